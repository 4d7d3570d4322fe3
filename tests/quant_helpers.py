"""Shared by the GPU tests of the 4-bit cache: seeded caches and runs, and the derived bounds."""
import numpy as np
import torch

import paged_kv_decode_attn_gb300 as oxd
import quant_ref as R
import workloads as W


def bf16(x, device="cuda"):
    return torch.as_tensor(np.asarray(x, np.float32), device=device).to(torch.bfloat16)


def f64(t):
    return t.double().cpu().numpy()


class Cache:
    """A 4-bit cache of normal values over the block tables of `lengths`; slots past a request's
    last token and pages of nobody hold random codes and NaN scales."""

    def __init__(self, lengths, G, Hkv, ps, layout, seed, sigma=1.0, extra_pages=3, q_sigma=1.0):
        rng = np.random.default_rng(seed)
        self.lengths, self.G, self.Hkv, self.ps, self.layout = list(lengths), G, Hkv, ps, layout
        self.batch, self.Hq = len(self.lengths), G * Hkv
        t = W.build_block_tables(np.asarray(lengths, np.int64), ps, rng)
        self.indptr, self.last = t.indptr, t.last_page_len
        self.num_pages = t.num_pages + extra_pages
        perm = rng.permutation(self.num_pages).astype(np.int32)
        self.indices = perm[t.indices]
        shape = (self.num_pages, ps, Hkv) if layout == "NHD" else (self.num_pages, Hkv, ps)
        live = np.zeros((self.num_pages, ps), bool)
        for b, n in enumerate(self.lengths):
            for j, p in enumerate(self.indices[self.indptr[b]:self.indptr[b + 1]]):
                live[p, :max(0, min(ps, n - j * ps))] = True
        dead = ~np.broadcast_to(live[:, None], (self.num_pages, Hkv, ps))
        self.codes, self.scales = [], []
        for _ in "kv":
            c, s = R.hold(R.round_bf16(rng.normal(size=shape + (128,)) * sigma))
            s = np.ascontiguousarray(s.swapaxes(1, 2)) if layout == "NHD" else s
            s[dead] = np.float16(np.nan)
            self.codes.append(c)
            self.scales.append(s)
        self.q = R.round_bf16(rng.normal(size=(self.batch, self.Hq, 128)) * q_sigma)
        self.d_codes = [torch.as_tensor(c, device="cuda") for c in self.codes]
        self.d_scales = [torch.as_tensor(s, device="cuda") for s in self.scales]
        self.pools = oxd.KvPools(*self.d_codes, *self.d_scales)
        self.d_q = bf16(self.q)
        self.d_indptr, self.d_indices, self.d_last = (
            torch.as_tensor(a, device="cuda") for a in (self.indptr, self.indices, self.last))

    def plan(self, **kw):
        desc = oxd.make_desc(self.batch, self.Hq, self.Hkv, self.ps, self.layout, self.num_pages, **kw)
        return oxd.oxd_quant_decode_plan(desc, self.indptr, self.last, torch.cuda.current_device())

    def run(self, plan, sm_scale=128 ** -0.5, want_lse=True, ws=None, out=None, lse=None, stream=None):
        out = torch.full((self.batch, self.Hq, 128), float("nan"), dtype=torch.bfloat16,
                         device="cuda") if out is None else out
        if lse is None and want_lse:
            lse = torch.full((self.batch, self.Hq), float("nan"), device="cuda")
        ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda") if ws is None else ws
        oxd.oxd_quant_decode_run(plan, self.d_q, self.pools, self.d_indptr, self.d_indices,
                                 self.d_last, sm_scale, out, lse, ws, stream=stream)
        return out, lse, ws

    def reference(self, sm_scale=128 ** -0.5):
        with np.errstate(invalid="ignore"):
            k, v = (R.pool_values(c, s, self.layout) for c, s in zip(self.codes, self.scales))
        return R.decode(self.q, k, v, self.indptr, self.indices, self.lengths, self.layout, sm_scale)


def assert_decode(out, lse, ref, what=""):
    """Bounds, from the roundings of one row (half a step each: f16 2^-11, bf16 2^-8, f32 2^-24):

    * a logit is a sum of 128 products in F32 with exact f16 operands (a column of q is exact, or
      off by 2^-25 of the head's largest), scaled per group: off by at most 128 * 2^-23 of the sum
      of sizes (a fused multiply-add chain that truncates loses 2^-23 a step), plus exp2's own
      2^-22 and the scaled argument's rounding: d = 2^-16 * size + 2^-20;
    * a weight then carries a factor e^d and one f16 rounding, a V value one f16 rounding; the
      denominator the same e^d: out is off by (2 d + 2^-11 + 2^-11 + 2^-14) * sum w |v|, the last
      for F32 sums over at most 2^9 steps per warp, and by half a bf16 step of itself;
    * f16 ends at steps of 2^-24, and the largest weight is held as 2^10 or more: a weight far below
      it is off by up to 2^-25 / 2^10 of it, whatever its size: 2^-35 * sum |v| more;
    * lse is off by d, by half a step of F32 of itself and 2^-22 of the logarithm.
    """
    r_out, r_lse, spread, size, total = ref
    d = 2.0 ** -16 * size + 2.0 ** -20
    o = f64(out)
    assert np.isfinite(o).all(), what
    err = np.abs(o - r_out)
    bound = (2 * d + 2.0 ** -10 + 2.0 ** -14)[..., None] * spread + 2.0 ** -8 * np.abs(r_out)
    bound = bound + 2.0 ** -35 * total
    assert (err <= bound).all(), f"{what}: out {(err / bound).max():.2f} of its bound"
    if lse is not None:
        e = np.abs(f64(lse) - r_lse)
        b = d + 2.0 ** -22 * (1 + np.abs(r_lse))
        assert (e <= b).all(), f"{what}: lse {(e / b).max():.2f} of its bound"
