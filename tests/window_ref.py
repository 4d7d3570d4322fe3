"""Attention with a sliding window and sinks in f64, and seeded paged caches for its tests.

A query at position p sees the tokens j <= p with j > p - window or j < sinks.
"""
import numpy as np

import quant_ref as R


def seen(p, length, window, sinks):
    """The tokens that a query at position p of a request of `length` tokens sees."""
    j = np.arange(length)
    return j[(j <= p) & ((j > p - window) | (j < sinks))]


def attend(q, k, v, sm_scale):
    """One query's heads [G, 128] over rows [n, 128]: (out, lse, spread, size, total); spread =
    sum w |v| bounds what relative errors of w and v move, size = the largest sum |q k| sm_scale,
    total = sum |v|."""
    x = q @ k.T * sm_scale
    m = x.max(-1, keepdims=True)
    w = np.exp(x - m)
    z = w.sum(-1, keepdims=True)
    size = (np.abs(q) @ np.abs(k).T * abs(sm_scale)).max(-1)
    return (w @ v / z, (m + np.log(z))[:, 0], w @ np.abs(v) / z, size,
            np.broadcast_to(np.abs(v).sum(0), q.shape))


def attention(q, k, v, lengths, q_lens, window, sinks, sm_scale):
    """q [sum q_lens, Hq, 128], k, v: per request [Hkv, L, 128]; query i of a request sits at
    L - q_len + i. Requests without tokens get 0 and -inf."""
    n, Hq, _ = q.shape
    got = [np.zeros((n, Hq, 128)), np.full((n, Hq), -np.inf), np.zeros((n, Hq, 128)),
           np.zeros((n, Hq)), np.zeros((n, Hq, 128))]
    at = 0
    for b, (length, ql) in enumerate(zip(lengths, q_lens)):
        for i in range(ql if length else 0):
            t = seen(length - ql + i, length, window, sinks)
            G = Hq // len(k[b])
            for h in range(len(k[b])):
                rows = slice(h * G, (h + 1) * G)
                for dst, x in zip(got, attend(q[at + i, rows], k[b][h][t], v[b][h][t], sm_scale)):
                    dst[at + i, rows] = x
        at += ql
    return got


class Paged:
    """Tables and bf16 pools of requests whose queries are their last q_lens tokens. What no query
    sees is poison: NaN rows in the pools, and pages wholly unseen listed as `unseen`."""

    def __init__(self, lengths, q_lens, Hkv, ps, layout, window, sinks, seed, sigma=1.0, unseen=-1,
                 poison=np.nan, spare=3):
        rng = np.random.default_rng(seed)
        self.lengths, self.q_lens, self.Hkv, self.ps, self.layout = lengths, q_lens, Hkv, ps, layout
        pages = [-(-n // ps) for n in lengths]
        self.indptr = np.concatenate([[0], np.cumsum(pages)]).astype(np.int32)
        self.last = np.asarray([n - (p - 1) * ps if p else 0 for n, p in zip(lengths, pages)], np.int32)
        self.num_pages = int(self.indptr[-1]) + spare
        self.indices = rng.permutation(self.num_pages)[:self.indptr[-1]].astype(np.int32)
        self.k, self.v = [], []  # per request [Hkv, L, 128]
        for n in lengths:
            for dst in (self.k, self.v):
                dst.append(R.round_bf16(rng.normal(size=(Hkv, n, 128)) * sigma))
        shape = (self.num_pages, ps, Hkv, 128)
        pools = [np.full(shape, poison), np.full(shape, poison)]
        for b, (n, ql) in enumerate(zip(lengths, q_lens)):
            live = np.zeros(n, bool)
            for i in range(ql):
                live[seen(n - ql + i, n, window, sinks)] = True
            for j in range(pages[b]):
                t = np.arange(j * ps, min(n, (j + 1) * ps))
                at = self.indptr[b] + j
                for pool, src in zip(pools, (self.k, self.v)):
                    pool[self.indices[at], t[live[t]] - j * ps] = src[b][:, t[live[t]]].swapaxes(0, 1)
                if not live[t].any():
                    self.indices[at] = unseen
        if layout == "HND":
            pools = [p.swapaxes(1, 2) for p in pools]
        self.pools = [np.ascontiguousarray(p) for p in pools]
        self.rng = rng

    def queries(self, Hq, sigma=1.0):
        return R.round_bf16(self.rng.normal(size=(sum(self.q_lens), Hq, 128)) * sigma)


def assert_close(out, lse, ref, what=""):
    """Bounds, from the roundings of one row (half a step each: bf16 2^-8, f32 2^-24):

    * a logit is a sum of 128 products of bf16 numbers in F32, exact products, sums that may
      truncate (2^-23 a step of the sum of sizes); its scale and the reference it is counted from
      round once each in the log2 domain, exp2 is good to 2^-22: d = 2^-16 * size + 2^-20;
    * a weight then carries a factor e^d and one bf16 rounding, a V value none, the denominator
      the same e^d: out is off by (2 d + 2^-8 + 2^-14) * sum w |v|, the last for F32 sums over at
      most 2^9 steps a warp, and by half a bf16 step of itself;
    * lse is off by d, by half a step of F32 of itself and 2^-22 of the logarithm.
    """
    r_out, r_lse, spread, size, _ = ref
    d = 2.0 ** -16 * size + 2.0 ** -20
    assert np.isfinite(out).all(), what
    err = np.abs(out - r_out)
    bound = (2 * d + 2.0 ** -8 + 2.0 ** -14)[..., None] * spread + 2.0 ** -8 * np.abs(r_out)
    assert (err <= bound).all(), f"{what}: out {(err / np.maximum(bound, 1e-300)).max():.2f} of its bound"
    if lse is not None:
        none = np.isneginf(r_lse)
        assert (np.isneginf(lse) == none).all(), what
        e = np.abs(np.where(none, 0, lse) - np.where(none, 0, r_lse))
        b = d + 2.0 ** -22 * (1 + np.abs(np.where(none, 0, r_lse)))
        assert (e <= b).all(), f"{what}: lse {(e / b).max():.2f} of its bound"


def attention_torch(q, k, v, lengths, q_lens, window, sinks, sm_scale, device="cuda"):
    """`attention` by torch in f64, for larger cases; the same outputs, as numpy arrays."""
    import torch

    n, Hq, _ = q.shape
    qd = torch.as_tensor(q, dtype=torch.float64, device=device)
    got = [torch.zeros((n, Hq, 128), dtype=torch.float64, device=device) for _ in range(3)]
    lse, size = (torch.zeros((n, Hq), dtype=torch.float64, device=device) for _ in range(2))
    lse -= np.inf
    at = 0
    for b, (length, ql) in enumerate(zip(lengths, q_lens)):
        G = Hq // len(k[b])
        pos = torch.arange(length - ql, length, device=device)[:, None]
        j = torch.arange(length, device=device)
        mask = (j <= pos) & ((j > pos - window) | (j < sinks))
        for h in range(Hq):
            kd, vd = (torch.as_tensor(x[b][h // G], dtype=torch.float64, device=device) for x in (k, v))
            rows = qd[at:at + ql, h]
            x = (rows @ kd.T * sm_scale).masked_fill(~mask, -np.inf)
            w = torch.softmax(x, -1)
            got[0][at:at + ql, h] = w @ vd
            got[1][at:at + ql, h] = w @ vd.abs()
            lse[at:at + ql, h] = torch.logsumexp(x, -1)
            size[at:at + ql, h] = (rows.abs() @ kd.abs().T * abs(sm_scale)).masked_fill(~mask, 0).amax(-1)
        at += ql
    return [t.cpu().numpy() for t in (got[0], lse, got[1], size, got[2])]
