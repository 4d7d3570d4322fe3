"""Decode with a sliding window and sinks against f64, bf16 and 4-bit pages (GPU)."""
import os

import numpy as np
import pytest
import torch

import paged_kv_decode_attn_gb300 as oxd
import quant_ref as R
import window_ref as Wr
from quant_helpers import assert_decode, bf16, f64

pytestmark = pytest.mark.gpu

SCALE = 128 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    oxd.build()


def dev(a):
    return torch.as_tensor(np.asarray(a, np.int32), device="cuda")


class Case:
    """One call over poisoned bf16 pages: guard bands around out and lse."""

    def __init__(self, lengths, G, Hkv, ps, layout, window, sinks, seed=0, sigma=1.0, q_sigma=1.0, **kw):
        self.p = Wr.Paged(lengths, [1] * len(lengths), Hkv, ps, layout, window, sinks, seed, sigma, **kw)
        self.B, self.Hq, self.window, self.sinks = len(lengths), G * Hkv, window, sinks
        self.q = self.p.queries(self.Hq, q_sigma)
        self.d_q, self.d_k, self.d_v = bf16(self.q), *(bf16(x) for x in self.p.pools)
        self.tables = [dev(self.p.indptr), dev(np.append(self.p.indices, 0)), dev(self.p.last)]
        self.ws = torch.empty(256, dtype=torch.uint8, device="cuda")

    def desc(self, **kw):
        p = self.p
        return oxd.make_window_decode_desc(self.B, self.Hq, p.Hkv, p.ps, p.layout, p.num_pages,
                                           len(self.tables[1]), self.window, self.sinks, **kw)

    def run(self, scale=SCALE, want_lse=True, stream=None, **kw):
        n = self.B * self.Hq
        out = torch.full((n * 128 + 256,), 77.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((n + 8,), 77.0, device="cuda")
        oxd.oxd_window_decode(self.desc(**kw), self.d_q, self.d_k, self.d_v, *self.tables, scale,
                              out[128:-128], lse[4:-4] if want_lse else None, self.ws, stream=stream)
        self.code = oxd.oxd_read_device_status(self.ws, stream)
        assert (out[:128] == 77).all() and (out[-128:] == 77).all()
        assert (lse[:4] == 77).all() and (lse[-4:] == 77).all()
        return out[128:-128].view(self.B, self.Hq, 128), lse[4:-4].view(self.B, self.Hq) if want_lse else None

    def reference(self, scale=SCALE):
        return Wr.attention(self.q, self.p.k, self.p.v, self.p.lengths, self.p.q_lens, self.window,
                            self.sinks, scale)

    def check(self, scale=SCALE, what="", **kw):
        out, lse = self.run(scale, **kw)
        assert self.code == 0, what
        Wr.assert_close(f64(out), f64(lse), self.reference(scale), what)
        return out, lse


LENGTHS = [1, 2, 15, 16, 17, 100, 129, 300, 640, 1000]


@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("ps", [8, 16, 32, 64])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (37, 0), (100, 17), (256, 65),
                                          (1000, 3), (5000, 8)])
def test_lengths_windows_and_sinks(layout, ps, window, sinks):
    Case(LENGTHS, 4, 2, ps, layout, window, sinks, seed=window + ps).check()


@pytest.mark.parametrize("G", [1, 2, 3, 7, 8, 9, 12, 16, 17, 24, 31, 32])
@pytest.mark.parametrize("Hkv", [1, 3])
def test_groups(G, Hkv):
    Case([700, 33, 5], G, Hkv, 16, "NHD", 130, 5, seed=G).check()


@pytest.mark.parametrize("splits", range(1, 17))
@pytest.mark.parametrize("G", [1, 5, 8, 16, 32])
def test_every_split(splits, G):
    """A stream shared by any number of CTAs, more of them than chunks too."""
    Case([900, 40], G, 1, 16, "HND", 500, 20, seed=splits).check(max_splits=splits)


def test_splits_that_the_launch_picks_for_long_windows():
    c = Case([9000], 4, 1, 64, "NHD", 8192, 64, seed=3)
    c.check()
    Case([9000], 32, 1, 16, "HND", 8500, 100, seed=4).check()


def test_requests_without_tokens():
    c = Case([0, 50, 0, 0, 7, 0], 4, 2, 16, "NHD", 20, 2, seed=1)
    out, lse = c.check()
    assert (out[0] == 0).all() and torch.isneginf(lse[5]).all()
    for splits in (2, 5):
        c.check(max_splits=splits)


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0, 4.0])
def test_scales(scale):
    Case([200, 31], 4, 2, 16, "NHD", 90, 4, seed=8).check(scale)


def test_far_logits_raise_the_maximum_often():
    """Keys that grow along the window: nearly every chunk raises the reference."""
    c = Case([600], 4, 1, 16, "NHD", 512, 4, seed=2)
    p = c.p
    grow = np.linspace(0.1, 20, 600)[None, :, None]
    p.k[0] = R.round_bf16(p.k[0] * 0 + grow * np.sign(c.q[0, 0]))
    pool = np.full_like(p.pools[0], np.nan)
    for j, page in enumerate(p.indices):
        if page >= 0:
            t = np.arange(j * 16, min(600, j * 16 + 16))
            pool[page, :len(t)] = p.k[0][:, t].swapaxes(0, 1)
    c.d_k = bf16(pool)
    c.check()
    c.check(max_splits=3)


def test_no_lse_and_another_stream():
    c = Case([100, 300], 8, 2, 32, "HND", 64, 2, seed=5)
    want, _ = c.check()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, _ = c.run(want_lse=False, stream=s)
    assert torch.equal(out, want)


def test_a_window_over_everything_is_the_plain_decode():
    c = Case([513, 40, 64], 4, 2, 16, "NHD", 1 << 20, 0, seed=6)
    out, lse = c.check()
    p = c.p
    desc = oxd.make_desc(3, 8, 2, 16, "NHD", p.num_pages)
    plan = oxd.oxd_paged_decode_plan(desc, p.indptr, p.last)
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    oxd.oxd_paged_decode_run(plan, c.d_q, c.d_k, c.d_v, *c.tables, SCALE, o2, l2, ws)
    Wr.assert_close(f64(o2), f64(l2), c.reference())


def test_runs_are_bitwise_equal():
    c = Case([4000, 77, 900], 8, 4, 16, "NHD", 700, 9, seed=7)
    out, lse = c.run()
    for _ in range(20):
        o, z = c.run()
        assert torch.equal(o, out) and torch.equal(z, lse)


@pytest.mark.parametrize("unseen", [-1, 1 << 30])
def test_unseen_pages_are_not_looked_at(unseen):
    Case([3000, 500], 4, 2, 8, "NHD", 100, 10, unseen=unseen, seed=9).check()


def test_bad_pages_are_recorded_and_confined():
    c = Case([100, 100, 100], 4, 2, 16, "NHD", 40, 0, seed=10)
    ref = c.reference()
    for bad in (-1, c.p.num_pages, 1 << 30):
        idx = np.append(c.p.indices, 0)
        idx[c.p.indptr[2] - 1] = bad  # request 1's last page
        c.tables[1] = dev(idx)
        out, lse = c.run()
        assert c.code == oxd.OXD_DEVICE_BAD_PAGE
        keep = [0, 2]
        Wr.assert_close(f64(out)[keep], f64(lse)[keep], [x[keep] for x in ref])


def test_bad_tables_are_recorded_and_confined():
    c = Case([100, 100, 100], 4, 2, 16, "HND", 40, 3, seed=11)
    ref, good = c.reference(), [t.clone() for t in c.tables]
    n = len(c.p.indices)
    for which, at, value, hit in [(2, 1, 0, [1]), (2, 1, 17, [1]), (2, 2, -5, [2]),
                                  (0, 3, n + 2, [2]), (0, 0, -1, [0]), (0, 3, -7, [2]),
                                  (0, 1, 2 ** 31 - 1, [0, 1])]:
        c.tables = [t.clone() for t in good]
        c.tables[which][at] = value
        for splits in (1, 4):
            out, lse = c.run(max_splits=splits)
            assert c.code == oxd.OXD_DEVICE_BAD_POSITION
            keep = [b for b in range(3) if b not in hit]
            Wr.assert_close(f64(out)[keep], f64(lse)[keep], [x[keep] for x in ref])
            assert (out[hit] == 0).all() and torch.isneginf(lse[hit]).all()


def test_a_request_of_more_than_2_30_tokens_is_refused():
    n = (1 << 24) + 2
    indices = torch.full((n,), 0, dtype=torch.int32, device="cuda")
    k = torch.zeros((2, 64, 1, 128), dtype=torch.bfloat16, device="cuda")
    q = torch.ones((1, 1, 128), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    for pages, code in ((n, oxd.OXD_DEVICE_BAD_POSITION), (1 << 24, 0)):
        out, lse = torch.empty_like(q), torch.empty((1, 1), device="cuda")
        d = oxd.make_window_decode_desc(1, 1, 1, 64, "NHD", 2, n, 100, 10)
        oxd.oxd_window_decode(d, q, k, k, dev([0, pages]), indices, dev([64]), 1.0, out, lse, ws)
        assert oxd.oxd_read_device_status(ws) == code
        if code == 0:
            assert abs(lse.item() - np.log(110)) < 1e-5


def test_a_captured_call_follows_the_lengths():
    c = Case([400, 400, 400], 4, 2, 16, "NHD", 64, 4, seed=12)
    desc = c.desc()
    out = torch.empty((3, 8, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((3, 8), device="cuda")

    def call():
        oxd.oxd_window_decode(desc, c.d_q, c.d_k, c.d_v, *c.tables, SCALE, out, lse, c.ws)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    g.replay()
    first = Case([400, 400, 400], 4, 2, 16, "NHD", 64, 4, seed=12)
    Wr.assert_close(f64(out), f64(lse), first.reference())
    # shorter requests: their windows are other tokens of the same pages (no poison there)
    c2 = Case([400, 400, 400], 4, 2, 16, "NHD", 400, 0, seed=12)
    c.d_k.copy_(c2.d_k)
    c.d_v.copy_(c2.d_v)
    c.tables[1].copy_(c2.tables[1])
    p = c2.p
    lengths = [0, 33, 256]
    c.tables[0].copy_(dev([0, 0, 3, 19]))
    idx = np.concatenate([p.indices[25:28], p.indices[50:66]])
    c.tables[1][:len(idx)] = dev(idx)
    c.tables[2].copy_(dev([0, 1, 16]))
    g.replay()
    k = [x[:, :n] for x, n in zip(p.k, lengths)]
    v = [x[:, :n] for x, n in zip(p.v, lengths)]
    Wr.assert_close(f64(out), f64(lse), Wr.attention(c.q, k, v, lengths, [1] * 3, 64, 4, SCALE))
    assert oxd.oxd_read_device_status(c.ws) == 0


@pytest.mark.parametrize("four", [False, True])
def test_behind_an_append_as_its_programmatic_dependent(four):
    """The append writes the step's q and rows; pdl gives the same result as a plain launch."""
    rng = np.random.default_rng(13)
    B, Hq, Hkv, ps, n = 20, 8, 2, 16, 6
    pool = B * n
    shape = (pool, ps, Hkv, 64 if four else 128)
    indptr, last = dev(np.arange(B + 1) * n), dev([ps] * B)
    idx = dev(rng.permutation(pool))
    ones = torch.ones(pool, dtype=torch.int32, device="cuda")
    q, k, v = (bf16(rng.normal(size=(B, h, 128))) for h in (Hq, Hkv, Hkv))
    req, pos = dev(range(B)), dev([n * ps - 1] * B)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    ad = oxd.make_axes_append_desc(B, B, Hq, Hkv, ps, "NHD", pool, pool)
    got = []
    if four:
        codes = [torch.as_tensor(rng.integers(0, 256, shape, np.uint8), device="cuda") for _ in "kv"]
        scales = [torch.as_tensor(rng.uniform(0.1, 0.5, (pool, Hkv, ps, 4)).astype(np.float16),
                                  device="cuda") for _ in "kv"]
    else:
        pools = [bf16(rng.normal(size=shape)) for _ in "kv"]
    for pdl in (0, 1):
        q_out, out = torch.empty_like(q), torch.empty_like(q)
        lse = torch.empty((B, Hq), device="cuda")
        wd = oxd.make_window_decode_desc(B, Hq, Hkv, ps, "NHD", pool, pool, 64, 4, pdl=pdl)
        for _ in range(5):
            if four:
                c = oxd.KvPools(*(x.clone() for x in codes + scales))
                oxd.oxd_quant_rope_append(ad, q, k, v, req, pos, None, indptr, idx, ones, q_out, c, ws)
                oxd.oxd_quant_window_decode(wd, q_out, c, indptr, idx, last, SCALE, out, lse, ws)
            else:
                c = [x.clone() for x in pools]
                oxd.oxd_rope_axes_append(ad, q, k, v, req, pos, None, indptr, idx, ones, q_out, *c, ws)
                oxd.oxd_window_decode(wd, q_out, *c, indptr, idx, last, SCALE, out, lse, ws)
            assert oxd.oxd_read_device_status(ws) == 0
            got.append((out.clone(), lse.clone()))
    for o, z in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(z, got[0][1])


# ------------------------------------------------------------------ 4-bit pages

class QuantCase(Case):
    """Over a 4-bit cache: unseen rows have random codes and NaN scales."""

    def __init__(self, lengths, G, Hkv, ps, layout, window, sinks, seed=0, sigma=1.0, q_sigma=1.0, **kw):
        self.p = p = Wr.Paged(lengths, [1] * len(lengths), Hkv, ps, layout, window, sinks, seed, sigma, **kw)
        self.B, self.Hq, self.window, self.sinks = len(lengths), G * Hkv, window, sinks
        self.q = p.queries(self.Hq, q_sigma)
        self.d_q = bf16(self.q)
        arrays = []
        for pool in p.pools:
            dead = np.isnan(pool).all(-1)
            codes, scales = R.hold(np.where(dead[..., None], 1.0, pool))
            codes[dead] = p.rng.integers(0, 256, (int(dead.sum()), 64))
            scales[dead] = np.float16(np.nan)
            arrays.append((codes, scales))
        self.codes = [torch.as_tensor(np.ascontiguousarray(c), device="cuda") for c, _ in arrays]
        self.scales = [torch.as_tensor(np.ascontiguousarray(
            s.swapaxes(1, 2) if layout == "NHD" else s), device="cuda") for _, s in arrays]
        self.pools = oxd.KvPools(*self.codes, *self.scales)
        # what the cache stands for
        p.k, p.v = ([R.values(*R.hold(x)) for x in y] for y in (p.k, p.v))
        self.tables = [dev(p.indptr), dev(np.append(p.indices, 0)), dev(p.last)]
        self.ws = torch.empty(256, dtype=torch.uint8, device="cuda")

    def run(self, scale=SCALE, want_lse=True, stream=None, **kw):
        n = self.B * self.Hq
        out = torch.full((n * 128 + 256,), 77.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((n + 8,), 77.0, device="cuda")
        oxd.oxd_quant_window_decode(self.desc(**kw), self.d_q, self.pools, *self.tables, scale,
                                    out[128:-128], lse[4:-4] if want_lse else None, self.ws,
                                    stream=stream)
        self.code = oxd.oxd_read_device_status(self.ws, stream)
        assert (out[:128] == 77).all() and (out[-128:] == 77).all()
        assert (lse[:4] == 77).all() and (lse[-4:] == 77).all()
        return out[128:-128].view(self.B, self.Hq, 128), lse[4:-4].view(self.B, self.Hq) if want_lse else None

    def check(self, scale=SCALE, what="", **kw):
        out, lse = self.run(scale, **kw)
        assert self.code == 0, what
        ref = self.reference(scale)
        live = np.asarray(self.p.lengths) > 0
        assert_decode(out[live], lse[live], [x[live] for x in ref], what)
        assert (out[~live] == 0).all() and torch.isneginf(lse[~live]).all()
        return out, lse


@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("ps", [8, 16, 32, 64])
@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 4), (37, 1), (256, 65), (5000, 8)])
def test_4bit_lengths_windows_and_sinks(layout, ps, window, sinks):
    QuantCase(LENGTHS + [0], 4, 2, ps, layout, window, sinks, seed=window + ps).check()


@pytest.mark.parametrize("G", [1, 2, 7, 8, 9, 16, 20, 32])
@pytest.mark.parametrize("Hkv,layout", [(1, "NHD"), (2, "HND"), (3, "NHD"), (4, "NHD")])
def test_4bit_groups(G, Hkv, layout):
    QuantCase([700, 33, 5], G, Hkv, 16, layout, 130, 5, seed=G).check()


@pytest.mark.parametrize("splits", [1, 2, 3, 5, 8, 13, 16])
@pytest.mark.parametrize("G,Hkv", [(4, 2), (8, 1), (12, 2)])
def test_4bit_every_split(splits, G, Hkv):
    QuantCase([900, 40, 0], G, Hkv, 16, "NHD", 500, 20, seed=splits).check(max_splits=splits)


@pytest.mark.parametrize("G", [1, 3, 8, 12])
@pytest.mark.parametrize("batch,window,sinks", [(700, 40, 3), (330, 4096, 5), (330, 4100, 0), (900, 4096, 17)])
def test_4bit_more_streams_than_the_gpu_holds(batch, window, sinks, G):
    """Two KV heads a CTA, and (from 4096 tokens) streams cut in two although not all fit."""
    rng = np.random.default_rng(batch + G)
    lengths = rng.integers(0, 80, batch)
    lengths[[3, batch - 1]] = 5000, 4400
    c = QuantCase(list(map(int, lengths)), G, 2, 16, "NHD", window, sinks, seed=G)
    out, lse = c.check()
    o, z = c.check(max_splits=1)
    if window < 4096:
        assert torch.equal(o, out) and torch.equal(z, lse)


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0])
def test_4bit_scales(scale):
    QuantCase([200, 31], 4, 2, 16, "NHD", 90, 4, seed=8).check(scale)


def test_4bit_runs_are_bitwise_equal():
    c = QuantCase([4000, 77, 900], 8, 4, 16, "NHD", 700, 9, seed=7)
    out, lse = c.run()
    for _ in range(20):
        o, z = c.run()
        assert torch.equal(o, out) and torch.equal(z, lse)


def test_4bit_bad_pages_and_tables():
    c = QuantCase([100, 100, 100], 4, 2, 16, "NHD", 40, 0, seed=10)
    ref, good = c.reference(), [t.clone() for t in c.tables]
    keep = [0, 2]
    for which, at, value, code in [(1, int(c.p.indptr[2]) - 1, -1, oxd.OXD_DEVICE_BAD_PAGE),
                                   (1, int(c.p.indptr[2]) - 1, c.p.num_pages, oxd.OXD_DEVICE_BAD_PAGE),
                                   (2, 1, 0, oxd.OXD_DEVICE_BAD_POSITION)]:
        c.tables = [t.clone() for t in good]
        c.tables[which][at] = value
        out, lse = c.run()
        assert c.code == code
        assert_decode(out[keep], lse[keep], [x[keep] for x in ref])


# ------------------------------------------------------------------ at random

@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("seed", range(30 * int(os.environ.get("OXD_FUZZ_SCALE", "1"))))
def test_random_decodes(seed, four):
    rng = np.random.default_rng(2000 + seed)
    B = int(rng.integers(1, 20))
    lengths = [int(np.exp(rng.uniform(0, np.log(2000)))) * int(rng.random() > 0.1) for _ in range(B)]
    G, Hkv = int(rng.integers(1, 33)), int(rng.choice([1, 2, 3, 4, 8]))
    window, sinks = int(np.exp(rng.uniform(0, np.log(2500)))), int(rng.choice([0, 1, 4, 33, 130]))
    ps, layout = int(rng.choice([8, 16, 32, 64])), str(rng.choice(["NHD", "HND"]))
    c = (QuantCase if four else Case)(lengths, G, Hkv, ps, layout, window, sinks, seed=seed,
                                      sigma=float(rng.choice([0.5, 1, 2])))
    c.check(float(rng.choice([SCALE, -SCALE, 0.5])), f"{lengths} {G} {Hkv} {window} {sinks} {ps} {layout}",
            max_splits=int(rng.choice([0, 0, 1, 5])))


# ------------------------------------------------------------------ far pages

@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("layout", ["NHD", "HND"])
def test_pools_past_2_32_bytes(layout, four):
    """Pages at both ends of pools of more than 4 GiB each."""
    ps, Hkv, G, n = 64, 2, 4, 300
    width = 64 if four else 128
    pages = (1 << 32) // (ps * Hkv * (64 if four else 256)) + 1000
    rng = np.random.default_rng(21)
    p = Wr.Paged([n], [1], Hkv, ps, layout, 200, 10, 21, spare=0)
    at = np.asarray([3, pages - 1, 0, pages - 700, pages // 2])[:len(p.indices)]
    shape = (pages, ps, Hkv, width) if layout == "NHD" else (pages, Hkv, ps, width)
    dtype = torch.uint8 if four else torch.bfloat16
    pools = [torch.empty(shape, dtype=dtype, device="cuda") for _ in "kv"]
    scales = [torch.empty((pages, Hkv, ps, 4), dtype=torch.float16, device="cuda") for _ in "kv"] if four else []
    k, v = p.k, p.v
    for i, pool in enumerate(p.pools):
        for j, page in enumerate(p.indices):
            if page < 0:
                continue
            x = np.nan_to_num(pool[page])
            if four:
                c, s = R.hold(x)
                pools[i][at[j]] = torch.as_tensor(c, device="cuda")
                scales[i][at[j]] = torch.as_tensor(
                    np.ascontiguousarray(s.swapaxes(0, 1) if layout == "NHD" else s), device="cuda")
            else:
                pools[i][at[j]] = bf16(x)
    if four:
        k, v = ([R.values(*R.hold(x)) for x in y] for y in (k, v))
    q = p.queries(G * Hkv)
    out, lse = torch.empty((1, G * Hkv, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((1, G * Hkv), device="cuda")
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    d = oxd.make_window_decode_desc(1, G * Hkv, Hkv, ps, layout, pages, len(at), 200, 10)
    tables = (dev(p.indptr), dev(np.where(p.indices < 0, -1, at)), dev(p.last))
    if four:
        oxd.oxd_quant_window_decode(d, bf16(q), oxd.KvPools(*pools, *scales), *tables, SCALE, out, lse, ws)
    else:
        oxd.oxd_window_decode(d, bf16(q), *pools, *tables, SCALE, out, lse, ws)
    assert oxd.oxd_read_device_status(ws) == 0
    ref = Wr.attention(q, k, v, [n], [1], 200, 10, SCALE)
    if four:
        assert_decode(out, lse, ref)
    else:
        Wr.assert_close(f64(out), f64(lse), ref)
