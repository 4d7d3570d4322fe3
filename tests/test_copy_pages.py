"""Page copies and conversions on the GPU: bit for bit against the f64 reference."""
import numpy as np
import pytest
import torch

import paged_kv_decode_attn_gb300 as oxd
import quant_ref as R
from quant_helpers import bf16, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    oxd.build()


def shape(pages, ps, H, layout, width):
    return (pages, ps, H, width) if layout == "NHD" else (pages, H, ps, width)


class Pools:
    """Random pools of one format (numpy and device)."""

    def __init__(self, fmt, layout, pages, ps, H, seed, sigma=1.0):
        rng = np.random.default_rng(seed)
        self.fmt, self.layout, self.pages, self.ps, self.H = fmt, layout, pages, ps, H
        x = [R.round_bf16(rng.normal(size=shape(pages, ps, H, layout, 128)) * sigma) for _ in "kv"]
        if fmt == "bf16":
            self.data = x
            self.dev = [bf16(a) for a in x]
            self.pools = oxd.KvPools(*self.dev)
        else:
            held = [R.hold(a) for a in x]
            self.data = [c for c, _ in held]
            self.scales = [np.ascontiguousarray(R.code_order(s, layout)) for _, s in held]
            self.dev = [torch.as_tensor(c, device="cuda") for c in self.data]
            self.dev_s = [torch.as_tensor(s, device="cuda") for s in self.scales]
            self.pools = oxd.KvPools(*self.dev, *self.dev_s)

    def rows(self, i):
        """Tensor i as [pages, H, ps, ...] rows: what the reference copies."""
        if self.fmt == "bf16":
            return self.data[i] if self.layout == "HND" else self.data[i].swapaxes(1, 2)
        v = R.pool_values(self.data[i], self.scales[i], self.layout)
        return v if self.layout == "HND" else v.swapaxes(1, 2)

    def got(self, i):
        """The device's tensor i: bf16 bits, or (codes, scale bits), with heads before tokens."""
        d = self.dev[i].view(torch.int16) if self.fmt == "bf16" else self.dev[i]
        d = d.cpu().numpy()
        d = d if self.layout == "HND" else d.swapaxes(1, 2)
        return d if self.fmt == "bf16" else (d, self.dev_s[i].view(torch.int16).cpu().numpy())


def bits(x):
    return bf16(x, "cpu").view(torch.int16).numpy()


def run(src, dst, sp, dp, refcount=None, n=None):
    n = len(sp) if n is None else n
    desc = oxd.make_copy_pages_desc(n, src.H, src.ps, src.fmt, src.layout, src.pages, dst.fmt,
                                    dst.layout, dst.pages)
    dev = [torch.as_tensor(np.asarray(a, np.int32), device="cuda") for a in (sp, dp)]
    ref = None if refcount is None else torch.as_tensor(refcount, dtype=torch.int32, device="cuda")
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    oxd.oxd_copy_pages(desc, src.pools, dst.pools, *dev, ref, ws)
    return oxd.oxd_read_device_status(ws)


def expect(src, dst, before, sp, dp):
    """dst's contents after the pairs, as got() gives them."""
    want = []
    for i in range(2):
        if dst.fmt == "bf16":
            w = before[i].copy()
            for s, d in zip(sp, dp):
                w[d] = bits(src.rows(i)[s])
        else:
            codes, scales = before[i][0].copy(), before[i][1].copy()
            for s, d in zip(sp, dp):
                if src.fmt == "e2m1":
                    c = src.data[i][s] if src.layout == "HND" else src.data[i][s].swapaxes(0, 1)
                    codes[d], scales[d] = c, src.scales[i][s].view(np.int16)
                else:
                    c, sc = R.hold(src.rows(i)[s])
                    codes[d], scales[d] = c, sc.view(np.int16)
            w = (codes, scales)
        want.append(w)
    return want


def assert_same(dst, want):
    for i in range(2):
        got = dst.got(i)
        if dst.fmt == "bf16":
            np.testing.assert_array_equal(got, want[i])
        else:
            np.testing.assert_array_equal(got[1], want[i][1])
            np.testing.assert_array_equal(R.plain_zero(got[0]), R.plain_zero(want[i][0]))


@pytest.mark.parametrize("src_fmt,dst_fmt", [("bf16", "bf16"), ("bf16", "e2m1"), ("e2m1", "bf16"),
                                             ("e2m1", "e2m1")])
@pytest.mark.parametrize("src_layout,dst_layout", [("NHD", "NHD"), ("HND", "HND"), ("NHD", "HND"),
                                                   ("HND", "NHD")])
@pytest.mark.parametrize("ps,H", [(8, 1), (16, 8), (32, 3), (64, 2), (16, 5)])
def test_between_two_caches(src_fmt, dst_fmt, src_layout, dst_layout, ps, H):
    src = Pools(src_fmt, src_layout, 11, ps, H, seed=1, sigma=2.0)
    dst = Pools(dst_fmt, dst_layout, 9, ps, H, seed=2)
    sp, dp = [3, 0, 10, 3, 7], [8, 1, 0, 4, 5]  # one source twice, pages of neither left alone
    want = expect(src, dst, [dst.got(0), dst.got(1)], sp, dp)
    assert run(src, dst, sp, dp) == 0
    assert_same(dst, want)


@pytest.mark.parametrize("fmt", ["bf16", "e2m1"])
@pytest.mark.parametrize("n", [1, 2, 63, 500])
def test_inside_one_cache(fmt, n):
    p = Pools(fmt, "NHD", 2 * n + 3, 16, 2, seed=n)
    order = np.random.default_rng(n).permutation(2 * n + 3)
    sp, dp = order[:n], order[n:2 * n]
    want = expect(p, p, [p.got(0), p.got(1)], sp, dp)
    assert run(p, p, sp, dp, refcount=np.ones(p.pages)) == 0
    assert_same(p, want)


def test_a_page_onto_itself_and_no_pairs():
    p = Pools("bf16", "HND", 4, 8, 2, seed=3)
    before = [p.got(0), p.got(1)]
    assert run(p, p, [2], [2]) == 0
    assert run(p, p, [], []) == 0
    assert_same(p, before)


def test_skipped_bad_and_shared_pages():
    src, dst = Pools("bf16", "NHD", 6, 16, 2, seed=4), Pools("e2m1", "NHD", 5, 16, 2, seed=5)
    before = [dst.got(0), dst.got(1)]
    ref = np.array([1, 2, 0, 1, 1])
    # a skipped pair says nothing, whatever its destination
    assert run(src, dst, [-1, 0, -1], [99, 0, -7], ref) == 0
    want = expect(src, dst, before, [0], [0])
    assert_same(dst, want)
    for sp, dp, code in (([6, 1], [3, 4], 1), ([-2, 1], [3, 4], 1), ([0, 1], [5, 4], 1),
                         ([0, 1], [-1, 4], 1), ([2 ** 31 - 1, 1], [0, 4], 1), ([0, 1], [1, 4], 4),
                         ([0, 1], [2, 4], 4)):
        assert run(src, dst, sp, dp, ref) == code
        assert_same(dst, expect(src, dst, want, [1], [4]))


def test_values_at_the_edges_of_the_format():
    H, ps = 1, 8
    src = Pools("bf16", "HND", 1, ps, H, seed=6)
    rng = np.random.default_rng(7)
    x = np.zeros((1, H, ps, 128))
    x[0, 0, 0] = R.round_bf16(rng.normal(size=128) * 2.0 ** rng.integers(-30, 20, 128))
    x[0, 0, 1, ::32] = [2.0 ** -24, 2.0 ** -25 * 3, 2.0 ** -22, 2.0 ** -126]
    x[0, 0, 2] = np.tile(R.round_bf16(np.linspace(-6, 6, 32)), 4)      # many ties
    x[0, 0, 3] = R.round_bf16(np.tile([6 * 1.375, 5 * 1.375, 3.5 * 1.375, -2.5 * 1.375], 32))
    x[0, 0, 4] = 65536.0
    x[0, 0, 5, 5] = R.round_bf16(3e38)
    x[0, 0, 6] = R.round_bf16(rng.normal(size=128) * 1e-5)
    x[0, 0, 7] = -0.0
    src.data = [x, -x]
    for d, v in zip(src.dev, src.data):
        d.copy_(bf16(v))
    dst = Pools("e2m1", "HND", 1, ps, H, seed=8)
    assert run(src, dst, [0], [0]) == 0
    for i in range(2):
        codes, scales = R.hold(src.rows(i))
        np.testing.assert_array_equal(dst.got(i)[1][0], scales[0].view(np.int16))
        # a zero's sign may be kept or not: compare what the codes stand for
        got = R.values(dst.got(i)[0], dst.got(i)[1].view(np.float16))
        np.testing.assert_array_equal(got, R.values(codes, scales))


def test_infinities_and_nan_become_finite():
    src, dst = Pools("bf16", "NHD", 1, 8, 1, seed=9), Pools("e2m1", "NHD", 1, 8, 1, seed=9)
    src.dev[0][0, 0, 0, 5] = float("inf")
    src.dev[0][0, 1, 0, 40] = -float("inf")
    src.dev[0][0, 2, 0, 100] = float("nan")
    assert run(src, dst, [0], [0]) == 0
    v = R.values(dst.got(0)[0], dst.got(0)[1].view(np.float16))[0, 0]
    assert np.isfinite(v).all() and v[0, 5] == 65472 and v[1, 40] == -65472
    keep = np.ones(128, bool)
    keep[96:] = False  # the other groups of the row with the NaN are as ever
    codes, scales = R.hold(src.rows(0)[0, 0, 2])
    np.testing.assert_array_equal(v[2][keep], R.values(codes, scales)[keep])


def test_every_code_and_scale_reads_back():
    p = Pools("e2m1", "HND", 3, 64, 2, seed=10)
    rng = np.random.default_rng(11)
    for i in range(2):
        p.data[i] = rng.integers(0, 256, p.data[i].shape).astype(np.uint8)
        p.scales[i] = rng.integers(0, 0x7154, p.scales[i].shape).astype(np.uint16).view(np.float16)
        p.dev[i].copy_(torch.as_tensor(p.data[i]))
        p.dev_s[i].copy_(torch.as_tensor(p.scales[i]))
    out = Pools("bf16", "NHD", 3, 64, 2, seed=12)
    assert run(p, out, [0, 1, 2], [2, 0, 1]) == 0
    for i in range(2):
        got = f64(out.dev[i]).swapaxes(1, 2)[[2, 0, 1]]
        # code x scale is exact in F32 (2 + 11 bits) and rounded once
        np.testing.assert_array_equal(got, f64(bf16(p.rows(i))))


def test_captured_call_replays_on_new_lists():
    p = Pools("bf16", "NHD", 40, 16, 2, seed=13)
    desc = oxd.make_copy_pages_desc(8, 2, 16, "bf16", "NHD", 40, "bf16", "NHD", 40)
    sp = torch.full((8,), -1, dtype=torch.int32, device="cuda")
    dp = torch.zeros(8, dtype=torch.int32, device="cuda")
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    oxd.oxd_copy_pages(desc, p.pools, p.pools, sp, dp, None, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        oxd.oxd_copy_pages(desc, p.pools, p.pools, sp, dp, None, ws)
    want = [p.got(0), p.got(1)]
    for s, d in (([1, 2, 3], [30, 31, 32]), ([5], [33]), (list(range(8)), list(range(20, 28)))):
        sp.fill_(-1)
        sp[:len(s)] = torch.tensor(s, dtype=torch.int32)
        dp[:len(d)] = torch.tensor(d, dtype=torch.int32)
        g.replay()
        assert oxd.oxd_read_device_status(ws) == 0
        for w in want:
            w[d] = w[s]
        assert_same(p, want)


def test_pools_past_32_bits():
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    ps, H, pages = 64, 8, 70_000  # 9 GB a pool
    k = torch.zeros(pages, ps, H, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    g = torch.Generator(device="cuda").manual_seed(1)
    for x in (k, v):
        x[0] = torch.randn(x[0].shape, generator=g, device="cuda").bfloat16()
        x[pages - 2] = torch.randn(x[0].shape, generator=g, device="cuda").bfloat16()
    desc = oxd.make_copy_pages_desc(2, H, ps, "bf16", "NHD", pages, "bf16", "NHD", pages)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    lists = [torch.tensor(a, dtype=torch.int32, device="cuda") for a in ([0, pages - 2], [pages - 1, 1])]
    oxd.oxd_copy_pages(desc, oxd.KvPools(k, v), oxd.KvPools(k, v), *lists, None, ws)
    assert oxd.oxd_read_device_status(ws) == 0
    for x in (k, v):
        assert torch.equal(x[pages - 1], x[0]) and torch.equal(x[1], x[pages - 2])
        assert not x[2].any() and not x[pages // 2].any() and not x[pages - 3].any()


@pytest.mark.parametrize("column", [0, 1, 7, 38, 69, 127])
def test_a_nan_leaves_the_other_columns_of_its_group(column):
    src, dst = Pools("bf16", "HND", 1, 8, 1, seed=12), Pools("e2m1", "HND", 1, 8, 1, seed=12)
    x = src.rows(0)[0, 0].copy()
    group = column // 32 * 32
    x[:, group:group + 32] *= 1 + 9 * (np.arange(32) % 2 == column % 2)  # the NaN's like are largest
    x = R.round_bf16(x)
    src.dev[0][0, 0] = bf16(x)
    src.dev[0][0, 0, :, column] = float("nan")
    assert run(src, dst, [0], [0]) == 0
    x[:, column] = 0
    codes, scales = R.hold(x)
    np.testing.assert_array_equal(dst.got(0)[1][0, 0], scales.view(np.int16))
    v = R.values(dst.got(0)[0], dst.got(0)[1].view(np.float16))[0, 0]
    keep = np.arange(128) != column
    assert np.isfinite(v).all()
    np.testing.assert_array_equal(v[:, keep], R.values(codes, scales)[:, keep])
