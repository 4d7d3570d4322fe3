"""Multi-axis rotary append into bf16 and 4-bit pages on the GPU against the f64 reference."""
from decimal import Decimal, localcontext

import numpy as np
import pytest
import torch

import paged_kv_decode_attn_gb300 as oxd
import quant_ref as R
import workloads as W
from quant_helpers import bf16, f64

pytestmark = pytest.mark.gpu

SECTIONS = {1: (64,), 2: (20, 44), 3: (16, 24, 24), 4: (16, 16, 16, 16)}


@pytest.fixture(scope="module", autouse=True)
def setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    oxd.build()


class Job:
    """New tokens for requests whose block tables cover them; pools filled with a pattern."""

    def __init__(self, first, add, Hq, Hkv, ps, layout, axes, four, seed, far=0, shuffle=True):
        rng = np.random.default_rng(seed)
        self.ps, self.layout, self.Hq, self.Hkv, self.four = ps, layout, Hq, Hkv, four
        ends = np.asarray(first) + np.asarray(add)
        t = W.build_block_tables(np.maximum(ends, 1).astype(np.int64), ps, rng)
        self.indptr, self.indices, self.pages = t.indptr, t.indices, t.num_pages + 2
        req = np.concatenate([np.full(n, b) for b, n in enumerate(add)])
        pos = np.concatenate([f + np.arange(n) for f, n in zip(first, add)])
        if shuffle:
            o = rng.permutation(len(req))
            req, pos = req[o], pos[o]
        self.req, self.pos, self.T = req, pos, len(req)
        self.rope = pos[None] if axes == 1 else rng.integers(0, far or 40, (axes, self.T))
        self.axes, self.theta = axes, 10000.0
        self.pair_axis = np.repeat(np.arange(axes), SECTIONS[axes])
        self.q, self.k, self.v = (R.round_bf16(rng.normal(size=(self.T, h, 128)))
                                  for h in (Hq, Hkv, Hkv))
        self.ref = np.ones(self.pages, np.int32)
        lead = (self.pages, ps, Hkv) if layout == "NHD" else (self.pages, Hkv, ps)
        if four:
            self.dev = [torch.full(lead + (64,), 0xA5, dtype=torch.uint8, device="cuda") for _ in "kv"]
            self.dev_s = [torch.full((self.pages, Hkv, ps, 4), 3.0, dtype=torch.float16,
                                     device="cuda") for _ in "kv"]
        else:
            self.dev = [torch.full(lead + (128,), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]

    def run(self, q_out=None, null_rope=False, stream=None):
        d = lambda a: torch.as_tensor(np.asarray(a, np.int32), device="cuda")  # noqa: E731
        desc = oxd.make_axes_append_desc(self.T, len(self.indptr) - 1, self.Hq, self.Hkv, self.ps,
                                         self.layout, self.pages, len(self.indices),
                                         rope_theta=self.theta, pair_axis=list(map(int, self.pair_axis)))
        dq = bf16(self.q)
        self.q_out = torch.empty_like(dq) if q_out is None else dq
        ws = torch.empty(256, dtype=torch.uint8, device="cuda")
        args = (desc, dq, bf16(self.k), bf16(self.v), d(self.req), d(self.pos),
                None if null_rope else d(self.rope), d(self.indptr), d(self.indices), d(self.ref),
                self.q_out)
        if self.four:
            oxd.oxd_quant_rope_append(*args, oxd.KvPools(*self.dev, *self.dev_s), ws, stream=stream)
        else:
            oxd.oxd_rope_axes_append(*args, *self.dev, ws, stream=stream)
        return oxd.oxd_read_device_status(ws)

    def rotated(self, x):
        return R.rotate(x, self.rope, self.pair_axis, self.theta)

    def check(self, skip=()):
        written = np.array([t not in skip for t in range(self.T)])
        page = self.indices[np.minimum(self.indptr[self.req] + self.pos // self.ps,
                                       len(self.indices) - 1)]
        slot = self.pos % self.ps
        close(f64(self.q_out), self.rotated(self.q), self.q)
        k = self.rotated(self.k)
        for i, rows in enumerate((k, self.v)):
            pool = self.dev[i].cpu() if self.four else self.dev[i].view(torch.int16).cpu()
            pool = pool.numpy() if self.layout == "HND" else pool.numpy().swapaxes(1, 2)
            got = pool[page[written], :, slot[written]]
            rest = np.ones(pool.shape[:3], bool)
            rest[page[written], :, slot[written]] = False
            if not self.four:
                assert (pool[rest] == bf16([7.0], "cpu").view(torch.int16).item()).all()
                got = f64(torch.as_tensor(got).view(torch.bfloat16))
                if i == 0:
                    close(got, rows[written], self.k[written])
                else:
                    np.testing.assert_array_equal(got, rows[written])
                continue
            scales = self.dev_s[i].cpu().numpy()
            assert (pool[rest] == 0xA5).all() and (scales[rest] == 3).all()
            codes, sc = R.hold(R.round_bf16(rows[written]))
            np.testing.assert_array_equal(scales[page[written], :, slot[written]], sc)
            # every code is the reference's (the sign of a zero aside)
            np.testing.assert_array_equal(R.values(got, sc), R.values(codes, sc))


def close(got, want, x):
    """A rotated row rounded once to bf16: half a step (2^-8 of the value) plus float error. The
    angle is good to 2^-25 turns (2e-7 rad) and two products and a sum round at 2^-24 each:
    within 2^-21 of the pair's norm."""
    norm = np.sqrt(x[..., :64] ** 2 + x[..., 64:] ** 2)
    norm = np.concatenate([norm, norm], -1)
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -21 * norm).all()


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("axes", [1, 2, 3, 4])
@pytest.mark.parametrize("ps,layout", [(8, "NHD"), (16, "HND"), (16, "NHD"), (32, "NHD"), (64, "HND")])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 8), (32, 8), (7, 1), (15, 3), (36, 9)])
def test_append(four, axes, ps, layout, Hq, Hkv):
    j = Job([0, 5, 100, 63, 40], [3, 1, 30, 17, 1], Hq, Hkv, ps, layout, axes, four, seed=axes + ps)
    assert j.run() == 0
    j.check()


@pytest.mark.parametrize("four", [False, True])
def test_one_token(four):
    j = Job([0], [1], 4, 2, 16, "NHD", 3, four, seed=1)
    j.rope[:] = 0
    assert j.run() == 0
    j.check()


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("theta", [10000.0, 1.5, 5e6])
def test_far_positions_and_other_bases(four, theta):
    j = Job([0, 30], [70, 60], 4, 2, 16, "NHD", 3, four, seed=2, far=1 << 17)
    j.theta = theta
    j.rope[:, :8] = [[0] * 8, [1 << 17] * 8, range((1 << 17) - 8, 1 << 17)]
    assert j.run() == 0
    j.check()


def test_the_last_position_the_angle_allows():
    # the reference's own f64 angle is good to 2^-53 * 2^24 * 1 rad = 2^-29 there
    j = Job([0], [40], 4, 2, 16, "NHD", 2, False, seed=3, far=1 << 24)
    j.rope[1, :] = (1 << 24) - 1
    assert j.run() == 0
    j.check()


@pytest.mark.parametrize("four", [False, True])
def test_one_axis_is_the_plain_append(four):
    j = Job([7, 100], [30, 20], 8, 2, 16, "NHD", 1, four, seed=4)
    assert j.run(null_rope=True) == 0
    j.check()
    first, q = [x.clone() for x in j.dev], j.q_out.clone()
    assert j.run() == 0
    assert all(torch.equal(a, b) for a, b in zip(first, j.dev)) and torch.equal(q, j.q_out)


@pytest.mark.parametrize("four", [False, True])
def test_interleaved_axes(four):
    j = Job([0, 9], [33, 20], 8, 2, 16, "HND", 3, four, seed=5)
    j.pair_axis = np.arange(64) % 3
    assert j.run() == 0
    j.check()


@pytest.mark.parametrize("four", [False, True])
def test_q_in_place(four):
    j = Job([0, 9], [33, 20], 32, 8, 16, "NHD", 3, four, seed=6)
    assert j.run(q_out="in place") == 0
    j.check()


def test_append_is_the_bf16_append_of_one_axis():
    """Bits of oxd_rope_append, which rotates in float too."""
    j = Job([0, 50], [40, 30], 16, 4, 16, "NHD", 1, False, seed=7)
    assert j.run() == 0
    d = lambda a: torch.as_tensor(np.asarray(a, np.int32), device="cuda")  # noqa: E731
    desc = oxd.make_rope_append_desc(j.T, 2, 16, 4, 16, "NHD", j.pages, len(j.indices))
    dq = bf16(j.q)
    out, pools = torch.empty_like(dq), [torch.full_like(x, 7.0) for x in j.dev]
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    oxd.oxd_rope_append(desc, dq, bf16(j.k), bf16(j.v), d(j.req), d(j.pos), d(j.indptr),
                        d(j.indices), d(j.ref), out, *pools, ws)
    assert torch.equal(pools[1], j.dev[1])
    for a, b in ((out, j.q_out), (pools[0], j.dev[0])):
        assert (a != b).float().mean() < 1e-3  # a value within float error of a bf16 midpoint


@pytest.mark.parametrize("four", [False, True])
def test_tokens_that_are_refused(four):
    def job():
        return Job([0, 20], [12, 12], 8, 4, 8, "NHD", 3, four, seed=8, shuffle=False)

    for change, code, skip in (
            (lambda j: j.req.__setitem__(3, -1), 5, [3]),
            (lambda j: j.req.__setitem__(3, 2), 5, [3]),
            (lambda j: j.pos.__setitem__(5, 99), 5, [5]),
            (lambda j: j.pos.__setitem__(5, -1), 5, [5]),
            (lambda j: j.rope.__setitem__((2, 7), -1), 5, [7]),
            (lambda j: j.rope.__setitem__((0, 7), 1 << 24), 5, [7])):
        j = job()
        change(j)
        assert j.run() == code
        j.rope = j.rope & ((1 << 24) - 1)
        j.check(skip)
    j = job()
    j.ref[j.indices[0]] = 2  # the first page of request 0: its tokens 0..7
    assert j.run() == 4
    j.check(range(8))
    j = job()
    page = j.indices[j.indptr[1] + 2]  # token 20 .. 23 of request 1
    j.indices = j.indices.copy()
    j.indices[j.indptr[1] + 2] = j.pages
    assert j.run() == 1
    j.indices[j.indptr[1] + 2] = page
    j.check([12, 13, 14, 15])
    j = job()
    j.indptr = j.indptr.copy()
    j.indptr[2] = len(j.indices) + 1
    assert j.run() == 5


def test_quant_append_equals_packing_the_bf16_pages():
    """K and V appended to 4-bit pages = appended as bf16, then packed (where the float rotation
    rounds like the exact one, all but a few in ten thousand rows' values)."""
    a = Job([0, 40], [64, 24], 4, 2, 16, "NHD", 3, True, seed=9)
    b = Job([0, 40], [64, 24], 4, 2, 16, "NHD", 3, False, seed=9)
    assert a.run() == 0 and b.run() == 0
    packed = [torch.full_like(x, 0xA5) for x in a.dev]
    scales = [torch.full_like(x, 3.0) for x in a.dev_s]
    n = a.pages
    desc = oxd.make_copy_pages_desc(n, 2, 16, "bf16", "NHD", n, "e2m1", "NHD", n)
    ids = torch.arange(n, dtype=torch.int32, device="cuda")
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    oxd.oxd_copy_pages(desc, oxd.KvPools(*b.dev), oxd.KvPools(*packed, *scales), ids, ids, None, ws)
    page, slot = a.indices[a.indptr[a.req] + a.pos // 16], a.pos % 16
    page, slot = torch.as_tensor(page, device="cuda").long(), torch.as_tensor(slot, device="cuda").long()
    assert torch.equal(packed[1][page, slot], a.dev[1][page, slot])
    assert torch.equal(scales[1][page, :, slot], a.dev_s[1][page, :, slot])
    assert (packed[0][page, slot] != a.dev[0][page, slot]).float().mean() < 1e-3


@pytest.mark.parametrize("four", [False, True])
def test_many_tokens(four):
    j = Job([0, 3, 1000], [2100, 700, 1300], 8, 2, 16, "NHD", 3, four, seed=10, far=5000)
    assert j.run() == 0
    j.check()


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("Hq,Hkv", [(512, 64), (3, 50), (1000, 1)])
def test_many_heads(four, Hq, Hkv):
    j = Job([5, 0, 16], [2, 1, 1], Hq, Hkv, 8, "NHD", 2, four, seed=31)
    assert j.run() == 0
    j.check()


@pytest.mark.parametrize("four", [False, True])
def test_a_captured_step_replays_on_new_rows_and_positions(four):
    """A decode step's append, captured once: the rows, slots and rope positions are what the tensors
    hold at each replay, and a replayed call leaves what an eager one would."""
    B, Hq, Hkv, ps, pages = 5, 8, 2, 8, 20
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.zeros(B, Hq, 128, dtype=torch.bfloat16, device="cuda")
    k, v = (torch.zeros(B, Hkv, 128, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    i32 = lambda a: torch.as_tensor(np.asarray(a, np.int32), device="cuda")  # noqa: E731
    req, pos, rope = i32(np.arange(B)), i32(np.zeros(B)), i32(np.zeros((3, B)))
    indptr, indices = i32(np.arange(0, pages + 1, pages // B)), i32(np.arange(pages)[::-1].copy())
    ref = torch.ones(pages, dtype=torch.int32, device="cuda")
    desc = oxd.make_axes_append_desc(B, B, Hq, Hkv, ps, "NHD", pages, pages, sections=[16, 24, 24])

    def pools():
        if not four:
            return [torch.zeros(pages, ps, Hkv, 128, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        return ([torch.zeros(pages, ps, Hkv, 64, dtype=torch.uint8, device="cuda") for _ in "kv"] +
                [torch.zeros(pages, Hkv, ps, 4, dtype=torch.float16, device="cuda") for _ in "kv"])

    def call(to, q_out, ws):
        args = (desc, q, k, v, req, pos, rope, indptr, indices, ref, q_out)
        if four:
            oxd.oxd_quant_rope_append(*args, oxd.KvPools(*to), ws)
        else:
            oxd.oxd_rope_axes_append(*args, *to, ws)

    a, b = pools(), pools()
    qa, qb = torch.empty_like(q), torch.empty_like(q)
    wa, wb = (torch.zeros(256, dtype=torch.uint8, device="cuda") for _ in "ab")
    call(a, qa, wa)
    torch.cuda.synchronize()
    for x in a:
        x.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(a, qa, wa)
    for step in range(6):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, device="cuda", generator=g))
        pos.copy_(torch.arange(B, device="cuda") + 5 * step)
        rope.copy_(torch.randint(0, 3000, rope.shape, device="cuda", generator=g))
        graph.replay()
        call(b, qb, wb)
        assert torch.equal(qa, qb)
        for x, y in zip(a, b):
            assert torch.equal(x, y)
        assert oxd.oxd_read_device_status(wa) == oxd.oxd_read_device_status(wb) == 0


@pytest.mark.parametrize("T", [40, 700])
def test_infinite_and_overflowing_keys_are_held_as_the_formats_ends(T):
    """A rotation that ends at an infinity, from an infinite column or past the largest float, is held
    as +-65472 with its sign, in even and odd columns alike, and its group's other columns against
    that scale; the bf16 append and a pack of its pages come to the same."""
    j = Job([1], [T], 1, 2, 16, "NHD", 1, True, seed=31)
    rng = np.random.default_rng(32)
    kinds = np.array([np.inf, -np.inf, 3e38, -3e38, 1.8e38])
    for t in range(T):
        # one column of a pair infinite, or both large: no inf - inf, which is a NaN by the formula
        col = rng.integers(0, 64)
        x = R.round_bf16(rng.choice(kinds))
        j.k[t, 0, col + 64 * rng.integers(0, 2)] = x
        if np.isfinite(x):
            j.k[t, 0, [col, col + 64]] = x * rng.choice([-1, 1], 2)
    assert np.isnan(j.rotated(j.k)).sum() == 0
    assert j.run() == 0
    j.check()


def far_rotation(x, rope, pair_axis, theta):
    """As R.rotate, the angles reduced in whole numbers: good to 2^-52 at any position."""
    with localcontext() as c:
        c.prec = 60
        pi = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
        turn = 1 << 120
        f = [int((-Decimal(theta).ln() * i / 64).exp() / (2 * pi) * turn) for i in range(64)]
    part = np.array([[int(p) * f[i] % turn / turn for i, p in enumerate(row)]
                     for row in np.asarray(rope)[np.asarray(pair_axis)].T])
    cos, sin = np.cos(2 * np.pi * part)[:, None], np.sin(2 * np.pi * part)[:, None]
    lo, hi = x[..., :64], x[..., 64:]
    return np.concatenate([lo * cos - hi * sin, hi * cos + lo * sin], -1)


@pytest.mark.parametrize("theta", [10000.0, 5e6])
def test_codes_at_the_farthest_positions(theta):
    """Every code and scale is the exactly rotated row's up to position 2^24 - 1."""
    j = Job([0], [2500], 1, 5, 16, "HND", 2, True, seed=33)
    j.theta = theta
    j.rope = np.random.default_rng(34).integers(1 << 23, 1 << 24, (2, j.T))
    j.rope[:, :4] = (1 << 24) - 1 - np.arange(8).reshape(2, 4)
    j.rotated = lambda x: far_rotation(x, j.rope, j.pair_axis, theta)
    assert j.run() == 0
    j.check()
