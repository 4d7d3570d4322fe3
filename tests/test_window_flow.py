"""A windowed model served as a program would: tables built on the GPU, prompts appended and
prefilled, then decode steps in one captured graph whose lengths advance on the device."""
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


def ints(*shape, dtype=torch.int32):
    return torch.full(shape, -9, dtype=dtype, device="cuda")


class Server:
    """The state of a serving loop on the device: page rows, free list, pools and tables."""

    def __init__(self, B, G, Hkv, ps, layout, window, sinks, four, pool=64, width=16):
        self.B, self.Hq, self.Hkv, self.ps, self.layout = B, G * Hkv, Hkv, ps, layout
        self.window, self.sinks, self.four, self.pool = window, sinks, four, pool
        rng = np.random.default_rng(B + G)
        self.lengths, self.rows = dev([0] * B), ints(B, width)
        self.held, self.taken = dev([0] * B), dev([0])
        self.free, self.refcount = dev(rng.permutation(pool)), dev([0] * pool)
        self.indptr, self.last, self.qo = ints(B + 1), ints(B), ints(B + 1)
        self.indices = ints(B * width)
        self.ws = torch.empty(256, dtype=torch.uint8, device="cuda")
        shape = (lambda n: (pool, ps, Hkv, n) if layout == "NHD" else (pool, Hkv, ps, n))
        if four:
            self.pools = [torch.zeros(shape(64), dtype=torch.uint8, device="cuda") for _ in "kv"]
            self.pools += [torch.full((pool, Hkv, ps, 4), float("nan"), dtype=torch.float16,
                                      device="cuda") for _ in "kv"]
        else:
            self.pools = [torch.full(shape(128), float("nan"), dtype=torch.bfloat16, device="cuda")
                          for _ in "kv"]
        self.cache = oxd.KvPools(*self.pools)

    def tables(self, new, T, maps):
        d = oxd.make_build_tables_desc(self.B, self.ps, self.rows.shape[1], self.pool,
                                       len(self.indices), T, len(self.free), self.window, self.sinks)
        oxd.oxd_build_tables(d, self.lengths, new, self.rows, self.held, self.held, self.free,
                             self.taken, self.taken, self.refcount, self.indptr, self.indices,
                             self.last, self.qo, *maps, None, self.ws)

    def append(self, q, k, v, maps, q_out):
        d = oxd.make_axes_append_desc(len(q), self.B, self.Hq, self.Hkv, self.ps, self.layout,
                                      self.pool, len(self.indices))
        args = (d, q, k, v, *maps, None, self.indptr, self.indices, self.refcount, q_out)
        if self.four:
            oxd.oxd_quant_rope_append(*args, self.cache, self.ws)
        else:
            oxd.oxd_rope_axes_append(*args, *self.pools, self.ws)

    def decode(self, q, out, lse, pdl):
        d = oxd.make_window_decode_desc(self.B, self.Hq, self.Hkv, self.ps, self.layout, self.pool,
                                        len(self.indices), self.window, self.sinks, pdl=pdl)
        args = (self.indptr, self.indices, self.last, SCALE, out, lse, self.ws)
        if self.four:
            oxd.oxd_quant_window_decode(d, q, self.cache, *args)
        else:
            oxd.oxd_window_decode(d, q, *self.pools, *args)

    def cached(self):
        """The rows of every request as the pools hold them, by the rows of pages: [Hkv, L, 128]."""
        pools = [p.cpu().numpy() if self.four else f64(p) for p in self.pools]
        if self.four:
            with np.errstate(invalid="ignore"):
                pools = [R.pool_values(pools[i], pools[2 + i], self.layout) for i in range(2)]
        rows = self.rows.cpu().numpy()
        got = []
        for pool in pools:
            got.append([R.tokens(pool, rows[b, :-(-n // self.ps)], self.layout)[:, :n] if n else
                        np.zeros((self.Hkv, 0, 128)) for b, n in enumerate(self.lengths.tolist())])
        return got


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("layout,G,Hkv,window,sinks", [("NHD", 4, 2, 40, 4), ("HND", 1, 3, 17, 0),
                                                       ("NHD", 16, 1, 64, 20)])
def test_prompts_then_captured_decode_steps(four, layout, G, Hkv, window, sinks):
    B, ps, steps = 3, 16, 20
    s = Server(B, G, Hkv, ps, layout, window, sinks, four)
    rng = np.random.default_rng(1)
    n = [50, 7, 33]
    T = sum(n)
    rows = (lambda t, h: bf16(rng.normal(size=(t, h, 128))))
    # ---- prompts: tables, append and, over bf16 pages, the prefill
    s.lengths.copy_(dev(n))
    maps = ints(T), ints(T)
    s.tables(dev(n), T, maps)
    assert oxd.oxd_read_device_status(s.ws) == 0
    assert s.taken.item() == sum(-(-x // ps) for x in n)
    q = rows(T, s.Hq)
    s.append(q, rows(T, Hkv), rows(T, Hkv), maps, q)
    assert oxd.oxd_read_device_status(s.ws) == 0
    if not four:
        pages = [-(-x // ps) for x in n]
        qo, indptr = np.concatenate([[0], np.cumsum(n)]), np.concatenate([[0], np.cumsum(pages)])
        assert s.qo.tolist() == qo.tolist() and s.indptr.tolist() == indptr.tolist()
        desc = oxd.make_prefill_desc(B, s.Hq, Hkv, ps, layout, s.pool)
        plan = oxd.oxd_window_prefill_plan(desc, window, sinks, qo, indptr, s.last.cpu().numpy())
        ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
        out, lse = torch.empty_like(q), torch.empty((T, s.Hq), device="cuda")
        oxd.oxd_paged_prefill_run(plan, q, *s.pools, s.qo, s.indptr, s.indices, s.last, SCALE, out,
                                  lse, ws)
        assert oxd.oxd_read_device_status(ws) == 0
        k, v = s.cached()
        Wr.assert_close(f64(out), f64(lse), Wr.attention(f64(q), k, v, n, n, window, sinks, SCALE))
    # ---- decode steps: one graph, replayed; nothing on the host knows the lengths
    q, k, v = rows(B, s.Hq), rows(B, Hkv), rows(B, Hkv)
    q_out, out, lse = torch.empty_like(q), torch.empty_like(q), torch.empty((B, s.Hq), device="cuda")
    maps, ones = (ints(B), ints(B)), dev([1] * B)

    def step():
        s.lengths += 1
        s.tables(ones, B, maps)
        s.append(q, k, v, maps, q_out)
        s.decode(q_out, out, lse, pdl=1)

    before = [x.clone() for x in (s.lengths, s.rows, s.held, s.taken, s.refcount, *s.pools)]
    step()  # (first use outside the capture)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for x, y in zip((s.lengths, s.rows, s.held, s.taken, s.refcount, *s.pools), before):
        x.copy_(y)
    for i in range(steps):
        for x, h in ((q, s.Hq), (k, Hkv), (v, Hkv)):
            x.copy_(rows(B, h))
        g.replay()
        assert oxd.oxd_read_device_status(s.ws) == 0
        lengths = [x + i + 1 for x in n]
        assert s.lengths.tolist() == lengths
        kc, vc = s.cached()
        ref = Wr.attention(f64(q_out), kc, vc, lengths, [1] * B, window, sinks, SCALE)
        if four:
            assert_decode(out, lse, ref, f"step {i}")
        else:
            Wr.assert_close(f64(out), f64(lse), ref, f"step {i}")
    # pages out of the window are not listed any more, and may go to others
    idx, indptr = s.indices.cpu().numpy(), s.indptr.cpu().numpy()
    gone = [j for j, p in enumerate(idx[indptr[0]:indptr[1]]) if p < 0]
    first = lengths[0] - window
    assert gone == [j for j in range(-(-lengths[0] // ps)) if j * ps >= sinks and (j + 1) * ps <= first]


def test_two_streams_at_once():
    """Two servers' steps on two streams, each with its own state and workspace."""
    servers = [Server(2, 4, 2, 16, "NHD", 30, 3, False) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in servers]
    rng = np.random.default_rng(3)
    data = [[bf16(rng.normal(size=(2, h, 128))) for h in (8, 2, 2)] for _ in range(30)]
    torch.cuda.synchronize()
    outs = []
    for s, stream in zip(servers, streams):
        with torch.cuda.stream(stream):
            s.lengths.copy_(dev([5, 90]))
            s.tables(dev([5, 90]), 0, (None, None))
            for p in s.pools:
                p.fill_(0.5)
    torch.cuda.synchronize()
    ones = dev([1, 1])
    for q, k, v in data:
        for s, stream in zip(servers, streams):
            with torch.cuda.stream(stream):
                s.lengths += 1
                maps = ints(2), ints(2)
                s.tables(ones, 2, maps)
                q_out, out, lse = torch.empty_like(q), torch.empty_like(q), torch.empty((2, 8), device="cuda")
                s.append(q, k, v, maps, q_out)
                s.decode(q_out, out, lse, pdl=1)
                outs.append((out, lse))
    torch.cuda.synchronize()
    for a, b in zip(outs[::2], outs[1::2]):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for s in servers:
        assert oxd.oxd_read_device_status(s.ws) == 0
