"""Windowed servers of different data on two streams at once, tables of two streams in flight together, copies
between captured launches, and more bf16 streams than the GPU holds (GPU)."""
import numpy as np
import pytest
import torch

import paged_kv_decode_attn_gb300 as oxd
import test_build_tables as T
import test_window_decode as D
import window_ref as Wr
from quant_helpers import bf16, f64
from test_window_flow import SCALE, Server, dev, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    oxd.build()


def test_two_servers_of_different_data():
    """Different sizes, lengths, windows and rows; each step's outputs against f64 over the server's own pools."""
    shapes = [dict(B=2, G=4, Hkv=2, ps=16, layout="NHD", window=30, sinks=3), dict(B=5, G=8, Hkv=1, ps=8,
              layout="HND", window=100, sinks=0)]
    starts = [[5, 90], [60, 1, 17, 33, 64]]
    steps, servers = 12, []
    rng = np.random.default_rng(3)
    for c, n in zip(shapes, starts):
        s = Server(four=False, **c)
        s.n, s.stream = n, torch.cuda.Stream()
        s.data = [[bf16(rng.normal(size=(s.B, h, 128))) for h in (s.Hq, s.Hkv, s.Hkv)] for _ in range(steps)]
        s.fill = [bf16(rng.normal(size=tuple(p.shape))) for p in s.pools]
        s.maps = [(ints(s.B), ints(s.B)) for _ in range(steps)]
        s.outs = [(torch.empty_like(q), torch.empty_like(q), torch.empty((s.B, s.Hq), device="cuda"))
                  for q, _, _ in s.data]
        s.ones, s.start = dev([1] * s.B), dev(n)
        s.kept = [[] for _ in range(steps)]
        servers.append(s)
    torch.cuda.synchronize()
    for s in servers:
        with torch.cuda.stream(s.stream):
            s.lengths.copy_(s.start)
            s.tables(s.start, 0, (None, None))
            for p, x in zip(s.pools, s.fill):
                p.copy_(x)
    for i in range(steps):
        for s in servers:
            with torch.cuda.stream(s.stream):
                s.lengths += 1
                s.tables(s.ones, s.B, s.maps[i])
                s.append(*s.data[i], s.maps[i], s.outs[i][0])
                s.decode(*s.outs[i], pdl=1)
                s.kept[i] = [x.clone() for x in (*s.pools, s.rows)]
    torch.cuda.synchronize()
    for s in servers:
        assert oxd.oxd_read_device_status(s.ws) == 0
        rows = s.rows.cpu().numpy()
        used = [rows[b, j] for b in range(s.B) for j in range(-(-(s.n[b] + steps) // s.ps))]
        assert len(set(used)) == len(used) == s.taken.item() and min(used) >= 0
        for i in range(steps):
            lengths = [x + i + 1 for x in s.n]
            assert s.maps[i][0].tolist() == list(range(s.B))
            assert s.maps[i][1].tolist() == [x - 1 for x in lengths]
            now = s.lengths.clone()
            s.lengths.copy_(dev(lengths))
            *pools, s.rows = s.kept[i]
            s.pools = pools
            k, v = s.cached()
            s.lengths.copy_(now)
            for b, length in enumerate(lengths):  # the step's V row is where the tables put it
                assert np.array_equal(v[b][:, length - 1], f64(s.data[i][2])[b])
            ref = Wr.attention(f64(s.outs[i][0]), k, v, lengths, [1] * s.B, s.window, s.sinks, SCALE)
            Wr.assert_close(f64(s.outs[i][1]), f64(s.outs[i][2]), ref, f"step {i}")


def test_tables_of_two_streams_in_flight_together():
    """Twenty calls a stream, in place, enqueued before anything is read."""
    runs = []
    for k, (B, ps, window) in enumerate(((200, 16, 500), (70, 8, 0))):
        rng = np.random.default_rng(20 + k)
        lengths = rng.integers(1, 400, B)
        s = T.state(lengths, np.ones(B, int), ps, seed=k, width=80, extra_free=B * 4)
        n_idx = B * 80
        o = dict(rows=dev(s["rows"]), held_out=dev(s["held"]), taken_out=dev([0]), refcount=dev(s["refcount"]),
                 indptr=ints(B + 1), indices=ints(n_idx), last_page_len=ints(B), qo_indptr=ints(B + 1),
                 token_request=ints(B), positions=ints(B), slots=ints(B, dtype=torch.int64))
        runs.append(dict(s=s, o=o, B=B, ps=ps, window=window, n_idx=n_idx, lengths=dev(lengths), ones=dev([1] * B),
                         free=dev(s["free"]), ws=torch.empty(256, dtype=torch.uint8, device="cuda"),
                         stream=torch.cuda.Stream()))
    torch.cuda.synchronize()
    steps = 20
    for _ in range(steps):
        for r in runs:
            o = r["o"]
            d = oxd.make_build_tables_desc(r["B"], r["ps"], 80, len(r["s"]["refcount"]), r["n_idx"], r["B"],
                                           len(r["free"]), r["window"], 4)
            with torch.cuda.stream(r["stream"]):
                oxd.oxd_build_tables(d, r["lengths"], r["ones"], o["rows"], o["held_out"], o["held_out"], r["free"],
                                     o["taken_out"], o["taken_out"], o["refcount"], o["indptr"], o["indices"],
                                     o["last_page_len"], o["qo_indptr"], o["token_request"], o["positions"],
                                     o["slots"], r["ws"])
                r["lengths"] += 1
    torch.cuda.synchronize()
    for r in runs:
        assert oxd.oxd_read_device_status(r["ws"]) == 0
        at = {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in r["s"].items()}
        for _ in range(steps):
            ref = T.reference(at, r["ps"], r["window"], 4, r["n_idx"], r["B"])
            at.update(lengths=at["lengths"] + 1, held=ref["held_out"], rows=ref["rows"].astype(np.int32),
                      taken=int(ref["taken_out"][0]), refcount=ref["refcount"])
        got = {n: t.cpu().numpy().astype(np.int64) for n, t in r["o"].items()}
        n = ref["indptr"][-1]  # (entries behind it are earlier steps')
        got["indices"], ref["indices"] = got["indices"][:n], ref["indices"][:n]
        T.compare(got, ref)


def test_copies_between_captured_launches():
    """A copy or a fill between two launches of a graph makes the second a plain one: it sees what was copied."""
    c = D.Case([300, 40, 500], 4, 2, 16, "NHD", 64, 4, seed=12)
    other = D.Case([300, 40, 500], 4, 2, 16, "NHD", 64, 4, seed=13)
    desc = c.desc()
    out = [torch.zeros_like(c.d_q) for _ in range(2)]
    lse = [torch.zeros((3, 8), device="cuda") for _ in range(2)]
    q, k, v = (torch.empty_like(x) for x in (c.d_q, c.d_k, c.d_v))
    tables = [torch.empty_like(x) for x in c.tables]

    def step():
        for i, x in enumerate((c, other)):
            for dst, src in zip((q, k, v, *tables), (x.d_q, x.d_k, x.d_v, *x.tables)):
                dst.copy_(src)
            oxd.oxd_window_decode(desc, q, k, v, *tables, SCALE, out[i], lse[i], c.ws)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(10):
        for o, z in zip(out, lse):
            o.zero_()
            z.zero_()
        g.replay()
        for x, o, z in zip((c, other), out, lse):
            Wr.assert_close(f64(o), f64(z), x.reference())


@pytest.mark.parametrize("G", [1, 8, 12, 32])
@pytest.mark.parametrize("batch,window,sinks", [(700, 40, 3), (330, 4096, 5), (900, 4096, 17)])
def test_more_bf16_streams_than_the_gpu_holds(batch, window, sinks, G):
    """Several waves, and from 4096 tokens clusters of two although not all are resident."""
    rng = np.random.default_rng(batch + G)
    lengths = rng.integers(0, 80, batch)
    lengths[[3, batch - 1]] = 5000, 4400
    c = D.Case(list(map(int, lengths)), G, 2, 16, "NHD", window, sinks, seed=G)
    out, lse = c.check()
    o, z = c.check(max_splits=1)
    if window < 4096:
        assert torch.equal(o, out) and torch.equal(z, lse)
