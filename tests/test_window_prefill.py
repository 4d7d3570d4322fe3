"""Causal prefill with a sliding window and sinks: planning on the CPU, runs against f64 (GPU)."""
import os

import numpy as np
import pytest
import torch

import paged_kv_decode_attn_gb300 as oxd
import window_ref as Wr
from quant_helpers import bf16, f64

SCALE = 128 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def built():
    oxd.build()


def tables(lengths, ps):
    pages = -(-np.asarray(lengths) // ps)
    indptr = np.concatenate([[0], np.cumsum(pages)])
    return indptr, np.asarray(lengths) - (pages - 1) * ps


def plan(lengths, q_lens, window, sinks, G=4, Hkv=2, ps=16, num_sms=152, **kw):
    indptr, last = tables(lengths, ps)
    desc = oxd.make_prefill_desc(len(lengths), G * Hkv, Hkv, ps, "NHD", int(indptr[-1]),
                                 num_sms=num_sms, **kw)
    return oxd.oxd_window_prefill_plan(desc, window, sinks, np.concatenate([[0], np.cumsum(q_lens)]),
                                       indptr, last)


def status(call):
    try:
        call()
    except oxd.OxdError as e:
        return e.status
    return 0


@pytest.mark.parametrize("window,sinks,want", [(0, 0, 1), (-1, 0, 1), (1, -1, 1), (1 << 30, 1, 2),
                                               (1 << 30, 0, 0), (1, (1 << 30) - 1, 0)])
def test_plan_refusals(window, sinks, want):
    assert status(lambda: plan([100], [10], window, sinks)) == want


def test_plan_refuses_what_the_plain_plan_refuses():
    assert status(lambda: plan([100], [101], 5, 0)) == 1
    assert status(lambda: plan([100], [0], 5, 0)) == 1
    assert status(lambda: plan([100], [10], 5, 0, ps=12)) == 2
    assert status(lambda: plan([100], [10], 5, 0, G=129, Hkv=1)) == 2


@pytest.mark.parametrize("lengths,q_lens,window,sinks", [
    ([100], [100], 7, 0), ([100], [100], 7, 3), ([100, 40], [30, 40], 20, 30), ([500], [1], 64, 4),
    ([64, 64], [64, 0], 100, 0), ([10], [10], 4, 20)])
def test_plan_counts_the_pairs_that_the_window_leaves(lengths, q_lens, window, sinks):
    want = sum(len(Wr.seen(n - q + i, n, window, sinks))
               for n, q in zip(lengths, q_lens) for i in range(q))
    assert plan(lengths, q_lens, window, sinks).info.causal_pairs == want


# ------------------------------------------------------------------ runs

gpu = pytest.mark.gpu


def dev(a):
    return torch.as_tensor(np.asarray(a, np.int32), device="cuda")


class Case:
    def __init__(self, lengths, q_lens, G, Hkv, ps, layout, window, sinks, seed=0, sigma=1.0, **kw):
        if not torch.cuda.is_available():
            pytest.skip("no CUDA device")
        self.p = Wr.Paged(lengths, q_lens, Hkv, ps, layout, window, sinks, seed, sigma, **kw)
        self.Hq, self.window, self.sinks = G * Hkv, window, sinks
        self.q = self.p.queries(self.Hq)
        self.d_q, self.d_k, self.d_v = bf16(self.q), *(bf16(x) for x in self.p.pools)
        self.qo = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        self.tables = [dev(self.qo), dev(self.p.indptr), dev(self.p.indices), dev(self.p.last)]

    def plan(self, **kw):
        p = self.p
        desc = oxd.make_prefill_desc(len(p.lengths), self.Hq, p.Hkv, p.ps, p.layout, p.num_pages, **kw)
        return oxd.oxd_window_prefill_plan(desc, self.window, self.sinks, self.qo, p.indptr, p.last,
                                           torch.cuda.current_device())

    def run(self, plan, scale=SCALE, bind=False, stream=None):
        n = len(self.q) * self.Hq
        out = torch.full((n * 128 + 256,), 77.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((n + 8,), 77.0, device="cuda")
        ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
        if bind:
            oxd.oxd_prefill_plan_bind_workspace(plan, ws)
        oxd.oxd_paged_prefill_run(plan, self.d_q, self.d_k, self.d_v, *self.tables, scale,
                                  out[128:-128], lse[4:-4], ws, stream=stream)
        self.code = oxd.oxd_read_device_status(ws, stream)
        assert (out[:128] == 77).all() and (out[-128:] == 77).all()
        assert (lse[:4] == 77).all() and (lse[-4:] == 77).all()
        return out[128:-128].view(-1, self.Hq, 128), lse[4:-4].view(-1, self.Hq)

    def reference(self, scale=SCALE):
        return Wr.attention(self.q, self.p.k, self.p.v, self.p.lengths, self.p.q_lens, self.window,
                            self.sinks, scale)

    def check(self, scale=SCALE, bind=False, **kw):
        out, lse = self.run(self.plan(**kw), scale, bind)
        assert self.code == 0
        Wr.assert_close(f64(out), f64(lse), self.reference(scale), str(kw))
        return out, lse


WINDOWS = [(1, 0), (1, 1), (5, 3), (64, 0), (100, 4), (128, 64), (129, 130), (300, 17), (1000, 0)]


@gpu
@pytest.mark.parametrize("rows", [128, 256])
@pytest.mark.parametrize("layout,ps", [("NHD", 8), ("HND", 16), ("NHD", 32), ("HND", 64), ("NHD", 16)])
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_prompts_windows_and_sinks(rows, layout, ps, window, sinks):
    """Rows that no query sees, and pages, are NaN or not listed."""
    c = Case([300, 1, 65, 700, 129], [300, 1, 10, 90, 128], 4, 1, ps, layout, window, sinks,
             seed=window + ps)
    c.check(tile_rows=rows)
    c.check(tile_rows=rows, max_splits=1, bind=True)


@gpu
@pytest.mark.parametrize("rows", [128, 256])
@pytest.mark.parametrize("G", [1, 2, 3, 5, 8, 16, 32, 100, 128])
def test_groups(rows, G):
    Case([200, 97], [70, 33], G, 1, 16, "NHD", 50, 6, seed=G).check(tile_rows=rows)


@gpu
@pytest.mark.parametrize("rows", [128, 256])
@pytest.mark.parametrize("splits", [1, 2, 3, 7, 0])
@pytest.mark.parametrize("window,sinks", [(700, 0), (600, 200), (1500, 1)])
def test_pieces_of_long_tiles(rows, splits, window, sinks):
    """Pieces that start among the sinks, cross the gap, and start behind it."""
    Case([2000], [20], 4, 1, 16, "NHD", window, sinks, seed=splits).check(tile_rows=rows,
                                                                        max_splits=splits)


@gpu
@pytest.mark.parametrize("rows", [128, 256])
@pytest.mark.parametrize("q_len", [1, 2, 31, 33, 63, 64, 65, 127, 128])
def test_few_queries_at_the_end_of_a_long_request(rows, q_len):
    Case([1500], [q_len], 4, 2, 16, "HND", 333, 40, seed=q_len).check(tile_rows=rows)


@gpu
@pytest.mark.parametrize("rows", [128, 256])
@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0, 4.0])
def test_scales(rows, scale):
    Case([400], [300], 4, 1, 16, "NHD", 90, 4, seed=8).check(scale, tile_rows=rows)


@gpu
@pytest.mark.parametrize("rows", [128, 256])
def test_growing_keys_raise_the_maximum(rows):
    c = Case([600], [500], 4, 1, 16, "NHD", 257, 4, seed=2, poison=0.0)
    grow = torch.linspace(0.1, 20, 600, device="cuda")
    sign = torch.sign(c.d_q[0, 0].float())
    p = c.p
    k = (grow[:, None] * sign).to(torch.bfloat16)
    for j, page in enumerate(p.indices):
        if page >= 0:
            rows_here = k[j * 16:j * 16 + 16]
            c.d_k[int(page), :len(rows_here), 0] = rows_here
    p.k[0] = f64(k)[None]
    c.check(tile_rows=rows)


@gpu
@pytest.mark.parametrize("rows", [128, 256])
def test_a_window_over_everything_is_the_plain_prefill(rows):
    c = Case([500, 64], [500, 3], 4, 2, 16, "NHD", 500, 3, seed=4)
    out, lse = c.check(tile_rows=rows)
    p = c.p
    desc = oxd.make_prefill_desc(2, 8, 2, 16, "NHD", p.num_pages, tile_rows=rows)
    plain = oxd.oxd_paged_prefill_plan(desc, c.qo, p.indptr, p.last)
    o2, l2 = c.run(plain)
    assert torch.equal(out, o2) and torch.equal(lse, l2)


@gpu
@pytest.mark.parametrize("rows", [128, 256])
def test_the_last_query_is_the_window_decode(rows):
    c = Case([900, 300], [40, 1], 4, 2, 16, "NHD", 200, 10, seed=5)
    out, lse = c.check(tile_rows=rows)
    p = c.p
    last = [39, 40]
    d = oxd.make_window_decode_desc(2, 8, 2, 16, "NHD", p.num_pages, len(p.indices), 200, 10)
    o, z = torch.empty_like(out[last]), torch.empty_like(lse[last])
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    oxd.oxd_window_decode(d, c.d_q[last].contiguous(), c.d_k, c.d_v, *c.tables[1:], SCALE, o, z, ws)
    ref = [x[last] for x in c.reference()]
    Wr.assert_close(f64(o), f64(z), ref)
    Wr.assert_close(f64(out[last]), f64(lse[last]), ref)


@gpu
@pytest.mark.parametrize("rows", [128, 256])
def test_runs_are_bitwise_equal_on_any_stream(rows):
    c = Case([2000, 150], [333, 150], 4, 2, 16, "NHD", 300, 9, seed=6)
    plan = c.plan(tile_rows=rows)
    out, lse = c.run(plan)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for i in range(10):
        o, z = c.run(plan, stream=s if i % 2 else None)
        assert torch.equal(o, out) and torch.equal(z, lse)


@gpu
@pytest.mark.parametrize("rows", [128, 256])
def test_unseen_pages_are_not_looked_at_and_bad_ones_recorded(rows):
    c = Case([1000, 60], [30, 20], 4, 1, 16, "NHD", 100, 20, unseen=1 << 30, seed=7)
    c.check(tile_rows=rows)
    idx = c.p.indices.copy()
    idx[c.p.indptr[1] - 1] = -1  # request 0's last page, which is seen
    c.tables[2] = dev(idx)
    out, lse = c.run(c.plan(tile_rows=rows))
    assert c.code == oxd.OXD_DEVICE_BAD_PAGE
    ref = [x[30:] for x in c.reference()]
    Wr.assert_close(f64(out[30:]), f64(lse[30:]), ref)


@gpu
@pytest.mark.parametrize("rows", [128, 256])
def test_tables_that_differ_from_the_plan_are_recorded(rows):
    c = Case([1000, 60], [30, 20], 4, 1, 16, "NHD", 100, 20, seed=7)
    c.tables[3][0] -= 1
    c.run(c.plan(tile_rows=rows))
    assert c.code == oxd.OXD_DEVICE_PLAN_MISMATCH


@gpu
@pytest.mark.parametrize("rows", [128, 256])
def test_a_wait_that_runs_out_is_reported(rows):
    c = Case([1500], [300], 4, 2, 16, "NHD", 700, 9, seed=8)
    for _ in range(5):
        c.run(c.plan(tile_rows=rows, wait_timeout_ns=1))
        if c.code == oxd.OXD_DEVICE_WAIT_TIMEOUT:
            break
    assert c.code == oxd.OXD_DEVICE_WAIT_TIMEOUT
    c.check(tile_rows=rows)  # the next run is unaffected


@gpu
@pytest.mark.parametrize("rows", [128, 256])
def test_a_captured_run(rows):
    c = Case([800], [200], 4, 1, 16, "NHD", 150, 5, seed=9)
    plan = c.plan(tile_rows=rows)
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    oxd.oxd_prefill_plan_bind_workspace(plan, ws)
    out = torch.empty_like(c.d_q)
    lse = torch.empty(c.d_q.shape[:2], device="cuda")

    def call():
        oxd.oxd_paged_prefill_run(plan, c.d_q, c.d_k, c.d_v, *c.tables, SCALE, out, lse, ws)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    out.zero_()
    g.replay()
    Wr.assert_close(f64(out), f64(lse), c.reference())


# ------------------------------------------------------------------ many pieces a CTA, and at random

@gpu
@pytest.mark.parametrize("rows", [128, 256])
@pytest.mark.parametrize("layout,G,Hkv,window,sinks", [("NHD", 4, 8, 200, 4), ("HND", 1, 16, 40, 0),
                                                       ("NHD", 12, 3, 333, 20)])
def test_more_tiles_than_resident_ctas(rows, layout, G, Hkv, window, sinks):
    lengths = [700, 64, 1300, 65, 900, 1, 500, 640, 777, 1000]
    q_lens = [700, 64, 900, 1, 300, 1, 500, 63, 700, 640]
    c = Case(lengths, q_lens, G, Hkv, 16, layout, window, sinks, seed=rows + G)
    for splits in (0, 1):
        out, lse = c.run(c.plan(tile_rows=rows, max_splits=splits), bind=True)
        assert c.code == 0
        ref = Wr.attention_torch(c.q, c.p.k, c.p.v, lengths, q_lens, window, sinks, SCALE)
        Wr.assert_close(f64(out), f64(lse), ref, f"splits {splits}")


@gpu
@pytest.mark.parametrize("seed", range(40 * int(os.environ.get("OXD_FUZZ_SCALE", "1"))))
def test_random_prefills(seed):
    rng = np.random.default_rng(1000 + seed)
    B = int(rng.integers(1, 6))
    lengths = [int(np.exp(rng.uniform(0, np.log(1500)))) for _ in range(B)]
    q_lens = [int(rng.integers(0, n + 1)) for n in lengths]
    q_lens[0] = max(q_lens[0], 1)
    G, Hkv = int(rng.choice([1, 2, 3, 4, 6, 8, 16, 40])), int(rng.choice([1, 2, 3]))
    window, sinks = int(np.exp(rng.uniform(0, np.log(1200)))), int(rng.choice([0, 1, 4, 33, 130, 300]))
    ps, layout = int(rng.choice([8, 16, 32, 64])), str(rng.choice(["NHD", "HND"]))
    scale = float(rng.choice([SCALE, -SCALE, 0.5]))
    c = Case(lengths, q_lens, G, Hkv, ps, layout, window, sinks, seed=seed, sigma=float(rng.choice([0.5, 1, 2])))
    out, lse = c.run(c.plan(tile_rows=int(rng.choice([0, 128, 256])), max_splits=int(rng.choice([0, 1, 3]))),
                     scale)
    assert c.code == 0
    ref = Wr.attention_torch(c.q, c.p.k, c.p.v, lengths, q_lens, window, sinks, scale)
    Wr.assert_close(f64(out), f64(lse), ref, f"{lengths} {q_lens} {G} {Hkv} {window} {sinks} {ps}")


@gpu
@pytest.mark.parametrize("rows", [128, 256])
def test_a_damaged_bound_list_is_reported_and_not_followed(rows):
    """Random words over a bound work list: reported, nothing written outside the outputs."""
    c = Case([1500, 300], [300, 40], 4, 2, 16, "NHD", 200, 9, seed=8)
    plan = c.plan(tile_rows=rows)
    n = len(c.q) * c.Hq
    rng = np.random.default_rng(5)
    out = torch.full((n * 128 + 256,), 77.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n + 8,), 77.0, device="cuda")
    ws = torch.empty(plan.workspace_bytes + 256, dtype=torch.uint8, device="cuda")
    for trial in range(12):
        ws[plan.workspace_bytes:] = 55
        oxd.oxd_prefill_plan_bind_workspace(plan, ws, plan.workspace_bytes)
        words = ws[256:256 + plan.info.num_units * 64].view(torch.int32)
        at = torch.as_tensor(rng.integers(0, len(words), 1 + trial * 5), device="cuda")
        words[at] = torch.as_tensor(rng.integers(-2 ** 31, 2 ** 31, len(at)).astype(np.int32), device="cuda")
        oxd.oxd_paged_prefill_run(plan, c.d_q, c.d_k, c.d_v, *c.tables, SCALE, out[128:-128], lse[4:-4],
                                  ws, plan.workspace_bytes)
        oxd.oxd_read_device_status(ws)
        assert (out[:128] == 77).all() and (out[-128:] == 77).all() and (ws[plan.workspace_bytes:] == 55).all()
        assert (lse[:4] == 77).all() and (lse[-4:] == 77).all()
    # every field of every unit at the ends of its type
    for field in range(16):
        for value in (-2 ** 31, -1, 0, 2 ** 30, 2 ** 31 - 1):
            oxd.oxd_prefill_plan_bind_workspace(plan, ws, plan.workspace_bytes)
            words.view(-1, 16)[:, field] = value
            oxd.oxd_paged_prefill_run(plan, c.d_q, c.d_k, c.d_v, *c.tables, SCALE, out[128:-128],
                                      lse[4:-4], ws, plan.workspace_bytes)
            oxd.oxd_read_device_status(ws)
            assert (out[:128] == 77).all() and (out[-128:] == 77).all()
            assert (lse[:4] == 77).all() and (lse[-4:] == 77).all()
            assert (ws[plan.workspace_bytes:] == 55).all()
    words[:] = -1
    oxd.oxd_paged_prefill_run(plan, c.d_q, c.d_k, c.d_v, *c.tables, SCALE, out[128:-128], lse[4:-4], ws,
                              plan.workspace_bytes)
    assert oxd.oxd_read_device_status(ws) == oxd.OXD_DEVICE_PLAN_MISMATCH
    c.check(tile_rows=rows)
