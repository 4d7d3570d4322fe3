"""Decode over a 4-bit cache on the GPU against the f64 reference."""
import numpy as np
import pytest
import torch

import paged_kv_decode_attn_gb300 as oxd
from quant_helpers import Cache, assert_decode, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    oxd.build()


RAGGED = [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 95, 127, 128, 129, 200, 257, 500]


def check(c, sm_scale=128 ** -0.5, **kw):
    plan = c.plan(**kw)
    out, lse, ws = c.run(plan, sm_scale)
    assert oxd.oxd_read_device_status(ws) == 0
    assert_decode(out, lse, c.reference(sm_scale), f"{kw}")
    return plan, out, lse


@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("ps", [8, 16, 32, 64])
@pytest.mark.parametrize("G,Hkv", [(1, 3), (2, 2), (4, 8), (8, 1), (12, 2), (16, 1), (17, 1), (32, 2)])
def test_ragged_batch(G, Hkv, ps, layout):
    check(Cache(RAGGED, G, Hkv, ps, layout, seed=G * 100 + ps))


@pytest.mark.parametrize("G", range(1, 33))
def test_every_group_size(G):
    check(Cache([1, 33, 190], G, 1, 16, "NHD", seed=G))


@pytest.mark.parametrize("L", list(range(1, 70)) + [255, 256, 257, 511, 512, 513])
def test_every_short_length(L):
    check(Cache([L], 4, 2, 8, "HND", seed=L))


@pytest.mark.parametrize("splits", [1, 2, 3, 7, 40])
@pytest.mark.parametrize("G,ps", [(1, 16), (4, 8), (8, 64), (16, 32), (32, 16)])
def test_forced_splits(G, ps, splits):
    check(Cache([1, 64, 300, 1025], G, 2, ps, "NHD", seed=splits), force_splits=splits)
    check(Cache([1, 64, 300, 1025], G, 2, ps, "HND", seed=splits), max_splits=splits)


@pytest.mark.parametrize("G,Hkv,ps,layout,lengths", [
    (4, 8, 16, "NHD", [4096, 512, 1733, 2999]),
    (1, 8, 16, "NHD", [512]),
    (8, 8, 16, "HND", [5000, 128, 9000]),
    (32, 1, 64, "NHD", [20000, 32768]),
    (16, 1, 8, "HND", [12345]),
])
def test_long(G, Hkv, ps, layout, lengths):
    check(Cache(lengths, G, Hkv, ps, layout, seed=5))


@pytest.mark.parametrize("G", [4, 16, 32])
@pytest.mark.parametrize("sm_scale", [0.0, -0.09, 0.5, 3.0])
def test_scales_of_the_logits(G, sm_scale):
    check(Cache([5, 77, 333], G, 2, 16, "NHD", seed=3), sm_scale)


@pytest.mark.parametrize("sigma,q_sigma", [(1e-3, 1.0), (300.0, 1.0), (1.0, 1e-20), (1.0, 1e4),
                                           (40.0, 30.0)])
def test_sizes_of_values(sigma, q_sigma):
    # from weights all equal to a softmax that is one token's
    check(Cache([3, 70, 400], 8, 1, 16, "NHD", seed=4, sigma=sigma, q_sigma=q_sigma),
          128 ** -0.5 / (q_sigma * sigma))
    check(Cache([3, 70, 400], 8, 1, 16, "NHD", seed=4, sigma=sigma, q_sigma=q_sigma),
          30.0 / (q_sigma * sigma))


def test_rising_and_falling_logits():
    # the running maximum moves at every step, or never again after the first
    for order in (1, -1):
        c = Cache([700], 4, 1, 16, "NHD", seed=9)
        k = np.argsort(order * (R_rows(c) @ c.q[0, 0]))
        reorder(c, k)
        check(c, 0.5)


def R_rows(c):
    import quant_ref as R

    return R.tokens(R.pool_values(c.codes[0], c.scales[0], c.layout), c.indices, c.layout)[0][:c.lengths[0]]


def reorder(c, order):
    """The tokens of the only request and head, in another order."""
    n = len(order)
    page, slot = c.indices[np.arange(n) // c.ps], np.arange(n) % c.ps
    for codes, scales, dc, ds in zip(c.codes, c.scales, c.d_codes, c.d_scales):
        codes[page, slot] = codes[page[order], slot[order]]
        scales[page, :, slot] = scales[page[order], :, slot[order]]
        dc.copy_(torch.as_tensor(codes))
        ds.copy_(torch.as_tensor(scales))


def test_extreme_scales_of_v():
    c = Cache([90], 4, 1, 16, "NHD", seed=10)
    live = ~np.isnan(c.scales[1])
    rng = np.random.default_rng(0)
    c.scales[1][live] = (rng.choice([6e-8, 1e-4, 1.0, 10912.0], size=live.sum())).astype(np.float16)
    c.d_scales[1].copy_(torch.as_tensor(c.scales[1]))
    out, lse, _ = c.run(c.plan())
    ref = c.reference()
    # code x scale below f16's normal range is off by up to half its last place, 2^-25, a token
    o = f64(out)
    d = 2.0 ** -16 * ref[3] + 2.0 ** -20
    bound = (2 * d + 2.0 ** -10 + 2.0 ** -14)[..., None] * ref[2] + 2.0 ** -8 * np.abs(ref[0])
    bound = bound + 2.0 ** -35 * ref[4] + 2.0 ** -25
    assert (np.abs(o - ref[0]) <= bound).all()


def test_no_lse_and_poisoned_guard_rows():
    c = Cache([40, 7], 4, 2, 16, "NHD", seed=11)
    plan = c.plan()
    big = torch.full((c.batch + 2, c.Hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    out, _, _ = c.run(plan, want_lse=False, out=big[1:-1])
    assert_decode(out, None, c.reference())
    assert (big[0] == 7).all() and (big[-1] == 7).all()


def test_same_plan_is_bitwise_repeatable_bound_and_not():
    c = Cache([2000, 33, 700, 1], 8, 4, 16, "NHD", seed=12)
    plan = c.plan()
    first, l0, ws = c.run(plan)
    oxd.oxd_plan_bind_workspace(plan, ws)
    for _ in range(20):
        out, lse, _ = c.run(plan, ws=ws)
        assert torch.equal(out, first) and torch.equal(lse, l0)
    assert oxd.oxd_read_device_status(ws) == 0


def test_long_work_list_is_uploaded():
    # more requests than the parameter buffer holds units for
    c = Cache([3] * 2500, 1, 1, 8, "NHD", seed=13)
    plan, _, _ = check(c, max_splits=1)
    assert plan.info.upload_bytes > 0


def test_captured_graphs_with_their_own_workspaces_on_two_streams():
    a, b = Cache([900, 17], 4, 2, 16, "NHD", seed=14), Cache([333, 64, 5], 16, 1, 8, "HND", seed=15)
    graphs = []
    for c in (a, b):
        plan = c.plan()
        out, lse, ws = c.run(plan)
        oxd.oxd_plan_bind_workspace(plan, ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(plan, ws=ws, out=out, lse=lse)
        out.zero_(), lse.zero_()
        graphs.append((c, g, out, lse, plan, ws))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for s, (_, g, *_) in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for c, _, out, lse, _, _ in graphs:
        assert_decode(out, lse, c.reference())


def test_bad_page_is_reported_and_others_are_right():
    c = Cache([40, 40, 40], 4, 2, 16, "NHD", seed=16)
    good = c.reference()
    for bad in (-1, c.num_pages, 2 ** 31 - 1):
        c.d_indices.copy_(torch.as_tensor(c.indices))
        c.d_indices[int(c.indptr[1]) + 1] = bad
        out, lse, ws = c.run(c.plan())
        assert oxd.oxd_read_device_status(ws) == 1
        keep = [0, 2]
        assert_decode(out[keep], lse[keep], tuple(x[keep] for x in good))


def test_device_tables_that_differ_are_reported():
    c = Cache([40, 40], 4, 2, 16, "NHD", seed=17)
    plan = c.plan()
    c.d_last[1] = 3
    _, _, ws = c.run(plan)
    assert oxd.oxd_read_device_status(ws) == 2


def test_stale_binding_computes_nothing():
    c = Cache([40, 700], 4, 2, 16, "NHD", seed=18)
    plan = c.plan()
    ws = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    oxd.oxd_plan_bind_workspace(plan, ws)
    ws.zero_()
    out = torch.full((c.batch, c.Hq, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    c.run(plan, ws=ws, out=out)
    assert oxd.oxd_read_device_status(ws) == 2
    assert (out == 3).all()


def test_dependent_launch_behind_another_kernel():
    c = Cache([900, 17, 64], 4, 2, 16, "NHD", seed=19)
    plan = c.plan(pdl=1)
    ref = c.reference()
    q = c.d_q.clone()
    for _ in range(10):
        c.d_q.zero_()
        c.d_q.copy_(q)
        out, lse, _ = c.run(plan)
        assert_decode(out, lse, ref)


def test_the_plans_of_two_caches_are_not_mixed_up():
    c = Cache([40], 4, 2, 16, "NHD", seed=20)
    k = torch.zeros(c.num_pages, 16, 2, 128, dtype=torch.bfloat16, device="cuda")
    plan = c.plan()
    out, lse, ws = c.run(plan)
    with pytest.raises(oxd.OxdError) as e:
        oxd.oxd_paged_decode_run(plan, c.d_q, k, k, c.d_indptr, c.d_indices, c.d_last, 1.0, out,
                                 lse, ws)
    assert e.value.status == 6
    desc = oxd.make_desc(1, 8, 2, 16, "NHD", c.num_pages)
    bf = oxd.oxd_paged_decode_plan(desc, c.indptr, c.last)
    with pytest.raises(oxd.OxdError) as e:
        c.run(bf, ws=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 6


def test_offsets_past_32_bits():
    # a pool whose codes pass 2^32 bytes; the request's pages lie at its end
    ps, Hkv, pages = 64, 8, 140_000
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    c = Cache([200], 4, Hkv, ps, "NHD", seed=21)
    codes = [torch.zeros(pages, ps, Hkv, 64, dtype=torch.uint8, device="cuda") for _ in "kv"]
    scales = [torch.zeros(pages, Hkv, ps, 4, dtype=torch.float16, device="cuda") for _ in "kv"]
    far = torch.arange(pages - c.num_pages, pages, device="cuda")
    for x, y in zip(codes + scales, c.d_codes + c.d_scales):
        x[far] = y
    desc = oxd.make_desc(1, c.Hq, Hkv, ps, "NHD", pages)
    plan = oxd.oxd_quant_decode_plan(desc, c.indptr, c.last)
    c.pools = oxd.KvPools(*codes, *scales)
    c.d_indices = c.d_indices + (pages - c.num_pages)
    out, lse, ws = c.run(plan)
    assert oxd.oxd_read_device_status(ws) == 0
    assert_decode(out, lse, c.reference())


@pytest.mark.parametrize("G", [4, 16, 32])
def test_a_wait_that_runs_out_is_reported_and_the_next_run_is_right(G):
    """A wait limit of a nanosecond on a batch that HBM needs tens of microseconds for. Each warp has
    several chunks in flight, so a run may still find every wait satisfied in time: it either says
    that a wait ran out or is right."""
    n, L, ps, Hkv = 256, 2048, 16, 2
    pages = n * L // ps
    g = torch.Generator(device="cuda").manual_seed(1)
    codes = [torch.randint(0, 256, (pages, ps, Hkv, 64), dtype=torch.uint8, device="cuda", generator=g)
             for _ in "kv"]
    scales = [torch.rand(pages, Hkv, ps, 4, device="cuda", generator=g).half() for _ in "kv"]
    q = torch.randn(n, G * Hkv, 128, device="cuda", generator=g).bfloat16()
    indptr = np.arange(0, pages + 1, L // ps, dtype=np.int32)
    last = np.full(n, ps, np.int32)
    d = [torch.as_tensor(a, device="cuda") for a in (indptr, np.arange(pages, dtype=np.int32), last)]
    guard = torch.full((n + 2, G * Hkv, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(n, G * Hkv, device="cuda")

    def run(**kw):
        desc = oxd.make_desc(n, G * Hkv, Hkv, ps, "NHD", pages, **kw)
        plan = oxd.oxd_quant_decode_plan(desc, indptr, last)
        ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
        oxd.oxd_quant_decode_run(plan, q, oxd.KvPools(*codes, *scales), *d, 0.1, guard[1:-1], lse, ws)
        return oxd.oxd_read_device_status(ws)

    assert run() == 0
    out, l0 = guard.clone(), lse.clone()
    for _ in range(5):
        guard[1:-1] = 0
        status = run(wait_timeout_ns=1)
        assert status == 3 or (status == 0 and torch.equal(guard, out) and torch.equal(lse, l0))
    assert (guard[0] == 7).all() and (guard[-1] == 7).all()
    assert run() == 0
    assert torch.equal(guard, out) and torch.equal(lse, l0)


@pytest.mark.parametrize("G,Hkv,layout", [(1, 8, "NHD"), (4, 2, "HND"), (8, 3, "NHD")])
def test_any_workspace_contents_and_two_plans_on_one(G, Hkv, layout):
    """Split streams, whatever the workspace held before, replayed from an unbound capture, and with
    another plan's run on the same workspace in between."""
    c = Cache([512, 900, 64, 130], G, Hkv, 16, layout, seed=23)
    plan, other = c.plan(force_splits=4), c.plan(force_splits=3)
    ref = c.reference()
    g = torch.Generator(device="cuda").manual_seed(2)
    n = max(plan.workspace_bytes, other.workspace_bytes)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    for fill in (torch.zeros(n, dtype=torch.uint8, device="cuda"),
                 torch.randint(0, 256, (n,), dtype=torch.uint8, device="cuda", generator=g)):
        ws.copy_(fill)
        out, lse, _ = c.run(plan, ws=ws)
        assert oxd.oxd_read_device_status(ws) == 0
        assert_decode(out, lse, ref)
        first, l0 = out.clone(), lse.clone()
        c.run(other, ws=ws)
        c.run(plan, ws=ws, out=out, lse=lse)
        assert torch.equal(out, first) and torch.equal(lse, l0)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        c.run(plan, ws=ws, out=out, lse=lse)
    for _ in range(5):
        out.zero_(), lse.zero_()
        graph.replay()
        assert torch.equal(out, first) and torch.equal(lse, l0)


@pytest.mark.parametrize("G,Hkv", [(1, 8), (2, 4), (5, 3), (8, 1)])
@pytest.mark.parametrize("lengths", [[512], [129], [4000], [300, 1000, 77, 130], [2048] * 3, [200] * 8])
def test_small_batches_in_one_launch(G, Hkv, lengths):
    """Streams cut into pieces that a cluster's first CTA merges, or run whole."""
    for layout in ("NHD", "HND"):
        c = Cache(lengths, G, Hkv, 16, layout, seed=25)
        plan, out, lse = check(c)
        assert plan.info.launches_per_run == 1 or max(lengths) > 2048
        ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
        oxd.oxd_plan_bind_workspace(plan, ws)
        for _ in range(5):
            o2, l2, _ = c.run(plan, ws=ws)
            assert torch.equal(out, o2) and torch.equal(lse, l2)
        ws.zero_()  # the binding is gone: nothing is computed, and that is said
        keep = torch.full_like(out, 3.0)
        c.run(plan, ws=ws, out=keep)
        assert oxd.oxd_read_device_status(ws) == 2 and (keep == 3).all()


@pytest.mark.parametrize("G,Hkv,layout,n,L", [(16, 8, "HND", 2600, 3), (32, 4, "NHD", 2600, 9),
                                              (32, 8, "NHD", 2600, 9), (4, 8, "NHD", 5000, 8),
                                              (8, 8, "HND", 2600, 2)])
def test_tens_of_units_a_cta(G, Hkv, layout, n, L):
    """From the call's own list, bound and replayed. (A CTA holds 32 units decoded: all cases but that
    of 10408 units pass it.)"""
    c = Cache([L] * n + [300, 1], G, Hkv, 8, layout, seed=26)
    plan, out, lse = check(c)
    assert plan.info.num_work_items > (32 if n * Hkv > 10400 else 20) * plan.info.grid_ctas
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    oxd.oxd_plan_bind_workspace(plan, ws)
    o2, l2, _ = c.run(plan, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(plan, ws=ws, out=o2, lse=l2)
    o2.zero_(), l2.zero_()
    graph.replay()
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    assert oxd.oxd_read_device_status(ws) == 0


@pytest.mark.parametrize("G,Hkv", [(1, 200), (8, 65), (32, 40)])
@pytest.mark.parametrize("layout", ["NHD", "HND"])
def test_many_heads(G, Hkv, layout):
    check(Cache([70, 9], G, Hkv, 16, layout, seed=27))


@pytest.mark.parametrize("G", [4, 16, 32])
def test_two_runs_of_one_plan_at_once(G):
    """One plan, two workspaces, two streams, neither waiting for the other."""
    c = Cache([3000, 33, 700, 1], G, 2, 16, "NHD", seed=28)
    plan, out, lse = check(c)
    streams = [torch.cuda.Stream() for _ in range(2)]
    runs = []
    torch.cuda.synchronize()
    for _ in range(10):
        for s in streams:
            with torch.cuda.stream(s):
                runs.append(c.run(plan))
    torch.cuda.synchronize()
    for o, l, ws in runs:
        assert oxd.oxd_read_device_status(ws) == 0
        assert torch.equal(o, out) and torch.equal(l, lse)


@pytest.mark.parametrize("n,Hkv", [(5, 8), (6, 8), (7, 8), (8, 8), (37, 1)])
def test_clusters_of_every_size_that_fits(n, Hkv):
    """37 to 64 streams: as many CTAs a stream as are resident at once, odd numbers among them."""
    c = Cache([1024, 129, 1000, 512, 700, 1023, 333, 64][:n] + [1024] * (n - 8), 4, Hkv, 16, "HND", seed=29)
    plan, out, lse = check(c)
    size = plan.info.cluster_size
    assert 4 <= size < 8 and plan.info.grid_ctas == size * n * Hkv
    for _ in range(5):
        o2, l2, _ = c.run(plan)
        assert torch.equal(out, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("G", [1, 4, 8, 16, 32])
def test_a_wait_that_runs_out_does_so(G):
    """Every CTA's first wait is for query rows that come from memory (L2 holds something else), with
    a limit of a nanosecond: at least one of the runs says that a wait ran out. The rows are waited
    for all the same, so each run's outputs are those of a plan without the limit."""
    n, ps = 600, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    codes = [torch.randint(0, 256, (n, 1, ps, 64), dtype=torch.uint8, device="cuda", generator=g)
             for _ in "kv"]
    scales = [torch.rand(n, 1, ps, 4, device="cuda", generator=g).half() for _ in "kv"]
    q = torch.randn(n, G, 128, device="cuda", generator=g).bfloat16()
    indptr, last = np.arange(n + 1, dtype=np.int32), np.full(n, ps, np.int32)
    d = [torch.as_tensor(a, device="cuda") for a in (indptr, indptr[:-1].copy(), last)]
    out, lse = torch.empty_like(q), torch.empty(n, G, device="cuda")
    other = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")

    def run(**kw):
        plan = oxd.oxd_quant_decode_plan(oxd.make_desc(n, G, 1, ps, "HND", n, **kw), indptr, last)
        ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
        oxd.oxd_plan_bind_workspace(plan, ws)
        out.zero_(), lse.zero_(), other.fill_(1)
        oxd.oxd_quant_decode_run(plan, q, oxd.KvPools(*codes, *scales), *d, 0.1, out, lse, ws)
        return oxd.oxd_read_device_status(ws)

    assert run() == 0
    o0, l0 = out.clone(), lse.clone()
    seen = []
    for _ in range(10):
        seen.append(run(wait_timeout_ns=1))
        assert torch.equal(out, o0) and torch.equal(lse, l0)
    assert set(seen) <= {0, 3} and 3 in seen, seen
    assert run() == 0
