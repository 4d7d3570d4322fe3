"""Block tables and token maps built on the GPU against plain Python (GPU)."""
import os

import numpy as np
import pytest
import torch

import paged_kv_decode_attn_gb300 as oxd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    oxd.build()


def reference(s, ps, window, sinks, n_idx, n_tok):
    """What the definition gives, request by request; the outputs that are cut off or behind the
    last entry as they were (-9) or -1."""
    got = {n: np.full(k, -9, np.int64) for n, k in (("indices", n_idx), ("token_request", n_tok),
                                                    ("positions", n_tok), ("slots", n_tok))}
    rows, refcount = s["rows"].astype(np.int64), s["refcount"].copy()
    indptr, qo, last, held, taken = [0], [0], [], [], int(s["taken"])
    listed, token = [], []
    for b, (n, new) in enumerate(zip(s["lengths"], s["new"])):
        need = -(-n // ps)
        have = s["held"][b]
        for j in range(have, need):
            if taken < len(s["free"]):
                rows[b, j] = s["free"][taken]
                if 0 <= rows[b, j] < len(refcount):
                    refcount[rows[b, j]] = 1
                have += 1
            taken += 1
        pages = [rows[b, j] if j < have else -1 for j in range(need)]
        for t in range(n - new, n):
            page = pages[t // ps]
            token.append((b, t, -1 if page < 0 else page * ps + t % ps))
        if window:
            first = n - max(new, 1) - window + 1
            pages = [-1 if j * ps >= sinks and (j + 1) * ps <= first else p for j, p in enumerate(pages)]
        listed += pages
        indptr.append(min(len(listed), n_idx))
        qo.append(min(len(token), n_tok))
        last.append(n - (need - 1) * ps if need else 0)
        held.append(have)
    listed, token = listed[:n_idx], token[:n_tok]
    got["indices"][:len(listed)] = listed
    for i, n in enumerate(("token_request", "positions", "slots")):
        got[n][:] = -1
        got[n][:len(token)] = [t[i] for t in token]
    got.update(indptr=indptr, qo_indptr=qo, last_page_len=last, rows=rows, held_out=held,
               taken_out=[min(taken, len(s["free"]))], refcount=refcount)
    return {n: np.asarray(x, np.int64) for n, x in got.items()}


def state(lengths, new, ps, seed, width=None, held=None, extra_free=5, taken=0, pool=None):
    rng = np.random.default_rng(seed)
    lengths, new = np.asarray(lengths), np.asarray(new)
    held = -(-(lengths - new) // ps) if held is None else np.asarray(held)
    need = -(-lengths // ps)
    width = width or int(max(need.max(), held.max(), 1)) + 1
    lack = int(np.maximum(need - held, 0).sum())
    n_free = max(taken + lack + extra_free, 0)
    pool = pool or int(held.sum()) + n_free + 3
    order = rng.permutation(max(pool, int(held.sum()) + n_free)).astype(np.int32)
    rows = np.full((len(lengths), width), -5, np.int32)
    at = 0
    for b, h in enumerate(held):
        rows[b, :h] = order[at:at + h]
        at += h
    return dict(lengths=lengths, new=new, held=held, rows=rows, free=order[at:at + n_free], taken=taken,
                refcount=np.zeros(pool, np.int64))


def dev(a, dtype=np.int32):
    return torch.as_tensor(np.asarray(a, dtype), device="cuda")


def run(s, ps, window=0, sinks=0, n_idx=None, n_tok=None, in_place=False, maps=True, slots=True,
        refcount=True, call=None):
    B = len(s["lengths"])
    n_idx = n_idx or max(int((-(-s["lengths"] // ps)).sum()), 1) + 7
    n_tok = (int(s["new"].sum()) + 6 if n_tok is None else n_tok) if maps else 0
    full = lambda n, t=torch.int32: torch.full((max(n, 1) + 4,), -9, dtype=t, device="cuda")  # noqa: E731
    o = dict(rows=dev(s["rows"]), refcount=dev(s["refcount"]), indptr=full(B + 1),
             indices=full(n_idx), last_page_len=full(B), qo_indptr=full(B + 1),
             token_request=full(n_tok), positions=full(n_tok), slots=full(n_tok, torch.int64))
    held, taken = dev(s["held"]), dev([s["taken"]])
    o["held_out"], o["taken_out"] = (held, taken) if in_place else (full(B), full(1))
    free = dev(s["free"]) if len(s["free"]) else None
    d = oxd.make_build_tables_desc(B, ps, s["rows"].shape[1], len(s["refcount"]), n_idx, n_tok,
                                   len(s["free"]), window, sinks)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    lengths, new = dev(s["lengths"]), dev(s["new"]) if maps else None

    def go():
        oxd.oxd_build_tables(
            d, lengths, new, o["rows"], held, o["held_out"], free,
            taken if free is not None else None, o["taken_out"] if free is not None else None,
            o["refcount"] if refcount else None, o["indptr"], o["indices"], o["last_page_len"],
            *((o[n] if maps else None) for n in ("qo_indptr", "token_request", "positions")),
            o["slots"] if slots and maps else None, ws)

    (call or (lambda f, *_: f()))(go, lengths, o)
    code = oxd.oxd_read_device_status(ws)
    sizes = dict(indptr=B + 1, indices=n_idx, last_page_len=B, qo_indptr=B + 1, token_request=n_tok,
                 positions=n_tok, slots=n_tok, held_out=B, taken_out=1)
    got = {}
    for n, t in o.items():
        x = t.cpu().numpy()
        if n in sizes and not (in_place and n in ("held_out", "taken_out")):
            assert (x[sizes[n]:] == -9).all(), n  # nothing behind the array
            x = x[:sizes[n]]
        got[n] = x.astype(np.int64)
    return got, code, n_idx, n_tok


def compare(got, ref, skip=()):
    for n, want in ref.items():
        if n not in skip:
            assert np.array_equal(got[n].reshape(want.shape), want), n


def check(s, ps, window=0, sinks=0, code=0, skip=(), **kw):
    got, was, n_idx, n_tok = run(s, ps, window, sinks, **kw)
    assert was == code
    skip = set(skip)
    if not len(s["free"]):
        skip.add("taken_out")
    if not n_tok:
        skip |= {"qo_indptr", "token_request", "positions", "slots"}
    compare(got, reference(s, ps, window, sinks, n_idx, n_tok), skip)


@pytest.mark.parametrize("ps", [8, 16, 32, 64])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (20, 4), (64, 65), (1000, 0)])
def test_mixed_requests(ps, window, sinks):
    lengths = [0, 1, 8, 9, 64, 65, 200, 1000, 0, 513, 100]
    new = [0, 1, 8, 1, 0, 1, 200, 37, 0, 1, 99]
    check(state(lengths, new, ps, seed=ps), ps, window, sinks)
    check(state(lengths, new, ps, seed=ps), ps, window, sinks, in_place=True)


@pytest.mark.parametrize("B", [1, 2, 31, 32, 33, 100, 512, 1023, 1024, 1025, 2500])
def test_batches(B):
    rng = np.random.default_rng(B)
    lengths = rng.integers(0, 400, B)
    new = np.minimum(lengths, rng.integers(0, 20, B))
    check(state(lengths, new, 16, seed=B), 16, 50, 3)


@pytest.mark.parametrize("lengths,new", [([100000], [100000]), ([70000, 3], [1, 3]),
                                         ([16384] * 40, [1] * 40), ([9000] * 3, [9000] * 3)])
def test_long_requests(lengths, new):
    """Several CTAs, several warps a request."""
    check(state(lengths, new, 8, seed=1), 8, 4096, 4)


def test_pages_that_a_request_holds_beyond_its_need_stay_its():
    """Dropped tokens (rejected drafts) keep their pages, which serve when it grows again."""
    check(state([5, 40, 0], [0, 1, 0], 16, seed=2, held=[3, 3, 2]), 16)


def test_without_a_free_list_without_maps_without_slots_and_refcounts():
    s = state([30, 7, 64], [1, 1, 0], 16, seed=3, held=[2, 1, 4], extra_free=0)
    assert len(s["free"]) == 0
    check(s, 16)
    s = state([30, 7, 64], [0, 0, 0], 16, seed=4, held=[0, 0, 2])
    check(s, 16, 20, 1, maps=False)
    s = state([30, 7, 64], [3, 1, 9], 16, seed=5)
    check(s, 16, slots=False, refcount=False, skip=("slots", "refcount"))


def test_the_free_list_goes_on_from_what_is_taken():
    check(state([33, 64, 1], [1, 64, 1], 16, seed=6, taken=4), 16)


def test_too_few_free_pages():
    s = state([100, 50, 40, 16], [100, 50, 40, 16], 16, seed=7, extra_free=-5)
    check(s, 16, code=oxd.OXD_DEVICE_NO_PAGES)
    s = state([100, 50], [100, 50], 16, seed=7, extra_free=-5, taken=3)
    check(s, 16, 32, 4, code=oxd.OXD_DEVICE_NO_PAGES, in_place=True)
    s = state([20, 50], [20, 50], 16, seed=7, held=[0, 0], extra_free=-6)
    assert len(s["free"]) == 0  # no free list at all
    check(s, 16, code=oxd.OXD_DEVICE_NO_PAGES)


def test_tables_that_do_not_fit_are_cut_off():
    s = state([100, 50, 40], [10, 50, 1], 16, seed=8)
    for n_idx, n_tok in ((9, 61), (7, 70), (1, 100), (14, 30), (14, 1)):
        check(s, 16, n_idx=n_idx, n_tok=n_tok, code=oxd.OXD_DEVICE_BAD_POSITION)


@pytest.mark.parametrize("name,value", [("lengths", -1), ("lengths", 16 * 40 + 1), ("lengths", 2 ** 31 - 1),
                                        ("new", -1), ("new", 51), ("held", -1), ("held", 41)])
def test_a_request_out_of_bounds_is_listed_as_empty(name, value):
    s = state([100, 50, 40], [10, 5, 1], 16, seed=9, width=40)
    got_held = value if name == "held" else s["held"][1]
    empty = {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in s.items()}
    s[name] = s[name].copy()
    s[name][1] = value
    got, code, n_idx, n_tok = run(s, 16, n_idx=40, n_tok=20)
    assert code == oxd.OXD_DEVICE_BAD_POSITION
    empty["lengths"][1] = empty["new"][1] = 0
    ref = reference(empty, 16, 0, 0, 40, 20)
    ref["held_out"][1] = got_held
    compare(got, ref)


@pytest.mark.parametrize("taken", [-1, 10 ** 6, 2 ** 31 - 1])
def test_a_count_of_taken_pages_out_of_bounds_takes_none(taken):
    s = state([30, 30], [30, 1], 16, seed=10)
    s["taken"] = taken
    got, code, n_idx, n_tok = run(s, 16)
    assert code in (oxd.OXD_DEVICE_BAD_POSITION, oxd.OXD_DEVICE_NO_PAGES)
    assert got["taken_out"][0] == taken and got["held_out"].tolist() == [0, 2]
    assert got["indices"][:4].tolist() == [-1, -1, *s["rows"][1, :2]]
    assert (got["refcount"] == 0).all()


def test_free_pages_outside_the_pool_are_recorded():
    s = state([30, 30], [30, 30], 16, seed=11, pool=3, extra_free=0)
    s["free"] = np.asarray([0, 7, 2, 1], np.int32)
    check(s, 16, code=oxd.OXD_DEVICE_BAD_PAGE)


def test_a_captured_loop_grows_the_requests_on_the_device():
    """Lengths advanced on the device, state in place: each replay is one step."""
    ps, B, steps = 8, 3, 40
    s = state([5, 16, 1], [1, 1, 1], ps, seed=12, width=10, held=[1, 2, 0], extra_free=30)
    steps_ref = []
    ref_s = {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in s.items()}
    for i in range(steps):
        r = reference(ref_s, ps, 12, 2, 60, B + 2)
        steps_ref.append(r)
        ref_s.update(lengths=ref_s["lengths"] + 1, held=r["held_out"], rows=r["rows"].astype(np.int32),
                     taken=int(r["taken_out"][0]), refcount=r["refcount"])

    def call(go, lengths, o):
        before = {n: t.clone() for n, t in [("lengths", lengths), *o.items()]}
        go()  # (first use outside the capture)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            go()
            lengths += 1
        for n, t in [("lengths", lengths), *o.items()]:
            t.copy_(before[n])
        for i in range(steps):
            g.replay()
            for n, want in steps_ref[i].items():
                if n != "indices":
                    x = o[n].cpu().numpy().astype(np.int64).reshape(-1)
                    assert np.array_equal(x[:want.size], want.reshape(-1)), (i, n)
                else:
                    k = steps_ref[i]["indptr"][-1]
                    assert np.array_equal(o[n].cpu().numpy()[:k], want[:k]), i

    run(s, ps, 12, 2, n_idx=60, n_tok=B + 2, in_place=True, call=call)


def test_runs_are_equal_on_two_streams():
    rng = np.random.default_rng(13)
    lengths = rng.integers(1, 3000, 200)
    s = state(lengths, np.ones(200, int), 16, seed=13)
    first, _, n_idx, n_tok = run(s, 16, 500, 4)
    for _ in range(5):
        with torch.cuda.stream(torch.cuda.Stream()):
            got, code, _, _ = run(s, 16, 500, 4)
        assert code == 0
        compare(got, first)


def test_slots_past_2_32():
    """Page numbers near 2^31: slots are 64-bit."""
    s = state([40, 9], [40, 1], 16, seed=14, held=[0, 1])
    s["free"] = (np.arange(len(s["free"])) + 2 ** 31 - 100).astype(np.int32)
    s["rows"][1, 0] = 2 ** 30 + 5
    got, code, n_idx, n_tok = run({**s, "refcount": np.zeros(1)}, 16, refcount=False)
    # (the pool of this call is declared as large as its reference counts: one page)
    assert code == oxd.OXD_DEVICE_BAD_PAGE
    ref = reference(s, 16, 0, 0, n_idx, n_tok)
    compare(got, ref, skip=("refcount",))
    assert got["slots"].max() > 2 ** 34


def test_twenty_six_calls_in_a_row_in_place():
    """Back to back, each a programmatic dependent of the one before."""
    ps, B = 8, 70
    s = state([3] * B, [1] * B, ps, seed=15, width=20, held=[1] * B, extra_free=B * 4)
    lengths = dev(s["lengths"])
    rows, held, taken = dev(s["rows"]), dev(s["held"]), dev([0])
    free, ref_count = dev(s["free"]), dev(s["refcount"])
    new = dev(s["new"])
    n_idx = B * 20
    d = oxd.make_build_tables_desc(B, ps, 20, len(s["refcount"]), n_idx, B, len(s["free"]))
    outs = [torch.full((n,), -9, dtype=torch.int32, device="cuda") for n in (B + 1, n_idx, B, B + 1, B, B)]
    slots = torch.full((B,), -9, dtype=torch.int64, device="cuda")
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    for _ in range(26):
        oxd.oxd_build_tables(d, lengths, new, rows, held, held, free, taken, taken, ref_count, *outs[:3],
                             *outs[3:], slots, ws)
        lengths += 1
    assert oxd.oxd_read_device_status(ws) == 0
    at = {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in s.items()}
    for _ in range(26):
        r = reference(at, ps, 0, 0, n_idx, B)
        at.update(lengths=at["lengths"] + 1, held=r["held_out"], rows=r["rows"].astype(np.int32),
                  taken=int(r["taken_out"][0]), refcount=r["refcount"])
    assert np.array_equal(rows.cpu().numpy(), r["rows"]) and taken.item() == r["taken_out"][0]
    assert np.array_equal(slots.cpu().numpy(), r["slots"])
    assert np.array_equal(outs[0].cpu().numpy(), r["indptr"])


@pytest.mark.parametrize("seed", range(30 * int(os.environ.get("OXD_FUZZ_SCALE", "1"))))
def test_random_tables(seed):
    rng = np.random.default_rng(3000 + seed)
    B = int(np.exp(rng.uniform(0, np.log(1500))))
    hi = int(np.exp(rng.uniform(0, np.log(3000))))
    lengths = rng.integers(0, hi + 1, B)
    new = np.minimum(lengths, rng.integers(0, int(np.exp(rng.uniform(0, np.log(hi + 1)))) + 1, B))
    ps = int(rng.choice([8, 16, 32, 64]))
    held = np.maximum(-(-(lengths - new) // ps) + rng.integers(-1, 3, B), 0)
    window = int(rng.choice([0, 1, 30, 500]))
    check(state(lengths, new, ps, seed, held=held, taken=int(rng.choice([0, 7]))), ps, window,
          int(rng.choice([0, 1, 20, 100])), in_place=bool(rng.integers(2)))
