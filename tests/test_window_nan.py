"""NaN in what a query of a windowed prefill sees: its row is NaN, out and lse, whether or not its tile is cut
into pieces; the rows that do not see it are as they would be (GPU)."""
import numpy as np
import pytest
import torch

import paged_kv_decode_attn_gb300 as oxd
import window_ref as Wr
from quant_helpers import f64
from test_window_prefill import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    oxd.build()


def plant(c, request, token, head):
    """NaN in one column of one K row."""
    p = c.p
    page = int(p.indices[p.indptr[request] + token // p.ps])
    at = (page, token % p.ps, head) if p.layout == "NHD" else (page, head, token % p.ps)
    c.d_k[at][5] = float("nan")


def hit_rows(c, request, token, head):
    """[rows, Hq]: the (query, head) pairs that see the row."""
    p, hit = c.p, np.zeros((len(c.q), c.Hq), bool)
    G = c.Hq // p.Hkv
    length, ql = p.lengths[request], p.q_lens[request]
    for i in range(ql):
        if token in Wr.seen(length - ql + i, length, c.window, c.sinks):
            hit[c.qo[request] + i, head * G:(head + 1) * G] = True
    return hit


def check(c, hit, **kw):
    out, lse = (f64(x) for x in c.run(c.plan(**kw)))
    assert c.code == 0
    assert np.isnan(out[hit]).all(), "out of rows that see NaN"
    assert np.isnan(lse[hit]).all(), "lse of rows that see NaN"
    Wr.assert_close(out[~hit], lse[~hit], [x[~hit] for x in c.reference()], str(kw))


@pytest.mark.parametrize("rows", [128, 256])
@pytest.mark.parametrize("splits", [1, 3, 0])
@pytest.mark.parametrize("token", [0, 5, 700, 1290, 1499])
def test_a_key_that_some_queries_see(rows, splits, token):
    """Among the sinks, in the window of some queries, of all, and the last query's own."""
    c = Case([200, 1500], [30, 200], 4, 2, 16, "NHD", 600, 6, seed=token)
    plant(c, 1, token, 1)
    hit = hit_rows(c, 1, token, 1)
    check(c, hit, tile_rows=rows, max_splits=splits)


@pytest.mark.parametrize("rows", [128, 256])
@pytest.mark.parametrize("token", [2, 500, 511, 1700, 2990, 2999])
def test_a_key_in_one_piece_of_a_tile(rows, token):
    c = Case([70, 3000], [70, 20], 4, 2, 16, "HND", 2500, 3, seed=token)
    assert c.plan(tile_rows=rows).info.max_pieces > 1
    plant(c, 1, token, 0)
    check(c, hit_rows(c, 1, token, 0), tile_rows=rows)


@pytest.mark.parametrize("rows", [128, 256])
@pytest.mark.parametrize("splits", [1, 2, 5, 0])
@pytest.mark.parametrize("G", [1, 4, 5])
def test_a_query_row(rows, splits, G):
    """All of its scores are NaN, in every piece."""
    c = Case([2000, 70], [20, 70], G, 2, 16, "HND", 1500, 3, seed=G)
    hit = np.zeros((len(c.q), c.Hq), bool)
    for row, head in ((0, 0), (19, 2 * G - 1), (40, G)):
        c.d_q[row, head, 77] = float("nan")
        hit[row, head] = True
    check(c, hit, tile_rows=rows, max_splits=splits)


@pytest.mark.parametrize("rows", [128, 256])
@pytest.mark.parametrize("splits", [0, 3])
def test_a_window_over_everything(rows, splits):
    c = Case([500, 900], [300, 9], 4, 2, 16, "NHD", 900, 0, seed=3)
    plant(c, 1, 10, 0)
    hit = hit_rows(c, 1, 10, 0)
    c.d_q[250, 3, 0] = float("nan")
    hit[250, 3] = True
    check(c, hit, tile_rows=rows, max_splits=splits)


def test_more_than_sixteen_pieces():
    """Rows merged by two warps."""
    c = Case([20000], [4], 4, 1, 64, "NHD", 19000, 3, seed=1)
    plan = c.plan(tile_rows=128)
    assert plan.info.max_pieces > 16
    for token in (2, 19996, 10000):
        c = Case([20000], [4], 4, 1, 64, "NHD", 19000, 3, seed=1)
        plant(c, 0, token, 0)
        check(c, hit_rows(c, 0, token, 0), tile_rows=128)


@pytest.mark.parametrize("splits", [0, 1, 5])
def test_the_window_decode_says_the_same(splits):
    import test_window_decode as D

    c = D.Case([900, 40], 4, 2, 16, "NHD", 500, 20, seed=2)
    p = c.p
    c.d_k[int(p.indices[p.indptr[0] + 880 // 16]), 880 % 16, 1, 5] = float("nan")
    c.d_q[1, 0, 3] = float("nan")
    out, lse = (f64(x) for x in c.run(max_splits=splits))
    hit = np.zeros((2, 8), bool)
    hit[0, 4:] = hit[1, 0] = True
    assert c.code == 0 and np.isnan(out[hit]).all() and np.isnan(lse[hit]).all()
    Wr.assert_close(out[~hit], lse[~hit], [x[~hit] for x in c.reference()])
