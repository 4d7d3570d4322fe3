"""Free lists with entries that are no pages, padded ones among them: recorded, and never a page that the row
listed before (GPU)."""
import numpy as np
import pytest
import torch

import paged_kv_decode_attn_gb300 as oxd
from test_build_tables import check, compare, reference, run, state

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    oxd.build()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 4), (1, 0)])
@pytest.mark.parametrize("bad", [-1, -7, -2 ** 31, 12, 2 ** 31 - 1])
def test_an_entry_outside_the_pool_is_listed_as_it_is(bad, window, sinks, in_place):
    """Requests that take the first, a middle and the last page of a list with one bad entry."""
    for at in range(5):
        s = state([30, 5, 40], [30, 5, 8], 16, seed=at, pool=12)
        assert len(s["free"]) >= 5
        s["free"] = s["free"].copy()
        s["free"][at] = bad
        takes = 2 + 1 + 1  # pages of this step
        check(s, 16, window, sinks, code=oxd.OXD_DEVICE_BAD_PAGE if at < takes else 0, in_place=in_place)


def test_a_padded_list_that_runs_into_its_padding():
    """A list of fixed size whose end is -1: the pages are recorded as no pages, request by request."""
    s = state([100, 50, 40, 16], [100, 50, 40, 16], 16, seed=7)
    s["free"] = s["free"].copy()
    s["free"][6:] = -1
    check(s, 16, code=oxd.OXD_DEVICE_BAD_PAGE)
    check(s, 16, 32, 4, code=oxd.OXD_DEVICE_BAD_PAGE, in_place=True)


@pytest.mark.parametrize("window,sinks", [(0, 0), (30, 2)])
@pytest.mark.parametrize("bad", [-1, -2 ** 31])
def test_the_next_steps_do_not_list_what_the_row_held_before(bad, window, sinks):
    """The rows behind the held pages are full of other requests' pages: a step that takes a bad entry and
    those after it, in place, list the entry and not the old page."""
    ps, steps = 8, 12
    s = state([7, 3], [1, 1], ps, seed=3, width=6, held=[1, 1], extra_free=20)
    s["rows"][0, 1:], s["rows"][1, 1:] = s["rows"][1, 0], s["rows"][0, 0]
    s["free"] = s["free"].copy()
    s["free"][0] = bad
    want, at = [], {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in s.items()}
    for _ in range(steps):
        r = reference(at, ps, window, sinks, 14, 3)
        want.append(r)
        at.update(lengths=at["lengths"] + 1, held=r["held_out"], rows=r["rows"].astype(np.int32),
                  taken=int(r["taken_out"][0]), refcount=r["refcount"])
    assert any((r["rows"][0, 1] == bad) and r["held_out"][0] > 1 for r in want)

    def call(go, lengths, o):
        for i in range(steps):
            o["indices"].fill_(-9)
            go()
            got = {n: t.cpu().numpy().astype(np.int64).reshape(-1)[:want[i][n].size] for n, t in o.items()}
            compare(got, want[i])
            lengths += 1

    run(s, ps, window, sinks, n_idx=14, n_tok=3, in_place=True, call=call)
