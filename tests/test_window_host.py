"""Refusals of the window decodes and of the table builder, on the CPU with addresses that are
never dereferenced."""
import numpy as np
import pytest

import paged_kv_decode_attn_gb300 as oxd

BASE = 1 << 40
GAP = 1 << 36


@pytest.fixture(scope="module", autouse=True)
def built():
    oxd.build()


def at(i, off=0):
    return BASE + i * GAP + off


def status(call):
    try:
        call()
    except oxd.OxdError as e:
        return e.status
    return 0


def window_call(four, over, desc_over):
    d = dict(batch=3, num_qo_heads=8, num_kv_heads=2, page_size=16, layout="NHD", num_pages=50,
             num_indices=20, window=64, sinks=4)
    d.update({k: v for k, v in desc_over.items() if k != "reserved"})
    desc = oxd.make_window_decode_desc(**d)
    if "reserved" in desc_over:
        desc.reserved[1] = desc_over["reserved"]
    a = dict(q=at(0), k=at(1), v=at(2), ks=at(3), vs=at(4), indptr=at(5), indices=at(6), last=at(7),
             scale=0.1, out=at(8), lse=at(9), ws=at(10), ws_bytes=256)
    a.update(over)
    tail = (a["indptr"], a["indices"], a["last"], a["scale"], a["out"], a["lse"], a["ws"], a["ws_bytes"])
    if four:
        return status(lambda: oxd.oxd_quant_window_decode(
            desc, a["q"], oxd.KvPools(a["k"], a["v"], a["ks"], a["vs"]), *tail, stream=0))
    return status(lambda: oxd.oxd_window_decode(desc, a["q"], a["k"], a["v"], *tail, stream=0))


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("over,desc_over,want", [
    (dict(q=None), {}, 1), (dict(k=None), {}, 1), (dict(v=None), {}, 1), (dict(indptr=None), {}, 1),
    (dict(indices=None), {}, 1), (dict(last=None), {}, 1), (dict(out=None), {}, 1),
    (dict(ws=None), {}, 1), (dict(scale=float("nan")), {}, 1), (dict(scale=float("inf")), {}, 1),
    ({}, dict(batch=0), 1), ({}, dict(num_qo_heads=0), 1), ({}, dict(num_kv_heads=0), 1),
    ({}, dict(num_qo_heads=9), 1), ({}, dict(layout=2), 1), ({}, dict(num_pages=0), 1),
    ({}, dict(num_indices=0), 1), ({}, dict(window=0), 1), ({}, dict(window=-1), 1),
    ({}, dict(sinks=-1), 1), ({}, dict(max_splits=-1), 1), ({}, dict(reserved=1), 1),
    ({}, dict(head_dim=64), 2), ({}, dict(page_size=12), 2), ({}, dict(num_qo_heads=66), 2),
    ({}, dict(window=1 << 30, sinks=1), 2), ({}, dict(num_pages=1 << 31), 2),
    ({}, dict(num_pages=(1 << 27) + 1), 2), ({}, dict(batch=1 << 25), 2),
    (dict(q=at(0, 8)), {}, 3), (dict(k=at(1, 8)), {}, 3), (dict(out=at(8, 8)), {}, 3),
    (dict(indptr=at(5, 2)), {}, 3), (dict(lse=at(9, 2)), {}, 3), (dict(ws=at(10, 128)), {}, 3),
    (dict(out=at(0)), {}, 4), (dict(out=at(1, 4096)), {}, 4), (dict(lse=at(8, 16)), {}, 4),
    (dict(lse=at(5)), {}, 4), (dict(ws=at(2)), {}, 4), (dict(ws=at(6)), {}, 4),
    (dict(ws_bytes=255), {}, 5),
])
def test_window_decode_refusals(four, over, desc_over, want):
    assert window_call(four, over, desc_over) == want


@pytest.mark.parametrize("over,want", [(dict(ks=None), 1), (dict(vs=None), 1), (dict(ks=at(3, 8)), 3),
                                       (dict(out=at(4)), 4)])
def test_4bit_window_decode_refusals(over, want):
    assert window_call(True, over, {}) == want


def test_quant_window_decode_refuses_no_cache():
    d = oxd.make_window_decode_desc(3, 8, 2, 16, "NHD", 50, 20, 64)
    assert oxd.lib().oxd_quant_window_decode(d, at(0), None, at(5), at(6), at(7), 0.1, at(8), None,
                                             at(10), 256, None) == 1
    assert oxd.lib().oxd_window_decode(None, at(0), at(1), at(2), at(5), at(6), at(7), 0.1, at(8),
                                       None, at(10), 256, None) == 1


ARGS = ["lengths", "new_tokens", "page_rows", "held", "held_out", "free_pages", "taken", "taken_out",
        "page_refcount", "indptr", "indices", "last_page_len", "qo_indptr", "token_request",
        "positions", "slots", "ws"]


def tables_call(over, desc_over):
    d = dict(batch=5, page_size=16, row_pages=30, num_pages=200, num_indices=150, num_tokens=40,
             num_free=100, window=64, sinks=4)
    d.update({k: v for k, v in desc_over.items() if k != "reserved"})
    desc = oxd.make_build_tables_desc(**d)
    desc.reserved = desc_over.get("reserved", 0)
    a = {n: at(i) for i, n in enumerate(ARGS)}
    a.update(ws_bytes=256)
    a.update(over)
    return status(lambda: oxd.oxd_build_tables(desc, *(a[n] for n in ARGS), a["ws_bytes"], stream=0))


@pytest.mark.parametrize("over,desc_over,want", [
    *[({n: None}, {}, 1) for n in ARGS if n not in ("page_refcount", "slots")],
    ({}, dict(batch=0), 1), ({}, dict(row_pages=0), 1), ({}, dict(num_indices=0), 1),
    ({}, dict(num_tokens=-1), 1), ({}, dict(num_free=-1), 1), ({}, dict(num_pages=0), 1),
    ({}, dict(window=-1), 1), ({}, dict(sinks=-1), 1), ({}, dict(reserved=1), 1),
    ({}, dict(page_size=10), 2), ({}, dict(num_pages=1 << 31), 2), ({}, dict(row_pages=1 << 27), 2),
    ({}, dict(batch=1 << 22, row_pages=17), 2), ({}, dict(window=(1 << 30) + 1), 2),
    *[({n: at(i, 2)}, {}, 3) for i, n in enumerate(ARGS)],
    (dict(slots=at(15, 4)), {}, 3), (dict(ws=at(16, 128)), {}, 3),
    (dict(indices=at(9)), {}, 4), (dict(indptr=at(0)), {}, 4), (dict(held_out=at(3, 4)), {}, 4),
    (dict(held_out=at(6)), {}, 4), (dict(taken_out=at(3)), {}, 4), (dict(page_rows=at(5)), {}, 4),
    (dict(slots=at(14)), {}, 4), (dict(ws=at(10)), {}, 4), (dict(page_refcount=at(5)), {}, 4),
    (dict(ws_bytes=255), {}, 5),
])
def test_build_tables_refusals(over, desc_over, want):
    assert tables_call(over, desc_over) == want


def test_build_tables_arguments_that_may_be_missing():
    """They pass every check and fail at the launch, for want of a device."""
    import torch

    if torch.cuda.is_available():
        pytest.skip("a kernel would follow the addresses")
    for over, desc_over in [
            (dict(page_refcount=None, slots=None), {}),
            (dict(free_pages=None, taken=None, taken_out=None), dict(num_free=0)),
            (dict(new_tokens=None, qo_indptr=None, token_request=None, positions=None, slots=None),
             dict(num_tokens=0)),
            (dict(held_out=at(3), taken_out=at(6)), {})]:
        assert tables_call(over, desc_over) == 7


def test_device_status_string_of_an_empty_free_list():
    assert "free pages" in oxd.oxd_device_status_string(oxd.OXD_DEVICE_NO_PAGES)
