"""Refusals and planning of the 4-bit cache's entry points, the multi-axis append and the page
copies, on the CPU with addresses that are never dereferenced."""
import ctypes

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


# ------------------------------------------------------------------ decode

def quant_plan(lengths, G=4, Hkv=2, ps=16, num_sms=152, **kw):
    lengths = np.asarray(lengths)
    pages = -(-lengths // ps)
    indptr = np.concatenate([[0], np.cumsum(pages)]).astype(np.int32)
    last = (lengths - (pages - 1) * ps).astype(np.int32)
    desc = oxd.make_desc(len(lengths), G * Hkv, Hkv, ps, kw.pop("layout", "NHD"), int(indptr[-1]),
                         num_sms=num_sms, **kw)
    return oxd.oxd_quant_decode_plan(desc, indptr, last)


@pytest.mark.parametrize("G,variant", [(1, 6), (8, 6), (9, 7), (16, 7), (17, 8), (32, 8)])
def test_plan_picks_the_variant_by_group(G, variant):
    info = quant_plan([100, 5000], G=G).info
    assert info.kernel_variant == variant
    assert info.total_kv_tokens == 5100


@pytest.mark.parametrize("kw,want", [
    (dict(shared_prefix_tokens=32, share_group=2), 2),
    (dict(G=33), 2),
    (dict(layout=7), 1),
    (dict(wait_timeout_ns=-1), 1),
])
def test_plan_refusals(kw, want):
    assert status(lambda: quant_plan([100, 200], **kw)) == want


def test_plan_refuses_bad_tables():
    desc = oxd.make_desc(2, 8, 2, 16, "NHD", 10, num_sms=152)
    for indptr, last in (([0, 2, 2], [16, 1]), ([0, 2, 4], [0, 1]), ([0, 2, 4], [17, 1]),
                         ([-1, 2, 4], [1, 1])):
        assert status(lambda: oxd.oxd_quant_decode_plan(desc, indptr, last)) == 1
    desc = oxd.make_desc(1, 8, 2, 12, "NHD", 10, num_sms=152)
    assert status(lambda: oxd.oxd_quant_decode_plan(desc, [0, 1], [1])) == 2
    desc = oxd.make_desc(1, 8, 2, 16, "NHD", 10, head_dim=64, num_sms=152)
    assert status(lambda: oxd.oxd_quant_decode_plan(desc, [0, 1], [1])) == 2


def run_args(plan, **over):
    a = dict(q=at(0), k=at(1), v=at(2), ks=at(3), vs=at(4), indptr=at(5), indices=at(6), last=at(7),
             scale=0.1, out=at(8), lse=at(9), ws=at(10), ws_bytes=plan.workspace_bytes)
    a.update(over)
    return lambda: oxd.oxd_quant_decode_run(
        plan, a["q"], oxd.KvPools(a["k"], a["v"], a["ks"], a["vs"]), a["indptr"], a["indices"],
        a["last"], a["scale"], a["out"], a["lse"], a["ws"], a["ws_bytes"], stream=0)


@pytest.mark.parametrize("over,want", [
    *[({n: None}, 1) for n in ("q", "k", "v", "ks", "vs", "indptr", "indices", "last", "out", "ws")],
    ({"scale": float("nan")}, 1), ({"scale": float("inf")}, 1),
    *[({n: at(20, 8)}, 3) for n in ("q", "k", "v", "ks", "vs", "out")],
    *[({n: at(20, 2)}, 3) for n in ("indptr", "indices", "last", "lse")],
    ({"ws": at(20, 128)}, 3), ({"ws_bytes": 0}, 5),
    *[({"out": at(i)}, 4) for i in (0, 1, 2, 3, 4, 9)],
    ({"lse": at(4, 4)}, 4), ({"ws": at(2)}, 4), ({"ws": at(3)}, 4),
])
def test_run_refusals(over, want):
    plan = quant_plan([100, 200])
    assert status(run_args(plan, **over)) == want


def test_run_refuses_the_other_caches_plans():
    plan = quant_plan([100])
    st = oxd.lib().oxd_paged_decode_run(plan.handle, at(0), at(1), at(2), at(5), at(6), at(7),
                                        ctypes.c_float(0.1), at(8), at(9), at(10), 1 << 30, 0)
    assert st == 6
    desc = oxd.make_desc(1, 8, 2, 16, "NHD", 10, num_sms=152)
    bf = oxd.oxd_paged_decode_plan(desc, [0, 1], [1])
    assert status(run_args(bf)) == 6
    plan.destroy()
    assert oxd.lib().oxd_quant_decode_run(plan.handle, *[at(0)] * 5, ctypes.c_float(0.1), at(8),
                                          at(9), at(10), 1 << 30, 0) == 6


def test_null_cache_struct():
    plan = quant_plan([100])
    assert oxd.lib().oxd_quant_decode_run(plan.handle, at(0), None, at(5), at(6), at(7),
                                          ctypes.c_float(0.1), at(8), at(9), at(10), 1 << 30, 0) == 1


# ------------------------------------------------------------------ appends

def append_call(four, desc_over=(), **over):
    desc = oxd.make_axes_append_desc(10, 3, 8, 2, 16, "NHD", 50, 20, sections=(16, 24, 24))
    for n, v in dict(desc_over).items():
        if n == "axis0":
            desc.pair_axis[0] = v
        else:
            setattr(desc, n, v)
    a = dict(q=at(0), k=at(1), v=at(2), req=at(3), pos=at(4), rope=at(5), indptr=at(6), indices=at(7),
             ref=at(8), q_out=at(9), kp=at(10), vp=at(11), ks=at(12), vs=at(13), ws=at(14),
             ws_bytes=256)
    a.update(over)
    head = [a[n] for n in ("q", "k", "v", "req", "pos", "rope", "indptr", "indices", "ref", "q_out")]
    if four:
        return lambda: oxd.oxd_quant_rope_append(
            desc, *head, oxd.KvPools(a["kp"], a["vp"], a["ks"], a["vs"]), a["ws"], a["ws_bytes"],
            stream=0)
    return lambda: oxd.oxd_rope_axes_append(desc, *head, a["kp"], a["vp"], a["ws"], a["ws_bytes"],
                                            stream=0)


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("desc,over,want", [
    *[({}, {n: None}, 1) for n in ("q", "k", "v", "req", "pos", "indptr", "indices", "ref", "q_out",
                                   "kp", "vp", "ws")],
    ({"num_tokens": 0}, {}, 1), ({"batch": 0}, {}, 1), ({"num_indices": 0}, {}, 1),
    ({"num_pages": 0}, {}, 1), ({"layout": 2}, {}, 1), ({"reserved": 1}, {}, 1),
    ({"num_axes": 0}, {}, 1), ({"num_axes": 5}, {}, 1), ({"num_axes": 2}, {}, 1),
    ({"axis0": 3}, {}, 1), ({"rope_theta": 1.0}, {}, 1), ({"rope_theta": float("inf")}, {}, 1),
    ({"head_dim": 64}, {}, 2), ({"page_size": 12}, {}, 2), ({"num_pages": 1 << 31}, {}, 2),
    ({"num_tokens": 2 ** 31 - 1}, {}, 2), ({"num_qo_heads": 2 ** 31 - 1}, {}, 2),
    *[({}, {n: at(20, 8)}, 3) for n in ("q", "k", "v", "q_out", "kp", "vp")],
    *[({}, {n: at(20, 2)}, 3) for n in ("req", "pos", "rope", "indptr", "indices", "ref")],
    ({}, {"ws": at(20, 64)}, 3), ({}, {"ws_bytes": 255}, 5),
    *[({}, {"q_out": at(i)}, 4) for i in (1, 2, 3, 4, 5, 6, 7, 8, 10, 11)],
    ({}, {"q_out": at(0, 16)}, 4), ({}, {"kp": at(0)}, 4), ({}, {"kp": at(11)}, 4),
    ({}, {"ws": at(0)}, 4), ({}, {"ws": at(5)}, 4), ({}, {"vp": at(8)}, 4),
])
def test_append_refusals(four, desc, over, want):
    assert status(append_call(four, desc, **over)) == want


@pytest.mark.parametrize("over,want", [({"ks": None}, 1), ({"vs": None}, 1), ({"ks": at(20, 8)}, 3),
                                       ({"vs": at(10)}, 4), ({"ks": at(1)}, 4), ({"ks": at(9)}, 4)])
def test_quant_append_refusals(over, want):
    assert status(append_call(True, **over)) == want


def test_sections_must_cover_all_pairs():
    with pytest.raises(oxd.OxdError):
        oxd.make_axes_append_desc(1, 1, 1, 1, 16, "NHD", 1, 1, sections=(16, 24))
    d = oxd.make_axes_append_desc(1, 1, 1, 1, 16, "NHD", 1, 1, pair_axis=[i % 3 for i in range(64)])
    assert d.num_axes == 3 and list(d.pair_axis[:4]) == [0, 1, 2, 0]


# ------------------------------------------------------------------ page copies

def copy_call(desc_over=(), src=None, dst=None, **over):
    desc = oxd.make_copy_pages_desc(4, 2, 16, "bf16", "NHD", 30, "e2m1", "NHD", 20)
    for n, v in dict(desc_over).items():
        setattr(desc, n, v)
    a = dict(sp=at(6), dp=at(7), ref=at(8), ws=at(9), ws_bytes=256)
    a.update(over)
    src = (at(0), at(1)) if src is None else src
    dst = (at(2), at(3), at(4), at(5)) if dst is None else dst
    return lambda: oxd.oxd_copy_pages(desc, oxd.KvPools(*src), oxd.KvPools(*dst), a["sp"], a["dp"],
                                      a["ref"], a["ws"], a["ws_bytes"], stream=0)


BF = {"dst_format": 0}


@pytest.mark.parametrize("desc,kw,want", [
    ({}, dict(src=(None, at(1))), 1), ({}, dict(src=(at(0), None)), 1),
    ({}, dict(dst=(at(2), at(3))), 1), ({}, dict(dst=(at(2), at(3), at(4), None)), 1),
    ({}, dict(src=(at(0), at(1), at(20), at(21))), 1),
    ({}, dict(sp=None), 1), ({}, dict(dp=None), 1), ({}, dict(ws=None, ws_bytes=256), 1),
    ({"num_pairs": -1}, {}, 1), ({"num_kv_heads": 0}, {}, 1), ({"src_num_pages": 0}, {}, 1),
    ({"dst_num_pages": 0}, {}, 1), ({"src_format": 2}, {}, 1), ({"dst_format": -1}, {}, 1),
    ({"src_layout": 2}, {}, 1), ({"dst_layout": -1}, {}, 1),
    ({"head_dim": 64}, {}, 2), ({"page_size": 24}, {}, 2), ({"dst_num_pages": 1 << 31}, {}, 2),
    ({}, dict(src=(at(20, 8), at(1))), 3), ({}, dict(dst=(at(2), at(3), at(20, 8), at(5))), 3),
    ({}, dict(sp=at(20, 2)), 3), ({}, dict(ref=at(20, 1)), 3), ({}, dict(ws=at(20, 16)), 3),
    ({}, dict(ws_bytes=128), 5),
    ({}, dict(dst=(at(0), at(3), at(4), at(5))), 4), ({}, dict(dst=(at(2), at(2), at(4), at(5))), 4),
    ({}, dict(sp=at(4)), 4), ({}, dict(ref=at(2)), 4), ({}, dict(ws=at(2)), 4), ({}, dict(ws=at(0)), 4),
    # one pool under two shapes, or K and V exchanged
    (BF, dict(dst=(at(0), at(1))), 4),
    ({**BF, "dst_num_pages": 30, "dst_layout": 1}, dict(dst=(at(0), at(1))), 4),
    ({**BF, "dst_num_pages": 30}, dict(dst=(at(1), at(0))), 4),
    ({**BF, "dst_num_pages": 30}, dict(dst=(at(0, 16), at(1, 16))), 4),
])
def test_copy_refusals(desc, kw, want):
    assert status(copy_call(desc, **kw)) == want


def test_reserved_fields_must_be_zero():
    desc = oxd.make_copy_pages_desc(4, 2, 16, "bf16", "NHD", 30, "bf16", "NHD", 20)
    desc.reserved[1] = 1
    assert status(lambda: oxd.oxd_copy_pages(desc, oxd.KvPools(at(0), at(1)), oxd.KvPools(at(2), at(3)),
                                             at(6), at(7), None, at(9), 256, stream=0)) == 1


@pytest.mark.parametrize("n", [2 ** 31 - 65534, 2 ** 31 - 1])
def test_copy_refuses_lists_its_counter_cannot_walk(n):
    # (far pools, so that nothing overlaps a list of 8 GB)
    desc = oxd.make_copy_pages_desc(n, 2, 16, "bf16", "NHD", 30, "bf16", "NHD", 20)
    assert status(lambda: oxd.oxd_copy_pages(desc, oxd.KvPools(at(0), at(1)), oxd.KvPools(at(2), at(3)),
                                             at(6), at(7), None, at(9), 256, stream=0)) == 2


@pytest.mark.parametrize("B,Hkv", [(38, 1), (5, 8), (7, 8), (8, 8), (64, 1), (63, 1)])
@pytest.mark.parametrize("L", [512, 1024, 2048, 4000])
@pytest.mark.parametrize("num_sms", [152, 100])
def test_the_clusters_of_a_plan_are_resident_at_once(B, Hkv, L, num_sms):
    # the instance that merges in its first CTA asks for 80 KB of a SM's 228
    info = quant_plan([L] * B, Hkv=Hkv, layout="HND", num_sms=num_sms).info
    assert info.grid_ctas <= 2 * num_sms or info.cluster_size == 0
    if L == 1024 and num_sms == 152:
        assert info.cluster_size == 304 // (B * Hkv) and info.launches_per_run == 1
