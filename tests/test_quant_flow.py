"""The 4-bit cache's operators as a serving program uses them, in one run."""
import numpy as np
import pytest
import torch

import paged_kv_decode_attn_gb300 as oxd
import quant_ref as R
from quant_helpers import assert_decode, bf16, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def setup():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    oxd.build()


def dev(a):
    return torch.as_tensor(np.asarray(a, np.int32), device="cuda")


@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("G,Hkv", [(4, 2), (16, 1), (1, 4)])
def test_prompt_pack_fork_decode_unpack_prefill(layout, G, Hkv):
    """A prompt with an image is appended on three axes as bf16, prefilled, and its pages packed
    into a 4-bit cache; the sequence is forked (full pages shared, the last made private by a page
    copy); both branches append new tokens and decode; a branch's pages are unpacked and another
    chunk is prefilled against them."""
    ps, n, Hq = 16, 75, G * Hkv
    rng = np.random.default_rng(G)
    axis = np.repeat(np.arange(3), (16, 24, 24))
    rope = np.stack([np.arange(n)] * 3)
    rope[:, 20:60] = [[20] * 40, 20 + np.arange(40) // 8, 20 + np.arange(40) % 8]
    q, k, v = (R.round_bf16(rng.normal(size=(n, h, 128))) for h in (Hq, Hkv, Hkv))
    pages = -(-n // ps)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    ones = torch.ones(64, dtype=torch.int32, device="cuda")

    def bf_pools(count):
        s = (count, ps, Hkv, 128) if layout == "NHD" else (count, Hkv, ps, 128)
        return [torch.zeros(s, dtype=torch.bfloat16, device="cuda") for _ in "kv"]

    # prompt into bf16 pages 0..4, and its prefill
    bf = bf_pools(8)
    desc = oxd.make_axes_append_desc(n, 1, Hq, Hkv, ps, layout, 8, pages, sections=(16, 24, 24))
    dq = bf16(q)
    oxd.oxd_rope_axes_append(desc, dq, bf16(k), bf16(v), dev([0] * n), dev(range(n)), dev(rope),
                             dev([0, pages]), dev(range(pages)), ones, dq, *bf, ws)
    assert oxd.oxd_read_device_status(ws) == 0
    last = n - (pages - 1) * ps

    def prefill(pools, count, q_rows, table, kv_len):
        p = -(-kv_len // ps)
        pd = oxd.make_prefill_desc(1, Hq, Hkv, ps, layout, count)
        lens = [kv_len - (p - 1) * ps]
        plan = oxd.oxd_paged_prefill_plan(pd, [0, len(q_rows)], [0, p], lens)
        out = torch.empty_like(q_rows)
        w = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
        oxd.oxd_paged_prefill_run(plan, q_rows, *pools, dev([0, len(q_rows)]), dev([0, p]), dev(table),
                                  dev(lens), 128 ** -0.5, out, None, w)
        assert oxd.oxd_read_device_status(w) == 0
        return out

    assert torch.isfinite(prefill(bf, 8, dq, range(pages), n)).all()

    # packed into pages 3..7 of a 4-bit cache of 16
    s = (16, ps, Hkv, 64) if layout == "NHD" else (16, Hkv, ps, 64)
    codes = [torch.zeros(s, dtype=torch.uint8, device="cuda") for _ in "kv"]
    scales = [torch.zeros(16, Hkv, ps, 4, dtype=torch.float16, device="cuda") for _ in "kv"]
    cache = oxd.KvPools(*codes, *scales)
    cd = oxd.make_copy_pages_desc(pages, Hkv, ps, "bf16", layout, 8, "e2m1", layout, 16)
    oxd.oxd_copy_pages(cd, oxd.KvPools(*bf), cache, dev(range(pages)), dev(range(3, 3 + pages)), ones, ws)
    assert oxd.oxd_read_device_status(ws) == 0

    # fork: full pages 3..6 shared, page 7 copied to 12; both branches get a page more
    fd = oxd.make_copy_pages_desc(1, Hkv, ps, "e2m1", layout, 16, "e2m1", layout, 16)
    refcount = torch.ones(16, dtype=torch.int32, device="cuda")
    refcount[3:7] = 2
    oxd.oxd_copy_pages(fd, cache, cache, dev([7]), dev([12]), refcount, ws)
    assert oxd.oxd_read_device_status(ws) == 0
    tables = [[3, 4, 5, 6, 7, 0], [3, 4, 5, 6, 12, 15]]

    # both branches append 7 tokens (across a page's end) and decode after each
    indices, grown = np.concatenate(tables), []
    for step in range(7):
        at = n + step
        qn, kn, vn = (R.round_bf16(rng.normal(size=(2, h, 128))) for h in (Hq, Hkv, Hkv))
        ad = oxd.make_axes_append_desc(2, 2, Hq, Hkv, ps, layout, 16, 12, sections=(16, 24, 24))
        q_out = torch.empty(2, Hq, 128, dtype=torch.bfloat16, device="cuda")
        new_rope = np.full((3, 2), at - 32)
        oxd.oxd_quant_rope_append(ad, bf16(qn), bf16(kn), bf16(vn), dev([0, 1]), dev([at, at]),
                                  dev(new_rope), dev([0, 6, 12]), dev(indices), refcount, q_out,
                                  cache, ws)
        assert oxd.oxd_read_device_status(ws) == 0
        grown.append((R.round_bf16(R.rotate(kn, new_rope, axis, 1e4)), vn))
        L = at + 1
        p = -(-L // ps)
        table = np.concatenate([t[:p] for t in tables])
        indptr, lens = np.array([0, p, 2 * p], np.int32), np.array([L - (p - 1) * ps] * 2, np.int32)
        plan = oxd.oxd_quant_decode_plan(oxd.make_desc(2, Hq, Hkv, ps, layout, 16), indptr, lens)
        out, lse = torch.empty_like(q_out), torch.empty(2, Hq, device="cuda")
        w = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
        oxd.oxd_quant_decode_run(plan, q_out, cache, dev(indptr), dev(table), dev(lens), 128 ** -0.5,
                                 out, lse, w)
        assert oxd.oxd_read_device_status(w) == 0
        kv, vv = (R.pool_values(c.cpu().numpy(), x.cpu().numpy(), layout) for c, x in zip(codes, scales))
        assert_decode(out, lse, R.decode(f64(q_out), kv, vv, indptr, table, [L, L], layout, 128 ** -0.5))

    # what the cache holds is the prompt's rows (bf16, then 4 bits) and the appended ones
    for i, name in enumerate("kv"):
        held = R.pool_values(codes[i].cpu().numpy(), scales[i].cpu().numpy(), layout)
        src = f64(bf[i])
        for b, t in enumerate(tables):
            rows = R.tokens(held, np.array(t), layout)
            prompt = R.tokens(src, np.arange(pages), layout)[:, :n]
            np.testing.assert_array_equal(rows[:, :n], R.values(*R.hold(prompt)))
            for step, pair in enumerate(grown):
                np.testing.assert_array_equal(rows[:, n + step], R.values(*R.hold(pair[i][b])))

    # branch 1 unpacked into bf16 pages, and a prefill of its last 5 tokens against them
    back = bf_pools(6)
    ud = oxd.make_copy_pages_desc(6, Hkv, ps, "e2m1", layout, 16, "bf16", layout, 6)
    oxd.oxd_copy_pages(ud, cache, oxd.KvPools(*back), dev(tables[1]), dev(range(6)), None, ws)
    assert oxd.oxd_read_device_status(ws) == 0
    kv, vv = (R.pool_values(c.cpu().numpy(), x.cpu().numpy(), layout) for c, x in zip(codes, scales))
    for pool, held in zip(back, (kv, vv)):
        np.testing.assert_array_equal(f64(pool), f64(bf16(held[tables[1]])))
    q5 = bf16(R.round_bf16(rng.normal(size=(5, Hq, 128))))
    out = prefill(back, 6, q5, range(6), n + 7)
    for i in range(5):
        L = n + 7 - 4 + i
        p = -(-L // ps)
        want = R.decode(f64(q5[i:i + 1]), f64(back[0]), f64(back[1]), [0, p], np.arange(p), [L], layout,
                        128 ** -0.5)[0]
        assert (np.abs(f64(out[i:i + 1]) - want) <= 1.5e-2 + 1e-2 * np.abs(want)).all()
