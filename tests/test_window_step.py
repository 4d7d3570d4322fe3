"""The step of a windowed model as the README documents it: a workspace for every launch whose errors matter."""
import ast
import os
import re

import numpy as np
import pytest
import torch

import paged_kv_decode_attn_gb300 as oxd
import window_ref as Wr
from quant_helpers import bf16, f64

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LAUNCHES = ("oxd_build_tables", "oxd_rope_axes_append", "oxd_window_decode")


def documented_step():
    with open(os.path.join(ROOT, "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    return next(b for b in blocks if "oxd_build_tables(" in b)


def workspaces(step):
    """The expression that each launch passes as its workspace, by the launch."""
    calls = [n for n in ast.walk(ast.parse(step)) if isinstance(n, ast.Call)]
    return {n.func.attr: ast.unparse(n.args[-1]) for n in calls
            if isinstance(n.func, ast.Attribute) and n.func.attr in LAUNCHES}


def test_every_launch_has_a_workspace_of_its_own():
    """A run replaces the status of the one before it on the same workspace."""
    ws = workspaces(documented_step())
    assert sorted(ws) == sorted(LAUNCHES)
    assert len(set(ws.values())) == len(LAUNCHES), ws


def test_every_name_is_made_by_the_step_or_a_users_tensor():
    made = {"oxd", "torch", "B", "pages", "len", "lengths", "ones", "page_rows", "held", "free", "taken", "refcount",
            "indptr", "indices", "last_page_len", "qo_indptr", "token_request", "positions", "q", "k", "v",
            "q_out", "k_pages", "v_pages", "sm_scale", "out", "lse", "range"}
    tree = ast.parse(documented_step())
    names = [n for n in ast.walk(tree) if isinstance(n, ast.Name)]
    made |= {n.id for n in names if isinstance(n.ctx, ast.Store)}
    assert {n.id for n in names if isinstance(n.ctx, ast.Load)} <= made


@pytest.mark.gpu
def test_a_request_that_outgrows_its_row_is_reported():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    oxd.build()
    rng = np.random.default_rng(1)
    B, pages, row = 3, 400, 256  # (the step's rows list 256 pages of 16 tokens)
    n = [100, 40, row * 16]
    dev = (lambda a, t=np.int32: torch.as_tensor(np.asarray(a, t), device="cuda"))  # noqa: E731
    order = rng.permutation(pages).astype(np.int32)
    held = [-(-x // 16) for x in n]
    page_rows, at = np.full((B, row), -1, np.int32), 0
    for b, h in enumerate(held):
        page_rows[b, :h] = order[at:at + h]
        at += h
    refcount = np.ones(pages, np.int32)
    k_pages, v_pages = (rng.normal(size=(pages, 16, 8, 128)) for _ in "kv")
    names = dict(
        oxd=oxd, torch=torch, B=B, pages=pages, lengths=dev(n), ones=dev([1] * B), page_rows=dev(page_rows),
        held=dev(held), free=dev(order[at:]), taken=dev([0]), refcount=dev(refcount),
        indptr=dev([0] * (B + 1)), indices=dev([-9] * (B * row)), last_page_len=dev([0] * B),
        qo_indptr=dev([0] * (B + 1)), token_request=dev([-9] * B), positions=dev([-9] * B),
        q=bf16(rng.normal(size=(B, 32, 128))), k=bf16(rng.normal(size=(B, 8, 128))),
        v=bf16(rng.normal(size=(B, 8, 128))), k_pages=bf16(k_pages), v_pages=bf16(v_pages), sm_scale=128 ** -0.5,
        lse=torch.empty((B, 32), device="cuda"))
    names["q_out"], names["out"] = torch.empty_like(names["q"]), torch.empty_like(names["q"])
    # (what an older text of the step takes from the blocks before it)
    names["ws"] = torch.empty(256, dtype=torch.uint8, device="cuda")
    names["ad"] = oxd.make_axes_append_desc(B, B, 32, 8, 16, "NHD", pages, B * row)
    step = documented_step()
    exec(step, names)
    code = {f: oxd.oxd_read_device_status(eval(w, names)) for f, w in workspaces(step).items()}
    assert code["oxd_build_tables"] == oxd.OXD_DEVICE_BAD_POSITION
    assert code["oxd_window_decode"] == 0
    # the request is listed as empty, the two before it are served
    out, lse = f64(names["out"]), f64(names["lse"])
    assert (out[2] == 0).all() and np.isneginf(lse[2]).all()
    kc, vc = [], []
    for pool, dst in ((names["k_pages"], kc), (names["v_pages"], vc)):
        p = f64(pool)
        for b in range(2):
            dst.append(p[names["page_rows"].cpu().numpy()[b, :-(-(n[b] + 1) // 16)]].reshape(-1, 8, 128)
                       [:n[b] + 1].swapaxes(0, 1))
    ref = Wr.attention(f64(names["q_out"])[:2], kc, vc, [n[0] + 1, n[1] + 1], [1, 1], 1024, 4, 128 ** -0.5)
    Wr.assert_close(out[:2], lse[:2], ref)
