"""The device status: its texts, and that a workspace may hold any data before a run without it reading as one."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest

import paged_kv_decode_attn_gb300 as oxd

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    oxd.build()


def next_epochs(n):
    f = getattr(oxd.lib(), "_ZN3oxd14next_run_epochEv")  # oxd::next_run_epoch()
    f.restype = ctypes.c_uint32
    return np.asarray([f() for _ in range(n)], np.uint32)


def test_epochs_are_words_that_data_does_not_hold():
    e = next_epochs(1000)
    assert len(set(e.tolist())) == 1000
    assert (e.view(np.int32) < -2 ** 28).all()          # no lengths, pages, positions or counts
    assert (e.view(np.float32) < -2.0 ** 32).all()      # no activations in F32 ...
    assert ((e & 0xffff0000).view(np.float32) < -2.0 ** 32).all()  # ... or, as its upper half, bf16


def test_epochs_of_two_processes_differ():
    """Both start anywhere (they are alike once in 2^29 times)."""
    code = ("import sys; sys.path[:0] = [%r, %r]; import test_status_epochs as t; print(t.next_epochs(1)[0])"
            % (ROOT, os.path.join(ROOT, "tests")))
    got = {subprocess.run([sys.executable, "-c", code], check=True, capture_output=True, text=True).stdout
           for _ in range(2)}
    assert len(got) == 2


CHILD = """
import sys
sys.path[:0] = [%r]
import numpy as np, torch
import paged_kv_decode_attn_gb300 as oxd
oxd.build()
B = 2
ints = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
k = torch.zeros((4, 16, 1, 128), dtype=torch.bfloat16, device="cuda")
q = torch.zeros((B, 4, 128), dtype=torch.bfloat16, device="cuda")
out, lse = torch.empty_like(q), torch.empty((B, 4), device="cuda")
d = oxd.make_window_decode_desc(B, 4, 1, 16, "NHD", 4, 2, 64, 4)
tables = ints(0, 1, 2), ints(0, 1), ints(5, 9)
for run in range(1, 61):  # the workspace holds lengths: 30 tokens, then as many as runs so far
    ws = torch.tensor([30, run] * 32, dtype=torch.int32, device="cuda").view(torch.uint8)
    oxd.oxd_window_decode(d, q, k, k, *tables, 0.1, out, lse, ws)
    assert oxd.oxd_read_device_status(ws) == 0, run
bad = ints(0, 7)  # a page outside the pool
for run in range(61, 121):
    ws = torch.tensor([30, run] * 32, dtype=torch.int32, device="cuda").view(torch.uint8)
    oxd.oxd_window_decode(d, q, k, k, tables[0], bad, tables[2], 0.1, out, lse, ws)
    assert oxd.oxd_read_device_status(ws) == oxd.OXD_DEVICE_BAD_PAGE, run
"""


@pytest.mark.gpu
def test_lengths_left_in_the_workspace_are_no_status():
    import torch

    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    r = subprocess.run([sys.executable, "-c", CHILD % ROOT], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_the_text_of_a_bad_position_fits_the_tables_and_decodes_too():
    text = oxd.oxd_device_status_string(oxd.OXD_DEVICE_BAD_POSITION)
    assert "append" not in text and all(w in text for w in ("position", "length", "table entry"))
