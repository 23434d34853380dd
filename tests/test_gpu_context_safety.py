"""What the rotation, norm and draft-tree calls report, and what they hold up while they run."""
import os
import subprocess
import sys

import numpy as np
import pytest

from test_gpu_tree import _case, _run

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def msa(cuda_device):
    import long_context_memory_b200 as m

    return m


@pytest.mark.parametrize("B", [1, 32, 33, 70])
@pytest.mark.parametrize("bad", ["only", "beside an empty one", "nothing drafted"])
def test_bad_documents_are_reported_in_every_batch(msa, cuda_device, B, bad):
    """A document id out of range raises the device error whatever the batch, also where its query has
    no pooled row left or no draft in use."""
    k = 2 if bad == "beside an empty one" else 1
    c = _case(B, B, 3, 4, 2, 64, 20, np.full(B, 20), k, False, cuda_device)
    ids = len(c["off"]) - 1
    _run(msa, c, cuda_device)
    assert msa.check_device_errors() == 0
    if bad == "beside an empty one":  # the last document has no rows
        c["off"] = np.append(c["off"], c["off"][-1])
        c["top"][-1] = ids
        ids += 1
        _run(msa, c, cuda_device)
        assert msa.check_device_errors() == 0
    if bad == "nothing drafted":
        c["n_draft"] = np.zeros(B, dtype=np.int32)
    for value in (ids, -1):
        c["top"][-1, -1] = value
        _run(msa, c, cuda_device)
        with pytest.raises(msa.MSAError):
            msa.check_device_errors()


@pytest.mark.parametrize("B,k", [(1, 2), (32, 1), (33, 1), (40, 0)])
def test_kernels_are_traced_under_their_own_names(msa, cuda_device, B, k):
    """The attention alone: no time of the plan's, and the counting of large batches' rows by its name."""
    c = _case(B, B, 3, 4, 2, 64, 20, np.full(B, 20), k, False, cuda_device)
    _run(msa, c, cuda_device)
    msa.trace_enable(True)
    try:
        msa.trace_reset()
        _run(msa, c, cuda_device)
        launches = {name: n for name, (_, n) in msa.trace_read().items() if n}
    finally:
        msa.trace_enable(False)
    want = {"tree_attend": 1, "tree_combine": 1}
    if B > 32 and k:
        want["tree_select"] = 1
    assert launches == want


SLOW = r"""
#include <time.h>
extern "C" {
static int slow() { timespec t{0, 300000000}; nanosleep(&t, nullptr); return 0; }
int msa_rotate() { return slow(); }
int msa_head_norm_rotate() { return slow(); }
int msa_head_norm_append() { return slow(); }
int msa_head_norm_rotate_grad() { return slow(); }
int msa_tree_plan() { return slow(); }
int msa_tree_attend() { return slow(); }
int msa_tree_commit() { return slow(); }
}
"""

BESIDE = r"""
import ctypes, importlib.util, sys, threading, time
sys.path.insert(0, sys.argv[1])
import torch
import long_context_memory_b200 as msa
from long_context_memory_b200 import workloads as W
spec = importlib.util.spec_from_file_location("_fastcall", sys.argv[1] + "/long_context_memory_b200/_fastcall.so")
fast = importlib.util.module_from_spec(spec)
spec.loader.exec_module(fast)
fast.bind(sys.argv[2])  # a library whose calls only take their time
bf = dict(dtype=torch.bfloat16, device="cuda")
z = lambda *s: torch.zeros(*s, **bf)
i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
f = lambda *s: torch.zeros(*s, device="cuda")
r, d, ws = msa.rotary(64), msa.Dims.of(W.Dims(hidden=256, n_q=2, n_kv=1, head_dim=64, n_r=4, d_r=64)), i(1 << 20)
q, k, p, K, V = z(2, 2, 64), z(2, 1, 64), i(2), z(2, 8, 1, 64), z(2, 8, 1, 64)
D = lambda: z(2, 3, 1, 64)
calls = dict(
    rotate=(r, q, p, k, False, z(2, 2, 64), z(2, 1, 64), None),
    head_norm_rotate=(r, q, k, None, None, p, 1e-6, 0.0, z(2, 2, 64), z(2, 1, 64), None),
    head_norm_append=(r, q, k, z(2, 1, 64), None, None, p, i(2), K, V, 1e-6, 0.0, z(2, 2, 64), None),
    head_norm_rotate_grad=(r, q, k, None, None, p, z(2, 2, 64), z(2, 1, 64), 1e-6, 0.0, z(2, 2, 64), z(2, 1, 64), f(64), f(64), ws, None),
    tree_plan=(i(2, 3), i(2), 0, None, i(2, 3, 1), i(2, 3), None),
    tree_attend=(d, z(2, 3, 2, 64), D(), D(), i(2, 3, 1), K, V, i(2), None, None, None, None, None, 0.0, z(2, 3, 2, 64), ws, None),
    tree_commit=(D(), D(), i(2, 2), i(2), K, V, i(2), i(2), None))
for name, args in calls.items():
    state, steps = [], 0
    t = threading.Thread(target=lambda: state.append(getattr(fast, name)(*args)))
    t.start()
    while t.is_alive() and steps < 10000:
        time.sleep(0.005)
        steps += 1
    t.join()
    print(name, state, steps)
    assert state == [0] and steps >= 10, name
"""


def test_other_threads_run_beside_a_call(msa, cuda_device, tmp_path):
    """A call that has to wait in the library (a full launch queue, say) leaves the interpreter to the other
    threads: against a library whose calls take 0.3 s, this one counts on in steps of 5 ms."""
    src, so = tmp_path / "slow.cpp", tmp_path / "slow.so"
    src.write_text(SLOW)
    subprocess.run(["g++", "-shared", "-fPIC", str(src), "-o", str(so)], check=True)
    r = subprocess.run([sys.executable, "-c", BESIDE, ROOT, str(so)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
