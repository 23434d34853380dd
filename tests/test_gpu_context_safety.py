"""What the rotation, norm and draft-tree calls report, and what they hold up while they run."""
import os
import subprocess
import sys

import numpy as np
import pytest

from test_gpu_tree import _case, _check, _run

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def msa(cuda_device):
    import long_context_memory_b200 as m

    return m


@pytest.mark.parametrize("B", [1, 8, 9, 32, 33, 70])
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


@pytest.mark.parametrize("B,k", [(1, 2), (8, 1), (9, 1), (33, 1), (40, 0)])
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
    if B > 8 and k:
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
    assert state == [0] and steps >= 5, name
"""


def test_other_threads_run_beside_a_call(msa, cuda_device, tmp_path):
    """A call that has to wait in the library (a full launch queue, say) leaves the interpreter to the other
    threads: against a library whose calls take 0.3 s, this one counts on in steps of 5 ms."""
    src, so = tmp_path / "slow.cpp", tmp_path / "slow.so"
    src.write_text(SLOW)
    subprocess.run(["g++", "-shared", "-fPIC", str(src), "-o", str(so)], check=True)
    r = subprocess.run([sys.executable, "-c", BESIDE, ROOT, str(so)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr


@pytest.mark.parametrize("D,n_q,n_kv", [(64, 8, 2), (128, 32, 8)])
def test_normalised_heads_in_the_decode_attention(msa, cuda_device, D, n_q, n_kv):
    """sparse_attend rotates its query and its new key itself: it takes heads that head_norm_rotate normalised
    at position 0, where nothing is turned.  The norm is rounded once (2^-8 of its value, and fp32 arithmetic
    within 2^-19 of it); the attention has its own tolerance on the heads that it was given."""
    import torch

    import context_oracle as C
    import oracle as O
    from long_context_memory_b200 import workloads as W

    rng = np.random.default_rng(D)
    B, T, off = 2, 40, 5
    dev, dims = cuda_device, W.Dims(hidden=256, n_q=n_q, n_kv=n_kv, head_dim=D, n_r=4, d_r=64)
    bf = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(dev).to(torch.bfloat16)
    bits = lambda t: t.cpu().view(torch.int16).numpy().view(np.uint16)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)
    fused, wq, wk = bf(B, n_q + 2 * n_kv, D), bf(D), bf(D)
    q0, k0, v = fused[:, :n_q], fused[:, n_q:n_q + n_kv], fused[:, n_q + n_kv:].contiguous()
    rot = msa.rotary(D, base=dims.rope_base)
    q, k = msa.head_norm_rotate(rot, q0, k0, wq, wk, i32([0] * B))
    f64 = lambda t: t.cpu().double().numpy()
    for x, w, y in ((q0, wq, q), (k0, wk, k)):
        n = C.head_norm(f64(x), f64(w))
        assert np.all(np.abs(f64(y) - n) <= (2.0 ** -8 + 2.0 ** -19) * np.abs(n) + 1e-30)
    co, idx, loc = np.array([0, 4, 9, 11], dtype=np.int32), np.array([[2, 0], [1, 2]], dtype=np.int32), np.array([T, 7], dtype=np.int32)
    Kb, Vb, K, V = bf(11, n_kv, D), bf(11, n_kv, D), bf(B, T, n_kv, D), bf(B, T, n_kv, D)
    Kr = msa.rotate(rot, K.view(B * T, n_kv, D), (torch.arange(T, device=dev, dtype=torch.int32) + off).repeat(B)).view(K.shape)
    Vr = V.clone()
    got = msa.sparse_attend(dims, q, Kb, Vb, i32(co), i32(idx), Kr, Vr, i32(loc), off, k_loc_rotated=True, k_new=k, v_new=v)
    for b in range(B):
        K[b, loc[b] - 1], V[b, loc[b] - 1] = k[b], v[b]
    ref = O.sparse_attend(bits(q), bits(Kb), bits(Vb), co, idx, bits(K), bits(V), loc, off, dims.rope_base)
    err = np.abs(f64(got.view(B, n_q, D)) - ref)
    assert np.all(err <= 2e-2 + 2e-2 * np.abs(ref)) and msa.check_device_errors() == 0
    # the token's key stands in the cache as head_norm_rotate turns it, but for one more rounding
    _, at = msa.head_norm_rotate(rot, q0, k0, wq, wk, i32(loc - 1 + off))
    for b in range(B):
        a = np.abs(f64(k[b]))
        pair = a + np.roll(a, D // 2, axis=-1)
        assert np.all(np.abs(f64(Kr[b, loc[b] - 1]) - f64(at[b])) <= (3 * 2.0 ** -8 + 2.0 ** -18) * pair)


@pytest.mark.parametrize("B,M,n_q,n_kv,D,T,k", [(8, 5, 8, 2, 64, 200, 7), (9, 5, 8, 2, 64, 200, 7), (20, 40, 8, 2, 64, 150, 3),
                                               (32, 3, 16, 8, 128, 90, 16), (12, 17, 32, 8, 128, 300, 0)])
def test_batches_about_the_planning_s_limit(msa, cuda_device, B, M, n_q, n_kv, D, T, k):
    """Ragged batches on both sides of the size from which a kernel counts the documents' rows."""
    import torch

    loc = np.random.default_rng(B).integers(0, T + 1, size=B)
    c = _case(B + k, B, M, n_q, n_kv, D, T, loc, k, True, cuda_device)
    got = _run(msa, c, cuda_device)
    _check(got, c)
    assert torch.equal(got, _run(msa, c, cuda_device)) and msa.check_device_errors() == 0


@pytest.mark.parametrize("rows", [2367, 2369, 4000, 8193])
@pytest.mark.parametrize("form", ["rotate", "norm"])
def test_long_rows_in_shares(msa, cuda_device, rows, form):
    """Rows that are taken whole or in two shares: a row's result does not depend on the rows beside it."""
    import torch

    gen = torch.Generator(device=cuda_device).manual_seed(rows)
    rn = lambda *s: torch.randn(*s, generator=gen, device=cuda_device)
    q, k, w = rn(rows, 32, 128), rn(rows, 7, 128), rn(128)
    p = torch.randint(0, 1 << 20, (rows,), generator=gen, device=cuda_device, dtype=torch.int32)
    rot = msa.rotary(128, 64, layout="interleaved")
    f = (lambda q, k, p: msa.rotate(rot, q, p, k=k)) if form == "rotate" else (lambda q, k, p: msa.head_norm_rotate(rot, q, k, w, w, p))
    out = f(q, k, p)
    for lo in range(0, rows, 100):
        part = f(q[lo:lo + 100], k[lo:lo + 100], p[lo:lo + 100])
        assert torch.equal(out[0][lo:lo + 100], part[0]) and torch.equal(out[1][lo:lo + 100], part[1])
    assert msa.check_device_errors() == 0


def test_two_threads_call_at_once(msa, cuda_device):
    """Calls of two Python threads, each on a stream of its own, give what one thread's calls give."""
    import threading

    import torch

    cs = [_case(41, 2, 24, 16, 4, 64, 900, [900, 333], 3, False, cuda_device), _case(42, 12, 9, 8, 2, 128, 200, [1, 199] * 6, 2, True, cuda_device)]
    rots = [msa.rotary(64, scaling="linear", factor=2.0), msa.rotary(64, 32, layout="interleaved")]
    x = torch.randn(50, 8, 64, device=cuda_device, dtype=torch.bfloat16)
    pos = torch.arange(50, device=cuda_device, dtype=torch.int32)
    ref = [(_run(msa, c, cuda_device), msa.rotate(r, x, pos)) for c, r in zip(cs, rots)]
    torch.cuda.synchronize()
    got, errors = [[], []], []

    def work(i):
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                for _ in range(60):
                    got[i].append((_run(msa, cs[i], cuda_device), msa.rotate(rots[i], x, pos)))
            st.synchronize()
        except Exception as e:  # (a thread's exception is the test's)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    assert all(torch.equal(a, ref[i][0]) and torch.equal(b, ref[i][1]) for i in range(2) for a, b in got[i])
    assert len(got[0]) == len(got[1]) == 60 and msa.check_device_errors() == 0
