"""Host-side tests of the rotation, per-head norm and draft-tree calls: the frequency tables, the
oracle's gradients against differences, and the refusals of the C ABI and the binding (no GPU)."""
import ctypes
import struct

import numpy as np
import pytest

import context_oracle as O

FAKE = 0x10000  # 16-byte aligned non-null "device" address; never dereferenced
FAR = 0x10000000000  # far behind it: tensors that must not overlap


@pytest.fixture(scope="module")
def msa():
    from long_context_memory_b200 import build

    if build.needs_build():
        build.build()
    import long_context_memory_b200 as m

    return m


SCALINGS = [dict(), dict(scaling="linear", factor=8.0), dict(scaling="ntk", factor=4.0),
            dict(scaling="parts", factor=8.0, orig_len=8192, low=1.0, high=4.0),
            dict(scaling="yarn", factor=4.0, orig_len=32768), dict(scaling="yarn", factor=2.5, orig_len=1)]


@pytest.mark.parametrize("kw", SCALINGS)
@pytest.mark.parametrize("rot_dim", [2, 4, 26, 64, 128, 256])
def test_turns_match_the_definition(msa, kw, rot_dim):
    r = msa.rotary(256, rot_dim, base=5e5, **kw)
    turns = msa.rotary_turns(r)
    theta = O.rotary_theta(rot_dim, 5e5, **kw)
    # the fraction is cut at 2^-64 of a turn; the definition in 64-bit floats is good to ~1e-13
    got = turns.astype(np.float64) * 2.0 ** -64
    assert np.max(np.abs(got - theta / (2 * np.pi)) / (theta / (2 * np.pi)) - 2.0 ** -64 * 2 * np.pi / theta) < 1e-11


def test_oracle_gradients_match_differences():
    rng = np.random.default_rng(1)
    theta = O.rotary_theta(6, 100.0)
    pos = np.array([3, -7])
    x, w, dy = rng.standard_normal((2, 3, 10)), rng.standard_normal(10), rng.standard_normal((2, 3, 10))
    for layout in ("half", "interleaved"):
        f = lambda x, w: np.sum(dy * O.rotate_heads(O.head_norm(x, w, 1.0, 1e-3), pos, theta, layout, 1.3))
        dx, dw = O.head_norm_rotate_grad(x, w, dy, pos, theta, layout, 1.3, 1.0, 1e-3)
        h = 1e-6
        for idx in [(0, 0, 0), (0, 2, 4), (1, 1, 5), (1, 0, 9)]:
            d = np.zeros_like(x)
            d[idx] = h
            assert abs((f(x + d, w) - f(x - d, w)) / (2 * h) - dx[idx]) < 1e-7
        for i in (0, 5, 9):
            d = np.zeros_like(w)
            d[i] = h
            assert abs((f(x, w + d) - f(x, w - d)) / (2 * h) - dw[i]) < 1e-7


def _heads(msa, heads=4, D=64, inp=FAKE, out=FAKE, in_row=None, in_head=None, out_row=None, out_head=None):
    pick = lambda v, d: d if v is None else v
    return struct.pack("@PPqqqqii", inp or 0, out or 0, pick(in_row, heads * D), pick(in_head, D), pick(out_row, heads * D),
                           pick(out_head, D), heads, 0)


def _rotate(msa, rot=None, dtype=0, rows=3, pos=FAKE, q=None, k=None):
    rot = rot or msa.rotary(64)
    q = q or _heads(msa)
    return msa.lib.msa_rotate(ctypes.byref(rot), dtype, q, k, rows, pos, 0, None)


@pytest.fixture
def no_launch(monkeypatch):
    """Valid calls stop with MSA_ERR_CUDA before their first launch."""
    monkeypatch.setenv("MSA_FAULT", "launch")


def test_rotate_validation(msa, no_launch):
    assert _rotate(msa) == 4
    assert _rotate(msa, k=_heads(msa, 2)) == 4
    for bad in (dict(head_dim=0), dict(head_dim=258)):
        assert _rotate(msa, msa.rotary(**bad)) == 2
    for bad in (dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=66), dict(base=1.0), dict(base=float("inf")),
                dict(factor=0.5), dict(factor=float("nan")), dict(magnitude=0.0),
                dict(scaling="parts", factor=2.0), dict(scaling="yarn", factor=2.0, orig_len=100, low=4.0, high=4.0),
                dict(scaling="yarn", factor=2.0, orig_len=100, low=0.0)):
        assert _rotate(msa, msa.rotary(64, **bad)) == 1, bad
    bad = msa.rotary(64)
    bad.layout = 2
    assert _rotate(msa, bad) == 1
    bad = msa.rotary(64)
    bad.scaling = 5
    assert _rotate(msa, bad) == 1
    assert _rotate(msa, dtype=3) == 1
    assert _rotate(msa, rows=-1) == 1
    assert _rotate(msa, rows=2 ** 31) == 1
    assert _rotate(msa, pos=None) == 1
    assert _rotate(msa, pos=FAKE + 2) == 1
    assert _rotate(msa, q=_heads(msa, heads=0)) == 1
    assert _rotate(msa, q=_heads(msa, inp=None)) == 1
    assert _rotate(msa, q=_heads(msa, out=None)) == 1
    assert _rotate(msa, q=_heads(msa, inp=FAKE + 1)) == 1
    assert _rotate(msa, q=_heads(msa, in_row=-1)) == 1
    assert _rotate(msa, q=_heads(msa, out=2 * FAKE, in_row=0, in_head=0)) == 4  # a broadcast input is read
    assert _rotate(msa, q=_heads(msa, out_row=0)) == 1      # rows of the output on top of each other
    assert _rotate(msa, q=_heads(msa, out_head=32)) == 1
    assert _rotate(msa, q=_heads(msa, out_row=128)) == 1    # rows reach into each other's heads
    assert _rotate(msa, q=_heads(msa, in_row=512, out_row=256)) == 1  # in place with other strides
    assert _rotate(msa, q=_heads(msa, in_row=64, in_head=192, out_row=64, out_head=192)) == 4  # head-major
    with pytest.raises(ValueError):
        msa.rotary(64, layout="quarter")
    with pytest.raises(ValueError):
        msa.rotary(64, scaling="longer")


def _norm(msa, form, eps=1e-6, off=0.0, qw=FAKE, kw=FAKE, rows=4, ws=FAKE * 16, ws_bytes=1 << 24, B=2, T=8, slots=FAKE,
          K=FAKE, V=FAR, v=None, k="k", dk="k", dkw=FAKE):
    r, q = msa.rotary(64), _heads(msa)
    kk = _heads(msa, 2) if k else None
    L = msa.lib
    if form == "forward":
        return L.msa_head_norm_rotate(ctypes.byref(r), 0, q, kk, rows, qw, kw, off, eps, FAKE, None)
    if form == "append":
        return L.msa_head_norm_append(ctypes.byref(r), 0, q, kk, v or _heads(msa, 2), rows, qw, kw, off, eps, FAKE,
                                      slots, K, V, B, T, None)
    return L.msa_head_norm_rotate_grad(ctypes.byref(r), 0, q, kk, q, _heads(msa, 2) if dk else None, rows, qw, kw, off,
                                       eps, FAKE, FAKE, dkw, ws, ws_bytes, None)


@pytest.mark.parametrize("form", ["forward", "append", "backward"])
def test_head_norm_validation(msa, no_launch, form):
    assert _norm(msa, form) == 4
    assert _norm(msa, form, qw=None, kw=None) == 4
    assert _norm(msa, form, eps=-1.0) == 1
    assert _norm(msa, form, eps=float("nan")) == 1
    assert _norm(msa, form, off=float("inf")) == 1
    assert _norm(msa, form, qw=FAKE + 1) == 1
    assert _norm(msa, form, kw=FAKE + 1) == 1
    assert _norm(msa, form, rows=-4) == 1


def test_head_norm_append_and_grad_validation(msa, no_launch):
    assert _norm(msa, "append", rows=5) == 1          # not a multiple of B
    assert _norm(msa, "append", B=0) == 1
    assert _norm(msa, "append", T=0) == 1
    assert _norm(msa, "append", slots=None) == 1
    assert _norm(msa, "append", K=None) == 1
    cache = 2 * 8 * 2 * 64 * 2
    assert _norm(msa, "append", V=FAKE + cache - 16) == 1 and _norm(msa, "append", V=FAKE + cache) == 4
    assert _norm(msa, "append", v=_heads(msa, 3)) == 1  # as many value heads as key heads
    assert _norm(msa, "append", k=None) == 1
    assert _norm(msa, "backward", ws_bytes=16) == 3
    assert "workspace too small" in msa.lib.msa_last_error().decode()
    assert _norm(msa, "backward", ws=FAKE + 16) == 1
    assert _norm(msa, "backward", dk=None) == 1
    assert _norm(msa, "backward", k=None, dk=None) == 1  # dk_weight without k
    assert _norm(msa, "backward", k=None, dk=None, dkw=None) == 4
    assert msa.head_norm_grad_workspace_size(msa.rotary(64), -1, 4, 2) == 0


def _dims(msa, **kw):
    d = dict(hidden=64, n_q=8, n_kv=2, head_dim=64, n_r=1, d_r=64, chunk=64, rope_base=1e6)
    d.update(kw)
    return msa.Dims(*d.values())


def _plan(msa, B=2, M=5, off=0, parents=FAKE, n=None, loc=FAKE, mask=FAR, pos=2 * FAR):
    return msa.lib.msa_tree_plan(parents, n, loc, B, M, off, mask, pos, None)


def test_tree_plan_validation(msa, no_launch):
    assert _plan(msa) == 4
    assert _plan(msa, M=256) == 4
    for bad in (dict(B=0), dict(B=65536), dict(M=0), dict(M=257), dict(off=-1), dict(parents=None), dict(loc=None),
                dict(mask=None), dict(pos=None), dict(mask=FAR + 4), dict(n=FAKE + 8),
                dict(mask=FAKE), dict(pos=FAKE + 16), dict(pos=FAR), dict(n=3 * FAR, mask=3 * FAR)):
        assert _plan(msa, **bad) == 1, bad


def _attend(msa, dims=None, B=2, M=5, T=10, k=0, n_docs=4, n_chunks=9, scale=0.0, ws_bytes=None, q=FAKE, K=FAKE, mem=FAKE,
            mask=FAKE, loc=FAKE, out=FAR):
    d = dims or _dims(msa)
    need = msa.lib.msa_tree_attend_workspace_size(ctypes.byref(d), B, M, k, T)
    return msa.lib.msa_tree_attend(ctypes.byref(d), q, FAKE, FAKE, mask, None, B, M, K, K, loc, T, mem, mem, mem, n_docs,
                                   n_chunks, mem, k, scale, out, FAKE * 16, need if ws_bytes is None else ws_bytes, None)


def test_tree_attend_validation(msa, no_launch):
    assert _attend(msa) == 4
    assert _attend(msa, k=3) == 4
    assert _attend(msa, T=0, K=None) == 4              # drafts alone
    assert _attend(msa, mem=None) == 4
    assert _attend(msa, out=FAR, q=FAR + 2 * 5 * 8 * 64 * 2) == 4
    assert _attend(msa, k=256, n_docs=300, n_chunks=(1 << 23) - 1) == 4
    for bad in (dict(B=0), dict(B=4097), dict(M=0), dict(M=257), dict(T=-1), dict(k=-1), dict(k=257, n_docs=300, n_chunks=400),
                dict(k=5), dict(k=3, n_chunks=3), dict(k=3, mem=None), dict(K=None), dict(q=None), dict(q=FAKE + 8),
                dict(mask=None), dict(loc=None), dict(scale=-1.0), dict(scale=float("nan")),
                dict(dims=_dims(msa, n_q=7)), dict(out=FAKE), dict(out=FAKE + 16), dict(out=FAR, K=FAR), dict(out=FAR, k=3, mem=FAR),
                dict(out=FAR, q=FAR + 2 * 5 * 8 * 64 * 2 - 16), dict(k=256, n_docs=300, n_chunks=1 << 23)):
        assert _attend(msa, **{**dict(ws_bytes=1 << 30), **bad}) == 1, bad
    for bad in (dict(head_dim=96), dict(n_q=34), dict(n_q=16, n_kv=16), dict(chunk=32)):
        assert _attend(msa, dims=_dims(msa, **bad), ws_bytes=1 << 30) == 2, bad
    assert _attend(msa, ws_bytes=0) == 3
    assert msa.lib.msa_tree_attend_workspace_size(ctypes.byref(_dims(msa, head_dim=96)), 1, 1, 0, 1) == 0


def _commit(msa, B=2, M=5, A=3, T=9, path=FAKE, new=2 * FAR, K=FAR, V=3 * FAR, Kd=FAKE):
    return msa.lib.msa_tree_commit(ctypes.byref(_dims(msa)), Kd, FAKE, path, FAKE, B, M, A, K, V, FAKE, T, new, None)


def test_tree_commit_validation(msa, no_launch):
    assert _commit(msa) == 4
    cache, drafts = 2 * 9 * 2 * 64 * 2, 2 * 5 * 2 * 64 * 2
    for bad in (dict(B=0), dict(M=257), dict(A=0), dict(A=6), dict(T=0), dict(path=None), dict(new=None), dict(new=FAKE),
                dict(K=FAR + 2), dict(V=FAR), dict(V=FAR + cache - 16), dict(Kd=FAR), dict(Kd=FAR - drafts + 16), dict(K=FAKE),
                dict(path=2 * FAR)):
        assert _commit(msa, **bad) == 1, bad
    assert _commit(msa, Kd=FAR - drafts) == 4 and _commit(msa, V=FAR + cache) == 4


def test_binding_refuses_tensors_off_the_device(msa):
    import torch

    q, pos = torch.zeros(2, 3, 64), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        msa.rotate(msa.rotary(64), q, pos)
    with pytest.raises(ValueError, match="CUDA"):
        msa.tree_plan(torch.zeros(1, 4, dtype=torch.int32), pos[:1], 0)
    kv, n = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        msa.tree_commit(kv, kv, torch.zeros(1, 2, dtype=torch.int32), n, kv, kv, n)
    with pytest.raises(ValueError, match="expected a tensor"):
        msa.tree_commit(kv, None, torch.zeros(1, 2, dtype=torch.int32), n, kv, kv, n)
    with pytest.raises(ValueError, match="structure"):
        msa.rotate(_dims(msa), q, pos)


def test_binding_refuses_wrong_shapes_and_types(msa):
    """Shapes, types and strides are checked before the device: host tensors are told what was expected
    of them (the call whose tensors fit is told that it wants CUDA tensors)."""
    import torch

    r = msa.rotary(64)
    q, k, pos = torch.zeros(4, 3, 64), torch.zeros(4, 2, 64), torch.zeros(4, dtype=torch.int32)
    for args, kw in [((r, q.double(), pos), {}), ((r, q[..., :32], pos), {}), ((r, q.reshape(12, 64), pos), {}),
                     ((r, q.transpose(1, 2).contiguous().transpose(1, 2), pos), {}), ((r, q, pos[:3]), {}),
                     ((r, q, pos.long()), {}), ((r, q, pos), dict(k=k[:3])), ((r, q, pos), dict(k=k.half())),
                     ((r, q, pos), dict(out=q[:3])), ((r, q, pos), dict(k_out=k)), ((r, q, pos), dict(k=k, k_out=q))]:
        with pytest.raises(ValueError, match="expected [^C]|k_out without k"):
            msa.rotate(*args, **kw)
    w = torch.ones(64)
    with pytest.raises(ValueError, match="expected [^C]|k_out without k"):
        msa.head_norm_rotate(r, q, k, w[:32], w, pos)
    with pytest.raises(ValueError, match="expected [^C]|k_out without k"):
        msa.head_norm_rotate_grad(r, q, k, w, w, pos, q, None)
    with pytest.raises(ValueError, match="expected [^C]|k_out without k"):
        msa.head_norm_rotate_grad(r, q, k, w, w, pos, q[:, :2], k)
    cache = torch.zeros(2, 9, 2, 64)
    for bad in (dict(v=q), dict(slots=pos[:2]), dict(K_loc=cache[:, :, :1]), dict(V_loc=cache.half()), dict(K_loc=k)):
        a = {**dict(v=k, slots=pos, K_loc=cache, V_loc=cache), **bad}
        with pytest.raises(ValueError, match="expected [^C]|k_out without k"):
            msa.head_norm_append(r, q, k, a["v"], w, w, pos, a["slots"], a["K_loc"], a["V_loc"])
    par = torch.zeros(2, 40, dtype=torch.int32)
    for bad in (dict(parents=par[0]), dict(parents=par.long()), dict(loc=pos[:3]), dict(n=pos[:3])):
        a = {**dict(parents=par, loc=pos[:2], n=None), **bad}
        with pytest.raises(ValueError, match="expected [^C]|k_out without k"):
            msa.tree_plan(a["parents"], a["loc"], 0, n_draft=a["n"])
    bf = torch.bfloat16
    d = _dims(msa)
    t = dict(q=torch.zeros(2, 40, 8, 64, dtype=bf), K_draft=torch.zeros(2, 40, 2, 64, dtype=bf),
             V_draft=torch.zeros(2, 40, 2, 64, dtype=bf), mask=torch.zeros(2, 40, 2, dtype=torch.int32),
             K_loc=torch.zeros(2, 9, 2, 64, dtype=bf), V_loc=torch.zeros(2, 9, 2, 64, dtype=bf), loc_len=pos[:2])
    for bad in (dict(q=t["q"][:, :, :4]), dict(q=t["q"].float()), dict(mask=t["mask"][..., :1]), dict(K_loc=None),
                dict(loc_len=pos), dict(V_draft=t["V_draft"][:, :39]), dict(K_bar=t["K_loc"][0]),
                dict(out=t["q"][:1]), dict(n_draft=pos), dict(V_loc=t["V_loc"][:, :8])):
        with pytest.raises(ValueError, match="expected [^C]|k_out without k"):
            msa.tree_attend(d, **{**t, **bad})
    with pytest.raises(ValueError, match="expected [^C]|k_out without k"):
        msa.tree_commit(t["K_draft"], t["V_draft"], par[:1], pos[:2], t["K_loc"], t["V_loc"], pos[:2])
    with pytest.raises(ValueError, match="ws: expected a contiguous tensor"):  # one byte, however long it looks
        msa.tree_attend(d, **t, ws=torch.zeros(1, dtype=torch.uint8).expand(1 << 24))
