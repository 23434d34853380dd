"""GPU parity of the rotation and the per-head norms against the float64 oracle.

Tolerances.  An output is rounded once: at most finfo.eps / 2 of its value.  Before that, in fp32:
cosine and sine are within 2^-22 (the reduced angle's rounding, 2^-24 of at most pi/4, and
sincospif's error), the magnitude and the two products and their sum add four roundings of 2^-24, so
a rotated element is within 2^-21 m (|a| + |b|).  A norm's factor adds 2^-20 (at most 24 roundings
of the sum of squares, halved by the root, and the root's and the products' own).
"""
import numpy as np
import pytest

import context_oracle as O

pytestmark = pytest.mark.gpu

KINDS = {"none": {}, "linear": dict(factor=8.0), "ntk": dict(factor=4.0),
         "parts": dict(factor=8.0, orig_len=8192, low=1.0, high=4.0), "yarn": dict(factor=4.0, orig_len=32768, magnitude=1.1386)}


@pytest.fixture(scope="module")
def msa(cuda_device):
    import long_context_memory_b200 as m

    return m


def _dtype(name):
    import torch

    return {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[name]


def _f64(t):
    return t.detach().cpu().double().numpy()


def _theta(rot_dim, scaling):
    kw = {k: v for k, v in KINDS[scaling].items() if k != "magnitude"}
    return O.rotary_theta(rot_dim, 1e6, scaling, **kw), KINDS[scaling].get("magnitude", 1.0)


def _pair_l1(x, theta, layout):
    """|a| + |b| of the pair of each element (|x| where nothing is rotated)."""
    h = len(theta)
    y = np.abs(x).copy()
    a = list(range(h)) if layout == "half" else [2 * i for i in range(h)]
    b = [h + i for i in range(h)] if layout == "half" else [2 * i + 1 for i in range(h)]
    y[..., a] = y[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y


def _check(got, ref, scale, rel, where=""):
    import torch

    fin = torch.finfo(got.dtype)
    err = np.abs(_f64(got) - ref)
    tol = fin.eps / 2 * np.abs(ref) * (1 + 2.0 ** -7) + rel * scale + fin.smallest_normal * fin.eps
    assert np.all(err <= tol), f"{where}: worst {np.max(err / tol):.2f} of the tolerance at {np.unravel_index(np.argmax(err / tol), err.shape)}"


def _inputs(rng, rows, n_q, n_kv, D, dtype, dev, sliced):
    """q, k, v heads [rows, heads, D]: slices of one fused tensor, or tensors of their own."""
    import torch

    x = torch.from_numpy(rng.standard_normal((rows, n_q + 2 * n_kv, D)).astype(np.float32)).to(dev).to(_dtype(dtype))
    q, k, v = x[:, :n_q], x[:, n_q:n_q + n_kv], x[:, n_q + n_kv:]
    return (q, k, v) if sliced else (q.contiguous(), k.contiguous(), v.contiguous())


CASES = [  # rows, n_q, n_kv, head_dim, rot_dim, layout, scaling, dtype, sliced
    (1, 32, 8, 128, 128, "half", "yarn", "bf16", False),
    (3, 32, 8, 128, 64, "interleaved", "none", "fp16", True),
    (65, 8, 2, 64, 64, "half", "parts", "fp32", True),
    (7, 5, 1, 80, 80, "half", "linear", "bf16", False),      # R/2 = 40: 8-element vectors
    (7, 5, 1, 72, 72, "half", "ntk", "fp16", True),          # R/2 = 36: 4-element vectors
    (9, 3, 3, 72, 24, "half", "none", "bf16", False),
    (9, 3, 3, 72, 24, "interleaved", "none", "bf16", False),
    (5, 2, 1, 80, 26, "half", "yarn", "bf16", False),        # R/2 = 13: element by element
    (5, 2, 1, 80, 26, "interleaved", "yarn", "fp32", False),
    (4, 1, 1, 7, 2, "half", "none", "fp32", False),          # an odd head
    (4, 1, 1, 2, 2, "interleaved", "none", "bf16", False),
    (33, 12, 12, 192, 96, "half", "none", "bf16", True),
    (17, 7, 1, 256, 256, "interleaved", "parts", "fp16", False),
    (17, 7, 1, 256, 84, "half", "parts", "fp32", False),
    (2500, 4, 2, 96, 64, "half", "none", "bf16", True),
    (301, 40, 8, 128, 128, "half", "none", "bf16", False),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("grad", [False, True])
def test_rotate(msa, cuda_device, case, grad):
    import torch

    rows, n_q, n_kv, D, R, layout, scaling, dtype, sliced = case
    rng = np.random.default_rng(rows * 131 + D + R)
    q, k, _ = _inputs(rng, rows, n_q, n_kv, D, dtype, cuda_device, sliced)
    pos = rng.integers(-5, 1 << 20, size=rows).astype(np.int32)
    pos[0] = 2 ** 31 - 1
    theta, mag = _theta(R, scaling)
    rot = msa.rotary(D, R, layout=layout, scaling=scaling, **KINDS[scaling])
    p = torch.from_numpy(pos).to(cuda_device)
    out, k_out = msa.rotate(rot, q, p, k=k, grad=grad)
    for x, y, name in ((q, out, "q"), (k, k_out, "k")):
        ref = O.rotate_heads(_f64(x), pos, theta, layout, mag, grad)
        _check(y, ref, mag * _pair_l1(_f64(x), theta, layout), 2.0 ** -21, name)
        assert torch.equal(y[..., R:], x[..., R:])  # what is not rotated is copied
    # in place, and the queries alone, give the same bits
    q2, k2 = q.clone(memory_format=torch.contiguous_format), k.clone(memory_format=torch.contiguous_format)
    msa.rotate(rot, q2, p, k=k2, grad=grad, out=q2, k_out=k2)
    assert torch.equal(q2, out) and torch.equal(k2, k_out)
    assert torch.equal(msa.rotate(rot, q, p, grad=grad), out)
    torch.cuda.synchronize()
    assert msa.check_device_errors() == 0


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("offset", [0.0, 1.0])
def test_head_norm_rotate(msa, cuda_device, case, offset):
    import torch

    rows, n_q, n_kv, D, R, layout, scaling, dtype, sliced = case
    rng = np.random.default_rng(rows * 77 + D + R)
    q, k, _ = _inputs(rng, rows, n_q, n_kv, D, dtype, cuda_device, sliced)
    pos = rng.integers(0, 1 << 20, size=rows).astype(np.int32)
    w = [torch.from_numpy((0.3 * rng.standard_normal(D) + 1 - offset).astype(np.float32)).to(cuda_device).to(q.dtype)
         for _ in range(2)]
    theta, mag = _theta(R, scaling)
    rot = msa.rotary(D, R, layout=layout, scaling=scaling, **KINDS[scaling])
    p = torch.from_numpy(pos).to(cuda_device)
    out, k_out = msa.head_norm_rotate(rot, q, k, w[0], w[1], p, eps=1e-5, weight_offset=offset)
    for x, wt, y in ((q, w[0], out), (k, w[1], k_out)):
        n = O.head_norm(_f64(x), _f64(wt), offset, 1e-5)
        _check(y, O.rotate_heads(n, pos, theta, layout, mag), mag * _pair_l1(n, theta, layout), 2.0 ** -19)
    # without weights; the keys alone as "queries"; in place
    y = msa.head_norm_rotate(rot, k, None, None, None, p, eps=1e-5)
    n = O.head_norm(_f64(k), None, 0.0, 1e-5)
    _check(y, O.rotate_heads(n, pos, theta, layout, mag), mag * _pair_l1(n, theta, layout), 2.0 ** -19)
    q2 = q.clone()
    msa.head_norm_rotate(rot, q2, k, w[0], w[1], p, eps=1e-5, weight_offset=offset, out=q2)
    assert torch.equal(q2, out)


@pytest.mark.parametrize("case", CASES)
def test_head_norm_rotate_grad(msa, cuda_device, case):
    import torch

    rows, n_q, n_kv, D, R, layout, scaling, dtype, sliced = case
    rng = np.random.default_rng(rows * 31 + D + R)
    q, k, _ = _inputs(rng, rows, n_q, n_kv, D, dtype, cuda_device, sliced)
    dq, dk, _ = _inputs(rng, rows, n_q, n_kv, D, dtype, cuda_device, not sliced)
    pos = rng.integers(0, 1 << 20, size=rows).astype(np.int32)
    w = [torch.from_numpy((0.3 * rng.standard_normal(D) + 1).astype(np.float32)).to(cuda_device).to(q.dtype)
         for _ in range(2)]
    theta, mag = _theta(R, scaling)
    rot = msa.rotary(D, R, layout=layout, scaling=scaling, **KINDS[scaling])
    p = torch.from_numpy(pos).to(cuda_device)
    got = msa.head_norm_rotate_grad(rot, q, k, w[0], w[1], p, dq, dk, eps=1e-5)
    for i, (x, wt, g) in enumerate(((q, w[0], dq), (k, w[1], dk))):
        dx, dw = O.head_norm_rotate_grad(_f64(x), _f64(wt), _f64(g), pos, theta, layout, mag, 0.0, 1e-5)
        # dx = r (u - n mean(u n)): u carries the rotation's error, the two means the sums' (as r)
        z = mag * _pair_l1(_f64(g), theta, layout)
        u = z * np.abs(_f64(wt))
        r = 1 / np.sqrt(np.mean(_f64(x) ** 2, -1, keepdims=True) + 1e-5)
        n = np.abs(_f64(x)) * r
        _check(got[i], dx, r * (u + n * np.mean(u * n, -1, keepdims=True)), 2.0 ** -18, "dx")
        # a lane adds up at most 128 terms, then trees over lanes, warps and CTAs (48 more)
        err = np.abs(_f64(got[2 + i]) - dw)
        assert np.all(err <= (2.0 ** -18 + 176 * 2.0 ** -24) * np.sum(z * n, (0, 1)) + 2.0 ** -24 * np.abs(dw)), "dw"
    again = msa.head_norm_rotate_grad(rot, q, k, w[0], w[1], p, dq, dk, eps=1e-5)
    assert all(torch.equal(a, b) for a, b in zip(got, again))  # sums in a fixed order
    # the queries alone, without a weight
    alone = msa.head_norm_rotate_grad(rot, q, None, None, None, p, dq, None, eps=1e-5)
    dx, _ = O.head_norm_rotate_grad(_f64(q), None, _f64(dq), pos, theta, layout, mag, 0.0, 1e-5)
    z = mag * _pair_l1(_f64(dq), theta, layout)
    r = 1 / np.sqrt(np.mean(_f64(q) ** 2, -1, keepdims=True) + 1e-5)
    n = np.abs(_f64(q)) * r
    _check(alone[0], dx, r * (z + n * np.mean(z * n, -1, keepdims=True)), 2.0 ** -18)
    assert alone[1] is None and alone[3] is None


@pytest.mark.parametrize("case", [CASES[0], CASES[2], CASES[4], CASES[7], CASES[11], CASES[15]])
@pytest.mark.parametrize("B", [1, 3])
def test_head_norm_append(msa, cuda_device, case, B):
    import torch

    rows, n_q, n_kv, D, R, layout, scaling, dtype, sliced = case
    rows, T = B * min(rows, 9), 23
    M = rows // B
    rng = np.random.default_rng(rows + D)
    q, k, v = _inputs(rng, rows, n_q, n_kv, D, dtype, cuda_device, sliced)
    slots = np.concatenate([rng.permutation(T)[:M] for _ in range(B)]).astype(np.int32)
    slots[-1] = -1 if M > 1 else slots[-1]  # a padded row
    pos = (1000 + slots).astype(np.int32)
    w = torch.from_numpy((0.3 * rng.standard_normal(D) + 1).astype(np.float32)).to(cuda_device).to(q.dtype)
    rot = msa.rotary(D, R, layout=layout, scaling=scaling, **KINDS[scaling])
    p, sl = torch.from_numpy(pos).to(cuda_device), torch.from_numpy(slots).to(cuda_device)
    K = torch.full((B, T, n_kv, D), float("nan"), dtype=q.dtype, device=cuda_device)
    V = K.clone()
    out = msa.head_norm_append(rot, q, k, v, w, w, p, sl, K, V)
    ref_q, ref_k = msa.head_norm_rotate(rot, q, k, w, w, p)
    assert torch.equal(out, ref_q)
    K2, V2 = torch.full_like(K, float("nan")), torch.full_like(V, float("nan"))
    for r in range(rows):
        if slots[r] >= 0:
            K2[r // M, slots[r]], V2[r // M, slots[r]] = ref_k[r], v[r]
    assert torch.equal(K.nan_to_num(77.0), K2.nan_to_num(77.0)) and torch.equal(V.nan_to_num(77.0), V2.nan_to_num(77.0))
    assert msa.check_device_errors() == 0


def test_bad_slots_are_left_out_and_reported(msa, cuda_device):
    import torch

    rot = msa.rotary(64)
    q = torch.randn(4, 2, 64, device=cuda_device)
    K, V = (torch.zeros(2, 5, 2, 64, device=cuda_device) for _ in range(2))
    pos = torch.zeros(4, dtype=torch.int32, device=cuda_device)
    slots = torch.tensor([0, 5, -2, 4], dtype=torch.int32, device=cuda_device)
    msa.head_norm_append(rot, q, q, q, None, None, pos, slots, K, V)
    with pytest.raises(msa.MSAError):
        msa.check_device_errors()
    assert V[0, 0].abs().sum() > 0 and V[1, 4].abs().sum() > 0
    assert V[0, 1:].abs().sum() == 0 and V[1, :4].abs().sum() == 0


def test_zero_rows_zero_heads_and_eps(msa, cuda_device):
    """No rows: nothing happens (weight gradients 0).  A head of zeros: 0 out, finite gradients."""
    import torch

    rot = msa.rotary(128)
    e = torch.empty(0, 4, 128, dtype=torch.bfloat16, device=cuda_device)
    pos = torch.empty(0, dtype=torch.int32, device=cuda_device)
    assert msa.rotate(rot, e, pos).shape == (0, 4, 128)
    assert msa.head_norm_rotate(rot, e, e, None, None, pos)[1].shape == (0, 4, 128)
    g = msa.head_norm_rotate_grad(rot, e, e, None, None, pos, e, e)
    assert float(g[2].abs().sum()) == 0 and float(g[3].abs().sum()) == 0
    x = torch.zeros(3, 5, 128, device=cuda_device)
    x[1, 2] = 1.0
    p = torch.arange(3, dtype=torch.int32, device=cuda_device)
    y = msa.head_norm_rotate(rot, x, None, None, None, p)
    assert float(y[0].abs().sum()) == 0 and torch.isfinite(y).all()
    g = msa.head_norm_rotate_grad(rot, x, None, None, None, p, torch.ones_like(x), None)
    assert torch.isfinite(g[0]).all() and torch.isfinite(g[2]).all()
    # eps = 0 is the caller's business for zero heads, and exact for others: 5 heads leave lanes idle
    x = torch.randn(3, 5, 128, device=cuda_device)
    g = msa.head_norm_rotate_grad(rot, x, None, None, None, p, torch.ones_like(x), None, eps=0.0)
    assert torch.isfinite(g[0]).all() and torch.isfinite(g[2]).all()


def test_values_outside_the_rotation_do_not_mix(msa, cuda_device):
    """NaN and infinities stay in their own head and pair."""
    import torch

    rot = msa.rotary(128, 64)
    x = torch.randn(4, 8, 128, device=cuda_device, dtype=torch.bfloat16)
    pos = torch.arange(4, dtype=torch.int32, device=cuda_device) + 5
    ref = msa.rotate(rot, x, pos)
    y = x.clone()
    y[1, 3, 100], y[2, 4, 5] = float("inf"), float("nan")
    got = msa.rotate(rot, y, pos)
    ok = torch.ones_like(x, dtype=torch.bool)
    ok[1, 3, 100] = ok[2, 4, 5] = ok[2, 4, 37] = False
    assert torch.equal(got[ok], ref[ok]) and torch.isinf(got[1, 3, 100])
    n_ref, n_got = (msa.head_norm_rotate(rot, t, None, None, None, pos) for t in (x, y))
    ok = torch.ones(4, 8, dtype=torch.bool, device=cuda_device)
    ok[1, 3] = ok[2, 4] = False
    assert torch.equal(n_got[ok], n_ref[ok])


def test_layouts_of_memory_agree(msa, cuda_device):
    """Head-major tensors, a broadcast input, an unaligned slice: the same values as contiguous ones."""
    import torch

    rot = msa.rotary(64, scaling="linear", factor=2.0)
    x = torch.randn(6, 4, 64, device=cuda_device, dtype=torch.bfloat16)
    w = torch.randn(64, device=cuda_device, dtype=torch.bfloat16)
    pos = torch.arange(6, dtype=torch.int32, device=cuda_device)
    ref = msa.head_norm_rotate(rot, x, None, w, None, pos)
    hm = x.transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.empty_like(hm)
    assert torch.equal(msa.head_norm_rotate(rot, hm, None, w, None, pos, out=out), ref) and out.stride() == hm.stride()
    flat = torch.empty(6 * 4 * 64 + 1, device=cuda_device, dtype=torch.bfloat16)
    un = flat[1:].view(6, 4, 64)
    un.copy_(x)
    _check(msa.head_norm_rotate(rot, un, None, w, None, pos), _f64(ref), np.abs(_f64(ref)) + 1, 2.0 ** -8)
    b = x[:1, :1].expand(6, 4, 64)
    assert torch.equal(msa.rotate(rot, b, pos), msa.rotate(rot, b.contiguous(), pos))


def test_rows_past_2_31_elements(msa, cuda_device):
    import torch

    gen = torch.Generator(device=cuda_device).manual_seed(2)
    step = 1_100_000_000
    big = torch.empty(2 * step + 256, dtype=torch.bfloat16, device=cuda_device)
    x = big.as_strided((3, 4, 64), (step, 64, 1))
    x.copy_(torch.randn(3, 4, 64, generator=gen, device=cuda_device))
    small, rot = x.contiguous(), msa.rotary(64)
    pos = torch.tensor([1, -2, 2 ** 31 - 1], dtype=torch.int32, device=cuda_device)
    w = small[0, 0].contiguous()
    ref = msa.head_norm_rotate(rot, small, small, w, w, pos)
    assert all(torch.equal(a, b) for a, b in zip(msa.head_norm_rotate(rot, x, x, w, w, pos), ref))
    ref = msa.head_norm_rotate_grad(rot, small, None, w, None, pos, small, None)
    assert all(torch.equal(a, b) for a, b in zip(msa.head_norm_rotate_grad(rot, x, None, w, None, pos, x, None)[::2], ref[::2]))
    ref = msa.rotate(rot, small, pos)
    msa.rotate(rot, x, pos, out=x)  # in place
    assert torch.equal(x, ref)


def test_streams_and_graphs(msa, cuda_device):
    import torch

    rot = msa.rotary(128, scaling="yarn", factor=4.0, orig_len=4096)
    B, n_q, n_kv, D, T = 3, 8, 2, 128, 16
    gen = torch.Generator(device=cuda_device).manual_seed(3)
    rn = lambda *s: torch.randn(*s, generator=gen, device=cuda_device).to(torch.bfloat16)
    q, k, v, w = rn(B, n_q, D), rn(B, n_kv, D), rn(B, n_kv, D), rn(D)
    slots = torch.tensor([0, 3, 9], dtype=torch.int32, device=cuda_device)
    pos = slots + 100
    caches = [torch.zeros(B, T, n_kv, D, dtype=torch.bfloat16, device=cuda_device) for _ in range(4)]
    dq, dk = rn(B, n_q, D), rn(B, n_kv, D)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    a = msa.head_norm_append(rot, q, k, v, w, w, pos, slots, caches[0], caches[1], stream=st)
    b = msa.head_norm_rotate_grad(rot, q, k, w, w, pos, dq, dk, stream=st.cuda_stream)
    st.synchronize()
    with torch.cuda.stream(st):  # warm, then capture
        out = msa.head_norm_append(rot, q, k, v, w, w, pos, slots, caches[2], caches[3])
        msa.head_norm_rotate_grad(rot, q, k, w, w, pos, dq, dk)
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = msa.head_norm_append(rot, q, k, v, w, w, pos, slots, caches[2], caches[3])
        grads = msa.head_norm_rotate_grad(rot, q, k, w, w, pos, dq, dk)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, a) and all(torch.equal(x, y) for x, y in zip(caches[:2], caches[2:]))
    assert all(torch.equal(x, y) for x, y in zip(grads, b))
    q.copy_(rn(B, n_q, D))
    slots.add_(1)
    pos.add_(1)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, msa.head_norm_rotate(rot, q, None, w, None, pos))
    assert torch.equal(caches[3][0, 1], v[0]) and msa.check_device_errors() == 0
