"""GPU parity of the draft-tree calls against the float64 oracle.

Tolerance of the attention: the output's rounding, eps / 2 = 2^-8 of its value; each weight's rounding
to bf16 before it multiplies its value, 2^-8 of A = sum_j p_j |v_j|; the scores' fp32 sums of at most
128 products and the exponentials, within 2^-12 of A for the score sizes used here
(128 * 2^-24 * scale * sum |q k| below 2^-13, and two exp2 roundings).
"""
import numpy as np
import pytest

import context_oracle as O
from long_context_memory_b200 import workloads as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def msa(cuda_device):
    import long_context_memory_b200 as m

    return m


def _f64(t):
    return t.detach().cpu().double().numpy()


def _dims(n_q, n_kv, D):
    return W.Dims(hidden=256, n_q=n_q, n_kv=n_kv, head_dim=D, n_r=4, d_r=64)


def _trees(rng, B, M, ragged):
    parents = np.full((B, M), -1, dtype=np.int32)
    for t in range(1, M):
        parents[:, t] = rng.integers(max(-1, t - 6), t, size=B)
    n = rng.integers(0, M + 1, size=B).astype(np.int32) if ragged else np.full(B, M, dtype=np.int32)
    if ragged:
        n[-1] = M
    return parents, n


def _case(seed, B, M, n_q, n_kv, D, T, loc, k, ragged, dev, scale=1.0):
    import torch

    rng = np.random.default_rng(seed)
    bf = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(dev).to(torch.bfloat16)
    c = dict(dims=_dims(n_q, n_kv, D), B=B, M=M, k=k)
    c["parents"], c["n_draft"] = _trees(rng, B, M, ragged)
    c["loc_len"] = np.array(loc, dtype=np.int32)
    c["see"], c["pos"] = O.tree_plan(c["parents"], c["n_draft"], c["loc_len"], 7)
    c["q"] = (bf(B, M, n_q, D) * scale).contiguous()
    c["Kd"], c["Vd"] = bf(B, M, n_kv, D), bf(B, M, n_kv, D)
    c["Kl"], c["Vl"] = (bf(B, T, n_kv, D), bf(B, T, n_kv, D)) if T else (None, None)
    if k:
        sizes = rng.integers(1, 40, size=max(2 * k, 4))
        sizes[0] = 1
        c["off"] = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
        c["top"] = np.stack([rng.permutation(len(sizes))[:k] for _ in range(B)]).astype(np.int32)
        c["Kb"], c["Vb"] = bf(int(c["off"][-1]), n_kv, D), bf(int(c["off"][-1]), n_kv, D)
    return c


def _run(msa, c, dev, **kw):
    import torch

    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)
    mem = dict(K_bar=c["Kb"], V_bar=c["Vb"], chunk_off=t(c["off"]), topk_idx=t(c["top"])) if c["k"] else {}
    mask = t(O.pack_mask(c["see"]))
    return msa.tree_attend(c["dims"], c["q"], c["Kd"], c["Vd"], mask, c["Kl"], c["Vl"], t(c["loc_len"]),
                           n_draft=t(c["n_draft"]), **mem, **kw)


def _oracle(c, absv=False, scale=None):
    v = (lambda x: None if x is None else np.abs(_f64(x))) if absv else (lambda x: None if x is None else _f64(x))
    f = lambda x: None if x is None else _f64(x)
    mem = (f(c["Kb"]), v(c["Vb"]), c["off"], c["top"]) if c["k"] else (None,) * 4
    T = 0 if c["Kl"] is None else c["Kl"].shape[1]
    return O.tree_attend(f(c["q"]), f(c["Kd"]), v(c["Vd"]), c["see"], np.clip(c["n_draft"], 0, c["M"]), f(c["Kl"]), v(c["Vl"]),
                         np.clip(c["loc_len"], 0, T), *mem, scale)


def _check(got, c, scale=None, more=0.0):
    ref, A = _oracle(c, scale=scale), _oracle(c, True, scale)
    err = np.abs(_f64(got) - ref)
    tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -12 + more) * A + 1e-30
    assert np.all(err <= tol), f"worst {np.nanmax(err / tol):.2f} of the tolerance at {np.unravel_index(np.argmax(err / tol), err.shape)}"


CASES = [  # B, M, n_q, n_kv, D, t_loc_max, loc_len, k, ragged drafts
    (1, 1, 8, 2, 64, 5, [0], 0, False),
    (1, 1, 8, 2, 128, 5, [1], 1, False),
    (2, 5, 8, 2, 64, 130, [130, 3], 0, True),
    (3, 33, 8, 2, 64, 300, [127, 128, 129], 3, True),
    (2, 16, 32, 8, 128, 700, [700, 641], 4, False),
    (2, 64, 16, 4, 128, 260, [255, 256], 2, True),
    (1, 100, 16, 1, 64, 200, [77], 3, False),
    (2, 31, 7, 7, 64, 64, [64, 1], 1, True),
    (1, 127, 20, 4, 128, 90, [63], 0, False),
    (1, 256, 8, 1, 64, 140, [140], 2, False),
    (5, 3, 4, 4, 128, 513, [512, 0, 511, 513, 257], 0, True),
    (3, 20, 8, 2, 64, 0, [0, 0, 0], 0, True),
    (2, 20, 6, 2, 128, 0, [0, 0], 5, True),
]


@pytest.mark.parametrize("case", CASES)
def test_tree_attend(msa, cuda_device, case):
    import torch

    B, M, n_q, n_kv, D, T, loc, k, ragged = case
    c = _case(sum(case[:6]) + k, B, M, n_q, n_kv, D, T, loc, k, ragged, cuda_device)
    got = _run(msa, c, cuda_device)
    torch.cuda.synchronize()
    assert msa.check_device_errors() == 0
    _check(got, c)
    assert torch.equal(got, _run(msa, c, cuda_device))


@pytest.mark.parametrize("T,loc,k", [(3000, [2999], 0), (5000, [1300], 16), (9000, [9000], 1)])
def test_tree_attend_long(msa, cuda_device, T, loc, k):
    """Enough keys for many splits; the scale given by the caller."""
    c = _case(T, 1, 6, 4, 1, 128, T, loc, k, False, cuda_device)
    _check(_run(msa, c, cuda_device, softmax_scale=0.05), c, scale=0.05)


def test_tree_attend_large_scores(msa, cuda_device):
    """Scores of a few hundred: weights concentrated on a few keys, running maxima that rise late."""
    c = _case(5, 2, 17, 8, 2, 64, 400, [400, 333], 2, True, cuda_device, scale=30.0)
    # scores' absolute error grows with them: 64 * 2^-24 * sum |q k| / 8 ~ 64 * 2^-24 * 30 * 41 / 8 * 2 < 2^-9
    _check(_run(msa, c, cuda_device), c, more=2.0 ** -8)


def test_rows_without_keys_are_zero(msa, cuda_device):
    import torch

    c = _case(9, 3, 40, 8, 2, 64, 50, [0, 0, 20], 0, False, cuda_device)
    c["n_draft"] = np.array([40, 0, 31], dtype=np.int32)
    c["see"][0, 5] = False
    c["see"][0, 39] = False
    c["see"][2] = False
    got = _run(msa, c, cuda_device)
    assert float(got[0, 5].abs().sum()) == 0 and float(got[0, 39].abs().sum()) == 0
    assert float(got[1].abs().sum()) == 0 and float(got[2, 31:].abs().sum()) == 0
    assert float(got[2, :31].abs().sum(-1).min()) > 0
    _check(got, c)


def test_what_nobody_sees_may_hold_anything(msa, cuda_device):
    import torch

    c = _case(11, 3, 37, 8, 2, 128, 300, [130, 0, 299], 2, False, cuda_device)
    c["n_draft"] = np.array([30, 37, 1], dtype=np.int32)
    c["see"][1, :, 3] = False  # draft 3 of query 1: seen by nobody
    c["see"][1, :, 36] = False
    clean = _run(msa, c, cuda_device)
    _check(clean, c)
    for bad in (float("nan"), float("inf"), -float("inf")):
        for b in range(3):
            for x in (c["Kl"], c["Vl"]):
                x[b, c["loc_len"][b]:] = bad
            for x in (c["Kd"], c["Vd"], c["q"]):
                x[b, c["n_draft"][b]:] = bad
        for x in (c["Kd"], c["Vd"]):
            x[1, 3] = x[1, 36] = bad
        free = np.setdiff1d(np.arange(len(c["off"]) - 1), c["top"].reshape(-1))
        for d in free:  # documents that no query routed to
            c["Kb"][c["off"][d]:c["off"][d + 1]] = bad
            c["Vb"][c["off"][d]:c["off"][d + 1]] = bad
        # a masked key (seen by others) may be NaN or infinite in the rows that do not see it
        c["Kd"][0, 2] = bad
        got = _run(msa, c, cuda_device)
        hide = ~c["see"][0, :30, 2]
        assert torch.equal(got[1:], clean[1:])
        assert torch.equal(got[0, :30][torch.from_numpy(hide).to(cuda_device)], clean[0, :30][torch.from_numpy(hide).to(cuda_device)])
        assert float(got[0, 30:].abs().sum()) == 0
        c["Kd"][0, 2] = 0.0
        c["see"][0, :, 2] = False
        clean = _run(msa, c, cuda_device)


def test_lengths_are_clamped_and_bad_documents_reported(msa, cuda_device):
    c = _case(13, 2, 9, 8, 2, 64, 33, [33, 40], 2, False, cuda_device)
    c["n_draft"] = np.array([11, -2], dtype=np.int32)
    _check(_run(msa, c, cuda_device), c)
    assert msa.check_device_errors() == 0
    c["top"][0, 1] = len(c["off"]) - 1
    _run(msa, c, cuda_device)
    with pytest.raises(msa.MSAError):
        msa.check_device_errors()


def test_streams_and_graphs(msa, cuda_device):
    """A captured call replayed after its lengths, mask and cache changed; another stream."""
    import torch

    c = _case(17, 2, 24, 16, 4, 64, 600, [600, 40], 3, False, cuda_device)
    dev = cuda_device
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)
    loc, n, mask = t(c["loc_len"]), t(c["n_draft"]), t(O.pack_mask(c["see"]))
    a = (c["dims"], c["q"], c["Kd"], c["Vd"], mask, c["Kl"], c["Vl"], loc)
    kw = dict(n_draft=n, K_bar=c["Kb"], V_bar=c["Vb"], chunk_off=t(c["off"]), topk_idx=t(c["top"]))
    ref = msa.tree_attend(*a, **kw)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    other = msa.tree_attend(*a, **kw, stream=st)
    st.synchronize()
    assert torch.equal(other, ref)
    with torch.cuda.stream(st):
        msa.tree_attend(*a, **kw)
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = msa.tree_attend(*a, **kw)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref)
    c["loc_len"], c["n_draft"] = np.array([5, 599], dtype=np.int32), np.array([24, 13], dtype=np.int32)
    loc.copy_(t(c["loc_len"]))
    n.copy_(t(c["n_draft"]))
    c["Kl"].mul_(-0.5)
    g.replay()
    torch.cuda.synchronize()
    _check(out, c)
    assert msa.check_device_errors() == 0


def _memory(c, rng, sizes, top, dev):
    """Documents of ``sizes`` pooled rows, ``top`` [B, k] of them for each query."""
    import torch

    bf = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(dev).to(torch.bfloat16)
    n_kv, D = c["Kd"].shape[2:]
    c["off"] = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    c["top"] = np.asarray(top, dtype=np.int32)
    c["k"] = c["top"].shape[1]
    c["Kb"], c["Vb"] = bf(int(c["off"][-1]), n_kv, D), bf(int(c["off"][-1]), n_kv, D)


@pytest.mark.parametrize("case", [  # B, M, n_q, n_kv, D, t_loc_max, k
    (33, 4, 8, 2, 64, 150, 3), (70, 3, 16, 8, 128, 40, 2), (400, 2, 4, 1, 64, 20, 1), (200, 1, 8, 8, 64, 300, 0),
    (64, 40, 8, 2, 64, 260, 0), (40, 70, 8, 4, 128, 70, 1)])
def test_tree_attend_many_queries(msa, cuda_device, case):
    """More queries than the kernel plans in shared memory; more items than SMs, cut at any place."""
    import torch

    B, M, n_q, n_kv, D, T, k = case
    loc = np.random.default_rng(B).integers(0, T + 1, size=B)
    c = _case(B, B, M, n_q, n_kv, D, T, loc, k, True, cuda_device)
    got = _run(msa, c, cuda_device)
    _check(got, c)
    assert torch.equal(got, _run(msa, c, cuda_device)) and msa.check_device_errors() == 0


@pytest.mark.parametrize("B,M,n_q,n_kv,D", [(1, 256, 16, 1, 64), (2, 255, 32, 2, 128), (1, 9, 16, 1, 128)])
def test_tree_attend_widest_groups(msa, cuda_device, B, M, n_q, n_kv, D):
    c = _case(M, B, M, n_q, n_kv, D, 200, [200, 31][:B], 2, B > 1, cuda_device)
    _check(_run(msa, c, cuda_device), c)


@pytest.mark.parametrize("B,k,D", [(1, 256, 64), (3, 255, 128), (40, 100, 64)])
def test_tree_attend_many_documents(msa, cuda_device, B, k, D):
    """Empty documents, documents of one row, of exactly a tile and longer than two; the same one twice."""
    rng = np.random.default_rng(k)
    c = _case(k, B, 3, 4, 2, D, 20, rng.integers(0, 21, size=B), 0, True, cuda_device)
    sizes = rng.choice([0, 1, 2, 3, 7, 31, 64, 65], size=300)
    sizes[[3, 50, 200]] = [128, 300, 129]
    top = np.stack([rng.permutation(300)[:k] for _ in range(B)])
    top[:, -1] = top[:, 0]
    top[:, :3] = [200, 50, 3]
    _memory(c, rng, sizes, top, cuda_device)
    _check(_run(msa, c, cuda_device), c)
    assert msa.check_device_errors() == 0


def test_nothing_drafted(msa, cuda_device):
    c = _case(23, 4, 20, 8, 2, 64, 50, [50, 0, 7, 9], 1, False, cuda_device)
    c["n_draft"][:] = 0
    assert float(_run(msa, c, cuda_device).abs().sum()) == 0 and msa.check_device_errors() == 0


@pytest.mark.parametrize("D", [64, 128])
def test_one_query_s_values_stay_its_own(msa, cuda_device, D):
    """Values that are not finite, in some queries' caches, documents and drafts: the others' rows do
    not change, although their tiles take the same places."""
    import torch

    B = 64
    rng = np.random.default_rng(D)
    loc = rng.integers(1, 300, size=B)
    c = _case(D, B, 5, 8, 8, D, 300, loc, 0, False, cuda_device)
    _memory(c, rng, rng.integers(1, 30, size=2 * B), np.arange(2 * B).reshape(B, 2), cuda_device)
    clean = _run(msa, c, cuda_device)
    bad = np.arange(0, B, 3)
    for x in (float("nan"), float("inf")):
        for b in bad:
            c["Vl"][b], c["Vd"][b] = x, x
            c["Vb"][c["off"][2 * b]:c["off"][2 * b + 2]] = x
        got = _run(msa, c, cuda_device)
        good = np.setdiff1d(np.arange(B), bad)
        assert torch.equal(got[good], clean[good])
        assert not torch.isfinite(got[bad]).any()


def test_calls_side_by_side_and_shared_workspaces(msa, cuda_device):
    """Two streams at once with workspaces of their own; two shapes back to back, and two graphs, over
    one workspace."""
    import torch

    dev = cuda_device
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)
    cs = [_case(31, 2, 24, 16, 4, 64, 900, [900, 333], 3, False, dev), _case(32, 3, 9, 8, 2, 128, 500, [1, 499, 0], 2, True, dev)]
    args = []
    for c in cs:
        kw = dict(n_draft=t(c["n_draft"]), K_bar=c["Kb"], V_bar=c["Vb"], chunk_off=t(c["off"]), topk_idx=t(c["top"]))
        args.append(((c["dims"], c["q"], c["Kd"], c["Vd"], t(O.pack_mask(c["see"])), c["Kl"], c["Vl"], t(c["loc_len"])), kw))
    ref = [msa.tree_attend(*a, **kw) for a, kw in args]
    for c, r in zip(cs, ref):
        _check(r, c)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    got = [[] for _ in cs]
    for _ in range(8):
        for i, (a, kw) in enumerate(args):
            got[i].append(msa.tree_attend(*a, **kw, stream=streams[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(g, ref[i]) for i in range(2) for g in got[i])
    size = max(msa.tree_attend_workspace_size(c["dims"], c["B"], c["M"], c["k"], c["Kl"].shape[1]) for c in cs)
    ws = torch.full((size + 256,), 0xFF, dtype=torch.uint8, device=dev)
    for i in (0, 1, 1, 0, 0, 1):
        a, kw = args[i]
        assert torch.equal(msa.tree_attend(*a, **kw, ws=ws), ref[i])
    graphs, outs = [], []
    for a, kw in args:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(msa.tree_attend(*a, **kw, ws=ws))
        graphs.append(g)
    for i in (0, 1, 0, 0, 1, 1):
        outs[i].zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], ref[i])
    assert msa.check_device_errors() == 0


def test_caches_past_2_31_elements(msa, cuda_device):
    """Appends, commits and attention at the far end of a cache of 2.5e9 elements.  Keys and values are
    zero except the last 500: a zero key has weight exp(0), so the exact result is short."""
    import torch

    dev, B, T, n_kv, D, M, tail = cuda_device, 2, 1_210_000, 8, 128, 3, 500
    gen = torch.Generator(device=dev).manual_seed(8)
    rn = lambda *s: torch.randn(*s, generator=gen, device=dev).to(torch.bfloat16)
    K, V = (torch.zeros(B, T, n_kv, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=dev)
    L = T - 10
    K[1, L - tail:L], V[1, L - tail:L] = rn(tail, n_kv, D), rn(tail, n_kv, D)
    rot = msa.rotary(D)
    q, k, v = rn(B, 8, D), rn(B, n_kv, D), rn(B, n_kv, D)
    msa.head_norm_append(rot, q, k, v, None, None, i32(5, L), i32(0, L), K, V)
    _, kr = msa.head_norm_rotate(rot, q, k, None, None, i32(5, L))
    assert torch.equal(K[1, L], kr[1]) and torch.equal(V[1, L], v[1]) and torch.equal(K[0, 0], kr[0])
    Kd, Vd = rn(B, M, n_kv, D), rn(B, M, n_kv, D)
    new = msa.tree_commit(Kd, Vd, i32(0, 2, 1, 2).view(2, 2), i32(0, 2), K, V, i32(0, L + 1))
    assert new.tolist() == [0, L + 3]
    assert torch.equal(K[1, L + 1:L + 3], Kd[1, 1:3]) and torch.equal(V[1, L + 1:L + 3], Vd[1, 1:3])
    assert float(K[1, L + 3:].abs().sum()) == 0 and float(V[1, :L - tail].abs().max()) == 0
    d = _dims(16, n_kv, D)
    see = np.zeros((B, M, M), dtype=bool)
    see[:, :, 0] = see[:, 2, 1] = True
    qq = rn(B, M, 16, D)
    got = msa.tree_attend(d, qq, Kd, Vd, torch.from_numpy(O.pack_mask(see)).to(dev), K, V, new)
    Kt, Vt = K[1, L - tail:L + 3].double(), V[1, L - tail:L + 3].double()
    for b, h, r in [(1, 0, 0), (1, 15, 1), (1, 6, 2), (0, 3, 2)]:
        js = np.nonzero(see[b, r])[0]
        Kr, Vr = (torch.cat([x[:, h // 2] if b else x[:0, 0], y[b, js][:, h // 2].double()]) for x, y in ((Kt, Kd), (Vt, Vd)))
        s = Kr @ qq[b, r, h].double() * D ** -0.5
        w = torch.exp(s - s.max())
        total = w.sum() + (L - tail if b else 0) * torch.exp(-s.max())  # the zero keys
        ref, A = w @ Vr / total, w @ Vr.abs() / total
        assert bool(((got[b, r, h].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -12) * A).all())
    assert msa.check_device_errors() == 0


# ----------------------------------------------------------------------------
# plan and commit
# ----------------------------------------------------------------------------
@pytest.mark.parametrize("B,M,ragged", [(1, 1, False), (1, 16, False), (3, 32, True), (4, 33, True), (2, 255, True), (70, 256, False)])
def test_tree_plan(msa, cuda_device, B, M, ragged):
    import torch

    rng = np.random.default_rng(B * M)
    parents, n = _trees(rng, B, M, ragged)
    if B == 2:
        parents[0] = np.arange(M) - 1  # one chain of every draft
    loc = rng.integers(0, 1 << 20, size=B).astype(np.int32)
    t = lambda a: torch.from_numpy(a).to(cuda_device)
    mask, pos = msa.tree_plan(t(parents), t(loc), 16, n_draft=t(n) if ragged else None)
    see, ref = O.tree_plan(parents, n, loc, 16)
    assert np.array_equal(mask.cpu().numpy(), O.pack_mask(see)) and np.array_equal(pos.cpu().numpy(), ref)
    assert msa.check_device_errors() == 0


def test_tree_plan_reports_bad_parents(msa, cuda_device):
    import torch

    t = lambda *a: torch.tensor(a, dtype=torch.int32, device=cuda_device)
    mask, pos = msa.tree_plan(t([-1, 0, 2, -2, 9]), t(10), 0)
    with pytest.raises(msa.MSAError):
        msa.check_device_errors()
    assert mask[0, :, 0].tolist() == [1, 3, 4, 8, 16] and pos[0].tolist() == [10, 11, 10, 10, 10]
    # parents behind the drafts in use are not read
    mask, pos = msa.tree_plan(t([-1, 0, 7, 9]), t(10), 0, n_draft=t(2))
    assert msa.check_device_errors() == 0 and mask[0, :, 0].tolist() == [1, 3, 0, 0]


@pytest.mark.parametrize("B,M,A,n_kv,D,T", [(1, 1, 1, 1, 64, 1), (1, 16, 5, 8, 128, 40), (7, 40, 9, 3, 64, 33), (90, 64, 17, 8, 128, 64)])
def test_tree_commit(msa, cuda_device, B, M, A, n_kv, D, T):
    import torch

    rng = np.random.default_rng(B + M)
    gen = torch.Generator(device=cuda_device).manual_seed(B)
    rn = lambda *s: torch.randn(*s, generator=gen, device=cuda_device).to(torch.bfloat16)
    Kd, Vd, K, V = rn(B, M, n_kv, D), rn(B, M, n_kv, D), rn(B, T, n_kv, D), rn(B, T, n_kv, D)
    path = np.sort(np.argsort(rng.random((B, M)), 1)[:, :A], 1).astype(np.int32)
    n = rng.integers(0, A + 1, size=B).astype(np.int32)
    loc = rng.integers(0, T - A + 1, size=B).astype(np.int32)
    Kr, Vr = K.clone(), V.clone()
    for b in range(B):
        for i in range(n[b]):
            Kr[b, loc[b] + i], Vr[b, loc[b] + i] = Kd[b, path[b, i]], Vd[b, path[b, i]]
    t = lambda a: torch.from_numpy(a).to(cuda_device)
    new = msa.tree_commit(Kd, Vd, t(path), t(n), K, V, t(loc))
    assert torch.equal(K, Kr) and torch.equal(V, Vr) and np.array_equal(new.cpu().numpy(), loc + n)
    assert msa.check_device_errors() == 0


def test_tree_commit_leaves_out_what_does_not_fit(msa, cuda_device):
    import torch

    t = lambda a: torch.tensor(a, dtype=torch.int32, device=cuda_device)
    Kd = torch.randn(2, 4, 1, 64, device=cuda_device).to(torch.bfloat16)
    K, V = (torch.zeros(2, 6, 1, 64, dtype=torch.bfloat16, device=cuda_device) for _ in range(2))
    new = msa.tree_commit(Kd, Kd, t([[0, 3, 3], [0, 4, 1]]), t([3, 5]), K, V, t([4, 0]))
    with pytest.raises(msa.MSAError):
        msa.check_device_errors()
    assert new.tolist() == [6, 3]
    assert torch.equal(K[0, 4], Kd[0, 0]) and torch.equal(K[0, 5], Kd[0, 3]) and float(K[0, :4].abs().sum()) == 0
    assert torch.equal(V[1, 0], Kd[1, 0]) and float(V[1, 1].abs().sum()) == 0 and torch.equal(V[1, 2], Kd[1, 1])


# ----------------------------------------------------------------------------
# together
# ----------------------------------------------------------------------------
def test_a_chain_of_drafts_equals_the_query_prefill(msa, cuda_device):
    """A tree that is one chain attends as sparse_attend's M query tokens do (which rotates its own
    queries): both within the attention's tolerance of each other."""
    import torch

    rng = np.random.default_rng(3)
    d = W.Dims(hidden=256, n_q=8, n_kv=2, head_dim=64, n_r=4, d_r=64)
    B, M, L, T, off = 2, 6, 50, 64, 5
    dev = cuda_device
    bf = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(dev).to(torch.bfloat16)
    sizes = rng.integers(1, 20, size=12)
    co = torch.from_numpy(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)).to(dev)
    Kb, Vb = bf(int(sizes.sum()), 2, 64), bf(int(sizes.sum()), 2, 64)
    idx = torch.tensor([[0, 3, 5], [11, 2, 7]], dtype=torch.int32, device=dev)
    rot = msa.rotary(64, base=d.rope_base)
    K, V, q = bf(B, T, 2, 64), bf(B, T, 2, 64), bf(B, M, 8, 64)
    Kr = msa.rotate(rot, K.view(B * T, 2, 64), (torch.arange(T, device=dev, dtype=torch.int32) + off).repeat(B)).view(K.shape)
    ll = torch.full((B,), L + M, dtype=torch.int32, device=dev)
    ref = msa.sparse_attend(d, q, Kb, Vb, co, idx, Kr, V, ll, off, k_loc_rotated=True)
    parents = (torch.arange(M, dtype=torch.int32, device=dev) - 1).repeat(B, 1)
    loc = torch.full((B,), L, dtype=torch.int32, device=dev)
    mask, pos = msa.tree_plan(parents, loc, off)
    qr = msa.rotate(rot, q.view(B * M, 8, 64), pos.view(-1)).view(q.shape)
    Kd, Vd = Kr[:, L:L + M].contiguous(), V[:, L:L + M].contiguous()
    got = msa.tree_attend(d, qr, Kd, Vd, mask, Kr, V, loc, K_bar=Kb, V_bar=Vb, chunk_off=co, topk_idx=idx)
    assert float((got.float() - ref.float()).abs().max()) < 2e-2  # the existing call's own tolerance
    # and committing the chain gives the cache that the prefill attended over
    K2, V2 = Kr.clone(), V.clone()
    K2[:, L:], V2[:, L:] = 0, 0
    path = torch.arange(M, dtype=torch.int32, device=dev).repeat(B, 1)
    new = msa.tree_commit(Kd, Vd, path, torch.full((B,), M, dtype=torch.int32, device=dev), K2, V2, loc)
    assert torch.equal(new, ll) and torch.equal(K2[:, :L + M], Kr[:, :L + M]) and torch.equal(V2[:, :L + M], V[:, :L + M])


def test_a_whole_step(msa, cuda_device):
    """Plan, norms and rotation, attention, commit, then the next decode token through
    head_norm_append: against the oracle's composition of the same steps."""
    import torch

    rng = np.random.default_rng(21)
    d = W.Dims(hidden=256, n_q=8, n_kv=2, head_dim=64, n_r=4, d_r=64)
    B, M, T, off = 2, 11, 90, 3
    dev = cuda_device
    bf = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(dev).to(torch.bfloat16)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)
    parents, n = _trees(rng, B, M, True)
    loc = np.array([70, 12], dtype=np.int32)
    K, V = bf(B, T, 2, 64), bf(B, T, 2, 64)
    fused = bf(B * M, 12, 64)  # one projection's output: 8 query, 2 key, 2 value heads
    wq, wk = bf(64), bf(64)
    rot = msa.rotary(64, 32, layout="interleaved", scaling="parts", factor=8.0, orig_len=64, low=1.0, high=4.0)
    theta = O.rotary_theta(32, 1e6, "parts", 8.0, 64, 1.0, 4.0)
    mask, pos = msa.tree_plan(t(parents), t(loc), off, n_draft=t(n))
    q, Kd = msa.head_norm_rotate(rot, fused[:, :8], fused[:, 8:10], wq, wk, pos.view(-1))
    Vd = fused[:, 10:].contiguous()
    q, Kd, Vd = q.view(B, M, 8, 64), Kd.view(B, M, 2, 64), Vd.view(B, M, 2, 64)
    out = msa.tree_attend(d, q, Kd, Vd, mask, K, V, t(loc), n_draft=t(n))
    see, opos = O.tree_plan(parents, n, loc, off)
    c = dict(q=q, Kd=Kd, Vd=Vd, Kl=K, Vl=V, see=see, n_draft=n, loc_len=loc, M=M, k=0)
    _check(out, c)
    oq = O.rotate_heads(O.head_norm(_f64(fused[:, :8]), _f64(wq)), opos.reshape(-1), theta, "interleaved")
    assert np.max(np.abs(_f64(q).reshape(oq.shape) - oq) / (np.abs(oq) + 1e-3)) < 2.0 ** -8 * 1.01
    # the deepest path of each query is accepted
    path, n_path = np.zeros((B, M), dtype=np.int32), np.zeros(B, dtype=np.int32)
    for b in range(B):
        if n[b]:
            leaf = int(np.argmax(see[b, :n[b]].sum(1)))
            ids = np.nonzero(see[b, leaf])[0]
            path[b, :len(ids)], n_path[b] = ids, len(ids)
    before = K.clone()
    new = msa.tree_commit(Kd, Vd, t(path), t(n_path), K, V, t(loc))
    for b in range(B):
        assert torch.equal(K[b, :loc[b]], before[b, :loc[b]])
        for i in range(n_path[b]):
            assert torch.equal(K[b, loc[b] + i], Kd[b, path[b, i]]) and torch.equal(V[b, loc[b] + i], Vd[b, path[b, i]])
            assert opos[b, path[b, i]] == off + loc[b] + i  # rotated for the slot it now has
    # one more token, decoded over the committed cache: a tree of one draft and head_norm_append agree
    tok = bf(B, 12, 64)
    slot = new.clone()
    K3, V3 = K.clone(), V.clone()
    q1 = msa.head_norm_append(rot, tok[:, :8], tok[:, 8:10], tok[:, 10:], wq, wk, slot + off, slot, K3, V3)
    m1, p1 = msa.tree_plan(torch.full((B, 1), -1, dtype=torch.int32, device=dev), new, off)
    q2, k2 = msa.head_norm_rotate(rot, tok[:, :8], tok[:, 8:10], wq, wk, p1.view(-1))
    assert torch.equal(q1, q2) and all(torch.equal(K3[b, int(slot[b])], k2[b]) for b in range(B))
    o1 = msa.tree_attend(d, q1.view(B, 1, 8, 64), K3[:, :1].contiguous(), V3[:, :1].contiguous(), torch.zeros_like(m1), K3, V3, new + 1)
    o2 = msa.tree_attend(d, q2.view(B, 1, 8, 64), k2.view(B, 1, 2, 64), tok[:, 10:].contiguous().view(B, 1, 2, 64), m1, K, V, new)
    assert float((o1.float() - o2.float()).abs().max()) < 2.0 ** -6 and msa.check_device_errors() == 0
