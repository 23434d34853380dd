"""Operators of the active context, as cases to be measured: the position rotation of queries and
keys, their per-head norms with the rotation in the same pass, and a decode step over a tree of
drafted tokens (its plan, its attention over routed documents, local cache and drafts, and the
append of the accepted drafts to the cache).

``run`` computes a case in plain torch operations, or, with ``own`` set, through this
framework's entry points; ``exact`` computes it from the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEVICE = "cuda"


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def _rotary(head_dim, rot_dim, layout, scaling):
    return {"head_dim": head_dim, "rot_dim": rot_dim, "layout": layout, "scaling": scaling}


def _rotate(rows, n_q, n_kv, rot, dtype, grad, sliced):
    return dict(op="rotate", rows=rows, n_q=n_q, n_kv=n_kv, dtype=dtype, grad=grad, sliced=sliced, **rot)


def _head_norm(form, rows, n_q, n_kv, rot, dtype, sliced=False, batch=1, t_loc=0):
    return dict(op="head_norm", form=form, rows=rows, n_q=n_q, n_kv=n_kv, dtype=dtype, sliced=sliced, batch=batch,
                t_loc=t_loc, **rot)


def _tree_attend(batch, drafts, n_q, n_kv, head_dim, t_loc, k, ragged):
    return dict(op="tree_attend", batch=batch, drafts=drafts, n_q=n_q, n_kv=n_kv, head_dim=head_dim, t_loc=t_loc, k=k,
                ragged=ragged)


def listed():
    half128 = _rotary(128, 128, "half", "none")
    return [
        # the query and key heads of one decoded token of a 1M-token session (32 query, 8 key heads of
        # 128), positions scaled past the trained context: the smallest call of all, latency only
        dict(_rotate(1, 32, 8, _rotary(128, 128, "half", "yarn"), "bf16", False, False), name="rotate_decode"),
        # a training step's gradients through an interleaved rotation of half of each head, in 32 bits,
        # an odd number of tokens, read from slices of a fused projection
        dict(_rotate(8193, 32, 8, _rotary(128, 64, "interleaved", "parts"), "fp32", True, True),
             name="rotate_backward"),
        # a decode step of 16 queries: norms, rotation, and the new keys and values into their cache slots
        dict(_head_norm("append", 16, 32, 8, half128, "bf16", batch=16, t_loc=4096), name="head_norm_append_decode"),
        # a long prompt's queries and keys, read from slices of the fused projection
        dict(_head_norm("forward", 16384, 32, 8, half128, "bf16", sliced=True), name="head_norm_prefill"),
        # the backward pass of the same norms in a training step, fp16, odd length, two thirds of the
        # head rotated
        dict(_head_norm("backward", 8191, 32, 8, _rotary(96, 64, "half", "none"), "fp16"), name="head_norm_backward"),
        # one query's 16 drafts over the 1M-token memory's routed documents and a 4K local cache
        dict(_tree_attend(1, 16, 32, 8, 128, 4096, 16, False), name="tree_attend_1m"),
        # 32 queries, 32 drafts each, over 16 routed documents and 8K local tokens: the largest call
        dict(_tree_attend(32, 32, 32, 8, 128, 8192, 16, False), name="tree_attend_16m"),
        # wide trees, smaller heads, no routed documents, every query another length and draft count
        dict(_tree_attend(7, 127, 16, 4, 64, 20000, 0, True), name="tree_attend_ragged"),
        # the plan of one small tree, and of a batch of wide ones: masks and positions from parents
        dict(op="tree_plan", batch=1, drafts=16, ragged=False, name="tree_plan_one"),
        dict(op="tree_plan", batch=32, drafts=127, ragged=True, name="tree_plan_batch"),
        # the accepted drafts of one query, and of a batch, into their local caches
        dict(op="tree_commit", batch=1, drafts=16, depth=5, n_kv=8, head_dim=128, t_loc=512, name="tree_commit_one"),
        dict(op="tree_commit", batch=64, drafts=64, depth=17, n_kv=8, head_dim=128, t_loc=1024,
             name="tree_commit_batch"),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotate", "head_norm", "head_norm", "tree_attend", "tree_attend", "tree_plan", "tree_commit"])
    if op in ("rotate", "head_norm"):
        head_dim = rng.choice([64, 72, 80, 96, 128, 128, 192, 256])
        rot_dim = rng.choice([head_dim, head_dim, head_dim // 2, 2 * (head_dim // 6)])
        rot = _rotary(head_dim, rot_dim, rng.choice(["half", "interleaved"]),
                      rng.choice(["none", "linear", "ntk", "parts", "yarn"]))
        n_q, n_kv = rng.choice([(32, 8), (8, 2), (16, 4), (12, 12), (7, 1), (24, 3)])
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        cap = (16384 * 40 * 128) // ((n_q + n_kv) * head_dim) // (2 if dtype == "fp32" else 1)
        rows = _log_uniform(rng, 1, cap)
        sliced = rng.random() < 0.5
        if op == "rotate":
            return _rotate(rows, n_q, n_kv, rot, dtype, rng.random() < 0.5, sliced)
        form = rng.choice(["forward", "append", "backward"])
        if form == "append":
            batch = _log_uniform(rng, 1, 64)
            per = _log_uniform(rng, 1, 64)
            return _head_norm(form, batch * per, n_q, n_kv, rot, dtype, sliced, batch, per + rng.randrange(1, 500))
        return _head_norm(form, rows, n_q, n_kv, rot, dtype, sliced)
    if op == "tree_attend":
        n_q, n_kv, head_dim = rng.choice([(32, 8, 128), (8, 2, 64), (16, 4, 64), (16, 1, 128), (8, 8, 64), (20, 4, 128)])
        drafts = _log_uniform(rng, 1, 200)
        t_loc = _log_uniform(rng, 1, 32768)
        k = rng.choice([0, 1, 5, 16])
        keys = t_loc + drafts + 40 * k
        budget = min(32 * 32 * 32 * 128 * 8900 // (drafts * n_q * head_dim * keys),
                     32 * 8 * 128 * 8900 // (n_kv * head_dim * keys))
        return _tree_attend(_log_uniform(rng, 1, max(1, min(48, budget))), drafts, n_q, n_kv, head_dim, t_loc, k,
                            rng.random() < 0.6)
    if op == "tree_plan":
        return dict(op="tree_plan", batch=_log_uniform(rng, 1, 128), drafts=_log_uniform(rng, 1, 256),
                    ragged=rng.random() < 0.5)
    drafts = _log_uniform(rng, 1, 200)
    return dict(op="tree_commit", batch=_log_uniform(rng, 1, 64), drafts=drafts, depth=rng.randrange(1, min(drafts, 40) + 1),
                n_kv=rng.choice([1, 2, 4, 8]), head_dim=rng.choice([64, 128]), t_loc=rng.randrange(64, 1025))


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
SCALING = {  # base, factor, orig_len, low, high, magnitude of each kind of frequency scaling
    "none": (1.0e6, 1.0, 0, 0.0, 0.0, 1.0),
    "linear": (1.0e6, 8.0, 0, 0.0, 0.0, 1.0),
    "ntk": (1.0e6, 4.0, 0, 0.0, 0.0, 1.0),
    "parts": (5.0e5, 8.0, 8192, 1.0, 4.0, 1.0),
    "yarn": (1.0e6, 4.0, 32768, 1.0, 32.0, 0.1 * math.log(4.0) + 1.0),
}


def _randn(g, shape, dtype, scale=1.0, shift=0.0):
    return (torch.randn(shape, generator=g, device=DEVICE, dtype=torch.float32) * scale + shift).to(dtype)


def _qkv(case, g, with_v):
    """Query, key (and value) heads [rows, heads, head_dim]: tensors of their own, or slices of the
    output [rows, all heads x head_dim] of one fused projection."""
    rows, n_q, n_kv, d = case["rows"], case["n_q"], case["n_kv"], case["head_dim"]
    dtype = DTYPES[case["dtype"]]
    if case["sliced"]:
        x = _randn(g, (rows, n_q + 2 * n_kv, d), dtype)
        parts = x[:, :n_q], x[:, n_q:n_q + n_kv], x[:, n_q + n_kv:]
    else:
        parts = tuple(_randn(g, (rows, h, d), dtype) for h in (n_q, n_kv, n_kv))
    return parts if with_v else parts[:2]


def _trees(rng, batch, drafts, ragged):
    """Parents of each query's drafted tokens (earlier drafts, -1: the committed context) and the
    drafts in use."""
    parents = np.full((batch, drafts), -1, dtype=np.int32)
    for t in range(1, drafts):
        lo = max(0, t - 8)
        parents[:, t] = rng.integers(lo, t, size=batch)
        parents[rng.random(batch) < 0.03, t] = -1
    n = np.full(batch, drafts, dtype=np.int32)
    if ragged:
        n = rng.integers(0, drafts + 1, size=batch).astype(np.int32)
        n[rng.integers(0, batch)] = drafts
    return parents, n


def _tree_masks(parents, n):
    """[batch, drafts, words] int32: bit j of row t set where draft j is t itself or an ancestor."""
    batch, drafts = parents.shape
    words = (drafts + 31) // 32
    see = np.zeros((batch, drafts, 32 * words), dtype=bool)
    for t in range(drafts):
        p = parents[:, t]
        has = p >= 0
        see[has, t] = see[has, p[has]]
        see[:, t, t] = True
    live = np.arange(drafts)[None] < n[:, None]
    see &= live[:, :, None]
    return np.packbits(see, axis=2, bitorder="little").view(np.uint32).view(np.int32).reshape(batch, drafts, words)


def _dims(case):
    import long_context_memory_b200.workloads as W

    return W.Dims(hidden=2560, n_q=case["n_q"], n_kv=case["n_kv"], head_dim=case["head_dim"], n_r=8, d_r=128)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    rng = np.random.default_rng(seed)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEVICE)
    st = {"case": case}
    op = case["op"]
    if op in ("rotate", "head_norm"):
        rows, d = case["rows"], case["head_dim"]
        dtype = DTYPES[case["dtype"]]
        form = case.get("form")
        if form == "append":
            st["q"], st["k"], st["v"] = _qkv(case, g, True)
        else:
            st["q"], st["k"] = _qkv(case, g, False)
        start = int(rng.integers(0, 900_000))  # a place in a long session
        st["positions"] = dev((start + np.arange(rows)).astype(np.int32))
        if op == "head_norm":
            st["w_q"] = _randn(g, (d,), dtype, 0.2, 1.0)
            st["w_k"] = _randn(g, (d,), dtype, 0.2, 1.0)
            if form == "backward":
                st["dq"] = _randn(g, (rows, case["n_q"], d), dtype)
                st["dk"] = _randn(g, (rows, case["n_kv"], d), dtype)
            if form == "append":
                B, T = case["batch"], case["t_loc"]
                M = rows // B
                first = rng.integers(0, T - M + 1, size=B)
                slots = (first[:, None] + np.arange(M)[None]).astype(np.int32)
                st["slots"] = dev(slots.reshape(-1))
                st["positions"] = dev((start + slots).reshape(-1).astype(np.int32))
                st["K_loc"] = _randn(g, (B, T, case["n_kv"], d), dtype)
                st["V_loc"] = _randn(g, (B, T, case["n_kv"], d), dtype)
        if own:
            import long_context_memory_b200 as msa

            base, factor, orig, low, high, mag = SCALING[case["scaling"]]
            st["rot"] = msa.rotary(d, case["rot_dim"], layout=case["layout"], base=base, scaling=case["scaling"],
                                   factor=factor, orig_len=orig, low=low, high=high, magnitude=mag)
            # buffers that a program keeps from one step to the next
            st["out"] = torch.empty((rows, case["n_q"], d), dtype=dtype, device=DEVICE)
            if form != "append":
                st["k_out"] = torch.empty((rows, case["n_kv"], d), dtype=dtype, device=DEVICE)
            if form == "backward":
                st["dw"] = torch.empty((2, d), dtype=torch.float32, device=DEVICE)
                nbytes = msa.head_norm_grad_workspace_size(st["rot"], rows, case["n_q"], case["n_kv"])
                st["ws"] = torch.empty(nbytes + 256, dtype=torch.uint8, device=DEVICE)
        return st
    B, M = case["batch"], case["drafts"]
    parents, n = _trees(rng, B, M, case.get("ragged", False))
    if op == "tree_plan":
        st["parents"], st["n_draft"] = dev(parents), dev(n)
        st["loc_len"] = dev(rng.integers(0, 100_000, size=B).astype(np.int32))
        if own:
            st["out"] = (torch.empty((B, M, (M + 31) // 32), dtype=torch.int32, device=DEVICE),
                         torch.empty((B, M), dtype=torch.int32, device=DEVICE))
        return st
    d, n_kv, T = case["head_dim"], case["n_kv"], case["t_loc"]
    bf = torch.bfloat16
    if op == "tree_commit":
        A = case["depth"]
        st["K_draft"], st["V_draft"] = _randn(g, (B, M, n_kv, d), bf), _randn(g, (B, M, n_kv, d), bf)
        st["K_loc"], st["V_loc"] = _randn(g, (B, T, n_kv, d), bf), _randn(g, (B, T, n_kv, d), bf)
        path = np.sort(np.argsort(rng.random((B, M)), axis=1)[:, :A], axis=1).astype(np.int32)
        st["path"] = dev(path)
        st["n_path"] = dev(rng.integers(1, A + 1, size=B).astype(np.int32))
        st["loc_len"] = dev(rng.integers(0, T - A + 1, size=B).astype(np.int32))
        if own:
            st["new_len"] = torch.empty_like(st["loc_len"])
        return st
    loc = np.full(B, T, dtype=np.int32)
    if case["ragged"]:
        loc = rng.integers(0, T + 1, size=B).astype(np.int32)
        loc[rng.integers(0, B)] = T
    st["q"] = _randn(g, (B, M, case["n_q"], d), bf)
    st["K_draft"], st["V_draft"] = _randn(g, (B, M, n_kv, d), bf), _randn(g, (B, M, n_kv, d), bf)
    st["K_loc"], st["V_loc"] = _randn(g, (B, T, n_kv, d), bf), _randn(g, (B, T, n_kv, d), bf)
    st["loc_len"], st["n_draft"] = dev(loc), dev(n)
    st["mask"] = dev(_tree_masks(parents, n))
    k = case["k"]
    if k:  # a memory of documents of about 32 pooled chunks, and each query's routed ones
        n_docs = max(64, 8 * k)
        chunks = np.maximum(1, np.round(rng.lognormal(math.log(32), 0.5, size=n_docs))).astype(np.int64)
        off = np.zeros(n_docs + 1, dtype=np.int32)
        off[1:] = np.cumsum(chunks)
        top = np.stack([rng.permutation(n_docs)[:k] for _ in range(B)]).astype(np.int32)
        C = int(off[-1])
        st["K_bar"], st["V_bar"] = _randn(g, (C, n_kv, d), bf), _randn(g, (C, n_kv, d), bf)
        st["chunk_off"], st["topk_idx"] = dev(off), dev(top)
        st["sel_max"] = int(chunks[top].sum(axis=1).max())
    if own:
        import long_context_memory_b200 as msa

        st["dims"] = _dims(case)
        nbytes = msa.tree_attend_workspace_size(st["dims"], B, M, k, T)
        st["ws"] = torch.empty(nbytes + 256, dtype=torch.uint8, device=DEVICE)
        st["out"] = torch.empty_like(st["q"])
    return st


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(st):
    import long_context_memory_b200 as msa

    case = st["case"]
    op = case["op"]
    if op == "rotate":
        return msa.rotate(st["rot"], st["q"], st["positions"], k=st["k"], grad=case["grad"], out=st["out"],
                          k_out=st["k_out"])
    if op == "head_norm":
        a = (st["rot"], st["q"], st["k"])
        if case["form"] == "forward":
            return msa.head_norm_rotate(*a, st["w_q"], st["w_k"], st["positions"], out=st["out"], k_out=st["k_out"])
        if case["form"] == "backward":
            return msa.head_norm_rotate_grad(*a, st["w_q"], st["w_k"], st["positions"], st["dq"], st["dk"],
                                             out=(st["out"], st["k_out"], st["dw"][0], st["dw"][1]), ws=st["ws"])
        q = msa.head_norm_append(*a, st["v"], st["w_q"], st["w_k"], st["positions"], st["slots"], st["K_loc"],
                                 st["V_loc"], out=st["out"])
        return q, st["K_loc"], st["V_loc"]
    if op == "tree_plan":
        return msa.tree_plan(st["parents"], st["loc_len"], 16, n_draft=st["n_draft"], out=st["out"])
    if op == "tree_commit":
        new_len = msa.tree_commit(st["K_draft"], st["V_draft"], st["path"], st["n_path"], st["K_loc"], st["V_loc"],
                                  st["loc_len"], out=st["new_len"])
        return st["K_loc"], st["V_loc"], new_len
    return msa.tree_attend(st["dims"], st["q"], st["K_draft"], st["V_draft"], st["mask"], st["K_loc"], st["V_loc"],
                           st["loc_len"], n_draft=st["n_draft"], K_bar=st.get("K_bar"), V_bar=st.get("V_bar"),
                           chunk_off=st.get("chunk_off"), topk_idx=st.get("topk_idx"), out=st["out"], ws=st["ws"])


def _theta_plain(case):
    """Radians per position of each rotated pair, and the magnitude of cosine and sine."""
    base, s, orig, low, high, mag = SCALING[case["scaling"]]
    r = case["rot_dim"]
    i = torch.arange(r // 2, dtype=torch.float64, device=DEVICE)
    kind = case["scaling"]
    if kind == "ntk":
        base = base * s ** (r / (r - 2)) if r > 2 else base
    theta = torch.exp(i * (-2.0 * math.log(base) / r))
    if kind == "linear":
        theta = theta / s
    elif kind == "parts":
        keep = ((theta * (orig / (2 * math.pi)) - low) / (high - low)).clamp(0, 1)
        theta = theta * (keep + (1 - keep) / s)
    elif kind == "yarn":
        at = lambda turns: r * math.log(orig / (2 * math.pi * turns)) / (2 * math.log(base))
        first, last = max(math.floor(at(high)), 0), min(math.ceil(at(low)), r - 1)
        ramp = ((i - first) / (last - first if last > first else 0.001)).clamp(0, 1)
        theta = theta * (1 - ramp + ramp / s)
    return theta, mag


def _cos_sin_plain(case, positions):
    theta, mag = _theta_plain(case)
    ang = positions.double()[:, None] * theta[None]
    return (ang.cos() * mag).float()[:, None], (ang.sin() * mag).float()[:, None]


def _turn(case, x, cos, sin, grad=False):
    """Rotate the first rot_dim dims of each head of x (32 bits); grad: the transposed rotation."""
    r = case["rot_dim"]
    if grad:
        sin = -sin
    y = x.clone()
    if case["layout"] == "half":
        a, b = x[..., : r // 2], x[..., r // 2: r]
        y[..., : r // 2], y[..., r // 2: r] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = a * cos - b * sin, b * cos + a * sin
    return y


EPS = 1e-6


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "rotate":
        cos, sin = _cos_sin_plain(case, st["positions"])
        return tuple(_turn(case, x.float(), cos, sin, case["grad"]).to(x.dtype) for x in (st["q"], st["k"]))
    if op == "head_norm":
        cos, sin = _cos_sin_plain(case, st["positions"])
        if case["form"] == "backward":
            outs, dws = [], []
            for x, w, g in ((st["q"], st["w_q"], st["dq"]), (st["k"], st["w_k"], st["dk"])):
                xf = x.float()
                inv = torch.rsqrt((xf * xf).mean(-1, keepdim=True) + EPS)
                n = xf * inv
                z = _turn(case, g.float(), cos, sin, grad=True)
                u = z * w.float()
                outs.append(((u - n * (u * n).mean(-1, keepdim=True)) * inv).to(x.dtype))
                dws.append((z * n).double().sum((0, 1)).float())
            return outs[0], outs[1], dws[0], dws[1]

        def norm(x, w):
            xf = x.float()
            n = xf * torch.rsqrt((xf * xf).mean(-1, keepdim=True) + EPS) * w.float()
            return _turn(case, n, cos, sin).to(x.dtype)

        q, k = norm(st["q"], st["w_q"]), norm(st["k"], st["w_k"])
        if case["form"] == "forward":
            return q, k
        B = case["batch"]
        b = torch.arange(B, device=DEVICE).repeat_interleave(case["rows"] // B)
        slots = st["slots"].long()
        st["K_loc"][b, slots] = k
        st["V_loc"][b, slots] = st["v"]
        return q, st["K_loc"], st["V_loc"]
    if op == "tree_plan":
        return _plan_plain(st)
    if op == "tree_commit":
        B, A = st["path"].shape
        i = torch.arange(A, device=DEVICE)
        b = torch.arange(B, device=DEVICE)[:, None]
        slots = st["loc_len"].long()[:, None] + i[None]
        take = (i[None] < st["n_path"][:, None])[..., None, None]
        path = st["path"].long()
        for cache, draft in ((st["K_loc"], st["K_draft"]), (st["V_loc"], st["V_draft"])):
            cache[b, slots] = torch.where(take, draft[b, path], cache[b, slots])
        return st["K_loc"], st["V_loc"], st["loc_len"] + st["n_path"]
    return _tree_attend_plain(st)


def _plan_plain(st):
    parents, n = st["parents"].long(), st["n_draft"].long()
    B, M = parents.shape
    t = torch.arange(M, device=DEVICE)
    see = torch.eye(M, device=DEVICE).repeat(B, 1, 1)
    step = see + (parents[:, :, None] == t[None, None]).float()
    reach = 1
    see = step
    while reach < M:  # paths of up to twice the length at each product
        see = (see @ see).clamp(max=1.0)
        reach *= 2
    live = t[None] < n[:, None]
    see = see * live[:, :, None]
    depth = (see.sum(-1) - 1).clamp(min=0).long()
    words = (M + 31) // 32
    bits = torch.zeros((B, M, words * 32), dtype=torch.int64, device=DEVICE)
    bits[..., :M] = see.long()
    packed = (bits.view(B, M, words, 32) << torch.arange(32, device=DEVICE)).sum(-1)
    packed = torch.where(packed >= 2 ** 31, packed - 2 ** 32, packed).int()
    return packed, (st["loc_len"].long()[:, None] + 16 + depth).int()


def _tree_attend_plain(st):
    q, K_loc, mask = st["q"], st["K_loc"], st["mask"]
    B, M, n_q, d = q.shape
    T, n_kv = K_loc.shape[1], K_loc.shape[2]
    G = n_q // n_kv
    t, j = torch.arange(T, device=DEVICE), torch.arange(M, device=DEVICE)
    live = j[None] < st["n_draft"][:, None]
    see_loc = (t[None] < st["loc_len"][:, None])[:, None].expand(B, M, T)
    see_draft = ((mask[:, :, j // 32] >> (j % 32)) & 1).bool() & live[:, None, :]
    K, V, see = [K_loc, st["K_draft"]], [st["V_loc"], st["V_draft"]], [see_loc, see_draft]
    if "K_bar" in st:  # the routed documents' pooled rows, padded to the longest selection
        off, top = st["chunk_off"].long(), st["topk_idx"].long()
        size = off[top + 1] - off[top]
        end = size.cumsum(1)
        s = torch.arange(st["sel_max"], device=DEVICE).expand(B, -1).contiguous()
        doc = torch.searchsorted(end, s, right=True).clamp(max=top.shape[1] - 1)
        row = off[top].gather(1, doc) + s - (end - size).gather(1, doc)
        in_sel = s < end[:, -1:]
        row = torch.where(in_sel, row, torch.zeros_like(row))
        K, V = [st["K_bar"][row]] + K, [st["V_bar"][row]] + V
        see = [in_sel[:, None].expand(B, M, -1)] + see
    K = torch.cat([x.float() for x in K], 1).permute(0, 2, 3, 1)  # [B, n_kv, d, keys]
    V = torch.cat([x.float() for x in V], 1).permute(0, 2, 1, 3)
    see = (torch.cat(see, 2) & live[:, :, None])[:, None, :, None]  # [B, 1, M, 1, keys]
    qf = q.float().view(B, M, n_kv, G, d).permute(0, 2, 1, 3, 4).reshape(B, n_kv, M * G, d)
    s = (qf @ K).mul_(d ** -0.5).view(B, n_kv, M, G, -1).masked_fill_(~see, -math.inf)
    top_s = s.amax(-1, keepdim=True)
    p = torch.exp_(s.sub_(torch.where(top_s == -math.inf, torch.zeros_like(top_s), top_s)))
    total = p.sum(-1)
    o = (p.view(B, n_kv, M * G, -1) @ V).view(B, n_kv, M, G, d)
    o = torch.where(total[..., None] > 0, o / total[..., None], torch.zeros_like(o))
    return o.permute(0, 2, 1, 3, 4).reshape(B, M, n_q, d).to(q.dtype)


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op in ("rotate", "head_norm"):
        size = 4 if case["dtype"] == "fp32" else 2
        rows, n_q, n_kv, d = case["rows"], case["n_q"], case["n_kv"], case["head_dim"]
        heads = rows * (n_q + n_kv)
        tensors = 2
        extra = rows * 4
        ops = 6 * (case["rot_dim"] // 2)
        if op == "head_norm":
            ops += 4 * d
            extra += 2 * d * size
            if case["form"] == "backward":
                tensors, ops, extra = 3, ops + 8 * d, extra + 2 * d * 4
            if case["form"] == "append":
                extra += rows * 4 + 2 * rows * n_kv * d * size
        return {"bytes": tensors * heads * d * size + extra, "flops": heads * ops}
    B, M = case["batch"], case["drafts"]
    if op == "tree_plan":
        words = (M + 31) // 32
        return {"bytes": B * (4 * M + 8 + 4 * M * words + 4 * M), "flops": B * M}
    d, n_kv = case["head_dim"], case["n_kv"]
    if op == "tree_commit":
        rows = B * (case["depth"] + 1) / 2  # the mean of the accepted counts
        return {"bytes": int(rows * n_kv * d * 2 * 4 + B * (4 * case["depth"] + 12)), "flops": 0}
    loc = case["t_loc"] * (0.5 if case["ragged"] else 1.0)  # the means of ragged lengths
    rows = M * (0.5 if case["ragged"] else 1.0)
    keys = loc + rows + 36 * case["k"]
    return {"bytes": int(B * keys * n_kv * d * 4 + 2 * B * M * case["n_q"] * d * 2),
            "flops": int(4 * B * rows * case["n_q"] * d * keys)}


# ----------------------------------------------------------------------------
# the definition in 64 bits
# ----------------------------------------------------------------------------
def _angles_exact(case, positions):
    base, s, orig, low, high, mag = SCALING[case["scaling"]]
    r, kind = case["rot_dim"], case["scaling"]
    theta = []
    for i in range(r // 2):
        if kind == "ntk" and r > 2:
            th = (base * s ** (r / (r - 2.0))) ** (-2.0 * i / r)
        else:
            th = base ** (-2.0 * i / r)
        if kind == "linear":
            th /= s
        if kind == "parts":  # slow pairs stretched, fast ones kept, a ramp in turns between
            turns = orig * th / (2 * math.pi)
            g = min(1.0, max(0.0, (turns - low) / (high - low)))
            th = (1 - g) * th / s + g * th
        if kind == "yarn":  # the ramp runs over the pair's index
            lo = max(math.floor(r * math.log(orig / (high * 2 * math.pi)) / (2 * math.log(base))), 0)
            hi = min(math.ceil(r * math.log(orig / (low * 2 * math.pi)) / (2 * math.log(base))), r - 1)
            g = min(1.0, max(0.0, (i - lo) / (hi - lo if hi > lo else 0.001)))
            th = g * th / s + (1 - g) * th
        theta.append(th)
    return torch.outer(positions.double(), torch.tensor(theta, dtype=torch.float64, device=positions.device)), mag


def _rotated_exact(case, x, ang, mag, sign=1.0):
    """Pairs as complex numbers, turned by exp(i angle)."""
    r = case["rot_dim"]
    head, rest = x[..., :r], x[..., r:]
    if case["layout"] == "half":
        pairs = torch.stack((head[..., : r // 2], head[..., r // 2:]), -1)
    else:
        pairs = head.reshape(*head.shape[:-1], r // 2, 2)
    z = torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.full_like(ang, mag), sign * ang)[:, None]
    pairs = torch.view_as_real(z)
    head = torch.cat((pairs[..., 0], pairs[..., 1]), -1) if case["layout"] == "half" else pairs.reshape(head.shape)
    return torch.cat((head, rest), -1)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "rotate":
        ang, mag = _angles_exact(case, st["positions"])
        return tuple(_rotated_exact(case, x.double(), ang, mag, -1.0 if case["grad"] else 1.0)
                     for x in (st["q"], st["k"]))
    if op == "head_norm":
        ang, mag = _angles_exact(case, st["positions"])
        d = case["head_dim"]
        if case["form"] == "backward":
            dx, dw = [], []
            for x, w, g in ((st["q"], st["w_q"], st["dq"]), (st["k"], st["w_k"], st["dk"])):
                x, w = x.double(), w.double()
                rms = (x.square().sum(-1, keepdim=True) / d + EPS).sqrt()
                z = _rotated_exact(case, g.double(), ang, mag, -1.0)
                dw.append((z * x / rms).sum((0, 1)))
                dx.append(z * w / rms - x * (z * w * x).sum(-1, keepdim=True) / (d * rms ** 3))
            return dx[0], dx[1], dw[0], dw[1]

        def norm(x, w):
            x = x.double()
            return _rotated_exact(case, x / (x.square().sum(-1, keepdim=True) / d + EPS).sqrt() * w.double(), ang, mag)

        q, k = norm(st["q"], st["w_q"]), norm(st["k"], st["w_k"])
        if case["form"] == "forward":
            return q, k
        K, V = st["K_loc"].double(), st["V_loc"].double()
        M = case["rows"] // case["batch"]
        for r, slot in enumerate(st["slots"].tolist()):
            K[r // M, slot] = k[r]
            V[r // M, slot] = st["v"][r].double()
        return q, K, V
    if op == "tree_plan":
        parents, n, loc = (st[x].cpu().numpy() for x in ("parents", "n_draft", "loc_len"))
        pos = np.zeros(parents.shape, dtype=np.int32)
        for b in range(parents.shape[0]):
            for t in range(parents.shape[1]):
                p, depth = int(parents[b, t]), 0
                while p >= 0 and t < n[b]:
                    p, depth = int(parents[b, p]), depth + 1
                pos[b, t] = loc[b] + 16 + depth
        dev = st["parents"].device
        return torch.from_numpy(_tree_masks(parents, n)).to(dev), torch.from_numpy(pos).to(dev)
    if op == "tree_commit":
        K, V = st["K_loc"].double(), st["V_loc"].double()
        new = st["loc_len"].clone()
        path, n, loc = st["path"].tolist(), st["n_path"].tolist(), st["loc_len"].tolist()
        for b in range(case["batch"]):
            for i in range(n[b]):
                K[b, loc[b] + i] = st["K_draft"][b, path[b][i]].double()
                V[b, loc[b] + i] = st["V_draft"][b, path[b][i]].double()
            new[b] = loc[b] + n[b]
        return K, V, new
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=st["q"].device)
    loc, n = st["loc_len"].tolist(), st["n_draft"].tolist()
    off = st["chunk_off"].tolist() if case["k"] else []
    for b in range(case["batch"]):
        K, V = [st["K_loc"][b, :loc[b]]], [st["V_loc"][b, :loc[b]]]
        for doc in st["topk_idx"][b].tolist() if case["k"] else []:
            K.append(st["K_bar"][off[doc]:off[doc + 1]])
            V.append(st["V_bar"][off[doc]:off[doc + 1]])
        K, V = torch.cat(K).double(), torch.cat(V).double()
        Kd, Vd = st["K_draft"][b, :n[b]].double(), st["V_draft"][b, :n[b]].double()
        bits = st["mask"][b, :n[b]].cpu().numpy().view(np.uint8)
        see = np.unpackbits(bits, axis=1, bitorder="little")[:, :n[b]].astype(bool).reshape(n[b], n[b])
        see = torch.from_numpy(see).to(K.device)
        for h in range(case["n_q"]):
            hk = h // (case["n_q"] // case["n_kv"])
            q = st["q"][b, :n[b], h].double()
            s = torch.cat((q @ K[:, hk].T, (q @ Kd[:, hk].T).masked_fill(~see, -math.inf)), 1) / math.sqrt(case["head_dim"])
            out[b, :n[b], h] = torch.softmax(s, -1) @ torch.cat((V[:, hk], Vd[:, hk]))
    return out
