"""Plain float64 definitions of the rotation, the per-head norms and the draft-tree calls (numpy only,
no code shared with the package): what the GPU parity tests of those calls compare against."""
import math

import numpy as np


# ----------------------------------------------------------------------------
# rotary positions of any layout, per-head norms, trees of drafted tokens
# ----------------------------------------------------------------------------
def rotary_theta(rot_dim: int, base: float, scaling: str = "none", factor: float = 1.0, orig_len: int = 0,
                 low: float = 1.0, high: float = 32.0) -> np.ndarray:
    """Radians per position of each pair, with the frequency scalings of long contexts."""
    R = rot_dim
    i = np.arange(R // 2, dtype=np.float64)
    if scaling == "ntk" and R > 2:
        base = base * factor ** (R / (R - 2.0))
    th = base ** (-2.0 * i / R)
    if scaling == "linear":
        th = th / factor
    if scaling == "parts":
        g = np.clip((orig_len * th / (2 * math.pi) - low) / (high - low), 0.0, 1.0)
        th = (1 - g) * th / factor + g * th
    if scaling == "yarn":
        at = lambda t: R * math.log(orig_len / (2 * math.pi * t)) / (2 * math.log(base))
        first, last = max(math.floor(at(high)), 0), min(math.ceil(at(low)), R - 1)
        g = 1 - np.clip((i - first) / (last - first if last > first else 0.001), 0.0, 1.0)
        th = (1 - g) * th / factor + g * th
    return th


def rotate_heads(x, positions, theta, layout: str = "half", magnitude: float = 1.0, grad: bool = False) -> np.ndarray:
    """x [rows, heads, head_dim] float64, its first 2 len(theta) elements turned at positions [rows]."""
    x = np.asarray(x, dtype=np.float64)
    h = len(theta)
    a = [i for i in range(h)] if layout == "half" else [2 * i for i in range(h)]
    b = [h + i for i in range(h)] if layout == "half" else [2 * i + 1 for i in range(h)]
    ang = np.asarray(positions, dtype=np.float64)[:, None, None] * theta
    c, s = magnitude * np.cos(ang), magnitude * np.sin(ang) * (-1.0 if grad else 1.0)
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def head_norm(x, weight, weight_offset: float = 0.0, eps: float = 1e-6) -> np.ndarray:
    """RMS norm of each head: x / sqrt(mean(x^2) + eps) * (weight_offset + weight) (None: factor 1)."""
    x = np.asarray(x, dtype=np.float64)
    n = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    return n if weight is None else n * (weight_offset + np.asarray(weight, dtype=np.float64))


def head_norm_rotate_grad(x, weight, dy, positions, theta, layout="half", magnitude=1.0, weight_offset=0.0, eps=1e-6):
    """(dx, dweight) of rotate_heads(head_norm(x, weight))."""
    x = np.asarray(x, dtype=np.float64)
    z = rotate_heads(dy, positions, theta, layout, magnitude, grad=True)
    r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    n = x * r
    u = z if weight is None else z * (weight_offset + np.asarray(weight, dtype=np.float64))
    dx = r * (u - n * np.mean(u * n, axis=-1, keepdims=True))
    return dx, np.sum(z * n, axis=(0, 1))


def tree_plan(parents, n_draft, loc_len, pos_offset: int):
    """(see [B, M, M] bool, positions [B, M]) of drafted trees."""
    parents = np.asarray(parents)
    B, M = parents.shape
    see = np.zeros((B, M, M), dtype=bool)
    pos = np.zeros((B, M), dtype=np.int64)
    for b in range(B):
        for t in range(M):
            depth = 0
            if t < n_draft[b]:
                j = t
                while j >= 0:
                    see[b, t, j] = True
                    j = int(parents[b, j])
                    depth += j >= 0
            pos[b, t] = pos_offset + loc_len[b] + depth
    return see, pos


def pack_mask(see) -> np.ndarray:
    """[B, M, M] bool -> [B, M, ceil(M/32)] int32, bit j % 32 of word j // 32."""
    B, M, _ = see.shape
    W = (M + 31) // 32
    bits = np.zeros((B, M, 32 * W), dtype=bool)
    bits[:, :, :M] = see
    return np.packbits(bits, axis=2, bitorder="little").view(np.uint32).view(np.int32).reshape(B, M, W)


def tree_attend(q, K_draft, V_draft, see, n_draft, K_loc, V_loc, loc_len, K_bar=None, V_bar=None, chunk_off=None,
                topk_idx=None, scale=None) -> np.ndarray:
    """float64 attention of drafts over [pooled rows of the selected documents; local keys; drafts seen].

    Every tensor float64; keys that a row does not see are left out of its products entirely."""
    B, M, n_q, D = q.shape
    n_kv = K_draft.shape[2]
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    out = np.zeros_like(q)
    for b in range(B):
        Ks, Vs = [], []
        if topk_idx is not None:
            for doc in topk_idx[b]:
                Ks.append(K_bar[chunk_off[doc]:chunk_off[doc + 1]])
                Vs.append(V_bar[chunk_off[doc]:chunk_off[doc + 1]])
        if K_loc is not None:
            Ks.append(K_loc[b, :loc_len[b]])
            Vs.append(V_loc[b, :loc_len[b]])
        for t in range(min(int(n_draft[b]), M)):
            js = [j for j in range(int(n_draft[b])) if see[b, t, j]]
            K = np.concatenate(Ks + [K_draft[b, js]])
            V = np.concatenate(Vs + [V_draft[b, js]])
            if len(K) == 0:
                continue
            for h in range(n_q):
                g = h // (n_q // n_kv)
                s = K[:, g] @ q[b, t, h] * scale
                p = np.exp(s - s.max())
                out[b, t, h] = (p / p.sum()) @ V[:, g]
    return out
