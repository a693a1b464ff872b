"""fp64 oracle of a speculative step over trees of drafted tokens (test code only).

Definitions (the pages have no such step; the reading is stated here):
  * a sequence's rows are its tree: parents[i] < i, -1 for a root; row i's token
    has the cache place past + i, its position is past + depth(i);
  * row i sees every place before `past`, and past + j for j on its way up to
    its root, itself included (or what another mask says);
  * the walk of the verification, with w and Z as in mla_tree_verify's
    definition, and the next token drawn at whole-number weights floor(2^40 w);
  * the kept rows move to places past, past + 1, ...
"""

import math

import numpy as np

from .mla_oracle import out_proj

STEP = 1 << 40


def depths(parents):
    d = []
    for p in parents:
        d.append(0 if p < 0 else d[p] + 1)
    return np.array(d, np.int64)


def ancestors(parents) -> np.ndarray:
    """[T, T] bool: row i's way up, itself included."""
    t = len(parents)
    m = np.zeros((t, t), bool)
    for i in range(t):
        j = i
        while j >= 0:
            m[i, j] = True
            j = parents[j]
    return m


def words(mask: np.ndarray, n: int) -> np.ndarray:
    """A bool mask [T, T] as [T, n] words of 64 bits (int64)."""
    out = np.zeros((mask.shape[0], n), np.uint64)
    for i, j in zip(*np.nonzero(mask)):
        out[i, j // 64] |= np.uint64(1) << np.uint64(j % 64)
    return out.view(np.int64)


def attend(q_abs, rows, mask, scale, W_uv):
    """q_abs [T, H, 576]; rows [past + T, 576]; mask [T, T] bool. Returns the
    output [T, H, 128], and for a tolerance: each weight's share of it,
    g = sum_t p_t |v_t| |W_uv|, and the largest half score |S_h| of a seen token
    (in units of the softmax's exponent)."""
    T, H, _ = q_abs.shape
    past = len(rows) - T
    seen = np.concatenate([np.ones((T, past), bool), np.asarray(mask, bool)], 1)
    out, g, half = np.zeros((T, H, 128)), np.zeros((T, H, 128)), np.zeros((T, H))
    for i in range(T):
        at = np.nonzero(seen[i])[0]
        if not len(at):
            continue
        kv = rows[at]
        s = (q_abs[i] @ kv.T) * scale                            # [H, n]
        part = (q_abs[i][:, :256] @ kv[:, :256].T) * scale
        half[i] = np.maximum(np.abs(part), np.abs(s - part)).max(1)
        p = np.exp(s - s.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        out[i] = out_proj((p @ kv[:, :512])[None], W_uv)[0]
        g[i] = np.einsum("hc,hcv->hv", p @ np.abs(kv[:, :512]), np.abs(W_uv))
    return out, g, half


def _clamp(p):
    return np.clip(np.nan_to_num(np.asarray(p, np.float32), nan=0.0, posinf=1.0, neginf=0.0), 0, 1)


def _whole(w) -> list:
    """floor(w 2^40) of float32 weights, as Python integers."""
    return [int(x) for x in np.floor(w.astype(np.float64) * STEP)]


def verify(target, draft, tokens, parents, u, u_last, max_path=None):
    """One sequence: (kept rows, next token)."""
    T, V = target.shape
    cur, path = 0, [0]
    w, z, gone = _clamp(target[0]), 1.0, False
    i = 1
    while i < T and (max_path is None or len(path) < max_path):
        if parents[i] != cur:
            i += 1
            continue
        x = int(tokens[i])
        if not 0 <= x < V:
            i += 1
            continue
        share = float(draft[cur][x]) if draft is not None else 1.0
        if float(u[i]) * share * z < float(w[x]):
            cur = i
            path.append(i)
            w, z = _clamp(target[cur]), 1.0
        elif draft is not None:
            # one rounding, as a fused multiply-add has
            less = w.astype(np.float64) - z * draft[cur].astype(np.float64)
            w = np.fmax(less.astype(np.float32), np.float32(0))   # (of a NaN: 0)
            z = float(np.float32(math.ldexp(float(sum(_whole(w))), -40)))
        else:
            z = max(z - float(w[x]), 0.0)
            w = w.copy()
            w[x] = 0
        i += 1
    k = _whole(w)
    total = sum(k)
    if total == 0:
        k = _whole(_clamp(target[cur]))
        total = sum(k)
    if total == 0:
        return path, -1
    goal = min(int(math.floor(max(float(u_last), 0.0) * float(total))), total - 1)
    run = 0
    for t, x in enumerate(k):
        run += x
        if run > goal:
            return path, t
    raise AssertionError


def commit(rows, past, path):
    """rows [places, ...] of one sequence, after the kept rows have moved."""
    out = rows.copy()
    for i, p in enumerate(path):
        out[past + i] = rows[past + p]
    return out
