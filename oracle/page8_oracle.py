"""fp64 oracle of the page-scaled 8-bit cache and of eviction (test code only).

Definitions (the pages name neither; the reading is stated here):
  * page p holds e4m3 codes of c_hat / S_p, S_p = 2^e a power of two, e the
    least integer in [-64, 64] with amax <= 448 * 2^e over the page's new rows,
    never below the scale the page had; codes in a page whose scale grows
    become e4m3(code * old / new);
  * attention reads the row [S_p * code || k_rot];
  * the mass of a cached token is decay * mass + the sum over its sequence's
    query rows and all heads of the attention weight;
  * eviction keeps the first `sinks`, the last `recent` and, of the others, the
    tokens of largest mass (ties: lower index; NaN least) up to `budget`;
  * compaction moves the kept rows, in order, to other pages, whose scale is
    the largest among the pages the rows come from.
"""

import math

import numpy as np

from .mla_oracle import (e4m3_decode, e4m3_encode, e4m3_round, latent_attention, out_proj,
                         rms_norm, rope)

E_MIN, E_MAX = -64, 64


def scale_for(amax: float) -> float:
    """2^e, e the least integer in [E_MIN, E_MAX] with amax <= 448 * 2^e."""
    for e in range(E_MIN, E_MAX + 1):
        if amax <= math.ldexp(448.0, e):
            return math.ldexp(1.0, e)
    return math.ldexp(1.0, E_MAX)


def recode(codes, factor: float) -> np.ndarray:
    """e4m3 codes of (value * factor); NaN codes stay NaN of either sign."""
    codes = np.asarray(codes, np.uint8)
    v = e4m3_decode(codes)
    nan = np.isnan(v)
    out = e4m3_encode(e4m3_round(np.where(nan, 0.0, v) * factor)).astype(np.uint8)
    return np.where(nan, codes, out)


def write(codes, rope_rows, scales, c_kv, k_pe, positions, slots, weight, eps, base,
          interleaved=False):
    """The cache after a write: (codes [nb, bs, 512] uint8, rope [nb, bs, 64]
    float64, scales [nb]); the inputs are not changed. Negative slots and slots
    past the cache are skipped; of two tokens with one slot the later stays."""
    codes, rope_rows, scales = codes.copy(), rope_rows.copy(), np.asarray(scales, np.float64).copy()
    nb, bs = codes.shape[:2]
    c_hat = rms_norm(c_kv, weight, eps)
    rot = rope(k_pe, positions, base, interleaved)
    pages = {}
    for t, s in enumerate(np.asarray(slots)):
        if 0 <= s < nb * bs:
            pages.setdefault(int(s) // bs, {})[int(s) % bs] = t
    for p, rows in pages.items():
        toks = list(rows.values())
        amax = np.nanmax(np.abs(c_hat[toks])) if np.isfinite(c_hat[toks]).any() else 0.0
        new = max(scales[p], scale_for(amax))
        if 0 < scales[p] < new:
            codes[p] = recode(codes[p], scales[p] / new)
        scales[p] = new
        for r, t in rows.items():
            codes[p, r] = e4m3_encode(e4m3_round(c_hat[t] / new))
            rope_rows[p, r] = rot[t]
    return codes, rope_rows, scales


def rows_of(codes, rope_rows, scales) -> np.ndarray:
    """The cache as float64 rows [nb, bs, 576]."""
    s = np.maximum(np.asarray(scales, np.float64), math.ldexp(1.0, E_MIN))
    return np.concatenate([e4m3_decode(codes) * s[:, None, None], rope_rows], -1)


def decode(q_abs, rows, block_table, seq_lens, query_start_loc, scale, W_uv, mass=None, decay=1.0):
    """(out [num_q, H, 128], mass after the step or None); rows [nb, bs, 576]."""
    bs = rows.shape[1]
    out = np.zeros((q_abs.shape[0], q_abs.shape[1], W_uv.shape[2]))
    mass = None if mass is None else np.asarray(mass, np.float64).copy()
    for b, n in enumerate(seq_lens):
        q0, q1 = int(query_start_loc[b]), int(query_start_loc[b + 1])
        if q1 <= q0:
            continue
        n = int(n)
        pages = np.asarray(block_table[b][:(n + bs - 1) // bs], np.int64)
        kv = rows[pages].reshape(-1, rows.shape[2])[:n]
        pos = np.arange(n - (q1 - q0), n)
        o, lse = latent_attention(q_abs[q0:q1], kv, pos, scale)
        out[q0:q1] = out_proj(o, W_uv)
        if mass is not None:
            s = scale * np.einsum("nhk,tk->nht", np.asarray(q_abs[q0:q1], np.float64), kv)
            p = np.exp(s - lse[..., None]) * (np.arange(n)[None, None] <= pos[:, None, None])
            at = (pages[:, None] * bs + np.arange(bs)[None]).reshape(-1)[:n]
            flat = mass.reshape(-1)
            flat[at] = (decay * flat[at] if decay > 0 else 0.0) + p.sum((0, 1))
    return out, mass


def select(mass, block_table, seq_lens, sinks, recent, budget):
    """(keep [B, budget] int32 padded with -1, new_lens [B] int32)."""
    bs = mass.shape[1]
    keep = np.full((len(seq_lens), budget), -1, np.int32)
    new = np.zeros(len(seq_lens), np.int32)
    for b, n in enumerate(int(x) for x in seq_lens):
        m = np.asarray(mass, np.float64)[np.asarray(block_table[b][:(n + bs - 1) // bs], np.int64)].reshape(-1)[:n]
        if n <= budget:
            chosen = list(range(n))
        else:
            middle = sorted(range(sinks, n - recent),
                            key=lambda t: (math.isnan(m[t]), -m[t] if not math.isnan(m[t]) else 0.0, t))
            chosen = sorted(list(range(sinks)) + list(range(n - recent, n)) +
                            middle[:budget - sinks - recent])
        keep[b, :len(chosen)] = chosen
        new[b] = len(chosen)
    return keep, new


def compact(codes, rope_rows, scales, mass, block_table, keep, new_lens, dst_table):
    """The cache after compaction; the inputs are not changed."""
    c2, r2, s2, m2 = codes.copy(), rope_rows.copy(), scales.copy(), mass.copy()
    bs = codes.shape[1]
    for b, n in enumerate(int(x) for x in new_lens):
        for j in range((n + bs - 1) // bs):
            toks = [int(t) for t in keep[b][j * bs:min(n, (j + 1) * bs)]]
            src = [int(block_table[b][t // bs]) for t in toks]
            d = int(dst_table[b][j])
            s2[d] = max(scales[p] for p in src)
            for r, (t, p) in enumerate(zip(toks, src)):
                c2[d, r] = codes[p, t % bs] if scales[p] == s2[d] else recode(codes[p, t % bs], scales[p] / s2[d])
                r2[d, r] = rope_rows[p, t % bs]
                m2[d, r] = mass[p, t % bs]
    return c2, r2, s2, m2
