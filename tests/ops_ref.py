"""Plain float64 references of the operators around a step's attention (numpy, no library code), and
their input builders."""
from __future__ import annotations

import math

import numpy as np

BS = 16


def bf16_values(bits: np.ndarray) -> np.ndarray:
    return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def to_bf16(x: np.ndarray) -> np.ndarray:
    """Bit patterns of float values rounded to bf16 (nearest even; NaN kept)."""
    f = np.ascontiguousarray(x, dtype=np.float32)
    u = f.view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    r[np.isnan(f)] = 0x7FC0
    return r


def e4m3_table() -> np.ndarray:
    """The value of each e4m3 code (bias 7, 3 mantissa bits, no infinities, 0x7F / 0xFF NaN)."""
    t = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        t[c] = math.nan if c & 127 == 127 else (-v if c >> 7 else v)
    return t


# ------------------------------------------------------------------------------------ rotation
def rope(x: np.ndarray, pos: np.ndarray, inv_freq: np.ndarray, interleaved: bool) -> np.ndarray:
    """x [n, heads, H] turned by pos [n]; angles reduced exactly (integers times a float64, by fmod of the
    product taken in extended steps)."""
    R = 2 * len(inv_freq)
    ang = np.empty((len(pos), R // 2))
    for j, f in enumerate(inv_freq):
        # exact product of the integer position and the float64 frequency, modulo 2 pi in 200-bit integers
        m, e = math.frexp(float(f))
        num = int(m * (1 << 53))                               # f = num 2^(e - 53)
        two_pi = 6283185307179586476925286766559005768394338798750  # 2 pi 10^48
        for i, p in enumerate(pos):
            top = num * int(p) * 10 ** 48                      # times 2^(e - 53)
            bot = two_pi
            if e - 53 >= 0:
                top <<= e - 53
            else:
                bot <<= 53 - e
            r = top % bot if top >= 0 else -((-top) % bot)
            ang[i, j] = 2 * math.pi * (r * 10 ** 25 // bot) / 10 ** 25
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    y = x.copy()
    a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    return y


# ------------------------------------------------------------------------- blocks and selection
def tables(rng, ctx, width=None, spare=2, shuffle=True):
    """(block_tables int32 [B, width] with -1 tails, pool size) of private blocks in random order."""
    nb = [-(-int(c) // BS) for c in ctx]
    width = max([1] + nb) if width is None else width
    pool = sum(nb) + spare
    order = rng.permutation(pool) if shuffle else np.arange(pool)
    out = np.full((len(ctx), width), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(nb):
        out[b, :n] = order[at:at + n]
        at += n
    return out, pool


def key_bounds(keys: np.ndarray, block_tables, ctx, num_new, bounds: np.ndarray) -> np.ndarray:
    """bounds [pool, K, 2, H] with the touched blocks' minima and maxima of keys [pool, 16, K, H]."""
    out = bounds.copy()
    for b, c in enumerate(ctx):
        for j in range(max(0, int(c) - num_new) // BS, -(-int(c) // BS)):
            rows = keys[block_tables[b, j], :min(BS, int(c) - BS * j)]
            out[block_tables[b, j], :, 0] = rows.min(0)
            out[block_tables[b, j], :, 1] = rows.max(0)
    return out


def exact_sum(terms: np.ndarray) -> float:
    return math.fsum(terms.tolist()) if np.all(np.isfinite(terms)) else float(terms.sum())


def select(q, bounds, block_tables, ctx, M, first, last) -> np.ndarray:
    """q [B, N, H], bounds [pool, K, 2, H] float64: exact scores (math.fsum), ties to the lowest index."""
    B, N, H = q.shape
    K = bounds.shape[1]
    G = N // K
    out = np.full((B, K, M), -1, dtype=np.int32)
    for b, c in enumerate(ctx):
        nb = -(-int(c) // BS)
        if nb <= M:
            out[b, :, :nb] = np.arange(nb)
            continue
        for k in range(K):
            scored = []
            for j in range(first, nb - last):
                blk = block_tables[b, j]
                if not 0 <= blk < bounds.shape[0]:
                    scored.append((-math.inf, j))
                    continue
                lo, hi = bounds[blk, k]
                s = []
                for g in range(G):
                    x = q[b, k * G + g]
                    s.append(exact_sum(np.where(x > 0, x * hi, x * lo)))
                scored.append((math.inf if any(math.isnan(v) for v in s) else max(s), j))
            best = sorted(scored, key=lambda t: (-t[0], t[1]))[:M - first - last]
            out[b, k] = sorted(list(range(first)) + [j for _, j in best] + list(range(nb - last, nb)))
    return out


# ------------------------------------------------------------------------------------ attention
def blocks_attention(q, keys, values, block_tables, ctx, selected, scale):
    """(out, lse, spread): spread [B, N, H] = the weighted mean of |v|, which scales the error bound of 16-bit
    weights.  keys, values [pool, 16, K, H] float64."""
    B, N, H = q.shape
    K = keys.shape[2]
    G = N // K
    out, lse, spread = np.zeros((B, N, H)), np.full((B, N), -np.inf), np.zeros((B, N, H))
    for b, c in enumerate(ctx):
        nb = -(-int(c) // BS)
        for k in range(K):
            rows_k, rows_v = [], []
            for j in selected[b, k, :min(nb, selected.shape[2])]:
                if j < 0 or j >= nb or not 0 <= block_tables[b, j] < keys.shape[0]:
                    continue
                n = min(BS, int(c) - BS * int(j))
                rows_k.append(keys[block_tables[b, j], :n, k])
                rows_v.append(values[block_tables[b, j], :n, k])
            if not rows_k:
                continue
            kk, vv = np.concatenate(rows_k), np.concatenate(rows_v)
            for g in range(G):
                z = scale * (kk @ q[b, k * G + g])
                m = z.max()
                w = np.exp(z - m)
                out[b, k * G + g] = w @ vv / w.sum()
                spread[b, k * G + g] = w @ np.abs(vv) / w.sum()
                lse[b, k * G + g] = m + math.log(w.sum())
    return out, lse, spread


# --------------------------------------------------------------------------------- verification
def clean(p):
    """Probabilities as the definition reads them: clamped to [0, 1], NaN is 0."""
    p = np.asarray(p, dtype=np.float64)
    return np.where(np.isnan(p), 0.0, np.clip(p, 0.0, 1.0))


def verify(p, q, tokens, u, r, lens=None, V=None):
    """(accepted, tokens_out): p [B, T + 1, >= V], q [B, T, >= V] or None, float64; running sums by math.fsum where
    they decide."""
    B, T = tokens.shape
    V = p.shape[2] if V is None else V
    p, q = clean(p[..., :V]), None if q is None else clean(q[..., :V])
    acc, out = np.zeros(B, np.int32), np.full((B, T + 1), -1, np.int32)
    for b in range(B):
        m = T if lens is None else int(lens[b])
        t = 0
        while t < m:
            x = int(tokens[b, t])
            if not 0 <= x < V:
                break
            if not float(u[b, t]) * (1.0 if q is None else q[b, t, x]) < p[b, t, x]:
                break
            out[b, t] = x
            t += 1
        w = p[b, t].copy()
        if t < m:
            if q is not None:
                w = np.maximum(w - q[b, t], 0.0)
            elif 0 <= int(tokens[b, t]) < V:
                w[int(tokens[b, t])] = max(0.0, w[int(tokens[b, t])] - 1.0)
            if w.sum() == 0.0:
                w = p[b, t].copy()
        total = math.fsum(w.tolist())
        acc[b] = t
        if total == 0.0:
            continue
        run = np.cumsum(w)
        bar = min(max(float(r[b]), 0.0), 1.0 - 2.0 ** -53) * total
        hit = np.nonzero(run > bar)[0]
        out[b, t] = hit[0] if len(hit) else np.nonzero(w)[0][-1]
    return acc, out
