"""Plain references of the latent cache's operators (float64) and of the operators on sequences' blocks (row by row, in
order), in numpy without library code."""
from __future__ import annotations

import math

import numpy as np

import ops_ref as R

DIM, ROPE = 512, 64
ROW = DIM + ROPE


def append_rows(kv, pos, inv_freq, interleaved, weight, eps):
    """kv [n, 576] float64 -> rows of the cache."""
    c = kv[:, :DIM]
    if weight is not None:
        c = c / np.sqrt((c * c).mean(-1, keepdims=True) + eps) * weight
    return np.concatenate([c, R.rope(kv[:, None, DIM:], pos, inv_freq, interleaved)[:, 0]], -1)


def attention(q, cache, tables, ctx, scale):
    """q [B, T, N, 576], cache [blocks, 16, 576] float64 -> out [B, T, N, 512], lse, sum w |v| / l, and the largest sum of
    |q| |c| a row meets.  Blocks outside the pool are left out."""
    B, T, N, _ = q.shape
    out, spread = np.zeros((B, T, N, DIM)), np.zeros((B, T, N, DIM))
    lse, size = np.full((B, T, N), -math.inf), np.zeros((B, T, N))
    for b in range(B):
        c = int(ctx[b])
        if not 0 < c <= tables.shape[1] * 16:
            continue
        ids = tables[b, :-(-c // 16)]
        good = np.repeat((ids >= 0) & (ids < len(cache)), 16)[:c]
        rows = cache[np.clip(ids, 0, len(cache) - 1)].reshape(-1, ROW)[:c]
        for t in range(T):
            seen = good & (np.arange(c) < c - T + t + 1)
            if not seen.any():
                continue
            k = rows[seen]
            z = scale * (q[b, t] @ k.T)
            top = z.max(-1, keepdims=True)
            w = np.exp(z - top)
            l = w.sum(-1, keepdims=True)
            out[b, t], spread[b, t] = w @ k[:, :DIM] / l, w @ np.abs(k[:, :DIM]) / l
            lse[b, t] = (top + np.log(l))[:, 0]
            size[b, t] = (np.abs(q[b, t]) @ np.abs(k).T).max(-1)
    return out, lse, spread, size


# ------------------------------------------------------------------- rows and the blocks they hold
def counts(tables, ctx, num_blocks):
    ref = np.zeros(num_blocks, dtype=np.int64)
    for row, c in zip(tables, ctx):
        for id_ in row[:-(-int(c) // 16)]:
            ref[id_] += 1
    return ref


def fork(tables, ctx, parents, num_blocks):
    """New tables and lengths, and their counts."""
    out, lens = np.full((len(parents), tables.shape[1]), -1, dtype=np.int32), np.zeros(len(parents), dtype=np.int32)
    for b, p in enumerate(parents):
        if 0 <= p < len(ctx):
            nb = -(-int(ctx[p]) // 16)
            out[b, :nb], lens[b] = tables[p, :nb], ctx[p]
    return out, lens, counts(out, lens, num_blocks)


def extend(tables, ctx, num_new, ref):
    """One row after the other; -> tables, lengths, counts, copies, whether a row was refused."""
    tables, ctx, ref = tables.copy(), ctx.copy(), ref.copy()
    copies = np.full((len(ctx), 2), -1, dtype=np.int32)
    free = sorted(np.flatnonzero(ref == 0).tolist(), reverse=True)
    for b, t in enumerate(num_new):
        n, t = int(ctx[b]), int(t)
        if t <= 0 or n < 0 or n + t > 16 * tables.shape[1]:
            continue
        shared = n % 16 != 0 and ref[tables[b, n // 16]] > 1
        before, after = -(-n // 16), -(-(n + t) // 16)
        if shared + after - before > len(free):
            return tables, ctx, ref, copies, True
        if shared:
            old, new = tables[b, n // 16], free.pop()
            copies[b], tables[b, n // 16] = (old, new), new
            ref[old] -= 1
            ref[new] = 1
        for j in range(before, after):
            tables[b, j] = free.pop()
            ref[tables[b, j]] = 1
        ctx[b] = n + t
    return tables, ctx, ref, copies, False


def compact(tables, ctx, ref, max_moves):
    tables, ref = tables.copy(), ref.copy()
    moves, to = np.full((max_moves, 2), -1, dtype=np.int32), {}
    lo, hi, n = 0, len(ref) - 1, 0
    while n < max_moves:
        while lo < len(ref) and ref[lo]:
            lo += 1
        while hi >= 0 and not ref[hi]:
            hi -= 1
        if lo >= hi:
            break
        moves[n], to[hi] = (hi, lo), lo
        ref[lo], ref[hi] = ref[hi], 0
        n += 1
    for b, c in enumerate(ctx):
        for j in range(-(-int(c) // 16)):
            tables[b, j] = to.get(int(tables[b, j]), tables[b, j])
    return tables, ref, moves, n


def random_rows(r, rows, width, num_blocks, fill=0.5):
    """Rows of random lengths over a pool, some sharing their leading (full) blocks, some everything with another row."""
    tables, ctx = np.full((rows, width), -1, dtype=np.int32), np.zeros(rows, dtype=np.int32)
    free = r.permutation(num_blocks)[:int(num_blocks * fill)].tolist()
    for b in range(rows):
        kind = r.random()
        like = int(r.integers(0, b)) if b else 0
        if b and kind < 0.3:
            tables[b], ctx[b] = tables[like], ctx[like]
            continue
        n = int(r.integers(0, 16 * width + 1))
        head = int(r.integers(0, min(n, int(ctx[like])) // 16 + 1)) if b and kind < 0.6 else 0
        need = -(-n // 16) - head
        if need > len(free):
            n, need = 16 * head, 0
        tables[b, :head] = tables[like, :head]
        for j in range(need):
            tables[b, head + j] = free.pop()
        ctx[b] = n
    return tables, ctx, counts(tables, ctx, num_blocks).astype(np.int32)
