"""What is measured of the latent cache (its append, its attention) and of the life of a cache's blocks (growing,
forking and compacting sequences).

Each operator in its plain form (elementary torch operations) and, with ``own`` true, as calls of the library.
``listed()`` holds the measured cases, ``draw()`` gives more of the same ranges.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16
LATENT, ROPE = 512, 64      # a cached row: the shared latent vector, then the shared rotary key
ROW = LATENT + ROPE
EPS = 1e-6


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # One decode step of 64 ragged sequences, 128 query heads: the newest tokens' latents are normed, their
        # rotary parts turned, both appended; a call this small is latency.
        dict(name="append_step_b64", op="append_step", B=64, T=1, N=128, lo=512, hi=8192, inter=True, norm=True),
        # A prefill chunk of 8,192 prompt tokens of eight sequences, 16 heads, somewhere in long contexts.
        dict(name="append_prompt_8k", op="append", tokens=8192, seqs=8, N=16, far=131072, inter=True, norm=True),
        # An odd number of prompt tokens, 40 heads, half layout, latents that come normed.
        dict(name="append_prompt_5001", op="append", tokens=5001, seqs=7, N=40, far=4096, inter=False, norm=False),
        # One short sequence, 16 heads: the latency end.
        dict(name="attend_b1_n16", op="attend", B=1, T=1, N=16, lo=2000, hi=2000),
        # One sequence of 128K tokens, 128 heads: all of the chip on one sequence.
        dict(name="attend_b1_128k", op="attend", B=1, T=1, N=128, lo=131072, hi=131072),
        # A ragged batch of 64, 128 heads.
        dict(name="attend_b64", op="attend", B=64, T=1, N=128, lo=512, hi=8192),
        # Verification of drafted tokens: three new tokens of 20 long sequences, 16 heads.
        dict(name="attend_b20_t3", op="attend", B=20, T=3, N=16, lo=1000, hi=32520),
        # Each step: 64 sequences take one more token, a few of them share their last block after a fork, in the
        # pools of four layers.
        dict(name="extend_step_b64", op="extend", B=64, lo=512, hi=8192, new=1, full=0.8, shared=0.2, layers=4, K=0, H=ROW),
        # A scheduler's tick: 250 sequences take up to 700 tokens each, in a large pool with few free blocks.
        dict(name="extend_chunk_b250", op="extend", B=250, lo=0, hi=8192, new=700, full=0.93, shared=0.1, layers=1, K=2, H=128),
        # Beam search: 16 beams of 4 choose their parents anew.
        dict(name="fork_beams_b64", op="fork", B=64, lo=512, hi=8192, group=4, gone=0.0),
        # Parallel sampling of long prompts: 250 rows, some of them done, the others moved up or forked.
        dict(name="fork_b250", op="fork", B=250, lo=16008, hi=32520, group=10, gone=0.3),
        # After a burst: the pools of eight layers are compacted.
        dict(name="compact_l8", op="compact", B=20, lo=512, hi=8192, full=0.5, layers=8, K=0, H=ROW),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append_step", "attend", "attend", "extend", "fork", "compact"])
    N = rng.choice([1, 4, 8, 16, 20, 32, 40, 64, 96, 128])
    inter, norm = rng.random() < 0.5, rng.random() < 0.7
    if op == "append":
        return dict(op=op, tokens=_log(rng, 1, 8000), seqs=rng.randint(1, 9), N=min(N, 40), far=_log(rng, 16, 1000000),
                    inter=inter, norm=norm)
    if op == "append_step":
        return dict(op=op, B=_log(rng, 1, 200), T=rng.choice([1, 1, 2, 3, 5, 8]), N=N, lo=1, hi=_log(rng, 16, 9000),
                    inter=inter, norm=norm)
    if op == "attend":
        B, T = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 3, 4])
        most = 64 * 128 * 8192 // (B * max(T * N, 128))      # no more work than the ragged batch's
        hi = _log(rng, 16, min(30000, most))
        return dict(op=op, B=B, T=T, N=N, lo=min(hi, rng.choice([0, 1, 40])), hi=hi)
    latent = rng.random() < 0.5
    K, H = (0, ROW) if latent else (rng.choice([1, 2, 5, 8]), rng.choice([64, 128]))
    layers = rng.randint(1, 4)
    size = 2 * BLOCK * H * max(2 * K, 1) * layers            # bytes of a block in every pool
    if op == "extend":
        B, full = _log(rng, 1, 250), rng.uniform(0.4, 0.98)
        hi = _log(rng, 17, max(17, min(8192, int(2 * BLOCK * full * 2e9 / (B * size)))))
        return dict(op=op, B=B, lo=0, hi=hi, new=_log(rng, 1, 700), full=full, shared=rng.choice([0.0, 0.2, 0.5]),
                    layers=layers, K=K, H=H)
    if op == "fork":
        hi = _log(rng, 17, 32000)
        return dict(op=op, B=_log(rng, 1, 250), lo=0, hi=hi, group=rng.randint(1, 10), gone=rng.uniform(0.0, 0.6))
    B, full = _log(rng, 1, 40), rng.uniform(0.2, 0.95)
    hi = _log(rng, 17, max(17, min(8192, int(2 * BLOCK * full * 1.6e9 / (B * size)))))
    return dict(op=op, B=B, lo=0, hi=hi, full=full, layers=layers, K=K, H=H)


# ----------------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _blocks(n):
    return -(-n // BLOCK)


def _tables(seed, ctx, longest, pool=None):
    """Block tables over a shuffled pool with room for every sequence at its longest: int32 [B, most blocks] on the
    host, -1 behind a sequence's last block."""
    nb = _blocks(ctx.astype(np.int64))
    width = max(1, _blocks(longest))
    pool = pool or len(ctx) * width + 3
    order = np.random.default_rng(seed + 1).permutation(pool).astype(np.int32)
    tables = np.full((len(ctx), width), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(nb):
        tables[b, :n] = order[at:at + n]
        at += int(n)
    return tables, pool


def _state(s, tables, ctx, refs, extra=()):
    """The integers that describe the sequences, in one tensor (`now`) so that a pass can start from the saved ones
    (`then`) with one copy."""
    parts = [tables.reshape(-1), ctx, refs, *extra]
    s["then"] = torch.from_numpy(np.concatenate([p.reshape(-1) for p in parts]).astype(np.int32)).cuda()
    s["now"] = s["then"].clone()
    at, views = 0, []
    for p in parts:
        views.append(s["now"][at:at + p.size])
        at += p.size
    s["tables"], s["ctx"], s["refs"] = views[0].view(tables.shape), views[1], views[2]
    return views[3:]


def _pools(g, s, pool):
    shape = (pool, BLOCK, s["K"], s["H"]) if s["K"] else (pool, BLOCK, s["H"])
    s["pools"] = [_randn(g, *shape) for _ in range(s["layers"] * (2 if s["K"] else 1))]


def prepare(case, seed):
    c, g, r = case, _gen(seed), np.random.default_rng(seed)
    op = c["op"]
    s = dict(c)
    s["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if op in ("append", "append_step"):
        N = c["N"]
        if op == "append":
            n, lead = c["tokens"], (c["tokens"],)
            # consecutive runs of tokens, each starting somewhere below `far`
            run = np.sort(r.integers(0, c["seqs"], size=n))
            start = r.integers(0, c["far"], size=c["seqs"])
            first = np.searchsorted(run, np.arange(c["seqs"]))
            s["positions"] = torch.from_numpy((start[run] + np.arange(n) - first[run]).astype(np.int32)).cuda()
            pool = _blocks(n) + 2
            slots = r.permutation(pool * BLOCK)[:n].astype(np.int64)
            if n > 4:
                slots[r.integers(0, n, size=2)] = -1   # padding rows of the batch
            s["slots"] = torch.from_numpy(slots).cuda()
        else:
            lead = (c["B"], c["T"])
            ctx = np.maximum(r.integers(c["lo"], c["hi"] + 1, size=c["B"]), c["T"]).astype(np.int32)
            tables, pool = _tables(seed, ctx, max(c["hi"], c["T"]))
            s["tables"], s["ctx"] = torch.from_numpy(tables).cuda(), torch.from_numpy(ctx).cuda()
            s["slots"] = torch.empty(lead, dtype=torch.int64, device="cuda")
        # a projection's rows: latents of some magnitude, rotary parts behind them; queries 192 wide, of which the
        # last 64 turn, and the buffer that attention takes, its latent parts filled by another projection
        s["kv_new"] = _randn(g, *lead, ROW) * (0.5 + 2.0 * torch.rand(*lead, 1, generator=g, device="cuda")).bfloat16()
        s["q_rope"] = _randn(g, *lead, N, 3 * ROPE)[..., 2 * ROPE:]
        s["q"] = _randn(g, *lead, N, ROW)
        s["weight"] = (1.0 + 0.1 * _randn(g, LATENT)) if c["norm"] else None
        s["cache"] = torch.zeros(pool, BLOCK, ROW, dtype=torch.bfloat16, device="cuda")
        s["inv_freq"] = torch.tensor([10000.0 ** (-2.0 * j / ROPE) for j in range(ROPE // 2)], dtype=torch.float64,
                                     device="cuda")
    elif op == "attend":
        B, T, N = c["B"], c["T"], c["N"]
        ctx = r.integers(c["lo"], c["hi"] + 1, size=B).astype(np.int32)
        tables, pool = _tables(seed, ctx, c["hi"])
        s["tables"], s["ctx"] = torch.from_numpy(tables).cuda(), torch.from_numpy(ctx).cuda()
        s["cache"] = _randn(g, pool, BLOCK, ROW)
        s["q"] = _randn(g, B, T, N, ROW)
        s["scale"] = 1.0 / math.sqrt(192.0)           # heads 128 + 64 wide before their keys were absorbed
        s["out"] = torch.empty(B, T, N, LATENT, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(B, T, N, dtype=torch.float32, device="cuda")
        if own:
            import paged_kv_decode_slot_gb300 as pkv
            s["ws"] = torch.zeros(pkv.pkv_latent_workspace_bytes(B, T, N), dtype=torch.uint8, device="cuda")
    else:
        B = c["B"]
        # lengths evenly over the range, in any order: a case's pool has one size whatever the seed
        ctx = r.permutation(np.linspace(c["lo"], c["hi"], B).round()).astype(np.int32)
        used = int(_blocks(ctx.astype(np.int64)).sum())
        longest = c["hi"] + (c["new"] if op == "extend" else 0)
        pool = B * max(1, _blocks(longest)) + 64 if op == "fork" else max(used + 1, int(used / c["full"]))
        parent = np.arange(B)
        if op == "extend":        # some rows are fresh forks of others: all blocks shared
            child = r.random(B) < c["shared"]
            child[0] = False
            parent = np.where(child, r.integers(0, np.maximum(np.arange(B), 1)), np.arange(B))
            for b in range(B):
                parent[b] = parent[parent[b]]
        elif op == "fork":        # beams: the rows of a group share the first half of their blocks
            ctx = np.maximum(ctx, ctx[np.arange(B) // c["group"] * c["group"]] // 2 // BLOCK * BLOCK).astype(np.int32)
        ctx = ctx[parent]
        own_rows = np.where(parent == np.arange(B), ctx, 0).astype(np.int32)
        tables, _ = _tables(seed, own_rows, longest, pool)
        tables = tables[parent]
        if op == "fork":
            for b in range(B):
                first = b // c["group"] * c["group"]
                head = int(ctx[first]) // 2 // BLOCK
                tables[b, :head] = tables[first, :head]
        refs = np.bincount(tables[tables >= 0], minlength=pool).astype(np.int32)
        if op == "extend":
            s["num_new"] = torch.from_numpy((r.integers(0, c["new"] + 1, size=B) if c["new"] > 1 else
                                             np.ones(B)).astype(np.int32)).cuda()
            (copies,) = _state(s, tables, ctx, refs, [np.full((B, 2), -1)])
            s["copies"] = copies.view(B, 2)
            _pools(g, s, pool)
        elif op == "fork":
            s["tables_out"] = torch.empty(tables.shape, dtype=torch.int32, device="cuda")
            s["ctx_out"] = torch.empty(B, dtype=torch.int32, device="cuda")
            _state(s, tables, ctx, refs)
            # every row takes a row of its own group (itself, most often), or nothing
            pick = np.arange(B) // c["group"] * c["group"] + r.integers(0, c["group"], size=B)
            pick = np.where((pick >= B) | (r.random(B) < 0.4), np.arange(B), pick)
            s["parents"] = torch.from_numpy(np.where(r.random(B) < c["gone"], -1, pick).astype(np.int32)).cuda()
        else:
            _state(s, tables, ctx, refs)
            s["moves"] = torch.empty(max(1, pool // 2), 2, dtype=torch.int32, device="cuda")
            s["num_moves"] = torch.empty(1, dtype=torch.int32, device="cuda")
            _pools(g, s, pool)
        if own and op != "fork":
            import paged_kv_decode_slot_gb300 as pkv
            s["ws"] = torch.zeros(pkv.pkv_blocks_workspace_bytes(pool), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------------- the operators
def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _own_append(s):
    import paged_kv_decode_slot_gb300 as pkv
    pkv.check(pkv.pkv_latent_append(s["kv_new"], s["q_rope"], s["positions"], s["inv_freq"], s["slots"], s["cache"], s["q"],
                                    norm_weight=s["weight"], eps=EPS, interleaved=s["inter"], err_flag=s["err"]))
    return s["q"], s["cache"]


def _own_append_step(s):
    import paged_kv_decode_slot_gb300 as pkv
    pkv.check(pkv.pkv_latent_append_multi(s["kv_new"], s["q_rope"], s["tables"], s["ctx"], s["inv_freq"], s["cache"],
                                          s["q"], s["slots"], norm_weight=s["weight"], eps=EPS, interleaved=s["inter"],
                                          err_flag=s["err"]))
    return s["q"], s["slots"], s["cache"]


def _own_attend(s):
    import paged_kv_decode_slot_gb300 as pkv
    pkv.check(pkv.pkv_decode_attn_latent(s["q"], s["cache"], s["tables"], s["ctx"], s["scale"], s["out"], s["lse"],
                                         s["ws"], s["err"]))
    return s["out"], s["lse"]


def _own_extend(s):
    import paged_kv_decode_slot_gb300 as pkv
    s["now"].copy_(s["then"])
    pkv.check(pkv.pkv_extend_sequences(s["tables"], s["ctx"], s["num_new"], s["refs"], s["copies"], s["ws"], s["err"]))
    pkv.check(pkv.pkv_copy_blocks_pools(s["pools"], s["copies"], s["err"]))
    return s["tables"], s["ctx"], s["refs"], s["copies"], *s["pools"]


def _own_fork(s):
    import paged_kv_decode_slot_gb300 as pkv
    s["now"].copy_(s["then"])
    pkv.check(pkv.pkv_fork_sequences(s["tables"], s["ctx"], s["parents"], s["refs"], s["tables_out"], s["ctx_out"], s["err"]))
    return s["tables_out"], s["ctx_out"], s["refs"]


def _own_compact(s):
    import paged_kv_decode_slot_gb300 as pkv
    s["now"].copy_(s["then"])
    pkv.check(pkv.pkv_compact_blocks(s["tables"], s["ctx"], s["refs"], s["moves"], s["num_moves"], s["ws"], s["err"]))
    pkv.check(pkv.pkv_copy_blocks_pools(s["pools"], s["moves"], s["err"]))
    return s["tables"], s["refs"], s["moves"], s["num_moves"], *s["pools"]


# the plain forms ------------------------------------------------------------------------------------
def _turn(x, cos, sin, inter):
    """x [..., heads, 64] rotated by the angles whose cosines and sines are [..., 1, 32], in 32 bits."""
    x = x.float()
    if inter:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    a, b = x[..., :ROPE // 2], x[..., ROPE // 2:]
    return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)


def _plain_put(s, kv, q_rope, q, pos, slots):
    ang = pos.double()[:, None] * s["inv_freq"]
    cos, sin = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]
    c = kv[:, :LATENT].float()
    if s["weight"] is not None:
        c = c * torch.rsqrt((c * c).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    rows = torch.cat([c, _turn(kv[:, None, LATENT:], cos, sin, s["inter"])[:, 0]], -1).to(kv.dtype)
    live = slots >= 0
    s["cache"].view(-1, ROW)[slots[live]] = rows[live]
    turned = _turn(q_rope, cos, sin, s["inter"]).to(q.dtype)
    q[..., LATENT:] = torch.where(live[:, None, None], turned, q[..., LATENT:])


def _plain_append(s):
    _plain_put(s, s["kv_new"], s["q_rope"], s["q"], s["positions"], s["slots"])
    return s["q"], s["cache"]


def _plain_append_step(s):
    B, T = s["slots"].shape
    pos = s["ctx"].long()[:, None] - T + torch.arange(T, device="cuda")
    blk = torch.gather(s["tables"].long(), 1, pos.clamp(min=0) // BLOCK)
    s["slots"].copy_(torch.where(pos >= 0, blk * BLOCK + pos % BLOCK, -1))
    n = B * T
    _plain_put(s, s["kv_new"].view(n, ROW), s["q_rope"].flatten(0, 1), s["q"].view(n, *s["q"].shape[2:]), pos.view(-1),
               s["slots"].view(-1))
    return s["q"], s["slots"], s["cache"]


def _plain_attend(s):
    B, T, N, _ = s["q"].shape
    width = s["tables"].shape[1]
    L = width * BLOCK
    ctx = s["ctx"].long()
    rows = s["cache"][s["tables"].clamp(min=0).long()].view(B, L, ROW).float()
    at = torch.arange(L, device="cuda")
    rows.masked_fill_((at >= ctx[:, None])[..., None], 0.0)
    logit = (s["q"].float().view(B, T * N, ROW) * s["scale"]) @ rows.transpose(1, 2)
    seen = ctx[:, None] - T + 1 + torch.arange(T, device="cuda")                     # tokens that new token t sees
    logit = logit.view(B, T, N, L).masked_fill_((at >= seen[..., None])[:, :, None], -math.inf)
    top = logit.amax(-1, keepdim=True)
    w = torch.exp_(logit.sub_(top.clamp(min=-1e30)))
    total = w.sum(-1, keepdim=True)
    out = (w.view(B, T * N, L) @ rows[..., :LATENT]).view(B, T, N, LATENT) / total.clamp(min=1e-30)
    s["out"].copy_(out)
    s["lse"].copy_((top + torch.log(total))[..., 0])
    return s["out"], s["lse"]


def _plain_copies(s, pairs):
    there = pairs[:, 0] >= 0
    src, dst = pairs[there].long().unbind(1)
    for p in s["pools"]:
        p[dst] = p[src]


def _free_ids(refs):
    """The free blocks' ids in ascending order at the front (as many as there are), and their number."""
    free = refs == 0
    rank = torch.where(free, torch.cumsum(free, 0) - 1, refs.numel())
    ids = torch.zeros(refs.numel() + 1, dtype=torch.int64, device="cuda")
    ids[rank] = torch.arange(refs.numel(), device="cuda")
    return ids, free.sum()


def _plain_extend(s):
    s["now"].copy_(s["then"])
    tables, ctx, refs, B = s["tables"], s["ctx"].long(), s["refs"], s["ctx"].numel()
    new, row = s["num_new"].long(), torch.arange(B, device="cuda")
    width = tables.shape[1]
    partial = (new > 0) & (ctx % BLOCK != 0)
    last = torch.gather(tables.long(), 1, (ctx // BLOCK).clamp(max=width - 1)[:, None])[:, 0].clamp(min=0)
    # of the rows that grow into one block the last one keeps it, if no other row holds it
    holders = torch.zeros_like(refs).index_add_(0, last, partial.to(torch.int32))
    keeper = torch.full_like(refs, -1).scatter_reduce_(0, last, torch.where(partial, row, -1).to(torch.int32), "amax")
    cow = partial & ~((refs[last] == holders[last]) & (keeper[last] == row))
    before, after = (ctx + BLOCK - 1) // BLOCK, (ctx + new + BLOCK - 1) // BLOCK
    need = cow.long() + after - before
    upto = torch.cumsum(need, 0)
    ids, count = _free_ids(refs)
    go = (new > 0) & (upto <= count)
    j = torch.arange(width, device="cuda")
    first = torch.where(cow, ctx // BLOCK, before)
    fresh = go[:, None] & (j >= first[:, None]) & (j < after[:, None])
    which = (upto - need)[:, None] + j - first[:, None]
    got = ids[torch.where(fresh, which, 0)]
    moved = go & cow
    s["copies"][:, 0] = torch.where(moved, last, -1)
    s["copies"][:, 1] = torch.where(moved, ids[torch.where(moved, upto - need, 0)], -1)
    tables.copy_(torch.where(fresh, got, tables.long()))
    refs.index_add_(0, got[fresh], torch.ones_like(got[fresh], dtype=torch.int32))
    refs.index_add_(0, last, -moved.to(torch.int32))
    s["ctx"].add_(torch.where(go, new, 0).to(torch.int32))
    _plain_copies(s, s["copies"])
    return s["tables"], s["ctx"], s["refs"], s["copies"], *s["pools"]


def _plain_fork(s):
    s["now"].copy_(s["then"])
    tables, ctx, par = s["tables"], s["ctx"], s["parents"].long()
    held = torch.arange(tables.shape[1], device="cuda") < (ctx[:, None] + BLOCK - 1) // BLOCK
    children = torch.zeros_like(ctx).index_add_(0, par.clamp(min=0), (par >= 0).to(torch.int32))
    s["refs"].index_add_(0, tables[held].long(), (children - 1)[:, None].expand_as(tables)[held])
    s["tables_out"].copy_(torch.where((par >= 0)[:, None] & held[par.clamp(min=0)], tables[par.clamp(min=0)], -1))
    s["ctx_out"].copy_(torch.where(par >= 0, ctx[par.clamp(min=0)], 0))
    return s["tables_out"], s["ctx_out"], s["refs"]


def _plain_compact(s):
    s["now"].copy_(s["then"])
    refs, tables = s["refs"], s["tables"]
    P = refs.numel()
    free, _ = _free_ids(refs)
    down, _ = _free_ids((refs.flip(0) == 0).to(torch.int32))          # used ids in descending order, counted from the end
    used = (refs != 0).sum()
    i = torch.arange(s["moves"].shape[0], device="cuda")
    src, dst = P - 1 - down[i], free[i]
    go = (i < used) & (i < P - used) & (src > dst)
    s["moves"].copy_(torch.where(go[:, None], torch.stack([src, dst], 1), -1))
    s["num_moves"].copy_(go.sum())
    to = torch.arange(P, device="cuda")
    to[src[go]] = dst[go]
    refs[dst[go]] = refs[src[go]]
    refs[src[go]] = 0
    held = torch.arange(tables.shape[1], device="cuda") < (s["ctx"][:, None] + BLOCK - 1) // BLOCK
    tables.copy_(torch.where(held, to[tables.clamp(min=0).long()], tables.long()))
    _plain_copies(s, s["moves"])
    return s["tables"], s["refs"], s["moves"], s["num_moves"], *s["pools"]


_plain = dict(append=_plain_append, append_step=_plain_append_step, attend=_plain_attend, extend=_plain_extend,
              fork=_plain_fork, compact=_plain_compact)
_own = dict(append=_own_append, append_step=_own_append_step, attend=_own_attend, extend=_own_extend, fork=_own_fork,
            compact=_own_compact)


# ------------------------------------------------------------------------------------------- work
def _lengths(c):
    return np.linspace(c["lo"], c["hi"], 257)


def work(case):
    c = case
    op = c["op"]
    if op in ("append", "append_step"):
        n = c["tokens"] if op == "append" else c["B"] * c["T"]
        return dict(bytes=n * 4 * (ROW + c["N"] * ROPE), flops=n * (LATENT * 4 + (c["N"] + 1) * ROPE * 3))
    if op == "attend":
        tokens, q = c["B"] * float(_lengths(c).mean()), c["B"] * c["T"] * c["N"]
        return dict(bytes=tokens * ROW * 2 + q * (2 * ROW + 2 * LATENT + 4),
                    flops=tokens * c["T"] * c["N"] * 2 * (ROW + LATENT))
    blocks = c["B"] * float(np.ceil(_lengths(c) / BLOCK).mean())
    if op == "fork":      # a row's entries read and written, the reference counts of those that change
        return dict(bytes=blocks * 16, flops=blocks)
    size = 2 * BLOCK * c["H"] * (2 * c["K"] if c["K"] else 1) * c["layers"]
    pool = blocks / c["full"]
    if op == "extend":    # the counts read once; new entries, and a share of copies on write
        grown = c["B"] * ((c["new"] + 1) // 2 if c["new"] > 1 else 1) / BLOCK
        return dict(bytes=4 * pool + 8 * grown + c["B"] * (24 + c["shared"] * 0.9 * 2 * size), flops=pool)
    moved = blocks * (1.0 - c["full"])
    return dict(bytes=4 * pool + 8 * blocks + moved * 2 * size, flops=pool)


# ------------------------------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return dict(append=_exact_append, append_step=_exact_append, attend=_exact_attend, extend=_exact_extend,
                fork=_exact_fork, compact=_exact_compact)[case["op"]](s)


def _exact_append(s):
    step = s["op"] == "append_step"
    if step:
        B, T = s["B"], s["T"]
        ctx, tab = s["ctx"].cpu().numpy().astype(np.int64), s["tables"].cpu().numpy().astype(np.int64)
        pos = (ctx[:, None] + np.arange(-T, 0)).reshape(-1)
        slots = np.where(pos >= 0, tab[np.repeat(np.arange(B), T), np.maximum(pos, 0) // 16] * 16 + pos % 16, -1)
    else:
        pos, slots = s["positions"].cpu().numpy().astype(np.int64), s["slots"].cpu().numpy()
    i = np.arange(64)
    pair, mate = (i // 2, i ^ 1) if s["inter"] else (i % 32, (i + 32) % 64)
    sign = np.where((i % 2 == 0) if s["inter"] else (i < 32), -1.0, 1.0)
    ang = torch.from_numpy(pos.astype(np.float64)).cuda()[:, None] * s["inv_freq"][torch.from_numpy(pair).cuda()]
    co, si = torch.cos(ang), torch.sin(ang) * torch.from_numpy(sign).cuda()
    turn = lambda x, c, d: x * c + x[..., torch.from_numpy(mate).cuda()] * d
    live = torch.from_numpy(np.flatnonzero(slots >= 0)).cuda()
    kv = s["kv_new"].reshape(-1, 576).double()
    lat = kv[:, :512]
    if s["weight"] is not None:
        lat = lat / torch.sqrt(lat.pow(2).sum(-1, keepdim=True) / 512 + EPS) * s["weight"].double()
    rows = torch.cat([lat, turn(kv[:, 512:], co, si)], -1)
    cache = s["cache"].double()
    cache.view(-1, 576).index_copy_(0, torch.from_numpy(slots[slots >= 0]).cuda(), rows[live])
    q = s["q"].double()
    flat = q.view(len(pos), -1, 576)
    qr = s["q_rope"].reshape(len(pos), -1, 64).double()
    flat[live, :, 512:] = turn(qr, co[:, None], si[:, None])[live]
    return (q, torch.from_numpy(slots).cuda().view(s["slots"].shape), cache) if step else (q, cache)


def _exact_attend(s):
    B, T, N, _ = s["q"].shape
    out = torch.zeros(B, T, N, 512, dtype=torch.float64, device="cuda")
    lse = torch.full((B, T, N), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["ctx"].tolist()):
        rows = s["cache"][s["tables"][b, :-(-n // 16)].long()].reshape(-1, 576)[:n].double()
        for t in range(T):
            m = n - T + t + 1
            if m > 0:
                z = s["scale"] * (s["q"][b, t].double() @ rows[:m].T)
                lse[b, t] = torch.logsumexp(z, -1)
                out[b, t] = torch.softmax(z, -1) @ rows[:m, :512]
    return out, lse


def _host(s):
    return s["tables"].cpu().numpy().copy(), s["ctx"].cpu().numpy().copy(), s["refs"].cpu().numpy().copy()


def _copied(s, pairs):
    for p in s["pools"]:
        for a, b in pairs:
            p[b] = p[a]
    return s["pools"]


def _exact_extend(s):
    tab, ctx, ref = _host(s)
    copies = np.full((len(ctx), 2), -1, dtype=np.int32)
    free = list(np.flatnonzero(ref == 0)[::-1])
    for b, t in enumerate(s["num_new"].tolist()):
        n = int(ctx[b])
        if t == 0:
            continue
        cow = n % 16 != 0 and ref[tab[b, n // 16]] > 1
        nb = -(-(n + t) // 16)
        if cow + nb - -(-n // 16) > len(free):
            break
        if cow:
            copies[b] = tab[b, n // 16], free.pop()
            ref[copies[b, 0]] -= 1
            tab[b, n // 16], ref[copies[b, 1]] = copies[b, 1], 1
        for j in range(-(-n // 16), nb):
            tab[b, j] = free.pop()
            ref[tab[b, j]] = 1
        ctx[b] = n + t
    pools = _copied(s, [p for p in copies.tolist() if p[0] >= 0])
    return (*(torch.from_numpy(x) for x in (tab, ctx, ref, copies)), *pools)


def _exact_fork(s):
    tab, ctx, ref = _host(s)
    out, lens = np.full_like(tab, -1), np.zeros_like(ctx)
    for b in range(len(ctx)):
        np.subtract.at(ref, tab[b, :-(-int(ctx[b]) // 16)], 1)
    for b, p in enumerate(s["parents"].tolist()):
        if p >= 0:
            nb = -(-int(ctx[p]) // 16)
            out[b, :nb], lens[b] = tab[p, :nb], ctx[p]
            np.add.at(ref, tab[p, :nb], 1)
    return tuple(torch.from_numpy(x) for x in (out, lens, ref))


def _exact_compact(s):
    tab, ctx, ref = _host(s)
    moves = np.full(s["moves"].shape, -1, dtype=np.int32)
    to, n, lo, hi = {}, 0, 0, len(ref) - 1
    while n < len(moves):
        while lo < len(ref) and ref[lo] != 0:
            lo += 1
        while hi >= 0 and ref[hi] == 0:
            hi -= 1
        if lo >= hi:
            break
        moves[n], to[hi] = (hi, lo), lo
        ref[lo], ref[hi] = ref[hi], 0
        n += 1
    for b in range(len(ctx)):
        for j in range(-(-int(ctx[b]) // 16)):
            tab[b, j] = to.get(int(tab[b, j]), tab[b, j])
    pools = _copied(s, moves[:n].tolist())
    return (*(torch.from_numpy(x) for x in (tab, ref, moves, np.array([n], dtype=np.int32))), *pools)
