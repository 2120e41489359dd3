"""What is measured of the operators around paged decode attention: the rotating append, the key bounds of
a block, the choice of blocks, attention over the chosen blocks, and the verification of drafted tokens.

Each operator in its plain form (elementary torch operations) and, with ``own`` true, as calls of the
library.  ``listed()`` holds the measured cases, ``draw()`` gives more of the same ranges.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16
E4M3_MAX = 448.0


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # One decode step of a ragged batch of 64 sequences (32 query / 8 KV heads of 128): the
        # batch's newest tokens are rotated and appended; a call this small is latency.
        dict(name="rope_step_b64", op="rope_step", B=64, T=1, N=32, K=8, H=128, R=128, inter=False,
             lo=512, hi=8192, kv="bf16"),
        # A prefill chunk of 8,192 prompt tokens of eight sequences, somewhere in long contexts.
        dict(name="rope_prompt_8k", op="rope", tokens=8192, seqs=8, N=32, K=8, H=128, R=128,
             inter=False, far=131072, kv="bf16"),
        # An odd number of prompt tokens, as many KV heads as query heads, half of each head
        # rotated in neighbouring pairs, into an e4m3 cache with a scale per (block, head).
        dict(name="rope_prompt_e4m3", op="rope", tokens=5001, seqs=7, N=40, K=40, H=128, R=64,
             inter=True, far=4096, kv="e4m3_block"),
        # After a prefill: the bounds of every block of 16 prompts.
        dict(name="bounds_prompt_b16", op="bounds", B=16, K=8, H=128, lo=512, hi=8192, new=0, kv="bf16"),
        # In a decode step over an e4m3 cache: the bounds of each sequence's newest block.
        dict(name="bounds_step_e4m3", op="bounds", B=64, K=8, H=128, lo=512, hi=8192, new=1, kv="e4m3_head"),
        # One sequence of 32K tokens: 64 of its 2,048 blocks (the latency end).
        dict(name="select_b1_32k", op="select", B=1, N=32, K=8, H=128, lo=32768, hi=32768, M=64, first=1, last=2),
        # A batch of 64 long sequences, 128 blocks each.
        dict(name="select_b64_32k", op="select", B=64, N=32, K=8, H=128, lo=8192, hi=32768, M=128, first=1, last=2),
        # One sequence of 128K tokens attending to 128 chosen blocks.
        dict(name="attend_b1_128k", op="attend", B=1, N=32, K=8, H=128, lo=131072, hi=131072, M=128, kv="bf16"),
        # A batch of 64 ragged sequences, some of them shorter than the 128 blocks they may choose.
        dict(name="attend_b64", op="attend", B=64, N=32, K=8, H=128, lo=512, hi=8192, M=128, kv="bf16"),
        # 20 sequences, eight query heads a KV head, an e4m3 cache with a scale per (block, head).
        dict(name="attend_e4m3_b20", op="attend", B=20, N=64, K=8, H=128, lo=16008, hi=32520, M=250,
             kv="e4m3_block"),
        # One sequence, three drafted tokens, a small vocabulary, 16-bit probabilities.
        dict(name="verify_b1", op="verify", B=1, T=3, V=32000, ragged=False, onehot=False, dtype="bf16"),
        # A batch of 64, four drafted tokens, a large vocabulary, 32-bit probabilities.
        dict(name="verify_b64", op="verify", B=64, T=4, V=128256, ragged=False, onehot=False, dtype="fp32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    K = rng.choice([1, 2, 4, 5, 8, 10])
    return K * rng.choice([1, 2, 4, 8]), K


def draw(rng):
    op = rng.choice(["rope", "rope_step", "bounds", "select", "attend", "verify"])
    N, K = _heads(rng)
    H = rng.choice([64, 128, 128])
    kv = rng.choice(["bf16", "e4m3_head", "e4m3_block"]) if H == 128 else "bf16"
    if op == "rope":
        return dict(op=op, tokens=_log(rng, 1, 8000), seqs=rng.randint(1, 9), N=N, K=K, H=H,
                    R=rng.choice([r for r in (16, 32, 64, 96, 128) if r <= H]), inter=rng.random() < 0.5,
                    far=_log(rng, 16, 1000000), kv=kv)
    if op == "rope_step":
        return dict(op=op, B=_log(rng, 1, 200), T=rng.choice([1, 1, 2, 3, 5, 8]), N=N, K=K, H=H,
                    R=rng.choice([r for r in (32, 64, 128) if r <= H]), inter=rng.random() < 0.5, lo=1,
                    hi=_log(rng, 16, 2500), kv=kv)
    if op == "bounds":
        return dict(op=op, B=_log(rng, 1, 60), K=K, H=H, lo=0, hi=_log(rng, 17, 8000),
                    new=rng.choice([0, 1, 1, 4, 33]), kv=kv)
    if op == "verify":
        return dict(op=op, B=_log(rng, 1, 60), T=rng.randint(1, 8), V=_log(rng, 100, 120000),
                    ragged=rng.random() < 0.5, onehot=rng.random() < 0.3, dtype=rng.choice(["fp32", "bf16"]))
    M = _log(rng, 4, 250)
    B = _log(rng, 1, 40)
    hi = _log(rng, 64, 30000)
    if op == "select":
        first = rng.choice([0, 1, 2])
        return dict(op=op, B=B, N=N, K=K, H=H, lo=min(hi, rng.choice([0, 1, 40])), hi=hi, M=M, first=first,
                    last=rng.randint(0 if first else 1, 2))
    return dict(op=op, B=B, N=N, K=K, H=H, lo=min(hi, rng.choice([0, 1, 40])), hi=hi, M=M, kv=kv)


# ----------------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _lengths(seed, B, lo, hi):
    return np.random.default_rng(seed).integers(lo, hi + 1, size=B).astype(np.int32)


def _tables(seed, ctx, longest):
    """Block tables over a shuffled pool with room for every sequence at its longest: int32
    [B, most blocks], -1 behind a sequence's last block."""
    nb = -(-ctx.astype(np.int64) // BLOCK)
    width = max(1, -(-longest // BLOCK))
    pool = len(ctx) * width + 3
    order = np.random.default_rng(seed + 1).permutation(pool).astype(np.int32)
    tables = np.full((len(ctx), width), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(nb):
        tables[b, :n] = order[at:at + n]
        at += int(n)
    return torch.from_numpy(tables).cuda(), pool


def _inv_freq(R):
    return torch.tensor([500000.0 ** (-2.0 * j / R) for j in range(R // 2)], dtype=torch.float64, device="cuda")


def _scales(g, kv, pool, K):
    """Scales of an e4m3 cache that holds values of about unit variance, one per head or per (block, head)."""
    shape = (pool, K) if kv == "e4m3_block" else (K,)
    return (3.0 + 3.0 * torch.rand(*shape, generator=g, device="cuda")) / E4M3_MAX


def _codes(x, scale):
    return (x.float() / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)


def _pool(g, kv, pool, K, H):
    """One pool of keys or values: bf16, or e4m3 codes of normal values in units of the scale."""
    x = _randn(g, pool, BLOCK, K, H)
    return x if kv == "bf16" else _codes(x, 4.5 / E4M3_MAX)


def prepare(case, seed):
    c, g = case, _gen(seed)
    op, kv = c["op"], c.get("kv", "bf16")
    s = dict(c)
    s["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if op in ("rope", "rope_step"):
        N, K, H = c["N"], c["K"], c["H"]
        if op == "rope":
            n, lead = c["tokens"], (c["tokens"],)
            # consecutive runs of tokens, each starting somewhere below `far`
            r = np.random.default_rng(seed)
            run = np.sort(r.integers(0, c["seqs"], size=n))
            start = r.integers(0, c["far"], size=c["seqs"])
            first = np.searchsorted(run, np.arange(c["seqs"]))
            s["positions"] = torch.from_numpy((start[run] + np.arange(n) - first[run]).astype(np.int32)).cuda()
            pool = -(-n // BLOCK) + 2
            slots = r.permutation(pool * BLOCK)[:n].astype(np.int64)
            if n > 4:
                slots[r.integers(0, n, size=2)] = -1   # padding rows of the batch
            s["slots"] = torch.from_numpy(slots).cuda()
        else:
            lead = (c["B"], c["T"])
            ctx = np.maximum(_lengths(seed, c["B"], c["lo"], c["hi"]), c["T"])
            s["tables"], pool = _tables(seed, ctx, max(c["hi"], c["T"]))
            s["ctx"] = torch.from_numpy(ctx.astype(np.int32)).cuda()
            s["slots"] = torch.empty(lead, dtype=torch.int64, device="cuda")
        s["q"], s["k_new"], s["v_new"] = _randn(g, *lead, N, H), _randn(g, *lead, K, H), _randn(g, *lead, K, H)
        s["q_out"] = s["q"].clone()
        s["inv_freq"] = _inv_freq(c["R"])
        kind = torch.bfloat16 if kv == "bf16" else torch.uint8
        s["k_cache"] = torch.zeros(pool, BLOCK, K, H, dtype=kind, device="cuda")
        s["v_cache"] = torch.zeros_like(s["k_cache"])
        if kv != "bf16":
            s["k_scale"], s["v_scale"] = _scales(g, kv, pool, K), _scales(g, kv, pool, K)
    elif op == "verify":
        B, T, V = c["B"], c["T"], c["V"]
        dt = torch.float32 if c["dtype"] == "fp32" else torch.bfloat16
        # a draft model's logits are its target's with an error
        logits = 2.5 * torch.randn(B, T + 1, V, generator=g, device="cuda")
        near = logits[:, :T] + 0.5 * torch.randn(B, T, V, generator=g, device="cuda")
        s["p"] = torch.softmax(logits, -1).to(dt)
        q = torch.softmax(near, -1)
        pick = (near - torch.log(-torch.log(torch.rand(B, T, V, generator=g, device="cuda").clamp(1e-12, 1 - 1e-7)))).argmax(-1)
        s["q"] = None if c["onehot"] else q.to(dt)
        if c["onehot"]:                     # a draft without probabilities: its likeliest token
            pick = near.argmax(-1)
        s["tokens"] = pick.to(torch.int32)
        s["u"] = torch.rand(B, T, generator=g, device="cuda")
        s["r"] = torch.rand(B, generator=g, device="cuda")
        s["lens"] = torch.randint(0, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32) if c["ragged"] else None
        s["ctx"] = torch.randint(T + 1, 9000, (B,), generator=g, device="cuda", dtype=torch.int32)
        s["accepted"] = torch.empty(B, dtype=torch.int32, device="cuda")
        s["out"] = torch.empty(B, T + 1, dtype=torch.int32, device="cuda")
        s["ctx_out"] = torch.empty(B, dtype=torch.int32, device="cuda")
        if own:
            import paged_kv_decode_slot_gb300 as pkv
            s["ws"] = torch.zeros(pkv.pkv_verify_workspace_bytes(B, V), dtype=torch.uint8, device="cuda")
    else:
        K, H, B = c["K"], c["H"], c["B"]
        ctx = _lengths(seed, B, c["lo"], c["hi"])
        s["tables"], pool = _tables(seed, ctx, c["hi"])
        s["ctx"] = torch.from_numpy(ctx).cuda()
        width = s["tables"].shape[1]
        if op == "bounds":
            s["k_cache"] = _pool(g, kv, pool, K, H)
            if kv != "bf16":
                s["k_scale"] = _scales(g, kv, pool, K)
            s["new"] = c["new"] or width * BLOCK
            s["bounds"] = torch.zeros(pool, K, 2, H, dtype=torch.bfloat16, device="cuda")
        elif op == "select":
            # a block's keys scatter by about one around a centre of their own
            s["q"] = _randn(g, B, c["N"], H)
            centre, reach = 0.7 * _randn(g, pool, K, H), 1.2 + 0.3 * _randn(g, pool, K, H)
            s["bounds"] = torch.stack([centre - reach.abs(), centre + reach.abs()], 2)
            s["selected"] = torch.empty(B, K, c["M"], dtype=torch.int32, device="cuda")
            if own:
                import paged_kv_decode_slot_gb300 as pkv
                s["ws"] = torch.zeros(pkv.pkv_select_workspace_bytes(B, K, width), dtype=torch.uint8, device="cuda")
        else:
            N, M = c["N"], c["M"]
            s["q"] = _randn(g, B, N, H)
            s["k_cache"], s["v_cache"] = _pool(g, kv, pool, K, H), _pool(g, kv, pool, K, H)
            if kv != "bf16":
                s["k_scale"], s["v_scale"] = _scales(g, kv, pool, K), _scales(g, kv, pool, K)
            s["scale"] = 1.0 / math.sqrt(H)
            # each (sequence, KV head) has chosen M of its blocks (all, where it has no more), the last among them
            nb = ((s["ctx"] + BLOCK - 1) // BLOCK).long()[:, None, None]
            j = torch.arange(width, device="cuda")
            key = torch.rand(B, K, width, generator=g, device="cuda") + (j == nb - 1) - 4.0 * (j >= nb)
            if width < M:
                key = torch.nn.functional.pad(key, (0, M - width), value=-4.0)
            best = key.topk(M, -1)
            s["selected"] = torch.where(best.values >= 0, best.indices, 1 << 30).sort(-1).values.to(torch.int32)
            s["selected"][s["selected"] == 1 << 30] = -1
            s["out"] = torch.empty(B, N, H, dtype=torch.bfloat16, device="cuda")
            s["lse"] = torch.empty(B, N, dtype=torch.float32, device="cuda")
            if own:
                import paged_kv_decode_slot_gb300 as pkv
                from paged_kv_decode_slot_gb300.step import plan_blocks_attention
                plan = plan_blocks_attention(B, K, M, torch.cuda.get_device_properties(0).multi_processor_count)
                s["pb"], s["parts"] = plan.partition_blocks, plan.max_partitions
                s["ws"] = torch.zeros(pkv.pkv_splitk_workspace_bytes(B, N, H, s["parts"]), dtype=torch.uint8,
                                      device="cuda")
    return s


# ---------------------------------------------------------------------------------- the operators
def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _values(codes):
    """An e4m3 pool as the values of its codes (in units of the scales)."""
    return codes.view(torch.float8_e4m3fn) if codes.dtype == torch.uint8 else codes


def _own_rope(s):
    import paged_kv_decode_slot_gb300 as pkv
    tail = dict(interleaved=s["inter"], err_flag=s["err"])
    if s["kv"] == "bf16":
        pkv.check(pkv.pkv_rope_append(s["q"], s["k_new"], s["v_new"], s["positions"], s["inv_freq"], s["slots"],
                                      s["k_cache"], s["v_cache"], s["q_out"], **tail))
    else:
        pkv.check(pkv.pkv_rope_append_fp8(s["q"], s["k_new"], s["v_new"], s["positions"], s["inv_freq"],
                                          s["k_scale"], s["v_scale"], s["slots"], s["k_cache"], s["v_cache"],
                                          s["q_out"], **tail))
    return s["q_out"], _values(s["k_cache"]), _values(s["v_cache"])


def _own_rope_step(s):
    import paged_kv_decode_slot_gb300 as pkv
    tail = dict(interleaved=s["inter"], err_flag=s["err"])
    if s["kv"] == "bf16":
        pkv.check(pkv.pkv_rope_append_multi(s["q"], s["k_new"], s["v_new"], s["tables"], s["ctx"], s["inv_freq"],
                                            s["k_cache"], s["v_cache"], s["q_out"], s["slots"], **tail))
    else:
        pkv.check(pkv.pkv_rope_append_multi_fp8(s["q"], s["k_new"], s["v_new"], s["tables"], s["ctx"],
                                                s["inv_freq"], s["k_scale"], s["v_scale"], s["k_cache"],
                                                s["v_cache"], s["q_out"], s["slots"], **tail))
    return s["q_out"], s["slots"], _values(s["k_cache"]), _values(s["v_cache"])


def _own_bounds(s):
    import paged_kv_decode_slot_gb300 as pkv
    if s["kv"] == "bf16":
        pkv.check(pkv.pkv_key_bounds(s["k_cache"], s["tables"], s["ctx"], s["new"], s["bounds"], s["err"]))
    else:
        pkv.check(pkv.pkv_key_bounds_fp8(s["k_cache"], s["k_scale"], s["tables"], s["ctx"], s["new"], s["bounds"],
                                         s["err"]))
    return s["bounds"]


def _own_select(s):
    import paged_kv_decode_slot_gb300 as pkv
    pkv.check(pkv.pkv_select_blocks(s["q"], s["bounds"], s["tables"], s["ctx"], s["selected"], s["ws"],
                                    first_blocks=s["first"], last_blocks=s["last"], err_flag=s["err"]))
    return s["selected"]


def _own_attend(s):
    import paged_kv_decode_slot_gb300 as pkv
    if s["kv"] == "bf16":
        pkv.check(pkv.pkv_decode_attn_blocks(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["ctx"],
                                             s["selected"], s["scale"], s["out"], s["lse"], s["pb"], s["parts"],
                                             s["ws"], s["err"]))
    else:
        pkv.check(pkv.pkv_decode_attn_blocks_fp8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                                 s["tables"], s["ctx"], s["selected"], s["scale"], s["out"],
                                                 s["lse"], s["pb"], s["parts"], s["ws"], s["err"]))
    return s["out"], s["lse"]


def _own_verify(s):
    import paged_kv_decode_slot_gb300 as pkv
    pkv.check(pkv.pkv_verify_draft(s["p"], s["q"], s["tokens"], s["u"], s["r"], s["accepted"], s["out"], s["ws"],
                                   draft_lens=s["lens"], context_lens=s["ctx"], context_lens_out=s["ctx_out"],
                                   err_flag=s["err"]))
    return s["accepted"], s["out"], s["ctx_out"]


# the plain forms ------------------------------------------------------------------------------------
def _rotate(x, cos, sin, R, inter):
    """x [..., heads, H] rotated by the angles whose cosines and sines are [..., 1, R / 2], in 32 bits."""
    x = x.float()
    if inter:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, x[..., R:]], -1)


def _plain_put(s, q, k, v, pos, slots):
    """Rotated q, and the rotated keys and the values written behind their slots; -1 leaves a row alone."""
    ang = pos.double()[:, None] * s["inv_freq"]
    cos, sin = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]
    live = slots >= 0
    s["q_out"].view(q.shape).copy_(torch.where(live[:, None, None], _rotate(q, cos, sin, s["R"], s["inter"]).to(q.dtype), q))
    at = slots[live]
    for new, pool, scale in ((_rotate(k, cos, sin, s["R"], s["inter"]), s["k_cache"], s.get("k_scale")),
                             (v.float(), s["v_cache"], s.get("v_scale"))):
        new = new[live]
        if scale is None:
            rows = new.to(pool.dtype)
        else:
            rows = _codes(new, (scale[at // BLOCK] if scale.dim() == 2 else scale[None])[..., None])
        pool.view(-1, *pool.shape[2:])[at] = rows


def _plain_rope(s):
    _plain_put(s, s["q"], s["k_new"], s["v_new"], s["positions"], s["slots"])
    return s["q_out"], _values(s["k_cache"]), _values(s["v_cache"])


def _plain_rope_step(s):
    B, T = s["slots"].shape
    pos = (s["ctx"].long()[:, None] - T + torch.arange(T, device="cuda"))
    blk = torch.gather(s["tables"].long(), 1, pos.clamp(min=0) // BLOCK)
    s["slots"].copy_(torch.where(pos >= 0, blk * BLOCK + pos % BLOCK, -1))
    flat = [s[n].view(B * T, *s[n].shape[2:]) for n in ("q", "k_new", "v_new")]
    _plain_put(s, *flat, pos.view(-1), s["slots"].view(-1))
    return s["q_out"], s["slots"], _values(s["k_cache"]), _values(s["v_cache"])


def _plain_bounds(s):
    ctx, width = s["ctx"].long(), s["tables"].shape[1]
    j = torch.arange(width, device="cuda")
    hit = (j * BLOCK < ctx[:, None]) & ((j + 1) * BLOCK > ctx[:, None] - s["new"])
    seq, blk = hit.nonzero(as_tuple=True)
    phys = s["tables"][seq, blk].long()
    keys = _values(s["k_cache"][phys]).float()                               # [n, 16, K, H]
    if s["kv"] != "bf16":
        sc = s["k_scale"][phys][:, None, :, None] if s["kv"] == "e4m3_block" else s["k_scale"][:, None]
        keys = keys * sc
    there = (blk[:, None] * BLOCK + torch.arange(BLOCK, device="cuda") < ctx[seq][:, None])[..., None, None]
    lo = keys.masked_fill(~there, math.inf).amin(1)
    hi = keys.masked_fill(~there, -math.inf).amax(1)
    s["bounds"][phys] = torch.stack([lo, hi], 2).to(torch.bfloat16)
    return s["bounds"]


def _plain_select(s):
    (B, N, H), (K, M) = s["q"].shape, s["selected"].shape[1:]
    width = s["tables"].shape[1]
    nb = ((s["ctx"].long() + BLOCK - 1) // BLOCK)[:, None, None]
    j = torch.arange(width, device="cuda")
    # in 64 bits: which of two near scores is the larger one decides
    bounds = s["bounds"][s["tables"].clamp(min=0).long()].double()           # [B, width, K, 2, H]
    q = s["q"].double().view(B, K, N // K, H)
    score = q.clamp(max=0) @ bounds[:, :, :, 0].permute(0, 2, 3, 1) + q.clamp(min=0) @ bounds[:, :, :, 1].permute(0, 2, 3, 1)
    score = score.amax(2)
    always = (j < s["first"]) | (j >= nb - s["last"])
    score = torch.where(j >= nb, -math.inf, torch.where(always, math.inf, score))
    order = score.sort(dim=-1, descending=True, stable=True).indices[..., :M]
    order = torch.where(order < nb, order, 1 << 30).sort(-1).values
    s["selected"].fill_(-1)
    s["selected"][..., :order.shape[-1]] = torch.where(order < nb, order, -1).to(torch.int32)
    return s["selected"]


def _plain_attend(s):
    (B, N, H), (K, M) = s["q"].shape, s["selected"].shape[1:]
    sel, ctx = s["selected"].long(), s["ctx"].long()
    phys = torch.gather(s["tables"].long()[:, None].expand(B, K, -1), 2, sel.clamp(min=0)).clamp(min=0)
    head = torch.arange(K, device="cuda")[None, :, None]
    k, v = (_values(s[n][phys, :, head]).float() for n in ("k_cache", "v_cache"))     # [B, K, M, 16, H]
    if s["kv"] != "bf16":
        ks, vs = ((s[n][phys, head] if s["kv"] == "e4m3_block" else s[n][None, :, None]) for n in ("k_scale", "v_scale"))
        k, v = k * ks[..., None, None], v * vs[..., None, None]
    at = sel[..., None] * BLOCK + torch.arange(BLOCK, device="cuda")
    there = ((sel >= 0)[..., None] & (at < ctx[:, None, None, None])).reshape(B, K, 1, M * BLOCK)
    q = s["q"].float().view(B, K, N // K, H) * s["scale"]
    logit = (q @ k.reshape(B, K, M * BLOCK, H).transpose(-1, -2)).masked_fill(~there, -math.inf)
    top = logit.amax(-1, keepdim=True)
    w = torch.exp(logit - top.clamp(min=-1e30))
    total = w.sum(-1, keepdim=True)
    v = v.reshape(B, K, M * BLOCK, H).masked_fill(~there.transpose(-1, -2), 0.0)
    out = (w @ v) / total.clamp(min=1e-30)
    s["out"].copy_(out.view(B, N, H))
    s["lse"].copy_((top + torch.log(total)).view(B, N))
    return s["out"], s["lse"]


def _plain_verify(s):
    p, q, tok = s["p"], s["q"], s["tokens"].long()
    B, T = tok.shape
    rows = torch.arange(B, device="cuda")
    lens = s["lens"].long() if s["lens"] is not None else torch.full((B,), T, device="cuda")
    # products and running sums in 64 bits: a draw next to a border falls on its own side of it
    pt = torch.gather(p[:, :T], 2, tok[..., None])[..., 0].double()
    qt = torch.gather(q, 2, tok[..., None])[..., 0].double() if q is not None else torch.ones_like(pt)
    ok = (s["u"].double() * qt < pt) & (torch.arange(T, device="cuda") < lens[:, None])
    n = ok.long().cumprod(-1).sum(-1)
    refused = n < lens
    rest = p[rows, n].double()
    at = n.clamp(max=T - 1)
    if q is not None:
        other = q[rows, at].double()
    else:
        other = torch.zeros_like(rest).scatter_(1, tok[rows, at][:, None], 1.0)
    rest = torch.where(refused[:, None], (rest - other).clamp(min=0.0), rest)
    run_ = rest.cumsum(-1)
    new = (run_ > s["r"].double()[:, None] * run_[:, -1:]).int().argmax(-1)
    i = torch.arange(T + 1, device="cuda")
    drafted = torch.nn.functional.pad(tok, (0, 1))
    out = torch.where(i < n[:, None], drafted, torch.where(i == n[:, None], new[:, None], -1))
    s["accepted"].copy_(n)
    s["out"].copy_(out)
    s["ctx_out"].copy_(s["ctx"] - lens + n)
    return s["accepted"], s["out"], s["ctx_out"]


_plain = dict(rope=_plain_rope, rope_step=_plain_rope_step, bounds=_plain_bounds, select=_plain_select,
              attend=_plain_attend, verify=_plain_verify)
_own = dict(rope=_own_rope, rope_step=_own_rope_step, bounds=_own_bounds, select=_own_select, attend=_own_attend,
            verify=_own_verify)


# ------------------------------------------------------------------------------------------- work
def _mean_blocks(c, most):
    """Expected min(blocks, most) of a sequence whose length is uniform between lo and hi."""
    lo, hi = c["lo"], c["hi"]
    n = np.unique(np.linspace(lo, hi, 513).astype(np.int64))
    return float(np.minimum(-(-n // BLOCK), most).mean())


def work(case):
    c = case
    op, es = c["op"], 1 if c.get("kv", "bf16") != "bf16" else 2
    if op in ("rope", "rope_step"):
        n = c["tokens"] if op == "rope" else c["B"] * c["T"]
        heads = c["N"] + c["K"]
        return dict(bytes=n * c["H"] * (2 * (c["N"] + 2 * c["K"]) + 2 * c["N"] + 2 * c["K"] * es),
                    flops=n * heads * c["R"] * 3)
    if op == "bounds":
        most = 1 << 30 if c["new"] == 0 else 1 + (c["new"] - 1) / BLOCK
        blocks = c["B"] * min(_mean_blocks(c, 1 << 30), most)
        return dict(bytes=blocks * c["K"] * c["H"] * (BLOCK * es + 4), flops=blocks * BLOCK * c["K"] * c["H"] * 2)
    if op == "select":
        # a sequence with no more blocks than may be chosen needs none of their bounds
        n = np.unique(np.linspace(c["lo"], c["hi"], 513).astype(np.int64))
        nb = -(-n // BLOCK)
        scored = c["B"] * float(np.where(nb > c["M"], nb - c["first"] - c["last"], 0).mean())
        return dict(bytes=scored * (c["K"] * c["H"] * 4 + 4) + c["B"] * (c["N"] * c["H"] * 2 + c["K"] * c["M"] * 4),
                    flops=scored * c["N"] * c["H"] * 4)
    if op == "attend":
        got = c["B"] * _mean_blocks(c, c["M"]) * c["K"]
        return dict(bytes=got * (2 * BLOCK * c["H"] * es + 8) + c["B"] * c["N"] * (c["H"] * 4 + 4),
                    flops=got * BLOCK * c["H"] * 4 * (c["N"] // c["K"]))
    es = 4 if c["dtype"] == "fp32" else 2
    # the row of the target's probabilities, and the draft's beside it where a token was refused (about two in three)
    rows = 1.0 if c["onehot"] else 1.67
    return dict(bytes=c["B"] * (rows * c["V"] * es + c["T"] * 16), flops=c["B"] * c["V"] * 4)


# ------------------------------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return dict(rope=_exact_rope, rope_step=_exact_rope, bounds=_exact_bounds, select=_exact_select,
                attend=_exact_attend, verify=_exact_verify)[case["op"]](s)


def _pool_f64(s, name):
    """[pool, 16, K, H] float64 values of a pool's codes without their scales, on the host."""
    x = s[name]
    return (x.view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x).double()


def _exact_rope(s):
    step = s["op"] == "rope_step"
    H, R = s["H"], s["R"]
    if step:
        B, T = s["B"], s["T"]
        ctx, tab = s["ctx"].cpu().numpy().astype(np.int64), s["tables"].cpu().numpy().astype(np.int64)
        pos = (ctx[:, None] + np.arange(-T, 0)).reshape(-1)
        slots = np.where(pos >= 0, tab[np.repeat(np.arange(B), T), np.maximum(pos, 0) // 16] * 16 + pos % 16, -1)
    else:
        pos, slots = s["positions"].cpu().numpy().astype(np.int64), s["slots"].cpu().numpy()
    half = R // 2
    i = np.arange(R)
    pair = i // 2 if s["inter"] else i % half
    mate = (i ^ 1) if s["inter"] else (i + half) % R
    sign = np.where((i % 2 == 0) if s["inter"] else (i < half), -1.0, 1.0)
    ang = torch.from_numpy(pos.astype(np.float64)).cuda()[:, None] * s["inv_freq"][torch.from_numpy(pair).cuda()]
    co, si = torch.cos(ang)[:, None], (torch.sin(ang) * torch.from_numpy(sign).cuda())[:, None]
    live = torch.from_numpy(slots >= 0).cuda()

    def turn(x):
        x = x.reshape(-1, x.shape[-2], H).double()
        y = x.clone()
        y[..., :R] = x[..., :R] * co + x[..., torch.from_numpy(mate).cuda()] * si
        return x, y
    q0, q1 = turn(s["q"])
    q = torch.where(live[:, None, None], q1, q0).view(s["q"].shape)
    at = torch.from_numpy(slots[slots >= 0]).cuda()
    pools = []
    for name, rows in (("k", turn(s["k_new"])[1]), ("v", turn(s["v_new"])[0])):
        pool = _pool_f64(s, name + "_cache")
        rows = rows[live]
        if s["kv"] != "bf16":
            sc = s[name + "_scale"].double()
            rows = (rows / (sc[at // 16] if sc.dim() == 2 else sc[None])[..., None]).clamp(-E4M3_MAX, E4M3_MAX)
        pool.view(-1, *pool.shape[2:]).index_copy_(0, at, rows)
        pools.append(pool)
    return (q, torch.from_numpy(slots).cuda().view(s["slots"].shape), *pools) if step else (q, *pools)


def _exact_bounds(s):
    pool, out = _pool_f64(s, "k_cache"), s["bounds"].double()
    if s["kv"] != "bf16":
        sc = s["k_scale"].double()
        pool *= sc[:, None, :, None] if sc.dim() == 2 else sc[:, None]
    tab = s["tables"].cpu().numpy()
    for b, n in enumerate(s["ctx"].tolist()):
        for j in range(max(0, n - s["new"]) // 16, -(-n // 16)):
            rows = pool[int(tab[b, j]), :min(16, n - 16 * j)]
            out[int(tab[b, j])] = torch.stack([rows.min(0).values, rows.max(0).values], 1)
    return out


def _exact_select(s):
    B, N, H = s["q"].shape
    K, M = s["selected"].shape[1:]
    out = np.full((B, K, M), -1, dtype=np.int32)
    for b, n in enumerate(s["ctx"].tolist()):
        nb = -(-n // 16)
        if nb <= M:
            out[b, :, :nb] = np.arange(nb)
            continue
        box = s["bounds"][s["tables"][b, :nb].long()].double()                # [nb, K, 2, H]
        for kv in range(K):
            q = s["q"][b, kv * (N // K):(kv + 1) * (N // K)].double()
            sc = torch.maximum(q[:, None] * box[:, kv, 0], q[:, None] * box[:, kv, 1]).sum(-1).amax(0).cpu().numpy()
            keep = list(range(s["first"])) + list(range(nb - s["last"], nb))
            mid = np.arange(s["first"], nb - s["last"])
            best = mid[np.lexsort((mid, -sc[mid]))][:M - len(keep)]
            out[b, kv] = np.sort(np.concatenate([np.array(keep, dtype=np.int64), best]))
    return torch.from_numpy(out)


def _exact_attend(s):
    B, N, H = s["q"].shape
    K = s["selected"].shape[1]
    G = N // K
    out = torch.zeros(B, N, H, dtype=torch.float64)
    lse = torch.full((B, N), -math.inf, dtype=torch.float64)
    for b, n in enumerate(s["ctx"].tolist()):
        for kv in range(K):
            sel = [j for j in s["selected"][b, kv].tolist() if j >= 0]
            if not sel or n == 0:
                continue
            at = s["tables"][b, sel].long()
            k, v = (_pool_f64({"x": s[x][at, :, kv]}, "x") for x in ("k_cache", "v_cache"))
            if s["kv"] != "bf16":
                for x, name in ((k, "k_scale"), (v, "v_scale")):
                    sc = s[name].double()
                    x *= sc[at, kv][:, None, None] if sc.dim() == 2 else sc[kv]
            last = n - 16 * torch.tensor(sel, device="cuda")[:, None]
            live = (torch.arange(16, device="cuda") < last).reshape(-1)
            k, v = k.reshape(-1, H)[live], v.reshape(-1, H)[live]
            z = s["scale"] * (s["q"][b, kv * G:(kv + 1) * G].double() @ k.T)
            lse[b, kv * G:(kv + 1) * G] = torch.logsumexp(z, -1).cpu()
            out[b, kv * G:(kv + 1) * G] = (torch.softmax(z, -1) @ v).cpu()
    return out, lse


def _exact_verify(s):
    B, T = s["tokens"].shape
    acc, out, ctx = np.zeros(B, np.int32), np.full((B, T + 1), -1, np.int32), s["ctx"].cpu().numpy().copy()
    tok, u, r = s["tokens"].cpu().numpy(), s["u"].double().cpu().numpy(), s["r"].double().cpu().numpy()
    for b in range(B):
        m = T if s["lens"] is None else int(s["lens"][b])
        t = 0
        while t < m:
            x = int(tok[b, t])
            if u[b, t] * (1.0 if s["q"] is None else float(s["q"][b, t, x])) >= float(s["p"][b, t, x]):
                break
            out[b, t] = x
            t += 1
        left = s["p"][b, t].double().cpu().numpy().copy()
        if t < m:
            if s["q"] is None:
                left[tok[b, t]] -= 1.0
            else:
                left -= s["q"][b, t].double().cpu().numpy()
            left = np.maximum(left, 0.0)
        run_ = np.cumsum(left)
        out[b, t] = int(np.argmax(run_ > r[b] * run_[-1]))
        acc[b], ctx[b] = t, ctx[b] - m + t
    return torch.from_numpy(acc), torch.from_numpy(out), torch.from_numpy(ctx)
