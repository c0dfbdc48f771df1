"""Cases of the 4-bit cache operators and of the step preparation around them.

Four operators, each with its plain form in elementary torch operations, its
call through the package (where `own` is true) and its definition in 64 bits:

* store   -- a chunk's K/V rows written into a 4-bit paged cache, and the
             written blocks read back as bf16 blocks;
* decode  -- single-query attention over a 4-bit paged cache;
* rope    -- RMS norm of every query and key head, position rotation, and the
             cache write of K and V, from a fused projection;
* batch   -- block tables, lengths, positions and slots of a ragged batch from
             the requests' lengths and a stack of free blocks.

A 4-bit cache is uint8 [num_blocks, num_kv_heads, block_size * (head_dim/2 + 4)]:
block_size rows of head_dim/2 code bytes (even dims in the low nibble), then
one (scale, zero) pair of bf16 per row; a code c stands for zero + scale * c.
"""

import math

import numpy as np
import torch

own = False


def _ops():
    from paged_kv_cache_379_b200 import ops
    return ops


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step's 128 new tokens of the grouped-query batch
        {"name": "store step 128x8x128", "op": "store", "tokens": 128, "kv_heads": 8, "head_dim": 128, "block_size": 16},
        # a short ragged chunk, small heads, 8-token blocks
        {"name": "store chunk 333x4x64", "op": "store", "tokens": 333, "kv_heads": 4, "head_dim": 64, "block_size": 8},
        # 8 prompts of 2048 tokens
        {"name": "store prompts 16384x8x128", "op": "store", "tokens": 16384, "kv_heads": 8, "head_dim": 128,
         "block_size": 16},
        # four short sequences: latency of a small interactive batch
        {"name": "decode small 4 seqs", "op": "decode", "seqs": 4, "heads": 4, "kv_heads": 4, "head_dim": 64,
         "block_size": 8, "low": 7, "high": 50, "len_seed": 379},
        # one conversation of about 8K tokens alone on the GPU
        {"name": "decode one 8K", "op": "decode", "seqs": 1, "heads": 32, "kv_heads": 8, "head_dim": 128,
         "block_size": 16, "low": 8001, "high": 8001, "len_seed": 380},
        # the grouped-query serving batch (64 query heads on 8)
        {"name": "decode gqa 128 seqs", "op": "decode", "seqs": 128, "heads": 64, "kv_heads": 8, "head_dim": 128,
         "block_size": 16, "low": 16, "high": 4096, "len_seed": 381},
        # the multi-head batch (32 heads, one query head per KV head)
        {"name": "decode mha 64 seqs", "op": "decode", "seqs": 64, "heads": 32, "kv_heads": 32, "head_dim": 128,
         "block_size": 16, "low": 128, "high": 2048, "len_seed": 382},
        # eight long documents
        {"name": "decode long 8 seqs", "op": "decode", "seqs": 8, "heads": 32, "kv_heads": 8, "head_dim": 128,
         "block_size": 16, "low": 32768, "high": 131072, "len_seed": 383},
        # one decode step of 128 sequences
        {"name": "rope step 128 tokens", "op": "rope", "tokens": 128, "heads": 64, "kv_heads": 8, "head_dim": 128,
         "rot_dim": 128, "interleaved": False, "block_size": 16},
        # 8 prompts of 2048 tokens, interleaved pairs, half of the head rotated
        {"name": "rope prompts 16384 tokens", "op": "rope", "tokens": 16384, "heads": 32, "kv_heads": 8,
         "head_dim": 128, "rot_dim": 64, "interleaved": True, "block_size": 16},
        # a decode step: 256 requests, one token each
        {"name": "batch step 256 reqs", "op": "batch", "seqs": 256, "ctx_high": 1280, "new_low": 1, "new_high": 1,
         "block_size": 16, "len_seed": 384},
        # a mixed step: prompt chunks of up to 2048 tokens
        {"name": "batch chunks 64 reqs", "op": "batch", "seqs": 64, "ctx_high": 4096, "new_low": 1, "new_high": 2048,
         "block_size": 16, "len_seed": 385},
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["store", "decode", "decode", "rope", "batch"])
    d = rng.choice([64, 128])
    if op == "store":
        return {"op": op, "tokens": _log_int(rng, 1, 16384), "kv_heads": rng.choice([1, 2, 3, 4, 8]), "head_dim": d,
                "block_size": rng.choice([8, 16, 32])}
    if op == "decode":
        kv = rng.choice([1, 2, 3, 4, 8])
        group = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
        seqs = _log_int(rng, 1, 200)
        high = _log_int(rng, 20, min(131072, 400000 // seqs))
        return {"op": op, "seqs": seqs, "heads": kv * group, "kv_heads": kv, "head_dim": d,
                "block_size": rng.choice([8, 16, 32]), "low": rng.choice([0, 1, high // 2]), "high": high,
                "len_seed": rng.randrange(1 << 30)}
    if op == "rope":
        kv = rng.choice([1, 2, 3, 4, 8])
        return {"op": op, "tokens": _log_int(rng, 1, 12000), "heads": kv * rng.choice([1, 2, 3, 4, 5, 7, 8]),
                "kv_heads": kv, "head_dim": d, "rot_dim": rng.choice([16, d // 2, d]),
                "interleaved": rng.random() < 0.5, "block_size": rng.choice([8, 16, 32])}
    high = rng.choice([1, 1, _log_int(rng, 2, 2048)])
    return {"op": op, "seqs": _log_int(rng, 1, 2000 if high == 1 else 100), "ctx_high": _log_int(rng, 16, 8192),
            "new_low": rng.choice([0, 1]) if high > 1 else 1, "new_high": high,
            "block_size": rng.choice([8, 16, 32]), "len_seed": rng.randrange(1 << 30)}


# ------------------------------------------------------------- sizes that a case fixes

def _decode_lens(case):
    g = np.random.Generator(np.random.PCG64(case["len_seed"]))
    low, high, n = case["low"], case["high"], case["seqs"]
    if high <= 4096 and low == 16:  # the serving batch's long-tailed lengths
        return np.clip(np.rint(np.exp(math.log(1024.0) + 0.8 * g.standard_normal(n))), low, high).astype(np.int64)
    return g.integers(low, high, size=n, endpoint=True)


def _batch_lens(case):
    g = np.random.Generator(np.random.PCG64(case["len_seed"]))
    n = case["seqs"]
    ctx = g.integers(0, case["ctx_high"], size=n, endpoint=True)
    new = g.integers(case["new_low"], case["new_high"], size=n, endpoint=True)
    return ctx, new


def _blocks(lens, block_size):
    return -(-np.asarray(lens, dtype=np.int64) // block_size)


def _row_bytes(head_dim):
    return head_dim // 2 + 4


# -------------------------------------------------------------------------- prepare

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) & 0x7FFFFFFFFFFF)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _perm(g, n):
    return torch.randperm(n, generator=g, device="cuda")


def prepare(case, seed):
    g = _gen(seed)
    return {"store": _prepare_store, "decode": _prepare_decode, "rope": _prepare_rope,
            "batch": _prepare_batch}[case["op"]](case, g)


def _slots(g, tokens, block_size):
    """Slots of `tokens` consecutive positions in blocks in random order, and those blocks."""
    n = -(-tokens // block_size)
    blocks = _perm(g, n)
    t = torch.arange(tokens, device="cuda")
    return blocks[t // block_size] * block_size + t % block_size, blocks.to(torch.int32)


def _prepare_store(case, g):
    T, H, D, bs = case["tokens"], case["kv_heads"], case["head_dim"], case["block_size"]
    qkv = _normal(g, T, 2 * H * D)  # K and V as a fused projection leaves them
    slots, blocks = _slots(g, T, bs)
    n = blocks.numel()
    cache = lambda: torch.zeros(n, H, bs * _row_bytes(D), dtype=torch.uint8, device="cuda")  # noqa: E731
    out = lambda: torch.empty(n, bs, H, D, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    return {"case": case, "key": qkv[:, :H * D].view(T, H, D), "value": qkv[:, H * D:].view(T, H, D), "slots": slots,
            "blocks": blocks, "key_cache": cache(), "value_cache": cache(), "key_out": out(), "value_out": out()}


def _random_cache(g, blocks, heads, block_size, head_dim):
    """A 4-bit cache of standard normal rows, filled in pieces."""
    cache = torch.empty(blocks, heads, block_size * _row_bytes(head_dim), dtype=torch.uint8, device="cuda")
    codes = cache[:, :, :block_size * head_dim // 2].view(blocks, heads, block_size, head_dim // 2)
    step = max(1, (1 << 28) // (heads * block_size * head_dim))
    for a in range(0, blocks, step):
        b = min(blocks, a + step)
        x = torch.randn(b - a, heads, block_size, head_dim, generator=g, device="cuda")
        zero = x.amin(-1, keepdim=True).to(torch.bfloat16)
        scale = ((x.amax(-1, keepdim=True) - zero.float()) / 15).to(torch.bfloat16)
        c = ((x - zero.float()) / scale.float()).round().clamp(0, 15).to(torch.uint8)
        codes[a:b] = c[..., 0::2] | (c[..., 1::2] << 4)
        cache[a:b, :, block_size * head_dim // 2:] = torch.cat([scale, zero], -1).view(torch.uint8).reshape(
            b - a, heads, block_size * 4)
    return cache


def _prepare_decode(case, g):
    B, Hq, H, D, bs = case["seqs"], case["heads"], case["kv_heads"], case["head_dim"], case["block_size"]
    lens = _decode_lens(case)
    need = _blocks(lens, bs)
    total, width = int(need.sum()), max(1, int(need.max()))
    pool = total + max(1, total // 50)
    perm = _perm(g, pool).to(torch.int32)
    start = torch.from_numpy(np.concatenate([[0], np.cumsum(need)[:-1]])).cuda()
    n = torch.from_numpy(need).cuda()
    j = torch.arange(width, device="cuda")
    tables = torch.where(j[None] < n[:, None], perm[(start[:, None] + j[None]).clamp(max=pool - 1)], -1)
    return {"case": case, "query": _normal(g, B, Hq, D), "tables": tables.to(torch.int32).contiguous(),
            "lens": torch.from_numpy(lens.astype(np.int32)).cuda(), "scale": 1.0 / math.sqrt(D),
            "key_cache": _random_cache(g, pool, H, bs, D), "value_cache": _random_cache(g, pool, H, bs, D),
            "out": torch.empty(B, Hq, D, dtype=torch.bfloat16, device="cuda"),
            # the scratch that a program keeps beside its cache, zeroed once
            "workspace": torch.zeros(8 << 20, dtype=torch.uint8, device="cuda")}


def _prepare_rope(case, g):
    T, Hq, H, D, bs = case["tokens"], case["heads"], case["kv_heads"], case["head_dim"], case["block_size"]
    qkv = _normal(g, T, (Hq + 2 * H) * D)
    rot, positions = case["rot_dim"], 8192
    angle = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * (
        10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot))[None]
    slots, blocks = _slots(g, T, bs)
    cache = lambda: torch.zeros(blocks.numel(), bs, H, D, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    weight = lambda: (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16)  # noqa: E731
    return {"case": case, "query": qkv[:, :Hq * D].view(T, Hq, D),
            "key": qkv[:, Hq * D:(Hq + H) * D].view(T, H, D), "value": qkv[:, (Hq + H) * D:].view(T, H, D),
            "q_weight": weight(), "k_weight": weight(), "cos_sin": torch.cat([angle.cos(), angle.sin()], -1).float(),
            "positions": torch.randint(0, positions, (T,), generator=g, device="cuda"), "slots": slots,
            "key_cache": cache(), "value_cache": cache(),
            "query_out": torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda"), "eps": 1e-6}


def _prepare_batch(case, g):
    ctx, new = _batch_lens(case)
    bs = case["block_size"]
    B, T = case["seqs"], int(new.sum())
    have, need = _blocks(ctx, bs), _blocks(ctx + new, bs)
    width = int(need.max()) + 1
    used, fresh = int(have.sum()), int((need - have).sum())
    pool = used + fresh + 64
    perm = _perm(g, pool).to(torch.int32)
    start = torch.from_numpy(np.concatenate([[0], np.cumsum(have)[:-1]])).cuda()
    j = torch.arange(width, device="cuda")
    tables = torch.where(j[None] < torch.from_numpy(have).cuda()[:, None],
                         perm[(start[:, None] + j[None]).clamp(max=pool - 1)], -1)
    i32 = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    i64 = lambda *s: torch.empty(*s, dtype=torch.int64, device="cuda")  # noqa: E731
    room = T + T // 8 + 1  # a step's arrays are padded to a fixed size
    return {"case": case, "tables": tables.to(torch.int32).contiguous(), "room": room, "pool": pool,
            "ctx": torch.from_numpy(ctx.astype(np.int32)).cuda(), "new": torch.from_numpy(new.astype(np.int32)).cuda(),
            "free": torch.cat([perm[used:], perm[:used]]).contiguous(),
            "num_free": torch.tensor([pool - used], dtype=torch.int32, device="cuda"),
            "seq_lens": i32(B), "q_start": i32(B + 1), "seq_ids": i32(room), "positions": i64(room), "slots": i64(room),
            "num_free_out": i32(1), "status": i32(1)}


# ------------------------------------------------------------------------------ run

def run(state):
    return {"store": _run_store, "decode": _run_decode, "rope": _run_rope, "batch": _run_batch}[state["case"]["op"]](state)


def _quantise(x):
    """(codes, scale, zero) of bf16 rows, all in fp32: zero = the row's minimum, scale =
    bf16(max/15 - min/15), code = the nearest integer to (x - zero) * (1/scale)."""
    x = x.float()
    r15 = float(np.float32(1.0 / 15.0))
    zero = x.amin(-1, keepdim=True)
    scale = (x.amax(-1, keepdim=True) * r15 - zero * r15).to(torch.bfloat16).float()
    flat = scale < 2.0 ** -126
    inverse = torch.where(flat, torch.zeros_like(scale), 1.0 / scale)
    codes = ((x - zero) * inverse).round().clamp(0, 15)
    return codes, torch.where(flat, torch.zeros_like(scale), scale), zero


def _run_store(s):
    if own:
        ops = _ops()
        ops.reshape_and_cache_int4(s["key"], s["value"], s["key_cache"], s["value_cache"], s["slots"])
        ops.dequantize_blocks_int4(s["key_cache"], s["value_cache"], s["blocks"], s["case"]["head_dim"],
                                   key_out=s["key_out"], value_out=s["value_out"])
        return {"key": s["key_out"], "value": s["value_out"]}
    c = s["case"]
    n, bs, H, D = s["blocks"].numel(), c["block_size"], c["kv_heads"], c["head_dim"]
    got = {}
    for name in ("key", "value"):
        codes, scale, zero = _quantise(s[name])
        rows = torch.zeros(n * bs, H, D, dtype=torch.bfloat16, device="cuda")
        rows[s["slots"]] = (zero + scale * codes).to(torch.bfloat16)
        got[name] = rows.view(n, bs, H, D)[s["blocks"].long()]
    return got


def _expand(cache, tables, block_size, head_dim):
    """fp32 [seqs, heads, width * block_size, head_dim] of the blocks in `tables`."""
    B, W = tables.shape
    rec = cache[tables.long().clamp(min=0)]
    H, cb = rec.shape[2], block_size * head_dim // 2
    code = rec[..., :cb].view(B, W, H, block_size, head_dim // 2)
    code = torch.stack([code & 15, code >> 4], -1).view(B, W, H, block_size, head_dim).float()
    par = rec[..., cb:].contiguous().view(torch.bfloat16).view(B, W, H, block_size, 2).float()
    x = code.mul_(par[..., :1]).add_(par[..., 1:])
    return x.transpose(1, 2).reshape(B, H, W * block_size, head_dim)


def _run_decode(s):
    if own:
        _ops().decode_int4(s["query"], s["key_cache"], s["value_cache"], s["tables"], s["lens"], s["scale"],
                           s["workspace"], out=s["out"])
        return s["out"]
    c = s["case"]
    B, Hq, H, D = c["seqs"], c["heads"], c["kv_heads"], c["head_dim"]
    q = s["query"].float().view(B, H, Hq // H, D)
    k = _expand(s["key_cache"], s["tables"], c["block_size"], D)
    x = torch.matmul(q, k.transpose(-1, -2)) * s["scale"]
    del k
    dead = torch.arange(x.shape[-1], device="cuda")[None] >= s["lens"][:, None]
    x = x.masked_fill(dead[:, None, None], float("-inf"))
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    v = _expand(s["value_cache"], s["tables"], c["block_size"], D).masked_fill(dead[:, None, :, None], 0.0)
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return o.reshape(B, Hq, D).to(torch.bfloat16)


def _norm_rope(x, weight, cos, sin, rot, interleaved, eps):
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * weight.float()
    r, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, rest], -1).to(torch.bfloat16)


def _run_rope(s):
    c = s["case"]
    if own:
        _ops().qk_norm_rope_cache(s["query"], s["key"], s["value"], s["q_weight"], s["k_weight"], s["cos_sin"],
                                  s["positions"], s["slots"], s["key_cache"], s["value_cache"], eps=s["eps"],
                                  interleaved=c["interleaved"], query_out=s["query_out"])
        return {"query": s["query_out"], "key_cache": s["key_cache"], "value_cache": s["value_cache"]}
    rot = c["rot_dim"]
    cs = s["cos_sin"][s["positions"]][:, None]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    s["key_cache"].view(-1, c["kv_heads"], c["head_dim"])[s["slots"]] = _norm_rope(
        s["key"], s["k_weight"], cos, sin, rot, c["interleaved"], s["eps"])
    s["value_cache"].view(-1, c["kv_heads"], c["head_dim"])[s["slots"]] = s["value"]
    return {"query": _norm_rope(s["query"], s["q_weight"], cos, sin, rot, c["interleaved"], s["eps"]),
            "key_cache": s["key_cache"], "value_cache": s["value_cache"]}


def _run_batch(s):
    bs, room = s["case"]["block_size"], s["room"]
    if own:
        _ops().prepare_batch(s["tables"], s["ctx"], s["new"], s["free"], s["num_free"], bs, s["pool"],
                             seq_lens=s["seq_lens"], q_start=s["q_start"], seq_ids=s["seq_ids"],
                             positions=s["positions"], slot_mapping=s["slots"], num_free_out=s["num_free_out"],
                             status=s["status"])
        return {k: s[k] for k in ("tables", "seq_lens", "q_start", "seq_ids", "positions", "slots", "num_free_out")}
    ctx, new = s["ctx"].long(), s["new"].long()
    have = (ctx + bs - 1) // bs
    need = (ctx + new + bs - 1) // bs - have
    before = need.cumsum(0) - need
    j = torch.arange(s["tables"].shape[1], device="cuda")[None]
    fresh = (j >= have[:, None]) & (j < (have + need)[:, None])
    at = s["num_free"].long() - 1 - (before[:, None] + j - have[:, None])
    s["tables"].copy_(torch.where(fresh, s["free"][at.clamp(0, s["pool"] - 1)], s["tables"]))
    ends = new.cumsum(0)
    start = torch.cat([torch.zeros_like(ends[:1]), ends])
    t = torch.arange(room, device="cuda")
    seq = torch.searchsorted(ends, t, right=True)
    live = t < ends[-1]
    q = seq.clamp(max=new.numel() - 1)
    pos = ctx[q] + t - start[q]
    blk = s["tables"][q, (pos // bs).clamp(0, s["tables"].shape[1] - 1)].long()
    return {"tables": s["tables"], "seq_lens": (ctx + new).int(), "q_start": start.int(),
            "seq_ids": torch.where(live, seq, -1).int(), "positions": torch.where(live, pos, -1),
            "slots": torch.where(live, blk * bs + pos % bs, -1), "num_free_out": s["num_free"] - need.sum().int()}


# ----------------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "store":
        rows, D = case["tokens"] * case["kv_heads"] * 2, case["head_dim"]
        # rows in, codes out, codes in again, bf16 blocks out, slots and block ids
        return {"bytes": rows * (2 * D + 2 * _row_bytes(D) + 2 * D) + case["tokens"] * 8, "flops": rows * D * 8}
    if op == "decode":
        lens = _decode_lens(case)
        n, D = int(lens.sum()), case["head_dim"]
        return {"bytes": n * case["kv_heads"] * 2 * _row_bytes(D) + int(_blocks(lens, case["block_size"]).sum()) * 4 +
                case["seqs"] * (case["heads"] * D * 4 + 4), "flops": n * case["heads"] * D * 4}
    if op == "rope":
        T, D = case["tokens"], case["head_dim"]
        rows = T * (case["heads"] + 2 * case["kv_heads"])
        return {"bytes": rows * D * 4 + T * (16 + case["rot_dim"] * 4), "flops": rows * D * 8}
    ctx, new = _batch_lens(case)
    bs, T = case["block_size"], int(new.sum())
    fresh = int((_blocks(ctx + new, bs) - _blocks(ctx, bs)).sum())
    room = T + T // 8 + 1
    return {"bytes": case["seqs"] * 16 + fresh * 8 + room * 20, "flops": room * 4}


# ---------------------------------------------------------------------------- exact

def exact(case, seed):
    s = prepare(case, seed)
    return {"store": _exact_store, "decode": _exact_decode, "rope": _exact_rope, "batch": _exact_batch}[case["op"]](s, case)


def _f32(x):
    """A value of 64 bits rounded to 32 and held in 64: one rounding of the definition."""
    return x.to(torch.float32).to(torch.float64)


def _exact_store(s, case):
    """The cached values by their definition; the roundings that define a code are taken one by one."""
    n, bs, H, D = s["blocks"].numel(), case["block_size"], case["kv_heads"], case["head_dim"]
    got = {}
    for name in ("key", "value"):
        x = s[name].double()
        low, high = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
        third = float(np.float32(1.0 / 15.0))
        step = _f32(_f32(high * third) - _f32(low * third)).to(torch.float32).to(torch.bfloat16).double()
        step = torch.where(step < 2.0 ** -126, 0.0, step)
        inv = torch.where(step > 0, _f32(1.0 / step), 0.0)
        code = torch.clamp(torch.round(_f32(_f32(x - low) * inv)), 0, 15)
        full = torch.zeros(n * bs, H, D, dtype=torch.float64, device="cuda")
        full.index_copy_(0, s["slots"], low + step * code)
        got[name] = full.view(n, bs, H, D).index_select(0, s["blocks"].long())
    return got


def _exact_decode(s, case):
    """One sequence at a time, the codes taken apart on their own."""
    Hq, H, D, bs = case["heads"], case["kv_heads"], case["head_dim"], case["block_size"]
    lens, out = s["lens"].tolist(), torch.zeros(case["seqs"], Hq, D, dtype=torch.float64, device="cuda")

    def rows(cache, ids, length):  # [heads, length, D]
        r = cache[ids.long()].permute(1, 0, 2)
        code = r[:, :, :bs * D // 2].reshape(H, -1, D // 2)[:, :length]
        pair = r[:, :, bs * D // 2:].reshape(H, -1, 4)[:, :length].contiguous().view(torch.bfloat16).double()
        x = torch.empty(H, length, D, dtype=torch.float64, device="cuda")
        x[..., 0::2] = (code % 16).double()
        x[..., 1::2] = torch.div(code, 16, rounding_mode="floor").double()
        return pair[..., 1:] + pair[..., :1] * x

    for i, length in enumerate(lens):
        if length <= 0:
            continue
        ids = s["tables"][i, :-(-length // bs)]
        q = s["query"][i].double().view(H, Hq // H, D)
        w = torch.softmax(torch.einsum("hgd,htd->hgt", q, rows(s["key_cache"], ids, length)) * s["scale"], -1)
        out[i] = torch.einsum("hgt,htd->hgd", w, rows(s["value_cache"], ids, length)).reshape(Hq, D)
    return out


def _exact_rope(s, case):
    rot = case["rot_dim"]
    first = torch.arange(0, rot, 2, device="cuda") if case["interleaved"] else torch.arange(rot // 2, device="cuda")
    second = first + (1 if case["interleaved"] else rot // 2)
    table = s["cos_sin"].double()[s["positions"]]

    def turn(x, w):
        x = x.double()
        y = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]) * w.double()
        co, si = table[:, None, :rot // 2], table[:, None, rot // 2:]
        z = y.clone()
        z[..., first] = y[..., first] * co - y[..., second] * si
        z[..., second] = y[..., first] * si + y[..., second] * co
        return z

    shape = s["key_cache"].shape
    caches = {}
    for name, rows in (("key_cache", turn(s["key"], s["k_weight"])), ("value_cache", s["value"].double())):
        caches[name] = torch.zeros(shape, dtype=torch.float64, device="cuda").view(-1, *shape[2:]).index_copy(
            0, s["slots"], rows).view(shape)
    return {"query": turn(s["query"], s["q_weight"]), **caches}


def _exact_batch(s, case):
    """The same integers, request by request on the host."""
    bs, tables = case["block_size"], s["tables"].cpu().numpy().copy()
    free, left = s["free"].cpu().numpy(), int(s["num_free"].item())
    ctx, new = _batch_lens(case)
    ids, pos, slots = (np.full(s["room"], -1, dtype=np.int64) for _ in range(3))
    at, starts = 0, [0]
    for i, (c, n) in enumerate(zip(ctx.tolist(), new.tolist())):
        for b in range(-(-c // bs), -(-(c + n) // bs)):
            left -= 1
            tables[i, b] = free[left]
        p = np.arange(c, c + n)
        ids[at:at + n], pos[at:at + n], slots[at:at + n] = i, p, tables[i, p // bs].astype(np.int64) * bs + p % bs
        at += n
        starts.append(at)
    return {"tables": tables, "seq_lens": (ctx + new).astype(np.int32), "q_start": np.array(starts, dtype=np.int32),
            "seq_ids": ids.astype(np.int32), "positions": pos, "slots": slots,
            "num_free_out": np.array([left], dtype=np.int32)}
