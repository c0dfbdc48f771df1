"""Plain forms of the 4-bit cache, head norm + rotation and batch preparation
operators: torch on the CPU in 64 bits (single fp32 roundings where the format
is defined by them), and numpy integers."""

from __future__ import annotations

import numpy as np
import torch

F32 = torch.float32
F64 = torch.float64


def half_step(dtype) -> float:
    """Largest relative error of rounding to `dtype`."""
    return torch.finfo(dtype).eps / 2


def quantise(x: torch.Tensor):
    """bf16 rows [..., D] -> (codes uint8 [..., D], pair bf16 [..., 2] of scale and zero)."""
    xf = x.to(F32)
    bad = ~torch.isfinite(xf).all(-1, keepdim=True)
    xf = torch.where(bad, torch.zeros_like(xf), xf)
    lo, hi = xf.amin(-1, keepdim=True), xf.amax(-1, keepdim=True)
    r = torch.tensor(np.float32(1.0 / 15.0))
    scale = (hi * r - lo * r).to(torch.bfloat16).to(F32)
    flat = scale < 2.0 ** -126
    inv = torch.where(flat, torch.zeros_like(scale), 1.0 / torch.where(flat, torch.ones_like(scale), scale))
    codes = ((xf - lo) * inv).round().clamp(0, 15)
    scale = torch.where(flat, torch.zeros_like(scale), scale)
    zero = torch.where(bad, torch.full_like(lo, float("nan")), lo + 0.0)
    codes = torch.where(bad, torch.zeros_like(codes), codes)
    scale = torch.where(bad, torch.zeros_like(scale), scale)
    return codes.to(torch.uint8), torch.cat([scale, zero], -1).to(torch.bfloat16)


def pack_row(codes: torch.Tensor, pair: torch.Tensor):
    """(bytes [..., D/2], pair bytes [..., 4])."""
    return codes[..., 0::2] | (codes[..., 1::2] << 4), pair.contiguous().view(torch.uint8)


def write_rows(cache: torch.Tensor, rows: torch.Tensor, slots, block_size: int) -> None:
    """bf16 rows [T, H, D] into a uint8 CPU cache [nb, H, record] at their slots."""
    nb, H, _ = cache.shape
    D = rows.shape[-1]
    b, p = pack_row(*quantise(rows))
    for t, slot in enumerate(slots.tolist()):
        if slot < 0 or slot >= nb * block_size:
            continue
        blk, o = divmod(slot, block_size)
        cache[blk, :, o * D // 2:(o + 1) * D // 2] = b[t]
        at = block_size * D // 2 + 4 * o
        cache[blk, :, at:at + 4] = p[t]


def values(cache: torch.Tensor, block_size: int, head_dim: int):
    """fp64 [nb, block_size, H, D]: what the codes of a CPU cache stand for."""
    nb, H, _ = cache.shape
    cb = block_size * head_dim // 2
    raw = cache[:, :, :cb].reshape(nb, H, block_size, head_dim // 2)
    code = torch.stack([raw & 15, raw >> 4], -1).reshape(nb, H, block_size, head_dim).to(F64)
    pair = cache[:, :, cb:].contiguous().view(torch.bfloat16).reshape(nb, H, block_size, 2).to(F64)
    return (pair[..., 1:] + pair[..., :1] * code).permute(0, 2, 1, 3).contiguous()


def pairs(cache: torch.Tensor, block_size: int, head_dim: int):
    """fp64 (scale, zero) [nb, block_size, H] of a CPU cache."""
    nb, H, _ = cache.shape
    p = cache[:, :, block_size * head_dim // 2:].contiguous().view(torch.bfloat16).reshape(nb, H, block_size, 2).to(F64)
    return p[..., 0].permute(0, 2, 1), p[..., 1].permute(0, 2, 1)


def decode(query, key_cache, value_cache, tables, lens, scale, block_size):
    """(out fp64 [B, Hq, D], bound fp64): single-query attention over 4-bit CPU caches, and how far a bf16
    result may be off element by element:
      * the output's rounding to bf16,
      * weights w_t = p_t s'_t rounded to fp16 before they multiply the value codes (at most half a step of
        15 s'_t, averaged with weights p_t / l),
      * fp32 logits: (D + 8) roundings of the sum of |q| (|z| + 15 s), which move a weight by that much
        relative, twice (numerator and denominator),
      * the query as 16-bit integers: multiples of 2^(e - 14) where 2^e is the binade of the head's largest
        entry; what an entry is off by counts with 15 s, twice,
      * fp32 sums over L tokens and the exponential's 2^-22."""
    B, Hq, D = query.shape
    k, v = values(key_cache, block_size, D), values(value_cache, block_size, D)
    ks, kz = pairs(key_cache, block_size, D)
    vs, _ = pairs(value_cache, block_size, D)
    H = k.shape[2]
    G = Hq // H
    out = torch.zeros(B, Hq, D, dtype=F64)
    bound = torch.zeros(B, Hq, D, dtype=F64)
    for i in range(B):
        L = min(int(lens[i]), tables.shape[1] * block_size)
        if L <= 0:
            continue
        ids = tables[i, :-(-L // block_size)].long()
        kk, vv = k[ids].reshape(-1, H, D)[:L], v[ids].reshape(-1, H, D)[:L]
        sk = (ks[ids].reshape(-1, H)[:L].abs() * 15 + kz[ids].reshape(-1, H)[:L].abs())
        sv = vs[ids].reshape(-1, H)[:L] * 15
        q = query[i].to(F64).view(H, G, D)
        x = torch.einsum("hgd,thd->hgt", q, kk) * scale
        p = torch.softmax(x, -1)
        o = torch.einsum("hgt,thd->hgd", p, vv)
        out[i] = o.reshape(Hq, D)
        mag = (q.abs().sum(-1, keepdim=True) * sk.t()[:, None] * abs(scale)).amax(-1)        # [H, G]
        step = torch.exp2(torch.floor(torch.log2(q.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -100))) - 14)
        off = (q - torch.round(q / step) * step).abs().sum(-1)                               # [H, G]
        off = off * (ks[ids].reshape(-1, H)[:L].abs().amax(0) * 15)[:, None] * abs(scale)
        rel = 2 * (D + 8) * half_step(F32) * mag + 2 * off + (L + 16) * half_step(F32) + 2.0 ** -21
        span = (vv.amax((0, 2)) - vv.amin((0, 2))).abs() + vv.abs().amax((0, 2))             # [H]
        wq = half_step(torch.float16) * torch.einsum("hgt,th->hg", p, sv)
        b = (wq + rel * span[:, None])[..., None] + half_step(torch.bfloat16) * 1.01 * o.abs()
        bound[i] = b.expand(H, G, D).reshape(Hq, D)
    return out, bound + 1e-30


def norm_rope(x, weight, cos_sin, positions, interleaved, eps):
    """(y fp64, bound fp64) of [T, heads, D] rows: RMS norm, then rotation of the first rot dims."""
    rot = cos_sin.shape[1]
    xd = x.to(F64)
    D = xd.shape[-1]
    y = xd / torch.sqrt((xd * xd).mean(-1, keepdim=True) + eps)
    if weight is not None:
        y = y * weight.to(F64)
    a_i = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    b_i = a_i + (1 if interleaved else rot // 2)
    cs = cos_sin.to(F64)[positions]
    c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    out, mag = y.clone(), y.abs()
    out[..., a_i] = y[..., a_i] * c - y[..., b_i] * s
    out[..., b_i] = y[..., b_i] * c + y[..., a_i] * s
    mag[..., a_i] = (y[..., a_i] * c).abs() + (y[..., b_i] * s).abs()
    mag[..., b_i] = (y[..., b_i] * c).abs() + (y[..., a_i] * s).abs()
    # fp32: 8 + log2(lanes) sums of squares, a reciprocal root, the products: below 32 half steps
    return out, half_step(torch.bfloat16) * 1.01 * out.abs() + 32 * half_step(F32) * mag


def prepare_batch(tables, ctx, new, free, num_free, bs, num_blocks, room):
    """Integers by the definition, request by request (a step that fits)."""
    tables = tables.copy()
    B = len(ctx)
    ids, pos, slots = (np.full(room, -1, dtype=np.int64) for _ in range(3))
    starts, at, left = [0], 0, int(num_free)
    for i in range(B):
        c, n = int(ctx[i]), int(new[i])
        for b in range(-(-c // bs), -(-(c + n) // bs)):
            left -= 1
            tables[i, b] = free[left] if 0 <= free[left] < num_blocks else -1
        p = np.arange(c, c + n)
        blk = tables[i, p // bs].astype(np.int64)
        ids[at:at + n], pos[at:at + n] = i, p
        slots[at:at + n] = np.where(blk >= 0, blk * bs + p % bs, -1)
        at += n
        starts.append(at)
    return tables, (np.asarray(ctx) + np.asarray(new)).astype(np.int32), np.array(starts, np.int32), ids, pos, slots, left
