"""GPU: head norm + rotation of many tokens, where a warp takes 8 groups of rows instead of 2 (from 37888 groups on, but
for the 4-bit cache), in every cache form, and a table of cosines past 2^31 bytes."""

import pytest
import torch

import _int4_ref as ref
from paged_kv_cache_379_b200 import ops
from test_gpu_rows import _close, _inputs, _table, _views

pytestmark = pytest.mark.gpu
DEV = "cuda"
WIDE = 148 * 32 * 8  # groups of 32 / (D / 8) rows


def _new(form, nb, bs, H, D):
    if form == "int4":
        return [ops.new_int4_cache(nb, bs, H, D) for _ in range(2)]
    return [torch.zeros(nb, bs, H, D, device=DEV, dtype=torch.uint8 if form == "fp8" else torch.bfloat16)
            for _ in range(2)]


def _call(form, q, k, v, qw, kw, cs, pos, slots, caches, interleaved, out):
    args = (q, k, v, qw, kw, cs, pos, slots, *caches)
    kw_ = dict(interleaved=interleaved, query_out=out)
    if form == "fp8":
        ops.qk_norm_rope_cache_fp8(*args, 0.02, 0.03, **kw_)
    elif form == "int4":
        ops.qk_norm_rope_cache_int4(*args, **kw_)
    else:
        ops.qk_norm_rope_cache(*args, **kw_)


@pytest.mark.parametrize("form", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("D,rot,interleaved,Hq,H,bs,T", [(128, 128, False, 32, 8, 16, 3201), (64, 32, True, 40, 5, 8, 6317),
                                                         (128, 48, True, 5, 3, 32, 12700)])
def test_cache_forms_with_many_rows(form, D, rot, interleaved, Hq, H, bs, T):
    """One wide call against pieces of it that take 2 groups a warp, bit for bit, and against the separate write."""
    groups = -(-(Hq + 2 * H) // (32 // (D // 8)))
    piece = (WIDE - 1) // groups
    assert T * groups >= WIDE > piece * groups
    nb = -(-T // bs) + 2
    qkv, _, _, _, qw, kw, cs, pos = _inputs(T, Hq, H, D, rot, seed=T)
    pos[4], pos[T - 1] = -1, 500                    # padding rows
    live = (pos >= 0) & (pos < 500)
    slots = torch.randperm(nb * bs, generator=torch.Generator().manual_seed(2))[:T]
    slots[11], slots[T - 2] = -1, nb * bs           # queries only
    q, k, v = _views(qkv.to(DEV), Hq, H, D)
    dev = [t.to(DEV) for t in (qw, kw, cs)]
    pos, slots = pos.to(DEV), slots.to(DEV)
    a, b, c = (_new(form, nb, bs, H, D) for _ in range(3))
    qa, qb = (torch.full((T, Hq, D), 3.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    _call(form, q, k, v, *dev, pos, slots, a, interleaved, qa)
    for t in range(0, T, piece):
        s = slice(t, min(T, t + piece))
        _call(form, q[s], k[s], v[s], *dev, pos[s], slots[s], b, interleaved, qb[s])
    assert torch.equal(qa, qb) and all(torch.equal(x, y) for x, y in zip(a, b))
    want, key = ops.qk_norm_rope(q, k, *dev, pos, interleaved=interleaved)
    on = live.to(DEV)
    assert torch.equal(qa[on], want[on]) and bool((qa[~on] == 3.0).all())
    write = torch.where(on & (slots < nb * bs), slots, torch.tensor(-1, device=DEV))
    if form == "bf16":
        ops.reshape_and_cache(key, v.contiguous(), *c, write)
    elif form == "fp8":
        ops.reshape_and_cache_fp8(key, v.contiguous(), *c, write, 0.02, 0.03)
    else:
        ops.reshape_and_cache_int4(key, v, *c, write)
    assert all(torch.equal(x, y) for x, y in zip(a, c))


@pytest.mark.parametrize("D,rot,interleaved,Hq,H,T", [(128, 128, False, 30, 7, 4500), (64, 64, True, 33, 9, 7001)])
def test_norm_rope_with_many_rows(D, rot, interleaved, Hq, H, T):
    assert T * -(-(Hq + H) // (32 // (D // 8))) >= WIDE
    qkv, q, k, _, qw, kw, cs, pos = _inputs(T, Hq, H, D, rot, seed=T)
    dq, dk, _ = _views(qkv.to(DEV), Hq, H, D)
    qo, ko = ops.qk_norm_rope(dq, dk, qw.to(DEV), kw.to(DEV), cs.to(DEV), pos.to(DEV), interleaved=interleaved)
    _close(qo, *ref.norm_rope(q, qw, cs, pos, interleaved, 1e-6))
    _close(ko, *ref.norm_rope(k, kw, cs, pos, interleaved, 1e-6))


def test_table_past_2_31_bytes():
    """Positions whose rows of the table begin past byte 2^31: 2^22 + 4 rows of 128 floats."""
    D = rot = 128
    n = (1 << 22) + 4
    cs = torch.empty(n, rot, device=DEV)
    small = _table(rot, 4)
    cs[n - 4:] = small.to(DEV)
    q = torch.randn(4, 2, D, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    pos = torch.arange(4)
    qo, _ = ops.qk_norm_rope(q.to(DEV), q.to(DEV), None, None, cs, (pos + n - 4).to(DEV))
    _close(qo, *ref.norm_rope(q, None, small, pos, False, 1e-6))
