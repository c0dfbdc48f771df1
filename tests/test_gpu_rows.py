"""GPU: head norm + rotation against the 64-bit form, and its cache writes
against the separate cache write bit for bit."""

import math

import pytest
import torch

import _int4_ref as ref
from paged_kv_cache_379_b200 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _table(rot, n=500):
    a = torch.arange(n, dtype=torch.float64)[:, None] * 10000.0 ** (
        -torch.arange(0, rot, 2, dtype=torch.float64) / rot)[None]
    return torch.cat([a.cos(), a.sin()], -1).float()


def _inputs(T, Hq, H, D, rot, seed=0):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(T, (Hq + 2 * H) * D, generator=g).to(torch.bfloat16)
    w = [(1 + 0.2 * torch.randn(D, generator=g)).to(torch.bfloat16) for _ in range(2)]
    pos = torch.randint(0, 500, (T,), generator=g)
    q, k, v = (t.view(T, -1, D) for t in qkv.split([Hq * D, H * D, H * D], dim=1))
    return qkv, q, k, v, *w, _table(rot), pos


def _views(qkv, Hq, H, D):
    T = qkv.shape[0]
    return [t.view(T, -1, D) for t in qkv.split([Hq * D, H * D, H * D], dim=1)]


def _close(got, want, bound):
    err = (got.cpu().double() - want).abs()
    assert bool((err <= bound).all()), f"worst {float((err / bound).max()):.3f} of the bound"


@pytest.mark.parametrize("D,rot", [(64, 16), (64, 32), (64, 64), (128, 16), (128, 48), (128, 64), (128, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,H", [(1, 1, 1), (5, 8, 2), (37, 12, 4), (3, 64, 8), (130, 3, 3)])
def test_norm_rope(D, rot, interleaved, T, Hq, H):
    qkv, q, k, v, qw, kw, cs, pos = _inputs(T, Hq, H, D, rot, seed=T + rot)
    dq, dk, _ = _views(qkv.to(DEV), Hq, H, D)
    qo, ko = ops.qk_norm_rope(dq, dk, qw.to(DEV), kw.to(DEV), cs.to(DEV), pos.to(DEV), eps=1e-5,
                              interleaved=interleaved)
    _close(qo, *ref.norm_rope(q, qw, cs, pos, interleaved, 1e-5))
    _close(ko, *ref.norm_rope(k, kw, cs, pos, interleaved, 1e-5))


@pytest.mark.parametrize("form", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("D,rot,interleaved,Hq,H,bs", [(64, 32, True, 6, 3, 8), (128, 128, False, 16, 2, 16),
                                                       (128, 64, True, 8, 8, 32)])
def test_cache_forms_equal_the_separate_write(form, D, rot, interleaved, Hq, H, bs):
    T, nb = 45, 16
    qkv, _, _, _, qw, kw, cs, pos = _inputs(T, Hq, H, D, rot, seed=7)
    pos[4], pos[9] = -1, 500              # padding rows
    q, k, v = _views(qkv.to(DEV), Hq, H, D)
    slots = torch.randperm(nb * bs, generator=torch.Generator().manual_seed(2))[:T]
    slots[11], slots[12] = -1, nb * bs    # queries only
    args = (qw.to(DEV), kw.to(DEV), cs.to(DEV), pos.to(DEV))
    live = torch.ones(T, dtype=torch.bool)
    live[4] = live[9] = False
    want_q, key = ops.qk_norm_rope(q, k, *args, interleaved=interleaved)
    write = torch.where(live & (slots < nb * bs), slots, torch.tensor(-1)).to(DEV)
    if form == "int4":
        new = lambda: ops.new_int4_cache(nb, bs, H, D)  # noqa: E731
    else:
        new = lambda: torch.zeros(nb, bs, H, D, device=DEV,  # noqa: E731
                                  dtype=torch.uint8 if form == "fp8" else torch.bfloat16)
    a, b = [new(), new()], [new(), new()]
    qo = torch.full((T, Hq, D), 3.0, dtype=torch.bfloat16, device=DEV)
    slots = slots.to(DEV)
    if form == "bf16":
        ops.qk_norm_rope_cache(q, k, v, *args, slots, *a, interleaved=interleaved, query_out=qo)
        ops.reshape_and_cache(key, v.contiguous(), *b, write)
    elif form == "fp8":
        ops.qk_norm_rope_cache_fp8(q, k, v, *args, slots, *a, 0.02, 0.03, interleaved=interleaved, query_out=qo)
        ops.reshape_and_cache_fp8(key, v.contiguous(), *b, write, 0.02, 0.03)
    else:
        ops.qk_norm_rope_cache_int4(q, k, v, *args, slots, *a, interleaved=interleaved, query_out=qo)
        ops.reshape_and_cache_int4(key, v, *b, write)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert torch.equal(qo[live], want_q[live])
    assert bool((qo[~live] == 3.0).all())  # padding rows are left as they were


def test_in_place_and_without_weights():
    qkv, q, k, v, qw, kw, cs, pos = _inputs(19, 8, 2, 128, 128, seed=1)
    buf = qkv.to(DEV)
    dq, dk, dv = _views(buf, 8, 2, 128)
    want = ops.qk_norm_rope(dq, dk, None, None, cs.to(DEV), pos.to(DEV))
    before = dv.clone()
    got = ops.qk_norm_rope(dq, dk, None, None, cs.to(DEV), pos.to(DEV), query_out=dq, key_out=dk)
    assert got[0] is dq and torch.equal(dq, want[0]) and torch.equal(dk, want[1]) and torch.equal(dv, before)
    _close(dq, *ref.norm_rope(q, None, cs, pos, False, 1e-6))
    _close(dk, *ref.norm_rope(k, None, cs, pos, False, 1e-6))


def test_magnitudes_and_zero_rows():
    qkv, q, k, v, qw, kw, cs, pos = _inputs(8, 4, 2, 64, 64, seed=3)
    for t, f in enumerate((0.0, 1e-30, 1e-12, 1e-3, 1e3, 1e9, 1e17, 1.0)):
        qkv[t] = (qkv[t].float() * f).to(torch.bfloat16)
    q, k, v = _views(qkv, 4, 2, 64)
    dq, dk, _ = _views(qkv.to(DEV), 4, 2, 64)
    qo, ko = ops.qk_norm_rope(dq, dk, qw.to(DEV), kw.to(DEV), cs.to(DEV), pos.to(DEV), eps=1e-6)
    for got, x, w in ((qo, q, qw), (ko, k, kw)):
        want, bound = ref.norm_rope(x, w, cs, pos, False, 1e-6)
        _close(got, want, bound + 1e-38)
    # a NaN stays in its head
    qkv[7, 5] = float("nan")
    dq, dk, _ = _views(qkv.to(DEV), 4, 2, 64)
    qn, _ = ops.qk_norm_rope(dq, dk, qw.to(DEV), kw.to(DEV), cs.to(DEV), pos.to(DEV), eps=1e-6)
    assert bool(qn[7, 0].isnan().all()) and torch.equal(qn[7, 1:], qo[7, 1:]) and torch.equal(qn[:7], qo[:7])


def test_far_positions():
    """A table row 2^17 away; offsets of a table beyond 2^31 bytes are 64-bit sums (position * rot)."""
    D = rot = 128
    n = 1 << 17
    g = torch.Generator().manual_seed(2)
    cs = torch.empty(n, rot, device=DEV)
    small = _table(rot, 4)
    cs[n - 4:] = small.to(DEV)
    q = torch.randn(4, 2, D, generator=g).to(torch.bfloat16)
    pos = torch.arange(4)
    qo, _ = ops.qk_norm_rope(q.to(DEV), q.to(DEV), None, None, cs, (pos + n - 4).to(DEV))
    _close(qo, *ref.norm_rope(q, None, small, pos, False, 1e-6))


def test_refusals_and_empty():
    qkv, q, k, v, qw, kw, cs, pos = [t.to(DEV) if isinstance(t, torch.Tensor) else t
                                     for t in _inputs(6, 4, 2, 64, 64)]
    q, k, v = _views(qkv, 4, 2, 64)
    with pytest.raises(ops.PagedKVError, match="unsupported"):
        ops.qk_norm_rope(q, k, None, None, cs[:, :24].contiguous(), pos)
    with pytest.raises(ops.PagedKVError):
        ops.qk_norm_rope(q, k, None, None, cs, pos, eps=math.inf)
    with pytest.raises(ValueError):
        ops.qk_norm_rope(q, k, qw[:32], None, cs, pos)
    with pytest.raises(ValueError):
        ops.qk_norm_rope(q, k, None, None, cs, pos[:5])
    with pytest.raises(ValueError):
        ops.qk_norm_rope(q, k[:5], None, None, cs, pos)
    with pytest.raises(TypeError):
        ops.qk_norm_rope(q, k, None, None, cs.double(), pos)
    with pytest.raises(ops.PagedKVError):   # rows that start off a 16-byte boundary
        odd = torch.zeros(6 * 4 * 64 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(6, 4, 64)
        ops.qk_norm_rope(odd, k, None, None, cs, pos)
    a, b = ops.qk_norm_rope(q[:0], k[:0], None, None, cs, pos[:0])
    assert a.shape == (0, 4, 64) and b.shape == (0, 2, 64)
