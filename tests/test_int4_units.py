"""4-bit cache, head norm + rotation and batch preparation: argument errors on
the host (no GPU), and the plain forms the GPU tests compare with."""

import ctypes

import numpy as np
import pytest
import torch

import _int4_ref as ref
from paged_kv_cache_379_b200 import _lib, ops

P = ctypes.c_void_p
FAKE = P(4096)


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def _caller(fn, defaults):
    def call(**kw):
        args = dict(defaults)
        assert set(kw) <= set(args), set(kw) - set(args)
        args.update(kw)
        return fn(*args.values())
    return call


def test_store_argument_errors(lib):
    call = _caller(lib.pa_reshape_and_cache_int4, dict(
        k=FAKE, v=FAKE, ks=1024, vs=1024, kc=FAKE, vc=FAKE, slots=FAKE, t=3, h=8, d=128, bs=16, nb=10, st=None))
    assert call(t=-1) == -2
    assert call(h=0) == -2
    assert call(nb=0) == -2
    assert call(nb=1 << 28) == -2          # slots past 31 bits
    assert call(d=96) == -3
    assert call(bs=4) == -3
    assert call(bs=64) == -3
    assert call(k=None) == -1
    assert call(slots=None) == -1
    assert call(kc=None) == -1
    assert call(v=P(4104)) == -8
    assert call(vc=P(4100)) == -8
    assert call(ks=1016) == -2             # tokens overlap
    assert call(vs=1028) == -8             # rows not 16-byte aligned
    assert call(t=0, k=None, v=None, slots=None, kc=None, vc=None) == 0


def test_append_argument_errors(lib):
    call = _caller(lib.pa_append_decode_kv_int4, dict(
        k=FAKE, v=FAKE, ks=1024, vs=1024, kc=FAKE, vc=FAKE, bt=FAKE, sl=FAKE, slots=None, b=3, mb=8, h=8, d=128,
        bs=16, nb=10, st=None))
    assert call(mb=0) == -2
    assert call(b=-1) == -2
    assert call(bt=None) == -1
    assert call(sl=None) == -1
    assert call(d=32) == -3
    assert call(b=0, k=None, v=None, bt=None, sl=None) == 0


def test_dequantize_argument_errors(lib):
    call = _caller(lib.pa_dequantize_blocks_int4, dict(
        ko=FAKE, vo=FAKE, kc=FAKE, vc=FAKE, ids=FAKE, n=3, h=8, d=128, bs=16, nb=10, st=None))
    assert call(n=-1) == -2
    assert call(ids=None) == -1
    assert call(ko=None) == -1
    assert call(vo=P(4098)) == -8
    assert call(bs=12) == -3
    assert call(n=0, ko=None, vo=None, ids=None) == 0


def test_decode_argument_errors(lib):
    need = lib.pa_decode_int4_workspace_size(64, 8, 128)
    assert need > 0
    assert lib.pa_decode_int4_workspace_size(63, 8, 128) == 0
    assert lib.pa_decode_int4_workspace_size(0, 8, 128) == 0
    call = _caller(lib.pa_decode_int4, dict(
        out=FAKE, q=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, sl=FAKE, scale=0.1, bs=16, h=8, b=4, hq=64, d=128, mb=8, nb=100,
        ws=FAKE, wb=need, st=None))
    assert call(hq=63) == -2
    assert call(hq=136) == -3              # 17 query heads per KV head
    assert call(b=-1) == -2
    for bad in (float("nan"), float("inf"), float("-inf")):
        assert call(scale=bad) == -2
    assert call(b=65536) == -2
    assert call(mb=0) == -2
    assert call(mb=1 << 28) == -2
    assert call(d=96) == -3
    assert call(bs=4) == -3
    assert call(q=None) == -1
    assert call(kc=None) == -1
    assert call(out=P(4100)) == -8
    assert call(ws=None) == -4
    assert call(wb=need - 1) == -4
    assert call(ws=P(4104)) == -4
    assert call(b=0, out=None, q=None, bt=None, sl=None, ws=None, wb=0) == 0


def _rope_defaults():
    return dict(qo=FAKE, q=FAKE, k=FAKE, v=FAKE, qw=None, kw=None, cs=FAKE, pos=FAKE, slots=FAKE, kc=FAKE, vc=FAKE,
                eps=1e-6, qos=1024, qs=1024, ks=256, vs=256, rot=128, inter=0, mp=100, t=3, hq=8, h=2, d=128, bs=16,
                nb=10)


@pytest.mark.parametrize("form", ["pa_qk_norm_rope_cache", "pa_qk_norm_rope_cache_fp8", "pa_qk_norm_rope_cache_int4"])
def test_rope_cache_argument_errors(lib, form):
    defaults = _rope_defaults()
    if form.endswith("fp8"):
        defaults.update(k_scale=1.0, v_scale=1.0)
    call = _caller(getattr(lib, form), dict(defaults, st=None))
    assert call(t=-1) == -2
    assert call(hq=0) == -2
    assert call(mp=0) == -2
    for eps in (-1e-6, float("nan"), float("inf")):
        assert call(eps=eps) == -2
    for rot in (0, 8, 24, 144):
        assert call(rot=rot) == -3
    assert call(d=96) == -3
    assert call(nb=0) == -2
    assert call(q=None) == -1
    assert call(pos=None) == -1
    assert call(slots=None) == -1
    assert call(kc=None) == -1
    assert call(cs=P(4104)) == -8
    assert call(qw=P(4098)) == -8
    assert call(qs=1000) == -2
    assert call(ks=260) == -8
    assert call(t=0, q=None, k=None, v=None, qo=None) == 0
    if form.endswith("fp8"):
        assert call(k_scale=0.0) == -2
        assert call(v_scale=float("nan")) == -2
    if form.endswith("int4"):
        assert call(bs=4) == -3


def test_rope_argument_errors(lib):
    call = _caller(lib.pa_qk_norm_rope, dict(
        qo=FAKE, ko=FAKE, q=FAKE, k=FAKE, qw=None, kw=None, cs=FAKE, pos=FAKE, eps=1e-6, qos=1024, kos=256, qs=1024,
        ks=256, rot=128, inter=0, mp=100, t=3, hq=8, h=2, d=128, st=None))
    assert call(ko=None) == -1
    assert call(kos=8) == -2
    assert call(rot=4) == -3
    assert call(t=0) == 0


def test_batch_argument_errors(lib):
    call = _caller(lib.pa_prepare_batch, dict(
        bt=FAKE, ctx=FAKE, new=FAKE, free=FAKE, nf=FAKE, sl=FAKE, qs=FAKE, ids=None, pos=None, slots=None, nfo=FAKE,
        status=FAKE, b=4, mb=8, t=16, fc=100, bs=16, nb=100, st=None))
    for kw in (dict(b=-1), dict(mb=0), dict(t=-1), dict(fc=-1), dict(bs=0), dict(nb=0), dict(mb=1 << 28)):
        assert call(**kw) == -2, kw
    for kw in (dict(bt=None), dict(ctx=None), dict(free=None), dict(nf=None), dict(qs=None), dict(status=None)):
        assert call(**kw) == -1, kw
    call = _caller(lib.pa_release_blocks, dict(
        bt=FAKE, sl=FAKE, rel=FAKE, free=FAKE, nf=FAKE, status=FAKE, b=4, mb=8, fc=100, bs=16, nb=100, st=None))
    for kw in (dict(b=-1), dict(mb=0), dict(fc=-1), dict(bs=0), dict(nb=0)):
        assert call(**kw) == -2, kw
    for kw in (dict(bt=None), dict(rel=None), dict(free=None), dict(nf=None), dict(status=None)):
        assert call(**kw) == -1, kw


def test_binding_refuses_wrong_tensors():
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    cache = torch.zeros(4, 2, ops.int4_record_bytes(16, 64), dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        ops.reshape_and_cache_int4(bf(3, 2, 64), bf(3, 2, 64), cache, cache, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(TypeError, match="bfloat16"):
        ops._rows(-1, torch.zeros(3, 2, 64), "query", 3, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        ops.qk_norm_rope(torch.zeros(3, 2, 64), bf(3, 2, 64), None, None, torch.zeros(8, 64),
                         torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        ops.decode_int4(bf(1, 2, 64), cache, cache, torch.zeros(1, 4, dtype=torch.int32),
                        torch.zeros(1, dtype=torch.int32), 0.1, torch.zeros(16, dtype=torch.uint8))


def test_binding_refuses_another_device(monkeypatch):
    class Fake(torch.Tensor):
        def get_device(self):
            return 1
    t = torch.zeros(1).as_subclass(Fake)
    monkeypatch.setattr(ops, "_current_device", lambda: 0)
    with pytest.raises(ValueError, match="current device is cuda:0"):
        ops._device(t, "query")
    with pytest.raises(ValueError, match="not on cuda:0"):
        ops._arr(0, t, torch.float32, "out", 1)
    monkeypatch.setattr(ops, "_current_device", lambda: 1)
    assert ops._device(t, "query") == 1
    assert ops._arr(1, t, torch.float32, "out", 1, 1) == t.data_ptr()


def test_record_bytes():
    assert ops.int4_record_bytes(16, 128) == 1088
    assert ops.int4_record_bytes(8, 64) == 288
    assert ops.new_int4_cache(3, 16, 2, 128, device="cpu").shape == (3, 2, 1088)


def test_plain_quantiser_is_within_half_a_step():
    """|value - x| <= scale / 2 plus the scale's own rounding over 15 codes."""
    g = torch.Generator().manual_seed(5)
    x = (torch.randn(4000, 64, generator=g) * torch.exp(torch.randn(4000, 1, generator=g) * 4)).to(torch.bfloat16)
    codes, pair = ref.quantise(x)
    s, z = pair[..., :1].double(), pair[..., 1:].double()
    err = (z + s * codes.double() - x.double()).abs()
    assert bool((err <= s * (0.5 + 15 * ref.half_step(torch.bfloat16) + 1e-5)).all())
    assert codes.max() == 15 and codes.min() == 0


def test_plain_quantiser_edges():
    x = torch.zeros(6, 64)
    x[1] = 3.0                      # constant
    x[2, 5] = float("nan")
    x[3, 7] = float("-inf")
    x[4, 0], x[4, 1] = 3.3e38, -3.3e38   # max - min past the fp32 range
    x[5, 3] = 1e-39                 # a range below the smallest scale
    codes, pair = ref.quantise(x.to(torch.bfloat16))
    assert pair[0].tolist() == [0.0, 0.0] and pair[1].tolist() == [0.0, 3.0]
    assert bool(pair[2:4, 1].isnan().all()) and not codes[2:4].any()
    assert bool(torch.isfinite(pair[4].float()).all()) and codes[4, 0] == 15 and codes[4, 1] == 0
    assert pair[5, 0] == 0


def test_plain_batch_matches_the_host_pool():
    """The device operator's definition hands out the blocks that the host pool would."""
    from paged_kv_cache_379_b200.pool import BlockPool
    rng = np.random.default_rng(3)
    bs, B, nb, width = 16, 9, 200, 12
    ctx = rng.integers(0, 150, B).astype(np.int32)
    pool = BlockPool(nb, bs)
    tables = np.full((B, width), -1, np.int32)
    nblk = (-(-ctx // bs)).astype(np.int32)
    for s in range(B):
        tables[s, :nblk[s]] = pool.allocate(int(nblk[s]))
    free = np.arange(nb, dtype=np.int32)[:nb - int(nblk.sum())]
    got = ref.prepare_batch(tables, ctx, np.ones(B, np.int32), free, len(free), bs, nb, B + 2)
    slots, pairs_ = pool.prepare_decode(tables, nblk, ctx.astype(np.int64))
    assert (got[0] == tables).all() and got[5][:B].tolist() == slots.tolist() and len(pairs_) == 0
    assert got[6] == pool.get_num_free_blocks()
