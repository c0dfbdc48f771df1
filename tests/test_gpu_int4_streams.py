"""GPU: what lies between two calls of the 4-bit cache.  Default outputs on a stream
that is not the current one: the current stream's late work must not land on them.
Results that the next call of the stream reads ahead of its own wait."""

import pytest
import torch

from paged_kv_cache_379_b200 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda"
SLEEP = 100_000_000  # cycles that the current stream is kept busy, about 50 ms


def _rows(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).to(DEV)


def _caches(nb=6, bs=16, H=2, D=128):
    kc, vc = ops.new_int4_cache(nb, bs, H, D), ops.new_int4_cache(nb, bs, H, D)
    ops.reshape_and_cache_int4(_rows(nb * bs, H, D, seed=1), _rows(nb * bs, H, D, seed=2), kc, vc,
                               torch.arange(nb * bs, device=DEV))
    return kc, vc


def _late_fills(shapes):
    """Work queued on the current stream, behind a pause, on memory that goes back to the allocator at once."""
    torch.cuda._sleep(SLEEP)
    for s in shapes:
        torch.zeros(s, dtype=torch.bfloat16, device=DEV)


@pytest.mark.parametrize("as_handle", [False, True])
def test_read_back_on_another_stream(as_handle):
    kc, vc = _caches()
    ids = torch.tensor([3, -1, 0, 5], dtype=torch.int32, device=DEV)
    want = [t.clone() for t in ops.dequantize_blocks_int4(kc, vc, ids, 128)]
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(SLEEP)
    got = ops.dequantize_blocks_int4(kc, vc, ids, 128, stream=other.cuda_stream if as_handle else other)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g, w) and not bool(g[1].any()) and bool(g[0].any())


def test_read_back_on_the_default_stream_by_handle():
    """Handle 0 while another stream is current."""
    kc, vc = _caches()
    ids = torch.tensor([3, -1, 0, 5], dtype=torch.int32, device=DEV)
    want = [t.clone() for t in ops.dequantize_blocks_int4(kc, vc, ids, 128)]
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        torch.cuda._sleep(SLEEP)
        got = ops.dequantize_blocks_int4(kc, vc, ids, 128, stream=0)
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want))


@pytest.mark.parametrize("form", ["decode", "rope", "rope_cache"])
def test_results_on_another_stream(form):
    kc, vc = _caches()
    T, Hq, H, D = 5, 8, 2, 128
    q, k, v = _rows(T, Hq, D, seed=3), _rows(T, H, D, seed=4), _rows(T, H, D, seed=5)
    tables = torch.arange(5, dtype=torch.int32, device=DEV)[:, None]
    lens = torch.tensor([16, 1, 9, 0, 12], dtype=torch.int32, device=DEV)
    ws = ops.new_int4_workspace(Hq, H, D)
    cs, pos = torch.rand(8, D, device=DEV), torch.arange(T, device=DEV)
    slots = torch.full((T,), -1, dtype=torch.int64, device=DEV)

    def run(stream=None):
        if form == "decode":
            return [ops.decode_int4(q, kc, vc, tables, lens, 0.09, ws, stream=stream)]
        if form == "rope":
            return ops.qk_norm_rope(q, k, None, None, cs, pos, stream=stream)
        return [ops.qk_norm_rope_cache_int4(q, k, v, None, None, cs, pos, slots, kc, vc, stream=stream)]

    want = [t.clone() for t in run()]
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    _late_fills([w.shape for w in want])
    got = run(other)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g, w) and bool(w.any())


def test_read_back_rows_appended_at_once():
    """Rows of the read-back as the new rows of the next call, which reads them ahead of its own wait."""
    nb, bs, H, D = 2000, 16, 8, 128
    kc, vc = _caches(nb, bs, H, D)
    ids = torch.randperm(nb, generator=torch.Generator().manual_seed(3)).to(torch.int32).to(DEV)
    B = nb * bs
    tables = torch.arange(nb, dtype=torch.int32, device=DEV).repeat_interleave(bs)[:, None].contiguous()
    lens = (torch.arange(B, device=DEV) % bs + 1).to(torch.int32)
    ko, vo = (torch.zeros(nb, bs, H, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    a, b = torch.zeros_like(ko), torch.zeros_like(vo)
    for shift in range(4):
        order = ids.roll(shift)
        ops.dequantize_blocks_int4(kc, vc, order, D, key_out=ko, value_out=vo)
        ops.append_decode_kv(ko.view(B, H, D), vo.view(B, H, D), a, b, tables, lens)
        torch.cuda.synchronize()
        assert torch.equal(a, ko) and torch.equal(b, vo)


def test_result_as_the_next_query():
    """The 4-bit decode's result as the query of a bf16 decode right after it."""
    nb, bs, H, D, B, Hq = 600, 16, 2, 128, 6, 16
    kc, vc = _caches(nb, bs, H, D)
    kb, vb = ops.dequantize_blocks_int4(kc, vc, torch.arange(nb, dtype=torch.int32, device=DEV), D)
    tables = torch.randperm(nb, generator=torch.Generator().manual_seed(4)).to(torch.int32).to(DEV).view(B, -1).contiguous()
    lens = torch.tensor([1600, 3, 900, 1599, 64, 1000], dtype=torch.int32, device=DEV)
    ws, ws2 = ops.new_int4_workspace(Hq, H, D), ops.new_workspace(B, Hq, H, D, 1600)
    q = _rows(B, Hq, D, seed=9)
    mid, out = torch.zeros_like(q), torch.zeros_like(q)

    def second(query):
        return ops.decode(query, kb, vb, tables, lens, 0.3, 1600, workspace=ws2, out=out)

    want = second(ops.decode_int4(q, kc, vc, tables, lens, 0.3, ws).clone()).clone()
    for _ in range(20):
        mid.zero_()
        ops.decode_int4(q, kc, vc, tables, lens, 0.3, ws, out=mid)
        second(mid)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
