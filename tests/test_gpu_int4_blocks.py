"""GPU: whole blocks of a 4-bit cache -- copied, copied on write and swapped through the block calls of the bf16
cache, and read back under a prompt chunk."""

import numpy as np
import pytest
import torch

import _int4_exact as exact
import _int4_ref as ref
import oracle
from _helpers import assert_close
from paged_kv_cache_379_b200 import ops
from paged_kv_cache_379_b200.step import bf16_to_host_bits

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _rows(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).to(DEV)


def _caches(nb, bs, H, D, seed=1):
    kc, vc = ops.new_int4_cache(nb, bs, H, D), ops.new_int4_cache(nb, bs, H, D)
    ops.reshape_and_cache_int4(_rows(nb * bs, H, D, seed=seed), _rows(nb * bs, H, D, seed=seed + 1), kc, vc,
                               torch.arange(nb * bs, device=DEV))
    return kc, vc


def _as_blocks(cache):
    """A 4-bit cache as the block calls take it: bf16 [num_blocks, 1, num_kv_heads, record / 2], the same memory."""
    return cache.view(torch.bfloat16).unsqueeze(1)


@pytest.mark.parametrize("D,bs,H", [(64, 8, 1), (128, 16, 3), (128, 32, 8)])
def test_copy_and_swap(D, bs, H):
    nb = 12
    kc, vc = _caches(nb, bs, H, D)
    k0, v0 = kc.clone(), vc.clone()
    pairs = torch.tensor([[3, 7], [0, 11], [5, 5 + 1]], dtype=torch.int64, device=DEV)
    ops.copy_blocks(_as_blocks(kc), _as_blocks(vc), pairs)
    for src, dst in pairs.tolist():
        k0[dst], v0[dst] = k0[src].clone(), v0[src].clone()
    assert torch.equal(kc, k0) and torch.equal(vc, v0)
    host = [torch.zeros(4, H, ops.int4_record_bytes(bs, D), dtype=torch.uint8).pin_memory() for _ in range(2)]
    out = torch.tensor([[7, 0], [2, 3]], dtype=torch.int64, device=DEV)
    ops.swap_blocks(*map(_as_blocks, host), _as_blocks(kc), _as_blocks(vc), out)
    torch.cuda.synchronize()
    for h, c in zip(host, (k0, v0)):
        assert torch.equal(h[0], c[7].cpu()) and torch.equal(h[3], c[2].cpu()) and not bool(h[1:3].any())
    back = torch.tensor([[3, 9]], dtype=torch.int64, device=DEV)
    ops.swap_blocks(_as_blocks(kc), _as_blocks(vc), *map(_as_blocks, host), back)
    torch.cuda.synchronize()
    assert torch.equal(kc[9], k0[2]) and torch.equal(vc[9], v0[2]) and torch.equal(kc[:9], k0[:9])


def test_copy_on_write_before_an_append():
    """Two sequences share a partly filled block; the one that writes gets a copy first."""
    D, bs, H, L = 128, 16, 2, 21
    kc, vc = _caches(6, bs, H, D)
    tables = torch.tensor([[0, 1], [0, 1]], dtype=torch.int32, device=DEV)
    before = kc.clone(), vc.clone()
    ops.copy_blocks(_as_blocks(kc), _as_blocks(vc), torch.tensor([[1, 4]], dtype=torch.int64, device=DEV))
    tables[1, 1] = 4
    k, v = _rows(2, H, D, seed=8), _rows(2, H, D, seed=9)
    lens = torch.tensor([0, L + 1], dtype=torch.int32, device=DEV)      # only the second one writes
    ops.append_decode_kv_int4(k, v, kc, vc, tables, lens)
    assert torch.equal(kc[:4], before[0][:4]) and torch.equal(vc[:4], before[1][:4])
    for cache, was, x in ((kc, before[0], k), (vc, before[1], v)):
        want = was[1][None].cpu().clone()
        ref.write_rows(want, x[1:].cpu(), torch.tensor([L - bs]), bs)
        assert torch.equal(cache[4].cpu(), want[0])


@pytest.mark.parametrize("D,bs,Hq,H,L,n", [(128, 16, 8, 2, 100, 30), (64, 8, 6, 3, 333, 129), (128, 16, 16, 1, 700, 1),
                                           (128, 8, 4, 4, 40, 40)])
def test_prompt_chunk_over_read_back_blocks(D, bs, Hq, H, L, n):
    """The chunk's n tokens and their context in 4 bits: blocks read back, then the prefill, against the 64-bit
    prefill over the same bf16 blocks; the chunk's last token decoded from the 4-bit cache beside it."""
    width = -(-L // bs)
    kc, vc = _caches(width + 3, bs, H, D, seed=L)
    table = torch.randperm(width + 3, generator=torch.Generator().manual_seed(1))[:width].to(torch.int32)
    kb, vb = ops.dequantize_blocks_int4(kc, vc, table.to(DEV), D)
    q = _rows(n, Hq, D, seed=5)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    near = torch.arange(width, dtype=torch.int32, device=DEV)[None]
    out = ops.prefill(q, kb, vb, near, i32(L), i32(0, n), D ** -0.5)
    torch.cuda.synchronize()
    want = oracle.paged_prefill(*(bf16_to_host_bits(t) for t in (q, kb, vb)), near.cpu().numpy(),
                                np.array([L], np.int32), [n], float(np.float32(D ** -0.5)), threads=8)
    assert_close(bf16_to_host_bits(out), want, f"prefill over read-back blocks D{D} bs{bs} L{L}")
    assert float((np.abs(want) > 2e-3 + 1e-2 * np.abs(want)).mean()) > 0.9, "zeros would pass"
    tok = ops.decode_int4(q[-1:], kc, vc, table[None].to(DEV), i32(L), D ** -0.5, ops.new_int4_workspace(Hq, H, D))
    exact.check(tok.cpu().double(), *exact.decode(q[-1:].cpu(), kc.cpu(), vc.cpu(), table[None],
                                                  torch.tensor([L], dtype=torch.int32), D ** -0.5, bs))
    assert ops.device_status() == 0
