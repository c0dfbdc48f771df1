"""GPU: the 4-bit cache -- quantising writes bit for bit, blocks read back, and
paged decode against the 64-bit form within a bound counted from its roundings."""

import numpy as np
import pytest
import torch

import _int4_ref as ref
from _helpers import ERROR_LOG
from paged_kv_cache_379_b200 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _bf(*shape, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(torch.bfloat16)


def _equal_caches(got: torch.Tensor, want: torch.Tensor, block_size, head_dim):
    """Codes equal; pairs equal, a NaN zero matching any NaN."""
    cb = block_size * head_dim // 2
    assert torch.equal(got[:, :, :cb], want[:, :, :cb])
    a = got[:, :, cb:].contiguous().view(torch.bfloat16)
    b = want[:, :, cb:].contiguous().view(torch.bfloat16)
    same = (a.view(torch.int16) == b.view(torch.int16)) | (a.isnan() & b.isnan())
    assert bool(same.all()), (~same).nonzero()[:4].tolist()


# ---- cache write ----------------------------------------------------------------------

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("T,H", [(1, 1), (5, 3), (67, 8)])
def test_store_bit_exact(D, bs, T, H):
    nb = -(-T // bs) + 2
    rows = _bf(2, T, H, D, seed=T * H + D + bs)
    rows[0, 0] *= 100
    slots = torch.from_numpy(np.random.default_rng(T).permutation(nb * bs)[:T].astype(np.int64))
    if T > 4:
        slots[1], slots[3] = -1, nb * bs  # padding, and a slot past the cache
    want = [torch.full((nb, H, ops.int4_record_bytes(bs, D)), 0xA5, dtype=torch.uint8) for _ in range(2)]
    got = [w.to(DEV) for w in want]
    for w, r in zip(want, rows):
        ref.write_rows(w, r, slots, bs)
    ops.reshape_and_cache_int4(rows[0].to(DEV), rows[1].to(DEV), *got, slots.to(DEV))
    for g, w in zip(got, want):
        _equal_caches(g.cpu(), w, bs, D)


def test_store_every_bf16_pattern():
    """All 65536 bit patterns, in rows of neighbouring patterns and in shuffled rows (infinities and NaNs)."""
    D, bs, H = 128, 16, 2
    pats = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    mixed = np.random.default_rng(1).permutation(pats)
    finite = pats[(pats & 0x7F80) != 0x7F80]
    near = np.sort(finite.view(np.int16))[:65024].view(np.uint16)
    key = torch.from_numpy(np.concatenate([pats, mixed]).view(np.int16)).view(torch.bfloat16).view(-1, H, D)
    val = torch.from_numpy(np.concatenate([near, pats, mixed[:512]]).view(np.int16)).view(torch.bfloat16).view(-1, H, D)
    T = key.shape[0]
    nb = T // bs
    slots = torch.arange(T)
    want = [torch.zeros(nb, H, ops.int4_record_bytes(bs, D), dtype=torch.uint8) for _ in range(2)]
    got = [w.to(DEV) for w in want]
    for w, r in zip(want, (key, val)):
        ref.write_rows(w, r, slots, bs)
    ops.reshape_and_cache_int4(key.to(DEV), val.to(DEV), *got, slots.to(DEV))
    for g, w in zip(got, want):
        _equal_caches(g.cpu(), w, bs, D)


def test_store_strided_views_of_a_projection():
    T, H, D, bs = 21, 4, 64, 8
    qkv = _bf(T, (2 + 2 * H) * D, seed=3).to(DEV)
    k = qkv[:, 2 * D:(2 + H) * D].view(T, H, D)
    v = qkv[:, (2 + H) * D:].view(T, H, D)
    slots = torch.randperm(32, generator=torch.Generator().manual_seed(1))[:T].to(DEV)
    a = [ops.new_int4_cache(4, bs, H, D) for _ in range(2)]
    b = [ops.new_int4_cache(4, bs, H, D) for _ in range(2)]
    ops.reshape_and_cache_int4(k, v, *a, slots)
    ops.reshape_and_cache_int4(k.contiguous(), v.contiguous(), *b, slots)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    with pytest.raises(ValueError, match="contiguous"):
        ops.reshape_and_cache_int4(k.transpose(1, 2).contiguous().transpose(1, 2), v, *a, slots)
    with pytest.raises(ValueError):
        ops.reshape_and_cache_int4(k[:, :2], v, *a, slots)
    with pytest.raises(ValueError):
        ops.reshape_and_cache_int4(k, v, *a, slots[:-1])


@pytest.mark.parametrize("bs", [8, 16, 32])
def test_append_equals_slot_mapping_and_store(bs):
    B, H, D, width = 13, 3, 128, 5
    rng = np.random.default_rng(bs)
    nb = B * width + 4
    tables = torch.from_numpy(rng.permutation(nb)[:B * width].reshape(B, width).astype(np.int32)).to(DEV)
    lens = torch.from_numpy(rng.integers(1, width * bs + 1, B).astype(np.int32)).to(DEV)
    lens[2], lens[5] = 0, width * bs + 1            # no token; a position past the row
    tables[7, (int(lens[7]) - 1) // bs] = -1
    k, v = _bf(B, H, D, seed=1).to(DEV), _bf(B, H, D, seed=2).to(DEV)
    a = [ops.new_int4_cache(nb, bs, H, D) for _ in range(2)]
    b = [ops.new_int4_cache(nb, bs, H, D) for _ in range(2)]
    slots = torch.full((B,), 7, dtype=torch.int64, device=DEV)
    ops.append_decode_kv_int4(k, v, *a, tables, lens, slot_mapping=slots)
    want = ops.slot_mapping(tables, bs, seq_lens=lens)
    ops.reshape_and_cache_int4(k, v, *b, want)
    assert torch.equal(slots, want)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ops.append_decode_kv_int4(k, v, *a, tables, lens)   # without the slots


@pytest.mark.parametrize("D,bs,H", [(64, 8, 3), (128, 16, 2), (128, 32, 1), (64, 32, 5)])
def test_dequantize_blocks(D, bs, H):
    nb = 9
    k, v = _bf(nb * bs, H, D, seed=1), _bf(nb * bs, H, D, seed=2, scale=1e-3)
    kc, vc = ops.new_int4_cache(nb, bs, H, D), ops.new_int4_cache(nb, bs, H, D)
    ops.reshape_and_cache_int4(k.to(DEV), v.to(DEV), kc, vc, torch.arange(nb * bs, device=DEV))
    ids = torch.tensor([4, 0, 4, -1, 8, nb, 1], dtype=torch.int32, device=DEV)
    ko = torch.full((7, bs, H, D), 5.0, dtype=torch.bfloat16, device=DEV)
    vo = ko.clone()
    ops.dequantize_blocks_int4(kc, vc, ids, D, key_out=ko, value_out=vo)
    for got, cache in ((ko, kc), (vo, vc)):
        full = ref.values(cache.cpu(), bs, D)
        for i, b in enumerate(ids.tolist()):
            if 0 <= b < nb:   # fma rounds to fp32 before bf16: one fp32 half step above the bf16 one
                err = (got[i].cpu().double() - full[b]).abs()
                assert bool((err <= full[b].abs() * (ref.half_step(torch.bfloat16) + 2.0 ** -23)).all())
            else:
                assert bool((got[i] == 5.0).all())
    a, b = ops.dequantize_blocks_int4(kc, vc, ids[:3], D)
    assert torch.equal(a, ko[:3]) and torch.equal(b, vo[:3])
    with pytest.raises(ValueError):
        ops.dequantize_blocks_int4(kc, vc, ids, D, key_out=ko[:2], value_out=vo)


# ---- decode ---------------------------------------------------------------------------

def _problem(lens, Hq, H, D, bs, seed=0, qscale=1.0, vscale=1.0, width=None, extra=3, offset=0.0):
    """Random 4-bit caches on the CPU and tables of distinct blocks; unused table entries name blocks out of range."""
    rng = np.random.default_rng(seed)
    need = [-(-max(0, n) // bs) for n in lens]
    width = width or max(1, max(need))
    nb = sum(need) + extra
    perm = rng.permutation(nb).astype(np.int32)
    tables = np.full((len(lens), width), nb + 1000, np.int32)
    at = 0
    for i, n in enumerate(need):
        tables[i, :n] = perm[at:at + n]
        at += n
    g = torch.Generator().manual_seed(seed + 1)
    caches = []
    for sc in (1.0, vscale):
        rows = ((torch.randn(nb, H, bs, D, generator=g) + offset) * sc).to(torch.bfloat16)
        b, p = ref.pack_row(*ref.quantise(rows))
        caches.append(torch.cat([b.reshape(nb, H, -1), p.reshape(nb, H, -1)], -1).contiguous())
    q = (torch.randn(len(lens), Hq, D, generator=g) * qscale).to(torch.bfloat16)
    return q, caches[0], caches[1], torch.from_numpy(tables), torch.tensor(lens, dtype=torch.int32)


def _run(q, kc, vc, tables, lens, scale, ws=None, **kw):
    H, D = kc.shape[1], q.shape[2]
    if ws is None:
        ws = ops.new_int4_workspace(q.shape[1], H, D)
    return ops.decode_int4(q.to(DEV), kc.to(DEV), vc.to(DEV), tables.to(DEV), lens.to(DEV), scale, ws, **kw)


def _check(label, out, want, bound):
    got = out.cpu().double()
    err = (got - want).abs()
    ok = err <= bound
    ERROR_LOG.append((label, got.numel(), float(err.max()), float((err / want.abs().clamp(min=1e-30)).max()),
                      float((err / want.abs().clamp(min=0.2))[want.abs() >= 0.2].max()) if bool(
                          (want.abs() >= 0.2).any()) else 0.0, float((err / bound).max())))
    assert bool(ok.all()), f"{label}: worst {float((err / bound).max()):.3f} of the bound at " \
                           f"{(~ok).nonzero()[0].tolist()}, {int((~ok).sum())} elements"
    assert ops.device_status() == 0


LENS = {
    "edges": [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, -3],
    "one": [777],
    "ragged": [300, 5, 1200, 64, 1, 511],
}


@pytest.mark.parametrize("D,bs", [(64, 8), (64, 16), (64, 32), (128, 8), (128, 16), (128, 32)])
@pytest.mark.parametrize("G,H", [(1, 4), (2, 3), (4, 2), (5, 1), (7, 2), (8, 2), (9, 1), (12, 3), (16, 1)])
@pytest.mark.parametrize("which", ["edges", "ragged"])
def test_decode(D, bs, G, H, which):
    lens = LENS[which]
    q, kc, vc, tables, ln = _problem(lens, G * H, H, D, bs, seed=G * 100 + D + bs)
    scale = 1.0 / D ** 0.5
    want, bound = ref.decode(q, kc, vc, tables, ln, scale, bs)
    out = _run(q, kc, vc, tables, ln, scale)
    _check(f"int4 decode {which} D{D} bs{bs} G{G} H{H}", out, want, bound)
    for i, n in enumerate(lens):
        if n <= 0:
            assert bool((out[i] == 0).all())


@pytest.mark.parametrize("G,H,L", [(1, 1, 20000), (4, 2, 9001), (8, 1, 30011), (16, 1, 5000), (1, 8, 4097)])
def test_decode_one_long_sequence(G, H, L):
    """A single sequence split over the whole GPU."""
    q, kc, vc, tables, ln = _problem([L], G * H, H, 128, 16, seed=L)
    want, bound = ref.decode(q, kc, vc, tables, ln, 0.09, 16)
    out = _run(q, kc, vc, tables, ln, 0.09)
    _check(f"int4 decode one {L} G{G} H{H}", out, want, bound)


@pytest.mark.parametrize("B", [130, 700, 2500])
def test_decode_many_sequences(B):
    """More sequences than threads of a CTA; most lengths short, some zero."""
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 90, B)
    lens[B // 2] = 900
    q, kc, vc, tables, ln = _problem(lens.tolist(), 4, 2, 64, 16, seed=B)
    want, bound = ref.decode(q, kc, vc, tables, ln, 0.125, 16)
    _check(f"int4 decode {B} seqs", _run(q, kc, vc, tables, ln, 0.125), want, bound)


@pytest.mark.parametrize("seed", range(16))
def test_decode_random_mixes(seed):
    """Lengths from none to thousands in one batch, so that units are cut between warps and between CTAs in every way."""
    rng = np.random.default_rng(1000 + seed)
    D, bs = int(rng.choice([64, 128])), int(rng.choice([8, 16, 32]))
    H, G = int(rng.integers(1, 6)), int(rng.choice([1, 2, 3, 4, 6, 8, 11, 16]))
    lens = np.exp(rng.uniform(0, np.log(6000), int(rng.integers(1, 40)))).astype(int) - 1
    q, kc, vc, tables, ln = _problem(lens.tolist(), G * H, H, D, bs, seed=seed)
    want, bound = ref.decode(q, kc, vc, tables, ln, 0.1, bs)
    _check(f"int4 decode mix {seed}: D{D} bs{bs} H{H} G{G}", _run(q, kc, vc, tables, ln, 0.1), want, bound)


@pytest.mark.parametrize("scale", [0.0, -0.09, 1e-30, 3.0])
def test_decode_scales(scale):
    """No, negative, vanishing and large softmax scales."""
    q, kc, vc, tables, ln = _problem([1, 40, 333, 700], 8, 2, 128, 16, seed=17)
    want, bound = ref.decode(q, kc, vc, tables, ln, scale, 16)
    _check(f"int4 decode scale {scale:g}", _run(q, kc, vc, tables, ln, scale), want, bound)


def test_decode_all_empty():
    q, kc, vc, tables, ln = _problem([0, 0, -1], 4, 2, 64, 16)
    out = torch.full_like(q, 9.0).to(DEV)
    _run(q, kc, vc, tables, ln, 0.125, out=out)
    assert bool((out == 0).all())


@pytest.mark.parametrize("qscale,vscale,offset", [(30.0, 1.0, 0.0), (1e-3, 1e4, 0.0), (1.0, 1e-6, 0.0), (1.0, 1e30, 0.0),
                                                  (1.0, 1.0, 5.0), (1e4, 1e-30, 0.0)])
def test_decode_magnitudes(qscale, vscale, offset):
    """Sharp and flat softmaxes, values past the fp16 range both ways, rows far from zero."""
    q, kc, vc, tables, ln = _problem([1, 40, 333, 700], 8, 2, 128, 16, seed=11, qscale=qscale, vscale=vscale,
                                     offset=offset)
    want, bound = ref.decode(q, kc, vc, tables, ln, 0.088, 16)
    _check(f"int4 decode q{qscale:g} v{vscale:g} +{offset:g}", _run(q, kc, vc, tables, ln, 0.088), want, bound)


def test_decode_rising_logits():
    """Every token's logit above the ones before it: the running maximum moves all along."""
    L, D, bs = 600, 64, 16
    q, kc, vc, tables, ln = _problem([L], 4, 1, D, bs, seed=4)
    rows = torch.linspace(-4, 4, L)[:, None].expand(L, D).clone()
    rows[:, ::2] += 0.25
    codes, p = ref.pack_row(*ref.quantise(rows.to(torch.bfloat16)))
    for t in range(L):
        blk = int(tables[0, t // bs])
        kc[blk, 0, (t % bs) * D // 2:(t % bs + 1) * D // 2] = codes[t]
        kc[blk, 0, bs * D // 2 + 4 * (t % bs):bs * D // 2 + 4 * (t % bs) + 4] = p[t]
    q = torch.stack([q[0, 0].abs(), -q[0, 1].abs(), q[0, 2].abs() * 8, q[0, 3].abs() * 0])[None].contiguous()
    want, bound = ref.decode(q, kc, vc, tables, ln, 0.125, bs)
    _check("int4 decode rising logits", _run(q, kc, vc, tables, ln, 0.125), want, bound)


def test_decode_mixed_value_scales():
    """Value rows whose scales differ by up to 2^20 in one sequence."""
    L, D, bs, H = 500, 128, 16, 1
    q, kc, vc, tables, ln = _problem([L], 4, H, D, bs, seed=6)
    g = torch.Generator().manual_seed(9)
    nb = vc.shape[0]
    mag = torch.exp2(torch.randint(-10, 11, (nb, H, bs, 1), generator=g).float())
    b, p = ref.pack_row(*ref.quantise((torch.randn(nb, H, bs, D, generator=g) * mag).to(torch.bfloat16)))
    vc = torch.cat([b.reshape(nb, H, -1), p.reshape(nb, H, -1)], -1).contiguous()
    want, bound = ref.decode(q, kc, vc, tables, ln, 0.088, bs)
    _check("int4 decode mixed value scales", _run(q, kc, vc, tables, ln, 0.088), want, bound)


def test_decode_nan_rows_and_queries_stay_in_their_head():
    q, kc, vc, tables, ln = _problem([100, 100, 100], 8, 2, 128, 16, seed=8)
    D, bs = 128, 16
    nan = torch.tensor([0.0, float("nan")]).to(torch.bfloat16).view(torch.uint8)
    at = bs * D // 2
    kc[int(tables[0, 3]), 1, at + 4 * 5:at + 4 * 5 + 4] = nan     # key row 53 of sequence 0, KV head 1
    vc[int(tables[1, 0]), 0, at:at + 4] = nan                     # value row 0 of sequence 1, KV head 0
    q[2, 3, 17] = float("inf")
    vc[int(tables[0, 6]), :, at + 4 * 4:] = 0xFF                  # rows past the length are not read
    kc[int(tables[0, 6]), :, at + 4 * 4:] = 0xFF
    want, bound = ref.decode(q, kc, vc, tables, ln, 0.088, bs)
    out = _run(q, kc, vc, tables, ln, 0.088).cpu().double()
    bad = torch.zeros(3, 8, dtype=torch.bool)
    bad[0, 4:], bad[1, :4], bad[2, 3] = True, True, True
    assert bool(out[bad].isnan().all()) and not bool(out[~bad].isnan().any())
    assert bool(((out - want).abs() <= bound)[~bad].all())


def test_decode_bad_table_entry():
    """An entry outside the cache is not followed: that sequence is NaN, the status says so, the others hold."""
    q, kc, vc, tables, ln = _problem([70, 200, 90], 4, 2, 64, 16, seed=2)
    want, bound = ref.decode(q, kc, vc, tables, ln, 0.125, 16)
    for entry in (-1, kc.shape[0], 2 ** 31 - 1, -2 ** 31):
        t = tables.clone()
        t[1, 7] = entry
        out = _run(q, kc, vc, t, ln, 0.125).cpu().double()
        assert ops.device_status() == -7
        assert bool(out[1].isnan().all())
        for i in (0, 2):
            assert bool(((out[i] - want[i]).abs() <= bound[i]).all())
    assert ops.device_status() == 0


def test_decode_length_past_the_table_row():
    q, kc, vc, tables, ln = _problem([64, 50], 4, 2, 64, 16, seed=2)
    want, bound = ref.decode(q, kc, vc, tables, ln, 0.125, 16)
    ln[0] = 65
    _check("int4 decode length past the row", _run(q, kc, vc, tables, ln, 0.125), want, bound)
    ln[0] = 2 ** 31 - 1
    _check("int4 decode huge length", _run(q, kc, vc, tables, ln, 0.125), want, bound)


def test_decode_shared_blocks():
    """The same blocks in several sequences and twice in one."""
    q, kc, vc, tables, ln = _problem([100, 100, 100], 4, 2, 64, 16, seed=2)
    tables[1] = tables[0]
    tables[2, 3:5] = tables[2, 0]
    want, bound = ref.decode(q, kc, vc, tables, ln, 0.125, 16)
    _check("int4 decode shared blocks", _run(q, kc, vc, tables, ln, 0.125), want, bound)


def test_decode_repeats_bit_for_bit():
    """The same call gives the same bits (partial results are joined in a fixed order), on one workspace."""
    q, kc, vc, tables, ln = _problem([5000, 3, 900, 0, 77], 16, 2, 128, 16, seed=3)
    ws = ops.new_int4_workspace(16, 2, 128)
    dev = [t.to(DEV) for t in (q, kc, vc, tables, ln)]
    first = ops.decode_int4(*dev, 0.088, ws).clone()
    for _ in range(20):
        assert torch.equal(ops.decode_int4(*dev, 0.088, ws), first)
    # another shape on the same workspace in between
    q2, kc2, vc2, t2, l2 = _problem([64, 2000], 4, 4, 64, 8, seed=5)
    want, bound = ref.decode(q2, kc2, vc2, t2, l2, 0.125, 8)
    _check("int4 decode on a used workspace", _run(q2, kc2, vc2, t2, l2, 0.125, ws=ws), want, bound)
    assert torch.equal(ops.decode_int4(*dev, 0.088, ws), first)


def test_decode_two_streams_and_a_graph():
    """Two calls at once on two workspaces, and a captured call replayed on new lengths and queries."""
    q, kc, vc, tables, ln = _problem([4000, 100, 9], 8, 2, 128, 16, seed=13)
    want, bound = ref.decode(q, kc, vc, tables, ln, 0.088, 16)
    dev = [t.to(DEV) for t in (q, kc, vc, tables, ln)]
    wss = [ops.new_int4_workspace(8, 2, 128) for _ in range(2)]
    outs = [torch.zeros_like(dev[0]) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, w, o in zip(streams, wss, outs):
            ops.decode_int4(*dev, 0.088, w, out=o, stream=s)
    torch.cuda.synchronize()
    for o in outs:
        _check("int4 decode two streams", o, want, bound)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.decode_int4(*dev, 0.088, wss[0], out=outs[0])
    ln2 = torch.tensor([1000, 0, 16], dtype=torch.int32)
    dev[4].copy_(ln2)
    dev[0].copy_(-q.to(DEV))
    for _ in range(3):
        graph.replay()
    want, bound = ref.decode(-q, kc, vc, tables, ln2, 0.088, 16)
    _check("int4 decode replayed", outs[0], want, bound)


def test_decode_cache_past_2_31_bytes():
    """Blocks beyond byte 2^31 of the caches."""
    D, bs, H = 128, 16, 8
    rec = ops.int4_record_bytes(bs, D)
    nb = (2 ** 31) // (rec * H) + 4000
    q, kc, vc, tables, ln = _problem([50, 300, 1], 16, H, D, bs, seed=21)
    n = kc.shape[0]
    big = [torch.zeros(nb, H, rec, dtype=torch.uint8, device=DEV) for _ in range(2)]
    for b, c in zip(big, (kc, vc)):
        b[nb - n:] = c.to(DEV)
    want, bound = ref.decode(q, kc, vc, tables, ln, 0.088, bs)
    moved = torch.where(tables < n, tables + (nb - n), tables)
    out = ops.decode_int4(q.to(DEV), *big, moved.to(DEV), ln.to(DEV), 0.088, ops.new_int4_workspace(16, H, D))
    _check("int4 decode past 2^31 bytes", out, want, bound)
    # the write and the read-back reach the same blocks
    rows = _bf(2, H, D, seed=1).to(DEV)
    slots = torch.tensor([nb * bs - 1, 5], device=DEV)
    ops.reshape_and_cache_int4(rows, rows, *big, slots)
    ko, _ = ops.dequantize_blocks_int4(*big, torch.tensor([nb - 1], dtype=torch.int32, device=DEV), D)
    codes, p = ref.quantise(rows[0].cpu())
    val = p[..., 1:].double() + p[..., :1].double() * codes.double()
    assert bool(((ko[0, bs - 1].cpu().double() - val).abs() <= val.abs() * 2.0 ** -8 * 1.001).all())


def test_decode_refusals():
    q, kc, vc, tables, ln = [t.to(DEV) for t in _problem([20], 4, 2, 64, 16)]
    ws = ops.new_int4_workspace(4, 2, 64)
    with pytest.raises(ops.PagedKVError, match="workspace"):
        ops.decode_int4(q, kc, vc, tables, ln, 0.1, ws[:-16])
    with pytest.raises(ops.PagedKVError, match="unsupported"):
        ops.decode_int4(torch.zeros(1, 34, 64, dtype=torch.bfloat16, device=DEV), kc, vc, tables, ln, 0.1, ws)
    with pytest.raises(ValueError):
        ops.decode_int4(q, kc, vc[:1], tables, ln, 0.1, ws)
    with pytest.raises(ValueError):
        ops.decode_int4(q, kc, vc, tables, ln.repeat(2), 0.1, ws)
    with pytest.raises(ValueError):
        ops.decode_int4(q, kc, vc, tables, ln, 0.1, ws, out=torch.zeros(1, 2, 64, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(TypeError):
        ops.decode_int4(q.float(), kc, vc, tables, ln, 0.1, ws)
    empty = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    assert ops.decode_int4(empty, kc, vc, tables[:0], ln[:0], 0.1, ws).shape == (0, 4, 64)
