"""GPU: a step's tables, lengths, positions and slots against the definition, and
the whole 4-bit serving step run as a user would."""

import numpy as np
import pytest
import torch

import _int4_ref as ref
from paged_kv_cache_379_b200 import ops

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).to(DEV)


class Step:
    """A batch's device arrays, poisoned where the operator has to write."""

    def __init__(self, ctx, new, bs, nb, width, room, seed=0, num_free=None, free=None):
        rng = np.random.default_rng(seed)
        B = len(ctx)
        self.ctx, self.new, self.bs, self.nb, self.room = np.array(ctx), np.array(new), bs, nb, room
        have = np.maximum(0, -(-self.ctx // bs))
        perm = rng.permutation(nb).astype(np.int32)
        used = int(have.sum())
        tables = np.full((B, width), -7, np.int32)
        at = 0
        for s in range(B):
            n = min(int(have[s]), width)
            tables[s, :n] = perm[at:at + n]
            at += n
        self.free = np.concatenate([perm[used:], np.full(used, 1 << 30, np.int32)]) if free is None else free
        self.num_free = nb - used if num_free is None else num_free
        self.tables = tables
        i32, i64 = torch.int32, torch.int64
        self.d = dict(block_tables=_dev(tables, i32), context_lens=_dev(ctx, i32), query_lens=_dev(new, i32),
                      free_blocks=_dev(self.free, i32), num_free=_dev([self.num_free], i32))
        self.o = dict(seq_lens=_dev(np.full(B, 99), i32), q_start=_dev(np.full(B + 1, 99), i32),
                      seq_ids=_dev(np.full(room, 99), i32), positions=_dev(np.full(room, 99), i64),
                      slot_mapping=_dev(np.full(room, 99), i64), num_free_out=_dev([99], i32), status=_dev([99], i32))

    def run(self, **over):
        o = dict(self.o, **over)
        ops.prepare_batch(*self.d.values(), self.bs, self.nb, **o)
        return {k: v.cpu().numpy() for k, v in o.items() if isinstance(v, torch.Tensor)}

    def check(self, got):
        t, sl, qs, ids, pos, slots, left = ref.prepare_batch(self.tables, self.ctx, self.new, self.free, self.num_free,
                                                             self.bs, self.nb, self.room)
        assert (self.d["block_tables"].cpu().numpy() == t).all()
        assert (got["seq_lens"] == sl).all() and (got["q_start"] == qs).all()
        assert (got["seq_ids"] == ids).all() and (got["positions"] == pos).all()
        assert (got["slot_mapping"] == slots).all()
        assert got["num_free_out"][0] == left and got["status"][0] == 0


def _batch(B, ctx_high, new_low, new_high, bs, seed, pad=5):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, ctx_high + 1, B)
    new = rng.integers(new_low, new_high + 1, B)
    need = -(-(ctx + new) // bs)
    return Step(ctx, new, bs, int(need.sum()) + 3, int(need.max(initial=0)) + 2, int(new.sum()) + pad, seed)


@pytest.mark.parametrize("B,ctx_high,new_low,new_high", [
    (1, 0, 0, 0), (1, 40, 1, 1), (7, 50, 0, 3), (256, 300, 1, 1), (33, 100, 0, 90), (1024, 60, 1, 1), (1025, 60, 0, 2),
    (2500, 20, 0, 3), (5000, 9, 1, 1), (64, 500, 1, 400)])
@pytest.mark.parametrize("bs", [4, 8, 16, 32, 5])
def test_prepare(B, ctx_high, new_low, new_high, bs):
    s = _batch(B, ctx_high, new_low, new_high, bs, seed=B + bs)
    s.check(s.run())


def test_prepare_optional_outputs_and_aliases():
    """Without per-token arrays; lengths and the free count updated in place."""
    s = _batch(40, 100, 0, 9, 16, 3)
    got = s.run()
    s2 = _batch(40, 100, 0, 9, 16, 3)
    n = s2.room
    o = s2.run(seq_ids=None, positions=None, slot_mapping=None, seq_lens=s2.d["context_lens"],
               num_free_out=s2.d["num_free"], num_tokens=n)
    assert (o["seq_lens"] == got["seq_lens"]).all() and o["num_free_out"][0] == got["num_free_out"][0]
    assert torch.equal(s.d["block_tables"], s2.d["block_tables"])
    with pytest.raises(ValueError, match="num_tokens"):
        s2.run(seq_ids=None, positions=None, slot_mapping=None)


def _refused(s, status):
    """Nothing handed out: tables as they were, lengths the cached ones, every row -1."""
    before = s.d["block_tables"].clone()
    got = s.run()
    width = s.tables.shape[1]
    assert got["status"][0] == status
    assert torch.equal(before, s.d["block_tables"])
    assert (got["seq_lens"] == np.clip(s.ctx, 0, width * s.bs)).all()
    assert (got["q_start"] == 0).all() and (got["slot_mapping"] == -1).all()
    assert (got["positions"] == -1).all() and (got["seq_ids"] == -1).all()
    assert got["num_free_out"][0] == s.num_free


def test_prepare_refusals():
    mk = lambda **kw: Step([17, 32, 5], [4, 1, 40], 16, 40, 6, 60, **kw)  # noqa: E731
    s = mk()
    s.check(s.run())
    for n in (4, 3):       # 0 + 1 + 2 blocks are needed: 17+4 stay in 2, 32+1 open a third, 5+40 take 1 to 3
        s = mk(num_free=n)
        s.check(s.run())
    _refused(mk(num_free=2), -6)
    _refused(mk(num_free=-1), -2)
    _refused(mk(num_free=41), -2)                                   # above the stack's capacity
    _refused(Step([17, 32, 5], [4, 1, 40], 16, 40, 6, 44), -2)      # 45 new tokens, 44 rows
    _refused(Step([17, 95, 5], [4, 2, 40], 16, 40, 6, 60), -2)      # past the table row
    _refused(Step([17, -1, 5], [4, 1, 40], 16, 40, 6, 60), -2)
    _refused(Step([17, 32, 5], [4, -1, 40], 16, 40, 6, 60), -2)
    _refused(Step([17, 32, 5], [4, 2 ** 31 - 1, 40], 16, 40, 6, 60), -2)


def test_prepare_bad_free_block():
    """A free block outside the cache: its entry and slots are -1, the status says so, the rest holds."""
    free = np.arange(40, dtype=np.int32)
    free[38] = 40
    s = Step([16, 16, 3], [1, 2, 4], 16, 40, 4, 9, free=free, num_free=40)
    got = s.run()
    t, _, _, _, _, slots, left = ref.prepare_batch(s.tables, s.ctx, s.new, free, 40, 16, 40, 9)
    assert got["status"][0] == -7 and (s.d["block_tables"].cpu().numpy() == t).all()
    assert (got["slot_mapping"] == slots).all() and (slots == -1).sum() == 4 and got["num_free_out"][0] == left


@pytest.mark.parametrize("B", [1, 40, 1500])
def test_release_returns_what_prepare_took(B):
    s = _batch(B, 60, 1, 5, 8, B)
    s.run(num_free_out=s.d["num_free"])
    rng = np.random.default_rng(B)
    mark = (rng.random(B) < 0.5).astype(np.int32) * 3
    tables, lens = s.d["block_tables"].cpu().numpy(), s.o["seq_lens"].cpu().numpy()
    nf = int(s.d["num_free"])
    stack = s.d["free_blocks"].cpu().numpy()[:nf].tolist()
    want_t, want_l = tables.copy(), lens.copy()
    for i in np.flatnonzero(mark):
        n = -(-int(lens[i]) // 8)
        stack += tables[i, :n].tolist()
        want_t[i, :n] = -1
        want_l[i] = 0
    status = _dev([99], torch.int32)
    ops.release_blocks(s.d["block_tables"], s.o["seq_lens"], _dev(mark, torch.int32), s.d["free_blocks"],
                       s.d["num_free"], 8, s.nb, status=status)
    assert int(status) == 0 and int(s.d["num_free"]) == len(stack)
    assert s.d["free_blocks"].cpu().numpy()[:len(stack)].tolist() == stack
    assert (s.d["block_tables"].cpu().numpy() == want_t).all() and (s.o["seq_lens"].cpu().numpy() == want_l).all()


@pytest.mark.parametrize("fault,status", [("entry", -7), ("length", -2), ("full", -2), ("count", -2)])
def test_release_refusals_change_nothing(fault, status):
    s = Step([17, 32, 5], [0, 0, 0], 16, 40, 6, 0)
    lens = _dev([17, 32, 5], torch.int32)
    mark = _dev([1, 0, 1], torch.int32)
    if fault == "entry":
        s.d["block_tables"][2, 0] = 40
    elif fault == "length":
        lens[0] = 97
    elif fault == "full":
        s.d["free_blocks"] = s.d["free_blocks"][:37].contiguous()   # 35 free + 3 released > 37
    else:
        s.d["num_free"].fill_(-2)
    keep = [t.clone() for t in (s.d["block_tables"], lens, s.d["free_blocks"], s.d["num_free"])]
    st = _dev([99], torch.int32)
    ops.release_blocks(s.d["block_tables"], lens, mark, s.d["free_blocks"], s.d["num_free"], 16, 40, status=st)
    assert int(st) == status
    for a, b in zip(keep, (s.d["block_tables"], lens, s.d["free_blocks"], s.d["num_free"])):
        assert torch.equal(a, b)


# ---- the operators together --------------------------------------------------------------

def _serve(Hq, H, D, bs, B, steps, graph):
    """A chunk for every request, then single tokens: tables and slots on the device, norm + rotation + 4-bit
    write, decode -- every output against the 64-bit form over the caches that the step left."""
    rng = np.random.default_rng(B)
    g = torch.Generator().manual_seed(B)
    width, nb, room = 8, 8 * B + 5, 12 * B
    rot = D
    a = torch.arange(width * bs, dtype=torch.float64)[:, None] * 10000.0 ** (
        -torch.arange(0, rot, 2, dtype=torch.float64) / rot)[None]
    cs = torch.cat([a.cos(), a.sin()], -1).float().to(DEV)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)  # noqa: E731
    i64 = lambda *s: torch.zeros(*s, dtype=torch.int64, device=DEV)  # noqa: E731
    tables = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    lens, new, free, nf = i32(B), i32(B), torch.randperm(nb, generator=g).to(torch.int32).to(DEV), i32(1)
    nf.fill_(nb)
    out = dict(q_start=i32(B + 1), positions=i64(room), slot_mapping=i64(room), status=i32(1))
    kc, vc = ops.new_int4_cache(nb, bs, H, D), ops.new_int4_cache(nb, bs, H, D)
    ws = ops.new_int4_workspace(Hq, H, D)
    qkv = torch.zeros(room, (Hq + 2 * H) * D, dtype=torch.bfloat16, device=DEV)
    qw = (1 + 0.1 * torch.randn(D, generator=g)).to(torch.bfloat16).to(DEV)
    q, k, v = qkv.split([Hq * D, H * D, H * D], dim=1)
    q, k, v = q.view(room, Hq, D), k.view(room, H, D), v.view(room, H, D)
    qo = torch.zeros(room, Hq, D, dtype=torch.bfloat16, device=DEV)
    last = torch.zeros(B, Hq, D, dtype=torch.bfloat16, device=DEV)
    o = torch.zeros_like(last)
    scale = 1 / D ** 0.5

    def step():
        ops.prepare_batch(tables, lens, new, free, nf, bs, nb, seq_lens=lens, num_free_out=nf, **out)
        ops.qk_norm_rope_cache_int4(q, k, v, qw, None, cs, out["positions"], out["slot_mapping"], kc, vc, query_out=qo)
        last.copy_(qo[(out["q_start"][1:] - 1).clamp(min=0).long()])
        ops.decode_int4(last, kc, vc, tables, lens, scale, ws, out=o)

    captured = None
    total = np.zeros(B, np.int64)
    for i in range(steps):
        n = rng.integers(1, 12, B) if i == 0 else np.ones(B, np.int64)
        new.copy_(_dev(n, torch.int32))
        qkv.copy_(torch.randn(*qkv.shape, generator=g).to(torch.bfloat16))
        if graph and i == 1:
            keep = [t.clone() for t in (tables, lens, nf)]
            captured = torch.cuda.CUDAGraph()
            with torch.cuda.graph(captured):
                step()
            for t, was in zip((tables, lens, nf), keep):
                assert torch.equal(t, was)
        captured.replay() if captured else step()
        total += n
        assert int(out["status"]) == 0 and (lens.cpu().numpy() == total).all()
        used = tables.cpu().numpy()
        ids = np.concatenate([used[s, :-(-int(total[s]) // bs)] for s in range(B)])
        assert len(set(ids.tolist())) == len(ids) and int(nf) == nb - len(ids)
        want, bound = ref.decode(last.cpu(), kc.cpu(), vc.cpu(), tables.cpu(), lens.cpu(), scale, bs)
        assert bool(((o.cpu().double() - want).abs() <= bound).all())
        # the cached keys are the plain form's, within the norm's bound and half a code
        rows, pos = int(out["q_start"][-1]), out["positions"].cpu()
        yk, bk = ref.norm_rope(k[:rows].cpu(), None, cs.cpu(), pos[:rows], False, 1e-6)
        slot = out["slot_mapping"].cpu()[:rows]
        got = ref.values(kc.cpu(), bs, D).reshape(-1, H, D)[slot]
        sc = ref.pairs(kc.cpu(), bs, D)[0].reshape(-1, H, 1)[slot]
        assert bool(((got - yk).abs() <= bk + sc * (0.5 + 15 * 2.0 ** -8 + 1e-3)).all())
    # finished requests give their blocks back
    st = i32(1)
    ops.release_blocks(tables, lens, torch.ones(B, dtype=torch.int32, device=DEV), free, nf, bs, nb, status=st)
    assert int(st) == 0 and int(nf) == nb and sorted(free.tolist()) == list(range(nb)) and not bool(lens.any())
    assert ops.device_status() == 0


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("Hq,H,D,bs,B", [(8, 2, 128, 16, 5), (4, 4, 64, 8, 9), (12, 1, 128, 32, 3)])
def test_serving_step(Hq, H, D, bs, B, graph):
    _serve(Hq, H, D, bs, B, steps=4, graph=graph)


def test_chunk_over_4bit_context_by_prefill():
    """A prompt chunk whose context is in the 4-bit cache: its blocks read back as bf16, then the prefill."""
    D, bs, H, Hq, L, n = 128, 16, 2, 8, 100, 30
    g = torch.Generator().manual_seed(1)
    nb = 12
    rows = torch.randn(2, L, H, D, generator=g).to(torch.bfloat16).to(DEV)
    table = torch.randperm(nb, generator=g)[:7].to(torch.int32)
    slots = (table.long()[torch.arange(L) // bs] * bs + torch.arange(L) % bs).to(DEV)
    kc, vc = ops.new_int4_cache(nb, bs, H, D), ops.new_int4_cache(nb, bs, H, D)
    ops.reshape_and_cache_int4(rows[0], rows[1], kc, vc, slots)
    kb, vb = ops.dequantize_blocks_int4(kc, vc, table.to(DEV), D)
    q = torch.randn(n, Hq, D, generator=g).to(torch.bfloat16)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    out = ops.prefill(q.to(DEV), kb, vb, torch.arange(7, dtype=torch.int32, device=DEV)[None], i32(L), i32(0, n), 0.088)
    tok = ops.decode_int4(q[-1:].to(DEV), kc, vc, table[None].to(DEV), i32(L), 0.088, ops.new_int4_workspace(Hq, H, D))
    # the chunk's last row is the decode of that token; bf16 key and value blocks: half a bf16 step of keys
    # (|q||k| summed over D, times the scale) and of values, and the bf16 outputs' own rounding
    k = kb.cpu().double().abs().amax()
    mag = float(q[-1].double().abs().sum(-1).max() * k * 0.088) * 2.0 ** -8
    v = float(vb.cpu().double().abs().amax())
    assert float((out[-1].double() - tok[0].double()).abs().max()) <= 2 * mag * v + 3 * v * 2.0 ** -8


@pytest.mark.parametrize("B,new_high", [(7, 3), (64, 400), (1500, 9)])
def test_prepare_in_place_equals_apart(B, new_high):
    """Lengths and the free count updated in place: the same integers, small steps and large ones."""
    a, b = (_batch(B, 100, 0, new_high, 16, B) for _ in range(2))
    want = a.run()
    got = b.run(seq_lens=b.d["context_lens"], num_free_out=b.d["num_free"])
    assert torch.equal(a.d["block_tables"], b.d["block_tables"])
    for k in want:
        assert (want[k] == got[k]).all(), k
    a.check(want)


def test_prepare_largest_rows():
    """The last positions of the widest row (15 blocks of 2^27: a 16th would pass 31 bits), one token past it,
    and a block size of one."""
    s = Step([15 * 2 ** 27 - 40], [9], 1 << 27, 40, 15, 12)
    s.check(s.run())
    _refused(Step([15 * 2 ** 27 - 8], [9], 1 << 27, 40, 15, 12), -2)
    s = Step([5, 0, 3], [2, 0, 4], 1, 40, 9, 8)
    s.check(s.run())
