"""GPU: batch preparation with lengths updated in place, on both sides of the sizes where its form changes, and with
as many rows as the entry point takes."""

import pytest
import torch

import _int4_ref as ref
from paged_kv_cache_379_b200 import ops
from test_gpu_batch import _batch

pytestmark = pytest.mark.gpu


# 4096 rows are filled by the one CTA, more by a second launch; 2048 requests fit its copies
@pytest.mark.parametrize("B,new_high", [(7, 3), (64, 60), (64, 400), (2048, 1), (2049, 1), (2500, 9)])
@pytest.mark.parametrize("which", ["context_lens", "query_lens"])
def test_lengths_in_place(B, new_high, which):
    """seq_lens as either of the two inputs."""
    s = _batch(B, 100, 0, new_high, 16, B + new_high)
    got = s.run(seq_lens=s.d[which])
    tables, lens, starts, ids, pos, slots, left = ref.prepare_batch(s.tables, s.ctx, s.new, s.free, s.num_free, s.bs,
                                                                    s.nb, s.room)
    assert got["status"][0] == 0 and got["num_free_out"][0] == left
    assert (s.d["block_tables"].cpu().numpy() == tables).all()
    assert (s.d[which].cpu().numpy() == lens).all() and (got["q_start"] == starts).all()
    assert (got["seq_ids"] == ids).all() and (got["positions"] == pos).all() and (got["slot_mapping"] == slots).all()


@pytest.mark.parametrize("rows", [2 ** 31 - 1, 2 ** 31 - 1500])
def test_most_rows(rows):
    """Row arrays of nearly 2^31 entries (8.6 GB): every one is written, those past the last token with -1."""
    s = _batch(40, 100, 0, 9, 16, 3)
    ids = torch.zeros(rows, dtype=torch.int32, device="cuda")
    o = dict(s.o, seq_ids=ids, positions=None, slot_mapping=None)
    ops.prepare_batch(*s.d.values(), s.bs, s.nb, **o)
    want = ref.prepare_batch(s.tables, s.ctx, s.new, s.free, s.num_free, s.bs, s.nb, s.room)
    n = s.room
    assert int(o["status"]) == 0 and (ids[:n].cpu().numpy() == want[3]).all()
    for a in range(n, rows, 1 << 28):
        assert bool((ids[a:a + (1 << 28)] == -1).all())
