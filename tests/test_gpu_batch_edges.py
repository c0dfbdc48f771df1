"""GPU: batch preparation with lengths updated in place, on both sides of the sizes where its form changes."""

import pytest
import torch

import _int4_ref as ref
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
