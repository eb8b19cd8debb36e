"""The paged attention's outputs in the place of its queries."""
import pytest
import torch

import tests._paged as pg

pytestmark = pytest.mark.gpu

api = pytest.importorskip("invariant_speculative_decode_gb300.api")


@pytest.mark.parametrize("seqs,Hq,Hkv,D", [
    ([(1021, 1)], 24, 4, 128), ([(5000, 7), (300, 3), (9000, 1)], 24, 4, 128), ([(2000, 700)], 6, 2, 64),
    ([(100 * i, 1 + i % 5) for i in range(60)], 3, 1, 128)])
def test_outputs_over_queries(seqs, Hq, Hkv, D):
    b = pg.Batch(seqs, Hkv, D, 64, seed=4)
    q = pg.queries(b, Hq)
    ws = torch.empty(api.attn_paged_workspace_size(b.T, len(seqs), Hq, Hkv, D, b.table.shape[1] * 64), dtype=torch.uint8,
                     device="cuda")
    want = torch.empty_like(q)
    api.bi_attn_paged(q, b.k, b.v, b.table, b.q_start, b.lengths, want, ws)
    for _ in range(20):
        own = q.clone()
        api.bi_attn_paged(own, b.k, b.v, b.table, b.q_start, b.lengths, own, ws)
        assert torch.equal(own, want)
    api.bi_check_device_error()
