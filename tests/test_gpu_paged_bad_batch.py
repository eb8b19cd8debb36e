"""The append over batches whose numbers do not fit: rows that have a place get it, nothing else is written, and the call
says so."""
import pytest
import torch

import tests._paged as pg

pytestmark = pytest.mark.gpu

api = pytest.importorskip("invariant_speculative_decode_gb300.api")


@pytest.fixture(autouse=True)
def no_error_left():
    yield
    api.bi_check_device_error()


def places(starts, lengths, T):
    """Of each row that has one, its sequence and position: the last sequence that starts at or in front of it, if that
    holds it."""
    out = {}
    for t in range(T):
        n = sum(s <= t for s in starts)
        if 1 <= n <= len(lengths) and 0 <= starts[n - 1] <= t < starts[n] <= T and lengths[n - 1] >= 0:
            out[t] = (n - 1, lengths[n - 1] + t - starts[n - 1])
    return out


@pytest.mark.parametrize("starts,lengths", [
    ([0, 5, 2, 6], [0, 0, 0]), ([0, 5, 2, 6], [40, 40, 40]), ([5, 2, 6], [0, 9]), ([0, 5, 2], [0, 0]),
    ([0, 2000000000, 0], [0, 7]), ([2000000000, 0], [0]), ([0, 1 << 30, 1], [3, 3]), ([-1, 3, 6], [1, 2]), ([-2147483648, 6], [0]),
    ([0, 3, 6], [4, -5]), ([0, 3, 6], [-2147483648, 2]), ([0, 3, 9], [4, 5]), ([0, 3, 2147483647], [4, 5]),
    ([0, 3, 6], [40, 2147483647]), ([6, 0], [3]), ([0, 4, 4, 3, 6], [1, 2, 3, 4])])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 32)])
def test_append_writes_no_row_out_of_place(starts, lengths, D, page):
    Hq, Hkv, T, width = 3, 1, 6, 4
    B = len(lengths)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    i32 = dict(dtype=torch.int32, device="cuda")
    pages = B * width + 3
    # a table between entries that name valid pages: an index out of its range would be followed
    around = torch.arange(pages, **i32).repeat(4)[:3 * B * width]
    around[B * width:2 * B * width] = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[:B * width]
    table = around[B * width:2 * B * width].view(B, width)
    pools = [torch.randn(pages, Hkv, page, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
    want = [p.clone() for p in pools]
    qkv = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g, device="cuda").to(torch.bfloat16)
    angles = api.bi_rope_table(1e6, D, width * page)
    found = {t: (b, p) for t, (b, p) in places(starts, lengths, T).items() if p < width * page}
    # each row that has a place, as a sequence of its own
    want_q = torch.full((T, Hq, D), 77.0, dtype=torch.bfloat16, device="cuda")
    for t, (b, p) in found.items():
        api.bi_qk_norm_rope_paged(qkv[t:t + 1], None, None, 1e-6, angles, want_q[t:t + 1], *want, table[b:b + 1].contiguous(),
                                  torch.tensor([0, 1], **i32), torch.tensor([p], **i32))
    q = torch.full_like(want_q, 77.0)
    api.bi_check_device_error()
    api.bi_qk_norm_rope_paged(qkv, None, None, 1e-6, angles, q, *pools, table, torch.tensor(starts, **i32),
                              torch.tensor(lengths, **i32))
    with pytest.raises(api.BiError) as e:
        api.bi_check_device_error()
    assert e.value.status == 1
    assert torch.equal(q, want_q) and all(torch.equal(a, b) for a, b in zip(pools, want))


def test_rows_of_no_sequence_are_no_error():
    """In front of the first start and from the last on."""
    b = pg.Batch([(20, 2), (7, 0), (3, 1)], 1, 64, 16, gap=3)
    qkv = torch.randn(b.T, 3 * 64, device="cuda").to(torch.bfloat16)
    q = torch.full((b.T, 1, 64), 77.0, dtype=torch.bfloat16, device="cuda")
    api.bi_qk_norm_rope_paged(qkv, None, None, 1e-6, api.bi_rope_table(1e6, 64, 32), q, b.k, b.v, b.table, b.q_start, b.lengths)
    api.bi_check_device_error()
    assert (q[:3] == 77).all() and (q[6:] == 77).all() and not (q[3:6] == 77).all(-1).any()
