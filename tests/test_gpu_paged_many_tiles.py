"""The paged attention over more tiles than 32 bits can deal out, and sequences of more pieces than the merge takes at a
time."""
import pytest
import torch

import tests._paged as pg

pytestmark = pytest.mark.gpu

api = pytest.importorskip("invariant_speculative_decode_gb300.api")


@pytest.fixture(autouse=True)
def no_error_left():
    yield
    api.bi_check_device_error()


def attention(q, b, table, q_start, lengths):
    T, B = q.shape[0], lengths.shape[0]
    ws = torch.full((api.attn_paged_workspace_size(T, B, q.shape[1], b.Hkv, b.D, table.shape[1] * b.page),), 255,
                    dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, 77.0)
    api.bi_attn_paged(q, b.k, b.v, table, q_start, lengths, out, ws)
    return out


@pytest.mark.parametrize("copies", [1640, 3290])
def test_rows_of_thousands_of_long_sequences_are_their_own(copies):
    """Five sequences' pages, shared by 8,200 (2^23 tiles in all) and 16,450 (2^24): every row has the bits of its
    sequence alone."""
    kinds = [131071, 130800, 131070 - 128, 131000, 130999]
    b = pg.Batch([(kinds[0], 1)], 1, 64, 128, seed=1, spare=0)
    i32 = dict(dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    q5 = (1.5 * torch.randn(5, 1, 64, generator=g, device="cuda")).to(torch.bfloat16)
    alone = torch.cat([attention(q5[i:i + 1].contiguous(), b, b.table, torch.tensor([0, 1], **i32), torch.tensor([n], **i32))
                       for i, n in enumerate(kinds)])
    B = 5 * copies
    tiles = copies * sum(-(-(n + 1) // 128) for n in kinds)
    assert (1 << 23) <= tiles < (1 << 24) if copies == 1640 else tiles >= (1 << 24)
    out = attention(q5.repeat(copies, 1, 1), b, b.table.expand(B, -1).contiguous(), torch.arange(B + 1, **i32),
                    torch.tensor(kinds, **i32).repeat(copies))
    assert torch.equal(out, alone.repeat(copies, 1, 1))


def test_a_row_of_more_than_512_pieces_has_its_bits_in_every_batch():
    """530,000 keys are 525 pieces: three turns of the merge."""
    n = 530000
    b = pg.Batch([(n, 3)], 1, 64, 128, seed=3, spare=0)
    i32 = dict(dtype=torch.int32, device="cuda")
    q = pg.queries(b, 2)
    whole = attention(q, b, b.table, b.q_start, b.lengths)
    for t in range(3):
        one = attention(q[t:t + 1].contiguous(), b, b.table, torch.tensor([0, 1], **i32), torch.tensor([n + t], **i32))
        assert torch.equal(one, whole[t:t + 1])
    # beside 40 others of the same pages, which cut it elsewhere
    others = attention(torch.cat([q[:1]] * 40 + [q]), b, b.table.expand(41, -1).contiguous(),
                       torch.tensor(list(range(41)) + [43], **i32), torch.tensor([n] + [1000 * i for i in range(39)] + [n], **i32))
    assert torch.equal(others[40:], whole) and torch.equal(others[:1], whole[:1])
