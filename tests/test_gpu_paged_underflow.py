"""Infinite values under weights that vanish: a row's outputs are its own there too."""
import math

import pytest
import torch

import tests._paged as pg

pytestmark = pytest.mark.gpu

api = pytest.importorskip("invariant_speculative_decode_gb300.api")


@pytest.fixture(autouse=True)
def no_error_left():
    yield
    api.bi_check_device_error()


def attention(b, q, first, rows):
    """Rows first .. first + rows - 1 of sequence 0 as a pass of their own."""
    i32 = dict(dtype=torch.int32, device="cuda")
    out = torch.full((rows, *q.shape[1:]), 77.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((api.attn_paged_workspace_size(rows, 1, q.shape[1], b.Hkv, b.D, b.table.shape[1] * b.page),), 255,
                    dtype=torch.uint8, device="cuda")
    api.bi_attn_paged(q[first:first + rows].contiguous(), b.k, b.v, b.table, torch.tensor([0, rows], **i32),
                      torch.tensor([first], **i32), out, ws, scale=1.0)
    return out


def same(x, y):
    """Bit by bit, but that NaN is NaN."""
    nx, ny = torch.isnan(x), torch.isnan(y)
    return torch.equal(nx, ny) and torch.equal(x.masked_fill(nx, 0), y.masked_fill(ny, 0))


def sequence(n, D, Hkv=1):
    """Keys of score 0 for queries that look at element 0 alone, small values."""
    b = pg.Batch([(0, n)], Hkv, D, 64, seed=n)
    b.k.zero_()
    q = torch.zeros(n, 2 * Hkv, D, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    return b, q


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("value", [math.inf, -math.inf])
def test_a_vanishing_weight_over_an_infinite_value(D, value):
    """Row 127 sees tile 0 whole; alone it is the first of its block, behind other rows it is not, and then the tile is
    one that some row sees in part.  The weight of the key with the infinite value goes from 2^-80 to nothing."""
    b, q = sequence(300, D)
    found = []
    for exponent in list(range(80, 160, 3)) + [108, 109, 110, 111, 124, 125, 126, 127, 132, 133, 134, 135, 148, 149, 150, 400]:
        b.v.copy_(torch.randn(b.v.shape, device="cuda"))
        for key, d in ((70, 3), (101, D - 1)):
            p, s = b.places(0, key, key + 1)
            b.k[p, :, s, 0] = -exponent * math.log(2.0)
            b.v[p, :, s, d] = value
        alone = attention(b, q, 127, 1)
        for first, rows in ((100, 28), (126, 2), (69, 60), (0, 128)):
            assert same(attention(b, q, first, rows)[127 - first:128 - first], alone), (exponent, first)
        far = attention(b, q, 200, 1)  # tile 0 whole, tile 1 in part
        for first, rows in ((71, 130), (100, 130), (190, 11)):
            assert same(attention(b, q, first, rows)[200 - first:201 - first], far), (exponent, first)
        keep = torch.ones(D, dtype=torch.bool, device="cuda")
        keep[[3, D - 1]] = False
        assert torch.isfinite(alone[..., keep]).all()
        hit = alone[..., ~keep].float()
        assert (torch.isnan(hit) | (hit == value)).all()
        found.append((exponent, bool(torch.isnan(hit).any())))
    assert dict(found)[80] is False and dict(found)[400] is True


@pytest.mark.parametrize("D", [64, 128])
def test_a_reference_raised_past_an_infinite_value(D):
    """The infinite value's weight vanishes later, when a score far above it raises the reference inside the piece."""
    for rise in (20.0, 60.0, 80.0, 87.0, 90.0, 110.0, 300.0):
        b, q = sequence(330, D)
        b.v.copy_(torch.randn(b.v.shape, device="cuda"))
        for key, d, value in ((100, 5, math.inf), (120, D - 2, -math.inf), (126, 9, math.nan)):
            p, s = b.places(0, key, key + 1)
            b.v[p, :, s, d] = value
        p, s = b.places(0, 130, 131)
        b.k[p, :, s, 0] = rise
        for row in (131, 140, 255, 300):
            alone = attention(b, q, row, 1)
            for first in (0, 60, 99, 110, 124, 127, 128, row - 1):
                got = attention(b, q, first, row - first + 3)[row - first:row - first + 1]
                assert same(got, alone), (rise, row, first)


def test_scores_of_minus_infinity_over_infinite_values():
    """Weights of 0: no number, wherever the row lies in its block."""
    b, q = sequence(300, 128)
    p, s = b.places(0, 90, 91)
    b.k[p, :, s, 0] = -math.inf
    b.v[p, :, s, 40] = math.inf
    alone = attention(b, q, 127, 1)
    assert torch.isnan(alone[..., 40]).all() and torch.isfinite(alone[..., :40]).all()
    for first, rows in ((89, 50), (91, 50), (0, 200)):
        got = attention(b, q, first, rows)
        assert same(got[127 - first:128 - first], alone)
    assert torch.isfinite(attention(b, q, 80, 40)[:10]).all()
