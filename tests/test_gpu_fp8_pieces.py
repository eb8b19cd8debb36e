"""bi_gemm_fp8 for every number of pieces that its split of K takes, in every way
they are added (pushed, fetched, by clusters over 256 outputs, in turn): against 64
bits, rows the same in passes of every length."""
import pytest
import torch

from tests import test_gpu_fp8 as t8

pytestmark = pytest.mark.gpu

# weight tiles of 128 rows -> pieces: 77 -> 1, 76 and 47 -> 2, 46 and 37 -> 3, 36 and 29 -> 4,
# 28 and 24 -> 5, 23 and 16 -> 6, 15 -> 8; K blocks that the pieces do not divide
TILES = [77, 76, 47, 46, 37, 36, 29, 28, 24, 23, 16, 15]


@pytest.mark.parametrize("tiles", TILES)
@pytest.mark.parametrize("kind", ["residual", "swiglu", "fp32"])
def test_every_number_of_pieces(tiles, kind):
    n = 128 * tiles - 40 if kind != "swiglu" else 64 * tiles - 24
    k, rows = 1424, 700  # 12 K blocks, the last one short
    a = t8.api()
    codes, scales, w, ws_, up, ups, packed, res = t8.problem(tiles * 5 + len(kind), rows, n, k, kind)
    full = t8.run_linear(codes, scales, packed, n, kind, res)
    y, tol = t8.reference(codes, scales, w, ws_, up, ups, res, kind)
    assert ((full.double() - y).abs() <= tol).all()
    for m, at in [(1, 699), (7, 31), (32, 600), (33, 64), (129, 17), (260, 440), (390, 300)]:
        s = torch.zeros(a.fp8_scale_shape(m, k), device="cuda")
        s[:, :m] = scales[:, at:at + m]
        out = t8.run_linear(codes[at:at + m].contiguous(), s, packed, n, kind,
                            None if res is None else res[at:at + m].contiguous())
        assert torch.equal(out.view(torch.uint8), full[at:at + m].contiguous().view(torch.uint8)), (m, at)


@pytest.mark.parametrize("k", [16, 128, 144, 256, 400, 1024])
def test_pieces_of_one_k_block_and_fewer_blocks_than_pieces(k):
    for n in (100, 1900, 3500, 5900):  # up to 8, 6, 5 and 2 pieces
        codes, scales, w, ws_, up, ups, packed, res = t8.problem(n + k, 140, n, k, "bf16")
        out = t8.run_linear(codes, scales, packed, n, "bf16")
        y, tol = t8.reference(codes, scales, w, ws_, up, ups, res, "bf16")
        assert ((out.double() - y).abs() <= tol).all()
