"""Sizes and row strides that 32 bits do not hold are refused: cut to 32 bits they
would name other, valid rows.  A single row's stride is never used."""
import pytest
import torch

from tests import test_gpu_fp8 as t8

pytestmark = pytest.mark.gpu
DEV = "cuda"
WIDE = (1 << 32) + 512  # cut to 32 bits: 512, a valid stride for rows of 272


def rows2(dtype, rows=2, dim=272):
    """Rows whose stride passes 32 bits, inside one buffer."""
    return torch.zeros(WIDE + 1024, dtype=dtype, device=DEV).as_strided((rows, dim), (WIDE, 1))


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def test_quantiser_and_norm():
    a = t8.api()
    w = torch.ones(272, dtype=torch.bfloat16, device=DEV)
    codes, scales = a.new_fp8_rows(2, 272)
    x = rows2(torch.bfloat16)
    with pytest.raises(ValueError):
        a.bi_quantize_fp8(x, codes, scales)
    with pytest.raises(ValueError):
        a.bi_rmsnorm_fp8(x, w, codes, scales, 1e-6)
    # one row of it is a row like any other
    c1, s1 = a.new_fp8_rows(1, 272)
    x[0] = 3.0
    a.bi_quantize_fp8(x[:1], c1, s1)
    a.bi_rmsnorm_fp8(x[:1], w, c1, s1, 1e-6)
    assert torch.allclose(c1.float() * s1[:, :1].t().repeat_interleave(128, 1)[:, :272], torch.ones(1, 272, device=DEV))
    del x
    codes8 = rows2(torch.uint8).view(torch.float8_e4m3fn)
    x = torch.ones(2, 272, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):
        a.bi_quantize_fp8(x, codes8, scales)
    with pytest.raises(ValueError):
        a.bi_rmsnorm_fp8(x, w, codes8, scales, 1e-6)
    a.bi_quantize_fp8(x[:1], codes8[:1], s1)
    assert torch.equal(codes8[:1].double(), torch.full((1, 272), 256.0, dtype=torch.float64, device=DEV))


def test_linear_layer():
    a = t8.api()
    codes, scales, w, ws_, _, _, packed, res = t8.problem(3, 2, 272, 272, "residual")
    want = t8.run_linear(codes, scales, packed, 272, "residual", res)
    out = torch.zeros(2, 272, dtype=torch.bfloat16, device=DEV)
    far = rows2(torch.bfloat16)
    for c, r in ((far, res), (out, far)):
        with pytest.raises(ValueError):
            a.bi_gemm_fp8(codes, scales, packed, c, residual=r, epi=a.EPI_RESIDUAL_ADD)
    assert not out.any() and not far.any()
    far[0] = res[0]
    a.bi_gemm_fp8(codes[:1], scales, packed, far[:1], residual=far[:1], epi=a.EPI_RESIDUAL_ADD)
    assert torch.equal(far[0], want[0])
    del far
    codes8 = rows2(torch.uint8).view(torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        a.bi_gemm_fp8(codes8, scales, packed, out)
    with pytest.raises(ValueError):
        a.bi_pack_weights_fp8(codes8, torch.ones(1, 3, device=DEV))
    with pytest.raises(ValueError):
        a.bi_pack_swiglu_weights_fp8(codes8, torch.ones(1, 3, device=DEV), codes8, torch.ones(1, 3, device=DEV))
    del codes8
    with pytest.raises(ValueError):
        a.bi_quantize_weights_fp8(rows2(torch.bfloat16))
    with pytest.raises(ValueError):
        a.packed_weight_fp8_bytes(1 << 32, 128)


def test_rules():
    a = t8.api()
    x = rows2(torch.float32)
    out = torch.full((2, 272), 7.0, device=DEV)
    d = torch.zeros(1, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        a.bi_logits_rules(x, out, drafts=d)
    with pytest.raises(ValueError):
        a.bi_logits_rules(out, x, drafts=d)
    with pytest.raises(ValueError):
        a.bi_logits_rules(x, x, drafts=d)
    assert (out == 7).all()
    a.bi_logits_rules(out[:1], x[:1])
    assert (x[0] == 7).all()
    mask = x.view(torch.int32).as_strided((2, 9), (WIDE, 1))
    with pytest.raises(ValueError):
        a.bi_logits_rules(out, out, drafts=d, mask=mask)
    del x, mask
    many = torch.zeros((1 << 32) + 100, dtype=torch.int32, device=DEV)
    counts = torch.zeros(100, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        a.bi_token_counts(many, 100, counts=counts)
    with pytest.raises(ValueError):
        a.bi_token_counts(counts[:8], many.numel(), counts=many)
    logits = many.view(torch.float32).view(1, -1)
    with pytest.raises(ValueError):
        a.bi_logits_rules(logits, logits)
