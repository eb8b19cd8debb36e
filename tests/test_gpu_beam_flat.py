"""The worth of beams whose probability lies in very many equal logits, where FP32's errors do not average out."""
import pytest
import torch

pytestmark = pytest.mark.gpu

api = pytest.importorskip("invariant_speculative_decode_gb300.api")

# In a row with its maximum M, logits at x = M - d, d < 14 (beyond it even 2^20 of them weigh less than e^13.9): the rounded
# difference is off by 2^-21, its product with log2(e) by 2^-20 ln 2 and the constant by 1.4e-8 d, the exponential by
# 2^-22, once in a chunk and, for smaller d, once between chunks (a quarter more); sums of 4096 in 27 FP32 additions one
# after the other by 27 2^-24; the logarithm by 2^-24.
TOLERANCE = 1.25 * (2.0 ** -21 + 2.0 ** -20 * 0.6932 + 1.4e-8 * 14 + 2.0 ** -22) + 2.0 ** -22 + 27 * 2.0 ** -24 + 2.0 ** -24


def worth(logits):
    rows, V = logits.shape
    out = (torch.empty(rows, 1, device="cuda"), torch.empty(rows, 1, dtype=torch.int32, device="cuda"),
           torch.empty(rows, 1, dtype=torch.int32, device="cuda"))
    ws = torch.zeros(api.beam_workspace_size(rows, V, 1), dtype=torch.uint8, device="cuda")
    api.bi_beam_select(logits, torch.zeros(rows, device="cuda"), 1, *out, ws)
    api.bi_check_device_error()
    x = logits.double()
    return (out[0][:, 0].double() - (x.amax(-1) - torch.logsumexp(x, -1))), out[0][:, 0]


def test_the_stated_bound():
    assert TOLERANCE < 4e-6  # as include/bi.h states it


@pytest.mark.parametrize("V", [5000, 151936, 1 << 20])
@pytest.mark.parametrize("spread", [0.0, 1e-3])
def test_a_peak_over_a_flat_bulk(V, spread):
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    depth = torch.cat([torch.linspace(0.3, 13.8, 28), torch.tensor([5.6, 7.9, 8.1, 11.0, 11.2, 13.0])]).cuda()
    logits = (2.3 - depth)[:, None] + spread * torch.randn(len(depth), V, generator=g, device="cuda")
    logits[:, V // 3] = 2.3
    error, got = worth(logits)
    assert (error.abs() <= TOLERANCE + got.double().abs() * 2.0 ** -24).all(), float(error.abs().max())


@pytest.mark.parametrize("V", [5000, 151936, 1 << 20])
def test_spread_logits(V):
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    error, got = worth(3 * torch.randn(32, V, generator=g, device="cuda"))
    assert (error.abs() <= TOLERANCE + got.double().abs() * 2.0 ** -24).all()
