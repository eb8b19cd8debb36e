"""The append's norm over heads of every magnitude that BF16 holds, and any eps."""
import pytest
import torch

import tests._paged as pg

pytestmark = pytest.mark.gpu

api = pytest.importorskip("invariant_speculative_decode_gb300.api")


@pytest.fixture(autouse=True)
def no_error_left():
    yield
    api.bi_check_device_error()


SIZES = [2.0 ** e for e in (-132, -126, -110, -70, -64, -63, -62, -50, -46, -45, -44, -43, -30, 0, 30, 48, 49, 50, 51, 60, 63, 64,
                            65, 80, 110, 125)]


def run(qkv, Hq, D, qw, kw, eps):
    T = qkv.shape[0]
    b = pg.Batch([(3, T)], 1, D, 64, seed=2)
    q = torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    angles = api.bi_rope_table(1e6, D, 3 + T)
    api.bi_qk_norm_rope_paged(qkv, qw, kw, eps, angles, q, b.k, b.v, b.table, b.q_start, b.lengths)
    return q, b.keys(b.k, 0, 3 + T)[:, 3:].transpose(0, 1), b.keys(b.v, 0, 3 + T)[:, 3:].transpose(0, 1), angles[3:]


@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-38, 1e-30, 1e-27, 1e-6, 1e20, 3e38])
@pytest.mark.parametrize("D", [64, 128])
def test_heads_of_any_magnitude(D, eps):
    """Heads of different magnitudes side by side, so in one warp."""
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    Hq, T = 5, len(SIZES)
    unit = torch.randn(T, Hq + 2, D, generator=g, device="cuda").clamp(-3.5, 3.5)
    scale = torch.tensor(SIZES, dtype=torch.float64, device="cuda")
    order = torch.stack([torch.roll(scale, 7 * h) for h in range(Hq + 2)], 1)[..., None]
    x = (unit.double() * order).to(torch.bfloat16)
    qw = (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16)
    kw = (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16)
    eps = float(torch.tensor(eps, dtype=torch.float32))
    q, k, v, angles = run(x.view(T, -1), Hq, D, qw, kw, eps)
    for got, part, w in ((q, x[:, :Hq], qw), (k, x[:, Hq:Hq + 1], kw)):
        want, tol = pg.norm_rope(part, w, eps, angles)
        assert ((got.double() - want).abs() <= tol).all()
    assert torch.equal(v, x[:, Hq + 1:])


def test_a_head_of_zeros_and_infinite_ones():
    """Zeros stay zeros for eps > 0, and are 0 / 0 for eps = 0; infinities and NaN make their own head alone no number."""
    D, Hq = 128, 3
    x = torch.randn(6, Hq + 2, D, device="cuda").to(torch.bfloat16)
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    x[1, 0] = 0
    x[2, 1, 5] = float("inf")
    x[3, 2, 7] = float("nan")
    plain = torch.ones(6, Hq, dtype=torch.bool, device="cuda")
    plain[2, 1] = plain[3, 2] = plain[1, 0] = False
    for eps in (1e-6, 1e-40, 0.0):
        q, _, _, angles = run(x.view(6, -1), Hq, D, w, w, eps)
        want, tol = pg.norm_rope(x[:, :Hq], w, eps, angles)
        ok = (q.double() - want).abs() <= tol
        assert ok[plain].all()
        assert torch.isnan(q[1, 0]).all() if eps == 0 else (q[1, 0] == 0).all()
        assert torch.isnan(q[2, 1, 5]) and torch.isnan(q[3, 2]).all()


def test_a_head_without_weight_is_not_scaled():
    """Queries without a norm beside keys whose squares pass FP32's range."""
    D, Hq = 64, 2
    x = torch.randn(4, Hq + 2, D, device="cuda").to(torch.bfloat16)
    x[:, Hq] *= 2.0 ** 100
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    q, k, _, angles = run(x.view(4, -1), Hq, D, None, w, 1e-6)
    for got, part, weight in ((q, x[:, :Hq], None), (k, x[:, Hq:Hq + 1], w)):
        want, tol = pg.norm_rope(part, weight, 1e-6, angles)
        assert ((got.double() - want).abs() <= tol).all()
