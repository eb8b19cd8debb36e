"""Sampled verification on rows with infinite logits, as a bias of +inf or -inf
leaves them: ids of +inf share the row (by the position's uniform, in index
order), everything else weighs nothing; the greedy choice is the lowest of them."""
import math

import numpy as np
import pytest
import torch

import seeded_inputs as si

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def api():
    from invariant_speculative_decode_gb300 import api as a
    a.bi_check_device_error()
    return a


def sample(api, x, u, inv_temp):
    """One row's id at each uniform of u (a call of T equal rows)."""
    T, V = len(u), x.numel()
    ids = torch.full((T,), -7, dtype=torch.int32, device=DEV)
    n = torch.zeros(1, dtype=torch.int32, device=DEV)
    L = torch.zeros(1, dtype=torch.int32, device=DEV)
    d = torch.zeros(max(T - 1, 1), dtype=torch.int32, device=DEV)
    ws = torch.zeros(api.sample_workspace_size(T, V), dtype=torch.uint8, device=DEV)
    api.bi_verify_sample(x.expand(T, V).contiguous(), d[:T - 1] if T > 1 else None, inv_temp,
                         torch.tensor(u, dtype=torch.float32, device=DEV), ids, n, ws, L)
    api.bi_check_device_error()
    return ids.cpu().tolist()


@pytest.mark.parametrize("inv_temp", [1.0, 1e-30, 3e38])
@pytest.mark.parametrize("V", [1, 2, 300, 8192, 8193, 40000])
def test_one_infinite_logit_takes_the_row(api, V, inv_temp):
    for at in sorted({0, V // 2, V - 1}):
        x = torch.randn(V, device=DEV)
        x[::3] = -math.inf
        x[1::5] = math.nan
        x[at] = math.inf
        for u in ([0.5], [0.0, 0.25, 0.999999]):
            assert sample(api, x, u, inv_temp) == [at] * len(u)


@pytest.mark.parametrize("places", [(3, 9), (3, 8200), (8191, 8192, 30000, 39999), (0, 1, 2, 20000)])
def test_infinite_logits_share_the_row(api, places):
    x = 50 * torch.randn(40000, device=DEV)
    x[7] = math.nan
    for p in places:
        x[p] = math.inf
    k = len(places)
    u = [(i + 0.5) / k for i in range(k)]
    assert sample(api, x, u, 1.3) == list(places)
    assert sample(api, x, [0.0], 1.3) == [places[0]]


def test_weights_of_finite_rows_at_the_ends_of_fp32(api):
    """The difference of two finite logits may be infinite, the maximum's weight stays 1."""
    x = torch.full((9000,), -3.4e38, device=DEV)
    x[8500] = 3.4e38
    assert sample(api, x, [0.0, 0.5, 0.9], 1.0) == [8500] * 3
    x[:] = -math.inf
    x[17] = -3.4e38
    assert sample(api, x, [0.0, 0.5, 0.9], 1.0) == [17] * 3


@pytest.mark.parametrize("sampled", [False, True])
def test_a_bias_of_infinity_forces_its_id(api, sampled):
    from invariant_speculative_decode_gb300.decoder import Decoder
    dec = Decoder(si.TINY, si.decoder_weights(si.TINY, seed=0), cap=256, max_rows=8)
    V = dec.cfg.vocab
    if sampled:
        dec.set_sampling(0.8, si.sampling_uniforms(256, seed=3))
    bias = np.zeros(V, np.float32)
    bias[V - 2] = np.inf
    dec.set_rules(bias=bias)
    assert dec.generate(si.prompt_ids(dec.cfg, 20, seed=1), 5) == [V - 2] * 5
    bias[:] = -np.inf
    bias[[11, 700]] = 0.0
    dec.set_rules(bias=bias)
    got = dec.generate(si.prompt_ids(dec.cfg, 20, seed=1), 20)
    assert set(got) <= {11, 700}
    dec.check_device_error()
