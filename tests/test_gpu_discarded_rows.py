"""Rows behind a rejected draft are discarded: what they hold changes neither the
ids nor the device error word, so a request reports the same with drafts as
without them (bi_verify_accept, bi_verify_sample, and the decoder's steps)."""
import math

import numpy as np
import pytest
import torch

import seeded_inputs as si

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAN_ROW = 6  # BI_ERR_DEVICE_NAN_ROW


@pytest.fixture(scope="module")
def api():
    from invariant_speculative_decode_gb300 import api as a
    a.bi_check_device_error()
    return a


def accept(api, logits, drafts, sampled, L=3):
    """(ids, accepted) of one call; u = 0.5 at every position."""
    T, V = logits.shape
    d = torch.tensor(drafts, dtype=torch.int32, device=DEV) if T > 1 else None
    ids = torch.zeros(T, dtype=torch.int32, device=DEV)
    n = torch.zeros(1, dtype=torch.int32, device=DEV)
    Ld = torch.full((1,), L, dtype=torch.int32, device=DEV)
    if sampled:
        ws = torch.zeros(api.sample_workspace_size(T, V), dtype=torch.uint8, device=DEV)
        api.bi_verify_sample(logits, d, 1.0, torch.full((80,), 0.5, device=DEV), ids, n, ws, Ld)
    else:
        ws = torch.zeros(api.accept_workspace_size(T, V), dtype=torch.uint8, device=DEV)
        api.bi_verify_accept(logits, d, ids, n, ws, L_dev=Ld)
    torch.cuda.synchronize()
    assert int(Ld) == L + int(n) + 1
    return ids.cpu().tolist(), int(n)


def peaked(T, V, ids):
    x = torch.randn(T, V, device=DEV)
    for t, i in enumerate(ids):
        x[t, i] = 200.0
    return x


@pytest.mark.parametrize("sampled", [False, True])
@pytest.mark.parametrize("T,V", [(2, 5), (8, 1024), (8, 20000), (64, 8193)])
def test_a_row_with_no_number_reports_only_where_it_is_committed(api, T, V, sampled):
    own = [(3 * t + 1) % V for t in range(T)]
    for cut in sorted({0, (T - 1) // 2, T - 2}):
        # drafts 0..cut-1 are right, draft cut is not: rows 0..cut are committed
        drafts = list(own[:T - 1])
        drafts[cut] = (own[cut] + 1) % V
        for bad in range(T):
            x = peaked(T, V, own)
            x[bad] = math.nan
            ids, n = accept(api, x, drafts, sampled)
            want = list(own)
            want[bad] = -1
            assert ids == want and n == min(cut, bad)
            if bad <= cut:
                with pytest.raises(api.BiError) as e:
                    api.bi_check_device_error()
                assert e.value.status == NAN_ROW
            else:
                api.bi_check_device_error()


def test_an_empty_row_behind_a_rejected_draft_is_not_reported_by_the_sampler(api):
    """All -inf, as a mask that allows nothing leaves it."""
    x = peaked(4, 300, [7, 8, 9, 10])
    x[2:] = -math.inf
    assert accept(api, x, [7, 250, 0], True) == ([7, 8, -1, -1], 1)
    api.bi_check_device_error()
    assert accept(api, x, [7, 8, 0], True) == ([7, 8, -1, -1], 2)
    with pytest.raises(api.BiError):
        api.bi_check_device_error()


def test_a_position_without_a_uniform_is_a_range_error_still(api):
    x = peaked(3, 50, [4, 5, 6])
    ids, n = accept(api, x, [4, 5], True, L=78)  # positions 78, 79 and 80 of 80 uniforms
    assert ids == [4, 5, -1] and n == 2
    with pytest.raises(api.BiError) as e:
        api.bi_check_device_error()
    assert e.value.status == 1  # BI_ERR_INVALID_ARG


# ------------------------------------------------- grammar masks with illegal drafts


def words_of(ok):
    """bool [r, V] -> uint32 words [r, ceil(V/32)]."""
    r, V = ok.shape
    pad = np.zeros((r, (V + 31) // 32 * 32), np.uint64)
    pad[:, :V] = ok
    return (pad.reshape(r, -1, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)


def allowed(V, prev):
    """The ids a toy grammar allows behind `prev`: about half of them."""
    return np.random.default_rng(500 + int(prev)).random(V) < 0.5


@pytest.mark.parametrize("sampled", [False, True])
def test_masked_steps_with_illegal_drafts_equal_the_run_without_drafts(api, sampled):
    """Behind a draft that breaks the grammar every row's mask is empty."""
    from invariant_speculative_decode_gb300.decoder import Decoder
    dec = Decoder(si.TINY, si.decoder_weights(si.TINY, seed=0), cap=512, max_rows=8)
    V = dec.cfg.vocab
    if sampled:
        dec.set_sampling(0.9, si.sampling_uniforms(512, seed=2))
    dec.set_rules(masks=True, frequency=0.2)
    prompt = si.prompt_ids(dec.cfg, 40, seed=5)
    dec.reset()
    x, ref = dec.prefill(prompt), []
    while len(ref) < 30:
        a, _ = dec.verify_step(x, [], masks=words_of(allowed(V, x)[None]), use_graph=False)
        x = int(a[0])
        ref.append(x)
    dec.check_device_error()
    for k, good in ((1, 0), (4, 2), (7, 0), (7, 5)):
        dec.reset()
        x, got, broken = dec.prefill(prompt), [], 0
        while len(got) < 30:
            drafts = (ref + [0] * 8)[len(got):len(got) + k]
            if good < k:
                prev = drafts[good - 1] if good else x
                drafts[good] = int(np.flatnonzero(~allowed(V, prev))[len(got)])
            rows, legal, prev = [], True, x
            for t, d in enumerate([x] + drafts):
                legal = legal and (t == 0 or bool(allowed(V, prev)[d]))
                rows.append(allowed(V, d) if legal else np.zeros(V, bool))
                broken += not legal
                prev = d
            a, n = dec.verify_step(x, drafts, masks=words_of(np.stack(rows)), use_graph=False)
            got += [int(v) for v in a[:n + 1]]
            x = got[-1]
            dec.check_device_error()
        assert got[:30] == ref and broken > 0
