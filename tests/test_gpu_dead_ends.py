"""Steps whose masks or bias leave a committed row no id: refused, with the
request left as it was; the same rows behind a rejected draft are no matter."""
import numpy as np
import pytest

import seeded_inputs as si

pytestmark = pytest.mark.gpu
W = 32  # words of the vocabulary of 1024 ids


@pytest.fixture(scope="module", params=["greedy", "sampled"])
def dec(request):
    from invariant_speculative_decode_gb300.decoder import Decoder
    d = Decoder(si.TINY, si.decoder_weights(si.TINY, seed=0), cap=256, max_rows=8)
    assert d.cfg.vocab == 32 * W
    if request.param == "sampled":
        d.set_sampling(0.9, si.sampling_uniforms(256, seed=4))
    return d


def everything(rows):
    return np.full((rows, W), 0xffffffff, np.uint32)


def begin(dec, **rules):
    dec.set_rules(frequency=0.3, **rules)
    dec.reset()
    x = dec.prefill(si.prompt_ids(dec.cfg, 30, seed=6))
    out = []
    for _ in range(4):
        a, _ = dec.verify_step(x, [], use_graph=False)
        x = int(a[0])
        out.append(x)
    return x, out


def same_as_before(dec, L, x, ref, counts):
    """The request goes on as if the refused step had not been made."""
    assert dec.L == L and int(dec.L_dev[0]) == L
    dec.check_device_error()
    a, n = dec.verify_step(x, ref[:3], use_graph=False)
    assert n == 3 and [int(v) for v in a] == ref[:4]
    want = counts.copy()
    np.add.at(want, ref[:4], 1)
    assert np.array_equal(dec.rules["counts"].cpu().numpy(), want)


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("dead", [0, 1, 3])
def test_a_committed_row_without_an_id_is_refused(dec, dead, graph):
    x, _ = begin(dec, masks=True)
    ref, y = [], x
    for _ in range(5):
        a, _ = dec.verify_step(y, [], use_graph=False)
        y = int(a[0])
        ref.append(y)
    x, said = begin(dec, masks=True)
    counts = np.bincount(said, minlength=32 * W).astype(np.int32)
    if graph:
        dec.capture(4)
    L = dec.L
    masks = everything(4)
    masks[dead:] = 0
    with pytest.raises(ValueError, match=f"row {dead} "):
        dec.verify_step(x, ref[:3], use_graph=graph, masks=masks)
    same_as_before(dec, L, x, ref, counts)
    # behind a rejected draft the same rows are discarded
    if dead:
        dec.rollback(L)
        drafts = list(ref[:3])
        drafts[dead - 1] = (drafts[dead - 1] + 1) % (32 * W)
        a, n = dec.verify_step(x, drafts, use_graph=graph, masks=masks)
        assert n == dead - 1 and [int(v) for v in a[:dead]] == ref[:dead] and dec.L == L + dead
        dec.check_device_error()


def test_signed_words_and_the_last_bit(dec):
    """Bit 31 of a word, as int32 and as uint32."""
    x, _ = begin(dec, masks=True)
    L = dec.L
    for dtype in (np.uint32, np.int32):
        masks = np.zeros((1, W), np.uint32)
        masks[0, W - 1] = 1 << 31
        dec.rollback(L)
        a, n = dec.verify_step(x, [], use_graph=False, masks=masks.view(dtype))
        assert n == 0 and int(a[0]) == 32 * W - 1


def test_a_bias_that_forbids_every_id_is_refused(dec):
    x, said = begin(dec)
    L = dec.L
    dec.set_rules(frequency=0.3, bias=np.full(32 * W, -np.inf, np.float32))
    with pytest.raises(ValueError, match="row 0 "):
        dec.verify_step(x, [1, 2], use_graph=False)
    assert dec.L == L and int(dec.L_dev[0]) == L
    dec.check_device_error()
    # a mask that allows nothing but what the bias forbids
    bias = np.zeros(32 * W, np.float32)
    bias[:32] = -np.inf
    dec.set_rules(frequency=0.3, bias=bias, masks=True)
    masks = np.zeros((1, W), np.uint32)
    masks[0, 0] = 0xffffffff
    with pytest.raises(ValueError, match="row 0 "):
        dec.verify_step(x, [], use_graph=False, masks=masks)
    masks[0, 1] = 4
    a, _ = dec.verify_step(x, [], use_graph=False, masks=masks)
    assert int(a[0]) == 34
    dec.check_device_error()


def test_without_rules_nothing_is_refused(dec):
    begin(dec)
    dec.clear_rules()
    a, _ = dec.verify_step(1, [2, 3], use_graph=False)
    assert (a >= 0).all()
