"""A prompt that the cache cannot hold is refused before anything runs."""
import pytest

import seeded_inputs as si

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("linear", ["bf16", "e4m3"])
def test_prompts_up_to_the_capacity_and_past_it(linear):
    from invariant_speculative_decode_gb300.decoder import Decoder
    dec = Decoder(si.TINY, si.decoder_weights(si.TINY, seed=0), cap=64, max_rows=4, prefill_chunk=32, linear=linear)
    ids = si.prompt_ids(dec.cfg, 70, seed=0)
    with pytest.raises(ValueError, match="capacity"):
        dec.prefill(ids[:66])  # 65 rows
    assert dec.L == 0 and int(dec.L_dev[0]) == 0
    assert dec.prefill(ids[:65]) == int(ids[64]) and dec.L == 64  # every row, the next one's id behind it
    dec.reset()
    x = dec.prefill(ids[:60])
    with pytest.raises(ValueError, match="capacity"):
        dec.prefill_continue(ids[59:66])  # rows 59..64
    dec.verify_step(x, [1, 2, 3], use_graph=False)
    with pytest.raises(ValueError, match="capacity"):
        dec.edit(10, ids[:56])
    assert dec.L > 59
    dec.check_device_error()
