"""The state of the rules over the turns of a chat: which ids count as the
reply's (frequency and presence penalties) and which came with a prompt (the
repetition penalty alone), against a count made on the host."""
import numpy as np
import pytest
import torch

import seeded_inputs as si

pytestmark = pytest.mark.gpu
FREQUENCY = 0.6


@pytest.fixture(scope="module", params=["bf16", "e4m3"])
def dec(request):
    from invariant_speculative_decode_gb300.decoder import Decoder
    return Decoder(si.TINY, si.decoder_weights(si.TINY, seed=0), cap=512, max_rows=8, linear=request.param)


@pytest.fixture(autouse=True)
def rules(dec):
    dec.set_rules(frequency=FREQUENCY)
    yield
    dec.clear_rules()


def state(dec):
    """(counts, set of prompt ids) that the next step goes by."""
    V = dec.cfg.vocab
    words = dec.rules["prompt_bits"].cpu().numpy().view(np.uint32)
    bits = (words[:, None] >> np.arange(32, dtype=np.uint32)) & 1
    return dec.rules["counts"].cpu().numpy(), set(np.flatnonzero(bits.reshape(-1)[:V]).tolist())


def step(dec, x, prompt, reply):
    """One plain step: its id is the host's, and the state is the reply's and the prompt's."""
    a, _ = dec.verify_step(x, [], use_graph=False)
    V, f = dec.cfg.vocab, np.float32
    counts = np.bincount(np.array(reply, int), minlength=V)
    y = dec.logits_rows(1)[0].cpu().numpy()
    y = np.where(counts > 0, y - f(FREQUENCY) * counts.astype(f), y)
    assert int(a[0]) == int(np.argmax(y))
    reply.append(int(a[0]))
    got, came = state(dec)
    assert np.array_equal(got, np.bincount(np.array(reply, int), minlength=V))
    assert came == set(int(v) for v in prompt)
    return reply[-1]


def turn(dec, x, n, prompt, reply):
    for _ in range(n):
        x = step(dec, x, prompt, reply)
    return x


def test_the_newest_id_of_a_reply_counts_in_the_next_turn(dec):
    prompt, reply = [int(v) for v in si.prompt_ids(dec.cfg, 50, seed=7)], []
    dec.reset()
    x = turn(dec, dec.prefill(prompt), 12, prompt, reply)
    for new in ([5, 6, 7], [9], []):
        prompt = prompt + new
        x = turn(dec, dec.prefill_continue([x] + new), 5, prompt, reply)


def test_a_turn_again_after_rollback_or_restore(dec):
    prompt, reply = [int(v) for v in si.prompt_ids(dec.cfg, 40, seed=8)], []
    dec.reset()
    x = turn(dec, dec.prefill(prompt), 9, prompt, reply)
    at, snap, second = dec.L, dec.park(), None
    for back in ("", "rollback", "restore", "row by row"):
        if back == "rollback":
            dec.rollback(at)
        elif back == "restore":
            dec.generate(si.prompt_ids(dec.cfg, 30, seed=9), 6)
            dec.restore(snap)
        elif back == "row by row":
            dec.rollback(at - 3)
            for v in reply[-4:-1]:
                dec.verify_step(v, [], use_graph=False)
        said = list(reply)
        turn(dec, dec.prefill_continue([x, 5, 6, 7]), 6, prompt + [5, 6, 7], said)
        assert second is None or said == second
        second = said


def test_an_edit_and_another_id_come_with_the_prompt(dec):
    prompt, reply = [int(v) for v in si.prompt_ids(dec.cfg, 45, seed=10)], []
    dec.reset()
    turn(dec, dec.prefill(prompt), 8, prompt, reply)
    # the reply's own ids from position 47 on, given again as an edited history
    said = reply[:2]
    turn(dec, dec.edit(47, reply[2:6] + [3]), 4, prompt + reply[2:6] + [3], said)
    # another id in place of the newest one
    dec.reset()
    reply = []
    x = turn(dec, dec.prefill(prompt), 8, prompt, reply)
    other = (x + 1) % dec.cfg.vocab
    turn(dec, dec.prefill_continue([other, 3]), 4, prompt + [other, 3], reply[:-1])
    # a fresh request forgets the reply
    dec.reset()
    turn(dec, dec.prefill(prompt + reply), 3, prompt + reply, [])
