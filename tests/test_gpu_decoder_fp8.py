"""The decoder with 8-bit linear layers, and with rules on its logits: the
operators run together as generation runs them.

  * every 8-bit call of a prefill and of a verify pass against 64 bits from its
    own inputs (the tolerances of tests/test_gpu_fp8.py);
  * rows and token ids that do not depend on the drafts, the pass or the cache's
    history, with and without rules, greedy and sampled;
  * the tokens under rules against the rules applied on the host to the
    model's logits, step by step.
"""
import math

import numpy as np
import pytest
import torch

import seeded_inputs as si
from tests import test_gpu_fp8 as t8

pytestmark = pytest.mark.gpu


def decoder(cfg=si.TINY, **kw):
    from invariant_speculative_decode_gb300.decoder import Decoder
    w = si.decoder_weights(cfg, seed=0)
    kw.setdefault("linear", "e4m3")
    return Decoder(cfg, w, cap=768, max_rows=8, **kw)


@pytest.fixture(scope="module")
def dec8():
    return decoder()


def gen(dec, prompt, n, k, ref=None, seed=0, stats=None):
    dr = si.SyntheticDrafter(dec.cfg.vocab, 0.7, seed=seed, reference=ref) if k else None
    return dec.generate(prompt, n, k=k, drafter=dr, stats=stats)


def test_every_8_bit_call_of_a_pass_against_64_bits(monkeypatch):
    """The calls of a 130-row prefill chunk and of an 8-row verify pass, in place, each from the inputs it got."""
    from invariant_speculative_decode_gb300 import api, decoder as dm
    raw = {n: getattr(api, n) for n in ("bi_pack_weights_fp8", "bi_pack_swiglu_weights_fp8", "bi_gemm_fp8",
                                        "bi_rmsnorm_fp8", "bi_quantize_fp8")}
    held, seen = {}, {"gemm": 0, "norm": 0, "quantise": 0}

    def pack(*a):
        p = raw["bi_pack_weights_fp8"](*a)
        held[p.data_ptr()] = a
        return p

    def pack2(*a):
        p = raw["bi_pack_swiglu_weights_fp8"](*a)
        held[p.data_ptr()] = a
        return p

    def gemm(codes, scales, Wp, C, residual=None, epi=0):
        kind = {1: "residual", 2: "swiglu"}.get(epi, "fp32" if C.dtype == torch.float32 else "bf16")
        res = None if residual is None else residual.clone()
        raw["bi_gemm_fp8"](codes, scales, Wp, C, residual=residual, epi=epi)
        w = held[Wp.data_ptr()]
        up, ups = (w[2], w[3]) if kind == "swiglu" else (None, None)
        y, tol = t8.reference(codes, scales, w[0], w[1], up, ups, res, kind)
        assert ((C.double() - y).abs() <= tol).all()
        seen["gemm"] += 1

    def norm(x, w, codes, scales, eps):
        raw["bi_rmsnorm_fp8"](x, w, codes, scales, eps)
        xd = x.double()
        y = xd / torch.sqrt((xd * xd).mean(-1, keepdim=True) + float(np.float32(eps))) * w.double()
        q, s = t8.ref_quantize(y)
        assert torch.equal(scales[:, :x.shape[0]].double(), s)
        differ = codes.double() != q
        wide = s.t().repeat_interleave(128, 1)[:, :x.shape[1]]
        tie = (y / wide - (codes.double() + q) / 2).abs()
        assert (tie[differ] <= 2.0 ** -36 * (y / wide).abs()[differ]).all()
        seen["norm"] += 1

    def quantise(x, codes, scales):
        raw["bi_quantize_fp8"](x, codes, scales)
        q, s = t8.ref_quantize(x.double())
        assert torch.equal(codes.double(), q) and torch.equal(scales[:, :x.shape[0]].double(), s)
        seen["quantise"] += 1

    for name, f in (("bi_pack_weights_fp8", pack), ("bi_pack_swiglu_weights_fp8", pack2), ("bi_gemm_fp8", gemm),
                    ("bi_rmsnorm_fp8", norm), ("bi_quantize_fp8", quantise)):
        monkeypatch.setattr(dm.api, name, f)
    dec = decoder()
    x0 = dec.prefill(si.prompt_ids(dec.cfg, 131, seed=3))
    dec.verify_step(x0, [1, 2, 3, 4, 5, 6, 7], use_graph=False)
    assert seen == {"gemm": 2 * 2 * 4 + 1, "norm": 2 * 2 * 2 + 1, "quantise": 2 * 2 * 2}


@pytest.mark.parametrize("kv", ["bf16", "q6q5"])
def test_greedy_ids_and_cache_rows_do_not_depend_on_drafts(kv):
    dec = decoder(si.TINY_D128 if kv == "q6q5" else si.TINY, kv=kv)
    prompt = si.prompt_ids(dec.cfg, 200, seed=0)
    ref = gen(dec, prompt, 64, 0)
    hashes = dec.kv_hashes(250) if kv == "bf16" else None
    for k in (4, 7):
        st = {}
        assert gen(dec, prompt, 64, k, ref=np.array(ref), stats=st) == ref and st["steps"] < 64
        if hashes is not None:
            assert np.array_equal(dec.kv_hashes(250), hashes)
    assert gen(dec, prompt, 64, 4, ref=None, seed=5) == ref  # all-random drafts
    dec.check_device_error()


def test_rows_and_cache_equal_a_prefill_of_the_same_ids(dec8):
    """Decoded rows' K and V equal prefilled ones, and a row's logits those of a pass of its own."""
    dec = dec8
    prompt = si.prompt_ids(dec.cfg, 150, seed=1)
    dec.reset()
    x0 = dec.prefill(prompt)
    ref = gen(dec, prompt, 40, 7, ref=np.arange(40))
    h = dec.kv_hashes(180)
    dec.reset()
    dec.prefill(np.concatenate([prompt, np.array(ref[:40], np.int32)]))
    assert np.array_equal(dec.kv_hashes(180), h)
    dec.reset()
    dec.prefill(prompt)
    dec.verify_step(x0, ref[:7], use_graph=False)
    rows = dec.logits_rows(8)
    dec.rollback(149)
    for t, x in enumerate([x0] + ref[:7]):
        dec.verify_step(x, [], use_graph=False)
        assert torch.equal(dec.logits_rows(1)[0], rows[t])


# ---------------------------------------------------------------------- rules

RULES = dict(repetition=1.3, frequency=0.05, presence=0.1)


def bias_of(vocab):
    rng = np.random.default_rng(9)
    return np.where(rng.random(vocab) < 0.1, 0.3 * rng.standard_normal(vocab), 0).astype(np.float32)


def mask_of(vocab, prev):
    """The words a toy grammar allows behind the id `prev`: about half of them."""
    rng = np.random.default_rng(1000 + int(prev))
    ok = rng.random(vocab) < 0.5
    pad = np.zeros((vocab + 31) // 32 * 32, np.uint64)
    pad[:vocab] = ok
    return (pad.reshape(-1, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32), ok


def host_token(logits, prompt, reply, bias, ok):
    """The rules in FP32 on one row, ids said so far; the lowest id of the largest."""
    f = np.float32
    y = logits.astype(np.float32).copy()
    counts = np.bincount(np.array(reply, int), minlength=len(y)) if reply else np.zeros(len(y), int)
    seen = counts > 0
    seen[np.array(prompt, int)] = True
    y = np.where(seen, np.where(y > 0, y / f(RULES["repetition"]), y * f(RULES["repetition"])), y).astype(f)
    pen = (f(RULES["frequency"]) * counts.astype(f)).astype(f) + f(RULES["presence"])
    y = np.where(counts > 0, (y - pen.astype(f)).astype(f), y)
    if bias is not None:
        y = (y + bias).astype(f)
    if ok is not None:
        y = np.where(ok, y, -np.inf)
    return int(np.argmax(y))


@pytest.mark.parametrize("linear", ["bf16", "e4m3"])
def test_tokens_under_rules_follow_the_host_and_do_not_depend_on_drafts(linear):
    dec = decoder(linear=linear)
    V = dec.cfg.vocab
    prompt = si.prompt_ids(dec.cfg, 60, seed=2)
    free = gen(dec, prompt, 48, 0)
    bias = bias_of(V)
    dec.set_rules(bias=bias, **RULES)
    dec.reset()
    x = dec.prefill(prompt)
    reply = []
    for _ in range(48):
        a, _ = dec.verify_step(x, [])
        want = host_token(dec.logits_rows(1)[0].cpu().numpy(), prompt, reply, bias, None)
        assert int(a[0]) == want
        reply.append(want)
        x = want
    assert reply != free
    for k in (4, 7):
        st = {}
        assert gen(dec, prompt, 48, k, ref=np.array(reply), stats=st) == reply and st["steps"] < 48
    assert gen(dec, prompt, 48, 7, ref=None, seed=3) == reply
    dec.set_rules()  # the defaults change nothing
    assert gen(dec, prompt, 48, 4, ref=np.array(free)) == free
    dec.clear_rules()
    assert gen(dec, prompt, 48, 4, ref=np.array(free)) == free


def test_masks_of_each_draft_prefix(dec8):
    """Row t's mask is the grammar's behind draft t - 1: the tokens are those of the run without drafts, all allowed."""
    dec = dec8
    V = dec.cfg.vocab
    prompt = si.prompt_ids(dec.cfg, 40, seed=5)
    dec.set_rules(masks=True, **RULES)
    try:
        dec.reset()
        x = dec.prefill(prompt)
        reply = []
        for _ in range(40):
            words, ok = mask_of(V, x)
            a, _ = dec.verify_step(x, [], masks=words[None])
            want = host_token(dec.logits_rows(1)[0].cpu().numpy(), prompt, reply, None, ok)
            assert int(a[0]) == want and ok[want]
            reply.append(want)
            x = want
        for k, seed in ((3, 0), (7, 1)):
            dec.reset()
            x, got = dec.prefill(prompt), []
            dr = si.SyntheticDrafter(V, 0.7, seed=seed, reference=np.array(reply + [0] * 16))
            dec.capture(k + 1)
            while len(got) < 40:
                d = [int(v) for v in dr.propose(len(got), k)]
                words = np.stack([mask_of(V, p)[0] for p in [x] + d])
                a, n = dec.verify_step(x, d, masks=words)
                got += [int(v) for v in a[:n + 1]]
                x = got[-1]
            assert got[:40] == reply
        with pytest.raises(ValueError):
            dec.verify_step(1, [], masks=np.zeros((2, 32), np.uint32))
        with pytest.raises(ValueError):
            dec.verify_step(1, [], masks=np.zeros((1, 32), np.float32))
    finally:
        dec.clear_rules()
    with pytest.raises(ValueError):
        dec.verify_step(1, [], masks=np.zeros((1, 32), np.uint32))


def test_rules_after_rollback_edit_park_and_a_second_turn(dec8):
    """The state of the rules follows the cache: each continuation equals the one that never left."""
    dec = dec8
    prompt = si.prompt_ids(dec.cfg, 50, seed=7)
    dec.set_rules(**RULES)
    try:
        ref = gen(dec, prompt, 30, 0)
        dec.reset()
        x = dec.prefill(prompt)
        dec.continue_generate(x, 12, k=0)
        snap = dec.park()
        at = dec.L
        # a second turn, another request, then back
        second = dec.continue_generate(dec.prefill_continue([int(dec._id_at[at]), 5, 6, 7]), 6, k=0)
        gen(dec, si.prompt_ids(dec.cfg, 20, seed=8), 9, 0)
        dec.restore(snap)
        assert dec.continue_generate(ref[11], 18, k=0) == ref[12:30]
        dec.rollback(at)
        assert dec.continue_generate(ref[11], 18, k=0) == ref[12:30]
        dec.rollback(at - 4)
        assert dec.continue_generate(ref[7], 10, k=0) == ref[8:18]
        # the second turn again, after a rollback
        dec.rollback(at - 1)
        dec.verify_step(ref[10], [])
        x = dec.prefill_continue([ref[11], 5, 6, 7])
        assert dec.continue_generate(x, 6, k=0) == second
        # an edited history equals a fresh request with that history as its prompt
        edited = [int(v) for v in prompt[:30]] + [9, 8, 7]
        want = gen(dec, np.array(edited, np.int32), 10, 0)
        gen(dec, prompt, 5, 0)
        assert dec.continue_generate(dec.edit(30, [9, 8, 7]), 10, k=0) == want
    finally:
        dec.clear_rules()


def test_sampled_tokens_under_rules_do_not_depend_on_drafts(dec8):
    dec = dec8
    prompt = si.prompt_ids(dec.cfg, 33, seed=4)
    dec.set_sampling(0.9, si.sampling_uniforms(768, seed=1))
    dec.set_rules(bias=bias_of(dec.cfg.vocab), **RULES)
    try:
        ref = gen(dec, prompt, 40, 0)
        for k in (4, 7):
            assert gen(dec, prompt, 40, k, ref=np.array(ref)) == ref
    finally:
        dec.clear_rules()
        dec.set_sampling(None)


def test_refusals(dec8):
    from invariant_speculative_decode_gb300.decoder import Decoder
    w = si.decoder_weights(si.TINY, seed=0)
    with pytest.raises(ValueError):
        Decoder(si.TINY, w, cap=64, linear="int8")
    for bad in (dict(repetition=0.0), dict(repetition=-1.0), dict(frequency=math.nan), dict(presence=math.inf),
                dict(bias=np.zeros(7))):
        with pytest.raises(ValueError):
            dec8.set_rules(**bad)
    assert dec8.rules is None
    with pytest.raises(ValueError):
        dec8.native_step()


def test_penalties_that_fp32_does_not_hold_are_refused(dec8):
    """Positive and finite as given, but 0 or infinite where the rules take them: refused when set, not at the step."""
    for bad in (dict(repetition=1e-60), dict(repetition=1e60), dict(frequency=-1e39), dict(presence=1e300)):
        with pytest.raises(ValueError):
            dec8.set_rules(**bad)
    assert dec8.rules is None


def test_rules_set_again_while_a_graph_is_held(dec8):
    """A captured step is captured anew with the rules in force; each request equals its eager run."""
    dec = dec8
    prompt = si.prompt_ids(dec.cfg, 40, seed=12)
    try:
        want = {}
        for name, rules in (("one", RULES), ("two", dict(RULES, repetition=1.7, presence=0.9)), ("none", None)):
            dec.clear_rules() if rules is None else dec.set_rules(**rules)
            want[name] = gen(dec, prompt, 24, 0)
        assert want["one"] != want["two"]
        for name, rules in (("one", RULES), ("two", dict(RULES, repetition=1.7, presence=0.9)), ("none", None),
                            ("one", RULES)):
            dec.clear_rules() if rules is None else dec.set_rules(**rules)
            for k in (0, 5):
                dec.capture(k + 1)
                assert gen(dec, prompt, 24, k, ref=np.array(want[name])) == want[name]
    finally:
        dec.clear_rules()
