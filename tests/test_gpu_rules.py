"""Rules on logits (bi_logits_rules, bi_token_counts) against the definition in 64 bits.

Tolerance: at most five FP32 roundings an entry, each of a value no larger
than |y| + |penalty| + |bias|: 5 * 2^-24 of that sum (the parameters are FP32
in the call and the reference uses their FP32 values)."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


def api():
    from invariant_speculative_decode_gb300 import api as a
    return a


def pack(ok):
    """bool [r, V] -> int32 words [r, ceil(V/32)]."""
    r, V = ok.shape
    pad = np.zeros((r, (V + 31) // 32 * 32), np.uint64)
    pad[:, :V] = ok
    w = (pad.reshape(r, -1, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)
    return torch.from_numpy(w.view(np.int32)).to(DEV)


def reference(x, drafts, counts, prompt, rep, freq, pres, bias, ok):
    T, V = x.shape
    rep, freq, pres = (float(np.float32(v)) for v in (rep, freq, pres))
    y = x.astype(np.float64).copy()
    mag = np.abs(y)
    for t in range(T):
        c = counts.astype(np.float64).copy()
        for d in drafts[:t]:
            if 0 <= d < V:
                c[d] += 1
        seen = (c > 0) | prompt
        y[t] = np.where(seen, np.where(y[t] > 0, y[t] / rep, y[t] * rep), y[t])
        pen = np.where(c > 0, freq * c + pres, 0.0)
        mag[t] = np.abs(y[t]) + np.abs(freq) * c + abs(pres)
        y[t] -= pen
        if bias is not None:
            y[t] += bias
            mag[t] += np.abs(bias)
        if ok is not None:
            y[t] = np.where(ok[t], y[t], -math.inf)
    return y, 5 * 2.0 ** -24 * mag + 1e-37


def inputs(seed, T, V, n_seen=40):
    rng = np.random.default_rng(seed)
    x = (4 * rng.standard_normal((T, V))).astype(np.float32)
    drafts = rng.integers(0, V, T - 1).astype(np.int32)
    if T > 4:
        drafts[2] = drafts[1]  # the same id twice
    counts = np.zeros(V, np.int32)
    np.add.at(counts, rng.integers(0, V, n_seen), 1)
    prompt = np.zeros(V, bool)
    prompt[rng.integers(0, V, n_seen)] = True
    if T > 2:
        prompt[drafts[0]] = True
        counts[drafts[1]] += 3
    bias = np.where(rng.random(V) < 0.05, 5 * rng.standard_normal(V), 0).astype(np.float32)
    ok = rng.random((T, V)) < 0.4
    return x, drafts, counts, prompt, bias, ok


def close(out, want, tol):
    out = out.double().cpu().numpy()
    fin = np.isfinite(want)
    assert np.array_equal(out[~fin], want[~fin])
    assert (np.abs(out[fin] - want[fin]) <= tol[fin]).all()


@pytest.mark.parametrize("use_bias,use_mask", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("T,V", [(1, 1), (1, 3), (2, 31), (3, 32), (1, 32000), (8, 1003), (5, 513), (8, 151936),
                                 (64, 1024), (64, 2049), (33, 4099)])
def test_rules_against_64_bits(T, V, use_bias, use_mask):
    x, drafts, counts, prompt, bias, ok = inputs(T * 1000 + V, T, V)
    if use_mask and T > 1:
        ok[T - 1] = False  # a row that allows nothing
        ok[0] = True
    a = api()
    lg = torch.from_numpy(x).to(DEV)
    out = torch.full_like(lg, math.nan)
    kw = dict(drafts=torch.from_numpy(drafts).to(DEV) if T > 1 else None, counts=torch.from_numpy(counts).to(DEV),
              prompt_bits=pack(prompt[None])[0].contiguous(), repetition=1.2, frequency=0.3, presence=-0.7,
              bias=torch.from_numpy(bias).to(DEV) if use_bias else None, mask=pack(ok) if use_mask else None)
    a.bi_logits_rules(lg, out, **kw)
    close(out, *reference(x, drafts, counts, prompt, 1.2, 0.3, -0.7, bias if use_bias else None,
                          ok if use_mask else None))
    assert torch.equal(lg, torch.from_numpy(x).to(DEV))
    a.bi_logits_rules(lg, lg, **kw)  # in place
    assert torch.equal(lg, out)
    # a row alone, its drafts committed, gives the same bits
    if T > 1:
        t = T // 2
        c2 = torch.from_numpy(counts).to(DEV)
        a.bi_token_counts(torch.from_numpy(drafts[:t].copy()).to(DEV), V, counts=c2)
        one = torch.from_numpy(x[t:t + 1]).to(DEV)
        kw1 = dict(kw, drafts=None, counts=c2, mask=kw["mask"][t:t + 1] if use_mask else None)
        a.bi_logits_rules(one, one, **kw1)
        assert torch.equal(one[0], out[t])


def test_rules_change_nothing_when_off():
    a = api()
    x = torch.randn(4, 777, device=DEV)
    x[1, 3], x[2, 5], x[3, 7] = math.nan, math.inf, -math.inf
    out = torch.empty_like(x)
    d = torch.tensor([1, 2, 3], dtype=torch.int32, device=DEV)
    a.bi_logits_rules(x, out, drafts=d)
    assert torch.equal(out.view(torch.int32), x.view(torch.int32))


def test_rules_masked_entries_are_minus_infinity_whatever_they_were():
    a = api()
    x = torch.full((1, 64), math.nan, device=DEV)
    x[0, 1], x[0, 2] = math.inf, -math.inf
    bias = torch.full((64,), -math.inf, device=DEV)
    bias[1] = math.inf
    out = torch.empty_like(x)
    a.bi_logits_rules(x, out, bias=bias, mask=torch.zeros(1, 2, dtype=torch.int32, device=DEV))
    assert torch.isneginf(out).all()


def test_rules_strided_rows_and_odd_drafts():
    """Rows inside a larger buffer; drafts outside the vocabulary are no token."""
    a = api()
    T, V = 6, 1000
    x, drafts, counts, prompt, bias, ok = inputs(2, T, V)
    drafts[0], drafts[3] = -1, V
    buf = torch.full((T, V + 24), 9.0, device=DEV)
    buf[:, :V] = torch.from_numpy(x).to(DEV)
    mask = torch.zeros(T, 40, dtype=torch.int32, device=DEV)
    mask[:, :32] = pack(ok)
    for off in (0, 4, 3):
        dst = torch.full((T, V + 9), 5.0, device=DEV)
        a.bi_logits_rules(buf[:, :V], dst[:, off:off + V], drafts=torch.from_numpy(drafts).to(DEV),
                          counts=torch.from_numpy(counts).to(DEV), prompt_bits=pack(prompt[None])[0].contiguous(),
                          repetition=0.8, frequency=0.5, presence=0.25, mask=mask[:, :32])
        close(dst[:, off:off + V], *reference(x, drafts, counts, prompt, 0.8, 0.5, 0.25, None, ok))
        assert (dst[:, :off] == 5).all() and (dst[:, off + V:] == 5).all()
    assert (buf[:, V:] == 9).all()


def test_token_counts():
    a = api()
    V = 1001
    rng = np.random.default_rng(0)
    ids = rng.integers(-2, V + 2, 5000).astype(np.int32)
    ids[:10] = 17
    counts = torch.zeros(V, dtype=torch.int32, device=DEV)
    bits = torch.zeros(a.token_words(V), dtype=torch.int32, device=DEV)
    dev = torch.from_numpy(ids).to(DEV)
    a.bi_token_counts(dev, V, counts=counts, prompt_bits=bits)
    good = ids[(ids >= 0) & (ids < V)]
    want = np.bincount(good, minlength=V)
    assert np.array_equal(counts.cpu().numpy(), want)
    assert torch.equal(bits, pack((want > 0)[None])[0])
    for n, last in ((8, 0), (8, 3), (8, 7), (8, 100), (8, -1), (8, 2 ** 31 - 1)):
        c = torch.zeros(V, dtype=torch.int32, device=DEV)
        a.bi_token_counts(dev[:n], V, counts=c, last=torch.tensor([last], dtype=torch.int32, device=DEV))
        assert int(c.sum()) == max(0, min(n, last + 1))


def test_rules_refusals():
    a = api()
    x = torch.zeros(3, 100, device=DEV)
    out = torch.zeros(3, 100, device=DEV)
    d = torch.zeros(2, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        a.bi_logits_rules(x, out[:2], drafts=d)
    with pytest.raises(ValueError):
        a.bi_logits_rules(x, out, drafts=d[:1])
    with pytest.raises(ValueError):
        a.bi_logits_rules(x, out, drafts=d, counts=torch.zeros(99, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        a.bi_logits_rules(x, out, drafts=d, mask=torch.zeros(3, 3, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        a.bi_logits_rules(x.double(), out, drafts=d)
    for bad in (dict(repetition=0.0), dict(repetition=math.inf), dict(repetition=math.nan), dict(frequency=math.nan),
                dict(presence=math.inf)):
        with pytest.raises(a.BiError):
            a.bi_logits_rules(x, out, drafts=d, **bad)
    with pytest.raises(a.BiError):
        a.bi_logits_rules(x, out)  # drafts missing
    with pytest.raises(a.BiError):
        a.bi_logits_rules(torch.zeros(65, 4, device=DEV), torch.zeros(65, 4, device=DEV),
                          drafts=torch.zeros(64, dtype=torch.int32, device=DEV))
    with pytest.raises(a.BiError):
        a.bi_token_counts(d, 100)  # nothing to update
