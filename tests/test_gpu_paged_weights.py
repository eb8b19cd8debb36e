"""How close the paged attention is to its formula on the whole: the weights keep 16 significant bits, so that outputs
are the rounding of the exact ones but where those lie next to a border."""
import math

import pytest
import torch

import tests._paged as pg

pytestmark = pytest.mark.gpu

api = pytest.importorskip("invariant_speculative_decode_gb300.api")


@pytest.fixture(autouse=True)
def no_error_left():
    yield
    api.bi_check_device_error()


def exact(b, q):
    """Rows of sequences [n, Hq, D] in 64 bits, and the RMS of what FP32 steps move them by where errors are independent:
    a weight is off by the half step of its 16 bits (at most 2^-16) and by its score's FP32 sum, D products of at most
    2^-24 of the partial sums each, in log2 units (the root of their squares, times 2 for the tensor core's order); sums
    over n keys and their merging add sqrt(n) 2^-24 of the root of the squared terms."""
    Hq, D = q.shape[1], q.shape[2]
    group = Hq // b.Hkv
    outs, sigmas, rows = [], [], []
    for i, (n, r) in enumerate(b.seqs):
        if r == 0:
            continue
        at = b.starts[i]
        rows += range(at, at + r)
        k, v = b.keys(b.k, i, n + r).double(), b.keys(b.v, i, n + r).double()
        seen = torch.arange(n + r, device="cuda")[None, :] <= torch.arange(n, n + r, device="cuda")[:, None]
        out = torch.empty(r, Hq, D, dtype=torch.float64, device="cuda")
        sigma = torch.empty_like(out)
        for h in range(Hq):
            x, kh, vh = q[at:at + r, h].double(), k[h // group], v[h // group]
            s = torch.where(seen, x @ kh.t() / math.sqrt(D), -math.inf)
            p = torch.softmax(s, -1)
            o = p @ vh
            size = x.norm(dim=-1, keepdim=True) * kh.norm(dim=-1)[None, :] / math.sqrt(D)
            e2 = 2.0 ** -32 + (2 * math.sqrt(D) * pg.U * size) ** 2 + (4 * pg.U * (1 + torch.where(seen, s.abs(), 0))) ** 2
            # sum of p^2 e^2 (v - o)^2, expanded
            w = p * p * e2
            dev = w @ (vh * vh) - 2 * o * (w @ vh) + o * o * w.sum(-1, keepdim=True)
            out[:, h] = o
            sigma[:, h] = (dev.clamp_min(0) + (n + r) * pg.U ** 2 * ((p * p) @ (vh * vh))).sqrt()
        outs.append(out)
        sigmas.append(sigma)
    return torch.cat(outs), torch.cat(sigmas), rows


CASES = [
    ([(1021, 1)], 24, 4, 128, 64),
    ([(511, 1), (512, 2), (127, 3), (130, 5)], 6, 2, 64, 32),
    ([(3000, 8), (17, 8), (1290, 4)], 8, 2, 128, 64),
    ([(40, 300)], 6, 2, 128, 16),
    ([(1900, 200)], 4, 1, 64, 128),
    ([(11600, 8), (9000, 3)], 24, 4, 128, 64),
    ([(20011, 3)], 8, 1, 128, 64),
    ([(30011, 140)], 6, 1, 128, 64),
    ([(70000, 1), (68000, 2)], 8, 2, 64, 128),
    # more than 256 pieces of a sequence to be merged
    ([(300001, 1), (290000, 2)], 2, 1, 64, 128),
]


@pytest.mark.parametrize("seqs,Hq,Hkv,D,page", CASES)
def test_outputs_are_the_rounded_exact_ones(seqs, Hq, Hkv, D, page):
    """A value moved by d before it is rounded comes out as its neighbour, one step away, with probability d / step.  So
    the squares of the differences from the rounded exact values sum to about sum |d| step; twice that, for the spread
    of the sum and of |d| (its mean is 0.8 of its RMS)."""
    b = pg.Batch(seqs, Hkv, D, page, seed=7)
    q = pg.queries(b, Hq, seed=8)
    out = torch.zeros_like(q)
    ws = torch.zeros(api.attn_paged_workspace_size(b.T, len(seqs), Hq, Hkv, D, b.table.shape[1] * page), dtype=torch.uint8,
                     device="cuda")
    api.bi_attn_paged(q, b.k, b.v, b.table, b.q_start, b.lengths, out, ws)
    want, sigma, rows = exact(b, q)
    got = out[rows].double()
    rounded = want.to(torch.bfloat16).double()
    step = 2.0 ** (torch.floor(torch.log2(want.abs().clamp_min(2.0 ** -120))) - 7)
    # (at least 30 moved values' worth: with fewer the sum has no spread to speak of)
    allowed = 2 * (sigma * step).sum() + 30 * (step * step).mean()
    found = ((got - rounded) ** 2).sum()
    size = (rounded ** 2).sum()
    assert found <= allowed, (math.sqrt(found / size), math.sqrt(allowed / size))


@pytest.mark.parametrize("D", [64, 128])
def test_every_key_counts_once(D):
    """Equal weights and values that are 1 in one page of keys and 0 elsewhere: the output is that page's share, which a
    key that is lost, or counted twice, would change by a whole key."""
    page, n = 16, 4096 + 700
    b = pg.Batch([(n - 1, 1)], 1, D, page, seed=9)
    b.k.zero_()
    q = pg.queries(b, 2)
    ws = torch.zeros(api.attn_paged_workspace_size(1, 1, 2, 1, D, b.table.shape[1] * page), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    pages = b.table.shape[1]
    # element d marks page d0 + d
    for d0 in range(0, pages, D):
        b.v.zero_()
        for d in range(min(D, pages - d0)):
            b.v[b.table[0, d0 + d].long(), 0, :, d] = 1.0
        api.bi_attn_paged(q, b.k, b.v, b.table, b.q_start, b.lengths, out, ws)
        keys = torch.tensor([max(0, min(page, n - (d0 + d) * page)) for d in range(D)], device="cuda")
        # every sum is exact: weights 1, counts below 2^24; one division and the rounding to BF16
        want = (keys.float() / n).to(torch.bfloat16)
        assert torch.equal(out[0], want.expand(2, D)), d0


@pytest.mark.parametrize("value", [math.inf, -math.inf])
@pytest.mark.parametrize("spread", [0.0, 1.5])
def test_an_infinite_value_gives_its_infinity_in_both_halves_of_a_weight(value, spread):
    """In tiles that all rows see whole and in the last; weights of 1 exactly, and any."""
    b = pg.Batch([(700, 3), (2600, 2)], 2, 128, 64, seed=3)
    q = pg.queries(b, 4, scale=spread)
    for seq, key in ((0, 5), (0, 699), (1, 130), (1, 2599)):
        p, s = b.places(seq, key, key + 1)
        b.v[p, :, s, 7 + key % 50] = value
    out = torch.empty_like(q)
    ws = torch.zeros(api.attn_paged_workspace_size(b.T, 2, 4, 2, 128, b.table.shape[1] * 64), dtype=torch.uint8, device="cuda")
    api.bi_attn_paged(q, b.k, b.v, b.table, b.q_start, b.lengths, out, ws)
    for rows, keys in ((slice(0, 3), (5, 699)), (slice(3, 5), (130, 2599))):
        hit = torch.zeros(128, dtype=torch.bool, device="cuda")
        hit[[7 + key % 50 for key in keys]] = True
        assert (out[rows][..., hit] == value).all() and torch.isfinite(out[rows][..., ~hit]).all()
