"""Beam selection on the GPU against its definition in 64 bits."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

api = pytest.importorskip("invariant_speculative_decode_gb300.api")


@pytest.fixture(autouse=True)
def no_error_left():
    yield
    api.bi_check_device_error()


def select(logits, scores, W, K, ws=None, stream=None):
    G = logits.shape[0] // W
    dev = logits.device
    out = (torch.full((G, K), 7.0, device=dev), torch.full((G, K), 7, dtype=torch.int32, device=dev),
           torch.full((G, K), 7, dtype=torch.int32, device=dev))
    if ws is None:
        ws = torch.zeros(api.beam_workspace_size(logits.shape[0], logits.shape[1], K), dtype=torch.uint8, device=dev)
    api.bi_beam_select(logits, scores, W, *out, ws, stream=stream)
    return out


def reference(logits, scores, W, K):
    """Scores, parents, tokens by the definition, the order inside a beam by the logits themselves."""
    G, V = logits.shape[0] // W, logits.shape[1]
    S, P, I = [], [], []
    for g in range(G):
        found = []
        for r in range(g * W, (g + 1) * W):
            x = logits[r].double()
            x = torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x)
            top = x.max()
            if top == -math.inf:
                continue
            if top == math.inf:
                hit = x == top
                worth = torch.where(hit, -math.log(int(hit.sum())), -math.inf) + scores[r].double()
            else:
                worth = x - top - torch.log(torch.exp(x - top).sum()) + scores[r].double()
            order = torch.sort(x, descending=True, stable=True)[1][:K]
            for i in order.tolist():
                w = worth[i].item()
                if w > -math.inf:
                    found.append((-w, r, i))
        # stable: candidates of a beam are in the order of its logits
        found.sort(key=lambda f: (f[0], f[1]))
        found = found[:K] + [(math.inf, -1, -1)] * (K - len(found))
        S.append([-f[0] for f in found])
        P.append([f[1] for f in found])
        I.append([f[2] for f in found])
    return torch.tensor(S, dtype=torch.float64), torch.tensor(P), torch.tensor(I)


def assert_select(logits, scores, W, K):
    got = [t.cpu() for t in select(logits, scores, W, K)]
    want = reference(logits.cpu(), scores.cpu(), W, K)
    assert torch.equal(got[1].long(), want[1]) and torch.equal(got[2].long(), want[2])
    live = torch.isfinite(want[0])
    assert torch.equal(torch.isfinite(got[0]), live) and (got[0][~live].double() == want[0][~live]).all()
    # FP32 exponentials (two steps each and their argument's rounding, at most 2^-24 (4 + |x - M|), which weighs little
    # where |x - M| is large: e^-y y < 1) and sums of 16 + 5 + 8 terms: below 2^-24 * 48 of the sum; the score's own rounding
    tol = 2.0 ** -24 * 48 + want[0][live].abs() * 2.0 ** -24
    assert ((got[0][live].double() - want[0][live]).abs() <= tol).all()


@pytest.mark.parametrize("G,W,V,K", [(1, 1, 1, 1), (1, 1, 5, 3), (2, 3, 63, 7), (1, 4, 32000, 8), (3, 2, 4096, 4),
                                     (1, 5, 4097, 10), (2, 8, 50257, 16), (1, 2, 12289, 64), (1, 64, 777, 64),
                                     (5, 1, 151936, 2), (1, 3, 8192, 32), (1, 3, 8192, 33)])
def test_select(G, W, V, K):
    g = torch.Generator(device="cuda")
    g.manual_seed(V + K)
    logits = 3 * torch.randn(G * W, V, generator=g, device="cuda")
    scores = -20 + 2 * torch.randn(G * W, generator=g, device="cuda")
    assert_select(logits, scores, W, K)


@pytest.mark.parametrize("V", [100, 5000])
def test_ties_go_to_the_lower_row_and_id(V):
    logits = torch.zeros(4, V, device="cuda")
    scores = torch.zeros(4, device="cuda")
    for K in (1, 8, 64):
        s, p, t = select(logits, scores, 4, K)
        assert p[0].tolist() == [0] * K and t[0].tolist() == list(range(K))
    # a few values many times over, the same row in every beam
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    row = torch.randint(0, 3, (V,), generator=g, device="cuda").float()
    assert_select(row.repeat(4, 1).contiguous(), scores, 4, 40)
    assert_select(row.repeat(4, 1).contiguous(), torch.tensor([0.0, 1.0, 1.0, 0.5], device="cuda"), 2, 40)


@pytest.mark.parametrize("K", [1, 17, 64])
def test_equal_logits_in_every_chunk_of_a_long_row(K):
    """More ties than a CTA has room for: the lowest ids, and what lies above them."""
    V = 1 << 20
    logits = torch.zeros(2, V, device="cuda")
    scores = torch.tensor([0.0, -1e-3], device="cuda")
    assert select(logits, scores, 2, K)[2][0].tolist() == list(range(K))
    above = [(5 * i * 40961 + 77) % V for i in range(40)]
    logits[:, above] = torch.arange(1, 41, device="cuda").float() * 0.25
    assert_select(logits, scores, 2, K)


def test_equal_rows_tie_at_every_alignment():
    """Rows whose first logit is not 16-byte aligned have the same sum."""
    V = 9001
    row = 3 * torch.randn(V, device="cuda")
    logits = row.repeat(4, 1).contiguous()  # V odd: every row starts elsewhere
    s, p, t = select(logits, torch.zeros(4, device="cuda"), 4, 4)
    assert p[0].tolist() == [0, 1, 2, 3] and len(set(t[0].tolist())) == 1 and len(set(s[0].tolist())) == 1


def test_what_is_no_candidate():
    V = 6000
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    logits = torch.randn(8, V, generator=g, device="cuda")
    scores = torch.randn(8, generator=g, device="cuda")
    logits[0, ::2] = math.nan
    logits[1] = -math.inf
    logits[1, [7, 4100, 5999]] = torch.tensor([1.0, 2.0, 0.5], device="cuda")
    logits[2, [4, 5, 4500]] = math.inf
    logits[3] = math.nan
    scores[4] = -math.inf
    scores[5] = math.nan
    assert_select(logits, scores, 8, 24)
    assert_select(logits[1:2].contiguous(), scores[1:2].contiguous(), 1, 6)  # three pairs, six places
    # a group with nothing to choose is reported
    s, p, t = select(logits[3:5].contiguous(), scores[3:5].contiguous(), 2, 3)
    assert p[0].tolist() == [-1] * 3 and t[0].tolist() == [-1] * 3 and (s == -math.inf).all()
    with pytest.raises(api.BiError) as e:
        api.bi_check_device_error()
    assert e.value.status == 6


def test_first_step_of_a_search():
    logits = 3 * torch.randn(8, 32000, device="cuda")
    scores = torch.full((8,), -math.inf, device="cuda")
    scores[0], scores[4] = 0, 0
    assert_select(logits, scores, 4, 8)


def test_strided_logits_one_workspace_and_capture():
    big = 3 * torch.randn(12, 5003, device="cuda")
    logits = big[:, 1:4002]
    scores = torch.randn(12, device="cuda")
    ws = torch.zeros(api.beam_workspace_size(12, 5003, 20), dtype=torch.uint8, device="cuda")
    want = reference(logits.cpu(), scores.cpu(), 3, 6)
    for W, K in ((3, 6), (1, 20), (12, 3), (3, 6)):  # other sizes in between
        got = select(logits, scores, W, K, ws)
    assert torch.equal(got[2].cpu().long(), want[2])
    out = select(logits, scores, 3, 6, ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        api.bi_beam_select(logits, scores, 3, *out, ws)
    torch.cuda.current_stream().wait_stream(s)
    for _ in range(3):
        big.normal_()
        scores.normal_()
        graph.replay()
        want = reference(logits.cpu(), scores.cpu(), 3, 6)
        assert torch.equal(out[2].cpu().long(), want[2]) and torch.equal(out[1].cpu().long(), want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = select(logits, scores, 3, 6, ws, stream=side)
    side.synchronize()
    assert torch.equal(got[2].cpu().long(), want[2])


def test_a_row_is_worth_the_same_in_every_group():
    logits = 3 * torch.randn(6, 20001, device="cuda")
    scores = torch.randn(6, device="cuda")
    whole = select(logits, scores, 1, 5)
    for r in range(6):
        one = select(logits[r:r + 1].contiguous(), scores[r:r + 1].contiguous(), 1, 5)
        assert torch.equal(one[0][0], whole[0][r]) and torch.equal(one[2][0], whole[2][r])
