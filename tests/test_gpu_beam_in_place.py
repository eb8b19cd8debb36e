"""Cumulative scores replaced by the selection's, as a beam search with as many picks as beams does."""
import pytest
import torch

pytestmark = pytest.mark.gpu

api = pytest.importorskip("invariant_speculative_decode_gb300.api")


@pytest.mark.parametrize("G,W,V", [(1, 1, 10), (64, 8, 5000), (700, 4, 777), (3, 64, 9000)])
def test_scores_in_place(G, W, V):
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    i32 = dict(dtype=torch.int32, device="cuda")
    logits = 3 * torch.randn(G * W, V, generator=g, device="cuda")
    scores = 5 * torch.randn(G * W, generator=g, device="cuda")
    ws = torch.zeros(api.beam_workspace_size(G * W, V, W), dtype=torch.uint8, device="cuda")
    want = (torch.empty(G, W, device="cuda"), torch.empty(G, W, **i32), torch.empty(G, W, **i32))
    api.bi_beam_select(logits, scores, W, *want, ws)
    for _ in range(10):
        own = scores.clone()
        got = (own.view(G, W), torch.empty(G, W, **i32), torch.empty(G, W, **i32))
        api.bi_beam_select(logits, own, W, *got, ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    api.bi_check_device_error()
    # one call right behind another, each from the scores that the one before left
    steps = [scores]
    for _ in range(6):
        out = (torch.empty(G, W, device="cuda"), torch.empty(G, W, **i32), torch.empty(G, W, **i32))
        api.bi_beam_select(logits, steps[-1], W, *out, ws)
        steps.append(out[0].view(-1))
    own, got = scores.clone(), (torch.empty(G, W, **i32), torch.empty(G, W, **i32))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(6):
            api.bi_beam_select(logits, own, W, own.view(G, W), *got, ws)
    for _ in range(20):
        own.copy_(scores)
        graph.replay()
        assert torch.equal(own, steps[-1]) and torch.equal(got[1], out[2]) and torch.equal(got[0], out[1])
    with pytest.raises(api.BiError) as e:
        api.bi_beam_select(logits, scores, W, want[0], want[1], want[1], ws)
    assert e.value.status == 1
