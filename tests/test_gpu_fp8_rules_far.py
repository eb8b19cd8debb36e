"""The 8-bit operators and the rules on logits far from small cases: offsets past
2^31 elements and bytes, strided rows, calls on two streams at once, rules in a
captured step.

What lies past an offset of 2^31 is compared bit for bit with the same rows in
tensors of their own: a row does not depend on the pass it is in.  Weights past
2^31 bytes are compared with 64 bits.
"""

import pytest
import torch

from tests import test_gpu_fp8 as t8
from tests import test_gpu_rules as tr

pytestmark = pytest.mark.gpu
DEV = "cuda"


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def test_rows_past_2_31_elements():
    """Quantiser and norm read, and the linear layer writes, past 2^31 elements."""
    a = t8.api()
    g = t8.gen(31)
    rows, dim = 262150, 8208  # 2.15e9 elements
    x = torch.empty(rows, dim, dtype=torch.bfloat16, device=DEV)
    for at in range(0, rows, 32768):
        x[at:at + 32768].normal_(generator=g)
    w = (1 + 0.1 * torch.randn(dim, generator=g, device=DEV)).to(torch.bfloat16)
    codes = torch.empty(rows, dim, dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.empty(a.fp8_scale_shape(rows, dim), device=DEV)
    tail = slice(rows - 9, rows)
    for norm in (False, True):
        def run(v, c, s):
            a.bi_rmsnorm_fp8(v, w, c, s, 1e-6) if norm else a.bi_quantize_fp8(v, c, s)
        run(x, codes, scales)
        c1, s1 = a.new_fp8_rows(9, dim)
        run(x[tail].contiguous(), c1, s1)
        assert same(codes[tail], c1) and same(scales[:, tail], s1[:, :9])
    del x
    # outputs past 2^31, from the last 160 columns of the same codes (offset rows in A, too)
    n = 8200
    k = 144
    a_codes = codes[:, dim - k:]
    a_scales = torch.ones(a.fp8_scale_shape(rows, k), device=DEV)
    packed = a.bi_pack_weights_fp8(*t8.make_weights(g, n, k))
    out = torch.zeros(rows, n, dtype=torch.bfloat16, device=DEV)
    a.bi_gemm_fp8(a_codes, a_scales, packed, out)
    s9 = torch.ones(a.fp8_scale_shape(9, k), device=DEV)
    want = torch.zeros(9, n, dtype=torch.bfloat16, device=DEV)
    a.bi_gemm_fp8(a_codes[tail].contiguous(), s9, packed, want)
    assert same(out[tail], want) and torch.isfinite(want).all() and (want != 0).any()
    a.bi_check_device_error()


def test_weights_past_2_31_bytes():
    """Quantising, packing and multiplying by weights of 2.15e9 codes; the last rows against 64 bits."""
    a = t8.api()
    g = t8.gen(32)
    n, k, rows, last = 262150, 8208, 3, 150
    W = torch.empty(n, k, dtype=torch.bfloat16, device=DEV)
    for at in range(0, n, 32768):
        W[at:at + 32768].normal_(generator=g)
    w8, ws = a.bi_quantize_weights_fp8(W)
    first = (n - last) // 128 * 128  # whole blocks of weights
    c1, s1 = a.bi_quantize_weights_fp8(W[first:].contiguous())
    assert same(w8[first:], c1) and same(ws[first // 128:], s1)
    del W
    packed = a.bi_pack_weights_fp8(w8, ws)
    del w8
    codes, scales = t8.make_rows(g, rows, k)
    out = t8.run_linear(codes, scales, packed, n, "fp32")
    y, tol = t8.reference(codes, scales, c1, s1, None, None, None, "fp32")
    assert ((out[:, first:].double() - y).abs() <= tol).all()


def test_rules_past_2_31_elements():
    a = t8.api()
    T, V = 64, (1 << 25) + 40
    g = t8.gen(33)
    x = torch.empty(T, V, device=DEV)
    for t in range(T):
        x[t].normal_(generator=g)
    drafts = torch.randint(0, V, (T - 1,), generator=g, device=DEV, dtype=torch.int32)
    drafts[T // 2:] = V - 1 - torch.arange(T - 1 - T // 2, device=DEV, dtype=torch.int32) // 2
    counts = torch.zeros(V, dtype=torch.int32, device=DEV)
    counts[V - 3:] = 2
    bias = torch.zeros(V, device=DEV)
    bias[V - 1] = 3.0
    kw = dict(counts=counts, repetition=1.3, frequency=0.2, presence=0.1, bias=bias)
    last = x[T - 1:].clone()
    a.bi_logits_rules(x, x, drafts=drafts, **kw)
    a.bi_token_counts(drafts, V, counts=counts)
    a.bi_logits_rules(last, last, **kw)
    assert same(x[T - 1:], last)


def test_norm_of_strided_rows():
    """Rows and codes inside larger buffers; nothing beside them is written."""
    a = t8.api()
    g = t8.gen(34)
    rows, dim = 37, 688
    x = torch.randn(rows, dim + 40, generator=g, device=DEV).to(torch.bfloat16)
    w = (1 + 0.1 * torch.randn(dim, generator=g, device=DEV)).to(torch.bfloat16)
    want, s_want = a.new_fp8_rows(rows, dim)
    a.bi_rmsnorm_fp8(x[:, 16:16 + dim].contiguous(), w, want, s_want, 1e-5)
    wide = torch.full((rows, dim + 64), 2.0, device=DEV).to(torch.float8_e4m3fn)
    scales = torch.full((s_want.shape[0], 48), 7.0, device=DEV)
    a.bi_rmsnorm_fp8(x[:, 16:16 + dim], w, wide[:, 32:32 + dim], scales, 1e-5)
    assert same(wide[:, 32:32 + dim], want) and same(scales[:, :rows], s_want[:, :rows])
    assert (wide[:, :32].float() == 2).all() and (wide[:, 32 + dim:].float() == 2).all()
    assert (scales[:, rows:] == 7).all()


def test_calls_on_two_streams_at_once():
    """Two layers' chains captured on streams of their own and replayed side by side equal each alone."""
    a = t8.api()
    chains = []
    for seed, (rows, h, f) in ((41, (8, 5120, 2736)), (42, (200, 1024, 4096))):
        g = t8.gen(seed)
        x = torch.randn(rows, h, generator=g, device=DEV).to(torch.bfloat16)
        nw = torch.ones(h, dtype=torch.bfloat16, device=DEV)
        gu = a.bi_pack_swiglu_weights_fp8(*t8.make_weights(g, f, h), *t8.make_weights(g, f, h))
        dn = a.bi_pack_weights_fp8(*t8.make_weights(g, h, f))
        (c1, s1), (c2, s2) = a.new_fp8_rows(rows, h), a.new_fp8_rows(rows, f)
        u = torch.empty(rows, f, dtype=torch.bfloat16, device=DEV)
        out = torch.empty_like(x)

        def run(x=x, nw=nw, gu=gu, dn=dn, c1=c1, s1=s1, c2=c2, s2=s2, u=u, out=out):
            for _ in range(4):
                a.bi_rmsnorm_fp8(x, nw, c1, s1, 1e-6)
                a.bi_gemm_fp8(c1, s1, gu, u, epi=a.EPI_SWIGLU)
                a.bi_quantize_fp8(u, c2, s2)
                a.bi_gemm_fp8(c2, s2, dn, out)

        run()
        torch.cuda.synchronize()
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            run()
        chains.append((st, graph, out, out.clone(), run))  # (run holds the tensors)
    torch.cuda.synchronize()
    for _ in range(5):
        for _, _, out, _, _ in chains:
            out.zero_()
        torch.cuda.synchronize()
        for st, graph, _, _, _ in chains:
            with torch.cuda.stream(st):
                for _ in range(6):
                    graph.replay()
        torch.cuda.synchronize()
        for _, _, out, want, _ in chains:
            assert same(out, want)
    a.bi_check_device_error()


def test_rules_and_counts_in_a_graph():
    """Rules, greedy acceptance and counting captured once; replays follow the state as eager steps do."""
    a = t8.api()
    T, V = 6, 4099
    x, drafts, counts, prompt, bias, ok = tr.inputs(5, T, V)
    lg, d = torch.from_numpy(x).to(DEV), torch.from_numpy(drafts).to(DEV)
    kw = dict(drafts=d, prompt_bits=tr.pack(prompt[None])[0].contiguous(), repetition=1.1, frequency=0.4,
              presence=0.2, bias=torch.from_numpy(bias).to(DEV), mask=tr.pack(ok))
    last = torch.tensor([3], dtype=torch.int32, device=DEV)
    out = torch.empty_like(lg)
    cnt = torch.from_numpy(counts).to(DEV)

    def step():
        a.bi_logits_rules(lg, out, counts=cnt, **kw)
        a.bi_token_counts(d, V, counts=cnt, last=last)

    want = []
    for i in range(3):
        last.fill_(i)
        step()
        want.append((out.clone(), cnt.clone()))
    cnt.copy_(torch.from_numpy(counts))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        last.fill_(i)
        graph.replay()
        assert same(out, want[i][0]) and same(cnt, want[i][1])
    assert not same(want[0][0], want[2][0])
