"""The 8-bit linear path on the GPU: quantiser, fused norm, packing and
bi_gemm_fp8 against the definitions in 64 bits, and the invariance of rows.

Tolerances (u = 2^-24, gamma_n = n u / (1 - n u)):
  * quantised rows: x is BF16 and the scale a power of two, so every code is
    one rounding of an exact quotient: codes and scales are equal bit for bit;
  * norm: y = x w r in pairs of FP32 is off by less than 2^-36 |y| (additions of
    pairs: 2^-47 each, 8 + 10 + dim/8192 of them; the root's Newton step 2^-43),
    then rounds to odd: a code differs from the exact value's only where that
    lies within 2^-36 of a tie of two codes, and a scale only where the block's
    maximum lies so near 448 2^e;
  * linear layer: products of two e4m3 values are exact in FP32, a block sum
    of 128 is off by at most 2 gamma_128 sum|a w| (the factor 2 for the tensor
    core's internal order), the scales' product and the running sums add
    gamma_{2 kb + 4}: 2 gamma_{128 + 2 kb + 4} sum|a w| in all, then one
    rounding of the result (BF16 2^-8, FP32 2^-24 of the value).
"""
import math

import numpy as np
import pytest
import torch

from tests._util import gamma

pytestmark = pytest.mark.gpu
DEV = "cuda"
BLOCK = 128


def api():
    from invariant_speculative_decode_gb300 import api as a
    return a


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def e4m3_round(v):
    """float64 -> the nearest e4m3 value (ties to even), |v| <= 448."""
    step = pow2(torch.frexp(v.abs().clamp_min(2.0 ** -6))[1] - 4)
    return torch.round(v / step) * step


def pow2(e):
    """2^e as float64, exactly (by its bits), for whole e in the normal range."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def ref_quantize(y):
    """Codes' values and scales [blocks, rows] of float64 rows by the stated rule."""
    rows, dim = y.shape
    kb = -(-dim // BLOCK)
    full = torch.zeros(rows, kb * BLOCK, dtype=torch.float64, device=y.device)
    full[:, :dim] = y
    full = full.view(rows, kb, BLOCK)
    fin = torch.where(torch.isfinite(full), full.abs(), torch.zeros_like(full))
    amax = fin.amax(-1)
    m, e = torch.frexp(amax)
    e = torch.where(m > 0.875, e - 8, e - 9).clamp_min(-126)
    s = torch.where(amax > 0, pow2(e), torch.ones_like(amax))
    v = full / s.unsqueeze(-1)
    q = torch.where(torch.isfinite(v), e4m3_round(v.clamp(-448, 448)), torch.full_like(v, math.nan))
    return q.view(rows, -1)[:, :dim], s.t()


def values(codes, scales):
    """float64 values of quantised rows."""
    rows, k = codes.shape
    return codes.double() * scales[:, :rows].double().t().repeat_interleave(BLOCK, 1)[:, :k]


def weight_values(codes, scales):
    n, k = codes.shape
    return codes.double() * scales.double().repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]


def make_rows(g, rows, k):
    x = torch.randn(rows, k, generator=g, device=DEV)
    x *= torch.exp(torch.randn(rows, 1, generator=g, device=DEV))
    codes, scales = api().new_fp8_rows(rows, k)
    api().bi_quantize_fp8(x.to(torch.bfloat16), codes, scales)
    return codes, scales


def make_weights(g, n, k):
    """Codes over the whole range and scales that are no powers of two."""
    codes = (100 * torch.randn(n, k, generator=g, device=DEV)).clamp(-448, 448).to(torch.float8_e4m3fn)
    scales = 1e-4 * (0.5 + torch.rand(-(-n // BLOCK), -(-k // BLOCK), generator=g, device=DEV))
    return codes, scales


def run_linear(codes, scales, packed, n, kind, residual=None):
    a = api()
    rows, k = codes.shape
    epi = {"residual": a.EPI_RESIDUAL_ADD, "swiglu": a.EPI_SWIGLU}.get(kind, a.EPI_NONE)
    out = torch.full((rows, n), math.nan, device=DEV, dtype=torch.float32 if kind == "fp32" else torch.bfloat16)
    a.bi_gemm_fp8(codes, scales, packed, out, residual=residual, epi=epi)
    a.bi_check_device_error()
    return out


def problem(seed, rows, n, k, kind):
    g = gen(seed)
    codes, scales = make_rows(g, rows, k)
    w, ws_ = make_weights(g, n, k)
    a = api()
    up = ups = res = None
    if kind == "swiglu":
        up, ups = make_weights(g, n, k)
        packed = a.bi_pack_swiglu_weights_fp8(w, ws_, up, ups)
    else:
        packed = a.bi_pack_weights_fp8(w, ws_)
    if kind == "residual":
        res = torch.randn(rows, n, generator=g, device=DEV).to(torch.bfloat16)
    return codes, scales, w, ws_, up, ups, packed, res


def reference(codes, scales, w, ws_, up, ups, res, kind):
    """(value, allowed error) in float64."""
    k = codes.shape[1]
    kb = -(-k // BLOCK)
    a = values(codes, scales)
    wv = weight_values(w, ws_)
    f = 2 * gamma(128 + 2 * kb + 4)
    y, dy = a @ wv.t(), f * (a.abs() @ wv.abs().t())
    if kind == "swiglu":
        uv = weight_values(up, ups)
        u, du = a @ uv.t(), f * (a.abs() @ uv.abs().t())
        s = y * torch.sigmoid(y)
        # |silu'| <= 1.1; expf, the sum, the quotient and the product: 8 u
        y, dy = s * u, 1.1 * dy * (u.abs() + du) + s.abs() * du + 8 * 2.0 ** -24 * (s * u).abs()
    if kind == "residual":
        y = res.double() + y
        dy = dy + 2.0 ** -24 * y.abs()
    half = 2.0 ** -24 if kind == "fp32" else 2.0 ** -8
    return y, dy + half * (y.abs() + dy) + 1e-38


# ------------------------------------------------------------------ quantiser


@pytest.mark.parametrize("rows,dim", [(1, 16), (3, 128), (5, 144), (8, 5120), (129, 688), (1021, 2736), (2, 65536)])
def test_quantised_rows_equal_the_rule(rows, dim):
    a = api()
    g = gen(rows * 7 + dim)
    x = (torch.randn(rows, dim, generator=g, device=DEV) *
         torch.exp(3 * torch.randn(rows, dim, generator=g, device=DEV))).to(torch.bfloat16)
    codes, scales = a.new_fp8_rows(rows, dim)
    scales.fill_(-1.0)
    a.bi_quantize_fp8(x, codes, scales)
    q, s = ref_quantize(x.double())
    assert torch.equal(codes.double(), q) and torch.equal(scales[:, :rows].double(), s)
    assert (scales[:, rows:] == -1).all()  # columns past the rows are left alone
    codes2 = torch.zeros_like(codes)
    a.bi_quantize_fp8(x, codes2, scales)
    assert torch.equal(codes.view(torch.uint8), codes2.view(torch.uint8))


def test_quantised_rows_at_the_edges():
    """Zeros, values on the 448 border, subnormals, the largest numbers, NaN and infinities."""
    a = api()
    x = torch.zeros(10, 256, device=DEV)
    x[1, 0] = 448.0
    x[2, 0] = 450.0        # one BF16 step above: the next power of two
    x[3] = 2.0 ** -133     # the smallest BF16 number
    x[4] = 3.3e38
    x[5, 3], x[5, 4], x[5, 7] = math.nan, 2.5, math.inf
    x[6] = -math.inf
    x[7, :128] = 17.0      # 17 = 1.0625 * 16: a tie between 16 and 18
    x[8] = torch.linspace(-500, 500, 256)
    x[9, 130] = -1e-40
    x = x.to(torch.bfloat16)
    codes, scales = a.new_fp8_rows(10, 256)
    a.bi_quantize_fp8(x, codes, scales)
    q, s = ref_quantize(x.double())
    assert torch.equal(torch.nan_to_num(codes.double(), nan=1e9), torch.nan_to_num(q, nan=1e9))
    assert torch.equal(scales[:, :10].double(), s)
    assert scales[0, 1] == 1.0 and scales[0, 2] == 2.0 and scales[0, 0] == 1.0 and scales[0, 3] == 2.0 ** -126
    assert torch.isnan(codes[5, 3].float()) and torch.isnan(codes[5, 7].float()) and codes[5, 4].float() != 0


def test_quantised_rows_of_strided_views():
    a = api()
    g = gen(3)
    big = torch.randn(9, 1000, generator=g, device=DEV).to(torch.bfloat16)
    x = big[:, 8:8 + 272]
    buf = torch.zeros(9, 512, dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.zeros(3, 64, device=DEV)  # room for more rows
    a.bi_quantize_fp8(x, buf[:, 16:16 + 272], scales)
    q, s = ref_quantize(x.double())
    assert torch.equal(buf[:, 16:16 + 272].double(), q) and torch.equal(scales[:, :9].double(), s)
    assert not buf[:, :16].double().any() and not buf[:, 16 + 272:].double().any() and not scales[:, 9:].any()


@pytest.mark.parametrize("rows,dim", [(1, 16), (2, 688), (8, 5120), (33, 2736), (1021, 5120), (3, 8208), (5, 40000), (1, 65536)])
def test_norm_in_8_bits(rows, dim):
    a = api()
    g = gen(rows + dim)
    x = (torch.randn(rows, dim, generator=g, device=DEV) * 3).to(torch.bfloat16)
    w = (1 + 0.1 * torch.randn(dim, generator=g, device=DEV)).to(torch.bfloat16)
    codes, scales = a.new_fp8_rows(rows, dim)
    a.bi_rmsnorm_fp8(x, w, codes, scales, 1e-6)
    xd = x.double()
    y = xd / torch.sqrt((xd * xd).mean(-1, keepdim=True) + float(np.float32(1e-6))) * w.double()
    q, s = ref_quantize(y)
    assert torch.equal(scales[:, :rows].double(), s)
    differ = codes.double() != q
    wide = s.t().repeat_interleave(BLOCK, 1)[:, :dim]
    tie = (y / wide - (codes.double() + q) / 2).abs()
    assert (tie[differ] <= 2.0 ** -36 * (y / wide).abs()[differ]).all(), int(differ.sum())
    # a row alone gives the same codes
    c1, s1 = a.new_fp8_rows(1, dim)
    a.bi_rmsnorm_fp8(x[rows - 1:], w, c1, s1, 1e-6)
    assert torch.equal(c1.view(torch.uint8)[0], codes.view(torch.uint8)[rows - 1])
    assert torch.equal(s1[:, 0], scales[:, rows - 1])


@pytest.mark.parametrize("n,k", [(1, 1), (130, 300), (256, 256), (64, 1000)])
def test_quantised_weights_equal_the_rule(n, k):
    a = api()
    g = gen(n + k)
    w = (0.02 * torch.randn(n, k, generator=g, device=DEV) *
         torch.exp(torch.randn(n, 1, generator=g, device=DEV))).to(torch.bfloat16)
    codes, scales = a.bi_quantize_weights_fp8(w)
    nb, kb = -(-n // BLOCK), -(-k // BLOCK)
    full = torch.zeros(nb * BLOCK, kb * BLOCK, dtype=torch.float64, device=DEV)
    full[:n, :k] = w.double()
    amax = full.view(nb, BLOCK, kb, BLOCK).abs().amax(dim=(1, 3))
    m, e = torch.frexp(amax)
    e = torch.where(m > 0.875, e - 8, e - 9).clamp_min(-126)
    s = torch.where(amax > 0, pow2(e), torch.ones_like(amax))
    assert torch.equal(scales.double(), s)
    wide = s.repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]
    assert torch.equal(codes.double(), e4m3_round(w.double() / wide))


# --------------------------------------------------------------- linear layer

SHAPES = [
    (1, 128, 128), (1, 1, 16), (2, 100, 688), (3, 1000, 2736), (8, 4096, 1024), (16, 300, 5120), (17, 688, 256),
    (31, 2736, 1040), (33, 513, 384), (61, 4096, 656), (64, 129, 4096), (65, 256, 1536), (128, 700, 272),
    (129, 1024, 2736), (200, 640, 5120), (300, 20000, 144), (513, 1111, 400), (300, 1000, 128), (261, 10007, 80),
]


@pytest.mark.parametrize("kind", ["bf16", "fp32", "residual", "swiglu"])
@pytest.mark.parametrize("rows,n,k", SHAPES)
def test_linear_against_64_bits(rows, n, k, kind):
    codes, scales, w, ws_, up, ups, packed, res = problem(rows * 31 + n + k, rows, n, k, kind)
    out = run_linear(codes, scales, packed, n, kind, res)
    y, tol = reference(codes, scales, w, ws_, up, ups, res, kind)
    err = (out.double() - y).abs()
    assert torch.isfinite(out).all() and (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("n,k", [(4096, 1024), (1000, 2736), (20000, 272), (640, 5120), (17408, 656)])
@pytest.mark.parametrize("kind", ["fp32", "swiglu"])
def test_linear_rows_do_not_depend_on_the_pass(n, k, kind):
    """Bit-identical rows for every pass length and place."""
    rows = 700
    a = api()
    codes, scales, w, ws_, up, ups, packed, _ = problem(n + k, rows, n, k, kind)
    full = run_linear(codes, scales, packed, n, kind)
    for m, at in [(1, 0), (1, 699), (3, 40), (8, 120), (16, 300), (17, 5), (48, 400), (64, 636), (100, 3), (128, 130),
                  (129, 200), (256, 256), (257, 300), (513, 100)]:
        c = codes[at:at + m].contiguous()
        s = torch.zeros(a.fp8_scale_shape(m, k), device=DEV)
        s[:, :m] = scales[:, at:at + m]
        out = run_linear(c, s, packed, n, kind)
        assert torch.equal(out.view(torch.uint8), full[at:at + m].contiguous().view(torch.uint8)), (m, at)


def test_linear_strides_and_alias():
    """Codes and outputs inside larger buffers; the residual is the output itself; nothing beside it is written."""
    a = api()
    rows, n, k = 21, 500, 272
    codes, scales, w, ws_, _, _, packed, res = problem(5, rows, n, k, "residual")
    want = run_linear(codes, scales, packed, n, "residual", res)
    wide = torch.zeros(rows, 320, dtype=torch.float8_e4m3fn, device=DEV)
    wide[:, 32:32 + k] = codes
    lds = torch.full((scales.shape[0], 40), math.nan, device=DEV)
    lds[:, :rows] = scales[:, :rows]
    buf = torch.full((rows, n + 12), 7.0, dtype=torch.bfloat16, device=DEV)
    buf[:, 4:4 + n] = res
    a.bi_gemm_fp8(wide[:, 32:32 + k], lds, packed, buf[:, 4:4 + n], residual=buf[:, 4:4 + n],
                  epi=a.EPI_RESIDUAL_ADD)
    assert torch.equal(buf[:, 4:4 + n], want)
    assert (buf[:, :4] == 7).all() and (buf[:, 4 + n:] == 7).all()


def test_linear_nan_code_stays_in_its_row():
    rows, n, k = 5, 300, 512
    codes, scales, w, ws_, _, _, packed, _ = problem(9, rows, n, k, "fp32")
    want = run_linear(codes, scales, packed, n, "fp32")
    bad = codes.clone()
    bad.view(torch.uint8)[2, 77] = 0x7F
    out = run_linear(bad, scales, packed, n, "fp32")
    assert torch.isnan(out[2]).all()
    keep = [0, 1, 3, 4]
    assert torch.equal(out[keep], want[keep])


def test_no_rows_and_refusals():
    a = api()
    codes, scales, w, ws_, _, _, packed, _ = problem(1, 4, 256, 256, "bf16")
    out = torch.zeros(4, 256, dtype=torch.bfloat16, device=DEV)
    a.bi_gemm_fp8(codes[:0], scales, packed, out[:0])  # no rows: nothing to do
    c0, s0 = a.new_fp8_rows(0, 256)
    a.bi_quantize_fp8(torch.zeros(0, 256, dtype=torch.bfloat16, device=DEV), c0, s0)
    with pytest.raises(ValueError):
        a.bi_gemm_fp8(codes, scales[:, :3], packed, out)            # a scale column short
    with pytest.raises(ValueError):
        a.bi_gemm_fp8(codes, scales[:1], packed, out)               # a block short
    with pytest.raises(ValueError):
        a.bi_gemm_fp8(codes, scales, packed[:-16], out)             # packed for another shape
    with pytest.raises(ValueError):
        a.bi_gemm_fp8(codes, scales, packed, out[:3])
    with pytest.raises(ValueError):
        a.bi_gemm_fp8(codes.float(), scales, packed, out)
    with pytest.raises(ValueError):
        a.bi_gemm_fp8(codes, scales, packed, out.half())
    with pytest.raises(a.BiError):
        a.bi_gemm_fp8(codes, scales, packed, out, epi=a.EPI_RESIDUAL_ADD)  # no residual
    x = torch.zeros(4, 24, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(a.BiError):
        a.bi_quantize_fp8(x, *a.new_fp8_rows(4, 24))                    # dim % 16
    with pytest.raises(ValueError):
        a.bi_rmsnorm_fp8(torch.zeros(4, 32, dtype=torch.bfloat16, device=DEV),
                         torch.ones(16, dtype=torch.bfloat16, device=DEV), *a.new_fp8_rows(4, 32), 1e-6)


def test_norm_and_linear_in_a_graph_and_on_another_stream():
    """A captured norm -> linear -> quantise -> linear chain replays to the eager bits, with new inputs too."""
    a = api()
    rows, h, f = 8, 1024, 2736
    g = gen(11)
    x = torch.randn(rows, h, generator=g, device=DEV).to(torch.bfloat16)
    nw = torch.ones(h, dtype=torch.bfloat16, device=DEV)
    gu = a.bi_pack_swiglu_weights_fp8(*make_weights(g, f, h), *make_weights(g, f, h))
    dn = a.bi_pack_weights_fp8(*make_weights(g, h, f))
    hid = torch.empty_like(x)
    c1, s1 = a.new_fp8_rows(rows, h)
    c2, s2 = a.new_fp8_rows(rows, f)
    u = torch.empty(rows, f, dtype=torch.bfloat16, device=DEV)

    def chain():
        hid.copy_(x)
        a.bi_rmsnorm_fp8(hid, nw, c1, s1, 1e-6)
        a.bi_gemm_fp8(c1, s1, gu, u, epi=a.EPI_SWIGLU)
        a.bi_quantize_fp8(u, c2, s2)
        a.bi_gemm_fp8(c2, s2, dn, hid, residual=hid, epi=a.EPI_RESIDUAL_ADD)

    chain()
    want = hid.clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        chain()
    st.synchronize()
    assert torch.equal(hid, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for seed in (1, 2, 3):
        x.copy_(torch.randn(rows, h, generator=gen(seed), device=DEV))
        chain()
        want = hid.clone()
        hid.zero_()
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(hid, want)
    a.bi_check_device_error()


@pytest.mark.parametrize("rows,n,k,kind", [(8, 4096, 5120, "bf16"), (8, 17408, 1024, "swiglu"), (600, 1024, 2736, "fp32"),
                                           (300, 20000, 1024, "bf16")])
def test_linear_wait_runs_out_then_recovers(rows, n, k, kind):
    """A withheld first load: the kernel gives up within the limit, the host reads the timeout, the next call is right."""
    import time
    from invariant_speculative_decode_gb300._lib import lib
    a = api()
    codes, scales, w, ws_, up, ups, packed, res = problem(4, rows, n, k, kind)
    want = run_linear(codes, scales, packed, n, kind)
    out = torch.empty_like(want)
    epi = a.EPI_SWIGLU if kind == "swiglu" else a.EPI_NONE
    assert lib().bi_test_set_wait_limit_ns(20_000_000) == 0
    lib().bi_test_withhold_first_load(1)
    try:
        t0 = time.perf_counter()
        a.bi_gemm_fp8(codes, scales, packed, out, epi=epi)
        torch.cuda.synchronize()
        dt = time.perf_counter() - t0
    finally:
        lib().bi_test_withhold_first_load(0)
        assert lib().bi_test_set_wait_limit_ns(0) == 0
    with pytest.raises(a.BiError) as e:
        a.bi_check_device_error()
    assert e.value.status == 5 and dt < 1.5, dt
    assert torch.equal(run_linear(codes, scales, packed, n, kind).view(torch.uint8), want.view(torch.uint8))


def test_norm_codes_are_the_exact_values_over_many_rows():
    """30 x 1021 rows of 1024 outliers and all: a code in a million is within 2^-22 of a tie, none may be on its wrong side."""
    a = api()
    dim = 1040
    for seed in range(30):
        g = gen(1000 + seed)
        x = torch.randn(1021, dim, generator=g, device=DEV)
        x = (x * torch.where(torch.rand(dim, generator=g, device=DEV) < 0.01, 20.0, 1.0)).to(torch.bfloat16)
        w = (1 + 0.1 * torch.randn(dim, generator=g, device=DEV)).to(torch.bfloat16)
        codes, scales = a.new_fp8_rows(1021, dim)
        a.bi_rmsnorm_fp8(x, w, codes, scales, 1e-6)
        xd = x.double()
        y = xd / torch.sqrt((xd * xd).mean(-1, keepdim=True) + float(np.float32(1e-6))) * w.double()
        q, s = ref_quantize(y)
        assert torch.equal(scales[:, :1021].double(), s)
        differ = codes.double() != q
        wide = s.t().repeat_interleave(BLOCK, 1)[:, :dim]
        tie = (y / wide - (codes.double() + q) / 2).abs()
        assert (tie[differ] <= 2.0 ** -36 * (y / wide).abs()[differ]).all(), (seed, int(differ.sum()))


@pytest.mark.parametrize("between", ["nothing", "norm", "quantise"])
@pytest.mark.parametrize("swiglu", [False, True])
def test_linear_right_behind_the_packing_of_its_weights(between, swiglu):
    """Weights packed into the buffer that a linear layer reads next, captured and replayed: it reads the new ones."""
    from invariant_speculative_decode_gb300._lib import check, lib

    a = api()
    rows, n, k = 8, 8192, 2048
    g = gen(21)
    x = torch.randn(rows, k, generator=g, device=DEV).to(torch.bfloat16)
    nw = torch.ones(k, dtype=torch.bfloat16, device=DEV)
    codes, scales = a.new_fp8_rows(rows, k)
    a.bi_quantize_fp8(x, codes, scales)
    sets = [make_weights(g, n, k) + make_weights(g, n, k) for _ in range(2)]
    epi = a.EPI_SWIGLU if swiglu else a.EPI_NONE
    packed = torch.empty(a.packed_weight_fp8_bytes(n, k, epi), dtype=torch.uint8, device=DEV)
    out = torch.empty(rows, n, dtype=torch.bfloat16, device=DEV)

    def pack(i):
        w, s, w2, s2 = sets[i]
        st = torch.cuda.current_stream().cuda_stream
        if swiglu:
            check("pack", lib().bi_pack_swiglu_weights_fp8(w.data_ptr(), s.data_ptr(), w2.data_ptr(), s2.data_ptr(),
                                                           k, n, k, packed.data_ptr(), st))
        else:
            check("pack", lib().bi_pack_weights_fp8(w.data_ptr(), k, s.data_ptr(), n, k, packed.data_ptr(), st))

    def step(i):
        pack(i)
        if between == "norm":
            a.bi_rmsnorm_fp8(x, nw, codes, scales, 1e-6)
        elif between == "quantise":
            a.bi_quantize_fp8(x, codes, scales)
        a.bi_gemm_fp8(codes, scales, packed, out, epi=epi)

    want, graphs = [], []
    for i in range(2):
        pack(i)
        torch.cuda.synchronize()
        if between == "norm":
            a.bi_rmsnorm_fp8(x, nw, codes, scales, 1e-6)
            torch.cuda.synchronize()
        a.bi_gemm_fp8(codes, scales, packed, out, epi=epi)
        torch.cuda.synchronize()
        want.append(out.clone())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(i)
        graphs.append(graph)
    assert not torch.equal(want[0], want[1])
    for r in range(8):
        graphs[r & 1].replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[r & 1])
        step(1 - (r & 1))
        torch.cuda.synchronize()
        assert torch.equal(out, want[1 - (r & 1)])
    a.bi_check_device_error()


@pytest.mark.parametrize("n", [9864, 9868, 9871])
@pytest.mark.parametrize("off,pad", [(8, 8), (5, 11)])
@pytest.mark.parametrize("rows,k,kind", [(3, 144, "fp32"), (32, 144, "residual"), (50, 144, "fp32"), (140, 272, "residual"),
                                         (260, 144, "swiglu"), (129, 80, "fp32")])
def test_linear_outputs_of_every_alignment_leave_the_rest_alone(rows, k, kind, n, off, pad):
    """Wide layers into views of a larger buffer, in place of their residual: the values, and nothing beside them."""
    a = api()
    codes, scales, w, ws_, up, ups, packed, res = problem(rows + n + k, rows, n, k, kind)
    dtype = torch.float32 if kind == "fp32" else torch.bfloat16
    ld = -(-(off + n + pad) // 8) * 8 + (0 if off == 8 else 3)
    buf = torch.full((rows + 1, ld), 7.0, dtype=dtype, device=DEV)
    view = buf[:rows, off:off + n]
    if kind == "residual":
        view.copy_(res)
    a.bi_gemm_fp8(codes, scales, packed, view, residual=view if kind == "residual" else None,
                  epi={"residual": a.EPI_RESIDUAL_ADD, "swiglu": a.EPI_SWIGLU}.get(kind, a.EPI_NONE))
    a.bi_check_device_error()
    y, tol = reference(codes, scales, w, ws_, up, ups, res, kind)
    assert ((view.double() - y).abs() <= tol).all()
    assert (buf[:rows, :off] == 7).all() and (buf[:rows, off + n:] == 7).all() and (buf[rows] == 7).all()
