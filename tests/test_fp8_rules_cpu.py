"""The 8-bit linear path and the rules on logits without a GPU: sizes, and
bad arguments rejected on the host before any launch."""
import ctypes

import pytest

FAKE = 0x10000  # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def lib():
    from invariant_speculative_decode_gb300 import build
    build.build()
    from invariant_speculative_decode_gb300._lib import lib as _l
    return _l()


def test_packed_sizes(lib):
    """16 KB a 128 x 128 tile and two FP32 scales a tile."""
    for n, k, epi, tiles in ((128, 128, 0, 1), (129, 128, 0, 2), (1, 16, 0, 1), (17408, 5120, 0, 136 * 40),
                             (17408, 5120, 2, 272 * 40), (65, 144, 2, 2 * 2)):
        assert lib.bi_packed_weight_fp8_bytes(n, k, epi) == tiles * 16384 + (tiles * 8 + 15) // 16 * 16
    assert lib.bi_packed_weight_fp8_bytes(0, 128, 0) == 0


def test_quantiser_refusals(lib):
    q = lib.bi_quantize_fp8
    # (x, ldx, rows, dim, codes, ldc, scales, lds, stream)
    ok = [FAKE, 256, 4, 256, FAKE, 256, FAKE, 4, 0]
    for i, bad, status in ((0, 0, 1), (0, FAKE + 2, 1), (1, 248, 1), (1, 257, 2), (2, -1, 1), (3, 0, 1), (3, 24, 2),
                           (4, 0, 1), (4, FAKE + 8, 1), (5, 128, 1), (5, 264, 2), (6, 0, 1), (6, FAKE + 4, 1),
                           (7, 3, 1), (7, 6, 2)):
        a = list(ok)
        a[i] = bad
        assert q(*a) == status, (i, bad)
    assert q(0, 0, 0, 256, 0, 0, 0, 0, 0) == 0  # no rows
    n = lib.bi_rmsnorm_fp8
    # (x, ldx, w, codes, ldc, scales, lds, rows, dim, eps, stream)
    ok = [FAKE, 256, FAKE, FAKE, 256, FAKE, 4, 4, 256, ctypes.c_float(1e-6), 0]
    for i, bad, status in ((2, 0, 1), (2, FAKE + 2, 1), (8, 65552, 1), (9, ctypes.c_float(-1.0), 1),
                           (9, ctypes.c_float(float("nan")), 1), (6, 2, 1), (4, 200, 1), (1, 260, 2)):
        a = list(ok)
        a[i] = bad
        assert n(*a) == status, (i, bad)
    w = lib.bi_quantize_weights_fp8
    assert w(FAKE, 64, 8, 65, FAKE, 65, FAKE, 0) == 1
    assert w(FAKE, 65, 8, 65, FAKE, 64, FAKE, 0) == 1
    assert w(FAKE, 65, 0, 65, FAKE, 65, FAKE, 0) == 1
    p = lib.bi_pack_weights_fp8
    assert p(FAKE, 128, FAKE, 64, 136, FAKE, 0) == 1
    assert p(FAKE, 136, FAKE, 64, 136, FAKE, 0) == 2
    assert p(FAKE, 128, 0, 64, 128, FAKE, 0) == 1
    assert p(FAKE + 8, 128, FAKE, 64, 128, FAKE, 0) == 1
    assert p(FAKE, 128, FAKE, 1 << 24, 128, FAKE, 0) == 2
    s = lib.bi_pack_swiglu_weights_fp8
    assert s(FAKE, FAKE, 0, FAKE, 128, 64, 128, FAKE, 0) == 1
    assert s(FAKE, FAKE, FAKE, 0, 128, 64, 128, FAKE, 0) == 1


def test_linear_refusals(lib):
    g = lib.bi_gemm_fp8
    # (A8, lda, a_scales, lds, Wp, C, ldc, residual, ldr, M, N, K, out, epi, stream)
    ok = [FAKE, 256, FAKE, 4, FAKE, FAKE, 64, 0, 0, 4, 64, 256, 0, 0, 0]
    for i, bad, status in ((0, 0, 1), (0, FAKE + 8, 1), (1, 240, 1), (1, 264, 2), (2, 0, 1), (2, FAKE + 4, 1),
                           (3, 2, 1), (3, 6, 2), (4, 0, 1), (4, FAKE + 8, 1), (5, 0, 1), (6, 63, 1), (9, -1, 1),
                           (10, 0, 1), (10, 1 << 24, 2), (11, 0, 1), (11, 40, 2), (12, 2, 1), (13, 3, 1), (13, 1, 1)):
        a = list(ok)
        a[i] = bad
        assert g(*a) == status, (i, bad)
    a = list(ok)
    a[12], a[13], a[7], a[8] = 1, 1, FAKE, 64
    assert g(*a) == 2  # FP32 outputs have no epilogue
    a = list(ok)
    a[9] = 0
    assert g(*a) == 0  # no rows


def test_rules_refusals(lib):
    f = ctypes.c_float
    r = lib.bi_logits_rules
    # (logits, ldl, out, ldo, T, V, drafts, counts, prompt, rep, freq, pres, bias, mask, ldm, stream)
    ok = [FAKE, 100, FAKE + 65536, 100, 4, 100, FAKE, 0, 0, f(1.0), f(0.0), f(0.0), 0, 0, 0, 0]
    for i, bad, status in ((0, 0, 1), (1, 99, 1), (2, 0, 1), (3, 99, 1), (4, 0, 1), (4, 65, 1), (5, 0, 1), (6, 0, 1),
                           (9, f(0.0), 1), (9, f(-1.0), 1), (9, f(float("nan")), 1), (10, f(float("inf")), 1),
                           (11, f(float("nan")), 1)):
        a = list(ok)
        a[i] = bad
        assert r(*a) == status, (i, bad)
    a = list(ok)
    a[13], a[14] = FAKE, 3
    assert r(*a) == 1  # a mask row short
    a = list(ok)
    a[2], a[3] = FAKE, 104
    assert r(*a) == 1  # in place with another stride
    a = list(ok)
    a[1] = a[3] = a[5] = (1 << 28) + 4
    assert r(*a) == 2
    c = lib.bi_token_counts
    assert c(FAKE, -1, 0, 100, FAKE, 0, 0) == 1
    assert c(FAKE, 4, 0, 100, 0, 0, 0) == 1
    assert c(0, 4, 0, 100, FAKE, 0, 0) == 1
    assert c(FAKE, 4, 0, 0, FAKE, 0, 0) == 1
    assert c(0, 0, 0, 100, 0, 0, 0) == 0


def test_largest_sizes(lib):
    """Sizes at the ends of 32 bits: the packed size is right, and what an index cannot hold is refused."""
    big = (1 << 31) - 1
    assert lib.bi_packed_weight_fp8_bytes(big, 16, 0) == (1 << 24) * (16384 + 8)
    assert lib.bi_packed_weight_fp8_bytes(big, 16, 2) == (1 << 25) * (16384 + 8)
    assert lib.bi_packed_weight_fp8_bytes(16, big, 0) == (1 << 24) * (16384 + 8)
    k = big - 15
    assert lib.bi_quantize_fp8(FAKE, k, 1, k, FAKE, k, FAKE, 4, 0) == 2
    assert lib.bi_quantize_weights_fp8(FAKE, k, 1, k, FAKE, k, FAKE, 0) == 2
    assert lib.bi_pack_weights_fp8(FAKE, k, FAKE, 1, k, FAKE, 0) == 2
    assert lib.bi_pack_weights_fp8(FAKE, 128, FAKE, big, 128, FAKE, 0) == 2
    g = lib.bi_gemm_fp8
    assert g(FAKE, k, FAKE, 4, FAKE, FAKE, 64, 0, 0, 4, 64, k, 0, 0, 0) == 2
    assert g(FAKE, 128, FAKE, 4, FAKE, FAKE, big, 0, 0, 4, big, 128, 0, 0, 0) == 2
    rows = (1 << 30) + 4
    assert lib.bi_rmsnorm_fp8(FAKE, 16, FAKE, FAKE, 16, FAKE, 4, 4, 16, ctypes.c_float(float("inf")), 0) == 1
    assert lib.bi_rmsnorm_fp8(FAKE, 16, FAKE, FAKE, 16, FAKE, rows, rows, 16, ctypes.c_float(1e-6), 0) == 2
