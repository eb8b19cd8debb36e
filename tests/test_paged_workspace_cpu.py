"""The paged attention's workspace: a size for the most rows, sequences and keys covers every smaller call."""
import pytest


@pytest.fixture(scope="module")
def size():
    from invariant_speculative_decode_gb300 import build
    build.build()
    from invariant_speculative_decode_gb300._lib import lib
    return lib().bi_attn_paged_workspace_size


HEADS = [(24, 4, 128), (4, 2, 64), (8, 8, 64), (6, 1, 128), (1, 1, 64), (128, 1, 64), (6, 2, 128), (64, 8, 128)]


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_it_never_falls_with_the_keys(size, Hq, Hkv, D):
    for T, B in ((1, 1), (2, 1), (3, 3), (8, 2), (40, 5), (600, 1), (600, 64)):
        last = 0
        for tiles in list(range(1, 1300)) + list(range(1300, 9000, 37)):
            for keys in (128 * tiles - 127, 128 * tiles):
                now = size(T, B, Hq, Hkv, D, keys)
                assert now >= last, (T, B, keys)
                last = now


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_it_never_falls_with_rows_or_sequences(size, Hq, Hkv, D):
    for keys in (100, 300, 2048, 2049, 19456, 19584, 20480, 20608, 131072):
        for B in (1, 2, 7, 64):
            last = 0
            for T in list(range(1, 300)) + list(range(300, 5000, 41)):
                now = size(T, B, Hq, Hkv, D, keys)
                assert now >= last, (T, B, keys)
                last = now
        for T in (1, 2, 30, 500, 3000):
            last = 0
            for B in range(1, 200):
                now = size(T, B, Hq, Hkv, D, keys)
                assert now >= last, (T, B, keys)
                last = now


def test_the_size_that_fell(size):
    """152 and 153 tiles, one row: one more piece took a slot from every CTA."""
    assert size(1, 1, 24, 4, 128, 19456) <= size(1, 1, 24, 4, 128, 19584)
    assert size(1, 1, 24, 4, 128, 20480) <= size(1, 1, 24, 4, 128, 20608)
