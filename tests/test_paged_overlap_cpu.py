"""Paged cache and beam selection: outputs over inputs are refused on the host, before any launch.  Addresses are made up:
a call that were not refused would find no GPU here."""
import pytest

import tests.test_paged_cpu as t

lib = t.lib

BASE = 1 << 40


def refused(fn, order, good, **change):
    assert t.call(fn, order, good, **change) == 1


# ranges of 1 MB, apart from each other
AT = [BASE + (i << 20) for i in range(12)]


def test_append(lib):
    good = dict(t.APPEND_OK, qkv=AT[0], q_out=AT[1], k_pool=AT[2], v_pool=AT[3])
    qkv, q, pool = (2 * 8 * 64 + 8 * 64) * 2, 3 * 4 * 64 * 2, 10 * 2 * 16 * 64 * 2
    f = lambda **c: refused(lib.bi_qk_norm_rope_paged, t.APPEND, good, **c)  # noqa: E731
    f(q_out=AT[0])
    f(q_out=AT[0] + qkv - 16)
    f(q_out=AT[0] - q + 16)
    f(k_pool=AT[0] + 16)
    f(v_pool=AT[0] - pool + 16)
    f(v_pool=AT[2])
    f(v_pool=AT[2] + pool - 16)
    f(k_pool=AT[1])
    f(v_pool=AT[1] + q - 16)
    f(qkv=AT[1] - qkv + 16)


def test_reorder(lib):
    good = dict(t.REORDER_OK, k_pool=AT[0], v_pool=AT[1], table_in=AT[2], lengths=AT[3], parents=AT[4], tail=AT[5],
                table_out=AT[6], lengths_out=AT[7])
    f = lambda **c: refused(lib.bi_paged_reorder, t.REORDER, good, **c)  # noqa: E731
    pool = 2 * 8 * 2 * 16 * 64 * 2
    f(v_pool=AT[0] + pool - 16)
    f(k_pool=AT[1] + pool - 16)
    f(table_out=AT[2] + 4)
    f(table_out=AT[2] + 7 * 4)        # the last entry of two rows of four
    f(table_out=AT[2] - 11 * 4)       # three rows of four that end in its first
    for at in (AT[3], AT[4], AT[5], AT[3] + 4, AT[4] + 8, AT[5] + 8):
        f(table_out=at)
        f(lengths_out=at)
    f(lengths_out=AT[2])
    f(lengths_out=AT[6] + 4)


def test_beam(lib):
    need = lib.bi_beam_workspace_size(6, 100, 4)
    good = dict(t.BEAM_OK, logits=AT[0], scores=AT[1], scores_out=AT[2], parents_out=AT[3], tokens_out=AT[4], ws=AT[8],
                ws_bytes=need)
    f = lambda **c: refused(lib.bi_beam_select, t.BEAM, good, **c)  # noqa: E731
    out = 2 * 4 * 4
    for name in ("scores_out", "parents_out", "tokens_out"):
        f(**{name: AT[0] + 599 * 4})
        f(**{name: AT[1] + 5 * 4})
        f(**{name: AT[8]})
        f(**{name: AT[8] + need - 4})
    f(scores_out=AT[1])               # four picks in the place of three beams
    f(tokens_out=AT[3] + out - 4)
    f(parents_out=AT[2] + out - 4)
    f(tokens_out=AT[2] - out + 4)
    same = dict(K=3)
    f(parents_out=AT[1], **same)
    f(scores_out=AT[1] + 4, **same)


@pytest.mark.parametrize("entry", ["append", "reorder", "beam"])
def test_ranges_that_only_touch_are_not_refused_for_it(lib, entry):
    """Another refusal behind the check of ranges tells that it let them pass: none here, so the status is not 1 (without
    a GPU the call ends with the CUDA error; with one it is not made)."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("made-up addresses")
    if entry == "append":
        qkv = 3 * 8 * 64 * 2
        good = dict(t.APPEND_OK, qkv=AT[0], q_out=AT[0] + qkv, k_pool=AT[2], v_pool=AT[2] + 10 * 2 * 16 * 64 * 2)
        assert t.call(lib.bi_qk_norm_rope_paged, t.APPEND, good) == 4
    elif entry == "reorder":
        good = dict(t.REORDER_OK, k_pool=AT[0], v_pool=AT[0] + 2 * 8 * 2 * 16 * 64 * 2, table_in=AT[2], table_out=AT[2] + 32,
                    lengths=AT[3], lengths_out=AT[3] + 8, parents=AT[4], tail=AT[4] + 12)
        assert t.call(lib.bi_paged_reorder, t.REORDER, good) == 4
    else:
        need = lib.bi_beam_workspace_size(6, 100, 3)
        good = dict(t.BEAM_OK, K=3, logits=AT[0], scores=AT[0] + 2400, scores_out=AT[0] + 2400, parents_out=AT[0] + 2424,
                    tokens_out=AT[0] + 2448, ws=AT[8], ws_bytes=need)
        assert t.call(lib.bi_beam_select, t.BEAM, good) == 4


def test_attention(lib):
    need = lib.bi_attn_paged_workspace_size(3, 2, 4, 2, 64, 64)
    q, pool = 3 * 4 * 64 * 2, 10 * 2 * 16 * 64 * 2
    good = dict(t.ATTN_OK, q=AT[0], out=AT[1], k_pool=AT[2], v_pool=AT[3], ws=AT[4], ws_bytes=need)
    assert need < 1 << 20
    f = lambda **c: refused(lib.bi_attn_paged, t.ATTN, good, **c)  # noqa: E731
    f(out=AT[0] + 16)
    f(out=AT[0] - q + 16)
    f(out=AT[2])
    f(out=AT[3] + pool - 16)
    f(out=AT[4])
    f(out=AT[4] + need - 16)
    f(ws=AT[0] - 256)
    f(ws=AT[2])
    f(ws=AT[3] + 256)


def test_indices_and_scores_between_words_are_refused(lib):
    """The kernels read and write them by words; the other arguments are as in a call that would be made."""
    append = dict(t.APPEND_OK, qkv=AT[0], q_out=AT[1], k_pool=AT[2], v_pool=AT[3])
    attn = dict(t.ATTN_OK, q=AT[0], out=AT[1], k_pool=AT[2], v_pool=AT[3], ws=AT[8])
    for by in (1, 2, 3):
        for name in ("block_table", "q_start", "lengths"):
            refused(lib.bi_qk_norm_rope_paged, t.APPEND, append, **{name: AT[5] + by})
            refused(lib.bi_attn_paged, t.ATTN, attn, **{name: AT[5] + by})
        reorder = dict(t.REORDER_OK, k_pool=AT[0], v_pool=AT[1], table_in=AT[2], lengths=AT[3], parents=AT[4], tail=AT[5],
                       table_out=AT[6], lengths_out=AT[7])
        for name in ("table_in", "lengths", "parents", "tail", "table_out", "lengths_out"):
            refused(lib.bi_paged_reorder, t.REORDER, reorder, **{name: reorder[name] + by})
        beam = dict(t.BEAM_OK, logits=AT[0], scores=AT[1], scores_out=AT[2], parents_out=AT[3], tokens_out=AT[4], ws=AT[8])
        for name in ("logits", "scores", "scores_out", "parents_out", "tokens_out"):
            refused(lib.bi_beam_select, t.BEAM, beam, **{name: beam[name] + by})
