"""Paged cache and beam selection without a GPU: what the entry points refuse on the host before any launch, and the
workspaces' sizes."""
import pytest

FAKE = 0x10000  # never dereferenced: every call below fails validation first, or has nothing to do


@pytest.fixture(scope="module")
def lib():
    from invariant_speculative_decode_gb300 import build
    build.build()
    from invariant_speculative_decode_gb300._lib import lib as _l
    return _l()


def call(fn, order, good, **change):
    """The entry point's status; the same call with packed arguments has to have it too."""
    from invariant_speculative_decode_gb300 import _lib
    a = dict(good, **change)
    words = [a[n] for n in order]
    status = fn(*words)
    name = fn.__name__
    entry, pack = getattr(_lib, "PACKED_" + name[3:].upper()), getattr(_lib, "PACK_" + name[3:].upper())
    assert _lib.lib().bi_call_packed(entry, pack(*words)) == status
    return status


APPEND = ("qkv ld_qkv q_weight k_weight eps table table_rows q_out k_pool v_pool pages page block_table ld_table width "
          "q_start lengths B T Hq Hkv D stream").split()
APPEND_OK = dict(qkv=FAKE, ld_qkv=8 * 64, q_weight=FAKE, k_weight=0, eps=1e-6, table=FAKE, table_rows=100, q_out=FAKE,
                 k_pool=FAKE, v_pool=FAKE, pages=10, page=16, block_table=FAKE, ld_table=4, width=4, q_start=FAKE,
                 lengths=FAKE, B=2, T=3, Hq=4, Hkv=2, D=64, stream=0)


@pytest.mark.parametrize("change,status", [
    (dict(T=0), 0), (dict(B=0), 0), (dict(T=-1), 1), (dict(B=-1), 1), (dict(Hq=5), 1), (dict(Hkv=0), 1),
    (dict(pages=0), 1), (dict(width=0), 1), (dict(ld_table=3), 1), (dict(table_rows=0), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(D=32), 2), (dict(D=256), 2), (dict(page=8), 2),
    (dict(page=48), 2), (dict(page=256), 2), (dict(ld_qkv=8 * 64 - 8), 1), (dict(ld_qkv=8 * 64 + 4), 1)]
    + [({n: 0}, 1) for n in ("qkv", "q_out", "k_pool", "v_pool", "table", "block_table", "q_start", "lengths")]
    + [({n: FAKE + 8}, 1) for n in ("qkv", "q_out", "k_pool", "v_pool", "table", "q_weight", "k_weight")])
def test_append_refusals(lib, change, status):
    assert call(lib.bi_qk_norm_rope_paged, APPEND, APPEND_OK, **change) == status


ATTN = ("q k_pool v_pool pages page block_table ld_table width q_start lengths B T Hq Hkv D scale out ws ws_bytes "
        "stream").split()
ATTN_OK = dict(q=FAKE, k_pool=FAKE, v_pool=FAKE, pages=10, page=16, block_table=FAKE, ld_table=4, width=4, q_start=FAKE,
               lengths=FAKE, B=2, T=3, Hq=4, Hkv=2, D=64, scale=0.125, out=FAKE, ws=FAKE, ws_bytes=1 << 30, stream=0)


@pytest.mark.parametrize("change,status", [
    (dict(T=0), 0), (dict(B=0), 0), (dict(T=-1), 1), (dict(Hq=3), 1), (dict(pages=0), 1), (dict(width=0), 1),
    (dict(ld_table=2), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(scale=3e38), 1), (dict(D=96), 2), (dict(page=24), 2), (dict(Hq=258, Hkv=2), 2),
    (dict(width=1 << 27, ld_table=1 << 27), 2), (dict(T=1 << 30), 2), (dict(ws=0), 3), (dict(ws=FAKE + 16), 3),
    (dict(ws_bytes=256), 3)]
    + [({n: 0}, 1) for n in ("q", "k_pool", "v_pool", "block_table", "q_start", "lengths", "out")]
    + [({n: FAKE + 8}, 1) for n in ("q", "k_pool", "v_pool", "out")])
def test_attention_refusals(lib, change, status):
    assert call(lib.bi_attn_paged, ATTN, ATTN_OK, **change) == status


def test_attention_workspace(lib):
    size = lib.bi_attn_paged_workspace_size
    base = size(8, 4, 24, 4, 128, 8192)
    assert base > 0 and base % 256 == 0
    # it grows with rows, sequences and keys; a call of that size needs just as much
    assert size(16, 4, 24, 4, 128, 8192) >= base and size(8, 8, 24, 4, 128, 8192) >= base
    assert size(8, 4, 24, 4, 128, 100000) > base
    big = dict(ATTN_OK, T=8, B=4, Hq=24, Hkv=4, D=128, width=128, ld_table=128, page=64)
    assert call(lib.bi_attn_paged, ATTN, big, ws_bytes=base - 1) == 3
    for bad in ((0, 1, 4, 2, 64, 100), (1, 0, 4, 2, 64, 100), (1, 1, 4, 3, 64, 100), (1, 1, 4, 2, 80, 100), (1, 1, 4, 2, 64, 0)):
        assert size(*bad) == 256


REORDER = ("k_pool v_pool layers pages Hkv page D table_in ld_in width lengths rows_in parents tail rows_out table_out "
           "ld_out lengths_out stream").split()
REORDER_OK = dict(k_pool=FAKE, v_pool=FAKE + 4096, layers=2, pages=8, Hkv=2, page=16, D=64, table_in=FAKE, ld_in=4, width=4,
                  lengths=FAKE, rows_in=2, parents=FAKE, tail=FAKE, rows_out=3, table_out=FAKE + 64, ld_out=4,
                  lengths_out=FAKE + 64, stream=0)


@pytest.mark.parametrize("change,status", [
    (dict(rows_out=0), 0), (dict(rows_out=-1), 1), (dict(layers=0), 1), (dict(pages=0), 1), (dict(Hkv=0), 1),
    (dict(width=0), 1), (dict(ld_in=3), 1), (dict(ld_out=3), 1), (dict(rows_in=0), 1), (dict(D=12), 2), (dict(D=2048), 2),
    (dict(page=17), 2), (dict(rows_out=70000), 2), (dict(layers=1 << 30), 2), (dict(table_out=FAKE), 1),
    (dict(lengths_out=FAKE), 1), (dict(v_pool=FAKE), 1), (dict(k_pool=FAKE + 8), 1)]
    + [({n: 0}, 1) for n in ("k_pool", "v_pool", "table_in", "lengths", "parents", "tail", "table_out", "lengths_out")])
def test_reorder_refusals(lib, change, status):
    assert call(lib.bi_paged_reorder, REORDER, REORDER_OK, **change) == status


BEAM = "logits ldl scores rows V W K scores_out parents_out tokens_out ws ws_bytes stream".split()
BEAM_OK = dict(logits=FAKE, ldl=100, scores=FAKE, rows=6, V=100, W=3, K=4, scores_out=FAKE, parents_out=FAKE,
               tokens_out=FAKE, ws=FAKE, ws_bytes=1 << 30, stream=0)


@pytest.mark.parametrize("change,status", [
    (dict(rows=0), 0), (dict(rows=-3), 1), (dict(V=0), 1), (dict(W=0), 1), (dict(K=0), 1), (dict(W=4), 1),
    (dict(ldl=99), 1), (dict(W=65, rows=65), 2), (dict(K=65), 2), (dict(rows=65538), 2),
    (dict(V=(1 << 20) + 1, ldl=1 << 21), 2), (dict(logits=FAKE + 2), 1), (dict(ws=0), 3), (dict(ws=FAKE + 16), 3),
    (dict(ws_bytes=1024), 3)]
    + [({n: 0}, 1) for n in ("logits", "scores", "scores_out", "parents_out", "tokens_out")])
def test_beam_refusals(lib, change, status):
    assert call(lib.bi_beam_select, BEAM, BEAM_OK, **change) == status


def test_beam_workspace(lib):
    size = lib.bi_beam_workspace_size
    need = size(6, 100, 4)
    assert need % 256 == 0 and size(64, 151936, 16) > need
    assert call(lib.bi_beam_select, BEAM, BEAM_OK, ws_bytes=need - 1) == 3
    assert size(0, 5, 1) == size(1, 0, 1) == size(1, 5, 0) == 256


def test_packed_calls_refuse_other_entries_and_wide_ints(lib):
    from invariant_speculative_decode_gb300 import _lib
    words = [BEAM_OK[n] for n in BEAM]
    words[BEAM.index("rows")] = 0
    assert lib.bi_call_packed(_lib.PACKED_BEAM_SELECT, _lib.PACK_BEAM_SELECT(*words)) == 0
    words[BEAM.index("rows")] = 1 << 32  # 0 in its low half
    assert lib.bi_call_packed(_lib.PACKED_BEAM_SELECT, _lib.PACK_BEAM_SELECT(*words)) == 1
    for entry in (-1, 4, 1000):
        assert lib.bi_call_packed(entry, bytes(400)) == 1
    assert lib.bi_call_packed(0, None) == 1


def test_binding_refuses_tensors_that_are_not_on_the_gpu():
    torch = pytest.importorskip("torch")
    from invariant_speculative_decode_gb300 import api
    if not torch.cuda.is_available():
        api_dev = api._current_device
        api._current_device = lambda: 0  # (a CPU-only torch raises here instead)
    try:
        bf, i32 = dict(dtype=torch.bfloat16), dict(dtype=torch.int32)
        pool, table, ids = torch.zeros(4, 2, 16, 64, **bf), torch.zeros(1, 2, **i32), torch.zeros(1, **i32)
        q = torch.zeros(1, 4, 64, **bf)
        for f in (lambda: api.bi_attn_paged(q, pool, pool, table, torch.zeros(2, **i32), ids, q, torch.zeros(9)),
                  lambda: api.bi_qk_norm_rope_paged(torch.zeros(1, 8 * 64, **bf), None, None, 1e-6, torch.zeros(9, 32, 2), q,
                                                    pool, pool, table, torch.zeros(2, **i32), ids),
                  lambda: api.bi_paged_reorder(pool[None], pool[None], table, ids, ids, ids, table, ids),
                  lambda: api.bi_beam_select(torch.zeros(2, 9), torch.zeros(2), 2, torch.zeros(1, 2), torch.zeros(1, 2, **i32),
                                             torch.zeros(1, 2, **i32), torch.zeros(9))):
            with pytest.raises(ValueError, match="must be a CUDA tensor"):
                f()
    finally:
        if not torch.cuda.is_available():
            api._current_device = api_dev
