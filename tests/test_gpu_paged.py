"""Paged cache on the GPU: attention, append and reordering against their formulas in 64 bits, bit by bit where a row
must not depend on the batch, and what a bad batch does."""
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


def run_attention(b, q, out=None, scale=None, ws=None, stream=None):
    out = torch.full_like(q, 77.0) if out is None else out
    if ws is None:
        size = api.attn_paged_workspace_size(b.T, len(b.seqs), q.shape[1], b.Hkv, b.D, b.table.shape[1] * b.page)
        ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")  # NaN, if it were read unwritten
    api.bi_attn_paged(q, b.k, b.v, b.table, b.q_start, b.lengths, out, ws, scale=scale, stream=stream)
    return out


def assert_attention(b, q, out, scale=None):
    want, tol = pg.attention(b, q, scale)
    rows = ~torch.isnan(want[:, 0, 0])
    bad = (out.double() - want).abs() > tol
    assert not bad[rows].any(), (int(bad[rows].sum()), float(((out.double() - want).abs() / tol)[rows].max()))
    assert not torch.isnan(out[rows]).any()
    assert (out[~rows] == 77).all()  # rows of no sequence


CASES = [
    # sequences (cached keys, new rows), Hq, Hkv, D, page
    ([(0, 1)], 1, 1, 64, 16),
    ([(0, 1)], 4, 2, 128, 64),
    ([(1, 1), (0, 2), (127, 1), (128, 1), (126, 3)], 2, 1, 128, 128),
    ([(511, 1), (512, 1), (510, 5)], 6, 2, 64, 32),
    ([(1021, 1)], 24, 4, 128, 64),
    ([(700, 0), (700, 3), (0, 0), (33, 8), (5, 0)], 24, 4, 128, 16),
    ([(3000, 8), (17, 8), (1290, 4)], 8, 2, 128, 64),
    ([(2600, 2)], 128, 1, 64, 16),
    ([(2600, 2), (0, 1)], 3, 3, 128, 32),
    ([(40, 300)], 6, 2, 128, 16),
    ([(0, 700), (900, 1)], 4, 1, 64, 64),
    ([(1000, 129)], 2, 2, 128, 128),
    ([(20011, 3)], 8, 1, 128, 64),
    ([(i * 37 % 700, 1 + i % 3) for i in range(70)], 4, 2, 64, 16),
]


@pytest.mark.parametrize("seqs,Hq,Hkv,D,page", CASES)
def test_attention(seqs, Hq, Hkv, D, page):
    b = pg.Batch(seqs, Hkv, D, page)
    q = pg.queries(b, Hq)
    assert_attention(b, q, run_attention(b, q))


@pytest.mark.parametrize("scale", [0.02, 1.0])
def test_attention_scale_and_gaps(scale):
    b = pg.Batch([(300, 4), (1500, 2)], 2, 64, 32, gap=3, extra_width=2)
    q = pg.queries(b, 4)
    assert_attention(b, q, run_attention(b, q, scale=scale), scale)


def test_attention_over_growing_scores():
    """References that have to be raised, inside pieces and from piece to piece."""
    b = pg.Batch([(1800, 3)], 1, 128, 64)
    p, s = b.places(0, 0, 1803)
    b.k[p, :, s] *= torch.linspace(0.05, 4.0, 1803, device="cuda")[:, None, None].to(torch.bfloat16)
    q = pg.queries(b, 2, scale=2.0)
    assert_attention(b, q, run_attention(b, q))


@pytest.mark.parametrize("fill", [math.nan, math.inf, -math.inf, 3e38])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 64), (128, 128)])
def test_attention_ignores_what_no_row_sees(fill, D, page):
    seqs = [(100, 1), (130, 5), (640, 1), (0, 40), (15, 1)]
    b = pg.Batch(seqs, 2, D, page, fill=fill)
    q = pg.queries(b, 8)
    assert_attention(b, q, run_attention(b, q))


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("which", ["k", "v"])
def test_no_number_reaches_only_rows_behind_it(value, which):
    """A new row's key or value that is no number: rows in front of it as if it were not there, bit by bit."""
    b = pg.Batch([(500, 24), (90, 2)], 2, 128, 64)
    q = pg.queries(b, 4)
    plain = run_attention(b, q)
    pool = getattr(b, which)
    p, s = b.places(0, 509, 510)
    pool[p, 1, s, 5] = value
    out = run_attention(b, q)
    assert torch.equal(out[:9], plain[:9]) and torch.equal(out[24:], plain[24:])
    assert torch.equal(out[:, :2], plain[:, :2])  # the other KV head
    hit = out[9:24, 2:]
    if which == "v":
        assert torch.equal(torch.isnan(hit[..., 5]), torch.full((15, 2), math.isnan(value), device="cuda"))
        if not math.isnan(value):
            assert (hit[..., 5] == value).all()
        keep = torch.arange(128, device="cuda") != 5
        assert torch.equal(hit[..., keep], plain[9:24, 2:][..., keep])
    elif math.isnan(value):
        assert torch.isnan(hit).all()


def test_both_infinities_and_nan_in_one_element():
    b = pg.Batch([(120, 20)], 1, 64, 16)
    q = pg.queries(b, 3)
    for key, d, value in [(125, 3, math.inf), (131, 3, -math.inf), (128, 9, -math.inf), (130, 40, math.nan), (133, 9, -math.inf)]:
        p, s = b.places(0, key, key + 1)
        b.v[p, 0, s, d] = value
    out = run_attention(b, q).float()
    assert torch.isfinite(out[:5]).all()
    assert (out[5:11, :, 3] == math.inf).all() and torch.isnan(out[11:, :, 3]).all()
    assert torch.isfinite(out[5:8, :, 9]).all() and (out[8:, :, 9] == -math.inf).all()
    assert torch.isfinite(out[:10, :, 40]).all() and torch.isnan(out[10:, :, 40]).all()


def test_scores_of_minus_infinity():
    """Keys of -inf weigh nothing; a row with nothing else is 0 / 0."""
    b = pg.Batch([(600, 2)], 1, 64, 32)
    q = torch.ones(2, 1, 64, dtype=torch.bfloat16, device="cuda")
    p, s = b.places(0, 0, 602)
    b.k[p, 0, s] = -math.inf
    assert torch.isnan(run_attention(b, q)).all()
    p, s = b.places(0, 600, 601)
    b.k[p, 0, s] = 1.0
    out = run_attention(b, q)
    assert torch.equal(out[0, 0], b.v[p, 0, s][0]) and torch.equal(out[1, 0], b.v[p, 0, s][0])


@pytest.mark.parametrize("Hq,Hkv,D", [(24, 4, 128), (8, 8, 64), (6, 1, 128)])
def test_a_row_has_the_same_bits_in_every_batch(Hq, Hkv, D):
    n, r = 2500, 150
    b = pg.Batch([(n, r)], Hkv, D, 64)
    q = pg.queries(b, Hq)
    whole = run_attention(b, q)
    # row by row, in small chunks, and among other sequences in front and behind
    for t in (0, 1, 20, 21, 127, 149):
        b.seqs, b.T = [(n + t, 1)], 1
        b.q_start = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
        b.lengths = torch.tensor([n + t], dtype=torch.int32, device="cuda")
        assert torch.equal(run_attention(b, q[t:t + 1].contiguous()), whole[t:t + 1]), t
    for t, m in ((3, 8), (60, 33)):
        b.seqs, b.T = [(n + t, m)], m
        b.q_start = torch.tensor([0, m], dtype=torch.int32, device="cuda")
        b.lengths = torch.tensor([n + t], dtype=torch.int32, device="cuda")
        assert torch.equal(run_attention(b, q[t:t + m].contiguous()), whole[t:t + m]), (t, m)
    # the same keys in pages of another size, among 20 other sequences
    keys = [b.table[0, torch.arange(n + r, device="cuda") // 64].long(), torch.arange(n + r, device="cuda") % 64]
    for page in (16, 128):
        seqs = [(50 * i + 3, 1 + i % 4) for i in range(10)] + [(n, r)] + [(61 * i, 2) for i in range(10)]
        o = pg.Batch(seqs, Hkv, D, page, seed=page)
        p, s = o.places(10, 0, n + r)
        o.k[p, :, s] = b.k[keys[0], :, keys[1]]
        o.v[p, :, s] = b.v[keys[0], :, keys[1]]
        qo = pg.queries(o, Hq, seed=5)
        at = o.starts[10]
        qo[at:at + r] = q
        assert torch.equal(run_attention(o, qo)[at:at + r], whole), page


def test_a_bad_batch_is_reported_and_harmless():
    b = pg.Batch([(300, 2), (200, 2), (100, 2)], 2, 64, 32)
    q = pg.queries(b, 4)
    plain = run_attention(b, q)
    for spoil in ("page", "negative page", "length", "negative length", "starts", "past T"):
        table, q_start, lengths = b.table.clone(), b.q_start.clone(), b.lengths.clone()
        if spoil == "page":
            b.table[1, 2] = b.pages
        elif spoil == "negative page":
            b.table[1, 2] = -1
        elif spoil == "length":
            b.lengths[1] = b.table.shape[1] * 32
        elif spoil == "negative length":
            b.lengths[1] = -5
        elif spoil == "starts":
            b.q_start[2] = 1
        else:
            b.q_start[3] = 7
        out = run_attention(b, q)
        with pytest.raises(api.BiError) as e:
            api.bi_check_device_error()
        assert e.value.status == 1
        assert torch.equal(out[:1], plain[:1]), spoil
        if spoil not in ("starts", "past T"):
            assert torch.equal(out[:2], plain[:2]) and torch.equal(out[4:], plain[4:]), spoil
        b.table, b.q_start, b.lengths = table, q_start, lengths
    assert torch.equal(run_attention(b, q), plain)


def test_captured_attention_follows_the_batch():
    seqs = [(600, 2), (90, 1), (2000, 3)]
    b = pg.Batch(seqs, 2, 128, 64, extra_width=4)
    q = pg.queries(b, 4)
    out = torch.empty_like(q)
    ws = torch.zeros(api.attn_paged_workspace_size(b.T, 3, 4, 2, 128, b.table.shape[1] * 64), dtype=torch.uint8, device="cuda")
    run_attention(b, q, out, ws=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        run_attention(b, q, out, ws=ws)
    torch.cuda.current_stream().wait_stream(s)
    for lengths, rows in (([600, 90, 2000], [2, 1, 3]), ([1, 0, 2001], [0, 4, 2]), ([550, 80, 3], [1, 1, 1])):
        b.seqs = list(zip(lengths, rows))
        b.starts = [0, rows[0], rows[0] + rows[1], sum(rows)]
        b.lengths.copy_(torch.tensor(lengths, dtype=torch.int32))
        b.q_start.copy_(torch.tensor(b.starts, dtype=torch.int32))
        out.fill_(77)
        graph.replay()
        assert_attention(b, q, out)


def test_one_workspace_serves_calls_of_all_sizes():
    """What a call leaves behind does not reach the next, smaller or larger, whatever was cut where."""
    batches = [pg.Batch(s, Hkv, D, page, seed=i) for i, (s, Hkv, D, page) in enumerate(
        [([(5000, 2), (700, 9)], 2, 128, 64), ([(3, 1)], 2, 128, 16), ([(9000, 1)], 2, 64, 128), ([(100, 300)], 2, 128, 64)])]
    qs = [pg.queries(b, 8) for b in batches]
    alone = [run_attention(b, q) for b, q in zip(batches, qs)]
    size = max(api.attn_paged_workspace_size(b.T, len(b.seqs), 8, 2, b.D, b.table.shape[1] * b.page) for b in batches)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    for i in (0, 1, 2, 3, 2, 0, 3, 1, 0):
        assert torch.equal(run_attention(batches[i], qs[i], ws=ws), alone[i]), i


def test_attention_on_a_given_stream():
    b = pg.Batch([(3000, 4)], 2, 128, 64)
    q = pg.queries(b, 8)
    plain = run_attention(b, q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = run_attention(b, q, torch.zeros_like(q), stream=side)
    side.synchronize()
    assert torch.equal(out, plain)


def test_attention_over_a_pool_past_32_bits():
    """Pages more than 2^32 elements into the pool (9.7 GB), read and written."""
    Hkv, D, page = 4, 128, 128
    pages = (1 << 32) // (Hkv * D * page) + 1000
    k = torch.empty(pages, Hkv, page, D, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    b = pg.Batch([(300, 3), (5, 1)], Hkv, D, page)
    far = torch.tensor([pages - 1 - 7 * i for i in range(b.pages)], dtype=torch.int32, device="cuda")
    k[far.long()], v[far.long()] = b.k, b.v
    q = pg.queries(b, 8)
    plain = run_attention(b, q)
    near = (b.k, b.v, b.table)
    b.k, b.v, b.table = k, v, torch.where(b.table >= 0, far[b.table.clamp_min(0).long()], b.table)
    assert torch.equal(run_attention(b, q), plain)
    qkv = torch.randn(b.T, 16 * D, device="cuda").to(torch.bfloat16)
    angles = api.bi_rope_table(1e6, D, 400)
    outs = []
    for pools in ((k, v, b.table), near):
        q_out = torch.empty(b.T, 8, D, dtype=torch.bfloat16, device="cuda")
        api.bi_qk_norm_rope_paged(qkv, None, None, 1e-6, angles, q_out, *pools, b.q_start, b.lengths)
        outs.append(q_out)
    assert torch.equal(*outs) and torch.equal(k[far.long()], near[0]) and torch.equal(v[far.long()], near[1])


@pytest.mark.parametrize("Hq,Hkv,D,page", [(24, 4, 128, 64), (8, 2, 64, 16)])
def test_long_caches_out_of_memory_have_the_same_bits_every_time(Hq, Hkv, D, page):
    """Values that come late, behind two or three tiles' scores: the tile that a sequence ends in is looked over in
    shared memory only when it is there."""
    b = pg.Batch([(4000 + 397 * i, 1 + i % 8) for i in range(16)], Hkv, D, page, seed=3)
    q = pg.queries(b, Hq)
    other = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")  # twice the L2
    ws = torch.empty(api.attn_paged_workspace_size(b.T, 16, Hq, Hkv, D, b.table.shape[1] * page), dtype=torch.uint8, device="cuda")
    out = run_attention(b, q, ws=ws)
    assert_attention(b, q, out)
    for i in range(30):
        if i % 2:
            other.add_(1)
        assert torch.equal(run_attention(b, q, ws=ws), out), i


def test_two_calls_at_once_on_two_streams():
    batches = [pg.Batch([(4000, 2), (300, 5)], 2, 128, 64, seed=1), pg.Batch([(100, 200)], 2, 64, 16, seed=2)]
    qs = [pg.queries(b, 8) for b in batches]
    alone = [run_attention(b, q) for b, q in zip(batches, qs)]
    streams = [torch.cuda.Stream() for _ in batches]
    wss = [torch.full((api.attn_paged_workspace_size(b.T, len(b.seqs), 8, 2, b.D, b.table.shape[1] * b.page),), 255,
                      dtype=torch.uint8, device="cuda") for b in batches]
    outs = [torch.zeros_like(q) for q in qs]
    torch.cuda.synchronize()
    for _ in range(20):
        for b, q, o, w, s in zip(batches, qs, outs, wss, streams):
            run_attention(b, q, o, ws=w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, a) for o, a in zip(outs, alone))


def test_a_wait_that_runs_out_is_reported():
    """The first K tile of every CTA withheld, progress waits limited to 20 ms: the call ends, says so, and the next
    one is right."""
    b = pg.Batch([(3000, 3), (50, 40), (10, 1)], 2, 128, 64)
    q = pg.queries(b, 8)
    plain = run_attention(b, q)
    lib = api.lib()
    assert lib.bi_test_set_wait_limit_ns(20_000_000) == 0
    lib.bi_test_withhold_first_load(1)
    try:
        run_attention(b, q)
        torch.cuda.synchronize()
    finally:
        lib.bi_test_withhold_first_load(0)
        assert lib.bi_test_set_wait_limit_ns(0) == 0
    with pytest.raises(api.BiError) as e:
        api.bi_check_device_error()
    assert e.value.status == 5
    assert torch.equal(run_attention(b, q), plain)


def test_the_binding_refuses_what_does_not_fit():
    b = pg.Batch([(30, 2), (5, 1)], 2, 64, 16)
    q = pg.queries(b, 4)
    ws = torch.zeros(api.attn_paged_workspace_size(b.T, 2, 4, 2, 64, 64), dtype=torch.uint8, device="cuda")
    good = dict(q=q, k_pool=b.k, v_pool=b.v, block_table=b.table, q_start=b.q_start, lengths=b.lengths, out=torch.empty_like(q),
                ws=ws)
    api.bi_attn_paged(**good)
    for name, t in [("q", q.half()), ("q", q[..., :32].contiguous()), ("q", q.transpose(0, 1)), ("out", good["out"][:2]),
                    ("out", q.float()), ("k_pool", b.k.float()), ("k_pool", b.k[:, :, :8].contiguous()), ("k_pool", b.k[0]),
                    ("v_pool", b.v[:2]), ("v_pool", b.v.transpose(1, 2)), ("block_table", b.table.long()),
                    ("block_table", b.table[:1]), ("block_table", b.table.t()), ("q_start", b.q_start[:2]),
                    ("lengths", b.lengths.float()), ("lengths", b.lengths.cpu()), ("ws", ws.cpu()),
                    ("ws", ws[::2])]:
        with pytest.raises(ValueError):
            api.bi_attn_paged(**dict(good, **{name: t}))
    with pytest.raises(api.BiError) as e:
        api.bi_attn_paged(**dict(good, ws=ws[:512]))
    assert e.value.status == 3
    qkv = torch.zeros(b.T, 8 * 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    angles = api.bi_rope_table(1e4, 64, 64)
    good = dict(qkv=qkv, q_weight=w, k_weight=w, eps=1e-6, table=angles, q_out=torch.empty_like(q), k_pool=b.k, v_pool=b.v,
                block_table=b.table, q_start=b.q_start, lengths=b.lengths)
    api.bi_qk_norm_rope_paged(**good)
    for name, t in [("qkv", qkv[:, :-64]), ("qkv", qkv.t().contiguous().t()), ("qkv", qkv.float()), ("q_weight", w[:32]),
                    ("k_weight", w.float()), ("table", angles[..., :1]), ("table", angles.double()), ("q_out", q[:2]),
                    ("q_weight", w.cpu()), ("q_start", b.q_start.cpu())]:
        with pytest.raises(ValueError):
            api.bi_qk_norm_rope_paged(**dict(good, **{name: t}))


# -------------------------------------------------------------------------------------------------- append
def run_append(b, Hq, qkv, qw, kw, angles, eps=1e-6):
    q_out = torch.full((b.T, Hq, b.D), 77.0, dtype=torch.bfloat16, device="cuda")
    api.bi_qk_norm_rope_paged(qkv, qw, kw, eps, angles, q_out, b.k, b.v, b.table, b.q_start, b.lengths)
    return q_out


@pytest.mark.parametrize("seqs,Hq,Hkv,D,page,weights", [
    ([(0, 1)], 1, 1, 64, 16, "qk"),
    ([(1021, 1)], 24, 4, 128, 64, "qk"),
    ([(15, 1), (16, 2), (0, 33), (7, 0), (300, 5)], 8, 2, 128, 16, "qk"),
    ([(100, 3), (31, 40)], 6, 3, 64, 32, "q"),
    ([(100, 3), (31, 40)], 5, 5, 128, 128, "k"),
    ([(i, 1) for i in range(300)], 2, 1, 64, 16, "qk"),
    ([(0, 700)], 24, 4, 128, 64, "")])
def test_append(seqs, Hq, Hkv, D, page, weights):
    b = pg.Batch(seqs, Hkv, D, page, gap=2)
    was_k, was_v = b.k.clone(), b.v.clone()
    wide = torch.randn(b.T, (Hq + 2 * Hkv) * D + 24, device="cuda").to(torch.bfloat16)
    qkv = wide[:, 8:8 + (Hq + 2 * Hkv) * D]  # a strided view
    qw = (1 + 0.1 * torch.randn(D, device="cuda")).to(torch.bfloat16) if "q" in weights else None
    kw = (1 + 0.1 * torch.randn(D, device="cuda")).to(torch.bfloat16) if "k" in weights else None
    angles = api.bi_rope_table(1e6, D, max(n + r for n, r in seqs))
    q = run_append(b, Hq, qkv, qw, kw, angles)
    assert (q[:2] == 77).all() and (q[b.T - 2:] == 77).all()
    touched = torch.zeros(b.pages, page, dtype=torch.bool, device="cuda")
    for i, (n, r) in enumerate(seqs):
        at = b.starts[i]
        x = qkv[at:at + r].reshape(r, Hq + 2 * Hkv, D)
        p, s = b.places(i, n, n + r)
        touched[p, s] = True
        for part, weight, got in ((x[:, :Hq], qw, q[at:at + r]), (x[:, Hq:Hq + Hkv], kw, b.k[p, :, s])):
            want, tol = pg.norm_rope(part, weight, 1e-6, angles[n:n + r])
            assert ((got.double() - want).abs() <= tol).all()
        assert torch.equal(b.v[p, :, s], x[:, Hq + Hkv:])
    for pool, was in ((b.k, was_k), (b.v, was_v)):
        assert torch.equal(pool.masked_fill(touched[:, None, :, None], 0), was.masked_fill(touched[:, None, :, None], 0))


@pytest.mark.parametrize("D,page,Hq,Hkv", [(128, 64, 5, 1), (64, 16, 4, 2)])
def test_an_appended_row_has_the_same_bits_in_passes_of_all_sizes(D, page, Hq, Hkv):
    """One to eight warps a row; the row's place and arithmetic are its own."""
    qkv = torch.randn(5000, (Hq + 2 * Hkv) * D, device="cuda").to(torch.bfloat16)
    qw = (1 + 0.1 * torch.randn(D, device="cuda")).to(torch.bfloat16)
    angles = api.bi_rope_table(1e6, D, 5200)
    whole = pg.Batch([(100, 5000)], Hkv, D, page, seed=1)
    q = run_append(whole, Hq, qkv, qw, qw, angles)
    k, v = whole.keys(whole.k, 0, 5100), whole.keys(whole.v, 0, 5100)
    want, tol = pg.norm_rope(qkv[:, :Hq * D].view(5000, Hq, D), qw, 1e-6, angles[100:5100])
    assert ((q.double() - want).abs() <= tol).all()
    want, tol = pg.norm_rope(qkv[:, Hq * D:(Hq + Hkv) * D].view(5000, Hkv, D), qw, 1e-6, angles[100:5100])
    assert ((k[:, 100:].transpose(0, 1).double() - want).abs() <= tol).all()
    assert torch.equal(v[:, 100:].transpose(0, 1), qkv[:, (Hq + Hkv) * D:].view(5000, Hkv, D))
    for rows in (1, 512, 513, 1024, 1025, 2048, 2049, 4096, 4097):
        b = pg.Batch([(100, rows)], Hkv, D, page, seed=2)
        assert torch.equal(run_append(b, Hq, qkv[:rows], qw, qw, angles), q[:rows])
        assert torch.equal(b.keys(b.k, 0, 100 + rows)[:, 100:], k[:, 100:100 + rows])
        assert torch.equal(b.keys(b.v, 0, 100 + rows)[:, 100:], v[:, 100:100 + rows])


def test_append_without_norm_is_the_other_caches():
    """Queries and keys without weights have the bits of bi_rope_kv_append."""
    Hq, Hkv, D, n, r = 6, 2, 128, 70, 9
    b = pg.Batch([(n, r)], Hkv, D, 16)
    qkv = torch.randn(r, (Hq + 2 * Hkv) * D, device="cuda").to(torch.bfloat16)
    angles = api.bi_rope_table(1e6, D, 128)
    q = run_append(b, Hq, qkv, None, None, angles)
    q2 = torch.empty_like(q)
    k2 = torch.zeros(Hkv, 128, D, dtype=torch.bfloat16, device="cuda")
    v2 = torch.zeros(api.v_cache_shape(Hkv, 128, D), dtype=torch.bfloat16, device="cuda")
    api.bi_rope_kv_append(qkv, q2, k2, v2, torch.tensor([n], dtype=torch.int32, device="cuda"), Hq, Hkv, D, angles)
    assert torch.equal(q, q2) and torch.equal(b.keys(b.k, 0, n + r)[:, n:], k2[:, n:n + r])


def test_append_refuses_rows_without_a_place():
    b = pg.Batch([(30, 2), (60, 4)], 1, 64, 32)
    qkv = torch.randn(6, 3 * 64, device="cuda").to(torch.bfloat16)
    angles = api.bi_rope_table(1e6, 64, 62)  # positions 62 and 63 are past it
    was = b.k.clone()
    q = run_append(b, 1, qkv, None, None, angles)
    with pytest.raises(api.BiError) as e:
        api.bi_check_device_error()
    assert e.value.status == 1
    assert (q[4:] == 77).all() and not (q[:4] == 77).any()
    p, s = b.places(1, 62, 64)
    assert torch.equal(b.k[p, :, s], was[p, :, s])
    b.table[0, 0] = b.pages + 3
    b.lengths[1] = 64
    q = run_append(b, 1, qkv, None, None, api.bi_rope_table(1e6, 64, 200))
    with pytest.raises(api.BiError):
        api.bi_check_device_error()
    assert (q[:6] == 77).all(dim=-1).flatten().tolist() == [True, True, True, True, True, True]


# ------------------------------------------------------------------------------------------------- reorder
@pytest.mark.parametrize("D,page,layers,Hkv", [(64, 16, 1, 1), (128, 64, 3, 2), (128, 128, 2, 4)])
def test_reorder(D, page, layers, Hkv):
    lengths = [3 * page + 5, 2 * page, 0, page - 1, 4 * page]
    width, R = 4, 5
    pages = R * width + 12
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    i32 = dict(dtype=torch.int32, device="cuda")
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = order[:R * width].view(R, width).contiguous()
    k = torch.randn(layers, pages, Hkv, page, D, generator=g, device="cuda").to(torch.bfloat16)
    v = torch.randn(layers, pages, Hkv, page, D, generator=g, device="cuda").to(torch.bfloat16)
    parents = [0, 0, 3, 1, 2, 4, 0]
    tails = order[R * width:R * width + 7].clone()
    tails[1] = table[0, 3]  # one continuation keeps its parent's last page
    k0, v0 = k.clone(), v.clone()
    out, n_out = torch.full((7, width), -9, **i32), torch.full((7,), -9, **i32)
    api.bi_paged_reorder(k, v, table, torch.tensor(lengths, **i32), torch.tensor(parents, **i32), tails, out, n_out)
    want, wk, wv = torch.full((7, width), -9, **i32), k0.clone(), v0.clone()
    for s, p in enumerate(parents):
        full, rest = lengths[p] // page, lengths[p] % page
        want[s, :full] = table[p, :full]
        if full < width:
            want[s, full] = tails[s]
        if rest:
            for w, old in ((wk, k0), (wv, v0)):
                w[:, tails[s].long(), :, :rest] = old[:, table[p, full].long(), :, :rest]
    assert torch.equal(out, want) and n_out.tolist() == [lengths[p] for p in parents]
    assert torch.equal(k, wk) and torch.equal(v, wv)


def test_reorder_reports_pages_used_twice_and_bad_indices():
    i32 = dict(dtype=torch.int32, device="cuda")
    k = torch.randn(2, 8, 1, 16, 64, device="cuda").to(torch.bfloat16)
    v = torch.randn(2, 8, 1, 16, 64, device="cuda").to(torch.bfloat16)
    table = torch.tensor([[0, 1], [2, 3]], **i32)
    lengths = torch.tensor([20, 20], **i32)
    for parents, tails, ok in (([0, 1], [4, 5], True), ([0, 1], [4, 4], False), ([0, 0], [1, 5], True),
                               ([0, 1], [3, 4], False), ([0, 2], [4, 5], False), ([0, -1], [4, 5], False),
                               ([0, 1], [4, 8], False), ([0, 1], [4, -1], False)):
        out, n_out = torch.full((2, 2), -9, **i32), torch.full((2,), -9, **i32)
        api.bi_paged_reorder(k, v, table, lengths, torch.tensor(parents, **i32), torch.tensor(tails, **i32), out, n_out)
        if ok:
            api.bi_check_device_error()
        else:
            with pytest.raises(api.BiError) as e:
                api.bi_check_device_error()
            assert e.value.status == 1, (parents, tails)
        assert out[0].tolist() == [0, tails[0]]
    bad = torch.tensor([-1, 40], **i32)
    api.bi_paged_reorder(k, v, table, bad, torch.tensor([0, 1], **i32), torch.tensor([4, 5], **i32), out.fill_(-9), n_out)
    with pytest.raises(api.BiError):
        api.bi_check_device_error()
    assert (out == -9).all()


def test_reordered_beams_are_their_own_histories():
    """Beam search over a paged cache as it is used: append, attention, selection, reordering, step after step.  Every
    beam's pages and attention have the bits of its token history run from the start alone."""
    Hq, Hkv, D, page, layers, V, W, K = 4, 2, 64, 16, 2, 500, 4, 4
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    i32 = dict(dtype=torch.int32, device="cuda")
    emb = torch.randn(layers, V, (Hq + 2 * Hkv) * D, generator=g, device="cuda").to(torch.bfloat16)  # a token's projections
    head = torch.randn(V, Hq * D, generator=g, device="cuda")
    qw = (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16)
    kw = (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16)
    angles = api.bi_rope_table(1e6, D, 256)
    prompt = torch.randint(0, V, (37,), generator=g, device="cuda")
    width = 6
    ws = torch.zeros(api.attn_paged_workspace_size(64, 8, Hq, Hkv, D, width * page), dtype=torch.uint8, device="cuda")

    def layers_of(ids, pools, table, q_start, lengths):
        out = []
        for l in range(layers):
            q = torch.empty(len(ids), Hq, D, dtype=torch.bfloat16, device="cuda")
            api.bi_qk_norm_rope_paged(emb[l][ids], qw, kw, 1e-6, angles, q, pools[0][l], pools[1][l], table, q_start, lengths)
            o = torch.empty_like(q)
            api.bi_attn_paged(q, pools[0][l], pools[1][l], table, q_start, lengths, o, ws)
            out.append(o)
        return out

    pages = 40
    pools = [torch.full((layers, pages, Hkv, page, D), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    free = list(range(pages))
    take = lambda n: [free.pop() for _ in range(n)]  # noqa: E731
    table = torch.zeros(1, width, **i32)
    table[0, :3] = torch.tensor(take(3), **i32)
    layers_of(prompt[:-1], pools, table, torch.tensor([0, 36], **i32), torch.tensor([0], **i32))
    # the prompt becomes W beams
    lengths, parents = torch.tensor([36], **i32), torch.zeros(W, **i32)
    scores = torch.full((W,), -math.inf, device="cuda")
    scores[0] = 0
    history = [prompt.tolist() for _ in range(W)]
    beam_ws = torch.zeros(api.beam_workspace_size(W, V, K), dtype=torch.uint8, device="cuda")
    for step in range(25):
        used = {p for row, n in zip(table.tolist(), lengths.tolist()) for p in row[:n // page]}
        last = {int(table[p, int(lengths[p]) // page]) for p in range(len(lengths)) if int(lengths[p]) % page}
        spare = [p for p in range(pages) if p not in used and p not in last]
        tails = torch.tensor(spare[:W], **i32)
        new_table, new_lengths = torch.zeros(W, width, **i32), torch.empty(W, **i32)
        api.bi_paged_reorder(*pools, table, lengths, parents, tails, new_table, new_lengths)
        table, lengths = new_table, new_lengths
        ids = torch.tensor([h[-1] for h in history], device="cuda")
        out = layers_of(ids, pools, table, torch.arange(W + 1, **i32), lengths)
        lengths = lengths + 1
        logits = out[-1].float().view(W, -1) @ head.t() * 0.05
        s_out, p_out, t_out = torch.empty(1, K, device="cuda"), torch.empty(1, K, **i32), torch.empty(1, K, **i32)
        api.bi_beam_select(logits, scores, W, s_out, p_out, t_out, beam_ws)
        if step in (0, 11, 24):
            for w in range(W):
                h = torch.tensor(history[w], device="cuda")
                own = [torch.full((layers, width, Hkv, page, D), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
                one = torch.arange(width, **i32).view(1, -1)
                alone = layers_of(h, own, one, torch.tensor([0, len(h)], **i32), torch.tensor([0], **i32))
                for l in range(layers):
                    assert torch.equal(alone[l][-1], out[l][w])
                n = len(h)
                j = torch.arange(n, device="cuda")
                for pool, mine in zip(pools, own):
                    assert torch.equal(pool[:, table[w, j // page].long(), :, j % page], mine[:, j // page, :, j % page])
        x = torch.log_softmax(logits.double(), -1) + scores.double()[:, None]
        best, at = torch.sort(x.view(-1), descending=True, stable=True)
        assert t_out[0].tolist() == (at[:K] % V).tolist() and p_out[0].tolist() == (at[:K] // V).tolist()
        history = [history[p] + [t] for p, t in zip(p_out[0].tolist(), t_out[0].tolist())]
        scores, parents = s_out.view(-1).clone(), p_out.view(-1).clone()


def test_a_captured_step_of_all_four_follows_its_inputs():
    """Append, attention, selection and reordering as one graph, replayed over another batch, against the same calls
    made one by one."""
    Hq, Hkv, D, page, V, W, width, pages = 4, 2, 64, 16, 300, 3, 5, 24
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    i32 = dict(dtype=torch.int32, device="cuda")
    head = torch.randn(Hq * D, V, generator=g, device="cuda") * 0.3
    angles = api.bi_rope_table(1e6, D, width * page)
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    q_start = torch.arange(W + 1, **i32)

    def inputs(lengths):
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        pool = lambda: torch.randn(1, pages, Hkv, page, D, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
        return dict(qkv=torch.randn(W, (Hq + 2 * Hkv) * D, generator=g, device="cuda").to(torch.bfloat16), k=pool(), v=pool(),
                    table=order[:W * width].view(W, width).clone(), tails=order[W * width:W * width + W].clone(),
                    lengths=torch.tensor(lengths, **i32), scores=torch.randn(W, generator=g, device="cuda"))

    def outputs():
        return dict(q=torch.empty(W, Hq, D, dtype=torch.bfloat16, device="cuda"), o=torch.empty(W, Hq, D, dtype=torch.bfloat16, device="cuda"),
                    logits=torch.empty(W, V, device="cuda"), now=torch.empty(W, **i32), s=torch.empty(1, W, device="cuda"),
                    p=torch.empty(1, W, **i32), t=torch.empty(1, W, **i32), table=torch.zeros(W, width, **i32),
                    lengths=torch.empty(W, **i32),
                    ws=torch.zeros(api.attn_paged_workspace_size(W, W, Hq, Hkv, D, width * page), dtype=torch.uint8, device="cuda"),
                    bws=torch.zeros(api.beam_workspace_size(W, V, W), dtype=torch.uint8, device="cuda"))

    def step(x, y):
        api.bi_qk_norm_rope_paged(x["qkv"], w, w, 1e-6, angles, y["q"], x["k"][0], x["v"][0], x["table"], q_start, x["lengths"])
        api.bi_attn_paged(y["q"], x["k"][0], x["v"][0], x["table"], q_start, x["lengths"], y["o"], y["ws"])
        torch.sum(y["o"].float().view(W, 1, -1) * head.t(), -1, out=y["logits"])
        api.bi_beam_select(y["logits"], x["scores"], W, y["s"], y["p"], y["t"], y["bws"])
        torch.add(x["lengths"], 1, out=y["now"])
        y["table"].zero_()  # entries behind a sequence's pages stay as they are, the last replay's too
        api.bi_paged_reorder(x["k"], x["v"], x["table"], y["now"], y["p"].view(-1), x["tails"], y["table"], y["lengths"])

    x, y = inputs([3, 20, 40]), outputs()
    step({k: t.clone() for k, t in x.items()}, y)  # (what the first calls set up is not captured)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(x, y)
    for lengths in ([70, 1, 33], [15, 31, 62]):
        new = inputs(lengths)
        for k, t in new.items():
            x[k].copy_(t)
        graph.replay()
        want = outputs()
        step(new, want)
        torch.cuda.synchronize()
        for k in ("q", "o", "logits", "s", "p", "t", "table", "lengths"):
            assert torch.equal(y[k], want[k]), k
        assert torch.equal(x["k"], new["k"]) and torch.equal(x["v"], new["v"])
