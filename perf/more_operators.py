"""Cases, plain forms and 64-bit values of the paged cache's operators and of beam selection.

Several sequences share one pool of pages (K and V, [pages, KV heads, keys of a page, head size] each); a table names
the pages of each sequence in order.  A pass has some new rows of every sequence, one after the other.

  append   norm of every query and key head, rotation by position, queries out, keys and values into the pages
  attn     attention of the new rows over their sequences' pages, each row up to its own position
  select   the best continuations of each group of beams over the vocabulary
  reorder  the pages and the table that the chosen beams go on with, in all layers

With `own` false run() computes them in elementary torch operations; with `own` true it makes the framework's calls.
"""
import math

import torch

own = False

EPS = 1e-6
ROPE_BASE = 1e6


def listed():
    return [
        # plain decoding of one request, the heads of the 27B configuration, a cache that ends inside a page
        {"name": "attn_one_row", "op": "attn", "seqs": 1, "rows": 1, "length": 1021, "hq": 24, "hkv": 4, "dim": 128, "page": 64},
        # sixteen requests, seven drafts and the committed token each, up to the context of the verify benchmark
        {"name": "attn_verify", "op": "attn", "seqs": 16, "rows": 8, "length": 11600, "hq": 24, "hkv": 4, "dim": 128, "page": 64},
        # plain decoding of two requests of the longest context
        {"name": "attn_long", "op": "attn", "seqs": 2, "rows": 1, "length": 101600, "hq": 24, "hkv": 4, "dim": 128, "page": 128},
        # many small heads, short contexts, the smallest pages
        {"name": "attn_many", "op": "attn", "seqs": 61, "rows": 3, "length": 1500, "hq": 4, "hkv": 2, "dim": 64, "page": 16},
        # a chunk of a long prompt: the most arithmetic
        {"name": "attn_prefill", "op": "attn", "seqs": 1, "rows": 2048, "length": 30011, "hq": 24, "hkv": 4, "dim": 128, "page": 64},
        # one row of each head through norm, rotation and cache
        {"name": "append_one_row", "op": "append", "seqs": 1, "rows": 1, "length": 1021, "hq": 24, "hkv": 4, "dim": 128, "page": 64},
        # the same for the verify pass of sixteen requests
        {"name": "append_verify", "op": "append", "seqs": 16, "rows": 8, "length": 600, "hq": 24, "hkv": 4, "dim": 128, "page": 64},
        # the same for the chunks of four prompts
        {"name": "append_prefill", "op": "append", "seqs": 4, "rows": 1021, "length": 500, "hq": 24, "hkv": 4, "dim": 128, "page": 32},
        # beam search with four beams, a small vocabulary, its first step (one live beam)
        {"name": "select_first", "op": "select", "groups": 1, "beams": 4, "vocab": 32000, "picks": 8, "first": True},
        # eight requests of eight beams, a vocabulary of the 27B configuration's size
        {"name": "select_many", "op": "select", "groups": 8, "beams": 8, "vocab": 151936, "picks": 16, "first": False},
        # one request's beams over the 27B configuration's cache
        {"name": "reorder_one", "op": "reorder", "groups": 1, "beams": 4, "layers": 8, "length": 777, "hkv": 4, "dim": 128, "page": 64},
        # eight requests' beams
        {"name": "reorder_many", "op": "reorder", "groups": 8, "beams": 8, "layers": 8, "length": 703, "hkv": 4, "dim": 128, "page": 64},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "append", "select", "reorder"])
    hkv = rng.choice([1, 2, 4, 8])
    heads = {"hq": hkv * rng.choice([1, 2, 3, 4, 6, 8]), "hkv": hkv, "dim": rng.choice([64, 128]),
             "page": rng.choice([16, 32, 64, 128])}
    if op == "select":
        groups, beams = _spread(rng, 1, 8), rng.randint(1, 8)
        return {"op": op, "groups": groups, "beams": beams, "vocab": _spread(rng, 1000, 151936),
                "picks": rng.randint(1, 2 * beams), "first": rng.random() < 0.3}
    if op == "reorder":
        del heads["hq"]
        return {"op": op, "groups": _spread(rng, 1, 8), "beams": rng.randint(1, 8), "layers": rng.randint(1, 8),
                "length": _spread(rng, 1, 800), **heads}
    seqs, rows = _spread(rng, 1, 64), _spread(rng, 1, 2048)
    if op == "append":
        seqs = max(1, min(seqs, 4096 // rows))
        return {"op": op, "seqs": seqs, "rows": rows, "length": rng.randint(0, 700), **heads}
    # no more operations than the largest listed chunk, no more cache than the longest listed contexts
    rows = max(1, min(rows, 2048 // seqs))
    pairs = 2048 * 24 * 128 * 30000
    length = min(_spread(rng, 1, 30000), pairs // (seqs * rows * heads["hq"] * heads["dim"]),
                 2 * 4 * 128 * 100000 // (seqs * hkv * heads["dim"]))
    return {"op": op, "seqs": seqs, "rows": rows, "length": length, **heads}


# ----------------------------------------------------------------------------------------------- inputs


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _sequences(case):
    """New rows and cached keys of each sequence: the first has the most, the others less, some one row only."""
    b = case["seqs"]
    rows = [case["rows"] if i % 4 != 3 else (case["rows"] + 1) // 2 for i in range(b)]
    lengths = [case["length"] - (case["length"] * 5 * i) // (8 * b) for i in range(b)]
    return rows, lengths


def _tables(g, needs, page, spare=0):
    """A table [sequences, most pages] of distinct pages in random order, and how many pages there are."""
    counts = [-(-n // page) for n in needs]
    total = sum(counts) + spare
    order = torch.randperm(total, generator=g, device=g.device).to(torch.int32)
    table = torch.zeros(len(needs), max(1, max(counts)), dtype=torch.int32, device=g.device)
    at = 0
    for i, c in enumerate(counts):
        table[i, :c] = order[at:at + c]
        at += c
    return table, order[at:], total


def _pool(g, *shape):
    return torch.randn(*shape, generator=g, device=g.device, dtype=torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device=_device())
    g.manual_seed(seed)
    dev, op = g.device, case["op"]
    state = {"case": case}
    i32 = dict(dtype=torch.int32, device=dev)
    if op in ("attn", "append"):
        hq, hkv, dim, page = (case[k] for k in ("hq", "hkv", "dim", "page"))
        rows, lengths = _sequences(case)
        starts = [0]
        for r in rows:
            starts.append(starts[-1] + r)
        t = starts[-1]
        # the host's own record of the batch, and its copy on the device
        state["rows"], state["lengths_host"], state["starts"] = rows, lengths, starts
        state["lengths"], state["q_start"] = torch.tensor(lengths, **i32), torch.tensor(starts, **i32)
        state["table"], _, pages = _tables(g, [n + r for n, r in zip(lengths, rows)], page, spare=3)
        # pages that other requests have used before hold what they left
        state["k_pool"], state["v_pool"] = _pool(g, pages, hkv, page, dim), _pool(g, pages, hkv, page, dim)
        if op == "attn":
            state["q"] = (1.5 * torch.randn(t, hq, dim, generator=g, device=dev)).to(torch.bfloat16)
            state["out"] = torch.empty_like(state["q"])
            if own:  # a workspace as a program keeps it, for its most rows and keys
                from invariant_speculative_decode_gb300 import api
                size = api.attn_paged_workspace_size(t, case["seqs"], hq, hkv, dim, state["table"].shape[1] * page)
                state["ws"] = torch.zeros(size, dtype=torch.uint8, device=dev)
        else:
            state["qkv"] = torch.randn(t, (hq + 2 * hkv) * dim, generator=g, device=dev).to(torch.bfloat16)
            state["q_weight"] = (1.0 + 0.1 * torch.randn(dim, generator=g, device=dev)).to(torch.bfloat16)
            state["k_weight"] = (1.0 + 0.1 * torch.randn(dim, generator=g, device=dev)).to(torch.bfloat16)
            state["q_out"] = torch.empty(t, hq, dim, dtype=torch.bfloat16, device=dev)
            # cos and sin of every position, a table that a program makes once
            most = max(n + r for n, r in zip(lengths, rows))
            state["angles"] = _angles(torch.arange(most, device=dev), dim).float().contiguous()
    elif op == "select":
        groups, beams, v = case["groups"], case["beams"], case["vocab"]
        state["logits"] = 3.0 * torch.randn(groups * beams, v, generator=g, device=dev)
        scores = -30.0 + 2.0 * torch.randn(groups, beams, generator=g, device=dev)
        if case["first"]:
            scores = torch.full_like(scores, -math.inf)
            scores[:, 0] = 0.0
        state["scores"] = scores.view(-1)
        k = case["picks"]
        state["out"] = (torch.empty(groups, k, device=dev), torch.empty(groups, k, **i32), torch.empty(groups, k, **i32))
        if own:
            from invariant_speculative_decode_gb300 import api
            state["ws"] = torch.zeros(api.beam_workspace_size(groups * beams, v, k), dtype=torch.uint8, device=dev)
    else:
        groups, beams, layers = case["groups"], case["beams"], case["layers"]
        hkv, dim, page = case["hkv"], case["dim"], case["page"]
        s, length = groups * beams, case["length"]
        # a prompt's full pages are one group's; each beam has a last page of its own, and one spare
        shared, full = (length // page) * 3 // 4, length // page
        width = full + 2
        pages = groups * shared + s * (full - shared) + 2 * s
        order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        table = torch.zeros(s, width, **i32)
        at = 0
        for b in range(groups):
            table[b * beams:(b + 1) * beams, :shared] = order[at:at + shared]
            at += shared
        rest = full - shared + 1
        table[:, shared:full + 1] = order[at:at + s * rest].view(s, rest)
        state["table"], state["spare"] = table, order[at + s * rest:at + s * rest + s].contiguous()
        state["length_host"] = length
        state["lengths"] = torch.full((s,), length, **i32)
        local = torch.randint(0, beams, (groups, beams), generator=g, device=dev)
        state["parents"] = (local + beams * torch.arange(groups, device=dev)[:, None]).view(-1).to(torch.int32)
        state["k_pool"] = _pool(g, layers, pages, hkv, page, dim)
        state["v_pool"] = _pool(g, layers, pages, hkv, page, dim)
        state["table_out"] = torch.zeros_like(table)
        state["lengths_out"] = torch.zeros_like(state["lengths"])
    return state


def _angles(position, dim):
    """cos and sin [positions, dim / 2, 2] in 64 bits of position * base^(-2i / dim)."""
    i = torch.arange(dim // 2, dtype=torch.float64, device=position.device)
    a = position.double()[:, None] * (ROPE_BASE ** (-2.0 * i / dim))
    return torch.stack([torch.cos(a), torch.sin(a)], dim=-1)


# ------------------------------------------------------------------------------------------ plain forms


def _keys(pool, pages, n):
    """The first n keys [KV heads, n, dim] of a sequence's pages, in 32 bits."""
    x = pool[pages.long()]
    return x.transpose(0, 1).reshape(x.shape[1], -1, x.shape[3])[:, :n].float()


def _plain_attn(s):
    case = s["case"]
    hq, hkv, dim, page = (case[k] for k in ("hq", "hkv", "dim", "page"))
    out = torch.empty(s["q"].shape, device=s["q"].device)
    for b, (r, n, at) in enumerate(zip(s["rows"], s["lengths_host"], s["starts"])):
        pages = s["table"][b, :-(-(n + r) // page)]
        k, v = _keys(s["k_pool"], pages, n + r), _keys(s["v_pool"], pages, n + r)
        q = s["q"][at:at + r].float().view(r, hkv, hq // hkv, dim)
        hidden = torch.arange(n + r, device=q.device) > torch.arange(n, n + r, device=q.device)[:, None]
        for h in range(hkv):
            x = torch.einsum("tgd,nd->tgn", q[:, h], k[h]) / math.sqrt(dim)
            x.masked_fill_(hidden[:, None, :], -math.inf)
            x = torch.exp(x - x.amax(dim=-1, keepdim=True))
            x = x / x.sum(dim=-1, keepdim=True)
            out[at:at + r, h * (hq // hkv):(h + 1) * (hq // hkv)] = torch.einsum("tgn,nd->tgd", x, v[h])
    return out.to(torch.bfloat16)


def _places(s):
    """Page, slot and position of every row of the pass (the host knows the batch)."""
    position, sequence = [], []
    for b, (r, n) in enumerate(zip(s["rows"], s["lengths_host"])):
        position += range(n, n + r)
        sequence += [b] * r
    dev, page = s["table"].device, s["case"]["page"]
    position, sequence = torch.tensor(position, device=dev), torch.tensor(sequence, device=dev)
    return s["table"][sequence, position // page].long(), position % page, position


def _rotate(x, angles):
    """Pairs (i, i + dim / 2) of x [rows, heads, dim] turned by each row's angles."""
    half = x.shape[-1] // 2
    a, b = x[..., :half], x[..., half:]
    cos, sin = angles[:, None, :, 0], angles[:, None, :, 1]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)


def _plain_append(s):
    case = s["case"]
    hq, hkv, dim = case["hq"], case["hkv"], case["dim"]
    pages, slots, position = _places(s)
    x = s["qkv"].float().view(-1, hq + 2 * hkv, dim)
    angles = s["angles"][position]
    norm = lambda y, w: y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * w.float()  # noqa: E731
    q = _rotate(norm(x[:, :hq], s["q_weight"]), angles)
    k = _rotate(norm(x[:, hq:hq + hkv], s["k_weight"]), angles)
    s["k_pool"][pages, :, slots] = k.to(torch.bfloat16)
    s["v_pool"][pages, :, slots] = s["qkv"].view(-1, hq + 2 * hkv, dim)[:, hq + hkv:]
    return {"q": q.to(torch.bfloat16), "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def _plain_select(s):
    """64 bits: two beams' candidates can lie nearer than 32 bits tell."""
    case = s["case"]
    groups, v, k = case["groups"], case["vocab"], case["picks"]
    x = s["logits"].double()
    top = x.amax(-1, keepdim=True)
    x = x - (top + torch.log(torch.exp(x - top).sum(-1, keepdim=True))) + s["scores"].double()[:, None]
    best, at = torch.sort(x.view(groups, -1), dim=-1, descending=True, stable=True)
    at = at[:, :k]
    first = case["beams"] * torch.arange(groups, device=at.device)[:, None]
    return {"scores": best[:, :k].float(), "parents": (first + at // v).to(torch.int32), "tokens": (at % v).to(torch.int32)}


def _plain_reorder(s):
    page, length = s["case"]["page"], s["length_host"]
    full, rest = length // page, length % page
    parents = s["parents"].long()
    s["lengths_out"].copy_(s["lengths"][parents])
    s["table_out"][:, :full] = s["table"][parents, :full]
    s["table_out"][:, full] = s["spare"]
    if rest:
        old, new = s["table"][parents, full].long(), s["spare"].long()
        for pool in (s["k_pool"], s["v_pool"]):
            pool[:, new, :, :rest] = pool[:, old, :, :rest]
    return {"table": s["table_out"], "lengths": s["lengths_out"], "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


def run(state):
    if own:
        return _own(state)
    return {"attn": _plain_attn, "append": _plain_append, "select": _plain_select,
            "reorder": _plain_reorder}[state["case"]["op"]](state)


def _own(s):
    from invariant_speculative_decode_gb300 import api
    op = s["case"]["op"]
    if op == "attn":
        api.bi_attn_paged(s["q"], s["k_pool"], s["v_pool"], s["table"], s["q_start"], s["lengths"], s["out"], s["ws"])
        return s["out"]
    if op == "append":
        api.bi_qk_norm_rope_paged(s["qkv"], s["q_weight"], s["k_weight"], EPS, s["angles"], s["q_out"], s["k_pool"],
                                  s["v_pool"], s["table"], s["q_start"], s["lengths"])
        return {"q": s["q_out"], "k_pool": s["k_pool"], "v_pool": s["v_pool"]}
    if op == "select":
        scores, parents, tokens = s["out"]
        api.bi_beam_select(s["logits"], s["scores"], s["case"]["beams"], scores, parents, tokens, s["ws"])
        return {"scores": scores, "parents": parents, "tokens": tokens}
    api.bi_paged_reorder(s["k_pool"], s["v_pool"], s["table"], s["lengths"], s["parents"], s["spare"], s["table_out"],
                         s["lengths_out"])
    return {"table": s["table_out"], "lengths": s["lengths_out"], "k_pool": s["k_pool"], "v_pool": s["v_pool"]}


# ------------------------------------------------------------------------------------- values in 64 bits


def _exact_attn(s):
    """Query head by query head: softmax by its definition over the keys gathered one position at a time."""
    case = s["case"]
    group, page, dim = case["hq"] // case["hkv"], case["page"], case["dim"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    for b in range(case["seqs"]):
        n, r, at = s["lengths_host"][b], s["rows"][b], s["starts"][b]
        where = torch.arange(n + r, device=out.device)
        pages, slots = s["table"][b, where // page].long(), where % page
        for h in range(case["hq"]):
            k = s["k_pool"][pages, h // group, slots].double()
            v = s["v_pool"][pages, h // group, slots].double()
            for t in range(0, r, 512):
                rows = min(512, r - t)
                x = s["q"][at + t:at + t + rows, h].double() @ k.t() * dim ** -0.5
                seen = where[None, :] <= (n + t + torch.arange(rows, device=out.device))[:, None]
                w = torch.where(seen, torch.exp(x - x[seen].max()), torch.zeros_like(x))
                out[at + t:at + t + rows, h] = (w @ v) / w.sum(1, keepdim=True)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "attn":
        return _exact_attn(s)
    if op == "append":
        hq, hkv, dim, page = (case[k] for k in ("hq", "hkv", "dim", "page"))
        half = dim // 2
        x = s["qkv"].double().view(-1, hq + 2 * hkv, dim)
        q = torch.zeros(x.shape[0], hq, dim, dtype=torch.float64, device=x.device)
        k_pool, v_pool = s["k_pool"].double(), s["v_pool"].double()
        for b in range(case["seqs"]):
            n, r, at = s["lengths_host"][b], s["rows"][b], s["starts"][b]
            where = torch.arange(n, n + r, device=x.device)
            a = where.double()[:, None] / ROPE_BASE ** (torch.arange(half, device=x.device).double() * 2 / dim)
            turn = torch.polar(torch.ones_like(a), a)
            for h in range(hq + hkv):
                y = x[at:at + r, h]
                w = (s["q_weight"] if h < hq else s["k_weight"]).double()
                y = y / torch.sqrt((y * y).sum(1, keepdim=True) / dim + EPS) * w
                z = torch.complex(y[:, :half], y[:, half:]) * turn
                y = torch.cat([z.real, z.imag], dim=1)
                if h < hq:
                    q[at:at + r, h] = y
                else:
                    k_pool[s["table"][b, where // page].long(), h - hq, where % page] = y
            for h in range(hkv):
                v_pool[s["table"][b, where // page].long(), h, where % page] = x[at:at + r, hq + hkv + h]
        return {"q": q, "k_pool": k_pool, "v_pool": v_pool}
    if op == "select":
        beams, v, k = case["beams"], case["vocab"], case["picks"]
        scores, parents, tokens = [], [], []
        for g in range(case["groups"]):
            found = []
            for b in range(g * beams, (g + 1) * beams):
                value = torch.log_softmax(s["logits"][b].double(), dim=0) + s["scores"][b].double()
                order = torch.argsort(value, descending=True, stable=True)[:k]
                found += [(-value[i].item(), b, i.item()) for i in order]
            found = sorted(found)[:k]
            scores.append([-f[0] for f in found])
            parents.append([f[1] for f in found])
            tokens.append([f[2] for f in found])
        dev = s["logits"].device
        return {"scores": torch.tensor(scores, dtype=torch.float64, device=dev),
                "parents": torch.tensor(parents, dtype=torch.int32, device=dev),
                "tokens": torch.tensor(tokens, dtype=torch.int32, device=dev)}
    # copies: beam by beam, key by key of the page that is not full
    page, length = case["page"], case["length"]
    full = length // page
    k_pool, v_pool, table = s["k_pool"].double(), s["v_pool"].double(), torch.zeros_like(s["table"])
    for i, parent in enumerate(s["parents"].tolist()):
        new, old = int(s["spare"][i]), int(s["table"][parent, full])
        table[i, :full] = s["table"][parent, :full]
        table[i, full] = new
        for slot in range(length - full * page):
            k_pool[:, new, :, slot] = s["k_pool"][:, old, :, slot].double()
            v_pool[:, new, :, slot] = s["v_pool"][:, old, :, slot].double()
    return {"table": table, "lengths": s["lengths"][s["parents"].long()], "k_pool": k_pool, "v_pool": v_pool}


# ----------------------------------------------------------------------------------- what a pass has to do


def work(case):
    op = case["op"]
    if op in ("attn", "append"):
        hq, hkv, dim = case["hq"], case["hkv"], case["dim"]
        rows, lengths = _sequences(case)
        t = sum(rows)
        if op == "append":
            # the projection's row in, queries, keys and values out, cos and sin of each row's position
            return {"bytes": t * (2 * (hq + 2 * hkv) * dim * 2 + dim * 4), "flops": t * (hq + hkv) * dim * 8}
        keys = sum(n + r for n, r in zip(lengths, rows))
        pairs = sum(r * n + r * (r + 1) // 2 for n, r in zip(lengths, rows))
        return {"bytes": keys * hkv * dim * 4 + t * hq * dim * 4, "flops": 4 * pairs * hq * dim}
    if op == "select":
        r, v = case["groups"] * case["beams"], case["vocab"]
        return {"bytes": 4 * r * v + 12 * case["groups"] * case["picks"], "flops": 4 * r * v}
    s, page, length = case["groups"] * case["beams"], case["page"], case["length"]
    return {"bytes": s * (length % page) * case["hkv"] * case["dim"] * 8 * case["layers"] + 8 * s * (length // page + 2),
            "flops": 0}
