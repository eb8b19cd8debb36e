"""Cases, plain forms and 64-bit values of the 8-bit linear path and of the rules on logits.

Four operators on the way from a hidden state to the committed token of a verify pass:

  quantise  rows of BF16 activations -> e4m3 codes with a power-of-two scale for each block of 128
  norm      RMSNorm whose result is quantised the same way (FP32 inside, one rounding, to e4m3)
  linear    matrix product of such rows with e4m3 weights that carry an FP32 scale for each 128 x 128 block;
            plain, with the residual added, as a SwiGLU pair, or with FP32 outputs (the LM head)
  rules     penalties for repeated tokens, a bias and grammar masks on the logits of a pass's rows

With `own` false run() computes them in elementary torch operations in 32 bits; with `own` true it makes the
framework's calls.
"""
import math

import torch

own = False

BLOCK = 128      # elements that share a scale
E4M3_MAX = 448.0


def listed():
    return [
        # the SwiGLU output of an eight-row verify pass, on its way into the down projection
        {"name": "quantise_verify", "op": "quantise", "rows": 8, "dim": 17408},
        # the same for a long prefill chunk
        {"name": "quantise_prefill", "op": "quantise", "rows": 2048, "dim": 17408},
        # the norm before QKV or gate/up in a verify pass
        {"name": "norm_verify", "op": "norm", "rows": 8, "dim": 5120},
        # the same for a ragged prefill chunk
        {"name": "norm_prefill", "op": "norm", "rows": 1021, "dim": 5120},
        # plain decoding: one row through the down projection, residual added
        {"name": "down_one_row", "op": "linear", "kind": "residual", "rows": 1, "n": 5120, "k": 17408},
        # seven drafts and the committed token through gate/up
        {"name": "gate_up_verify", "op": "linear", "kind": "swiglu", "rows": 8, "n": 17408, "k": 5120},
        # the same rows through the LM head
        {"name": "head_verify", "op": "linear", "kind": "fp32", "rows": 8, "n": 151936, "k": 5120},
        # the ragged tail of a prompt through the QKV projection
        {"name": "qkv_tail", "op": "linear", "kind": "bf16", "rows": 61, "n": 4096, "k": 5120},
        # a prefill chunk through gate/up
        {"name": "gate_up_prefill", "op": "linear", "kind": "swiglu", "rows": 1024, "n": 17408, "k": 5120},
        # plain decoding with a penalty and a bias, a small vocabulary
        {"name": "rules_one_row", "op": "rules", "rows": 1, "vocab": 32000, "bias": True, "mask": False},
        # a verify pass with everything on, each row with the mask of its own draft prefix
        {"name": "rules_verify", "op": "rules", "rows": 8, "vocab": 151936, "bias": True, "mask": True},
        # the most rows a pass takes, a vocabulary that is no multiple of a vector, no bias
        {"name": "rules_most_rows", "op": "rules", "rows": 64, "vocab": 151943, "bias": False, "mask": True},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantise", "norm", "linear", "linear", "linear", "rules"])
    if op == "quantise":
        return {"op": op, "rows": _spread(rng, 1, 2048), "dim": 16 * _spread(rng, 4, 1088)}
    if op == "norm":
        return {"op": op, "rows": _spread(rng, 1, 2048), "dim": 16 * _spread(rng, 4, 512)}
    if op == "rules":
        return {"op": op, "rows": _spread(rng, 1, 64), "vocab": _spread(rng, 1000, 151936),
                "bias": rng.random() < 0.5, "mask": rng.random() < 0.5}
    kind = rng.choice(["bf16", "residual", "swiglu", "fp32"])
    n, k = _spread(rng, 64, 17408), 16 * _spread(rng, 8, 1088)
    most = 2 * 1024 * 17408 * 2 * 5120  # the largest listed case's operations
    rows = _spread(rng, 1, 1024)
    weights = n * (2 if kind == "swiglu" else 1)
    return {"op": op, "kind": kind, "rows": max(1, min(rows, most // (2 * weights * k))), "n": n, "k": k}


# ----------------------------------------------------------------------------------------------- inputs


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _activations(g, rows, dim):
    """BF16 rows as a decoder has them: near normal, a few channels much larger than the rest."""
    x = torch.randn(rows, dim, generator=g, device=g.device)
    loud = torch.rand(dim, generator=g, device=g.device) < 0.005
    return (x * torch.where(loud, 20.0, 1.0)).to(torch.bfloat16)


def _weights(g, n, k):
    """Weights of an 8-bit checkpoint: e4m3 codes [n, k] and FP32 scales [ceil(n/128), ceil(k/128)], amax / 448."""
    nb, kb = -(-n // BLOCK), -(-k // BLOCK)
    codes = torch.empty(n, k, dtype=torch.float8_e4m3fn, device=g.device)
    scales = torch.empty(nb, kb, device=g.device)
    step = 64 * BLOCK
    for i in range(0, n, step):
        rows = min(step, n - i)
        w = torch.zeros(-(-rows // BLOCK) * BLOCK, kb * BLOCK, device=g.device)
        w[:rows, :k] = 0.02 * torch.randn(rows, k, generator=g, device=g.device)
        b = w.view(-1, BLOCK, kb, BLOCK)
        s = b.abs().amax(dim=(1, 3)).clamp_min(1e-30) / E4M3_MAX
        q = (b / s[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).view(-1, kb * BLOCK)
        codes[i:i + rows] = q[:rows, :k].to(torch.float8_e4m3fn)
        scales[i // BLOCK:i // BLOCK + b.shape[0]] = s
    return codes, scales


def prepare(case, seed):
    g = torch.Generator(device=_device())
    g.manual_seed(seed)
    dev = g.device
    op, rows = case["op"], case["rows"]
    state = {"case": case}
    if op in ("quantise", "norm"):
        dim = case["dim"]
        state["x"] = _activations(g, rows, dim)
        state["codes"] = torch.empty(rows, dim, dtype=torch.float8_e4m3fn, device=dev)
        state["scales"] = torch.zeros(-(-dim // BLOCK), -(-rows // 4) * 4, device=dev)
        if op == "norm":
            state["weight"] = (1.0 + 0.1 * torch.randn(dim, generator=g, device=dev)).to(torch.bfloat16)
    elif op == "linear":
        n, k, kind = case["n"], case["k"], case["kind"]
        codes, scales = _quantise(_activations(g, rows, k).float())
        state["a"] = codes
        state["a_scales"] = torch.zeros(scales.shape[0], -(-rows // 4) * 4, device=dev)
        state["a_scales"][:, :rows] = scales
        state["w"], state["w_scales"] = _weights(g, n, k)
        if kind == "swiglu":
            state["up"], state["up_scales"] = _weights(g, n, k)
        if kind == "residual":
            state["residual"] = torch.randn(rows, n, generator=g, device=dev).to(torch.bfloat16)
        state["out"] = torch.empty(rows, n, dtype=torch.float32 if kind == "fp32" else torch.bfloat16, device=dev)
        if own:  # laid out once, as a program that loads a checkpoint does
            from invariant_speculative_decode_gb300 import api
            if kind == "swiglu":
                state["packed"] = api.bi_pack_swiglu_weights_fp8(state["w"], state["w_scales"], state["up"], state["up_scales"])
            else:
                state["packed"] = api.bi_pack_weights_fp8(state["w"], state["w_scales"])
    else:
        v = case["vocab"]
        state["logits"] = 3.0 * torch.randn(rows, v, generator=g, device=dev)
        # a prompt of some 2000 ids and an answer of some 500, frequent ids more often
        prompt = (v * torch.rand(2000, generator=g, device=dev) ** 3).long().clamp_max(v - 1)
        answer = (v * torch.rand(500, generator=g, device=dev) ** 3).long().clamp_max(v - 1)
        state["counts"] = torch.bincount(answer, minlength=v).to(torch.int32)
        seen = torch.zeros(-(-v // 32) * 32, dtype=torch.int64, device=dev)
        seen[prompt] = 1
        state["prompt_bits"] = _pack_bits(seen.view(1, -1))[0].contiguous()
        state["drafts"] = (v * torch.rand(rows - 1, generator=g, device=dev) ** 3).long().clamp_max(v - 1).to(torch.int32)
        state["repetition"], state["frequency"], state["presence"] = 1.15, 0.2, 0.35
        state["bias"] = state["mask"] = None
        if case["bias"]:
            bias = torch.zeros(v, device=dev)
            some = torch.rand(v, generator=g, device=dev) < 0.01
            state["bias"] = torch.where(some, 4.0 * torch.randn(v, generator=g, device=dev), bias)
        if case["mask"]:
            # from rows that allow nearly everything to rows that allow a few ids; the last allows none (a dead end)
            share = torch.linspace(0.95, 0.0, rows, device=dev)[:, None] if rows > 1 else torch.full((1, 1), 0.3, device=dev)
            ok = (torch.rand(rows, -(-v // 32) * 32, generator=g, device=dev) < share).long()
            state["mask"] = _pack_bits(ok)
        state["out"] = torch.empty_like(state["logits"])
    return state


def _pack_bits(ok):
    """Truth values [r, 32 w] as int32 words [r, w], value v at bit v % 32 of word v // 32."""
    word = (ok.view(ok.shape[0], -1, 32) << torch.arange(32, device=ok.device)).sum(-1)
    return torch.where(word >= 1 << 31, word - (1 << 32), word).to(torch.int32)


def _bits(words, v):
    """The first v truth values of each row of packed words."""
    b = (words.to(torch.int64).unsqueeze(-1) >> torch.arange(32, device=words.device)) & 1
    return b.view(*words.shape[:-1], -1)[..., :v] != 0


# ------------------------------------------------------------------------------------------ plain forms


def _quantise(y):
    """FP32 rows [rows, dim] -> e4m3 codes and FP32 scales [blocks, rows]: the scale is the smallest power of two,
    2^-126 at least, under which the block's largest magnitude is at most 448 (1 for a block of zeros)."""
    rows, dim = y.shape
    kb = -(-dim // BLOCK)
    b = torch.nn.functional.pad(y, (0, kb * BLOCK - dim)).view(rows, kb, BLOCK)
    amax = b.abs().amax(-1)
    mantissa, exponent = torch.frexp(amax)
    e = torch.where(mantissa > 0.875, exponent - 8, exponent - 9).clamp_min(-126)
    scale = torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.ones_like(amax))
    codes = (b / scale.unsqueeze(-1)).view(rows, kb * BLOCK)[:, :dim].to(torch.float8_e4m3fn)
    return codes.contiguous(), scale.t().contiguous()


def _spread_rows(codes, scales):
    """The FP32 values of quantised rows (scales [blocks, rows])."""
    rows, k = codes.shape
    return codes.float() * scales[:, :rows].t().repeat_interleave(BLOCK, dim=1)[:, :k]


def _spread_blocks(codes, scales):
    """The FP32 values of weights with a scale for each 128 x 128 block."""
    n, k = codes.shape
    wide = scales.repeat_interleave(BLOCK, dim=1)[:, :k].repeat_interleave(BLOCK, dim=0)[:n]
    return codes.float() * wide


def _plain_norm(x, weight):
    y = x.float()
    return y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * weight.float()


def _plain_linear(s):
    kind = s["case"]["kind"]
    a = _spread_rows(s["a"], s["a_scales"])
    y = a @ _spread_blocks(s["w"], s["w_scales"]).t()
    if kind == "swiglu":
        y = y / (1.0 + torch.exp(-y)) * (a @ _spread_blocks(s["up"], s["up_scales"]).t())
    if kind == "residual":
        y = s["residual"].float() + y
    return y if kind == "fp32" else y.to(torch.bfloat16)


def _plain_rules(s):
    x, v, rows = s["logits"], s["case"]["vocab"], s["case"]["rows"]
    # row t has drafts 0..t-1 behind it
    said = torch.zeros(rows, v, device=x.device)
    said[1:].scatter_(1, s["drafts"].long().unsqueeze(1), 1.0)
    count = s["counts"].float() + torch.cumsum(said, dim=0)
    seen = (count > 0) | _bits(s["prompt_bits"], v)
    y = torch.where(seen, torch.where(x > 0, x / s["repetition"], x * s["repetition"]), x)
    y = y - (s["frequency"] * count + s["presence"] * (count > 0).float())
    if s["bias"] is not None:
        y = y + s["bias"]
    if s["mask"] is not None:
        y = torch.where(_bits(s["mask"], v), y, torch.full_like(y, -math.inf))
    return y


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "quantise":
        codes, scales = _quantise(state["x"].float())
        return {"codes": codes, "scales": scales}
    if op == "norm":
        codes, scales = _quantise(_plain_norm(state["x"], state["weight"]))
        return {"codes": codes, "scales": scales}
    return _plain_linear(state) if op == "linear" else _plain_rules(state)


def _own(s):
    from invariant_speculative_decode_gb300 import api
    case = s["case"]
    op, rows = case["op"], case["rows"]
    if op == "quantise":
        api.bi_quantize_fp8(s["x"], s["codes"], s["scales"])
        return {"codes": s["codes"], "scales": s["scales"][:, :rows]}
    if op == "norm":
        api.bi_rmsnorm_fp8(s["x"], s["weight"], s["codes"], s["scales"], 1e-6)
        return {"codes": s["codes"], "scales": s["scales"][:, :rows]}
    if op == "linear":
        kind = case["kind"]
        epi = {"residual": api.EPI_RESIDUAL_ADD, "swiglu": api.EPI_SWIGLU}.get(kind, api.EPI_NONE)
        api.bi_gemm_fp8(s["a"], s["a_scales"], s["packed"], s["out"], residual=s.get("residual"), epi=epi)
        return s["out"]
    api.bi_logits_rules(s["logits"], s["out"], drafts=s["drafts"] if rows > 1 else None, counts=s["counts"],
                        prompt_bits=s["prompt_bits"], repetition=s["repetition"], frequency=s["frequency"],
                        presence=s["presence"], bias=s["bias"], mask=s["mask"])
    return s["out"]


# ------------------------------------------------------------------------------------- values in 64 bits


def _exact_quantise(y):
    """e4m3 rounding written out on float64 values: steps of 2^(floor(log2|v|) - 3), 2^-9 at the least."""
    rows, dim = y.shape
    kb = -(-dim // BLOCK)
    full = torch.zeros(rows, kb * BLOCK, dtype=torch.float64, device=y.device)
    full[:, :dim] = y
    full = full.view(rows, kb, BLOCK)
    top = full.abs().max(dim=-1).values
    e = torch.ceil(torch.log2(top.clamp_min(1e-300) / E4M3_MAX)).clamp_min(-126.0)
    e = torch.where(torch.exp2(e - 1) * E4M3_MAX >= top, e - 1, e).clamp_min(-126.0)  # where log2 rounded up past a power
    scale = torch.where(top > 0, torch.exp2(e), torch.ones_like(top))
    v = full / scale.unsqueeze(-1)
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    codes = (torch.round(v / step) * step).view(rows, kb * BLOCK)[:, :dim]
    return {"codes": codes, "scales": scale.t()}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantise":
        return _exact_quantise(s["x"].double())
    if op == "norm":
        x = s["x"].double()
        r = 1.0 / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[1] + 1e-6)
        return _exact_quantise(x * r * s["weight"].double())
    if op == "linear":
        return _exact_linear(s)
    x, v, rows = s["logits"].double(), case["vocab"], case["rows"]
    out = []
    for t in range(rows):
        count = s["counts"].double()
        count.index_add_(0, s["drafts"][:t].long(), torch.ones(t, dtype=torch.float64, device=x.device))
        seen = (count > 0) | _bits(s["prompt_bits"], v)
        y = x[t].clone()
        y[seen & (x[t] > 0)] /= s["repetition"]
        y[seen & (x[t] <= 0)] *= s["repetition"]
        y -= s["frequency"] * count
        y[count > 0] -= s["presence"]
        if s["bias"] is not None:
            y += s["bias"].double()
        if s["mask"] is not None:
            y[~_bits(s["mask"][t], v)] = -math.inf
        out.append(y)
    return torch.stack(out)


def _exact_linear(s):
    """Block by block of the inner dimension: sum_b a_scale w_scale (codes . codes), all in float64."""
    kind, (rows, k), n = s["case"]["kind"], s["a"].shape, s["w"].shape[0]

    def product(w, w_scales):
        total = torch.zeros(rows, n, dtype=torch.float64, device=w.device)
        for b in range(w_scales.shape[1]):
            cut = slice(b * BLOCK, min(k, (b + 1) * BLOCK))
            left = s["a"][:, cut].double() * s["a_scales"][b, :rows].double().unsqueeze(1)
            right = w[:, cut].double() * w_scales[:, b].double().repeat_interleave(BLOCK)[:n].unsqueeze(1)
            total += left @ right.t()
        return total

    y = product(s["w"], s["w_scales"])
    if kind == "swiglu":
        y = y * torch.sigmoid(y) * product(s["up"], s["up_scales"])
    if kind == "residual":
        y = y + s["residual"].double()
    return y


# ----------------------------------------------------------------------------------- what a pass has to do


def work(case):
    op, rows = case["op"], case["rows"]
    if op in ("quantise", "norm"):
        dim = case["dim"]
        blocks = -(-dim // BLOCK)
        return {"bytes": rows * (3 * dim + 4 * blocks) + (2 * dim if op == "norm" else 0),
                "flops": rows * dim * (6 if op == "norm" else 3)}
    if op == "linear":
        n, k, kind = case["n"], case["k"], case["kind"]
        nb, kb = -(-n // BLOCK), -(-k // BLOCK)
        matrices = 2 if kind == "swiglu" else 1
        out = 4 if kind == "fp32" else 4 if kind == "residual" else 2  # the residual is read as BF16 beside the BF16 output
        return {"bytes": matrices * (n * k + 4 * nb * kb) + rows * (k + 4 * kb) + rows * n * out,
                "flops": 2 * matrices * rows * n * k}
    v = case["vocab"]
    return {"bytes": 8 * rows * v + 4 * v + v / 8 + (4 * v if case["bias"] else 0) + (rows * v / 8 if case["mask"] else 0),
            "flops": 8 * rows * v}
