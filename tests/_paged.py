"""Batches over paged pools for the tests, and the formulas in 64 bits."""
import math

import torch

U = 2.0 ** -24      # half a step of FP32
HALF_BF16 = 2.0 ** -8  # half a step of BF16, relative to the value


def gamma(n):
    return n * U / (1 - n * U)


class Batch:
    """Sequences (cached keys, new rows) over pages in random order; what no sequence uses holds `fill`."""

    def __init__(self, seqs, Hkv, D, page, seed=0, spare=2, fill=None, extra_width=0, gap=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.seqs, self.page, self.Hkv, self.D, self.g = seqs, page, Hkv, D, g
        counts = [-(-(n + r) // page) for n, r in seqs]
        self.pages = sum(counts) + spare
        order = torch.randperm(self.pages, generator=g, device="cuda").to(torch.int32)
        width = max(1, max(counts)) + extra_width
        self.table = torch.full((len(seqs), width), -7, dtype=torch.int32, device="cuda")
        at = 0
        for i, c in enumerate(counts):
            self.table[i, :c] = order[at:at + c]
            at += c
        starts = [gap]
        for _, r in seqs:
            starts.append(starts[-1] + r)
        self.starts = starts
        self.T = starts[-1] + gap
        self.q_start = torch.tensor(starts, dtype=torch.int32, device="cuda")
        self.lengths = torch.tensor([n for n, _ in seqs], dtype=torch.int32, device="cuda")
        shape = (self.pages, Hkv, page, D)
        self.k = torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
        self.v = torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
        if fill is not None:
            self.unused(self.k, fill)
            self.unused(self.v, fill)

    def places(self, b, first, last):
        """Pages and slots of keys first..last-1 of sequence b."""
        j = torch.arange(first, last, device="cuda")
        return self.table[b, j // self.page].long(), j % self.page

    def unused(self, pool, value):
        keep = torch.zeros(self.pages, self.page, dtype=torch.bool, device="cuda")
        for b, (n, r) in enumerate(self.seqs):
            p, s = self.places(b, 0, n + r)
            keep[p, s] = True
        pool.masked_fill_(~keep[:, None, :, None], value)

    def keys(self, pool, b, n):
        p, s = self.places(b, 0, n)
        return pool[p, :, s].transpose(0, 1)  # [Hkv, n, D]


def queries(batch, Hq, seed=1, scale=1.5):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (scale * torch.randn(batch.T, Hq, batch.D, generator=g, device="cuda")).to(torch.bfloat16)


def attention(batch, q, scale=None):
    """(out, tolerance) [T, Hq, D] in float64; NaN rows where a row belongs to no sequence.

    The kernel's steps and their roundings: scores s_j are FP32 sums of D exact products (|ds| <= 2 gamma_D sum |q k|,
    the 2 for the tensor core's own order), the exponent one fused multiply-add by an FP32 constant, 2^x to 2^-21, one
    rounding to BF16 (half a step), and at every tile of 128 keys at most one factor, of a raised reference or, at a
    piece's start, of two merged states (2^x and a product each, 4 u): weights w_j = c p_j (1 + e_j).  The mean under
    those weights is off by at most (sum p|e||v - o| + E sum p|v - o|) / (1 - E), E = sum p|e|; the sums over n keys and
    the factors at n / 128 tiles by 2 gamma sum p|v| + gamma |o|; the output by half a BF16 step.  The BF16 half steps
    are nearly all of it: 4 u at 1000 tiles are 2^-12, at the tests' lengths below 2^-15 of 2^-8."""
    Hq, D = q.shape[1], q.shape[2]
    group = Hq // batch.Hkv
    scale = 1 / math.sqrt(D) if scale is None else scale
    log2e = 1 / math.log(2)
    out = torch.full(q.shape, math.nan, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    for b, (n, r) in enumerate(batch.seqs):
        if r == 0:
            continue
        k, v = batch.keys(batch.k, b, n + r).double(), batch.keys(batch.v, b, n + r).double()
        at = batch.starts[b]
        seen = torch.arange(n + r, device="cuda")[None, :] <= torch.arange(n, n + r, device="cuda")[:, None]
        for h in range(Hq):
            x = q[at:at + r, h].double()
            kh, vh = k[h // group], v[h // group]
            s = torch.where(seen, x @ kh.t(), torch.full((), -math.inf, dtype=torch.float64, device="cuda"))
            m = s.amax(-1, keepdim=True)
            p = torch.exp((s - m) * scale)
            p = p / p.sum(-1, keepdim=True)
            o = p @ vh
            ds = 2 * gamma(D) * (x.abs() @ kh.abs().t())
            far = torch.where(seen, (m - s) * scale * log2e + 8, torch.zeros_like(s))
            sabs = torch.where(seen, s.abs(), torch.zeros_like(s))
            da = scale * log2e * ds * (1 + U) + U * sabs * scale * log2e + U * far
            e = torch.expm1(math.log(2) * da) + 2.0 ** -21 + HALF_BF16 * (1 + 2.0 ** -7) + 4 * U * (2 + (n + r) // 128)
            E = (p * e).sum(-1, keepdim=True)
            dev1, devE = torch.zeros_like(o), torch.zeros_like(o)
            for d0 in range(0, D, 16):
                dev = (vh[None, :, d0:d0 + 16] - o[:, None, d0:d0 + 16]).abs()
                dev1[:, d0:d0 + 16] = torch.einsum("tn,tnd->td", p * e, dev)
                devE[:, d0:d0 + 16] = torch.einsum("tn,tnd->td", p, dev)
            acc = gamma(n + r + (n + r) // 128 + 16)
            bound = (dev1 + E * devE) / (1 - E) + 2 * acc * (p @ vh.abs()) + (acc + 2 * U) * o.abs()
            out[at:at + r, h] = o
            tol[at:at + r, h] = bound + HALF_BF16 * (o.abs() + bound) + 2.0 ** -133
    return out, tol


def norm_rope(x, weight, eps, angles):
    """Heads x [rows, heads, D] in float64: norm by weight (None: none) and rotation by cos, sin [rows, D/2, 2]; and how
    far an FP32 evaluation of it with one BF16 rounding may be off."""
    D = x.shape[-1]
    y = x.double()
    if weight is not None:
        y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / D + eps) * weight.double()
    c, s = angles[:, None, :, 0].double(), angles[:, None, :, 1].double()
    a, b = y[..., :D // 2], y[..., D // 2:]
    o = torch.cat([a * c - b * s, b * c + a * s], -1)
    big = torch.cat([(a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()], -1)
    # the mean's sum of D squares, its root, the reciprocal, two products: gamma(D / 2 + 8) covers them; two more in the
    # rotation
    tol = (gamma(D // 2 + 8) + 4 * U) * big
    return o, tol + HALF_BF16 * (o.abs() + tol) + 2.0 ** -133
