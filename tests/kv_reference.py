"""Plain 64-bit forms of the paged KV cache's operators, for the tests.

Everything is written out from the definitions in include/hbl.h: codes bit by
bit, one sequence and one head at a time, sums in float64.
"""
import math

import torch

import hadamard_rotated_int4_b200 as hbl


def unpack(codes, D, bits):
    """[..., D*bits/8] bytes -> codes [..., D] (int64): code j at bits [bits*j, bits*j+bits)."""
    j = torch.arange(D, device=codes.device) * bits
    u = torch.zeros(*codes.shape[:-1], D, dtype=torch.int64, device=codes.device)
    for k in range(bits):
        at = j + k
        u |= ((codes[..., at // 8].long() >> (at % 8)) & 1) << k
    return u


def values(codes, scales, D, bits):
    return (unpack(codes, D, bits) - (1 << (bits - 1))).double() * scales.double()[..., None]


def quantise(x, bits, eps=1e-5):
    """Codes and scales of head rows: the quotient is one fp32 division, the
    product is rounded once, half to even."""
    qp = (1 << (bits - 1)) - 1
    gamma = x.float().abs().amax(-1, keepdim=True)
    den = gamma + torch.tensor(eps, dtype=torch.float32)
    inv = torch.where(den > 0, qp / den, torch.zeros_like(den))
    u = torch.round(x.double() * inv.double()).long() + (1 << (bits - 1))
    return u, (gamma / qp)[..., 0]


class Case:
    """A batch over a cache: `new` and `lens` per sequence, pages in a shuffled
    order, stored rows from random codes; slots past a sequence's end and unused
    pages hold 0xFF bytes and NaN scales."""

    def __init__(self, new, lens, heads=4, kv_heads=2, D=64, bits=4, page=16, seed=0, dev="cuda:0",
                 extra_rows=0, extra_pages=2, qscale=2.0, wide=None):
        g = torch.Generator().manual_seed(seed)
        self.new, self.lens, self.heads, self.D, self.bits, self.page = (list(new), list(lens),
                                                                         heads, D, bits, page)
        need = [-(-n // page) for n in lens]
        wide = max(need + [1]) if wide is None else wide
        pages = sum(need) + extra_pages
        order = torch.randperm(pages, generator=g).to(torch.int32)
        table = torch.full((len(lens), wide), 1 << 30, dtype=torch.int32)  # unused: out of range
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        self.rows = sum(new) + extra_rows
        self.cu = torch.tensor([0] + list(new)).cumsum(0).to(torch.int32).to(dev)
        self.kv_lens = torch.tensor(list(lens), dtype=torch.int32, device=dev)
        self.table = table.to(dev)
        shape = (pages, kv_heads, page)
        codes = [torch.full(shape + (D * bits // 8,), 255, dtype=torch.uint8) for _ in range(2)]
        scales = [torch.full(shape, math.nan) for _ in range(2)]
        for c, s in zip(codes, scales):
            for b, n in enumerate(lens):
                for i in range(need[b]):
                    m = min(page, n - i * page)
                    p = int(table[b, i])
                    c[p, :, :m] = torch.randint(0, 256, (kv_heads, m, D * bits // 8), generator=g,
                                                dtype=torch.uint8)
                    s[p, :, :m] = (torch.rand(kv_heads, m, generator=g) + 0.25) * \
                        (3.0 / (1 << (bits - 1)))
        self.cache = hbl.KvCache(codes[0].to(dev), scales[0].to(dev), codes[1].to(dev),
                                 scales[1].to(dev), D)
        self.q = (qscale * torch.randn(self.rows, heads, D, generator=g)).to(torch.bfloat16).to(dev)
        self.k, self.v = (torch.randn(self.rows, kv_heads, D, generator=g).to(torch.bfloat16).to(dev)
                          for _ in range(2))
        self.batch = (self.cu, self.kv_lens, self.table)

    def stored(self, b, h, which):
        """fp64 values [len, D] of sequence b, cached head h."""
        c = self.cache
        codes, scales = (c.k_codes, c.k_scales) if which == "k" else (c.v_codes, c.v_scales)
        pos = torch.arange(self.lens[b], device=codes.device)
        page = self.table[b].long()[pos // self.page]
        return values(codes[page, h, pos % self.page], scales[page, h, pos % self.page], self.D,
                      self.bits)


def attention(case, scale=None, causal=True, window=0):
    """(O, lse, tolerance of O, tolerance of lse), fp64 [rows, heads, ...]; rows of no
    sequence are NaN.

    Tolerances, to first order.  u = 2^-24 is an fp32 rounding's half step.
    A score is a sum of D exact products in fp32, in any order, by a unit that may
    truncate (4u a step): off by at most D * 4u * sum|q_d k_d|, scaled; two
    more roundings scale it.  e = that bound in nats, largest over the row's keys,
    plus 8u for the exponential itself, plus 2^-19 for the exponent's own
    rounding (|x| log2(e) below 64 in these cases, its half step 2^-19).
    A weight is then off by 2e relative (its own and the normaliser's) and by
    2^-11 for its rounding to fp16, and below the smallest normal number by half
    a step of 2^-24 against a largest weight of at least 1/2: 2^-24 of the largest
    weight * |v| for each key.  The weighted sum's accumulation: n keys, 4u each.
    O is rounded to bf16: 2^-8.
    lse is off by e, its own rounding (2^-23 |lse|) and the sum's (n * u)."""
    c, u = case, 2.0 ** -24
    dev = c.q.device
    group = c.heads // c.cache.num_kv_heads
    scale = c.D ** -0.5 if scale is None else scale
    O = torch.full((c.rows, c.heads, c.D), math.nan, dtype=torch.float64, device=dev)
    lse = torch.full((c.rows, c.heads), math.nan, dtype=torch.float64, device=dev)
    tol_O, tol_lse = torch.zeros_like(O), torch.zeros_like(lse)
    r0 = 0
    for b, (n, m) in enumerate(zip(c.new, c.lens)):
        pos = torch.arange(m - n, m, device=dev)[:, None]
        key = torch.arange(m, device=dev)[None]
        seen = torch.ones(n, m, dtype=torch.bool, device=dev)
        if causal:
            seen &= key <= pos
        if window > 0:
            seen &= key > pos - window
        for h in range(c.cache.num_kv_heads if n else 0):
            k, v = c.stored(b, h, "k"), c.stored(b, h, "v")
            for j in range(h * group, (h + 1) * group):
                q = c.q[r0:r0 + n, j].double()
                s = (scale * (q @ k.T)).masked_fill(~seen, -math.inf)
                z = torch.logsumexp(s, 1) if m else torch.full((n,), -math.inf, device=dev,
                                                               dtype=torch.float64)
                p = torch.where(seen, torch.exp(s - torch.where(z > -math.inf, z,
                                                               torch.zeros_like(z))[:, None]),
                                torch.zeros_like(s))
                O[r0:r0 + n, j], lse[r0:r0 + n, j] = p @ v, z
                if m == 0:
                    continue
                big = (abs(scale) * (q.abs() @ k.abs().T)).masked_fill(~seen, 0).amax(1)
                e = (4 * c.D + 2) * u * big + 8 * u + 2.0 ** -19
                top = (p[:, :, None] * v.abs()[None]).amax(1) if n * m * c.D < 1 << 27 else \
                    torch.stack([(p[i][:, None] * v.abs()).amax(0) for i in range(n)])
                tol_O[r0:r0 + n, j] = 2.0 ** -8 * O[r0:r0 + n, j].abs() + \
                    (2 * e + 2.0 ** -11 + 4 * m * u)[:, None] * (p @ v.abs()) + \
                    2.0 ** -24 * seen.sum(1)[:, None] * (2 * top.amax(1, keepdim=True))
                tol_lse[r0:r0 + n, j] = e + 2.0 ** -23 * z.abs().nan_to_num(posinf=0) + m * u
        r0 += n
    return O, lse, tol_O, tol_lse


def check_attention(case, got, lse=None, **kw):
    """Asserts a kernel's O (bf16) and lse against attention(); rows of no sequence are
    not looked at."""
    O, z, tol_O, tol_z = attention(case, **kw)
    n = sum(case.new)
    err = (got.double() - O)[:n].abs()
    assert torch.isfinite(got[:n].float()).all()
    over = (err - tol_O[:n])
    assert not n or float(over.max()) <= 0, (
        "O off by %g, %g allowed, at %s" % (float(err.flatten()[over.argmax()]),
                                            float(tol_O[:n].flatten()[over.argmax()]),
                                            torch.unravel_index(over.argmax(), over.shape)))
    if lse is not None:
        none = z[:n] == -math.inf
        assert torch.equal(lse[:n] == -math.inf, none)
        d = torch.where(none, torch.zeros_like(z[:n]), lse[:n].double() - z[:n]).abs()
        assert not n or bool((d <= tol_z[:n]).all()), float((d - tol_z[:n]).max())
