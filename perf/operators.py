"""The paged low-bit KV cache's operators and the calls that time them.

Three operators, on a cache of `bits`-bit codes (2, 3, 4 or 8) with one fp32
scale per token and head, kept in pages that a block table strings together:

  write      quantise the new tokens' K and V and store them in their pages
  read       dequantise a range of each sequence's tokens back to rows
  attention  attend from the new tokens to everything their sequence has cached

A batch is packed: sequence b's new rows are rows cu[b] to cu[b + 1], its
length with them is kv_lens[b], so its row i stands at position
kv_lens[b] - (cu[b + 1] - cu[b]) + i.

Plain forms are elementary torch operations in fp32 (fp64 where a code is
rounded); with `own` set, run() makes the library's calls instead.
"""
import math
import random

import torch

own = False

EPS = 1e-5


# ------------------------------------------------------------------- cases

def _case(name, op, bits, heads, kv_heads, dim, page, seqs, rows, kv, lens, window=0, causal=True,
          fp32=False, fixed=False):
    c = {"op": op, "bits": bits, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page,
         "seqs": seqs, "rows": rows, "kv": kv, "lens": lens, "window": window, "causal": causal,
         "fp32": fp32, "fixed": fixed}
    if name:
        c["name"] = name
    return c


def listed():
    """`rows` and `kv` bound the new rows and the length of each of `seqs`
    sequences; `fixed`: every sequence has exactly those, else `lens` seeds a
    ragged draw below them (empty sequences among them)."""
    return [
        # a decoding step of 64 sequences stores its 64 tokens: all latency
        _case("write_step", "write", 4, 8, 8, 128, 64, 64, 1, 4000, 1, fixed=True),
        # prompts of 8192 tokens in all, the K and V halves of the benchmark's 96-head Q/K/V states
        _case("write_prompt", "write", 3, 32, 32, 128, 64, 4, 2048, 2048, 2, fixed=True),
        # ragged prompts, an odd head count, small pages; the rows come back in fp32
        _case("write_ragged", "write", 8, 5, 5, 64, 16, 37, 301, 900, 3, fp32=True),
        # one whole long sequence taken out of the cache
        _case("read_long", "read", 4, 8, 8, 128, 64, 1, 131071, 131071, 4, fixed=True),
        # the tails of 48 sequences, heads of 256, in fp32
        _case("read_ragged", "read", 2, 2, 2, 256, 32, 48, 700, 2500, 5, fp32=True),
        # a single user's next token, early on: latency
        _case("decode_one", "attention", 4, 32, 8, 128, 64, 1, 1, 517, 6, fixed=True),
        # a serving step: 64 sequences of uneven lengths, grouped heads
        _case("decode_batch", "attention", 4, 32, 8, 128, 64, 64, 1, 8192, 7),
        # two users far into a long context, on the 3-bit cache
        _case("decode_long", "attention", 3, 32, 8, 128, 64, 2, 1, 131071, 8, fixed=True),
        # five drafted tokens a sequence to verify, a head of its own for each query head (hidden 2048)
        _case("verify", "attention", 8, 32, 32, 64, 16, 16, 5, 4100, 9, fixed=True),
        # a whole prompt against itself: the largest
        _case("chunk_prompt", "attention", 4, 32, 8, 128, 64, 1, 8192, 8192, 10, fixed=True),
        # a step that mixes chunks of prompts with decoding sequences
        _case("chunk_mixed", "attention", 8, 32, 8, 128, 64, 6, 700, 12000, 11),
        # a sliding window, wide heads, the 2-bit cache
        _case("chunk_window", "attention", 2, 16, 2, 256, 32, 2, 2000, 6001, 12, window=1025,
              fixed=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    """One more case of the same ranges; its work stays below the largest listed one's."""
    op = rng.choice(("write", "read", "attention", "attention", "attention"))
    while True:
        bits, dim = rng.choice((2, 3, 4, 8)), rng.choice((32, 64, 128, 128, 256))
        kv_heads = rng.randint(1, 16)
        group = rng.choice((1, 2, 3, 4, 5, 7, 8)) if op == "attention" else 1
        page = rng.choice((16, 32, 48, 64, 128))
        seqs = _log(rng, 1, 64)
        kv = _log(rng, 1, 131072)
        if op == "attention":
            kind = rng.choice(("step", "few", "chunk"))
            rows = 1 if kind == "step" else rng.randint(2, 8) if kind == "few" else _log(rng, 9, 8192)
            rows = min(rows, kv)
            window = rng.choice((0, 0, 0, _log(rng, 1, 8192)))
            causal = rng.random() < 0.9
        else:
            rows, window, causal = _log(rng, 1, kv), 0, True
        c = _case("", op, bits, kv_heads * group, kv_heads, dim, page, seqs, rows, kv,
                  rng.randrange(1 << 30), window, causal, op != "attention" and rng.random() < 0.5,
                  rng.random() < 0.3)
        # what the plain form holds at once, and what the path has to do, both bounded
        scores = seqs * kv_heads * group * rows * kv if op == "attention" else 0
        cells = seqs * (kv + page) * kv_heads * dim
        if scores > 2 ** 31 or cells > 3 * 2 ** 28:
            continue
        w = work(c)
        if w["bytes"] > 6.5e8 or w["flops"] > 5e11:
            continue
        return c


def _lens(case):
    """(new rows, length) of each sequence, from the case alone."""
    r = random.Random(case["lens"])
    b, rows, kv = case["seqs"], case["rows"], case["kv"]
    if case["fixed"]:
        return [rows] * b, [kv] * b
    n, m = [], []
    for i in range(b):
        length = kv if i == 0 else r.randint(max(1, kv // 8), kv)
        new = min(length, rows if i == 0 or rows == 1 else
                  r.choice((0, 1, r.randint(1, rows), r.randint(1, rows), rows)))
        n.append(new)
        m.append(length)
    return n, m


def _pairs(case, new, length):
    """(query, key) pairs that one sequence's mask leaves, and its first visible key."""
    if new == 0:
        return 0, length
    w = case["window"] if case["window"] > 0 else 1 << 40
    first = max(0, length - new - w + 1)
    total = 0
    if case["causal"]:
        # row at position p sees min(p + 1, w) keys
        lo, hi = length - new, length - 1
        full = max(0, hi - max(lo, w - 1) + 1) if w <= hi + 1 else 0
        total = full * w if full else 0
        top = min(hi, w - 2)
        if top >= lo:
            total += (lo + 1 + top + 1) * (top - lo + 1) // 2
    else:
        # row at position p sees keys max(0, p - w + 1) .. length - 1
        for p in (range(length - new, length) if w < length else ()):
            total += length - max(0, p - w + 1)
        if w >= length:
            total = new * length
    return total, first


def work(case):
    new, length = _lens(case)
    t, d, kvh = sum(new), case["dim"], case["kv_heads"]
    row = d * case["bits"] / 8 + 4  # one head's codes and scale
    out = 4 if case["fp32"] else 2
    if case["op"] == "write":  # K, V in; codes and scales out; the values they stand for
        return {"bytes": 2 * t * kvh * (2 * d + row + out * d), "flops": 0}
    if case["op"] == "read":
        return {"bytes": 2 * t * kvh * (row + out * d), "flops": 0}
    seen = pairs = 0
    for n, m in zip(new, length):
        p, first = _pairs(case, n, m)
        pairs += p
        seen += m - first if n else 0
    return {"bytes": 2 * seen * kvh * row + t * case["heads"] * (4 * d + 4),
            "flops": 4 * pairs * case["heads"] * d}


# ------------------------------------------------------------- plain forms

def _quantise(x, bits):
    """Rows of the last dimension -> (codes int32 in [0, 2^bits), scales fp32).
    The quotient is one fp32 division; x * inv is rounded once, half to even."""
    qp = (1 << (bits - 1)) - 1
    gamma = x.float().abs().amax(-1)
    den = gamma + torch.tensor(EPS, dtype=torch.float32, device=x.device)
    inv = torch.where(den > 0, qp / den, torch.zeros_like(den))
    q = torch.round(x.double() * inv.double()[..., None]).clamp(-qp - 1, qp)
    return (q + (qp + 1)).to(torch.int32), gamma / qp


def _pack(u, bits):
    """Codes [..., D] -> bytes [..., D * bits / 8]: code j of a group of 32 at
    bits [bits * j, bits * j + bits) of the group's little-endian integer."""
    planes = (u[..., None] >> torch.arange(bits, device=u.device, dtype=u.dtype)) & 1
    planes = planes.to(torch.uint8).reshape(*u.shape[:-1], u.shape[-1] * bits // 8, 8)
    weights = torch.tensor([1, 2, 4, 8, 16, 32, 64, 128], dtype=torch.uint8, device=u.device)
    return (planes * weights).sum(-1, dtype=torch.uint8)


def _unpack(codes, bits, d):
    """Bytes [..., D * bits / 8] -> codes as fp32 [..., D]."""
    if bits == 8:
        return codes.float()
    if bits in (2, 4):
        shift = torch.arange(0, 8, bits, device=codes.device, dtype=torch.uint8)
        return ((codes[..., None] >> shift) & ((1 << bits) - 1)).flatten(-2).float()
    at = torch.arange(d, device=codes.device) * bits
    wide = torch.nn.functional.pad(codes, (0, 1)).to(torch.int16)
    two = wide[..., at // 8] | (wide[..., at // 8 + 1] << 8)
    return ((two >> (at % 8).to(torch.int16)) & 7).float()


def _rows(s):
    """Of each packed row: its sequence, its position, its page and slot there."""
    c = s["case"]
    t = torch.arange(s["total"], device=s["cu"].device)
    seq = torch.searchsorted(s["cu"].long(), t, right=True) - 1
    pos = s["kv_lens"].long()[seq] - s["cu"].long()[seq + 1] + t
    return seq, pos, s["table"].long()[seq, pos // c["page"]], pos % c["page"]


def _plain_write(s):
    c = s["case"]
    _, _, page, slot = _rows(s)
    for x, codes, scales in ((s["k"], s["k_codes"], s["k_scales"]),
                             (s["v"], s["v_codes"], s["v_scales"])):
        u, scale = _quantise(x, c["bits"])
        codes[page, :, slot] = _pack(u, c["bits"])
        scales[page, :, slot] = scale


def _plain_read(s):
    c = s["case"]
    _, _, page, slot = _rows(s)
    half = 1 << (c["bits"] - 1)
    dtype = torch.float32 if c["fp32"] else torch.bfloat16
    value = lambda codes, scales: ((_unpack(codes[page, :, slot], c["bits"], c["dim"]) - half) *
                                   scales[page, :, slot][..., None]).to(dtype)
    return value(s["k_codes"], s["k_scales"]), value(s["v_codes"], s["v_scales"])


def _plain_attention(s):
    c = s["case"]
    dev, b, d = s["q"].device, c["seqs"], c["dim"]
    kvh, g, n, m = c["kv_heads"], c["heads"] // c["kv_heads"], s["max_rows"], s["max_kv"]
    half = 1 << (c["bits"] - 1)
    cu, lens = s["cu"].long(), s["kv_lens"].long()
    pos = torch.arange(m, device=dev)
    page = s["table"].long()[:, pos // c["page"]]
    slot = (pos % c["page"]).expand(b, m)
    value = lambda codes, scales: ((_unpack(codes[page, :, slot], c["bits"], d) - half) *
                                   scales[page, :, slot][..., None]).transpose(1, 2)
    i = torch.arange(n, device=dev)
    at = (cu[:-1, None] + i).clamp(max=max(0, s["total"] - 1))
    q = s["q"][at].float().reshape(b, n, kvh, g, d).permute(0, 2, 3, 1, 4).reshape(b, kvh, g * n, d)
    x = torch.matmul(q, value(s["k_codes"], s["k_scales"]).transpose(2, 3)).mul_(1 / math.sqrt(d))
    p = (lens - cu[1:] + cu[:-1])[:, None] + i  # each row's position
    seen = pos < lens[:, None, None]
    if c["causal"]:
        seen = seen & (pos <= p[..., None])
    if c["window"] > 0:
        seen = seen & (pos > p[..., None] - c["window"])
    x = x.view(b, kvh, g, n, m).masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(top > -math.inf, top, torch.zeros_like(top))).exp_()
    total = x.sum(-1, keepdim=True)
    y = torch.matmul(x.view(b, kvh, g * n, m), value(s["v_codes"], s["v_scales"]))
    y = y.view(b, kvh, g, n, d) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (total.log() + top).squeeze(-1)
    seq = torch.searchsorted(cu, torch.arange(s["total"], device=dev), right=True) - 1
    row = torch.arange(s["total"], device=dev) - cu[seq]
    take = lambda z: z.permute(0, 3, 1, 2, *range(4, z.dim()))[seq, row].flatten(1, 2)
    return take(y).to(torch.bfloat16), take(lse)


# ------------------------------------------------------------------- a case

def prepare(case, seed):
    """The batch's descriptors, the cache as earlier steps left it, the new rows."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    c = dict(case)
    new, length = _lens(c)
    page, kvh, d, bits = c["page"], c["kv_heads"], c["dim"], c["bits"]
    wide = max(-(-m // page) for m in length)
    pages = sum(-(-m // page) for m in length) + 3
    order = torch.randperm(pages, device=dev, generator=g).to(torch.int32)
    # every entry is a page of the pool; those past a sequence's end are never used
    used = torch.tensor([0] + [-(-m // page) for m in length], device=dev).cumsum(0)
    at = (used[:-1, None] + torch.arange(wide, device=dev)).clamp(max=pages - 1)
    s = {"case": c, "total": sum(new), "max_rows": max(max(new), 1), "max_kv": max(length),
         "cu": torch.tensor([0] + new, device=dev).cumsum(0).to(torch.int32),
         "kv_lens": torch.tensor(length, device=dev, dtype=torch.int32),
         "table": order[at].contiguous()}
    # a few channels stand out, as they do in keys; values are even
    stand = 1 + 4 * (torch.rand(kvh, 1, d, device=dev, generator=g) < 0.04).float()

    def states(rows, heads, channels):
        x = torch.randn(rows, heads, d, device=dev, generator=g)
        return (x * channels.transpose(0, 1) if channels is not None else x).to(torch.bfloat16)

    if c["op"] == "write":
        # slices of one projection's output, as a layer has them
        x = torch.cat((states(s["total"], kvh, stand), states(s["total"], kvh, None)), 1)
        s["k"], s["v"] = x[:, :kvh], x[:, kvh:]
        s["k_codes"], s["v_codes"] = (torch.zeros(pages, kvh, page, d * bits // 8, device=dev,
                                                  dtype=torch.uint8) for _ in range(2))
        s["k_scales"], s["v_scales"] = (torch.zeros(pages, kvh, page, device=dev)
                                        for _ in range(2))
    else:
        for name, channels in (("k", stand), ("v", None)):
            codes = torch.empty(pages, kvh, page, d * bits // 8, device=dev, dtype=torch.uint8)
            scales = torch.empty(pages, kvh, page, device=dev)
            step = max(1, (1 << 26) // (kvh * page * d))
            for i in range(0, pages, step):
                x = states(min(step, pages - i) * page, kvh, channels)
                x = x.view(-1, page, kvh, d).transpose(1, 2)
                u, scale = _quantise(x, bits)
                codes[i:i + step], scales[i:i + step] = _pack(u, bits), scale
            s[name + "_codes"], s[name + "_scales"] = codes, scales
    if c["op"] == "attention":
        s["q"] = (2 * torch.randn(s["total"], c["heads"], d, device=dev, generator=g)).to(
            torch.bfloat16)
    return s


def run(s):
    """One call as a program makes it.  A write is followed by the read of its
    rows: their packed codes are returned as the values they stand for."""
    c = s["case"]
    if not own:
        if c["op"] == "attention":
            return _plain_attention(s)
        if c["op"] == "write":
            _plain_write(s)
        return _plain_read(s)
    import hadamard_rotated_int4_b200 as hbl

    cache = hbl.KvCache(s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], c["dim"])
    batch = (s["cu"], s["kv_lens"], s["table"])
    if c["op"] == "attention":
        return hbl.kv_attention(s["q"], cache, *batch, max_rows=s["max_rows"], max_kv=s["max_kv"],
                                causal=c["causal"], window=c["window"], want_lse=True)
    if c["op"] == "write":
        hbl.kv_cache_write(cache, s["k"], s["v"], *batch, eps=EPS)
    return hbl.kv_cache_read(cache, *batch, s["total"],
                             dtype=torch.float32 if c["fp32"] else torch.bfloat16)


# -------------------------------------------------------------------- exact

def _values64(codes, scales, bits, d):
    """What stored rows stand for, in fp64, bit by bit from the layout's definition."""
    j = torch.arange(d, device=codes.device)
    u = torch.zeros(*codes.shape[:-1], d, dtype=torch.int64, device=codes.device)
    for k in range(bits):
        bit = j * bits + k
        u |= ((codes[..., bit // 8].long() >> (bit % 8)) & 1) << k
    return (u - 2 ** (bits - 1)).double() * scales.double()[..., None]


def exact(case, seed):
    """The same outputs in fp64, one sequence and one head at a time."""
    s = prepare(case, seed)
    c = s["case"]
    cu, lens, table = s["cu"].tolist(), s["kv_lens"].tolist(), s["table"].long()
    d, page, bits = c["dim"], c["page"], c["bits"]
    kvh, group = c["kv_heads"], c["heads"] // c["kv_heads"]
    if c["op"] == "write":
        qp = 2 ** (bits - 1) - 1
        out = []
        for x in (s["k"], s["v"]):
            x = x.double()
            big = x.abs().max(-1, keepdim=True).values
            # the quotient that the codes round by is defined as an fp32 one
            step = (qp / (big.float() + EPS)).double()
            out.append((x * step).round().clamp(-qp - 1, qp) * (big / qp))
        return tuple(out)
    dev = s["k_codes"].device

    def fetch(b, h, first, last):
        pos = torch.arange(first, last, device=dev)
        at = table[b, pos // page], pos % page
        return (_values64(s["k_codes"][at[0], h, at[1]], s["k_scales"][at[0], h, at[1]], bits, d),
                _values64(s["v_codes"][at[0], h, at[1]], s["v_scales"][at[0], h, at[1]], bits, d))

    if c["op"] == "read":
        k, v = (torch.empty(s["total"], kvh, d, dtype=torch.float64, device=dev) for _ in range(2))
        for b in range(c["seqs"]):
            n = cu[b + 1] - cu[b]
            for h in range(kvh if n else 0):
                k[cu[b]:cu[b + 1], h], v[cu[b]:cu[b + 1], h] = fetch(b, h, lens[b] - n, lens[b])
        return k, v
    y = torch.zeros(s["total"], c["heads"], d, dtype=torch.float64, device=dev)
    lse = torch.full((s["total"], c["heads"]), -math.inf, dtype=torch.float64, device=dev)
    for b in range(c["seqs"]):
        n = cu[b + 1] - cu[b]
        if n == 0:
            continue
        here, key = torch.arange(lens[b] - n, lens[b], device=dev), torch.arange(lens[b], device=dev)
        hidden = torch.zeros(n, lens[b], dtype=torch.bool, device=dev)
        if c["causal"]:
            hidden |= key[None] > here[:, None]
        if c["window"] > 0:
            hidden |= key[None] <= here[:, None] - c["window"]
        for h in range(kvh):
            k, v = fetch(b, h, 0, lens[b])
            for j in range(h * group, (h + 1) * group):
                x = s["q"][cu[b]:cu[b + 1], j].double() @ k.T / math.sqrt(d)
                x = x.masked_fill(hidden, -math.inf)
                z = torch.logsumexp(x, 1)
                y[cu[b]:cu[b + 1], j] = torch.exp(x - z[:, None]).nan_to_num(0.0) @ v
                lse[cu[b]:cu[b + 1], j] = z
    return y, lse
