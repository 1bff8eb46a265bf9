"""The paged KV cache at the ends of what its calls take: descriptors outside
their bounds, buffers that move or overlap, scales and rows near the ends of
fp32, calls that run side by side.  Plain 64-bit forms: tests/kv_reference.py.
"""
import math

import numpy as np
import pytest
import torch

import hadamard_rotated_int4_b200 as hbl
import oracle
from tests import kv_reference as ref

DEV = "cuda:0"
gpu = pytest.mark.gpu


def pools(cache):
    return [t.cpu().clone() for t in (cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales)]


def same_bytes(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def written(case, before, rows):
    """The pools after a write of `rows`: (packed row, sequence, position) each."""
    want = [t.clone() for t in before]
    table = case.table.cpu()
    for t, b, p in rows:
        at = (int(table[b, p // case.page]), slice(None), p % case.page)
        for x, o in ((case.k, 0), (case.v, 2)):
            row = x[t].contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
            codes, scales = oracle.kv_quant(row, case.bits)
            want[o][at], want[o + 1][at] = torch.from_numpy(codes), torch.from_numpy(scales)
    return want


# ------------------------------------------------- descriptors outside their bounds

# (cu_seqlens, kv_lens) of two sequences with a table of 32 positions each, 6 packed rows, and
# the rows that have a place by the definition: row t of sequence b at kv_len - (cu[b + 1] - t)
OUTSIDE = [
    # a length past the table: the rows past position 31 are left out, the others stay theirs
    ([0, 4, 6], [34, 20], [(0, 0, 30), (1, 0, 31), (4, 1, 18), (5, 1, 19)]),
    ([0, 1, 6], [33, 20], [(i, 1, 14 + i) for i in range(1, 6)]),
    ([0, 4, 6], [2 ** 31 - 1, 20], [(4, 1, 18), (5, 1, 19)]),
    ([0, 4, 6], [-3, 20], [(4, 1, 18), (5, 1, 19)]),
    # rows past the packed ones: those there keep their positions
    ([0, 2, 8], [20, 30], [(0, 0, 18), (1, 0, 19)] + [(2 + i, 1, 24 + i) for i in range(4)]),
    ([0, 2, 2 ** 31 - 1], [20, 30], [(0, 0, 18), (1, 0, 19)]),
    # rows before the packed ones
    ([-2, 3, 6], [20, 30], [(i, 0, 17 + i) for i in range(3)] + [(3 + i, 1, 27 + i) for i in range(3)]),
    ([-2 ** 31, 3, 6], [20, 30], [(i, 0, 17 + i) for i in range(3)] + [(3 + i, 1, 27 + i) for i in range(3)]),
]


@gpu
@pytest.mark.parametrize("cu,lens,rows", OUTSIDE)
def test_rows_outside_the_bounds_are_left_out_where_they_stand(cu, lens, rows):
    c = ref.Case([3, 3], [32, 32], heads=4, kv_heads=2, D=64, bits=4, page=16, seed=5)
    c.cu.copy_(torch.tensor(cu, dtype=torch.int32))
    c.kv_lens.copy_(torch.tensor(lens, dtype=torch.int32))
    before = pools(c.cache)
    status = hbl.new_status(DEV)
    hbl.kv_cache_write(c.cache, c.k, c.v, *c.batch, status=status)
    assert int(status[0]) == 1
    for got, want in zip(pools(c.cache), written(c, before, rows)):
        assert same_bytes(got, want)

    # read back, and attended from, by the same descriptors: the rows with a place as by good ones
    status.zero_()
    K, V = hbl.kv_cache_read(c.cache, *c.batch, 6, dtype=torch.float32, status=status)
    assert int(status[0]) == 1
    status.zero_()
    O = hbl.kv_attention(c.q, c.cache, *c.batch, status=status)
    assert int(status[0]) == 1
    for t, b, p in rows:
        u, s = ref.quantise(c.k[t].cpu(), 4)
        assert torch.equal(K[t].cpu(), (u - 8).float() * s[..., None])
        one = (torch.tensor([0, 1], dtype=torch.int32, device=DEV),
               torch.tensor([p + 1], dtype=torch.int32, device=DEV), c.table[b:b + 1])
        alone = hbl.kv_attention(c.q[t:t + 1].contiguous(), c.cache, *one)
        # (both within the attention's tolerance, mostly the output's half step of 2^-8)
        assert torch.allclose(O[t].float(), alone[0].float(), rtol=2.0 ** -6, atol=1e-3)

# ------------------------------------------------------------- a cache's tensors

@gpu
def test_a_cache_keeps_the_tensors_it_was_made_of():
    c = ref.Case([2], [20], heads=2, kv_heads=2, D=64, bits=4)
    cache = c.cache
    for name in ("k_codes", "k_scales", "v_codes", "v_scales", "num_pages", "num_kv_heads",
                 "page_size", "head_dim", "bits", "device"):
        with pytest.raises(AttributeError):
            setattr(cache, name, getattr(cache, name))
    # a tensor whose memory has moved is refused, by each call
    cache.v_codes.resize_(64, *cache.v_codes.shape[1:])
    for call in (lambda: hbl.kv_cache_write(cache, c.k, c.v, *c.batch),
                 lambda: hbl.kv_cache_read(cache, *c.batch, c.rows),
                 lambda: hbl.kv_attention(c.q, cache, *c.batch)):
        with pytest.raises(ValueError):
            call()

# ------------------------------------------------------------ rows of tiny values

def tiny_rows(D):
    """bf16 bits [8, D]: the quotient Qp / max|x| passes fp32 in some, in others just not."""
    g = np.random.default_rng(D)
    x = np.zeros((8, D), dtype=np.uint16)
    x[0] = g.integers(0, 4, D)                      # the smallest subnormal numbers
    x[1] = g.integers(0, 4, D) | 0x8000
    x[2] = g.integers(0, 0x80, D) | (g.integers(0, 2, D) << 15)  # subnormal ones of either sign
    x[3, 5] = 1                                     # one value, the rest zero
    x[4] = g.integers(0, 0x0100, D) | (g.integers(0, 2, D) << 15)
    x[5] = g.integers(0, 0x0800, D) | (g.integers(0, 2, D) << 15)
    x[6] = g.integers(0, 0x7f00, D)                 # all sizes
    return x


@gpu
@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-38, 1e-5])
@pytest.mark.parametrize("bits", [2, 3, 4, 8])
@pytest.mark.parametrize("D", [32, 64, 128, 256])
def test_tiny_rows_quantise_as_defined(D, bits, eps):
    x = tiny_rows(D)
    codes, scales = oracle.kv_quant(x, bits, eps=eps)
    dev = torch.from_numpy(x.view(np.int16).copy()).view(torch.bfloat16).to(DEV)
    got = hbl.kv_quant(dev, bits, eps=eps)
    assert np.array_equal(got[0].cpu().numpy(), codes)
    assert np.array_equal(got[1].cpu().numpy().view(np.uint32), scales.view(np.uint32))
    c = ref.Case([8], [8], heads=1, kv_heads=1, D=D, bits=bits, page=16)
    hbl.kv_cache_write(c.cache, dev.view(8, 1, D), dev.flip(0).view(8, 1, D), *c.batch, eps=eps)
    page = int(c.table[0, 0])
    for pool, want in zip(pools(c.cache), (codes, scales, codes[::-1], scales[::-1])):
        assert same_bytes(pool[page, 0, :8], torch.from_numpy(want.copy()))

# --------------------------------------------------------- V's scales, all of fp32

def expected(c, causal=True, window=0):
    """(O, lse, tolerance of each), fp64, for scales of any size.

    As kv_reference.attention, with what wide scales add.  Exponents in log2 reach
    |s| + |log2 sv| < 256, where fp32's half step is 2^-17: three roundings of the
    exponent, the logarithm of the scale to 2^-22 of itself (150 * 2^-22), and the
    difference of two reference points (2^-16): together below 2^-14 in nats.  A weight
    p_i sv_i is held to 2^-12 of itself (here 2^-11), or to 2^-31 of the row's
    largest one: 2^-30 of that times |code|.  A bf16's least half step is 2^-134."""
    u = 2.0 ** -24
    O = torch.zeros(c.rows, c.heads, c.D, dtype=torch.float64, device=DEV)
    z = torch.full((c.rows, c.heads), -math.inf, dtype=torch.float64, device=DEV)
    tol_O, tol_z = torch.zeros_like(O), torch.zeros_like(z)
    group, r0 = c.heads // c.cache.num_kv_heads, 0
    for b, (n, m) in enumerate(zip(c.new, c.lens)):
        pos, key = torch.arange(m - n, m, device=DEV)[:, None], torch.arange(m, device=DEV)[None]
        hidden = (key > pos) if causal else torch.zeros(n, m, dtype=torch.bool, device=DEV)
        if window:
            hidden = hidden | (key <= pos - window)
        at = c.table[b].long()[key[0] // c.page], key[0] % c.page
        for j in range(c.heads if n else 0):
            h = j // group
            k = c.stored(b, h, "k")
            code = ref.unpack(c.cache.v_codes[at[0], h, at[1]], c.D, c.bits).double() - (
                1 << (c.bits - 1))
            sv = c.cache.v_scales[at[0], h, at[1]].double()
            q = c.q[r0:r0 + n, j].double() * c.D ** -0.5
            s = (q @ k.T).masked_fill(hidden, -math.inf)
            lse = torch.logsumexp(s, 1)
            p = torch.exp(s - lse[:, None].nan_to_num(neginf=0.0)) * sv
            e = (4 * c.D + 2) * u * (q.abs() @ k.abs().T).masked_fill(hidden, 0).amax(1) + 2.0 ** -14
            rows = slice(r0, r0 + n)
            O[rows, j], z[rows, j] = p @ code, lse
            tol_O[rows, j] = 2.0 ** -8 * O[rows, j].abs() + 2.0 ** -134 + \
                (2 * e + 2.0 ** -11 + 4 * m * u)[:, None] * (p @ code.abs()) + \
                2.0 ** -30 * p.amax(1, keepdim=True) * ((~hidden).double() @ code.abs())
            tol_z[rows, j] = e + 2.0 ** -23 * lse.abs().nan_to_num(posinf=0.0) + m * u
        r0 += n
    return O, z, tol_O, tol_z


def check(c, **kw):
    O, lse = hbl.kv_attention(c.q, c.cache, *c.batch, max_rows=max(c.new), want_lse=True, **kw)
    want, z, tol_O, tol_z = expected(c, **kw)
    assert torch.isfinite(O.float()).all()
    d = (O.double() - want).abs() - tol_O
    assert float(d.max()) <= 0, (float(O.flatten()[d.argmax()]), float(want.flatten()[d.argmax()]))
    none = z == -math.inf
    assert torch.equal(lse == -math.inf, none)
    d = (lse.double() - z).abs().masked_fill(none, 0) - tol_z
    assert float(d.max()) <= 0, (float(lse.flatten()[d.argmax()]), float(z.flatten()[d.argmax()]))


def scales_of(kind, shape, g):
    """V scales [.., positions] of one kind (exponents; zero where nan)."""
    e = torch.rand(shape, generator=g) - 0.5
    pos = torch.arange(shape[-1]).expand(shape)
    if kind == "tiny":
        e = e - 110
    elif kind == "subnormal":
        e = 6 * e - 140
    elif kind == "huge":
        e = e + 125
    elif kind == "spread":
        e = 240 * e
    elif kind == "zero_rows":       # beside rows of 2^34
        e = torch.where(pos % 7 == 3, math.nan, e + 34)
    elif kind == "zeros":
        e = torch.full(shape, math.nan)
    elif kind == "zeros_among":     # small ones and large ones that need no form of their own
        e = torch.where(pos % 5 == 1, math.nan, 78 * e)
    elif kind == "late":            # ordinary ones, then a few wild ones
        e = torch.where(pos > shape[-1] - 9, 200 * e, e)
    elif kind == "early":
        e = torch.where(pos < 9, 200 * e, e)
    elif kind == "edges":           # at and around where the kernels change their form
        e = torch.where(pos % 2 == 0, -40.0, 40.0) + 0.02 * e
    return torch.exp2(e.double()).float().nan_to_num(nan=0.0)


KINDS = ["tiny", "subnormal", "huge", "spread", "zero_rows", "zeros", "zeros_among", "late", "early", "edges"]


def wide_case(kind, new, lens, D, bits, qscale=2.0, **kw):
    c = ref.Case(new, lens, D=D, bits=bits, page=16, seed=D + bits, qscale=qscale, **kw)
    g = torch.Generator().manual_seed(D * bits)
    for b, m in enumerate(lens):
        pos = torch.arange(m)
        sv = scales_of(kind, (c.cache.num_kv_heads, m), g).to(DEV)
        page = c.table[b].long()[pos.to(DEV) // 16]
        c.cache.v_scales[page, :, pos.to(DEV) % 16] = sv.T.contiguous()
        # zero rows as the write leaves them: zero scales, zero values
        zero = torch.from_numpy(oracle.kv_quant(np.zeros((1, D), np.uint16), bits)[0][0].copy())
        for i in (sv[0] == 0).nonzero().flatten().tolist():
            c.cache.v_codes[page[i], :, i % 16] = zero.to(DEV)
    return c


@gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,bits", [(32, 8), (64, 3), (128, 4), (256, 2)])
@pytest.mark.parametrize("new,lens", [([1, 3], [200, 777]), ([5, 1], [1500, 90]), ([40, 130], [300, 333])])
def test_attention_of_any_value_scale(kind, D, bits, new, lens):
    if kind == "huge" and bits > 2:     # (their values would pass fp32)
        bits = 2
    c = wide_case(kind, new, lens, D, bits, heads=4, kv_heads=2)
    check(c)
    # equal scores, where every row's share of the sum counts
    c.q.zero_()
    check(c)


@gpu
@pytest.mark.parametrize("kind", ["spread", "late", "zero_rows"])
@pytest.mark.parametrize("causal,window", [(True, 100), (False, 0), (False, 50)])
@pytest.mark.parametrize("new", [[2, 1], [70, 200]])
def test_attention_of_any_value_scale_under_masks(kind, causal, window, new):
    c = wide_case(kind, new, [260, 400], 64, 4, heads=4, kv_heads=2, qscale=0.5)
    check(c, causal=causal, window=window)


@gpu
@pytest.mark.parametrize("new", [[1, 2], [150, 40]])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_scores_that_make_up_for_the_scales(D, new):
    # position i's score is -log of its V scale, between 2^-60 and 2^60: every term of O
    # counts alike, and the normaliser is that of the rows of the smallest scales
    c = wide_case("spread", new, [500, 3000], D, 4, heads=2, kv_heads=2)
    c.q.zero_()
    c.q[..., 0] = 1.0
    for b, m in enumerate(c.lens):
        pos = torch.arange(m, device=DEV)
        page, slot = c.table[b].long()[pos // 16], pos % 16
        e = (120 * torch.rand(2, m, generator=torch.Generator().manual_seed(b)) - 60).to(DEV)
        c.cache.v_scales[page, :, slot] = torch.exp2(e).T.contiguous()
        c.cache.k_scales[page, :, slot] = (e.abs() * math.log(2) * D ** 0.5).T.contiguous()
        codes = torch.full((m, 2, D // 2), 0x88, dtype=torch.uint8, device=DEV)
        codes[:, :, 0] = torch.where(e.T > 0, 0x87, 0x89).to(torch.uint8)  # the first value -1 or 1
        c.cache.k_codes[page, :, slot] = codes
    check(c)

# ------------------------------------------------------------ buffers that overlap

def test_overlap_of_strided_rows():
    # against all elements of both, over small layouts
    g = np.random.default_rng(0)
    seen = {True: 0, False: 0}
    for _ in range(4000):
        rows, heads, D = (int(g.integers(1, 5)) for _ in range(3))
        a = (int(g.integers(0, 40)), int(g.integers(0, 12)), int(g.integers(0, 12)))
        b = a if g.random() < 0.1 else tuple(int(v) for v in (g.integers(0, 40), g.integers(0, 12),
                                                              g.integers(0, 12)))
        if g.random() < 0.5:
            b = (b[0], a[1], b[2])
        cells = [{at + i * r + j * h + d for i in range(rows) for j in range(heads) for d in range(D)}
                 for at, r, h in (a, b)]
        want = bool(cells[0] & cells[1])
        assert hbl._kv_overlap(rows, heads, D, a, b) == want, (rows, heads, D, a, b)
        alone = len(cells[0]) < rows * heads * D
        assert hbl._kv_overlap(rows, heads, D, a) == alone, (rows, heads, D, a)
        seen[want] += 1
    assert min(seen.values()) > 500


@gpu
@pytest.mark.parametrize("rows", [2, 150])
def test_attention_outputs_that_overlap(rows):
    c = ref.Case([rows], [rows + 300], heads=4, kv_heads=2, D=64, bits=4, seed=rows)
    want = hbl.kv_attention(c.q, c.cache, *c.batch)
    wide = torch.zeros(rows + 1, 4, 64, dtype=torch.bfloat16, device=DEV)
    wide[:-1] = c.q
    for out in (wide[1:], wide.view(-1)[8:8 + c.q.numel()].view(rows, 4, 64)):
        with pytest.raises(ValueError):
            hbl.kv_attention(wide[:-1], c.cache, *c.batch, out=out)
    # rows or heads of the output over one another
    flat = torch.zeros(4 * rows * 256, dtype=torch.bfloat16, device=DEV)
    for strides in ((128, 64, 1), (256, 56, 1), (64, 64, 1)):
        with pytest.raises(ValueError):
            hbl.kv_attention(c.q, c.cache, *c.batch, out=flat.as_strided((rows, 4, 64), strides))
    # side by side in one buffer, in either order of strides, and the queries themselves
    fused = torch.zeros(rows, 8, 64, dtype=torch.bfloat16, device=DEV)
    fused[:, :4] = c.q
    assert torch.equal(hbl.kv_attention(fused[:, :4], c.cache, *c.batch, out=fused[:, 4:]), want)
    assert torch.equal(fused[:, :4], c.q)
    out = flat.as_strided((rows, 4, 64), (64, 64 * rows, 1))
    assert torch.equal(hbl.kv_attention(c.q, c.cache, *c.batch, out=out), want)
    q = c.q.clone()
    assert torch.equal(hbl.kv_attention(q, c.cache, *c.batch, out=q), want)


@gpu
def test_read_outputs_that_overlap():
    c = ref.Case([6], [20], heads=2, kv_heads=2, D=64, bits=4)
    x = torch.zeros(9, 2, 64, dtype=torch.bfloat16, device=DEV)
    for out in ((x[:6], x[:6]), (x[:6], x[3:])):
        with pytest.raises(ValueError):
            hbl.kv_cache_read(c.cache, *c.batch, 6, out=out)

# --------------------------------------------------------------------- lost waits

def test_clock_wait_probe_is_checked_on_the_host():
    call = hbl.lib().hbl_selftest_clock_wait
    assert call(0, 0, 1000, None, None) == 1
    assert call(0, 0, 0, 0x10000, None) == 1 and call(0, 0, 2000000001, 0x10000, None) == 1
    assert call(0, 0, 1000, 0x10004, None) == 3


@gpu
@pytest.mark.parametrize("arrive,aborted,limit,want",
                         [(1, 0, 1000, 0), (0, 0, 2000000, 7), (0, 1, 2000000000, 7), (1, 1, 1000, 0)])
def test_the_attention_s_wait_gives_up_by_time_and_by_its_flag(arrive, aborted, limit, want):
    status = hbl.new_status(DEV)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    hbl.selftest_clock_wait(1, 0, 1000, status)  # (loaded)
    begin.record()
    hbl.selftest_clock_wait(arrive, aborted, limit, status)
    end.record()
    torch.cuda.synchronize()
    assert int(status[0]) == want
    # 2e6 clocks are some 1 to 2 ms; the flag does not wait for its second
    ms = begin.elapsed_time(end)
    assert ms < 100 and (want == 0 or aborted or ms > 0.5)
    c = ref.Case([1, 40], [70, 90], heads=4, kv_heads=2, D=64, bits=4)  # the context is usable
    O, lse = hbl.kv_attention(c.q, c.cache, *c.batch, want_lse=True)
    ref.check_attention(c, O, lse)

# ------------------------------------------------------------------- side by side

@gpu
@pytest.mark.parametrize("new,lens", [([1, 1], [5000, 300]), ([70], [4000]), ([40, 1, 130], [900, 3000, 1500])])
def test_calls_on_several_streams_give_what_one_gives(new, lens):
    # split pieces, split ranges and both kernels of a mixed batch, three streams at once,
    # a workspace of the call's own each time
    cases = [ref.Case(new, lens, heads=8, kv_heads=2, D=128, bits=4, seed=s) for s in range(3)]
    call = lambda c: hbl.kv_attention(c.q, c.cache, *c.batch, max_rows=max(new), want_lse=True)
    alone = [call(c) for c in cases]
    assert hbl.kv_attention_workspace_size(sum(new), 8, cases[0].cache, len(new),
                                           cases[0].table.shape[1], max_rows=max(new)) > 0
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = []
    for _ in range(8):
        for i, (c, s) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(s):
                outs.append((i, call(c)))
    torch.cuda.synchronize()
    for i, (O, lse) in outs:
        assert torch.equal(O, alone[i][0]) and torch.equal(lse, alone[i][1])
