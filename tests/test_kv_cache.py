"""The paged low-bit KV cache: writing new rows, reading rows back, and the
attention over it, against plain 64-bit forms (tests/kv_reference.py).

Codes and scales are bit-exact by definition.  Read values are one fp32
product (half a step, 2^-24) and, in bf16, one more rounding (2^-8).  The
attention's tolerances are derived in kv_reference.attention.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

import hadamard_rotated_int4_b200 as hbl
import oracle
from hadamard_rotated_int4_b200 import inputs
from tests import kv_reference as ref

DEV = "cuda:0"
gpu = pytest.mark.gpu
BITS, DIMS = [2, 3, 4, 8], [32, 64, 128, 256]


# ---------------------------------------------------------------- on the CPU

A = 0x10000


def _args(**kw):
    c = dict(k_codes=A, k_scales=A, v_codes=A, v_scales=A, num_pages=4, page_size=16,
             num_kv_heads=2, head_dim=64, bits=4)
    b = dict(cu_seqlens=A, kv_lens=A, block_table=A, num_seqs=2, pages_per_seq=2, rows=3)
    a = dict(Q=A, q_row_stride=256, q_head_stride=64, O=A, o_row_stride=256, o_head_stride=64,
             lse=None, num_heads=4, max_rows=0, max_kv=0, scale=0.125, causal=1, window=0)
    for k, v in kw.items():
        (c if k in c else b if k in b else a)[k] = v
    return hbl._CacheArgs(**c), hbl._BatchArgs(**b), hbl._AttnArgs(**a)


def _write(K=A, kr=128, kh=64, V=A, vr=128, vh=64, eps=1e-5, **kw):
    c, b, _ = _args(**kw)
    return hbl.lib().hbl_kv_cache_write(c, b, K, kr, kh, V, vr, vh, eps, None, None)


def _read(K=A, V=A, fp32=0, **kw):
    c, b, _ = _args(**kw)
    return hbl.lib().hbl_kv_cache_read(c, b, K, V, fp32, None, None)


def _attend(ws=None, ws_bytes=0, **kw):
    c, b, a = _args(**kw)
    return hbl.lib().hbl_kv_attention(c, b, a, ws, ws_bytes, None, None)


SHARED = [(dict(bits=5), 1), (dict(bits=0), 1), (dict(head_dim=96), 2), (dict(head_dim=512), 2),
          (dict(num_pages=0), 2), (dict(num_kv_heads=0), 2), (dict(num_kv_heads=1 << 16, num_heads=1 << 16), 2),
          (dict(page_size=8), 2), (dict(page_size=24), 2), (dict(page_size=1 << 17), 2),
          (dict(num_seqs=-1), 2), (dict(pages_per_seq=-1), 2), (dict(rows=-1), 2),
          (dict(pages_per_seq=1 << 27), 2), (dict(pages_per_seq=(1 << 27) - 255), 2),
          (dict(k_codes=None), 1), (dict(v_scales=None), 1),
          (dict(cu_seqlens=None), 1), (dict(block_table=None), 1), (dict(v_codes=A + 8), 3),
          (dict(k_scales=A + 4), 3), (dict(kv_lens=A + 2), 3), (dict(rows=0), 0),
          (dict(num_seqs=0), 0)]


@pytest.mark.parametrize("kw,want", SHARED)
def test_cache_and_batch_are_checked_on_the_host(kw, want):
    for call in (_write, _read, _attend):
        if call is not _attend and "num_heads" in kw:
            assert call(num_kv_heads=kw["num_kv_heads"]) == want
        else:
            assert call(**kw) == want, call


def test_call_arguments_are_checked_on_the_host():
    assert _write(eps=-1.0) == 1 and _write(eps=math.inf) == 1
    assert _write(K=None) == 1 and _write(V=A + 2) == 3
    assert _write(kr=132) == 3 and _write(vh=65) == 3
    assert _read(K=None) == 1 and _read(V=A + 8) == 3 and _read(fp32=2) == 1
    assert _attend(scale=math.nan) == 1 and _attend(window=-1) == 1 and _attend(causal=2) == 1
    assert _attend(num_heads=3) == 2 and _attend(num_heads=0) == 2 and _attend(max_rows=-1) == 2
    assert _attend(max_kv=-1) == 2 and _attend(rows=1 << 29) == 2
    assert _attend(Q=None) == 1 and _attend(O=A + 8) == 3 and _attend(lse=A + 2) == 3
    assert _attend(q_row_stride=252) == 3 and _attend(o_head_stride=4) == 3
    lib = hbl.lib()
    c, b, a = _args()
    assert lib.hbl_kv_attention_workspace(c, b, a, None) == 1
    need = ctypes.c_size_t(7)
    assert lib.hbl_kv_attention_workspace(None, b, a, ctypes.byref(need)) == 1 and need.value == 0
    c, b, a = _args(rows=0)
    assert lib.hbl_kv_attention_workspace(c, b, a, ctypes.byref(need)) == 0 and need.value == 0


def test_binding_refuses_host_tensors_and_bad_shapes():
    z = torch.zeros(4, 2, 16, 32, dtype=torch.uint8)
    with pytest.raises(TypeError):
        hbl.KvCache(z, torch.zeros(4, 2, 16), z, torch.zeros(4, 2, 16), 64)


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("D", DIMS)
def test_reference_codec_agrees_with_the_oracle(bits, D):
    X = inputs.qkv_states(T=5, H=3, D=D, seed=bits * D)
    codes, scales = oracle.kv_quant(X, bits)
    x = torch.from_numpy(X.view(np.int16).copy()).view(torch.bfloat16)
    u, s = ref.quantise(x, bits)
    assert np.array_equal(ref.unpack(torch.from_numpy(codes), D, bits).numpy(),
                          u.reshape(-1, D).numpy())
    assert np.array_equal(oracle.kv_unpack(codes, D, bits), u.reshape(-1, D).numpy())
    assert np.array_equal(s.reshape(-1).numpy(), scales)


# ---------------------------------------------------------------- write, read

RAGGED = ([3, 0, 1, 40, 17, 2], [50, 7, 1, 40, 100, 0])  # the last one's rows have no place


def _written(case, k_like, v_like, before):
    """The pools that writing case.k, case.v should leave, from `before`."""
    want = [t.clone() for t in before]
    r0 = 0
    for n, m, table in zip(case.new, case.lens, case.table.cpu()):
        for i in range(n):
            p = m - n + i
            if p < 0:
                continue
            at = (int(table[p // case.page]), slice(None), p % case.page)
            for x, o in ((k_like, 0), (v_like, 2)):
                row = x[r0 + i].contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
                codes, scales = oracle.kv_quant(row, case.bits)
                want[o][at], want[o + 1][at] = torch.from_numpy(codes), torch.from_numpy(scales)
        r0 += n
    return want


def _pools(case):
    c = case.cache
    return [t.cpu().clone() for t in (c.k_codes, c.k_scales, c.v_codes, c.v_scales)]


def _same(a, b):
    return torch.equal(a.view(torch.uint8) if a.dtype == torch.uint8 else a.view(torch.int32),
                       b.view(torch.uint8) if b.dtype == torch.uint8 else b.view(torch.int32))


@gpu
@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("kv_heads,page", [(1, 16), (5, 48)])
def test_write_is_bit_exact_and_touches_nothing_else(bits, D, kv_heads, page):
    c = ref.Case(*RAGGED, heads=kv_heads, kv_heads=kv_heads, D=D, bits=bits, page=page, seed=D + bits,
                 extra_rows=3)
    before = _pools(c)
    hbl.kv_cache_write(c.cache, c.k, c.v, *c.batch)
    for got, want in zip(_pools(c), _written(c, c.k, c.v, before)):
        assert _same(got, want)


@gpu
@pytest.mark.parametrize("bits", BITS)
def test_write_of_strided_states_and_edge_rows(bits):
    c = ref.Case([5, 9], [5, 30], heads=3, kv_heads=3, D=64, bits=bits, seed=1)
    # slices of a fused projection, and a transposed layout
    qkv = torch.randn(14, 8, 64, device=DEV).to(torch.bfloat16)
    k = qkv[:, 1:4]
    v = torch.randn(3, 14, 64, device=DEV).to(torch.bfloat16).transpose(0, 1)
    qkv[2, 1] = 0                       # a zero row: codes 2^(bits-1), scale 0
    qkv[3, 2] = 0
    qkv[3, 2, 7] = -10.0                # one spike
    qkv[4, 1] = 1.0
    qkv[5, 3, ::2] = 3e38               # very large values
    before = _pools(c)
    for eps in (1e-5, 0.0):
        hbl.kv_cache_write(c.cache, k, v, *c.batch, eps=eps)
        if eps:
            for got, want in zip(_pools(c), _written(c, k, v, before)):
                assert _same(got, want)
    hbl.kv_cache_write(c.cache, k, v, *c.batch)
    K, _ = hbl.kv_cache_read(c.cache, *c.batch, c.rows)
    assert not K[2, 0].any()


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("D", DIMS)
def test_read(bits, D, dtype):
    c = ref.Case(*RAGGED, heads=3, kv_heads=3, D=D, bits=bits, page=32, seed=D - bits, extra_rows=4)
    out = tuple(torch.full((c.rows, 3, D), 7.0, dtype=dtype, device=DEV) for _ in range(2))
    K, V = hbl.kv_cache_read(c.cache, *c.batch, c.rows, dtype=dtype, out=out)
    assert K is out[0] and V is out[1]
    step = 2.0 ** -24 + (2.0 ** -8 if dtype == torch.bfloat16 else 0)
    r0 = 0
    for b, (n, m) in enumerate(zip(c.new, c.lens)):
        skip = max(0, n - m)  # rows without a place
        for got, which in ((K, "k"), (V, "v")):
            assert not got[r0:r0 + skip].any()
            for h in range(3):
                want = c.stored(b, h, which)[m - n + skip:]
                x = got[r0 + skip:r0 + n, h].double()
                assert bool(((x - want).abs() <= step * want.abs()).all())
        r0 += n
    assert bool((K[r0:] == 7).all()) and bool((V[r0:] == 7).all())  # rows of no sequence


@gpu
def test_many_sequences_and_one_long_one():
    # more sequences than a warp looks at in one step, most of them one row
    new = [1] * 70 + [0] * 5 + [300] + [1] * 60
    lens = [(7 * i) % 90 + 1 for i in range(75)] + [1000] + [3] * 60
    c = ref.Case(new, lens, heads=2, kv_heads=2, D=32, bits=3, seed=4)
    before = _pools(c)
    hbl.kv_cache_write(c.cache, c.k, c.v, *c.batch)
    for got, want in zip(_pools(c), _written(c, c.k, c.v, before)):
        assert _same(got, want)
    K, V = hbl.kv_cache_read(c.cache, *c.batch, c.rows, dtype=torch.float32)
    u, s = ref.quantise(c.k.cpu(), 3)
    assert torch.equal(K.cpu(), (u - 4).float() * s[..., None])


@gpu
def test_bad_descriptors_are_reported_and_touch_nothing():
    def run(change):
        c = ref.Case([2, 3], [20, 40], heads=2, kv_heads=2, D=64, bits=4, seed=9)
        change(c)
        before = _pools(c)
        status = hbl.new_status(DEV)
        hbl.kv_cache_write(c.cache, c.k, c.v, *c.batch, status=status)
        st = [int(status[0])]
        after = _pools(c)
        touched = [int((a.flatten(2).view(torch.uint8) != b.flatten(2).view(torch.uint8)).any(-1).sum())
                   for a, b in zip(before, after)]
        for call in (lambda s: hbl.kv_cache_read(c.cache, *c.batch, c.rows, status=s),
                     lambda s: hbl.kv_attention(c.q, c.cache, *c.batch, status=s)):
            status.zero_()
            call(status)
            st.append(int(status[0]))
        return st, touched, c

    st, touched, _ = run(lambda c: None)
    assert st == [0, 0, 0] and touched[0] > 0

    def bad_page(v):
        def f(c):
            c.table[1, 2] = v  # positions 32..39: the second sequence's new rows
        return f

    for v in (-1, 1 << 20, -(1 << 31)):
        st, touched, c = run(bad_page(v))
        assert st == [1, 1, 1]
        K, _ = hbl.kv_cache_read(c.cache, *c.batch, c.rows)
        assert not K[2:].any()
        # the first sequence is not affected
        O, lse = hbl.kv_attention(c.q, c.cache, *c.batch, want_lse=True)
        c2 = c
        c2.new, c2.lens = [2], [20]
        ref.check_attention(c2, O, lse)

    def far_len(c):
        c.kv_lens[1] = 1 << 30
    assert run(far_len)[0] == [1, 1, 1]

    def negative_len(c):
        c.kv_lens[1] = -5
    assert run(negative_len)[0] == [1, 1, 1]

    def far_rows(c):
        c.cu[2] = 100
    assert run(far_rows)[0] == [1, 1, 1]

    def falling_rows(c):
        c.cu[1] = 5
        c.cu[2] = 2
    assert run(falling_rows)[0] == [1, 1, 1]


# ---------------------------------------------------------------- attention

def attend(c, **kw):
    out = torch.full((c.rows, c.heads, c.D), 7.0, dtype=torch.bfloat16, device=DEV)
    O, lse = hbl.kv_attention(c.q, c.cache, *c.batch, want_lse=True, out=out, **kw)
    assert O is out
    assert bool((O[sum(c.new):] == 7).all())  # rows of no sequence are left as they were
    return O, lse


@gpu
@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("group", [1, 4])
def test_attention_one_row_each(bits, D, group):
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 129, 333, 0]
    c = ref.Case([1] * len(lens), lens, heads=3 * group, kv_heads=3, D=D, bits=bits, page=16,
                 seed=D * bits + group, extra_rows=2)
    ref.check_attention(c, *attend(c, max_rows=1))


@gpu
@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("D", DIMS)
def test_attention_ragged_chunks(bits, D):
    # chunks of every kind: whole prompts, appended ones, empty ones, and one
    # with more rows than positions (its first rows see nothing)
    new = [130, 1, 0, 37, 300, 5, 9]
    lens = [130, 77, 50, 400, 301, 3, 0]
    c = ref.Case(new, lens, heads=6, kv_heads=2, D=D, bits=bits, page=48, seed=D + 7 * bits,
                 extra_rows=3)
    ref.check_attention(c, *attend(c, max_rows=300))
    O, lse = attend(c)
    ref.check_attention(c, O, lse)


@gpu
@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 8, 9, 16, 17, 33, 64, 65, 129, 257])
@pytest.mark.parametrize("group", [1, 3, 8])
def test_attention_row_counts(rows, group):
    c = ref.Case([rows, max(1, rows - 1)], [rows + 190, rows], heads=2 * group, kv_heads=2, D=64,
                 bits=4, page=16, seed=rows + group)
    ref.check_attention(c, *attend(c, max_rows=rows))


@gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 2, 16, 100, 5000])
@pytest.mark.parametrize("D", [64, 256])
def test_attention_windows_and_masks(causal, window, D):
    new, lens = [1, 140, 3, 4], [700, 500, 3, 2]
    c = ref.Case(new, lens, heads=4, kv_heads=2, D=D, bits=4, page=32, seed=window + D)
    ref.check_attention(c, *attend(c, causal=causal, window=window), causal=causal, window=window)
    one = ref.Case([1, 1, 2], [700, 1, 90], heads=4, kv_heads=2, D=D, bits=3, page=32, seed=window)
    ref.check_attention(one, *attend(one, causal=causal, window=window, max_rows=2), causal=causal,
                        window=window)


@gpu
@pytest.mark.parametrize("new,lens", [([1, 1], [20000, 4099]), ([3, 2], [9000, 8191]),
                                      ([150], [6000])])
@pytest.mark.parametrize("bits", [3, 8])
def test_attention_long_contexts(new, lens, bits):
    # work that is split over the positions and joined
    c = ref.Case(new, lens, heads=8, kv_heads=2, D=128, bits=bits, page=64, seed=bits)
    ref.check_attention(c, *attend(c, max_rows=max(new), max_kv=max(lens)))
    # the hint is only a hint: a wrong one changes no result beyond the tolerance
    ref.check_attention(c, *attend(c, max_rows=max(new), max_kv=16))


@gpu
@pytest.mark.parametrize("rows,group", [(1, 1), (3, 8)])
def test_attention_of_many_sequences(rows, group):
    # more sequences than a CTA has threads, uneven and empty ones among them, so
    # that the pieces of the common line begin and end anywhere
    lens = [(37 * i) % 200 + (900 if i % 71 == 0 else 0) for i in range(700)]
    new = [min(rows, n) if i % 5 else 0 for i, n in enumerate(lens)]
    c = ref.Case(new, lens, heads=group, kv_heads=1, D=32, bits=4, page=16, seed=rows, extra_rows=2)
    ref.check_attention(c, *attend(c, max_rows=rows))
    # and one chunk among them
    new[333], lens[333] = 150, 400
    c = ref.Case(new, lens, heads=group, kv_heads=1, D=32, bits=4, page=16, seed=rows, extra_rows=2)
    ref.check_attention(c, *attend(c, max_rows=150))


@gpu
@pytest.mark.parametrize("D,bits", [(32, 8), (64, 4), (256, 3)])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 30)])
def test_attention_of_many_chunks(D, bits, causal, window):
    # more chunked sequences than a warp has lanes, uneven, short and empty ones among
    # them, so that row blocks of all of them are put in order
    lens = [(53 * i) % 170 + 9 for i in range(70)]
    new = [0 if i % 9 == 4 else min(n, 7 + (29 * i) % 90) for i, n in enumerate(lens)]
    c = ref.Case(new, lens, heads=8, kv_heads=2, D=D, bits=bits, page=16, seed=D, extra_rows=1)
    O, lse = attend(c, max_rows=max(new), causal=causal, window=window)
    ref.check_attention(c, O, lse, causal=causal, window=window)


@gpu
@pytest.mark.parametrize("group", [33, 128, 300])
@pytest.mark.parametrize("D", [64, 256])
def test_attention_of_wide_groups(group, D):
    # one token's query heads fill a row block, or more than one
    c = ref.Case([1, 1, 3, 0, 2], [200, 1, 90, 5, 700], heads=group, kv_heads=1, D=D, bits=4,
                 page=32, seed=group, extra_rows=1)
    ref.check_attention(c, *attend(c, max_rows=3))
    one = ref.Case([1], [1500], heads=group, kv_heads=1, D=D, bits=2, page=32, seed=group)
    ref.check_attention(one, *attend(one))


@gpu
@pytest.mark.parametrize("new", [[1, 2, 1], [40, 1, 130]])
def test_rows_before_the_first_sequence(new):
    c = ref.Case(new, [200, 50, 131], heads=4, kv_heads=2, D=64, bits=4, seed=1, extra_rows=3)
    want, _ = attend(c)
    c.cu += 3
    c.q = c.q.roll(3, 0)
    out = torch.full_like(c.q, 7.0)
    hbl.kv_attention(c.q, c.cache, *c.batch, out=out)
    assert torch.equal(out[3:], want[:-3]) and bool((out[:3] == 7).all())


@gpu
def test_attention_under_a_wide_block_table():
    # a table with room for 2^30 positions a sequence: the plan goes by its width, the
    # work by the lengths
    c = ref.Case([1, 2, 40, 1], [700, 90, 41, 3], heads=32, kv_heads=32, D=32, bits=2, page=16,
                 wide=1 << 26)
    ref.check_attention(c, *attend(c, max_rows=40))
    c = ref.Case([1, 2, 1, 1], [700, 90, 41, 3], heads=32, kv_heads=32, D=32, bits=2, page=16,
                 wide=1 << 26)
    ref.check_attention(c, *attend(c, max_rows=2))
    ref.check_attention(c, *attend(c, max_rows=2, window=0x7fffffff), window=0x7fffffff)


@gpu
@pytest.mark.parametrize("rows", [1, 6, 200])
def test_attention_extreme_scores_scales_and_zero_rows(rows):
    c = ref.Case([rows], [260], heads=4, kv_heads=2, D=64, bits=4, seed=rows)
    c.cache.v_scales[c.table[0, 0].long(), :, 3] = 0    # a zero row: code 8 everywhere
    c.cache.v_codes[c.table[0, 0].long(), :, 3] = 0x88
    c.cache.k_scales[c.table[0, 1].long(), :, 5] = 0
    c.cache.v_scales[c.table[0, 2].long(), :, 1] = 1e4  # a value far above the others
    c.cache.v_scales[c.table[0, 3].long(), :, 1] = 1e-6
    ref.check_attention(c, *attend(c))
    for scale in (0.0, 1.0, -0.3, 1e-3):
        ref.check_attention(c, *attend(c, scale=scale), scale=scale)


@gpu
@pytest.mark.parametrize("rows", [1, 140])
def test_attention_of_strided_queries_and_outputs(rows):
    c = ref.Case([rows], [rows + 60], heads=6, kv_heads=2, D=64, bits=8, seed=rows)
    fused = torch.zeros(rows, 10, 64, dtype=torch.bfloat16, device=DEV)
    fused[:, 2:8] = c.q
    wide = torch.full((6, rows, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    O = hbl.kv_attention(fused[:, 2:8], c.cache, *c.batch, out=wide.transpose(0, 1))
    ref.check_attention(c, O)
    with pytest.raises(ValueError):
        hbl.kv_attention(c.q[..., ::2], c.cache, *c.batch)
    with pytest.raises(hbl.HblError):
        hbl.kv_attention(torch.zeros(rows, 6, 68, dtype=torch.bfloat16, device=DEV)[..., 4:],
                         c.cache, *c.batch)


@gpu
def test_a_row_of_nan_stays_its_own():
    for rows in (8, 150):
        c = ref.Case([rows, 1], [rows + 40, 30], heads=4, kv_heads=2, D=64, bits=4, seed=rows)
        clean, _ = attend(c)
        c.q[3] = math.nan
        c.q[5, 1] = math.inf
        O, _ = attend(c)
        keep = torch.ones(c.rows, 4, dtype=torch.bool, device=DEV)
        keep[3] = False
        keep[5, 1] = False
        assert torch.equal(O[keep], clean[keep])


@gpu
@pytest.mark.parametrize("new,lens", [([1, 1, 1], [3000, 40, 777]), ([200, 1], [1500, 900])])
def test_attention_repeats_bit_for_bit(new, lens):
    c = ref.Case(new, lens, heads=8, kv_heads=2, D=128, bits=4, seed=2)
    first = attend(c, max_rows=max(new))
    for _ in range(3):
        again = attend(c, max_rows=max(new))
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@gpu
@pytest.mark.parametrize("D", DIMS)
def test_many_tiles_many_times(D):
    # long non-causal chunks on every SM, launched back to back: no wait of the
    # kernel's pipeline may be missed
    c = ref.Case([17], [2100], heads=148 * 4, kv_heads=148, D=D, bits=2, page=64, seed=D)
    status = hbl.new_status(DEV)
    outs = [hbl.kv_attention(c.q, c.cache, *c.batch, causal=False, status=status) for _ in range(60)]
    torch.cuda.synchronize()
    assert int(status[0]) == 0
    assert all(torch.equal(o, outs[0]) for o in outs[1:])


@gpu
def test_rows_past_max_rows_are_left_out_and_reported():
    c = ref.Case([5, 40], [50, 60], heads=2, kv_heads=2, D=64, bits=4, seed=3)
    status = hbl.new_status(DEV)
    out = torch.full((c.rows, 2, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    hbl.kv_attention(c.q, c.cache, *c.batch, max_rows=8, out=out, status=status)
    assert int(status[0]) == 1
    assert bool((out[13:] == 7).all())
    full = hbl.kv_attention(c.q, c.cache, *c.batch)
    assert torch.allclose(out[:13].float(), full[:13].float(), rtol=2.0 ** -6, atol=1e-3)


@gpu
@pytest.mark.parametrize("D", [64, 256])
def test_rows_past_max_rows_under_a_wide_window(D):
    # 2000 rows where 2 were announced: those two, far back, see nearly the whole
    # sequence, which the plan (a window of 40 rows) made no room to split
    c = ref.Case([2000, 1], [2010, 30], heads=4, kv_heads=2, D=D, bits=4, seed=D)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    assert hbl.kv_attention_workspace_size(c.rows, 4, c.cache, 2, c.table.shape[1], max_rows=2,
                                           causal=False, window=40) == 0
    O, lse = attend(c, causal=False, window=40, max_rows=2, status=st)
    assert st.item() == 1
    want, z, tol, tol_z = ref.attention(c, causal=False, window=40)
    for r in (0, 1, 2000):
        assert bool(((O[r].double() - want[r]).abs() <= tol[r]).all())
        assert bool(((lse[r].double() - z[r]).abs() <= tol_z[r]).all())
    assert bool((O[2:2000] == 7).all())


@gpu
def test_offsets_past_32_bits():
    # a pool of over 2^31 bytes of codes whose last pages are used
    pages, heads, page, D = 18000, 8, 64, 256
    cache = hbl.kv_cache_alloc(pages, page, heads, D, 8, DEV)
    n = 150
    table = torch.tensor([[pages - 1, 0, pages - 2]], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    k, v, q = (torch.randn(n, heads, D, device=DEV).to(torch.bfloat16) for _ in range(3))
    hbl.kv_cache_write(cache, k, v, cu, lens, table)
    K, V = hbl.kv_cache_read(cache, cu, lens, table, n, dtype=torch.float32)
    u, s = ref.quantise(k.cpu(), 8)
    assert torch.equal(K.cpu(), (u - 128).float() * s[..., None])
    small = hbl.kv_cache_alloc(3, page, heads, D, 8, DEV)
    t2 = torch.tensor([[2, 0, 1]], dtype=torch.int32, device=DEV)
    hbl.kv_cache_write(small, k, v, cu, lens, t2)
    assert torch.equal(hbl.kv_attention(q, cache, cu, lens, table),
                       hbl.kv_attention(q, small, cu, lens, t2))


# ---------------------------------------------------------------- together

@gpu
def test_prefill_then_decode_then_projection():
    """A prompt in two chunks, then tokens one by one, each attention's output
    through the H-BitLinear output projection; against the 64-bit attention of
    the same cache and the oracle's layer."""
    H, KV, D, bits = 8, 2, 64, 4
    cache = hbl.kv_cache_alloc(40, 16, KV, D, bits, DEV)
    g = torch.Generator().manual_seed(0)
    table = torch.randperm(40, generator=g).to(torch.int32).view(2, 20).to(DEV)
    packed, alpha = hbl.pack_ternary(torch.from_numpy(inputs.latent_weights(256, H * D, seed=3)).to(DEV))
    lens = [0, 0]
    for new in ([70, 33], [50, 1], [1, 1], [1, 1], [1, 0]):
        lens = [a + b for a, b in zip(lens, new)]
        rows = sum(new)
        qkv = torch.randn(rows, H + 2 * KV, D, generator=g).to(torch.bfloat16).to(DEV)
        cu = torch.tensor([0] + new).cumsum(0).to(torch.int32).to(DEV)
        kv_lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        status = hbl.new_status(DEV)
        hbl.kv_cache_write(cache, qkv[:, H:H + KV], qkv[:, H + KV:], cu, kv_lens, table, status=status)
        O, lse = hbl.kv_attention(qkv[:, :H], cache, cu, kv_lens, table, max_rows=max(new),
                                  want_lse=True, status=status)
        Y = hbl.hbitlinear_forward(O.view(rows, H * D), packed, alpha, 4)
        assert int(status[0]) == 0
        c = ref.Case(new, lens, heads=H, kv_heads=KV, D=D, bits=bits)
        c.cache, c.table, c.q, c.cu, c.kv_lens = cache, table, qkv[:, :H], cu, kv_lens
        ref.check_attention(c, O, lse)
        wp, wa = (packed.cpu().numpy().view(np.uint32), float(alpha[0]))
        want = oracle.hbitlinear_forward(
            O.view(rows, H * D).view(torch.int16).cpu().numpy().view(np.uint16), wp, wa, 4)
        assert np.array_equal(Y.view(torch.int16).cpu().numpy().view(np.uint16), want)


@gpu
@pytest.mark.parametrize("new,lens", [([1, 1, 1], [800, 5, 300]), ([90, 1], [600, 80])])
def test_captured_steps_replay_with_new_lengths(new, lens):
    """Two graphs over one cache, a workspace each, replayed with other lengths
    than they were captured with."""
    c = ref.Case(new, lens, heads=8, kv_heads=2, D=64, bits=4, seed=6, wide=60)
    graphs = []
    side = torch.cuda.Stream()
    need = hbl.kv_attention_workspace_size(c.rows, 8, c.cache, len(new), 60, max_rows=max(new))
    for _ in range(2):
        out = torch.zeros(c.rows, 8, 64, dtype=torch.bfloat16, device=DEV)
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
        run = lambda: hbl.kv_attention(c.q, c.cache, *c.batch, max_rows=max(new), out=out, ws=ws)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            run()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            hbl.kv_cache_write(c.cache, c.k, c.v, *c.batch)
            run()
        graphs.append((graph, out, ws))
    for shorter in ([0, 0, 0][:len(new)], [7, 0, 11][:len(new)]):
        c.lens = [m - s for m, s in zip(lens, shorter)]
        c.kv_lens.copy_(torch.tensor(c.lens, dtype=torch.int32))
        for graph, out, _ in graphs:
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            ref.check_attention(c, out)


@gpu
def test_two_streams_at_once():
    cases = [ref.Case([1, 1], [5000, 300], heads=8, kv_heads=2, D=128, bits=4, seed=s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                outs.append((c, hbl.kv_attention(c.q, c.cache, *c.batch, max_rows=1)))
    torch.cuda.synchronize()
    for c, O in outs[-2:]:
        ref.check_attention(c, O)


@gpu
def test_binding_refusals_on_the_device():
    c = ref.Case([2], [20], heads=2, kv_heads=2, D=64, bits=4)
    with pytest.raises(ValueError):
        hbl.kv_cache_write(c.cache, c.k[:, :1], c.v[:, :1], *c.batch)
    with pytest.raises(TypeError):
        hbl.kv_cache_write(c.cache, c.k.float(), c.v.float(), *c.batch)
    with pytest.raises(TypeError):
        hbl.kv_attention(c.q, c.cache, c.cu.long(), c.kv_lens, c.table)
    with pytest.raises(ValueError):
        hbl.kv_attention(c.q, c.cache, c.cu[:1], c.kv_lens, c.table)
    with pytest.raises(TypeError):
        hbl.kv_cache_read(c.cache, *c.batch, c.rows, dtype=torch.float16)
    with pytest.raises(ValueError):
        hbl.KvCache(c.cache.k_codes, c.cache.k_scales, c.cache.v_codes, c.cache.v_scales, 100)
    with pytest.raises(hbl.HblError):
        hbl.kv_attention(torch.zeros(2, 3, 64, dtype=torch.bfloat16, device=DEV), c.cache, *c.batch)
    one = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device=DEV)
    for out in (one.expand(2, 2, 64), one[:, :1].expand(2, 2, 64)):
        with pytest.raises(ValueError):
            hbl.kv_attention(c.q, c.cache, *c.batch, out=out)
