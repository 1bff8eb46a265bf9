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
