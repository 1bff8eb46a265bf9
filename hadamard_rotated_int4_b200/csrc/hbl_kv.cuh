// hbl_kv.cuh -- device helpers shared by the KV kernels: the absmax quantiser of
// one head row, the packed-code layout, and the paged batch's addressing.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "hbl_internal.cuh"
#include "hbl_launch.h"

namespace hbl {

// ------------------------------------------------------------ codes of 16 values
// A lane holds 16 values of a row, D/16 lanes a row.  Its 16 codes are 16*B
// contiguous bits: two halves of 8 codes, code i of a half at bits [B*i, B*i+B).
constexpr int kKvVpl = 16;

template <int B>
using KvHalf = typename std::conditional<(8 * B <= 32), uint32_t, uint64_t>::type;

// Quantises a row spread over D/16 neighbouring lanes (bf16 bits in raw):
// gamma = max|x| over those lanes, inv = Qp / (gamma + eps) (one division),
// u = clip(rhe(x * inv), -Qp - 1, Qp) + 2^(B-1), each product rounded once by an
// fma with 1.5 * 2^23.  Where inv is finite, no product needs the clip: |x| <= gamma,
// so |x * inv| <= Qp up to the rounding of inv (well under half a unit).  It is infinite
// exactly where gamma + eps <= Qp * 2^-128, with eps = 0 or nearly: then *over is set,
// and the codes are kv_ends16's, from the row loaded once more (kept in registers for
// that rare case, it costs K11 spills).  Returns gamma / Qp.
// Every lane of the warp calls it (the max goes through shuffles).
template <int D, int B>
__device__ __forceinline__ float kv_quant16(const uint4 (&raw)[2], float eps, KvHalf<B> (&h)[2],
                                            bool* over) {
    constexpr int QP = (1 << (B - 1)) - 1;
    constexpr int32_t kMagicBits = 0x4B400000;  // 1.5 * 2^23
    const float qp = (float)QP;
    float x[kKvVpl];
    const uint32_t w[8] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w,
                           raw[1].x, raw[1].y, raw[1].z, raw[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 f = bf16x2_to_f2(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
    float g = 0.f;
#pragma unroll
    for (int i = 0; i < kKvVpl; ++i) g = fmaxf(g, fabsf(x[i]));
#pragma unroll
    for (int o = 1; o < D / kKvVpl; o <<= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
    const float den = __fadd_rn(g, eps);
    *over = den <= qp * 0x1p-128f;
    const float inv = __fdiv_rn(qp, den);
    h[0] = 0;
    h[1] = 0;
#pragma unroll
    for (int i = 0; i < kKvVpl; ++i) {
        const int32_t b = __float_as_int(__fmaf_rn(x[i], inv, 12582912.0f));
        const uint32_t code = (uint32_t)(b - kMagicBits + (QP + 1));
        h[i / 8] |= (KvHalf<B>)code << (B * (i % 8));
    }
    return __fdiv_rn(g, qp);
}

// Codes of 16 values for an infinite inv: the clip's ends by their signs, zero for zeros
// (gamma + eps = 0 among them).
template <int B>
__device__ __forceinline__ void kv_ends16(const uint4 (&raw)[2], KvHalf<B> (&h)[2]) {
    const uint32_t w[8] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w,
                           raw[1].x, raw[1].y, raw[1].z, raw[1].w};
    h[0] = 0;
    h[1] = 0;
#pragma unroll
    for (int i = 0; i < kKvVpl; ++i) {
        const uint32_t x = w[i / 2] >> (16 * (i % 2));
        const uint32_t code = (x & 0x7fffu) == 0    ? 1u << (B - 1)
                              : (x & 0x8000u) != 0 ? 0u
                                                   : (1u << B) - 1u;
        h[i / 8] |= (KvHalf<B>)code << (B * (i % 8));
    }
}

// Stores lane li's 16 codes of the row at dst (D*B/8 bytes).  Every lane of the
// warp calls it (3-bit lane pairs share a 12-byte group through a shuffle).
template <int B>
__device__ __forceinline__ void kv_store16(uint8_t* dst, int li, const KvHalf<B> (&h)[2], bool ok) {
    if constexpr (B == 8) {  // 16 bytes per lane
        if (ok)
            *reinterpret_cast<uint4*>(dst + li * 16) =
                make_uint4((uint32_t)h[0], (uint32_t)((uint64_t)h[0] >> 32), (uint32_t)h[1],
                           (uint32_t)((uint64_t)h[1] >> 32));
    } else if constexpr (B == 4) {  // 8 bytes per lane
        if (ok) *reinterpret_cast<uint2*>(dst + li * 8) = make_uint2(h[0], h[1]);
    } else if constexpr (B == 2) {  // 4 bytes per lane
        if (ok) *reinterpret_cast<uint32_t*>(dst + li * 4) = h[0] | (h[1] << 16);
    } else {  // B == 3: 48 bits per lane; a lane pair makes one 12-byte group
        const uint64_t mine = (uint64_t)h[0] | ((uint64_t)h[1] << 24);
        const uint64_t next = __shfl_down_sync(0xffffffffu, mine, 1);
        if (ok && (li & 1) == 0) {
            uint32_t* d32 = reinterpret_cast<uint32_t*>(dst + (li >> 1) * 12);
            d32[0] = (uint32_t)mine;
            d32[1] = (uint32_t)(mine >> 32) | ((uint32_t)next << 16);
            d32[2] = (uint32_t)(next >> 16);
        }
    }
}

// Loads lane li's 16 codes of the row at src: h as kv_quant16 leaves them.
template <int B>
__device__ __forceinline__ void kv_load16(const uint8_t* src, int li, KvHalf<B> (&h)[2]) {
    if constexpr (B == 8) {
        const uint4 v = *reinterpret_cast<const uint4*>(src + li * 16);
        h[0] = (uint64_t)v.x | ((uint64_t)v.y << 32);
        h[1] = (uint64_t)v.z | ((uint64_t)v.w << 32);
    } else if constexpr (B == 4) {
        const uint2 v = *reinterpret_cast<const uint2*>(src + li * 8);
        h[0] = v.x;
        h[1] = v.y;
    } else if constexpr (B == 2) {
        const uint32_t v = *reinterpret_cast<const uint32_t*>(src + li * 4);
        h[0] = v & 0xffffu;
        h[1] = v >> 16;
    } else {  // 48 bits at bit 48 * (li & 1) of the pair's 96
        const uint32_t* s32 = reinterpret_cast<const uint32_t*>(src + (li >> 1) * 12) + (li & 1);
        const uint64_t v = ((uint64_t)s32[0] | ((uint64_t)s32[1] << 32)) >> ((li & 1) * 16);
        h[0] = (uint32_t)v & 0xffffffu;
        h[1] = (uint32_t)(v >> 24) & 0xffffffu;
    }
}

// Two fp32 -> a bf16 pair (low half = first), round to nearest even.
__device__ __forceinline__ uint32_t f2_to_bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Calls f(ic<D>, ic<bits>) for the cache's head size and code width.
template <class F>
hbl_status kv_dispatch(int D, int bits, F&& f) {
    auto by_bits = [&](auto d) -> hbl_status {
        switch (bits) {
            case 2: return f(d, ic<2>{});
            case 3: return f(d, ic<3>{});
            case 4: return f(d, ic<4>{});
            case 8: return f(d, ic<8>{});
            default: return HBL_ERR_INVALID_ARG;
        }
    };
    switch (D) {
        case 32: return by_bits(ic<32>{});
        case 64: return by_bits(ic<64>{});
        case 128: return by_bits(ic<128>{});
        case 256: return by_bits(ic<256>{});
        default: return HBL_ERR_SHAPE;
    }
}

__device__ __forceinline__ void sts32(uint32_t at, uint32_t v) {
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

__device__ __forceinline__ void or_shared(uint32_t at, uint32_t v) {
    asm volatile("red.shared.or.b32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

// ------------------------------------------------------------ waits of a pipeline

// Waits for an mbarrier phase, for at most `limit` SM clocks (about two seconds), and
// while *abort_flag (if given) is zero.  Polls in a bare loop and looks at the flag
// and the clock now and then only: in kernels that hand over every few hundred
// cycles, reading the global timer at each failed poll costs more than the wait.
constexpr int64_t kWaitClocks = 4000000000ll;
__device__ __forceinline__ bool mbar_wait_clock(uint32_t bar, uint32_t parity,
                                                const volatile int* abort_flag,
                                                int64_t limit = kWaitClocks) {
    int64_t t0 = 0;
    for (uint32_t n = 1;; ++n) {
        if (mbar_test_parity(bar, parity)) return true;
        if ((n & 127u) == 0) {
            if (abort_flag != nullptr && *abort_flag) return false;
            const int64_t t = clock64();
            if (t0 == 0) t0 = t;
            if (t - t0 > limit) return false;
        }
    }
}

// ------------------------------------------------------------ the paged batch

// One sequence of the batch: rows [r0, r1) of the packed new rows, `len`
// positions in all; row t stands at position len - (c1 - t) = first + (t - r0), c1 the
// end that the descriptors give (negative for rows that the length does not reach).
// Of descriptors outside their bounds the rows and positions that do not exist are cut
// off, so nothing out of range is ever addressed, and `bad` is set; the others stay
// where the descriptors put them: a row moved to another position would take the place
// of one that is cached there.
struct KvSeq {
    int r0, r1, first, len;
    bool bad;
};
__device__ __forceinline__ bool kv_bad(const KvBatch& kb, int cap, int c0, int c1, int n) {
    return c0 < 0 || c1 < c0 || c1 > kb.rows || (unsigned)n > (unsigned)cap;
}
__device__ __forceinline__ int kv_capacity(const KvBatch& kb, int page_size) {
    return kb.pages_per_seq * page_size;  // (at most 2^31 - 4096)
}
__device__ __forceinline__ KvSeq kv_seq(const KvBatch& kb, int page_size, int b) {
    const int c0 = __ldg(kb.cu + b), c1 = __ldg(kb.cu + b + 1), n = __ldg(kb.lens + b);
    const int cap = kv_capacity(kb, page_size);
    KvSeq s;
    s.r0 = min(max(c0, 0), kb.rows);
    s.r1 = min(max(c1, s.r0), kb.rows);
    s.len = min(max(n, 0), cap);
    // (where there are rows, r0 < c1: no overflow; where n < 0, all have no place)
    s.first = (int)((unsigned)max(n, 0) - (unsigned)c1 + (unsigned)s.r0);
    if (n > cap) s.r1 = max(s.r0, min(s.r1, c1 - (n - cap)));  // rows past the table
    s.bad = kv_bad(kb, cap, c0, c1, n);
    return s;
}

// The sequence and position of packed row t, found by the whole warp (every lane calls
// it with the same t): the sequence is that whose rows end first behind t.  One round
// of loads for 32 sequences: their ends and lengths come together, and the found one's
// are handed round.  in_seq is false for a row before the first sequence, behind the
// last one or past the table; pos is below the sequence's clamped length, and negative
// for a row without a place.  bad is set on lanes that met a descriptor outside its
// bounds on the way.
struct KvRow {
    int b, pos;
    bool in_seq;
};
__device__ __forceinline__ KvRow kv_row(const KvBatch& kb, int page_size, int t, bool* bad) {
    const int lane = threadIdx.x & 31, cap = kv_capacity(kb, page_size);
    KvRow r = {kb.num_seqs, 0, false};
    int before = __ldg(kb.cu);  // where the sequences looked at begin
    for (int i = 0; i < kb.num_seqs; i += 32) {
        const bool in = i + lane < kb.num_seqs;
        const int end = in ? __ldg(kb.cu + i + lane + 1) : 0;
        const int n = in ? __ldg(kb.lens + i + lane) : 0;
        const uint32_t after = __ballot_sync(0xffffffffu, in && end > t);
        // the descriptors are checked as they come by (a falling or far end, a length
        // past the table), whether row t is theirs or not
        int start = __shfl_up_sync(0xffffffffu, end, 1);
        if (lane == 0) start = before;
        if (in && kv_bad(kb, cap, start, end, n)) *bad = true;
        if (after != 0) {
            const int k = __ffs(after) - 1;
            const int c1 = __shfl_sync(0xffffffffu, end, k), len = __shfl_sync(0xffffffffu, n, k);
            const int c0 = __shfl_sync(0xffffffffu, start, k);
            r.b = i + k;
            r.pos = max(len, 0) - (c1 - t);
            r.in_seq = t >= c0 && r.pos < cap;
            break;
        }
        before = __shfl_sync(0xffffffffu, end, 31);
    }
    return r;
}

// The page that holds position pos of sequence b, or -1 if the block table names
// a page outside the pool.  0 <= pos < the sequence's clamped length.
__device__ __forceinline__ int kv_page(const KvBatch& kb, int num_pages, int b, int page_index) {
    const int page = __ldg(kb.table + (int64_t)b * kb.pages_per_seq + page_index);
    return (unsigned)page < (unsigned)num_pages ? page : -1;
}

}  // namespace hbl
