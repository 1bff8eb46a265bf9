// hbl_kv_codes.cuh -- packed cache codes widened to 16-bit floats for the tensor
// cores, exactly (u - 2^(B-1) is an integer of at most 8 bits).
//
// The widening works on "half words": 16 bits holding kHalf<B> consecutive codes
// (8 of 2 bits, 4 of 4, 2 of 8; 3-bit codes are first laid out as 12 of every 16
// bits), two half words to a register.  Masking code i of both halves and
// or-ing an exponent above it gives two floats 2^m + u * 2^(B*i) at once (m the
// mantissa width: 10 for fp16, 7 for bf16); one packed fma takes the offset off
// and scales u back.  Codes whose bits pass the mantissa are shifted down first,
// several codes to a shift.  Per pair that is one logic operation, one fma and
// a share of a shift: about one instruction per code.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "hbl_kv.cuh"

namespace hbl {

template <int B>
constexpr int kKvHalfCodes = B == 2 ? 8 : B == 8 ? 2 : 4;

__device__ __forceinline__ uint32_t hfma2_u(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t bfma2_u(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
// (x & mask) | bits in one operation (written as two, the compiler makes two of
// them: only one of its operands can be a constant).
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(x), "r"(mask), "r"(bits));
    return d;
}
__device__ __forceinline__ uint32_t and_xor(uint32_t x, uint32_t mask, uint32_t bits) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(d) : "r"(x), "r"(mask), "r"(bits));
    return d;
}
// Bits of a small power-of-two or integer-valued constant, both halves.
__host__ __device__ constexpr uint32_t pow2_f16(int e) { return (uint32_t)((e + 15) << 10); }
__host__ __device__ constexpr uint32_t pow2_bf16(int e) { return (uint32_t)((e + 127) << 7); }
__host__ __device__ constexpr uint32_t neg_int_bits(int v, int mant, int bias) {  // -v, v > 0
    int e = 0;
    while ((v >> (e + 1)) != 0) ++e;
    return 0x8000u | (uint32_t)((e + bias) << mant) |
           (uint32_t)(((v << mant) >> e) & ((1 << mant) - 1));
}
__host__ __device__ constexpr uint32_t twice(uint32_t h) { return h | (h << 16); }

// out[i] = (code i of the low half, code i of the high half), minus 2^(B-1), as
// fp16 pairs, for the first N codes.
template <int B, int N>
__device__ __forceinline__ void kv_widen_f16(uint32_t x, uint32_t (&out)[N]) {
    constexpr int kPer = B == 8 ? 1 : B == 2 ? 4 : 2;  // codes that fit 10 mantissa bits
    constexpr int kOff = 1 << (B - 1);
    static_for<0, N>([&](auto ii) {
        constexpr int i = decltype(ii)::value, at = B * (i % kPer), sh = B * (i - i % kPer);
        constexpr uint32_t mask = twice(((1u << B) - 1u) << at);
        const uint32_t v = and_or(x >> sh, mask, 0x64006400u);  // 1024 + u * 2^at
        out[i] = hfma2_u(v, twice(pow2_f16(-at)), twice(neg_int_bits((1024 >> at) + kOff, 10, 15)));
    });
}
// The same as bf16 pairs.
template <int B, int N>
__device__ __forceinline__ void kv_widen_bf16(uint32_t x, uint32_t (&out)[N]) {
    constexpr int kPer = B == 2 ? 3 : B == 3 ? 2 : 1;  // codes that fit 7 mantissa bits
    constexpr int kOff = 1 << (B - 1);
    static_for<0, N>([&](auto ii) {
        constexpr int i = decltype(ii)::value;
        if constexpr (B == 8) {
            // 128 + (u & 127), then -256, or -128 where u's top bit is set (the
            // two constants differ in that bit): u - 128 either way
            const uint32_t y = x >> (8 * i);
            out[i] = bfma2_u(and_or(y, 0x007f007fu, 0x43004300u), twice(pow2_bf16(0)),
                             and_xor(y, 0x00800080u, 0xC380C380u));
        } else {
            constexpr int at = B * (i % kPer), sh = B * (i - i % kPer);
            constexpr uint32_t mask = twice(((1u << B) - 1u) << at);
            const uint32_t v = and_or(x >> sh, mask, 0x43004300u);  // 128 + u * 2^at
            out[i] = bfma2_u(v, twice(pow2_bf16(-at)),
                             twice(neg_int_bits((128 >> at) + kOff, 7, 127)));
        }
    });
}

// N consecutive codes of a row in shared memory, from code index i * N (row at
// byte address `row`, a multiple of 4), as half words, two to a register.
template <int B, int N>
constexpr int kKvWords = (N + 2 * kKvHalfCodes<B> - 1) / (2 * kKvHalfCodes<B>);

// 24 bits of eight 3-bit codes -> two 12-bit halves (what lies above them in
// either half is not cleared: every code is masked out by itself).
__device__ __forceinline__ uint32_t kv_spread3(uint32_t c) {
    return __byte_perm(c, c << 4, 0x7610);
}

template <int B, int N>
__device__ __forceinline__ void kv_lds_codes(uint32_t row, int i, uint32_t (&w)[kKvWords<B, N>]) {
    constexpr int kBits = B * N;
    if constexpr (kBits % 32 == 0) {
        constexpr int kRaw = kBits / 32;
        uint32_t raw[kRaw];
        const uint32_t at = row + i * (kBits / 8);
        if constexpr (kRaw % 4 == 0) {
#pragma unroll
            for (int k = 0; k < kRaw / 4; ++k) {
                const uint4 v = lds128(at + 16 * k);
                raw[4 * k] = v.x;
                raw[4 * k + 1] = v.y;
                raw[4 * k + 2] = v.z;
                raw[4 * k + 3] = v.w;
            }
        } else if constexpr (kRaw % 2 == 0) {
#pragma unroll
            for (int k = 0; k < kRaw / 2; ++k)
                asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                             : "=r"(raw[2 * k]), "=r"(raw[2 * k + 1])
                             : "r"(at + 8 * k)
                             : "memory");
        } else {
#pragma unroll
            for (int k = 0; k < kRaw; ++k) raw[k] = lds32(at + 4 * k);
        }
        if constexpr (B == 3) {  // kRaw is a multiple of 3: four chunks of 24 bits in each
#pragma unroll
            for (int k = 0; k < kRaw / 3; ++k) {
                w[4 * k] = kv_spread3(raw[3 * k]);
                w[4 * k + 1] = kv_spread3(__funnelshift_r(raw[3 * k], raw[3 * k + 1], 24));
                w[4 * k + 2] = kv_spread3(__funnelshift_r(raw[3 * k + 1], raw[3 * k + 2], 16));
                w[4 * k + 3] = kv_spread3(raw[3 * k + 2] >> 8);
            }
        } else {
#pragma unroll
            for (int k = 0; k < kRaw; ++k) w[k] = raw[k];
        }
    } else {
        // 8, 12, 16, 24 or 48 bits at any bit: a window of two words.  The second
        // one of the row's last window may lie behind the row (its bits are
        // not used then); the buffer goes on there.
        const uint32_t bit = (uint32_t)i * kBits, at = row + (bit >> 5) * 4, sh = bit & 31u;
        const uint32_t w0 = lds32(at), w1 = lds32(at + 4);
        const uint32_t lo = __funnelshift_r(w0, w1, sh);
        if constexpr (B == 3 && N >= 8) {
            w[0] = kv_spread3(lo);
            if constexpr (N == 16) w[1] = kv_spread3(__funnelshift_r(lo, w1 >> sh, 24));
        } else {
            w[0] = lo;
        }
    }
}

}  // namespace hbl
