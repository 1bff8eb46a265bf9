// k13_kv_decode.cuh -- attention of few rows (one token, or a few, per sequence)
// over the paged low-bit cache.
//
// For a row at position p and a query head over cached head h, with the stored
// codes k, v (integers in [-2^(b-1), 2^(b-1))) and scales sk, sv:
//   x_i = scale * log2(e) * sk_i * (q . k_i) + log2(sv_i)
//   O   = sum_i 2^(x_i - m) v_i / sum_i 2^(x_i - m) / sv_i,   m = max x_i
// in one pass with the running m: taking V's scale into the exponent leaves the
// integer codes as the second product's operand, and the weights 2^(x_i - m)
// in (0, 1], so that fp16 holds them (times 2^14; what is below 2^-39 of
// the row's largest term is lost, a term's rounding is 2^-12 of itself).
//
// What bounds it: the codes and scales of every visible position are read once
// per cached head, 2*D*b/8 + 8 bytes a position (HBM).  Per code it can afford
// about 3 (4 bits) to 1.5 (2 bits) lane instructions at that rate, and the G
// query heads of a cached head share the codes: so the products run on
// mma.sync, whose A fragments are widened in registers straight from the codes
// (a tcgen05 operand would have to go through shared or tensor memory first; the
// tensor rate is far from the limit here, a warp's 16 positions x D codes
// are two m16n8k16 per 256 codes).
//
// One CTA: one sequence, cached head, block of 8*NT rows (query heads of the
// sequence's new tokens) and a range of positions; its warps take 32 positions
// in turn, each through a ring of cp.async stages of its own (no CTA barrier in
// the loop), and join their (m, sum, O) in shared memory.  Ranges of one
// sequence are joined by the combine kernel.
//
// Fragments.  Positions are the M of both products (S^T = K Q^T, 16 positions x
// 8 rows; O^T = V^T P^T, 16 values x 8 rows), so eight rows waste nothing.
// The contraction may run over D in any order: lane t of a quad takes D/4
// consecutive codes of its position, in the pair order that widening gives, and
// Q's fragment is laid out to match.  Slot r of a block of 16 positions is
// position (r >> 1 & 3) + 4 * (r & 1) + (r & 8), so that lane t's four V rows are t,
// t + 4, t + 8, t + 12 (neighbouring lanes read neighbouring rows).  P^T becomes
// the second product's B fragment by an 8x8 transpose of each half.
#pragma once

#include <math_constants.h>

#include "hbl_kv_codes.cuh"
#include "k12_kv_attention.cuh"

namespace hbl {
namespace k13 {

using k12::Plan;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int KW = 32;                     // positions of one warp step
constexpr float kShift = 14.f;             // weights are held times 2^14

template <int D, int B>
struct Stage {
    static constexpr int kRow = D * B / 8;
    static constexpr int kCodes = KW * kRow;                        // K's or V's
    static constexpr int kScales = KW * 4;
    static constexpr int kBytes = 2 * kCodes + 2 * kScales + 16;    // + the flags word
    // stages of one warp: about 12 KB in flight, at least two
    static constexpr int kCount = kBytes * 4 <= 20480 ? 4 : kBytes * 3 <= 26000 ? 3 : 2;
};
template <int D, int B, int NT>
constexpr int smem_bytes() {
    const int ring = kWarps * Stage<D, B>::kCount * Stage<D, B>::kBytes + 16;
    const int join = kWarps * 8 * NT * (D + 4) * 4 + kWarps * 8 * NT * 8;
    return ring > join ? ring : join;
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
__device__ __forceinline__ uint32_t f2_to_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float lg2(float x) {
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

template <int D, int B, int NT>
__global__ void __launch_bounds__(kThreads) decode_kernel(KvCache c, KvBatch kb, KvAttn a, Plan pl,
                                                          float* part, int32_t* status) {
    using St = Stage<D, B>;
    constexpr int R = 8 * NT;            // rows of the block
    constexpr int NK = D / 4, NV = D / 8;  // codes of a lane's K row, of its V rows
    constexpr int kPairs = D / 8;        // K pairs of a lane
    constexpr int H = kKvHalfCodes<B>;
    extern __shared__ __align__(16) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;

    // ---- which rows, which positions
    const int split = (int)(blockIdx.x % pl.splits);
    const int rb = (int)(blockIdx.x / pl.splits % pl.row_blocks);
    const int b = (int)(blockIdx.x / pl.splits / pl.row_blocks), h = (int)blockIdx.y;
    const k12::Rows s = k12::rows_of(kb, c.page_size, a, b);
    if (s.bad && split == 0 && rb == 0 && h == 0 && threadIdx.x == 0)
        report_status(status, HBL_ERR_INVALID_ARG);
    const int nr = s.n * a.group;  // this sequence's rows on this head
    if (nr < pl.min_rows || nr > pl.max_rows || rb * R >= nr) return;
    const k12::Range rg = k12::range_of(a, s, rb * R, min(nr, rb * R + R) - 1);
    const k12::Split sp = k12::split_of(pl, rg, split);
    if (split >= max(sp.count, 1)) return;
    pdl_launch_dependents();

    // per lane: the visible range of rows 2t, 2t + 1 of each tile
    int lo[NT][2], hi[NT][2];
    int all_lo = 0, all_hi = 0x7fffffff;  // every row sees [all_lo, all_hi)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = min(rb * R + 8 * n + 2 * t + e, nr - 1);
            const k12::Range w = k12::range_of(a, s, r, r);
            lo[n][e] = w.begin;
            hi[n][e] = w.end;
            all_lo = max(all_lo, w.begin);
            all_hi = min(all_hi, w.end);
        }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        all_lo = max(all_lo, __shfl_xor_sync(0xffffffffu, all_lo, o));
        all_hi = min(all_hi, __shfl_xor_sync(0xffffffffu, all_hi, o));
    }

    // ---- the ring of this warp
    const uint32_t ring = smem_addr(smem) + warp * St::kCount * St::kBytes;
    const int step = kWarps * KW;
    const int first = sp.begin + warp * KW;
    const int steps = first < sp.end ? (sp.end - first + step - 1) / step : 0;
    // lanes 0, 1 (and all others alike): the page of segment lane & 1 of a step
    auto page_of = [&](int it) {
        const int key = first + it * step + 16 * (lane & 1);
        if (it >= steps || key >= sp.end) return -2;  // nothing there
        return kv_page(kb, c.num_pages, b, (int)pl.div_page(key));
    };
    auto issue = [&](int it, int page) {
        if (it < steps) {
            const uint32_t st = ring + (it % St::kCount) * St::kBytes;
            const int key = first + it * step + 16 * (lane & 1);
            int64_t base = 0;
            if (page >= 0)
                base = ((int64_t)page * c.heads + h) * c.page_size +
                       (key - (int)pl.div_page(key) * c.page_size);
            int64_t row[2];
            bool ok[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                row[e] = __shfl_sync(0xffffffffu, base, e);
                ok[e] = __shfl_sync(0xffffffffu, page, e) >= 0;
            }
            constexpr int kChunks = 2 * St::kRow;  // 16-byte pieces: 16 rows of kRow bytes, twice
#pragma unroll
            for (int k = 0; k < (kChunks + 31) / 32; ++k) {
                const int ch = lane + 32 * k;
                if (kChunks % 32 == 0 || ch < kChunks) {
                    const int seg = ch >= St::kRow, off = (ch - seg * St::kRow) * 16;
                    const int64_t at = (seg ? row[1] : row[0]) * St::kRow + off;
                    const int bytes = (seg ? ok[1] : ok[0]) ? 16 : 0;
                    cp_async16(st + ch * 16, c.kc + at, bytes);
                    cp_async16(st + St::kCodes + ch * 16, c.vc + at, bytes);
                }
            }
            if (lane < 16) {  // the scales: 2 segments x 4 pieces, of K and of V
                const int seg = (lane >> 2) & 1, off = (lane & 3) * 4;
                const float* src = (lane < 8 ? c.ks : c.vs) + (seg ? row[1] : row[0]) + off;
                cp_async16(st + 2 * St::kCodes + lane * 16, src, (seg ? ok[1] : ok[0]) ? 16 : 0);
            }
            if (lane == 0) {
                const uint32_t flags = (ok[0] ? 1u : 0u) | (ok[1] ? 2u : 0u);
                asm volatile("st.shared.u32 [%0], %1;" ::"r"(st + 2 * St::kCodes + 2 * St::kScales),
                             "r"(flags)
                             : "memory");
            }
            if (page == -1) report_status(status, HBL_ERR_INVALID_ARG);
        }
        cp_async_commit();
    };
#pragma unroll
    for (int it = 0; it < St::kCount - 1; ++it) issue(it, page_of(it));
    int next_page = page_of(St::kCount - 1);

    // ---- Q's fragments: pair p of lane t is codes (C w + i, C w + i + C/2), C = 2H
    uint32_t q[NT][kPairs];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int r = rb * R + 8 * n + g;
        uint32_t raw[NK / 2];
        const int i = r / a.group;
        const uint16_t* src = a.q + (int64_t)(s.row0 + i) * a.q_row +
                              (int64_t)(h * a.group + (r - i * a.group)) * a.q_head + t * NK;
#pragma unroll
        for (int k = 0; k < NK / 8; ++k) {
            const uint4 v = r < nr ? reinterpret_cast<const uint4*>(src)[k] : make_uint4(0, 0, 0, 0);
            raw[4 * k] = v.x;
            raw[4 * k + 1] = v.y;
            raw[4 * k + 2] = v.z;
            raw[4 * k + 3] = v.w;
        }
        constexpr int C = NK < 2 * H ? NK : 2 * H;
        static_for<0, kPairs>([&](auto pp) {
            constexpr int p = decltype(pp)::value, w = p / (C / 2), i0 = p % (C / 2);
            constexpr int e0 = C * w + i0, e1 = e0 + C / 2;
            q[n][p] = __byte_perm(raw[e0 / 2], raw[e1 / 2],
                                  (e0 & 1 ? 0x32 : 0x10) | (e1 & 1 ? 0x7600 : 0x5400));
        });
    }

    float O[NV / 2][NT][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int k = 0; k < NV / 2; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) O[k][n][e] = 0.f;
        m[n][0] = m[n][1] = -CUDART_INF_F;
        l[n][0] = l[n][1] = 0.f;
    }
    const float xscale = a.scale * 1.4426950408889634f;
    const int kslot = (g >> 1) + 4 * (g & 1);  // this lane's K rows: kslot, kslot + 8

    for (int it = 0; it < steps; ++it) {
        asm volatile("cp.async.wait_group %0;" ::"n"(St::kCount - 2) : "memory");
        __syncwarp();
        issue(it + St::kCount - 1, next_page);
        next_page = page_of(it + St::kCount);
        const uint32_t st = ring + (it % St::kCount) * St::kBytes;
        const int key0 = first + it * step;
        const uint32_t flags = lds32(st + 2 * St::kCodes + 2 * St::kScales);
        const bool plain = flags == 3u && key0 >= all_lo && key0 + KW <= min(all_hi, sp.end);

        float S[2][NT][4];
        float rsv[2][2];  // 1 / sv of positions kslot, kslot + 8 of each block
#pragma unroll
        for (int blk = 0; blk < 2; ++blk) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) S[blk][n][e] = 0.f;
            const uint32_t r0 = st + (16 * blk + kslot) * St::kRow;
            uint32_t w0[kKvWords<B, NK>], w1[kKvWords<B, NK>];
            kv_lds_codes<B, NK>(r0, t, w0);
            kv_lds_codes<B, NK>(r0 + 8 * St::kRow, t, w1);
            if constexpr (NK < 2 * H) {  // 8 codes of 2 bits: one half word, split in two of 4
                w0[0] = (w0[0] & 0xffu) | ((w0[0] & 0xff00u) << 8);
                w1[0] = (w1[0] & 0xffu) | ((w1[0] & 0xff00u) << 8);
            }
            constexpr int P = NK < 2 * H ? NK / 2 : H;  // pairs of a word
            static_for<0, kKvWords<B, NK>>([&](auto ww) {
                constexpr int w = decltype(ww)::value;
                uint32_t a0[P], a1[P];
                kv_widen_bf16<B, P>(w0[w], a0);
                kv_widen_bf16<B, P>(w1[w], a1);
#pragma unroll
                for (int p = 0; p < P; p += 2)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma_bf16(S[blk][n], a0[p], a1[p], a0[p + 1], a1[p + 1], q[n][P * w + p],
                                 q[n][P * w + p + 1]);
            });
        }
        // ---- exponents; what is not visible becomes -inf, whatever is stored there
        float mx[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) mx[n][0] = mx[n][1] = -CUDART_INF_F;
#pragma unroll
        for (int blk = 0; blk < 2; ++blk)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int slot = 16 * blk + kslot + 8 * u, key = key0 + slot;
                const uint32_t sc = st + 2 * St::kCodes + 4 * slot;
                const float sk = __uint_as_float(lds32(sc));
                const float sv = __uint_as_float(lds32(sc + St::kScales));
                const bool there = plain || (((flags >> blk) & 1u) != 0 && key < sp.end);
                const float ck = there ? __fmul_rn(sk, xscale) : 0.f;
                // a zero scale (an all-zero row: its codes are zero too) as 2^-100
                const float lv = there ? fmaxf(lg2(sv), -100.f) : 0.f;
                rsv[blk][u] = ex2(-lv);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = __fmaf_rn(S[blk][n][2 * u + e], ck, lv);
                        if (!plain && !(there && key >= lo[n][e] && key < hi[n][e]))
                            x = -CUDART_INF_F;
                        S[blk][n][2 * u + e] = x;
                        mx[n][e] = fmaxf(mx[n][e], x);
                    }
            }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int o = 4; o < 32; o <<= 1)
                    mx[n][e] = fmaxf(mx[n][e], __shfl_xor_sync(0xffffffffu, mx[n][e], o));
        bool grew = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) grew |= mx[n][0] > m[n][0] || mx[n][1] > m[n][1];
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float nm = fmaxf(m[n][e], mx[n][e]);
                    const float f = nm == m[n][e] ? 1.f : ex2(m[n][e] - nm);
                    m[n][e] = nm;
                    l[n][e] *= f;
#pragma unroll
                    for (int k = 0; k < NV / 2; ++k) {
                        O[k][n][e] *= f;
                        O[k][n][2 + e] *= f;
                    }
                }
        }
        // ---- weights and the second product
#pragma unroll
        for (int blk = 0; blk < 2; ++blk) {
            uint32_t p[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    float w[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        // a row that has seen nothing yet: 2^(-inf) = 0 against any base
                        const float base = m[n][e] == -CUDART_INF_F ? 0.f : kShift - m[n][e];
                        w[e] = ex2(S[blk][n][2 * u + e] + base);
                        l[n][e] = __fmaf_rn(w[e], rsv[blk][u], l[n][e]);
                    }
                    p[n][u] = transpose8(f2_to_f16x2(w[0], w[1]));
                }
            const uint32_t r0 = st + St::kCodes + (16 * blk + t) * St::kRow;
            constexpr int W = kKvWords<B, NV>;
            uint32_t v[4][W];
#pragma unroll
            for (int k = 0; k < 4; ++k) kv_lds_codes<B, NV>(r0 + 4 * k * St::kRow, g, v[k]);
            constexpr int P = NV < H ? NV : H;  // values of a half word
            static_for<0, NV / P>([&](auto hh) {
                constexpr int hw = decltype(hh)::value, w = hw / 2;
                constexpr uint32_t sel = hw & 1 ? 0x7632 : 0x5410;
                uint32_t a0[P], a2[P];
                kv_widen_f16<B, P>(__byte_perm(v[0][w], v[1][w], sel), a0);
                kv_widen_f16<B, P>(__byte_perm(v[2][w], v[3][w], sel), a2);
#pragma unroll
                for (int i = 0; i < P; i += 2)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma_f16(O[(P * hw + i) / 2][n], a0[i], a0[i + 1], a2[i], a2[i + 1],
                                p[n][0], p[n][1]);
            });
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");

    // ---- join the warps.  Lane (g, t): values NV g .. of rows 2t, 2t + 1
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], o);
    __syncthreads();  // the rings are free
    float* so = reinterpret_cast<float*>(smem);         // [warp][R][D + 4]
    float* sm = so + kWarps * R * (D + 4);              // [warp][R]: m, then l
    float* sl = sm + kWarps * R;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = 8 * n + 2 * t + e;
            float* dst = so + (warp * R + r) * (D + 4) + g * NV;
            if constexpr (NV >= 4) {
#pragma unroll
                for (int k = 0; k < NV / 4; ++k)
                    reinterpret_cast<float4*>(dst)[k] =
                        make_float4(O[2 * k][n][e], O[2 * k][n][2 + e], O[2 * k + 1][n][e],
                                    O[2 * k + 1][n][2 + e]);
            }
            if (g == 0) {
                sm[warp * R + r] = m[n][e];
                sl[warp * R + r] = l[n][e];
            }
        }
    __syncthreads();
    constexpr int kPer = D / 4;  // threads of a row, four values each
    for (int x = threadIdx.x; x < R * kPer; x += kThreads) {
        const int r = x / kPer, d = (x % kPer) * 4, row = rb * R + r;
        if (row >= nr) break;
        float M = -CUDART_INF_F;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w * R + r]);
        float L = 0.f;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float mw = sm[w * R + r];
            const float f = mw == -CUDART_INF_F ? 0.f : ex2(mw - M);
            const float4 v = *reinterpret_cast<const float4*>(so + (w * R + r) * (D + 4) + d);
            L = __fmaf_rn(sl[w * R + r], f, L);
            y.x = __fmaf_rn(v.x, f, y.x);
            y.y = __fmaf_rn(v.y, f, y.y);
            y.z = __fmaf_rn(v.z, f, y.z);
            y.w = __fmaf_rn(v.w, f, y.w);
        }
        if (sp.count <= 1) {
            k12::store_row<4>(a, s, h, row, d, &y.x, M - kShift, L);
        } else {
            float* dst = part + k12::part_index(pl, c, b, h, split, row) * (D + 4);
            *reinterpret_cast<float4*>(dst + d) = y;
            if (d == 0) *reinterpret_cast<float2*>(dst + D) = make_float2(M - kShift, L);
        }
    }
}

template <int D, int B, int NT>
hbl_status launch(const KvCache& c, const KvBatch& kb, const KvAttn& a, const Plan& pl, float* part,
                  int32_t* status, cudaStream_t stream) {
    constexpr int kSmem = smem_bytes<D, B, NT>();
    auto kern = decode_kernel<D, B, NT>;
    if (!smem_attr_once(reinterpret_cast<const void*>(kern), kSmem)) return HBL_ERR_CUDA;
    const dim3 grid((unsigned)(kb.num_seqs * pl.row_blocks * pl.splits), (unsigned)c.heads);
    kern<<<grid, kThreads, kSmem, stream>>>(c, kb, a, pl, part, status);
    return cudaGetLastError() == cudaSuccess ? HBL_OK : HBL_ERR_CUDA;
}

template <int D>
hbl_status launch_d(const KvCache& c, const KvBatch& kb, const KvAttn& a, const Plan& pl, float* part,
                    int32_t* status, cudaStream_t stream) {
    auto by_nt = [&](auto bits) -> hbl_status {
        constexpr int B = decltype(bits)::value;
        if constexpr (D <= 128) {
            if (pl.block_rows == 16) return launch<D, B, 2>(c, kb, a, pl, part, status, stream);
        }
        return launch<D, B, 1>(c, kb, a, pl, part, status, stream);
    };
    switch (c.bits) {
        case 2: return by_nt(ic<2>{});
        case 3: return by_nt(ic<3>{});
        case 4: return by_nt(ic<4>{});
        default: return by_nt(ic<8>{});
    }
}

}  // namespace k13
}  // namespace hbl
