// k13_kv_decode.cuh -- attention of few rows (one token, or a few, per sequence)
// over the paged low-bit cache.
//
// For a row at position p and a query head over cached head h, with the stored
// codes k, v (integers in [-2^(b-1), 2^(b-1))) and scales sk, sv:
//   x_i = scale * log2(e) * sk_i * (q . k_i) + log2(sv_i)
//   O   = sum_i 2^(x_i - m) v_i / sum_i 2^(x_i - m) / sv_i,   m = max x_i
// in one pass with the running m: taking V's scale into the exponent leaves the
// integer codes as the second product's operand, and the weights 2^(x_i - m)
// in (0, 2^8], so that fp16 holds them (times 2^6; what is below 2^-31 of
// the reference is lost, a term's rounding is 2^-11 of itself).  Where 1 / sv or a weight
// leaves fp32's range, which takes V scales outside 2^-40 .. 2^40, a part is worked on
// once more with its normaliser summed apart (k12_kv_attention.cuh).
//
// What bounds it: the codes and scales of every visible position are read once
// per cached head, 2*D*b/8 + 8 bytes a position (HBM), and close behind it the
// integer unit, which masks the codes out (one operation to two lanes' worth of
// cycles).  The G query heads of a cached head share the codes, so the products
// run on mma.sync, whose A fragments are made in registers straight from the
// codes (a tcgen05 operand would have to go through shared or tensor memory
// first; the tensor rate is far from the limit here).  Both products run on
// exact integers in fp16, whose ten mantissa bits take two 4-bit codes of a half
// word unshifted (bf16: one).  Q is fp16 times a power of two of its row that
// brings its largest value to [2^14, 2^15): values down to 2^-31 of that are
// exact, smaller ones are off by 2^-39 of it at most.  (Codes left masked as
// subnormal fp16, with the offset taken off the sums, save the fma, but the
// tensor cores align such products by their exponent field and lose ten bits.)
//
// One CTA: an equal piece of the line of all work (k12_kv_attention.cuh): one after
// the other, parts of one sequence, cached head and block of 8*NT rows (query heads
// of the sequence's new tokens).  Its warps take KW positions in turn, each through a
// ring of bulk copies of its own (no CTA barrier in the loop), and join their
// (m, sum, O) in shared memory.  What pieces share of one head is joined by the next
// kernel.  The reference point m follows the running maximum only when a score
// passes it by more than 2^8.
//
// Measured, graph replay, D = 128, 32 query heads over 8: 64 sequences of 1024 to
// 8192 on the 4-bit cache 75 us (44 to read it once), two of 131071 on the 3-bit one
// 75 us (33); five rows of each of 16 sequences, 8-bit, 32 heads of 64, 69 us (44).
// Loads alone take 60 and 43 us in the first two, all but the widening 63 and 54.  With
// a V scale outside 2^-40 .. 2^40 in every part the first takes 167 us, with zero rows
// 95 (a look at all scales; both timed as calls, 83 without).
// Tried and slower: four CTAs an SM with steps of 32 positions (84 against 76 us),
// 16 or 32 positions at a time within a step (82, 78), copies that run ahead into the
// next part (79: the other CTAs of the SM cover the gap already).
//
// Fragments.  Positions are the M of both products (S^T = K Q^T, 16 positions x
// 8 rows; O^T = V^T P^T, 16 values x 8 rows), so eight rows waste nothing.
// The contraction may run over D in any order: lane t of a quad takes D/4
// consecutive codes of its position, in the pair order that masking gives, and
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
constexpr float kShift = 6.f;              // weights are held times 2^6 ...
constexpr float kLazy = 8.f;               // ... and may pass the reference by 2^8

// A warp's step: 64 positions, fewer of long rows, so that two or three stages a
// warp leave room for three CTAs an SM.
template <int D, int B>
struct Stage {
    static constexpr int kRow = D * B / 8;
    static constexpr int KW = kRow <= 64 ? 64 : kRow <= 128 ? 32 : 16;
    static constexpr int kCodes = KW * kRow;                        // K's or V's
    static constexpr int kScales = KW * 4;
    static constexpr int kBytes = 2 * kCodes + 2 * kScales + 16;    // + the flags word
    static constexpr int kCount = kBytes * 3 <= 14000 ? 3 : 2;
};
template <int D, int B, int NT>
__host__ __device__ constexpr int smem_bytes() {
    const int ring = kWarps * Stage<D, B>::kCount * Stage<D, B>::kBytes + 16;
    const int join = kWarps * 8 * NT * (D + 4) * 4 + kWarps * 8 * NT * 8;
    return (ring > join ? ring : join) + kWarps * 32;  // + the barriers
}

// CTAs to an SM that the registers leave room for.
template <int D, int NT>
constexpr int kCtas = NT == 1 && D <= 128 ? 3 : 2;

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

template <int D, int B, int NT>
__global__ void __launch_bounds__(kThreads, kCtas<D, NT>)
    decode_kernel(KvCache c, KvBatch kb, KvAttn a, Plan pl, float* part, int32_t* status) {
    using St = Stage<D, B>;
    constexpr int R = 8 * NT;            // rows of the block
    constexpr int NK = D / 4, NV = D / 8;  // codes of a lane's K row, of its V rows
    constexpr int kPairs = D / 8;        // K pairs of a lane
    constexpr int H = kKvHalfCodes<B>;
    constexpr int KW = St::KW, NB = KW / 16;
    extern __shared__ __align__(16) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;

    // ---- this CTA's piece of the line
    const k12::Line line = k12::line_of<kThreads, false>(pl, c, kb, a, blockIdx.x,
                                                         blockIdx.x == 0 ? status : nullptr);
    int at = line.at;
    if (at >= line.total) return;
    const int stop = (int)min((int64_t)at + line.per, (int64_t)line.total);
    pdl_launch_dependents();

    const uint32_t ring = smem_addr(smem) + warp * St::kCount * St::kBytes;
    const uint32_t bars = smem_addr(smem) + smem_bytes<D, B, NT>() - kWarps * 32 + warp * 32;
    if (lane < St::kCount) mbar_init_count(bars + 8 * lane, 1);
    // flags behind the first warp's barriers (at most three): 1, V's scales need a second pass;
    // 2, a wait gave up
    const uint32_t flags_s = smem_addr(smem) + smem_bytes<D, B, NT>() - kWarps * 32 + 24;
    if (threadIdx.x == 0) sts32(flags_s, 0);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncwarp();
    int done = 0;  // stages of this warp's ring that have been used
    int item = line.item;
    k12::Item im = k12::item_of(pl, c, kb, a, item);
    int before = line.before;  // the line's units before this item
    while (true) {
        // ---- one head's part of an item: units [u0, u1) of im.units
        while (at >= before + im.units * c.heads) {
            before += im.units * c.heads;
            im = k12::item_of(pl, c, kb, a, ++item);
        }
        const int b = item / pl.row_blocks, rb = item - b * pl.row_blocks;
        const int h = (at - before) / im.units, u0 = (at - before) - h * im.units;
        const int u1 = min(im.units, u0 + (stop - at));
        at += u1 - u0;
        const k12::Rows s = im.s;
        const int nr = im.nr;
        const int begin = im.from + u0 * pl.unit;
        const int end = u1 == im.units ? im.rg.end : im.from + u1 * pl.unit;

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
        const int step = kWarps * KW;
        const int first = begin + warp * KW;
        const int steps = first < end ? (end - first + step - 1) / step : 0;
        // one copy takes the positions of one page: seg of them, and a lane to each of
        // K's and V's codes and scales (lane >> 2) of each segment (lane & 3)
        const int seg_shift = min(pl.seg_shift, ilog2(KW)), seg = 1 << seg_shift;
        const int my_seg = lane & 3, my_kind = lane >> 2;
        const bool copies = my_kind < 4 && my_seg < (KW >> seg_shift);
        auto page_of = [&](int it) {
            const int key = first + it * step + (my_seg << seg_shift);
            if (it >= steps || !copies || key >= end) return -2;  // nothing there
            return kv_page(kb, c.num_pages, b, (int)pl.div_page(key));
        };
        uint8_t* const my_base = my_kind == 0 ? c.kc : my_kind == 1 ? c.vc
                                 : reinterpret_cast<uint8_t*>(my_kind == 2 ? c.ks : c.vs);
        const int my_row = my_kind < 2 ? St::kRow : 4;
        const uint32_t my_dst = (my_kind < 2 ? my_kind * St::kCodes
                                             : 2 * St::kCodes + (my_kind - 2) * St::kScales) +
                                (my_seg << seg_shift) * my_row;
        auto issue = [&](int it, int page) {
            if (it >= steps) return;
            const int slot = (done + it) % St::kCount;
            const uint32_t st = ring + slot * St::kBytes, bar = bars + 8 * slot;
            const uint32_t there = __ballot_sync(0xffffffffu, page >= 0);
            if (page == -1) report_status(status, HBL_ERR_INVALID_ARG);
            if (lane == 0) {
                asm volatile("st.shared.u32 [%0], %1;" ::"r"(st + 2 * St::kCodes + 2 * St::kScales),
                             "r"(there & 15u)
                             : "memory");
                asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar),
                             "r"((uint32_t)(__popc(there & 15u) * seg * (2 * St::kRow + 8)))
                             : "memory");
            }
            __syncwarp();
            if (page >= 0) {
                const int key = first + it * step + (my_seg << seg_shift);
                const int64_t row = ((int64_t)page * c.heads + h) * c.page_size +
                                    (key - (int)pl.div_page(key) * c.page_size);
                asm volatile(
                    "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], "
                    "[%1], %2, [%3];" ::"r"(st + my_dst),
                    "l"(my_base + row * my_row), "r"((uint32_t)(seg * my_row)), "r"(bar)
                    : "memory");
            }
        };
        int next_page;
        auto start = [&] {
#pragma unroll
            for (int it = 0; it < St::kCount; ++it) issue(it, page_of(it));
            next_page = page_of(St::kCount);
        };
        start();

        // ---- Q's fragments: pair p of lane t is codes (C w + i, C w + i + C/2), C = 2H
        uint32_t q[NT][kPairs];
        float xs[NT][2];  // scale * log2(e) of rows 2t, 2t + 1, and their power of two taken back
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = rb * R + 8 * n + g;
            uint32_t raw[NK / 2];
            const int i = r / a.group;
            const uint16_t* src = a.q + (int64_t)(s.row0 + i) * a.q_row +
                                  (int64_t)(h * a.group + (r - i * a.group)) * a.q_head + t * NK;
#pragma unroll
            for (int k = 0; k < NK / 8; ++k) {
                const uint4 v =
                    r < nr ? reinterpret_cast<const uint4*>(src)[k] : make_uint4(0, 0, 0, 0);
                raw[4 * k] = v.x;
                raw[4 * k + 1] = v.y;
                raw[4 * k + 2] = v.z;
                raw[4 * k + 3] = v.w;
            }
            float big = 0.f;
#pragma unroll
            for (int k = 0; k < NK / 2; ++k) {
                const float2 f = bf16x2_to_f2(raw[k]);
                big = fmaxf(big, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
            // 2^(14 - e), e the exponent of the row's largest value
            const int e = max((int)(__float_as_uint(big) >> 23) - 127, -112);
            const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
            constexpr int C = NK < 2 * H ? NK : 2 * H;
            static_for<0, kPairs>([&](auto pp) {
                constexpr int p = decltype(pp)::value, w = p / (C / 2), i0 = p % (C / 2);
                constexpr int e0 = C * w + i0, e1 = e0 + C / 2;
                auto value = [&](int x) {
                    return __uint_as_float((x & 1) ? raw[x / 2] & 0xffff0000u : raw[x / 2] << 16);
                };
                q[n][p] = f2_to_f16x2(value(e0) * up, value(e1) * up);
            });
            // row 8n + g's lane holds e; lanes (., t) need rows 2t, 2t + 1
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int ee = __shfl_sync(0xffffffffu, e, (2 * t + u) * 4);
                xs[n][u] = a.scale * 1.4426950408889634f * 0x1p-14f *
                           __uint_as_float((uint32_t)(127 + ee) << 23);
            }
        }

        float O[NV / 2][NT][4];
        float m[NT][2], base[NT][2], l[NT][2];
        float ref[NT][2];  // what l counts against
        const int kslot = (g >> 1) + 4 * (g & 1);  // this lane's K rows: kslot, kslot + 8
        // One pass over the part's positions; whether a wait gave up.  APART: the normaliser
        // is summed apart; otherwise `odd` says whether it has to be.
        bool odd = false;
        auto pass = [&](auto apart) {
            constexpr bool APART = decltype(apart)::value;
            constexpr int NBP = APART ? 1 : NB;  // blocks of a step at once (few: less code)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int k = 0; k < NV / 2; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) O[k][n][e] = 0.f;
                m[n][0] = m[n][1] = -CUDART_INF_F;
                l[n][0] = l[n][1] = base[n][0] = base[n][1] = 0.f;
                ref[n][0] = ref[n][1] = -CUDART_INF_F;
            }

            int it = 0;
            for (; it < steps; ++it) {
                const int use = done + it, ring_slot = use % St::kCount;
                const uint32_t st = ring + ring_slot * St::kBytes;
                if (!__all_sync(0xffffffffu, mbar_wait_clock(bars + 8 * ring_slot,
                                                             (use / St::kCount) & 1, nullptr))) {
                    if (lane == 0) report_status(status, HBL_ERR_TIMEOUT);
                    break;
                }
                const int key0 = first + it * step;
                const uint32_t flags = lds32(st + 2 * St::kCodes + 2 * St::kScales);
                const bool plain = flags == (1u << (KW >> seg_shift)) - 1u && key0 >= all_lo &&
                                   key0 + KW <= min(all_hi, end);

#pragma unroll 1
                for (int b0 = 0; b0 < NB; b0 += NBP) {
                    float S[NBP][NT][4];
#pragma unroll
                    for (int blk = 0; blk < NBP; ++blk) {
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e) S[blk][n][e] = 0.f;
                        const uint32_t r0 = st + (16 * (b0 + blk) + kslot) * St::kRow;
                        uint32_t w0[kKvWords<B, NK>], w1[kKvWords<B, NK>];
                        kv_lds_codes<B, NK>(r0, t, w0);
                        kv_lds_codes<B, NK>(r0 + 8 * St::kRow, t, w1);
                        if constexpr (NK < 2 * H) {  // 8 codes of 2 bits: a half word, in two of 4
                            w0[0] = (w0[0] & 0xffu) | ((w0[0] & 0xff00u) << 8);
                            w1[0] = (w1[0] & 0xffu) | ((w1[0] & 0xff00u) << 8);
                        }
                        constexpr int P = NK < 2 * H ? NK / 2 : H;  // pairs of a word
                        static_for<0, kKvWords<B, NK>>([&](auto ww) {
                            constexpr int w = decltype(ww)::value;
                            uint32_t a0[P], a1[P];
                            kv_widen_f16<B, P>(w0[w], a0);
                            kv_widen_f16<B, P>(w1[w], a1);
#pragma unroll
                            for (int p = 0; p < P; p += 2)
#pragma unroll
                                for (int n = 0; n < NT; ++n)
                                    mma_f16(S[blk][n], a0[p], a1[p], a0[p + 1], a1[p + 1],
                                            q[n][P * w + p], q[n][P * w + p + 1]);
                        });
                    }
                    // ---- exponents
                    float mx[NT][2], rsv[NBP][2];  // rsv: 1 / sv of positions kslot, kslot + 8
                    float step_far = 0.f;  // of this lane's positions, the largest |log2(sv)|
#pragma unroll
                    for (int blk = 0; blk < NBP; ++blk) {
                        float lvs[2];
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const uint32_t sc =
                                st + 2 * St::kCodes + 4 * (16 * (b0 + blk) + kslot + 8 * u);
                            const float sk = __uint_as_float(lds32(sc));
                            const float any =
                                APART ? 0.f : lg2(__uint_as_float(lds32(sc + St::kScales)));
                            lvs[u] = fabsf(any);
                            const float lv = APART ? 0.f : fmaxf(any, k12::kZeroFold);
                            rsv[blk][u] = ex2(-lv);
#pragma unroll
                            for (int n = 0; n < NT; ++n)
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    S[blk][n][2 * u + e] = __fmaf_rn(
                                        S[blk][n][2 * u + e], __fmul_rn(sk, xs[n][e]), lv);
                        }
                        step_far = max3(step_far, lvs[0], lvs[1]);
                    }
                    if (!plain) {  // what is not visible becomes -inf, whatever is stored there
                        step_far = 0.f;
#pragma unroll
                        for (int blk = 0; blk < NBP; ++blk)
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                const int slot = 16 * (b0 + blk) + kslot + 8 * u, key = key0 + slot;
                                const bool there =
                                    ((flags >> (slot >> seg_shift)) & 1u) != 0 && key < end;
                                if (!there)
                                    rsv[blk][u] = 0.f;
                                else if (!(rsv[blk][u] >= 0x1p-40f && rsv[blk][u] <= 0x1p40f))
                                    step_far = CUDART_INF_F;
#pragma unroll
                                for (int n = 0; n < NT; ++n)
#pragma unroll
                                    for (int e = 0; e < 2; ++e)
                                        if (!(there && key >= lo[n][e] && key < hi[n][e]))
                                            S[blk][n][2 * u + e] = -CUDART_INF_F;
                            }
                    }
                    odd |= step_far > k12::kFold;
                    auto largest = [&] {
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                mx[n][e] = fmaxf(S[0][n][e], S[0][n][2 + e]);
#pragma unroll
                                for (int blk = 1; blk < NBP; ++blk)
                                    mx[n][e] = max3(mx[n][e], S[blk][n][e], S[blk][n][2 + e]);
                            }
                    };
                    largest();
                    if constexpr (APART) {  // the scores' own largest and sum; then V's scales
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
#pragma unroll
                                for (int o = 4; o < 32; o <<= 1)
                                    mx[n][e] =
                                        fmaxf(mx[n][e], __shfl_xor_sync(0xffffffffu, mx[n][e], o));
                                const float to = fmaxf(ref[n][e], mx[n][e]);
                                const float rb = to == -CUDART_INF_F ? 0.f : kShift - to;
                                if (to != ref[n][e]) l[n][e] *= ex2(ref[n][e] - to);
                                ref[n][e] = to;
#pragma unroll
                                for (int blk = 0; blk < NBP; ++blk)
                                    l[n][e] += ex2(S[blk][n][e] + rb) + ex2(S[blk][n][2 + e] + rb);
                            }
#pragma unroll
                        for (int blk = 0; blk < NBP; ++blk)
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                // (stored where nothing is, it may be anything: -inf stays -inf)
                                const uint32_t sc = st + 2 * St::kCodes + St::kScales +
                                                    4 * (16 * (b0 + blk) + kslot + 8 * u);
                                const float any = lg2_any(__uint_as_float(lds32(sc)));
                                const float lv = fminf(fmaxf(any, k12::kNoScale), 128.f);
                                rsv[blk][u] = 0.f;
#pragma unroll
                                for (int n = 0; n < NT; ++n)
#pragma unroll
                                    for (int e = 0; e < 2; ++e) S[blk][n][2 * u + e] += lv;
                            }
                        largest();
                    }
                    // each lane looks at its own positions' largest; only when one is too far
                    // above the reference do the lanes of a row find their common one
                    bool far = false;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        far |= mx[n][0] > m[n][0] + kLazy || mx[n][1] > m[n][1] + kLazy;
                    if (__any_sync(0xffffffffu, far)) {
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
#pragma unroll
                                for (int o = 4; o < 32; o <<= 1)
                                    mx[n][e] =
                                        fmaxf(mx[n][e], __shfl_xor_sync(0xffffffffu, mx[n][e], o));
                                const float nm = fmaxf(m[n][e], mx[n][e]);
                                const float f = nm == m[n][e] ? 1.f : ex2(m[n][e] - nm);
                                m[n][e] = nm;
                                // a row that has seen nothing: 2^(-inf) = 0 against any base
                                base[n][e] = nm == -CUDART_INF_F ? 0.f : kShift - nm;
                                if constexpr (!APART) l[n][e] *= f;
#pragma unroll
                                for (int k = 0; k < NV / 2; ++k) {
                                    O[k][n][e] *= f;
                                    O[k][n][2 + e] *= f;
                                }
                            }
                    }
                    // ---- weights and the second product
#pragma unroll
                    for (int blk = 0; blk < NBP; ++blk) {
                        uint32_t p[NT][2];
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                float w[2];
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    w[e] = ex2(S[blk][n][2 * u + e] + base[n][e]);
                                    if constexpr (!APART)
                                        l[n][e] = __fmaf_rn(w[e], rsv[blk][u], l[n][e]);
                                }
                                p[n][u] = transpose8(f2_to_f16x2(w[0], w[1]));
                            }
                        const uint32_t r0 = st + St::kCodes + (16 * (b0 + blk) + t) * St::kRow;
                        constexpr int VW = kKvWords<B, NV>;
                        uint32_t v[4][VW];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            kv_lds_codes<B, NV>(r0 + 4 * k * St::kRow, g, v[k]);
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
                                    mma_f16(O[(P * hw + i) / 2][n], a0[i], a0[i + 1], a2[i],
                                            a2[i + 1], p[n][0], p[n][1]);
                        });
                    }
                }
                __syncwarp();  // the stage is read
                issue(it + St::kCount, next_page);
                next_page = page_of(it + St::kCount + 1);
            }
            // after a timeout: the copies still in flight, the late one among them
            for (int j = it; j < steps && j < it + St::kCount; ++j)
                mbar_wait_clock(bars + 8 * ((done + j) % St::kCount), ((done + j) / St::kCount) & 1,
                                nullptr);
            done += steps;
            return it < steps;
        };
        if (pass(ic_bool<false>{})) or_shared(flags_s, 2);
        if (odd) or_shared(flags_s, 1);
        __syncthreads();  // (the rings are free as well)
        const uint32_t raised = lds32(flags_s);
        bool apart = __builtin_expect(raised != 0, 0);
        if (apart) {  // unless they were zero scales alone
            if (raised & 2u) return;  // nothing is stored of a part that lacks positions
            bool far = false;
            for (int key = begin + threadIdx.x; key < end; key += kThreads) {
                const int pi = (int)pl.div_page(key), page = kv_page(kb, c.num_pages, b, pi);
                if (page >= 0)
                    far |= !k12::folds(c.vs[((int64_t)page * c.heads + h) * c.page_size +
                                            (key - pi * c.page_size)]);
            }
            apart = __syncthreads_or(far);
            if (threadIdx.x == 0) sts32(flags_s, 0);
        }
        if (__builtin_expect(apart, 0)) {
            start();
            const bool late = pass(ic_bool<true>{});
            // both sums against the point half way between theirs
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (ref[n][e] == -CUDART_INF_F) continue;
                    const float C = 0.5f * (m[n][e] + ref[n][e]), up = ex2(m[n][e] - C);
                    l[n][e] *= ex2(ref[n][e] - C);
                    m[n][e] = C;
#pragma unroll
                    for (int k = 0; k < NV / 2; ++k) {
                        O[k][n][e] *= up;
                        O[k][n][2 + e] *= up;
                    }
                }
            if (__syncthreads_or(late)) return;
        }
        // ---- join the warps.  Lane (g, t): values NV g .. of rows 2t, 2t + 1
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int o = 4; o < 32; o <<= 1)
                    l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], o);
        float* so = reinterpret_cast<float*>(smem);         // [warp][R][D + 4]
        float* sm = so + kWarps * R * (D + 4);              // [warp][R]: m, then l
        float* sl = sm + kWarps * R;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * n + 2 * t + e;
                float* dst = so + (warp * R + r) * (D + 4) + g * NV;
#pragma unroll
                for (int k = 0; k < NV / 4; ++k)
                    reinterpret_cast<float4*>(dst)[k] =
                        make_float4(O[2 * k][n][e], O[2 * k][n][2 + e], O[2 * k + 1][n][e],
                                    O[2 * k + 1][n][2 + e]);
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
            if (u0 == 0 && u1 == im.units) {
                k12::store_row4(a, s, h, row, d, y, M - kShift, L);
            } else {
                float* dst = k12::slot_of(part, pl, D, blockIdx.x, u0 == 0) + r * (D + 4);
                *reinterpret_cast<float4*>(dst + d) = y;
                if (d == 0) *reinterpret_cast<float2*>(dst + D) = make_float2(M - kShift, L);
            }
        }
        // the rings' memory goes back to the copies
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncthreads();
        if (at >= stop) return;
    }
}

template <int D, int B, int NT>
hbl_status launch(const KvCache& c, const KvBatch& kb, const KvAttn& a, const Plan& pl, float* part,
                  int32_t* status, cudaStream_t stream) {
    constexpr int kSmem = smem_bytes<D, B, NT>();
    auto kern = decode_kernel<D, B, NT>;
    if (!smem_attr_once(reinterpret_cast<const void*>(kern), kSmem)) return HBL_ERR_CUDA;
    kern<<<(unsigned)pl.ctas, kThreads, kSmem, stream>>>(c, kb, a, pl, part, status);
    return cudaGetLastError() == cudaSuccess ? HBL_OK : HBL_ERR_CUDA;
}

template <int D>
hbl_status launch_d(const KvCache& c, const KvBatch& kb, const KvAttn& a, const Plan& pl,
                    float* part, int32_t* status, cudaStream_t stream) {
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
