// k14_kv_chunk.cuh -- attention of a chunk of new rows over the paged low-bit
// cache, on the tcgen05 tensor cores.
//
// The mathematics is k13_kv_decode.cuh's: with integer codes k, v and scales,
//   x_i = scale * log2(e) * sk_i * (q . k_i) + log2(sv_i),
//   O = sum_i 2^(x_i - m) v_i / sum_i 2^(x_i - m) / sv_i
// so both products run on exact integers (bf16 keys against bf16 queries, fp16
// values against fp16 weights) and the scales cost one packed fma per pair of
// scores.  The reference point m follows the running maximum only when a
// score passes it by more than 2^8 (weights stay below 2^14 in fp16): the
// accumulator in tensor memory is rescaled a few times a row, not every tile.  Where V's
// scales are too small or too large for 1 / sv, a CTA takes its positions once more and
// sums the normaliser apart (k12_kv_attention.cuh).
//
// One CTA: one sequence, cached head and 2 x 128 head rows (128 at D = 256),
// and a range of positions, widened in tiles of KT and worked on in parts of 64.
// Sixteen warps:
//   0..7    softmax, four warps to each 128 rows: scores out of tensor memory,
//           weights back into it in the scores' place; at the end the results
//   8..14   (and 4..7 at D = 256, which has one row set) widen K and V codes from
//           HBM straight into swizzled operand tiles (two stages each, loaded a
//           tile ahead) and lay out the tiles' scales
//   15      issues the MMAs: S = Q K^T (both operands in shared
//           memory), O += P V (P in tensor memory, V read down its rows, which
//           is the transposed operand that the second product needs)
// Scores have two buffers a row set: part i + 1's are computed while part i is
// in its softmax, so the softmax warps never wait for the tensor core.
//
// What bounds it: 128 positions are 4 * 128^3 * 2 products for the two row sets,
// 2048 tensor cycles at D = 128, and 2 * 128 * 128 exponentials, 2048 cycles of
// the 16-a-cycle special-function units: both at once at best.  Shared memory is
// as busy (2048 cycles of MMA operand reads with scores of 64 columns, 512 of
// operand tiles stored), which is why scores leave tensor memory in the
// 16x256b shape: a thread then needs a quarter of a part's scales, not all.
// (Parts of 128 with one score buffer read less, but then every part's softmax
// waits for the product before it and the scores after that: 6270 cycles for
// 128 positions.)  At D = 256 a widened tile serves only 128 rows, and the widening
// bounds it: 3300 cycles for 64 positions, where the products take 1300.
//
// Measured, graph replay: 4-bit, D = 128, a prompt of 8192 against itself with 32
// query heads over 8: 699 us, 786 TFLOP/s, 0.48 of the measured bf16 rate; 5100 cycles
// for 128 positions and two row sets, of which the products with their hand-overs
// alone (nothing widened, no exponentials) take 3700; some 12 us of every CTA are its
// start (block, barriers, queries: 5) and end (last products, results: 3) and
// the filling of its pipeline.
//
// Measured as well: heads of 64 634 us, of 32 572 us (the exponentials are as many);
// 16 heads over 2 of 256 and 4096 positions 253 us.  The second pass that wide V scales
// take: 2.4 ms instead of 0.7.  It works on 16 rows at a time: with all 32 of a warp at
// once its registers cost the first pass 2 % (725 us).
//
// Tried and slower: 24 warps with a pair to each row quarter, half the columns each
// (6380 cycles); weights computed against the reference of the part before while the
// maximum is found (6654); at D = 256, parts dealt to two softmax groups in turn (as
// fast: the softmax does not bound it).
//
// D order.  Widening gives codes in pairs (i, i + C/2) of C; queries are laid
// out in the same order, and O's columns are put back when it is stored.
#pragma once

#include "hbl_kv_codes.cuh"
#include "hbl_tmem.cuh"
#include "k12_kv_attention.cuh"

namespace hbl {
namespace k14 {

using k12::Plan;

constexpr int kThreads = 512;
constexpr int kMmaWarp = 15;
constexpr float kShift = 6.f;        // weights are held times 2^6 ...
constexpr float kLazy = 8.f;         // ... and may pass the reference by 2^8
constexpr int kScaleStages = 4;
constexpr float kNowhere = -1e30f;   // in a scale's place: no position

template <int D>
struct Tile {
    static constexpr int NQ = D == 256 ? 1 : 2;       // sets of 128 rows
    static constexpr int KT = D == 256 ? 64 : 128;    // positions of a tile
    static constexpr int kPanels = D >= 64 ? D / 64 : 1;  // 128-byte panels of a row
    static constexpr int kParts = KT / 64;            // parts of a tile
    static constexpr uint32_t kOCol = 256;            // first accumulator column
    static constexpr int kQ = NQ * 128 * kPanels * 128;  // bytes
    static constexpr int kStage = KT * kPanels * 128;    // one operand tile
    static constexpr int kScale = KT * 12;               // (ck, ck, lv, lv) a pair, then 1/sv
    static constexpr int kBars = 512;                    // two sets: one to a pass
    static constexpr int kUnits = KT * (D / 32) / 32;    // warp units of 32 x 32 codes
    static constexpr int kConv = 15 - 4 * NQ;            // widening warps
    static constexpr int kMine = (kUnits + kConv - 1) / kConv;
    static constexpr int kSmem = kQ + 4 * kStage + kScaleStages * kScale + kBars + 1024;
};

// K-major (queries, keys) and row-major-down (values) descriptors of operand
// tiles in 128-byte swizzled panels: eight rows of 128 bytes to an atom.
__device__ __forceinline__ uint64_t desc_k(uint32_t saddr) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)1 << 16) |
           ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// leading offset: from one panel of 64 columns to the next
__device__ __forceinline__ uint64_t desc_v(uint32_t saddr, uint32_t panel_bytes) {
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(panel_bytes >> 4) << 16) |
           ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// kind::f16: D fp32 (bits 4-5 = 1), A and B types (bits 7-9, 10-12: 0 fp16, 1
// bf16), B transposed (bit 16), N >> 3 at bit 17, M >> 4 at bit 24.
__host__ __device__ constexpr uint32_t idesc(bool bf16, bool b_mn, int N) {
    return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn ? 1u << 16 : 0u) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
// MMAs and commits by the whole, converged warp, of which one lane is elected: the
// operands are then uniform and need not be moved from one thread's registers,
// which took some 75 cycles an MMA.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id,
                                       uint32_t accum) {
    asm volatile(
        "{\n.reg .pred p, e;\n"
        "elect.sync _|e, 0xffffffff;\n"
        "setp.ne.b32 p, %4, 0;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(accum)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id,
                                       uint32_t accum) {
    asm volatile(
        "{\n.reg .pred p, e;\n"
        "elect.sync _|e, 0xffffffff;\n"
        "setp.ne.b32 p, %4, 0;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(id), "r"(accum)
        : "memory");
}
__device__ __forceinline__ void commit(uint32_t mbar) {
    asm volatile(
        "{\n.reg .pred e;\n"
        "elect.sync _|e, 0xffffffff;\n"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(
            mbar)
        : "memory");
}
__device__ __forceinline__ void fence_async() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void reg_alloc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dealloc() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Bounded wait; on expiry (here or, through the flag, anywhere in the CTA) false.
// one(): by a single thread.  all(): by a whole warp, whose lanes leave it
// together -- the tensor-memory instructions that follow need the warp
// converged, and lanes that poll for themselves come out one after another.
struct Waiter {
    volatile int* abort_flag;
    int32_t* status;
    __device__ __forceinline__ bool all(uint32_t bar, uint32_t parity) const {
        return __all_sync(0xffffffffu, one(bar, parity));
    }
    __device__ __forceinline__ bool one(uint32_t bar, uint32_t parity) const {
        if (mbar_wait_clock(bar, parity, abort_flag)) return true;
        if (!*abort_flag) report_status(status, HBL_ERR_TIMEOUT);
        *abort_flag = 1;
        return false;
    }
};

// A lane's place in a unit of 32 lanes x 32 codes: eight neighbouring lanes take
// four rows and two groups of a row, so that their 16-byte stores fall into
// different banks of the swizzled tile.
template <int D>
struct Lane {
    static constexpr int kGroups = D / 32;          // groups of 32 codes in a row
    static constexpr int kRows = 32 / kGroups;      // rows of a unit
    int row, group;
    __device__ __forceinline__ explicit Lane(int lane) {
        if constexpr (kGroups == 1) {
            row = lane;
            group = 0;
        } else {
            const int lo = lane & 1, k = (lane >> 1) & 3, rest = lane >> 3;
            constexpr int kHigh = kGroups / 2;  // 1, 2, 4
            group = (rest % kHigh) * 2 + lo;
            row = (rest / kHigh) * 4 + k;
        }
    }
};
// Byte offset of 16-byte chunk q (0..3) of a group in a tile of `rows` rows.
__device__ __forceinline__ uint32_t chunk_at(int rows, int row, int group, int q) {
    const int chunk = (group & 1) * 4 + q;
    return (uint32_t)((group >> 1) * rows * 128 + row * 128 + ((chunk ^ (row & 7)) << 4));
}

// 32 codes (B words) -> 16 pairs, as bf16 or fp16.
template <int B, bool BF16>
__device__ __forceinline__ void widen32(const uint32_t (&raw)[B], uint32_t (&out)[16]) {
    constexpr int H = kKvHalfCodes<B>, W = 16 / H;
    uint32_t w[W];
    if constexpr (B == 3) {
        w[0] = kv_spread3(raw[0]);
        w[1] = kv_spread3(__funnelshift_r(raw[0], raw[1], 24));
        w[2] = kv_spread3(__funnelshift_r(raw[1], raw[2], 16));
        w[3] = kv_spread3(raw[2] >> 8);
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = raw[i];
    }
#pragma unroll
    for (int i = 0; i < W; ++i) {
        uint32_t p[H];
        if constexpr (BF16)
            kv_widen_bf16<B, H>(w[i], p);
        else
            kv_widen_f16<B, H>(w[i], p);
#pragma unroll
        for (int k = 0; k < H; ++k) out[H * i + k] = p[k];
    }
}
// Within a group of 32: the value at place n of the order that widening gives.
template <int B>
__host__ __device__ constexpr int place_of(int n) {
    const int H = kKvHalfCodes<B>, p = n / 2;
    return p / H * 2 * H + p % H + (n & 1) * H;
}

// What a CTA has to do: rows from row0 on of sequence b, over the positions of sp.
template <int D>
struct Task {
    k12::Rows s;
    k12::Split sp;
    int b, row0, nr, parts, tiles, sets;  // sets: row sets that have rows
    bool work;
    // what all sets report is reported twice where one is missing
    __device__ __forceinline__ void arrive_for_all(uint32_t bar) const {
        for (int k = sets; k <= Tile<D>::NQ; ++k) mbar_arrive_one(bar);
    }
};
template <int D>
__device__ __forceinline__ Task<D> task_of(const Plan& pl, const KvCache& c, const KvBatch& kb,
                                           const KvAttn& a, const volatile int* where, int split) {
    using T = Tile<D>;
    Task<D> k = {};
    k.b = where[0];
    k.row0 = where[1] * 128 * T::NQ;
    if (k.b >= 0) {
        k.s = k12::rows_of(kb, c.page_size, a, k.b);
        k.nr = k.s.n * a.group;
        k.sp = k12::split_of(
            pl, k12::range_of(a, k.s, k.row0, min(k.nr, k.row0 + 128 * T::NQ) - 1), split);
    }
    k.work = k.b >= 0 && split < max(k.sp.count, 1);
    k.parts = !k.work || k.sp.count == 0 ? 0 : (k.sp.end - k.sp.begin + 63) / 64;
    k.tiles = (k.parts + T::kParts - 1) / T::kParts;
    k.sets = !k.work ? 0 : T::NQ == 2 && k.nr - k.row0 > 128 ? 2 : 1;
    return k;
}

// The barriers of one pass.
struct Barriers {
    uint32_t at;
    __device__ __forceinline__ uint32_t kfull(int s) const { return at + 8u * s; }
    __device__ __forceinline__ uint32_t kempty(int s) const { return at + 8u * (2 + s); }
    __device__ __forceinline__ uint32_t vfull(int s) const { return at + 8u * (4 + s); }
    __device__ __forceinline__ uint32_t vempty(int s) const { return at + 8u * (6 + s); }
    __device__ __forceinline__ uint32_t scfull(int s) const { return at + 8u * (8 + s); }
    __device__ __forceinline__ uint32_t scempty(int s) const { return at + 8u * (12 + s); }
    // 2 * set + buffer
    __device__ __forceinline__ uint32_t sfull(int s) const { return at + 8u * (16 + s); }
    __device__ __forceinline__ uint32_t pfull(int s) const { return at + 8u * (20 + s); }
    __device__ __forceinline__ uint32_t ofull(int set) const { return at + 8u * (24 + set); }
    __device__ __forceinline__ uint32_t drain() const { return at + 8u * 27; }
    static constexpr int kCount = 28;
    template <int CONV, int NQ>
    static __device__ __forceinline__ uint32_t arrivals(int i) {
        if (i < 8) return (i & 2) == 0 ? CONV : 1;          // kfull, vfull; kempty, vempty
        if (i >= 12 && i < 16) return 4 * NQ;                // scempty
        return i >= 20 && i < 24 ? 4 : i == 26 ? 4 * NQ : 1;  // pfull; the queries'; the rest
    }
};

template <int D, int B>
__global__ void __launch_bounds__(kThreads, 1) chunk_kernel(KvCache c, KvBatch kb, KvAttn a,
                                                            Plan pl, float* part,
                                                            int32_t* status) {
    using T = Tile<D>;
    constexpr int KT = T::KT, NQ = T::NQ;
    constexpr int ROW_BYTES = D * B / 8;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_s = smem_addr(smem_raw);
    const uint32_t base_s = (raw_s + 1023u) & ~1023u;
    uint8_t* smem_base = smem_raw + (base_s - raw_s);
    const uint32_t q_s = base_s, k_s = q_s + T::kQ, v_s = k_s + 2 * T::kStage;
    const uint32_t sc_s = v_s + 2 * T::kStage, bar_s = sc_s + kScaleStages * T::kScale;
    uint8_t* bar_p = smem_base + (bar_s - base_s);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_p + 240);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(bar_p + 244);
    const uint32_t odd_s = bar_s + 256 + 240;  // a flag: V's scales need a second pass
    const uint32_t qfull = bar_s + 8u * 26;

    // ---- which rows, which positions: all heads of one block, then those of the next
    const int split = (int)(blockIdx.x % pl.splits), nth = (int)(blockIdx.x / pl.splits);
    const int h = nth % c.heads;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int* const where = reinterpret_cast<int*>(bar_p + 248);
    if (warp == 0) {
        const k12::Block blk = k12::block_of<128 * NQ>(pl, c, kb, a, nth / c.heads);
        if (lane == 0) {
            where[0] = blk.b;
            where[1] = blk.rb;
        }
    } else if (warp == 1) {
        // a lane to each barrier of a set (the queries' one, 26, is in the first alone)
        if (lane < Barriers::kCount) {
            const uint32_t n = Barriers::arrivals<T::kConv, NQ>(lane);
            mbar_init_count(bar_s + 8 * lane, n);
            mbar_init_count(bar_s + 256 + 8 * lane, n);
        }
        if (lane == 0) {
            sts32(odd_s, 0);
            *abort_flag = 0;
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    } else if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         smem_addr(tmem_slot))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tmem_fence_before();
    } else if (blockIdx.x == 0 && warp == 2) {  // the descriptors, by the first CTA
        for (int i = lane; i < kb.num_seqs; i += 32)
            if (k12::rows_of(kb, c.page_size, a, i).bad) report_status(status, HBL_ERR_INVALID_ARG);
    }
    __syncthreads();
    tmem_fence_after();
    const Task<D> first = task_of<D>(pl, c, kb, a, where, split);
    if (first.work) pdl_launch_dependents();
    const uint32_t tmem = *tmem_slot;
    const Waiter wait{abort_flag, status};

    // A pass over the positions, by each role.  Where V's scales need the normaliser summed
    // apart, which the warp that lays them out finds out, nothing is stored after the first
    // pass, and a second one (APART) takes its time; the queries stay.
    auto softmax = [&](auto apart, const Task<D>& task) {
        constexpr bool APART = decltype(apart)::value;
        const Barriers bar{bar_s + (APART ? 256u : 0u)};
        const k12::Rows& s = task.s;
        const k12::Split& sp = task.sp;
        const int row0 = task.row0, nr = task.nr, parts = task.parts;
        const int set = warp >> 2, quarter = warp & 3, g = lane >> 2, t = lane & 3;
        // ---- rows of this thread: 16 hf + 8 u + g of the warp's 32
        int lo[4], hi[4];
        int max_lo = 0, min_hi = 0x7fffffff;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int r = min(row0 + set * 128 + 32 * quarter + 8 * k + g, nr - 1);
            const int p = s.first + r / a.group;
            hi[k] = a.causal ? p + 1 : 0x7fffffff;
            lo[k] = k12::window_begin(a, p);
            max_lo = max(max_lo, lo[k]);
            min_hi = min(min_hi, hi[k]);
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            max_lo = max(max_lo, __shfl_xor_sync(0xffffffffu, max_lo, o));
            min_hi = min(min_hi, __shfl_xor_sync(0xffffffffu, min_hi, o));
        }
        float m[4], base[4], ref[4];  // (ref: what l counts against, APART)
        float2 l[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            m[k] = -CUDART_INF_F;
            base[k] = 0.f;
            ref[k] = -CUDART_INF_F;
            l[k] = make_float2(0.f, 0.f);
        }
        const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
        const uint32_t o_t = tmem + lanes + T::kOCol + set * D;
        // ---- the parts, APART: in the same steps, two references to a row
        bool ok = true;
        if constexpr (!APART) {
#pragma unroll 1
            for (int i = 0; i < parts; ++i) {
                const int sb = 2 * set + (i & 1), j = i / T::kParts;
                const uint32_t s_t = tmem + lanes + sb * 64;
                // this thread's scales of the part: (ck, ck, lv, lv) and 1/sv of columns
                // 8k + 2t, 8k + 2t + 1
                const uint8_t* const sc_p =
                    smem_base + (sc_s - base_s) + (j % kScaleStages) * T::kScale;
                const float4* const sc4 =
                    reinterpret_cast<const float4*>(sc_p + (i % T::kParts) * 512) + t;
                const float2* const rs2 =
                    reinterpret_cast<const float2*>(sc_p + KT * 8 + (i % T::kParts) * 256) + t;
                ok = wait.all(bar.scfull(j % kScaleStages), (j / kScaleStages) & 1) &&
                     wait.all(bar.sfull(sb), (i >> 1) & 1);
                if (!ok) break;
                tmem_fence_after();
                float x[2][32];
                tmem_ld_16x256b_x8(s_t, x[0]);
                tmem_ld_16x256b_x8(s_t + (16u << 16), x[1]);
                tmem_wait_ld(x[0]);
                tmem_wait_ld(x[1]);
                // ---- exponents
                const int key0 = sp.begin + i * 64;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float4 f = sc4[4 * k];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        float* v = &x[r >> 1][4 * k + 2 * (r & 1)];
                        const float2 y = __ffma2_rn(make_float2(v[0], v[1]), make_float2(f.x, f.y),
                                                    make_float2(f.z, f.w));
                        v[0] = y.x;
                        v[1] = y.y;
                    }
                }
                if (key0 < max_lo || key0 + 64 > min_hi) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int key = key0 + 8 * k + 2 * t + e;
                                if (key < lo[r] || key >= hi[r])
                                    x[r >> 1][4 * k + 2 * (r & 1) + e] = -CUDART_INF_F;
                            }
                }
                // each lane looks at its own columns' largest; only when one is too far
                // above the reference do the lanes of a row find their common one
                float mx[4];
                bool far = false;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    mx[r] = fmaxf(x[r >> 1][2 * (r & 1)], x[r >> 1][2 * (r & 1) + 1]);
#pragma unroll
                    for (int k = 1; k < 8; ++k)
                        mx[r] = max3(mx[r], x[r >> 1][4 * k + 2 * (r & 1)],
                                     x[r >> 1][4 * k + 2 * (r & 1) + 1]);
                    far |= mx[r] > m[r] + kLazy;
                }
                if (__any_sync(0xffffffffu, far)) {
                    float f[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
                        mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
                        const float nm = fmaxf(m[r], mx[r]);
                        f[r] = nm == m[r] ? 1.f : ex2(m[r] - nm);
                        m[r] = nm;
                        // a row that has seen nothing: 2^(-inf) = 0 against any base
                        base[r] = nm == -CUDART_INF_F ? 0.f : kShift - nm;
                        l[r] = __fmul2_rn(l[r], make_float2(f[r], f[r]));
                    }
                    if (i > 0) {  // the accumulator, once the product before has landed
                        ok = wait.all(bar.ofull(set), (i - 1) & 1);
                        if (!ok) break;
                        tmem_fence_after();
#pragma unroll 1
                        for (int cc = 0; cc < D / 32; ++cc)
#pragma unroll
                            for (int hf = 0; hf < 2; ++hf) {
                                const uint32_t at = o_t + ((uint32_t)(16 * hf) << 16) + 32 * cc;
                                float o[16];
                                tmem_ld_16x256b_x4(at, o);
                                tmem_wait_ld(o);
#pragma unroll
                                for (int k = 0; k < 4; ++k)
#pragma unroll
                                    for (int e = 0; e < 4; ++e) o[4 * k + e] *= f[2 * hf + e / 2];
                                tmem_st_16x256b_x4(at, o);
                            }
                    }
                }
                // ---- weights
                uint32_t p[2][16];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float2 rs = rs2[4 * k];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float* v = &x[r >> 1][4 * k + 2 * (r & 1)];
                        const float2 y = __fadd2_rn(make_float2(v[0], v[1]),
                                                    make_float2(base[r], base[r]));
                        const float2 w = make_float2(ex2(y.x), ex2(y.y));
                        l[r] = __ffma2_rn(w, rs, l[r]);
                        p[r >> 1][2 * k + (r & 1)] = f2_to_f16x2(w.x, w.y);
                    }
                }
                tmem_st_16x128b_x8(s_t, p[0]);
                tmem_st_16x128b_x8(s_t + (16u << 16), p[1]);
                tmem_wait_st();
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive_one(bar.pfull(sb));
                    if (i % T::kParts == T::kParts - 1 || i + 1 == parts)
                        task.arrive_for_all(bar.scempty(j % kScaleStages));
                }
            }
        } else {
#pragma unroll 1
            for (int i = 0; i < parts; ++i) {
                const int sb = 2 * set + (i & 1), j = i / T::kParts;
                const uint32_t s_t = tmem + lanes + sb * 64;
                const float4* const sc4 =
                    reinterpret_cast<const float4*>(smem_base + (sc_s - base_s) +
                                                    (j % kScaleStages) * T::kScale +
                                                    (i % T::kParts) * 512) + t;
                ok = wait.all(bar.scfull(j % kScaleStages), (j / kScaleStages) & 1) &&
                     wait.all(bar.sfull(sb), (i >> 1) & 1) &&
                     (i == 0 || wait.all(bar.ofull(set), (i - 1) & 1));
                if (!ok) break;
                tmem_fence_after();
                const int key0 = sp.begin + i * 64;
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {  // 16 rows at a time: registers before speed
                    const uint32_t half = (uint32_t)(16 * hf) << 16;
                    float x[32];
                    tmem_ld_16x256b_x8(s_t + half, x);
                    tmem_wait_ld(x);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {  // scores; -inf where nothing is or may be seen
                        const float4 f = sc4[4 * k];
                        const int key = key0 + 8 * k + 2 * t;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int r = 2 * hf + e / 2, at = key + (e & 1);
                            const bool there = (e & 1 ? f.w : f.z) != kNowhere;
                            x[4 * k + e] = there && at >= lo[r] && at < hi[r]
                                               ? x[4 * k + e] * (e & 1 ? f.y : f.x)
                                               : -CUDART_INF_F;
                        }
                    }
                    float f2[2];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {  // their largest and sum
                        const int r = 2 * hf + u;
                        float top = -CUDART_INF_F;
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            top = max3(top, x[4 * k + 2 * u], x[4 * k + 2 * u + 1]);
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                        const float to = fmaxf(ref[r], top);
                        if (to != ref[r]) l[r].x *= ex2(ref[r] - to);
                        ref[r] = to;
                        const float rb = to == -CUDART_INF_F ? 0.f : kShift - to;
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            l[r].x += ex2(x[4 * k + 2 * u] + rb) + ex2(x[4 * k + 2 * u + 1] + rb);
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k) {  // V's scales
                        const float4 f = sc4[4 * k];
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[4 * k + e] += e & 1 ? f.w : f.z;
                    }
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int r = 2 * hf + u;
                        float top = m[r];
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            top = max3(top, x[4 * k + 2 * u], x[4 * k + 2 * u + 1]);
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                        f2[u] = top == m[r] ? 1.f : ex2(m[r] - top);
                        m[r] = top;
                        base[r] = top == -CUDART_INF_F ? 0.f : kShift - top;
                    }
                    uint32_t p[16];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const float to = base[2 * hf + u];
                            p[2 * k + u] = f2_to_f16x2(ex2(x[4 * k + 2 * u] + to),
                                                       ex2(x[4 * k + 2 * u + 1] + to));
                        }
                    tmem_st_16x128b_x8(s_t + half, p);
                    if (i > 0) {
#pragma unroll 1
                        for (int cc = 0; cc < D / 32; ++cc) {
                            float o[16];
                            tmem_ld_16x256b_x4(o_t + half + 32 * cc, o);
                            tmem_wait_ld(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] *= f2[e % 4 / 2];
                            tmem_st_16x256b_x4(o_t + half + 32 * cc, o);
                        }
                    }
                }
                tmem_wait_st();
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive_one(bar.pfull(sb));
                    if (i % T::kParts == T::kParts - 1 || i + 1 == parts)
                        task.arrive_for_all(bar.scempty(j % kScaleStages));
                }
            }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float z = l[r].x + l[r].y;
            z += __shfl_xor_sync(0xffffffffu, z, 1);
            z += __shfl_xor_sync(0xffffffffu, z, 2);
            l[r].x = z;
        }
        // ---- the accumulator out, a lane to a row, 32 columns at a time.  Every product
        // has landed with the drain's single phase (a set's last product alone could not
        // be told from the one before the one before it by a parity).
        if (ok && parts > 0) ok = wait.all(bar.drain(), 0);
        // (Both flags stand: a wait that another warp lost, which left products out, since
        // before the drain; the scales' since the last part's, which this warp has waited for.)
        if (ok && *abort_flag == 0 && (APART || lds32(odd_s) == 0)) {
            tmem_fence_after();
            // row 8k + g's sum and reference sit in lane 4g
            float L = 0.f, M = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float lk = __shfl_sync(0xffffffffu, l[k].x, 4 * (lane & 7));
                const float mk = __shfl_sync(0xffffffffu, m[k], 4 * (lane & 7));
                if (lane >> 3 == k) {
                    L = lk;
                    M = mk - kShift;
                }
            }
            float up = 1.f;
            if constexpr (APART) {  // both sums against the point half way between theirs
                float R = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float rk = __shfl_sync(0xffffffffu, ref[k], 4 * (lane & 7));
                    if (lane >> 3 == k) R = rk - kShift;
                }
                if (R != -CUDART_INF_F) {
                    const float C = 0.5f * (M + R);
                    up = ex2(M - C);
                    L *= ex2(R - C);
                    M = C;
                }
            }
            const int row = row0 + set * 128 + 32 * quarter + lane;
            const bool there = row < nr, whole = sp.count <= 1;
            float inv = 1.f;
            uint8_t* dst;
            if (whole) {
                dst = reinterpret_cast<uint8_t*>(
                    k12::row_out(a, s, h, row, M, L, there, &inv));
            } else {
                const int i = row / a.group;
                float* to = part + k12::part_index(kb, a, split, s.row0 + i,
                                                   h * a.group + row - i * a.group) *
                                       (D + 4);
                if (there) *reinterpret_cast<float2*>(to + D) = make_float2(M, L);
                dst = reinterpret_cast<uint8_t*>(to);
            }
            // Two neighbouring lanes store 32 bytes of one's row, then of the other's:
            // whole sectors.  even and odd: those rows, from this lane's 16 bytes on.
            const bool is_odd = lane & 1;
            const uint64_t mine = reinterpret_cast<uint64_t>(dst);
            const uint64_t next = __shfl_xor_sync(0xffffffffu, mine, 1);
            const bool next_there = __shfl_xor_sync(0xffffffffu, (int)there, 1) != 0;
            uint8_t* const even =
                reinterpret_cast<uint8_t*>(is_odd ? next : mine) + 16 * (lane & 1);
            uint8_t* const odd =
                reinterpret_cast<uint8_t*>(is_odd ? mine : next) + 16 * (lane & 1);
            const bool even_there = is_odd ? next_there : there;
            const bool odd_there = is_odd ? there : next_there;
            auto store_pair = [&](const uint32_t* lo, const uint32_t* hi, int at) {
                uint32_t e[4], o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t got =
                        __shfl_xor_sync(0xffffffffu, is_odd ? lo[k] : hi[k], 1);
                    e[k] = is_odd ? got : lo[k];
                    o[k] = is_odd ? hi[k] : got;
                }
                if (even_there)
                    *reinterpret_cast<uint4*>(even + at) = make_uint4(e[0], e[1], e[2], e[3]);
                if (odd_there)
                    *reinterpret_cast<uint4*>(odd + at) = make_uint4(o[0], o[1], o[2], o[3]);
            };
#pragma unroll 1
            for (int cc = 0; cc < D / 32; ++cc) {
                float o[32];
                if (parts > 0) {
                    tmem_ld_32x32b_x32(o_t + 32 * cc, o);
                    tmem_wait_ld(o);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0.f;
                }
                float y[32];  // back in the order of D
                static_for<0, 32>([&](auto n) {
                    const float v = o[decltype(n)::value];
                    y[place_of<B>(decltype(n)::value)] = APART ? v * up * inv : v * inv;
                });
                if (whole) {
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) w[e] = f2_to_bf16x2(y[2 * e], y[2 * e + 1]);
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        store_pair(w + 8 * q, w + 8 * q + 4, 64 * cc + 32 * q);
                } else {
                    uint32_t w[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) w[e] = __float_as_uint(y[e]);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        store_pair(w + 8 * q, w + 8 * q + 4, 128 * cc + 32 * q);
                }
            }
        }
    };
    auto issue = [&](auto apart, const Task<D>& task) {
        const int parts = task.parts, sets = task.sets;
        const Barriers bar{bar_s + (decltype(apart)::value ? 256u : 0u)};
        if (parts > 0) {
            constexpr uint32_t kIdQk = idesc(true, false, 64), kIdPv = idesc(false, true, D);
            constexpr uint32_t kPanel = KT * 128;
            const uint64_t q_d = desc_k(q_s), k_d = desc_k(k_s), v_d = desc_v(v_s, kPanel);
            // bytes to descriptor units
            auto units = [](uint32_t bytes) { return (uint64_t)(bytes >> 4); };
            // scores of part i (64 rows of its tile's keys, score buffer i & 1) for both
            // sets; a tile's keys are done with its last part
            auto scores = [&](int i) {
                const int j = i / T::kParts;
                if (i % T::kParts == 0 && !wait.all(bar.kfull(j & 1), (j >> 1) & 1)) return false;
                tmem_fence_after();
                const uint64_t b0 = k_d + units((uint32_t)(j & 1) * T::kStage +
                                                (uint32_t)(i % T::kParts) * 8192);
                for (int set = 0; set < sets; ++set) {
                    const uint32_t sb = (uint32_t)(2 * set + (i & 1));
                    const uint64_t a0 = q_d + units((uint32_t)set * 128 * T::kPanels * 128);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        mma_ss(tmem + sb * 64, a0 + units((k / 4) * 128 * 128) + 2 * (k % 4),
                               b0 + units((k / 4) * kPanel) + 2 * (k % 4), kIdQk, k != 0);
                    commit(bar.sfull(sb));
                }
                if (i % T::kParts == T::kParts - 1) commit(bar.kempty(j & 1));
                return true;
            };
            bool ok = wait.all(qfull, 0) && scores(0);
            for (int i = 0; i < parts && ok; ++i) {
                // part i + 1's buffer held the weights of part i - 1, whose product was
                // issued before
                if (i + 1 < parts) ok = scores(i + 1);
                const int j = i / T::kParts;
                if (ok && i % T::kParts == 0) ok = wait.all(bar.vfull(j & 1), (j >> 1) & 1);
                const uint64_t b0 = v_d + units((uint32_t)(j & 1) * T::kStage +
                                                (uint32_t)(i % T::kParts) * 8192);
                for (int set = 0; set < sets && ok; ++set) {
                    const uint32_t sb = (uint32_t)(2 * set + (i & 1));
                    ok = wait.all(bar.pfull(sb), (i >> 1) & 1);
                    if (!ok) break;
                    tmem_fence_after();
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_ts(tmem + T::kOCol + set * D, tmem + sb * 64 + 8 * k,
                               b0 + units(k * 2048), kIdPv, i != 0 || k != 0);
                    commit(bar.ofull(set));
                }
                if (ok && i % T::kParts == T::kParts - 1) commit(bar.vempty(j & 1));
            }
            // every MMA issued has completed once this commit arrives
            commit(bar.drain());
            if (!mbar_wait_clock(bar.drain(), 0, nullptr)) {
                if (lane == 0) report_status(status, HBL_ERR_TIMEOUT);
                *abort_flag = 1;
            }
        }
    };
    auto widen = [&](auto apart, const Task<D>& task) {
        constexpr bool APART = decltype(apart)::value;
        const Barriers bar{bar_s + (APART ? 256u : 0u)};
        const k12::Split& sp = task.sp;
        const int b = task.b, tiles = task.tiles;
        const int cw = warp >= 8 ? warp - 8 : warp + 3;  // warps 8 .. 14, then 4 .. 7
        const Lane<D> ln(lane);
        uint32_t raw[2][T::kMine][B];  // keys, values: loaded a tile ahead
        int page[2][T::kMine];  // of the units that are loaded next: keys, values
        // this warp's i-th unit of a tile of K (values: dealt out from where the keys'
        // left off, so that all get about the same)
        constexpr int kConv = T::kConv, kTurn = kConv - T::kUnits % kConv;
        auto unit = [&](bool val, int i) { return (val ? (cw + kTurn) % kConv : cw) + kConv * i; };
        auto key_of = [&](int phase, int i) {  // phase 2j: keys of tile j, 2j + 1: values
            return sp.begin + (phase >> 1) * KT + unit(phase & 1, i) * Lane<D>::kRows + ln.row;
        };
        auto load_page = [&](int phase, int i) {
            const int key = key_of(phase, i);
            page[phase & 1][i] = unit(phase & 1, i) < T::kUnits && key < sp.end
                                     ? kv_page(kb, c.num_pages, b, (int)pl.div_page(key))
                                     : -1;
        };
        // the codes of a unit, whose page was looked up a tile ago
        auto load = [&](int phase, int i) {
            uint32_t(&to)[B] = raw[phase & 1][i];
            const int key = key_of(phase, i), pg = page[phase & 1][i];
            if (pg >= 0) {
                const int64_t row = ((int64_t)pg * c.heads + h) * c.page_size +
                                    (key - (int)pl.div_page(key) * c.page_size);
                const uint8_t* src = ((phase & 1) ? c.vc : c.kc) + row * ROW_BYTES +
                                     ln.group * (4 * B);
                if constexpr (B % 4 == 0) {
#pragma unroll
                    for (int k = 0; k < B / 4; ++k) {
                        const uint4 v = __ldg(reinterpret_cast<const uint4*>(src) + k);
                        to[4 * k] = v.x;
                        to[4 * k + 1] = v.y;
                        to[4 * k + 2] = v.z;
                        to[4 * k + 3] = v.w;
                    }
                } else if constexpr (B == 2) {
                    const uint2 v = __ldg(reinterpret_cast<const uint2*>(src));
                    to[0] = v.x;
                    to[1] = v.y;
                } else {
#pragma unroll
                    for (int k = 0; k < B; ++k)
                        to[k] = __ldg(reinterpret_cast<const uint32_t*>(src) + k);
                }
            } else {  // nothing there: any finite codes (their weight is zero)
#pragma unroll
                for (int k = 0; k < B; ++k) to[k] = 0;
            }
            load_page(phase + 2, i);
        };
        uint32_t lane_at[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) lane_at[k] = chunk_at(KT, ln.row, ln.group, k);
        auto store = [&](auto bf16, int i, int u, uint32_t dst) {
            uint32_t out[16];
            widen32<B, decltype(bf16)::value>(raw[decltype(bf16)::value ? 0 : 1][i], out);
            // (row & 7, which the swizzle goes by, is the lane's own where a unit
            // has a multiple of eight rows, and flips bit 2 in odd units of four)
            const uint32_t to = dst + u * Lane<D>::kRows * 128;
            const uint32_t flip = Lane<D>::kRows % 8 == 0 ? 0u : (uint32_t)(u & 1) << 6;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                sts128(to + (lane_at[k] ^ flip),
                       make_uint4(out[4 * k], out[4 * k + 1], out[4 * k + 2], out[4 * k + 3]));
        };
        const float xscale = a.scale * 1.4426950408889634f;
        // scales of a tile: four positions a lane, by the last widening warp, which
        // looks up their page a tile before
        float4 sk, sv;
        bool sc_there = false;
        int sc_page = -2;
        auto load_scales_page = [&](int j) {
            const int key = sp.begin + j * KT + 4 * lane;
            if (4 * lane < KT && key < sp.end) {
                sc_page = kv_page(kb, c.num_pages, b, (int)pl.div_page(key));
            } else {
                sc_page = -2;  // no position; -1: no such page
            }
        };
        auto load_scales = [&](int j) {
            const int key = sp.begin + j * KT + 4 * lane;
            sc_there = sc_page >= 0;
            if (sc_page == -1) report_status(status, HBL_ERR_INVALID_ARG);
            if (sc_there) {
                const int64_t row = ((int64_t)sc_page * c.heads + h) * c.page_size +
                                    (key - (int)pl.div_page(key) * c.page_size);
                sk = *reinterpret_cast<const float4*>(c.ks + row);
                sv = *reinterpret_cast<const float4*>(c.vs + row);
            }
            load_scales_page(j + 1);
        };
        auto store_scales = [&](int j) {
            if (4 * lane >= KT) return;
            const uint32_t sc = sc_s + (j % kScaleStages) * T::kScale;
            const int key = sp.begin + j * KT + 4 * lane;
            const float k4[4] = {sk.x, sk.y, sk.z, sk.w}, v4[4] = {sv.x, sv.y, sv.z, sv.w};
            float ck[4], lv[4], rs[4];
            bool odd = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                // a position that is not there: 0 * x - inf
                const bool there = sc_there && key + e < sp.end;
                ck[e] = there ? __fmul_rn(k4[e], xscale) : 0.f;
                if constexpr (APART) {
                    lv[e] = there ? fmaxf(lg2_any(v4[e]), k12::kNoScale) : kNowhere;
                    rs[e] = 0.f;  // (not used)
                } else {
                    lv[e] = there ? fmaxf(lg2(v4[e]), k12::kZeroFold) : -CUDART_INF_F;
                    rs[e] = there ? ex2(-lv[e]) : 0.f;
                    odd |= there && !k12::folds(v4[e]);
                }
            }
            if (odd) sts32(odd_s, 1);
            auto f = [](float v) { return __float_as_uint(v); };
            sts128(sc + lane * 32, make_uint4(f(ck[0]), f(ck[1]), f(lv[0]), f(lv[1])));
            sts128(sc + lane * 32 + 16, make_uint4(f(ck[2]), f(ck[3]), f(lv[2]), f(lv[3])));
            sts128(sc + KT * 8 + lane * 16, make_uint4(f(rs[0]), f(rs[1]), f(rs[2]), f(rs[3])));
        };
        const bool scales = cw == kConv - 1;
        if (scales) {
            load_scales_page(0);
            load_scales(0);
        }
#pragma unroll
        for (int i = 0; i < T::kMine; ++i) {
            load_page(0, i);
            load_page(1, i);
        }
#pragma unroll
        for (int i = 0; i < T::kMine; ++i) load(0, i);
#pragma unroll
        for (int i = 0; i < T::kMine; ++i) load(1, i);
        bool ok = true;
#pragma unroll 1
        for (int j = 0; j < tiles && ok; ++j) {
            const int st = j & 1;
            const uint32_t par = ((j >> 1) & 1) ^ 1;
            if (scales) {
                if (j >= kScaleStages)
                    ok = wait.all(bar.scempty(j % kScaleStages), ((j / kScaleStages) & 1) ^ 1);
                if (!ok) break;
                store_scales(j);
                __syncwarp();
                if (lane == 0) mbar_arrive_one(bar.scfull(j % kScaleStages));
                load_scales(j + 1);
            }
            if (j >= 2) ok = wait.all(bar.kempty(st), par);
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < T::kMine; ++i) {
                const int u = unit(false, i);
                if (u < T::kUnits) store(ic_bool<true>{}, i, u, k_s + st * T::kStage);
                load(2 * j + 2, i);
            }
            fence_async();
            __syncwarp();
            if (lane == 0) mbar_arrive_one(bar.kfull(st));
            if (j >= 2) ok = wait.all(bar.vempty(st), par);
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < T::kMine; ++i) {
                const int u = unit(true, i);
                if (u < T::kUnits) store(ic_bool<false>{}, i, u, v_s + st * T::kStage);
                load(2 * j + 3, i);
            }
            fence_async();
            __syncwarp();
            if (lane == 0) mbar_arrive_one(bar.vfull(st));
        }
    };
    // behind a pass: what tensor memory holds is read; all roles know of a second one
    auto done = [&] {
        __syncwarp();
        tmem_fence_before();
        asm volatile("barrier.sync 0;" ::: "memory");
        tmem_fence_after();
    };
    auto again = [&] {
        done();
        return lds32(odd_s) != 0 && *abort_flag == 0;
    };
    if (warp < 4 * NQ) {
        // ================= softmax
        reg_alloc<144>();
        const int set = warp >> 2, quarter = warp & 3;
        if (set < first.sets) {
            const k12::Rows& s = first.s;
            const int row0 = first.row0, nr = first.nr;
            // ---- this set's queries into the operand layout
            const Lane<D> ql(lane);
            const uint32_t qbase = q_s + set * 128 * T::kPanels * 128;
            constexpr int kUnits = 128 / Lane<D>::kRows;
            constexpr int kLoads = kUnits >= 16 ? 4 : kUnits / 4;  // units in flight
#pragma unroll 1
            for (int u0 = quarter; u0 < kUnits; u0 += 4 * kLoads) {
                uint32_t raw[kLoads][16];
#pragma unroll
                for (int v = 0; v < kLoads; ++v) {
                    const int u = u0 + 4 * v, row = u * Lane<D>::kRows + ql.row;
                    const int r = row0 + set * 128 + row, i = r / a.group;
                    const uint16_t* src = a.q + (int64_t)(s.row0 + i) * a.q_row +
                                          (int64_t)(h * a.group + (r - i * a.group)) * a.q_head +
                                          ql.group * 32;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint4 z = r < nr
                                            ? reinterpret_cast<const uint4*>(src)[k]
                                            : make_uint4(0, 0, 0, 0);
                        raw[v][4 * k] = z.x;
                        raw[v][4 * k + 1] = z.y;
                        raw[v][4 * k + 2] = z.z;
                        raw[v][4 * k + 3] = z.w;
                    }
                }
#pragma unroll
                for (int v = 0; v < kLoads; ++v) {
                    const int u = u0 + 4 * v;
                    uint32_t out[16];
                    static_for<0, 16>([&](auto pp) {
                        constexpr int e0 = place_of<B>(2 * decltype(pp)::value);
                        constexpr int e1 = place_of<B>(2 * decltype(pp)::value + 1);
                        out[decltype(pp)::value] =
                            __byte_perm(raw[v][e0 / 2], raw[v][e1 / 2],
                                        (e0 & 1 ? 0x32 : 0x10) | (e1 & 1 ? 0x7600 : 0x5400));
                    });
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        sts128(qbase + chunk_at(128, u * Lane<D>::kRows + ql.row, ql.group, k),
                               make_uint4(out[4 * k], out[4 * k + 1], out[4 * k + 2],
                                          out[4 * k + 3]));
                }
            }
            fence_async();
            __syncwarp();
            if (lane == 0) first.arrive_for_all(qfull);

            softmax(ic_bool<false>{}, first);
        }
        if (again()) {
            const Task<D> task = task_of<D>(pl, c, kb, a, where, split);
            if (set < task.sets) softmax(ic_bool<true>{}, task);
            done();
        }
    } else {
        if (warp >= 8) reg_dealloc<112>();  // (warps 4 .. 7 keep what they have)
        if (warp == kMmaWarp) {
            // ================= MMA issue
            issue(ic_bool<false>{}, first);
            if (again()) {
                issue(ic_bool<true>{}, task_of<D>(pl, c, kb, a, where, split));
                done();
            }
        } else {
            // ================= widening
            if (first.tiles > 0) widen(ic_bool<false>{}, first);
            if (again()) {
                widen(ic_bool<true>{}, task_of<D>(pl, c, kb, a, where, split));
                done();
            }
        }
    }
    __syncwarp();
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem)
                     : "memory");
    }
}

template <int D, int B>
hbl_status launch(const KvCache& c, const KvBatch& kb, const KvAttn& a, const Plan& pl, float* part,
                  int32_t* status, cudaStream_t stream) {
    auto kern = chunk_kernel<D, B>;
    if (!smem_attr_once(reinterpret_cast<const void*>(kern), Tile<D>::kSmem)) return HBL_ERR_CUDA;
    const unsigned grid = (unsigned)(pl.row_blocks * pl.splits * c.heads);  // (it fits 31 bits)
    kern<<<grid, kThreads, Tile<D>::kSmem, stream>>>(c, kb, a, pl, part, status);
    return cudaGetLastError() == cudaSuccess ? HBL_OK : HBL_ERR_CUDA;
}

template <int D>
hbl_status launch_d(const KvCache& c, const KvBatch& kb, const KvAttn& a, const Plan& pl,
                    float* part, int32_t* status, cudaStream_t stream) {
    switch (c.bits) {
        case 2: return launch<D, 2>(c, kb, a, pl, part, status, stream);
        case 3: return launch<D, 3>(c, kb, a, pl, part, status, stream);
        case 4: return launch<D, 4>(c, kb, a, pl, part, status, stream);
        default: return launch<D, 8>(c, kb, a, pl, part, status, stream);
    }
}

}  // namespace k14
}  // namespace hbl
