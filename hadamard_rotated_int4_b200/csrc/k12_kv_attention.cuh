// k12_kv_attention.cuh -- what the attention kernels over the paged cache share:
// a sequence's rows and their visible positions, the split of a range of
// positions over CTAs, and the final store of a row.
//
// Head rows.  A cached head's query rows of one sequence are numbered
// r = token * group + j (group = query heads per cached head), so all query
// heads of a cached head share its codes within a CTA.
#pragma once

#include <math_constants.h>

#include "hbl_kv.cuh"

namespace hbl {

// ---- arithmetic of the kernels
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
__device__ __forceinline__ float lg2_any(float x) {  // subnormal x too
    float r;
    asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// Two fp32 -> an fp16 pair (low half = first), round to nearest even.
__device__ __forceinline__ uint32_t f2_to_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

namespace k12 {

// How a launch is laid out; made on the host from sizes alone (few_plan,
// chunk_plan).
struct Plan {
    int block_rows;          // head rows of a CTA
    int row_blocks;          // few rows: most blocks to a sequence; chunks: most in all
    int min_rows, max_rows;  // the kernel takes sequences with so many head rows
    int splits;              // chunks: most ranges of positions of one row block
    int quantum;             // chunks: positions of a range (more where `splits` do not reach)
    int ctas, min_units;     // few rows: CTAs, and the fewest units that are worth one
    int unit;                // few rows: positions of a unit, a multiple of 64
    bool whole;              // few rows: an item is one unit, whatever it sees
    int seg_shift;           // 16, 32 or 64 positions (log2) that a page holds a multiple of
    uint32_t page_mul, page_shift;  // x / page_size = (mulhi(x, mul) + x) >> shift, x < 2^31

    __device__ __forceinline__ uint32_t div_page(uint32_t x) const {
        return (__umulhi(x, page_mul) + x) >> page_shift;
    }
};

struct Rows {
    int row0, n;  // packed rows of the sequence that this call attends from
    int first;    // position of the first (negative: no place)
    int len;
    bool bad;
};
__device__ __forceinline__ Rows rows_of(const KvBatch& kb, int page_size, const KvAttn& a, int b) {
    const KvSeq s = kv_seq(kb, page_size, b);
    Rows r;
    r.row0 = s.r0;
    r.n = min(s.r1 - s.r0, a.max_rows);
    r.first = s.first;
    r.len = s.len;
    r.bad = s.bad || r.n < s.r1 - s.r0;
    return r;
}

// First position that a window leaves visible from position p.
__device__ __forceinline__ int window_begin(const KvAttn& a, int p) {
    return a.window > 0 ? (int)max((int64_t)0, (int64_t)p - a.window + 1) : 0;
}

// Positions that head rows r0 .. r1 see between them (r0 == r1: that row's).
struct Range {
    int begin, end;
};
__device__ __forceinline__ Range range_of(const KvAttn& a, const Rows& s, int r0, int r1) {
    Range w;
    w.end = a.causal ? min(s.len, s.first + r1 / a.group + 1) : s.len;
    w.end = max(w.end, 0);
    w.begin = min(window_begin(a, s.first + r0 / a.group), w.end);
    return w;
}

// Range number `split` of a row block's positions: whole groups of 64 from a
// multiple of 64 on, equal ones, the last one shorter.
struct Split {
    int begin, end;
    int count;  // ranges of this row block
};
__device__ __forceinline__ Split split_of(const Plan& pl, const Range& rg, int split) {
    Split s;
    const int from = rg.begin & ~63, total = rg.end > rg.begin ? rg.end - from : 0;
    const int q = max(pl.quantum, ((total + pl.splits - 1) / pl.splits + 127) & ~127);
    s.count = (int)(((uint32_t)total + (uint32_t)q - 1u) / (uint32_t)q);
    s.begin = (int)((uint32_t)from + (uint32_t)split * (uint32_t)q);
    s.end = (int)min((int64_t)s.begin + q, (int64_t)rg.end);
    return s;
}

// ---- V's scales and the reference points of a row
// O's sum and its normaliser, with scores s and V's scales sv, both in log2:
//   O = sum_i 2^(s_i + sv_i - M) v_i / sum_i 2^(s_i - R) * 2^(M - R).
// M follows the largest s + sv.  Where all of V's scales lie in 2^-kFold .. 2^kFold, R is
// M, and the second sum is that of w_i / sv_i of the weights w_i that the product needs
// anyway; a zero scale counts as 2^kZeroFold (its codes are zeros, and only its score
// matters; weights of 2^-126 are 2^-32 of the largest score's at most).  Past
// that the weights of small scales, or 1 / sv, leave fp32's range.  A kernel
// that meets such a scale takes its positions once more and sums 2^(s_i - R) apart, R the
// largest s: an exponential a score more, and no scale is too large or too small.  What
// it hands on is O's sum and the normaliser against one point, half way between M
// and R (at most 150 apart): both stay in range.
constexpr float kFold = 40.f, kZeroFold = -60.f;
constexpr float kNoScale = -150.f;  // log2 of a zero scale apart: below every other
__device__ __forceinline__ bool folds(float sv) {  // zero, or of 2^-kFold .. 2^kFold
    constexpr uint32_t kLow = (uint32_t)(127 - (int)kFold) << 23;
    constexpr uint32_t kSpan = (uint32_t)(2 * (int)kFold) << 23;
    const uint32_t bits = __float_as_uint(sv);
    return bits == 0 || bits - kLow <= kSpan;
}

// Partial results of chunks: [split][packed row][query head] x (D values, m, sum, 2 unused).
__device__ __forceinline__ int64_t part_index(const KvBatch& kb, const KvAttn& a, int split,
                                              int64_t t, int head) {
    return ((int64_t)split * kb.rows + t) * a.heads + head;
}

// ---- chunks: which row block a CTA has
// The row blocks (of BLOCK head rows) of the sequences that the kernel takes, in the
// order that their CTAs start: of each 32 sequences the block that ends farthest back
// first, which under a causal mask is the one with the most to do, so that short ones
// fill the gaps at the end.  Block `index` is block rb of sequence b (b = -1: there
// are not so many); by one warp, a lane to a sequence.
struct Block {
    int b, rb;
};
template <int BLOCK>
__device__ __forceinline__ Block block_of(const Plan& pl, const KvCache& c, const KvBatch& kb,
                                          const KvAttn& a, int index) {
    auto sum = [](int v) { return (int)__reduce_add_sync(0xffffffffu, (unsigned)v); };
    const int lane = threadIdx.x & 31;
    for (int i = 0; i < kb.num_seqs; i += 32) {
        // of sequence i + lane: its row blocks, the position of its first token and how
        // many follow it (without a causal mask all blocks end with the sequence)
        int n = 0, first = -1, tokens = 0;
        if (i + lane < kb.num_seqs) {
            const Rows s = rows_of(kb, c.page_size, a, i + lane);
            const int nr = s.n * a.group;
            if (nr >= pl.min_rows && nr <= pl.max_rows) {
                n = (nr + BLOCK - 1) / BLOCK;
                first = a.causal ? s.first : s.len - 1;
                tokens = a.causal ? s.n - 1 : 0;
            }
        }
        const int total = sum(n);
        if (index < total) {
            // this lane's blocks that end at position `end` or behind it: those from the
            // block of token x on
            auto count = [&](int end) {
                const unsigned x = (unsigned)(end - 1) - (unsigned)first;
                const int from = (int)(x * (unsigned)a.group / BLOCK);
                return end <= 0 || end - 1 < first ? n : x > (unsigned)tokens ? 0 : n - from;
            };
            int lo = 0, hi = (int)__reduce_max_sync(0xffffffffu,
                                                    (unsigned)max(first + tokens + 1, 0)) + 1;
            while (hi - lo > 1) {  // more than `index` end at lo or behind, not at hi
                const int mid = lo + (hi - lo) / 2;
                if (sum(count(mid)) > index)
                    lo = mid;
                else
                    hi = mid;
            }
            // those that end at lo, sequence by sequence
            const int past = count(lo + 1), mine = count(lo) - past;
            int upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += u;
            }
            const int left = index - sum(past);
            const bool here = left < upto && left >= upto - mine;
            const int who = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
            const int rb = n - past - 1 - (left - (upto - mine));
            return {i + who, __shfl_sync(0xffffffffu, rb, who)};
        }
        index -= total;
    }
    return {-1, 0};
}

// ---- few rows: all work in one line, cut into equal pieces
// An item is one row block of one sequence on every cached head: heads times
// `units` units of pl.unit positions.  The line runs item by item, head by head;
// CTA i takes units [i * per, (i + 1) * per), whichever sequences they are of.  The
// host makes the unit large enough for the line to fit 31 bits.
struct Item {
    Rows s;
    Range rg;
    int nr, from, units;  // head rows of the sequence; first position; units of one head
};
__device__ __forceinline__ Item item_of(const Plan& pl, const KvCache& c, const KvBatch& kb,
                                        const KvAttn& a, int i) {
    Item t;
    const int b = i / pl.row_blocks, r0 = (i - b * pl.row_blocks) * pl.block_rows;
    t.s = rows_of(kb, c.page_size, a, b);
    t.nr = t.s.n * a.group;
    t.units = 0;
    if (t.nr >= pl.min_rows && t.nr <= pl.max_rows && r0 < t.nr) {
        t.rg = range_of(a, t.s, r0, min(t.nr, r0 + pl.block_rows) - 1);
        t.from = t.rg.begin & ~63;
        // a block that sees nothing still has its rows stored
        // (`whole`: one unit even of a sequence that breaks the caller's max_rows, whose
        // rows then reach further back than was said: there is no room for pieces)
        const uint32_t seen = (uint32_t)(t.rg.end - t.from), unit = (uint32_t)pl.unit;
        t.units = pl.whole ? 1 : max(1, (int)((seen + unit - 1) / unit));
    }
    return t;
}

// Units of a CTA of a line of `total`.
__device__ __forceinline__ int cut(const Plan& pl, int total) {
    const uint32_t n = min(max((uint32_t)total / (uint32_t)pl.min_units, 1u), (uint32_t)pl.ctas);
    return (int)(((uint32_t)total + n - 1) / n);
}

// The line's cut, and where the first unit of piece `cta` lies (LAST: its last
// unit); by all threads.  The items' units are summed once, and once more up to
// that unit where they are more than one to a thread.
struct Line {
    int total, per;
    int at;            // that unit; not below `total`: there is no such piece
    int item, before;  // of that unit; the line's units before the item
};
template <int kThreads, bool LAST>
__device__ __forceinline__ Line line_of(const Plan& pl, const KvCache& c, const KvBatch& kb,
                                        const KvAttn& a, int cta, int32_t* status) {
    __shared__ int warp_sum[kThreads / 32];
    __shared__ int found[2];
    const int items = kb.num_seqs * pl.row_blocks;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Line line;
    int mine = 0;
    bool bad = false;
    for (int i = threadIdx.x; i < items; i += kThreads) {
        const Item t = item_of(pl, c, kb, a, i);
        mine += t.units * c.heads;
        bad |= t.s.bad;
    }
    if (bad) report_status(status, HBL_ERR_INVALID_ARG);
    // inclusive sums over the CTA: v's up to this thread, and of all
    auto scan = [&](int v, int* all) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        if (lane == 31) warp_sum[warp] = v;
        __syncthreads();
        *all = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) v += warp_sum[w];
            *all += warp_sum[w];
        }
        return v;
    };
    const int upto = scan(mine, &line.total);
    line.per = cut(pl, line.total);
    const int64_t first = (int64_t)cta * line.per;
    line.at = line.total;
    if (first >= line.total) return line;  // the same for the whole CTA
    line.at = (int)(LAST ? min(first + line.per, (int64_t)line.total) - 1 : first);
    const int at = line.at;
    if (items <= kThreads) {
        if (at >= upto - mine && at < upto) {
            found[0] = threadIdx.x;
            found[1] = upto - mine;
        }
    } else {
        int before = 0;
        for (int i = 0; i < items && before <= at; i += kThreads) {
            int v = 0, all;
            if (i + (int)threadIdx.x < items)
                v = item_of(pl, c, kb, a, i + threadIdx.x).units * c.heads;
            __syncthreads();  // the sums of the step before are read
            const int u = before + scan(v, &all);
            if (at >= u - v && at < u) {
                found[0] = i + threadIdx.x;
                found[1] = u - v;
            }
            before += all;
        }
    }
    __syncthreads();
    line.item = found[0];
    line.before = found[1];
    return line;
}

// Partial results of few rows: two slots to a CTA, of the piece that goes on from
// the CTA before (0) and of one that begins here and ends elsewhere (1).
__device__ __forceinline__ float* slot_of(float* part, const Plan& pl, int D, int64_t cta, int slot) {
    return part + (cta * 2 + slot) * pl.block_rows * (D + 4);
}

// Where a head row's O goes, and 1 / L of its sum of weights L (against 2^M);
// stores the row's lse if this thread is the one to.
__device__ __forceinline__ uint16_t* row_out(const KvAttn& a, const Rows& s, int h, int row, float M,
                                             float L, bool store_lse, float* inv) {
    const int i = row / a.group, head = h * a.group + (row - i * a.group);
    const int64_t t = s.row0 + i;
    *inv = L == 0.f ? 0.f : __fdiv_rn(1.f, L);
    if (store_lse && a.lse != nullptr)
        a.lse[t * a.heads + head] =
            L == 0.f ? -CUDART_INF_F : __fmul_rn(M + log2f(L), 0.6931471805599453f);
    return a.o + t * a.o_row + (int64_t)head * a.o_head;
}
// Four values of a head row, from column d on, from their weighted sums y.
__device__ __forceinline__ void store_row4(const KvAttn& a, const Rows& s, int h, int row, int d,
                                           const float4& y, float M, float L) {
    float inv;
    uint16_t* dst = row_out(a, s, h, row, M, L, d == 0, &inv) + d;
    *reinterpret_cast<uint2*>(dst) = make_uint2(f2_to_bf16x2(y.x * inv, y.y * inv),
                                                f2_to_bf16x2(y.z * inv, y.w * inv));
}

}  // namespace k12

namespace k13 {
// Few rows: per head size, in files of their own (k13_kv_decode_d*.cu).
hbl_status launch_d32(const KvCache&, const KvBatch&, const KvAttn&, const k12::Plan&, float* part,
                      int32_t* status, cudaStream_t);
hbl_status launch_d64(const KvCache&, const KvBatch&, const KvAttn&, const k12::Plan&, float* part,
                      int32_t* status, cudaStream_t);
hbl_status launch_d128(const KvCache&, const KvBatch&, const KvAttn&, const k12::Plan&, float* part,
                       int32_t* status, cudaStream_t);
hbl_status launch_d256(const KvCache&, const KvBatch&, const KvAttn&, const k12::Plan&, float* part,
                       int32_t* status, cudaStream_t);
}  // namespace k13

namespace k14 {
// Chunks: per head size, in files of their own (k14_kv_chunk_d*.cu).
hbl_status launch_d32(const KvCache&, const KvBatch&, const KvAttn&, const k12::Plan&, float* part,
                      int32_t* status, cudaStream_t);
hbl_status launch_d64(const KvCache&, const KvBatch&, const KvAttn&, const k12::Plan&, float* part,
                      int32_t* status, cudaStream_t);
hbl_status launch_d128(const KvCache&, const KvBatch&, const KvAttn&, const k12::Plan&, float* part,
                       int32_t* status, cudaStream_t);
hbl_status launch_d256(const KvCache&, const KvBatch&, const KvAttn&, const k12::Plan&, float* part,
                       int32_t* status, cudaStream_t);
}  // namespace k14
}  // namespace hbl
