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
namespace k12 {

// How the launch is split; made on the host from sizes alone (few_plan, chunk_plan).
struct Plan {
    int block_rows;  // head rows of a CTA
    int row_blocks;  // CTAs to a sequence's head rows
    int min_rows, max_rows;  // the kernel takes sequences with so many head rows
    int splits;      // most ranges of positions of one row block
    int quantum;     // positions of a range (more where `splits` ranges would not reach)
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
    r.first = s.len - (s.r1 - s.r0);
    r.len = s.len;
    r.bad = s.bad || r.n < s.r1 - s.r0;
    return r;
}

// Positions that head rows r0 .. r1 see between them (r0 == r1: that row's).
struct Range {
    int begin, end;
};
__device__ __forceinline__ Range range_of(const KvAttn& a, const Rows& s, int r0, int r1) {
    Range w;
    w.end = a.causal ? min(s.len, s.first + r1 / a.group + 1) : s.len;
    w.end = max(w.end, 0);
    w.begin = a.window > 0 ? max(0, s.first + r0 / a.group - a.window + 1) : 0;
    w.begin = min(w.begin, w.end);
    return w;
}

// Range number `split` of a row block's positions: whole groups of 16 (a group
// never crosses a page), equal ones, the last one shorter.
struct Split {
    int begin, end;
    int count;  // ranges of this row block
};
__device__ __forceinline__ Split split_of(const Plan& pl, const Range& rg, int split) {
    Split s;
    const int from = rg.begin & ~15, total = rg.end > rg.begin ? rg.end - from : 0;
    const int q = max(pl.quantum, ((total + pl.splits - 1) / pl.splits + 127) & ~127);
    s.count = (total + q - 1) / q;
    s.begin = from + split * q;
    s.end = min(s.begin + q, rg.end);
    return s;
}

// Partial results: [seq][cached head][split][row] x (D values, m, sum, 2 unused).
__device__ __forceinline__ int64_t part_index(const Plan& pl, const KvCache& c, int b, int h,
                                              int split, int row) {
    return (((int64_t)b * c.heads + h) * pl.splits + split) * ((int64_t)pl.row_blocks *
                                                               pl.block_rows) + row;
}

// Values d .. d + N - 1 of a head row from its weighted sum y and sum of weights
// L, both against 2^M; the thread with d == 0 stores the row's lse.
template <int N>
__device__ __forceinline__ void store_row(const KvAttn& a, const Rows& s, int h, int row, int d,
                                          const float* y, float M, float L) {
    const int i = row / a.group, head = h * a.group + (row - i * a.group);
    const int64_t t = s.row0 + i;
    const float inv = L == 0.f ? 0.f : __fdiv_rn(1.f, L);
    uint32_t w[N / 2];
#pragma unroll
    for (int k = 0; k < N / 2; ++k) w[k] = f2_to_bf16x2(y[2 * k] * inv, y[2 * k + 1] * inv);
    uint16_t* dst = a.o + t * a.o_row + (int64_t)head * a.o_head + d;
    if constexpr (N % 8 == 0) {
#pragma unroll
        for (int k = 0; k < N / 8; ++k)
            reinterpret_cast<uint4*>(dst)[k] =
                make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
    } else {
        static_assert(N == 4, "four values or whole 16-byte vectors");
        *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    }
    if (d == 0 && a.lse != nullptr)
        a.lse[t * a.heads + head] =
            L == 0.f ? -CUDART_INF_F : __fmul_rn(M + log2f(L), 0.6931471805599453f);
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
