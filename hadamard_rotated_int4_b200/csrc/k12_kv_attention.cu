// k12_kv_attention.cu -- attention over the paged low-bit cache: the launch plan
// and the joining of ranges of positions.
#include "k12_kv_attention.cuh"

namespace hbl {
namespace k12 {

// Joins the ranges of a head row: O = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s.
// One warp per head row, D/32 values a lane; a row with one range was stored by
// the kernel that computed it.
constexpr int kThreads = 128;

template <int D>
__global__ void __launch_bounds__(kThreads) combine_kernel(KvCache c, KvBatch kb, KvAttn a, Plan pl,
                                                           const float* part) {
    constexpr int N = D / 32;
    const int lane = threadIdx.x & 31;
    const int rows = pl.row_blocks * pl.block_rows;
    const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int row = (int)(w % rows), h = (int)(w / rows % c.heads), b = (int)(w / rows / c.heads);
    Rows s = {};
    int count = 0;
    if (b < kb.num_seqs) {
        s = rows_of(kb, c.page_size, a, b);
        const int nr = s.n * a.group, r0 = row / pl.block_rows * pl.block_rows;
        if (row < nr && nr <= pl.few_rows)
            count = split_of(pl, range_of(a, s, r0, min(nr, r0 + pl.block_rows) - 1), 0).count;
    }
    // every thread waits: the grid must not end before the one it depends on
    pdl_wait();
    if (count <= 1) return;
    const float* src = part + part_index(pl, c, b, h, 0, row) * (D + 4);
    const int64_t next = (int64_t)rows * (D + 4);
    float M = -CUDART_INF_F;
    for (int k = lane; k < count; k += 32) M = fmaxf(M, src[k * next + D]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float L = 0.f, y[N];
#pragma unroll
    for (int i = 0; i < N; ++i) y[i] = 0.f;
    for (int k = 0; k < count; ++k) {
        const float* p = src + k * next;
        const float m = p[D], f = m == -CUDART_INF_F ? 0.f : exp2f(m - M);
        L = __fmaf_rn(p[D + 1], f, L);
#pragma unroll
        for (int i = 0; i < N; ++i) y[i] = __fmaf_rn(p[32 * i + lane], f, y[i]);
    }
    const int i = row / a.group, head = h * a.group + (row - i * a.group);
    const int64_t t = s.row0 + i;
    const float inv = L == 0.f ? 0.f : __fdiv_rn(1.f, L);
    uint16_t* dst = a.o + t * a.o_row + (int64_t)head * a.o_head;
#pragma unroll
    for (int k = 0; k < N; ++k)
        dst[32 * k + lane] = (uint16_t)(f2_to_bf16x2(y[k] * inv, 0.f) & 0xffffu);
    if (a.lse != nullptr && lane == 0)
        a.lse[t * a.heads + head] =
            L == 0.f ? -CUDART_INF_F : __fmul_rn(M + log2f(L), 0.6931471805599453f);
}

static int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

Plan make_plan(const KvCache& c, const KvBatch& b, const KvAttn& a) {
    constexpr int kSizingSms = 148;  // the workspace must not depend on the device
    Plan p = {};
    const int64_t rows = (int64_t)a.max_rows * a.group;
    p.block_rows = c.D <= 128 && rows > 8 ? 16 : 8;
    p.row_blocks = (int)ceil_div(rows, p.block_rows);
    p.few_rows = 0x7fffffff;
    int64_t span = a.max_kv;
    if (a.window > 0 && span > (int64_t)a.window + a.max_rows)
        span = (int64_t)a.window + a.max_rows;
    const int64_t ctas = (int64_t)b.num_seqs * c.heads * p.row_blocks;
    int64_t q = ceil_div(ctas * span, kSizingSms * 6);
    q = (q < 256 ? 256 : q + 127) & ~127ll;
    p.splits = (int)ceil_div(span, q);
    if (p.splits < 1) p.splits = 1;
    if (p.splits > 256) p.splits = 256;
    p.quantum = (int)(q < 0x40000000 ? q : 0x40000000);
    // round-up reciprocal: exact for x < 2^31
    uint32_t l = 0;
    while ((1ull << l) < (uint32_t)c.page_size) ++l;
    p.page_shift = l;
    p.page_mul = (uint32_t)((((1ull << l) - c.page_size) << 32) / c.page_size + 1);
    return p;
}

}  // namespace k12

size_t kv_attention_workspace(const KvCache& c, const KvBatch& b, const KvAttn& a) {
    const k12::Plan p = k12::make_plan(c, b, a);
    if (p.splits == 1) return 0;
    return (size_t)b.num_seqs * c.heads * p.splits * p.row_blocks * p.block_rows * (c.D + 4) *
           sizeof(float);
}

hbl_status launch_kv_attention(const KvCache& c, const KvBatch& b, const KvAttn& a, void* ws,
                               int32_t* status, cudaStream_t stream, int num_sms) {
    (void)num_sms;
    const k12::Plan p = k12::make_plan(c, b, a);
    float* part = static_cast<float*>(ws);
    const int64_t ctas = (int64_t)b.num_seqs * p.row_blocks * p.splits;
    const int64_t join =
        k12::ceil_div((int64_t)b.num_seqs * c.heads * p.row_blocks * p.block_rows, 4);
    if (ctas > 0x7fffffffll || join > 0x7fffffffll) return HBL_ERR_SHAPE;
    hbl_status st;
    switch (c.D) {
        case 32: st = k13::launch_d32(c, b, a, p, part, status, stream); break;
        case 64: st = k13::launch_d64(c, b, a, p, part, status, stream); break;
        case 128: st = k13::launch_d128(c, b, a, p, part, status, stream); break;
        default: st = k13::launch_d256(c, b, a, p, part, status, stream); break;
    }
    if (st != HBL_OK || p.splits == 1) return st;
    const dim3 grid((unsigned)join), block(k12::kThreads);
    switch (c.D) {
        case 32: return launch_pdl(k12::combine_kernel<32>, grid, block, 0, stream, c, b, a, p, part);
        case 64: return launch_pdl(k12::combine_kernel<64>, grid, block, 0, stream, c, b, a, p, part);
        case 128:
            return launch_pdl(k12::combine_kernel<128>, grid, block, 0, stream, c, b, a, p, part);
        default:
            return launch_pdl(k12::combine_kernel<256>, grid, block, 0, stream, c, b, a, p, part);
    }
}

}  // namespace hbl
