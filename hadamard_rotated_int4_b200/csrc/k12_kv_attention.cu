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
        if (row < nr && nr >= pl.min_rows && nr <= pl.max_rows)
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

constexpr int kSizingSms = 148;  // the workspace must not depend on the device
// Sequences with at most this many head rows go to the few-rows kernel.
constexpr int kFewRows = 32;

// Round-up reciprocal of the page size: exact for x < 2^31.
static void set_page(Plan* p, int page_size) {
    uint32_t l = 0;
    while ((1ull << l) < (uint32_t)page_size) ++l;
    p->page_shift = l;
    p->page_mul = (uint32_t)((((1ull << l) - page_size) << 32) / page_size + 1);
}
// Positions that a row block can see, by the caller's hint.
static int64_t span_of(const KvAttn& a, int64_t rows) {
    const int64_t reach = (int64_t)a.window + rows;
    return a.window > 0 && a.max_kv > reach ? reach : a.max_kv;
}
static void set_splits(Plan* p, int64_t span, int64_t quantum) {
    const int64_t q = (quantum + 127) & ~127ll;
    int64_t n = ceil_div(span, q);
    n = n < 1 ? 1 : n > 256 ? 256 : n;
    p->splits = (int)n;
    p->quantum = (int)(q < 0x40000000 ? q : 0x40000000);
}

// Few rows: 8 or 16 head rows a CTA, ranges so that every SM has a few CTAs.
static Plan few_plan(const KvCache& c, const KvBatch& b, const KvAttn& a, int64_t rows) {
    Plan p = {};
    p.block_rows = c.D <= 128 && rows > 8 ? 16 : 8;
    p.row_blocks = (int)ceil_div(rows, p.block_rows);
    p.min_rows = 0;
    p.max_rows = (int)rows;
    const int64_t span = span_of(a, a.max_rows);
    const int64_t ctas = (int64_t)b.num_seqs * c.heads * p.row_blocks;
    const int64_t q = ceil_div(ctas * span, kSizingSms * 6);
    set_splits(&p, span, q < 256 ? 256 : q);
    set_page(&p, c.page_size);
    return p;
}

// Chunks: 256 head rows a CTA (128 at D = 256); ranges only where the row blocks
// leave SMs without work.
static Plan chunk_plan(const KvCache& c, const KvBatch& b, const KvAttn& a, int min_rows) {
    Plan p = {};
    const int64_t rows = (int64_t)a.max_rows * a.group;
    p.block_rows = c.D <= 128 ? 256 : 128;
    p.row_blocks = (int)ceil_div(rows, p.block_rows);
    p.min_rows = min_rows;
    p.max_rows = 0x7fffffff;
    // row blocks with rows in them: max_rows may be one sequence's alone
    int64_t blocks = (int64_t)b.num_seqs * p.row_blocks;
    const int64_t packed = (int64_t)b.rows * a.group / p.block_rows + b.num_seqs;
    if (blocks > packed) blocks = packed;
    const int64_t span = span_of(a, a.max_rows);
    const int64_t n = kSizingSms / (blocks * c.heads);
    const int64_t q = n <= 1 ? span : ceil_div(span, n);
    set_splits(&p, span, q < 512 ? 512 : q);
    set_page(&p, c.page_size);
    return p;
}

// The plans of a call: `few` and `chunk` say which kernels run.
struct Plans {
    bool few, chunk;
    Plan f, k;
};
static Plans plans_of(const KvCache& c, const KvBatch& b, const KvAttn& a) {
    Plans p = {};
    const int64_t rows = (int64_t)a.max_rows * a.group;
    p.chunk = rows > kFewRows;
    // one sequence that may be long is taken for long; among several, each goes
    // by its own rows
    p.few = !p.chunk || b.num_seqs > 1;
    if (p.few) p.f = few_plan(c, b, a, p.chunk ? kFewRows : rows);
    if (p.chunk) p.k = chunk_plan(c, b, a, p.few ? kFewRows + 1 : 0);
    return p;
}
static size_t part_bytes(const KvCache& c, const KvBatch& b, const Plan& p) {
    if (p.splits == 1) return 0;
    return (size_t)b.num_seqs * c.heads * p.splits * p.row_blocks * p.block_rows * (c.D + 4) *
           sizeof(float);
}
static bool fits(const KvCache& c, const KvBatch& b, const Plan& p) {
    return (int64_t)b.num_seqs * p.row_blocks * p.splits <= 0x7fffffffll &&
           ceil_div((int64_t)b.num_seqs * c.heads * p.row_blocks * p.block_rows, 4) <= 0x7fffffffll;
}

static hbl_status combine(const KvCache& c, const KvBatch& b, const KvAttn& a, const Plan& p,
                          const float* part, cudaStream_t stream) {
    if (p.splits == 1) return HBL_OK;
    const dim3 grid((unsigned)ceil_div(
        (int64_t)b.num_seqs * c.heads * p.row_blocks * p.block_rows, kThreads / 32)),
        block(kThreads);
    switch (c.D) {
        case 32: return launch_pdl(combine_kernel<32>, grid, block, 0, stream, c, b, a, p, part);
        case 64: return launch_pdl(combine_kernel<64>, grid, block, 0, stream, c, b, a, p, part);
        case 128: return launch_pdl(combine_kernel<128>, grid, block, 0, stream, c, b, a, p, part);
        default: return launch_pdl(combine_kernel<256>, grid, block, 0, stream, c, b, a, p, part);
    }
}

}  // namespace k12

size_t kv_attention_workspace(const KvCache& c, const KvBatch& b, const KvAttn& a) {
    const k12::Plans p = k12::plans_of(c, b, a);
    return (p.few ? k12::part_bytes(c, b, p.f) : 0) + (p.chunk ? k12::part_bytes(c, b, p.k) : 0);
}

hbl_status launch_kv_attention(const KvCache& c, const KvBatch& b, const KvAttn& a, void* ws,
                               int32_t* status, cudaStream_t stream, int num_sms) {
    (void)num_sms;
    const k12::Plans p = k12::plans_of(c, b, a);
    if ((p.few && !k12::fits(c, b, p.f)) || (p.chunk && !k12::fits(c, b, p.k))) return HBL_ERR_SHAPE;
    float* part = static_cast<float*>(ws);
    hbl_status st;
    if (p.chunk) {
        switch (c.D) {
            case 32: st = k14::launch_d32(c, b, a, p.k, part, status, stream); break;
            case 64: st = k14::launch_d64(c, b, a, p.k, part, status, stream); break;
            case 128: st = k14::launch_d128(c, b, a, p.k, part, status, stream); break;
            default: st = k14::launch_d256(c, b, a, p.k, part, status, stream); break;
        }
        if (st != HBL_OK) return st;
        st = k12::combine(c, b, a, p.k, part, stream);
        if (st != HBL_OK) return st;
        part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + k12::part_bytes(c, b, p.k));
    }
    if (p.few) {
        switch (c.D) {
            case 32: st = k13::launch_d32(c, b, a, p.f, part, status, stream); break;
            case 64: st = k13::launch_d64(c, b, a, p.f, part, status, stream); break;
            case 128: st = k13::launch_d128(c, b, a, p.f, part, status, stream); break;
            default: st = k13::launch_d256(c, b, a, p.f, part, status, stream); break;
        }
        if (st != HBL_OK) return st;
        return k12::combine(c, b, a, p.f, part, stream);
    }
    return HBL_OK;
}

}  // namespace hbl
