// k12_kv_attention.cu -- attention over the paged low-bit cache: the launch plan
// and the joining of ranges of positions.
#include "k12_kv_attention.cuh"

namespace hbl {
namespace k12 {

// Joins `count` parts of a head row: O = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s;
// D/4 threads (four values each) to a part, 4 * kThreads / D parts at once, four
// loads of each thread in flight.  Part 0 lies at src0, part k > 0 at src + k * next.
constexpr int kThreads = 128;

template <int D>
__device__ __forceinline__ void join_row(const KvAttn& a, const Rows& s, int h, int row, int count,
                                         const float* src0, const float* src, int64_t next) {
    constexpr int T = D / 4, G = kThreads / T;  // threads of a part, parts at once
    constexpr int U = 4;
    __shared__ float4 sy[kThreads];
    __shared__ float sl[G];
    const int t = threadIdx.x % T, g = threadIdx.x / T;
    auto part_of = [&](int k) { return k == 0 ? src0 : src + k * next; };
    float M = -CUDART_INF_F;  // every warp for itself
    for (int k = threadIdx.x & 31; k < count; k += 32) M = fmaxf(M, part_of(k)[D]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float L = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = g; k < count; k += G * U) {
        float4 v[U];
        float2 ml[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool in = k + u * G < count;
            const float* p = part_of(in ? k + u * G : k);
            v[u] = reinterpret_cast<const float4*>(p)[t];
            ml[u] = *reinterpret_cast<const float2*>(p + D);
            if (!in) ml[u].x = -CUDART_INF_F;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float f = ml[u].x == -CUDART_INF_F ? 0.f : exp2f(ml[u].x - M);
            L = __fmaf_rn(ml[u].y, f, L);
            y.x = __fmaf_rn(v[u].x, f, y.x);
            y.y = __fmaf_rn(v[u].y, f, y.y);
            y.z = __fmaf_rn(v[u].z, f, y.z);
            y.w = __fmaf_rn(v[u].w, f, y.w);
        }
    }
    sy[threadIdx.x] = y;
    if (t == 0) sl[g] = L;
    __syncthreads();
    if (g != 0) return;
    const int most = min(count, G);
    for (int k = 1; k < most; ++k) {
        const float4 z = sy[k * T + t];
        L += sl[k];
        y.x += z.x;
        y.y += z.y;
        y.z += z.z;
        y.w += z.w;
    }
    store_row4(a, s, h, row, 4 * t, y, M, L);
}

// Few rows: CTA (i, r) joins row r of the one head of an item that begins in piece
// i of the line and goes on past it (all others were stored by the kernel that
// computed them).
template <int D>
__global__ void __launch_bounds__(kThreads) join_pieces_kernel(KvCache c, KvBatch kb, KvAttn a,
                                                               Plan pl, float* part) {
    const Line line = line_of<kThreads, true>(pl, c, kb, a, blockIdx.x, nullptr);
    Item im = {};
    int h = 0, count = 0, row = 0;
    if (line.at < line.total) {
        im = item_of(pl, c, kb, a, line.item);
        h = (line.at - line.before) / im.units;
        const int first = line.before + h * im.units, last = first + im.units - 1;
        row = line.item % pl.row_blocks * pl.block_rows + (int)blockIdx.y;
        if (first >= (int)blockIdx.x * line.per && last > line.at && row < im.nr)
            count = last / line.per - (int)blockIdx.x + 1;
    }
    // every thread waits: the grid must not end before the one it depends on
    pdl_wait();
    if (count > 1)
        join_row<D>(a, im.s, h, row, count,
                    slot_of(part, pl, D, blockIdx.x, 1) + blockIdx.y * (D + 4),
                    slot_of(part, pl, D, blockIdx.x, 0) + blockIdx.y * (D + 4),
                    2 * pl.block_rows * (D + 4));
}

// Chunks: one CTA to a packed row and query head, whose ranges of positions it joins.
template <int D>
__global__ void __launch_bounds__(kThreads) join_ranges_kernel(KvCache c, KvBatch kb, KvAttn a,
                                                               Plan pl, const float* part) {
    const int t = (int)blockIdx.x, head = (int)blockIdx.y, h = head / a.group;
    int count = 0, row = 0;
    bool bad = false;
    const KvRow q = kv_row(kb, c.page_size, t, &bad);
    Rows s = {};
    if (q.in_seq) {
        s = rows_of(kb, c.page_size, a, q.b);
        const int nr = s.n * a.group;
        row = (t - s.row0) * a.group + head - h * a.group;
        const int r0 = row / pl.block_rows * pl.block_rows;
        if (row < nr && nr >= pl.min_rows && nr <= pl.max_rows)
            count = split_of(pl, range_of(a, s, r0, min(nr, r0 + pl.block_rows) - 1), 0).count;
    }
    pdl_wait();
    if (count <= 1) return;
    const float* src = part + part_index(kb, a, 0, t, head) * (D + 4);
    join_row<D>(a, s, h, row, count, src, src, (int64_t)kb.rows * a.heads * (D + 4));
}

static int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// SMs that the plans count on (the workspace must not depend on the device).
constexpr int kSizingSms = 148;
// Row blocks that see at most this many positions, by the block table's width and the
// window (a wider table counts as long, whatever the lengths in it), are not split.  Not splitting saves
// a launch (22 -> 17 us a call, host included), and on the GPU, 8 cached heads of 128
// at 4 bits, one sequence of 517: 9.5 against 11.4 us split, 8 of 1000: 11.5 / 14.0,
// 256 of 400: 43 / 71; one of 1000 takes 11.0 / 8.5, 64 of 1000: 30.9 / 29.4.  (With V's
// scales looked over, the first is 10.1 now, under a table of 2048 pages 12.8.)
constexpr int kWhole = 1024;
// Sequences with at most this many head rows go to the few-rows kernel.  16 sequences
// of 4000, 4 query heads to each of 8 cached ones: 32 head rows take 61 us there and
// 87.5 us in chunks, 48 take 83.5 and 87.9, 64 take 101.5 and 88.3.  (Measured at D = 128
// alone; other head sizes go by it.)
constexpr int kFewRows = 32;

// Round-up reciprocal of the page size: exact for x < 2^31.
static void set_page(Plan* p, int page_size) {
    uint32_t l = 0;
    while ((1ull << l) < (uint32_t)page_size) ++l;
    p->seg_shift = page_size % 64 == 0 ? 6 : page_size % 32 == 0 ? 5 : 4;
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

// Few rows: blocks of 8 head rows, or 16 where there are more than 8 (16 sequences of
// 4000 with 16 head rows each: 42 us, in blocks of 8 46.5; with 32: 61 and 76); as
// many CTAs as run at once, so that all work is one wave of equal pieces.
static Plan few_plan(const KvCache& c, const KvBatch& b, const KvAttn& a, int64_t rows) {
    Plan p = {};
    p.block_rows = c.D <= 128 && rows > 8 ? 16 : 8;
    p.row_blocks = (int)ceil_div(rows, p.block_rows);
    p.min_rows = 0;
    p.max_rows = (int)rows;
    p.ctas = kSizingSms * (p.block_rows == 8 && c.D <= 128 ? 3 : 2);
    // (one sequence of 2000: 9.3 us, 12.4 with pieces of one unit, 12.9 with sixteen)
    p.min_units = 4;
    // the whole line stays below 2^31 units
    const int64_t longest = (int64_t)b.pages_per_seq * c.page_size;
    const int64_t items = (int64_t)b.num_seqs * p.row_blocks * c.heads;
    p.unit = 64;
    // where no block can see many positions, one unit holds them all: nothing is
    // split, and nothing has to be joined
    const int64_t seen = a.window > 0 && (int64_t)a.window + a.max_rows < longest
                             ? (int64_t)a.window + a.max_rows
                             : longest;
    if (seen <= kWhole) {
        p.unit = kWhole + 64;  // a block begins at a multiple of 64
        p.min_units = 1;
        p.whole = true;
    }
    while (p.unit < (1 << 30) && items * (longest / p.unit + 2) > 0x7fffffffll) p.unit *= 2;
    // no more CTAs than the block table has room for pieces
    const int64_t most = ceil_div(items * (longest / p.unit + 2), p.min_units);
    if (most < p.ctas) p.ctas = (int)most;
    set_page(&p, c.page_size);
    return p;
}

// Chunks: 256 head rows a CTA (128 at D = 256), the grid as large as packed rows can
// fill; ranges only where the row blocks leave SMs without work, of 256 positions at
// least (64 rows of one sequence of 4000: 27.3 us; 32.3 with 512, 44.2 with 1024).
static Plan chunk_plan(const KvCache& c, const KvBatch& b, const KvAttn& a, int min_rows) {
    Plan p = {};
    p.block_rows = c.D <= 128 ? 256 : 128;
    p.min_rows = min_rows > 1 ? min_rows : 1;
    p.max_rows = 0x7fffffff;
    // every block but a sequence's last is full, and a sequence has min_rows at least
    const int64_t rows = (int64_t)b.rows * a.group;
    int64_t seqs = rows / p.min_rows;
    if (seqs > b.num_seqs) seqs = b.num_seqs;
    int64_t blocks = rows / p.block_rows + seqs;
    const int64_t most = b.num_seqs * ceil_div((int64_t)a.max_rows * a.group, p.block_rows);
    if (blocks > most) blocks = most;
    p.row_blocks = (int)(blocks < 0x7fffffff ? blocks : 0x7fffffff);
    const int64_t span = span_of(a, a.max_rows);
    const int64_t n = blocks > 0 ? kSizingSms / (blocks * c.heads) : 0;
    const int64_t q = n <= 1 ? span : ceil_div(span, n);
    set_splits(&p, span, q < 256 ? 256 : q);
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
static size_t part_bytes(const KvCache& c, const KvBatch& b, const KvAttn& a, const Plan& p) {
    if (p.whole) return 0;
    if (p.ctas > 0) return (size_t)p.ctas * 2 * p.block_rows * (c.D + 4) * sizeof(float);
    if (p.splits == 1) return 0;
    return (size_t)p.splits * b.rows * a.heads * (c.D + 4) * sizeof(float);
}
// Grids, and the few-rows kernel's line of units, fit 31 bits.
static bool fits(const KvCache& c, const KvBatch& b, const Plan& p) {
    const int64_t items = (int64_t)b.num_seqs * p.row_blocks;
    if (p.ctas > 0)
        return items <= 0x7fffffffll &&
               items * c.heads * ((int64_t)b.pages_per_seq * c.page_size / p.unit + 2) <=
                   0x7fffffffll;
    return (int64_t)p.row_blocks * p.splits * c.heads <= 0x7fffffffll;
}

template <int D>
static hbl_status combine_d(const KvCache& c, const KvBatch& b, const KvAttn& a, const Plan& p,
                            float* part, cudaStream_t stream) {
    if (p.ctas > 0)
        return launch_pdl(
            join_pieces_kernel<D>,
            dim3((unsigned)p.ctas, (unsigned)(p.max_rows < p.block_rows ? p.max_rows : p.block_rows)),
            dim3(kThreads), 0, stream, c, b, a, p, part);
    return launch_pdl(join_ranges_kernel<D>, dim3((unsigned)b.rows, (unsigned)a.heads),
                      dim3(kThreads), 0, stream, c, b, a, p, part);
}
static hbl_status combine(const KvCache& c, const KvBatch& b, const KvAttn& a, const Plan& p,
                          float* part, cudaStream_t stream) {
    if (p.whole || (p.ctas == 0 && p.splits == 1)) return HBL_OK;
    switch (c.D) {
        case 32: return combine_d<32>(c, b, a, p, part, stream);
        case 64: return combine_d<64>(c, b, a, p, part, stream);
        case 128: return combine_d<128>(c, b, a, p, part, stream);
        default: return combine_d<256>(c, b, a, p, part, stream);
    }
}

}  // namespace k12

size_t kv_attention_workspace(const KvCache& c, const KvBatch& b, const KvAttn& a) {
    const k12::Plans p = k12::plans_of(c, b, a);
    return (p.few ? k12::part_bytes(c, b, a, p.f) : 0) + (p.chunk ? k12::part_bytes(c, b, a, p.k) : 0);
}

hbl_status launch_kv_attention(const KvCache& c, const KvBatch& b, const KvAttn& a, void* ws,
                               int32_t* status, cudaStream_t stream) {
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
        part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + k12::part_bytes(c, b, a, p.k));
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
