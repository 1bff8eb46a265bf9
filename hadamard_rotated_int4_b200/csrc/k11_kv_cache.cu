// k11_kv_cache.cu -- the paged low-bit KV cache: new K/V rows quantised into
// their pages, and rows dequantised out of them.
//
// One head row (one token's D values of one head) is coded as K5 codes it:
//   gamma = max|x|;  inv = Qp / (gamma + eps);  u = rhe(x * inv) + 2^(b-1);
//   scale = gamma / Qp;  value = (u - 2^(b-1)) * scale
// and stored at row (page * heads + head) * page_size + slot of the codes and
// scales, page = block_table[seq][pos / page_size], slot = pos % page_size.  A
// head's rows of one page are contiguous, so the attention that reads them
// streams whole pages of its head.
//
// Both kernels are bound by HBM at large batches, close behind by the instructions of
// coding and placing a row (three quarters of all issue slots), and by launch
// latency at one decoding step.  Measured, graph replay: 131071 rows of 8 heads of 128
// out of the 4-bit cache as bf16 107 us, 0.97 of the measured copy bandwidth; 8192
// tokens of 32 heads into the 3-bit cache 37.4 us, 0.66 of it; 64 tokens of 8 heads
// 2.8 us to write and 3.2 us to read, 1024 tokens of as many sequences 11.4 and 11.0
// (a token's search goes over 32 sequences at a time).  A warp takes one token and
// 1..kSteps steps of its 2 * heads head rows (K heads, then V heads; D/16 lanes a row, 16 values a lane): the
// token's sequence, position and page are found once per warp, by one round of
// loads and a ballot per 32 sequences instead of a chain of dependent loads.
#include "hbl_kv_codes.cuh"

namespace hbl {
namespace k11 {

constexpr int kThreads = 128;
constexpr int kSteps = 4;  // most steps of one warp task
// CTAs to an SM, by the registers that they leave a thread: 32 warps whose four
// steps of rows are all in flight, 48 that hold codes only.
constexpr int kWriteCtas = 8, kReadCtas = 12;

struct Task {
    int tasks_per_row;  // warp tasks of one token
    int per_task;       // head rows of one task
    int64_t tasks;
};

// A task's token; by a division of 32 bits where they do, a tenth of the instructions.
__device__ __forceinline__ int row_of(const Task& k, int64_t task) {
    if (k.tasks <= 0xffffffffll) return (int)((uint32_t)task / (uint32_t)k.tasks_per_row);
    return (int)(task / k.tasks_per_row);
}

// Where the token of this warp's task stands in the cache.
struct Place {
    int64_t base;  // (page * heads) * page_size + slot
    bool in_seq;   // the row belongs to a sequence of the batch
    bool ok;       // and has a place in a page of the pool
};
__device__ __forceinline__ Place place_of(const KvCache& c, const KvBatch& kb, int t,
                                          int32_t* status) {
    Place p;
    p.base = 0;
    p.in_seq = p.ok = false;
    bool bad = false;
    const KvRow r = kv_row(kb, c.page_size, t, &bad);
    if (bad) report_status(status, HBL_ERR_INVALID_ARG);
    p.in_seq = r.in_seq;
    if (r.in_seq && r.pos >= 0) {
        const int pi = r.pos / c.page_size;
        const int page = kv_page(kb, c.num_pages, r.b, pi);
        if (page >= 0) {
            p.base = (int64_t)page * c.heads * c.page_size + (r.pos - pi * c.page_size);
            p.ok = true;
        } else if ((threadIdx.x & 31) == 0) {
            report_status(status, HBL_ERR_INVALID_ARG);
        }
    }
    return p;
}

// The descriptors that the rows' own searches, 32 sequences at a time, may not come
// to, looked over by the first warp of the grid behind its own rows.
__device__ __forceinline__ void check_batch(const KvCache& c, const KvBatch& kb, int32_t* status) {
    if (blockIdx.x != 0 || threadIdx.x >= 32) return;
    for (int b = 32 + threadIdx.x; b < kb.num_seqs; b += 32)
        if (kv_seq(kb, c.page_size, b).bad) report_status(status, HBL_ERR_INVALID_ARG);
}

template <int D, int B>
__global__ void __launch_bounds__(kThreads, kWriteCtas) write_kernel(KvCache c, KvBatch kb, KvStates x,
                                                         float eps, Task k, int32_t* status) {
    constexpr int LPR = D / kKvVpl;
    constexpr int RPW = 32 / LPR;
    constexpr int ROW_BYTES = D * B / 8;
    const int lane = threadIdx.x & 31, sub = lane / LPR, li = lane % LPR;
    const int64_t warps = ((int64_t)gridDim.x * kThreads) >> 5;
    for (int64_t task = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5; task < k.tasks;
         task += warps) {
        const int t = row_of(k, task);
        const int first = (int)(task - (int64_t)t * k.tasks_per_row) * k.per_task;
        const int last = min(first + k.per_task, 2 * c.heads);
        uint4 raw[kSteps][2];
        const uint16_t* const k0 = x.k + (int64_t)t * x.k_row + li * kKvVpl;
        const uint16_t* const v0 =
            x.v + (int64_t)t * x.v_row - (int64_t)c.heads * x.v_head + li * kKvVpl;
        auto load = [&](int step, uint4 (&to)[2]) {
            const int r = first + step * RPW + sub;  // K heads, then V heads
            const bool isv = r >= c.heads;
            const uint4* s = reinterpret_cast<const uint4*>((isv ? v0 : k0) +
                                                            r * (isv ? x.v_head : x.k_head));
            to[0] = r < last ? s[0] : make_uint4(0, 0, 0, 0);
            to[1] = r < last ? s[1] : make_uint4(0, 0, 0, 0);
        };
#pragma unroll
        for (int step = 0; step < kSteps; ++step) load(step, raw[step]);  // while their place is found
        const Place p = place_of(c, kb, t, status);
#pragma unroll
        for (int step = 0; step < kSteps; ++step) {
            if (first + step * RPW >= last) break;
            const int r = first + step * RPW + sub;
            KvHalf<B> h[2];
            bool over;
            const float scale = kv_quant16<D, B>(raw[step], eps, h, &over);
            if (over) {
                uint4 again[2];
                load(step, again);
                kv_ends16<B>(again, h);
            }
            const bool ok = p.ok && r < last, isv = r >= c.heads;
            const int64_t row = p.base + (int64_t)(isv ? r - c.heads : r) * c.page_size;
            kv_store16<B>((isv ? c.vc : c.kc) + row * ROW_BYTES, li, h, ok);
            if (ok && li == 0) (isv ? c.vs : c.ks)[row] = scale;
        }
    }
    check_batch(c, kb, status);
}

// value = (u - 2^(B-1)) * scale, one fp32 rounding, then one to bf16.  The codes
// become fp16 pairs first, which hold them exactly: about one instruction a code,
// where taking each out of its bits and converting it takes three.
template <int B>
__device__ __forceinline__ void values16(const KvHalf<B> (&h)[2], float scale, float (&v)[16]) {
    constexpr int H = kKvHalfCodes<B>, W = 16 / (2 * H);
    uint32_t w[W];
    if constexpr (B == 8) {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = (uint32_t)(h[i / 2] >> (32 * (i % 2)));
    } else if constexpr (B == 4) {
        w[0] = h[0];
        w[1] = h[1];
    } else if constexpr (B == 3) {
        w[0] = kv_spread3(h[0]);
        w[1] = kv_spread3(h[1]);
    } else {
        w[0] = h[0] | (h[1] << 16);
    }
#pragma unroll
    for (int i = 0; i < W; ++i) {
        uint32_t pair[H];
        kv_widen_f16<B, H>(w[i], pair);
#pragma unroll
        for (int k = 0; k < H; ++k) {
            const float2 f = __half22float2(reinterpret_cast<const __half2&>(pair[k]));
            v[2 * H * i + k] = __fmul_rn(f.x, scale);
            v[2 * H * i + k + H] = __fmul_rn(f.y, scale);
        }
    }
}

template <int D, int B, bool F32>
__global__ void __launch_bounds__(kThreads, kReadCtas) read_kernel(KvCache c, KvBatch kb, void* k_out,
                                                        void* v_out, Task k, int32_t* status) {
    constexpr int LPR = D / kKvVpl;
    constexpr int RPW = 32 / LPR;
    constexpr int ROW_BYTES = D * B / 8;
    const int lane = threadIdx.x & 31, sub = lane / LPR, li = lane % LPR;
    const int64_t warps = ((int64_t)gridDim.x * kThreads) >> 5;
    for (int64_t task = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5; task < k.tasks;
         task += warps) {
        const int t = row_of(k, task);
        const int first = (int)(task - (int64_t)t * k.tasks_per_row) * k.per_task;
        const int last = min(first + k.per_task, 2 * c.heads);
        const Place p = place_of(c, kb, t, status);
        if (!p.in_seq) continue;  // left as it was
        KvHalf<B> h[kSteps][2];
        float scale[kSteps];
#pragma unroll
        for (int step = 0; step < kSteps; ++step) {  // every load in flight before the first use
            const int r = first + step * RPW + sub;
            const bool isv = r >= c.heads;
            h[step][0] = h[step][1] = 0;
            scale[step] = 0.f;
            if (r < last && p.ok) {
                const int64_t row = p.base + (int64_t)(isv ? r - c.heads : r) * c.page_size;
                kv_load16<B>((isv ? c.vc : c.kc) + row * ROW_BYTES, li, h[step]);
                scale[step] = (isv ? c.vs : c.ks)[row];
            }
        }
#pragma unroll
        for (int step = 0; step < kSteps; ++step) {
            if (first + step * RPW >= last) break;
            const int r = first + step * RPW + sub;
            const bool isv = r >= c.heads;
            float v[16];
            values16<B>(h[step], scale[step], v);
            uint32_t w[F32 ? 16 : 8];
            if constexpr (F32) {
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(v[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = f2_to_bf16x2(v[2 * i], v[2 * i + 1]);
            }
            // A lane's 16-byte pieces are the halves of whole 32-byte sectors.  Two lanes
            // trade halves, so that one store writes both halves of a sector: the even
            // lane's sector first, then the odd lane's.
            const bool odd = li & 1;
            uint4* const row = reinterpret_cast<uint4*>(
                (isv ? static_cast<uint8_t*>(v_out) : static_cast<uint8_t*>(k_out)) +
                ((int64_t)t * c.heads + (isv ? r - c.heads : r)) * D * (F32 ? 4 : 2));
            constexpr int kSectors = F32 ? 2 : 1;  // of a lane
#pragma unroll
            for (int k = 0; k < kSectors; ++k) {
                uint32_t mine[4], theirs[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t lo = w[8 * k + i], hi = w[8 * k + 4 + i];
                    mine[i] = odd ? hi : lo;
                    theirs[i] = __shfl_xor_sync(0xffffffffu, odd ? lo : hi, 1);
                }
                const int even_at = (li & ~1) * 2 * kSectors + 2 * k + (odd ? 1 : 0);
                const int odd_at = even_at + 2 * kSectors;
                if (r < last) {
                    // even lane: its own low half, then the odd lane's; odd lane: the even
                    // lane's high half, then its own
                    row[even_at] = odd ? make_uint4(theirs[0], theirs[1], theirs[2], theirs[3])
                                       : make_uint4(mine[0], mine[1], mine[2], mine[3]);
                    row[odd_at] = odd ? make_uint4(mine[0], mine[1], mine[2], mine[3])
                                      : make_uint4(theirs[0], theirs[1], theirs[2], theirs[3]);
                }
            }
        }
    }
    check_batch(c, kb, status);
}

// Few head rows in all: one step a warp, for the most warps in flight (64 tokens of 8
// heads: 3.0 us to write, 3.8 with four).  Many: kSteps steps, which share the search
// for the token's page (8192 tokens of 32 heads: 38 us, 70 with one).  Going on to a
// second or fourth set of steps for one token gains no more (37 to write, 39 to read).
template <int D>
static Task plan(const KvCache& c, const KvBatch& b, int num_sms, unsigned* grid) {
    constexpr int RPW = 32 / (D / kKvVpl);
    const int64_t head_rows = 2ll * c.heads;
    Task k;
    int steps = kSteps;
    while (steps > 1 && (int64_t)b.rows * ((head_rows + steps * RPW - 1) / (steps * RPW)) <
                            (int64_t)num_sms * 32)
        steps >>= 1;
    k.per_task = steps * RPW;
    k.tasks_per_row = (int)((head_rows + k.per_task - 1) / k.per_task);
    k.tasks = (int64_t)b.rows * k.tasks_per_row;
    const int64_t ctas = (k.tasks + kThreads / 32 - 1) / (kThreads / 32);
    *grid = (unsigned)(ctas < (int64_t)num_sms * 128 ? ctas : (int64_t)num_sms * 128);
    return k;
}

static hbl_status done() { return cudaGetLastError() == cudaSuccess ? HBL_OK : HBL_ERR_CUDA; }

template <int D, int B>
static hbl_status write_one(const KvCache& c, const KvBatch& b, const KvStates& x, float eps,
                            int32_t* status, cudaStream_t s, int sms) {
    unsigned grid;
    const Task k = plan<D>(c, b, sms, &grid);
    write_kernel<D, B><<<grid, kThreads, 0, s>>>(c, b, x, eps, k, status);
    return done();
}
template <int D, int B>
static hbl_status read_one(const KvCache& c, const KvBatch& b, void* ko, void* vo, bool fp32,
                           int32_t* status, cudaStream_t s, int sms) {
    unsigned grid;
    const Task k = plan<D>(c, b, sms, &grid);
    if (fp32)
        read_kernel<D, B, true><<<grid, kThreads, 0, s>>>(c, b, ko, vo, k, status);
    else
        read_kernel<D, B, false><<<grid, kThreads, 0, s>>>(c, b, ko, vo, k, status);
    return done();
}

}  // namespace k11

hbl_status launch_kv_cache_write(const KvCache& c, const KvBatch& b, const KvStates& x, float eps,
                                 int32_t* status, cudaStream_t stream, int num_sms) {
    return kv_dispatch(c.D, c.bits, [&](auto d, auto bits) {
        return k11::write_one<decltype(d)::value, decltype(bits)::value>(c, b, x, eps, status,
                                                                         stream, num_sms);
    });
}

hbl_status launch_kv_cache_read(const KvCache& c, const KvBatch& b, void* k_out, void* v_out,
                                bool fp32, int32_t* status, cudaStream_t stream, int num_sms) {
    return kv_dispatch(c.D, c.bits, [&](auto d, auto bits) {
        return k11::read_one<decltype(d)::value, decltype(bits)::value>(c, b, k_out, v_out, fp32,
                                                                        status, stream, num_sms);
    });
}

}  // namespace hbl
