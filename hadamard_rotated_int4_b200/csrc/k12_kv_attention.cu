// k12_kv_attention.cu -- attention of new rows over the paged low-bit KV cache.
//
// For a row at position p and a query head over cached head h:
//   x_i = scale * log2(e) * (q . K_i),  O = sum_i 2^(x_i - m) V_i / sum_i 2^(x_i - m)
// in one pass over the visible positions with the running maximum m and sum.
// One warp per (row, query head), D/32 values a lane.
#include <cuda_bf16.h>
#include <math_constants.h>

#include "hbl_kv.cuh"

namespace hbl {
namespace k12 {

constexpr int kThreads = 256;

template <int D, int B>
__global__ void __launch_bounds__(kThreads) attention_kernel(KvCache c, KvBatch kb, KvAttn a,
                                                             int32_t* status) {
    constexpr int VPT = D / 32, ROW_BYTES = D * B / 8;
    const int lane = threadIdx.x & 31;
    const int64_t w = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5;
    if (w >= (int64_t)kb.rows * a.heads) return;
    const int t = (int)(w / a.heads), j = (int)(w % a.heads), h = j / a.group;
    const int b = kv_seq_of_row(kb, t);
    if (b >= kb.num_seqs) return;
    const KvSeq s = kv_seq(kb, c.page_size, b);
    if (s.bad || t - s.r0 >= a.max_rows) {
        if (lane == 0) report_status(status, HBL_ERR_INVALID_ARG);
    }
    if (t < s.r0 || t >= s.r1 || t - s.r0 >= a.max_rows) return;
    const int pos = s.len - (s.r1 - s.r0) + (t - s.r0);
    const int end = a.causal ? min(s.len, pos + 1) : s.len;
    const int begin = a.window > 0 ? max(0, pos - a.window + 1) : 0;
    float q[VPT], o[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        q[i] = __uint_as_float((uint32_t)a.q[t * a.q_row + j * a.q_head + 32 * i + lane] << 16);
        o[i] = 0.f;
    }
    float m = -CUDART_INF_F, l = 0.f;
    const float scale = a.scale * 1.4426950408889634f;
    auto code = [&](const uint8_t* row, int d) {
        const int bit = B * d;
        const uint8_t* p = row + bit / 8;
        uint32_t v = p[0];
        if (B == 3 && bit % 8 > 5) v |= (uint32_t)p[1] << 8;
        return (float)((int)((v >> (bit % 8)) & ((1u << B) - 1u)) - (1 << (B - 1)));
    };
    for (int i = begin; i < end; ++i) {
        const int pi = i / c.page_size;
        const int page = kv_page(kb, c.num_pages, b, pi);
        if (page < 0) {
            if (lane == 0) report_status(status, HBL_ERR_INVALID_ARG);
            continue;
        }
        const int64_t row = ((int64_t)page * c.heads + h) * c.page_size + (i - pi * c.page_size);
        float dot = 0.f;
#pragma unroll
        for (int k = 0; k < VPT; ++k)
            dot = __fmaf_rn(q[k], code(c.kc + row * ROW_BYTES, 32 * k + lane), dot);
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, k);
        const float x = dot * (c.ks[row] * scale), n = fmaxf(m, x);
        const float f = m == n ? 1.f : exp2f(m - n), p = exp2f(x - n), pv = p * c.vs[row];
        m = n;
        l = __fmaf_rn(l, f, p);
#pragma unroll
        for (int k = 0; k < VPT; ++k)
            o[k] = __fmaf_rn(o[k], f, pv * code(c.vc + row * ROW_BYTES, 32 * k + lane));
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int k = 0; k < VPT; ++k)
        a.o[t * a.o_row + j * a.o_head + 32 * k + lane] =
            __bfloat16_as_ushort(__float2bfloat16_rn(o[k] * inv));
    if (a.lse != nullptr && lane == 0)
        a.lse[(int64_t)t * a.heads + j] =
            l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -CUDART_INF_F;
}

}  // namespace k12

size_t kv_attention_workspace(const KvCache&, const KvBatch&, const KvAttn&) { return 0; }

hbl_status launch_kv_attention(const KvCache& c, const KvBatch& b, const KvAttn& a, void* ws,
                               int32_t* status, cudaStream_t stream, int num_sms) {
    (void)ws;
    (void)num_sms;
    return kv_dispatch(c.D, c.bits, [&](auto d, auto bits) {
        const int64_t ctas = ((int64_t)b.rows * a.heads + k12::kThreads / 32 - 1) / (k12::kThreads / 32);
        if (ctas > 0x7fffffffll) return HBL_ERR_SHAPE;
        k12::attention_kernel<decltype(d)::value, decltype(bits)::value>
            <<<(unsigned)ctas, k12::kThreads, 0, stream>>>(c, b, a, status);
        return cudaGetLastError() == cudaSuccess ? HBL_OK : HBL_ERR_CUDA;
    });
}

}  // namespace hbl
