// k5_kv_quant.cu -- per-head absmax quantiser of Q, K, V states (after RoPE)
// to unsigned `bits`-bit integers, for low-bit attention and the KV cache.
//
// BitNet v2 write-up (0755model.com), section "实验结果" (tables 2 and 3): the
// QKV states are quantised after RoPE, per head, with absmax, directly to
// unsigned integers and without calibration data; a 3-bit KV cache is
// reported.  The quantiser is the INT8 absmax quantiser of the activations
// taken to b bits and offset into the unsigned range:
//   Qp = 2^(b-1) - 1;  gamma = max|x|;  inv = Qp / (gamma + eps)  (one division)
//   q = clip(rhe(x * inv), -Qp-1, Qp);  u = q + 2^(b-1);  scale = gamma / Qp
// (inv = 0 when gamma + eps == 0, so a zero row gives u = 2^(b-1), scale 0).
// Each code rounds the exact product x * inv once (an fma with 1.5 * 2^23).
//
// Layout: a row of D codes is D*b/8 bytes; each group of 32 codes is 4*b bytes
// and code j of a group sits at bits [b*j, b*j + b) of the group read as a
// little-endian integer.
//
// Mapping: D/16 lanes per row, 16 values (two 16-byte loads) per lane, so a
// warp covers 32*16/D rows per step and a lane's 16 codes are 16*b contiguous
// bits; the per-step costs (the max over the row's lanes, the division, the
// scale) are shared by 16 values per lane.  For b = 3 lane pairs make one
// 12-byte group (one shuffle).  Memory-bound: 2*D bytes in, D*b/8 + 4 out per
// row; each warp keeps U steps of loads in flight.
#include <cuda_runtime.h>

#include "hbl_kv.cuh"

namespace hbl {
namespace k5 {

constexpr int kThreads = 256;
constexpr int U = 2;     // row steps per warp with their loads in flight together
constexpr int VPL = kKvVpl;  // values per lane

template <int D, int B>
__global__ void __launch_bounds__(kThreads) kv_quant_kernel(const uint16_t* __restrict__ X,
                                                            int64_t rows, float eps,
                                                            uint8_t* __restrict__ codes,
                                                            float* __restrict__ scales) {
    constexpr int LPR = D / VPL;     // lanes per row
    constexpr int RPW = 32 / LPR;    // rows per warp step
    constexpr int ROW_BYTES = D * B / 8;
    const int lane = threadIdx.x & 31;
    const int sub = lane / LPR, li = lane % LPR;
    const int64_t warp0 = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5;
    const int64_t nwarps = ((int64_t)gridDim.x * kThreads) >> 5;

    for (int64_t base = warp0 * (RPW * U); base < rows; base += nwarps * (RPW * U)) {
        uint4 raw[U][2];
        auto load = [&](int u, uint4 (&to)[2]) {
            const int64_t row = base + u * RPW + sub;
            const uint4* src = reinterpret_cast<const uint4*>(X + row * D + li * VPL);
            to[0] = row < rows ? src[0] : make_uint4(0, 0, 0, 0);
            to[1] = row < rows ? src[1] : make_uint4(0, 0, 0, 0);
        };
#pragma unroll
        for (int u = 0; u < U; ++u) load(u, raw[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = base + u * RPW + sub;
            KvHalf<B> h[2];
            bool over;
            const float scale = kv_quant16<D, B>(raw[u], eps, h, &over);
            if (over) {
                uint4 again[2];
                load(u, again);
                kv_ends16<B>(again, h);
            }
            const bool ok = row < rows;
            kv_store16<B>(codes + row * ROW_BYTES, li, h, ok);
            if (ok && li == 0) scales[row] = scale;
        }
    }
}

template <int D, int B>
static hbl_status launch_one(const uint16_t* X, int64_t rows, float eps, uint8_t* codes,
                             float* scales, cudaStream_t stream, int sms) {
    constexpr int RPW = 32 / (D / VPL);
    const int64_t per_cta = (int64_t)(kThreads / 32) * RPW * U;
    int64_t grid = (rows + per_cta - 1) / per_cta;
    const int64_t cap = (int64_t)sms * 8;
    if (grid > cap) grid = cap;
    kv_quant_kernel<D, B><<<(unsigned)grid, kThreads, 0, stream>>>(X, rows, eps, codes, scales);
    return cudaGetLastError() == cudaSuccess ? HBL_OK : HBL_ERR_CUDA;
}

template <int D>
static hbl_status by_bits(int bits, const uint16_t* X, int64_t rows, float eps, uint8_t* codes,
                          float* scales, cudaStream_t s, int sms) {
    switch (bits) {
        case 2: return launch_one<D, 2>(X, rows, eps, codes, scales, s, sms);
        case 3: return launch_one<D, 3>(X, rows, eps, codes, scales, s, sms);
        case 4: return launch_one<D, 4>(X, rows, eps, codes, scales, s, sms);
        case 8: return launch_one<D, 8>(X, rows, eps, codes, scales, s, sms);
        default: return HBL_ERR_INVALID_ARG;
    }
}

}  // namespace k5

hbl_status launch_kv_quant(const uint16_t* X, int64_t rows, int D, int bits, float eps,
                           uint8_t* codes, float* scales, cudaStream_t stream, int num_sms) {
    if (rows == 0) return HBL_OK;
    switch (D) {
        case 32: return k5::by_bits<32>(bits, X, rows, eps, codes, scales, stream, num_sms);
        case 64: return k5::by_bits<64>(bits, X, rows, eps, codes, scales, stream, num_sms);
        case 128: return k5::by_bits<128>(bits, X, rows, eps, codes, scales, stream, num_sms);
        case 256: return k5::by_bits<256>(bits, X, rows, eps, codes, scales, stream, num_sms);
        default: return HBL_ERR_SHAPE;
    }
}

}  // namespace hbl
