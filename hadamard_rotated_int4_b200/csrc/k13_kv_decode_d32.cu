// k13_kv_decode_d32.cu -- the few-rows attention kernel for head size 32.
#include "k13_kv_decode.cuh"

namespace hbl {
namespace k13 {
hbl_status launch_d32(const KvCache& c, const KvBatch& b, const KvAttn& a, const k12::Plan& pl,
                     float* part, int32_t* status, cudaStream_t stream) {
    return launch_d<32>(c, b, a, pl, part, status, stream);
}
}  // namespace k13
}  // namespace hbl
