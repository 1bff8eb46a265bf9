// k14_kv_chunk_d32.cu -- the chunk attention kernel for head size 32.
#include "k14_kv_chunk.cuh"

namespace hbl {
namespace k14 {
hbl_status launch_d32(const KvCache& c, const KvBatch& b, const KvAttn& a, const k12::Plan& pl,
                     float* part, int32_t* status, cudaStream_t stream) {
    return launch_d<32>(c, b, a, pl, part, status, stream);
}
}  // namespace k14
}  // namespace hbl
