// k14_kv_chunk_d64.cu -- the chunk attention kernel for head size 64.
#include "k14_kv_chunk.cuh"

namespace hbl {
namespace k14 {
hbl_status launch_d64(const KvCache& c, const KvBatch& b, const KvAttn& a, const k12::Plan& pl,
                     float* part, int32_t* status, cudaStream_t stream) {
    return launch_d<64>(c, b, a, pl, part, status, stream);
}
}  // namespace k14
}  // namespace hbl
