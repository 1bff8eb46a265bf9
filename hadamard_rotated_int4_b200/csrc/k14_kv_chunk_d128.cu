// k14_kv_chunk_d128.cu -- the chunk attention kernel for head size 128.
#include "k14_kv_chunk.cuh"

namespace hbl {
namespace k14 {
hbl_status launch_d128(const KvCache& c, const KvBatch& b, const KvAttn& a, const k12::Plan& pl,
                     float* part, int32_t* status, cudaStream_t stream) {
    return launch_d<128>(c, b, a, pl, part, status, stream);
}
}  // namespace k14
}  // namespace hbl
