// pa_shared_8.cu -- shared-prefix decode kernels for E4M3 and E5M2 caches.
#include "pa_shared_kernels.cuh"

namespace pa {
namespace shd {

KernelInfo pick_attend_8(int head_dim, int kv_dtype) {
  if (kv_dtype == PA_KV_FP8_E5M2) return head_dim == 64 ? attend_info<64, kKvE5M2>() : attend_info<128, kKvE5M2>();
  return head_dim == 64 ? attend_info<64, kKvFp8>() : attend_info<128, kKvFp8>();
}

}  // namespace shd
}  // namespace pa
