// pa_shared_16.cu -- shared-prefix decode kernels for bf16 and fp16 caches.
#include "pa_shared_kernels.cuh"

namespace pa {
namespace shd {

KernelInfo pick_attend_16(int head_dim, int kv_dtype) {
  if (kv_dtype == PA_KV_F16) return head_dim == 64 ? attend_info<64, kKvF16>() : attend_info<128, kKvF16>();
  return head_dim == 64 ? attend_info<64, kKvBf16>() : attend_info<128, kKvBf16>();
}

}  // namespace shd
}  // namespace pa
