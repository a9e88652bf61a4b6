// pkv_share_wide.cu -- the 128-row tiles of requests that share prefixes (pkv_tree_wide.cuh).
#include "pkv_tree_wide.cuh"

namespace pkv {

cudaError_t launch_shared_wide(const TcArgs& a, int64_t max_items, int num_sms, cudaStream_t st) {
  return a.p.D == 128 ? launch_items<Wide<128, true>>(tree_wide_kernel<128, true>, a, max_items, num_sms, st)
                      : launch_items<Wide<64, true>>(tree_wide_kernel<64, true>, a, max_items, num_sms, st);
}

}  // namespace pkv
