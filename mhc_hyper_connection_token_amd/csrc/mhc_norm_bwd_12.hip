// mhc_norm_bwd_12.hip -- the post mix's gradient with the norm, 1 and 2 streams.
#include "mhc_norm_bwd.h"

namespace mhc {

void launch_post_norm_bwd_12(const PostNormBwd& p, int T, int S, int HQ, int KB, float eps,
                             float* part, int n, float* gate_part, hipStream_t st) {
  S == 1 ? launch_post_norm_bwd_s<1>(p, T, HQ, KB, eps, part, n, gate_part, st)
         : launch_post_norm_bwd_s<2>(p, T, HQ, KB, eps, part, n, gate_part, st);
}

}  // namespace mhc
