// mhc_norm_bwd_34.hip -- the post mix's gradient with the norm, 3 and 4 streams.
#include "mhc_norm_bwd.h"

namespace mhc {

void launch_post_norm_bwd_34(const PostNormBwd& p, int T, int S, int HQ, int KB, float eps,
                             float* part, int n, float* gate_part, hipStream_t st) {
  S == 3 ? launch_post_norm_bwd_s<3>(p, T, HQ, KB, eps, part, n, gate_part, st)
         : launch_post_norm_bwd_s<4>(p, T, HQ, KB, eps, part, n, gate_part, st);
}

}  // namespace mhc
