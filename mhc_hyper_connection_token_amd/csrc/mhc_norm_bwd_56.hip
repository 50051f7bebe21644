// mhc_norm_bwd_56.hip -- the post mix's gradient with the norm, 5 and 6 streams.
#include "mhc_norm_bwd.h"

namespace mhc {

void launch_post_norm_bwd_56(const PostNormBwd& p, int T, int S, int HQ, int KB, float eps,
                             float* part, int n, float* gate_part, hipStream_t st) {
  S == 5 ? launch_post_norm_bwd_s<5>(p, T, HQ, KB, eps, part, n, gate_part, st)
         : launch_post_norm_bwd_s<6>(p, T, HQ, KB, eps, part, n, gate_part, st);
}

}  // namespace mhc
