// mhc_norm_bwd_78.hip -- the post mix's gradient with the norm, 7 and 8 streams.
#include "mhc_norm_bwd.h"

namespace mhc {

void launch_post_norm_bwd_78(const PostNormBwd& p, int T, int S, int HQ, int KB, float eps,
                             float* part, int n, float* gate_part, hipStream_t st) {
  S == 7 ? launch_post_norm_bwd_s<7>(p, T, HQ, KB, eps, part, n, gate_part, st)
         : launch_post_norm_bwd_s<8>(p, T, HQ, KB, eps, part, n, gate_part, st);
}

}  // namespace mhc
