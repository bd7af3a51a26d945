// The walk of k_decay.hpp that makes dq (state transposed, sums for dg).
#include "k_decay.hpp"

namespace gdn {

hipError_t launch_walk_dq(const DecayWalk& p, int K, int V, bool bf) {
    return launch_walk_of<false, true, 2, false>(p, K, V, bf);
}

}  // namespace gdn
