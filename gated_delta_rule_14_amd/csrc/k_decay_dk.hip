// The walk of k_decay.hpp that makes dk (reversed, state transposed, sums for dg).
#include "k_decay.hpp"

namespace gdn {

hipError_t launch_walk_dk(const DecayWalk& p, int K, int V, bool bf) {
    return launch_walk_of<true, true, 1, false>(p, K, V, bf);
}

}  // namespace gdn
