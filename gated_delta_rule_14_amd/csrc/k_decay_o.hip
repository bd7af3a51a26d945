// The walk of k_decay.hpp that makes the output.
#include "k_decay.hpp"

namespace gdn {

hipError_t launch_walk_o(const DecayWalk& p, int K, int V, bool bf) {
    return launch_walk_of<false, false, 0, false>(p, K, V, bf);
}

}  // namespace gdn
