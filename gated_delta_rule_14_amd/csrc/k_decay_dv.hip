// The walk of k_decay.hpp that makes dv and dh0 (reversed).
#include "k_decay.hpp"

namespace gdn {

hipError_t launch_walk_dv(const DecayWalk& p, int K, int V, bool bf) {
    return launch_walk_of<true, false, 0, false>(p, K, V, bf);
}

}  // namespace gdn
