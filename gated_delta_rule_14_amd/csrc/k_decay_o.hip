// The forward walks of k_decay.hpp: the output, and the segments' own states.
#include "k_decay.hpp"

namespace gdn {

template <typename T, int K, int V, bool LOCAL>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? (LOCAL ? 3 : 2) : 1) void decay_walk_kernel(DecayWalk p) {
    typedef DecayBody<T, K, V, false, false, 0, LOCAL> B;
    __shared__ typename B::Shared s;
    B::run(p, blockIdx.x, s);
}

template <typename T, int K, int V>
static hipError_t walk_of(const DecayWalk& p, bool local) {
    const unsigned blocks = walk_blocks(p, local);
    if (blocks == 0) return hipSuccess;
    if (local) hipLaunchKernelGGL((decay_walk_kernel<T, K, V, true>), dim3(blocks), dim3(256), 0, p.stream, p);
    else hipLaunchKernelGGL((decay_walk_kernel<T, K, V, false>), dim3(blocks), dim3(256), 0, p.stream, p);
    return hipGetLastError();
}

hipError_t launch_decay_walk(const DecayWalk& p, bool local, int K, int V, bool bf) {
    if (K == 64 && V == 64) return bf ? walk_of<bf16, 64, 64>(p, local) : walk_of<float, 64, 64>(p, local);
    if (K == 64 && V == 128) return bf ? walk_of<bf16, 64, 128>(p, local) : walk_of<float, 64, 128>(p, local);
    if (K == 128 && V == 64) return bf ? walk_of<bf16, 128, 64>(p, local) : walk_of<float, 128, 64>(p, local);
    if (K == 128 && V == 128) return bf ? walk_of<bf16, 128, 128>(p, local) : walk_of<float, 128, 128>(p, local);
    return hipErrorInvalidValue;
}

}  // namespace gdn
