// The walks of k_decay.hpp that make the gradients: dq (state transposed, sums for
// dg), dk (from the end, state transposed, sums for dg), dv and dh0 (from the end).
//
// They need nothing of each other, so one launch runs all three, the workgroups of
// a segment's head next to each other on one XCD: dk and dv read the same rows at
// about the same time, and no walk's end leaves the chip half idle (2 x 8192 tokens
// of 16 heads of 128: 257 us, as three launches 12 us more; 300 tokens of 4 heads, the
// whole backward 29 us, as three launches and with longer segments 64).
#include "k_decay.hpp"

namespace gdn {

template <typename T, int K, int V>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 2 : 1) void decay_grad_kernel(DecayWalk q, DecayWalk k, DecayWalk v) {
    typedef DecayBody<T, V, K, false, true, 2, false> Q;
    typedef DecayBody<T, V, K, true, true, 1, false> D;
    typedef DecayBody<T, K, V, true, false, 0, false> N;
    __shared__ union Any {
        typename Q::Shared q;
        typename D::Shared k;
        typename N::Shared v;
        __device__ Any() {}
    } s;
    const unsigned slot = blockIdx.x >> 3, which = slot % 3, block = slot / 3 * 8 + (blockIdx.x & 7);
    if (which == 0) Q::run(q, block, s.q);
    else if (which == 1) D::run(k, block, s.k);
    else N::run(v, block, s.v);
}

template <typename T, int K, int V>
static hipError_t grad_of(const DecayWalk& q, const DecayWalk& k, const DecayWalk& v) {
    const unsigned blocks = walk_blocks(q, false);
    if (blocks == 0) return hipSuccess;
    hipLaunchKernelGGL((decay_grad_kernel<T, K, V>), dim3(3 * blocks), dim3(256), 0, q.stream, q, k, v);
    return hipGetLastError();
}

hipError_t launch_decay_grad(const DecayWalk& q, const DecayWalk& k, const DecayWalk& v, int K, int V, bool bf) {
    if (K == 64 && V == 64) return bf ? grad_of<bf16, 64, 64>(q, k, v) : grad_of<float, 64, 64>(q, k, v);
    if (K == 64 && V == 128) return bf ? grad_of<bf16, 64, 128>(q, k, v) : grad_of<float, 64, 128>(q, k, v);
    if (K == 128 && V == 64) return bf ? grad_of<bf16, 128, 64>(q, k, v) : grad_of<float, 128, 64>(q, k, v);
    if (K == 128 && V == 128) return bf ? grad_of<bf16, 128, 128>(q, k, v) : grad_of<float, 128, 128>(q, k, v);
    return hipErrorInvalidValue;
}

}  // namespace gdn
