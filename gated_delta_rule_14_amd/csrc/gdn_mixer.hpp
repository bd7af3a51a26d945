// Internal launcher interface of the token mixers next to the delta rule
// (linear attention with a decay per head, append to a paged cache, attention
// of one token over it) between gdn_mixer_api.hip and their kernels.  Not part
// of the public ABI.
#pragma once

#include "gdn_layer.hpp"

namespace gdn {

// Rows of a tensor: element (token, head, d) is at p + token * ts + (head / div) * hs + d.
struct HeadRows {
    const void* p = nullptr;
    int64_t ts = 0, hs = 0;
    int div = 1;                  // state heads that share one of its heads
};

// One walk over the chunks of every segment (k_decay.hpp):
//   out_i = in_scale din_i a_i S + pair_scale sum_j gamma_ij (a_i b_j) c_j,
//   S <- dec S + up_scale sum_j dout_j b_j c_j^T
// with c the columns of S that the waves own.
struct DecayWalk {
    SeqMap map;                   // segments; sequences of up to map.tile tokens have none
    int64_t tiles = 0, singles = 0;   // workgroups for segments, then for whole sequences
    HeadRows a, b, c, x;          // x: what the output is multiplied with for dg
    const float* g = nullptr;     // natural-log gates, token stride gs (0: one for each head)
    int64_t gs = 0;
    float in_scale = 1.f, pair_scale = 1.f, up_scale = 1.f;
    const float* tile_state = nullptr;   // [tiles][H][K][V] states entering the segments
    int chain = 0;                       //   or, of sequences of up to `chain` segments, these alone
    const float* seq_state = nullptr;    // [N][H][K][V] entering whole sequences, or nullptr
    float* seq_out = nullptr;     // [N][H][K][V] states leaving the sequences, or nullptr
    // the gradients behind segments and whole sequences, and their products with the state that
    // leaves the chunk before the last one, decayed to the end: [tiles + singles][H]
    const float *tile_end = nullptr, *seq_end = nullptr;
    float* ends = nullptr;
    void* out = nullptr;          // [tokens][H][DC], element type
    float* out32 = nullptr;       // or in 32 bits
    float* dots = nullptr;        // [H][tokens]
    float *local = nullptr, *dec = nullptr;   // states of the segments alone [tiles][H][K][V], [tiles][H]
    int64_t H = 0, tokens = 0;
    int share = 1;                // state heads to a head of q and k
    hipStream_t stream = nullptr;
};
// the forward: the output, or (local) the segments' own states
hipError_t launch_decay_walk(const DecayWalk& w, bool local, int K, int V, bool bf16);
// dq, dk and dv, walks of one map
hipError_t launch_decay_grad(const DecayWalk& q, const DecayWalk& k, const DecayWalk& v, int K, int V, bool bf16);
// the segments alone for the gradients: f forward over (v, k), r from the end over (do, q)
hipError_t launch_decay_local2(const DecayWalk& f, const DecayWalk& r, int K, int V, bool bf16);

// Entering states of the segments out of their own, in place.
struct DecayJoin {
    SeqMap map;
    int64_t tiles;
    float* state;                 // [tiles][H][K][V]
    const float* dec;             // [tiles][H]
    const float* first;           // [N][H][K][V] or nullptr
    int64_t H, KV;
    int V;                        // with own_order the states' elements are in the forward walk's
    bool own_order;               //   order, but those of `first`, which are [K][V]
    bool rev;                     // from the last segment to the first
    int chain;                    // sequences of up to so many segments are left to the walk
    hipStream_t stream;
};
hipError_t launch_decay_join(const DecayJoin& a, const DecayJoin* b = nullptr);   // b: another one of its sizes

// dg out of the walks' dots: its running sum from each segment's end.
struct DecayGate {
    SeqMap map;
    int64_t tiles, singles;
    const float *dq, *dk;         // [H][tokens]
    const float* ends;            // [tiles + singles][H]
    const float* g;
    int64_t gs;
    float* dg;                    // [tokens][H]
    float* part;                  // or the segments' sums of it [tiles + singles][H]
    int64_t H, tokens;
    hipStream_t stream;
};
hipError_t launch_decay_gate(const DecayGate& a);

struct DecayStep {
    HeadRows q, k, v;             // rows are sequences
    const float* g;
    int64_t gs;
    float* state;
    void* o;
    float scale;
    int64_t N, H;
    int K, V;
    bool bf16;
    hipStream_t stream;
};
hipError_t launch_decay_step(const DecayStep& a);

// A cache of pages: element (page, slot, head, d) is at p + page * ps + slot * ts + head * hs + d.
struct Pages {
    void* p = nullptr;
    int64_t ps = 0, ts = 0, hs = 0;
};

struct PagedAppend {
    QkLaunch qk;                  // q, k and their options; qo: the rotated q (q may be nullptr); positions may be nullptr
    const void* v;
    int64_t vs, vhs;              // token and head strides of v
    Pages kc, vc;
    const int32_t* table;         // [N][M] pages of each sequence
    const int64_t* lens;          // [N] tokens that the cache holds
    const int64_t* cu;            // [N + 1] or nullptr: qk.T tokens to a sequence
    int64_t N, M, pages;
    int64_t page;                 // tokens of a page
};
hipError_t launch_paged_append(const PagedAppend& a);

struct PagedAttn {
    const void* q;
    int64_t qs, qhs;              // sequence and head strides
    Pages kc, vc;
    const int32_t* table;
    const int64_t* lens;          // [N] tokens to attend to
    int64_t N, M, pages, page, window;
    int Hq, Hk, D;
    float scale;                  // of the scores, times log2(e)
    void* o;                      // [N][Hq][D]
    int64_t share = 1;            // pieces that all sequences together are cut into (each at least one)
    float *part = nullptr, *ml = nullptr;   // [share + N][Hq][D], [share + N][Hq][2]
    bool bf16;
    hipStream_t stream;
};
int64_t paged_attn_share(int64_t Hq, int64_t Hk);
hipError_t launch_paged_attn(const PagedAttn& a);

}  // namespace gdn
