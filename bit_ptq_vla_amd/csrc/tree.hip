// Trees of drafted tokens, for gfx950: what their nodes see, and the path of
// them that sampled tokens confirm.
//
// A sequence's new tokens are the nodes; a node's parent is the index of an
// earlier one, anything else makes it a root.  A block takes a sequence, whose
// parents (and the child that each node's sampled token confirms) lie in LDS, so
// that a walk costs an LDS read a node: up the tree from every node at once, a
// lane to a node, for its mask words from the last to the first (parents come
// before their children, so a walk meets the bits in falling order), and down
// from node 0 by one lane.  The time is a launch and a chain of loads, walk and
// stores: a plan and an accepted path take 12 to 13 us for one tree of 16 nodes
// as for 64 of 256, two launches' 6.6 and what the calls cost on the host.

#include <hip/hip_runtime.h>

#include "kv_index.h"
#include "qlin_internal.h"

namespace qlin {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ int parent_of(const int32_t* parents, int64_t row0, int i) {
    const int p = parents[row0 + i];
    return p >= 0 && p < i ? p : -1;
}

__global__ __launch_bounds__(kThreads) void tree_plan_kernel(KvIndex ix, const int32_t* parents, uint32_t* mask,
                                                             int64_t mask_ld, int words, int32_t* positions) {
    __shared__ int16_t up[kMaxTreeNodes];
    const int b = blockIdx.x;
    const KvSeq s = kv_seq(ix, b);
    for (int i = threadIdx.x; i < s.n; i += kThreads) up[i] = static_cast<int16_t>(parent_of(parents, s.row0, i));
    __syncthreads();
    for (int i = threadIdx.x; i < s.n; i += kThreads) {
        uint32_t* row = mask + (s.row0 + i) * mask_ld;
        int at = i, depth = -1;
        for (int w = words - 1; w >= 0; --w) {
            uint32_t bits = 0;
            while (at >= 32 * w) {        // (at is -1 behind a root)
                bits |= 1u << (at - 32 * w);
                at = up[at];
                ++depth;
            }
            row[w] = bits;
        }
        positions[s.row0 + i] = s.first + depth;
    }
}

__global__ __launch_bounds__(kThreads) void tree_accept_kernel(KvIndex ix, const int32_t* parents, const int32_t* draft,
                                                               const int32_t* sampled, int32_t* path, int64_t path_ld,
                                                               int32_t* count, int32_t* token) {
    __shared__ int next[kMaxTreeNodes];      // the first confirmed child
    __shared__ int16_t taken[kMaxTreeNodes];
    __shared__ int length;
    const int b = blockIdx.x;
    const KvSeq s = kv_seq(ix, b);
    for (int i = threadIdx.x; i < s.n; i += kThreads) next[i] = kMaxTreeNodes;
    __syncthreads();
    for (int i = threadIdx.x; i < s.n; i += kThreads) {
        const int p = i > 0 ? parent_of(parents, s.row0, i) : -1;
        if (p >= 0 && draft[s.row0 + i] == sampled[s.row0 + p]) atomicMin(&next[p], i);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        int n = 0;
        for (int at = 0; at < s.n; at = next[at]) taken[n++] = static_cast<int16_t>(at);   // a child comes behind its parent
        length = n;
        count[b] = n;
        token[b] = n > 0 ? sampled[s.row0 + taken[n - 1]] : -1;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < ix.max_q; i += kThreads) path[b * path_ld + i] = i < length ? taken[i] : -1;
}

}  // namespace

hipError_t launch_tree_plan(const KvIndex& ix, const int32_t* parents, uint32_t* mask, int64_t mask_ld,
                            int32_t* positions, hipStream_t st) {
    tree_plan_kernel<<<dim3(static_cast<unsigned>(ix.batch)), kThreads, 0, st>>>(ix, parents, mask, mask_ld,
                                                                                 (ix.max_q + 31) / 32, positions);
    return hipGetLastError();
}

hipError_t launch_tree_accept(const KvIndex& ix, const int32_t* parents, const int32_t* draft, const int32_t* sampled,
                              int32_t* path, int64_t path_ld, int32_t* count, int32_t* token, hipStream_t st) {
    tree_accept_kernel<<<dim3(static_cast<unsigned>(ix.batch)), kThreads, 0, st>>>(ix, parents, draft, sampled, path,
                                                                                   path_ld, count, token);
    return hipGetLastError();
}

}  // namespace qlin
