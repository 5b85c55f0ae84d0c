// tree.cuh -- parameter block and device helpers of the drafted-tree kernels
// (tree.cu: attention of the nodes; tree_commit.cu: the accepted branch).
#pragma once

#include "rat_internal.cuh"

namespace rat {

// CTAs of tree_tc.cu, one an SM, at most
constexpr int kTreeTcCtas = 148;

// Nodes of one entry's tree, at most: a branch fits in one 64-bit mask.
constexpr int kTreeMaxNodes = 64;

// What the plan says of one head: in one place, as the first read of a kernel
// parameter's line by an SM takes as long as one of global memory.
struct TreeHead {
    int dil, win;
    int slab;        // ceil(cap / dil)
    int nsplit;      // pieces of one dilated set, at most
    int wsplit;      // pieces of the window's held rows (>= 1)
    int slab_ctas;   // CTAs that share the head's (set, piece) items
    int cta0;        // first CTA of the head within an entry
    int slot0;       // first partial slot
    int recur;
    int fused;       // one item has all the keys and writes the result itself
    int tc;          // place in tc_head with even shares, else -1
};

struct TreeParams {
    const void *q, *k, *v, *g;   // [B,N,H,d]
    const int *parent;           // device [B,N]
    const float *state[2];       // [B,H,d] fp32, read only
    const void *cache[2];        // [B,H,R,d] or the pools, read only
    const int *pos;              // device [B]
    void *o;                     // [B,N,H,d]
    float *lse;                  // [B,H,N] or null
    void *node_rows;             // [B][H][2][N][d] augmented rows of the nodes (cfg dtype)
    float *part;                 // [B][slots_per_b][N][d] unnormalised accumulators
    float2 *ml;                  // [B][slots_per_b][N] (max, sum); sum < 0: a page was not valid
    int *info;                   // [B][H][N] pieces of the node's dilated set; -1: absent, or entry skipped; -2: done
    long long cache_R;
    int cap, B, N, H, d;
    int grid, dedupe, sep;       // as in DecodeParams
    const int *page_table;
    int page_rows, pps, num_pages;
    float scale_log2;
    int ctas_per_b, slots_per_b;
    int ctas_per_head;           // when all heads have as many, else 0
    TreeHead head[kMaxHeads];
    // heads whose held rows tree_tc.cu takes (slab_ctas is 0): by pieces, as the other
    // heads' are, or (tc_even) in even shares: its CTA c then has the partial of pair
    // q = b * n_tc + i (i: place in tc_head) in slot tc_slot0 + q + c
    int n_tc, tc_same, tc_even;      // tc_same: they all have one dilation
    unsigned char tc_head[kMaxHeads];
    int tc_items_per_b;              // pieces of an entry, and the first of a head
    int tc_item0[kMaxHeads];
    int tc_slot0;
    int2 *tc_range;                  // [B * n_tc] first and last CTA of a pair with held rows
    WsHeader *hdr;
};

// The shape of one entry's tree, in shared memory.
struct TreeInfo {
    unsigned long long anc[kTreeMaxNodes];  // branch of node i, itself included (0: absent)
    unsigned long long far;                 // tree_masks()
    int jump[kTreeMaxNodes];
    signed char depth[kTreeMaxNodes];       // -1: absent
    int max_depth;                          // -1: no node
    int valid;                              // parents and position in range
};

// Depths and branches from the parents (one warp).  A node's branch is its
// parent's and itself; pointer doubling finds it in log2(depth) rounds.
// parent[i] is in [-1, i), or -2 for an absent node, which has no children.
__device__ __forceinline__ void tree_analyse(TreeInfo &ti, const int *parent, int N, int pos, int cap) {
    const int lane = threadIdx.x & 31;
    int par[2];
    bool ok = pos >= 0 && pos <= cap;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int i = lane + 32 * u;
        par[u] = i < N ? parent[i] : -2;
        ok = ok && par[u] >= -2 && par[u] < i;
        ti.jump[i] = par[u];
    }
    ok = __all_sync(0xffffffffu, ok);
    __syncwarp();
    if (ok) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
            if (par[u] >= 0) ok = ok && ti.jump[par[u]] != -2;
        ok = __all_sync(0xffffffffu, ok);
    }
    int dmax = -1;
    if (ok) {
        unsigned long long anc[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int i = lane + 32 * u;
            anc[u] = par[u] == -2 ? 0ull : 1ull << i;
            ti.anc[i] = anc[u];
        }
        __syncwarp();
        while (__any_sync(0xffffffffu, par[0] >= 0 || par[1] >= 0)) {
            int nj[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                nj[u] = par[u];
                if (par[u] >= 0) {
                    anc[u] |= ti.anc[par[u]];
                    nj[u] = ti.jump[par[u]];
                }
            }
            __syncwarp();
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int i = lane + 32 * u;
                par[u] = nj[u];
                ti.jump[i] = nj[u];
                ti.anc[i] = anc[u];
            }
            __syncwarp();
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int dep = __popcll(anc[u]) - 1;
            ti.depth[lane + 32 * u] = (signed char)dep;
            dmax = max(dmax, dep);
        }
        dmax = __reduce_max_sync(0xffffffffu, dmax);
        ok = pos + dmax < cap;   // every node's position has a row (pos <= cap: no overflow)
    }
    if (lane == 0) {
        ti.max_depth = dmax;
        ti.valid = ok ? 1 : 0;
    }
}

// The dilated sets of an entry's nodes.  Positions t and t' have the same held
// keys when t == t' mod D, so nodes are taken by depth mod D: set g holds the
// nodes of depth == g mod D, and reads slab (pos + g) mod D.  On the fixed grid
// (and for D = 1) every node reads the same rows.
__device__ __forceinline__ int tree_num_sets(const TreeParams &p, int D, int max_depth) {
    return p.grid ? (max_depth >= 0 ? 1 : 0) : min(D, max_depth + 1);
}
__device__ __forceinline__ int tree_set_of(const TreeParams &p, int D, int depth) {
    return p.grid || D == 1 ? 0 : depth % D;
}
// Held rows of set g, and the first cache row of its slab.
__device__ __forceinline__ int tree_set_rows(const TreeParams &p, int h, int pos, int g, long long &row0) {
    const int D = p.head[h].dil;
    if (p.grid) {
        row0 = 0;
        return pos / D;
    }
    const int r = (int)(((unsigned)pos + g) % (unsigned)D);
    row0 = (long long)r * p.head[h].slab;
    return pos > r ? (pos - 1 - r) / D + 1 : 0;
}
// How n rows are cut: at most `most` pieces of equal length, in whole 128 rows
// (but the last).
constexpr int kTreeMinRows = 128;
__device__ __forceinline__ int tree_piece_rows(int n, int most) {
    const int pieces = max(1, min(most, (n + kTreeMinRows - 1) / kTreeMinRows));
    return ((n + pieces - 1) / pieces + 127) & ~127;   // whole tiles, and whole pages of 128 rows or a divisor
}

// Gate of one channel: a = sigmoid(g) and 1 - a without cancellation, as in the
// decode step (logits beyond +-80 saturate).
__device__ __forceinline__ void gate_pair(float g, float &a, float &oma) {
    const float e = expf(-fminf(fmaxf(g, -80.f), 80.f));
    a = __fdividef(1.f, 1.f + e);   // within 2 units of the last place; 1 + e < 2^126
    oma = e * a;
}

__device__ __forceinline__ void gate4(const float4 &g, float4 &a, float4 &oma) {
    gate_pair(g.x, a.x, oma.x);
    gate_pair(g.y, a.y, oma.y);
    gate_pair(g.z, a.z, oma.z);
    gate_pair(g.w, a.w, oma.w);
}

// Split plan and workspace offsets of a tree step (host); returns the bytes the
// step needs after the workspace header.
struct TreeLayout {
    size_t node_rows, part, ml, info, tc_range, total;
};
TreeLayout tree_plan(const rat_cfg *c, int cap, int page_rows, TreeParams *p);

cudaError_t launch_tree(const TreeParams &p, int dtype, cudaStream_t s);
// recurrence, windows, nodes and the slabs of all heads but those in tc_head (tree_mma.cu)
cudaError_t launch_tree_mma(const TreeParams &p, int dtype, unsigned grid, cudaStream_t s);
// the held rows of its heads in tc_head (tree_tc.cu), and whether pages of
// page_rows rows suit its copies (0: a dense cache)
bool tree_tc_pages(int page_rows);
cudaError_t launch_tree_tc(const TreeParams &p, cudaStream_t s);

// Commit of the accepted branch (tree_commit.cu).
struct CommitParams {
    const void *k, *v, *g;       // [B,N,H,d]
    const int *parent, *leaf;    // device [B,N], [B]
    const float *state[2];       // [B,H,d] fp32
    float *out_state[2];         // [B,H,d] fp32, may be the same memory
    void *cache[2];              // [B,H,R,d] or the pools
    const int *pos;              // device [B]
    int *out_pos;                // device [B], may be the same memory
    long long cache_R;
    int cap, B, N, H, d;
    int grid, sep;
    const int *page_table;
    int page_rows, pps, num_pages;
    int dil[kMaxHeads];
    int win[kMaxHeads];
    int slab[kMaxHeads];
    unsigned char recur[kMaxHeads];
    WsHeader *hdr;
};
cudaError_t launch_tree_commit(const CommitParams &p, int dtype, cudaStream_t s);

}  // namespace rat
