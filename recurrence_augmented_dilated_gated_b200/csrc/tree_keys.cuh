// tree_keys.cuh -- what the two forms of the tree step share (tree.cu: CUDA
// cores, fp32; tree_mma.cu: tensor cores, bf16): which keys an item holds,
// where they are and for whom they count, and the recurrence down the tree.
#pragma once

#include "tree.cuh"

namespace rat {

__device__ __forceinline__ int find_tree_head(const TreeParams &p, int it) {
    int lo = 0, hi = p.H - 1;  // largest h with cta0[h] <= it
    while (lo < hi) {
        int mid = (lo + hi + 1) >> 1;
        if (p.cta0[mid] <= it) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// The keys of one item: rows of a slab, held rows of the window, or the nodes.
enum KeyKind { kSlab = 0, kWindow = 1, kNodes = 2 };

struct Keys {
    int kind;
    long long row0;   // slab: first cache row;  window: first position
    int n;            // keys
};

__device__ __forceinline__ long long key_offset(const TreeParams &p, const Keys &ks, int b, int h, int i) {
    if (ks.kind == kNodes) return ((((long long)b * p.H + h) * 2) * p.N + i) * p.d;   // keys; values N * d further
    long long row = ks.row0 + i;
    if (ks.kind == kWindow) {
        long long main_row, ring_row;
        cache_rows_of(row, p.dil[h], p.win[h], p.slab[h], p.grid, main_row, ring_row);
        row = ring_row >= 0 ? ring_row : main_row;
    }
    return cache_offset(p.page_table, p.pps, p.page_rows, p.num_pages, p.cache_R, p.H, p.d, b, h, row);
}

// How often key i counts for a node of depth `dep` and branch `anc` (0, 1 or 2).
__device__ __forceinline__ int key_count(const TreeParams &p, const Keys &ks, const TreeInfo &ti, int h, int pos,
                                         int dep, unsigned long long anc, int node, int i) {
    if (i >= ks.n) return 0;
    if (ks.kind == kSlab) return 1;
    const int D = p.dil[h], W = p.win[h];
    if (ks.kind == kWindow) {
        const int j = (int)ks.row0 + i, t = pos + dep;
        if (j <= t - W) return 0;
        if (p.dedupe && (p.grid ? j % D == D - 1 : (t - j) % D == 0)) return 0;
        return 1;
    }
    if (!((anc >> i) & 1ull)) return 0;
    const int back = dep - ti.depth[i];
    const int far = p.grid ? (i == node || (pos + ti.depth[i]) % D == D - 1) : back % D == 0;
    const int near = back < W && !(p.dedupe && far);
    return far + near;
}

__device__ __forceinline__ void store1(float *p, float x) { *p = x; }
__device__ __forceinline__ void store1(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// The keys of a head's local item `li`: a piece of the window's held rows, and
// in item 0 the nodes.  Returns the number of parts.
__device__ __forceinline__ int local_keys(const TreeParams &p, int h, int pos, int li, Keys *parts) {
    const int ws = p.wsplit[h], W = p.win[h];
    const int n_held = W > 0 ? min(W - 1, pos) : 0, len = (n_held + ws - 1) / ws;
    const int a = min(li * len, n_held);
    parts[0].kind = kWindow;
    parts[0].row0 = pos - n_held + a;
    parts[0].n = min(len, n_held - a);
    parts[1].kind = kNodes;
    parts[1].row0 = 0;
    parts[1].n = p.N;
    return li == 0 ? 2 : 1;
}

// The rows of piece `piece` of set g; false when there is none.
__device__ __forceinline__ bool slab_keys(const TreeParams &p, int h, int pos, int g, int piece, Keys &ks) {
    ks.kind = kSlab;
    const int n = tree_set_rows(p, h, pos, g, ks.row0);
    const int len = tree_piece_rows(n, p.nsplit[h]);
    if (n == 0 || (long long)piece * len >= n) return false;
    ks.row0 += piece * len;
    ks.n = min(len, n - piece * len);
    return true;
}

// The nodes of set g, in order (one warp).
__device__ __forceinline__ void list_nodes(const TreeParams &p, const TreeInfo &ti, int h, int g, int *nodes, int *n) {
    const int lane = threadIdx.x & 31;
    int cnt = 0;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int i = lane + 32 * u;
        const bool in = ti.depth[i] >= 0 && tree_set_of(p, p.dil[h], ti.depth[i]) == g;
        const unsigned mask = __ballot_sync(0xffffffffu, in);
        if (in) nodes[cnt + __popc(mask & ((1u << lane) - 1u))] = i;
        cnt += __popc(mask);
    }
    if (lane == 0) *n = cnt;
}

// The recurrence down the tree: one channel of one tensor per thread, nodes in
// order (a parent comes before its children), states kept in shared memory.
template <typename T, int D, int kThreads>
__device__ __forceinline__ void run_tree(const TreeParams &p, const int *parent, int b, int h,
                                         float *hist) {
    const size_t bh = (size_t)b * p.H + h;
    for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
        const int x = i / D, c = i % D;
        const T *src = static_cast<const T *>(x ? p.v : p.k);
        const T *gate = static_cast<const T *>(p.g) + (p.sep && x ? (size_t)p.B * p.N * p.H * D : 0);
        const float s0 = p.state[x][bh * D + c];
        T *out = static_cast<T *>(p.node_rows) + (bh * 2 + x) * p.N * D + c;
        float *hc = hist + threadIdx.x;   // this thread's column: no other thread reads it
        const bool rec = p.recur[h] != 0;
#pragma unroll 4
        for (int n = 0; n < p.N; ++n) {
            const size_t e = (((size_t)b * p.N + n) * p.H + h) * D + c;
            float a = 0.f, oma = 1.f;
            if (rec) gate_pair((float)gate[e], a, oma);
            const int par = parent[n];
            float s = a * (par >= 0 ? hc[(size_t)par * kThreads] : s0) + oma * (float)src[e];
            if (par == RAT_NODE_ABSENT) s = 0.f;   // its inputs may hold anything
            hc[(size_t)n * kThreads] = s;
            store1(out + (size_t)n * D, s);
        }
    }
}

}  // namespace rat
