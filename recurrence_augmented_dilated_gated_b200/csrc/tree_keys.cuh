// tree_keys.cuh -- what the two forms of the tree step share (tree.cu: CUDA
// cores, fp32; tree_mma.cu: tensor cores, bf16): which keys an item holds,
// where they are and for whom they count, and the recurrence down the tree.
#pragma once

#include "tree.cuh"
#include "tree_copy.cuh"

namespace rat {

__device__ __forceinline__ int find_tree_head(const TreeParams &p, int it) {
    if (p.ctas_per_head > 0) return it / p.ctas_per_head;
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

// Element offset of key i: of its cache row (-1: no valid page), or of the
// node's row.  Rows and positions fit in 32 bits (D * ceil(cap / D) < cap + D).
__device__ __forceinline__ long long key_offset(const TreeParams &p, const Keys &ks, int b, int h, int i) {
    const long long bh = (long long)b * p.H + h;
    if (ks.kind == kNodes) return (bh * 2 * p.N + i) * p.d;   // keys; values N * d further
    unsigned row = (unsigned)ks.row0 + i;
    if (ks.kind == kWindow) {
        const unsigned j = row, D = p.dil[h], S = p.slab[h];
        if (!p.grid) row = D == 1 ? j : j % D * S + j / D;
        else row = D > 1 ? S + j % (unsigned)p.win[h] : j;   // the ring
    }
    if (!p.page_table) return (bh * p.cache_R + row) * p.d;
    const unsigned pi = row / (unsigned)p.page_rows, pr = row - pi * p.page_rows;
    const int pg = p.page_table[(long long)b * p.pps + pi];
    if (pg < 0 || pg >= p.num_pages) return -1;
    return (((long long)pg * p.H + h) * p.page_rows + pr) * p.d;
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

// What tree_combine_kernel needs to know of the tree (item 0 of every head).
__device__ __forceinline__ void tell_pieces(const TreeParams &p, const TreeInfo &ti, int b, int h, int pos) {
    const int i = threadIdx.x;
    if (i >= p.N) return;
    int np = -1;
    if (ti.valid && ti.depth[i] >= 0) {
        long long row0;
        const int n = tree_set_rows(p, h, pos, tree_set_of(p, p.dil[h], ti.depth[i]), row0);
        const int len = tree_piece_rows(n, p.nsplit[h]);
        np = n == 0 ? 0 : (n + len - 1) / len;
    }
    p.info[((size_t)b * p.H + h) * p.N + i] = np;
}

// Programmatic dependent launch: the next kernel of the step may start once
// every CTA of this one has; it waits itself before it reads.
__device__ __forceinline__ void allow_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), unsigned grid, unsigned threads, size_t smem, cudaStream_t s, bool after, const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = after ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
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

// 16 bytes past L1; zeros when `on` is false (the address is not read then)
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// The recurrence down the tree (128 threads).  A thread owns one channel of both
// tensors (D = 128) or of one (D = 64: the upper half of the CTA takes the
// values) and walks the nodes in order, a parent before its children.  k, v and
// g of as many nodes as fit in kTreeStage bytes are staged together by
// asynchronous copies: one round trip to memory for 32 nodes of bf16, not one
// per node.  Shared memory: the states, a column per thread ([node][2 D] floats),
// then the stage.  The code is kept small (no unrolled chunk): it runs once per
// CTA, and fetching a straight line of instructions cold costs more than the
// loop (measured: 40 us a CTA with 16 nodes unrolled).
constexpr int kTreeStage = 32768;
template <int D> constexpr size_t tree_smem(int N) { return (size_t)N * 2 * D * sizeof(float) + kTreeStage; }

template <typename T, int D>
__device__ __forceinline__ void run_tree(const TreeParams &p, const int *parent, int b, int h, uint8_t *smem) {
    constexpr int kThreads = 128, kBoth = D == kThreads ? 2 : 1;
    constexpr int kChunks = D * (int)sizeof(T) / 16;                 // 16-byte chunks of a row
    constexpr int kNodes = kTreeStage / (4 * D * (int)sizeof(T));    // nodes staged at a time (k, v, two gates)
    static_assert(D * 2 == kThreads * kBoth, "the CTA's threads cover the channels of both tensors");
    const int tid = threadIdx.x, c = tid % D, x0 = tid / D;
    const size_t bh = (size_t)b * p.H + h;
    const bool rec = p.recur[h] != 0;
    const int n_src = !rec ? 2 : p.sep ? 4 : 3;
    float *hc = reinterpret_cast<float *>(smem) + tid;   // [node][kBoth][thread]: no other thread reads this column
    uint8_t *stage = smem + (size_t)p.N * 2 * D * sizeof(float);
    const float s0 = p.state[x0][bh * D + c], s1 = kBoth == 2 ? p.state[1][bh * D + c] : 0.f;
    T *out = static_cast<T *>(p.node_rows) + (bh * 2 + x0) * p.N * D + c;
    for (int n0 = 0; n0 < p.N; n0 += kNodes) {
        const int nn = min(kNodes, p.N - n0);
        __syncthreads();   // the stage is free
#pragma unroll 1
        for (int y = 0; y < n_src; ++y) {
            const char *src = static_cast<const char *>(y == 0 ? p.k : y == 1 ? p.v : p.g) +
                              (y == 3 ? (size_t)p.B * p.N * p.H * D * sizeof(T) : 0);
#pragma unroll 1
            for (int e = tid; e < nn * kChunks; e += kThreads) {
                const int n = e / kChunks, ch = e % kChunks;
                cp_async16(smem_u32(stage) + ((y * kNodes + n) * kChunks + ch) * 16,
                           src + ((((size_t)b * p.N + n0 + n) * p.H + h) * kChunks + ch) * 16, true);
            }
        }
        cp_commit();
        cp_wait<0>();
        __syncthreads();
        const T *st = reinterpret_cast<const T *>(stage) + c;
#pragma unroll 2
        for (int w = 0; w < nn; ++w) {
            const int n = n0 + w, par = parent[n];
            float a = 0.f, oma = 1.f;
            if (rec) gate_pair((float)st[((p.sep && x0 ? 3 : 2) * kNodes + w) * D], a, oma);
            float s = a * (par >= 0 ? hc[(size_t)par * kBoth * kThreads] : s0) + oma * (float)st[(x0 * kNodes + w) * D];
            if (par == RAT_NODE_ABSENT) s = 0.f;   // its inputs may hold anything
            hc[(size_t)n * kBoth * kThreads] = s;
            store1(out + (size_t)n * D, s);
            if (kBoth == 2) {
                if (rec && p.sep) gate_pair((float)st[(3 * kNodes + w) * D], a, oma);
                s = a * (par >= 0 ? hc[(size_t)(par * 2 + 1) * kThreads] : s1) + oma * (float)st[(kNodes + w) * D];
                if (par == RAT_NODE_ABSENT) s = 0.f;
                hc[(size_t)(n * 2 + 1) * kThreads] = s;
                store1(out + (size_t)(p.N + n) * D, s);
            }
        }
    }
    __threadfence();   // other threads copy these rows past L1
}

}  // namespace rat
