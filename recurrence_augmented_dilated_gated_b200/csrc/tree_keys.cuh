// tree_keys.cuh -- what the kernels of the tree step share (tree_mma.cu: every
// item; tree_tc.cu: held rows of large trees): which keys an item holds, where
// they are and for whom they count, and the recurrence down the tree.
#pragma once

#include "tree.cuh"
#include "tree_copy.cuh"

namespace rat {

__device__ __forceinline__ int find_tree_head(const TreeParams &p, int it) {
    if (p.ctas_per_head > 0) return it / p.ctas_per_head;
    int lo = 0, hi = p.H - 1;  // largest h with cta0[h] <= it
    while (lo < hi) {
        int mid = (lo + hi + 1) >> 1;
        if (p.head[mid].cta0 <= it) lo = mid; else hi = mid - 1;
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
        const unsigned j = row, D = p.head[h].dil, S = p.head[h].slab;
        if (!p.grid) row = D == 1 ? j : j % D * S + j / D;
        else row = D > 1 ? S + j % (unsigned)p.head[h].win : j;   // the ring
    }
    if (!p.page_table) return (bh * p.cache_R + row) * p.d;
    const unsigned pi = row / (unsigned)p.page_rows, pr = row - pi * p.page_rows;
    const int pg = p.page_table[(long long)b * p.pps + pi];
    if (pg < 0 || pg >= p.num_pages) return -1;
    return (((long long)pg * p.H + h) * p.page_rows + pr) * p.d;
}

// Depth differences that are multiples of a head's dilation, and the nodes on its
// grid, as bits (one warp).
__device__ __forceinline__ void tree_masks(const TreeParams &p, TreeInfo &ti, int h, int pos) {
    const int lane = threadIdx.x & 31;
    const unsigned D = p.head[h].dil;
    unsigned m[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int i = lane + 32 * u;
        m[u] = __ballot_sync(0xffffffffu, p.grid ? ti.depth[i] >= 0 && (unsigned)(pos + ti.depth[i]) % D == D - 1 : i % D == 0);
    }
    if (lane == 0) ti.far = (unsigned long long)m[1] << 32 | m[0];
}

// How often key i counts for a node of depth `dep` and branch `anc` (0, 1 or 2).
__device__ __forceinline__ int key_count(const TreeParams &p, const Keys &ks, const TreeInfo &ti, int h, int pos,
                                         int dep, unsigned long long anc, int node, int i) {
    if (i >= ks.n) return 0;
    if (ks.kind == kSlab) return 1;
    const int D = p.head[h].dil, W = p.head[h].win;
    if (ks.kind == kWindow) {
        const int j = (int)ks.row0 + i, t = pos + dep;
        if (j <= t - W) return 0;
        if (p.dedupe && (p.grid ? j % D == D - 1 : (t - j) % D == 0)) return 0;
        return 1;
    }
    if (!((anc >> i) & 1ull)) return 0;
    const int back = dep - ti.depth[i];
    const int far = p.grid ? i == node || ((ti.far >> i) & 1ull) : (int)((ti.far >> back) & 1ull);
    const int near = back < W && !(p.dedupe && far);
    return far + near;
}

__device__ __forceinline__ void store1(float *p, float x) { *p = x; }
__device__ __forceinline__ void store1(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// The rows of piece `piece` of set g; false when there is none.
__device__ __forceinline__ bool slab_keys(const TreeParams &p, int h, int pos, int g, int piece, Keys &ks) {
    ks.kind = kSlab;
    const int n = tree_set_rows(p, h, pos, g, ks.row0);
    const int len = tree_piece_rows(n, p.head[h].nsplit);
    if (n == 0 || (long long)piece * len >= n) return false;
    ks.row0 += piece * len;
    ks.n = min(len, n - piece * len);
    return true;
}

// The keys of a head's local item `li`: a piece of the window's held rows, in
// item 0 the nodes, and the held rows of the dilated set if the head's keys are
// all in one item.  Returns the number of parts.
__device__ __forceinline__ int local_keys(const TreeParams &p, int h, int pos, int li, Keys *parts) {
    const int ws = p.head[h].wsplit, W = p.head[h].win;
    const int n_held = W > 0 ? min(W - 1, pos) : 0, len = (n_held + ws - 1) / ws;
    const int a = min(li * len, n_held);
    int k = 0;
    if (p.head[h].fused && slab_keys(p, h, pos, 0, 0, parts[0])) k = 1;
    parts[k].kind = kWindow;
    parts[k].row0 = pos - n_held + a;
    parts[k].n = min(len, n_held - a);
    if (parts[k].n > 0) ++k;
    if (li == 0) {
        parts[k].kind = kNodes;
        parts[k].row0 = 0;
        parts[k].n = p.N;
        ++k;
    }
    return k;
}

// What tree_combine_kernel needs to know of the tree (item 0 of every head).
__device__ __forceinline__ void tell_pieces(const TreeParams &p, const TreeInfo &ti, int b, int h, int pos) {
    const int i = threadIdx.x;
    if (i >= p.N) return;
    int np = -1;
    if (ti.valid && ti.depth[i] >= 0) {
        long long row0;
        const int n = tree_set_rows(p, h, pos, tree_set_of(p, p.head[h].dil, ti.depth[i]), row0);
        const int len = tree_piece_rows(n, p.head[h].nsplit);
        np = n == 0 ? 0 : (n + len - 1) / len;
    }
    if (ti.valid && ti.max_depth >= 0 && p.head[h].fused) np = -2;   // absent nodes too
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
        const bool in = ti.depth[i] >= 0 && tree_set_of(p, p.head[h].dil, ti.depth[i]) == g;
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

// The recurrence down the tree (128 threads), 64 channels at a time, in shared
// memory as [node][array][64] floats: arrays k, v, gate and, with separate gates,
// the values' gate.
//   1  the tokens of all nodes are copied into their places (one round trip);
//   2  half a warp a node, each place is overwritten: k and v by (1 - a) x, a gate
//      by a;
//   3  a thread, one channel of one tensor, walks the nodes, a parent before its
//      children, adding a * parent: the rest is out of the chain;
//   4  the rows are rounded and written out together.
// (Gates inside the walk took 500 cycles a node, 23 us for 64 nodes.)  The code is
// kept small: it runs once per CTA, and a straight line of instructions fetched
// cold costs more than a loop.  The memory stays within a bf16 ring's 64 KB, so
// that three CTAs share an SM (two took the hybrid step from 377 to 412 us).
constexpr int kTreeChannels = 64;
constexpr size_t tree_smem(int N, int sep) { return (size_t)N * kTreeChannels * (sep ? 4 : 3) * sizeof(float); }

template <typename T, int D>
__device__ __forceinline__ void run_tree(const TreeParams &p, const int *parent, int b, int h, float *mem) {
    constexpr int kThreads = 128, kCh = kTreeChannels;
    constexpr int kChunks = kCh * (int)sizeof(T) / 16;               // 16-byte chunks of 64 channels
    const int tid = threadIdx.x, N = p.N;
    const int arrays = p.sep ? 4 : 3, row = arrays * kCh;            // floats of a node
    const size_t bh = (size_t)b * p.H + h;
    const bool rec = p.head[h].recur != 0;
    const int c = tid % kCh, x = tid / kCh;
#pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += kCh) {
        const float s0 = p.state[x][bh * D + c0 + c];
        __syncthreads();   // the channels before are written out
#pragma unroll 1
        for (int y = 0; y < (rec ? arrays : 2); ++y) {
            const T *src = static_cast<const T *>(y == 0 ? p.k : y == 1 ? p.v : p.g) + (y == 3 ? (size_t)p.B * N * p.H * D : 0) + c0;
#pragma unroll 2
            for (int e = tid; e < N * kChunks; e += kThreads) {
                const int n = e / kChunks, ch = e % kChunks;
                cp_async16(smem_u32(mem + n * row + y * kCh) + ch * 16,
                           src + (((size_t)b * N + n) * p.H + h) * D + ch * (16 / (int)sizeof(T)), true);
            }
        }
        cp_commit();
        cp_wait<0>();
        __syncthreads();
#pragma unroll 1
        for (int n0 = 0; n0 < N; n0 += kThreads / 16) {
            const int n = n0 + tid / 16;
            float *m = mem + n * row + (tid % 16) * 4;
            const T *raw = reinterpret_cast<const T *>(mem + n * row) + (tid % 16) * 4;
            constexpr int kStep = kCh * (int)(sizeof(float) / sizeof(T));   // from array to array
            float4 k, v, g, gv;
            if (n < N) {
                k = IO4<T>::load(raw);
                v = IO4<T>::load(raw + kStep);
                if (rec) g = IO4<T>::load(raw + 2 * kStep);
                if (rec && p.sep) gv = IO4<T>::load(raw + 3 * kStep);
            }
            __syncwarp();
            if (n < N) {
                float4 a = make_float4(0.f, 0.f, 0.f, 0.f), oma = make_float4(1.f, 1.f, 1.f, 1.f);
                if (rec) gate4(g, a, oma);
                *reinterpret_cast<float4 *>(m) = make_float4(oma.x * k.x, oma.y * k.y, oma.z * k.z, oma.w * k.w);
                *reinterpret_cast<float4 *>(m + 2 * kCh) = a;
                if (p.sep) {
                    if (rec) gate4(gv, a, oma);
                    *reinterpret_cast<float4 *>(m + 3 * kCh) = a;
                }
                *reinterpret_cast<float4 *>(m + kCh) = make_float4(oma.x * v.x, oma.y * v.y, oma.z * v.z, oma.w * v.w);
            }
        }
        __syncthreads();
        float *m = mem + x * kCh + c;
        const float *ga = mem + (2 + (p.sep ? x : 0)) * kCh + c;
#pragma unroll 1
        for (int n0 = 0; n0 < N; n0 += 4) {
            float a[4], u[4];
            int par[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int n = min(n0 + w, N - 1);
                par[w] = parent[n];
                u[w] = m[n * row];
                a[w] = ga[n * row];
            }
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                if (n0 + w < N) {
                    const float s = a[w] * (par[w] >= 0 ? m[par[w] * row] : s0) + u[w];
                    m[(n0 + w) * row] = par[w] == RAT_NODE_ABSENT ? 0.f : s;   // its inputs may hold anything
                }
            }
        }
        __syncthreads();
        T *out = static_cast<T *>(p.node_rows) + bh * 2 * N * D + c0;
#pragma unroll 2
        for (int e = tid; e < N * 2 * (kCh / 4); e += kThreads) {
            const int ch = e % (kCh / 4), nx = e / (kCh / 4), y = nx & 1, n = nx >> 1;
            IO4<T>::store(out + ((size_t)y * N + n) * D + ch * 4, *reinterpret_cast<const float4 *>(mem + n * row + y * kCh + ch * 4));
        }
    }
    __threadfence();   // other threads copy these rows past L1
}

}  // namespace rat
