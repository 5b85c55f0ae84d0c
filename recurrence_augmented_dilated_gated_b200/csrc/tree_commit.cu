// tree_commit.cu -- K8: the accepted branch of a drafted tree becomes part of
// the sequence (the decode step's "simple step update" of RAT+ Figure 2, taken
// for every node from the top of the branch to the accepted leaf).
//
// Entry b with leaf l and branch n_0 .. n_{m-1} (n_{m-1} = l): for x = k, v
//   s <- a_{n_i} s + (1 - a_{n_i}) x_{n_i},  cache row of position pos + i <- s,
// then the state is s and the length pos + m.  Nothing of the tree step is
// kept for this: the branch is walked again from the tokens, which is less
// than storing every node's state.
//
// A cluster of kCluster CTAs serves one entry, so that pos can be advanced in
// place: every CTA reads pos[b] before the cluster's barrier and one writes it
// after.  A thread owns four channels of one head and tensor and walks the
// branch, its loads issued kAhead nodes at a time.
// Bound: latency of the walk at small batches, bytes (k, v, g of the branch
// read, its rows written, the states both) at large ones.
#include <cooperative_groups.h>

#include "tree.cuh"

namespace rat {

namespace {

constexpr int kCluster = 8;
constexpr int kThreads = 256;
constexpr int kAhead = 4;

template <typename T>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads) tree_commit_kernel(const CommitParams p) {
    __shared__ int s_path[kTreeMaxNodes];
    __shared__ int s_len;
    const int tid = threadIdx.x;
    const int b = blockIdx.x / kCluster, rank = blockIdx.x % kCluster;
    const int N = p.N;
    const int *parent = p.parent + (size_t)b * N;
    const int pos = p.pos[b], leaf = p.leaf[b];
    if (tid == 0) {
        // the branch, leaf first; a parent is below its child's index, so the
        // walk ends.  -1: an argument out of range
        int n = 0, i = leaf;
        bool ok = pos >= 0 && pos <= p.cap && leaf >= -1 && leaf < N;
        while (ok && i >= 0) {
            const int up = parent[i];
            ok = up >= -1 && up < i;
            s_path[n++] = i;
            i = up;
        }
        ok = ok && pos + n <= p.cap;
        s_len = ok ? n : -1;
    }
    __syncthreads();
    int len = s_len;
    int bad = len < 0;
    if (!bad && p.page_table) {
        // every page that the branch's rows of any head touch has to be valid,
        // else the entry stays as it is; all CTAs check all of them and agree
        for (int x = tid; x < len * p.H; x += kThreads) {
            const int h = x % p.H;
            long long r0, r1;
            cache_rows_of((long long)pos + x / p.H, p.dil[h], p.win[h], p.slab[h], p.grid, r0, r1);
            if (r0 >= 0)
                bad |= cache_offset(p.page_table, p.pps, p.page_rows, p.num_pages, p.cache_R, p.H, p.d, b, h, r0) < 0;
            if (r1 >= 0)
                bad |= cache_offset(p.page_table, p.pps, p.page_rows, p.num_pages, p.cache_R, p.H, p.d, b, h, r1) < 0;
        }
    }
    bad = __syncthreads_or(bad);
    if (bad) {
        len = 0;
        if (tid == 0 && rank == 0) report_error(p.hdr, RAT_ERR_INVALID, b);
    }
    const int vec = p.d / 4, units = p.H * 2 * vec;
    for (int u = rank * kThreads + tid; u < units; u += kCluster * kThreads) {
        const int c = (u % vec) * 4, hx = u / vec, x = hx & 1, h = hx >> 1;
        const size_t e0 = ((size_t)b * p.H + h) * p.d + c;
        const T *src = static_cast<const T *>(x ? p.v : p.k);
        const T *gate = static_cast<const T *>(p.g) + (p.sep && x ? (size_t)p.B * N * p.H * p.d : 0);
        T *cache = static_cast<T *>(p.cache[x]);
        const bool rec = p.recur[h] != 0;
        float4 s = *reinterpret_cast<const float4 *>(p.state[x] + e0);
        for (int i0 = 0; i0 < len; i0 += kAhead) {
            float4 xs[kAhead], gs[kAhead];
#pragma unroll
            for (int w = 0; w < kAhead; ++w) {
                if (i0 + w >= len) break;
                const size_t e = (((size_t)b * N + s_path[len - 1 - i0 - w]) * p.H + h) * p.d + c;
                xs[w] = IO4<T>::load(src + e);
                if (rec) gs[w] = IO4<T>::load(gate + e);
            }
#pragma unroll
            for (int w = 0; w < kAhead; ++w) {
                if (i0 + w >= len) break;
                float a, oma;
                if (rec) {
                    gate_pair(gs[w].x, a, oma); s.x = a * s.x + oma * xs[w].x;
                    gate_pair(gs[w].y, a, oma); s.y = a * s.y + oma * xs[w].y;
                    gate_pair(gs[w].z, a, oma); s.z = a * s.z + oma * xs[w].z;
                    gate_pair(gs[w].w, a, oma); s.w = a * s.w + oma * xs[w].w;
                } else {
                    s = xs[w];
                }
                long long r0, r1;
                cache_rows_of((long long)pos + i0 + w, p.dil[h], p.win[h], p.slab[h], p.grid, r0, r1);
                if (r0 >= 0)
                    IO4<T>::store(cache + cache_offset(p.page_table, p.pps, p.page_rows, p.num_pages, p.cache_R, p.H,
                                                       p.d, b, h, r0) + c, s);
                if (r1 >= 0)   // a branch longer than the window wraps around the ring: the last position stays
                    IO4<T>::store(cache + cache_offset(p.page_table, p.pps, p.page_rows, p.num_pages, p.cache_R, p.H,
                                                       p.d, b, h, r1) + c, s);
            }
        }
        *reinterpret_cast<float4 *>(p.out_state[x] + e0) = s;
    }
    cooperative_groups::this_cluster().sync();   // every CTA of the entry has read pos[b]
    if (rank == 0 && tid == 0) p.out_pos[b] = pos + len;
}

}  // namespace

cudaError_t launch_tree_commit(const CommitParams &p, int dtype, cudaStream_t s) {
    if (p.B == 0) return cudaSuccess;
    const unsigned grid = (unsigned)p.B * kCluster;
    if (dtype == RAT_BF16) tree_commit_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(p);
    else tree_commit_kernel<float><<<grid, kThreads, 0, s>>>(p);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace rat
