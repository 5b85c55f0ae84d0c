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
// A cluster of up to kMaxCluster CTAs serves one entry (as many as its channels
// fill), so that pos can be advanced in place: every CTA reads pos[b] before
// the cluster's barrier and one writes it after.  A thread owns four channels of
// one head, keys and values (one gate for both), and walks the branch with the
// loads of kAhead nodes in flight; it steps row numbers along instead of
// dividing.
// Bound: latency of the walk at small batches, bytes (k, v, g of the branch
// read, its rows written, the states both) at large ones.
#include <cooperative_groups.h>

#include "tree.cuh"

namespace rat {

namespace {

constexpr int kMaxCluster = 8;   // portable
constexpr int kThreads = 128;
constexpr int kAhead = 4;

__device__ __forceinline__ void step4(float4 &s, const float4 &x, const float4 &a, const float4 &oma) {
    s.x = a.x * s.x + oma.x * x.x;
    s.y = a.y * s.y + oma.y * x.y;
    s.z = a.z * s.z + oma.z * x.z;
    s.w = a.w * s.w + oma.w * x.w;
}
template <typename T>
__global__ void __launch_bounds__(kThreads) tree_commit_kernel(const CommitParams p) {
    cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
    const int kCluster = (int)cluster.num_blocks();
    __shared__ int s_parent[kTreeMaxNodes], s_path[kTreeMaxNodes];
    __shared__ int s_len;
    const int tid = threadIdx.x;
    const int b = blockIdx.x / kCluster, rank = (int)cluster.block_rank();
    const int N = p.N;
    const int pos = p.pos[b], leaf = p.leaf[b];
    if (tid < N) s_parent[tid] = p.parent[(size_t)b * N + tid];
    __syncthreads();
    if (tid == 0) {
        // the branch, leaf first; a parent is below its child's index, so the
        // walk ends.  -1: an argument out of range
        int n = 0, i = leaf;
        bool ok = pos >= 0 && pos <= p.cap && leaf >= -1 && leaf < N;
        while (ok && i >= 0) {
            const int up = s_parent[i];
            ok = up >= -1 && up < i;
            s_path[n++] = i;
            i = up;
        }
        ok = ok && pos <= p.cap - n;
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
        bad = __syncthreads_or(bad);
    }
    if (bad) {
        len = 0;
        if (tid == 0 && rank == 0) report_error(p.hdr, RAT_ERR_INVALID, b);
    }
    const int vec = p.d / 4, units = p.H * vec;
    const T *kin = static_cast<const T *>(p.k), *vin = static_cast<const T *>(p.v), *gin = static_cast<const T *>(p.g);
    const T *gvin = gin + (p.sep ? (size_t)p.B * N * p.H * p.d : 0);
    T *ck = static_cast<T *>(p.cache[0]), *cv = static_cast<T *>(p.cache[1]);
    for (int u = rank * kThreads + tid; u < units; u += kCluster * kThreads) {
        const int c = (u % vec) * 4, h = u / vec;
        const size_t e0 = ((size_t)b * p.H + h) * p.d + c;
        const bool rec = p.recur[h] != 0;
        float4 sk = *reinterpret_cast<const float4 *>(p.state[0] + e0), sv = *reinterpret_cast<const float4 *>(p.state[1] + e0);
        const unsigned D = p.dil[h], S = p.slab[h], W = p.grid && D > 1 ? p.win[h] : 0;
        unsigned res = (unsigned)pos % D, quo = (unsigned)pos / D, ring = W ? (unsigned)pos % W : 0;
        auto put = [&](unsigned row) {
            const long long off = cache_offset(p.page_table, p.pps, p.page_rows, p.num_pages, p.cache_R, p.H, p.d, b, h, row) + c;
            IO4<T>::store(ck + off, sk);
            IO4<T>::store(cv + off, sv);
        };
        for (int i0 = 0; i0 < len; i0 += kAhead) {
            float4 xk[kAhead], xv[kAhead], g[kAhead], gv[kAhead];
#pragma unroll
            for (int w = 0; w < kAhead; ++w) {
                if (i0 + w >= len) break;
                const size_t e = (((size_t)b * N + s_path[len - 1 - i0 - w]) * p.H + h) * p.d + c;
                xk[w] = IO4<T>::load(kin + e);
                xv[w] = IO4<T>::load(vin + e);
                if (rec) g[w] = IO4<T>::load(gin + e);
                if (rec && p.sep) gv[w] = IO4<T>::load(gvin + e);
            }
#pragma unroll
            for (int w = 0; w < kAhead; ++w) {
                if (i0 + w >= len) break;
                if (rec) {
                    float4 a, oma;
                    gate4(g[w], a, oma);
                    step4(sk, xk[w], a, oma);
                    if (p.sep) gate4(gv[w], a, oma);
                    step4(sv, xv[w], a, oma);
                } else {
                    sk = xk[w];
                    sv = xv[w];
                }
                if (!p.grid) put(res * S + quo);
                else if (res == D - 1) put(quo);
                if (W) put(S + ring);   // a branch longer than the window wraps around: the last position stays
                if (++res == D) {
                    res = 0;
                    ++quo;
                }
                if (++ring == W) ring = 0;
            }
        }
        *reinterpret_cast<float4 *>(p.out_state[0] + e0) = sk;
        *reinterpret_cast<float4 *>(p.out_state[1] + e0) = sv;
    }
    cluster.sync();   // every CTA of the entry has read pos[b]
    if (rank == 0 && tid == 0) p.out_pos[b] = pos + len;
}

}  // namespace

cudaError_t launch_tree_commit(const CommitParams &p, int dtype, cudaStream_t s) {
    if (p.B == 0) return cudaSuccess;
    const int need = (p.H * (p.d / 4) + kThreads - 1) / kThreads;
    int size = 1;
    while (size < need && size < kMaxCluster) size *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.B * size);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = size;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    cudaError_t e = dtype == RAT_BF16 ? cudaLaunchKernelEx(&cfg, tree_commit_kernel<__nv_bfloat16>, p)
                                      : cudaLaunchKernelEx(&cfg, tree_commit_kernel<float>, p);
    if (e != cudaSuccess) return e;
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace rat
