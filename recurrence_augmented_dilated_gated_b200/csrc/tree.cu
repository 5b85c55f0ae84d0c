// tree.cu -- K7: one decode step for a tree of drafted tokens over the decode
// cache ("RAT+: Train Dense, Infer Sparse", Figure 2: decode updates the
// recurrence with a step and attends over the dilated KV cache; here the step
// is taken for every node of a tree of candidate continuations at once).
//
// Node i of entry b hangs below node p_i (-1: below the last held position),
// at depth n_i and position t_i = pos + n_i.  Its augmented key and value are
//   s_i = a_i s_{p_i} + (1 - a_i) x_i   (x = k, v),
// rounded to the cache's type as a cache row would be.  Its query attends, in
// one softmax over a multiset of keys, to
//   - the held rows of its dilated set { j < pos : j == t_i mod D } (on the
//     fixed grid: j mod D == D - 1) and of its window { t_i - W < j < pos },
//   - the nodes of its branch, once for the set and once for the window.
// A softmax over a multiset splits exactly into partial softmaxes (maximum,
// sum, accumulator) over any parts of it, so the step is cut into items:
//   - nodes whose depths agree mod D read the same slab of the cache; an item
//     is one piece of one slab with all the nodes that read it, so every cache
//     row is read once however many nodes need it;
//   - one item per (b, h) runs the recurrence down the tree, then scores the
//     window's held rows and the nodes against each other (a branch is a
//     64-bit mask); a long window is cut into further items.
// tree_combine_kernel joins the partials in a fixed order.
// Bound: the cache rows, each read once; 4 d operations per (node, row).
#include <stdlib.h>
#include "tree_keys.cuh"

namespace rat {

namespace {

constexpr int kThreads = 128;
constexpr int kTile = 32;   // keys per shared-memory tile

// Shared memory of one CTA (floats): Q [MQ][D], K [kTile][D + 4], V [kTile][D],
// P [MQ][kTile]; the recurrence's states and stage lie over them.
template <int D, int MQ> constexpr size_t simt_floats() {
    return (size_t)MQ * D + kTile * (D + 4) + kTile * D + (size_t)MQ * kTile;
}

// Running softmax of the item's nodes: each thread holds D * MQ / 128 sums
// (channel tid % D, nodes (tid / D) + u * (128 / D)), and the maxima and sums of
// the nodes tid / 8 + 16 u.
template <int D, int MQ> struct Running {
    static constexpr int kPer = MQ * D / kThreads;
    static constexpr int kRows = MQ / 16;
    float acc[kPer];
    float m[kRows], l[kRows];
};

template <typename T, int D, int MQ>
__device__ __forceinline__ void attend(const TreeParams &p, const Keys &ks, const TreeInfo &ti, int b, int h, int pos,
                                       const int *nodes, int n_nodes, float *sQ, float *sK, float *sV, float *sP,
                                       float *s_corr, int *s_flags, Running<D, MQ> &R) {
    constexpr int kRows = Running<D, MQ>::kRows, kPer = Running<D, MQ>::kPer;
    const int tid = threadIdx.x;
    const T *src[2];
    if (ks.kind == kNodes) {
        src[0] = static_cast<const T *>(p.node_rows);
        src[1] = src[0] + (size_t)p.N * D;
    } else {
        src[0] = static_cast<const T *>(p.cache[0]);
        src[1] = static_cast<const T *>(p.cache[1]);
    }
    const int qrow = tid / 8, kcol = tid % 8;
    int dep[kRows], node[kRows];
    unsigned long long anc[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
        const int r = qrow + 16 * u;
        node[u] = r < n_nodes ? nodes[r] : -1;
        dep[u] = node[u] >= 0 ? ti.depth[node[u]] : 0;
        anc[u] = node[u] >= 0 ? ti.anc[node[u]] : 0ull;
    }
    for (int k0 = 0; k0 < ks.n; k0 += kTile) {
        __syncthreads();
        if (tid == 0) s_flags[1] = 0;
        __syncthreads();
        // stage the tile's keys and values as floats (rows past the end: zero)
        constexpr int kVec = D / 4;
        for (int e = tid; e < kTile * kVec; e += kThreads) {
            const int r = e / kVec, c = (e % kVec) * 4;
            float4 kk = make_float4(0.f, 0.f, 0.f, 0.f), vv = kk;
            if (k0 + r < ks.n) {
                const long long off = key_offset(p, ks, b, h, k0 + r);
                if (off >= 0) {
                    kk = IO4<T>::load(src[0] + off + c);
                    vv = IO4<T>::load(src[1] + off + c);
                } else {
                    s_flags[0] = 1;
                }
                // inf - inf and NaN - NaN are NaN, x - x is 0 for every other x
                if (ks.kind != kSlab && (vv.x - vv.x) + (vv.y - vv.y) + (vv.z - vv.z) + (vv.w - vv.w) != 0.f) s_flags[1] = 1;
            }
            *reinterpret_cast<float4 *>(sK + r * (D + 4) + c) = kk;
            *reinterpret_cast<float4 *>(sV + r * D + c) = vv;
        }
        __syncthreads();
        // scores of nodes qrow + 16 u against keys kcol + 8 w
        float s[kRows][4];
#pragma unroll
        for (int u = 0; u < kRows; ++u)
#pragma unroll
            for (int w = 0; w < 4; ++w) s[u][w] = 0.f;
#pragma unroll 4
        for (int c = 0; c < D; c += 4) {
            float4 kk[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) kk[w] = *reinterpret_cast<const float4 *>(sK + (kcol + 8 * w) * (D + 4) + c);
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                const float4 qq = *reinterpret_cast<const float4 *>(sQ + (qrow + 16 * u) * D + c);
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    s[u][w] += qq.x * kk[w].x + qq.y * kk[w].y + qq.z * kk[w].z + qq.w * kk[w].w;
            }
        }
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            int cnt[4];
            float mx = -INFINITY;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                cnt[w] = node[u] < 0 ? 0 : key_count(p, ks, ti, h, pos, dep[u], anc[u], node[u], k0 + kcol + 8 * w);
                if (cnt[w]) mx = fmaxf(mx, s[u][w]);
            }
#pragma unroll
            for (int off = 4; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            const float mn = fmaxf(R.m[u], mx);
            const float corr = R.m[u] == -INFINITY ? 0.f : exp2f(R.m[u] - mn);
            const float ref = mn == -INFINITY ? 0.f : mn;   // scores of -inf weigh nothing, NaN stays NaN
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float e = cnt[w] ? cnt[w] * exp2f(s[u][w] - ref) : 0.f;
                sum += e;
                sP[(qrow + 16 * u) * kTile + kcol + 8 * w] = e;
            }
#pragma unroll
            for (int off = 4; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            R.l[u] = R.l[u] * corr + sum;
            R.m[u] = mn;
            if (kcol == 0) s_corr[qrow + 16 * u] = corr;
        }
        __syncthreads();
        const int c = tid % D, r0 = tid / D;
#pragma unroll
        for (int u = 0; u < kPer; ++u) R.acc[u] *= s_corr[r0 + u * (kThreads / D)];
        if (s_flags[1]) {
            // a value that is not finite reaches only the nodes that see its key
            for (int k = 0; k < kTile; ++k) {
                const float v = sV[k * D + c];
#pragma unroll
                for (int u = 0; u < kPer; ++u) {
                    const float e = sP[(r0 + u * (kThreads / D)) * kTile + k];
                    if (e != 0.f) R.acc[u] = fmaf(e, v, R.acc[u]);   // the other path's order: the same bits
                }
            }
            continue;
        }
        for (int k = 0; k < kTile; k += 4) {
            float vv[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) vv[w] = sV[(k + w) * D + c];
#pragma unroll
            for (int u = 0; u < kPer; ++u) {
                const float4 pp = *reinterpret_cast<const float4 *>(sP + (r0 + u * (kThreads / D)) * kTile + k);
                R.acc[u] = fmaf(pp.w, vv[3], fmaf(pp.z, vv[2], fmaf(pp.y, vv[1], fmaf(pp.x, vv[0], R.acc[u]))));
            }
        }
    }
}

template <typename T, int D, int MQ>
__device__ __forceinline__ void run_item(const TreeParams &p, const TreeInfo &ti, int b, int h, int pos,
                                         const Keys *parts, int n_parts, int slot, const int *nodes, int n_nodes,
                                         float *smem, float *s_corr, int *s_flags) {
    float *sQ = smem, *sK = sQ + MQ * D, *sV = sK + kTile * (D + 4), *sP = sV + kTile * D;
    const int tid = threadIdx.x;
    __syncthreads();   // the previous item's reads of sQ and of the recurrence's history
    if (tid == 0) s_flags[0] = 0;
    for (int e = tid; e < MQ * (D / 4); e += kThreads) {
        const int r = e / (D / 4), c = (e % (D / 4)) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < n_nodes) {
            x = IO4<T>::load(static_cast<const T *>(p.q) + (((size_t)b * p.N + nodes[r]) * p.H + h) * D + c);
            x.x *= p.scale_log2; x.y *= p.scale_log2; x.z *= p.scale_log2; x.w *= p.scale_log2;
        }
        *reinterpret_cast<float4 *>(sQ + r * D + c) = x;
    }
    Running<D, MQ> R;
#pragma unroll
    for (int u = 0; u < Running<D, MQ>::kPer; ++u) R.acc[u] = 0.f;
#pragma unroll
    for (int u = 0; u < Running<D, MQ>::kRows; ++u) {
        R.m[u] = -INFINITY;
        R.l[u] = 0.f;
    }
    for (int i = 0; i < n_parts; ++i)
        attend<T, D, MQ>(p, parts[i], ti, b, h, pos, nodes, n_nodes, sQ, sK, sV, sP, s_corr, s_flags, R);
    __syncthreads();
    const size_t base = ((size_t)b * p.slots_per_b + p.slot0[h] + slot) * p.N;
    const int bad = s_flags[0];
    if (tid % 8 == 0) {
#pragma unroll
        for (int u = 0; u < Running<D, MQ>::kRows; ++u) {
            const int r = tid / 8 + 16 * u;
            if (r < n_nodes) p.ml[base + nodes[r]] = make_float2(R.m[u], bad ? -1.f : R.l[u]);
        }
    }
#pragma unroll
    for (int u = 0; u < Running<D, MQ>::kPer; ++u) {
        const int r = tid / D + u * (kThreads / D);
        if (r < n_nodes) p.part[(base + nodes[r]) * D + tid % D] = R.acc[u];
    }
}

template <typename T, int D, int MQ>
__global__ void __launch_bounds__(kThreads) tree_simt_kernel(const TreeParams p) {
    extern __shared__ __align__(16) float smem[];
    __shared__ TreeInfo ti;
    __shared__ int s_parent[kTreeMaxNodes], s_nodes[kTreeMaxNodes];
    __shared__ int s_n, s_flags[2];   // a page was not valid; a value of the tile is not finite
    __shared__ float s_corr[kTreeMaxNodes];
    const int tid = threadIdx.x;
    allow_next();
    const int b = blockIdx.x / p.ctas_per_b, it = blockIdx.x % p.ctas_per_b;
    const int h = find_tree_head(p, it), li = it - p.cta0[h];
    const int pos = p.pos[b];
    if (tid < 32) tree_analyse(ti, p.parent + (size_t)b * p.N, p.N, pos, p.cap);
    if (tid < kTreeMaxNodes) s_parent[tid] = tid < p.N ? p.parent[(size_t)b * p.N + tid] : -2;
    __syncthreads();
    if (li == 0) tell_pieces(p, ti, b, h, pos);
    if (!ti.valid || ti.max_depth < 0) {
        if (!ti.valid && li == 0 && tid == 0) report_error(p.hdr, RAT_ERR_INVALID, b);
        return;
    }
    const int ws = p.wsplit[h];
    if (li < ws) {
        Keys parts[2];
        const int n_parts = local_keys(p, h, pos, li, parts);
        if (li == 0) run_tree<T, D>(p, s_parent, b, h, reinterpret_cast<uint8_t *>(smem));   // over Q, K, V and P
        if (tid == 0) s_n = p.N;
        if (tid < p.N) s_nodes[tid] = tid;
        __syncthreads();
        run_item<T, D, MQ>(p, ti, b, h, pos, parts, n_parts, p.nsplit[h] + li, s_nodes, p.N, smem, s_corr,
                           s_flags);
        return;
    }
    const int sets = tree_num_sets(p, p.dil[h], ti.max_depth), items = sets * p.nsplit[h];
    for (int x = li - ws; x < items; x += p.slab_ctas[h]) {
        const int g = x % sets, piece = x / sets;
        Keys ks;
        if (!slab_keys(p, h, pos, g, piece, ks)) continue;
        __syncthreads();
        if (tid < 32) list_nodes(p, ti, h, g, s_nodes, &s_n);
        __syncthreads();
        run_item<T, D, MQ>(p, ti, b, h, pos, &ks, 1, piece, s_nodes, s_n, smem, s_corr, s_flags);
    }
}

// Joins the partials of a node, pieces of its dilated set and then the window's,
// in that order: a warp a node, a lane the maximum and sum of one piece and then
// D / 32 channels of all of them.
constexpr int kCombineThreads = 128;

template <typename T, int D>
__global__ void __launch_bounds__(kCombineThreads) tree_combine_kernel(const TreeParams p) {
    constexpr int kNodes = kCombineThreads / 32, kC = D / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nb = (p.N + kNodes - 1) / kNodes;
    const int bh = blockIdx.x / nb, i = (blockIdx.x % nb) * kNodes + warp;
    const int b = bh / p.H, h = bh % p.H;
    const int S = p.nsplit[h], ws = p.wsplit[h];
    const size_t base = ((size_t)b * p.slots_per_b + p.slot0[h]) * p.N;
    wait_previous();
    int bad = 0;
    if (p.page_table) {
        // a page that was not valid anywhere in (b, h): the whole pair is skipped
        for (int e = threadIdx.x; e < (S + ws) * p.N; e += kCombineThreads) {
            const int s = e / p.N, np = p.info[(size_t)bh * p.N + e % p.N];
            if (np >= 0 && (s >= S || s < np)) bad |= p.ml[base + e].y < 0.f;
        }
        bad = __syncthreads_or(bad);
        if (bad && threadIdx.x == 0 && i == 0) report_error(p.hdr, RAT_ERR_INVALID, b);
    }
    if (i >= p.N) return;
    const int np = p.info[(size_t)bh * p.N + i];
    float M = -INFINITY, L = 0.f, o[kC] = {};
    if (np >= 0 && !bad) {
        const int n = np + ws;   // piece x is slot x, or S + x - np past the set's
        for (int x = lane; x < n; x += 32) M = fmaxf(M, p.ml[base + (size_t)(x < np ? x : S + x - np) * p.N + i].x);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
#pragma unroll 2
        for (int x = 0; x < n; ++x) {
            const size_t at = base + (size_t)(x < np ? x : S + x - np) * p.N + i;
            const float2 ml = p.ml[at];
            float a[kC];
            if (kC == 4) *reinterpret_cast<float4 *>(a) = *reinterpret_cast<const float4 *>(p.part + at * D + lane * kC);
            else *reinterpret_cast<float2 *>(a) = *reinterpret_cast<const float2 *>(p.part + at * D + lane * kC);
            const float w = ml.y == 0.f ? 0.f : exp2f(ml.x - M);   // a sum that is NaN makes the node NaN
            L += ml.y * w;
#pragma unroll
            for (int c = 0; c < kC; ++c) o[c] += ml.y == 0.f ? 0.f : a[c] * w;
        }
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    T *dst = static_cast<T *>(p.o) + (((size_t)b * p.N + i) * p.H + h) * D + lane * kC;
    if (kC == 4) {
        IO4<T>::store(dst, make_float4(o[0] * inv, o[1] * inv, o[kC - 2] * inv, o[kC - 1] * inv));
    } else {
        store1(dst, o[0] * inv);
        store1(dst + 1, o[1] * inv);
    }
    if (p.lse && lane == 0) p.lse[(size_t)bh * p.N + i] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
}

template <typename T, int D, int MQ> cudaError_t launch_simt(const TreeParams &p, unsigned grid, cudaStream_t s) {
    const size_t smem = simt_floats<D, MQ>() * sizeof(float) > tree_smem<D>(MQ) ? simt_floats<D, MQ>() * sizeof(float) : tree_smem<D>(MQ);
    static std::atomic<unsigned long long> smem_set{0};
    cudaError_t e = ensure_smem_limit(tree_simt_kernel<T, D, MQ>, smem, smem_set);
    if (e != cudaSuccess) return e;
    return launch_after(tree_simt_kernel<T, D, MQ>, grid, kThreads, smem, s, false, p);
}

template <typename T, int D> cudaError_t launch_typed(const TreeParams &p, cudaStream_t s) {
    const unsigned grid = (unsigned)p.B * (unsigned)p.ctas_per_b;
    cudaError_t e = cudaSuccess;
    if (p.n_tc > 0) {
        e = launch_tree_tc(p, s);
        if (e != cudaSuccess) return e;
        count_launches(1);
    }
    if constexpr (sizeof(T) == 2) e = launch_tree_mma(p, grid, s);
    else e = p.N <= 16 ? launch_simt<T, D, 16>(p, grid, s) : launch_simt<T, D, 64>(p, grid, s);
    if (e != cudaSuccess) return e;
    const unsigned nb = (p.N + kCombineThreads / 32 - 1) / (kCombineThreads / 32);
    e = launch_after(tree_combine_kernel<T, D>, (unsigned)p.B * p.H * nb, kCombineThreads, 0, s, true, p);
    if (e != cudaSuccess) return e;
    count_launches(2);
    return cudaSuccess;
}

}  // namespace

// Items are sized by the cache's capacity: pieces of at most `target` rows, cut
// further (down to kRowsMin) only while the batch's items would leave SMs idle.
// How many of a head's D slabs a tree touches is known on the device only (its
// depth): kSetsGuess CTAs per piece share them, and loop when there are more.
TreeLayout tree_plan(const rat_cfg *c, int cap, int page_rows, TreeParams *p) {
    const int kTcMinNodes = getenv("TCMIN") ? atoi(getenv("TCMIN")) : 16;
    constexpr int kRowsMax = 4096, kRowsMin = 256, kItemsWanted = 4 * 148, kSetsGuess = 8;
    const bool grid = (c->flags & RAT_FLAG_GRID_DILATION) != 0;
    const int N = c->T;
    auto sets_of = [&](int D) { return grid ? 1 : (D < kSetsGuess ? D : kSetsGuess) < N ? (D < kSetsGuess ? D : kSetsGuess) : N; };
    int target = kRowsMax;
    while (target > kRowsMin) {
        long long n = 0;
        for (int h = 0; h < c->H; ++h) {
            const long long slab = ((long long)cap + c->dil[h] - 1) / c->dil[h];
            n += sets_of(c->dil[h]) * ((slab + target - 1) / target);
        }
        if (n * c->B >= kItemsWanted) break;
        target /= 2;
    }
    // A CTA that takes several items looks at the tree once: no more CTAs than
    // kItemsWanted * 4 in all, however many items there are.
    long long share = c->B > 0 ? (4ll * kItemsWanted + (long long)c->B * c->H - 1) / ((long long)c->B * c->H) : 1;
    int ctas = 0, slots = 0, per_head = 0;
    p->n_tc = p->tc_items_per_b = 0;
    long long R = 0;
    for (int h = 0; h < c->H; ++h) {
        const int D = c->dil[h];
        const int slab = (int)(((long long)cap + D - 1) / D);
        const int ns = (slab + target - 1) / target;
        p->dil[h] = D;
        // with dedupe a D = 1 head's window keys are all in its dilated set
        p->win[h] = (c->flags & RAT_FLAG_DEDUPE) && D == 1 ? 0 : c->win[h];
        p->slab[h] = slab;
        p->nsplit[h] = ns;
        const int w = p->win[h] < cap ? p->win[h] : cap;
        p->wsplit[h] = w > target ? (w + target - 1) / target : 1;
        const long long most = (long long)sets_of(D) * ns;
        p->slab_ctas[h] = (int)(most < share ? most : share);
        if (c->dtype == RAT_BF16 && c->d == 128 && (grid || D == 1) && N > kTcMinNodes &&
            tree_tc_pages(page_rows)) {
            p->slab_ctas[h] = 0;
            p->tc_head[p->n_tc] = (unsigned char)h;
            p->tc_item0[p->n_tc++] = p->tc_items_per_b;
            p->tc_items_per_b += ns;
        }
        p->cta0[h] = ctas;
        p->slot0[h] = slots;
        p->recur[h] = (c->recur == nullptr || c->recur[h] != 0) ? 1 : 0;
        const int mine = p->wsplit[h] + p->slab_ctas[h];
        per_head = h == 0 ? mine : per_head == mine ? mine : -1;
        ctas += mine;
        slots += ns + p->wsplit[h];
        const long long rows = grid ? (long long)slab + (D > 1 ? c->win[h] : 0) : (long long)D * slab;
        R = R > rows ? R : rows;
    }
    p->cta0[c->H] = ctas;
    p->slot0[c->H] = slots;
    p->ctas_per_b = ctas;
    p->slots_per_b = slots;
    p->ctas_per_head = per_head > 0 ? per_head : 0;
    p->cache_R = R;
    p->grid = grid ? 1 : 0;
    p->dedupe = (c->flags & RAT_FLAG_DEDUPE) ? 1 : 0;
    p->sep = (c->flags & RAT_FLAG_SEPARATE_GATES) ? 1 : 0;
    auto al = [](size_t x) { return (x + 255) & ~(size_t)255; };
    const size_t elt = c->dtype == RAT_F32 ? 4 : 2;
    TreeLayout L;
    L.node_rows = 0;
    L.part = al((size_t)c->B * c->H * 2 * N * c->d * elt);
    L.ml = L.part + al((size_t)c->B * slots * N * c->d * sizeof(float));
    L.info = L.ml + al((size_t)c->B * slots * N * sizeof(float2));
    L.total = L.info + al((size_t)c->B * c->H * N * sizeof(int));
    return L;
}

cudaError_t launch_tree(const TreeParams &p, int dtype, cudaStream_t s) {
    if ((size_t)p.B * p.N == 0) return cudaSuccess;
    if (dtype == RAT_BF16)
        return p.d == 128 ? launch_typed<__nv_bfloat16, 128>(p, s) : launch_typed<__nv_bfloat16, 64>(p, s);
    return p.d == 128 ? launch_typed<float, 128>(p, s) : launch_typed<float, 64>(p, s);
}

}  // namespace rat
