// tree_mma.cu -- K7 with bf16 operands: the tree step's items (tree.cu) on the
// tensor cores.
//
// An item is a run of cache rows and the nodes that read it: scores S = Q K~^T,
// probabilities P, sums O = P V~, with 16 nodes as the rows of one matrix
// instruction (m16n8k16, fp32 accumulation).  A node's rows of S and O stay in
// registers for the whole item; K~ and V~ rows pass through a ring of shared
// memory filled by 16-byte asynchronous copies, in tiles of kTile rows.
//   - up to 16 nodes: the four warps take different keys of the tile and join
//     their partial softmaxes at the end; up to 32: two by two; up to 64: a
//     warp for every 16 nodes.  So every warp works whatever the tree's shape.
//   - 16-byte chunk c of row r sits at chunk c ^ (r & 7): the eight rows of an
//     ldmatrix fall on different banks.
//   - the softmax reference of a node is raised only when a score passes it by
//     more than 2^8 (P stays below 2^8, its sum in fp32): one vote per 16 keys
//     instead of reductions and rescaling.
//   - P is rounded to bf16 for the product with V~ (half a step, 2^-9 of each
//     probability; the sum of P keeps fp32): the same rounding as the prefill's.
// Bound: HBM for small node counts (a row's 4 d bytes are used for 4 d
// operations per node).
#include "tree_keys.cuh"

namespace rat {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 64;
constexpr int kStages = 3;
constexpr float kSlack = 8.f;   // log2 of how far P may pass 1

__device__ __forceinline__ uint32_t smem_u32(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// 16 bytes; zeros when `on` is false (the address is not read then)
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack2(float x, float y) {
    __nv_bfloat162 t = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<uint32_t *>(&t);
}
__device__ __forceinline__ bool not_finite2(uint32_t w) {   // either bf16 of a pair
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

template <int D> struct Shape {
    static constexpr int kChunks = D / 8;                   // 16-byte chunks of a row
    static constexpr uint32_t kRowBytes = D * 2;
    static constexpr uint32_t kHalf = kTile * kRowBytes;    // K~ of a stage, then V~
    static constexpr uint32_t kStage = 2 * kHalf;
    static constexpr int kRowsAtOnce = kThreads / kChunks;  // rows that one pass of the CTA copies
    static __device__ __forceinline__ uint32_t at(int r, int c) { return r * kRowBytes + ((c ^ (r & 7)) << 4); }
};

struct Shared {
    TreeInfo ti;
    int parent[kTreeMaxNodes], nodes[kTreeMaxNodes];
    int n, bad;
    unsigned long long odd[3];       // rows of local tile t with a value that is not finite, at t mod 3
    float m[kWarps][16], l[kWarps][16];
};

// One item: the keys of parts[0 .. n_parts), tile by tile.
template <int D, bool kLocal>
__device__ __forceinline__ void run_item(const TreeParams &p, Shared &sh, uint8_t *ring, const Keys *parts, int n_parts,
                                         int b, int h, int pos, int slot) {
    using S = Shape<D>;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    __syncthreads();   // sh.n and sh.nodes are set, and the ring is free
    const int n_nodes = sh.n;
    const int WM = n_nodes <= 16 ? 1 : n_nodes <= 32 ? 2 : 4, WK = kWarps / WM;
    const int wm = warp % WM, wk = warp / WM;
    const int r0 = lane >> 2, c0 = (lane & 3) * 2;   // this lane's row (and r0 + 8) and first column of a fragment
    int tiles[2] = {(parts[0].n + kTile - 1) / kTile, n_parts > 1 ? (parts[1].n + kTile - 1) / kTile : 0};
    const int n_tiles = tiles[0] + tiles[1];

    auto load = [&](int t) {
        const Keys &ks = parts[kLocal && t >= tiles[0] ? 1 : 0];
        const int k0 = (kLocal && t >= tiles[0] ? t - tiles[0] : t) * kTile;
        const __nv_bfloat16 *src[2];
        if (kLocal && ks.kind == kNodes) {
            src[0] = static_cast<const __nv_bfloat16 *>(p.node_rows);
            src[1] = src[0] + (size_t)p.N * D;
        } else {
            src[0] = static_cast<const __nv_bfloat16 *>(p.cache[0]);
            src[1] = static_cast<const __nv_bfloat16 *>(p.cache[1]);
        }
        const uint32_t dst = smem_u32(ring) + (t % kStages) * S::kStage;
        const int c = tid % S::kChunks;
#pragma unroll
        for (int r = tid / S::kChunks; r < kTile; r += S::kRowsAtOnce) {
            const bool in = k0 + r < ks.n;
            long long off = in ? key_offset(p, ks, b, h, k0 + r) : 0;
            const bool on = in && off >= 0;
            if (in && off < 0) sh.bad = 1;
            if (!on) off = 0;
            cp_async16(dst + S::at(r, c), src[0] + off + c * 8, on);
            cp_async16(dst + S::kHalf + S::at(r, c), src[1] + off + c * 8, on);
        }
    };

    if (tid == 0) sh.bad = 0;
    if (tid < 3) sh.odd[tid] = 0;
    __syncthreads();
#pragma unroll
    for (int t = 0; t < kStages - 1; ++t) {
        if (t < n_tiles) load(t);
        cp_commit();
    }
    // the warp's nodes: rows of Q as A fragments
    uint32_t q[D / 16][4];
    int node[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int r = wm * 16 + r0 + 8 * u;
        node[u] = r < n_nodes ? sh.nodes[r] : -1;
        const uint32_t *src = reinterpret_cast<const uint32_t *>(
            static_cast<const __nv_bfloat16 *>(p.q) + (((size_t)b * p.N + max(node[u], 0)) * p.H + h) * D);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            q[k][u] = node[u] >= 0 ? src[k * 8 + (lane & 3)] : 0u;
            q[k][u + 2] = node[u] >= 0 ? src[k * 8 + 4 + (lane & 3)] : 0u;
        }
    }
    int dep[2] = {0, 0};
    unsigned long long anc[2] = {0ull, 0ull};
    if (kLocal) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
            if (node[u] >= 0) {
                dep[u] = sh.ti.depth[node[u]];
                anc[u] = sh.ti.anc[node[u]];
            }
    }
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};   // references, this lane's part of the sums

    for (int t = 0; t < n_tiles; ++t) {
        cp_wait<kStages - 2>();
        const uint8_t *kt = ring + (t % kStages) * S::kStage;
        const Keys &ks = parts[kLocal && t >= tiles[0] ? 1 : 0];
        const int k0 = (kLocal && t >= tiles[0] ? t - tiles[0] : t) * kTile;
        if (kLocal) {
            // values that are not finite leave the tile (their keys are noted):
            // a zero probability times one of them would reach every node
            uint4 *v = reinterpret_cast<uint4 *>(const_cast<uint8_t *>(kt) + S::kHalf);
            const int c = tid % S::kChunks;
#pragma unroll 1
            for (int r = tid / S::kChunks; r < kTile; r += S::kRowsAtOnce) {
                uint4 *e = v + S::at(r, c) / 16;
                uint4 x = *e;
                if (not_finite2(x.x) || not_finite2(x.y) || not_finite2(x.z) || not_finite2(x.w)) {
                    uint32_t w[4] = {x.x, x.y, x.z, x.w};
                    for (int i = 0; i < 4; ++i) {
                        if ((w[i] & 0x7f80u) == 0x7f80u) w[i] &= 0xffff0000u;
                        if ((w[i] & 0x7f800000u) == 0x7f800000u) w[i] &= 0x0000ffffu;
                    }
                    *e = make_uint4(w[0], w[1], w[2], w[3]);
                    atomicOr(&sh.odd[t % 3], 1ull << r);
                }
            }
        }
        __syncthreads();   // the tile has landed for everyone, and the one before is done with
        if (t + kStages - 1 < n_tiles) load(t + kStages - 1);
        cp_commit();
        if (kLocal && tid == 0) sh.odd[(t + 2) % 3] = 0;   // read for tile t - 1, next set after tile t + 1's barrier
        const uint32_t sk = smem_u32(kt), sv = sk + S::kHalf;
        for (int kb = wk; kb < kTile / 16; kb += WK) {
            if (k0 + kb * 16 >= ks.n) break;
            float s[2][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) s[0][j] = s[1][j] = 0.f;
            // lane's row of the four 8 x 8 matrices: keys 0-7 / 8-15 by chunk
            const int kr = kb * 16 + (lane & 7) + ((lane >> 4) << 3), kc = (lane >> 3) & 1;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                uint32_t f[4];
                ldsm4(f, sk + S::at(kr, 2 * k + kc));
                mma16816(s[0], q[k], f[0], f[1]);
                mma16816(s[1], q[k], f[2], f[3]);
            }
            // s[n][2u + j]: node row r0 + 8u, key kb * 16 + 8n + c0 + j
            float cnt[2][4];
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int key = k0 + kb * 16 + 8 * n + c0 + j;
                        float w = key < ks.n ? 1.f : 0.f;
                        if (kLocal) w = node[u] < 0 ? 0.f : (float)key_count(p, ks, sh.ti, h, pos, dep[u], anc[u], node[u], key);
                        cnt[n][2 * u + j] = w;
                        s[n][2 * u + j] = w > 0.f ? s[n][2 * u + j] * p.scale_log2 : -INFINITY;
                        mx[u] = fmaxf(mx[u], s[n][2 * u + j]);
                    }
            if (__any_sync(0xffffffffu, mx[0] > m[0] + kSlack || mx[1] > m[1] + kSlack)) {
                // some node's reference is raised (the first keys always do)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 1));
                    mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 2));
                    if (mx[u] > m[u] + kSlack) {
                        const float corr = exp2f(m[u] - mx[u]);   // 0 from a reference of -inf
                        m[u] = mx[u];
                        l[u] *= corr;
#pragma unroll
                        for (int i = 0; i < D / 8; ++i) {
                            o[i][2 * u] *= corr;
                            o[i][2 * u + 1] *= corr;
                        }
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float ref = m[u] == -INFINITY ? 0.f : m[u];   // scores of -inf weigh nothing, NaN stays NaN
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float &x = s[n][2 * u + j];
                        x = exp2f(x - ref);
                        if (kLocal) x = cnt[n][2 * u + j] > 0.f ? x * cnt[n][2 * u + j] : 0.f;
                        l[u] += x;
                    }
            }
            const uint32_t pa[4] = {pack2(s[0][0], s[0][1]), pack2(s[0][2], s[0][3]), pack2(s[1][0], s[1][1]),
                                    pack2(s[1][2], s[1][3])};
            const int vr = kb * 16 + (lane & 15), vc = lane >> 4;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                uint32_t f[4];
                ldsm4t(f, sv + S::at(vr, 2 * i + vc));
                mma16816(o[2 * i], pa, f[0], f[1]);
                mma16816(o[2 * i + 1], pa, f[2], f[3]);
            }
            if (kLocal) {
                unsigned odd = (unsigned)(sh.odd[t % 3] >> (kb * 16)) & 0xffffu;
                while (odd) {
                    // rare: the values left out above, for the nodes that see their key
                    const int key = __ffs(odd) - 1;
                    odd &= odd - 1;
                    const long long off = key_offset(p, ks, b, h, k0 + kb * 16 + key);
                    const __nv_bfloat16 *v = ks.kind == kNodes
                                                 ? static_cast<const __nv_bfloat16 *>(p.node_rows) + (size_t)p.N * D + off
                                                 : static_cast<const __nv_bfloat16 *>(p.cache[1]) + off;
                    const int from = (lane & ~3) | ((key & 7) >> 1);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const float lo = __shfl_sync(0xffffffffu, key < 8 ? s[0][2 * u] : s[1][2 * u], from);
                        const float hi = __shfl_sync(0xffffffffu, key < 8 ? s[0][2 * u + 1] : s[1][2 * u + 1], from);
                        const float pr = (key & 1) ? hi : lo;
#pragma unroll
                        for (int i = 0; i < D / 8; ++i)
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const float x = __bfloat162float(v[i * 8 + c0 + j]);
                                if (pr != 0.f && !(fabsf(x) < INFINITY)) o[i][2 * u + j] += pr * x;
                            }
                    }
                }
            }
        }
    }

    // join the warps that hold the same nodes, then write the partial
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        l[u] += __shfl_xor_sync(0xffffffffu, l[u], 1);
        l[u] += __shfl_xor_sync(0xffffffffu, l[u], 2);
    }
    cp_wait<0>();
    __syncthreads();
    if (WK > 1) {
        float *so = reinterpret_cast<float *>(ring);   // [warp][16][D]
        if ((lane & 3) == 0) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                sh.m[warp][r0 + 8 * u] = m[u];
                sh.l[warp][r0 + 8 * u] = l[u];
            }
        }
        __syncthreads();
        float w[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float M = -INFINITY;
            for (int x = 0; x < WK; ++x) M = fmaxf(M, sh.m[x * WM + wm][r0 + 8 * u]);
            w[u] = m[u] == -INFINITY ? (l[u] == 0.f ? 0.f : 1.f) : exp2f(m[u] - M);
            float L = 0.f;
            for (int x = 0; x < WK; ++x) {
                const float mm = sh.m[x * WM + wm][r0 + 8 * u], ll = sh.l[x * WM + wm][r0 + 8 * u];
                L += mm == -INFINITY ? ll : ll * exp2f(mm - M);   // -inf: nothing seen (0), or NaN
            }
            m[u] = M;
            l[u] = L;
        }
        if (wk > 0) {
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    // row-wise rotation by 8 floats a row keeps the lanes of a store on different banks
                    const int r = r0 + 8 * u, c = (i * 8 + c0 + 8 * r) % D;
                    *reinterpret_cast<float2 *>(so + (warp * 16 + r) * D + c) = make_float2(o[i][2 * u] * w[u], o[i][2 * u + 1] * w[u]);
                }
        }
        __syncthreads();
        if (wk == 0) {
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int r = r0 + 8 * u, c = (i * 8 + c0 + 8 * r) % D;
                    float x = o[i][2 * u] * w[u], y = o[i][2 * u + 1] * w[u];
                    for (int k = 1; k < WK; ++k) {
                        const float2 z = *reinterpret_cast<const float2 *>(so + ((k * WM + wm) * 16 + r) * D + c);
                        x += z.x;
                        y += z.y;
                    }
                    o[i][2 * u] = x;
                    o[i][2 * u + 1] = y;
                }
        }
    }
    if (wk == 0) {
        const size_t base = ((size_t)b * p.slots_per_b + p.slot0[h] + slot) * p.N;
        const bool bad = sh.bad != 0;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (node[u] < 0) continue;
            if ((lane & 3) == 0) p.ml[base + node[u]] = make_float2(m[u], bad ? -1.f : l[u]);
            float *dst = p.part + (base + node[u]) * D + c0;
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
                *reinterpret_cast<float2 *>(dst + i * 8) = make_float2(o[i][2 * u], o[i][2 * u + 1]);
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads) tree_mma_kernel(const TreeParams p) {
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ Shared sh;
    const int tid = threadIdx.x;
    const int b = blockIdx.x / p.ctas_per_b, it = blockIdx.x % p.ctas_per_b;
    const int h = find_tree_head(p, it), li = it - p.cta0[h];
    const int pos = p.pos[b];
    if (tid < 32) tree_analyse(sh.ti, p.parent + (size_t)b * p.N, p.N, pos, p.cap);
    else if (tid < 32 + kTreeMaxNodes) sh.parent[tid - 32] = tid - 32 < p.N ? p.parent[(size_t)b * p.N + tid - 32] : RAT_NODE_ABSENT;
    __syncthreads();
    if (!sh.ti.valid || sh.ti.max_depth < 0) {
        if (!sh.ti.valid && li == 0 && tid == 0) report_error(p.hdr, RAT_ERR_INVALID, b);
        return;
    }
    const int ws = p.wsplit[h];
    if (li < ws) {
        Keys parts[2];
        const int n = local_keys(p, h, pos, li, parts);
        if (li == 0) {
            run_tree<__nv_bfloat16, D, kThreads>(p, sh.parent, b, h, reinterpret_cast<float *>(ring));
            __threadfence();   // the copies of these rows go past L1
        }
        if (tid == 0) sh.n = p.N;
        if (tid < p.N) sh.nodes[tid] = tid;
        run_item<D, true>(p, sh, ring, parts, n, b, h, pos, p.nsplit[h] + li);
        return;
    }
    const int sets = tree_num_sets(p, p.dil[h], sh.ti.max_depth), items = sets * p.nsplit[h];
    for (int x = li - ws; x < items; x += p.slab_ctas[h]) {
        const int g = x % sets, piece = x / sets;
        Keys ks;
        if (!slab_keys(p, h, pos, g, piece, ks)) continue;
        __syncthreads();
        if (tid < 32) list_nodes(p, sh.ti, h, g, sh.nodes, &sh.n);
        run_item<D, false>(p, sh, ring, &ks, 1, b, h, pos, piece);
    }
}

template <int D> cudaError_t launch_typed(const TreeParams &p, unsigned grid, cudaStream_t s) {
    const size_t smem = kStages * (size_t)Shape<D>::kStage;
    static_assert((size_t)kStages * Shape<D>::kStage >= kTreeMaxNodes * kThreads * sizeof(float), "the recurrence's history fits");
    static_assert((size_t)kStages * Shape<D>::kStage >= kWarps * 16 * D * sizeof(float), "the warps' sums fit");
    static std::atomic<unsigned long long> smem_set{0};
    cudaError_t e = ensure_smem_limit(tree_mma_kernel<D>, smem, smem_set);
    if (e != cudaSuccess) return e;
    tree_mma_kernel<D><<<grid, kThreads, smem, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_mma(const TreeParams &p, unsigned grid, cudaStream_t s) {
    return p.d == 128 ? launch_typed<128>(p, grid, s) : launch_typed<64>(p, grid, s);
}

}  // namespace rat
