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
#include "attn_tc.cuh"
#include "tree_keys.cuh"

namespace rat {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 64;
constexpr int kStages = 3;
constexpr float kSlack = 8.f;   // log2 of how far P may pass 1

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
    // 16-byte chunk c of row r: halves of 64 channels, 128-byte swizzled as TMA writes them
    static __device__ __forceinline__ uint32_t at(int r, int c) { return (c >> 3) * (kTile * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4); }
};

// TMA maps of a dense cache; a paged one is copied row by row.
struct Maps {
    CUtensorMap kv[2];
};

struct Shared {
    TreeInfo ti;
    int parent[kTreeMaxNodes], nodes[kTreeMaxNodes];
    int n, bad, odd;                      // odd: some local value is not finite
    uint64_t full[kStages];               // a slab's tile has landed
    volatile int abort;
    uint8_t count[kTreeMaxNodes][kTile];  // how often a key of a masked tile counts for a node
    float m[kWarps][16], l[kWarps][16];
};

// One item: the keys of parts[0 .. n_parts), tile by tile, for the sh.n nodes of
// sh.nodes.  One body serves slabs and local items (what differs is where a row
// is and which tiles carry a mask): a second copy of it would only thrash the
// instruction cache.
// False when a wait gave up.
template <int D>
__device__ __forceinline__ bool run_item(const TreeParams &p, const Maps &maps, Shared &sh, uint8_t *ring, const Keys *parts,
                                         int n_parts, int b, int h, int pos, int slot, int &fills) {
    using S = Shape<D>;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    fence_async();     // what was written to the ring by ordinary stores, before TMA writes there
    __syncthreads();   // sh.n and sh.nodes are set, and the ring is free
    const int n_nodes = sh.n;
    const int WM = n_nodes <= 16 ? 1 : n_nodes <= 32 ? 2 : 4, WK = kWarps / WM;
    const int wm = warp % WM, wk = warp / WM;
    const int r0 = lane >> 2, c0 = (lane & 3) * 2;   // this lane's row (and r0 + 8) and first column of a fragment
    const int tiles0 = (parts[0].n + kTile - 1) / kTile;
    const int n_tiles = tiles0 + (n_parts > 1 ? (parts[1].n + kTile - 1) / kTile : 0);
    if (tid == 0) sh.bad = sh.odd = 0;
    const bool bulk = parts[0].kind == kSlab && !p.page_table;   // the item's tiles come by TMA
    const int fill0 = fills;                                     // such tiles before this item's
    if (bulk) fills += n_tiles;

    // Q into the stage that no tile uses yet
    const uint32_t sq = smem_u32(ring) + ((fill0 + kStages - 1) % kStages) * S::kStage;
    for (int e = tid; e < WM * 16 * S::kChunks; e += kThreads) {
        const int r = e / S::kChunks, c = e % S::kChunks;
        const bool on = r < n_nodes;
        const int n = on ? sh.nodes[r] : 0;
        cp_async16(sq + S::at(r, c), static_cast<const __nv_bfloat16 *>(p.q) + (((size_t)b * p.N + n) * p.H + h) * D + c * 8, on);
    }
    cp_commit();
    auto load = [&](int t) {
        if (bulk) {
            if (tid == 0) {
                const int f = fill0 + t, y = (int)parts[0].row0 + t * kTile;
                uint64_t *bar = &sh.full[f % kStages];
                const uint32_t dst = smem_u32(ring) + (f % kStages) * S::kStage;
                mbar_expect(bar, S::kStage);
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int half = 0; half < D / 64; ++half)
                        tma_load(dst + x * S::kHalf + half * (kTile * 128), &maps.kv[x], bar, half * 64, y, b * p.H + h);
            }
            return;
        }
        const bool second = t >= tiles0;
        const Keys &ks = parts[second ? 1 : 0];
        const int k0 = (second ? t - tiles0 : t) * kTile;
        const __nv_bfloat16 *kb = static_cast<const __nv_bfloat16 *>(p.cache[0]), *vb = static_cast<const __nv_bfloat16 *>(p.cache[1]);
        if (ks.kind == kNodes) {
            kb = static_cast<const __nv_bfloat16 *>(p.node_rows);
            vb = kb + (size_t)p.N * D;
        }
        // a warp copies 16 rows; lane i finds the place of the i-th of them
        constexpr int kPerPass = 32 / S::kChunks;   // rows of a warp in one pass
        const int mine = (lane & 15) / kPerPass * S::kRowsAtOnce + warp * kPerPass + (lane & 15) % kPerPass;
        long long off = -1;
        if (k0 + mine < ks.n) {
            off = key_offset(p, ks, b, h, k0 + mine);
            if (off < 0) sh.bad = 1;
        }
        const uint32_t dst = smem_u32(ring) + ((fill0 + t) % kStages) * S::kStage;
        const int c = lane % S::kChunks;
#pragma unroll
        for (int i = 0; i < 16 / kPerPass; ++i) {
            const long long o = __shfl_sync(0xffffffffu, off, i * kPerPass + lane / S::kChunks);
            const int r = i * S::kRowsAtOnce + warp * kPerPass + lane / S::kChunks;
            const long long e = o < 0 ? 0 : o + c * 8;
            cp_async16(dst + S::at(r, c), kb + e, o >= 0);
            cp_async16(dst + S::kHalf + S::at(r, c), vb + e, o >= 0);
        }
    };
    __syncthreads();
#pragma unroll 1
    for (int t = 0; t < kStages - 1; ++t) {
        if (t < n_tiles) load(t);
        cp_commit();
    }
    cp_wait<kStages - 1>();
    __syncthreads();
    uint32_t q[D / 16][4];   // the warp's nodes: rows of Q as A fragments
#pragma unroll
    for (int k = 0; k < D / 16; ++k) ldsm4(q[k], sq + S::at(wm * 16 + (lane & 15), 2 * k + (lane >> 4)));
    fence_async();     // Q's stage is a tile's next
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
    bool ok = true;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};   // references, this lane's part of the sums

#pragma unroll 1
    for (int t = 0; t < n_tiles; ++t) {
        const int f = fill0 + t;
        uint8_t *stage = ring + (f % kStages) * S::kStage;
        if (bulk) ok = mbar_wait(&sh.full[f % kStages], (f / kStages) & 1, &sh.abort);
        else cp_wait<kStages - 2>();
        const uint32_t sk = smem_u32(stage), sv = sk + S::kHalf;
        const bool second = t >= tiles0;
        const Keys &ks = parts[second ? 1 : 0];
        const int k0 = (second ? t - tiles0 : t) * kTile;
        // nodes mask each other; the window's first keys are out of the deeper
        // nodes' reach; with dedupe any of its keys may be in the dilated set
        const bool local = ks.kind != kSlab;
        const bool masked = ks.kind == kNodes || (ks.kind == kWindow && (p.dedupe || k0 < sh.ti.max_depth));
        if (local) {
            // values that are not finite leave the tile: a zero probability times
            // one of them would reach every node.  add_odd() puts them back
            __syncwarp();
            uint4 *v = reinterpret_cast<uint4 *>(stage + S::kHalf);
#pragma unroll 1
            for (int r = tid / S::kChunks; r < kTile; r += S::kRowsAtOnce) {
                uint4 *e = v + S::at(r, tid % S::kChunks) / 16;
                const uint4 x = *e;
                if (not_finite2(x.x) || not_finite2(x.y) || not_finite2(x.z) || not_finite2(x.w)) {
                    __nv_bfloat16 *w = reinterpret_cast<__nv_bfloat16 *>(e);
#pragma unroll 1
                    for (int i = 0; i < 8; ++i)
                        if (!(fabsf(__bfloat162float(w[i])) < INFINITY)) w[i] = __float2bfloat16_rn(0.f);
                    sh.odd = 1;
                }
            }
        }
        if (bulk && k0 + kTile > ks.n) {
            // rows behind the item's last hold anything: their values are zeroed
            uint4 *v = reinterpret_cast<uint4 *>(stage + S::kHalf);
#pragma unroll 1
            for (int r = tid / S::kChunks; r < kTile; r += S::kRowsAtOnce)
                if (k0 + r >= ks.n) v[S::at(r, tid % S::kChunks) / 16] = make_uint4(0u, 0u, 0u, 0u);
        }
        // the tile has landed for everyone, and the one before is done with
        if (!__syncthreads_and(ok)) {
            if (tid == 0) {
                report_error(p.hdr, RAT_ERR_TIMEOUT, (int)blockIdx.x);
                volatile int never = 0;
                for (int q = f; q < fill0 + min(n_tiles, t + kStages - 1); ++q)   // copies in flight
                    mbar_wait(&sh.full[q % kStages], (q / kStages) & 1, &never);
            }
            __syncthreads();
            return false;
        }
        if (masked) {
#pragma unroll 1
            for (int e = tid; e < n_nodes * kTile; e += kThreads) {
                const int i = e / kTile, key = k0 + e % kTile, dep = sh.ti.depth[i];
                sh.count[i][e % kTile] = dep < 0 ? 0 : key_count(p, ks, sh.ti, h, pos, dep, sh.ti.anc[i], i, key);
            }
            __syncthreads();
        }
        if (t + kStages - 1 < n_tiles) load(t + kStages - 1);
        cp_commit();
#pragma unroll 1
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
            if (masked) {
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int r = wm * 16 + r0 + 8 * u;
                        const uint16_t w = r < n_nodes ? *reinterpret_cast<const uint16_t *>(&sh.count[r][kb * 16 + 8 * n + c0]) : (uint16_t)0;
                        cnt[n][2 * u] = (float)(w & 0xff);
                        cnt[n][2 * u + 1] = (float)(w >> 8);
                    }
            } else {
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) cnt[n][j] = k0 + kb * 16 + 8 * n + c0 + (j & 1) < ks.n ? 1.f : 0.f;
            }
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[n][j] = cnt[n][j] > 0.f ? s[n][j] * p.scale_log2 : -INFINITY;
                    mx[j >> 1] = fmaxf(mx[j >> 1], s[n][j]);
                }
            if (__any_sync(0xffffffffu, mx[0] > m[0] + kSlack || mx[1] > m[1] + kSlack)) {
                // some node's reference is raised (the first keys always do)
                float corr[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 1));
                    mx[u] = fmaxf(mx[u], __shfl_xor_sync(0xffffffffu, mx[u], 2));
                    const bool up = mx[u] > m[u] + kSlack;
                    corr[u] = up ? exp2f(m[u] - mx[u]) : 1.f;   // 0 from a reference of -inf
                    m[u] = up ? mx[u] : m[u];
                    l[u] *= corr[u];
                }
#pragma unroll
                for (int i = 0; i < D / 8; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[i][j] *= corr[j >> 1];
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float ref = m[u] == -INFINITY ? 0.f : m[u];   // scores of -inf weigh nothing, NaN stays NaN
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int j = 2 * u; j < 2 * u + 2; ++j) {
                        s[n][j] = cnt[n][j] > 0.f ? cnt[n][j] * exp2f(s[n][j] - ref) : 0.f;
                        l[u] += s[n][j];
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
        }
    }

    // Join the warps that hold the same nodes: sums go to shared memory, scaled
    // to the common reference, and leave it row by row.
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        l[u] += __shfl_xor_sync(0xffffffffu, l[u], 1);
        l[u] += __shfl_xor_sync(0xffffffffu, l[u], 2);
        if ((lane & 3) == 0) {
            sh.m[warp][r0 + 8 * u] = m[u];
            sh.l[warp][r0 + 8 * u] = l[u];
        }
    }
    cp_wait<0>();
    __syncthreads();
    float *so = reinterpret_cast<float *>(ring);   // [warp][16][D], a row's columns turned by 8 r (banks)
    float M[2], L[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int r = r0 + 8 * u;
        M[u] = -INFINITY;
        L[u] = 0.f;
#pragma unroll 1
        for (int x = 0; x < WK; ++x) M[u] = fmaxf(M[u], sh.m[x * WM + wm][r]);
#pragma unroll 1
        for (int x = 0; x < WK; ++x) {
            const float mm = sh.m[x * WM + wm][r], ll = sh.l[x * WM + wm][r];
            L[u] += mm == -INFINITY ? ll : ll * exp2f(mm - M[u]);   // -inf: nothing seen (0), or NaN
        }
        const float w = m[u] == -INFINITY ? 1.f : exp2f(m[u] - M[u]);
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
            *reinterpret_cast<float2 *>(so + (warp * 16 + r) * D + (i * 8 + c0 + 8 * r) % D) = make_float2(o[i][2 * u] * w, o[i][2 * u + 1] * w);
    }
    __syncthreads();
    const size_t base = ((size_t)b * p.slots_per_b + p.slot0[h] + slot) * p.N;
    if (wk == 0 && (lane & 3) == 0) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int r = wm * 16 + r0 + 8 * u;
            if (r < n_nodes) p.ml[base + sh.nodes[r]] = make_float2(M[u], sh.bad ? -1.f : L[u]);
        }
    }
    if (sh.odd) {
        // the values left out: each reaches the nodes that see its key (the
        // probability's size does not matter to an infinity or a NaN)
#pragma unroll 1
        for (int c = tid; c < D; c += kThreads)
#pragma unroll 1
            for (int part = 0; part < n_parts; ++part)
#pragma unroll 1
                for (int i = 0; i < parts[part].n; ++i) {
                    const long long off = key_offset(p, parts[part], b, h, i);
                    if (off < 0) continue;
                    const __nv_bfloat16 *v = parts[part].kind == kNodes
                                                 ? static_cast<const __nv_bfloat16 *>(p.node_rows) + (size_t)p.N * D
                                                 : static_cast<const __nv_bfloat16 *>(p.cache[1]);
                    const float x = __bfloat162float(v[off + c]);
                    if (fabsf(x) < INFINITY) continue;
#pragma unroll 1
                    for (int n = 0; n < n_nodes; ++n)
                        if (sh.ti.depth[n] >= 0 && key_count(p, parts[part], sh.ti, h, pos, sh.ti.depth[n], sh.ti.anc[n], n, i))
                            so[n * D + (c + 8 * (n & 15)) % D] += x;
                }
        __syncthreads();
    }
#pragma unroll 2
    for (int e = tid; e < n_nodes * (D / 4); e += kThreads) {
        const int r = e / (D / 4), c = (e % (D / 4)) * 4;
        const float *src = so + r * D + (c + 8 * (r & 15)) % D;
        float4 x = *reinterpret_cast<const float4 *>(src);
#pragma unroll 1
        for (int k = 1; k < WK; ++k) {
            const float4 y = *reinterpret_cast<const float4 *>(src + k * WM * 16 * D);
            x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
        }
        *reinterpret_cast<float4 *>(p.part + (base + sh.nodes[r]) * D + c) = x;
    }
    return true;
}

template <int D>
__global__ void __launch_bounds__(kThreads) tree_mma_kernel(const TreeParams p, const __grid_constant__ Maps maps) {
    extern __shared__ uint8_t raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    __shared__ Shared sh;
    const int tid = threadIdx.x;
    allow_next();
    const int b = blockIdx.x / p.ctas_per_b, it = blockIdx.x % p.ctas_per_b;
    const int h = find_tree_head(p, it), li = it - p.cta0[h];
    const int pos = p.pos[b];
    if (tid == kThreads - 1) {
        for (int i = 0; i < kStages; ++i) mbar_init(&sh.full[i], 1);
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    int fills = 0;
    if (tid < 32) tree_analyse(sh.ti, p.parent + (size_t)b * p.N, p.N, pos, p.cap);
    else if (tid < 32 + kTreeMaxNodes) sh.parent[tid - 32] = tid - 32 < p.N ? p.parent[(size_t)b * p.N + tid - 32] : RAT_NODE_ABSENT;
    __syncthreads();
    if (li == 0) tell_pieces(p, sh.ti, b, h, pos);
    if (!sh.ti.valid || sh.ti.max_depth < 0) {
        if (!sh.ti.valid && li == 0 && tid == 0) report_error(p.hdr, RAT_ERR_INVALID, b);
        if (blockIdx.x == gridDim.x - 1) wait_previous();
        return;
    }
    const int ws = p.wsplit[h];
    const int sets = tree_num_sets(p, p.dil[h], sh.ti.max_depth), items = sets * p.nsplit[h];
    // CTAs below ws take one local item, the others slab items x, x + slab_ctas, ...
#pragma unroll 1
    for (int x = li < ws ? items - 1 : li - ws; x < items; x += max(1, p.slab_ctas[h])) {
        Keys parts[2];
        int n = 1, slot = x / sets;
        if (li < ws) {
            slot = p.nsplit[h] + li;
            n = local_keys(p, h, pos, li, parts);
            if (li == 0) run_tree<__nv_bfloat16, D>(p, sh.parent, b, h, ring);
            if (tid == 0) sh.n = p.N;
            if (tid < p.N) sh.nodes[tid] = tid;
        } else {
            if (!slab_keys(p, h, pos, x % sets, slot, parts[0])) continue;
            __syncthreads();
            if (tid < 32) list_nodes(p, sh.ti, h, x % sets, sh.nodes, &sh.n);
        }
        if (!run_item<D>(p, maps, sh, ring, parts, n, b, h, pos, slot, fills)) break;
    }
    // this kernel ends after the one before it (tree_tc.cu's part of the step),
    // so that the one after, which waits for this one, has both
    if (blockIdx.x == gridDim.x - 1) wait_previous();
}

template <int D> cudaError_t launch_typed(const TreeParams &p, unsigned grid, cudaStream_t s) {
    constexpr size_t kRing = kStages * (size_t)Shape<D>::kStage;
    static_assert(kRing >= kWarps * 16 * D * sizeof(float), "the warps' sums fit");
    const size_t smem = (kRing > tree_smem<D>(kTreeMaxNodes) ? kRing : tree_smem<D>(kTreeMaxNodes)) + 1024;
    static std::atomic<unsigned long long> smem_set{0};
    cudaError_t e = ensure_smem_limit(tree_mma_kernel<D>, smem, smem_set);
    if (e != cudaSuccess) return e;
    Maps maps = {};
    if (!p.page_table)
        for (int x = 0; x < 2; ++x)
            if (!encode_map_rows(&maps.kv[x], p.cache[x], p.cache_R, (long long)p.B * p.H, D, kTile)) return cudaErrorInvalidValue;
    return launch_after(tree_mma_kernel<D>, grid, kThreads, smem, s, p.n_tc > 0, p, maps);
}

}  // namespace

cudaError_t launch_tree_mma(const TreeParams &p, unsigned grid, cudaStream_t s) {
    return p.d == 128 ? launch_typed<128>(p, grid, s) : launch_typed<64>(p, grid, s);
}

}  // namespace rat
