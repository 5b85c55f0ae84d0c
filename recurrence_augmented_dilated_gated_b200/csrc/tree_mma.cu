// tree_mma.cu -- K7: the tree step's items (tree.cu) on the register-fragment
// tensor-core instructions, bf16 and fp32.
//
// An item is a run of cache rows and the nodes that read it: scores S = Q K~^T,
// probabilities P, sums O = P V~, with 16 nodes as the rows of one matrix
// instruction.  A node's rows of S and O stay in registers for the whole item;
// K~ and V~ rows pass through a ring of shared memory, by TMA from a dense
// cache, by 16-byte asynchronous copies row by row from pages, the window and
// the tree.
//   - up to 16 nodes: the four warps take different keys of a tile and join
//     their partial softmaxes at the end; up to 32: two by two; up to 64: a
//     warp for every 16 nodes.  So every warp works whatever the tree's shape.
//   - 16-byte chunk c of row r sits at chunk c ^ (r & 7) of its 128 bytes: the
//     eight rows of an ldmatrix fall on different banks.
//   - the softmax reference of a node is raised only when a score passes it by
//     more than 2^8 (P stays below 2^8, its sum in fp32): one vote per block of
//     keys instead of reductions and rescaling.
//   - bf16: m16n8k16.  P goes into the product with V~ in two bf16 halves (2^-17 of
//     each probability; kHalves), so that what remains of the error is the output's
//     own rounding, 1.7e-3.  An item of up to 8 nodes has the small ones in the free
//     rows 8-15 of the same instruction (64 x 32 nodes at 16K positions, D = 16, sets of
//     six: 537 us with one bf16, 531 so); with more nodes there is a second one.  For
//     d = 64 and more than 16 nodes the instructions are the time and P is one bf16
//     (half a step, 2^-9; error 2.3e-3), as in the prefill: 9 x 38 nodes, 28 dense heads
//     of 4012 rows 142 us, with second instructions 163 (d = 128 at 0.24 M rows, 48 nodes,
//     the most that tree_tc.cu leaves: 69 and 77).  The sum of P is of fp32 values.
//   - fp32: m16n8k8 on tf32 halves: x = b + s with b = x rounded to tf32 (11
//     bits) and s = x - b, of which the instruction takes 11 bits too; x y = b b' +
//     b s' + s b' leaves out s s' and what s was cut by, 2^-22 of the product.
// Bound: HBM for small node counts (a row's bytes serve 4 d operations a node);
// with more than 16 nodes on the same rows the instruction rate, which is why
// tree_tc.cu takes those where it can.
#include "tree_keys.cuh"

namespace rat {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kTileMax = 64;
constexpr int kStagesMax = 2;
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
__device__ __forceinline__ void mma1688(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x = big + small, big with the 11 bits of tf32 (the instruction cuts small to as many).
// kInf: an infinity is the largest tf32 and an infinite small part, so that a product
// of halves has its sign; else it is (infinity, NaN).  The conversion that saturates
// took 441 us where this one takes 411 (16 x 8 nodes, 16 heads of 4000 rows), so an
// item uses it when its sums came out not finite, and is taken again.
template <bool kInf> __device__ __forceinline__ void split(uint32_t x, uint32_t &big, uint32_t &small) {
    uint32_t b;
    if (kInf) asm("cvt.rna.satfinite.tf32.f32 %0, %1;" : "=r"(b) : "f"(__uint_as_float(x)));
    else asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(b) : "f"(__uint_as_float(x)));
    small = __float_as_uint(__uint_as_float(x) - __uint_as_float(b));
    big = b;
}
__device__ __forceinline__ uint32_t pack2(float x, float y) {
    __nv_bfloat162 t = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<uint32_t *>(&t);
}
template <typename T> __device__ __forceinline__ bool not_finite(uint32_t w) {   // any value in a word
    if (sizeof(T) == 4) return (w & 0x7f800000u) == 0x7f800000u;
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ float value(float x) { return x; }
__device__ __forceinline__ float value(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T, int D> struct Shape {
    static constexpr bool kF32 = sizeof(T) == 4;
    static constexpr int kTile = kF32 && D == 128 ? 32 : 64;   // rows of a stage
    static constexpr int kBlocks = kF32 ? kTile / 8 : 4;    // of kBlock keys
    static constexpr int kBlock = kTile / kBlocks;          // keys that a warp takes at a time
    static constexpr int kStages = 2;
    static constexpr int kPer = 16 / (int)sizeof(T);        // channels of a 16-byte chunk
    static constexpr int kChunks = D / kPer;                // chunks of a row
    static constexpr uint32_t kHalf = kTile * D * sizeof(T);   // K~ of a stage, then V~
    static constexpr uint32_t kStage = 2 * kHalf;
    static constexpr uint32_t kRing = kStages * kStage;
    static constexpr int kRowsAtOnce = kThreads / kChunks;  // rows that one pass of the CTA copies
    static constexpr int kWarpRows = kTile / kWarps;        // rows that a warp copies of a tile
    // 16-byte chunk c of row r of `rows`: 128-byte columns, swizzled as TMA writes them
    static __device__ __forceinline__ uint32_t at(int r, int c, int rows = kTile) {
        return (c >> 3) * (rows * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
    }
};

// TMA maps of a dense cache; a paged one is copied row by row.
struct Maps {
    CUtensorMap kv[2];
};

// Rows of Q that the warps read: 16 for one, two or four of them; and the bytes of
// an fp32 Q, in halves for up to 32 nodes.
__host__ __device__ __forceinline__ int padded_nodes(int n) { return n <= 16 ? 16 : n <= 32 ? 32 : 64; }
template <int D> constexpr size_t q_bytes(int n) { return (size_t)(n <= 16 ? 16 : 32) * D * 8; }

struct Shared {
    TreeInfo ti;
    alignas(16) int parent[kTreeMaxNodes];   // read four at a time
    int nodes[kTreeMaxNodes];
    int n, bad, odd;                      // odd: some local value is not finite
    uint64_t full[kStagesMax];              // a slab's tile has landed
    Waits waits;
    uint8_t count[kTreeMaxNodes][kTileMax];  // how often a key of a masked tile counts for a node
    float m[kWarps][16], l[kWarps][16];
    float inv[kTreeMaxNodes];
};

// key_count() of a tile: of nodes without branches and four at a time, so that what
// is read of them does not wait for what is written (64 nodes: 14600 -> 6000
// cycles); of n held rows of the window, `held` positions back from pos.  Out of
// line, as it would take registers from the item's loop.
template <int kTile>
__device__ __noinline__ void count_keys(Shared &sh, int n_nodes, int k0, bool nodes, int held, int n, int pos, int W, int D, int dedupe, int grid) {
    constexpr int kStep = kThreads / kTile;
    const int key = threadIdx.x % kTile;   // a thread has one key
    if (!nodes) {
        const int j = pos - held + k0 + key;
        const bool left_out = k0 + key >= n || (dedupe && grid && j % D == D - 1);
#pragma unroll 1
        for (int i = threadIdx.x / kTile; i < n_nodes; i += kStep) {
            const int dep = sh.ti.depth[i], back = pos + dep - j;
            sh.count[i][key] = !(left_out || dep < 0 || back >= W || (dedupe && !grid && back % D == 0));
        }
        return;
    }
    const int k = min(k0 + key, kTreeMaxNodes - 1), kd = sh.ti.depth[k];
    const unsigned *half = reinterpret_cast<const unsigned *>(sh.ti.anc) + (k >> 5);   // the word with the key's bit
    const unsigned bit = 1u << (k & 31), far_lo = (unsigned)sh.ti.far, far_hi = (unsigned)(sh.ti.far >> 32);
    const bool far_key = (k < 32 ? far_lo : far_hi) & bit;
#pragma unroll 1
    for (int i0 = threadIdx.x / kTile; i0 < n_nodes; i0 += 4 * kStep) {
        int cnt[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const int i = min(i0 + w * kStep, n_nodes - 1), back = sh.ti.depth[i] - kd;
            const bool far = grid ? i == k || far_key : ((back < 32 ? far_lo : far_hi) >> (back & 31)) & 1u;
            const bool near = back < W && !(dedupe && far);
            cnt[w] = half[2 * i] & bit ? (int)far + (int)near : 0;
        }
#pragma unroll
        for (int w = 0; w < 4; ++w)
            if (i0 + w * kStep < n_nodes) sh.count[i0 + w * kStep][key] = (uint8_t)cnt[w];
    }
}

// One item: the keys of parts[0 .. n_parts), tile by tile, for the sh.n nodes of
// sh.nodes.  One body serves slabs and local items (what differs is where a row
// is and which tiles carry a mask): a second copy of it would only thrash the
// instruction cache.
enum ItemEnd { kDone, kGaveUp, kAgain };   // a wait gave up; nothing written, to be taken again with kInf
template <typename T, int D, bool kHalves, bool kInf>
__device__ __forceinline__ ItemEnd run_item(const TreeParams &p, const Maps &maps, Shared &sh, uint8_t *ring, const Keys *parts,
                                         int n_parts, int b, int h, int pos, int slot, int &fills) {
    using S = Shape<T, D>;
    constexpr int kTile = S::kTile, kStages = S::kStages, kBlock = S::kBlock, NB = kBlock / 8;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    fence_async();     // what was written to the ring by ordinary stores, before TMA writes there
    __syncthreads();   // sh.n and sh.nodes are set, and the ring is free
    const int n_nodes = sh.n;
    const int WM = padded_nodes(n_nodes) / 16, WK = kWarps / WM;
    const int wm = warp % WM, wk = warp / WM;
    const int r0 = lane >> 2, c0 = (lane & 3) * 2;   // this lane's row (and r0 + 8) and first column of a fragment
    const bool few = kHalves && n_nodes <= 8;        // rows 8-15 hold the small halves of P
    // tiles of the parts, one part after the other
    const int end0 = n_parts > 0 ? (parts[0].n + kTile - 1) / kTile : 0;
    const int end1 = end0 + (n_parts > 1 ? (parts[1].n + kTile - 1) / kTile : 0);
    const int n_tiles = end1 + (n_parts > 2 ? (parts[2].n + kTile - 1) / kTile : 0);
    auto part_of = [&](int t, int &k0) -> const Keys & {
        const int i = (t >= end0) + (t >= end1);
        k0 = (t - (i == 0 ? 0 : i == 1 ? end0 : end1)) * kTile;
        return parts[i];
    };
    if (tid == 0) sh.bad = sh.odd = 0;
    const int bulk = n_parts > 0 && parts[0].kind == kSlab && !p.page_table ? end0 : 0;   // tiles that come by TMA
    const int fill0 = fills;                                                              // such tiles before this item's
    fills += bulk;

    // Q: into the stage that no tile uses yet (bf16: it goes on to registers), or
    // a place of its own (fp32: in halves it would be 128 registers; the halves of
    // up to 32 nodes are made once, those of 64 nodes as they are used, so that
    // the place stays within 32 KB and two CTAs within an SM)
    const uint32_t sq = smem_u32(ring) + (S::kF32 ? S::kRing : ((fill0 + kStages - 1) % kStages) * S::kStage);
    const int q_rows = S::kF32 ? 16 * WM : kTreeMaxNodes;
    const bool halves = S::kF32 && WM < 4;
    for (int e = tid; e < WM * 16 * S::kChunks; e += kThreads) {
        const int r = e / S::kChunks, c = e % S::kChunks;
        const bool on = r < n_nodes;
        const int n = on ? sh.nodes[r] : 0;
        cp_async16(sq + S::at(r, c, q_rows), static_cast<const T *>(p.q) + (((size_t)b * p.N + n) * p.H + h) * D + c * S::kPer, on);
    }
    cp_commit();
    auto load = [&](int t) {
        if (t < bulk) {
            if (tid == 0) {
                const int f = fill0 + t, y = (int)parts[0].row0 + t * kTile;
                uint64_t *bar = &sh.full[f % kStages];
                const uint32_t dst = smem_u32(ring) + (f % kStages) * S::kStage;
                mbar_expect(bar, S::kStage);
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int col = 0; col < S::kChunks / 8; ++col)
                        tma_load(dst + x * S::kHalf + col * (kTile * 128), &maps.kv[x], bar, col * 8 * S::kPer, y, b * p.H + h);
            }
            return;
        }
        int k0;
        const Keys &ks = part_of(t, k0);
        const T *kb = static_cast<const T *>(p.cache[0]), *vb = static_cast<const T *>(p.cache[1]);
        if (ks.kind == kNodes) {
            kb = static_cast<const T *>(p.node_rows);
            vb = kb + (size_t)p.N * D;
        }
        // a warp copies kWarpRows rows; lane i finds the place of the i-th of them
        constexpr int kPerPass = 32 / S::kChunks;   // rows of a warp in one pass
        const int li = lane % S::kWarpRows, mine = li / kPerPass * S::kRowsAtOnce + warp * kPerPass + li % kPerPass;
        long long off = -1;
        if (k0 + mine < ks.n) {
            off = key_offset(p, ks, b, h, k0 + mine);
            if (off < 0) sh.bad = 1;
        }
        const uint32_t dst = smem_u32(ring) + ((fill0 + t) % kStages) * S::kStage;
        const int c = lane % S::kChunks;
#pragma unroll
        for (int i = 0; i < S::kWarpRows / kPerPass; ++i) {
            const long long o = __shfl_sync(0xffffffffu, off, i * kPerPass + lane / S::kChunks);
            const int r = i * S::kRowsAtOnce + warp * kPerPass + lane / S::kChunks;
            const long long e = o < 0 ? 0 : o + c * S::kPer;
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
    const uint32_t sq_small = sq + q_rows * D * 4;   // fp32: Q in halves, the small ones behind the big
    if (halves) {
        uint4 *x = reinterpret_cast<uint4 *>(ring + S::kRing);
        for (int e = tid; e < WM * 16 * S::kChunks; e += kThreads) {
            uint4 *big = x + S::at(e / S::kChunks, e % S::kChunks, q_rows) / 16, *small = big + q_rows * D / 4;
            const uint4 v = *big;
            split<kInf>(v.x, big->x, small->x);
            split<kInf>(v.y, big->y, small->y);
            split<kInf>(v.z, big->z, small->z);
            split<kInf>(v.w, big->w, small->w);
        }
        __syncthreads();
    }
    uint32_t q[S::kF32 ? 1 : D / 16][4];   // bf16: the warp's nodes, rows of Q as A fragments
    // rows 0-7 / 8-15 of a fragment by chunk
    const int qr = wm * 16 + (lane & 15), qc = lane >> 4;
    if constexpr (!S::kF32) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) ldsm4(q[k], sq + S::at(qr, 2 * k + qc, q_rows));
    }
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
        if (t < bulk) ok = mbar_wait(&sh.full[f % kStages], (f / kStages) & 1, &sh.waits);
        else cp_wait<kStages - 2>();
        const uint32_t sk = smem_u32(stage), sv = sk + S::kHalf;
        int k0;
        const Keys &ks = part_of(t, k0);
        // nodes mask each other; the window's first keys are out of the deeper
        // nodes' reach; with dedupe any of its keys may be in the dilated set
        const bool masked = ks.kind == kNodes || (ks.kind == kWindow && (p.dedupe || k0 < sh.ti.max_depth));
        if (masked) {
            // values that are not finite leave the tile: a zero probability times
            // one of them would reach every node.  add_odd() puts them back
            __syncwarp();
            uint4 *v = reinterpret_cast<uint4 *>(stage + S::kHalf);
#pragma unroll 1
            for (int r = tid / S::kChunks; r < kTile; r += S::kRowsAtOnce) {
                uint4 *e = v + S::at(r, tid % S::kChunks) / 16;
                const uint4 x = *e;
                if (not_finite<T>(x.x) || not_finite<T>(x.y) || not_finite<T>(x.z) || not_finite<T>(x.w)) {
                    T *w = reinterpret_cast<T *>(e);
#pragma unroll 1
                    for (int i = 0; i < S::kPer; ++i)
                        if (!(fabsf(value(w[i])) < INFINITY)) store1(w + i, 0.f);
                    sh.odd = 1;
                }
            }
        }
        if (t < bulk && k0 + kTile > ks.n) {
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
                static_assert(kStages == 2, "this tile's copies are the only ones in flight");
                mbar_drain(&sh.full[f % kStages], (f / kStages) & 1);
            }
            cp_wait<0>();
            __syncthreads();
            return kGaveUp;
        }
        if (masked) {
            count_keys<kTile>(sh, n_nodes, k0, ks.kind == kNodes, pos - (int)ks.row0, ks.n, pos, p.head[h].win, p.head[h].dil, p.dedupe, p.grid);
            __syncthreads();
        }
        if (t + kStages - 1 < n_tiles) load(t + kStages - 1);
        cp_commit();
#pragma unroll 1
        for (int kb = wk; kb < kTile / kBlock; kb += WK) {
            if (k0 + kb * kBlock >= ks.n) break;
            float s[NB][4];
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[n][j] = 0.f;
            if constexpr (!S::kF32) {
                // lane's row of the four 8 x 8 matrices: keys 0-7 / 8-15 by chunk
                const int kr = kb * 16 + (lane & 7) + ((lane >> 4) << 3), kc = (lane >> 3) & 1;
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    uint32_t f[4];
                    ldsm4(f, sk + S::at(kr, 2 * k + kc));
                    mma16816(s[0], q[k], f[0], f[1]);
                    mma16816(s[1], q[k], f[2], f[3]);
                }
            } else {
                // two steps of 8 channels: four chunks of the block's 8 keys.  Each
                // product of halves and each step has sums of its own: short chains
                // of instructions, and few roundings of the instruction's (which cut)
                const int kr = kb * 8 + (lane & 7), kc = lane >> 3;
                float part[2][3][4] = {};
#pragma unroll 2
                for (int k = 0; k < D / 16; ++k) {
                    uint32_t f[4];
                    ldsm4(f, sk + S::at(kr, 4 * k + kc));
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        uint32_t ab[4], as[4], bb[2], bs[2];
                        ldsm4(ab, sq + S::at(qr, 4 * k + 2 * y + qc, q_rows));
                        if (halves) {
                            ldsm4(as, sq_small + S::at(qr, 4 * k + 2 * y + qc, q_rows));
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i) split<kInf>(ab[i], ab[i], as[i]);
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i) split<kInf>(f[2 * y + i], bb[i], bs[i]);
                        mma1688(part[y][0], ab, bb[0], bb[1]);
                        mma1688(part[y][1], as, bb[0], bb[1]);
                        mma1688(part[y][2], ab, bs[0], bs[1]);
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    s[0][j] = (part[0][0][j] + part[1][0][j]) + ((part[0][1][j] + part[1][1][j]) + (part[0][2][j] + part[1][2][j]));
            }
            // s[n][2u + j]: node row r0 + 8u, key kb * kBlock + 8n + c0 + j
            float cnt[NB][4];
            if (masked) {
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int r = wm * 16 + r0 + 8 * u;
                        const uint16_t w = r < n_nodes ? *reinterpret_cast<const uint16_t *>(&sh.count[r][kb * kBlock + 8 * n + c0]) : (uint16_t)0;
                        cnt[n][2 * u] = (float)(w & 0xff);
                        cnt[n][2 * u + 1] = (float)(w >> 8);
                    }
            } else {
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) cnt[n][j] = k0 + kb * kBlock + 8 * n + c0 + (j & 1) < ks.n ? 1.f : 0.f;
            }
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int n = 0; n < NB; ++n)
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
                if (few) corr[1] = corr[0];
#pragma unroll
                for (int i = 0; i < D / 8; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[i][j] *= corr[j >> 1];
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float ref = m[u] == -INFINITY ? 0.f : m[u];   // scores of -inf weigh nothing, NaN stays NaN
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int j = 2 * u; j < 2 * u + 2; ++j) {
                        s[n][j] = cnt[n][j] > 0.f ? cnt[n][j] * exp2f(s[n][j] - ref) : 0.f;
                        l[u] += s[n][j];
                    }
            }
            if constexpr (!S::kF32) {
                uint32_t pa[4], pb[4];   // P: bf16 halves, or one bf16
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = s[i >> 1][2 * (i & 1)], y = s[i >> 1][2 * (i & 1) + 1];
                    if (kHalves) p_halves(x, y, pa[i], pb[i]);
                    else pa[i] = pack2(x, y);
                }
                if (few) {
                    pa[1] = pb[0];
                    pa[3] = pb[2];
                }
                const int vr = kb * 16 + (lane & 15), vc = lane >> 4;
#pragma unroll
                for (int i = 0; i < D / 16; i += 2) {
                    // two chunks at a time: instructions on the same sums are four apart
                    uint32_t f[4], e[4];
                    ldsm4t(f, sv + S::at(vr, 2 * i + vc));
                    ldsm4t(e, sv + S::at(vr, 2 * i + 2 + vc));
                    mma16816(o[2 * i], pa, f[0], f[1]);
                    mma16816(o[2 * i + 1], pa, f[2], f[3]);
                    mma16816(o[2 * i + 2], pa, e[0], e[1]);
                    mma16816(o[2 * i + 3], pa, e[2], e[3]);
                    if (!kHalves || few) continue;
                    mma16816(o[2 * i], pb, f[0], f[1]);
                    mma16816(o[2 * i + 1], pb, f[2], f[3]);
                    mma16816(o[2 * i + 2], pb, e[0], e[1]);
                    mma16816(o[2 * i + 3], pb, e[2], e[3]);
                }
            } else {
                // the instruction's key index x is key 2 x, x + 4 key 2 x + 1: P's own order
                uint32_t ab[4], as[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) split<false>(__float_as_uint(s[0][(i >> 1) + 2 * (i & 1)]), ab[i], as[i]);
                const int vr = kb * 8 + c0;
                const uint8_t *v = stage + S::kHalf + ((lane >> 2) & 3) * 4;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    const int c = 2 * i + (lane >> 4);
                    float t[4] = {};
                    uint32_t bb[2], bs[2];
                    split<kInf>(*reinterpret_cast<const uint32_t *>(v + S::at(vr, c)), bb[0], bs[0]);
                    split<kInf>(*reinterpret_cast<const uint32_t *>(v + S::at(vr + 1, c)), bb[1], bs[1]);
                    mma1688(t, as, bb[0], bb[1]);
                    mma1688(t, ab, bs[0], bs[1]);
                    mma1688(t, ab, bb[0], bb[1]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[i][j] += t[j];
                }
            }
        }
    }

    if (few) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
            o[i][0] += o[i][2];
            o[i][1] += o[i][3];
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
    if constexpr (S::kF32 && !kInf) {
        // a sum that is not finite, of a node that is there
        bool odd = false;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float z = l[u] * 0.f;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) z = fmaf(o[i][2 * u], 0.f, fmaf(o[i][2 * u + 1], 0.f, z));
            const int r = wm * 16 + r0 + 8 * u;
            odd |= z != z && r < n_nodes && sh.ti.depth[sh.nodes[min(r, kTreeMaxNodes - 1)]] >= 0;
        }
        if (__syncthreads_or(odd)) return kAgain;
    } else {
        __syncthreads();
    }
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
    const size_t base = ((size_t)b * p.slots_per_b + p.head[h].slot0 + slot) * p.N;
    const bool fused = p.head[h].fused != 0;
    if (wk == 0 && (lane & 3) == 0) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int r = wm * 16 + r0 + 8 * u;
            if (r >= n_nodes) continue;
            if (!fused) {
                p.ml[base + sh.nodes[r]] = make_float2(M[u], sh.bad ? -1.f : L[u]);
            } else {
                // the result itself: absent nodes and a pair with an invalid page are zero
                const float sum = sh.bad || sh.ti.depth[r] < 0 ? 0.f : L[u];
                sh.inv[r] = sum == 0.f ? 0.f : 1.f / sum;
                if (p.lse) p.lse[((size_t)b * p.H + h) * p.N + r] = sum == 0.f ? -INFINITY : (M[u] + log2f(sum)) * 0.69314718055994531f;
            }
        }
    }
    if (fused) {
        if (sh.bad && tid == 0) report_error(p.hdr, RAT_ERR_INVALID, b);
        __syncthreads();
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
                    const T *v = parts[part].kind == kNodes ? static_cast<const T *>(p.node_rows) + (size_t)p.N * D
                                                            : static_cast<const T *>(p.cache[1]);
                    const float x = value(v[off + c]);
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
        if (!fused) {
            *reinterpret_cast<float4 *>(p.part + (base + sh.nodes[r]) * D + c) = x;
        } else {
            const float w = sh.inv[r];   // 0: nothing to give, whatever the sums hold
            x = w == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(x.x * w, x.y * w, x.z * w, x.w * w);
            IO4<T>::store(static_cast<T *>(p.o) + (((size_t)b * p.N + r) * p.H + h) * D + c, x);
        }
    }
    return kDone;
}

template <typename T, int D, bool kHalves>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 3 : 2) tree_mma_kernel(const TreeParams p, const __grid_constant__ Maps maps) {
    extern __shared__ uint8_t raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    __shared__ Shared sh;
    const int tid = threadIdx.x;
    allow_next();
    const int b = blockIdx.x / p.ctas_per_b, it = blockIdx.x % p.ctas_per_b;
    const int h = find_tree_head(p, it), li = it - p.head[h].cta0;
    if (li == 0) {
        TreeWalk<T, D>::stage(p, b, h, 0, ring);
        TreeWalk<T, D>::ask_queries(p, b, h);
    }
    const int pos = p.pos[b];
    WaitSettings waits = {};
    if (tid == kThreads - 1) {
        for (int i = 0; i < kStagesMax; ++i) mbar_init(&sh.full[i], 1);
        waits = start_waits(sh.waits, p.hdr);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    int fills = 0;
    if (tid < 32) {
        tree_analyse(sh.ti, p.parent + (size_t)b * p.N, p.N, pos, p.cap);
        __syncwarp();
        if (li < p.head[h].wsplit) tree_masks(p, sh.ti, h, pos);
    }
    if (tid >= 32 && tid < 32 + kTreeMaxNodes) sh.parent[tid - 32] = tid - 32 < p.N ? p.parent[(size_t)b * p.N + tid - 32] : RAT_NODE_ABSENT;
    __syncthreads();
    if (tid == kThreads - 1) set_waits(sh.waits, waits, &sh.full[0]);
    if (li == 0) tell_pieces(p, sh.ti, b, h, pos);
    if (!sh.ti.valid || sh.ti.max_depth < 0) {
        if (!sh.ti.valid && li == 0 && tid == 0) report_error(p.hdr, RAT_ERR_INVALID, b);
        cp_wait<0>();
        if (blockIdx.x == gridDim.x - 1) wait_previous();
        return;
    }
    const int ws = p.head[h].wsplit;
    const int sets = tree_num_sets(p, p.head[h].dil, sh.ti.max_depth), items = sets * p.head[h].nsplit;
    // CTAs below ws take one local item, the others slab items x, x + slab_ctas, ...
#pragma unroll 1
    for (int x = li < ws ? max(items, 1) - 1 : li - ws; x < items; x += max(1, p.head[h].slab_ctas)) {
        Keys parts[3];
        int n = 1, slot = x / sets;
        if (li < ws) {
            slot = p.head[h].nsplit + li;
            n = local_keys(p, h, pos, li, parts);
            if (li == 0) TreeWalk<T, D>::run(p, sh.parent, b, h, ring);
            if (tid == 0) sh.n = p.N;
            if (tid < p.N) sh.nodes[tid] = tid;
        } else {
            if (!slab_keys(p, h, pos, x % sets, slot, parts[0])) continue;
            __syncthreads();
            if (tid < 32) list_nodes(p, sh.ti, h, x % sets, sh.nodes, &sh.n);
        }
        ItemEnd end = run_item<T, D, kHalves, false>(p, maps, sh, ring, parts, n, b, h, pos, slot, fills);
        if constexpr (sizeof(T) == 4) {
            if (end == kAgain) end = run_item<T, D, kHalves, true>(p, maps, sh, ring, parts, n, b, h, pos, slot, fills);
        }
        if (end == kGaveUp) break;
    }
    // this kernel ends after the one before it (tree_tc.cu's part of the step),
    // so that the one after, which waits for this one, has both
    if (blockIdx.x == gridDim.x - 1) wait_previous();
}

template <typename T, int D, bool kHalves> cudaError_t launch_typed(const TreeParams &p, unsigned grid, cudaStream_t s) {
    using S = Shape<T, D>;
    static_assert(S::kRing >= kWarps * 16 * D * sizeof(float), "the warps' sums fit");
    static_assert(S::kTile <= kTileMax && S::kStages <= kStagesMax, "tile and ring as declared");
    const size_t ring = S::kRing + (S::kF32 ? q_bytes<D>(p.N) : 0), tree = TreeWalk<T, D>::bytes(p.N, p.sep);
    const size_t smem = (ring > tree ? ring : tree) + 1024;   // bf16: three CTAs an SM
    static std::atomic<unsigned long long> smem_set{0};
    // the limit is raised once per device, so to the largest tree's
    const size_t most = S::kRing + (S::kF32 ? q_bytes<D>(kTreeMaxNodes) : 0), most_tree = TreeWalk<T, D>::bytes(kTreeMaxNodes, 1);
    cudaError_t e = ensure_smem_limit(tree_mma_kernel<T, D, kHalves>, (most > most_tree ? most : most_tree) + 1024, smem_set, true);
    if (e != cudaSuccess) return e;
    Maps maps = {};
    if (!p.page_table)
        for (int x = 0; x < 2; ++x)
            if (!encode_map_rows(&maps.kv[x], p.cache[x], sizeof(T) == 4 ? RAT_F32 : RAT_BF16, p.cache_R, (long long)p.B * p.H, D, S::kTile))
                return cudaErrorInvalidValue;
    return launch_after(tree_mma_kernel<T, D, kHalves>, grid, kThreads, smem, s, p.n_tc > 0, p, maps);
}

}  // namespace

cudaError_t launch_tree_mma(const TreeParams &p, int dtype, unsigned grid, cudaStream_t s) {
    if (dtype == RAT_F32) return p.d == 128 ? launch_typed<float, 128, false>(p, grid, s) : launch_typed<float, 64, false>(p, grid, s);
    if (p.d == 128) return launch_typed<__nv_bfloat16, 128, true>(p, grid, s);
    return p.N <= 16 ? launch_typed<__nv_bfloat16, 64, true>(p, grid, s) : launch_typed<__nv_bfloat16, 64, false>(p, grid, s);
}

}  // namespace rat
