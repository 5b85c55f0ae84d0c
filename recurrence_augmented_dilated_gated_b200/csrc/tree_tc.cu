// tree_tc.cu -- K7 for heads whose nodes all read the same rows (D = 1, or the
// fixed grid) and whose tree is large: the held rows on the 5th-generation
// tensor cores (tcgen05 + TMEM), bf16 operands, d = 128.
//
// The products are taken transposed, so that the 128 rows of an instruction are
// always full however many nodes N a tree has:
//   S^T [128 keys x N] = K~ Q^T      (A = the K~ tile, B = the nodes' queries)
//   O^T [128 channels x N] += V~^T P^T   (A = the V~ tile read along its rows)
// Up to 32 nodes P is in two bf16 halves side by side (p_halves; N is then 2 N, and the
// sums are added when an item ends): what remains of the error is the output's own
// rounding, 1.7e-3 (4 x 24 nodes, 16 heads over 16000 rows 105 us, 106 with them).  For
// more, P is one bf16 (half a step, 2^-9 of each; 2.3e-3), as in the prefill: the small
// halves would take a slot of the ring and twice the softmax's instructions (16 x 64
// nodes 348 and 380).  The sum of P is of fp32 values in both.
// A thread of the softmax warps owns one key (a TMEM lane) and all its scores;
// the reference a node's scores are measured from is shared by all keys and
// raised, for the whole CTA, only when a score passes it by more than 2^8.  The
// sums of P stay in registers, a node's share of each key, and are added
// across the CTA once per item.
//
// One persistent CTA per SM walks over items (its runs of rows of one (b, h)):
//   warps 0-3  softmax: S^T from TMEM, P^T (bf16) to shared memory, at an item's
//              end O^T from TMEM to the item's partial; they also stage the next
//              item's queries once its last scores are in
//   warp 4     copies: K~ and V~ tiles (32 KB each) into a ring of four or six slots, by
//              TMA, 128-byte swizzled; a page is a box of its own.  (16-byte
//              asynchronous copies by two warps instead, for any page size, took
//              3.3 TB/s at N = 32.)
//   warp 5     TMEM owner; one lane issues the instructions: the scores of tile
//              t + 1 before the product of tile t, so that one runs during the
//              softmax of the other
// TMEM: S0 [0,64) S1 [64,128) O [128,192) columns.
// Bound: HBM.  128 rows take 64 KB, 2830 cycles of an SM's share of the memory
// bandwidth, against 512 of the tensor core and about 700 of the softmax at
// N = 64.
//
// Every wait is bounded (globaltimer); on expiry the CTA records
// RAT_ERR_TIMEOUT, drains its copies and instructions, frees its TMEM, exits.
#include <float.h>

#include "tmem_io.cuh"
#include "tree_copy.cuh"
#include "tree_keys.cuh"

namespace rat {

namespace {

constexpr int kSoftmax = 128;
constexpr int kThreads = kSoftmax + 64;
constexpr int kD = 128;
constexpr int kTile = 128;               // keys per tile
constexpr int kSlotsMax = 6;
constexpr uint32_t kHalf = kTile * 128;  // 64 channels of a tile: rows of 128 bytes
constexpr uint32_t kSlot = 2 * kHalf;    // a K~ or a V~ tile
// Four slots for up to 32 nodes: beside them an SM has room for a CTA of
// tree_mma.cu (64 KB), which then does the windows and the nodes while this kernel
// streams (32 x 16 nodes on a paged grid 136 -> 121 us).  That takes no more than 168 registers a
// thread too, with which two of this kernel's warps and one of tree_mma.cu's fit in a quarter
// of the SM (4 x 24 nodes, 16 heads over 16000 rows 104 us, with 170 registers 119).  For 64 nodes Q leaves it no room, and six slots
// are 2 % faster than four.
template <int NP> struct Mem {
    static constexpr int kSlots = NP <= 32 ? 4 : kSlotsMax;
    static constexpr uint32_t kQHalf = NP * 128;
    static constexpr uint32_t kOffQ = kSlots * kSlot, kOffP = kOffQ + 2 * kQHalf, kBytes = kOffP + kTile * 128;
    static constexpr bool kHalves = NP <= 32;          // P in two halves
    static constexpr int kO = kHalves ? 2 * NP : NP;   // columns of P, and of O
};
constexpr int kTmemCols = 256;
constexpr float kSlack = 8.f;            // log2 of how far P may pass 1

__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}
// Shared-memory matrix descriptor: 128-byte swizzle, groups of eight 128-byte
// lines 1024 bytes apart; `lbo` is the distance of 64-element blocks for an
// operand that is contiguous along its rows (M or N), unused otherwise.
__device__ __forceinline__ uint64_t sdesc(uint32_t addr, uint32_t lbo) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// kind::f16, fp32 accumulation, bf16 operands, M = 128; `mn`: both operands are
// contiguous along M / N instead of along K.
__device__ __forceinline__ uint32_t idesc(int N, bool mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (mn ? 3u << 15 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
// two floats at once (f32x2 arithmetic: one instruction for both)
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t x, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// The softmax warps' barrier.  None of them leaves its loop early, however a
// wait ended, so every one of them comes here as often.
__device__ __forceinline__ void softmax_sync() { asm volatile("barrier.cta.sync 1, %0;" ::"n"(kSoftmax) : "memory"); }
__device__ __forceinline__ bool softmax_any(bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}\n"
        : "=r"(r) : "r"((uint32_t)x), "n"(kSoftmax) : "memory");
    return r != 0;
}

// What a CTA does: `tiles` tiles, the first `skip` of entry list[0] left out; n
// entries are listed, those behind them follow one by one.
constexpr int kList = 8;
struct Range {
    long long skip, tiles;
    int n, list[kList];
    long long sum[kThreads / 32];     // of a warp
    int count[kThreads / 32];
};

// All tiles of all pairs (b, h), in that order, are dealt out evenly: CTA c of G
// (of as many as there are tiles, if they are fewer) has tiles total * c / G ..
// total * (c + 1) / G - 1, whatever the positions.  (Pieces
// of equal length planned by the capacity left CTAs idle where entries are
// shorter: 16 x 64 nodes over 16000 dense rows 366 -> 333 us.)
// With many pairs (tree_plan) each is cut into pieces by the capacity, and the
// pieces go round: CTAs are then at neighbouring rows and heads, which for pages lie
// side by side (32 entries of 16 paged grid heads of 1800 rows: 124 us, even shares
// 128).
__device__ __forceinline__ int pair_tiles(const TreeParams &p, int i, int pos) {
    long long row0;
    return pos < 0 || pos > p.cap ? 0 : (tree_set_rows(p, p.tc_head[i], pos, 0, row0) + kTile - 1) / kTile;
}
__device__ __forceinline__ long long entry_tiles(const TreeParams &p, int b) {
    const int pos = p.pos[b];
    if (p.tc_same) return (long long)p.n_tc * pair_tiles(p, 0, pos);
    long long n = 0;
    for (int i = 0; i < p.n_tc; ++i) n += pair_tiles(p, i, pos);
    return n;
}
// Sums over the threads before this one, and over all of them (every thread).
__device__ __forceinline__ void scan_block(Range &r, long long v, int f, long long &v0, int &f0, long long &v_all, int &f_all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long x = v;
    int y = f;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long a = __shfl_up_sync(0xffffffffu, x, off);
        const int c = __shfl_up_sync(0xffffffffu, y, off);
        if (lane >= off) {
            x += a;
            y += c;
        }
    }
    __syncthreads();   // the sums before are read
    if (lane == 31) {
        r.sum[warp] = x;
        r.count[warp] = y;
    }
    __syncthreads();
    v0 = x - v;
    f0 = y - f;
    v_all = f_all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) {
            v0 += r.sum[w];
            f0 += r.count[w];
        }
        v_all += r.sum[w];
        f_all += r.count[w];
    }
}
__device__ __forceinline__ void find_range(const TreeParams &p, Range &r) {
    const int tid = threadIdx.x;
    long long mine = 0, first = 0, total, v0;
    int none, f0;
    for (int b = tid; b < p.B; b += kThreads) {
        const long long n = entry_tiles(p, b);
        if (b == tid) first = n;
        mine += n;
    }
    scan_block(r, mine, 0, v0, f0, total, none);
    // no more CTAs than tiles: those between a pair's first and last all have some of it
    const long long ctas = max(1LL, min((long long)gridDim.x, total)), c = min((long long)blockIdx.x, ctas);
    const long long begin = total * c / ctas, end = total * min(c + 1, ctas) / ctas;
    if (tid == 0) {
        r.skip = 0;
        r.tiles = end - begin;
    }
    long long before = 0;
    int listed = 0;
    for (int b0 = 0; b0 < p.B && before < end; b0 += kThreads) {
        const int b = b0 + tid;
        const long long n = b0 == 0 ? first : b < p.B ? entry_tiles(p, b) : 0;
        long long all = total;   // one round of entries: its sums are there
        int in_all;
        if (p.B > kThreads) scan_block(r, n, 0, v0, f0, all, in_all);
        const long long lo = before + v0;
        const bool in = n > 0 && lo < end && lo + n > begin;
        long long none0, none1;
        scan_block(r, 0, in, none0, f0, none1, in_all);
        if (in && listed + f0 < kList) r.list[listed + f0] = b;
        if (in && lo <= begin) r.skip = begin - lo;
        before += all;
        listed += in_all;
    }
    if (tid == 0) r.n = min(listed, kList);
    // the barrier that follows makes it visible
}

// The items of a CTA, in order: its runs of tiles of one pair.  Every role walks
// the same list.
struct Items {
    int k, b, i, pos;                 // even shares: place in the list; entry, head's place and position of the next pair
    long long left, off;              // tiles to come; tiles of the next pair to leave out
    int u;                            // pieces: the piece
    int h, pair, tiles, slot;
    bool first, last;                 // of the pair's items (even shares)
    Keys ks;
    __device__ __forceinline__ void start(const TreeParams &p, const Range &r) {
        u = (int)blockIdx.x - (int)gridDim.x;
        if (!p.tc_even) return;
        k = i = 0;
        left = r.tiles;
        off = r.skip;
        b = left > 0 ? r.list[0] : 0;
        pos = left > 0 ? p.pos[b] : 0;
    }
    __device__ __forceinline__ bool next_piece(const TreeParams &p) {
        const int total = p.B * p.tc_items_per_b;
        for (;;) {
            if (u >= total - (int)gridDim.x) return false;
            u += gridDim.x;
            b = u / p.tc_items_per_b;
            const int it = u - b * p.tc_items_per_b;
            int lo = 0, hi = p.n_tc - 1;   // largest i with tc_item0[i] <= it
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (p.tc_item0[mid] <= it) lo = mid; else hi = mid - 1;
            }
            h = p.tc_head[lo];
            const int piece = it - p.tc_item0[lo];
            pos = p.pos[b];
            if (pos < 0 || pos > p.cap || !slab_keys(p, h, pos, 0, piece, ks)) continue;
            tiles = (ks.n + kTile - 1) / kTile;
            slot = b * p.slots_per_b + p.head[h].slot0 + piece;
            first = last = false;
            return true;
        }
    }
    __device__ __forceinline__ bool next(const TreeParams &p, const Range &r) {
        if (!p.tc_even) return next_piece(p);
        while (left > 0) {
            if (i == p.n_tc) {
                i = 0;
                ++k;
                b = k < r.n ? r.list[k] : b + 1;
                pos = p.pos[b];
            }
            const int n = pair_tiles(p, i, pos);
            if (off >= n) {
                off -= n;
                ++i;
                continue;
            }
            h = p.tc_head[i];
            pair = b * p.n_tc + i;
            slot = p.tc_slot0 + pair + (int)blockIdx.x;
            tiles = (int)min(left, n - off);
            first = off == 0;
            last = off + tiles == n;
            ks.kind = kSlab;
            const int rows = tree_set_rows(p, h, pos, 0, ks.row0);
            ks.row0 += off * kTile;
            ks.n = (int)min((long long)tiles * kTile, rows - off * kTile);
            left -= tiles;
            off = 0;
            ++i;
            return true;
        }
        return false;
    }
};

struct Shared {
    uint64_t full[kSlotsMax], empty[kSlotsMax], sfull[2], sempty[2], qfull, pfull, pvdone, copied[4], drain;
    uint32_t tmem;
    Waits waits;
    int asked;                        // K~ and V~ tiles that the copies have been asked for
    int bad[4];                       // item number + 1 of an item with an invalid page, by item mod 4 (the copies
                                      // run at most three items ahead of the softmax, as does copied)
    alignas(16) float nref[kTreeMaxNodes];  // the references, negative; read four at a time
    float corr[kTreeMaxNodes];
    float part[4][kTreeMaxNodes];     // a warp's maxima or sums
    Range range;
};

// NP columns of this thread's TMEM lane
template <int NP> __device__ __forceinline__ void ld_cols(uint32_t addr, uint32_t *r) {
    if constexpr (NP == 16) {
        tmem_ld16(addr, r);
    } else {
#pragma unroll
        for (int n = 0; n < NP; n += 32) tmem_ld32(addr + n, r + n);
    }
}
template <int NP> __device__ __forceinline__ void st_cols(uint32_t addr, const uint32_t *r) {
    if constexpr (NP == 16) tmem_st16(addr, r);
    else tmem_st32(addr, r);
}

struct Maps {
    CUtensorMap kv[2];
    int box;             // rows of a box: a tile, or a page that is shorter
};

template <int NP>   // nodes, padded to 16, 32 or 64
__global__ void __launch_bounds__(kThreads, NP <= 32 ? 2 : 1)   // 168 registers: see Mem
tree_tc_kernel(const TreeParams p, const __grid_constant__ Maps maps) {
    constexpr int kSlots = Mem<NP>::kSlots;
    constexpr uint32_t kQHalf = Mem<NP>::kQHalf, kOffQ = Mem<NP>::kOffQ, kOffP = Mem<NP>::kOffP;
    extern __shared__ uint8_t raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    __shared__ Shared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    allow_next();
    WaitSettings waits = {};
    if (tid == 0) {
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.sfull[i], 1);
            mbar_init(&sh.sempty[i], kSoftmax);
        }
        mbar_init(&sh.qfull, kSoftmax);
        mbar_init(&sh.pfull, kSoftmax);
        mbar_init(&sh.pvdone, 1);
        for (int i = 0; i < 4; ++i) mbar_init(&sh.copied[i], 32);
        mbar_init(&sh.drain, 1);
        for (int i = 0; i < 4; ++i) sh.bad[i] = 0;
        waits = start_waits(sh.waits, p.hdr);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 5) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem)), "r"(kTmemCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (p.tc_even) find_range(p, sh.range);
    tc_before();
    __syncthreads();
    tc_after();
    if (tid == 0) set_waits(sh.waits, waits, &sh.full[0]);
    const uint32_t tmem = sh.tmem, base = smem_u32(smem);
    Items it;
    it.start(p, sh.range);
    bool ok = true;

    if (warp == 5) {
        // ------------------------------------------------ instruction issue
        if (lane == 0) {
            int j = 0, t_all = 0, items = 0, pv_slot = -1;   // ring slots and tiles so far; slot of a V~ tile not yet multiplied
            bool pv_first = false;
            const uint32_t iqk = idesc(NP, false), ipv = idesc(Mem<NP>::kO, true);
            auto product = [&](int t) {   // O^T += V~^T P^T of tile t
                const int s = pv_slot % kSlots;
                if (!mbar_wait(&sh.full[s], (pv_slot / kSlots) & 1, &sh.waits) || !mbar_wait(&sh.pfull, t & 1, &sh.waits)) return false;
                tc_after();
#pragma unroll
                for (int k = 0; k < kTile / 16; ++k)
                    tc_mma(tmem + 128, sdesc(base + s * kSlot + k * 2048, kHalf), sdesc(base + kOffP + k * 2048, 16), ipv, k > 0 || !pv_first);
                tc_commit(&sh.empty[s]);
                tc_commit(&sh.pvdone);
                return true;
            };
            while (ok && it.next(p, sh.range)) {
                ok = mbar_wait(&sh.qfull, items & 1, &sh.waits);
                ++items;
                for (int t = 0; ok && t < it.tiles; ++t, ++t_all) {
                    const int s = j % kSlots;
                    ok = mbar_wait(&sh.full[s], (j / kSlots) & 1, &sh.waits) &&
                         (t_all < 2 || mbar_wait(&sh.sempty[t_all & 1], (t_all / 2 - 1) & 1, &sh.waits));
                    if (!ok) break;
                    tc_after();
#pragma unroll
                    for (int k = 0; k < kD / 16; ++k)
                        tc_mma(tmem + (t_all & 1) * 64, sdesc(base + s * kSlot + (k >> 2) * kHalf + (k & 3) * 32, 16),
                               sdesc(base + kOffQ + (k >> 2) * kQHalf + (k & 3) * 32, 16), iqk, k > 0);
                    tc_commit(&sh.empty[s]);
                    tc_commit(&sh.sfull[t_all & 1]);
                    if (pv_slot >= 0) ok = product(t_all - 1);
                    pv_slot = j + 1;
                    pv_first = t == 0;
                    j += 2;
                }
            }
            if (ok && pv_slot >= 0) ok = product(t_all - 1);
            if (!ok) {
                sh.waits.abort = 1;
                report_error(p.hdr, RAT_ERR_TIMEOUT, (int)blockIdx.x);
            }
            tc_commit(&sh.drain);   // everything issued has finished before TMEM is freed
            mbar_drain(&sh.drain, 0);
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ------------------------------------------------ copies
        // lane 2 i + x brings half x (64 channels) of box i of a tile
        const int half = lane & 1, first = (lane >> 1) * maps.box;
        int j = 0, items = 0;
        while (ok && it.next(p, sh.range)) {
            bool bad = false;
            // the page of the lane's box in a tile, looked up a tile ahead: the next
            // copies do not wait for it
            auto page_of = [&](int t) {
                if (!p.page_table || first >= kTile || t * kTile + first >= it.ks.n) return 0;
                return p.page_table[(long long)it.b * p.pps + ((unsigned)it.ks.row0 + t * kTile + first) / (unsigned)p.page_rows];
            };
            int page = page_of(0);
            for (int t = 0; ok && t < it.tiles; ++t) {
                const unsigned row = (unsigned)it.ks.row0 + t * kTile + first;
                int y = (int)row, z = it.b * p.H + it.h;
                bool on = first < kTile && t * kTile + first < it.ks.n;
                if (on && p.page_table) {
                    y = (int)(row % (unsigned)p.page_rows);
                    z = page * p.H + it.h;
                    if (page < 0 || page >= p.num_pages) {
                        bad = true;
                        on = false;
                    }
                }
                page = t + 1 < it.tiles ? page_of(t + 1) : 0;
                const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, on)) * maps.box * 128;
#pragma unroll 1
                for (int x = 0; x < 2; ++x, ++j) {
                    const int s = j % kSlots;
                    if (j >= kSlots) ok = __all_sync(0xffffffffu, mbar_wait(&sh.empty[s], (j / kSlots - 1) & 1, &sh.waits));
                    if (!ok) break;
                    if (lane == 0) mbar_expect(&sh.full[s], bytes);
                    __syncwarp();
                    if (on) tma_load(base + s * kSlot + half * kHalf + first * 128, &maps.kv[x], &sh.full[s], half * 64, y, z);
                }
            }
            if (bad) sh.bad[items & 3] = items + 1;
            mbar_arrive(&sh.copied[items & 3]);
            ++items;
        }
        if (lane == 0) sh.asked = j;
        if (!ok) {
            sh.waits.abort = 1;
            if (lane == 0) report_error(p.hdr, RAT_ERR_TIMEOUT, (int)blockIdx.x);
        }
    } else {
        // ------------------------------------------------ softmax
        constexpr int kCols = NP < 32 ? NP : 32;   // columns of O at a time
        const uint32_t t_lane = tmem + ((uint32_t)(warp * 32) << 16);
        const uint64_t scale2 = pack2(p.scale_log2, p.scale_log2);
        int t_all = 0, items = 0;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            if (!ok || __all_sync(0xffffffffu, mbar_wait(bar, parity, &sh.waits))) return;
            ok = false;
            sh.waits.abort = 1;   // the waits that follow, everyone's, end at once
        };
        // queries of an item: row n of Q is node n (absent nodes: zeros)
        auto stage_q = [&](int b, int h) {
            for (int e = tid; e < NP * 16; e += kSoftmax) {
                const int n = e >> 4, c = e & 15;
                uint4 x = make_uint4(0u, 0u, 0u, 0u);
                if (n < p.N) {
                    const int up = p.parent[(size_t)b * p.N + n];   // at the same time as the query
                    x = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.q) + (((size_t)b * p.N + n) * p.H + h) * kD + c * 8);
                    if (up == RAT_NODE_ABSENT) x = make_uint4(0u, 0u, 0u, 0u);
                }
                *reinterpret_cast<uint4 *>(smem + kOffQ + (c >> 3) * kQHalf + n * 128 + (((c & 7) ^ (n & 7)) << 4)) = x;
            }
            fence_async();
            mbar_arrive(&sh.qfull);
        };
        bool more = it.next(p, sh.range);
        if (more) stage_q(it.b, it.h);
        while (more) {
            uint64_t l2[NP / 2];
#pragma unroll
            for (int n = 0; n < NP / 2; ++n) l2[n] = 0ull;
            for (int t = 0; t < it.tiles; ++t, ++t_all) {
                wait(&sh.sfull[t_all & 1], (t_all / 2) & 1);
                tc_after();
                const bool valid = t * kTile + tid < it.ks.n;
                // x = score * scale - reference, in the log2 domain
                uint64_t x2[NP / 2];
                auto scores = [&]() {
                    uint32_t s[NP];
                    ld_cols<NP>(t_lane + (t_all & 1) * 64, s);
#pragma unroll
                    for (int n = 0; n < NP; n += 4) {
                        const ulonglong2 r = *reinterpret_cast<const ulonglong2 *>(&sh.nref[n]);
                        x2[n / 2] = fma2(pack2(__uint_as_float(s[n]), __uint_as_float(s[n + 1])), scale2, r.x);
                        x2[n / 2 + 1] = fma2(pack2(__uint_as_float(s[n + 2]), __uint_as_float(s[n + 3])), scale2, r.y);
                    }
                };
                bool over = t == 0;
                if (!over) {
                    scores();
                    float mx = -INFINITY;
#pragma unroll
                    for (int n = 0; n < NP / 2; ++n) {
                        float a, c;
                        unpack2(x2[n], a, c);
                        mx = fmaxf(mx, fmaxf(a, c));
                    }
                    over = valid && mx > kSlack;
                }
                if (softmax_any(over)) {
                    // some reference is raised (the first tile sets all of them):
                    // maxima over the tile's keys, by the integers in the floats' order
                    {
                        uint32_t s[NP];
                        ld_cols<NP>(t_lane + (t_all & 1) * 64, s);
#pragma unroll
                        for (int n = 0; n < NP; ++n) {
                            const float x = __uint_as_float(s[n]) * p.scale_log2;
                            int i = __float_as_int(valid && x == x ? x : -INFINITY);
                            i ^= (i >> 31) & 0x7fffffff;
                            i = __reduce_max_sync(0xffffffffu, i);
                            i ^= (i >> 31) & 0x7fffffff;
                            if (lane == (n & 31)) sh.part[warp][n] = __int_as_float(i);
                        }
                    }
                    softmax_sync();
                    if (tid < NP) {
                        float mx = fmaxf(fmaxf(sh.part[0][tid], sh.part[1][tid]), fmaxf(sh.part[2][tid], sh.part[3][tid]));
                        // nothing but scores of -inf so far: they weigh nothing beside any
                        // reference, and the first that is more raises this one
                        mx = fmaxf(mx, -FLT_MAX);
                        const float old = -sh.nref[tid];
                        const bool up = t == 0 || mx > old + kSlack;
                        sh.corr[tid] = t > 0 && up ? exp2f(old - mx) : 1.f;
                        if (up) sh.nref[tid] = -mx;
                    }
                    softmax_sync();
                    if (t > 0) {
                        wait(&sh.pvdone, (t_all - 1) & 1);
                        tc_after();
#pragma unroll
                        for (int n = 0; n < NP; n += 2) {
                            float a, c;
                            unpack2(l2[n / 2], a, c);
                            l2[n / 2] = pack2(a * sh.corr[n], c * sh.corr[n + 1]);
                        }
#pragma unroll 1
                        for (int n = 0; n < Mem<NP>::kO; n += kCols) {
                            uint32_t o[kCols];
                            ld_cols<kCols>(t_lane + 128 + n, o);
#pragma unroll
                            for (int i = 0; i < kCols; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * sh.corr[n % NP + i]);
                            st_cols<kCols>(t_lane + 128 + n, o);
                        }
                    }
                    scores();
                }
                tc_before();
                mbar_arrive(&sh.sempty[t_all & 1]);
                const bool tail = t == it.tiles - 1 && it.ks.n % kTile != 0;
                if (tail && !valid) {
#pragma unroll
                    for (int n = 0; n < NP / 2; ++n) x2[n] = pack2(-INFINITY, -INFINITY);
                }
                if (t_all > 0) wait(&sh.pvdone, (t_all - 1) & 1);   // P of the tile before has been read
                uint8_t *row = smem + kOffP + tid * 128;
#pragma unroll
                for (int n = 0; n < NP; n += 8) {
                    uint32_t pk[4], ps[4];
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        float a, c;
                        unpack2(x2[(n + i) / 2], a, c);
                        a = exp2f_fast(a);
                        c = exp2f_fast(c);
                        l2[(n + i) / 2] = add2(l2[(n + i) / 2], pack2(a, c));
                        if constexpr (Mem<NP>::kHalves) {
                            p_halves(a, c, pk[i / 2], ps[i / 2]);
                        } else {
                            __nv_bfloat162 v = __floats2bfloat162_rn(a, c);
                            pk[i / 2] = *reinterpret_cast<uint32_t *>(&v);
                        }
                    }
                    *reinterpret_cast<uint4 *>(row + (((n >> 3) ^ (tid & 7)) << 4)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
                    if constexpr (Mem<NP>::kHalves)
                        *reinterpret_cast<uint4 *>(row + (((NP + n >> 3) ^ (tid & 7)) << 4)) = make_uint4(ps[0], ps[1], ps[2], ps[3]);
                }
                if (tail) {
                    // rows behind the item's last hold anything: their values are
                    // zeroed, as a probability of zero does not undo a NaN
                    const int v = 2 * t_all + 1;
                    wait(&sh.full[v % kSlots], (v / kSlots) & 1);
                    if (!valid) {
                        uint4 *x = reinterpret_cast<uint4 *>(smem + (v % kSlots) * kSlot + tid * 128);
#pragma unroll
                        for (int c = 0; c < 8; ++c) x[c] = x[kHalf / 16 + c] = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                fence_async();
                mbar_arrive(&sh.pfull);
            }
            // the item's last scores are in, so Q is free: the next item's go there
            const int pair = it.pair, slot = it.slot;
            const bool first = it.first, last = it.last;
            more = it.next(p, sh.range);
            if (more) stage_q(it.b, it.h);
            // sums over the keys: halves of the nodes change lanes until a lane
            // holds NP / 32 nodes' sums over its warp (or two lanes one node's)
            float l[NP];
#pragma unroll
            for (int n = 0; n < NP; n += 2) unpack2(l2[n / 2], l[n], l[n + 1]);
#pragma unroll
            for (int half = NP / 2, off = 16; off > 0; half >>= 1, off >>= 1) {
                const bool up = lane & off;
                if (half == 0) l[0] += __shfl_xor_sync(0xffffffffu, l[0], off);
#pragma unroll
                for (int n = 0; n < half; ++n) {
                    const float give = up ? l[n] : l[n + half], keep = up ? l[n + half] : l[n];
                    l[n] = keep + __shfl_xor_sync(0xffffffffu, give, off);
                }
            }
            // lane bits, highest first, chose the halves: lane i holds nodes i * NP / 32 ...
#pragma unroll
            for (int n = 0; n < (NP + 31) / 32; ++n) sh.part[warp][lane * NP / 32 + n] = l[n];
            softmax_sync();
            const size_t rowbase = (size_t)slot * p.N;
            if (tid == 0 && first) p.tc_range[pair].x = (int)blockIdx.x;
            if (tid == 0 && last) p.tc_range[pair].y = (int)blockIdx.x;
            wait(&sh.copied[items & 3], (items >> 2) & 1);
            wait(&sh.pvdone, (t_all - 1) & 1);
            if (tid < p.N) {
                const float sum = (sh.part[0][tid] + sh.part[1][tid]) + (sh.part[2][tid] + sh.part[3][tid]);
                const bool bad = *(volatile int *)&sh.bad[items & 3] == items + 1;
                p.ml[rowbase + tid] = make_float2(sum == 0.f ? -INFINITY : -sh.nref[tid], bad ? -1.f : sum);
            }
            ++items;
            tc_after();
#pragma unroll 1
            for (int n = 0; n < NP; n += kCols) {
                uint32_t o[kCols], e[kCols] = {};
                ld_cols<kCols>(t_lane + 128 + n, o);
                if constexpr (Mem<NP>::kHalves) ld_cols<kCols>(t_lane + 128 + NP + n, e);
#pragma unroll
                for (int i = 0; i < kCols; ++i)
                    if (n + i < p.N) p.part[(rowbase + n + i) * kD + tid] = __uint_as_float(o[i]) + __uint_as_float(e[i]);
            }
            tc_before();
            softmax_sync();   // sh.nref and sh.part are read
        }
        if (!ok && lane == 0) report_error(p.hdr, RAT_ERR_TIMEOUT, (int)blockIdx.x);
    }
    tc_before();
    __syncthreads();
    // whichever role gave up, the copies still in flight land before the CTA leaves
    if (warp == 4 && sh.waits.abort)
        for (int q = max(0, sh.asked - kSlots); q < sh.asked; ++q) mbar_drain(&sh.full[q % kSlots], (q / kSlots) & 1);
    if (warp == 5) {
        tc_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

template <int NP> cudaError_t launch_np(const TreeParams &p, cudaStream_t s) {
    static std::atomic<unsigned long long> smem_set{0};
    constexpr uint32_t kBytes = Mem<NP>::kBytes;
    cudaError_t e = ensure_smem_limit(tree_tc_kernel<NP>, kBytes + 1024, smem_set, true);
    if (e != cudaSuccess) return e;
    Maps maps;
    const long long rows = p.page_table ? p.page_rows : p.cache_R, blocks = (long long)(p.page_table ? p.num_pages : p.B) * p.H;
    maps.box = p.page_table && p.page_rows < kTile ? p.page_rows : kTile;
    for (int x = 0; x < 2; ++x)
        if (!encode_map_rows(&maps.kv[x], p.cache[x], RAT_BF16, rows, blocks, kD, maps.box)) return cudaErrorInvalidValue;
    tree_tc_kernel<NP><<<kTreeTcCtas, kThreads, kBytes + 1024, s>>>(p, maps);
    return cudaGetLastError();
}

}  // namespace

// A page has to be a whole number of tiles or a whole part of one, in eights of
// rows (the swizzle's period), so that a tile is a whole number of boxes.
bool tree_tc_pages(int page_rows) {
    return page_rows == 0 || page_rows % kTile == 0 || (page_rows % 8 == 0 && kTile % page_rows == 0);
}

cudaError_t launch_tree_tc(const TreeParams &p, cudaStream_t s) {
    return p.N <= 16 ? launch_np<16>(p, s) : p.N <= 32 ? launch_np<32>(p, s) : launch_np<64>(p, s);
}

}  // namespace rat
