// pages.cu -- K9: the page table of a paged decode cache, kept on the GPU.
//
// Update.  A page of entry b's logical rows is needed when some head holds one
// of the positions 0 .. n - 1 there, n = min(length + extra, cap).  With
// has(e) = "entry e of the table names a page":
//   has and not needed: the page goes back on the free stack,
//   needed and not has: a page comes off it,
// all in the order of the table's entries (b, then page), gives first, so the
// result does not depend on how the work is spread.  That takes the ranks of
// the entries among those that give and among those that take: two prefix sums
// over the table.  One cluster of eight or sixteen CTAs does it in one launch: every
// warp owns a contiguous run of entries and counts with ballots, the warps'
// counts are summed through distributed shared memory, and a second pass over
// the run turns ballots into ranks.
// Bound: latency (three sweeps of a run by its warp and three cluster
// barriers); a lane's first kHeld entries stay in registers between the sweeps
// (16 x 32 warps x 16 x 32 entries: 512 sequences of 512 pages), and their loads
// go out together.  A step of 8 sequences takes 9 us, of 256 sequences of 512
// pages 19 us (device time); a table of 131072 entries is 0.2 us of bandwidth.
//
// Slot map.  The row of the flat pool (or flat dense cache) that holds a
// position of a head: index arithmetic and one table read per value, bound by
// the 8 bytes written for each.
#include <cooperative_groups.h>

#include "pages.cuh"

namespace rat {

namespace {

namespace cg = cooperative_groups;

constexpr int kSmall = 8, kLarge = 16;   // CTAs of the cluster
constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

// Does a head of class c hold one of positions 0 .. n-1 in rows [p0, p1)?
// (p0 < 2^31: it is a row of the table; p1 may pass it.)
__device__ __forceinline__ bool page_needed(const HeadClass &c, int grid, unsigned p0, long long p1, int n) {
    if (grid) {
        if (p0 < c.by_d.div(n)) return true;
        return c.W > 0 && p1 > c.S && p0 < (long long)c.S + min(n, c.W);
    }
    // residue r fills rows r * S .. r * S + ceil((n - r) / D) - 1 of its slab
    const unsigned r = c.by_s.div(p0);
    if (r >= (unsigned)c.D) return false;
    const unsigned filled = n > (int)r ? c.by_d.div(n - 1 - (int)r) + 1 : 0;
    if (p0 - r * c.S < filled) return true;
    return (r + 1) * (long long)c.S < p1 && (int)r + 1 < c.D && (int)r + 1 < n;   // the next slab starts inside the page
}

constexpr int kHeld = 16;   // entries of a run that a lane keeps in registers between the sweeps

__global__ void __launch_bounds__(kThreads, 1) page_update_kernel(const PageUpdateParams p) {
    __shared__ int s_cnt[2][kWarps];       // entries of each warp that give / take a page
    __shared__ int s_sum[2];               // and of the CTA
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)cluster.block_rank(), kCluster = (int)cluster.num_blocks();
    const int total = p.B * p.pps;         // < 2^31
    const int run = (int)((((long long)total + kCluster * kWarps - 1) / (kCluster * kWarps) + 31) & ~31LL);
    const long long lo = (long long)(rank * kWarps + warp) * run;
    const int e_lo = (int)min(lo, (long long)total), e_hi = (int)min(lo + run, (long long)total);
    const int n_free = *p.n_free;
    const unsigned below = (1u << lane) - 1u;

    // state of one entry: bit 0 has, bit 1 needed; with both it stays as it is, and so does
    // whatever a sequence has whose length is out of range
    auto state = [&](int page, int e, int len) {
        if (len > p.cap) return 3;
        const int b = p.by_pps.div(e);
        bool need = false;
        if (len >= 0) {
            const int n = (int)min((long long)len + p.extra, (long long)p.cap);
            const unsigned p0 = (unsigned)(e - b * p.pps) * (unsigned)p.page_rows;
            const long long p1 = (long long)p0 + p.page_rows;
#pragma unroll 1
            for (int c = 0; c < p.ncls && !need; ++c) need = page_needed(p.cls[c], p.grid, p0, p1, n);
        }
        const bool has = page >= 0 && page < p.num_pages;
        return (has ? 1 : 0) | (need ? 2 : 0);
    };

    // the first kHeld * 32 entries of the run: loaded together, kept with their states
    int held[kHeld], lens[kHeld];
    unsigned states = 0;                   // two bits each
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        const int e = e_lo + i * 32 + lane;
        held[i] = e < e_hi ? p.table[e] : -1;
        lens[i] = e < e_hi ? p.length[p.by_pps.div(e)] : -1;
    }
    int give = 0, take = 0;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        if (e_lo + i * 32 >= e_hi) break;
        const int e = e_lo + i * 32 + lane, st = e < e_hi ? state(held[i], e, lens[i]) : 0;
        states |= (unsigned)st << (2 * i);
        give += __popc(__ballot_sync(0xffffffffu, st == 1));
        take += __popc(__ballot_sync(0xffffffffu, st == 2));
    }
    // the others are looked at again in every sweep
    auto look = [&](int e, int &page) {
        page = p.table[e];
        return state(page, e, p.length[p.by_pps.div(e)]);
    };
    int page;
    const int e_more = e_lo + kHeld * 32;
#pragma unroll 2
    for (int e = e_more; e < e_hi; e += 32) {
        const int st = e + lane < e_hi ? look(e + lane, page) : 0;
        give += __popc(__ballot_sync(0xffffffffu, st == 1));
        take += __popc(__ballot_sync(0xffffffffu, st == 2));
    }
    if (lane == 0) {
        s_cnt[0][warp] = give;
        s_cnt[1][warp] = take;
    }
    __syncthreads();
    if (warp < 2) {
        // exclusive sums over the CTA's warps
        const int v = s_cnt[warp][lane];
        int x = v;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, off);
            if (lane >= off) x += y;
        }
        s_cnt[warp][lane] = x - v;
        if (lane == 31) s_sum[warp] = x;
    }
    cluster.sync();
    // a lane reads one CTA's sums
    int give0 = s_cnt[0][warp], take0 = s_cnt[1][warp], gives = 0, takes = 0;
    if (lane < kCluster) {
        const int *sum = cluster.map_shared_rank(s_sum, lane);
        gives = sum[0];
        takes = sum[1];
    }
    give0 += __reduce_add_sync(0xffffffffu, lane < rank ? gives : 0);
    take0 += __reduce_add_sync(0xffffffffu, lane < rank ? takes : 0);
    gives = __reduce_add_sync(0xffffffffu, gives);
    takes = __reduce_add_sync(0xffffffffu, takes);
    // a stack that cannot be right (more pages given back than there are) is left alone
    const bool ok = n_free >= 0 && (long long)n_free + gives <= p.num_pages;
    const int top = n_free + gives;
    auto put_back = [&](int st, int page) {
        const unsigned m = __ballot_sync(0xffffffffu, st == 1);
        if (st == 1) p.free_pages[n_free + give0 + __popc(m & below)] = page;
        give0 += __popc(m);
    };
    // the stack's place for an entry that takes a page, -1 when it ran out
    auto place = [&](int st) {
        const unsigned m = __ballot_sync(0xffffffffu, st == 2);
        const int at = top - 1 - (take0 + __popc(m & below));
        take0 += __popc(m);
        return st == 2 && at >= 0 ? at : -1;
    };
    auto settle = [&](int st, int e, int at, int got) {
        if (e >= e_hi || st == 3) return;
        if (st != 2) {
            p.table[e] = -1;
            return;
        }
        if (at < 0) report_error(p.hdr, RAT_ERR_NO_PAGES, (int)p.by_pps.div(e));
        if (at >= 0 && (got < 0 || got >= p.num_pages)) {
            got = -1;
            report_error(p.hdr, RAT_ERR_INVALID, (int)p.by_pps.div(e));
        }
        p.table[e] = got;
    };
    if (ok) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            if (e_lo + i * 32 >= e_hi) break;
            put_back((states >> (2 * i)) & 3, held[i]);
        }
#pragma unroll 1
        for (int e = e_more; e < e_hi; e += 32) {
            const int st = e + lane < e_hi ? look(e + lane, page) : 0;
            put_back(st, page);
        }
    }
    cluster.sync();   // the pages given back are on the stack
    if (ok) {
        // a lane's pages are fetched together
        int at[kHeld], got[kHeld];
#pragma unroll
        for (int i = 0; i < kHeld; ++i) at[i] = place((states >> (2 * i)) & 3);
#pragma unroll
        for (int i = 0; i < kHeld; ++i) got[i] = at[i] >= 0 ? __ldcg(p.free_pages + at[i]) : -1;
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            if (e_lo + i * 32 >= e_hi) break;
            settle((states >> (2 * i)) & 3, e_lo + i * 32 + lane, at[i], got[i]);
        }
#pragma unroll 1
        for (int e = e_more; e < e_hi; e += 32) {
            const int st = e + lane < e_hi ? look(e + lane, page) : 0, where = place(st);
            settle(st, e + lane, where, where >= 0 ? __ldcg(p.free_pages + where) : -1);
        }
        for (int b = rank * kThreads + tid; b < p.B; b += kCluster * kThreads)
            if (p.length[b] > p.cap) report_error(p.hdr, RAT_ERR_INVALID, b);
    }
    if (rank == 0 && tid == 0) {
        if (ok) *p.n_free = max(0, top - takes);
        else report_error(p.hdr, RAT_ERR_INVALID, -1);
    }
    cluster.sync();   // no CTA leaves while another may still read its sums
}

constexpr int kSlotThreads = 256;
constexpr int kSlotPlaces = 2048; // places (position, row layout) of a CTA, at a time
constexpr int kSlotClasses = 64;  // row layouts handled at a time
// positions of one CTA: as many as the places allow, between 32 and 128 (32 for
// any number of layouts took 30 us for 8.2 M values: the CTAs' first loads,
// nine waves of them, were the time)
int slot_tokens(int ncls) { return ncls <= 16 ? 128 : ncls <= 32 ? 64 : 32; }

// Heads with the same layout have a position in the same page and line, so that
// is found once per (position, layout); a head's value is then one addition.
__global__ void __launch_bounds__(kSlotThreads) slot_map_kernel(const SlotParams p) {
    __shared__ long long s_at[2][kSlotPlaces];   // place of head 0's row (-1: none)
    __shared__ unsigned char s_cls[kMaxHeads];
    const int tid = threadIdx.x;
    const int chunks = (p.T + p.tokens - 1) / p.tokens;
    const int b = blockIdx.x / chunks, i0 = (blockIdx.x % chunks) * p.tokens;
    const int nt = min(p.tokens, p.T - i0);
    const int pos = p.pos[b], cnt = p.count ? p.count[b] : p.T;
    const bool ok = pos >= 0 && cnt >= 0 && cnt <= p.T && pos <= p.cap && cnt <= p.cap - pos;
    if (!ok && i0 == 0 && tid == 0) report_error(p.hdr, RAT_ERR_INVALID, b);
    for (int h = tid; h < p.H; h += kSlotThreads) s_cls[h] = p.cls_of[h];
    // place of logical row `row` of head 0; a head further is `stride` rows on
    const long long stride = p.page_table ? p.page_rows : p.cache_R;
    auto place = [&](unsigned row) -> long long {
        if (!p.page_table) return (long long)b * p.H * p.cache_R + row;
        const unsigned pi = p.by_page.div(row);
        const int pg = p.page_table[(long long)b * p.pps + pi];
        if (pg < 0 || pg >= p.num_pages) return -1;
        return (long long)pg * p.H * p.page_rows + (row - pi * p.page_rows);
    };
    for (int c0 = 0; c0 < p.ncls; c0 += kSlotClasses) {
        const int nc = min(kSlotClasses, p.ncls - c0);
        __syncthreads();
        for (int e = tid; e < nt * nc; e += kSlotThreads) {
            const int i = i0 + e / nc, c = e % nc;
            const HeadClass &k = p.cls[c0 + c];
            long long main_at = -1, ring_at = -1;
            if (ok && i < cnt) {
                const unsigned j = (unsigned)pos + i, q = k.by_d.div(j), r = j - q * k.D;
                if (!p.grid) main_at = place(r * k.S + q);
                else if (r == (unsigned)k.D - 1) main_at = place(q);
                // the ring's row, unless a later position of the run takes it
                if (p.ring && k.W > 0 && i >= cnt - k.W) ring_at = place(k.S + (j - k.by_w.div(j) * k.W));
            }
            s_at[0][e] = main_at;
            s_at[1][e] = ring_at;
        }
        __syncthreads();
        const size_t out0 = ((size_t)b * p.T + i0) * p.H;
        if (p.ncls <= kSlotClasses && p.H % 2 == 0) {
            // two heads of a position at a time: 16-byte stores
            auto value = [&](long long at, int h) { return at < 0 ? -1 : at + h * stride; };
            for (int e = 2 * tid; e < nt * p.H; e += 2 * kSlotThreads) {
                const int i = p.by_h.div(e), h = e - i * p.H, a = i * nc + s_cls[h], c = i * nc + s_cls[h + 1];
                *reinterpret_cast<longlong2 *>(p.slots + out0 + e) = make_longlong2(value(s_at[0][a], h), value(s_at[0][c], h + 1));
                if (p.ring) *reinterpret_cast<longlong2 *>(p.ring + out0 + e) = make_longlong2(value(s_at[1][a], h), value(s_at[1][c], h + 1));
            }
            continue;
        }
        for (int e = tid; e < nt * p.H; e += kSlotThreads) {
            const int i = p.by_h.div(e), h = e - i * p.H, c = s_cls[h] - c0;
            if (c < 0 || c >= nc) continue;
            const long long m = s_at[0][i * nc + c];
            p.slots[out0 + e] = m < 0 ? -1 : m + h * stride;
            if (p.ring) {
                const long long r = s_at[1][i * nc + c];
                p.ring[out0 + e] = r < 0 ? -1 : r + h * stride;
            }
        }
    }
}

}  // namespace

cudaError_t launch_page_update(const PageUpdateParams &p, cudaStream_t s) {
    // sixteen CTAs (not a portable size) for a table that eight would hold in more
    // than kHeld / 2 entries a lane, where the device can place them.  What was
    // found is kept for each device: the attribute is a device's own
    static std::atomic<unsigned long long> asked{0}, placed{0};
    int size = kSmall;
    if ((long long)p.B * p.pps > (long long)kSmall * kThreads * (kHeld / 2)) size = kLarge;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (size == kLarge) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
        bool can = (placed.load(std::memory_order_acquire) & bit) != 0;
        if (!can && !(asked.load(std::memory_order_acquire) & bit)) {
            cfg.gridDim = dim3(kLarge);
            attr.val.clusterDim.x = kLarge;
            int n = 0;
            can = cudaFuncSetAttribute(page_update_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                  cudaOccupancyMaxActiveClusters(&n, page_update_kernel, &cfg) == cudaSuccess && n > 0;
            if (!can) cudaGetLastError();
            if (can) placed.fetch_or(bit, std::memory_order_acq_rel);
            asked.fetch_or(bit, std::memory_order_acq_rel);
        }
        if (!can) size = kSmall;
    }
    cfg.gridDim = dim3(size);
    attr.val.clusterDim.x = size;
    cudaError_t e = cudaLaunchKernelEx(&cfg, page_update_kernel, p);
    if (e != cudaSuccess) return e;
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_slot_map(const SlotParams &p, cudaStream_t s) {
    if ((long long)p.B * p.T == 0) return cudaSuccess;
    SlotParams q = p;
    q.tokens = slot_tokens(p.ncls);
    const unsigned grid = (unsigned)p.B * (unsigned)((p.T + q.tokens - 1) / q.tokens);
    slot_map_kernel<<<grid, kSlotThreads, 0, s>>>(q);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace rat
