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
// over the table.  One cluster of kCluster CTAs does it in one launch: every
// warp owns a contiguous run of entries and counts with ballots, the warps'
// counts are summed through distributed shared memory, and a second pass over
// the run turns ballots into ranks.
// Bound: latency (three sweeps of a run by its warp and three cluster
// barriers); the table itself is read from DRAM once.
//
// Slot map.  The row of the flat pool (or flat dense cache) that holds a
// position of a head: index arithmetic and one table read per value, bound by
// the 8 bytes written for each.
#include <cooperative_groups.h>

#include "pages.cuh"

namespace rat {

namespace {

namespace cg = cooperative_groups;

constexpr int kCluster = 8;
constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

// Does a head of class c hold one of positions 0 .. n-1 in rows [p0, p1)?
__device__ __forceinline__ bool page_needed(const HeadClass &c, int grid, long long p0, long long p1, int n) {
    if (grid) {
        if (p0 < n / c.D) return true;
        return c.W > 0 && p1 > c.S && p0 < (long long)c.S + min(n, c.W);
    }
    // residue r fills rows r * S .. r * S + ceil((n - r) / D) - 1 of its slab
    const long long r = p0 / c.S;
    if (r >= c.D) return false;
    const long long filled = n > r ? (n - 1 - r) / c.D + 1 : 0;
    if (p0 - r * c.S < filled) return true;
    return (r + 1) * c.S < p1 && r + 1 < c.D && r + 1 < n;   // the next slab starts inside the page
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads) page_update_kernel(const PageUpdateParams p) {
    __shared__ int s_cnt[2][kWarps];       // entries of each warp that give / take a page
    __shared__ int s_sum[2];               // and of the CTA
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = (int)cluster.block_rank();
    const int total = p.B * p.pps;
    const int run = ((total + kCluster * kWarps - 1) / (kCluster * kWarps) + 31) & ~31;
    const long long e_lo = (long long)(rank * kWarps + warp) * run;
    const long long e_hi = min(e_lo + run, (long long)total);
    const int n_free = *p.n_free;
    const unsigned below = (1u << lane) - 1u;

    // state of one entry: bit 0 has, bit 1 needed
    auto state = [&](long long e, int &page) {
        page = -1;
        if (e >= e_hi) return 0;
        const int b = (int)(e / p.pps), pi = (int)(e % p.pps);
        page = p.table[e];
        const int len = p.length[b];
        bool need = false;
        if (len >= 0 && len <= p.cap) {
            const int n = (int)min((long long)len + p.extra, (long long)p.cap);
            const long long p0 = (long long)pi * p.page_rows;
            for (int c = 0; c < p.ncls && !need; ++c) need = page_needed(p.cls[c], p.grid, p0, p0 + p.page_rows, n);
        }
        const bool has = page >= 0 && page < p.num_pages;
        if (len > p.cap) need = has;   // a length out of range: the entry stays as it is
        return (has ? 1 : 0) | (need ? 2 : 0);
    };

    int give = 0, take = 0;
    for (long long e = e_lo; e < e_hi; e += 32) {
        int page;
        const int st = state(e + lane, page);
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
    int give0 = s_cnt[0][warp], take0 = s_cnt[1][warp], gives = 0, takes = 0;
    for (int r = 0; r < kCluster; ++r) {
        const int *sum = cluster.map_shared_rank(s_sum, r);
        const int g = sum[0], t = sum[1];
        gives += g;
        takes += t;
        if (r < rank) {
            give0 += g;
            take0 += t;
        }
    }
    // a stack that cannot be right (more pages given back than there are) is left alone
    const bool ok = n_free >= 0 && (long long)n_free + gives <= p.num_pages;
    const int top = n_free + gives;
    if (ok) {
        for (long long e = e_lo; e < e_hi; e += 32) {
            int page;
            const int st = state(e + lane, page);
            const unsigned m = __ballot_sync(0xffffffffu, st == 1);
            if (st == 1) p.free_pages[n_free + give0 + __popc(m & below)] = page;
            give0 += __popc(m);
        }
    }
    cluster.sync();   // the pages given back are on the stack
    if (ok) {
        for (long long e = e_lo; e < e_hi; e += 32) {
            int page;
            const int st = state(e + lane, page);
            const unsigned m = __ballot_sync(0xffffffffu, st == 2);
            if (e + lane < e_hi) {
                if (st == 2) {
                    const int at = top - 1 - (take0 + __popc(m & below));
                    int got = at >= 0 ? __ldcg(p.free_pages + at) : -1;
                    if (at < 0) {
                        report_error(p.hdr, RAT_ERR_NO_PAGES, (int)((e + lane) / p.pps));
                    } else if (got < 0 || got >= p.num_pages) {
                        got = -1;
                        report_error(p.hdr, RAT_ERR_INVALID, (int)((e + lane) / p.pps));
                    }
                    p.table[e + lane] = got;
                } else if (st != 3) {
                    p.table[e + lane] = -1;
                }
            }
            take0 += __popc(m);
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

__global__ void __launch_bounds__(kSlotThreads) slot_map_kernel(const SlotParams p) {
    const long long n = (long long)p.B * p.T * p.H;
    for (long long e = (long long)blockIdx.x * kSlotThreads + threadIdx.x; e < n; e += (long long)gridDim.x * kSlotThreads) {
        const int h = (int)(e % p.H);
        const long long bt = e / p.H;
        const int i = (int)(bt % p.T), b = (int)(bt / p.T);
        const int pos = p.pos[b], cnt = p.count ? p.count[b] : p.T;
        const bool ok = pos >= 0 && cnt >= 0 && cnt <= p.T && (long long)pos + cnt <= p.cap;
        if (!ok && i == 0 && h == 0) report_error(p.hdr, RAT_ERR_INVALID, b);
        long long row[2] = {-1, -1};
        if (ok && i < cnt) {
            cache_rows_of((long long)pos + i, p.dil[h], p.win[h], p.slab[h], p.grid, row[0], row[1]);
            if (i < cnt - p.win[h]) row[1] = -1;   // a later position of the run takes the ring row
        }
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            long long *out = w ? p.ring : p.slots;
            if (!out) continue;
            // the offset of channel 0 in a cache of one channel is the row
            out[e] = row[w] < 0 ? -1 : cache_offset(p.page_table, p.pps, p.page_rows, p.num_pages, p.cache_R, p.H, 1, b, h, row[w]);
        }
    }
}

}  // namespace

cudaError_t launch_page_update(const PageUpdateParams &p, cudaStream_t s) {
    page_update_kernel<<<kCluster, kThreads, 0, s>>>(p);
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t launch_slot_map(const SlotParams &p, cudaStream_t s) {
    const long long n = (long long)p.B * p.T * p.H;
    if (n == 0) return cudaSuccess;
    const unsigned grid = (unsigned)min((n + kSlotThreads - 1) / kSlotThreads, 148ll * 16);
    slot_map_kernel<<<grid, kSlotThreads, 0, s>>>(p);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace rat
