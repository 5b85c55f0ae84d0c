// pages.cuh -- parameter blocks of the page-table kernels (pages.cu).
#pragma once

#include "rat_internal.cuh"

namespace rat {

// Quotients of a fixed divisor d >= 1 without a division (Granlund and Montgomery,
// "Division by invariant integers using multiplication", 1994): for n < 2^31,
// n / d = hi32(n * m) >> s with m = ceil(2^(32 + s) / d), 2^s >= d (m < 2^33 has
// its top bit implied: q = (hi32(n * (m - 2^32)) + n) >> s, and n + hi < 2^32).
struct Divisor {
    unsigned m, s;
    __host__ void set(unsigned d) {
        s = 0;
        while ((1ull << s) < d) ++s;
        m = (unsigned)((((1ull << s) - d) << 32) / d + 1);
    }
    __device__ __forceinline__ unsigned div(unsigned n) const { return (__umulhi(n, m) + n) >> s; }
};

// The heads of a call that keep the same rows: same dilation and ring.
struct HeadClass {
    int D, W;        // W = 0: no ring
    int S;           // ceil(cap / D)
    Divisor by_d, by_s, by_w;
};

struct PageUpdateParams {
    int *table;              // [B, pps]
    const int *length;       // [B], < 0: the entry holds nothing
    int *free_pages;         // [num_pages] stack, the next page last
    int *n_free;             // [1]
    int B, pps, page_rows, num_pages, cap, extra, grid;
    Divisor by_pps;
    int ncls;
    HeadClass cls[kMaxHeads];
    WsHeader *hdr;
};
cudaError_t launch_page_update(const PageUpdateParams &p, cudaStream_t s);

struct SlotParams {
    const int *pos, *count;      // [B]; count null: T
    long long *slots, *ring;     // [B,T,H]; ring may be null
    long long cache_R;
    int B, T, H, cap, grid;
    const int *page_table;
    int page_rows, pps, num_pages;
    Divisor by_page, by_h;
    int tokens;                  // positions of one CTA
    int ncls;                    // W of a class: the ring's length, 0 without one
    HeadClass cls[kMaxHeads];
    unsigned char cls_of[kMaxHeads];
    WsHeader *hdr;
};
cudaError_t launch_slot_map(const SlotParams &p, cudaStream_t s);

}  // namespace rat
