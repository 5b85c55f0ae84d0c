// pages.cuh -- parameter blocks of the page-table kernels (pages.cu).
#pragma once

#include "rat_internal.cuh"

namespace rat {

// The heads of a call that keep the same rows: same dilation and ring.
struct HeadClass {
    int D, W;        // W = 0: no ring
    int S;           // ceil(cap / D)
};

struct PageUpdateParams {
    int *table;              // [B, pps]
    const int *length;       // [B], < 0: the entry holds nothing
    int *free_pages;         // [num_pages] stack, the next page last
    int *n_free;             // [1]
    int B, pps, page_rows, num_pages, cap, extra, grid;
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
    int ncls;                    // W of a class: the ring's length, 0 without one
    HeadClass cls[kMaxHeads];
    unsigned char cls_of[kMaxHeads];
    WsHeader *hdr;
};
cudaError_t launch_slot_map(const SlotParams &p, cudaStream_t s);

}  // namespace rat
