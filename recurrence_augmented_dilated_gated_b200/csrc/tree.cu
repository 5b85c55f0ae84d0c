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
#include <algorithm>

#include "tree_keys.cuh"

namespace rat {

namespace {

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
    const int S = p.head[h].nsplit, ws = p.head[h].wsplit;
    const int tc = p.head[h].tc;
    // first slots of the set's pieces and of the window's
    int set0 = b * p.slots_per_b + p.head[h].slot0;
    const int w0 = set0 + S;
    wait_previous();
    // the set's pieces: as many as info says, or tree_tc.cu's
    int shared = 0;
    if (tc >= 0) {
        long long row0;
        const int pos = p.pos[b];
        if (pos > 0 && pos <= p.cap && tree_set_rows(p, h, pos, 0, row0) > 0) {
            const int q = b * p.n_tc + tc;
            const int2 r = p.tc_range[q];
            set0 = p.tc_slot0 + q + r.x;
            shared = r.y - r.x + 1;
        }
    }
    auto pieces = [&](int node) {
        const int np = p.info[(size_t)bh * p.N + node];
        return np > 0 && tc >= 0 ? shared : np;
    };
    int bad = 0;
    if (p.page_table) {
        // a page that was not valid anywhere in (b, h): the whole pair is skipped
        const int most = tc >= 0 ? shared : S;
        for (int e = threadIdx.x; e < (most + ws) * p.N; e += kCombineThreads) {
            const int s = e / p.N, n = e % p.N, np = pieces(n);
            if (np < 0) continue;
            if (s >= most || s < np) bad |= p.ml[(size_t)(s < most ? set0 + s : w0 + s - most) * p.N + n].y < 0.f;
        }
        bad = __syncthreads_or(bad);
        if (bad && threadIdx.x == 0 && i == 0) report_error(p.hdr, RAT_ERR_INVALID, b);
    }
    if (i >= p.N) return;
    const int np = pieces(i);
    if (np == -2) return;
    float M = -INFINITY, L = 0.f, o[kC] = {};
    if (np >= 0 && !bad) {
        const int n = np + ws;   // pieces of the set, then of the window
        auto place = [&](int x) { return (size_t)(x < np ? set0 + x : w0 + x - np) * p.N + i; };
        for (int x = lane; x < n; x += 32) M = fmaxf(M, p.ml[place(x)].x);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
#pragma unroll 2
        for (int x = 0; x < n; ++x) {
            const size_t at = place(x);
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

template <typename T, int D> cudaError_t launch_typed(const TreeParams &p, cudaStream_t s) {
    const unsigned grid = (unsigned)p.B * (unsigned)p.ctas_per_b;
    cudaError_t e = cudaSuccess;
    if (p.n_tc > 0) {
        e = launch_tree_tc(p, s);
        if (e != cudaSuccess) return e;
        count_launches(1);
    }
    e = launch_tree_mma(p, sizeof(T) == 4 ? RAT_F32 : RAT_BF16, grid, s);
    if (e != cudaSuccess) return e;
    const unsigned nb = (p.N + kCombineThreads / 32 - 1) / (kCombineThreads / 32);
    e = launch_after(tree_combine_kernel<T, D>, (unsigned)p.B * p.H * nb, kCombineThreads, 0, s, true, p);
    if (e != cudaSuccess) return e;
    count_launches(2);
    return cudaSuccess;
}

}  // namespace

namespace {

// Rows of one kind of dilated set, and how many of them an entry has.
struct SetRows {
    int rows;
    long long sets;
};

// rows / length, rounded up (rows up to 2^31 - 1)
int count_pieces(int rows, int length) { return (int)(((long long)rows + length - 1) / length); }

// The longest pieces to cut dilated sets into, for items that run `at_once` at a
// time and cost as much as `fixed` rows besides their own (a piece's first loads,
// its join and its partials, 5 us): the least number of rounds times the length
// of one, by the cache's capacity.
int piece_target(const SetRows *kinds, int n_kinds, long long B, int at_once, int fixed) {
    static const int kTargets[] = {128, 192, 256, 384, 512, 768, 1024, 1536, 2048, 4096};
    long long best = 0;
    int pick = 128;
    for (int target : kTargets) {
        long long items = 0;
        int longest = 0;
        for (int k = 0; k < n_kinds; ++k) {
            const int pieces = count_pieces(kinds[k].rows, target), len = count_pieces(kinds[k].rows, pieces);
            items += kinds[k].sets * pieces;
            if (len > longest) longest = len;
        }
        const long long cost = (items * B + at_once - 1) / at_once * (fixed + longest);
        if (best == 0 || cost <= best) {
            best = cost;
            pick = target;
        }
    }
    return pick;
}

}  // namespace

// How many of a head's D slabs a tree touches is known on the device only (its
// depth): the plan takes kSetsGuess, and a CTA loops when there are more.
TreeLayout tree_plan(const rat_cfg *c, int cap, int page_rows, TreeParams *p) {
    constexpr int kSetsGuess = 8, kSMs = 148;
    // tree_tc.cu takes heads whose nodes all read the same rows, from this many held
    // rows on (by capacity, with caches held to it).  Both forms measured warm, 16 heads, 8 / 24 / 48 nodes:
    // 1 x 16000 positions (0.24 M rows) tree_tc 43 / 50 / 82 us, tree_mma 38 / 51 / 78;
    // 4 x 8000 (0.49 M) 61 / 69 / 94 against 63 / 87 / 138; 4 x 16000 (0.98 M) 97 / 107 /
    // 127 against 107 / 142 / 240; 8 x 16000 (1.95 M) 172 / 180 / 198 against 194 / 250 / 414.
    // (6 x 20 nodes, 28 grid heads with W = 128, 0.63 M rows: 100 against 91.)
    const long long kTcMinRows = c->T > 32 ? 3 << 17 : 3 << 18;
    const bool grid = (c->flags & RAT_FLAG_GRID_DILATION) != 0;
    const int N = c->T;
    auto sets_of = [&](int D) {
        const int most = D < kSetsGuess ? D : kSetsGuess;
        return grid ? 1 : most < N ? most : N;
    };
    // the kinds of sets among the heads, for either form
    SetRows kinds[2][kMaxHeads];
    int dils[2][kMaxHeads], n_kinds[2] = {0, 0};
    long long one_set_rows = 0;
    for (int h = 0; h < c->H; ++h) {
        const int D = c->dil[h], x = grid || D == 1;
        int k = 0;
        while (k < n_kinds[x] && dils[x][k] != D) ++k;
        if (k == n_kinds[x]) {
            dils[x][k] = D;
            kinds[x][k].rows = (int)(((long long)cap + D - 1) / D);
            kinds[x][k].sets = 0;
            ++n_kinds[x];
        }
        kinds[x][k].sets += sets_of(D);
        if (x) one_set_rows += kinds[x][k].rows;
    }
    const bool tc = c->dtype == RAT_BF16 && c->d == 128 && one_set_rows * c->B >= kTcMinRows && tree_tc_pages(page_rows);
    const int n_sets = n_kinds[0];   // kinds of heads with several sets
    // Fewer pairs than three for each of its CTAs: even shares of all rows, whatever the
    // lengths; else pieces by the capacity.  16 entries x 16 heads of 14000 rows (1.7
    // pairs a CTA): 333 us, by pieces 366; 32 x 16 of 1800 rows, in pages (3.5): 128, by
    // pieces 124.
    long long one_set_heads = 0;
    for (int k = 0; k < n_kinds[1]; ++k) one_set_heads += kinds[1][k].sets;
    const bool even = tc && one_set_heads * c->B < 3 * kTreeTcCtas;
    int target_tc = 0;
    if (tc) {
        target_tc = piece_target(kinds[1], n_kinds[1], c->B, kSMs, 512);
    } else {
        for (int k = 0; k < n_kinds[1]; ++k) kinds[0][n_kinds[0] + k] = kinds[1][k];
        n_kinds[0] += n_kinds[1];
    }
    // in 5 us an item of tree_mma.cu alone on its SM reads 640 rows of bf16 or 160 of
    // fp32 for up to 16 nodes, half or a quarter for up to 32 or 64; a CTA of tree_tc.cu 512
    long long most_rows = -1;
    int nodes = N;
    for (int k = 0; k < n_kinds[0]; ++k)
        if (kinds[0][k].sets * kinds[0][k].rows > most_rows) {
            most_rows = kinds[0][k].sets * kinds[0][k].rows;
            nodes = k < n_sets ? (N + sets_of(dils[0][k]) - 1) / sets_of(dils[0][k]) : N;
        }
    const int fixed = (c->dtype == RAT_BF16 ? 640 : 160) / (nodes <= 16 ? 1 : nodes <= 32 ? 2 : 4);
    const int target = piece_target(kinds[0], n_kinds[0], c->B, 3 * kSMs, fixed);
    const int window_rows = target > 128 ? target : 128;
    // A CTA that takes several items looks at the tree once: not more CTAs than some
    // sixteen rounds of them (five rounds took 524 us where these take 520, 64
    // entries of 16 heads).
    const long long pairs = (long long)c->B * c->H;
    const long long share = pairs > 0 ? (48ll * kSMs + pairs - 1) / pairs : 1;
    // Nor more pieces of a head than 96 rounds of one item an SM: a piece has partials of
    // its own, which would grow with the capacity whatever is held (64 entries of 16 heads
    // of 2^20 positions, 64 nodes: 8.8 GB, so 0.5).
    const long long most_pieces = pairs > 0 ? (96ll * kSMs + pairs - 1) / pairs : 1;
    auto cut = [&](int rows, int length) { return (int)std::min<long long>(count_pieces(rows, length), most_pieces); };
    int ctas = 0, slots = 0, per_head = 0;
    p->n_tc = p->tc_items_per_b = 0;
    p->tc_same = 1;
    p->tc_even = even ? 1 : 0;
    long long R = 0;
    for (int h = 0; h < c->H; ++h) {
        const int D = c->dil[h];
        const int slab = (int)(((long long)cap + D - 1) / D);
        const bool one_set = grid || D == 1, by_tc = tc && one_set;
        const int ns = by_tc && even ? 1 : cut(slab, by_tc ? target_tc : target);
        p->head[h].dil = D;
        // with dedupe a D = 1 head's window keys are all in its dilated set
        p->head[h].win = (c->flags & RAT_FLAG_DEDUPE) && D == 1 ? 0 : c->win[h];
        p->head[h].slab = slab;
        p->head[h].nsplit = ns;
        const int w = p->head[h].win < cap ? p->head[h].win : cap;
        p->head[h].wsplit = w > window_rows ? cut(w, window_rows) : 1;
        const long long most = (long long)sets_of(D) * ns;
        p->head[h].slab_ctas = (int)(most < share ? most : share);
        p->head[h].fused = 0;
        p->head[h].tc = by_tc && even ? p->n_tc : -1;
        if (by_tc) {
            p->head[h].slab_ctas = 0;
            p->tc_item0[p->n_tc] = p->tc_items_per_b;
            p->tc_items_per_b += ns;
            p->tc_head[p->n_tc++] = (unsigned char)h;
            if (D != c->dil[p->tc_head[0]]) p->tc_same = 0;
        } else if (one_set && ns == 1 && p->head[h].wsplit == 1) {
            p->head[h].fused = 1;
            p->head[h].slab_ctas = 0;
        }
        p->head[h].cta0 = ctas;
        p->head[h].slot0 = slots;
        p->head[h].recur = (c->recur == nullptr || c->recur[h] != 0) ? 1 : 0;
        const int mine = p->head[h].wsplit + p->head[h].slab_ctas;
        per_head = h == 0 ? mine : per_head == mine ? mine : -1;
        ctas += mine;
        slots += ns + p->head[h].wsplit;
        const long long rows = grid ? (long long)slab + (D > 1 ? c->win[h] : 0) : (long long)D * slab;
        R = R > rows ? R : rows;
    }
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
    const size_t pairs_tc = even ? (size_t)c->B * p->n_tc : 0, all_slots = (size_t)c->B * slots + (even ? pairs_tc + kTreeTcCtas : 0);
    p->tc_slot0 = (int)((long long)c->B * slots);   // in range, or the step is refused
    L.node_rows = 0;
    L.part = al((size_t)c->B * c->H * 2 * N * c->d * elt);
    L.ml = L.part + al(all_slots * N * c->d * sizeof(float));
    L.info = L.ml + al(all_slots * N * sizeof(float2));
    L.tc_range = L.info + al((size_t)c->B * c->H * N * sizeof(int));
    L.total = L.tc_range + al(pairs_tc * sizeof(int2));
    return L;
}

cudaError_t launch_tree(const TreeParams &p, int dtype, cudaStream_t s) {
    if ((size_t)p.B * p.N == 0) return cudaSuccess;
    if (dtype == RAT_BF16)
        return p.d == 128 ? launch_typed<__nv_bfloat16, 128>(p, s) : launch_typed<__nv_bfloat16, 64>(p, s);
    return p.d == 128 ? launch_typed<float, 128>(p, s) : launch_typed<float, 64>(p, s);
}

}  // namespace rat
