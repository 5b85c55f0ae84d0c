// tree_keys.cuh -- what the kernels of the tree step share (tree_mma.cu: every
// item; tree_tc.cu: held rows of large trees): which keys an item holds, where
// they are and for whom they count, and the recurrence down the tree.
#pragma once

#include "tree.cuh"
#include "tree_copy.cuh"

namespace rat {

__device__ __forceinline__ int find_tree_head(const TreeParams &p, int it) {
    if (p.ctas_per_head > 0) return it / p.ctas_per_head;
    int lo = 0, hi = p.H - 1;  // largest h with cta0[h] <= it
    while (lo < hi) {
        int mid = (lo + hi + 1) >> 1;
        if (p.head[mid].cta0 <= it) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// The keys of one item: rows of a slab, held rows of the window, or the nodes.
enum KeyKind { kSlab = 0, kWindow = 1, kNodes = 2 };

struct Keys {
    int kind;
    long long row0;   // slab: first cache row;  window: first position
    int n;            // keys
};

// Element offset of key i: of its cache row (-1: no valid page), or of the
// node's row.  Rows and positions fit in 32 bits (D * ceil(cap / D) < cap + D).
__device__ __forceinline__ long long key_offset(const TreeParams &p, const Keys &ks, int b, int h, int i) {
    const long long bh = (long long)b * p.H + h;
    if (ks.kind == kNodes) return (bh * 2 * p.N + i) * p.d;   // keys; values N * d further
    unsigned row = (unsigned)ks.row0 + i;
    if (ks.kind == kWindow) {
        const unsigned j = row, D = p.head[h].dil, S = p.head[h].slab;
        if (!p.grid) row = D == 1 ? j : j % D * S + j / D;
        else row = D > 1 ? S + j % (unsigned)p.head[h].win : j;   // the ring
    }
    if (!p.page_table) return (bh * p.cache_R + row) * p.d;
    const unsigned pi = row / (unsigned)p.page_rows, pr = row - pi * p.page_rows;
    const int pg = p.page_table[(long long)b * p.pps + pi];
    if (pg < 0 || pg >= p.num_pages) return -1;
    return (((long long)pg * p.H + h) * p.page_rows + pr) * p.d;
}

// Depth differences that are multiples of a head's dilation, and the nodes on its
// grid, as bits (one warp).
__device__ __forceinline__ void tree_masks(const TreeParams &p, TreeInfo &ti, int h, int pos) {
    const int lane = threadIdx.x & 31;
    const unsigned D = p.head[h].dil;
    unsigned m[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int i = lane + 32 * u;
        m[u] = __ballot_sync(0xffffffffu, p.grid ? ti.depth[i] >= 0 && (unsigned)(pos + ti.depth[i]) % D == D - 1 : i % D == 0);
    }
    if (lane == 0) ti.far = (unsigned long long)m[1] << 32 | m[0];
}

// How often key i counts for a node of depth `dep` and branch `anc` (0, 1 or 2).
__device__ __forceinline__ int key_count(const TreeParams &p, const Keys &ks, const TreeInfo &ti, int h, int pos,
                                         int dep, unsigned long long anc, int node, int i) {
    if (i >= ks.n) return 0;
    if (ks.kind == kSlab) return 1;
    const int D = p.head[h].dil, W = p.head[h].win;
    if (ks.kind == kWindow) {
        const int j = (int)ks.row0 + i, t = pos + dep;
        if (j <= t - W) return 0;
        if (p.dedupe && (p.grid ? j % D == D - 1 : (t - j) % D == 0)) return 0;
        return 1;
    }
    if (!((anc >> i) & 1ull)) return 0;
    const int back = dep - ti.depth[i];
    const int far = p.grid ? i == node || ((ti.far >> i) & 1ull) : (int)((ti.far >> back) & 1ull);
    const int near = back < W && !(p.dedupe && far);
    return far + near;
}

__device__ __forceinline__ void store1(float *p, float x) { *p = x; }
__device__ __forceinline__ void store1(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }
// one or two adjacent values
template <int kN> __device__ __forceinline__ void loads(const float *p, float (&x)[kN]) {
    if constexpr (kN == 2) {
        const float2 v = *reinterpret_cast<const float2 *>(p);
        x[0] = v.x;
        x[1] = v.y;
    } else {
        x[0] = *p;
    }
}
template <int kN> __device__ __forceinline__ void loads(const __nv_bfloat16 *p, float (&x)[kN]) {
    if constexpr (kN == 2) {
        const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(p));
        x[0] = v.x;
        x[1] = v.y;
    } else {
        x[0] = __bfloat162float(*p);
    }
}
template <int kN> __device__ __forceinline__ void stores(float *p, const float (&x)[kN]) {
    if constexpr (kN == 2) *reinterpret_cast<float2 *>(p) = make_float2(x[0], x[1]);
    else *p = x[0];
}
template <int kN> __device__ __forceinline__ void stores(__nv_bfloat16 *p, const float (&x)[kN]) {
    if constexpr (kN == 2) *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(x[0], x[1]);
    else *p = __float2bfloat16_rn(x[0]);
}

__device__ __forceinline__ float exp2f_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two probabilities as bf16 halves, for products with bf16 values: x cut to bf16, and
// what that leaves, rounded (2^-9 of it, 2^-17 of x).  The last bit of x is set first
// (2^-23), so that both halves of a probability are above 0 and an infinite value comes
// out with its sign; a probability of 0 has halves of 0 (2^-149 rounds to it).  One
// rounded bf16 alone, 2^-9, would be most of the step's error.
__device__ __forceinline__ void p_halves(float x, float y, uint32_t &big, uint32_t &small) {
    const uint32_t xi = __float_as_uint(x) | 1u, yi = __float_as_uint(y) | 1u;
    big = __byte_perm(xi, yi, 0x7632);
    const __nv_bfloat162 t = __floats2bfloat162_rn(__uint_as_float(xi) - __uint_as_float(xi & 0xffff0000u),
                                                   __uint_as_float(yi) - __uint_as_float(yi & 0xffff0000u));
    small = *reinterpret_cast<const uint32_t *>(&t);
}

// The gate for a state that is rounded to T.  For bf16 rows the exponential is the
// hardware's: its error of 2^-22 and that of the rounded exponent, |g| 2^-24, pass
// into the gate times a (1 - a), under 2^-22 in all where the row keeps 2^-9.
template <typename T> __device__ __forceinline__ void tree_gate(float g, float &a, float &oma) {
    if constexpr (sizeof(T) == 4) {
        gate_pair(g, a, oma);
    } else {
        // logits beyond +-80 saturate: an infinity times a gate of 0 would be NaN
        const float e = exp2f_fast(fmaxf(fminf(g * -1.44269504f, 115.f), -115.f));
        a = __fdividef(1.f, 1.f + e);
        oma = e * a;
    }
}
__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// The rows of piece `piece` of set g; false when there is none.
__device__ __forceinline__ bool slab_keys(const TreeParams &p, int h, int pos, int g, int piece, Keys &ks) {
    ks.kind = kSlab;
    const int n = tree_set_rows(p, h, pos, g, ks.row0);
    const int len = tree_piece_rows(n, p.head[h].nsplit);
    if (n == 0 || (long long)piece * len >= n) return false;
    ks.row0 += piece * len;
    ks.n = min(len, n - piece * len);
    return true;
}

// The keys of a head's local item `li`: a piece of the window's held rows, in
// item 0 the nodes, and the held rows of the dilated set if the head's keys are
// all in one item.  Returns the number of parts.
__device__ __forceinline__ int local_keys(const TreeParams &p, int h, int pos, int li, Keys *parts) {
    const int ws = p.head[h].wsplit, W = p.head[h].win;
    const int n_held = W > 0 ? min(W - 1, pos) : 0, len = (n_held + ws - 1) / ws;
    const int a = min(li * len, n_held);
    int k = 0;
    if (p.head[h].fused && slab_keys(p, h, pos, 0, 0, parts[0])) k = 1;
    parts[k].kind = kWindow;
    parts[k].row0 = pos - n_held + a;
    parts[k].n = min(len, n_held - a);
    if (parts[k].n > 0) ++k;
    if (li == 0) {
        parts[k].kind = kNodes;
        parts[k].row0 = 0;
        parts[k].n = p.N;
        ++k;
    }
    return k;
}

// What tree_combine_kernel needs to know of the tree (item 0 of every head).
__device__ __forceinline__ void tell_pieces(const TreeParams &p, const TreeInfo &ti, int b, int h, int pos) {
    const int i = threadIdx.x;
    if (i >= p.N) return;
    int np = -1;
    if (ti.valid && ti.depth[i] >= 0) {
        long long row0;
        const int n = tree_set_rows(p, h, pos, tree_set_of(p, p.head[h].dil, ti.depth[i]), row0);
        const int len = tree_piece_rows(n, p.head[h].nsplit);
        np = n == 0 ? 0 : (n + len - 1) / len;
    }
    if (ti.valid && ti.max_depth >= 0 && p.head[h].fused) np = -2;   // absent nodes too
    p.info[((size_t)b * p.H + h) * p.N + i] = np;
}

// Programmatic dependent launch: the next kernel of the step may start once
// every CTA of this one has; it waits itself before it reads.
__device__ __forceinline__ void allow_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), unsigned grid, unsigned threads, size_t smem, cudaStream_t s, bool after, const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = after ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The nodes of set g, in order (one warp).
__device__ __forceinline__ void list_nodes(const TreeParams &p, const TreeInfo &ti, int h, int g, int *nodes, int *n) {
    const int lane = threadIdx.x & 31;
    int cnt = 0;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int i = lane + 32 * u;
        const bool in = ti.depth[i] >= 0 && tree_set_of(p, p.head[h].dil, ti.depth[i]) == g;
        const unsigned mask = __ballot_sync(0xffffffffu, in);
        if (in) nodes[cnt + __popc(mask & ((1u << lane) - 1u))] = i;
        cnt += __popc(mask);
    }
    if (lane == 0) *n = cnt;
}

// 16 bytes past L1; zeros when `on` is false (the address is not read then)
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// The recurrence down the tree (128 threads), in shared memory: the tokens of all
// nodes as they come ([node][array][kCh] of the tensors' type, arrays k, v, gate
// and, with separate gates, the values' gate), overwritten by the states
// ([node][k, v][kCh] floats).  stage() starts the copies of the tokens, before the
// tree has been looked at; walk() takes kBatch nodes at a time: their tokens go to
// registers and become a and (1 - a) x side by side, then every thread follows its
// channels from parent to child, adding a * parent, and writes the rounded rows.
// Tokens lie at the end of the memory, so states reach a batch's tokens only once
// that batch is in registers: node n's state ends at (n + 1) S <= N (S - R) + (n + 1) R,
// with S and R the bytes of a node's states and tokens.
// With one warp on each of the SM's schedulers an instruction takes some five
// cycles, so their number is the time: a thread has two adjacent channels of one
// tensor where there are 128 (one channel of both tensors: 33000 cycles for 64
// nodes, 17000 so).  bf16 states take the ring's 64 KB at 64 nodes, so three CTAs share
// an SM; fp32 tokens are taken 64 channels at a time.
template <typename T, int D> struct TreeWalk {
    static constexpr int kThreads = 128, kBatch = 8;
    static constexpr int kCh = sizeof(T) == 2 ? D : 64;
    static constexpr int kMine = 2 * kCh / kThreads;                  // adjacent channels of a thread, of k or of v
    static constexpr int kState = 2 * kCh * (int)sizeof(float);       // bytes of a node's states
    static constexpr int kRow = kCh * (int)sizeof(T);                 // of one of its tokens
    static_assert(kMine == 1 || kMine == 2, "one or two channels");

    static __host__ __device__ __forceinline__ int token_bytes(int sep) { return kRow * (sep ? 4 : 3); }
    static __host__ __device__ __forceinline__ size_t bytes(int N, int sep) {
        const int r = token_bytes(sep);
        return (size_t)N * (r > kState ? r : kState);
    }
    static __device__ __forceinline__ uint8_t *tokens(uint8_t *mem, int N, int sep) {
        return mem + bytes(N, sep) - (size_t)N * token_bytes(sep);
    }

    // starts the copies of channels c0 .. c0 + kCh - 1 of all nodes
    static __device__ __forceinline__ void stage(const TreeParams &p, int b, int h, int c0, uint8_t *mem) {
        constexpr int kChunks = kRow / 16;
        const int N = p.N, r = token_bytes(p.sep);
        uint8_t *to = tokens(mem, N, p.sep);
#pragma unroll 1
        for (int y = 0; y < (p.head[h].recur ? (p.sep ? 4 : 3) : 2); ++y) {
            const T *src = static_cast<const T *>(y == 0 ? p.k : y == 1 ? p.v : p.g) + (y == 3 ? (size_t)p.B * N * p.H * D : 0) + c0;
#pragma unroll 4
            for (int e = threadIdx.x; e < N * kChunks; e += kThreads) {
                const int n = e / kChunks, ch = e % kChunks;
                cp_async16(smem_u32(to + n * r + y * kRow) + ch * 16, src + (((size_t)b * N + n) * p.H + h) * D + ch * (16 / (int)sizeof(T)), true);
            }
        }
        cp_commit();
    }
    // the queries are read after the walk: from L2 then
    static __device__ __forceinline__ void ask_queries(const TreeParams &p, int b, int h) {
        constexpr int kLines = D * (int)sizeof(T) / 128;
        for (int e = threadIdx.x; e < p.N * kLines; e += kThreads)
            prefetch_l2(static_cast<const T *>(p.q) + (((size_t)b * p.N + e / kLines) * p.H + h) * D + e % kLines * (128 / (int)sizeof(T)));
    }

    // channels c0 .. c0 + kCh - 1, staged; s0: the entry's states of k and v, out: the
    // head's node rows, both from channel c0 on
    static __device__ __noinline__ void walk(const int *parent, int N, bool sep, bool rec, const float *s0k, const float *s0v, T *out,
                                             uint8_t *mem) {
        const int r = token_bytes(sep);
        const int x = threadIdx.x / (kThreads / 2), c = threadIdx.x % (kThreads / 2) * kMine;
        float *state = reinterpret_cast<float *>(mem) + x * kCh + c;
        const uint8_t *tok = tokens(mem, N, sep) + c * (int)sizeof(T), *gates = tok + (sep ? 2 + x : 2) * kRow;
        tok += x * kRow;
        out += x * N * D + c;
        float s0[kMine];
        loads<kMine>((x ? s0v : s0k) + c, s0);
        cp_wait<0>();
        __syncthreads();
#pragma unroll 1
        for (int n0 = 0; n0 < N; n0 += kBatch) {
            float a[kBatch][kMine], u[kBatch][kMine];
            int up[kBatch];
            const uint8_t *t = tok + n0 * r, *g = gates + n0 * r;
#pragma unroll
            for (int w = 0; w < kBatch; w += 4) *reinterpret_cast<int4 *>(up + w) = *reinterpret_cast<const int4 *>(parent + n0 + w);
#pragma unroll
            for (int w = 0; w < kBatch; ++w, t += r, g += r) {
                if (n0 + w >= N) break;
                loads<kMine>(reinterpret_cast<const T *>(t), u[w]);
                if (rec) {
                    float gate[kMine];
                    loads<kMine>(reinterpret_cast<const T *>(g), gate);
#pragma unroll
                    for (int i = 0; i < kMine; ++i) {
                        float add;
                        tree_gate<T>(gate[i], a[w][i], add);
                        u[w][i] *= add;
                    }
                }
            }
            __syncthreads();   // the batch is in registers
#pragma unroll
            for (int w = 0; w < kBatch; ++w) {
                const int n = n0 + w;
                if (n >= N) break;
                if (rec) {
                    float before[kMine];
#pragma unroll
                    for (int i = 0; i < kMine; ++i) before[i] = s0[i];
                    if (up[w] >= 0) loads<kMine>(state + up[w] * 2 * kCh, before);
#pragma unroll
                    for (int i = 0; i < kMine; ++i) u[w][i] = a[w][i] * before[i] + u[w][i];
                }
                if (up[w] == RAT_NODE_ABSENT) {   // its inputs may hold anything
#pragma unroll
                    for (int i = 0; i < kMine; ++i) u[w][i] = 0.f;
                }
                stores<kMine>(state + n * 2 * kCh, u[w]);
                stores<kMine>(out + n * D, u[w]);
            }
        }
        __threadfence();   // other threads copy these rows past L1
    }
    static __device__ __forceinline__ void run(const TreeParams &p, const int *parent, int b, int h, uint8_t *mem) {
        const size_t bh = (size_t)b * p.H + h;
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += kCh) {
            if (c0 > 0) {
                __syncthreads();   // the channels before are done with
                stage(p, b, h, c0, mem);
            }
            walk(parent, p.N, p.sep != 0, p.head[h].recur != 0, p.state[0] + bh * D + c0, p.state[1] + bh * D + c0,
                 static_cast<T *>(p.node_rows) + bh * 2 * p.N * D + c0, mem);
        }
    }
};

}  // namespace rat
