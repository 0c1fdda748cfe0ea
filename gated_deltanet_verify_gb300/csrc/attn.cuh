// attn.cuh -- argument blocks of the full-attention side of a verify step (append.cu, attend.cu, attend_f32.cu) and
// what its kernels share: how a paged cache is addressed, what a new token may see, and how the work is dealt out.
#pragma once

#include "check.cuh"
#include "internal.cuh"

namespace gdn {

// A paged key/value cache: position p of slot s, kv head h lies at
//   pool + table[s][p / page] * page_stride + (h * page + p % page) * D.
struct KvPages {
    void *k, *v;
    const int32_t *table;             // [B][max_pages]
    const int32_t *past;              // [B]: positions a slot holds before the batch
    long long page_stride;            // elements
    int n_pages, max_pages;
    int page_log2;                    // tokens a page: 2^page_log2
    size_t ext_past, ext_table, ext_pool;     // bytes, for a checked build (as all ext_...): of past (and lengths), table, k and v
};

// Rotation and append of a batch's keys and values (append.cu).
struct AppendArgs {
    int B, T, H, Hk, D;
    KvPages kv;
    const void *q, *k, *v;            // rows of H / Hk / Hk heads; q may be NULL
    long long ld_q, ld_k, ld_v;       // row strides (elements)
    void *q_out;                      // [B][T][H][D]
    int rope_dims, adjacent;
    const float *freq, *q_norm, *k_norm;
    float eps;
    const int32_t *length, *parent, *path;
    int *d_status;
    size_t ext_q, ext_k, ext_v, ext_out, ext_freq, ext_norm, ext_nodes;     // nodes: parent or path
};

// Attention of a batch over the cache (attend.cu, attend_f32.cu).
struct AttendArgs {
    int B, T, H, Hk, D, G;            // G = H / Hk query heads share a kv head
    KvPages kv;
    const void *q;                    // [B][T][H][D]
    void *out;
    const int32_t *length, *parent;
    float scale;
    int window, n_sink;
    int TB, n_tb;                     // tokens a block of rows takes (TB * G rows), blocks a slot
    int ctas;                         // of the launch
    int least;                        // tiles of a CTA's share, at least (if there are so many)
    int pad;                          // what a block costs beside its tiles, in tiles
    int part_rows;                    // rows of a part in the workspace
    float *partial;                   // [2 * ctas][part_rows][D]: unnormalised sums of split blocks
    float2 *stats;                    // [2 * ctas][part_rows]: their maxima (in powers of two) and sums
    int *d_status;
    size_t ext_q, ext_nodes, ext_partial, ext_stats;      // q and out; parent; the workspace's two halves
};

constexpr int kTileF32 = 32, kTileBf16 = 128;   // keys a tile

constexpr int kAttendCtas = 152;      // CTAs of a launch: one on every SM, or two (f32)

// How the rows of a slot and a kv head are cut up.
struct AttendBlock {
    int rows;                         // of a block, at most (what a part of the workspace holds)
    int tokens;                       // that a block takes
    int least;                        // tiles a CTA takes at least
    int pad;                          // what a block costs beside its tiles, in tiles
    int ctas;                         // of a launch, at most
};
AttendBlock attend_f32_block(int T, int G, int D);
AttendBlock attend_bf16_block(int T, int G, int D);
// What the workspace holds.
inline size_t attend_partial_bytes(const AttendBlock &b, int D) { return size_t(2) * b.ctas * b.rows * D * sizeof(float); }
inline size_t attend_stats_bytes(const AttendBlock &b) { return size_t(2) * b.ctas * b.rows * sizeof(float2); }

// Return a cudaError_t of the launch (cudaSuccess when enqueued).
cudaError_t launch_append(const AppendArgs &a, gdn_dtype dtype, int sm_count, cudaStream_t stream);
cudaError_t launch_attend_f32(const AttendArgs &a, cudaStream_t stream);
cudaError_t launch_attend_bf16(const AttendArgs &a, cudaStream_t stream);
// the rows of blocks that several CTAs shared, from their parts
cudaError_t launch_attend_join(const AttendArgs &a, gdn_dtype dtype, cudaStream_t stream);

#ifdef __CUDACC__

__device__ __forceinline__ void report(int *d_status, gdn_status code) {
    if (d_status) atomicCAS(d_status, int(GDN_OK), int(code));
}

// The real tokens of slot s, or -1 where its past or its length cannot be.
__device__ __forceinline__ int live_tokens(const KvPages &kv, const int32_t *length, int T, int s, int &past, int *d_status) {
    past = 0;
    if (!in_bounds(kv.past + s, 4, kv.past, kv.ext_past, d_status) ||
        (length && !in_bounds(length + s, 4, length, kv.ext_past, d_status)))
        return -1;
    past = kv.past[s];
    const int n = length ? length[s] : T;
    const long long room = (long long)kv.max_pages << kv.page_log2;
    if (n < 0 || n > T || past < 0 || (long long)past + n > room) return -1;
    return n;
}

// An entry of the page table.
__device__ __forceinline__ int page_at(const KvPages &kv, const int32_t *at, int *d_status) {
    return in_bounds(at, 4, kv.table, kv.ext_table, d_status) ? *at : -1;
}
// The parent of node t of slot s, of T nodes; one that cannot be (and a parent outside its buffer) hangs from the past.
__device__ __forceinline__ int parent_of(const int32_t *parent, int T, int s, int t, size_t extent, int *d_status, bool report_it) {
    const int32_t *at = parent + (size_t)s * T + t;
    const int p = in_bounds(at, 4, parent, extent, d_status) ? *at : -1;
    if (p >= -1 && p < t) return p;
    if (report_it) report(d_status, GDN_ERR_TREE);
    return -1;
}

// The key tiles (of TK positions) that a block of rows, tokens [t0, t1) of slot s, reads: those of the first positions that
// stay visible, then those from the window's lower end to the last position any of its tokens sees.
struct Span {
    int past, t0, t1;
    int lo, hi;                       // the block sees positions [lo, hi) and those below min(n_sink, lo)
    int sink_tiles, first, n;         // tiles: 0 .. sink_tiles - 1, then first ..; n in all
    __device__ __forceinline__ int tile(int j) const { return j < sink_tiles ? j : first + j - sink_tiles; }
};

template <int TK>
__device__ __forceinline__ Span block_span(const AttendArgs &a, int s, int tb) {
    Span p;
    const int n = live_tokens(a.kv, a.length, a.T, s, p.past, a.d_status);
    p.t0 = tb * a.TB;
    p.t1 = min(n, p.t0 + a.TB);
    p.sink_tiles = p.first = p.n = p.lo = p.hi = 0;
    if (p.t0 >= n) return p;
    p.hi = p.past + p.t1;
    // a tree's nodes lie at past + depth, which is 0 at the least
    const int lowest = p.past + (a.parent ? 0 : p.t0);
    p.lo = a.window ? max(0, lowest - a.window + 1) : 0;
    p.first = p.lo / TK;
    p.sink_tiles = min((min(a.n_sink, p.lo) + TK - 1) / TK, p.first);
    p.n = p.sink_tiles + (p.hi + TK - 1) / TK - p.first;
    return p;
}

// The whole work is a row of tiles (fewer than 2^31, as the host checks): blocks of rows in the order (slot, token block), kv
// heads within one, key tiles within one.  Of n CTAs, CTA c takes the tiles [start(c), start(c + 1)), so every SM has the
// same share whatever the lengths; the block at either end of its share may be split with its neighbours, whose partial
// sums are joined later.  A block begins with `pad` tiles that are not there, for what it costs beside its tiles: without
// them the CTAs with the most blocks ended last (64 slots in a window of 1024, 10 tiles a block: 46 us where it is 41 with
// them; trees of 64: 53 and 42).
struct Share {
    int total, ctas, base, more;      // the first `more` CTAs take base + 1 tiles, the others base
    __device__ __forceinline__ void set(int t, const AttendArgs &a) {
        total = t;
        ctas = min(a.ctas, (t + a.least - 1) / a.least);
        base = ctas ? t / ctas : 0;
        more = t - base * ctas;
    }
    __device__ __forceinline__ int start(int c) const { return base * c + min(c, more); }
    // the CTA that has this tile
    __device__ __forceinline__ int owner(int tile) const {
        const int wide = (base + 1) * more;
        return tile < wide ? tile / (base + 1) : more + (tile - wide) / base;
    }
};

// Where a tile lies: pair = slot * n_tb + token block, then tile `offset` of its Hk * (pad + n).
struct Place {
    int pair, offset;
};

// A warp finds its way by itself where there are at most kScanPairs pairs; more take the whole CTA.  (Rolled loops: a launch
// starts with a cold instruction cache, and unrolled by 8 this took 4600 cycles for one pair.)
constexpr int kScanPairs = 256;
constexpr unsigned kWarp = 0xffffffffu;

template <int TK> __device__ __forceinline__ int pair_tiles(const AttendArgs &a, int pair) {
    const int n = pair < a.B * a.n_tb ? block_span<TK>(a, pair / a.n_tb, pair % a.n_tb).n : 0;
    return n ? (n + a.pad) * a.Hk : 0;
}
__device__ __forceinline__ int scan_warp(int v) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(kWarp, v, d);
        if ((threadIdx.x & 31) >= d) v += o;
    }
    return v;
}
template <int TK> __device__ __forceinline__ int scan_total(const AttendArgs &a) {
    int sum = 0;
#pragma unroll 1
    for (int i = 0; i < a.B * a.n_tb; i += 32) sum += pair_tiles<TK>(a, i + (threadIdx.x & 31));
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(kWarp, sum, d);
    return sum;
}
// the pair that a tile (below the total) is in
template <int TK> __device__ __forceinline__ Place scan_find(const AttendArgs &a, int tile) {
    int before = 0, i = 0;
#pragma unroll 1
    for (;; i += 32) {
        const int n = pair_tiles<TK>(a, i + (threadIdx.x & 31)), upto = before + scan_warp(n);
        const unsigned past = __ballot_sync(kWarp, upto > tile);
        if (past || i + 32 >= a.B * a.n_tb) {
            const int l = past ? __ffs(past) - 1 : 0;
            return Place{i + l, tile - __shfl_sync(kWarp, upto - n, l)};
        }
        before = __shfl_sync(kWarp, upto, 31);
    }
}
// the first tile of a pair
template <int TK> __device__ __forceinline__ int scan_begin(const AttendArgs &a, int pair) {
    int before = 0;
#pragma unroll 1
    for (int i = 0; i < pair; i += 32) {
        const int at = i + (threadIdx.x & 31);
        before += at < pair ? pair_tiles<TK>(a, at) : 0;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) before += __shfl_xor_sync(kWarp, before, d);
    return before;
}

// a warp by itself, with at most kScanPairs pairs
template <int TK> __device__ __forceinline__ Place warp_place(const AttendArgs &a, int c, Share &share) {
    if (a.B * a.n_tb > 32) {
        share.set(scan_total<TK>(a), a);
        return c < share.ctas ? scan_find<TK>(a, share.start(c)) : Place{0, 0};
    }
    const int n = pair_tiles<TK>(a, threadIdx.x & 31), upto = scan_warp(n);
    share.set(__shfl_sync(kWarp, upto, 31), a);
    if (c >= share.ctas) return Place{0, 0};
    const int tile = share.start(c), l = __ffs(__ballot_sync(kWarp, upto > tile)) - 1;
    return Place{l, tile - __shfl_sync(kWarp, upto - n, l)};
}

// The sum of all tiles, then the pair that tile `share.start(c)` is in; called by the whole CTA (THREADS of them).
// scratch: THREADS / 32 + 2 words of shared memory.
template <int TK, int THREADS>
__device__ __forceinline__ Place find_place(const AttendArgs &a, int c, Share &share, int *scratch) {
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, pairs = a.B * a.n_tb;
    if (pairs <= kScanPairs) return warp_place<TK>(a, c, share);
    const int chunk = (pairs + THREADS - 1) / THREADS;
    const int i0 = min(pairs, tid * chunk), i1 = min(pairs, i0 + chunk);
    int mine = 0;
#pragma unroll 1
    for (int i = i0; i < i1; ++i) mine += pair_tiles<TK>(a, i);
    const int upto = scan_warp(mine);
    int *found = scratch + THREADS / 32;
    if (lane == 31) scratch[wid] = upto;
    if (tid < 2) found[tid] = 0;          // what a CTA without a share gets: a place that is there
    __syncthreads();
    int before = upto - mine, total = 0;
    for (int w = 0; w < THREADS / 32; ++w) {
        const int v = scratch[w];
        before += w < wid ? v : 0;
        total += v;
    }
    share.set(total, a);
    if (c < share.ctas) {
        int at = share.start(c) - before;
        if (at >= 0 && at < mine) {
            int i = i0;
#pragma unroll 1
            for (;; ++i) {
                const int n = pair_tiles<TK>(a, i);
                if (at < n || i + 1 == i1) break;
                at -= n;
            }
            found[0] = i;
            found[1] = at;
        }
    }
    __syncthreads();
    return Place{found[0], found[1]};
}

#endif  // __CUDACC__

}  // namespace gdn
