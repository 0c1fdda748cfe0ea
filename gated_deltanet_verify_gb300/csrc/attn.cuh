// attn.cuh -- argument blocks of the full-attention side of a verify step (append.cu, attend.cu, attend_f32.cu) and
// what its kernels share: how a paged cache is addressed, what a new token may see, and how the work is dealt out.
#pragma once

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
    size_t ext_kv, ext_table;         // bytes, for a checked build
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
    int ctas;
    float *partial;                   // [2 * ctas][TB * G][D]: unnormalised sums of split blocks
    float2 *stats;                    // [2 * ctas][TB * G]: their maxima (in powers of two) and sums
    int *d_status;
};

// What the workspace holds; rows: of a block, at most.
constexpr int kAttendCtas = 152;      // CTAs of a launch, at most: one on every SM
inline size_t attend_partial_bytes(int rows, int D) { return size_t(2) * kAttendCtas * rows * D * sizeof(float); }
inline size_t attend_stats_bytes(int rows) { return size_t(2) * kAttendCtas * rows * sizeof(float2); }

// Return a cudaError_t of the launch (cudaSuccess when enqueued).
cudaError_t launch_append(const AppendArgs &a, gdn_dtype dtype, int sm_count, cudaStream_t stream);
cudaError_t launch_attend_f32(AttendArgs a, int sm_count, cudaStream_t stream);
cudaError_t launch_attend_bf16(const AttendArgs &a, int sm_count, cudaStream_t stream);
// rows of a block at most, for the workspace
int attend_f32_block_rows(int T, int G);
int attend_bf16_block_rows(int T, int G, int D);

#ifdef __CUDACC__

__device__ __forceinline__ void report(int *d_status, gdn_status code) {
    if (d_status) atomicCAS(d_status, int(GDN_OK), int(code));
}

// The real tokens of slot s, or -1 where its past or its length cannot be.
__device__ __forceinline__ int live_tokens(const KvPages &kv, const int32_t *length, int T, int s, int &past) {
    past = kv.past[s];
    const int n = length ? length[s] : T;
    const long long room = (long long)kv.max_pages << kv.page_log2;
    if (n < 0 || n > T || past < 0 || (long long)past + n > room) return -1;
    return n;
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
    const int n = live_tokens(a.kv, a.length, a.T, s, p.past);
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

// The whole work is a row of tiles: blocks of rows in the order (slot, token block), kv heads within one, key tiles
// within one.  CTA c of n takes the tiles [start(c), start(c + 1)), so every SM has the same share whatever the
// lengths; the block at either end of its share may be split with its neighbours, whose partial sums are joined later.
struct Share {
    long long total;
    int ctas;
    __device__ __forceinline__ long long start(int c) const { return total * c / ctas; }
    // the CTA that has this tile
    __device__ __forceinline__ int owner(long long tile) const {
        int c = int(min((long long)ctas - 1, tile * ctas / total));
        while (c + 1 < ctas && start(c + 1) <= tile) ++c;
        while (c > 0 && start(c) > tile) --c;
        return c;
    }
};

// Where a tile lies: pair = slot * n_tb + token block, then tile `offset` of its Hk * n.
struct Place {
    int pair;
    long long offset;
};

// Found by the whole CTA together (THREADS of them): the sum of all tiles, then the pair that tile `share.start(c)` is
// in.  scratch: THREADS / 32 + 4 long longs of shared memory.
template <int TK, int THREADS>
__device__ __forceinline__ Place find_place(const AttendArgs &a, int c, Share &share, long long *scratch) {
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, pairs = a.B * a.n_tb;
    const int chunk = (pairs + THREADS - 1) / THREADS;
    const int i0 = min(pairs, tid * chunk), i1 = min(pairs, i0 + chunk);
    long long mine = 0;
    for (int i = i0; i < i1; ++i) mine += block_span<TK>(a, i / a.n_tb, i % a.n_tb).n;
    mine *= a.Hk;
    long long upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += o;
    }
    if (lane == 31) scratch[wid] = upto;
    __syncthreads();
    long long before = 0, total = 0;
    for (int w = 0; w < THREADS / 32; ++w) {
        const long long v = scratch[w];
        before += w < wid ? v : 0;
        total += v;
    }
    share.total = total;
    share.ctas = int(min((long long)a.ctas, total));
    long long *found = scratch + THREADS / 32;
    if (total > 0 && c < share.ctas) {
        const long long target = share.start(c);
        before += upto - mine;
        if (mine > 0 && target >= before && target < before + mine) {
            long long at = target - before;
            int i = i0;
            for (;; ++i) {
                const long long n = (long long)block_span<TK>(a, i / a.n_tb, i % a.n_tb).n * a.Hk;
                if (at < n) break;
                at -= n;
            }
            found[0] = i;
            found[1] = at;
        }
    }
    __syncthreads();
    return Place{int(found[0]), found[1]};
}

#endif  // __CUDACC__

}  // namespace gdn
