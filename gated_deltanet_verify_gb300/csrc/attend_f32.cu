// attend_f32.cu -- attention of a batch of new tokens over a paged cache, on the CUDA cores, all in fp32.
//
// Rows: the G query heads that share a kv head times a block's tokens, so that a key and a value are read once for all of
// them.  out = sum_k 2^(x_k - m) v_k / sum_k 2^(x_k - m) with x = scale log2(e) q.k and the running maximum m: one pass
// over the keys, a tile of 32 at a time, the sums rescaled when m grows.
//
// A CTA of 256 threads.  Many rows (64 a block): the scores of 64 rows x 32 keys (register tiles of rows x keys, operands from
// shared memory in 16-byte reads whose rows are padded by four words), a warp's softmax for each row (a lane a key), then
// the weighted sum of the values (a lane D / 32 columns of 8 rows).  Few rows (8, 16 or 32): the bytes bind, so every key and value
// leaves shared memory once for 8 rows.  The queries lie in registers, a lane D / 32 columns of 8 rows; a warp takes its share of the
// keys, 4 at a time, whose 32 partial scores its lanes add up in 31 exchanges; for the values a warp takes its share of the
// columns and its lanes the keys, their sums added up at the block's end.  Tiles stream through 2 to 6 buffers of asynchronous
// copies.  Positions that no row may see are filled with zeros, and the scores of those that a row may not see are
// replaced, so what lies there does not matter.
//
// What bounds it.  Few rows: the copies' issue and the steps between barriers beside the cache's bytes (8 single tokens behind 20000
// positions, 32 + 8 heads of 128: 300 us, 4.4 TB/s; 3 behind 57508, 24 + 4 of 256: 321 us, 4.4 TB/s).  Many rows: reads of
// shared memory beside the products (1024 tokens behind 2000 positions, 16 + 4 heads of 128: 703 us, 30 TFLOP/s).
#include "attn.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = kTileF32;       // a lane each in the softmax
constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ float4 read4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
template <int N> __device__ __forceinline__ void store_row(float *to, const float *x) {
#pragma unroll
    for (int i = 0; i < N; ++i) to[i] = x[i];
}
// N floats (2 or 4) in one read
template <int N> __device__ __forceinline__ void read_n(const float *p, float *x) {
    if constexpr (N == 4) {
        const float4 f = read4(p);
        x[0] = f.x; x[1] = f.y; x[2] = f.z; x[3] = f.w;
    } else {
        const float2 f = *reinterpret_cast<const float2 *>(p);
        x[0] = f.x; x[1] = f.y;
    }
}
// 32 values a lane -> of each the sum over the warp's lanes, the i-th in lane i: every step halves what is left
__device__ __forceinline__ float sums_by_lane(float (&x)[32], int lane) {
#pragma unroll
    for (int n = 16; n; n >>= 1)
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const bool up = lane & n;
            const float mine = up ? x[i + n] : x[i], other = up ? x[i] : x[i + n];
            x[i] = mine + __shfl_xor_sync(kFull, other, n);
        }
    return x[0];
}

// Few rows: 8, 16 or 32, in groups of 8, each with its own kWarps warps.
template <int D, int BM> struct Shape {
    static constexpr bool kFew = BM <= 32;
    // CTAs an SM: where their tiles fit, two, which cover each other's barriers (D = 128, 8 single tokens behind 20000 positions:
    // 309 us, with one 425; 1024 tokens behind 2000: 709 and 945)
    static constexpr int kCtas = D <= 128 ? 2 : 1;
    static constexpr int kBuffers = !kFew ? 2 : D == 64 ? 6 : 3;
    static constexpr int kGroups = kFew ? BM / 8 : 1, kWarps = 8 / kGroups;
    static constexpr int kQ = D / 32, kQV = kQ < 4 ? kQ : 4;                // of a row, a lane's columns, and as it reads them
    static constexpr int kLanes = D / (4 * kWarps), kParts = 32 / kLanes;   // lanes side by side, 4 columns each; parts of the keys
    static constexpr int kKeys = kTile / kParts, kKeysV = kKeys < 4 ? kKeys : 4;
};

template <int D, int BM> struct Smem {
    float q[Shape<D, BM>::kFew ? 1 : BM][D + 4];
    float k[Shape<D, BM>::kBuffers][kTile][D + 4];
    float v[Shape<D, BM>::kBuffers][kTile][Shape<D, BM>::kFew ? D + 4 : D];
    float p[BM][kTile + 4];
    float m[BM], l[BM], scale[BM];
    unsigned long long line[BM];      // a tree's nodes that a row sees
    int at[BM];                       // a row's token, -1: none
    int position[BM];                 // where a row's token is
    int parents[64], depth[64];
    int scratch[kThreads / 32 + 2];
};

template <int D, int BM>
__global__ void __launch_bounds__(kThreads, (Shape<D, BM>::kCtas)) attend_kernel(const __grid_constant__ AttendArgs a) {
    extern __shared__ __align__(16) unsigned char raw[];
    Smem<D, BM> &sm = *reinterpret_cast<Smem<D, BM> *>(raw);
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, c = blockIdx.x;
    auto chk = [&](const void *p, size_t bytes, const void *base, size_t extent) { return in_bounds(p, bytes, base, extent, a.d_status); };
    Share share;
    Place at = find_place<kTile, kThreads>(a, c, share, sm.scratch);
    if (c == 0)
        for (int s = tid; s < a.B; s += kThreads) {
            int past;
            if (live_tokens(a.kv, a.length, a.T, s, past, a.d_status) < 0) report(a.d_status, GDN_ERR_LENGTH);
        }
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    if (c >= share.ctas) return;
    int left = share.start(c + 1) - share.start(c);
    const int page = 1 << a.kv.page_log2;
    const float scale2 = a.scale * 1.4426950408889634f;

    constexpr int kCols = D / 32;                 // columns a lane holds of the sums
    constexpr int kRowsW = BM / 8;                // rows a warp holds
    using Sh = Shape<D, BM>;
    constexpr bool kFew = Sh::kFew;
    constexpr int kBuffers = Sh::kBuffers;
    // few rows: this warp's group of 8, its place among the group's, the lane's columns and its part of the keys
    const int row0 = wid / Sh::kWarps * 8, wg = wid % Sh::kWarps, column = (wg * Sh::kLanes + lane % Sh::kLanes) * 4, kpart = lane / Sh::kLanes;
    float qr[kFew ? 8 : 1][Sh::kQ];
    float o[kFew ? 8 : kRowsW][kFew ? 4 : kCols];

    bool first_block = true;
    int pair = at.pair;
    Span span = block_span<kTile>(a, pair / a.n_tb, pair % a.n_tb);
    int kvh = at.offset / span.n, j = at.offset % span.n;
    while (left > 0) {
        const int s = pair / a.n_tb;
        const int rows = (span.t1 - span.t0) * a.G;
        const int j0 = j, j1 = min(span.n, j0 + left);
        const int32_t *table = a.kv.table + (size_t)s * a.kv.max_pages;
        const int sink = min(a.n_sink, span.lo);

        // ---- a tile's copies.  Lane r knows where the tile's row r lies, its page id having been read a tile ahead
        auto page_id = [&](int jj) {
            if (jj >= j1) return -1;
            const int key = span.tile(jj) * kTile + lane;
            return key < span.hi && (key >= span.lo || key < sink) ? page_at(a.kv, table + (key >> a.kv.page_log2), a.d_status) : -1;
        };
        int id = page_id(j0);
        auto fetch = [&](int jj, int buf) {
            if (jj < j1) {
                const int key = span.tile(jj) * kTile + lane;
                long long row = -1;
                if (key < span.hi && (key >= span.lo || key < sink)) {
                    if (id < 0 || id >= a.kv.n_pages) report(a.d_status, GDN_ERR_PAGE);
                    else row = (long long)id * a.kv.page_stride + ((size_t)kvh * page + (key & (page - 1))) * D;
                }
                id = page_id(jj + 1);
                constexpr int kVecs = D / 4;
#pragma unroll
                for (int n = 0; n < kTile * kVecs / kThreads; ++n) {
                    const int i = tid + n * kThreads, r = i / kVecs, x = (i % kVecs) * 4;
                    const long long from = __shfl_sync(kFull, row, r);
                    const bool there = from >= 0 && chk(static_cast<const float *>(a.kv.k) + from + x, 16, a.kv.k, a.kv.ext_pool) &&
                                       chk(static_cast<const float *>(a.kv.v) + from + x, 16, a.kv.v, a.kv.ext_pool);
                    const int bytes = there ? 16 : 0;                // of the 16 written, those that are read
                    const long long off = there ? from + x : 0;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(
                                     (uint32_t)__cvta_generic_to_shared(&sm.k[buf][r][x])), "l"(static_cast<const float *>(a.kv.k) + off),
                                 "r"(bytes) : "memory");
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(
                                     (uint32_t)__cvta_generic_to_shared(&sm.v[buf][r][x])), "l"(static_cast<const float *>(a.kv.v) + off),
                                 "r"(bytes) : "memory");
                }
            }
            asm volatile("cp.async.commit_group;\n" ::: "memory");
        };

        __syncthreads();                          // the block before no longer reads shared memory
#pragma unroll 1
        for (int n = 0; n + 1 < kBuffers; ++n) fetch(j0 + n, n);
        // ---- the block's rows: to registers where they are few, else to shared memory
        auto query = [&](int r) {
            return static_cast<const float *>(a.q) +
                   (((size_t)s * a.T + span.t0 + r / a.G) * a.H + (size_t)kvh * a.G + r % a.G) * D;
        };
        if constexpr (kFew) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool on = row0 + i < rows && chk(query(row0 + i), D * 4, a.q, a.ext_q);
                const float *from = on || chk(query(0), D * 4, a.q, a.ext_q) ? query(on ? row0 + i : 0) : static_cast<const float *>(a.q);
#pragma unroll
                for (int e = 0; e < Sh::kQ; e += Sh::kQV) {
                    read_n<Sh::kQV>(from + e * 32 + lane * Sh::kQV, &qr[i][e]);
#pragma unroll
                    for (int f = 0; f < Sh::kQV; ++f) qr[i][e + f] = on ? qr[i][e + f] : 0.f;
                }
            }
        } else {
            for (int i = tid; i < BM * (D / 4); i += kThreads) {
                const int r = i / (D / 4), x = (i % (D / 4)) * 4;
                const bool on = r < rows && chk(query(r) + x, 16, a.q, a.ext_q);
                *reinterpret_cast<float4 *>(&sm.q[r][x]) = on ? read4(query(r) + x) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
        if (a.parent && tid < span.t1) sm.parents[tid] = parent_of(a.parent, a.T, s, tid, a.ext_nodes, a.d_status, true);
        __syncthreads();
        if (a.parent && tid < span.t1) {
            int d = 0;
            for (int p = sm.parents[tid]; p >= 0; p = sm.parents[p]) ++d;
            sm.depth[tid] = d;
        }
        __syncthreads();
        for (int r = tid; r < BM; r += kThreads) {
            const int t = r < rows ? span.t0 + r / a.G : -1;
            sm.at[r] = t;
            sm.m[r] = -INFINITY;
            sm.l[r] = 0.f;
            sm.scale[r] = 1.f;
            unsigned long long line = 0;
            if (a.parent)
                for (int p = t; p >= 0; p = sm.parents[p]) line |= 1ull << p;
            sm.line[r] = line;
            sm.position[r] = span.past + (a.parent && t >= 0 ? sm.depth[t] : t);
        }
#pragma unroll
        for (int i = 0; i < (int)(sizeof o / sizeof o[0]); ++i)
#pragma unroll
            for (int e = 0; e < (int)(sizeof o[0] / sizeof o[0][0]); ++e) o[i][e] = 0.f;

        int buf = 0;
        for (int jj = j0; jj < j1; ++jj, buf = buf + 1 == kBuffers ? 0 : buf + 1) {
            const int k0 = span.tile(jj) * kTile;
            asm volatile("cp.async.wait_group %0;\n" ::"n"(kBuffers - 2) : "memory");
            __syncthreads();
            if constexpr (kFew) {
                // ---- scores: a warp 32 / kWarps keys for 8 rows, four keys at a time
#pragma unroll
                for (int n = 0; n < kTile / Sh::kWarps; n += 4) {
                    const int key = wg * (kTile / Sh::kWarps) + n;
                    float x[32];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float kr[Sh::kQ];
#pragma unroll
                        for (int e = 0; e < Sh::kQ; e += Sh::kQV) read_n<Sh::kQV>(&sm.k[buf][key + k][e * 32 + lane * Sh::kQV], kr + e);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            x[k * 8 + i] = qr[i][0] * kr[0];
#pragma unroll
                            for (int e = 1; e < Sh::kQ; ++e) x[k * 8 + i] = fmaf(qr[i][e], kr[e], x[k * 8 + i]);
                        }
                    }
                    sm.p[row0 + lane % 8][key + lane / 8] = sums_by_lane(x, lane) * scale2;
                }
            } else {
                // ---- scores: rows rg + 16 i, keys kg + 16 n
                constexpr int kR = BM / 16;
                const int rg = tid >> 4, kg = tid & 15;
                float x[kR][2];
#pragma unroll
                for (int i = 0; i < kR; ++i) x[i][0] = x[i][1] = 0.f;
#pragma unroll 4
                for (int d = 0; d < D; d += 4) {
                    const float4 ka = *reinterpret_cast<const float4 *>(&sm.k[buf][kg][d]);
                    const float4 kb = *reinterpret_cast<const float4 *>(&sm.k[buf][kg + 16][d]);
#pragma unroll
                    for (int i = 0; i < kR; ++i) {
                        const float4 f = *reinterpret_cast<const float4 *>(&sm.q[rg + 16 * i][d]);
                        x[i][0] = fmaf(f.x, ka.x, fmaf(f.y, ka.y, fmaf(f.z, ka.z, fmaf(f.w, ka.w, x[i][0]))));
                        x[i][1] = fmaf(f.x, kb.x, fmaf(f.y, kb.y, fmaf(f.z, kb.z, fmaf(f.w, kb.w, x[i][1]))));
                    }
                }
#pragma unroll
                for (int i = 0; i < kR; ++i) {
                    sm.p[rg + 16 * i][kg] = x[i][0] * scale2;
                    sm.p[rg + 16 * i][kg + 16] = x[i][1] * scale2;
                }
            }
            __syncthreads();
            // The next tile's copies, to where the tile before was, which all have read by now (sent off here, beside the softmax,
            // and without a barrier at the loop's end: 300 us for 8 tokens behind 20000, before the scores 309).
            fetch(jj + kBuffers - 1, buf == 0 ? kBuffers - 1 : buf - 1);
            // ---- softmax: a warp a row, a lane a key
            for (int r = wid; r < (BM <= 16 ? BM : rows); r += 8) {
                const int t = sm.at[r], key = k0 + lane, node = key - span.past;
                bool sees = t >= 0 && node <= t;
                int where = key;
                if (a.parent && node >= 0 && node < span.t1) {
                    sees = sees && (sm.line[r] >> node & 1);
                    where = span.past + sm.depth[node];
                }
                if (a.window) sees = sees && (where > sm.position[r] - a.window || where < a.n_sink);
                const float x = sees ? sm.p[r][lane] : -INFINITY;
                float top = x;
#pragma unroll
                for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, d));
                const float m = sm.m[r], to = fmaxf(m, top);
                const float p = sees ? exp2f(x - to) : 0.f;
                float sum = p;
#pragma unroll
                for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(kFull, sum, d);
                sm.p[r][lane] = p;
                if (lane == 0) {
                    const float f = m == to ? 1.f : exp2f(m - to);
                    sm.scale[r] = f;
                    sm.l[r] = sm.l[r] * f + sum;
                    sm.m[r] = to;
                }
            }
            if constexpr (kFew) {
                __syncthreads();
                // ---- values: a group's warps share out the columns, a warp's lanes the keys
                bool moved = false;
                float f[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) moved |= (f[i] = sm.scale[row0 + i]) != 1.f;
                if (moved)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[i][e] *= f[i];
#pragma unroll
                for (int k = 0; k < Sh::kKeys; k += Sh::kKeysV) {
                    const int key = kpart * Sh::kKeys + k;
                    float v[Sh::kKeysV][4];
#pragma unroll
                    for (int n = 0; n < Sh::kKeysV; ++n) read_n<4>(&sm.v[buf][key + n][column], v[n]);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float w[Sh::kKeysV];
                        read_n<Sh::kKeysV>(&sm.p[row0 + i][key], w);
#pragma unroll
                        for (int n = 0; n < Sh::kKeysV; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[i][e] = fmaf(w[n], v[n][e], o[i][e]);
                    }
                }
            } else {
                __syncwarp();
                // ---- values: a warp's rows are its own (wid + 8 i), a lane's columns
                constexpr int V = kCols < 4 ? kCols : 4;
#pragma unroll
                for (int i = 0; i < kRowsW; ++i) {
                    const float f = sm.scale[wid + 8 * i];
#pragma unroll
                    for (int e = 0; e < kCols; ++e) o[i][e] *= f;
                }
#pragma unroll 2
                for (int k = 0; k < kTile; k += 4) {
                    float v[4][kCols];
#pragma unroll
                    for (int n = 0; n < 4; ++n)
#pragma unroll
                        for (int e = 0; e < kCols; e += V) {
                            const float *from = &sm.v[buf][k + n][(e / V * 32 + lane) * V];
                            if constexpr (V == 4) {
                                const float4 f = *reinterpret_cast<const float4 *>(from);
                                v[n][e] = f.x; v[n][e + 1] = f.y; v[n][e + 2] = f.z; v[n][e + 3] = f.w;
                            } else {
                                const float2 f = *reinterpret_cast<const float2 *>(from);
                                v[n][e] = f.x; v[n][e + 1] = f.y;
                            }
                        }
#pragma unroll
                    for (int i = 0; i < kRowsW; ++i) {
                        const float4 p = *reinterpret_cast<const float4 *>(&sm.p[wid + 8 * i][k]);
#pragma unroll
                        for (int e = 0; e < kCols; ++e)
                            o[i][e] = fmaf(p.x, v[0][e], fmaf(p.y, v[1][e], fmaf(p.z, v[2][e], fmaf(p.w, v[3][e], o[i][e]))));
                    }
                }
            }
        }
        // ---- the block's sums: its output, or a part of it
        const bool whole = j0 == 0 && j1 == span.n;
        const size_t part = size_t(2 * c + (first_block ? 0 : 1)) * a.part_rows;
        float *out = static_cast<float *>(a.out) + (((size_t)s * a.T + span.t0) * a.H + (size_t)kvh * a.G) * D;
        auto place = [&](int r) { return whole ? out + ((size_t)(r / a.G) * a.H + r % a.G) * D : a.partial + (part + r) * D; };
        auto put = [&](const float *to, size_t bytes) { return whole ? chk(to, bytes, a.out, a.ext_q) : chk(to, bytes, a.partial, a.ext_partial); };
        if constexpr (kFew) {
#pragma unroll
            for (int d = Sh::kLanes; d < 32; d *= 2)
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[i][e] += __shfl_xor_sync(kFull, o[i][e], d);
            if (!whole && tid < rows && chk(a.stats + part + tid, 8, a.stats, a.ext_stats)) a.stats[part + tid] = make_float2(sm.m[tid], sm.l[tid]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = row0 + i;
                if (r >= rows || kpart != i % Sh::kParts || !put(place(r) + column, 16)) continue;
                const float f = whole ? 1.f / sm.l[r] : 1.f;
                *reinterpret_cast<float4 *>(place(r) + column) = make_float4(o[i][0] * f, o[i][1] * f, o[i][2] * f, o[i][3] * f);
            }
        } else {
            constexpr int V = kCols < 4 ? kCols : 4;
#pragma unroll
            for (int i = 0; i < kRowsW; ++i) {
                const int r = wid + 8 * i;
                if (r >= rows) continue;
                const float l = sm.l[r], f = whole ? 1.f / l : 1.f;
                if (!whole && lane == 0 && chk(a.stats + part + r, 8, a.stats, a.ext_stats)) a.stats[part + r] = make_float2(sm.m[r], l);
#pragma unroll
                for (int e = 0; e < kCols; ++e) o[i][e] *= f;
#pragma unroll
                for (int e = 0; e < kCols; e += V)
                    if (put(place(r) + (e / V * 32 + lane) * V, 4 * V)) store_row<V>(place(r) + (e / V * 32 + lane) * V, &o[i][e]);
            }
        }
        // ---- the next block
        left -= j1 - j0;
        first_block = false;
        j = 0;
        if (left > 0 && ++kvh == a.Hk) {
            kvh = 0;
            do {
                if (++pair == a.B * a.n_tb) break;        // never, unless the lengths change under the call
                span = block_span<kTile>(a, pair / a.n_tb, pair % a.n_tb);
            } while (span.n == 0);
            if (pair == a.B * a.n_tb) break;
        }
    }
    asm volatile("cp.async.wait_all;\n" ::: "memory");
}

template <int D, int BM> cudaError_t launch(const AttendArgs &a, cudaStream_t stream) {
    const int smem = int(sizeof(Smem<D, BM>));
    static PerContext<int> limits;
    unsigned long long ctx = 0;
    int set = 0;
    if (!current_context_id(&ctx) || !limits.get(ctx, &set)) {
        const cudaError_t e = cudaFuncSetAttribute(attend_kernel<D, BM>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        if (current_context_id(&ctx)) limits.put(ctx, 1);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(a.ctas), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, attend_kernel<D, BM>, a);
    return e != cudaSuccess ? e : launch_attend_join(a, GDN_F32, stream);
}

template <int BM> cudaError_t launch_d(const AttendArgs &a, cudaStream_t stream) {
    return a.D == 64 ? launch<64, BM>(a, stream) : a.D == 128 ? launch<128, BM>(a, stream) : launch<256, BM>(a, stream);
}

}  // namespace

// Rows of a block: no more than a slot has, in steps of 2, up to 64: a wider block spends its time on rows that are not there (8
// single tokens behind 20000 positions with G = 4, D = 128: 309 us with 8 rows, 494 with 16; 8 slots of 20 rows over 4000:
// 97 us with 32, 128 with 64).
static int block_rows(int T, int G) {
    const long long rows = (long long)T * G;
    return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

AttendBlock attend_f32_block(int T, int G, int D) {
    const int rows = block_rows(T, G);
    return {rows, rows / G < T ? rows / G : T, 1, 0, (D <= 128 ? 2 : 1) * kAttendCtas};
}

cudaError_t launch_attend_f32(const AttendArgs &a, cudaStream_t stream) {
    const int rows = block_rows(a.T, a.G);
    return rows == 8 ? launch_d<8>(a, stream) : rows == 16 ? launch_d<16>(a, stream)
           : rows == 32 ? launch_d<32>(a, stream) : launch_d<64>(a, stream);
}

}  // namespace gdn
