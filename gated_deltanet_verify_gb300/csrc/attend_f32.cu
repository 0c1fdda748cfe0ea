// attend_f32.cu -- attention of a batch of new tokens over a paged cache, on the CUDA cores, all in fp32.
//
// Rows: the G query heads that share a kv head times a block's tokens, so that a key and a value are read once for all of
// them.  out = sum_k 2^(x_k - m) v_k / sum_k 2^(x_k - m) with x = scale log2(e) q.k and the running maximum m: one pass
// over the keys, a tile of 32 at a time, the sums rescaled when m grows.
//
// A CTA of 256 threads: the scores of BM rows x 32 keys (register tiles of rows x keys, operands from shared memory in
// 16-byte reads whose rows are padded by four words), a warp's softmax for each row (a lane a key), then the
// weighted sum of the values (a lane D / 32 columns of BM / 8 rows).  Tiles stream through two buffers of asynchronous
// copies.  Positions that no row may see are filled with zeros, and the scores of those that a row may not see are
// replaced, so what lies there does not matter.
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

template <int D, int BM> struct Smem {
    float q[BM][D + 4];
    float k[2][kTile][D + 4];
    float v[2][kTile][D];
    float p[BM][kTile + 4];
    float m[BM], l[BM], scale[BM];
    unsigned long long line[BM];      // a tree's nodes that a row sees
    int at[BM];                       // a row's token, -1: none
    int position[BM];                 // where a row's token is
    int parents[64], depth[64];
    int scratch[kThreads / 32 + 2];
};

template <int D, int BM>
__global__ void __launch_bounds__(kThreads) attend_kernel(const __grid_constant__ AttendArgs a) {
    extern __shared__ __align__(16) unsigned char raw[];
    Smem<D, BM> &sm = *reinterpret_cast<Smem<D, BM> *>(raw);
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, c = blockIdx.x;
    Share share;
    Place at = find_place<kTile, kThreads>(a, c, share, sm.scratch);
    if (c == 0)
        for (int s = tid; s < a.B; s += kThreads) {
            int past;
            if (live_tokens(a.kv, a.length, a.T, s, past) < 0) report(a.d_status, GDN_ERR_LENGTH);
        }
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    if (c >= share.ctas) return;
    int left = share.start(c + 1) - share.start(c);
    const int page = 1 << a.kv.page_log2;
    const float scale2 = a.scale * 1.4426950408889634f;

    constexpr int kCols = D / 32;                 // columns a lane holds of the sums
    constexpr int kRowsW = BM / 8;                // rows a warp holds
    float o[kRowsW][kCols];

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

        // ---- a tile's copies
        auto fetch = [&](int jj, int buf) {
            const int k0 = span.tile(jj) * kTile;
            constexpr int kVecs = D / 4;
            for (int i = tid; i < kTile * kVecs; i += kThreads) {
                const int r = i / kVecs, x = (i % kVecs) * 4, key = k0 + r;
                bool on = key < span.hi && (key >= span.lo || key < sink);
                const int id = on ? table[key >> a.kv.page_log2] : 0;
                if (on && (id < 0 || id >= a.kv.n_pages)) {
                    report(a.d_status, GDN_ERR_PAGE);
                    on = false;
                }
                const long long off = (long long)(on ? id : 0) * a.kv.page_stride +
                                      ((size_t)kvh * page + (key & (page - 1))) * D + x;
                const float *kp = static_cast<const float *>(a.kv.k) + off, *vp = static_cast<const float *>(a.kv.v) + off;
                float *ks = &sm.k[buf][r][x], *vs = &sm.v[buf][r][x];
                const int bytes = on ? 16 : 0;                   // of the 16 written, those that are read
                const void *kg = on ? (const void *)kp : a.kv.k, *vg = on ? (const void *)vp : a.kv.v;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(
                                 (uint32_t)__cvta_generic_to_shared(ks)), "l"(kg), "r"(bytes) : "memory");
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(
                                 (uint32_t)__cvta_generic_to_shared(vs)), "l"(vg), "r"(bytes) : "memory");
            }
            asm volatile("cp.async.commit_group;\n" ::: "memory");
        };

        __syncthreads();                          // the block before no longer reads shared memory
        fetch(j0, 0);
        // ---- the block's rows
        for (int i = tid; i < BM * (D / 4); i += kThreads) {
            const int r = i / (D / 4), x = (i % (D / 4)) * 4;
            float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows)
                f = read4(static_cast<const float *>(a.q) +
                             (((size_t)s * a.T + span.t0 + r / a.G) * a.H + (size_t)kvh * a.G + r % a.G) * D + x);
            *reinterpret_cast<float4 *>(&sm.q[r][x]) = f;
        }
        if (a.parent && tid < span.t1) {
            int p = a.parent[(size_t)s * a.T + tid];
            if (p < -1 || p >= tid) {
                report(a.d_status, GDN_ERR_TREE);
                p = -1;
            }
            sm.parents[tid] = p;
        }
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
            unsigned long long line = 0;
            if (a.parent)
                for (int p = t; p >= 0; p = sm.parents[p]) line |= 1ull << p;
            sm.line[r] = line;
            sm.position[r] = span.past + (a.parent && t >= 0 ? sm.depth[t] : t);
        }
#pragma unroll
        for (int i = 0; i < kRowsW; ++i)
#pragma unroll
            for (int e = 0; e < kCols; ++e) o[i][e] = 0.f;

        for (int jj = j0; jj < j1; ++jj) {
            const int buf = (jj - j0) & 1, k0 = span.tile(jj) * kTile;
            if (jj + 1 < j1) fetch(jj + 1, buf ^ 1);
            else asm volatile("cp.async.commit_group;\n" ::: "memory");
            asm volatile("cp.async.wait_group 1;\n" ::: "memory");
            __syncthreads();
            // ---- scores: rows rg + 16 i, keys kg + 16 n
            {
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
            // ---- softmax: a warp a row, a lane a key
            for (int r = wid; r < BM; r += 8) {
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
            __syncthreads();                      // the tile's buffer may be filled again
        }
        // ---- the block's sums: its output, or a part of it
        const bool whole = j0 == 0 && j1 == span.n;
        const size_t part = size_t(2 * c + (first_block ? 0 : 1)) * a.part_rows;
        constexpr int V = kCols < 4 ? kCols : 4;
#pragma unroll
        for (int i = 0; i < kRowsW; ++i) {
            const int r = wid + 8 * i;
            if (r >= rows) continue;
            const float l = sm.l[r];
            if (whole) {
                float *out = static_cast<float *>(a.out) +
                         (((size_t)s * a.T + span.t0 + r / a.G) * a.H + (size_t)kvh * a.G + r % a.G) * D;
                const float inv = 1.f / l;
#pragma unroll
                for (int e = 0; e < kCols; ++e) o[i][e] *= inv;
#pragma unroll
                for (int e = 0; e < kCols; e += V) store_row<V>(out + (e / V * 32 + lane) * V, &o[i][e]);
            } else {
                if (lane == 0) a.stats[part + r] = make_float2(sm.m[r], l);
                float *to = a.partial + (part + r) * D;
#pragma unroll
                for (int e = 0; e < kCols; e += V) store_row<V>(to + (e / V * 32 + lane) * V, &o[i][e]);
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

// rows of a block: 16 where a slot has no more (a wider block would spend its time on rows that are not there), else 64
static int block_rows(int T, int G) { return (long long)T * G <= 16 ? 16 : 64; }

AttendBlock attend_f32_block(int T, int G) {
    const int rows = block_rows(T, G);
    return {rows, rows / G < T ? rows / G : T, 1, 0, kAttendCtas};
}

cudaError_t launch_attend_f32(const AttendArgs &a, cudaStream_t stream) {
    return block_rows(a.T, a.G) == 16 ? launch_d<16>(a, stream) : launch_d<64>(a, stream);
}

}  // namespace gdn
