// attend_join.cu -- the blocks of rows whose keys several CTAs shared, joined from their partial sums.
//
// Part i of a row holds m_i (the maximum of its scores, in powers of two), l_i = sum 2^(x - m_i) and
// O_i = sum 2^(x - m_i) v; with m = max m_i the row is sum 2^(m_i - m) O_i / sum 2^(m_i - m) l_i, in the order of the parts.
// A part in which the row sees nothing has l_i = 0 and m_i = -inf.  The partial sums are still in L2, so round trips to
// it are what costs: a warp takes 128 columns of a row, its lanes fetch the parts' m and l at once (a part each), and several
// parts' sums are in flight together: 16 where a block may have many parts, 4 where it has a few (more warps an SM then).
#include "attn.cuh"

#include <cuda_bf16.h>

namespace gdn {
namespace {

constexpr int kJoinThreads = 128;
constexpr int kJoinWarps = kJoinThreads / 32;

template <int N> __device__ __forceinline__ void store_row(float *to, const float *x) {
#pragma unroll
    for (int i = 0; i < N; ++i) to[i] = x[i];
}
template <int N> __device__ __forceinline__ void store_row(__nv_bfloat16 *to, const float *x) {
#pragma unroll
    for (int i = 0; i < N; i += 2) *reinterpret_cast<__nv_bfloat162 *>(to + i) = __floats2bfloat162_rn(x[i], x[i + 1]);
}

// BATCH: parts in flight
template <typename E, int D, int TK, int BATCH>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ AttendArgs a, const bool by_item) {
    __shared__ int scratch[kJoinWarps + 2];
    constexpr int V = D / 32 < 4 ? D / 32 : 4;      // numbers a lane takes of a part
    constexpr int kWarpsRow = D / (32 * V);
    constexpr int kPartWords = ((sizeof(E) == 4 ? 2 : 1) * kAttendCtas + 31) / 32;      // parts a lane looks after
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    auto chk = [&](const void *p, size_t bytes, const void *base, size_t extent) { return in_bounds(p, bytes, base, extent, a.d_status); };
    // The lengths were there before the kernel whose sums are joined began, so this goes on beside its end.
    Share share;
    int c, s, kvh = 0, parts = 1;
    int begin = 0;
    Span span;
    if (by_item) {                                  // few blocks of rows: one after the other
        share.set(scan_total<TK>(a), a);
        const int pair = blockIdx.x / a.Hk;
        s = pair / a.n_tb;
        span = block_span<TK>(a, s, pair % a.n_tb);
        kvh = blockIdx.x % a.Hk;
        begin = scan_begin<TK>(a, pair) + kvh * (span.n + a.pad);
        c = span.n ? share.owner(begin + a.pad) : 0;
        if (span.n) parts = share.owner(begin + a.pad + span.n - 1) - c + 1;
    } else {                                        // the one that CTA c's share ends in
        c = blockIdx.x;
        const Place at = find_place<TK, kJoinThreads>(a, c + 1, share, scratch);
        s = at.pair / a.n_tb;
        span = block_span<TK>(a, s, at.pair % a.n_tb);
        if (c + 1 < share.ctas) {
            kvh = at.offset / (span.n + a.pad);
            begin = share.start(c + 1) - (at.offset - kvh * (span.n + a.pad));
            // else it begins there, or an earlier CTA has its beginning
            if (share.owner(begin + a.pad) == c) parts = share.owner(begin + a.pad + span.n - 1) - c + 1;
        }
    }
    // (every thread waits, so that this kernel does not end before the one whose sums are joined)
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    if (parts == 1) return;
    const int rows = (span.t1 - span.t0) * a.G, stride = a.part_rows;
    const size_t first = size_t(2 * c + (begin > share.start(c) ? 1 : 0)) * stride;
    const int column = (wid % kWarpsRow) * (32 * V) + lane * V;
    for (int r = blockIdx.y * (kJoinWarps / kWarpsRow) + wid / kWarpsRow; r < rows; r += gridDim.y * (kJoinWarps / kWarpsRow)) {
        auto part = [&](int i) { return (i == 0 ? first : size_t(2 * (c + i)) * stride) + r; };
        float w[kPartWords], m = -INFINITY, sum = 0.f;
        float2 st[kPartWords];
#pragma unroll
        for (int k = 0; k < kPartWords; ++k) {
            const int i = 32 * k + lane;
            st[k] = i < parts && chk(a.stats + part(i), 8, a.stats, a.ext_stats) ? a.stats[part(i)] : make_float2(-INFINITY, 0.f);
            m = fmaxf(m, st[k].x);
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(kWarp, m, d));
#pragma unroll
        for (int k = 0; k < kPartWords; ++k) {
            w[k] = st[k].x == -INFINITY ? 0.f : exp2f(st[k].x - m);
            sum += w[k] * st[k].y;
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(kWarp, sum, d);
        float o[V];
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = 0.f;
#pragma unroll
        for (int k = 0; k < kPartWords; ++k)
            for (int i0 = 32 * k; i0 < min(parts, 32 * k + 32); i0 += BATCH) {
                float x[BATCH][V];
#pragma unroll
                for (int q = 0; q < BATCH; ++q) {
                    const float *from = a.partial + part(i0 + q) * D + column;
                    const bool there = i0 + q < parts && chk(from, 4 * V, a.partial, a.ext_partial);
                    if constexpr (V == 4) {
                        const float4 f = there ? *reinterpret_cast<const float4 *>(from) : make_float4(0.f, 0.f, 0.f, 0.f);
                        x[q][0] = f.x; x[q][1] = f.y; x[q][2] = f.z; x[q][3] = f.w;
                    } else {
                        const float2 f = there ? *reinterpret_cast<const float2 *>(from) : make_float2(0.f, 0.f);
                        x[q][0] = f.x; x[q][1] = f.y;
                    }
                }
#pragma unroll
                for (int q = 0; q < BATCH; ++q) {      // past the last part the weight is 0
                    const float f = __shfl_sync(kWarp, w[k], (i0 + q) & 31);
#pragma unroll
                    for (int e = 0; e < V; ++e) o[e] += f == 0.f ? 0.f : f * x[q][e];
                }
            }
        const float inv = 1.f / sum;
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] *= inv;
        E *to = static_cast<E *>(a.out) + (((size_t)s * a.T + span.t0 + r / a.G) * a.H + (size_t)kvh * a.G + r % a.G) * D + column;
        if (chk(to, V * sizeof(E), a.out, a.ext_q)) store_row<V>(to, o);
    }
}

template <typename E, int D, int TK> cudaError_t launch(const AttendArgs &a, cudaStream_t stream) {
    // With no more blocks of rows than CTAs, a column of the grid for each; else one for each border between two CTAs, where
    // a block has two or three parts.  Some eight CTAs an SM: each looks for its block first.
    const long long items = (long long)a.B * a.n_tb * a.Hk;
    const bool by_item = items <= a.ctas;
    const int columns = by_item ? (int)items : a.ctas, most = 8 * kAttendCtas / columns;
    const int rows_cta = kJoinWarps / (D > 128 ? D / 128 : 1), groups = (a.TB * a.G + rows_cta - 1) / rows_cta;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(columns), unsigned(groups < most ? groups : most), 1);
    cfg.blockDim = dim3(kJoinThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // (16 tokens behind 8185 positions, 22 parts a block: 19.6 us for the whole call, 20.5 with 4 in flight; 32 slots, two or
    // three parts: 182.9 us with 4, 188.8 with 16.)
    auto kern = 8 * items <= a.ctas ? join_kernel<E, D, TK, 16> : join_kernel<E, D, TK, 4>;
    return cudaLaunchKernelEx(&cfg, kern, a, by_item);
}

}  // namespace

cudaError_t launch_attend_join(const AttendArgs &a, gdn_dtype dtype, cudaStream_t stream) {
    if (dtype == GDN_F32)
        return a.D == 64    ? launch<float, 64, kTileF32>(a, stream)
               : a.D == 128 ? launch<float, 128, kTileF32>(a, stream)
                            : launch<float, 256, kTileF32>(a, stream);
    return a.D == 64    ? launch<__nv_bfloat16, 64, kTileBf16>(a, stream)
           : a.D == 128 ? launch<__nv_bfloat16, 128, kTileBf16>(a, stream)
                        : launch<__nv_bfloat16, 256, kTileBf16>(a, stream);
}

}  // namespace gdn
