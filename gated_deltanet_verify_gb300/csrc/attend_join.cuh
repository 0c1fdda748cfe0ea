// attend_join.cuh -- the blocks of rows whose keys several CTAs shared, joined from their partial sums.
//
// Part i of a row holds m_i (the maximum of its scores, in powers of two), l_i = sum 2^(x - m_i) and
// O_i = sum 2^(x - m_i) v; with m = max m_i the row is sum 2^(m_i - m) O_i / sum 2^(m_i - m) l_i, in the order of the parts.
// A part in which the row sees nothing has l_i = 0 and m_i = -inf.  A warp takes a row; the partial sums are still in L2.
#pragma once

#include "attn.cuh"

#include <cuda_bf16.h>

namespace gdn {
namespace {

constexpr int kJoinThreads = 256;
constexpr int kJoinRows = kJoinThreads / 32;

template <int N> __device__ __forceinline__ void store_row(float *to, const float *x) {
#pragma unroll
    for (int i = 0; i < N; ++i) to[i] = x[i];
}
template <int N> __device__ __forceinline__ void store_row(__nv_bfloat16 *to, const float *x) {
#pragma unroll
    for (int i = 0; i < N; i += 2) *reinterpret_cast<__nv_bfloat162 *>(to + i) = __floats2bfloat162_rn(x[i], x[i + 1]);
}

template <typename E, int D, int TK>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ AttendArgs a) {
    __shared__ long long scratch[kJoinThreads / 32 + 4];
    constexpr int V = D / 32 < 4 ? D / 32 : 4;      // numbers a load; a lane holds D / 32
    constexpr int C = D / 32 / V;
    const int c = blockIdx.x, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    Share share;
    const Place at = find_place<TK, kJoinThreads>(a, c + 1, share, scratch);
    if (c + 1 >= share.ctas) return;
    const int s = at.pair / a.n_tb;
    const Span span = block_span<TK>(a, s, at.pair % a.n_tb);
    const int kvh = int(at.offset / span.n), j = int(at.offset % span.n);
    const long long next = share.start(c + 1), begin = next - j;
    if (j == 0 || begin < share.start(c)) return;   // nothing is split here, or an earlier CTA has its beginning
    const int last = share.owner(begin + span.n - 1), parts = last - c + 1;
    const int r = blockIdx.y * kJoinRows + (threadIdx.x >> 5), rows = a.TB * a.G;
    if (r >= (span.t1 - span.t0) * a.G) return;
    auto part = [&](int i) { return size_t(i == 0 ? 2 * c + (begin > share.start(c) ? 1 : 0) : 2 * (c + i)) * rows + r; };
    float m = -INFINITY;
    for (int i = lane; i < parts; i += 32) m = fmaxf(m, a.stats[part(i)].x);
#pragma unroll
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    float sum = 0.f, o[C][V];
#pragma unroll
    for (int q = 0; q < C; ++q)
#pragma unroll
        for (int e = 0; e < V; ++e) o[q][e] = 0.f;
#pragma unroll 4
    for (int i = 0; i < parts; ++i) {
        const size_t p = part(i);
        const float2 st = a.stats[p];
        const float w = st.x == -INFINITY ? 0.f : exp2f(st.x - m);
        sum += w * st.y;
        const float *from = a.partial + p * D;
#pragma unroll
        for (int q = 0; q < C; ++q) {
            float x[V];
            if constexpr (V == 4) {
                const float4 f = *reinterpret_cast<const float4 *>(from + (q * 32 + lane) * 4);
                x[0] = f.x; x[1] = f.y; x[2] = f.z; x[3] = f.w;
            } else {
                const float2 f = *reinterpret_cast<const float2 *>(from + lane * 2);
                x[0] = f.x; x[1] = f.y;
            }
#pragma unroll
            for (int e = 0; e < V; ++e) o[q][e] += w == 0.f ? 0.f : w * x[e];
        }
    }
    const float inv = 1.f / sum;
    E *out = static_cast<E *>(a.out) + (((size_t)s * a.T + span.t0 + r / a.G) * a.H + (size_t)kvh * a.G + r % a.G) * D;
#pragma unroll
    for (int q = 0; q < C; ++q) {
#pragma unroll
        for (int e = 0; e < V; ++e) o[q][e] *= inv;
        store_row<V>(out + (q * 32 + lane) * V, o[q]);
    }
}

template <typename E, int D, int TK> cudaError_t launch_join(const AttendArgs &a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(a.ctas), unsigned((a.TB * a.G + kJoinRows - 1) / kJoinRows), 1);
    cfg.blockDim = dim3(kJoinThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, join_kernel<E, D, TK>, a);
}

}  // namespace
}  // namespace gdn
