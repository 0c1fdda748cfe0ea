// append.cu -- a batch's queries and keys normalised and rotated by their positions, its keys and values appended to a
// paged cache, in one pass.
//
// A head's vector x (D numbers) becomes x' = R(p) (x / sqrt(mean x^2 + eps) * w): R(p) turns pair i of the first
// rope_dims numbers by the angle p * freq[i].  The new tokens' k' and v go to their slot's pages, q' to a dense matrix.
//
// Angles.  p * freq[i] in fp32 loses its turns at far positions (at p = 10^5 an error of 2^-8 radians).  Only the angle's
// part of a full turn counts, so freq / 2 pi less its whole turns is held as a 64-bit fraction of a turn, off by 2^-63 at
// most, and multiplied by p in wrapping integers; sincospif of the product's upper 32 bits follows.  The fraction comes from the
// 24 bits of freq times the 128 bits of 1 / 2 pi that its exponent asks for (Payne and Hanek, Radian reduction for
// trigonometric functions, 1983), for |freq| up to 2^40 and more.  No fp64: as one product of fp64 numbers it was off by |freq| 2^-56
// of a turn, and a few such operations in every CTA cost the trees below 1.8 us (an SM does two a cycle).  A
// token's angles are computed once and shared by its heads.
//
// Bytes bound it: every row is read once and written once.  A token is one CTA's (with few tokens several share its heads):
// its threads take 8 numbers of a head each (16-byte accesses in bf16), so D / 8 lanes hold a head, its norm is a few
// shuffles, and the other half of a rotated pair comes by a shuffle too (rope_dims / 2 is a multiple of 8).  Two or three
// heads a thread are in flight, the first while the angles are computed.  8192 tokens of 32 + 8 + 8 heads of 128: 39 us, 5.2 TB/s of the
// 6.7 that a copy has, with 70 % of the issue slots (46 us with the frequencies converted for every token and the
// sines read where their threads met in a bank); one token 2.4 us, 32 x 16 in trees 6.2 us, in a captured graph.
#include "attn.cuh"

#include <cuda_bf16.h>

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 8;               // numbers a thread holds of a head
constexpr unsigned kFull = 0xffffffffu;

template <typename E> struct Vec;
template <> struct Vec<float> {
    float4 a, b;
    __device__ __forceinline__ void get(float *x) const {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
    __device__ __forceinline__ void set(const float *x) {
        a = make_float4(x[0], x[1], x[2], x[3]);
        b = make_float4(x[4], x[5], x[6], x[7]);
    }
};
template <> struct Vec<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void get(float *x) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    __device__ __forceinline__ void set(const float *x) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        a = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// 1 / 2 pi, 64 bits a word behind the binary point, with zeros on both sides
__constant__ const unsigned long long kTurn[6] = {0, 0, 0x28be60db9391054aull, 0x7f09d5f47d4d3770ull, 0x36d8a5664f10e410ull, 0};
__device__ __forceinline__ unsigned long long turn_bits(int from) {
    const int w = from >> 6, s = from & 63;
    return s ? kTurn[w] << s | kTurn[w + 1] >> (64 - s) : kTurn[w];
}
// the part of a turn that f radians are, in 2^-64 of a turn: 24 bits of f times bits of 1 / 2 pi, of which those above the binary
// point of the product do not count
__device__ __forceinline__ unsigned long long turn_fraction(float f) {
    const uint32_t u = __float_as_uint(f), e = u >> 23 & 255;
    const unsigned long long m = (u & 0x7fffff) | (e ? 0x800000 : 0);
    const int shift = min(max((int)e, 1) - 150 + 64, 128);     // (of larger numbers, infinities and NaN the angles are no one's)
    const unsigned long long x = m * turn_bits(max(0, 64 + shift)) + __umul64hi(m, turn_bits(128 + shift));
    return u >> 31 ? 0 - x : x;
}

template <typename E, int D, bool ADJACENT>
__global__ void __launch_bounds__(kThreads, 4) append_kernel(const __grid_constant__ AppendArgs a) {
    constexpr int kLanes = D / kPer;              // threads a head
    constexpr int kHeads = kThreads / kLanes;     // heads at a time
    // Heads that a thread has in flight.  Three of 32 bytes (f32) do not stay in 64 registers; in bf16 they nearly do, and were
    // faster for heads of 128 alone (8192 tokens, us, three and two: f32 24 + 4 + 4 heads of 256 106 and 88, 40 + 8 + 8 of 64 58 and
    // 47; bf16 72 and 69, 44 and 42; bf16 32 + 8 + 8 of 128 56 and 58, with neither norms nor shuffles 40 and 44).
    constexpr int kBatch = sizeof(E) == 2 && D == 128 ? 3 : 2;
    // cos and sin of the token's angles; a thread's pairs are as far apart as there are threads, so that they do not meet in a bank
    __shared__ float2 turn[D / 2];
    constexpr int kPairs = ADJACENT ? kPer / 2 : kPer, kApart = D / 2 / kPairs;
    auto spot = [](int pair) { return pair % kPairs * kApart + pair / kPairs; };
    __shared__ int parents[64];
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const int tid = threadIdx.x, sub = tid % kLanes, group = tid / kLanes;
    const int half = a.rope_dims / 2, heads = a.H + 2 * a.Hk;
    // this CTA's heads: of every gridDim.y groups of kHeads one, kBatch of them in flight
    const int head0 = (a.q ? 0 : a.H) + blockIdx.y * kHeads + group, step = gridDim.y * kHeads;
    const int page = 1 << a.kv.page_log2;
    // where this thread's numbers are turned: pairs half apart (or beside one another), the lower ones first
    const int i0 = sub * kPer, apart = half / kPer, lane = tid & 31;
    const bool low = sub < apart, turned = i0 < a.rope_dims;
    const int other = (low ? lane + apart : lane - apart) & 31;
    const bool norms = a.q_norm || a.k_norm;
    auto chk = [&](const void *p, size_t bytes, const void *base, size_t extent) { return in_bounds(p, bytes, base, extent, a.d_status); };
    const unsigned long long part = tid < half && chk(a.freq + tid, 4, a.freq, a.ext_freq) ? turn_fraction(a.freq[tid]) : 0;  // of a turn, a position
    for (int row = blockIdx.x; row < a.B * a.T; row += gridDim.x) {
        const int s = row / a.T, t = row - s * a.T;
        int past;
        const int n = live_tokens(a.kv, a.length, a.T, s, past, a.d_status);
        if (n < 0 && t == 0 && tid == 0) report(a.d_status, GDN_ERR_LENGTH);
        if (t >= n) continue;
        int source = t, depth = t;
        if (a.path) {
            if (!chk(a.path + row, 4, a.path, a.ext_nodes)) continue;
            source = a.path[row];
            if (source == -1) continue;
            if (source < 0 || source >= a.T) {
                if (tid == 0) report(a.d_status, GDN_ERR_TREE);
                continue;
            }
        }
        const size_t from = (size_t)s * a.T + source;
        const int k_head = a.H, v_head = a.H + a.Hk;  // heads in one row: q, then k, then v
        const E *from_q = static_cast<const E *>(a.q) + from * a.ld_q + i0;
        const E *from_k = static_cast<const E *>(a.k) + from * a.ld_k - (size_t)k_head * D + i0;
        const E *from_v = static_cast<const E *>(a.v) + from * a.ld_v - (size_t)v_head * D + i0;
        auto load = [&](int h) {
            const E *from = (h < k_head ? from_q : h < v_head ? from_k : from_v) + (size_t)h * D;
            if (!(h < k_head ? chk(from, sizeof(Vec<E>), a.q, a.ext_q) : h < v_head ? chk(from, sizeof(Vec<E>), a.k, a.ext_k)
                                                                                   : chk(from, sizeof(Vec<E>), a.v, a.ext_v)))
                return Vec<E>{};
            return *reinterpret_cast<const Vec<E> *>(from);
        };
        // the first rows are on their way while the angles are computed
        Vec<E> v[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
            if (head0 + b * step < heads) v[b] = load(head0 + b * step);
        const int place = past + t;
        const int id = page_at(a.kv, a.kv.table + (size_t)s * a.kv.max_pages + (place >> a.kv.page_log2), a.d_status);
        const bool held = id >= 0 && id < a.kv.n_pages;
        if (!held && tid == 0) report(a.d_status, GDN_ERR_PAGE);
        __syncthreads();                          // the last token's angles are no longer read
        if (a.parent) {
            if (tid <= t) parents[tid] = parent_of(a.parent, a.T, s, tid, a.ext_nodes, a.d_status, tid == t);
            __syncthreads();
            depth = 0;
            for (int p = parents[t]; p >= 0; p = parents[p]) ++depth;
        }
        if (tid < half) {
            const int x = int(part * (unsigned long long)(past + depth) >> 32);
            float sn, cs;
            sincospif((float)x * 0x1p-31f, &sn, &cs);
            turn[spot(tid)] = make_float2(cs, sn);
        }
        __syncthreads();
        // the same for every head: y = x cos + (the pair's other number) sin, with the sine's sign
        float cs[kPer], sn[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const bool first = ADJACENT ? !(i & 1) : low;
            const float2 f = turned ? turn[spot(ADJACENT ? (i0 + i) / 2 : low ? i0 + i : i0 - half + i)] : make_float2(1.f, 0.f);
            cs[i] = f.x;
            sn[i] = first ? -f.y : f.y;
        }
        E *to_q = static_cast<E *>(a.q_out) + (size_t)row * a.H * D + i0;
        const long long at = (long long)id * a.kv.page_stride + (size_t)(place & (page - 1)) * D + i0;
        E *to_k = static_cast<E *>(a.kv.k) + at - (size_t)k_head * page * D, *to_v = static_cast<E *>(a.kv.v) + at - (size_t)v_head * page * D;
        for (int h0 = head0 - group; h0 < heads; h0 += kBatch * step) {        // (the same in all lanes: they shuffle)
            if (h0 != head0 - group)
#pragma unroll
                for (int b = 0; b < kBatch; ++b)
                    if (h0 + group + b * step < heads) v[b] = load(h0 + group + b * step);
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                if (h0 + b * step >= heads) break;
                const int h = h0 + group + b * step;
                if (h0 + b * step < v_head) {     // not all are v, which goes as it came
                    float x[kPer], y[kPer];
                    v[b].get(x);
                    if (norms) {
                        const float *w = h < k_head ? a.q_norm : a.k_norm;
                        float sum = 0.f;
#pragma unroll
                        for (int i = 0; i < kPer; ++i) sum += x[i] * x[i];
#pragma unroll
                        for (int d = kLanes / 2; d; d >>= 1) sum += __shfl_xor_sync(kFull, sum, d);
                        if (w && chk(w + i0, 4 * kPer, w, a.ext_norm)) {
                            const float r = rsqrtf(sum / D + a.eps);
                            const float4 w0 = *reinterpret_cast<const float4 *>(w + i0), w1 = *reinterpret_cast<const float4 *>(w + i0 + 4);
                            const float ww[kPer] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                            for (int i = 0; i < kPer; ++i) x[i] = x[i] * r * ww[i];
                        }
                    }
#pragma unroll
                    for (int i = 0; i < kPer; ++i) {
                        const float o = ADJACENT ? x[i ^ 1] : __shfl_sync(kFull, x[i], other);
                        y[i] = turned ? fmaf(o, sn[i], x[i] * cs[i]) : x[i];
                    }
                    if (h < v_head) v[b].set(y);
                }
                E *to = h < k_head ? to_q + (size_t)h * D : (h < v_head ? to_k : to_v) + (size_t)h * page * D;
                if (h < heads && (h < k_head || held) &&
                    (h < k_head ? chk(to, sizeof(Vec<E>), a.q_out, a.ext_out) : chk(to, sizeof(Vec<E>), h < v_head ? a.kv.k : a.kv.v, a.kv.ext_pool)))
                    *reinterpret_cast<Vec<E> *>(to) = v[b];
            }
        }
    }
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
}

template <typename E>
cudaError_t launch(const AppendArgs &a, int sms, cudaStream_t stream) {
    auto kern = a.D == 64    ? (a.adjacent ? append_kernel<E, 64, true> : append_kernel<E, 64, false>)
                : a.D == 128 ? (a.adjacent ? append_kernel<E, 128, true> : append_kernel<E, 128, false>)
                             : (a.adjacent ? append_kernel<E, 256, true> : append_kernel<E, 256, false>);
    cudaLaunchConfig_t cfg = {};
    // As many CTAs as the SMs hold at once, which share out the tokens; with few tokens their heads too, twice as many then
    // (32 x 16 tokens: in trees 6.2 us, with one CTA a token 6.5, in f32 6.8 and 8.4; in chains 7.2 and 6.5).
    const long long rows = (long long)a.B * a.T, most = 4LL * sms, spare = 2 * most / rows;
    const int groups = ((a.q ? a.H : 0) + 2 * a.Hk + kThreads * kPer / a.D - 1) / (kThreads * kPer / a.D);
    cfg.gridDim = dim3(unsigned(rows < most ? rows : most), unsigned(spare < 1 ? 1 : spare < groups ? spare : groups), 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace

cudaError_t launch_append(const AppendArgs &a, gdn_dtype dtype, int sm_count, cudaStream_t stream) {
    return dtype == GDN_F32 ? launch<float>(a, sm_count, stream) : launch<__nv_bfloat16>(a, sm_count, stream);
}

}  // namespace gdn
