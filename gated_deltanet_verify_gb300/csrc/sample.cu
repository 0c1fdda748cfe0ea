// sample.cu -- one token per row of logits: temperature, top-k, top-p and min-p
// from given uniforms.
//
// With x_i = (l_i - max l) / T and w_i = exp(x_i), tokens ordered by (logit
// descending, index ascending), each filter keeps a prefix of that order: top-k
// the first k, top-p the shortest prefix of those whose mass reaches p of
// theirs, min-p the tokens with w_i >= min_p.  The token is the smallest i with
// sum_{j <= i, kept} w_j > u * sum_{kept} w_j, in index order.
//
// A border of that last sum decides the token, so every sum is exact: a weight
// is a 64-bit integer in units of 2^-44 of the largest weight (weight() below),
// and the integer sums do not depend on the order they are taken in -- the
// token is the same whatever the launch shape, and equals the one of 64-bit
// arithmetic unless u lies within ~1e-11 of a border.
//
// Thresholds are found on the logits themselves, as order-preserving 32-bit
// keys: bisection for the largest key whose tokens and all above it reach the
// count or the mass; ties at that key are kept by index.
#include "internal.cuh"

#include <cuda_bf16.h>

#include "weight.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kFull = 0xffffffffu;
using u64 = unsigned long long;

__device__ __forceinline__ u64 shfl_xor64(u64 v, int m) { return __shfl_xor_sync(kFull, v, m); }

template <typename L>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleArgs a) {
    __shared__ WeightTable table;
    __shared__ u64 red[kWarps];
    __shared__ u64 red_out;
    __shared__ u64 warp_mass[kWarps];
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int row = blockIdx.x, slot = row / a.T, V = a.V;
    const L *logits = static_cast<const L *>(a.logits) + size_t(row) * a.ld;
    table.fill(tid, kThreads);

    auto report = [&]() {
        if (tid == 0 && a.d_status) atomicCAS(a.d_status, int(GDN_OK), int(GDN_ERR_SAMPLE));
    };
    auto finish = [&](int token, float logprob) {
        if (tid == 0) {
            a.tokens[row] = token;
            if (a.logprob) a.logprob[row] = logprob;
        }
    };
    // block-wide sum, maximum and minimum; every thread gets the result
    auto reduce = [&](u64 v, auto op) -> u64 {
#pragma unroll
        for (int m = 16; m; m >>= 1) v = op(v, shfl_xor64(v, m));
        __syncthreads();
        if (lane == 0) red[wid] = v;
        __syncthreads();
        if (wid == 0) {
            u64 t = red[lane & (kWarps - 1)];
#pragma unroll
            for (int m = kWarps / 2; m; m >>= 1) t = op(t, shfl_xor64(t, m));
            if (lane == 0) red_out = t;
        }
        __syncthreads();
        return red_out;
    };
    auto sum = [](u64 x, u64 y) { return x + y; };
    auto most = [](u64 x, u64 y) { return x > y ? x : y; };
    auto least = [](u64 x, u64 y) { return x < y ? x : y; };

    const float temp = a.temperature ? a.temperature[slot] : 1.0f;
    const float uu = a.u[row];
    const int k = a.top_k ? a.top_k[slot] : 0;
    const float p = a.top_p ? a.top_p[slot] : 1.0f, mp = a.min_p ? a.min_p[slot] : 0.0f;
    const bool fine = sample_params_ok(temp, p, mp) && uu >= 0.0f && uu < 1.0f;

    u64 mx = 0;
    for (int i = tid; i < V; i += kThreads) mx = most(mx, u64(key_of(clean(logits[i]))));
    const uint32_t kmax = uint32_t(reduce(mx, most));
    if (!fine || kmax == kNone) {
        report();
        finish(-1, -INFINITY);
        return;
    }
    const float top = value_of(kmax);
    if (temp == 0.0f) {
        u64 at = ~0ull;
        for (int i = tid; i < V; i += kThreads)
            if (key_of(clean(logits[i])) == kmax) at = least(at, u64(i));
        at = reduce(at, least);
        finish(int(at), 0.0f);
        return;
    }
    const Scale sc = scale_of(temp);
    // kept: key > K, or key == K and index <= I
    uint32_t K = kNone + 1;
    int I = V;
    auto kept = [&](uint32_t key, int i) { return key > K || (key == K && i <= I); };
    // the index of the need-th token of key K
    auto tie = [&](u64 need) -> int {
        int lo = 0, hi = V - 1;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            u64 n = 0;
            for (int i = tid; i <= mid; i += kThreads) n += key_of(clean(logits[i])) == K;
            if (reduce(n, sum) >= need) hi = mid;
            else lo = mid + 1;
        }
        return lo;
    };
    // the largest key at which stat, summed over the kept tokens of that key and above, reaches target
    auto cross = [&](u64 target, auto stat) {
        uint32_t lo = K, hi = kmax;
        while (lo < hi) {
            const uint32_t mid = lo + (hi - lo + 1) / 2;
            u64 n = 0;
            for (int i = tid; i < V; i += kThreads) {
                const float l = clean(logits[i]);
                const uint32_t key = key_of(l);
                if (key >= mid && kept(key, i)) n += stat(l);
            }
            if (reduce(n, sum) >= target) lo = mid;
            else hi = mid - 1;
        }
        u64 above = 0;
        for (int i = tid; i < V; i += kThreads) {
            const float l = clean(logits[i]);
            const uint32_t key = key_of(l);
            if (key > lo && kept(key, i)) above += stat(l);
        }
        above = reduce(above, sum);
        const u64 each = stat(value_of(lo));
        const bool same = lo == K;               // the old limit on ties may be the tighter one
        K = lo;
        const u64 need = target > above ? (target - above + each - 1) / each : 1;
        const int at = tie(need);
        I = same ? min(I, at) : at;
    };
    auto w = [&](float l) { return weight(l, top, sc, table); };
    if (k > 0 && k < V) {
        u64 n = 0;
        for (int i = tid; i < V; i += kThreads) n += kept(key_of(clean(logits[i])), i);
        if (reduce(n, sum) > u64(k)) cross(u64(k), [](float) { return u64(1); });
    }
    if (p < 1.0f) {
        u64 n = 0;
        for (int i = tid; i < V; i += kThreads) {
            const float l = clean(logits[i]);
            if (kept(key_of(l), i)) n += w(l);
        }
        cross(mass_target(p, reduce(n, sum)), w);
    }
    if (mp > 0.0f) {
        const uint32_t key = min_p_key(mp, temp, top);
        if (key > K) {
            K = key;
            I = V;
        }
    }
    // the kept mass by warp, each over a stretch of the row of its own; then the warp and the token
    const int seg = ((V + kWarps - 1) / kWarps + 31) & ~31;
    const int beg = min(V, wid * seg), end = min(V, beg + seg);
    u64 mine = 0;
    for (int i = beg + lane; i < end; i += 32) {
        const float l = clean(logits[i]);
        if (kept(key_of(l), i)) mine += w(l);
    }
#pragma unroll
    for (int m = 16; m; m >>= 1) mine += shfl_xor64(mine, m);
    if (lane == 0) warp_mass[wid] = mine;
    __syncthreads();
    u64 total = 0, before = 0;
    for (int i = 0; i < kWarps; ++i) {
        if (i < wid) before += warp_mass[i];
        total += warp_mass[i];
    }
    const u64 target = draw_target(uu, total);
    if (before <= target && target < before + mine) {
        for (int i0 = beg; i0 < end; i0 += 32) {
            const int i = i0 + lane;
            u64 c = 0;
            if (i < end) {
                const float l = clean(logits[i]);
                if (kept(key_of(l), i)) c = w(l);
            }
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const u64 o = __shfl_up_sync(kFull, c, m);
                if (lane >= m) c += o;
            }
            const unsigned hit = __ballot_sync(kFull, before + c > target);
            if (hit) {
                if (lane == __ffs(hit) - 1) {
                    a.tokens[row] = i;
                    if (a.logprob) a.logprob[row] = log_prob(clean(logits[i]), top, temp, total);
                }
                break;
            }
            before += __shfl_sync(kFull, c, 31);
        }
    }
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a, gdn_dtype dtype, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(a.B) * unsigned(a.T), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return dtype == GDN_BF16 ? cudaLaunchKernelEx(&cfg, sample_kernel<__nv_bfloat16>, a)
                             : cudaLaunchKernelEx(&cfg, sample_kernel<float>, a);
}

}  // namespace gdn
