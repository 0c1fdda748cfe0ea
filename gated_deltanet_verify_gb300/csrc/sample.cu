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
// is a 64-bit integer in units of 2^-44 of the largest weight (weight.cuh), and
// the integer sums do not depend on the order they are taken in -- the token is
// the same whatever the launch shape, and equals the one of 64-bit arithmetic
// unless u lies within ~1e-11 of a border.  For the same reason the atomics
// below (integer counts and masses) leave no trace of their order.
//
// A thread-block cluster holds a row in its CTAs' shared memory, so the logits
// are read from HBM once; what follows are passes over shared memory, joined by
// exchanges of a few words between the CTAs:
//   1. the top logit (and its lowest index: all that temperature 0 needs);
//   2. with top-k or top-p, a histogram of the tokens over bins of 1/16 octave
//      of weight (monotone in the logit), merged over the cluster: it gives the
//      bin in which top-k ends, and an estimate of the one in which top-p ends;
//   3. with top-p, the exact masses: of all, of the bins before a window of 32
//      around the estimate, and of each bin in it;
//   4. the border inside its bin: a finer histogram over the keys there, then the
//      few tokens of one of its cells by counting in the first CTA.  Where the
//      kept tokens are few from the start (up to kList), the first CTA takes them
//      all and ends the row alone;
//   5. the kept mass of every CTA, the CTA that holds the drawn place, the token.
#include "internal.cuh"

#include <cuda_bf16.h>

#include "weight.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kFull = 0xffffffffu;
constexpr int kBins = 768;               // 1/16 octave each: 45.5 octaves, where weights end, lie in bin 728
constexpr int kWindow = 32;
constexpr int kCells = 256;
constexpr int kList = 512;
constexpr int kMaxCluster = 16;
constexpr int kExchange = 2 + kWindow;
using u64 = unsigned long long;

struct Item {
    u64 order;                           // key, then the index counted down: larger comes first
    u64 stat;
};

struct Shared {
    WeightTable table;
    Item list[kList];
    u64 xch[2][kMaxCluster][kExchange];  // what each CTA of the cluster sent, two rounds
    u64 out[kExchange];                  // what this CTA sends
    u64 sum[kExchange];                  // summed over the cluster
    u64 cell_stat[kCells];
    u64 win[kWindow];
    u64 red[kWarps];
    u64 warp_sum[kWarps];
    u64 word[4];                         // broadcast within the cluster (bc) or the CTA
    double t_log_min_p;
    uint32_t cell_count[kCells];
    uint32_t hist[kBins];                // this CTA's counts
    uint32_t count[kBins];               // the cluster's, then summed up to and with each bin
    float fred[kWarps];
    uint32_t ured[kWarps];
    int n_list;
    int found;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint32_t smem_u32(const void *p) { return uint32_t(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ uint32_t map_cluster(const void *p, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ void st_cluster64(uint32_t addr, u64 v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;\n" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ void st_cluster32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;\n" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_cluster32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];\n" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void add_cluster64(uint32_t addr, u64 v) {
    asm volatile("red.relaxed.cluster.shared::cluster.add.u64 [%0], %1;\n" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t add_cluster32(uint32_t addr, uint32_t v) {
    uint32_t r;
    asm volatile("atom.relaxed.cluster.shared::cluster.add.u32 %0, [%1], %2;\n" : "=r"(r) : "r"(addr), "r"(v) : "memory");
    return r;
}

// the logits of one 16-byte vector
template <typename L> struct Vec;
template <> struct Vec<float> {
    static constexpr int N = 4;
    __device__ __forceinline__ static void get(const uint4 &v, float *f) {
        f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y); f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
    }
    __device__ __forceinline__ static uint4 put(const float *f) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    __device__ __forceinline__ static void get(const uint4 &v, float *f) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    // the values came from bf16: their upper halves hold all of them
    __device__ __forceinline__ static uint4 put(const float *f) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = (__float_as_uint(f[2 * i]) >> 16) | (__float_as_uint(f[2 * i + 1]) & 0xffff0000u);
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

template <typename L>
struct Sampler {
    static constexpr int E = Vec<L>::N;
    Shared &s;
    uint4 *data;                         // this CTA's vectors
    int nv, seg;                         // vectors of this CTA; of a warp
    int base;                            // index of element 0 of vector 0 (negative before a row's first token)
    int n_cta, rank, round;
    int tid, lane, wid;
    float top;
    Scale sc;
    float bin_scale;                     // bins per unit of logit
    uint32_t K;                          // kept: key > K, or key == K and index <= I
    int I;

    __device__ __forceinline__ bool kept(uint32_t key, int i) const { return key > K || (key == K && i <= I); }
    __device__ __forceinline__ Weight weigh(float l) const { return weight(l, top, sc, s.table); }
    __device__ __forceinline__ u64 units(float l) const { return weigh(l).units(); }
    // monotone in l; 0 for the top logit (inf - inf gives NaN, which converts to 0)
    __device__ __forceinline__ int bin(float l) const {
        const int b = __float2int_rz((top - l) * bin_scale);
        return b < kBins - 1 ? b : kBins - 1;
    }

    __device__ __forceinline__ void sync_cluster() const {
        __syncwarp();
        if (n_cta == 1) __syncthreads();
        else asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
    }

    // f(logit, index) for every element of this CTA, warps over stretches of their own, in index order within a lane
    // and between the lanes of one step; masked elements (and those beside the row) come as -inf
    template <typename F> __device__ __forceinline__ void each(F f) const {
        const int end = min(nv, (wid + 1) * seg);
        for (int v = wid * seg + lane; v < end; v += 32) {
            float l[E];
            Vec<L>::get(data[v], l);
#pragma unroll
            for (int e = 0; e < E; ++e) f(l[e], base + v * E + e);
        }
    }

    template <typename Op> __device__ __forceinline__ u64 warp_all(u64 v, Op op) const {
#pragma unroll
        for (int m = 16; m; m >>= 1) v = op(v, u64(__shfl_xor_sync(kFull, v, m)));
        return v;
    }
    // a sum or maximum (0 is neutral to op) over the block; threads 0 .. 31 hold the result
    template <typename Op> __device__ __forceinline__ u64 block_first(u64 v, Op op) const {
        v = warp_all(v, op);
        __syncthreads();
        if (lane == 0) s.red[wid] = v;
        __syncthreads();
        return wid == 0 ? warp_all(lane < kWarps ? s.red[lane] : 0ull, op) : 0;
    }
    // s.out[0 .. n) of every CTA to all: afterwards s.xch[round] holds them by rank
    __device__ __forceinline__ const u64 (*exchange(int n))[kExchange] {
        __syncthreads();
        round ^= 1;
        for (int t = tid; t < n * n_cta; t += kThreads) {
            const int to = t / n, j = t - to * n;
            st_cluster64(map_cluster(&s.xch[round][rank][j], to), s.out[j]);
        }
        sync_cluster();
        return s.xch[round];
    }
    // the same of one sum or maximum (0 is neutral to op) over each CTA: by rank in s.xch[round][rank][0]
    template <typename Op> __device__ __forceinline__ const u64 (*exchange_of(u64 v, Op op))[kExchange] {
        v = warp_all(v, op);
        __syncthreads();
        if (lane == 0) s.red[wid] = v;
        __syncthreads();
        round ^= 1;
        if (tid < n_cta) {
            v = s.red[0];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) v = op(v, s.red[w]);
            st_cluster64(map_cluster(&s.xch[round][rank][0], tid), v);
        }
        sync_cluster();
        return s.xch[round];
    }
    // one value of every thread, summed over the cluster: the same in all its threads
    __device__ __forceinline__ u64 cluster_sum(u64 v) {
        const auto x = exchange_of(v, [](u64 a, u64 b) { return a + b; });
        u64 t = 0;
        for (int r = 0; r < n_cta; ++r) t += x[r][0];
        return t;
    }

    // the merged histogram of the tokens' bins, summed up to and with each bin, in s.count
    __device__ __forceinline__ void histogram() {
        for (int i = tid; i < kBins; i += kThreads) s.hist[i] = 0;
        __syncthreads();
        each([&](float l, int) {
            if (l > -INFINITY) atomicAdd(&s.hist[bin(l)], 1u);
        });
        sync_cluster();
        if (n_cta == 1) {
            for (int i = tid; i < kBins; i += kThreads) s.count[i] = s.hist[i];
        } else {
            // lane r of a group of n_cta reads CTA r's count of a bin and, with their sum, writes CTA r's copy
            const int slice = kBins / n_cta;
            for (int t = tid; t < kBins; t += kThreads) {
                const int r = t & (n_cta - 1), b = rank * slice + t / n_cta;
                uint32_t c = ld_cluster32(map_cluster(&s.hist[b], r));
                for (int m = n_cta >> 1; m; m >>= 1) c += __shfl_xor_sync(kFull, c, m);     // whole warps: 768 bins
                st_cluster32(map_cluster(&s.count[b], r), c);
            }
        }
        sync_cluster();
        // 256 threads take three bins each
        uint32_t c[3] = {0, 0, 0};
        if (tid < 256) {
#pragma unroll
            for (int j = 0; j < 3; ++j) c[j] = s.count[3 * tid + j];
        }
        uint32_t t = c[0] + c[1] + c[2], run = t;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const uint32_t o = __shfl_up_sync(kFull, run, m);
            if (lane >= m) run += o;
        }
        if (lane == 31) s.ured[wid] = run;
        __syncthreads();
        for (int w = 0; w < wid; ++w) run += s.ured[w];
        run -= t;
        if (tid < 256) {
#pragma unroll
            for (int j = 0; j < 3; ++j) s.count[3 * tid + j] = run += c[j];
        }
        __syncthreads();
    }
    // the first bin up to which at least n tokens lie (n of them at least)
    __device__ __forceinline__ int bin_of_count(uint32_t n) {
        for (int b = tid; b < kBins; b += kThreads)
            if (s.count[b] >= n && (b == 0 || s.count[b - 1] < n)) s.found = b;
        __syncthreads();
        const int b = s.found;
        __syncthreads();
        return b;
    }
    // about where the mass reaches p of that of the bins up to `last`, each bin's tokens taken at its middle
    __device__ __forceinline__ int bin_of_mass(float p, int last) {
        float c[3] = {0.f, 0.f, 0.f};
        if (tid < 256) {
#pragma unroll
            for (int j = 0; j < 3; ++j) {
                const int b = 3 * tid + j;
                const uint32_t n = s.count[b] - (b ? s.count[b - 1] : 0);
                c[j] = b > last ? 0.f : float(n) * exp2f(-(b + 0.5f) * 0.0625f);
            }
        }
        const float t = c[0] + c[1] + c[2];
        float run = t;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const float o = __shfl_up_sync(kFull, run, m);
            if (lane >= m) run += o;
        }
        if (lane == 31) s.fred[wid] = run;
        if (tid == 0) s.found = last;
        __syncthreads();
        float all = 0.f;
        for (int w = 0; w < kWarps; ++w) {
            if (w < wid) run += s.fred[w];
            all += s.fred[w];
        }
        run -= t;
        const float need = p * all;
        if (tid < 256) {
#pragma unroll
            for (int j = 0; j < 3; ++j) {
                const float to = run + c[j];
                if (to >= need && (run < need || (tid == 0 && j == 0)) && 3 * tid + j < last) atomicMin(&s.found, 3 * tid + j);
                run = to;
            }
        }
        __syncthreads();
        const int b = s.found;
        __syncthreads();
        return b;
    }

    // tokens of the CTAs for which take(logit, key, index) holds, into the first CTA's list with their stat
    template <typename T, typename S> __device__ __forceinline__ void gather(T take, S stat) {
        const uint32_t n_at = map_cluster(&s.n_list, 0), list_at = map_cluster(s.list, 0);
        each([&](float l, int i) {
            const uint32_t key = key_of(l);
            if (!take(l, key, i)) return;
            const uint32_t at = add_cluster32(n_at, 1);
            if (at < kList) {
                st_cluster64(list_at + at * 16, (u64(key) << 32) | uint32_t(~i));
                st_cluster64(list_at + at * 16 + 8, stat(l));
            }
        });
    }

    // K and I where the stat of the kept tokens, of bin b from `before` on, reaches target
    template <typename S> __device__ __forceinline__ void resolve(int b, u64 before, u64 target, S stat) {
        // a bin of few tokens goes to the list whole; else cells over its keys, its edges widened by their own rounding,
        // keys beyond in the end cells
        uint32_t n = s.count[b] - (b ? s.count[b - 1] : 0), lo = 0;
        int shift = 32, at = kCells - 1;              // one cell
        auto cell = [&](uint32_t key) {
            const uint32_t c = key < lo || shift > 31 ? 0u : min((key - lo) >> shift, uint32_t(kCells - 1));
            return kCells - 1 - int(c);
        };
        if (tid == 0) s.n_list = 0;
        if (n > kList) {
            const float hi_l = fminf(top - b / bin_scale, 3.4028234e38f), lo_l = fmaxf(top - (b + 1) / bin_scale, -3.4028234e38f);
            const uint32_t hi = key_of(hi_l + 0.0f) + 512;
            lo = b == kBins - 1 ? kNone : key_of(lo_l + 0.0f) - 512;
            shift = max(0, 24 - __clz(max(1u, hi - lo)));
            for (int i = tid; i < kCells; i += kThreads) s.cell_stat[i] = s.cell_count[i] = 0;
            sync_cluster();
            const uint32_t stat_at = map_cluster(s.cell_stat, 0), count_at = map_cluster(s.cell_count, 0);
            each([&](float l, int i) {
                if (!(l > -INFINITY) || bin(l) != b) return;
                const uint32_t key = key_of(l);
                if (!kept(key, i)) return;
                const int c = cell(key);
                add_cluster64(stat_at + c * 8, stat(l));
                add_cluster32(count_at + c * 4, 1);
            });
            sync_cluster();
            if (rank == 0 && wid == 0) {
                u64 c[kCells / 32], t = 0;
#pragma unroll
                for (int j = 0; j < kCells / 32; ++j) t += c[j] = s.cell_stat[lane * (kCells / 32) + j];
                u64 run = t;
#pragma unroll
                for (int m = 1; m < 32; m <<= 1) {
                    const u64 o = __shfl_up_sync(kFull, run, m);
                    if (lane >= m) run += o;
                }
                run += before - t;
#pragma unroll
                for (int j = 0; j < kCells / 32; ++j) {
                    if (run < target && target <= run + c[j]) {
                        const int to = lane * (kCells / 32) + j;
                        const u64 head = (u64(to) << 32) | s.cell_count[to];
                        for (int r = 0; r < n_cta; ++r) {
                            st_cluster64(map_cluster(&s.word[0], r), head);
                            st_cluster64(map_cluster(&s.word[1], r), run);
                        }
                    }
                    run += c[j];
                }
            }
            sync_cluster();
            at = int(s.word[0] >> 32);
            n = uint32_t(s.word[0]);
            before = s.word[1];
        } else {
            sync_cluster();
        }
        auto here = [&](float l, uint32_t key, int i) {
            return l > -INFINITY && bin(l) == b && cell(key) == at && kept(key, i);
        };
        if (n <= kList) {
            gather(here, stat);
            sync_cluster();
            n = s.n_list;                             // without the tokens of the bin that top-k left out
            if (rank == 0 && tid < int(n)) {
                const Item me = s.list[tid];
                u64 run = before;
                for (int j = 0; j < int(n); ++j) {
                    const Item o = s.list[j];
                    if (o.order > me.order) run += o.stat;
                }
                if (run < target && target <= run + me.stat)
                    for (int r = 0; r < n_cta; ++r) st_cluster64(map_cluster(&s.word[2], r), me.order);
            }
            sync_cluster();
            K = uint32_t(s.word[2] >> 32);
            I = int(~uint32_t(s.word[2]));
            return;
        }
        // many tokens in one cell, most often equal ones: bisection over its keys, then the ties by index
        uint32_t k_lo = 0xffffffffu, k_hi = 0;
        each([&](float l, int i) {
            const uint32_t key = key_of(l);
            if (here(l, key, i)) {
                k_lo = min(k_lo, key);
                k_hi = max(k_hi, key);
            }
        });
        auto most = [](u64 x, u64 y) { return x > y ? x : y; };
        const u64 a = block_first(u64(~k_lo), most), z = block_first(u64(k_hi), most);
        if (tid == 0) {
            s.out[0] = a;
            s.out[1] = z;
        }
        const auto x = exchange(2);
        uint32_t lo_key = 0, hi_key = 0;
        for (int r = 0; r < n_cta; ++r) {
            lo_key = max(lo_key, uint32_t(x[r][0]));
            hi_key = max(hi_key, uint32_t(x[r][1]));
        }
        lo_key = ~lo_key;
        auto above = [&](uint32_t from) {           // the stat of the cell's tokens of that key and above, and `before`
            u64 m = 0;
            each([&](float l, int i) {
                const uint32_t key = key_of(l);
                if (key >= from && here(l, key, i)) m += stat(l);
            });
            return before + cluster_sum(m);
        };
        while (lo_key < hi_key) {
            const uint32_t mid = lo_key + (hi_key - lo_key + 1) / 2;
            if (above(mid) >= target) lo_key = mid;
            else hi_key = mid - 1;
        }
        const u64 run = above(lo_key + 1), one = stat(value_of(lo_key)), need = (target - run + one - 1) / one;
        // the need-th token of that key in index order
        u64 m = 0;
        each([&](float l, int i) {
            const uint32_t key = key_of(l);
            m += key == lo_key && kept(key, i);
        });
        auto tie = [&](float l, int i) -> u64 {
            const uint32_t key = key_of(l);
            return key == lo_key && kept(key, i);
        };
        warp_sums(m);
        pick(need - 1, tie, [&](float, int i) {
            for (int r = 0; r < n_cta; ++r) st_cluster64(map_cluster(&s.word[3], r), u64(uint32_t(i)));
        });
        sync_cluster();
        K = lo_key;
        I = int(uint32_t(s.word[3]));
    }

    // each warp's sum of `mine` in s.warp_sum
    __device__ __forceinline__ void warp_sums(u64 mine) {
        mine = warp_all(mine, [](u64 a, u64 b) { return a + b; });
        __syncthreads();
        if (lane == 0) s.warp_sum[wid] = mine;
        __syncthreads();
    }
    // with the warps' sums of stat in s.warp_sum: at(logit, index), by one thread of the cluster, of the first token in
    // index order up to which the stats sum to more than `place`
    template <typename S, typename A> __device__ __forceinline__ void pick(u64 place, S stat, A at) {
        u64 all = 0;
        for (int w = 0; w < kWarps; ++w) all += s.warp_sum[w];
        if (tid == 0) s.out[0] = all;
        const auto x = exchange(1);
        u64 run = 0;
        for (int r = 0; r < rank; ++r) run += x[r][0];
        find(place, run, stat, at);
    }
    // the same within this CTA, the sum before it being `run`
    template <typename S, typename A> __device__ __forceinline__ void find(u64 place, u64 run, S stat, A at) {
        for (int w = 0; w < wid; ++w) run += s.warp_sum[w];
        if (!(run <= place && place < run + s.warp_sum[wid])) return;
        const int end = min(nv, (wid + 1) * seg);
        for (int v0 = wid * seg; v0 < end; v0 += 32) {
            const int v = v0 + lane;
            float l[E];
            u64 c[E], t = 0;
            if (v < end) Vec<L>::get(data[v], l);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                c[e] = v < end ? stat(l[e], base + v * E + e) : 0;
                t += c[e];
            }
            u64 to = t;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const u64 o = __shfl_up_sync(kFull, to, m);
                if (lane >= m) to += o;
            }
            const unsigned hit = __ballot_sync(kFull, run + to > place);
            if (hit) {
                if (lane == __ffs(hit) - 1) {
                    u64 r = run + to - t;
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        if (r <= place && place < r + c[e]) at(l[e], base + v * E + e);
                        r += c[e];
                    }
                }
                return;
            }
            run += __shfl_sync(kFull, to, 31);
        }
    }
};

template <typename L>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs a, int n_cta, int cta_vecs) {
    extern __shared__ __align__(16) unsigned char smem[];
    Shared &s = *reinterpret_cast<Shared *>(smem);
    constexpr int E = Vec<L>::N;
    Sampler<L> x{s};
    x.data = reinterpret_cast<uint4 *>(smem + (sizeof(Shared) + 15) / 16 * 16);
    x.tid = threadIdx.x; x.lane = x.tid & 31; x.wid = x.tid >> 5;
    x.n_cta = n_cta; x.rank = int(blockIdx.x) & (n_cta - 1); x.round = 0;
    const int row = int(blockIdx.x) / n_cta, slot = row / a.T, V = a.V, tid = x.tid;

    // a CTA's shared memory may be written by its peers once it has started: the wait for all to have done so comes
    // before the first exchange
    if (n_cta > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;\n" ::: "memory");
    s.table.fill(tid, kThreads);
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    // the row as 16-byte vectors from the last 16-byte boundary before it
    const L *logits = static_cast<const L *>(a.logits) + size_t(row) * size_t(a.ld);
    const int head = int((reinterpret_cast<uintptr_t>(logits) & 15) / sizeof(L));
    const int row_vecs = (head + V + E - 1) / E;
    const int v0 = min(row_vecs, x.rank * cta_vecs);
    x.nv = min(row_vecs, v0 + cta_vecs) - v0;
    x.seg = (x.nv + kWarps - 1) / kWarps;
    x.base = v0 * E - head;
    const uint4 *src = reinterpret_cast<const uint4 *>(logits - head) + v0;
    const int seg_end = min(x.nv, (x.wid + 1) * x.seg);
    auto whole = [&](int v) { return x.base + v * E + E <= V; };      // ends inside the row
    for (int v = x.wid * x.seg + x.lane; v < seg_end; v += 32)
        if (whole(v)) cp_async16(smem_u32(x.data + v), src + v);
    const float temp = a.temperature ? a.temperature[slot] : 1.0f;
    const float u = a.u[row];
    const int k = a.top_k ? a.top_k[slot] : 0;
    const float p = a.top_p ? a.top_p[slot] : 1.0f, mp = a.min_p ? a.min_p[slot] : 0.0f;
    const bool fine = sample_params_ok(temp, p, mp) && u >= 0.0f && u < 1.0f;
    if (tid == 0 && mp > 0.0f) s.t_log_min_p = double(temp) * log(double(mp));       // while the copies are in flight
    asm volatile("cp.async.commit_group;\ncp.async.wait_group 0;\n" ::: "memory");

    // 1. the top logit; each thread cleans the vectors that it copied itself
    float best = -INFINITY;
    int best_i = 0;
    for (int v = x.wid * x.seg + x.lane; v < seg_end; v += 32) {
        float l[E];
        const int i0 = x.base + v * E;
        if (whole(v)) {
            Vec<L>::get(x.data[v], l);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) l[e] = i0 + e >= 0 && i0 + e < V ? to_float(logits[i0 + e]) : -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            l[e] = i0 + e < 0 ? -INFINITY : clean(l[e]);
            if (l[e] > best) {
                best = l[e];
                best_i = i0 + e;
            }
        }
        x.data[v] = Vec<L>::put(l);
    }
    auto most = [](u64 p, u64 q) { return p > q ? p : q; };
    u64 first = (u64(key_of(best)) << 32) | uint32_t(~best_i);
    __syncwarp();
    if (n_cta > 1) asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory");
    {
        const auto got = x.exchange_of(first, most);
        first = 0;
        for (int r = 0; r < n_cta; ++r) first = most(first, got[r][0]);
    }
    const uint32_t k_top = uint32_t(first >> 32);
    auto finish = [&](int token, float logprob) {
        a.tokens[row] = token;
        if (a.logprob) a.logprob[row] = logprob;
    };
    if (!fine || k_top == kNone || temp == 0.0f) {
        if (x.rank == 0 && tid == 0) {
            const bool greedy = fine && k_top != kNone;
            if (!greedy && a.d_status) atomicCAS(a.d_status, int(GDN_OK), int(GDN_ERR_SAMPLE));
            finish(greedy ? int(~uint32_t(first)) : -1, greedy ? 0.0f : -INFINITY);
        }
        return;
    }
    x.top = value_of(k_top);
    x.sc = scale_of(temp);
    x.bin_scale = 16.0f * x.sc.hi;
    x.K = kNone + 1;
    x.I = V;
    const uint32_t k_min_p = mp > 0.0f ? min_p_key(s.t_log_min_p, x.top) : 0u;
    bool by_k = k > 0 && k < V;
    const bool by_p = p < 1.0f;
    u64 all_mass = 0;                      // of what top-k left, where top-p needs it
    u64 my_mass = 0;                       // this CTA's kept mass, where it is known before the last pass
    bool know_mass = false;
    int list_to = -1;                      // >= 0: the kept tokens lie in the bins up to this one and fit the list
    if (by_k || by_p) {
        x.histogram();
        int last = kBins - 1;
        if (by_k && s.count[kBins - 1] <= uint32_t(k)) by_k = false;
        if (by_k) {
            last = x.bin_of_count(k);
            if (s.count[last] <= kList) list_to = last;
            else x.resolve(last, last ? s.count[last - 1] : 0, u64(k), [](float) { return u64(1); });
        }
        if (by_p && list_to < 0) {
            int b0 = max(0, min(x.bin_of_mass(p, last) - kWindow / 2, kBins - kWindow));
            for (;;) {
                for (int i = tid; i < kWindow; i += kThreads) s.win[i] = 0;
                __syncthreads();
                Weight m_all{0, 0}, m_before{0, 0};
                x.each([&](float l, int i) {
                    if (!x.kept(key_of(l), i)) return;
                    const Weight w = x.weigh(l);
                    const int b = x.bin(l) - b0;
                    m_all += w;
                    if (b < 0) m_before += w;
                    else if (b < kWindow) atomicAdd(&s.win[b], w.units());
                });
                auto add = [](u64 p, u64 q) { return p + q; };
                const u64 b_all = x.block_first(m_all.units(), add), b_before = x.block_first(m_before.units(), add);
                if (tid == 0) {
                    s.out[0] = b_all;
                    s.out[1] = b_before;
                }
                for (int i = tid; i < kWindow; i += kThreads) s.out[2 + i] = s.win[i];
                const auto got = x.exchange(kExchange);
                if (tid < kExchange) {
                    u64 t = 0;
                    for (int r = 0; r < n_cta; ++r) t += got[r][tid];
                    s.sum[tid] = t;
                }
                __syncthreads();
                all_mass = s.sum[0];
                const u64 target = mass_target(p, all_mass);
                u64 run = s.sum[1];
                int b = -1;
                u64 before = 0;
                my_mass = s.out[1];
                if (run < target)
                    for (int i = 0; i < kWindow; ++i) {
                        if (run < target && target <= run + s.sum[2 + i]) {
                            b = i;
                            before = run;
                        }
                        if (b < 0) my_mass += s.out[2 + i];
                        run += s.sum[2 + i];
                    }
                if (b >= 0) {
                    b += b0;
                    if (!by_k && s.count[b] <= kList) {
                        list_to = b;
                    } else {
                        x.resolve(b, before, target, [&](float l) { return x.units(l); });
                        know_mass = true;
                        // the kept tokens of this CTA in the bin itself
                        Weight in_bin{0, 0};
                        x.each([&](float l, int i) {
                            if (l > -INFINITY && x.bin(l) == b && x.kept(key_of(l), i)) in_bin += x.weigh(l);
                        });
                        const u64 m = x.block_first(in_bin.units(), add);
                        if (tid == 0) s.word[3] = my_mass + m;
                    }
                    break;
                }
                // the estimate was off: the window before or behind
                b0 = s.sum[1] >= target ? max(0, b0 - kWindow) : min(b0 + kWindow, kBins - kWindow);
                __syncthreads();
            }
        }
    }
    if (list_to >= 0) {
        // few tokens: the first CTA ranks them all by counting, and ends the row
        if (tid == 0) s.n_list = 0;
        x.sync_cluster();
        x.gather([&](float l, uint32_t, int) { return l > -INFINITY && x.bin(l) <= list_to; },
                 [&](float l) { return x.units(l); });
        x.sync_cluster();
        if (x.rank != 0) return;
        const int n = s.n_list;
        Item me{0, 0};
        u64 before = 0;
        int place = 0;
        if (tid < n) {
            me = s.list[tid];
            for (int j = 0; j < n; ++j) {
                const Item o = s.list[j];
                if (o.order > me.order) {
                    before += o.stat;
                    ++place;
                }
            }
        }
        auto add = [](u64 p, u64 q) { return p + q; };
        bool keep = tid < n && (!by_k || place < k);
        if (by_p) {
            if (by_k) {
                const u64 t = x.block_first(keep ? me.stat : 0, add);
                if (tid == 0) s.word[0] = t;
                __syncthreads();
                all_mass = s.word[0];
            }
            keep = keep && before < mass_target(p, all_mass);
        }
        keep = keep && uint32_t(me.order >> 32) >= k_min_p;
        const u64 total_first = x.block_first(keep ? me.stat : 0, add);
        if (tid == 0) s.word[0] = total_first;
        __syncthreads();
        if (tid < n) s.list[tid].stat = keep ? me.stat : 0;
        __syncthreads();
        const u64 total = s.word[0], target = draw_target(u, total);
        if (keep) {
            u64 run = 0;
            for (int j = 0; j < n; ++j) {
                const Item o = s.list[j];
                // a lower index is a larger lower word
                if (uint32_t(o.order) > uint32_t(me.order)) run += o.stat;
            }
            if (run <= target && target < run + me.stat)
                finish(int(~uint32_t(me.order)), log_prob(value_of(uint32_t(me.order >> 32)), x.top, temp, total));
        }
        return;
    }
    if (k_min_p > x.K) {
        x.K = k_min_p;
        x.I = V;
        know_mass = false;
    }
    auto stat = [&](float l, int i) -> u64 { return x.kept(key_of(l), i) ? x.units(l) : 0; };
    auto sums = [&]() {
        Weight m{0, 0};
        x.each([&](float l, int i) {
            if (x.kept(key_of(l), i)) m += x.weigh(l);
        });
        x.warp_sums(m.units());
    };
    if (!know_mass) {
        sums();
        if (tid == 0) {
            u64 t = 0;
            for (int w = 0; w < kWarps; ++w) t += s.warp_sum[w];
            s.out[0] = t;
        }
    } else if (tid == 0) {
        s.out[0] = s.word[3];
    }
    const auto got = x.exchange(1);
    u64 run = 0, total = 0;
    for (int r = 0; r < n_cta; ++r) {
        if (r < x.rank) run += got[r][0];
        total += got[r][0];
    }
    const u64 target = draw_target(u, total);
    if (!(run <= target && target < run + got[x.rank][0])) return;
    if (know_mass) sums();
    x.find(target, run, stat, [&](float l, int i) { finish(i, log_prob(l, x.top, temp, total)); });
}

// CTAs per row, a power of two up to 16
int row_ctas(int rows, int vocab, int elem, int sms) {
    const size_t bytes = size_t(vocab) * elem + 16;
    int n = 1;
    while (n < kMaxCluster && bytes / n > 64 * 1024) n *= 2;
    // few rows: more CTAs each, while they are not more than two per SM and have a few vectors a thread
    while (n < kMaxCluster && rows * n * 2 <= 2 * sms && bytes / (2 * n) >= 8 * 1024) n *= 2;
    return n;
}

template <typename L> cudaError_t launch_t(const SampleArgs &a, int sms, cudaStream_t stream) {
    const int n = row_ctas(a.B * a.T, a.V, sizeof(L), sms);
    constexpr int E = Vec<L>::N;
    const int row_vecs = (a.V + 2 * E - 2) / E;              // whatever its first vector's alignment
    const int vecs = (row_vecs + n - 1) / n;
    const size_t smem = (sizeof(Shared) + 15) / 16 * 16 + size_t(vecs) * 16;
    auto kern = sample_kernel<L>;
    // function attributes belong to the context: the limits raised so far, by context id
    struct Attrs {
        int smem = 0;
        bool nonportable = false;
    };
    static PerContext<Attrs> attrs;
    unsigned long long ctx = 0;
    Attrs have;
    const bool known = current_context_id(&ctx) && attrs.get(ctx, &have);
    if (!known || int(smem) > have.smem || (n > 8 && !have.nonportable)) {
        cudaError_t e = cudaSuccess;
        if (int(smem) > have.smem) {
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
            if (e != cudaSuccess) return e;
            have.smem = int(smem);
        }
        if (n > 8 && !have.nonportable) {
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess) return e;
            have.nonportable = true;
        }
        if (current_context_id(&ctx)) attrs.put(ctx, have);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(a.B) * unsigned(a.T) * unsigned(n), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = n;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, a, n, vecs);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a, gdn_dtype dtype, int sm_count, cudaStream_t stream) {
    return dtype == GDN_BF16 ? launch_t<__nv_bfloat16>(a, sm_count, stream) : launch_t<float>(a, sm_count, stream);
}

}  // namespace gdn
