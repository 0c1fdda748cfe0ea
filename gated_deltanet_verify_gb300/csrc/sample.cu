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
// is a 64-bit integer in units of about 2^-44 of the largest one (weight.cuh), and
// the integer sums do not depend on the order they are taken in -- the token is
// the same whatever the launch shape.  It equals the one of 64-bit arithmetic
// unless u lies nearer to a border than the weights' errors together: ~1e-12 of
// the sum as a rule, at most V 2^-45 + 2^-34 of it (1.5e-8 if 524288 light tokens
// all round the same way; u itself comes in steps of 6e-8).  A token lighter than
// half a unit is never drawn.  For the same reason the atomics below (integer
// counts and masses) leave no trace of their order.
//
// A thread-block cluster of 1 to 16 CTAs takes a row and goes over it two or
// three times; the first pass reads HBM, the others find it in L2:
//   1. the top logit and its lowest index (all that temperature 0 needs);
//   2. top-k: the tokens from a bound on, to the first CTA's list.  The bound is
//      the k-th largest of the threads' own tops, so it lies just below the k-th
//      token wherever threads rarely hold two of the first k.  If the list stays
//      short (kFew), the first CTA ranks it by counting and ends the row alone;
//   3. top-p (or a long top-k): a histogram of the tokens over bins of 1/64
//      octave of weight, merged over the cluster, gives about where the border
//      lies;
//   4. the exact masses of all tokens and of those before the border's bin; the
//      tokens of that bin (or two) go to the list, where a radix selection over
//      (key, index) finds the border.  If they are too many, once more with cells
//      of 1/1024 bin; if they are equal, they are counted off by index.  Without
//      top-k and top-p this pass only sums;
//   5. the warp that holds the drawn place goes over its stretch once more.
//
// What bounds it: with many rows instruction issue (60 instructions a token in
// all without filters, about 25 of them the exact weight; 64 % of the issue slots
// used); with few rows latency -- a cluster barrier costs ~0.7 us, a block-wide
// sum ~0.5 us, and code that is run once waits for its instructions.
//
// Measured, f32 (bf16), per call in a captured graph: one row of 32768, greedy
// 3.4 us (3.3), no filter 7.9 (8.9), top-k + top-p + min-p 10.0 (9.8), top-p alone
// 19.7 (23.4); 16 rows of 131072, top-p 36.2 (41.7); 128 rows of 100003, no filter
// 34.0 (29.3), top-p 69.5 (83); 256 rows of 200000, greedy 37 us (5.5 TB/s), no
// filter 113 (96), top-p 215 (199), mixed filters 157 (134).
#include "step.cuh"

#include <cuda_bf16.h>

#include "weight.cuh"

namespace gdn {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kBins = 2944;              // 1/64 octave each: 46 octaves; weights end at 45.5
constexpr float kBinOctaves = 1.0f / 64;
constexpr int kHead = 512;               // bins whose tokens' places inside them are summed too
constexpr int kFine = 1024;              // cells a bin, where a bin is too full
constexpr int kList = 2048;
constexpr int kFew = 512;
constexpr int kSmall = 256;              // items that are ranked by counting in a selection
constexpr int kCells = 512;
constexpr int kMaxCluster = 16;
constexpr int kExchange = 5;
using u64 = unsigned long long;

struct Item {
    u64 order;                           // key, then the index counted down: larger comes first
    u64 stat;
};

struct Shared {
    WeightTable table;
    Item list[kList];
    Item small[kSmall];
    u64 cell_stat[kCells];
    u64 xch[2][kMaxCluster][kExchange];  // what each CTA of the cluster sent, two rounds
    u64 out[kExchange], part[32][kExchange];     // what this CTA sends; its warps' parts of that
    u64 red[32];
    u64 warp_sum[32];                    // each warp's kept mass
    u64 warp_ties[32];
    u64 word, word2;                     // broadcast by the first CTA, or within a CTA
    double t_log_min_p;
    uint32_t hist[kBins];                // this CTA's counts
    uint32_t count[kBins];               // the cluster's, summed up to and with each bin
    uint32_t hist_in[kHead], in[kHead];  // the sums of places inside the first bins, in 1/256 bin: this CTA's, all
    float fred[32];
    u64 place;                           // a bin, and as a float the fraction of it
    uint32_t ured[32];
    uint32_t n_list, n_small;
    int found;
};

constexpr size_t kSharedBytes = (sizeof(Shared) + 15) / 16 * 16;

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
__device__ __forceinline__ void unpack(const uint4 &v, float (&f)[4], float) {
    f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y); f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ void unpack(const uint4 &v, float (&f)[8], __nv_bfloat16) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

struct Add {
    __device__ __forceinline__ u64 operator()(u64 a, u64 b) const { return a + b; }
};
struct Most {
    __device__ __forceinline__ u64 operator()(u64 a, u64 b) const { return a > b ? a : b; }
};

enum Border { kFound, kBefore, kBehind, kCrowded };

template <typename L, int NT>
struct Sampler {
    static constexpr int E = 16 / sizeof(L);
    static constexpr int kWarps = NT / 32;
    static constexpr int kRing = NT == 1024 ? 4 : 2;     // vectors of a thread on their way, a power of two
    static constexpr int kPer = (kBins + NT - 1) / NT;
    Shared &s;
    uint4 *ring;                         // [kRing][NT]
    const L *row;                        // the row's first logit
    const uint4 *vecs;                   // the row as 16-byte vectors from the last boundary before it
    int V, head;                         // head: elements of vector 0 before the row
    int row_vecs, cta_vecs;
    int v0, nv, seg;                     // this CTA's vectors: v0 .. v0 + nv; seg of them a warp
    int n_cta, rank, round;
    int tid, lane, wid;
    float top;
    Scale sc;
    float bin_scale;                     // bins per unit of logit
    float low;                           // kept: logit > low, or logit == low and index <= I (a masked one never is)
    int I;

    __device__ __forceinline__ bool kept(float l, int i) const { return l > low || (l == low && i <= I); }
    __device__ __forceinline__ u64 units(float l) const {
        Weight w;
        weights<1>(&l, l, sc, s.table, &w);
        return w.units();
    }
    // the logit at which bin b (or cell b of bins of 1/kFine) begins, going down; the top logit always lies in the first,
    // though a logit as large as a mask's lowest value swallows a bin's width
    __device__ __forceinline__ float edge_of(float b, float scale) const {
        return b <= 0.f ? INFINITY : fminf(top - __fdiv_rn(b, scale), value_of(key_of(top) - 1));
    }

    __device__ __forceinline__ void start_row(const SampleArgs &a, int r) {
        row = static_cast<const L *>(a.logits) + size_t(r) * size_t(a.ld);
        head = int((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(L));
        vecs = reinterpret_cast<const uint4 *>(row - head);
        row_vecs = (head + V + E - 1) / E;
        v0 = min(row_vecs, rank * cta_vecs);
        nv = min(row_vecs, v0 + cta_vecs) - v0;
        seg = (nv + kWarps - 1) / kWarps;
    }

    __device__ __forceinline__ void sync_cluster() const {
        __syncwarp();
        if (n_cta == 1) __syncthreads();
        else asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
    }

    // vector v of the row; what lies beside the row is masked (the last vector may end behind the buffer)
    __device__ __forceinline__ void load(int v, float (&l)[E]) const {
        const int i0 = v * E - head;
        if (i0 >= 0 && i0 + E <= V) {
            unpack(vecs[v], l, L());
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) l[e] = i0 + e >= 0 && i0 + e < V ? to_float(row[i0 + e]) : -INFINITY;
        }
    }
    // f(logits, v) for every vector of this CTA, warps over stretches of their own.  A thread's next vectors are on their
    // way to a ring of its own in shared memory meanwhile (with two of them in registers instead, a pass took as long as
    // the loads' latency allowed: 256 bf16 rows of 200000, the top logit alone, 36 us against 24)
    template <typename F> __device__ __forceinline__ void each_vec(F f) const {
        const int end = v0 + min(nv, (wid + 1) * seg), start = v0 + wid * seg + lane;
        const int first = head ? 1 : 0, n_whole = (head + V) / E - first;          // vectors inside the row
        const uint32_t slots = smem_u32(ring + tid);
        uint32_t slot = 0;
        const uint4 *src = vecs + start;
        auto fetch = [&](int v, uint32_t at) {
            if (v < end && unsigned(v - first) < unsigned(n_whole))
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(slots + at), "l"(src) : "memory");
            asm volatile("cp.async.commit_group;\n" ::: "memory");
            src += 32;
        };
#pragma unroll
        for (int j = 0; j < kRing - 1; ++j) fetch(start + 32 * j, uint32_t(j) * NT * 16);
        for (int v = start; v < end; v += 32) {
            fetch(v + 32 * (kRing - 1), (slot + (kRing - 1) * NT * 16) & (kRing * NT * 16 - 1));
            asm volatile("cp.async.wait_group %0;\n" ::"n"(kRing - 1) : "memory");
            float l[E];
            if (unsigned(v - first) < unsigned(n_whole)) {
                uint4 u;
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(slots + slot) : "memory");
                unpack(u, l, L());
            } else {
                load(v, l);
            }
            slot = (slot + NT * 16) & (kRing * NT * 16 - 1);
            f(l, v);
        }
    }
    // f(logit, index) for every element
    template <typename F> __device__ __forceinline__ void each(F f) const {
        each_vec([&](const float (&l)[E], int v) {
#pragma unroll
            for (int e = 0; e < E; ++e) f(l[e], v * E - head + e);
        });
    }
    // f(logit, weight, index in the vector, vector) for every element, four at a time, but those where all are below low; a
    // token is kept if the logit that f gets is at least low (that of one at low, but behind I, is -inf)
    template <typename F> __device__ __forceinline__ void each_weight(F f) const {
        each_vec([&](const float (&l)[E], int v) {
#pragma unroll
            for (int e = 0; e < E; e += 4) {
                float m[4] = {l[e], l[e + 1], l[e + 2], l[e + 3]};
                if (I < V)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (m[j] == low && v * E - head + e + j > I) m[j] = -INFINITY;
                const float most = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
                if (!(most >= low)) continue;      // none is kept
                Weight w[4];
                weights<4>(m, most, sc, s.table, w);
#pragma unroll
                for (int j = 0; j < 4; ++j) f(m[j], w[j], e + j, v);
            }
        });
    }

    template <typename Op> __device__ __forceinline__ u64 warp_all(u64 v, Op op) const {
#pragma unroll
        for (int m = 16; m; m >>= 1) v = op(v, u64(__shfl_xor_sync(kFull, v, m)));
        return v;
    }
    // a sum or maximum (0 is neutral to op) over the block, the same in all its threads
    template <typename Op> __device__ __forceinline__ u64 block_all(u64 v, Op op) const {
        v = warp_all(v, op);
        __syncthreads();
        if (lane == 0) s.red[wid] = v;
        __syncthreads();
        return warp_all(lane < kWarps ? s.red[lane] : 0ull, op);
    }
    // s.out[0 .. n) of every CTA to all: afterwards s.xch[round] holds them by rank
    __device__ __forceinline__ const u64 (*exchange(int n))[kExchange] {
        __syncthreads();
        round ^= 1;
        for (int t = tid; t < n * n_cta; t += NT) {
            const int to = t / n, j = t - to * n;
            st_cluster64(map_cluster(&s.xch[round][rank][j], to), s.out[j]);
        }
        sync_cluster();
        return s.xch[round];
    }
    // the same for N values of every warp in s.part, sums or (bit j of `largest`) maxima over the CTA's warps
    template <int N> __device__ __forceinline__ const u64 (*exchange_parts(unsigned largest))[kExchange] {
        __syncthreads();
        round ^= 1;
        for (int t = tid; t < N * n_cta; t += NT) {
            const int to = t / N, j = t - to * N;
            u64 v = s.part[0][j];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) {
                const u64 o = s.part[w][j];
                v = largest >> j & 1 ? (v > o ? v : o) : v + o;
            }
            st_cluster64(map_cluster(&s.xch[round][rank][j], to), v);
        }
        sync_cluster();
        return s.xch[round];
    }
    // one value of every thread over the cluster: the same in all its threads
    template <typename Op> __device__ __forceinline__ u64 cluster_all(u64 v, Op op) {
        v = block_all(v, op);
        if (n_cta == 1) return v;
        if (tid == 0) s.out[0] = v;
        const auto x = exchange(1);
        v = 0;
        for (int r = 0; r < n_cta; ++r) v = op(v, x[r][0]);
        return v;
    }
    template <typename T> __device__ __forceinline__ T warp_scan(T v) const {        // inclusive
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const T o = __shfl_up_sync(kFull, v, m);
            if (lane >= m) v += o;
        }
        return v;
    }

    __device__ __forceinline__ void clear() {
        for (int i = tid; i < kBins; i += NT) s.hist[i] = 0;
        for (int i = tid; i < kHead; i += NT) s.hist_in[i] = 0;
    }
    // the merged histogram of the kept tokens' places (top - l) scale - from, the last bin taking what lies beyond if
    // `open`, summed up to and with each bin, in s.count; with `open` also the sums of the places inside the first bins,
    // in s.in (a few heavy tokens taken at their bins' middles would spoil an estimate).  The list is empty afterwards.
    __device__ __forceinline__ void histogram(float scale, int first, bool open) {
        if (!open) clear();                      // at the start they are clear
        if (tid == 0) s.n_list = 0;
        __syncthreads();
        if (open && top < INFINITY) {
            const uint32_t counts = smem_u32(s.hist) - 4u * 0x4b400000u;
            const float heavy = top - __fdividef(kHead + 1.f, scale);
            each_vec([&](const float (&l)[E], int) {
                float most = l[0];
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    most = fmaxf(most, l[e]);
                    // the bin in the low bits of a sum that is rounded down, its ulp 1
                    const float x = fminf((top - l[e]) * scale, kBins - 0.5f);
                    const uint32_t at = counts + 4u * __float_as_uint(__fadd_rz(x, 12582912.f));
                    if (l[e] >= low) asm volatile("red.shared.add.u32 [%0], 1;\n" ::"r"(at) : "memory");
                }
                if (most > heavy)
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const float x = (top - l[e]) * scale;
                        const int b = __float2int_rz(x);
                        if (l[e] >= low && b < kHead) atomicAdd(&s.hist_in[b], uint32_t(__float2int_rz((x - b) * 256.f)));
                    }
            });
        } else {
            each([&](float l, int i) {
                if (!kept(l, i)) return;
                // 0 for the top logit (inf - inf gives NaN, which converts to 0)
                const int b = __float2int_rz((top - l) * scale) - first;
                if (unsigned(b) < unsigned(kBins)) atomicAdd(&s.hist[b], 1u);
            });
        }
        sync_cluster();
        const uint32_t *from = s.hist;
        if (n_cta > 1) {
            // lane r of a group of n_cta reads CTA r's count of a bin and, with their sum, writes CTA r's copy
            const int slice = kBins / n_cta, r = tid & (n_cta - 1);
            uint32_t c[kPer];                                       // whole warps: kBins is a multiple of 32
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                c[j] = tid + j * NT < kBins ? ld_cluster32(map_cluster(&s.hist[rank * slice + (tid + j * NT) / n_cta], r)) : 0;
            for (int m = n_cta >> 1; m; m >>= 1)
#pragma unroll
                for (int j = 0; j < kPer; ++j) c[j] += __shfl_xor_sync(kFull, c[j], m);
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                if (tid + j * NT < kBins) st_cluster32(map_cluster(&s.count[rank * slice + (tid + j * NT) / n_cta], r), c[j]);
            for (int t = tid; open && t < kHead; t += NT) {
                const int b = rank * (kHead / n_cta) + t / n_cta;
                uint32_t c = ld_cluster32(map_cluster(&s.hist_in[b], r));
                for (int m = n_cta >> 1; m; m >>= 1) c += __shfl_xor_sync(kFull, c, m);
                st_cluster32(map_cluster(&s.in[b], r), c);
            }
            sync_cluster();
            from = s.count;
        } else {
            for (int t = tid; t < kHead; t += NT) s.in[t] = s.hist_in[t];
        }
        uint32_t c[kPer], t = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) t += c[j] = kPer * tid + j < kBins ? from[kPer * tid + j] : 0;
        uint32_t run = warp_scan(t);
        if (lane == 31) s.ured[wid] = run;
        __syncthreads();
        const uint32_t w = warp_scan(lane < kWarps ? s.ured[lane] : 0u);
        run += (wid ? __shfl_sync(kFull, w, wid - 1) : 0u) - t;
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (kPer * tid + j < kBins) s.count[kPer * tid + j] = run += c[j];
        __syncthreads();
    }
    // the first bin up to which at least n tokens lie
    __device__ __forceinline__ int bin_of_count(uint32_t n) {
        for (int b = tid; b < kBins; b += NT)
            if (s.count[b] >= n && (b == 0 || s.count[b - 1] < n)) s.found = b;
        __syncthreads();
        const int b = s.found;
        __syncthreads();
        return b;
    }
    // about where the mass reaches `need` (or, need < 0, -need of that of the bins up to `last`), in units of the weight
    // at the start, bins `octaves` wide, each one's tokens taken at its middle (with `open`, in the first bins, at their
    // mean place): the bin and the fraction of it; past kBins if it is not reached
    __device__ __forceinline__ float place_of_mass(float need, int last, float octaves, bool open) {
        float c[kPer], t = 0.f;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int b = kPer * tid + j;
            const uint32_t n = b < kBins ? s.count[b] - (b ? s.count[b - 1] : 0) : 0;
            float in = open && b < kHead && n ? __fdividef(s.in[b] + 0.5f * n, 256.f * n) : 0.5f;
            if (sizeof(L) == 2 && open && b >= kHead) {
                // bf16 logits are sparse: the highest one that begins below the bin's edge, if it is the only one in it
                const uint32_t bits = __float_as_uint(top - __fdividef(float(b), bin_scale));
                const uint32_t v = (bits & 0x80000000u ? bits + 0xffffu : bits) & 0xffff0000u;
                const float at = (top - __uint_as_float(v)) * bin_scale - float(b);
                const float next = (top - __uint_as_float(bits & 0x80000000u ? v + 0x10000u : v - 0x10000u)) * bin_scale - float(b);
                if (at < 1.f && next >= 1.f) in = fmaxf(at, 0.f);
            }
            t += c[j] = b > last ? 0.f : float(n) * exp2f(-(b + in) * octaves);
        }
        float run = warp_scan(t);
        if (lane == 31) s.fred[wid] = run;
        if (tid == 0) s.place = u64(kBins) << 32;
        __syncthreads();
        const float w = warp_scan(lane < kWarps ? s.fred[lane] : 0.f);
        run += (wid ? __shfl_sync(kFull, w, wid - 1) : 0.f) - t;
        if (need < 0.f) need *= -__shfl_sync(kFull, w, 31);
        int mine = kBins;
        float fraction = 0.f;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            if (mine == kBins && run + c[j] >= need && c[j] > 0.f) {
                mine = kPer * tid + j;
                fraction = fminf(fmaxf(__fdividef(need - run, c[j]), 0.f), 1.f);
            }
            run += c[j];
        }
        if (mine < kBins) atomicMin(&s.place, (u64(mine) << 32) | __float_as_uint(fraction));
        __syncthreads();
        const u64 at = s.place;
        return float(at >> 32) + __uint_as_float(uint32_t(at));
    }

    // a token to the first CTA's list, if there is room; one atomic for the lanes that come here together
    __device__ __forceinline__ void push(uint32_t key, int i, u64 stat) const {
        const unsigned here = __activemask();
        const int first = __ffs(here) - 1;
        uint32_t at = 0;
        if (lane == first) at = add_cluster32(map_cluster(&s.n_list, 0), __popc(here));
        at = __shfl_sync(here, at, first) + __popc(here & ((1u << lane) - 1));
        if (at < kList) {
            const uint32_t to = map_cluster(s.list, 0) + at * 16;
            st_cluster64(to, (u64(key) << 32) | uint32_t(~i));
            st_cluster64(to + 8, stat);
        }
    }

    // with low: I, for this CTA, so that of the tokens of that logit (kept so far) the first `need` in index order are
    // kept; each warp's kept ones, times `one`, are added to s.warp_sum
    __device__ __forceinline__ void tie(float value, u64 need, u64 one) {
        auto same = [&](float l, int i) -> u64 { return l == value && kept(l, i); };
        u64 mine = 0;
        each([&](float l, int i) { mine += same(l, i); });
        mine = warp_all(mine, Add());
        __syncthreads();
        if (lane == 0) s.warp_ties[wid] = mine;
        __syncthreads();
        const u64 all = warp_all(lane < kWarps ? s.warp_ties[lane] : 0ull, Add());
        if (tid == 0) s.out[0] = all;
        const auto x = exchange(1);
        u64 run = 0;
        for (int r = 0; r < rank; ++r) run += x[r][0];
        if (tid == 0) {
            u64 to = run;
            for (int w = 0; w < kWarps; ++w) {
                const u64 n = s.warp_ties[w];
                s.warp_sum[w] += (need <= to ? 0 : min(need - to, n)) * one;
                to += n;
            }
        }
        int limit = run < need ? 0x7fffffff : -1;
        if (run < need && need < run + all) {
            find(need - 1, run, s.warp_ties, same, [&](float, int i) { s.found = i; });
            __syncthreads();
            limit = s.found;
        }
        __syncthreads();
        I = value == low ? min(I, limit) : limit;
        low = value;
    }

    // low and I where the stat of the kept tokens reaches target, by bisection over the keys
    template <typename S> __device__ __forceinline__ void slow_border(u64 target, S stat) {
        auto from = [&](uint32_t key) {
            const float least = value_of(key);
            u64 m = 0;
            each([&](float l, int i) {
                if (l >= least && kept(l, i)) m += stat(l);
            });
            return cluster_all(m, Add());
        };
        const uint32_t top_key = key_of(top);
        uint32_t lo = key_of(low), hi = top_key;
        while (lo < hi) {
            const uint32_t mid = lo + (hi - lo + 1) / 2;
            if (from(mid) >= target) lo = mid;
            else hi = mid - 1;
        }
        const float value = value_of(lo) + 0.0f;
        const u64 above = lo == top_key ? 0 : from(lo + 1), one = stat(value);
        tie(value, (target - above + one - 1) / one, 0);
    }

    // by the first CTA: the order of the list's item at which the stats, `before` and on, reach target, or 0
    __device__ __forceinline__ u64 select(int n, u64 before, u64 target) {
        u64 lo = 0, hi = 0;
        for (int t = tid; t < n; t += NT) {
            const u64 o = s.list[t].order;
            hi = max(hi, o);
            lo = max(lo, ~o);
        }
        hi = block_all(hi, Most());
        lo = ~block_all(lo, Most());
        int live = n;
        while (live > kSmall) {
            // cells of equal width from hi down
            const int shift = max(0, 55 - __clzll((long long)(hi - lo)));
            for (int t = tid; t < kCells; t += NT) {
                s.cell_stat[t] = 0;
                s.hist[t] = 0;
            }
            if (tid == 0) s.n_small = kCells;
            __syncthreads();
            for (int t = tid; t < n; t += NT) {
                const Item o = s.list[t];
                if (o.order < lo || o.order > hi) continue;
                const int c = int((hi - o.order) >> shift);
                atomicAdd(&s.cell_stat[c], o.stat);
                atomicAdd(&s.hist[c], 1u);
            }
            __syncthreads();
            if (wid == 0) {
                constexpr int kEach = kCells / 32;
                u64 t = 0;
                for (int j = 0; j < kEach; ++j) t += s.cell_stat[lane * kEach + j];
                u64 run = before + warp_scan(t) - t;
                for (int j = 0; j < kEach; ++j) {
                    const u64 c = s.cell_stat[lane * kEach + j];
                    if (run < target && target <= run + c) {
                        s.n_small = lane * kEach + j;
                        s.word2 = run;
                    }
                    run += c;
                }
            }
            __syncthreads();
            const u64 c = s.n_small;
            if (c == kCells) return 0;
            before = s.word2;
            live = int(s.hist[c]);
            if (c < ((hi - lo) >> shift)) lo = hi - ((c + 1) << shift) + 1;       // not the last cell
            hi -= c << shift;
            __syncthreads();
        }
        if (tid == 0) {
            s.n_small = 0;
            s.word2 = 0;
        }
        __syncthreads();
        for (int t = tid; t < n; t += NT) {
            const Item o = s.list[t];
            if (o.order >= lo && o.order <= hi) s.small[atomicAdd(&s.n_small, 1u)] = o;
        }
        __syncthreads();
        if (tid < live) {
            const Item me = s.small[tid];
            for (int j = 0; j < live; ++j) {
                const Item o = s.small[j];
                if (o.order > me.order) before += o.stat;
            }
            if (before < target && target <= before + me.stat) s.word2 = me.order;
        }
        __syncthreads();
        return s.word2;
    }

    // low and I where the stat of the kept tokens (MASS: their weights, else 1) reaches its target, among the tokens of
    // at most `from` and above `to`; target_of(all) gives it, from the stat of all kept tokens, which is returned, as is
    // that of the tokens above `from`.  With kFound s.warp_sum holds each warp's kept stat.  The list is empty before
    // and afterwards.
    template <bool MASS, typename T>
    __device__ __forceinline__ Border border(float from, float to, T target_of, u64 &all, u64 &before) {
        Weight w_all{0, 0}, w_before{0, 0};
        uint32_t n_all = 0, n_before = 0, n = 0, k_lo = 0xffffffffu, k_hi = 0;
        auto hold = [&](float l, int i, u64 stat) {
            const uint32_t key = key_of(l + 0.0f);
            ++n;
            k_lo = min(k_lo, key);
            k_hi = max(k_hi, key);
            push(key, i, stat);
        };
        if (MASS) {
            each_weight([&](float l, const Weight &w, int e, int v) {
                if (!(l >= low)) return;
                w_all += w;
                if (l > from) w_before += w;
                else if (l > to) hold(l, v * E - head + e, w.units());
            });
        } else {
            each([&](float l, int i) {
                if (!kept(l, i)) return;
                ++n_all;
                if (l > from) ++n_before;
                else if (l > to) hold(l, i, 1);
            });
        }
        const u64 p_before = warp_all(MASS ? w_before.units() : u64(n_before), Add());
        const u64 p_all = warp_all(MASS ? w_all.units() : u64(n_all), Add());
        n = __reduce_add_sync(kFull, n);
        k_lo = __reduce_min_sync(kFull, k_lo);
        k_hi = __reduce_max_sync(kFull, k_hi);
        if (lane == 0) {
            s.warp_sum[wid] = p_before;
            s.part[wid][0] = p_all;
            s.part[wid][1] = p_before;
            s.part[wid][2] = n;
            s.part[wid][3] = u64(~k_lo);
            s.part[wid][4] = k_hi;
        }
        const auto x = exchange_parts<5>(0x18);
        before = all = n = k_lo = k_hi = 0;
        for (int r = 0; r < n_cta; ++r) {
            all += x[r][0];
            before += x[r][1];
            n += uint32_t(x[r][2]);
            k_lo = max(k_lo, uint32_t(x[r][3]));
            k_hi = max(k_hi, uint32_t(x[r][4]));
        }
        k_lo = ~k_lo;
        const u64 target = target_of(all);
        const u64 one = n > kList && MASS ? units(value_of(k_lo)) : 1;
        const u64 need = one ? (target - before + one - 1) / one : u64(n) + 1;     // of equal tokens
        const Border got = before >= target ? kBefore : n == 0 ? kBehind : n <= kList ? kFound
                         : k_lo != k_hi ? kCrowded : need > n ? kBehind : kFound;
        if (got != kFound || n > kList) {
            if (tid == 0) s.n_list = 0;
            if (got == kFound) tie(value_of(k_lo), need, one);
            else sync_cluster();
            return got;
        }
        if (rank == 0) {
            const u64 at = select(int(n), before, target);
            if (at)
                for (int t = tid; t < int(n); t += NT) {
                    const Item o = s.list[t];
                    if (o.order < at) continue;
                    // a kept token: its mass to the warp in whose stretch it lies
                    const int v = (int(~uint32_t(o.order)) + head) / E, r = v / cta_vecs, first = r * cta_vecs;
                    const int its = (min(row_vecs, first + cta_vecs) - first + kWarps - 1) / kWarps;
                    add_cluster64(map_cluster(&s.warp_sum[(v - first) / its], r), o.stat);
                }
            if (tid < n_cta) st_cluster64(map_cluster(&s.word, tid), at);
            if (tid == 0) s.n_list = 0;
        }
        sync_cluster();
        const u64 at = s.word;
        if (at == 0) return kBehind;
        low = value_of(uint32_t(at >> 32));
        I = int(~uint32_t(at));
        return kFound;
    }

    // the same, the border being looked for: near `place` (in bins) first; whether s.warp_sum holds the kept stats
    template <bool MASS, typename T> __device__ __forceinline__ bool look_for(float place, T target_of) {
        u64 all = 0, before;
        // the estimate is good to a fraction of a bin
        float b0 = floorf(place - 0.45f), b1 = floorf(place + 0.45f) + 1.f;
        if (!MASS) b0 = floorf(place), b1 = b0 + 1.f;
        for (int turn = 0; turn < 6; ++turn) {
            Border got = border<MASS>(edge_of(b0, bin_scale), edge_of(b1, bin_scale), target_of, all, before);
            if (got == kFound) return true;
            if (got == kCrowded) {
                // cells of 1/kFine bin over three bins from b0 on
                const int first = int(fmaxf(b0, 0.f)) * kFine;
                const float scale = bin_scale * kFine;
                histogram(scale, first, false);
                const u64 need = target_of(all) - before;
                float c0, c1;
                if (MASS) {
                    const float at = place_of_mass(float(need) / float(units(top)) * exp2f(fmaxf(b0, 0.f) * kBinOctaves), kBins - 1,
                                                   kBinOctaves / kFine, false);
                    c0 = floorf(at) - 1.f;
                    c1 = floorf(at) + 2.f;
                } else {
                    c0 = bin_of_count(uint32_t(min(need, u64(s.count[kBins - 1]))));
                    c1 = c0 + 1.f;
                }
                if (border<MASS>(edge_of(first + c0, scale), edge_of(first + c1, scale), target_of, all, before) == kFound)
                    return true;
                break;
            }
            // off by a bin or more
            const float by = b1 - b0 + turn;
            if (got == kBefore) {
                b1 = b0 + 1.f;
                b0 = fmaxf(0.f, b0 - by);
            } else {
                b0 = b1 - 1.f;
                b1 += by;
            }
        }
        slow_border(target_of(all), [&](float l) { return MASS ? units(l) : u64(1); });
        return false;
    }

    // by the whole CTA, the sum of stat before it being `run` and its warps' sums `warp`: at(logit, index), by one
    // thread, of the first token in index order up to which the stats sum to more than `place`
    template <typename S, typename A> __device__ __forceinline__ void find(u64 place, u64 run, const u64 *warp, S stat, A at) {
        int w = 0;
        while (w < kWarps && place >= run + warp[w]) run += warp[w++];
        if (w == kWarps) return;
        // the stretch of warp w, one vector a thread and round
        const int end = v0 + min(nv, (w + 1) * seg);
        for (int u = v0 + w * seg; u < end && run <= place; u += NT) {
            const int v = u + tid;
            float l[E];
            u64 c[E], t = 0;
            if (v < end) load(v, l);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                c[e] = v < end ? stat(l[e], v * E - head + e) : 0;
                t += c[e];
            }
            const u64 to = warp_scan(t);
            __syncthreads();
            if (lane == 31) s.red[wid] = to;
            __syncthreads();
            const u64 ws = warp_scan(lane < kWarps ? s.red[lane] : 0ull);
            u64 before = run + (wid ? __shfl_sync(kFull, ws, wid - 1) : 0ull) + to - t;
            run += __shfl_sync(kFull, ws, 31);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (before <= place && place < before + c[e]) at(l[e], v * E - head + e);
                before += c[e];
            }
        }
    }
};

template <typename L, int NT, int PER_SM>
__global__ void __launch_bounds__(NT, PER_SM) sample_kernel(const SampleArgs a, int n_cta, int cta_vecs) {
    extern __shared__ __align__(16) unsigned char smem[];
    Shared &s = *reinterpret_cast<Shared *>(smem);
    Sampler<L, NT> x{s, reinterpret_cast<uint4 *>(smem + kSharedBytes)};
    constexpr int kWarps = NT / 32, E = Sampler<L, NT>::E;
    x.tid = threadIdx.x; x.lane = x.tid & 31; x.wid = x.tid >> 5;
    x.n_cta = n_cta; x.rank = int(blockIdx.x) & (n_cta - 1); x.round = 0;
    x.V = a.V; x.cta_vecs = cta_vecs;
    const int tid = x.tid, row = int(blockIdx.x) / n_cta, slot = row / a.T;

    // a CTA's shared memory may be written by its peers once it has started: the wait for all to have done so comes
    // before the first exchange
    if (n_cta > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;\n" ::: "memory");
    s.table.fill(tid, NT);
    x.clear();
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const float temp = a.temperature ? a.temperature[slot] : 1.0f;
    const float u = a.u[row];
    const int k = a.top_k ? a.top_k[slot] : 0;
    const float p = a.top_p ? a.top_p[slot] : 1.0f, mp = a.min_p ? a.min_p[slot] : 0.0f;
    const bool fine = sample_params_ok(temp, p, mp) && u >= 0.0f && u < 1.0f;
    x.start_row(a, row);

    bool by_k = k > 0 && k < a.V;
    const bool by_p = p < 1.0f;

    // 1. the top logit
    float best = -INFINITY;
    int best_v = 0, best_i = 0;
    x.each_vec([&](const float (&l)[E], int v) {
        float m = l[0];
#pragma unroll
        for (int e = 1; e < E; ++e) m = fmaxf(m, l[e]);         // of NaN and a number the number
        if (m > best) {
            best = m;
            best_v = v;
        }
    });
    if (best > -INFINITY) {
        float l[E];
        x.load(best_v, l);
#pragma unroll
        for (int e = E - 1; e >= 0; --e)
            if (l[e] == best) best_i = best_v * E - x.head + e;
    }
    const uint32_t k_best = key_of(best + 0.0f);
    if (tid == 0) {
        if (mp > 0.0f) s.t_log_min_p = double(temp) * log(double(mp));
        s.n_list = 0;
    }
    // top-k's bound: some key that at least k / n_cta of this CTA's threads reach (if that many hold a token at all);
    // the least of the CTAs' bounds is reached by k tokens
    const int share = (k + n_cta - 1) / n_cta;
    uint32_t bound = kNone + 1;
    const bool bounded = by_k && fine && temp != 0.0f && share <= NT / 4;
    if (bounded) {
        uint32_t lo = kNone + 1, hi = 0xff800000u;             // the key of +inf
        while (lo < hi) {
            const uint32_t mid = lo + (hi - lo + 1) / 2;
            const int n = __syncthreads_count(k_best >= mid);
            if (n >= share) lo = mid;
            else hi = mid - 1;
            if (n >= share && n <= share + share / 4) break;
        }
        bound = lo;
    }
    u64 first = x.warp_all((u64(k_best) << 32) | uint32_t(~best_i), Most());
    if (x.lane == 0) {
        s.part[x.wid][0] = first;
        s.part[x.wid][1] = uint32_t(~bound);
    }
    __syncwarp();
    if (n_cta > 1) asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory");
    {
        const auto got = x.template exchange_parts<2>(3);
        for (int r = 0; r < n_cta; ++r) {
            first = max(first, got[r][0]);
            bound = min(bound, uint32_t(~got[r][1]));
        }
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
    x.sc = scale_of(temp, x.top);
    x.bin_scale = scale_of(temp, 0.0f).hi / kBinOctaves;
    x.low = x.top == INFINITY ? INFINITY : -3.4028234e38f;       // of infinite logits all are equally likely, others out
    x.I = a.V;
    const uint32_t k_min_p = mp > 0.0f ? min_p_key(s.t_log_min_p, x.top) : 0u;
    bool short_list = false;
    if (bounded) {
        const float least = value_of(bound);
        x.each([&](float l, int i) {
            if (l >= least) x.push(key_of(l + 0.0f), i, 0);
        });
        x.sync_cluster();
        const uint32_t n = ld_cluster32(map_cluster(&s.n_list, 0));
        short_list = n <= kFew;
        // the first CTA stays until its peers have read n: it waits for them when it is done
        if (!short_list || x.rank != 0) x.sync_cluster();
        else if (n_cta > 1) asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
    }
    bool know_mass = false;                // s.warp_sum holds the kept masses
    if (!short_list && (by_k || by_p)) {
        x.histogram(x.bin_scale, 0, true);
        int last = kBins - 1;
        by_k = by_k && s.count[kBins - 1] > uint32_t(k);
        if (by_k) last = x.bin_of_count(k);
        const float place = by_p ? x.place_of_mass(-p, last, kBinOctaves, true) : 0.f;
        if (by_k) x.template look_for<false>(float(last), [&](u64) { return u64(k); });
        if (by_p) {
            know_mass = x.template look_for<true>(fminf(place, float(last)), [&](u64 all) { return mass_target(p, all); });
        }
    }
    if (short_list) {
        // the first CTA ranks them all by counting, and ends the row
        if (x.rank != 0) return;
        const int n = int(s.n_list);
        Item me{0, 0};
        u64 before = 0;
        int place = 0;
        if (tid < n) {
            me = s.list[tid];
            const float l = value_of(uint32_t(me.order >> 32));
            s.list[tid].stat = me.stat = l >= x.low ? x.units(l) : 0;
        }
        __syncthreads();
        if (tid < n) {
            for (int j = 0; j < n; ++j) {
                const Item o = s.list[j];
                if (o.order > me.order) {
                    before += o.stat;
                    ++place;
                }
            }
        }
        bool keep = tid < n && place < k;
        if (by_p) {
            const u64 all = x.block_all(keep ? me.stat : 0, Add());
            keep = keep && before < mass_target(p, all);
        }
        keep = keep && uint32_t(me.order >> 32) >= k_min_p;
        const u64 total = x.block_all(keep ? me.stat : 0, Add()), target = draw_target(u, total);
        if (tid < n) s.list[tid].stat = keep ? me.stat : 0;
        __syncthreads();
        if (keep) {
            u64 run = 0;
            for (int j = 0; j < n; ++j) {
                const Item o = s.list[j];
                // a lower index is a larger lower word
                if (uint32_t(o.order) > uint32_t(me.order)) run += o.stat;
            }
            if (run <= target && target < run + me.stat)
                finish(int(~uint32_t(me.order)), log_prob(value_of(uint32_t(me.order >> 32)), x.top, temp, x.units(x.top), total));
        }
        __syncwarp();
        if (n_cta > 1) asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
        return;
    }
    if (k_min_p > key_of(x.low)) {
        x.low = value_of(k_min_p);
        x.I = a.V;
        know_mass = false;
    }
    if (!know_mass) {
        Weight m{0, 0};
        x.each_weight([&](float l, const Weight &w, int, int) {
            if (l >= x.low) m += w;
        });
        const u64 mine = x.warp_all(m.units(), Add());
        __syncthreads();
        if (x.lane == 0) s.warp_sum[x.wid] = mine;
        __syncthreads();
    }
    const u64 mine = x.warp_all(x.lane < kWarps ? s.warp_sum[x.lane] : 0ull, Add());
    u64 run = 0, total = mine;
    if (n_cta > 1) {
        if (tid == 0) s.out[0] = mine;
        const auto got = x.exchange(1);
        total = 0;
        for (int r = 0; r < n_cta; ++r) {
            if (r < x.rank) run += got[r][0];
            total += got[r][0];
        }
    }
    const u64 target = draw_target(u, total);
    if (run <= target && target < run + mine)
        x.find(target, run, s.warp_sum, [&](float l, int i) -> u64 { return x.kept(l, i) ? x.units(l) : 0; },
               [&](float l, int i) { finish(i, log_prob(l, x.top, temp, x.units(x.top), total)); });
}

// CTAs per row, a power of two up to 16, threads per CTA and the CTAs that an SM has registers for
struct Plan {
    int n_cta, threads, per_sm;
};
Plan plan_of(int rows, int vocab, int sms) {
    // Few rows: a cluster each, of CTAs with an SM and its registers to themselves (one row of 32768, top-k: 8.3 us against
    // 9.0 with half the registers), 4096 tokens each at least.  Not every cluster finds that many SMs together: of four up
    // to 27/32 of the SMs (32 rows of 131072, top-p: 40 us; 38 rows: 62 us against 48 with two CTAs an SM), larger ones up
    // to 9/16 (10 rows, 8 CTAs: 31 us against 40 with 4; 16 rows: 54 against 36.5).
    const int most4 = int(sms * 27LL / 32), most = int(sms * 9LL / 16);
    int n = 1;
    while (n < kMaxCluster && (long long)rows * n * 2 <= (n <= 2 ? most4 : most) && vocab / (2 * n) >= 4096) n *= 2;
    // Up to almost half as many rows as SMs: four CTAs, two per SM, even out rows of different cost (64 mixed rows: 40 us
    // against 57 with two CTAs a row, one per SM).  The last SMs hold no cluster of four: 74 rows of 131072 with top-k take
    // 22 us, 76 would take 33, and 25 with one CTA a row.
    if (n < 4 && (long long)rows * 4 <= 2LL * sms - 8 && vocab / 4 >= 4096) return {4, 512, 2};
    // one CTA per row: 1024 threads while rows are fewer than two per SM (128 rows of 100003, top-p: 70 us against 88
    // with 512; 512 rows of 50000: 152 against 127); a thread's weights add up in 32 bits for 1000 tokens
    const bool wide = n == 1 && vocab > 8192 && (rows <= 2 * sms || vocab > 262144);
    return {n, wide ? 1024 : 512, wide || n > 1 || rows <= most4 ? 1 : 2};
}

template <typename L, int NT, int PER_SM> cudaError_t launch_t(const SampleArgs &a, int n, cudaStream_t stream) {
    constexpr int E = 16 / sizeof(L);
    const int row_vecs = (a.V + 2 * E - 2) / E;              // whatever its first vector's alignment
    const int vecs = (row_vecs + n - 1) / n;
    auto kern = sample_kernel<L, NT, PER_SM>;
    const size_t smem = kSharedBytes + size_t(Sampler<L, NT>::kRing) * NT * 16;
    // function attributes belong to the context: set once in each
    static PerContext<int> attrs;
    unsigned long long ctx = 0;
    int set = 0;
    if (!(current_context_id(&ctx) && attrs.get(ctx, &set))) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        if (current_context_id(&ctx)) attrs.put(ctx, 1);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(a.B) * unsigned(a.T) * unsigned(n), 1, 1);
    cfg.blockDim = dim3(NT, 1, 1);
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
    const Plan plan = plan_of(a.B * a.T, a.V, sm_count);
    auto launch = [&](auto logit) {
        using L = decltype(logit);
        return plan.threads == 1024 ? launch_t<L, 1024, 1>(a, plan.n_cta, stream)
               : plan.per_sm == 1   ? launch_t<L, 512, 1>(a, plan.n_cta, stream)
                                    : launch_t<L, 512, 2>(a, plan.n_cta, stream);
    };
    return dtype == GDN_BF16 ? launch(__nv_bfloat16()) : launch(float());
}

}  // namespace gdn
