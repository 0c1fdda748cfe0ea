// lora.cu -- the first half of a low-rank adapter: h = scale_a X A_a^T, each
// slot's rows with the slot's own adapter.  The second half, h B_a^T, goes
// through the tensor cores into the accumulators of the shared projection
// (proj.cu), so a projection with adapters rounds its output once, like one
// without.
//
// Unit of work: a pair of a slot and one of the aligned groups of 16 rows of X
// that its rows touch (rows of other slots count as zero), because the second
// half is a product over such groups.  h is summed in fp32 and stored as three
// bf16 numbers of 8 bits each, which together hold all 24 of it: the three
// products that this costs the tensor cores are cheaper than fp32 arithmetic, and
// h enters the output's sums unrounded.  (Two numbers, with 2^-17 of
// h lost: 94.5 us against 94.7 at 32 slots of rank 16, 104 against 106 at rank 64.)
//
// X and A are read once each per pair, straight from global memory into the
// fragments of mma.sync (m16n8k16, bf16, fp32 sums): with K permuted alike on
// both sides a lane's fragments of two k steps are 16 contiguous bytes of a
// row.  The work is a stream of A at best (r K elements a slot), and a chain of
// a few loads at one slot; so K is split over a cluster of up to 8 CTAs and
// their 8 warps, and the sums are joined through distributed shared memory in a
// fixed order.
//
// Measured, a projection with adapters against the same without (captured graph):
// input projection, hidden 5120, one slot of 16 rows, rank 16: 30.6 us against
// 28.1; 32 slots: 94.7 against 86.7; 8 slots of rank 128: 49.4 against 34.6; output
// projection, 8 slots of rank 64: 25.1 against 18.4.  This kernel runs beside the
// projection's weight stream, which does not wait for it; what is left are loads
// that take 4-5 us a round while that stream fills HBM's queues, and the adapters'
// own tiles at the end of the projection's ring.
#include "step.cuh"

#include <cuda_bf16.h>

namespace gdn {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxSplit = 8;

struct ShrinkArgs {
    const __nv_bfloat16 *X, *A;
    int M, K, T, r, P, n_adapters;
    const int32_t *adapter;
    const float *scale;
    __nv_bfloat16 *h;                // [pair][high, middle, low][16][r]
    int *d_status;
};

__device__ __forceinline__ uint32_t map_cluster(const void *p, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(uint32_t(__cvta_generic_to_shared(p))), "r"(rank));
    return r;
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];\n" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
__device__ __forceinline__ uint4 ld16(const __nv_bfloat16 *p, bool ok) {
    return ok ? *reinterpret_cast<const uint4 *>(p) : make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// R8: the tiles of eight rank columns held in registers, at most; more than 64 columns go to CTAs by 64
template <int R8>
__global__ void __launch_bounds__(kThreads) lora_shrink_kernel(const ShrinkArgs a) {
    extern __shared__ float part[];              // [kWarps / 2][16][rl]; the first [16][rl] holds the CTA's sum afterwards
    // The projection starts once every CTA here has seen the kernel before complete, so it may read X at once; it
    // waits for this grid's results itself.
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const int pair = blockIdx.x, s = pair / a.P, j = pair % a.P;
    const int group = s * a.T / 16 + j;
    if (group * 16 >= (s + 1) * a.T) return;     // the slot's rows end before: uniform over the cluster
    const int id = a.adapter[s];
    if (id < 0 || id >= a.n_adapters) {
        if (id != -1 && threadIdx.x == 0 && a.d_status) atomicCAS(a.d_status, int(GDN_OK), int(GDN_ERR_ADAPTER));
        return;
    }
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int r = a.r, j0 = blockIdx.z * 64, rl = min(64, r - j0), n8 = rl / 8, S = gridDim.y, split = blockIdx.y;
    const int m0 = group * 16 + g, m1 = m0 + 8, lo = s * a.T, hi = min(a.M, lo + a.T);
    const bool in0 = m0 >= lo && m0 < hi, in1 = m1 >= lo && m1 < hi;
    const __nv_bfloat16 *x0 = a.X + (size_t)m0 * a.K, *x1 = a.X + (size_t)m1 * a.K;
    const __nv_bfloat16 *w = a.A + ((size_t)id * r + j0 + g) * a.K;
    float acc[R8][4];
#pragma unroll
    for (int n = 0; n < R8; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
    // the loads of kAhead steps are in flight at once
    constexpr int kAhead = 4;
    const int step = S * kWarps * 32;
    for (int k0 = (split * kWarps + wid) * 32; k0 < a.K; k0 += kAhead * step) {
        uint4 p[kAhead], q[kAhead], b[kAhead][R8];
#pragma unroll
        for (int h = 0; h < kAhead; ++h) {
            const int k = k0 + h * step + 8 * t;
            const bool ok = k < a.K;             // K is a multiple of 8
            p[h] = ld16(x0 + k, ok && in0);
            q[h] = ld16(x1 + k, ok && in1);
#pragma unroll
            for (int n = 0; n < R8; ++n) b[h][n] = ld16(w + (size_t)n * 8 * a.K + k, ok && n < n8);
        }
#pragma unroll
        for (int h = 0; h < kAhead; ++h)
#pragma unroll
            for (int n = 0; n < R8; ++n) {
                mma16816(acc[n], p[h].x, q[h].x, p[h].y, q[h].y, b[h][n].x, b[h][n].y);
                mma16816(acc[n], p[h].z, q[h].z, p[h].w, q[h].w, b[h][n].z, b[h][n].w);
            }
    }
    // the upper half of the warps leave their sums, the lower half add theirs: half the shared memory, so that a CTA of the
    // projection finds room beside this one
    float *mine = part + (wid & (kWarps / 2 - 1)) * 16 * rl;
#pragma unroll
    for (int half = 1; half >= 0; --half) {
        if (wid / (kWarps / 2) == half)
#pragma unroll
            for (int n = 0; n < R8; ++n)
                if (n < n8) {
                    float2 *u = reinterpret_cast<float2 *>(mine + g * rl + n * 8 + 2 * t);
                    float2 *v = reinterpret_cast<float2 *>(mine + (g + 8) * rl + n * 8 + 2 * t);
                    const float2 x = half ? make_float2(0.f, 0.f) : *u, y = half ? make_float2(0.f, 0.f) : *v;
                    *u = make_float2(x.x + acc[n][0], x.y + acc[n][1]);
                    *v = make_float2(y.x + acc[n][2], y.y + acc[n][3]);
                }
        __syncthreads();
    }
    for (int i = threadIdx.x; i < 16 * rl; i += kThreads) {
        float v = part[i];
#pragma unroll
        for (int q = 1; q < kWarps / 2; ++q) v += part[q * 16 * rl + i];
        part[i] = v;                             // only this thread reads or writes element i of any part
    }
    const float scale = a.scale ? a.scale[id] : 1.0f;
    if (S > 1) cluster_sync();
    else __syncthreads();
    // the CTAs of the cluster share out the elements
    for (int i = split * kThreads + threadIdx.x; i < 16 * rl; i += S * kThreads) {
        float v = part[i];
        if (S > 1) {
            float w[kMaxSplit];                  // all in flight at once
#pragma unroll
            for (int q = 0; q < kMaxSplit; ++q) w[q] = q < S ? ld_cluster(map_cluster(part + i, q)) : 0.f;
            v = w[0];
#pragma unroll
            for (int q = 1; q < kMaxSplit; ++q) v += w[q];
        }
        // rows of other slots are zero whatever the adapter holds
        const int m = group * 16 + i / rl;
        v = m >= lo && m < hi ? v * scale : 0.f;
        // cut off, not rounded: the differences are exact, and a finite h stays finite
        const __nv_bfloat16 high = __float2bfloat16_rz(v);
        float rest = v - __bfloat162float(high);
        rest = rest - rest == 0.f ? rest : 0.f;  // an infinite or NaN h stays what it is
        const __nv_bfloat16 middle = __float2bfloat16_rz(rest);
        __nv_bfloat16 *to = a.h + ((size_t)pair * 48 + i / rl) * r + j0 + i % rl;
        to[0] = high;
        to[16 * r] = middle;
        to[32 * r] = __float2bfloat16_rn(rest - __bfloat162float(middle));
    }
    if (S > 1) cluster_sync();                   // the peers have read this CTA's sums
}

template <int R8> cudaError_t launch_t(const ShrinkArgs &a, int pairs, int sms, cudaStream_t stream) {
    // CTAs a pair and 64 rank columns: while there is an SM for each, and every warp has a k step (output projection,
    // 8 slots of rank 64: 45, 32, 28, 24.5 us with 1, 2, 4, 8; 32 slots, two CTAs an SM: 62 us against 54)
    const int parts = (a.r + 63) / 64;
    int S = 1;
    while (S < kMaxSplit && (long long)pairs * parts * S * 2 <= sms && a.K >= 2 * S * kWarps * 32) S *= 2;
    const size_t smem = size_t(kWarps / 2) * 16 * (a.r < 64 ? a.r : 64) * 4;
    auto kern = lora_shrink_kernel<R8>;
    // An SM that has its shared memory divided for a small kernel takes none of the projection's CTAs until it is empty
    // (input projection, 32 slots of one row: 40.5 us against 37; 32 of 16 rows: 97.6 against 95).  Function attributes
    // belong to the context: set once in each.
    static PerContext<int> attrs;
    unsigned long long ctx = 0;
    int set = 0;
    if (!(current_context_id(&ctx) && attrs.get(ctx, &set))) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout,
                                                   cudaSharedmemCarveoutMaxShared);
        if (e != cudaSuccess) return e;
        if (current_context_id(&ctx)) attrs.put(ctx, 1);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(pairs), unsigned(S), unsigned(parts));
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1;
    attr[1].val.clusterDim.y = S;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace

int lora_groups_per_slot(int T) { return T % 16 == 0 ? T / 16 : (T + 14) / 16 + 1; }

size_t lora_scratch_bytes(long long slots, int T, int rank) {
    return size_t(slots) * lora_groups_per_slot(T) * 48 * rank * 2;
}

cudaError_t launch_lora_shrink(const void *X, int M, int K, const LoraArgs &l, int sms, int *d_status, cudaStream_t stream) {
    const int P = lora_groups_per_slot(l.T);
    const ShrinkArgs a{static_cast<const __nv_bfloat16 *>(X), static_cast<const __nv_bfloat16 *>(l.a), M, K, l.T, l.rank, P,
                       l.n_adapters, l.adapter, l.scale, static_cast<__nv_bfloat16 *>(l.h), d_status};
    const int pairs = M / l.T * P;
    if (l.rank <= 16) return launch_t<2>(a, pairs, sms, stream);
    if (l.rank <= 32) return launch_t<4>(a, pairs, sms, stream);
    return launch_t<8>(a, pairs, sms, stream);
}

}  // namespace gdn
