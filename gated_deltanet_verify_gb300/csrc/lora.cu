// lora.cu -- the first half of a low-rank adapter: h = scale_a X A_a^T, each
// slot's rows with the slot's own adapter.  The second half, h B_a^T, is added
// to the shared projection's fp32 sums in the GEMM's epilogue (proj.cu), so a
// projection with adapters rounds once, like one without.  h stays in fp32.
#include "internal.cuh"

#include <cuda_bf16.h>

namespace gdn {
namespace {

constexpr int kThreads = 256;

// one warp per (row, rank column)
__global__ void __launch_bounds__(kThreads) lora_shrink_kernel(const __nv_bfloat16 *X, int M, int K, const LoraArgs a,
                                                               int *d_status) {
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const int lane = threadIdx.x & 31;
    const long long i = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (i >= (long long)M * a.rank) return;
    const int m = int(i / a.rank), j = int(i % a.rank);
    const int id = a.adapter[m / a.T];
    if (id < 0 || id >= a.n_adapters) {
        if ((id < -1 || id >= a.n_adapters) && lane == 0 && d_status)
            atomicCAS(d_status, int(GDN_OK), int(GDN_ERR_ADAPTER));
        return;
    }
    const __nv_bfloat16 *x = X + (size_t)m * K;
    const __nv_bfloat16 *w = static_cast<const __nv_bfloat16 *>(a.a) + ((size_t)id * a.rank + j) * K;
    float acc = 0.f;
    for (int k = lane; k < K; k += 32) acc = fmaf(__bfloat162float(x[k]), __bfloat162float(w[k]), acc);
#pragma unroll
    for (int s = 16; s; s >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, s);
    if (lane == 0) a.h[i] = a.scale ? a.scale[id] * acc : acc;
}

}  // namespace

size_t lora_scratch_bytes(long long M, int rank) { return size_t(M) * rank * 4; }

cudaError_t launch_lora_shrink(const void *X, int M, int K, const LoraArgs &lora, int *d_status, cudaStream_t stream) {
    const long long warps = (long long)M * lora.rank;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned((warps + kThreads / 32 - 1) / (kThreads / 32)), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, lora_shrink_kernel, static_cast<const __nv_bfloat16 *>(X), M, K, lora, d_status);
}

}  // namespace gdn
