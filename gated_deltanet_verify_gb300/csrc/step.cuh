// step.cuh -- argument blocks of the operators around the block: sampling, acceptance, adapters.  (Apart from
// internal.cuh, whose text is part of what recorded measurements of the block's kernels are keyed on.)
#pragma once

#include "internal.cuh"

namespace gdn {

// One token per row of logits (sample.cu).
struct SampleArgs {
    int B, T, V;
    long long ld;                     // row stride of the logits (elements)
    const void *logits;
    const float *u;                   // [B][T]
    const float *temperature, *top_p, *min_p;   // [B] each, NULL: 1, off, off
    const int32_t *top_k;             // [B], NULL: off
    int32_t *tokens;                  // [B][T]
    float *logprob;                   // [B][T] or NULL
    int *d_status;
};

// The accepted prefix or path of a draft (accept.cu).
struct AcceptArgs {
    int B, T;
    const int32_t *parent;            // [B][T]: a tree; NULL: a chain
    const int32_t *draft, *tokens;    // [B][T]
    const int32_t *length;            // [B] or NULL
    int32_t *place;                   // [B]: trim (chain) or accepted node (tree)
    int32_t *next;                    // [B] or NULL
    int32_t *emit, *path;             // [B][T] or NULL
    int *d_status;
};

// The low-rank adapters beside one projection (lora.cu, proj.cu).
struct LoraArgs {
    int n_adapters, rank, T;          // T: rows of X per slot
    const void *a, *b;                // [n_adapters][rank][K], [n_adapters][N][rank] bf16
    const float *scale;               // [n_adapters] or NULL (1)
    const int32_t *adapter;           // [slots]
    void *h;                          // scratch: lora_scratch_bytes
};

// Return a cudaError_t of the launch (cudaSuccess when enqueued).
cudaError_t launch_sample(const SampleArgs &a, gdn_dtype dtype, int sm_count, cudaStream_t stream);
cudaError_t launch_accept(const AcceptArgs &a, cudaStream_t stream);
// h = scale * X A^T per slot and group of 16 rows; reports an adapter id that names none.
cudaError_t launch_lora_shrink(const void *X, int M, int K, const LoraArgs &lora, int sms, int *d_status, cudaStream_t stream);
size_t lora_scratch_bytes(long long slots, int T, int rank);
// Aligned groups of 16 rows that the T rows of one slot may touch.
int lora_groups_per_slot(int T);

// gemm_xwt_bf16 with the low-rank term of each slot's adapter added to the fp32 sums.
bool gemm_xwt_lora_bf16(const void *W, const void *X, void *C, int M, int N, int K, long long ldc, const LoraArgs &lora,
                        int sms, int *d_status, cudaStream_t stream, std::string &why);

}  // namespace gdn
