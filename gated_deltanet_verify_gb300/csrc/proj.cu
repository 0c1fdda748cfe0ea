// proj.cu -- the projections either side of the GDN block: the fused input
// projection x -> [qkv | z | alpha | beta_raw] and the output projection
// out -> y, as one hand-written sm_103a GEMM kernel.
//
// Row-major C[M][N] (row stride ldc, bf16) = X[M][K] @ W[N][K]^T, bf16
// operands, fp32 accumulation.  In a verify step M = slots x tokens is small
// (16 rows for one slot) while W holds tens of MB, so the GEMM streams the
// weights: the weight rows are the tensor core's M dimension and the
// activation rows its N.
//
//   * One CTA per 128-row tile of W (and per split of K when the tiles are
//     too few to cover the SMs; a 256-row block of X per grid row).  The tile
//     is D = W_tile X^T (128 x Mt), fp32 in tensor memory (tcgen05.mma
//     kind::f16, bf16 A and B, both K-major from shared memory).
//   * Warp 0 is the TMA producer: each stage holds kKBlk columns of K of the
//     W tile and of X as 64-column (128-byte) TMA boxes in the 128-byte
//     swizzled K-major layout the tensor core reads directly.
//     Two threads issue the MMAs (8 per stage), warp 1 those of the ring's even
//     stages into one tensor-memory accumulator and warp 2 those of the odd
//     ones into a second, and
//     free each stage through tcgen05.commit on its "empty" barrier: one
//     thread's MMAs follow each other ~150 cycles apart whatever their size
//     (measured from M = 64, N = 16 to M = 128, N = 256), and two issuing
//     threads on an SM each keep that pace, so a second issuer doubles the
//     rate of these N = 16 MMAs.  The epilogue adds the two accumulators in a
//     fixed order.
//   * Programmatic dependent launch: the weight tiles of the first stages
//     are requested before the grid-dependency wait (the weights do not
//     depend on the previous kernel; X does), so the stream of weights starts
//     while the previous kernel finishes.
//   * Epilogue: thread t of the 128 reads TMEM lane t (weight row n0 + t)
//     and writes column n0 + t of every output row.  With K split S ways the
//     S CTAs of a tile form a thread-block cluster and share out its columns:
//     after a cluster barrier (every split's MMAs are done, so the pipeline
//     buffers are free) each writes the others' columns of its fp32 partial tile
//     into their shared memory (distributed shared memory), and after a second
//     barrier each adds up its own columns in split order and writes bf16.  No
//     global scratch, and the sum's order is fixed.
//   * With low-rank adapters (LoraTerm) the ring goes on after the K blocks with
//     the adapters' B tiles and the matching rows of h: the same MMAs with N = 16,
//     each into the columns of its 16 activation rows.  Warp 3 lists them while
//     the K blocks stream.  Only MMAs of one shape are ordered among themselves,
//     so the K blocks' sums are waited for before the first of them.
//   * Every wait is bounded; a wait that gives up reports GDN_ERR_TIMEOUT on
//     the caller's status word (when one is given) and the tile is skipped.
#include "step.cuh"

#include <cuda_bf16.h>
#include <type_traits>

namespace gdn {
namespace {

constexpr int kTileN = 128;             // weight rows per CTA (MMA M)
#ifndef GDN_GEMM_KBLK
#define GDN_GEMM_KBLK 128
#endif
constexpr int kKBlk = GDN_GEMM_KBLK;    // K columns per pipeline stage (a multiple of 64: one TMA box per 64)
constexpr int kBoxes = kKBlk / 64;      // 64-column (128-byte) boxes per operand per stage
static_assert(kKBlk % 64 == 0, "whole 128-byte boxes");
constexpr int kMaxMt = 256;             // activation rows per CTA (MMA N)
constexpr int kThreads = 128;
constexpr int kSpin = 1 << 22;          // mbarrier polls before a wait gives up
constexpr int kMaxStages = 16;

struct GemmArgs {
    CUtensorMap w_map, x_map;
    int M, N, K, Mt;                    // Mt: activation rows per CTA (multiple of 16, <= 256)
    int n_kb, kb_per_split, splits, stages;
    long long ldc;
    __nv_bfloat16 *C;
    int *d_status;
};

// A low-rank term beside the product, by the slot (T rows of X) a row belongs to (h by lora.cu): units of an aligned
// group of 16 rows, one slot's part of it and up to 64 rank columns, D[:, group] += B_tile (h_high + h_middle + h_low)^T.  They
// follow the K blocks through the same ring of stages; a stage holds several units (the B tile's box, 128 rows of
// `width` columns, then the 48 rows of h's three parts), whose swizzle is as wide as their rows: 32, 64 or 128 bytes.
struct LoraTerm {
    CUtensorMap b_map, h_map;           // [n_adapters * N][r]; [pairs * kPartRows][r]
    const int32_t *adapter;             // [slots]; outside [0, n_adapters): no term
    int n_adapters, r, T, P;            // P: groups a slot's rows may touch
    int width;                          // rank columns a unit: 16, 32 or 64
};
struct NoTerm {};
constexpr int kParts = 3, kPartRows = 16 * kParts;   // of h: bf16 numbers that add up to it
struct Unit {
    int h_row, b_row, column, box;      // column: of D
};
// the most units a block of Mt rows can have: its slots (T rows each) and the groups they cut, by 64 rank columns
__host__ __device__ constexpr int max_units(int Mt, int T, int r) {
    const int slots = (Mt + T - 1) / T + 1;
    return ((slots < Mt ? slots : Mt) + Mt / 16) * ((r + 63) / 64);
}
// rank columns a unit, and its bytes
__host__ __device__ constexpr int unit_width(int r) { return r <= 16 ? 16 : r <= 32 ? 32 : 64; }
__host__ __device__ constexpr uint32_t unit_bytes(int width) { return (uint32_t)(kTileN + kPartRows) * width * 2; }
// n units in steps of the ring: a stage's fill each, but both issuers busy
__device__ __forceinline__ int units_per_step(int n, uint32_t stage_bytes, int width) {
    const int fill = (int)(stage_bytes / unit_bytes(width));
    const int steps = max((n + fill - 1) / fill, min(n, 2));
    return steps ? (n + steps - 1) / steps : 1;
}

__device__ __forceinline__ uint32_t smem_u32(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.expect_tx.release.cta.shared::cta.b64 st, [%0], %1;\n\t}\n" ::"r"(bar),
                 "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}\n"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return ok != 0;
}
// bounded wait; false if it gave up
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity) {
    for (int i = 0; i < kSpin; ++i)
        if (mbar_try(bar, parity)) return true;
    return false;
}
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n" ::"r"(
            dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
// shared-memory matrix descriptor of a K-major tile with 128-byte rows in the 128-byte swizzle (the layout a
// SWIZZLE_128B TMA box of 64 bf16 columns leaves): 8-row groups 1024 bytes apart, the leading offset unused
// (one MMA's 16 columns lie inside a row); saddr may point 32 * j bytes into a 1024-aligned tile to select
// columns 16 j .. 16 j + 15
__device__ __forceinline__ uint64_t make_desc_sw128(uint32_t saddr) {
    uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFF);
    d |= (uint64_t)1 << 16;                                    // leading byte offset 16 (unused)
    d |= (uint64_t)(1024 >> 4) << 32;                          // stride byte offset: next 8-row group
    d |= (uint64_t)1 << 46;                                    // descriptor version (sm_100 family)
    d |= (uint64_t)2 << 61;                                    // layout: 128-byte swizzle
    return d;
}
// the same for rows of `width` bf16 columns (16, 32 or 64) in the swizzle of that width
__device__ __forceinline__ uint64_t make_desc_sw(uint32_t saddr, int width) {
    const uint64_t layout = width == 16 ? 6 : width == 32 ? 4 : 2;
    return (uint64_t)((saddr >> 4) & 0x3FFF) | (uint64_t)1 << 16 | (uint64_t)(width) << 32 | (uint64_t)1 << 46 | layout << 61;
}
// instruction descriptor: kind::f16 with bf16 A and B, fp32 D, both K-major, M = 128
__host__ __device__ constexpr uint32_t idesc_bf16(int N) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(bar)
                 : "memory");
}
// 16 fp32 columns of this thread's TMEM lane (activation rows come in multiples of 16)
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float *v) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
// the same 16 columns summed over the n accumulators (Mt columns apart), in accumulator order
__device__ __forceinline__ void tmem_ld16_sum(uint32_t taddr, int n, int Mt, float *v) {
    tmem_ld16(taddr, v);
    for (int q = 1; q < n; ++q) {
        float w[16];
        tmem_ld16(taddr + (uint32_t)(q * Mt), w);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] += w[i];
    }
}
__device__ __forceinline__ uint32_t map_cluster(uint32_t local, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(local), "r"(rank));
    return r;
}
__device__ __forceinline__ void st_cluster_f32x4(uint32_t addr, float a, float b, float c, float d) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};\n" ::"r"(addr), "f"(a), "f"(b), "f"(c), "f"(d) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void fence_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void fence_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }

// bytes of one pipeline stage: the W tile (128 rows) and the X block (Mt rows), 64 K-columns each
__host__ __device__ constexpr uint32_t w_stage_bytes() { return kTileN * kKBlk * 2; }
__host__ __device__ inline uint32_t x_stage_bytes(int Mt) { return (uint32_t)Mt * kKBlk * 2; }

// H: the parts a stage is filled and freed in (its boxes of 64 K columns shared out), each with its own barriers
template <typename Term, int H>
__global__ void __launch_bounds__(kThreads, 1) gemm_kernel(const __grid_constant__ GemmArgs a,
                                                        const __grid_constant__ Term term) {
    extern __shared__ __align__(1024) unsigned char sm[];
    // full and empty by stage and half, done (2 arrivals), units listed, each issuer's K blocks summed
    __shared__ __align__(8) uint64_t bars[2 * kMaxStages + 4];
    __shared__ uint32_t tslot;
    __shared__ int n_units;
    constexpr bool kLora = std::is_same<Term, LoraTerm>::value;
    const int tid = threadIdx.x, wid = tid >> 5;
    const int nt = blockIdx.x, mb = blockIdx.y, split = blockIdx.z;   // the splits of a tile: one cluster
    const int n0 = nt * kTileN, m0 = mb * a.Mt;
    const int kb0 = split * a.kb_per_split;
    const int kb1 = min(a.n_kb, kb0 + a.kb_per_split);
    // K blocks of this CTA; with a term both issuers' accumulators are in use, so both get one: past the split's own
    // it is one past the end of K, which reads zeros
    const int nb = kLora ? max(kb1 - kb0, 2) : kb1 - kb0;
    auto k_of = [&](int i) { return (kLora && kb0 + i >= kb1 ? a.n_kb : kb0 + i) * kKBlk; };
    const int S = a.stages;
    const uint32_t wbytes = w_stage_bytes(), xbytes = x_stage_bytes(a.Mt);
    const uint32_t stage_bytes = wbytes + xbytes;
    const uint32_t sbase = (smem_u32(sm) + 1023u) & ~1023u;   // swizzled tiles start on 1024 bytes
    constexpr int kPart = kBoxes / H;
    static_assert(kBoxes % H == 0, "whole boxes");
    auto full = [&](int s, int h = 0) { return smem_u32(&bars[s * H + h]); };
    auto empty = [&](int s, int h = 0) { return smem_u32(&bars[kMaxStages + s * H + h]); };
    const uint32_t done = smem_u32(&bars[2 * kMaxStages]), listed = smem_u32(&bars[2 * kMaxStages + 1]);
    auto summed = [&](int e) { return smem_u32(&bars[2 * kMaxStages + 2 + e]); };
    Unit *units = reinterpret_cast<Unit *>(sm + (sbase - smem_u32(sm)) + (size_t)S * stage_bytes);

    if (wid == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(&tslot)),
                     "r"(2 * kMaxMt));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
    }
    if (tid == 32) {
        for (int s = 0; s < S * H; ++s) {
            mbar_init(smem_u32(&bars[s]), 1);
            mbar_init(smem_u32(&bars[kMaxStages + s]), 1);
        }
        mbar_init(done, 2);
        mbar_init(listed, 1);
        mbar_init(summed(0), 1);
        mbar_init(summed(1), 1);
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tmem = tslot;
    bool ok = true;

    if (tid == 0) {
        // ---- producer: the weight boxes of the first stages go out before the dependency wait
        const int pre = min(S, nb);
        const uint32_t xbox = (uint32_t)a.Mt * 128;            // bytes of one X box
        for (int i = 0; i < pre; ++i) {
            const uint32_t st = sbase + (uint32_t)i * stage_bytes;
            for (int b = 0; b < kBoxes; ++b) {
                if (b % kPart == 0) mbar_expect_tx(full(i, b / kPart), stage_bytes / H);
                tma_box(st + b * 16384u, &a.w_map, k_of(i) + 64 * b, n0, full(i, b / kPart));
            }
        }
        // with adapters the kernel before is the one that computes h: it lets this one start only when X is there, and
        // the wait for h is warp 3's
        if constexpr (!kLora) asm volatile("griddepcontrol.wait;\n" ::: "memory");
        for (int i = 0; i < pre; ++i)
            for (int b = 0; b < kBoxes; ++b)
                tma_box(sbase + (uint32_t)i * stage_bytes + wbytes + b * xbox, &a.x_map, k_of(i) + 64 * b, m0,
                        full(i, b / kPart));
        for (int i = pre; i < nb && ok; ++i) {
            const int s = i % S;
            const uint32_t st = sbase + (uint32_t)s * stage_bytes;
            for (int h = 0; h < H && ok; ++h) {
                ok = mbar_wait(empty(s, h), ((i / S) - 1) & 1);       // the MMAs of stage use i - S are done
                mbar_expect_tx(full(s, h), stage_bytes / H);
                for (int b = h * kPart; b < (h + 1) * kPart; ++b)
                    tma_box(st + b * 16384u, &a.w_map, k_of(i) + 64 * b, n0, full(s, h));
                for (int b = h * kPart; b < (h + 1) * kPart; ++b)
                    tma_box(st + wbytes + b * xbox, &a.x_map, k_of(i) + 64 * b, m0, full(s, h));
            }
        }
        if constexpr (kLora) {
            ok = ok && mbar_wait(listed, 0);
            const int n = ok ? n_units : 0;
            const int per = units_per_step(n, stage_bytes, term.width);
            const uint32_t ub = unit_bytes(term.width), hb = (uint32_t)kTileN * term.width * 2;
            for (int i = nb, u0 = 0; u0 < n && ok; ++i, u0 += per) {
                const int s = i % S, un = min(per, n - u0);
                for (int h = 0; h < H; ++h)                          // units take the stage whole
                    if (i >= S) ok = ok && mbar_wait(empty(s, h), ((i / S) - 1) & 1);
                const uint32_t st = sbase + (uint32_t)s * stage_bytes;
                for (int h = 1; h < H; ++h) mbar_expect_tx(full(s, h), 0);
                mbar_expect_tx(full(s), (uint32_t)un * ub);
                for (int u = 0; u < un; ++u) {
                    const Unit q = units[u0 + u];
                    tma_box(st + (uint32_t)u * ub, &term.b_map, 64 * q.box, q.b_row, full(s));
                    tma_box(st + (uint32_t)u * ub + hb, &term.h_map, 64 * q.box, q.h_row, full(s));
                }
            }
        }
    } else if (tid == 32 || tid == 64) {
        // ---- MMA issuers: the even or the odd stages of the ring into accumulator e (8 MMAs of K = 16 per stage);
        // each stage is freed when its MMAs complete.  A stage always has the same issuer, which has then seen
        // every earlier use of it complete: with the K blocks dealt out by their own parity, a ring of an odd
        // number of stages would hand a stage from one issuer to the other and back, and a wait for its use u + 2
        // could take the phase of use u (the same parity) for it while the load of use u + 1 is still in flight
        const int e = wid - 1;
        const uint32_t acc = tmem + (uint32_t)(e * a.Mt);
        const uint32_t id = idesc_bf16(a.Mt);
        for (int i = e; i < nb && ok; ++i) {
            const int s = i % S;
            if ((s & 1) != e) continue;
            const uint32_t st = sbase + (uint32_t)s * stage_bytes;
            for (int h = 0; h < H; ++h) {
                ok = ok && mbar_wait(full(s, h), (i / S) & 1);
                fence_after_sync();
#pragma unroll
                for (int j = 0; j < kKBlk / 16; ++j) {          // 16 columns (32 bytes of each row) per MMA
                    const uint32_t b = j >> 2, c = 32u * (j & 3);
                    if ((int)b / kPart == h)
                        mma_bf16(acc, make_desc_sw128(st + b * 16384u + c),
                                 make_desc_sw128(st + wbytes + b * (uint32_t)a.Mt * 128u + c), id, (i > e || j > 0) ? 1u : 0u);
                }
                mma_commit(empty(s, h));
            }
        }
        if constexpr (kLora) {
            ok = ok && mbar_wait(listed, 0);
            const int n = ok ? n_units : 0;
            const int per = units_per_step(n, stage_bytes, term.width);
            const uint32_t ub = unit_bytes(term.width), hb = (uint32_t)kTileN * term.width * 2, part = 32u * term.width;
            // MMAs into the same accumulator follow one another in order only if their shapes are the same: before those
            // of N = 16 the K blocks' (of N = Mt) have to be complete.  The units' tiles are on their way meanwhile.
            if (n > 0 && a.Mt != 16) {
                mma_commit(summed(e));
                ok = ok && mbar_wait(summed(e), 0);
                fence_after_sync();
            }
            for (int i = nb, u0 = 0; u0 < n && ok; ++i, u0 += per) {
                const int s = i % S, un = min(per, n - u0);
                if ((s & 1) != e) continue;
                for (int h = 0; h < H; ++h) ok = ok && mbar_wait(full(s, h), (i / S) & 1);
                fence_after_sync();
                for (int u = 0; u < un; ++u) {
                    const Unit q = units[u0 + u];
                    const uint32_t b = sbase + (uint32_t)s * stage_bytes + (uint32_t)u * ub, h = b + hb;
                    const int steps = (min(64, term.r - 64 * q.box) + 15) / 16;
                    for (int j = 0; j < steps; ++j) {
                        const uint64_t bd = make_desc_sw(b + 32u * j, term.width);
#pragma unroll
                        for (int p = 0; p < kParts; ++p)
                            mma_bf16(acc + q.column, bd, make_desc_sw(h + p * part + 32u * j, term.width), idesc_bf16(16), 1u);
                    }
                }
                for (int h = 0; h < H; ++h) mma_commit(empty(s, h));
            }
        }
        mma_commit(done);
    } else if (kLora && wid == 3) {
        // ---- the units of this block and split, in slot order
        if constexpr (kLora) {
            asm volatile("griddepcontrol.wait;\n" ::: "memory");
            const int lane = tid & 31, rows = min(a.M, m0 + a.Mt), s0 = m0 / term.T, s1 = (rows - 1) / term.T;
            const int boxes = (term.r + 63) / 64;
            int n = 0;                                   // of all splits
            for (int sb = s0; sb <= s1; sb += 32) {
                const int s = sb + lane, id = s <= s1 ? term.adapter[s] : -1;
                const int first = s * term.T / 16;       // the slot's first group
                const int g0 = max(first, m0 / 16), g1 = min(((s + 1) * term.T - 1) / 16, (rows - 1) / 16);
                const int mine = id >= 0 && id < term.n_adapters ? (g1 - g0 + 1) * boxes : 0;
                int to = mine;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int o = __shfl_up_sync(0xffffffffu, to, d);
                    if (lane >= d) to += o;
                }
                for (int q = 0; q < mine; ++q) {
                    const int at = n + to - mine + q, g = g0 + q / boxes;
                    if (at % a.splits != split) continue;
                    const Unit u{(s * term.P + g - first) * kPartRows, id * a.N + n0, g * 16 - m0, q % boxes};
                    units[at / a.splits] = u;
                    // its B tile comes at the end of the ring: into L2 by then
                    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];\n" ::"l"(
                                     reinterpret_cast<uint64_t>(&term.b_map)),
                                 "r"(64 * u.box), "r"(u.b_row)
                                 : "memory");
                }
                n += __shfl_sync(0xffffffffu, to, 31);
            }
            if (lane == 0) n_units = (n - split + a.splits - 1) / a.splits;
            __syncwarp();
            if (lane == 0) asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.release.cta.shared::cta.b64 st, [%0];\n\t}\n" ::"r"(listed) : "memory");
        }
    }
    __syncwarp();
    // ---- epilogue: the accumulator of weight row n0 + tid, every activation row of the block
    const bool got = mbar_wait(done, 0);
    fence_after_sync();
    // one verdict for the whole CTA (the collective TMEM loads below need every lane of a warp)
    const bool good = __syncthreads_and(got && ok) != 0;
    if (!good && tid == 0 && a.d_status) atomicCAS(a.d_status, int(GDN_OK), int(GDN_ERR_TIMEOUT));
    const int n_acc = nb > 1 ? 2 : 1;                 // the odd stages' accumulator holds a sum only if used
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
    const int n = n0 + tid;
    const uint32_t taddr = tmem + ((uint32_t)(32 * wid) << 16);
    if (a.splits == 1) {
        if (good)
            for (int c0 = 0; c0 < a.Mt; c0 += 16) {
                float v[16];
                tmem_ld16_sum(taddr + c0, n_acc, a.Mt, v);
                if (n < a.N)
#pragma unroll
                    for (int q = 0; q < 16; ++q) {
                        const int m = m0 + c0 + q;
                        if (m < a.M) a.C[(size_t)m * a.ldc + n] = __float2bfloat16_rn(v[q]);
                    }
            }
    } else {
        // The splits share out the 16-column chunks (chunk c is split c % splits's): each sends the others' chunks of its
        // partial tile to their owners, as [sender][four columns][row][4], and adds up its own in split order.
        // (One owner for all and scalar stores took 0.17 us a column: 36 us for 128 rows of the output projection.)
        constexpr uint32_t kChunk = 16 * kTileN * 4;
        cluster_sync();                            // every split's MMAs are done: the pipeline buffers are free
        for (int c = 0; 16 * c < a.Mt; ++c) {
            const int owner = c % a.splits;
            if (owner == split) continue;
            float v[16];
            tmem_ld16_sum(taddr + 16 * c, n_acc, a.Mt, v);
            const int from = split < owner ? split : split - 1;
            const uint32_t dst = map_cluster(sbase, owner) + (uint32_t)((c / a.splits) * (a.splits - 1) + from) * kChunk + tid * 16u;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float *p = v + 4 * q;
                st_cluster_f32x4(dst + (uint32_t)q * kTileN * 16u, good ? p[0] : 0.f, good ? p[1] : 0.f, good ? p[2] : 0.f,
                                 good ? p[3] : 0.f);
            }
        }
        cluster_sync();                            // every partial has landed
        if (good)
            for (int c = split; 16 * c < a.Mt; c += a.splits) {
                float v[16], acc[16];
                tmem_ld16_sum(taddr + 16 * c, n_acc, a.Mt, v);
                const float4 *red = reinterpret_cast<const float4 *>(sm + (sbase - smem_u32(sm)) +
                                                                     (size_t)(c / a.splits) * (a.splits - 1) * kChunk) + tid;
                for (int sp = 0; sp < a.splits; ++sp) {
                    const int from = sp < split ? sp : sp - 1;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float4 w = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                        if (sp != split) w = red[(size_t)from * (kChunk / 16) + q * kTileN];
                        acc[4 * q] = sp ? acc[4 * q] + w.x : w.x;
                        acc[4 * q + 1] = sp ? acc[4 * q + 1] + w.y : w.y;
                        acc[4 * q + 2] = sp ? acc[4 * q + 2] + w.z : w.z;
                        acc[4 * q + 3] = sp ? acc[4 * q + 3] + w.w : w.w;
                    }
                }
                if (n < a.N)
#pragma unroll
                    for (int q = 0; q < 16; ++q) {
                        const int m = m0 + 16 * c + q;
                        if (m < a.M) a.C[(size_t)m * a.ldc + n] = __float2bfloat16_rn(acc[q]);
                    }
            }
    }
    fence_before_sync();
    __syncthreads();
    if (wid == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(2 * kMaxMt));
}

}  // namespace

// K splits of a tile: enough CTAs to cover the SMs when the output tiles are few, while the other splits' partial tiles
// would fit the pipeline buffers of one CTA (what its share of the columns takes of them is less)
static int gemm_splits(int n_tiles, int m_blocks, int n_kb, int Mt, size_t smem, int sms) {
    int splits = (int)(sms / ((long long)n_tiles * m_blocks));
    if (splits > 8) splits = 8;
    if (splits > n_kb) splits = n_kb;
    while (splits > 1 && (size_t)(splits - 1) * Mt * kTileN * 4 > smem) --splits;
    return splits < 1 ? 1 : splits;
}

constexpr uint32_t kRingBytes = 216u * 1024u;   // pipeline stages of a CTA
// with 1024 bytes to align the tiles by, and the longest list of units (256 rows, a slot each, rank 128)
template <typename Term> constexpr size_t max_smem() {
    return kRingBytes + 1024 + (std::is_same<Term, LoraTerm>::value ? max_units(kMaxMt, 1, 128) * sizeof(Unit) : 0);
}

// The kernel's shared memory limit, which belongs to the context: set once in each, to the most that any launch asks for.
// (Set to each launch's own size, one host thread's launch could meet the smaller limit of another's.)
template <typename Term, int H> static cudaError_t raise_smem_limit() {
    static PerContext<int> limits;
    unsigned long long ctx = 0;
    int set = 0;
    if (current_context_id(&ctx) && limits.get(ctx, &set)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(gemm_kernel<Term, H>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)max_smem<Term>());
    if (e == cudaSuccess && current_context_id(&ctx)) limits.put(ctx, 1);
    return e;
}

// before(): what goes on the stream ahead of the kernel, once nothing but the launches themselves can fail
template <typename Term, typename Before>
static bool gemm_launch(const void *W, const void *X, void *C, int M, int N, int K, long long ldc, Term &term,
                        int *d_status, cudaStream_t stream, std::string &why, Before before) {
    constexpr bool kLora = std::is_same<Term, LoraTerm>::value;
    PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (!encode) {
        why = "the driver's tensor-map encoder is unavailable";
        return false;
    }
    if (K % 8 || K < 8) {
        why = "K must be a positive multiple of 8";
        return false;
    }
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) !=
                                                   cudaSuccess) {
        why = "no usable CUDA device";
        return false;
    }
    GemmArgs a{};
    a.M = M; a.N = N; a.K = K; a.ldc = ldc;
    a.Mt = M >= kMaxMt ? kMaxMt : ((M + 15) / 16) * 16;
    const int m_blocks = (M + a.Mt - 1) / a.Mt;
    const int n_tiles = (N + kTileN - 1) / kTileN;
    a.n_kb = (K + kKBlk - 1) / kKBlk;
    const uint32_t stage = w_stage_bytes() + x_stage_bytes(a.Mt);
    // as many stages as fit in ~216 KB: a stage is held until its MMAs complete, so the bytes in flight per
    // SM set the intake (six 36 KB stages: output projection 14.6 us against 14.9 with five; two CTAs per SM
    // with 100 KB each, the K splits spread over every SM, measured slower: 26 us)
    a.stages = (int)(kRingBytes / stage);
    if (a.stages > kMaxStages) a.stages = kMaxStages;
    if (a.stages < 2) {                                           // one for each MMA issuer
        why = "pipeline stage larger than shared memory";
        return false;
    }
    // a ring of two stages (more than 160 activation rows) moves by halves, so that three of its four are in flight
    // while one feeds the MMAs
    const bool halves = a.stages == 2;
    auto kern = halves ? gemm_kernel<Term, kBoxes> : gemm_kernel<Term, 1>;
    size_t smem = (size_t)a.stages * stage + 1024;                // + room to align the tiles to 1024 bytes
    const int splits = gemm_splits(n_tiles, m_blocks, a.n_kb, a.Mt, smem - 1024, sms);
    if constexpr (kLora) {
        smem += (size_t)max_units(a.Mt, term.T, term.r) * sizeof(Unit);
    }
    a.kb_per_split = (a.n_kb + splits - 1) / splits;
    a.splits = (a.n_kb + a.kb_per_split - 1) / a.kb_per_split;
    a.C = static_cast<__nv_bfloat16 *>(C);
    a.d_status = d_status;
    // tensor maps: 64-column (128-byte) boxes in the 128-byte swizzle
    const cuuint32_t estr[2] = {1, 1};
    {
        const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)N};
        const cuuint64_t strides[1] = {(cuuint64_t)K * 2};
        const cuuint32_t box[2] = {64u, (cuuint32_t)kTileN};
        if (encode(&a.w_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(W), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS) {
            why = "weight tensor map";
            return false;
        }
    }
    {
        const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)M};
        const cuuint64_t strides[1] = {(cuuint64_t)K * 2};
        const cuuint32_t box[2] = {64u, (cuuint32_t)a.Mt};
        if (encode(&a.x_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(X), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS) {
            why = "activation tensor map";
            return false;
        }
    }
    cudaError_t e = halves ? raise_smem_limit<Term, kBoxes>() : raise_smem_limit<Term, 1>();
    if (e == cudaSuccess) e = before();
    if (e == cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(n_tiles, m_blocks, a.splits);
        cfg.blockDim = dim3(kThreads, 1, 1);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = 1;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = a.splits;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        e = cudaLaunchKernelEx(&cfg, kern, a, term);
    }
    if (e != cudaSuccess) {
        why = std::string("projection GEMM launch: ") + cudaGetErrorString(e);
        return false;
    }
    return true;
}

bool gemm_xwt_bf16(const void *W, const void *X, void *C, int M, int N, int K, long long ldc, int *d_status,
                   cudaStream_t stream, std::string &why) {
    NoTerm none;
    return gemm_launch(W, X, C, M, N, K, ldc, none, d_status, stream, why, [] { return cudaSuccess; });
}

bool gemm_xwt_lora_bf16(const void *W, const void *X, void *C, int M, int N, int K, long long ldc, const LoraArgs &lora,
                        int sms, int *d_status, cudaStream_t stream, std::string &why) {
    PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (!encode) {
        why = "the driver's tensor-map encoder is unavailable";
        return false;
    }
    LoraTerm term{};
    term.adapter = lora.adapter;
    term.n_adapters = lora.n_adapters; term.r = lora.rank; term.T = lora.T;
    term.P = lora_groups_per_slot(lora.T);
    term.width = unit_width(lora.rank);
    const CUtensorMapSwizzle swizzle = term.width == 16   ? CU_TENSOR_MAP_SWIZZLE_32B
                                       : term.width == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                          : CU_TENSOR_MAP_SWIZZLE_128B;
    // boxes of `width` columns: 128 rows of B, the rows of a pair's three parts of h
    const cuuint32_t estr[2] = {1, 1};
    auto map = [&](CUtensorMap *m, const void *p, cuuint64_t rows, cuuint32_t box_rows) {
        const cuuint64_t dims[2] = {(cuuint64_t)lora.rank, rows};
        const cuuint64_t strides[1] = {(cuuint64_t)lora.rank * 2};
        const cuuint32_t box[2] = {(cuuint32_t)term.width, box_rows};
        return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(p), dims, strides, box, estr,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    if (!map(&term.b_map, lora.b, (cuuint64_t)lora.n_adapters * N, kTileN) ||
        !map(&term.h_map, lora.h, (cuuint64_t)(M / lora.T) * term.P * kPartRows, kPartRows)) {
        why = "adapter tensor map";
        return false;
    }
    return gemm_launch(W, X, C, M, N, K, ldc, term, d_status, stream, why,
                       [&] { return launch_lora_shrink(X, M, K, lora, sms, d_status, stream); });
}

}  // namespace gdn
