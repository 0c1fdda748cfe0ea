// attend.cu -- attention of a batch of new tokens over a paged cache, bf16, on the tensor cores.
//
// Rows: the G query heads that share a kv head times a block's tokens, 128 to a tile (a chain's verify of 16 tokens with
// G = 6 fills 96), so that a key and a value are read once for all of them.  Per tile of 128 keys
//   S = Q K^T            (128 x 128, fp32 in tensor memory)
//   P = 2^(S scale log2 e - m)   rounded to bf16, in place of S; the row sums stay fp32
//   O += P V             (128 x D, fp32 in tensor memory)
// with the running maximum m: one pass over the cache (Milakov and Gimelshein, Online normalizer calculation for softmax,
// 2018).  m is only moved (and O rescaled) when it has grown by more than 2^8, a known variant of it: weights reach 2^8 and the
// rescale is rare.  The rounding of P to bf16 (half a step, 2^-8, of each weight) is what the tensor cores take, and of the
// order of the output's own rounding.  The row sums, in fp32, are of the rounded weights: so an output is a mean of the values
// that its row sees, and a row of equal values comes out as that value.  (A sum of the weights before their rounding left it off by
// up to 2^-8; it saves an instruction a pair of weights: 428 us for the prompt below against 442, and 1 % elsewhere at most.)
//
//   * A warp (two for D = 64) streams keys and values through a ring of 16 or 32 KB stages: one TMA box a page, straight into
//     the tensor cores' 128-byte swizzle.  A page's tokens come in groups of 8 (a swizzle atom's rows), all 64-column chunks of a group
//     side by side, so that boxes of any page size leave the same layout: group stride (D / 64) KB, chunk stride 1 KB.  It is
//     K-major for K (8-row groups by the stride offset) and, read the other way, MN-major for V.
//   * Two warps issue the MMAs, one those of S and one those of P V; S has as many buffers as tensor memory holds beside O
//     (three, or two for D = 256), so that the next S is made while this one's softmax runs.  (Two row tiles a CTA, each with
//     its own S, O and softmax warps, halve what the keys and values cost in shared memory, but ran slower: the chains
//     of one tile's S, softmax and P V are what binds, and two of them took 4950 cycles where a single one takes 2200.)
//   * Two threads do the softmax of a row (tensor memory's lane), half of the keys each, and exchange their maxima: S, softmax
//     and P V of a tile follow one another, so its time counts (4096 tokens of 32 + 8 heads of 128 over 8192 positions: 342 us, with
//     one thread a row 356; 8 trees of 64: 42 and 46).  Where a slot has at most 32 rows they lie there four times instead, and each copy's warp takes a quarter of
//     every tile's keys (its other weights are zeros); the four sums are added up at the end (64 slots of 2 tokens in a
//     window of 1024: 41 us, with one copy of the rows 52; one token behind 1001 positions: 10.8 and 13.5).
//   * The work is dealt out by tiles (attn.cuh): every CTA has the same number whatever the lengths, and the blocks of rows
//     at the ends of its share are joined with its neighbours' parts by attend_join.cu.
//
// Positions that no row of the block sees are not loaded by whole pages, and their rows of V are cleared in shared memory
// before the MMA (0 x NaN would be NaN); scores that a row may not see are replaced, whatever was there.
//
// What bounds it.  Few rows: the cache's bytes (4 single tokens behind 131000 positions, D = 128: 298 us, 7.2 TB/s; 32 slots of 16
// tokens over up to 16384, D = 256: 182 us, 6.1 TB/s).  Many rows: shared memory, which a tile of D = 256 asks for 320 KB (the
// loads write 128, S reads Q and K, 128, P V reads V, 64), 2500 cycles at 128 bytes each, where its MMAs take 2048 (4096 tokens over
// 8192 positions: 442 us in a captured graph, 1400 TFLOP/s).  Few keys: latency -- a launch, dependent loads of lengths, page ids and pages, one tile's S, softmax and
// P V, and instructions that come from L2 the first time.
//
// Every wait is bounded; one that gives up reports GDN_ERR_TIMEOUT and the CTA ends.
#include "attn.cuh"

#include <cuda_bf16.h>

namespace gdn {
namespace {

constexpr int kTile = kTileBf16;
constexpr int kLanes = 128;           // tensor memory's: rows of a block
constexpr int kSpin = 1 << 20;        // mbarrier polls before a wait gives up
constexpr float kSlack = 8.f;         // powers of two by which a maximum may grow unmoved

// C: copies of the rows, 128 / C of them, side by side in tensor memory; copy i takes the i-th C-th of every tile's keys.
template <int D, int C> struct Shape {
    static constexpr int kChunks = D / 64;                         // 128-byte columns of a row
    static constexpr int kStage = D == 64 ? 16384 : 32768;         // bytes
    static constexpr int kKChunks = kChunks < 2 ? kChunks : 2;     // of K in a stage: 128 keys x 64 kKChunks
    static constexpr int kKStages = kChunks / kKChunks;
    static constexpr int kVTokens = kStage / (2 * D);              // of V in a stage: kVTokens keys x D
    static constexpr int kVStages = kTile / kVTokens;
    static constexpr int kQTile = kLanes * D * 2;
    static constexpr int kQBuffers = D == 64 ? 2 : 1;   // where there is room, the next block's Q comes early
    static constexpr int kQBytes = kQBuffers * kQTile;
    static constexpr int kRing = (224 * 1024 - kQBytes) / kStage < 12 ? (224 * 1024 - kQBytes) / kStage : 12;
    static constexpr int kBuffers = D == 256 ? 2 : 3;              // of S, in tensor memory beside O
    static constexpr int kOColumn = 128 * 2;                       // O, between the second S and the third
    // a ring that reaches back past the tile whose S buffer this one's is, even if a block ends with each
    static constexpr bool kLongRing = kRing >= kBuffers * (kKStages + kVStages + 2);
    static constexpr int kRows = kLanes / C;                       // of a block
    // Without copies two threads share a row, each with half of a tile's keys (and of O where it is moved).
    static constexpr int kShare = C == 1 ? 2 : 1;
    static constexpr int kKeys = kTile / (C * kShare);             // of a tile that a thread takes
    static constexpr int kSoftmax = kShare * kLanes;               // threads
    // Warps that load.  A tile of D = 64 is only 32 KB, and one warp takes 1200 cycles to send off its boxes of pages of 32 tokens:
    // there one takes the keys and one the values (64 slots of 2 tokens in a window of 1024: 41.4 us against 43.1).  Larger
    // heads' tiles take longer to come than to send for, and one warp does (8 trees of 64 tokens, D = 128: 42.5 us against 43.7).
    static constexpr int kLoaders = D == 64 ? 2 : 1;
    static constexpr int kLoads = kSoftmax / 32, kMmas = kLoads + kLoaders;   // the first warps of loads and MMAs
    static constexpr int kThreads = kSoftmax + 32 * kLoaders + 64;
    // a row's sums on their way out: two stages are shared out among the softmax threads
    static constexpr int kOut = 2 * kStage / kLanes;
    static_assert(kRing >= 5, "a tile's V, the next one's K, and one more");
};

// What a CTA keeps beside its tiles, behind them.
template <int RING, int THREADS> struct Control {
    uint64_t full[RING], empty[RING];
    uint64_t q_full[2], q_empty[2];
    uint64_t s_full[3], p_full[3];    // S is there; P is there
    uint64_t o_done[3];               // P V is done: O is whole so far, the buffer free
    uint64_t o_free;                  // O has been read out
    int scratch[THREADS / 32 + 2];
    uint32_t tmem;
    union {                           // of a row:
        float2 stats[kLanes];         // maximum and sum, by copy
        float each[2][kLanes];        // each thread's maximum of a tile, at the end its sum
    };
    int parents[64];
    unsigned char depths[64];
};

struct TcArgs {
    CUtensorMap q_map, k_map, v_map;
    AttendArgs a;
};

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.expect_tx.release.cta.shared::cta.b64 st, [%0], %1;\n\t}\n" ::"r"(bar),
                 "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.release.cta.shared::cta.b64 st, [%0];\n\t}\n" ::"r"(bar) : "memory");
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
// The same by a whole warp, with one answer for all its lanes.  The first look stands by itself: mostly the phase is over by
// then, and the warp goes on without having entered a loop that its lanes could leave one by one (434 us against 474 for a
// prompt of 4096 tokens with 24 heads of 256; as one loop of votes, 465).
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
    if (__all_sync(0xffffffffu, mbar_try(bar, parity))) return true;
    return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ void tma_box5(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, int c3, int c4, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];\n" ::
            "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
// shared-memory matrix descriptor in the 128-byte swizzle, atoms of 8 rows x 128 bytes.  K-major: `stride` from one
// 8-row group to the next (one MMA's 16 columns lie inside a row; lead unused).  MN-major: `lead` from one 64-column chunk
// to the next, `stride` from one group of 8 k to the next.
__device__ __forceinline__ uint64_t make_desc(uint32_t saddr, uint32_t lead, uint32_t stride) {
    return (uint64_t)((saddr >> 4) & 0x3FFF) | (uint64_t)(lead >> 4) << 16 | (uint64_t)(stride >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)2 << 61;
}
// instruction descriptor: kind::f16, bf16 A and B, fp32 D, M = 128, A K-major, B K-major or MN-major
__host__ __device__ constexpr uint32_t idesc(int N, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
constexpr uint32_t kNegateA = 1u << 13;   // takes -A: a maximum of scores stays one of S under a negative scale
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
                 "l"(a), "l"(b), "r"(id), "r"(acc)
                 : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
                 "r"(a), "l"(b), "r"(id), "r"(acc)
                 : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

#define GDN_R32(r) \
    "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), \
    "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), \
    "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), \
    "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
#define GDN_I32(r) \
    "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), \
    "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), \
    "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), \
    "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
// 32 columns of this thread's tensor-memory lane (wait_ld / wait_st before the registers or the columns are used)
__device__ __forceinline__ void tmem_ld32(uint32_t at, uint32_t *r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
                 "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
                 : GDN_R32(r)
                 : "r"(at));
}
__device__ __forceinline__ void tmem_st32(uint32_t at, const uint32_t *r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,"
                 "%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};\n" ::GDN_I32(r),
                 "r"(at)
                 : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t *r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};\n" ::
                     "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
                     "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(at)
                 : "memory");
}
// the softmax warps
template <int THREADS> __device__ __forceinline__ void softmax_sync() { asm volatile("bar.sync 1, %0;\n" ::"n"(THREADS) : "memory"); }
template <int THREADS> __device__ __forceinline__ bool softmax_all(bool ok) {
    int r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbar.red.and.pred q, 1, %2, p;\n\tselp.b32 %0, 1, 0, q;\n\t}\n" :
                     "=r"(r) : "r"((int)ok), "n"(THREADS) : "memory");
    return r != 0;
}
// the two warps that share 32 rows
__device__ __forceinline__ void rows_sync(int warp) { asm volatile("bar.sync %0, 64;\n" ::"r"(2 + (warp & 3)) : "memory"); }
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// pairs of fp32 in one instruction
__device__ __forceinline__ uint64_t pair2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 split2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;\n" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// each of a pair of bf16 to an fp32 sum
__device__ __forceinline__ void add_pair(float &a, float &b, uint32_t p) {
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tadd.rn.f32.bf16 %0, lo, %0;\n\tadd.rn.f32.bf16 %1, hi, %1;\n\t}\n"
        : "+f"(a), "+f"(b)
        : "r"(p));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// bits [0, n) of a word, n any int
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

// A place in a ring of N stages (of keys and values, or S buffers): the stage, and how often the ring has gone round.
template <int N> struct Ring {
    uint32_t stage = 0, round = 0;
    __device__ __forceinline__ void next(int n = 1) {
        stage += n;
        if (stage >= N) {
            stage -= N;
            ++round;
        }
    }
    __device__ __forceinline__ Ring after(int n) const {
        Ring x = *this;
        x.next(n);
        return x;
    }
};

// A CTA's blocks of rows, one after the other: each role walks them by itself.
struct Walk {
    int left, pair, kvh, j0, j1;
    Span span;
    bool first, whole;
    // a block of one tile, of no slot
    __device__ __forceinline__ void none() {
        span = Span{0, 0, 1 << 20, 0, kTile, 0, 0, 1};
        left = j1 = 1;
        pair = kvh = j0 = 0;
        first = whole = true;
    }
    // the first block with tiles of a share of `tiles` tiles; false if there is none
    __device__ __forceinline__ bool begin(const AttendArgs &a, const Place &at, int tiles) {
        left = tiles;
        pair = at.pair;
        first = true;
        span = block_span<kTile>(a, pair / a.n_tb, pair % a.n_tb);
        kvh = at.offset / (span.n + a.pad);
        return cut(a, at.offset % (span.n + a.pad));
    }
    // from the block's tile `from`, the first a.pad of which are not there
    __device__ __forceinline__ bool cut(const AttendArgs &a, int from) {
        const int to = min(span.n + a.pad, from + left);
        left -= to - from;
        j0 = max(0, from - a.pad);
        j1 = max(0, to - a.pad);
        whole = j0 == 0 && j1 == span.n;
        return j1 > j0;
    }
    __device__ __forceinline__ bool next(const AttendArgs &a) {
        first = false;
        if (left <= 0) return false;
        if (++kvh == a.Hk) {
            kvh = 0;
            do {
                if (++pair == a.B * a.n_tb) return false;      // never, unless the lengths change under the call
                span = block_span<kTile>(a, pair / a.n_tb, pair % a.n_tb);
            } while (span.n == 0);
        }
        return cut(a, 0);
    }
};

template <int D, int C>
__global__ void __launch_bounds__((Shape<D, C>::kThreads), 1) attend_tc_kernel(const __grid_constant__ TcArgs args) {
    using Sh = Shape<D, C>;
    constexpr int kThreads = Sh::kThreads;
    using Ctl = Control<Sh::kRing, kThreads>;
    extern __shared__ __align__(1024) unsigned char sm[];         // no other shared memory, so that it starts at a swizzle atom
    Ctl &ctl = *reinterpret_cast<Ctl *>(sm + Sh::kQBytes + Sh::kRing * Sh::kStage);
    const AttendArgs &a = args.a;
    const int tid = threadIdx.x, wid = tid >> 5, lane = tid & 31, c = blockIdx.x;
    const uint32_t qbase = smem_u32(sm), ring = qbase + Sh::kQBytes;
    auto full = [&](uint32_t s) { return smem_u32(&ctl.full[s]); };
    auto empty = [&](uint32_t s) { return smem_u32(&ctl.empty[s]); };
    auto q_full = [&](int b) { return smem_u32(&ctl.q_full[b]); };
    auto q_empty = [&](int b) { return smem_u32(&ctl.q_empty[b]); };
    auto s_full = [&](int b) { return smem_u32(&ctl.s_full[b]); };
    auto p_full = [&](int b) { return smem_u32(&ctl.p_full[b]); };
    auto o_done = [&](int b) { return smem_u32(&ctl.o_done[b]); };
    const uint32_t o_free = smem_u32(&ctl.o_free);

    auto chk = [&](const void *p, size_t bytes, const void *base, size_t extent) { return in_bounds(p, bytes, base, extent, a.d_status); };

    if (wid == Sh::kMmas) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(smem_u32(&ctl.tmem)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n");
    } else if (wid == Sh::kLoads) {
        if (lane < Sh::kRing) {
            mbar_init(full(lane), Sh::kLoaders);
            mbar_init(empty(lane), 2);            // by both MMA warps
        }
        if (lane < 3) {
            mbar_init(s_full(lane), 1);
            mbar_init(p_full(lane), Sh::kLoads);      // a warp's lanes arrive together
            mbar_init(o_done(lane), 1);
        }
        if (lane < 2) {
            mbar_init(q_full(lane), 1);
            mbar_init(q_empty(lane), 1);
            if (lane) mbar_init(o_free, Sh::kLoads);
        }
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
        if (lane < 3) prefetch_map(lane == 0 ? &args.q_map : lane == 1 ? &args.k_map : &args.v_map);
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = ctl.tmem;
    bool ok = true;
    // What comes before the wait for the kernel ahead runs beside its end: for the softmax warps a dry pass through their
    // loop.  (Where the whole CTA looks for its work together there is none.)
    const bool together = a.B * a.n_tb > kScanPairs;
    Share share;
    Place at{0, 0};
    auto begin = [&] {
        asm volatile("griddepcontrol.wait;\n" ::: "memory");
        asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
        if (together) return;
        at = warp_place<kTile>(a, c, share);
    };
    if (together) {
        begin();
        at = find_place<kTile, kThreads>(a, c, share, ctl.scratch);
    }
    {
        if (wid < Sh::kLoads) {
            // ---- the softmax: tensor memory's lane = row (of one of C copies), a thread or two for each
            const int tl = tid % kLanes, half = tid / kLanes, copy = tl / Sh::kRows, row = tl % Sh::kRows;
            const uint32_t lanes = tmem + ((uint32_t)(32 * (wid & 3)) << 16), o_at = lanes + Sh::kOColumn;
            // (a negative scale's sign is in S: see the MMAs)  A scale of zero leaves all weights alike, and masked ones at none: it is
            // the smallest number, which brings no score to anything and leaves an infinity one
            const float sc = fmaxf(fabsf(a.scale) * 1.4426950408889634f, __uint_as_float(1u));
            Ring<Sh::kBuffers> u, before;         // this tile's S, and the tile's before it
            bool any = false;                     // was there one?
            Ring<Sh::kRing> r;                    // the first stage of this tile
            int last_pair = -1;
            unsigned long long line = 0;          // a tree's nodes that this row sees
            int position = 0;
            Walk w;
            // A launch starts with a cold instruction cache: the first pass through this loop takes 4000 cycles and more where
            // the next ones take 1400.  So it is a dry one, on a block of one tile that is not there, over whatever tensor
            // memory holds; it writes into O, which the first P V overwrites.
            bool dry = !together;
            if (dry) w.none();
            if (dry || (c < share.ctas && w.begin(a, at, share.start(c + 1) - share.start(c))))
            do {
                const int s = w.pair / a.n_tb, past = w.span.past, n = w.j1 - w.j0;
                const int first_t = w.span.t0, last_t = w.span.t1 - 1;
                const int t = row < a.TB * a.G ? first_t + row / a.G : w.span.t1;
                const bool on = t < w.span.t1;
                const bool busy = __any_sync(kWarp, on);
                if (w.pair != last_pair && !dry) {
                    last_pair = w.pair;
                    position = past + t;
                    if (a.parent) {
                        softmax_sync<Sh::kSoftmax>();
                        if (half == 0 && tl < w.span.t1)
                            ctl.parents[tl] = parent_of(a.parent, a.T, s, tl, a.ext_nodes, a.d_status, true);
                        softmax_sync<Sh::kSoftmax>();
                        if (half == 0 && tl < w.span.t1) {
                            int d = 0;
                            for (int p = ctl.parents[tl]; p >= 0; p = ctl.parents[p]) ++d;
                            ctl.depths[tl] = (unsigned char)d;
                        }
                        softmax_sync<Sh::kSoftmax>();
                        line = 0;
                        if (on) {
                            const int mine = ctl.depths[t];
                            position = past + mine;
                            for (int p = t; p >= 0; p = ctl.parents[p]) {
                                const int d = ctl.depths[p];
                                if (!a.window || mine - d < a.window || past + d < a.n_sink) line |= 1ull << p;
                            }
                        }
                    }
                }
                const int lim = a.parent ? past : position + 1;   // positions below: by the rule of a chain
                const int low = a.window ? position - a.window + 1 : 0;
                const int sink = min(a.n_sink, w.span.lo);
                float m = -INFINITY, l = 0.f;
                for (int q = 0; q < n; ++q) {
                    const uint32_t s_column = u.stage * 128 + (u.stage == 2 ? 128 : 0);
                    const int k0 = w.span.tile(w.j0 + q) * kTile, mine = (copy + half) * Sh::kKeys, mine0 = k0 + mine;
                    if (!dry) ok = ok && warp_wait(s_full(u.stage), u.round & 1);
                    // (after a wait that gave up all go on without waiting, as the barriers among them want, and leave together)
                    fence_after();
                    // O is whole up to the tile before
                    auto wait_o = [&] { return warp_wait(o_done(before.stage), before.round & 1); };
                    if (busy) {
                        const uint32_t s_at = lanes + s_column + mine, p_at = dry ? o_at : lanes + s_column;
                        uint32_t x[Sh::kKeys];
#pragma unroll
                        for (int e = 0; e < Sh::kKeys; e += 32) tmem_ld32(s_at + e, x + e);
                        wait_ld();
                        // The other copies' keys.  P takes the place of S, and a load and a store of tensor memory come in no order but
                        // by a wait: not before the scores are here.
                        if (C > 1) {
                            const uint32_t zero[16] = {};
#pragma unroll
                            for (int e = 1; e < C; ++e)
#pragma unroll
                                for (int f = 0; f < Sh::kKeys / 2; f += 16)
                                    tmem_st16(p_at + ((copy + e) & (C - 1)) * (Sh::kKeys / 2) + f, zero);
                        }
                        // does every row see all of the keys?  (One answer for the warp: its lanes are of one copy.)
                        const bool all = mine0 + Sh::kKeys <= past + (a.parent ? 0 : first_t + 1) &&
                                         (!a.window || mine0 > past + last_t - a.window);
                        if (!all) {
#pragma unroll
                            for (int e = 0; e < Sh::kKeys; e += 32) {
                                const int at0 = mine0 + e;
                                uint32_t see = below(lim - at0);
                                if (a.window) see &= ~below(low - at0) | below(a.n_sink - at0);
                                if (a.parent) {
                                    const int sh = past - at0;            // node 0's bit
                                    if (sh > -64 && sh < 32) see |= (uint32_t)(sh >= 0 ? line << sh : line >> -sh);
                                }
#pragma unroll
                                for (int f = 0; f < 32; ++f)
                                    if (!(see >> f & 1)) x[e + f] = 0xff800000u;
                            }
                        }
                        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int e = 0; e < Sh::kKeys; e += 2)
                            top[e / 2 & 3] = max3(top[e / 2 & 3], __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
                        float to = max3(fmaxf(top[0], top[1]), top[2], top[3]);
                        if constexpr (Sh::kShare == 2) {
                            // (the other thread's P goes over scores of this one's, so its store comes behind this load)
                            ctl.each[half][tl] = to;
                            fence_before();
                            rows_sync(wid);
                            fence_after();
                            to = fmaxf(to, ctl.each[half ^ 1][tl]);
                            rows_sync(wid);
                        }
                        const bool grows = on && (to - m) * sc > kSlack;
                        if (q == 0) {
                            m = fmaxf(m, to);
                        } else if (__any_sync(kWarp, grows)) {
                            const float up = fmaxf(m, to), f = m == up ? 1.f : ex2((m - up) * sc);
                            ok = ok && wait_o();
                            fence_after();
                            l *= f;
                            m = up;
#pragma unroll 1
                            for (int e = half * (D / Sh::kShare); e < (half + 1) * (D / Sh::kShare); e += 32) {
                                uint32_t o[32];
                                tmem_ld32(o_at + e, o);
                                wait_ld();
#pragma unroll
                                for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                                tmem_st32(o_at + e, o);
                            }
                        }
                        const float base = m == -INFINITY ? 0.f : -m * sc;
                        const uint64_t sc2 = pair2(sc, sc), base2 = pair2(base, base);
                        float sum[4] = {};
#pragma unroll
                        for (int e = 0; e < Sh::kKeys; e += 32) {
                            uint32_t p[16];
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                const float2 z = split2(fma2(pair2(__uint_as_float(x[e + 2 * k]), __uint_as_float(x[e + 2 * k + 1])), sc2, base2));
                                const float y0 = ex2(z.x), y1 = ex2(z.y);
                                p[k] = pack_bf16(y0, y1);
                                add_pair(sum[2 * (k & 1)], sum[2 * (k & 1) + 1], p[k]);
                            }
                            tmem_st16(p_at + mine / 2 + e / 2, p);
                        }
                        l += (sum[0] + sum[2]) + (sum[1] + sum[3]);
                        wait_st();
                    }
                    if (dry) break;
                    // ---- rows of V that no row of the block sees
                    if (k0 + kTile > w.span.hi || (k0 < w.span.lo && k0 + kTile > sink)) {
                        const int key = k0 + tl, part = tl / Sh::kVTokens, g = tl % Sh::kVTokens;
                        // The stage's last round has to be over (see the MMAs): it is where the ring is long, as the P V before
                        // this S buffer's is done; else the P V of the tile before is waited for, whose stages come ahead.
                        if (!Sh::kLongRing && any) ok = ok && wait_o();
                        const Ring<Sh::kRing> rv = r.after(((q == 0) + (q + 1 < n)) * Sh::kKStages + part);
                        ok = ok && warp_wait(full(rv.stage), rv.round & 1);
                        if (ok && !(key < w.span.hi && (key >= w.span.lo || key < sink))) {
                            const uint32_t to = ring + rv.stage * Sh::kStage + (g >> 3) * (Sh::kChunks * 1024) + (g & 7) * 128;
#pragma unroll 1
                            for (int e = half; e < Sh::kChunks; e += Sh::kShare)
#pragma unroll
                                for (int k = 0; k < 8; ++k)       // (turned, so that lanes do not meet in a bank)
                                    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};\n" ::"r"(to + e * 1024 + ((k + g) & 7) * 16), "r"(0)
                                                 : "memory");
                        }
                        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
                    }
                    // what the ring has moved on by, with this tile's V: the next tile's K comes before it
                    if (q == 0) r.next(Sh::kKStages);
                    if (q + 1 < n) r.next(Sh::kKStages);
                    r.next(Sh::kVStages);
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(p_full(u.stage));
                    before = u;
                    any = true;
                    u.next();
                }
                if (dry) {
                    dry = false;
                    begin();
                    if (c >= share.ctas || !w.begin(a, at, share.start(c + 1) - share.start(c))) break;
                    last_pair = -1;
                    continue;
                }
                // ---- the block's sums: its output, or a part of it
                float factor = 1.f;
                if constexpr (C > 1) {
                    // copies to a common maximum
                    ctl.stats[tl] = make_float2(m, l);
                    softmax_sync<Sh::kSoftmax>();
                    const float own = m;
                    m = -INFINITY;
                    l = 0.f;
#pragma unroll
                    for (int e = 0; e < C; ++e) m = fmaxf(m, ctl.stats[e * Sh::kRows + row].x);
#pragma unroll
                    for (int e = 0; e < C; ++e) {
                        const float2 st = ctl.stats[e * Sh::kRows + row];
                        l += st.x == -INFINITY ? 0.f : st.y * ex2((st.x - m) * sc);
                    }
                    factor = own == -INFINITY ? 0.f : ex2((own - m) * sc);
                }
                if constexpr (Sh::kShare == 2) {
                    ctl.each[half][tl] = l;
                    softmax_sync<Sh::kSoftmax>();
                    l = ctl.each[0][tl] + ctl.each[1][tl];
                }
                if (w.whole) factor /= l;
                const size_t part0 = size_t(2 * c + (w.first ? 0 : 1)) * a.part_rows;
                if (!w.whole && on && copy == 0 && half == 0 && chk(a.stats + part0 + row, 8, a.stats, a.ext_stats))
                    a.stats[part0 + row] = make_float2(m * sc, l);
                ok = ok && warp_wait(o_done(before.stage), before.round & 1);
                fence_after();
                // Rows go through the two stages, each turned by its number of 16 bytes (so that 32 lanes write 32 rows
                // without conflicts), and leave side by side, four 16-byte pieces a thread in flight.  (Written by its own
                // lane, 16 bytes a row at a time, 96 rows of 256 took 7400 cycles; as two bulk copies a row, 11500.)
                constexpr int kCols = Sh::kOut / 4 < D ? Sh::kOut / 4 : D, kPieces = kCols / 4, kStep = Sh::kSoftmax / kPieces;
                unsigned char *stage[2];
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    const Ring<Sh::kRing> st = r.after(p);
                    ok = ok && warp_wait(full(st.stage), st.round & 1);
                    stage[p] = sm + Sh::kQBytes + st.stage * Sh::kStage;
                }
                // row `from` of tensor memory, its 16-byte piece p
                auto spot = [&](int from, int p) {
                    return reinterpret_cast<float4 *>((from < kLanes / 2 ? stage[0] : stage[1]) + from % (kLanes / 2) * Sh::kOut +
                                                      ((p + from) & (kPieces - 1)) * 16);
                };
                const int rows = ok ? (last_t + 1 - first_t) * a.G : 0;            // as in every warp, unless a wait gave up
                const int piece = tid % kPieces, row0 = tid / kPieces;
                unsigned char *out0 = w.whole ? reinterpret_cast<unsigned char *>(static_cast<__nv_bfloat16 *>(a.out) +
                                                    (((size_t)s * a.T + first_t) * a.H + (size_t)w.kvh * a.G) * D + 4 * piece)
                                              : reinterpret_cast<unsigned char *>(a.partial + (part0 + row0) * D + 4 * piece);
#pragma unroll 1
                for (int at0 = 0; at0 < D; at0 += kCols) {
                    if (at0 > 0) softmax_sync<Sh::kSoftmax>();
                    if (ok && busy) {
#pragma unroll 1
                        for (int e = half * (kCols / Sh::kShare); e < (half + 1) * (kCols / Sh::kShare); e += 32) {
                            uint32_t o[32];
                            tmem_ld32(o_at + at0 + e, o);
                            wait_ld();
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                *spot(tl, e / 4 + k) = make_float4(__uint_as_float(o[4 * k]) * factor, __uint_as_float(o[4 * k + 1]) * factor,
                                                                  __uint_as_float(o[4 * k + 2]) * factor, __uint_as_float(o[4 * k + 3]) * factor);
                        }
                    }
                    if (at0 + kCols == D) {
                        fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(o_free);
                    }
                    softmax_sync<Sh::kSoftmax>();
#pragma unroll 1
                    for (int x = row0; x < rows; x += 4 * kStep) {
                        float4 y[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int rr = min(x + k * kStep, rows - 1);
                            y[k] = *spot(rr, piece);
#pragma unroll
                            for (int e = 1; e < C; ++e) {
                                const float4 z = *spot(e * Sh::kRows + rr, piece);
                                y[k].x += z.x; y[k].y += z.y; y[k].z += z.z; y[k].w += z.w;
                            }
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int rr = x + k * kStep;
                            if (rr >= rows) break;
                            if (w.whole) {
                                const int tt = rr / a.G;
                                uint2 *to = reinterpret_cast<uint2 *>(out0 + (((size_t)tt * a.H + rr - tt * a.G) * D + at0) * 2);
                                if (chk(to, 8, a.out, a.ext_q)) *to = make_uint2(pack_bf16(y[k].x, y[k].y), pack_bf16(y[k].z, y[k].w));
                            } else {
                                float4 *to = reinterpret_cast<float4 *>(out0 + ((rr - row0) * D + at0) * 4);
                                if (chk(to, 16, a.partial, a.ext_partial)) *to = y[k];
                            }
                        }
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
                ok = softmax_all<Sh::kSoftmax>(ok);
                if (tid < 4) mbar_arrive(empty(r.after(tid / 2).stage));
                r.next(2);
                if (!ok || !w.next(a)) break;
            } while (true);
        } else {
            if (!together) begin();
            Walk w;
            const bool some = c < share.ctas && w.begin(a, at, share.start(c + 1) - share.start(c));
            if (!some) {
                // nothing to do: fewer tiles than CTAs
            } else if (wid < Sh::kMmas) {
                // ---- the loads
                const int loader = wid - Sh::kLoads;
                const int page_log2 = a.kv.page_log2, page = 1 << page_log2;
                Ring<Sh::kRing> r;                // the next stage to fill
                auto free_stage = [&] {
                    if (r.round > 0) ok = ok && warp_wait(empty(r.stage), (r.round - 1) & 1);
                };
                int blocks = 0;
                do {
                    const int s = w.pair / a.n_tb, sink = min(a.n_sink, w.span.lo), lo = w.span.lo, hi = w.span.hi;
                    const int32_t *table = a.kv.table + (size_t)s * a.kv.max_pages;
                    // page p of a tile is lane p's (a page of more than a tile: lane 0's)
                    auto page_id = [&](int j) {
                        if (j >= w.j1) return -1;
                        const int from = w.span.tile(j) * kTile + (lane << page_log2), to = from + min(page, kTile);
                        const bool on = lane < max(1, kTile >> page_log2) && ((from < hi && to > lo) || from < sink);
                        return on ? page_at(a.kv, table + (from >> page_log2), a.d_status) : -1;
                    };
                    // a tile's K or V: of a stage kKChunks columns of all keys, or all columns of kVTokens keys
                    auto put = [&](int j, int id, bool value) {
                        const CUtensorMap *map = value ? &args.v_map : &args.k_map;
                        const int tokens = value ? Sh::kVTokens : kTile, box = min(page, tokens), stages = value ? Sh::kVStages : Sh::kKStages;
                        const uint32_t box_bytes = (uint32_t)box * (value ? D : 64 * Sh::kKChunks) * 2;
                        const int tile0 = w.span.tile(j) * kTile;
#pragma unroll 1
                        for (int part = 0; part < stages; ++part, r.next()) {
                            const uint32_t st = r.stage;
                            free_stage();
                            if (!ok) return;
                            // (A stage is only full when both loaders have passed it, so that neither can fall a round behind.)
                            if (Sh::kLoaders == 2 && value != (loader == 1)) {
                                if (lane == 0) mbar_arrive(full(st));
                                continue;
                            }
                            const int from = tile0 + (value ? part * Sh::kVTokens : 0) + lane * box, to = from + box;
                            const bool on = lane < tokens / box && ((from < hi && to > lo) || from < sink);
                            int g = __shfl_sync(kWarp, id, ((from >> page_log2) - (tile0 >> page_log2)) & 31);
                            if (on && (g < 0 || g >= a.kv.n_pages)) {
                                report(a.d_status, GDN_ERR_PAGE);
                                g = a.kv.n_pages; // outside the tensor: zeros
                            }
                            const uint32_t boxes = __popc(__ballot_sync(kWarp, on));
                            if (lane == 0) mbar_expect(full(st), boxes * box_bytes);
                            __syncwarp();
                            if (on)
                                tma_box5(ring + st * Sh::kStage + lane * box_bytes, map, 0, 0, value ? 0 : part * Sh::kKChunks,
                                         ((w.kvh << page_log2) + (from & (page - 1))) >> 3, g, full(st));
                        }
                    };
                    int id = page_id(w.j0), id1 = page_id(w.j0 + 1);
                    const int qb = blocks % Sh::kQBuffers, uses = blocks / Sh::kQBuffers;
                    if (loader == 0 && uses > 0) ok = ok && warp_wait(q_empty(qb), (uses - 1) & 1);
                    if (loader == 0 && ok) {
                        const int q = lane / C;   // lane: chunk, copy
                        if (lane == 0) mbar_expect(q_full(qb), (uint32_t)(a.TB * a.G * 128 * (Sh::kChunks * C)));
                        __syncwarp();
                        if (q < Sh::kChunks)
                            tma_box5(qbase + qb * Sh::kQTile + q * (kLanes * 128) + (lane % C) * (Sh::kRows * 128), &args.q_map, 0, q,
                                     w.kvh * a.G, w.span.t0, s, q_full(qb));
                    }
                    __syncwarp();
                    ++blocks;
                    // in the order in which the MMAs take them
                    put(w.j0, id, false);
#pragma unroll 1
                    for (int j = w.j0; j < w.j1 && ok; ++j) {
                        const int id2 = page_id(j + 2);
                        if (j + 1 < w.j1) put(j + 1, id1, false);
                        put(j, id, true);
                        id = id1;
                        id1 = id2;
                    }
                    // two stages for the block's sums on their way out
                    for (int p = 0; p < 2 && ok; ++p, r.next()) {
                        free_stage();
                        if (ok && lane == 0) mbar_arrive(full(r.stage));
                    }
                } while (ok && w.next(a));
                if (!ok)                          // the copies in flight land before the CTA ends
                    for (int i = 0; i < Sh::kRing; ++i) {
                        const uint32_t fills = r.round + (i < (int)r.stage);      // of stage i
                        if (fills > 0 && !mbar_wait(full(i), (fills - 1) & 1)) break;     // (they have, in that time)
                    }
            } else {
                // ---- the MMAs, from two warps: an MMA's end is known some 400 cycles after it, and what one warp waits for the
                // other need not: one makes S, the other takes P V.  Both pass every stage of the ring in its order, whether theirs or
                // not, and a stage is only filled again when both have: its barrier has two phases, so that who falls a
                // round behind would wait for ever, and who runs ahead would take the last round's for this one's.
                const int part = wid - Sh::kMmas;
                const uint32_t qk_desc = idesc(kTile, false) | (a.scale < 0.f ? kNegateA : 0);
                const bool leader = elect_one();  // one thread issues all of a warp's, so that its commits cover them
                Ring<Sh::kRing> r;                // the next stage
                Ring<Sh::kBuffers> x;             // this warp's next S
                int blocks = 0;
                auto arrived = [&](bool mine) {
                    ok = ok && warp_wait(full(r.stage), r.round & 1);
                    fence_after();
                    if (ok && leader && !mine) mbar_arrive(empty(r.stage));
                };
                // S.  Who does not take the stages passes them by
                auto column = [&] { return tmem + x.stage * 128 + (x.stage == 2 ? 128 : 0); };
                auto qk = [&](bool mine) {
#pragma unroll
                    for (int p = 0; p < Sh::kKStages; ++p, r.next()) {
                        arrived(mine);
                        if (ok && leader && mine) {
                            const uint64_t qd = make_desc(qbase + (blocks % Sh::kQBuffers) * Sh::kQTile + p * Sh::kKChunks * (kLanes * 128), 16, 1024);
                            const uint64_t kd = make_desc(ring + r.stage * Sh::kStage, 16, Sh::kKChunks * 1024);
#pragma unroll
                            for (int k = 0; k < 4 * Sh::kKChunks; ++k)
                                mma_ss(column(), qd + ((k / 4) * (kLanes * 128) + (k & 3) * 32) / 16, kd + ((k / 4) * 1024 + (k & 3) * 32) / 16,
                                       qk_desc, p > 0 || k > 0);
                            mma_commit(empty(r.stage));
                            if (p + 1 == Sh::kKStages) mma_commit(s_full(x.stage));
                        }
                        __syncwarp();
                    }
                };
                auto pv = [&](bool fresh, bool mine) {
#pragma unroll
                    for (int p = 0; p < Sh::kVStages; ++p, r.next()) {
                        arrived(mine);
                        if (ok && leader && mine) {
                            const uint64_t vd = make_desc(ring + r.stage * Sh::kStage, 1024, Sh::kChunks * 1024);
#pragma unroll
                            for (int k = 0; k < Sh::kVTokens / 16; ++k)
                                mma_ts(tmem + Sh::kOColumn, column() + (p * Sh::kVTokens / 16 + k) * 8,
                                       vd + k * 2 * Sh::kChunks * 1024 / 16, idesc(D, true), !fresh || p > 0 || k > 0);
                            mma_commit(empty(r.stage));
                            if (p + 1 == Sh::kVStages) mma_commit(o_done(x.stage));
                        }
                        __syncwarp();
                    }
                };
                do {
                    if (part == 0) ok = ok && warp_wait(q_full(blocks % Sh::kQBuffers), (blocks / Sh::kQBuffers) & 1);
                    const int n = w.j1 - w.j0;
                    // Q is free for the next block once the last S is made
                    auto q_done = [&](int t) {
                        if (t == n - 1 && ok && leader) mma_commit(q_empty(blocks % Sh::kQBuffers));
                        __syncwarp();
                    };
#pragma unroll 1
                    for (int t = -1; t < n && ok; ++t) {
                        if (t + 1 < n) {
                            // an S buffer is free once the P V of its last use is done
                            if (part == 0 && x.round > 0) ok = ok && warp_wait(o_done(x.stage), (x.round - 1) & 1);
                            qk(part == 0);
                            if (part == 0) {
                                q_done(t + 1);
                                x.next();
                            }
                        }
                        if (t >= 0) {
                            if (part == 1) {
                                ok = ok && warp_wait(p_full(x.stage), x.round & 1);
                                if (t == 0 && blocks > 0) ok = ok && warp_wait(o_free, (blocks - 1) & 1);
                            }
                            pv(t == 0, part == 1);
                            if (part == 1) x.next();
                        }
                    }
                    r.next(2);                    // those of the sums on their way out, which the softmax warps pass
                    ++blocks;
                } while (ok && w.next(a));
            }
        }
    }
    if (!ok && lane == 0) report(a.d_status, GDN_ERR_TIMEOUT);
    if (c + 1 == a.ctas)
        for (int s = tid; s < a.B; s += kThreads) {
            int past;
            if (live_tokens(a.kv, a.length, a.T, s, past, a.d_status) < 0) report(a.d_status, GDN_ERR_LENGTH);
        }
    fence_before();
    __syncthreads();
    fence_after();
    if (wid == Sh::kMmas) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tmem));
}

template <int D, int C> cudaError_t launch(TcArgs &t, cudaStream_t stream) {
    using Sh = Shape<D, C>;
    PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
    if (!encode) return cudaErrorNotSupported;
    const AttendArgs &a = t.a;
    const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
    auto map = [&](CUtensorMap *m, const void *p, const cuuint64_t *dims, const cuuint64_t *strides, const cuuint32_t *box) {
        return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void *>(p), dims, strides, box, ones,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    const cuuint64_t es = 2, page = 1ull << a.kv.page_log2;
    {
        // a block's rows: G heads of TB tokens of one slot (tokens past T read zeros)
        const cuuint64_t dims[5] = {64, D / 64, (cuuint64_t)a.H, (cuuint64_t)a.T, (cuuint64_t)a.B};
        const cuuint64_t strides[4] = {128, D * es, a.H * D * es, (cuuint64_t)a.T * a.H * D * es};
        const cuuint32_t box[5] = {64, 1, (cuuint32_t)a.G, (cuuint32_t)a.TB, 1};
        if (!map(&t.q_map, a.q, dims, strides, box)) return cudaErrorInvalidValue;
    }
    // a page of a kv head: groups of 8 tokens, in each the 64-column chunks, in each 8 rows
    const cuuint64_t dims[5] = {64, 8, D / 64, (cuuint64_t)a.Hk * (page / 8), (cuuint64_t)a.kv.n_pages};
    const cuuint64_t strides[4] = {D * es, 128, 8 * D * es, (cuuint64_t)a.kv.page_stride * es};
    const cuuint32_t kbox[5] = {64, 8, Sh::kKChunks, (cuuint32_t)(page < kTile ? page / 8 : kTile / 8), 1};
    const cuuint32_t vbox[5] = {64, 8, D / 64, (cuuint32_t)(page < Sh::kVTokens ? page / 8 : Sh::kVTokens / 8), 1};
    if (!map(&t.k_map, a.kv.k, dims, strides, kbox) || !map(&t.v_map, a.kv.v, dims, strides, vbox)) return cudaErrorInvalidValue;

    constexpr size_t smem = Sh::kQBytes + Sh::kRing * Sh::kStage + sizeof(Control<Sh::kRing, Sh::kThreads>);
    static_assert(smem <= 227 * 1024, "shared memory of a CTA");
    static PerContext<int> limits;
    unsigned long long ctx = 0;
    int set = 0;
    if (!current_context_id(&ctx) || !limits.get(ctx, &set)) {
        const cudaError_t e = cudaFuncSetAttribute(attend_tc_kernel<D, C>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        if (current_context_id(&ctx)) limits.put(ctx, 1);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(a.ctas), 1, 1);
    cfg.blockDim = dim3(Sh::kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, attend_tc_kernel<D, C>, t);
    return e != cudaSuccess ? e : launch_attend_join(a, GDN_BF16, stream);
}

// Copies of the rows: four where a slot has at most 32.
int copies(int T, int G) { return (long long)T * G <= 32 ? 4 : 1; }

template <int D> cudaError_t launch_d(TcArgs &t, cudaStream_t stream) {
    return copies(t.a.T, t.a.G) == 4 ? launch<D, 4>(t, stream) : launch<D, 1>(t, stream);
}

}  // namespace

AttendBlock attend_bf16_block(int T, int G, int D) {
    const int c = copies(T, G), rows = kLanes / c, tokens = rows / G < T ? rows / G : T;
    // A part of many rows costs as much as a tile's keys and values.  A block's beginning and end take 3 to 5 us, a tile of 128
    // keys 0.8 (D = 64), 1.5 (128) or 3 us (256).  Where a slot is one block the cache's bytes bind, and 128 CTAs take them a little
    // faster than one on each of 152 SMs (8 slots of 20000 positions: 100.1 and 104.2 us for one token with D = 128, 108.8 and
    // 113.7 for 16 with D = 256), or as fast where they come from L2 (8 of 1500: 17.8 and 17.9, 23.7 and 23.8; 64 single tokens of up
    // to 300 with D = 256 lose, 26.0 and 24.3) or under a window of 1024 (D = 128, 16 and 64 single tokens: 21.5 and 23.0, 55.9
    // and 55.8; D = 256, 32 slots of 16: 45.2 and 47.0).  With D = 64 (59.1 and 58.0; 64 slots of a window 44.7 and 41.0) or
    // several blocks (a prompt: 509 and 442; trees of 64: 46.0 and 42.4) they are slower.
    const int least = c > 1 ? 1 : 3, pad = D == 64 ? 4 : 3, ctas = D >= 128 && tokens == T ? 128 : kAttendCtas;
    return {rows, tokens, least, pad, ctas};
}

cudaError_t launch_attend_bf16(const AttendArgs &a, cudaStream_t stream) {
    TcArgs t{};
    t.a = a;
    return a.D == 64 ? launch_d<64>(t, stream) : a.D == 128 ? launch_d<128>(t, stream) : launch_d<256>(t, stream);
}

}  // namespace gdn
