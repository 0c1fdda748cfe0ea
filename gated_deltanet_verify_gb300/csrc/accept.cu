// accept.cu -- how much of a draft a verify step keeps, decided on the device.
//
// Chain: the target's token after input t is tokens[t], the draft's guess for
// that place is the next input draft[t+1].  With n the number of leading t at
// which they agree, inputs 0 .. n are kept (trim = T-1-n, what gdn_rollback
// takes) and tokens[0 .. n] are the step's output: the n accepted guesses, then
// the target's own token at the first place where the draft was wrong or ended.
// Tree: the same from node 0 along the children that hold the sampled token.
//
// This is lossless for any drafter: every emitted token is the one sampled from
// the target's distribution at its place, a draft only decides whether the
// state after it is at hand.
//
// A few hundred bytes per slot, so launch latency bounds it: one warp per slot,
// one load per lane and tensor (two past 32 tokens), then ballots; the walk
// down a tree keeps its nodes in registers (two per lane), so a step costs two
// ballots and a shuffle and no memory access.  In a captured graph a chain takes
// 1.2 us (8 slots of 16 to 1024 of 64), a tree 1.6 to 2.5 us.
#include "step.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 4;             // slots per CTA
constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ unsigned long long ballot2(bool lo, bool hi) {
    return (unsigned long long)__ballot_sync(kFull, lo) | ((unsigned long long)__ballot_sync(kFull, hi) << 32);
}
// value of element i of a 64-element row held as element lane in lo and lane + 32 in hi
__device__ __forceinline__ int pick(int lo, int hi, int i) {
    const int a = __shfl_sync(kFull, lo, i & 31), b = __shfl_sync(kFull, hi, i & 31);
    return i < 32 ? a : b;
}

template <bool TREE>
__global__ void __launch_bounds__(32 * kWarps) accept_kernel(const AcceptArgs a) {
    // programmatic dependent launch: the sampled tokens come from the kernel before; the kernel after waits
    // for this grid's completion itself
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    const int lane = threadIdx.x & 31, s = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (s >= a.B) return;
    auto chk = [&](const void *p, const void *base, size_t ext) { return in_bounds(p, 4, base, ext, a.d_status); };
    const int T = a.T;
    const size_t ext_bt = size_t(a.B) * T * 4, ext_b = size_t(a.B) * 4;
    auto load = [&](const int32_t *base, int t, int none) -> int {
        const int32_t *p = base + size_t(s) * T + t;
        return t < T && chk(p, base, ext_bt) ? *p : none;
    };
    auto report = [&](gdn_status code) {
        if (lane == 0 && a.d_status) atomicCAS(a.d_status, int(GDN_OK), int(code));
    };
    const int len = a.length == nullptr ? T : (chk(a.length + s, a.length, ext_b) ? a.length[s] : -1);
    int tok[2], dr[2], place, last, n_emit;
    int path[2] = {-1, -1};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        tok[q] = load(a.tokens, lane + 32 * q, -1);
        dr[q] = load(a.draft, lane + 32 * q, -1);
    }
    if (len < (TREE ? 0 : 1) || len > T) {
        report(GDN_ERR_LENGTH);
        place = -1; last = -1; n_emit = 0;
    } else if constexpr (!TREE) {
        // agreement at t: the guess for the place after t lies at t + 1
        const int up0 = __shfl_sync(kFull, dr[0], (lane + 1) & 31), up1 = __shfl_sync(kFull, dr[1], (lane + 1) & 31);
        const int next0 = lane == 31 ? up1 : up0, next1 = lane == 31 ? -1 : up1;
        const unsigned long long same = ballot2(tok[0] >= 0 && next0 == tok[0] && lane + 1 < len,
                                                tok[1] >= 0 && next1 == tok[1] && lane + 33 < len);
        last = __ffsll((long long)~same) - 1;         // bit 63 is never set: t + 1 < len <= 64
        place = T - 1 - last;
        n_emit = last + 1;
    } else {
        int par[2];
        bool bad = false;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int t = lane + 32 * q;
            par[q] = load(a.parent, t, -2);
            if (t >= len) par[q] = -2;                 // not a node
            else if (t == 0 ? par[q] != -1 : (par[q] < -1 || par[q] >= t)) {
                par[q] = -2;                           // not a tree in token order: the node is never reached
                bad = true;
            }
        }
        if (__any_sync(kFull, bad)) report(GDN_ERR_TREE);
        const bool root = __shfl_sync(kFull, par[0], 0) == -1;
        int cur = root ? 0 : -1, depth = root ? 1 : 0;
        if (root && lane == 0) path[0] = 0;
        while (cur >= 0) {                             // a child lies after its parent: at most len steps
            const int want = pick(tok[0], tok[1], cur);
            const unsigned long long kids = ballot2(want >= 0 && par[0] == cur && dr[0] == want,
                                                    want >= 0 && par[1] == cur && dr[1] == want);
            if (kids == 0) break;
            cur = __ffsll((long long)kids) - 1;
#pragma unroll
            for (int q = 0; q < 2; ++q)
                if (lane + 32 * q == depth) path[q] = cur;
            ++depth;
        }
        place = cur; last = cur; n_emit = depth;
    }
    const int next = last < 0 ? -1 : pick(tok[0], tok[1], last);
    if (lane == 0) {
        if (chk(a.place + s, a.place, ext_b)) a.place[s] = place;
        if (a.next && chk(a.next + s, a.next, ext_b)) a.next[s] = next;
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int t = lane + 32 * q;
        // every lane takes part in the shuffles
        const int from = TREE ? (path[q] < 0 ? 0 : path[q]) : t;
        const int e0 = __shfl_sync(kFull, tok[0], from & 31), e1 = __shfl_sync(kFull, tok[1], from & 31);
        if (t >= T) continue;
        const size_t i = size_t(s) * T + t;
        if (a.emit && chk(a.emit + i, a.emit, ext_bt)) a.emit[i] = t < n_emit ? (from < 32 ? e0 : e1) : -1;
        if (TREE && a.path && chk(a.path + i, a.path, ext_bt)) a.path[i] = path[q];
    }
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
}

}  // namespace

cudaError_t launch_accept(const AcceptArgs &a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned((a.B + kWarps - 1) / kWarps), 1, 1);
    cfg.blockDim = dim3(32 * kWarps, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return a.parent ? cudaLaunchKernelEx(&cfg, accept_kernel<true>, a) : cudaLaunchKernelEx(&cfg, accept_kernel<false>, a);
}

}  // namespace gdn
