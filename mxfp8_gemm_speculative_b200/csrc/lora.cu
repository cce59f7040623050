// Low-rank adapters of many requests at once, beside a shared projection:
//
//   Out[m] = Y[m] + s[a] * (X[m] A[a]^T) B[a]^T,    a = index[m],
//
// X bf16 [M][K], A bf16 [L][R][K], B bf16 [L][N][R], Y and Out bf16 [M][N];
// a token whose index names no adapter keeps its row of Y.
//
// What bounds it: 2 M R (K + N) flops against the bytes of the adapters in
// use (2 R (K + N) each) and of X, Y and Out.  With R <= 128 that is at most
// a few hundred flops per byte for one adapter and far fewer for many, so
// HBM bytes should bound a large batch, and latency bounds a small one.
// mma.sync, since a tcgen05 tile (128 rows of one adapter) would be mostly
// empty in a decode batch.  In the expand kernel of a prefill chunk its pipe is
// 24 % busy at R = 16, 37 % at R = 32 and 47 % at R = 128, and the one that
// takes T apart (logic and permutes) 50 %: from R = 32 on those two, and not
// bytes, are what the kernel takes its time for.
//
// Two kernels, joined by programmatic dependent launch:
//   shrink   T = s * X A^T, [M][R] in fp32;
//   expand   Out = Y + T B^T, T as three bf16 of eight bits of mantissa each
//            (the inner product keeps its 24 bits, at the price of three times
//            the MMAs), summed in fp32 and rounded once.
//
// Tokens come in any order.  Both kernels take blocks of 64 consecutive tokens
// and group a block's tokens by adapter with warp instructions (no sort
// kernel, no host plan, nothing read back), so an adapter is read once per
// block that uses it and once in all for up to 64 tokens.
//
// Measured (B200, graph of calls over rotating buffers): 8192 tokens,
// 5120 -> 17408, R = 16: 132 us for 658 MB (5.0 TB/s; shrink 23, expand 109),
// R = 32: 172 us; 37 tokens of 48 adapters, 17408 -> 5120, R = 64: 23 us for
// 72 MB; one token, 5120 -> 5120: 6.9 us (two kernels of a few dependent steps
// each).
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace mxg {
namespace {

typedef unsigned long long u64;

constexpr int kBlockTok = 64;     // tokens grouped together
constexpr int kShrinkWarps = 8;
constexpr int kFew = 16;          // tokens of a group that takes the smaller stages

struct LoraParams {
    const uint16_t *X, *A, *B, *Y;   // bf16
    uint16_t *Out;
    const float *scales;     // [L] or NULL (all 1)
    const int *index;        // [M]
    WsHeader *hdr;           // status word, cleared by the shrink kernel
    float4 *T;               // fp32 [M][R]
    long long ldx, ldy, ldo; // row strides in elements
    int M, N, K, R, L;
};

// The first wait that ran out in any call on the device since lora_status
// cleared it: the workspace of a call may be gone when the caller asks.
__device__ WsHeader g_lora_errors;

__device__ __forceinline__ void record_timeout(WsHeader *hdr, int where)
{
    record_error(hdr, MXG_ERR_TIMEOUT, where);
    record_error(&g_lora_errors, MXG_ERR_TIMEOUT, where);
}

// A wait that nothing ends, for the self-test of that record.
__global__ void lora_wait_timeout_kernel(unsigned long long limit_ns)
{
    __shared__ uint64_t bar;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        fence_barrier_init();
    }
    __syncthreads();
    const bool ok = __all_sync(0xffffffffu, mbar_wait(&bar, 0, limit_ns));
    if (!ok && threadIdx.x == 0)
        record_timeout(&g_lora_errors, 599);
}

// 16 bytes global -> shared, asynchronous; zeros when `in` is false.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool in)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(in ? 16 : 0)
                 : "memory");
}
// Arrives on a barrier once the thread's asynchronous copies so far have landed
// (one of the barrier's expected arrivals).
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

// -------------------------------------------------------- tokens by adapter
// The block's tokens grouped by adapter, in the registers of a warp: lane l
// knows tokens l and l + 32, with the tokens (a bit each) of their groups.
struct Groups {
    int a0, a1;        // adapters (-1: none, -2: no such token)
    u64 of0, of1;      // tokens of the same adapter
    u64 leaders;       // first token of every group
};

// raw0, raw1: the index of tokens lane and lane + 32 (anything behind ntok).
__device__ __forceinline__ Groups group_tokens(int raw0, int raw1, int ntok, int L, int lane)
{
    Groups g;
    g.a0 = lane >= ntok ? -2 : raw0 >= 0 && raw0 < L ? raw0 : -1;
    g.a1 = lane + 32 >= ntok ? -2 : raw1 >= 0 && raw1 < L ? raw1 : -1;
    unsigned m00, m01 = 0, m10 = 0, m11 = 0;
    const int a = __shfl_sync(0xffffffffu, g.a0, 0);
    if (__all_sync(0xffffffffu, (g.a0 == a || g.a0 == -2) && (g.a1 == a || g.a1 == -2))) {
        // one group
        const u64 all = ntok == 64 ? ~0ull : (1ull << ntok) - 1;
        g.of0 = g.of1 = all;
        g.leaders = 1;
        return g;
    }
    m00 = __match_any_sync(0xffffffffu, g.a0);
    m11 = ntok > 32 ? __match_any_sync(0xffffffffu, g.a1) : 0xffffffffu;
    if (ntok > 32)
        // the halves against each other, by independent shuffles (a loop over
        // one half's adapters takes four times as long for many of them)
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            m01 |= (unsigned)(__shfl_sync(0xffffffffu, g.a1, i) == g.a0) << i;
            m10 |= (unsigned)(__shfl_sync(0xffffffffu, g.a0, i) == g.a1) << i;
        }
    g.of0 = m00 | (u64)m01 << 32;
    g.of1 = m10 | (u64)m11 << 32;
    const unsigned lead0 = __ballot_sync(0xffffffffu, g.a0 != -2 && __ffs(m00) - 1 == lane);
    const unsigned lead1 =
        __ballot_sync(0xffffffffu, g.a1 != -2 && m10 == 0 && __ffs(m11) - 1 == lane);
    g.leaders = lead0 | (u64)lead1 << 32;
    return g;
}

// The same by a whole CTA, for more than 32 tokens: each of its first eight
// warps compares every token with eight others (by one warp, 64 shuffles; by
// all nine warps of two CTAs of an SM for themselves, a microsecond of them).
__device__ __forceinline__ Groups group_tokens_cta(int raw0, int raw1, int ntok, int L, int lane,
                                                   int warp, u64 (&masks)[kBlockTok])
{
    Groups g;
    g.a0 = lane >= ntok ? -2 : raw0 >= 0 && raw0 < L ? raw0 : -1;
    g.a1 = lane + 32 >= ntok ? -2 : raw1 >= 0 && raw1 < L ? raw1 : -1;
    if (warp < 8) {
        uint32_t e0 = 0, e1 = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int l = (8 * warp + i) & 31;
            const int a = __shfl_sync(0xffffffffu, warp < 4 ? g.a0 : g.a1, l);
            e0 |= (uint32_t)(a == g.a0) << i;
            e1 |= (uint32_t)(a == g.a1) << i;
        }
        reinterpret_cast<uint8_t *>(&masks[lane])[warp] = (uint8_t)e0;
        reinterpret_cast<uint8_t *>(&masks[lane + 32])[warp] = (uint8_t)e1;
    }
    __syncthreads();
    g.of0 = masks[lane];
    g.of1 = masks[lane + 32];
    const unsigned lead0 =
        __ballot_sync(0xffffffffu, g.a0 != -2 && __ffsll(g.of0) - 1 == lane);
    const unsigned lead1 =
        __ballot_sync(0xffffffffu, g.a1 != -2 && __ffsll(g.of1) - 1 == lane + 32);
    g.leaders = lead0 | (u64)lead1 << 32;
    return g;
}

// The group that token `first` leads: its adapter, its number of tokens, and
// those (offsets in the block, rising) in this warp's list.
__device__ __forceinline__ int take_group(const Groups &g, int first, uint8_t *list, int lane,
                                          int &adapter)
{
    const int l = first & 31;
    const bool up = first >= 32;
    adapter = __shfl_sync(0xffffffffu, up ? g.a1 : g.a0, l);
    const u64 of = __shfl_sync(0xffffffffu, up ? g.of1 : g.of0, l);
    __syncwarp();   // the list's last readers are done
    if (of >> lane & 1)
        list[__popcll(of & ((1ull << lane) - 1))] = (uint8_t)lane;
    if (of >> (lane + 32) & 1)
        list[__popcll(of & ((1ull << (lane + 32)) - 1))] = (uint8_t)(lane + 32);
    __syncwarp();
    return __popcll(of);
}

__device__ __forceinline__ float4 ld_peer_f4(const void *p, uint32_t rank)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(peer_addr(p, rank))
                 : "memory");
    return v;
}

// Four fp32 values as sums of three bf16 each, by truncation: eight bits of
// mantissa go to `hi`, the next eight to `mid`, the last to `lo` (all 24, but
// for bits below 2^-133).  Pairs, in the order of the values.
struct Split {
    uint32_t hi[2], mid[2], lo[2];
};
__device__ __forceinline__ Split split_f32(const uint4 &v)
{
    const uint32_t b[4] = {v.x, v.y, v.z, v.w};
    uint32_t m[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float r = __uint_as_float(b[i]) - __uint_as_float(b[i] & 0xFFFF0000u);
        m[i] = __float_as_uint(r);
        l[i] = __float_as_uint(r - __uint_as_float(m[i] & 0xFFFF0000u));
    }
    Split s;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        s.hi[i] = __byte_perm(b[2 * i], b[2 * i + 1], 0x7632);
        s.mid[i] = __byte_perm(m[2 * i], m[2 * i + 1], 0x7632);
        s.lo[i] = __byte_perm(l[2 * i], l[2 * i + 1], 0x7632);
    }
    return s;
}

// Infinities and NaN among bf16 pairs.  note: `seen` becomes nonzero (0 times
// one is NaN); mask: ones over each value that is finite.
__device__ __forceinline__ void note_nonfinite(uint32_t &seen, uint32_t pair)
{
    asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(seen) : "r"(pair), "r"(0u));
}
__device__ __forceinline__ uint32_t finite_mask(uint32_t pair)
{
    return ((pair & 0x7F80u) != 0x7F80u ? 0xFFFFu : 0u) |
           ((pair & 0x7F800000u) != 0x7F800000u ? 0xFFFF0000u : 0u);
}
// An infinity or NaN is its own `hi`: the rest of it, infinity less infinity,
// would be NaN.
__device__ __forceinline__ void drop_rest(Split &s, int pair)
{
    const uint32_t keep = finite_mask(s.hi[pair]);
    s.mid[pair] &= keep;
    s.lo[pair] &= keep;
}

// Values too small for a bf16 other than 0 become its smallest: an infinity
// times them is an infinity, not NaN.
__device__ __forceinline__ void lift(uint4 &v)
{
    uint32_t *b[4] = {&v.x, &v.y, &v.z, &v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if ((*b[i] & 0x7FFF0000u) == 0 && (*b[i] & 0xFFFFu) != 0)
            *b[i] = (*b[i] & 0x80000000u) | 0x10000u;
}

// Two fp32 values rounded to a bf16 pair.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// ------------------------------------------------------------------- shrink
// One cluster per (block of tokens, share of its groups, slice of ranks); its
// CTAs split K and are added through distributed shared memory in rank order
// (bitwise reproducible; no atomics, no partial sums in memory).  A producer
// warp streams a CTA's K range of a group's rows of X and of the adapter's
// rows of A through a ring in shared memory: A as tensor-map boxes of 64 k, X
// for more than 16 tokens as boxes of 16 rows of a run or as gathers of four
// rows, for fewer by asynchronous copies of 16 bytes (which for 64 scattered
// rows took the producer three times the stage's load: 47 us against 36 for 791
// tokens, 16608 to 3360, R = 32).  Eight consumer warps run MMAs with the ranks as their
// 16 rows and 8 tokens as their columns; a warp takes every other 16 bytes of
// a row, and the two halves are added at the end.
//
// Up to 16 tokens (decode and verify chunks) the bytes of A are what counts,
// and a stage holds more k of fewer rows.  Neither that nor a token's place
// in the batch changes the order of its sums.
template <int RT>
struct Shrink {
    static constexpr int kTok = kBlockTok;                  // most tokens of a group
    static constexpr int sub(int rows) { return (rows + 16 * RT) * 128; }   // 64 k of tokens, ranks
    static constexpr int kSubMany = RT == 1 ? 2 : 1, kSubFew = RT == 1 ? 4 : 2;   // per stage
    static constexpr int kMany = kSubMany * sub(kTok), kFewStage = kSubFew * sub(kFew);
    static constexpr int kSlot = kMany > kFewStage ? kMany : kFewStage;
    static constexpr int kSlots = RT == 1 ? 3 : (RT == 2 ? 7 : 3);
    static constexpr int ST = 16 * RT + 4;                  // row stride of a reduced tile
    static constexpr int kTile = kTok * ST * (int)sizeof(float);
    // ring (aligned to 1024 bytes), tiles of the two halves
    static constexpr size_t smem = (size_t)kSlots * kSlot + 2 * kTile + 1024;
    static constexpr int kThreads = (kShrinkWarps + 1) * 32;
};

// The consumers' part of one item: MMAs over the stages of up to ROWS tokens.
template <int RT, int ROWS, int SUB, typename W>
__device__ __forceinline__ void shrink_item(int ntok, int k0, int k1, uint32_t ring, float *tile,
                                            uint64_t *empty, int &slot, uint32_t &phase, W &&wait,
                                            const bool &ok)
{
    using C = Shrink<RT>;
    constexpr int kHalf = kShrinkWarps / 2;
    constexpr int kPer = (ROWS / 8 + kHalf - 1) / kHalf;   // token tiles per warp
    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int q = warp / kHalf, first = warp % kHalf;
    float acc[kPer][RT][4];
#pragma unroll
    for (int j = 0; j < kPer; ++j)
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[j][i][e] = 0.f;
    // Rows of 128 bytes with the 128-byte swizzle: 16-byte chunk c of row r
    // lies at c ^ (r % 8).  With the chunks 2 t + q, the two rows that eight
    // lanes load together use all banks.
    const uint32_t at = g * 128 + (((2 * t + q) ^ g) << 4);
    for (int k = k0; k < k1; k += 64 * SUB) {
        wait(slot, phase);
        if (ok && 8 * first < ntok) {
            const uint32_t st = ring + slot * C::kSlot + at;
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
                if (u > 0 && k + 64 * u >= k1)
                    break;
                const uint32_t x = st + u * C::sub(ROWS), a = x + ROWS * 128;
                uint4 xv[kPer];
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    xv[j] = lds128a(x + (first + j * kHalf) * 1024);
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    const uint4 a0 = lds128a(a + 2 * i * 1024), a1 = lds128a(a + (2 * i + 1) * 1024);
#pragma unroll
                    for (int j = 0; j < kPer; ++j) {
                        mma_bf16_16816(acc[j][i], a0.x, a1.x, a0.y, a1.y, xv[j].x, xv[j].y);
                        mma_bf16_16816(acc[j][i], a0.z, a1.z, a0.w, a1.w, xv[j].z, xv[j].w);
                    }
                }
            }
        }
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&empty[slot]);
        if (++slot == C::kSlots) {
            slot = 0;
            phase ^= 1;
        }
    }
    // this warp's half: tile[half][token][rank]
    float *mine = tile + q * (C::kTile / (int)sizeof(float));
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int c = 8 * (first + j * kHalf) + 2 * t;
        if (c - 2 * t < ntok)
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    mine[(c + (e & 1)) * C::ST + 16 * i + g + 8 * (e >> 1)] = acc[j][i][e];
    }
}

template <int RT>
__global__ void __launch_bounds__(Shrink<RT>::kThreads, 2)
    lora_shrink_kernel(const __grid_constant__ CUtensorMap x_map,
                       const __grid_constant__ CUtensorMap x_rows,
                       const __grid_constant__ CUtensorMap a_map, const LoraParams p, int slices,
                       int slice_ranks)
{
    using C = Shrink<RT>;
    constexpr int ST = C::ST;
    __shared__ uint8_t lists[kShrinkWarps + 1][kBlockTok];
    __shared__ u64 masks[kBlockTok];
    __shared__ uint64_t full[C::kSlots], empty[C::kSlots];
    extern __shared__ uint8_t dyn_raw[];
    // 1024-byte alignment for the swizzled boxes
    uint8_t *dyn = dyn_raw + ((1024 - (smem_u32(dyn_raw) & 1023)) & 1023);
    float *tile = reinterpret_cast<float *>(dyn + C::kSlots * C::kSlot);   // [halves][tokens][ST]

    const int tid = threadIdx.x, warp = uniform_warp(), lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < C::kSlots; ++i) {
            mbar_init(&full[i], 1 + 32);   // the boxes' bytes, and every lane's own copies
            mbar_init(&empty[i], kShrinkWarps);
        }
        fence_barrier_init();
    }
    __syncthreads();
    // The dependent launch is allowed only after this wait: the expand kernel
    // may then read the index, B and Y before its own wait, since everything
    // queued before this kernel has completed.
    pdl_wait();
    pdl_launch_dependents();
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && tid == 0)
        p.hdr->status = p.hdr->where = 0;

    const int block = blockIdx.z / slices, slice = blockIdx.z % slices;
    const int m0 = block * kBlockTok, r0 = slice * slice_ranks;
    const int ranks = min(slice_ranks, p.R - r0);
    const int btok = min(kBlockTok, p.M - m0);
    const int raw0 = lane < btok ? __ldcg(p.index + m0 + lane) : -1;
    const int raw1 = lane + 32 < btok ? __ldcg(p.index + m0 + lane + 32) : -1;
    const Groups grp = btok > 32 ? group_tokens_cta(raw0, raw1, btok, p.L, lane, warp, masks)
                                 : group_tokens(raw0, raw1, btok, p.L, lane);
    uint8_t *list = lists[warp];
    const int crank = (int)cluster_rank(), csize = (int)cluster_size();
    const int units = (p.K + 63) / 64;
    const int k0 = (int)((long long)crank * units / csize) * 64;
    const int k1 = min(p.K, (int)((long long)(crank + 1) * units / csize) * 64);

    // Every warp walks the items of this cluster, in the same order: every
    // gridDim.y-th group of the block that has an adapter.  Each ends with two
    // cluster barriers that all threads take part in.
    // (The lanes pick the groups at once: a walk that counts them costs 380
    // cycles a group, 5 us before the 24th one's first copy.)
    u64 rest;
    {
        const bool lead0 = (grp.leaders >> lane & 1) && grp.a0 >= 0;
        const bool lead1 = (grp.leaders >> (lane + 32) & 1) && grp.a1 >= 0;
        const unsigned all0 = __ballot_sync(0xffffffffu, lead0);
        const unsigned all1 = __ballot_sync(0xffffffffu, lead1);
        const unsigned below = (1u << lane) - 1;
        const unsigned n0 = __popc(all0 & below), n1 = __popc(all0) + __popc(all1 & below);
        const unsigned mine0 = __ballot_sync(0xffffffffu, lead0 && n0 % gridDim.y == blockIdx.y);
        const unsigned mine1 = __ballot_sync(0xffffffffu, lead1 && n1 % gridDim.y == blockIdx.y);
        rest = mine0 | (u64)mine1 << 32;
    }
    int a = -1, ntok = 0;
    auto next_item = [&]() {
        if (rest == 0)
            return false;
        const int first = __ffsll(rest) - 1;
        rest &= rest - 1;
        ntok = take_group(grp, first, list, lane, a);
        return true;
    };
    // waits by whole warps; after one that ran out the role only goes through
    // the barriers
    bool ok = true;
    auto wait_on = [&](uint64_t *bar, uint32_t parity, int where) {
        if (!ok)
            return;
        ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, kWaitLimitNs));
        if (!ok && lane == 0)
            record_timeout(p.hdr, where);
    };

    if (warp == kShrinkWarps) {
        // ------------------------------------------------------- producer
        const uint64_t pol_a = l2_policy_evict_first(), pol_x = l2_policy_evict_last();
        int slot = 0;
        uint32_t phase = 1;         // of the empty barriers: the first round is free
        bool wrapped = false;
        bool owed = false;          // the last item's barriers
        uint32_t copied = 0;        // slots that 16-byte copies wrote last
        auto barriers = [&]() {
            cluster_barrier();
            cluster_barrier();
            owed = false;
        };
        // One stage after another, by one warp: everything that does not
        // change within an item is worked out before its stages.
        auto stages = [&](auto few_) {
            constexpr bool kIsFew = decltype(few_)::value;
            constexpr int kRows = kIsFew ? kFew : C::kTok;
            constexpr int kSub = kIsFew ? C::kSubFew : C::kSubMany;
            constexpr int kFours = kRows / 4;
            const int n = ntok, m = m0 + list[0];
            // boxes of 16 tokens, for a run (a few rows are as well copied one by one)
            const bool run = !kIsFew && m0 + list[n - 1] - m == n - 1;
            const int xb = run ? (n + 15) / 16 : 0;
            const int fours = run ? 0 : (n + 3) / 4;
            // few: rows lane / 8 + 4 i, their 16 bytes lane % 8; else gathers
            // of rows 4 j .. 4 j + 3, j = lane % kFours
            const int c = lane & 7;
            const uint16_t *src[kIsFew ? kFours : 1];
            uint32_t dst[kIsFew ? kFours : 1];
            int row[4] = {};
            if constexpr (kIsFew) {
#pragma unroll
                for (int i = 0; i < kFours; ++i) {
                    const int r = (lane >> 3) + 4 * i;
                    src[i] = p.X + (m0 + list[r < n ? r : 0]) * p.ldx + 8 * c;
                    dst[i] = r * 128 + ((c ^ (r & 7)) << 4);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    row[i] = m0 + list[min(4 * (lane % kFours) + i, n - 1)];
            }
            const int arow = a * p.R + r0;
            int s = 0;
            for (int k = k0; k < k1; k += 64 * kSub, ++s) {
                // the ring may run ahead of the last item's end by its own size
                if (owed && s == C::kSlots)
                    barriers();
                wait_on(&empty[slot], phase, 531);
                if (!ok)
                    break;
                // Boxes of many tokens land where copies of few did: those are
                // complete now (the consumers that freed the slot waited for
                // them), and the fence puts them before the boxes.
                if (!kIsFew && copied >> slot & 1)
                    fence_proxy_async_smem();
                copied = kIsFew ? copied | 1u << slot : copied & ~(1u << slot);
                const int nsub = kSub == 1 ? 1 : min(kSub, (k1 - k + 63) / 64);
                uint8_t *st = dyn + slot * C::kSlot;
                if (lane == 0)
                    mbar_arrive_expect_tx(&full[slot], nsub * 128 *
                                                           (slice_ranks + 16 * xb +
                                                            (kIsFew ? 0 : 4 * fours)));
                __syncwarp();
                if (lane < nsub)
                    tma_load_2d(st + lane * C::sub(kRows) + kRows * 128, &a_map, k + 64 * lane, arow,
                                &full[slot], pol_a);
                if (!kIsFew && !run && lane < kSub * kFours) {
                    const int u = lane / kFours, j = lane % kFours;
                    if (u < nsub && j < fours)
                        tma_gather4(st + u * C::sub(kRows) + j * 512, &x_rows, k + 64 * u, row[0],
                                    row[1], row[2], row[3], &full[slot], pol_x);
                }
                if (!kIsFew && lane < kSub * (kRows / 16)) {
                    const int u = lane / (kRows / 16), j = lane % (kRows / 16);
                    if (u < nsub && j < xb)
                        tma_load_2d(st + u * C::sub(kRows) + j * 2048, &x_map, k + 64 * u,
                                    m + 16 * j, &full[slot], pol_x);
                }
                if constexpr (kIsFew) {
#pragma unroll
                    for (int u = 0; u < kSub; ++u) {
                        if (u >= nsub)
                            break;
                        const int kc = k + 64 * u;
                        const bool in = kc + 8 * c < p.K;
#pragma unroll
                        for (int i = 0; i < kFours; ++i) {
                            if (i >= fours)
                                break;
                            if ((lane >> 3) + 4 * i < n)
                                cp_async16(smem_u32(st) + u * C::sub(kRows) + dst[i],
                                           in ? src[i] + kc : src[i] - 8 * c, in);
                        }
                    }
                }
                cp_async_arrive(&full[slot]);
                if (++slot == C::kSlots) {
                    slot = 0;
                    phase ^= 1;
                    wrapped = true;
                }
            }
        };
        while (next_item()) {
            if (ntok <= kFew)
                stages(std::true_type());
            else
                stages(std::false_type());
            if (owed)
                barriers();
            owed = true;
        }
        if (owed)
            barriers();
        // (otherwise the consumers wait for every copy issued here)
        if (!ok)
            for (int s = 0; s < C::kSlots; ++s)
                if (s < slot || wrapped)
                    mbar_wait(&full[s], s < slot ? phase ^ 1 : phase, kWaitLimitNs);
        return;
    }

    int slot = 0;
    uint32_t phase = 0;
    auto wait_full = [&](int s, uint32_t parity) { wait_on(&full[s], parity, 541); };
    while (next_item()) {
        const int n = ntok;
        const float sc = p.scales ? __ldcg(p.scales + a) : 1.f;   // ahead of its use
        if (n <= kFew)
            shrink_item<RT, kFew, C::kSubFew>(n, k0, k1, smem_u32(dyn), tile, empty, slot, phase,
                                              wait_full, ok);
        else
            shrink_item<RT, C::kTok, C::kSubMany>(n, k0, k1, smem_u32(dyn), tile, empty, slot,
                                                  phase, wait_full, ok);
        cluster_barrier();
        // ---- add the halves of the CTAs of the cluster in rank order: every
        // CTA finishes a share of the (token, four ranks) entries
        const int quads = ranks / 4;
        float4 out{}, *to = nullptr;   // stored behind the arrival, which would wait for it
        for (int e = tid * csize + crank; e < n * quads; e += kShrinkWarps * 32 * csize) {
            const int c = e / quads, q = e % quads;
            const float *mine = tile + c * ST + 4 * q;
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int w = 0; w < csize; ++w)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float4 v = ld_peer_f4(mine + h * (C::kTile / (int)sizeof(float)), w);
                    s.x += v.x;
                    s.y += v.y;
                    s.z += v.z;
                    s.w += v.w;
                }
            if (to)
                *to = out;
            to = p.T + (size_t)(m0 + list[c]) * (p.R / 4) + r0 / 4 + q;
            out = make_float4(s.x * sc, s.y * sc, s.z * sc, s.w * sc);
        }
        cluster_arrive();   // the tiles are read before the next item's
        if (to)
            *to = out;
        cluster_wait();
    }
}

// ------------------------------------------------------------------- expand
// A CTA takes 256 columns and a list of parts, up to 16 tokens of one adapter
// each: those of a range of blocks, or (few blocks) of a share of one block's
// groups.  Y, Out and T are bytes that are used once, B once per run of parts
// of one adapter, so what counts is how many of them are in flight: a producer
// warp walks the parts and fills a ring of stages with Y (512 bytes a token)
// and T and a ring of B tiles (256 rows of B are one contiguous range), and
// eight consumer warps work on 32 columns each.  Sixteen consecutive tokens
// are one tensor-map box; others are copied row by row (a copy costs the
// engine some 35 cycles whatever its size: row copies alone made a prefill
// chunk 1.6 times slower than plain loads; gathers of four rows, even where no
// part took them, cost a prefill chunk 3 us of 117 and gave scattered tokens 3 %).
//
// MMAs have the part's tokens as their 16 rows and 8 columns each; column c of
// MMA i is column 8 (c / 2) + 2 i + c % 2 of the warp's 32, so a lane's
// results are eight consecutive columns and 16 bytes of a row of Y and Out.
// The sums start from Y.  S = 16-rank steps.
template <int S>
struct Expand {
    static constexpr int kCols = 256;
    static constexpr int kConsumers = kCols / 32;
    static constexpr int kThreads = (kConsumers + 1) * 32;   // + the producer
    static constexpr int kYRow = kCols * 2;
    static constexpr int kY = 16 * kYRow, kStage = kY + 16 * 64 * S;   // Y, then T rows of 4 R bytes
    static constexpr int kStages = S == 1 ? 5 : 3;
    static constexpr int kBTile = kCols * 32 * S;
    static constexpr int kBStages = S == 1 ? 3 : 2;
    static constexpr int kRing = kStages * kStage;
    static constexpr size_t smem = (size_t)kRing + kBStages * kBTile;
    // parts that can be filled ahead of T, each with a B of its own
    static constexpr int kAhead = kStages < kBStages ? kStages : kBStages;
};

// What a part is: its tokens (run: consecutive ones, box: 16 of those),
// whether its adapter's B is new, whether it has no adapter (Y is copied),
// whether it is the end of the list.
struct __align__(16) Part {
    int rows[16];
    int ntok, new_b, plain, end;
    int run, box;
};

// The parts of one block of tokens.
struct PartTable {
    int adapter[kBlockTok];
    uint8_t ntok[kBlockTok];
    uint8_t rows[kBlockTok][16];   // offsets in the block, rising
};

// Fills the table (one warp); returns the number of parts.  Every token finds
// its place at once, from the masks of its group and a sum over the groups
// before it: a walk through the groups costs a lone warp a microsecond a part.
__device__ __forceinline__ int list_parts(const Groups &g, PartTable &tab, bool skip_plain, int lane)
{
    const u64 below0 = (1ull << lane) - 1, below1 = (1ull << (lane + 32)) - 1;
    const int cnt0 = __popcll(g.of0), cnt1 = __popcll(g.of1);
    const bool lead0 = g.leaders >> lane & 1, lead1 = g.leaders >> (lane + 32) & 1;
    const int n0 = lead0 && !(skip_plain && g.a0 < 0) ? (cnt0 + 15) / 16 : 0;
    const int n1 = lead1 && !(skip_plain && g.a1 < 0) ? (cnt1 + 15) / 16 : 0;
    int s0 = n0, s1 = n1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u0 = __shfl_up_sync(0xffffffffu, s0, o), u1 = __shfl_up_sync(0xffffffffu, s1, o);
        if (lane >= o) {
            s0 += u0;
            s1 += u1;
        }
    }
    const int total0 = __shfl_sync(0xffffffffu, s0, 31);
    const int first0 = s0 - n0, first1 = total0 + s1 - n1;   // of the groups these lanes lead
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const u64 of = h ? g.of1 : g.of0;
        const int a = h ? g.a1 : g.a0;
        const int lead = of ? __ffsll(of) - 1 : 0;
        const int f0 = __shfl_sync(0xffffffffu, first0, lead & 31);
        const int f1 = __shfl_sync(0xffffffffu, first1, lead & 31);
        const int first = lead < 32 ? f0 : f1;
        if (a == -2 || (skip_plain && a < 0))
            continue;
        const int rank = __popcll(of & (h ? below1 : below0));
        tab.rows[first + rank / 16][rank % 16] = (uint8_t)(lane + 32 * h);
        if (rank % 16 == 0) {
            tab.adapter[first + rank / 16] = a;
            tab.ntok[first + rank / 16] = (uint8_t)min(16, __popcll(of) - rank);
        }
    }
    __syncwarp();
    return total0 + __shfl_sync(0xffffffffu, s1, 31);
}

template <int S>
__global__ void __launch_bounds__(Expand<S>::kThreads, S <= 2 ? 3 : (S == 4 ? 2 : 1))
    lora_expand_kernel(const __grid_constant__ CUtensorMap y_map, const LoraParams p, int blocks,
                       int subs)
{
    using C = Expand<S>;
    __shared__ Part parts[C::kStages];
    __shared__ uint64_t full[C::kStages], empty[C::kStages];
    __shared__ uint64_t b_empty[C::kBStages];
    __shared__ PartTable table;
    __shared__ u64 masks[kBlockTok];
    extern __shared__ __align__(128) uint8_t dyn[];
    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const int n0 = blockIdx.x * C::kCols;
    const int cols = min(C::kCols, p.N - n0);
    const int quads = p.R / 4;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], C::kConsumers);
        }
        for (int i = 0; i < C::kBStages; ++i)
            mbar_init(&b_empty[i], C::kConsumers);
        fence_barrier_init();
    }
    // the first block's index, grouped by all warps where that is work and
    // the CTA has no other block
    int block, block_end, sub = 0;
    if (subs > 1) {
        block = blocks == 1 ? 0 : blockIdx.y % blocks;
        block_end = block + 1;
        sub = blocks == 1 ? blockIdx.y : blockIdx.y / blocks;
    } else {
        // (blocks < 2^15 and a few hundred CTAs: 32 bits)
        block = (int)(blockIdx.y * (unsigned)blocks / gridDim.y);
        block_end = (int)((blockIdx.y + 1) * (unsigned)blocks / gridDim.y);
    }
    int raw0, raw1;
    auto peek = [&](int b) {
        const int m = b * kBlockTok + lane;
        const int end = b < block_end ? min(p.M, (b + 1) * kBlockTok) : 0;
        raw0 = m < end ? __ldcg(p.index + m) : -1;
        raw1 = m + 32 < end ? __ldcg(p.index + m + 32) : -1;
    };
    Groups grp{};
    bool grouped = subs > 1 && p.M - block * kBlockTok > 32;
    if (grouped) {
        peek(block);
        grp = group_tokens_cta(raw0, raw1, min(kBlockTok, p.M - block * kBlockTok), p.L, lane, warp,
                               masks);
    } else {
        __syncthreads();
    }
    pdl_launch_dependents();
    // by whole warps; once a wait has run out the role goes to its end
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity, int where) {
        if (!ok || __all_sync(0xffffffffu, mbar_test(bar, parity)))
            return;
        ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, kWaitLimitNs));
        if (!ok && lane == 0)
            record_timeout(p.hdr, where);
    };

    if (warp == C::kConsumers) {
        // ------------------------------------------------------- producer
        if (!grouped)
            peek(block);
        const bool in_place = p.Out == p.Y;
        const uint64_t pol_once = l2_policy_evict_first(), pol_keep = l2_policy_evict_last();
        int slot = 0, b_slot = 0;
        uint32_t phase = 1, b_phase = 1;     // of the empty barriers: the first round is free
        auto copy_t = [&](int s) {
            const Part &q = parts[s];
            const int i = lane - 16;
            if (q.plain || i < 0 || i >= (q.run ? 1 : q.ntok))
                return;
            bulk_g2s(dyn + s * C::kStage + C::kY + i * quads * 16,
                     p.T + (size_t)q.rows[i] * quads, (q.run ? q.ntok : 1) * quads * 16, &full[s],
                     pol_keep);
        };
        bool waited = false;
        int before = 0;   // stages filled ahead of the wait: their T comes after it
        auto wait_shrink = [&]() {
            // T is the shrink kernel's.  Without any part too: this kernel must
            // not complete before that one, whose inputs the next on the
            // stream may change
            pdl_wait();
            waited = true;
            for (int s = 0; s < before; ++s)
                copy_t(s);
        };
        bool wrapped = false, b_wrapped = false;
        int a_last = -1;
        for (; block < block_end && ok; ++block) {
            const int m0 = block * kBlockTok;
            // a whole block of one adapter (a prefill chunk's) needs no list
            const int a0 = __shfl_sync(0xffffffffu, raw0, 0);
            const bool one =
                m0 + kBlockTok <= p.M && __all_sync(0xffffffffu, raw0 == a0 && raw1 == a0);
            int nparts;
            if (one) {
                nparts = (a0 < 0 || a0 >= p.L) && in_place ? 0 : kBlockTok / 16;
            } else {
                if (!grouped)
                    grp = group_tokens(raw0, raw1, min(kBlockTok, p.M - m0), p.L, lane);
                __syncwarp();
                nparts = list_parts(grp, table, in_place, lane);
            }
            grouped = false;
            peek(block + 1);   // ahead of its use
            for (int i = sub; i < nparts; i += subs) {
                if (!waited && before == C::kAhead)
                    wait_shrink();
                int a = a0 < p.L ? a0 : -1, n = 16, first = m0 + 16 * i, mine = first + lane;
                bool run = true;
                if (!one) {
                    a = table.adapter[i];
                    n = table.ntok[i];
                    first = m0 + table.rows[i][0];
                    mine = m0 + table.rows[i][lane < n ? lane : 0];
                    run = m0 + table.rows[i][n - 1] - first == n - 1;
                }
                const bool box = run && n == 16;
                const bool new_b = a >= 0 && a != a_last;
                // (a test of a barrier takes 150 cycles: none in the first round)
                if (wrapped)
                    wait(&empty[slot], phase, 501);
                if (new_b && b_wrapped)
                    wait(&b_empty[b_slot], b_phase, 502);
                if (!ok)
                    break;
                Part &q = parts[slot];
                if (lane < 16)
                    q.rows[lane] = mine;
                if (lane == 0) {
                    *reinterpret_cast<int4 *>(&q.ntok) = make_int4(n, new_b, a < 0, 0);
                    q.run = run;
                    q.box = box;
                }
                __syncwarp();
                // a box is written whole: zeros stand for its columns past the end
                if (lane == 0)
                    mbar_arrive_expect_tx(&full[slot],
                                          n * ((box ? C::kCols : cols) * 2 +
                                               (a < 0 ? 0 : quads * 16)) +
                                              (new_b ? cols * p.R * 2 : 0));
                __syncwarp();
                // index, B and Y precede the shrink kernel's own wait: they are
                // read ahead of this kernel's
                if (new_b) {
                    a_last = a;
                    if (lane == 0)
                        bulk_g2s(dyn + C::kRing + b_slot * C::kBTile,
                                 p.B + ((size_t)a * p.N + n0) * p.R, cols * p.R * 2, &full[slot],
                                 pol_keep);
                    if (++b_slot == C::kBStages) {
                        b_slot = 0;
                        b_phase ^= 1;
                        b_wrapped = true;
                    }
                }
                if (box) {
                    if (lane == 0)
                        tma_load_2d(dyn + slot * C::kStage, &y_map, n0, first, &full[slot],
                                    pol_once);
                } else if (lane < n) {
                    bulk_g2s(dyn + slot * C::kStage + lane * C::kYRow, p.Y + mine * p.ldy + n0,
                             cols * 2, &full[slot], pol_once);
                }
                if (waited)
                    copy_t(slot);
                else
                    ++before;
                if (++slot == C::kStages) {
                    slot = 0;
                    phase ^= 1;
                    wrapped = true;
                }
            }
        }
        if (!waited)
            wait_shrink();
        if (ok && wrapped)
            wait(&empty[slot], phase, 503);
        if (ok) {
            // the end of the list
            if (lane == 0) {
                parts[slot].end = 1;
                parts[slot].ntok = 0;
                mbar_arrive(&full[slot]);
            }
        } else {
            // no role works on: every copy issued here has landed before the
            // CTA exits (otherwise the consumers wait for each of them)
            for (int s = 0; s < C::kStages; ++s)
                if (s < slot || wrapped)
                    mbar_wait(&full[s], s < slot ? phase ^ 1 : phase, kWaitLimitNs);
        }
    } else {
        // ------------------------------------------------------- consumers
        const int g = lane >> 2, t = lane & 3;
        uint32_t b[4][S][2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int s = 0; s < S; ++s)
                b[i][s][0] = b[i][s][1] = 0;
        uint32_t b_seen = 0;   // an infinity or NaN in this lane's B
        const uint32_t base = smem_u32(dyn);
        const int ncol = n0 + warp * 32 + 8 * t;
        const bool col_in = ncol < p.N;
        const uint32_t yoff = g * C::kYRow + warp * 64 + t * 16, toff = C::kY + g * quads * 16;
        int slot = 0, b_slot = 0;
        uint32_t phase = 0;
        while (true) {
            wait(&full[slot], phase, 521);
            const int4 q = *reinterpret_cast<const int4 *>(&parts[slot].ntok);
            if (!ok || q.w)   // end
                break;
            const uint32_t st = base + slot * C::kStage;
            const int2 row = make_int2(g < q.x ? parts[slot].rows[g] : -1,
                                       g + 8 < q.x ? parts[slot].rows[g + 8] : -1);
            uint32_t w[2][4];
            auto load_y = [&] {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint4 y = lds128a(st + yoff + 8 * r * C::kYRow);
                    w[r][0] = y.x;
                    w[r][1] = y.y;
                    w[r][2] = y.z;
                    w[r][3] = y.w;
                }
            };
            load_y();
            if (q.y) {   // new B
                // column (row of B) and ranks of this lane.  S = 1: four
                // consecutive ranks 4 t; else eight, 32 q + 8 t, for two steps
                const uint32_t tile = base + C::kRing + b_slot * C::kBTile;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t brow =
                        tile + (warp * 32 + 8 * (g >> 1) + 2 * i + (g & 1)) * p.R * 2;
                    if constexpr (S == 1) {
                        const uint2 v = 4 * t < p.R ? lds64a(brow + 8 * t) : make_uint2(0u, 0u);
                        b[i][0][0] = v.x;
                        b[i][0][1] = v.y;
                    } else {
#pragma unroll
                        for (int h = 0; h < S / 2; ++h) {
                            const uint4 v = 32 * h + 8 * t < p.R ? lds128a(brow + 64 * h + 16 * t)
                                                                 : make_uint4(0u, 0u, 0u, 0u);
                            b[i][2 * h][0] = v.x;
                            b[i][2 * h][1] = v.y;
                            b[i][2 * h + 1][0] = v.z;
                            b[i][2 * h + 1][1] = v.w;
                        }
                    }
                }
                b_seen = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (warp * 32 + 8 * (g >> 1) + 2 * i + (g & 1) < cols)   // else not B's
#pragma unroll
                        for (int s = 0; s < S; ++s) {
                            note_nonfinite(b_seen, b[i][s][0]);
                            note_nonfinite(b_seen, b[i][s][1]);
                        }
            }
            if (!q.z) {   // with an adapter
                float acc[4][4];
                uint32_t seen = b_seen;   // an infinity or NaN in B or T
                auto multiply = [&](auto careful) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            acc[i][e] = __uint_as_float(e & 1 ? w[e >> 1][i] & 0xFFFF0000u
                                                              : w[e >> 1][i] << 16);
#pragma unroll
                    for (int s = 0; s < S; ++s) {
                        const int r4 = S == 1 ? t : 8 * (s / 2) + 2 * t + (s & 1);   // rank / 4
                        uint4 ta = make_uint4(0u, 0u, 0u, 0u), tb = ta;
                        if (r4 < quads && row.x >= 0)
                            ta = lds128a(st + toff + 16 * r4);
                        if (r4 < quads && row.y >= 0)
                            tb = lds128a(st + toff + (8 * quads + r4) * 16);
                        if (decltype(careful)::value) {
                            lift(ta);
                            lift(tb);
                        }
                        Split u = split_f32(ta), v = split_f32(tb);
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if (decltype(careful)::value) {
                                drop_rest(u, h);
                                drop_rest(v, h);
                            } else {
                                note_nonfinite(seen, u.hi[h]);
                                note_nonfinite(seen, v.hi[h]);
                            }
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mma_bf16_16816(acc[i], u.hi[0], v.hi[0], u.hi[1], v.hi[1], b[i][s][0],
                                           b[i][s][1]);
                        // an infinity in B times `hi` is the product: 0 or a
                        // rest of the other sign would make it NaN
                        uint32_t bf[4][2];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                bf[i][h] = decltype(careful)::value
                                               ? b[i][s][h] & finite_mask(b[i][s][h])
                                               : b[i][s][h];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mma_bf16_16816(acc[i], u.mid[0], v.mid[0], u.mid[1], v.mid[1], bf[i][0],
                                           bf[i][1]);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mma_bf16_16816(acc[i], u.lo[0], v.lo[0], u.lo[1], v.lo[1], bf[i][0],
                                           bf[i][1]);
                    }
                };
                multiply(std::false_type());
                if (__any_sync(0xffffffffu, seen != 0)) {   // rare: once more, with care
                    load_y();
                    multiply(std::true_type());
                }
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w[r][i] = pack_bf16(acc[i][2 * r], acc[i][2 * r + 1]);
            }
            // every lane's reads of the stage have returned: it is free
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&empty[slot]);
                if (q.y)
                    mbar_arrive(&b_empty[b_slot]);
            }
            if (q.y && ++b_slot == C::kBStages)
                b_slot = 0;
            if (col_in && row.x >= 0)
                *reinterpret_cast<uint4 *>(p.Out + row.x * p.ldo + ncol) =
                    make_uint4(w[0][0], w[0][1], w[0][2], w[0][3]);
            if (col_in && row.y >= 0)
                *reinterpret_cast<uint4 *>(p.Out + row.y * p.ldo + ncol) =
                    make_uint4(w[1][0], w[1][1], w[1][2], w[1][3]);
            if (++slot == C::kStages) {
                slot = 0;
                phase ^= 1;
            }
        }
    }
}

// Attributes a kernel launch needs, set once per device.
cudaError_t allow_smem(const void *fn, std::atomic<bool> (&done)[kMaxDeviceCache], size_t smem)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= kMaxDeviceCache)
        return cudaErrorInvalidDevice;
    if (!done[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess)
            return e;
        done[dev].store(true, std::memory_order_release);
    }
    return cudaSuccess;
}

template <int RT>
cudaError_t launch_shrink(const LoraPlan &pl, const LoraParams &p, cudaStream_t stream)
{
    using C = Shrink<RT>;
    const void *fn = reinterpret_cast<const void *>(&lora_shrink_kernel<RT>);
    static std::atomic<bool> done[kMaxDeviceCache];
    const cudaError_t e = allow_smem(fn, done, C::smem);
    if (e != cudaSuccess)
        return e;
    // boxes of 64 k: a slice's ranks of A, 16 tokens or one of X (which only
    // groups of more than 16 tokens use)
    alignas(64) CUtensorMap xm{}, xr{}, am{};
    if (!encode_tensor_map_2d(&am, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.A, (uint64_t)p.K,
                              (uint64_t)p.L * p.R, (uint64_t)p.K * 2, 64,
                              (uint32_t)pl.slice_ranks, CU_TENSOR_MAP_SWIZZLE_128B) ||
        (p.M > kFew &&
         (!encode_tensor_map_2d(&xm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.X, (uint64_t)p.K,
                                (uint64_t)p.M, (uint64_t)p.ldx * 2, 64, 16,
                                CU_TENSOR_MAP_SWIZZLE_128B) ||
          !encode_tensor_map_2d(&xr, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.X, (uint64_t)p.K,
                                (uint64_t)p.M, (uint64_t)p.ldx * 2, 64, 1,
                                CU_TENSOR_MAP_SWIZZLE_128B))))
        return cudaErrorInvalidValue;
    LoraParams q = p;
    int slices = pl.slices, ranks = pl.slice_ranks;
    void *args[] = {&xm, &xr, &am, &q, &slices, &ranks};
    return launch_pdl_cluster(fn, dim3(pl.cluster, pl.shrink_subs, pl.blocks * pl.slices),
                              dim3(C::kThreads), pl.cluster, C::smem, stream, args);
}

template <int S>
cudaError_t launch_expand(const LoraPlan &pl, const LoraParams &p, cudaStream_t stream)
{
    const void *fn = reinterpret_cast<const void *>(&lora_expand_kernel<S>);
    static std::atomic<bool> done[kMaxDeviceCache];
    const cudaError_t e = allow_smem(fn, done, Expand<S>::smem);
    if (e != cudaSuccess)
        return e;
    // boxes of 16 tokens x 256 columns (a batch of fewer tokens has none)
    alignas(64) CUtensorMap ym{};
    if (p.M >= 16 &&
        !encode_tensor_map_2d(&ym, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.Y, (uint64_t)p.N,
                              (uint64_t)p.M, (uint64_t)p.ldy * 2, Expand<S>::kCols, 16,
                              CU_TENSOR_MAP_SWIZZLE_NONE))
        return cudaErrorInvalidValue;
    LoraParams q = p;
    int blocks = pl.blocks, subs = pl.expand_subs;
    void *args[] = {&ym, &q, &blocks, &subs};
    return launch_pdl(fn, dim3(pl.ntiles, pl.expand_shares), dim3(Expand<S>::kThreads),
                      Expand<S>::smem, stream, args);
}

}  // namespace

bool lora_shape_ok(int M, int N, int K, int R)
{
    // blocks (times two rank slices) are a grid dimension of at most 65535
    return M >= 1 && M <= 32767 * kBlockTok && N >= 8 && K >= 8 && R >= 8 && R <= 128 &&
           N % 8 == 0 && K % 8 == 0 && R % 8 == 0;
}

size_t lora_scratch_bytes(int M, int R)
{
    return sizeof(WsHeader) + (size_t)M * R * 4;
}

LoraPlan plan_lora(int device, int M, int N, int K, int R)
{
    const int sms = device_info(device).sms;
    LoraPlan pl{};
    const long long blocks = ((long long)M + kBlockTok - 1) / kBlockTok;
    // ranks above 64 in two slices
    pl.slices = R <= 64 ? 1 : 2;
    pl.slice_ranks = R <= 64 ? R : (R / 2 + 7) / 8 * 8;
    pl.rank_tiles = pl.slice_ranks <= 16 ? 1 : (pl.slice_ranks <= 32 ? 2 : 4);
    pl.blocks = (int)blocks;
    const int tok = std::min(M, kBlockTok);
    // shrink: K is split over a cluster while the blocks alone leave room (two
    // CTAs fit on an SM; clusters of eight do not fill every SM of a GPC, so an
    // eighth of that is left out), at least four stages of 64 k a CTA
    const int room = 2 * sms * 7 / 8;
    pl.cluster = 1;
    while (pl.cluster < 8 && 2 * pl.cluster * blocks * pl.slices <= room &&
           2 * pl.cluster * 256 <= K)
        pl.cluster *= 2;
    // groups of a block run side by side in what room is left: the host does
    // not know how many there are, and a share without any ends at once
    const long long shrink_ctas = blocks * pl.slices * pl.cluster;
    pl.shrink_subs = (int)std::max<long long>(1, std::min<long long>(tok, room / shrink_ctas));
    // expand: one wave of CTAs; they share the blocks out, or, with fewer
    // blocks than that, each block's groups
    const int steps = (R + 15) / 16;
    pl.expand_steps = steps <= 2 ? steps : (steps <= 4 ? 4 : 8);
    pl.ntiles = (N + 255) / 256;
    const int fit = pl.expand_steps <= 2 ? 3 : (pl.expand_steps == 4 ? 2 : 1);   // CTAs an SM
    const int shares = std::max(1, fit * sms / pl.ntiles);
    if (shares <= blocks) {
        pl.expand_subs = 1;
        pl.expand_shares = shares;
    } else {
        pl.expand_subs = std::min(tok, (int)(shares / blocks));
        pl.expand_shares = (int)(pl.expand_subs * blocks);
    }
    return pl;
}

cudaError_t lora_error_header(void **header)
{
    return cudaGetSymbolAddress(header, g_lora_errors);
}

cudaError_t launch_lora_wait_timeout(int limit_us, cudaStream_t stream)
{
    lora_wait_timeout_kernel<<<1, 32, 0, stream>>>((unsigned long long)limit_us * 1000ull);
    return cudaGetLastError();
}

cudaError_t launch_lora(const LoraPlan &pl, const LoraArgs &a, cudaStream_t stream)
{
    LoraParams p{};
    p.X = static_cast<const uint16_t *>(a.X);
    p.A = static_cast<const uint16_t *>(a.A);
    p.B = static_cast<const uint16_t *>(a.B);
    p.Y = static_cast<const uint16_t *>(a.Y);
    p.Out = static_cast<uint16_t *>(a.Out);
    p.scales = a.scales;
    p.index = a.index;
    p.hdr = static_cast<WsHeader *>(a.workspace);
    p.T = reinterpret_cast<float4 *>(p.hdr + 1);
    p.ldx = a.ldx;
    p.ldy = a.ldy;
    p.ldo = a.ldo;
    p.M = a.M;
    p.N = a.N;
    p.K = a.K;
    p.R = a.R;
    p.L = a.L;
    cudaError_t e;
    if (pl.rank_tiles == 1)
        e = launch_shrink<1>(pl, p, stream);
    else if (pl.rank_tiles == 2)
        e = launch_shrink<2>(pl, p, stream);
    else
        e = launch_shrink<4>(pl, p, stream);
    if (e != cudaSuccess)
        return e;
    switch (pl.expand_steps) {
    case 1: return launch_expand<1>(pl, p, stream);
    case 2: return launch_expand<2>(pl, p, stream);
    case 4: return launch_expand<4>(pl, p, stream);
    default: return launch_expand<8>(pl, p, stream);
    }
}

}  // namespace mxg
