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
// HBM bytes bound a large batch and launch latency a small one; the
// mma.sync tensor path is never the limit, and reading operands straight
// into its fragments needs no staging.
//
// Two kernels, joined by programmatic dependent launch:
//   shrink   T = s * X A^T, [M][R] in fp32, kept as two bf16 halves
//            (T = hi + lo, 16 bits of mantissa at least: the inner product
//            is not rounded to bf16 on its way);
//   expand   Out = Y + T B^T, summed in fp32 and rounded once.
//
// Tokens come in any order.  Both kernels take blocks of 64 consecutive
// tokens and group a block's tokens by adapter in shared memory (a few
// hundred cycles; no sort kernel, no host plan, nothing read back), so an
// adapter is read once per block that uses it and once in all for a decode
// batch.
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "kernels.h"

namespace mxg {
namespace {

constexpr int kBlockTok = 64;     // tokens grouped together
constexpr int kShrinkWarps = 8;   // warps that split K in a shrink CTA

struct LoraParams {
    const uint16_t *X, *A, *B, *Y;   // bf16
    uint16_t *Out;
    const float *scales;     // [L] or NULL (all 1)
    const int *index;        // [M]
    uint4 *T;                // [M][R / 4]: four hi halves, then four lo halves
    long long ldx, ldy, ldo; // row strides in elements
    int M, N, K, R, L;
};

// 16-byte load that bypasses L1 (adapters are read once per CTA).
__device__ __forceinline__ uint4 ldg128_once(const void *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// -------------------------------------------------------- tokens by adapter
struct Groups {
    int adapter[kBlockTok];          // per token of the block (-1: none)
    int group[kBlockTok];            // its group, numbered by first token
    int g_adapter[kBlockTok];        // per group
    int g_begin[kBlockTok + 1];      // its tokens are list[g_begin .. next g_begin)
    short list[kBlockTok];           // token offsets in the block, by group
    unsigned leaders[2];             // bit per token: the first of its group
};

// Groups the block's `ntok` tokens; returns the number of groups.  Called by
// every thread of a CTA of at least 64.
__device__ __forceinline__ int group_tokens(Groups &s, const int *index, int ntok, int L)
{
    const int i = threadIdx.x;
    if (i < kBlockTok) {
        const int a = i < ntok ? __ldcg(index + i) : -1;
        s.adapter[i] = a >= 0 && a < L ? a : -1;
    }
    __syncthreads();
    if (i < kBlockTok) {
        const int a = s.adapter[i];
        int first = i;
        for (int j = ntok - 1; j >= 0; --j)
            if (s.adapter[j] == a)
                first = j;
        s.group[i] = first;   // token that leads the group, renumbered below
        const unsigned lead = __ballot_sync(0xffffffffu, i < ntok && first == i);
        if ((i & 31) == 0)
            s.leaders[i >> 5] = lead;
    }
    __syncthreads();
    const unsigned lo = s.leaders[0], hi = s.leaders[1];
    int grp = -1;
    if (i < ntok) {
        const int f = s.group[i];
        grp = f < 32 ? __popc(lo & ((1u << f) - 1)) : __popc(lo) + __popc(hi & ((1u << (f - 32)) - 1));
        if (f == i)
            s.g_adapter[grp] = s.adapter[i];
    }
    __syncthreads();
    if (i < ntok)
        s.group[i] = grp;
    __syncthreads();
    if (i < ntok) {
        int before = 0, rank = 0;   // tokens of earlier groups; earlier tokens of this one
        for (int j = 0; j < ntok; ++j) {
            const int gj = s.group[j];
            before += gj < grp;
            rank += gj == grp && j < i;
        }
        s.list[before + rank] = (short)i;
        if (rank == 0)
            s.g_begin[grp] = before;
    }
    const int ngroups = __popc(lo) + __popc(hi);
    if (i == 0)
        s.g_begin[ngroups] = ntok;
    __syncthreads();
    return ngroups;
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

// fp32 v = hi + lo in bf16; a value without a finite hi has no lo.
__device__ __forceinline__ void split_bf16(float v, uint32_t &hi, uint32_t &lo)
{
    hi = f32_to_bf16_bits(v);
    const float back = __uint_as_float(hi << 16);
    const float rest = v - back;
    lo = (hi & 0x7F80u) == 0x7F80u ? 0u : f32_to_bf16_bits(rest);
}

// ------------------------------------------------------------------- shrink
// One cluster per (block of tokens, share of its groups, slice of 16 RT
// ranks); its CTAs split K, and each CTA's warps split that again in units of
// 32: a lane loads 16 bytes (eight k) per row, so the fragments of two
// m16n8k16 MMAs (ranks as the 16 rows, tokens as the 8 columns) come straight
// from global memory, X and A in the same k order.  Warps are added through
// shared memory and CTAs through distributed shared memory in a fixed order
// (bitwise reproducible; no atomics, no second pass over partial sums).
// 8 NT tokens of one adapter run together, so A is read once for them.
template <int RT, int NT>
__global__ void __launch_bounds__(kShrinkWarps * 32, 2) lora_shrink_kernel(const LoraParams p)
{
    constexpr int CT = 8 * NT;        // tokens per chunk
    constexpr int ST = 16 * RT + 4;   // row stride of the reduced tile (floats)
    __shared__ Groups grp;
    extern __shared__ float4 red[];   // [warps][RT * NT][32], then the CTA's tile
    float *tile = reinterpret_cast<float *>(red + kShrinkWarps * RT * NT * 32);   // [CT][ST]

    // The dependent launch is allowed only after this wait: the expand kernel
    // may then read the index, B and Y before its own wait, since everything
    // queued before this kernel has completed.
    pdl_wait();
    pdl_launch_dependents();

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int nslices = (p.R + 16 * RT - 1) / (16 * RT);
    const int block = blockIdx.z / nslices, slice = blockIdx.z % nslices;
    const int m0 = block * kBlockTok;
    const int ngroups = group_tokens(grp, p.index + m0, min(kBlockTok, p.M - m0), p.L);
    const int crank = (int)cluster_rank(), csize = (int)cluster_size();
    const int units = (p.K + 31) / 32;
    const int u0 = (int)((long long)crank * units / csize);
    const int u1 = (int)((long long)(crank + 1) * units / csize);
    const int r0 = slice * 16 * RT;

    int n = 0;   // chunks seen so far: this cluster takes every gridDim.y-th
    for (int gi = 0; gi < ngroups; ++gi) {
        const int a = grp.g_adapter[gi];
        if (a < 0)
            continue;
        const int end = grp.g_begin[gi + 1];
        for (int begin = grp.g_begin[gi]; begin < end; begin += CT, ++n) {
            if (n % gridDim.y != blockIdx.y)
                continue;
            const int ntok = min(CT, end - begin);
            const int nt_live = (ntok + 7) / 8;
            float acc[RT][NT][4];
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[i][j][e] = 0.f;
            // this lane's rows: ranks g and g + 8 of every rank tile, token
            // g of every token tile (absent ones stay zero)
            const uint16_t *xrow[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int slot = 8 * j + g;
                xrow[j] = slot < ntok ? p.X + (m0 + grp.list[begin + slot]) * p.ldx : nullptr;
            }
            const uint16_t *abase = p.A + (size_t)a * p.R * p.K + (size_t)(r0 + g) * p.K;
#pragma unroll 2
            for (int u = u0 + warp; u < u1; u += kShrinkWarps) {
                const int k = 32 * u + 8 * t;
                const bool in = k < p.K;
                uint4 av[RT][2], xv[NT];
#pragma unroll
                for (int i = 0; i < RT; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        av[i][h] = make_uint4(0u, 0u, 0u, 0u);
                        if (in && r0 + 16 * i + 8 * h + g < p.R)
                            av[i][h] = ldg128_once(abase + (size_t)(16 * i + 8 * h) * p.K + k);
                    }
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    xv[j] = make_uint4(0u, 0u, 0u, 0u);
                    if (in && xrow[j])
                        xv[j] = ldg128(xrow[j] + k);
                }
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    if (j < nt_live)
#pragma unroll
                        for (int i = 0; i < RT; ++i) {
                            mma_bf16_16816(acc[i][j], av[i][0].x, av[i][1].x, av[i][0].y,
                                           av[i][1].y, xv[j].x, xv[j].y);
                            mma_bf16_16816(acc[i][j], av[i][0].z, av[i][1].z, av[i][0].w,
                                           av[i][1].w, xv[j].z, xv[j].w);
                        }
            }
            // ---- add the warps, in warp order
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    if (j < nt_live)
                        red[((warp * NT + j) * RT + i) * 32 + lane] =
                            make_float4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
            __syncthreads();
            for (int e = threadIdx.x; e < nt_live * RT * 32; e += kShrinkWarps * 32) {
                float4 s = red[e];
#pragma unroll
                for (int w = 1; w < kShrinkWarps; ++w) {
                    const float4 v = red[w * NT * RT * 32 + e];
                    s.x += v.x;
                    s.y += v.y;
                    s.z += v.z;
                    s.w += v.w;
                }
                const int l = e & 31, i = (e >> 5) % RT, j = (e >> 5) / RT;
                const int r = 16 * i + (l >> 2), c = 8 * j + 2 * (l & 3);
                tile[c * ST + r] = s.x;
                tile[(c + 1) * ST + r] = s.y;
                tile[c * ST + r + 8] = s.z;
                tile[(c + 1) * ST + r + 8] = s.w;
            }
            cluster_barrier();
            // ---- add the CTAs of the cluster in rank order: every CTA
            // finishes a share of the (token, four ranks) entries
            const int quads = min(16 * RT, p.R - r0) / 4;
            const float sc = p.scales ? __ldg(p.scales + a) : 1.f;
            for (int e = threadIdx.x * csize + crank; e < ntok * quads;
                 e += kShrinkWarps * 32 * csize) {
                const int c = e / quads, q = e % quads;
                const float *mine = tile + c * ST + 4 * q;
                float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int w = 0; w < csize; ++w) {
                    const float4 v = ld_peer_f4(mine, w);
                    s.x += v.x;
                    s.y += v.y;
                    s.z += v.z;
                    s.w += v.w;
                }
                uint32_t hi[4], lo[4];
                split_bf16(s.x * sc, hi[0], lo[0]);
                split_bf16(s.y * sc, hi[1], lo[1]);
                split_bf16(s.z * sc, hi[2], lo[2]);
                split_bf16(s.w * sc, hi[3], lo[3]);
                p.T[(size_t)(m0 + grp.list[begin + c]) * (p.R / 4) + r0 / 4 + q] =
                    make_uint4(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16),
                               lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
            }
            cluster_barrier();   // the tiles are read before the next chunk's
        }
    }
}

// ------------------------------------------------------------------- expand
// One warp per 32 columns and (block of tokens, share of its groups): the
// rows of B for its columns stay in registers as MMA operands while the
// group's tokens pass, 16 at a time (tokens as the 16 rows, columns as the 8
// of four MMAs).  Column c of MMA i is column 8 (c / 2) + 2 i + c % 2 of the
// warp's 32, so a lane's results are eight consecutive columns and Y and Out
// move 16 bytes a lane, 64 contiguous bytes a row.  S = 16-rank steps.
template <int S>
__global__ void __launch_bounds__(256) lora_expand_kernel(const LoraParams p)
{
    __shared__ Groups grp;
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int m0 = blockIdx.z * kBlockTok;
    // index, B and Y precede the shrink kernel's own wait: readable now
    const int ngroups = group_tokens(grp, p.index + m0, min(kBlockTok, p.M - m0), p.L);
    const int n0 = (blockIdx.x * (blockDim.x >> 5) + warp) * 32;
    const int ncol = n0 + 8 * t;          // first of this lane's eight columns
    const bool col_in = ncol < p.N;
    const int quads = p.R / 4;
    bool waited = false;

    for (int gi = blockIdx.y; gi < ngroups; gi += gridDim.y) {
        const int a = grp.g_adapter[gi];
        const int begin = grp.g_begin[gi], end = grp.g_begin[gi + 1];
        if (a < 0) {
            if (p.Out == p.Y)
                continue;
            if (!waited)
                pdl_wait();
            waited = true;
            for (int o = begin + g; o < end; o += 8) {
                const long long m = m0 + grp.list[o];
                if (col_in)
                    *reinterpret_cast<uint4 *>(p.Out + m * p.ldo + ncol) =
                        __ldcg(reinterpret_cast<const uint4 *>(p.Y + m * p.ldy + ncol));
            }
            continue;
        }
        // B operands: column (row of B) and ranks of this lane.  S = 1: four
        // consecutive ranks 4 t; else eight, 32 q + 8 t, for two steps
        uint32_t b[4][S][2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = n0 + 8 * (g >> 1) + 2 * i + (g & 1);
            const uint16_t *row = p.B + ((size_t)a * p.N + n) * p.R;
            if constexpr (S == 1) {
                uint2 v = make_uint2(0u, 0u);
                if (n < p.N && 4 * t < p.R)
                    v = __ldcg(reinterpret_cast<const uint2 *>(row + 4 * t));
                b[i][0][0] = v.x;
                b[i][0][1] = v.y;
            } else {
#pragma unroll
                for (int q = 0; q < S / 2; ++q) {
                    uint4 v = make_uint4(0u, 0u, 0u, 0u);
                    if (n < p.N && 32 * q + 8 * t < p.R)
                        v = ldg128_once(row + 32 * q + 8 * t);
                    b[i][2 * q][0] = v.x;
                    b[i][2 * q][1] = v.y;
                    b[i][2 * q + 1][0] = v.z;
                    b[i][2 * q + 1][1] = v.w;
                }
            }
        }
        for (int o = begin; o < end; o += 16) {
            const bool in0 = o + g < end, in1 = o + g + 8 < end;
            const long long ma = in0 ? m0 + grp.list[o + g] : 0;
            const long long mb = in1 ? m0 + grp.list[o + g + 8] : 0;
            uint4 ya = make_uint4(0u, 0u, 0u, 0u), yb = ya;
            if (in0 && col_in)
                ya = __ldcg(reinterpret_cast<const uint4 *>(p.Y + ma * p.ldy + ncol));
            if (in1 && col_in)
                yb = __ldcg(reinterpret_cast<const uint4 *>(p.Y + mb * p.ldy + ncol));
            if (!waited)
                pdl_wait();   // T is the shrink kernel's
            waited = true;
            float acc[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[i][e] = 0.f;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const int q = S == 1 ? t : 8 * (s / 2) + 2 * t + (s & 1);   // rank / 4
                uint4 ta = make_uint4(0u, 0u, 0u, 0u), tb = ta;
                if (q < quads) {
                    if (in0)
                        ta = __ldcg(p.T + ma * quads + q);
                    if (in1)
                        tb = __ldcg(p.T + mb * quads + q);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    mma_bf16_16816(acc[i], ta.x, tb.x, ta.y, tb.y, b[i][s][0], b[i][s][1]);
                    mma_bf16_16816(acc[i], ta.z, tb.z, ta.w, tb.w, b[i][s][0], b[i][s][1]);
                }
            }
            const uint32_t y0[4] = {ya.x, ya.y, ya.z, ya.w}, y1[4] = {yb.x, yb.y, yb.z, yb.w};
            uint32_t w0[4], w1[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w0[i] = f32_to_bf16_bits(__uint_as_float(y0[i] << 16) + acc[i][0]) |
                        ((uint32_t)f32_to_bf16_bits(__uint_as_float(y0[i] & 0xFFFF0000u) + acc[i][1])
                         << 16);
                w1[i] = f32_to_bf16_bits(__uint_as_float(y1[i] << 16) + acc[i][2]) |
                        ((uint32_t)f32_to_bf16_bits(__uint_as_float(y1[i] & 0xFFFF0000u) + acc[i][3])
                         << 16);
            }
            if (in0 && col_in)
                *reinterpret_cast<uint4 *>(p.Out + ma * p.ldo + ncol) =
                    make_uint4(w0[0], w0[1], w0[2], w0[3]);
            if (in1 && col_in)
                *reinterpret_cast<uint4 *>(p.Out + mb * p.ldo + ncol) =
                    make_uint4(w1[0], w1[1], w1[2], w1[3]);
        }
    }
    // this kernel does not complete before the shrink kernel, even without
    // any group to work on: what follows on the stream may change the inputs
    if (!waited)
        pdl_wait();
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

template <int RT, int NT>
cudaError_t launch_shrink(const LoraPlan &pl, const LoraParams &p, cudaStream_t stream)
{
    const void *fn = reinterpret_cast<const void *>(&lora_shrink_kernel<RT, NT>);
    constexpr size_t smem =
        (size_t)kShrinkWarps * RT * NT * 512 + (size_t)8 * NT * (16 * RT + 4) * sizeof(float);
    static std::atomic<bool> done[kMaxDeviceCache];
    const cudaError_t e = allow_smem(fn, done, smem);
    if (e != cudaSuccess)
        return e;
    LoraParams q = p;
    void *args[] = {&q};
    return launch_pdl_cluster(fn, dim3(pl.cluster, pl.shrink_subs, pl.blocks * pl.slices),
                              dim3(kShrinkWarps * 32), pl.cluster, smem, stream, args);
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
    return (size_t)M * R * 4;
}

LoraPlan plan_lora(int device, int M, int N, int K, int R)
{
    const int sms = device_info(device).sms;
    LoraPlan pl{};
    const long long blocks = ((long long)M + kBlockTok - 1) / kBlockTok;
    pl.rank_tiles = R <= 16 ? 1 : (R <= 32 ? 2 : 4);
    pl.slices = (R + 16 * pl.rank_tiles - 1) / (16 * pl.rank_tiles);
    pl.blocks = (int)blocks;
    const int tok = std::min(M, kBlockTok);
    // shrink: K is split over a cluster while the blocks alone leave SMs idle
    // (two CTAs fit on one), with at least a unit of 32 k per warp
    const int units = (K + 31) / 32;
    pl.cluster = 1;
    while (pl.cluster < 8 && 2 * pl.cluster * blocks * pl.slices <= 2 * sms &&
           2 * pl.cluster * kShrinkWarps <= units)
        pl.cluster *= 2;
    // groups of a block run side by side while there is room for them: the
    // host does not know how many there are, and a share without any ends at
    // once
    const long long shrink_ctas = blocks * pl.slices * pl.cluster;
    pl.shrink_subs = (int)std::max<long long>(1, std::min<long long>(tok, 4 * sms / shrink_ctas));
    // expand: 128 columns a CTA while that leaves SMs idle, else 256
    pl.expand_warps = ((N + 255) / 256) * blocks < sms ? 4 : 8;
    pl.ntiles = (N + 32 * pl.expand_warps - 1) / (32 * pl.expand_warps);
    const long long expand_ctas = blocks * pl.ntiles;
    pl.expand_subs = (int)std::max<long long>(1, std::min<long long>(tok, 8 * sms / expand_ctas));
    return pl;
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
    p.T = static_cast<uint4 *>(a.workspace);
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
        e = launch_shrink<1, 8>(pl, p, stream);
    else if (pl.rank_tiles == 2)
        e = launch_shrink<2, 8>(pl, p, stream);
    else
        e = launch_shrink<4, 4>(pl, p, stream);
    if (e != cudaSuccess)
        return e;
    const int steps = (a.R + 15) / 16;
    const void *fn = steps == 1   ? reinterpret_cast<const void *>(&lora_expand_kernel<1>)
                     : steps == 2 ? reinterpret_cast<const void *>(&lora_expand_kernel<2>)
                     : steps <= 4 ? reinterpret_cast<const void *>(&lora_expand_kernel<4>)
                                  : reinterpret_cast<const void *>(&lora_expand_kernel<8>);
    void *args[] = {&p};
    return launch_pdl(fn, dim3(pl.ntiles, pl.expand_subs, pl.blocks), dim3(32 * pl.expand_warps), 0,
                      stream, args);
}

}  // namespace mxg
