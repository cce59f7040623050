// One token per row of logits from a given random number, after temperature,
// top-p, top-k and min-p (the definition is at sample_logits in mxg.h).
//
// What bounds it: the logits are read once, M V 2 (or 4) bytes; the rest is
// a weight exp((l - max) / T) per entry and the search for the border of the
// kept set.  One row of 248320 bf16 entries is 0.5 MB, 0.08 us of HBM time,
// so a few rows are bound by latency (the hops between the CTAs of a row) and
// many rows by the arithmetic per entry.
//
// A row is taken by one thread-block cluster: every CTA copies its share into
// shared memory and everything after that runs on chip, the CTAs exchanging
// histograms and sums through distributed shared memory.
//
//  * Sums are integers.  A weight is an fp64 value in (0, 1], rounded to a
//    multiple of 2^-44; sums of up to 2^19 of those fit 64 bits and do not
//    depend on their order, so atomics and any split of the row give the same
//    token.  fp32 weights would not do: a token is picked where a running sum
//    of up to 248320 terms crosses a border, and an error of 2^-22 moves
//    that border past whole tokens.
//  * The kept set is a cut (value, ties): every entry above a logit value,
//    and the first few in index order of those equal to it (bf16 logits tie
//    by the thousand).  It is found by histograms: 512 bins of 1/16 binade of
//    the weight first, over all entries, then only over the entries of the
//    bin in which the border falls, 512 bins of their key range at a time,
//    until a bin is a single key.  No sort.
//  * One last pass adds the kept weights per warp segment in index order; the
//    CTA, the warp and the lane in whose part u * (kept mass) falls are found
//    from the sums of the parts, and only that part is looked through.
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace mxg {
namespace {

typedef unsigned long long u64;

constexpr int kBins = 512;
constexpr int kListCap = 2048;    // entries of the border bin a CTA lists
constexpr int kMaxCluster = 8;
constexpr int kMaxWarps = 32;
constexpr int kFix = 44;          // weights are multiples of 2^-kFix
constexpr int kSmemSlice = 192 * 1024;   // most bytes of logits a CTA holds
constexpr int kSlack = 136;       // slots beyond a CTA's entries: skew and the last 128

struct SampleParams {
    const void *logits;
    long long ld;
    int M, V, per;
    const float *u, *temperature, *top_p, *min_p;
    const int *top_k;
    int *tokens;
    float *probs;
};

// ------------------------------------------------------------------ entries
// A CTA's entries lie in shared memory in slots: [0, skew) and those behind
// the last entry hold -inf, so that every loop runs over whole groups of
// four.  NaN is stored as -inf and -0 as +0.
__device__ __forceinline__ float canonical(float v)
{
    return fmaxf(v, -INFINITY) + 0.f;
}
__device__ __forceinline__ float value_of(uint16_t b)
{
    return __uint_as_float((uint32_t)b << 16);
}
__device__ __forceinline__ float value_of(uint32_t b)
{
    return __uint_as_float(b);
}
template <typename T>
__device__ __forceinline__ T bits_of(float v)
{
    return sizeof(T) == 2 ? (T)(__float_as_uint(v) >> 16) : (T)__float_as_uint(v);
}

// Four consecutive slots.
__device__ __forceinline__ void load4(const uint16_t *d, int slot, float (&v)[4])
{
    const uint2 w = *reinterpret_cast<const uint2 *>(d + slot);
    v[0] = __uint_as_float(w.x << 16);
    v[1] = __uint_as_float(w.x & 0xFFFF0000u);
    v[2] = __uint_as_float(w.y << 16);
    v[3] = __uint_as_float(w.y & 0xFFFF0000u);
}
__device__ __forceinline__ void load4(const uint32_t *d, int slot, float (&v)[4])
{
    const float4 w = *reinterpret_cast<const float4 *>(d + slot);
    v[0] = w.x;
    v[1] = w.y;
    v[2] = w.z;
    v[3] = w.w;
}

// Integer keys that rise with the value; those of bf16 have 16 bits.
__device__ __forceinline__ uint32_t key_of(float v, uint16_t)
{
    const uint32_t b = __float_as_uint(v) >> 16;
    return b & 0x8000u ? 0xFFFFu - b : b | 0x8000u;
}
__device__ __forceinline__ uint32_t key_of(float v, uint32_t)
{
    const uint32_t b = __float_as_uint(v);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k, uint16_t)
{
    return __uint_as_float((k & 0x8000u ? k & 0x7FFFu : 0xFFFFu - k) << 16);
}
__device__ __forceinline__ float key_value(uint32_t k, uint32_t)
{
    return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// Weights of one row, round(2^kFix * exp((v - top) / T)), for finite v.
struct Weights {
    float least;          // 48 binades below the top or lower: no weight
    double top;
    double c;             // 64 * log2(e) / T
    const double *table;  // 2^(j / 64)

    // (v - top) / T in units of 1/64 binade, its integer part in the low bits
    __device__ __forceinline__ double scaled(float v, double &d) const
    {
        constexpr double kMagic = 6755399441055744.0;   // 1.5 * 2^52
        d = (double)fmaxf(v, least) - top;
        return fma(d, c, kMagic);
    }

    // First-level bin: 1/16 binade of the weight, the last bin holding
    // everything from 32 binades down.  It never falls as v falls.
    __device__ __forceinline__ int bin(double m) const
    {
        return min(-__double2loint(m) >> 2, kBins - 1);
    }

    __device__ __forceinline__ int bin(float v) const
    {
        double d;
        return bin(scaled(v, d));
    }

    __device__ __forceinline__ u64 weight(double m, double d) const
    {
        constexpr double kMagic = 6755399441055744.0;
        const int n = __double2loint(m);
        const double f = fma(d, c, -(m - kMagic));
        // 2^(f / 64) - 1 by its series: |f| <= 1/2, |f ln2 / 64| <= 0.0055,
        // so the sixth-order term is below 2^-54
        constexpr double l = 0.69314718055994530942 / 64.0;
        const double q =
            f * (l + f * (l * l / 2.0 +
                          f * (l * l * l / 6.0 +
                               f * (l * l * l * l / 24.0 + f * (l * l * l * l * l / 120.0)))));
        const double t = table[n & 63];
        const double w = fma(t, q, t);
        // times 2^(n / 64 + kFix) by the exponent field, then rounded to an
        // integer by adding 2^52
        const double s = __hiloint2double(__double2hiint(w) + (((n >> 6) + kFix) << 20),
                                          __double2loint(w));
        const double r = s + 4503599627370496.0;
        return (u64)__double_as_longlong(r) & 0xFFFFFFFFFFFFFull;
    }

    __device__ __forceinline__ u64 operator()(float v) const
    {
        double d;
        const double m = scaled(v, d);
        return weight(m, d);
    }
};

// ------------------------------------------------------------ shared memory
struct Hist {
    uint32_t lo[kBins], hi[kBins];   // 64-bit sums in two words
};

struct Shared {
    double table[64];
    // [0], [1]: masses and counts of the first level; then [2] and [3], [0]
    // and [1] in turn
    Hist hist[4];
    uint32_t list[kListCap];     // keys of the border bin
    u64 wmass[kMaxWarps];        // kept mass above the cut, per warp segment
    uint32_t wtie[kMaxWarps];    // entries equal to the cut, per warp segment
    u64 scan[kMaxWarps];
    uint32_t red[kMaxWarps];
    // exchanged with the peers
    uint32_t top_key, first;     // largest key; first index of the maximum
    u64 mass;                    // kept mass above the cut
    uint32_t ties;               // entries equal to the cut
    // answers of a search
    int bin;
    u64 base, total;
    int listed;
};

__device__ __forceinline__ u64 warp_sum(u64 v)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ u64 warp_scan(u64 v, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 b = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o)
            v += b;
    }
    return v;
}

// Adds w to a bin of this CTA's histogram (all lanes of the warp; w = 0: an
// entry that does not count).  Integer sums: their order does not matter; the
// low words carry into the high ones (a 64-bit shared-memory atomic is a
// compare-and-swap loop, 43 cycles a warp against 9 for the two).  A warp
// whose entries fall into one bin (rows of few distinct values) adds them up
// first: 32 atomics on one word run one after another.
template <bool MASS>
__device__ __forceinline__ void hist_add(Hist &h, int bin, u64 w, int lane)
{
    const int b0 = __shfl_sync(0xffffffffu, bin, 0);
    if (__all_sync(0xffffffffu, bin == b0)) {
        w = MASS ? warp_sum(w) : (u64)__popc(__ballot_sync(0xffffffffu, w != 0));
        if (lane != 0)
            return;
    }
    if (w == 0)
        return;
    if (!MASS) {
        atomicAdd(&h.lo[bin], (uint32_t)w);
        return;
    }
    const uint32_t lo = (uint32_t)w;
    const uint32_t old = atomicAdd(&h.lo[bin], lo);
    const uint32_t hi = (uint32_t)(w >> 32) + (old + lo < old ? 1u : 0u);
    if (hi)
        atomicAdd(&h.hi[bin], hi);
}

__device__ __forceinline__ void hist_clear(Hist &h)
{
    for (int i = threadIdx.x; i < kBins; i += blockDim.x) {
        h.lo[i] = 0;
        h.hi[i] = 0;
    }
}

// The border in the cluster's histogram h (complete in every CTA): s.bin is
// the first bin whose running sum, from `base`, reaches the target, s.base
// the sum before it, s.total the sum of all bins; s.bin = -1 when no bin
// reaches it.  target = 0: ceil(p * total), at least 1.
__device__ __forceinline__ void hist_find(Shared &s, const Hist &h, u64 base, u64 target, double p)
{
    const int i = threadIdx.x, lane = i & 31, warp = i >> 5;
    const uint32_t n = cluster_size();
    u64 v = 0;
    if (i < kBins) {
        uint32_t lo[kMaxCluster], hi[kMaxCluster];
#pragma unroll
        for (uint32_t c = 0; c < kMaxCluster; ++c) {
            lo[c] = c < n ? ld_peer(&h.lo[i], c) : 0;
            hi[c] = c < n ? ld_peer(&h.hi[i], c) : 0;
        }
#pragma unroll
        for (uint32_t c = 0; c < kMaxCluster; ++c)
            v += (u64)lo[c] + ((u64)hi[c] << 32);
    }
    u64 incl = warp_scan(v, lane);
    if (lane == 31 && warp < kBins / 32)
        s.scan[warp] = incl;
    if (i == 0)
        s.bin = -1;
    __syncthreads();
    u64 total = 0;
#pragma unroll
    for (int w = 0; w < kBins / 32; ++w) {
        if (w < warp)
            incl += s.scan[w];
        total += s.scan[w];
    }
    if (target == 0)
        target = max(1ull, (u64)ceil(p * (double)total));
    incl += base;
    if (i < kBins && incl >= target && incl - v < target) {
        s.bin = i;
        s.base = incl - v;
    }
    if (i == 0)
        s.total = total;
    __syncthreads();
}

// Largest key in [lo, hi] for which `yes` holds, given that it holds for lo
// and for no key above one for which it does not; 32 keys at a time.
template <typename F>
__device__ __forceinline__ uint32_t last_key(uint32_t lo, uint32_t hi, int lane, F yes)
{
    while (lo < hi) {
        const uint32_t step = (hi - lo + 31) / 32;
        const uint32_t k = lo + step * (lane + 1);
        const bool in = k >= lo && k <= hi;   // no overflow
        const int n = __popc(__ballot_sync(0xffffffffu, in && yes(k)));
        lo += step * n;
        hi = min(hi, lo + (step - 1));
    }
    return lo;
}

// ------------------------------------------------------------------- kernel
template <typename T>
__global__ void __launch_bounds__(1024, 1) sample_kernel(const SampleParams p)
{
    __shared__ Shared s;
    extern __shared__ __align__(16) uint8_t dyn[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nwarps = blockDim.x >> 5;
    const uint32_t rank = cluster_rank(), ncta = cluster_size();
    const int row = blockIdx.x / ncta;
    const int lo = min((int)rank * p.per, p.V);            // this CTA's entries
    const int cnt = min(lo + p.per, p.V) - lo;
    const T *src = static_cast<const T *>(p.logits) + row * p.ld + lo;
    // slots at the source's address modulo 16 bytes; a segment of whole 128
    // slots per warp, in index order
    constexpr int kVec = 16 / sizeof(T);
    const int skew = (int)(reinterpret_cast<uintptr_t>(src) & 15u) / (int)sizeof(T);
    const int seg = (skew + cnt + 128 * nwarps - 1) / (128 * nwarps) * 128;
    const int used = (skew + cnt + 127) / 128 * 128;       // slots that any warp reads
    const int b0 = min(used, warp * seg), b1 = min(used, b0 + seg);
    T *data = reinterpret_cast<T *>(dyn);
    for (int i = tid; i < 64; i += blockDim.x)
        s.table[i] = exp2((double)i * (1.0 / 64.0));
    for (int i = 0; i < 4; ++i)
        hist_clear(s.hist[i]);
    if (tid == 0) {
        s.first = 0xFFFFFFFFu;
        s.listed = 0;
    }
    if (tid < skew)
        data[tid] = bits_of<T>(-INFINITY);
    for (int i = skew + cnt + tid; i < used; i += blockDim.x)
        data[i] = bits_of<T>(-INFINITY);
    pdl_wait();
    pdl_launch_dependents();
    const float temp = p.temperature ? __ldg(p.temperature + row) : 1.f;
    const float top_p = p.top_p ? __ldg(p.top_p + row) : 1.f;
    const float min_p = p.min_p ? __ldg(p.min_p + row) : 0.f;
    const int top_k = p.top_k ? __ldg(p.top_k + row) : 0;
    const float u = __ldg(p.u + row);

    // ---- copy the entries and find the maximum
    float mx = -INFINITY;
    {
        const int head = min(cnt, (kVec - skew) % kVec);
        const int vecs = (cnt - head) / kVec;
        const uint4 *vsrc = reinterpret_cast<const uint4 *>(src + head);
        uint4 *vdst = reinterpret_cast<uint4 *>(data + skew + head);
        for (int i0 = tid; i0 < vecs; i0 += 4 * blockDim.x) {
            uint4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i0 + j * (int)blockDim.x < vecs)
                    v[j] = __ldcs(vsrc + i0 + j * blockDim.x);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i0 + j * (int)blockDim.x < vecs) {
                    uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (sizeof(T) == 2) {
                            const float a = canonical(__uint_as_float(w[k] << 16));
                            const float b = canonical(__uint_as_float(w[k] & 0xFFFF0000u));
                            mx = fmaxf(mx, fmaxf(a, b));
                            w[k] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
                        } else {
                            const float a = canonical(__uint_as_float(w[k]));
                            mx = fmaxf(mx, a);
                            w[k] = __float_as_uint(a);
                        }
                    }
                    vdst[i0 + j * blockDim.x] = make_uint4(w[0], w[1], w[2], w[3]);
                }
        }
        if (tid < cnt - vecs * kVec) {   // what the vectors leave: fewer than 2 kVec entries
            const int i = tid < head ? tid : tid + vecs * kVec;
            const float a = canonical(value_of(src[i]));
            data[skew + i] = bits_of<T>(a);
            mx = fmaxf(mx, a);
        }
    }
    uint32_t mk = __reduce_max_sync(0xffffffffu, key_of(mx, (uint32_t)0));
    if (lane == 0)
        s.red[warp] = mk;
    __syncthreads();
    if (warp == 0) {
        mk = __reduce_max_sync(0xffffffffu, lane < nwarps ? s.red[lane] : 0u);
        if (lane == 0)
            s.top_key = mk;
    }
    cluster_barrier();
    mk = __reduce_max_sync(0xffffffffu, lane < (int)ncta ? ld_peer(&s.top_key, lane) : 0u);
    float top = key_value(mk, (uint32_t)0);

    if (top == -INFINITY || !(temp > 0.f)) {   // nothing to take, or greedy
        if (top > -INFINITY)
            for (int i = b0 + 4 * lane; i < b1; i += 128) {
                float v[4];
                load4(data, i, v);
                if (v[0] == top || v[1] == top || v[2] == top || v[3] == top) {
                    const int e = v[0] == top ? 0 : v[1] == top ? 1 : v[2] == top ? 2 : 3;
                    atomicMin(&s.first, (uint32_t)(lo + i + e - skew));
                    break;
                }
            }
        cluster_barrier();
        if (rank == 0 && warp == 0) {
            const uint32_t first = __reduce_min_sync(
                0xffffffffu, lane < (int)ncta ? ld_peer(&s.first, lane) : 0xFFFFFFFFu);
            if (lane == 0) {
                p.tokens[row] = (int)first;
                if (p.probs)
                    p.probs[row] = top > -INFINITY ? 1.f : 0.f;
            }
        }
        cluster_barrier();
        return;
    }
    if (top == INFINITY) {
        // the +inf entries share the mass: as zeros among -inf (every warp
        // reads its own segment only)
        for (int i = b0 + lane; i < b1; i += 32)
            data[i] = bits_of<T>(value_of(data[i]) == INFINITY ? 0.f : -INFINITY);
        __syncwarp();
        top = 0.f;
    }

    const double kLog2e = 1.4426950408889634074;
    Weights weight;
    weight.top = (double)top;
    weight.table = s.table;
    {
        // a temperature at which the next lower float has no weight is as
        // good as any below it, and keeps (v - top) / T in range
        const double gap = (double)top - (double)nextafterf(top, -INFINITY);
        const double t = fmax((double)temp, gap * (kLog2e / 48.0));
        weight.c = 64.0 * kLog2e / t;
        weight.least = fmaxf(__double2float_rd((double)top - 48.0 / kLog2e * t), -FLT_MAX);
    }

    // ---- min-p: the lowest value that passes (the test rises with the value)
    float low = -FLT_MAX;   // -inf never passes
    if (min_p > 0.f) {
        const double cut = (double)temp * log(fmin((double)min_p, 1.0));
        low = fmaxf(__double2float_rd(weight.top + cut), -FLT_MAX);
        for (int i = 0; i < 2 && low > -FLT_MAX; ++i) {
            const float below = nextafterf(low, -INFINITY);
            if ((double)below - weight.top >= cut)
                low = below;
        }
        for (int i = 0; i < 3 && (double)low - weight.top < cut; ++i)
            low = nextafterf(low, INFINITY);
    }

    // ---- the cut of top-p and top-k: keep values above it, and the first
    // cut_ties in index order of those equal to it
    const bool use_p = top_p < 1.f, use_k = top_k > 0;
    float cut = -INFINITY;
    u64 cut_ties = 0;
    if (use_p || use_k) {
        for (int i = b0 + 4 * lane; i < b1; i += 128) {
            float v[4];
            load4(data, i, v);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool in = v[e] > -INFINITY;
                double d;
                const double m = weight.scaled(v[e], d);
                const int bin = weight.bin(m);
                if (use_p)
                    hist_add<true>(s.hist[0], bin, in ? weight.weight(m, d) : 0ull, lane);
                if (use_k)
                    hist_add<false>(s.hist[1], bin, in ? 1ull : 0ull, lane);
            }
        }
        cluster_barrier();
        int bin_p = kBins, bin_k = kBins;
        u64 base_p = 0, base_k = 0, target_p = 0;
        const u64 target_k = (u64)max(top_k, 0);
        if (use_p) {
            hist_find(s, s.hist[0], 0, 0, (double)top_p);
            bin_p = s.bin;
            base_p = s.base;
            target_p = max(1ull, (u64)ceil((double)top_p * (double)s.total));
            __syncthreads();
        }
        if (use_k) {
            hist_find(s, s.hist[1], 0, target_k, 0.0);
            if (s.bin >= 0) {   // else the row has no more than top_k entries
                bin_k = s.bin;
                base_k = s.base;
            }
            __syncthreads();
        }
        // the stricter filter decides; both are followed when their borders
        // fall into one bin
        const int bin = min(bin_p, bin_k);
        if (bin < kBins) {
            const bool do_p = bin_p == bin, do_k = bin_k == bin;
            // the bin's keys are kl .. kh
            const uint32_t k_min = key_of(-FLT_MAX, T(0)), k_top = key_of(top, T(0));
            auto key_bin = [&](uint32_t k) { return weight.bin(key_value(k, T(0))); };
            const uint32_t kh = bin == 0 ? k_top
                                         : last_key(k_min, k_top, lane,
                                                    [&](uint32_t k) { return key_bin(k) >= bin; });
            uint32_t kl = k_min;
            if (key_bin(k_min) > bin)
                kl = last_key(k_min, kh, lane, [&](uint32_t k) { return key_bin(k) > bin; }) + 1;
            const float vl = key_value(kl, T(0)), vh = key_value(kh, T(0));
            const int sh0 = max(0, 32 - __clz(kh - kl) - 9);   // bins of 2^sh keys from kh down
            // second level: a histogram of those keys, and a list of them for
            // the levels behind it (when they are too many for the list, those
            // look through the slots again)
            for (int i = b0 + 4 * lane; i < b1; i += 128) {
                float v[4];
                load4(data, i, v);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const bool in = v[e] >= vl && v[e] <= vh;
                    const unsigned found = __ballot_sync(0xffffffffu, in);
                    if (!found)
                        continue;
                    const uint32_t k = key_of(v[e], T(0));
                    const int b = in ? (int)((kh - k) >> sh0) : 0;
                    if (do_p)
                        hist_add<true>(s.hist[2], b, in ? weight(v[e]) : 0ull, lane);
                    if (do_k)
                        hist_add<false>(s.hist[3], b, in ? 1ull : 0ull, lane);
                    if (sh0 > 0) {
                        int at = 0;
                        if (lane == 0)
                            at = atomicAdd(&s.listed, __popc(found));
                        at = __shfl_sync(0xffffffffu, at, 0) + __popc(found & ((1u << lane) - 1));
                        if (in && at < kListCap)
                            s.list[at] = k;
                    }
                }
            }
            cluster_barrier();
            const bool listed = s.listed <= kListCap;
            const int entries = listed ? s.listed : used;
            hist_clear(s.hist[0]);   // the peers have read these by now
            hist_clear(s.hist[1]);
            // the histogram of a further level: masses ([2] or [0]) or counts ([3] or [1])
            auto refine = [&](auto mass, u64 base, u64 target, uint32_t &key, u64 &ties) {
                constexpr bool MASS = decltype(mass)::value;
                Hist *h = MASS ? &s.hist[2] : &s.hist[3], *other = MASS ? &s.hist[0] : &s.hist[1];
                uint32_t l = kl, r = kh;
                int sh = sh0;
                while (true) {
                    hist_find(s, *h, base, target, 0.0);
                    base = s.base;
                    r -= (uint32_t)s.bin << sh;
                    l = max(l, r - ((1u << sh) - 1));
                    if (sh == 0)
                        break;
                    __syncthreads();
                    Hist *t = h;
                    h = other;
                    other = t;
                    sh = l < r ? max(0, 32 - __clz(r - l) - 9) : 0;
                    for (int i = tid; i - lane < entries; i += blockDim.x) {
                        uint32_t k = 0;
                        if (i < entries)
                            k = listed ? s.list[i] : key_of(value_of(data[i]), T(0));
                        const bool in = k >= l && k <= r;
                        const u64 w = !in ? 0ull : MASS ? weight(key_value(k, T(0))) : 1ull;
                        hist_add<MASS>(*h, in ? (int)((r - k) >> sh) : 0, w, lane);
                    }
                    cluster_barrier();
                    hist_clear(*other);   // read by the peers before this barrier
                }
                __syncthreads();
                key = r;
                const u64 each = MASS ? weight(key_value(r, T(0))) : 1ull;
                ties = (target - base + each - 1) / each;
            };
            uint32_t key = 0, cut_key = 0;
            u64 ties = 0;
            if (do_p) {
                refine(std::true_type(), base_p, target_p, key, ties);
                cut_key = key;
                cut_ties = ties;
            }
            if (do_k) {
                refine(std::false_type(), base_k, target_k, key, ties);
                if (key > cut_key || (key == cut_key && ties < cut_ties)) {
                    cut_key = key;
                    cut_ties = ties;
                }
            }
            cut = key_value(cut_key, T(0));
        }
    }

    // ---- kept mass per warp segment and CTA
    const float keep = fmaxf(low, cut);    // what is kept is at least this ...
    const bool tied = cut >= low;          // ... and above the cut or among the first ties
    u64 mass = 0;
    uint32_t tie = 0;
    for (int i = b0 + 4 * lane; i < b1; i += 128) {
        float v[4];
        load4(data, i, v);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (v[e] >= keep) {
                if (v[e] == cut)
                    ++tie;
                else
                    mass += weight(v[e]);
            }
    }
    mass = warp_sum(mass);
    tie = __reduce_add_sync(0xffffffffu, tie);
    if (lane == 0) {
        s.wmass[warp] = mass;
        s.wtie[warp] = tie;
    }
    __syncthreads();
    if (warp == 0) {
        const u64 m = warp_sum(lane < nwarps ? s.wmass[lane] : 0ull);
        const uint32_t n = __reduce_add_sync(0xffffffffu, lane < nwarps ? s.wtie[lane] : 0u);
        if (lane == 0) {
            s.mass = m;
            s.ties = n;
        }
    }
    cluster_barrier();
    // ---- where u * (kept mass) falls: the CTA, then its warp (every warp
    // works that out for itself), then the entry.  of() gives each lane the
    // kept mass of its part from the mass above the cut and the ties in it
    const u64 each = tied ? weight(cut) : 0ull;
    auto of = [&](u64 m, u64 n, u64 &before) {
        before += warp_scan(n, lane) - n;
        return m + each * (before >= cut_ties ? 0ull : min(n, cut_ties - before));
    };
    u64 ties_before = 0;
    u64 part = 0, n = 0;
    if (lane < (int)ncta) {
        part = ld_peer64(&s.mass, lane);
        n = ld_peer(&s.ties, lane);
    }
    // the peers' shared memory is not read after this point
    cluster_arrive();
    part = of(part, n, ties_before);
    u64 incl = warp_scan(part, lane);
    const u64 total = __shfl_sync(0xffffffffu, incl, 31);
    // the entry whose running sum first exceeds u * total (u >= 1 or NaN:
    // the last one with a weight)
    const double x = (double)u * (double)total;
    u64 target = total - 1;
    if (x < (double)target)
        target = x > 0.0 ? (u64)x : 0;
    int at = __ffs(__ballot_sync(0xffffffffu, incl > target)) - 1;
    if (at == (int)rank) {
        u64 before = __shfl_sync(0xffffffffu, incl - part, at);
        ties_before = __shfl_sync(0xffffffffu, ties_before, at);
        part = of(lane < nwarps ? s.wmass[lane] : 0ull, lane < nwarps ? s.wtie[lane] : 0u,
                  ties_before);
        incl = before + warp_scan(part, lane);
        at = __ffs(__ballot_sync(0xffffffffu, incl > target)) - 1;
        if (at == warp) {
            before = __shfl_sync(0xffffffffu, incl - part, at);
            ties_before = __shfl_sync(0xffffffffu, ties_before, at);
            // a 32nd of the segment per lane, then its entries
            const int sub = seg / 32;   // a multiple of 4
            mass = 0;
            tie = 0;
            for (int i = b0 + lane * sub; i < min(b1, b0 + (lane + 1) * sub); i += 4) {
                float v[4];
                load4(data, i, v);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (v[e] >= keep) {
                        if (v[e] == cut)
                            ++tie;
                        else
                            mass += weight(v[e]);
                    }
            }
            __syncwarp();
            part = of(mass, tie, ties_before);
            incl = before + warp_scan(part, lane);
            at = __ffs(__ballot_sync(0xffffffffu, incl > target)) - 1;
            u64 run = __shfl_sync(0xffffffffu, incl - part, at);
            ties_before = __shfl_sync(0xffffffffu, ties_before, at);
            const int e0 = b0 + at * sub, e1 = min(b1, e0 + sub);
            for (int i = e0 + lane; i - lane < e1; i += 32) {
                const float v = i < e1 ? value_of(data[i]) : -INFINITY;
                const bool in = v >= keep;
                const unsigned equal = __ballot_sync(0xffffffffu, in && v == cut);
                u64 w = 0;
                if (in && v != cut)
                    w = weight(v);
                else if (in && ties_before + __popc(equal & ((1u << lane) - 1)) < cut_ties)
                    w = each;
                ties_before += __popc(equal);
                const u64 sum = run + warp_scan(w, lane);
                const unsigned hit = __ballot_sync(0xffffffffu, sum > target);
                if (hit) {
                    if (lane == __ffs(hit) - 1) {
                        p.tokens[row] = lo + i - skew;
                        if (p.probs)
                            p.probs[row] = (float)((double)w / (double)total);
                    }
                    break;
                }
                run = __shfl_sync(0xffffffffu, sum, 31);
            }
        }
    }
    cluster_wait();
}

template <typename T>
cudaError_t launch_typed(const SamplePlan &pl, const SampleParams &p, cudaStream_t stream)
{
    const void *fn = reinterpret_cast<const void *>(&sample_kernel<T>);
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= kMaxDeviceCache)
        return cudaErrorInvalidDevice;
    static std::atomic<bool> done[kMaxDeviceCache];
    if (!done[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kSmemSlice + kSlack * (int)sizeof(T));
        if (e != cudaSuccess)
            return e;
        done[dev].store(true, std::memory_order_release);
    }
    SampleParams q = p;
    void *args[] = {&q};
    return launch_pdl_cluster(fn, dim3((unsigned)p.M * pl.cluster), dim3(pl.threads), pl.cluster,
                              pl.smem, stream, args);
}

}  // namespace

bool sample_shape_ok(int M, int V)
{
    // a row fits the shared memory of its cluster as fp32; rows times
    // clusters are a grid dimension
    return M >= 1 && M <= (1 << 27) && V >= 1 && V <= kMaxCluster * kSmemSlice / 4;
}

SamplePlan plan_sample(int device, int M, int V, bool fp32)
{
    const int size = fp32 ? 4 : 2;
    SamplePlan pl{};
    // a CTA per 4096 entries at least while that leaves SMs idle
    const int sms = device_info(device).sms;
    pl.cluster = 1;
    while (pl.cluster < kMaxCluster &&
           ((V > 4096 * pl.cluster && (long long)M * pl.cluster * 2 <= sms) ||
            (long long)(V + pl.cluster - 1) / pl.cluster * size > 72 * 1024))
        pl.cluster *= 2;
    pl.per = ((V + pl.cluster - 1) / pl.cluster + 7) / 8 * 8;
    pl.threads = (long long)M * pl.cluster <= sms ? 1024 : 512;
    pl.smem = ((size_t)pl.per + kSlack) * size;   // whole groups of 128 slots, and the skew
    return pl;
}

cudaError_t launch_sample(const SamplePlan &pl, const SampleArgs &a, cudaStream_t stream)
{
    SampleParams p{};
    p.logits = a.logits;
    p.ld = a.ld;
    p.M = a.M;
    p.V = a.V;
    p.per = pl.per;
    p.u = a.u;
    p.temperature = a.temperature;
    p.top_p = a.top_p;
    p.min_p = a.min_p;
    p.top_k = a.top_k;
    p.tokens = a.tokens;
    p.probs = a.probs;
    return a.fp32 ? launch_typed<uint32_t>(pl, p, stream) : launch_typed<uint16_t>(pl, p, stream);
}

}  // namespace mxg
