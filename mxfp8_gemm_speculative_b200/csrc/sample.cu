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
//  * The kept set is a cut (key, ties): every entry above a logit value, and
//    the first few in index order of those equal to it (bf16 logits tie by
//    the thousand).  It is found by histograms: 512 bins of 1/16 binade of
//    the weight first, over all entries, then only over the entries of the
//    bin in which the border falls, 512 bins of their key range at a time,
//    until a bin is a single key.  No sort.
//  * One last pass adds the kept weights per warp segment in index order; the
//    warp in whose segment u * (kept mass) falls walks its entries.
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
// The value of stored bits: NaN becomes -inf and -0 becomes +0.
__device__ __forceinline__ float value_of(uint16_t b)
{
    return fmaxf(__uint_as_float((uint32_t)b << 16), -INFINITY) + 0.f;
}
__device__ __forceinline__ float value_of(uint32_t b)
{
    return fmaxf(__uint_as_float(b), -INFINITY) + 0.f;
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

// Weights of one row: round(2^kFix * exp((v - top) / T)).
struct Weights {
    float top;
    double dtop;
    double c;             // 256 * log2(e) / T
    const double *table;  // 2^(j / 256)

    __device__ __forceinline__ u64 operator()(float v) const
    {
        if (v == top)
            return 1ull << kFix;   // also for +inf
        // (v - top) / T in units of 1/256 binade, not below -70 binades
        // (smaller weights round to none, and so does everything beside an
        // infinite top); split into an integer and a rest f in [-1/2, 1/2]
        const double x = fmax(((double)v - dtop) * c, -70.0 * 256.0);
        constexpr double kMagic = 6755399441055744.0;   // 1.5 * 2^52
        const double m = x + kMagic;
        const int n = __double2loint(m);
        const double f = x - (m - kMagic);
        // 2^(f / 256) - 1 by its series: |f ln2 / 256| <= 0.00136, so the
        // fifth-order term is below 2^-54
        constexpr double l = 0.69314718055994530942 / 256.0;
        const double q =
            f * (l + f * (l * l / 2.0 + f * (l * l * l / 6.0 + f * (l * l * l * l / 24.0))));
        const double t = table[n & 255];
        const double w = fma(t, q, t);
        // times 2^(n / 256 + kFix) by the exponent field, then rounded to an
        // integer by adding 2^52
        const double s = __hiloint2double(__double2hiint(w) + (((n >> 8) + kFix) << 20),
                                          __double2loint(w));
        const double r = s + 4503599627370496.0;
        return (u64)__double_as_longlong(r) & 0xFFFFFFFFFFFFFull;
    }
};

// First-level bin of an entry: 1/16 binade of its weight, the last one
// holding everything from 32 binades down.  fp32 is enough: the map only has
// to be the same everywhere and not to rise with the value.
__device__ __forceinline__ int coarse_bin(float v, float top, float c16)
{
    return v == top ? 0 : (int)fminf((top - v) * c16, (float)(kBins - 1));
}

// ------------------------------------------------------------ shared memory
struct Hist {
    uint32_t lo[kBins], hi[kBins];   // 64-bit sums in two words
};

struct Shared {
    double table[256];
    Hist hist[3];
    u64 wmass[kMaxWarps];        // kept mass above the cut, per warp segment
    uint32_t wtie[kMaxWarps];    // entries equal to the cut, per warp segment
    uint32_t list[kListCap];     // keys of the border bin
    u64 scan[kMaxWarps];
    uint32_t red[kMaxWarps];
    // exchanged with the peers
    uint32_t top_key, first;     // largest key; first index of the maximum
    uint32_t kmin, kmax;         // keys in the border bin
    // answers of a search
    int bin;
    u64 base;
    int listed;
    u64 total;
    int owner;
    u64 owner_base;
    uint32_t owner_tie;
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
// entry that does not count).  Integer sums: their order does not matter.
// The low words carry into the high ones.  A warp whose entries fall into one
// bin (rows of few distinct values) adds them up first: 32 atomics on one
// word run one after another.
template <bool MASS>
__device__ __forceinline__ void hist_add(Hist &h, int bin, u64 w, int lane)
{
    const unsigned live = __ballot_sync(0xffffffffu, w != 0);
    if (!live)
        return;
    const int b0 = __shfl_sync(0xffffffffu, bin, __ffs(live) - 1);
    if (__all_sync(0xffffffffu, w == 0 || bin == b0)) {
        const u64 s = MASS ? warp_sum(w) : (u64)__popc(live);
        if (lane != 0)
            return;
        w = s;
        bin = b0;
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
    if (i < kBins)
        for (uint32_t c = 0; c < n; ++c)
            v += (u64)ld_peer(&h.lo[i], c) + ((u64)ld_peer(&h.hi[i], c) << 32);
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
    for (int i = tid; i < 256; i += blockDim.x)
        s.table[i] = exp2((double)i * (1.0 / 256.0));
    for (int i = 0; i < 3; ++i)
        hist_clear(s.hist[i]);
    if (tid == 0) {
        s.first = 0xFFFFFFFFu;
        s.kmin = 0xFFFFFFFFu;
        s.kmax = 0;
        s.listed = 0;
    }
    pdl_wait();
    pdl_launch_dependents();

    // ---- copy the slice, at its address modulo 16, and find the maximum
    const T *src = static_cast<const T *>(p.logits) + row * p.ld + lo;
    const int skew = (int)(reinterpret_cast<uintptr_t>(src) & 15u) / (int)sizeof(T);
    T *data = reinterpret_cast<T *>(dyn) + skew;
    float mx = -INFINITY;
    {
        constexpr int kVec = 16 / sizeof(T);
        const int head = min(cnt, (kVec - skew) % kVec);
        const int vecs = (cnt - head) / kVec;
        const uint4 *vsrc = reinterpret_cast<const uint4 *>(src + head);
        uint4 *vdst = reinterpret_cast<uint4 *>(data + head);
        for (int i0 = tid; i0 < vecs; i0 += 4 * blockDim.x) {
            uint4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i0 + j * (int)blockDim.x < vecs)
                    v[j] = __ldcs(vsrc + i0 + j * blockDim.x);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i0 + j * (int)blockDim.x < vecs) {
                    vdst[i0 + j * blockDim.x] = v[j];
                    const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (sizeof(T) == 2) {
                            mx = fmaxf(mx, fmaxf(value_of((uint16_t)w[k]),
                                                 value_of((uint16_t)(w[k] >> 16))));
                        } else {
                            mx = fmaxf(mx, value_of((uint32_t)w[k]));
                        }
                    }
                }
        }
        if (tid < cnt - vecs * kVec) {   // what the vectors leave: fewer than 2 kVec entries
            const int i = tid < head ? tid : tid + vecs * kVec;
            data[i] = src[i];
            mx = fmaxf(mx, value_of(data[i]));
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
    for (uint32_t c = 0; c < ncta; ++c)
        mk = max(mk, ld_peer(&s.top_key, c));
    mk = __reduce_max_sync(0xffffffffu, mk);
    const float top = key_value(mk, (uint32_t)0);

    const float temp = p.temperature ? __ldg(p.temperature + row) : 1.f;
    // this warp's entries, in index order
    const int seg = (((cnt + nwarps - 1) / nwarps) + 31) / 32 * 32;
    const int b0 = min(cnt, warp * seg), b1 = min(cnt, b0 + seg);

    if (top == -INFINITY || !(temp > 0.f)) {   // nothing to take, or greedy
        if (top > -INFINITY)
            for (int i = b0 + lane; i < b1; i += 32)
                if (value_of(data[i]) == top) {
                    atomicMin(&s.first, (uint32_t)(lo + i));
                    break;
                }
        cluster_barrier();
        if (rank == 0 && tid == 0) {
            uint32_t first = s.first;
            for (uint32_t c = 1; c < ncta; ++c)
                first = min(first, ld_peer(&s.first, c));
            p.tokens[row] = (int)first;
            if (p.probs)
                p.probs[row] = top > -INFINITY ? 1.f : 0.f;
        }
        cluster_barrier();
        return;
    }

    const double kLog2e = 1.4426950408889634074;
    Weights weight;
    weight.top = top;
    weight.dtop = (double)top;
    weight.c = 256.0 * kLog2e / (double)temp;
    weight.table = s.table;
    const float c16 = (float)(16.0 * kLog2e / (double)temp);

    // ---- min-p: the lowest value that passes (the test rises with the value)
    float low = -FLT_MAX;   // -inf never passes
    const float min_p = p.min_p ? __ldg(p.min_p + row) : 0.f;
    if (min_p > 0.f && top < INFINITY) {
        const double cut = (double)temp * log(fmin((double)min_p, 1.0));
        const double dtop = weight.dtop;
        low = fmaxf(__double2float_rd(dtop + cut), -FLT_MAX);
        for (int i = 0; i < 2 && low > -FLT_MAX; ++i) {
            const float below = nextafterf(low, -INFINITY);
            if (below > -INFINITY && (double)below - dtop >= cut)
                low = below;
        }
        for (int i = 0; i < 3 && !((double)low - dtop >= cut); ++i)
            low = nextafterf(low, INFINITY);
        low += 0.f;   // no -0
    }
    uint32_t low_key = key_of(low, T(0));   // of the value truncated to T
    if (key_value(low_key, T(0)) < low)
        ++low_key;

    // ---- the cut of top-p and top-k
    const float top_p = p.top_p ? __ldg(p.top_p + row) : 1.f;
    const int top_k = p.top_k ? __ldg(p.top_k + row) : 0;
    const bool use_p = top_p < 1.f, use_k = top_k > 0;
    uint32_t cut_key = 0;              // keep keys above it, and ...
    u64 cut_ties = ~0ull;              // ... the first so many equal to it
    if (use_p || use_k) {
        for (int i = b0 + lane; i - lane < b1; i += 32) {
            const float v = i < b1 ? value_of(data[i]) : -INFINITY;
            const bool in = v > -INFINITY;
            const int bin = in ? coarse_bin(v, top, c16) : 0;
            if (use_p)
                hist_add<true>(s.hist[0], bin, in ? weight(v) : 0ull, lane);
            if (use_k)
                hist_add<false>(s.hist[1], bin, in ? 1ull : 0ull, lane);
        }
        cluster_barrier();
        int bin_p = kBins, bin_k = kBins;
        u64 base_p = 0, base_k = 0, target_p = 0;
        if (use_p) {
            hist_find(s, s.hist[0], 0, 0, (double)top_p);
            bin_p = s.bin;
            base_p = s.base;
            target_p = max(1ull, (u64)ceil((double)top_p * (double)s.total));
            __syncthreads();
        }
        if (use_k) {
            hist_find(s, s.hist[1], 0, (u64)top_k, 0.0);
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
            // list the keys of that bin (or, when they are too many, look
            // through the slice again each time)
            uint32_t least = 0xFFFFFFFFu, most = 0;
            for (int i = b0 + lane; i - lane < b1; i += 32) {
                const float v = i < b1 ? value_of(data[i]) : -INFINITY;
                const uint32_t k = key_of(v, T(0));
                const bool in = v > -INFINITY && coarse_bin(v, top, c16) == bin;
                const unsigned found = __ballot_sync(0xffffffffu, in);
                if (!found)
                    continue;
                int at = 0;
                if (lane == 0)
                    at = atomicAdd(&s.listed, __popc(found));
                at = __shfl_sync(0xffffffffu, at, 0) + __popc(found & ((1u << lane) - 1));
                if (in) {
                    if (at < kListCap)
                        s.list[at] = k;
                    least = min(least, k);
                    most = max(most, k);
                }
            }
            least = __reduce_min_sync(0xffffffffu, least);
            most = __reduce_max_sync(0xffffffffu, most);
            if (lane == 0 && least <= most) {
                atomicMin(&s.kmin, least);
                atomicMax(&s.kmax, most);
            }
            cluster_barrier();
            uint32_t kmin = 0xFFFFFFFFu, kmax = 0;
            for (uint32_t c = 0; c < ncta; ++c) {
                kmin = min(kmin, ld_peer(&s.kmin, c));
                kmax = max(kmax, ld_peer(&s.kmax, c));
            }
            const bool listed = s.listed <= kListCap;
            const int entries = listed ? s.listed : cnt;
            int level = 0;
            auto refine = [&](auto mass, u64 base, u64 target, uint32_t &key, u64 &ties) {
                constexpr bool MASS = decltype(mass)::value;
                uint32_t kl = kmin, kh = kmax;
                while (kl < kh) {
                    const uint32_t range = kh - kl;   // bins of 2^sh keys from kh down
                    const int sh = max(0, 32 - __clz(range) - 9);
                    Hist &h = s.hist[level & 1 ? 0 : 2];
                    for (int i = tid; i - lane < entries; i += blockDim.x) {
                        uint32_t k = 0;
                        bool in = i < entries;
                        if (in && listed) {
                            k = s.list[i];
                        } else if (in) {
                            const float v = value_of(data[i]);
                            in = v > -INFINITY;
                            k = key_of(v, T(0));
                        }
                        in = in && k >= kl && k <= kh;
                        const u64 w = !in ? 0ull : MASS ? weight(key_value(k, T(0))) : 1ull;
                        hist_add<MASS>(h, in ? (int)((kh - k) >> sh) : 0, w, lane);
                    }
                    cluster_barrier();
                    // the peers have read the other histogram by now
                    hist_clear(s.hist[level & 1 ? 2 : 0]);
                    hist_find(s, h, base, target, 0.0);
                    const uint32_t b = (uint32_t)s.bin;
                    base = s.base;
                    kh -= b << sh;
                    kl = max(kl, kh - ((1u << sh) - 1));
                    ++level;
                    __syncthreads();
                }
                key = kh;
                const u64 each = MASS ? weight(key_value(kh, T(0))) : 1ull;
                ties = (target - base + each - 1) / each;
            };
            uint32_t key = 0;
            u64 ties = 0;
            if (bin_p == bin) {
                refine(std::true_type(), base_p, target_p, key, ties);
                cut_key = key;
                cut_ties = ties;
            }
            if (bin_k == bin) {
                refine(std::false_type(), base_k, (u64)top_k, key, ties);
                if (key > cut_key || (key == cut_key && ties < cut_ties)) {
                    cut_key = key;
                    cut_ties = ties;
                }
            }
        }
    }

    // ---- kept mass per warp segment, in index order
    u64 mass = 0;
    uint32_t tie = 0;
    for (int i = b0 + lane; i < b1; i += 32) {
        const float v = value_of(data[i]);
        const uint32_t k = key_of(v, T(0));
        if (k >= low_key && k > cut_key)
            mass += weight(v);
        else if (k >= low_key && k == cut_key)
            ++tie;
    }
    mass = warp_sum(mass);
    tie = __reduce_add_sync(0xffffffffu, tie);
    if (lane == 0) {
        s.wmass[warp] = mass;
        s.wtie[warp] = tie;
    }
    cluster_barrier();
    // every CTA adds all segments: thread i takes segment i of the row
    const u64 each = cut_key ? weight(key_value(cut_key, T(0))) : 0;
    {
        const int n = (int)ncta * nwarps;   // at most 256, below blockDim
        u64 m = 0;
        u64 ti = 0;
        if (tid < n) {
            m = ld_peer64(&s.wmass[tid % nwarps], tid / nwarps);
            ti = ld_peer(&s.wtie[tid % nwarps], tid / nwarps);
        }
        // ties before each segment, then the mass each keeps
        u64 t_incl = warp_scan(ti, lane);
        if (lane == 31)
            s.scan[warp] = t_incl;
        __syncthreads();
        for (int w = 0; w < warp; ++w)
            t_incl += s.scan[w];
        const u64 before = t_incl - ti;
        const u64 kept_ties = before >= cut_ties ? 0 : min(ti, cut_ties - before);
        m += kept_ties * each;
        u64 incl = warp_scan(m, lane);
        __syncthreads();
        if (lane == 31)
            s.scan[warp] = incl;
        __syncthreads();
        u64 total = 0;
        for (int w = 0; w < nwarps; ++w) {
            if (w < warp)
                incl += s.scan[w];
            total += s.scan[w];
        }
        // first entry whose running sum exceeds u * total (u >= 1 or NaN:
        // the last one with a weight)
        const double x = (double)__ldg(p.u + row) * (double)total;
        u64 target = total - 1;
        if (x < (double)target)
            target = x > 0.0 ? (u64)x : 0;
        if (tid < n && incl > target && incl - m <= target) {
            s.owner = tid;
            s.owner_base = incl - m;
            s.owner_tie = (uint32_t)min(before, (u64)0xFFFFFFFFu);
            s.total = target;
        }
        __syncthreads();
        const int owner = s.owner;
        if ((int)rank == owner / nwarps && warp == owner % nwarps) {
            u64 run = s.owner_base;
            uint32_t ties = s.owner_tie;
            const u64 want = s.total;
            for (int i = b0 + lane; i - lane < b1; i += 32) {
                u64 w = 0;
                const float v = i < b1 ? value_of(data[i]) : -INFINITY;
                const uint32_t k = key_of(v, T(0));
                const bool in = i < b1 && k >= low_key;
                const unsigned equal = __ballot_sync(0xffffffffu, in && k == cut_key);
                if (in && k > cut_key)
                    w = weight(v);
                else if (in && k == cut_key &&
                         ties + __popc(equal & ((1u << lane) - 1)) < cut_ties)
                    w = each;
                ties += __popc(equal);
                const u64 sum = run + warp_scan(w, lane);
                const unsigned hit = __ballot_sync(0xffffffffu, sum > want);
                if (hit) {
                    if (lane == __ffs(hit) - 1) {
                        p.tokens[row] = lo + i;
                        if (p.probs)
                            p.probs[row] = (float)((double)w / (double)total);
                    }
                    break;
                }
                run = __shfl_sync(0xffffffffu, sum, 31);
            }
        }
    }
    cluster_barrier();   // the peers have read this CTA's shared memory
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
                                 kSmemSlice + 32);
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
    pl.smem = (size_t)pl.per * size + 32;
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
