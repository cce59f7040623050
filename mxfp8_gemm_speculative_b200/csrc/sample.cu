// One token per row of logits from a given random number, after temperature,
// top-p, top-k and min-p (the definition is at sample_logits in mxg.h).
//
// What bounds it: the logits are read once, M V 2 (or 4) bytes; the rest is
// a weight exp((l - max) / T) per entry and the search for the border of the
// kept set.  One row of 248320 bf16 entries is 0.5 MB, 0.08 us of HBM time,
// so a few rows are bound by latency (the steps of a row, one after another)
// and many rows by the arithmetic per entry.
//
// Here a row is taken by one thread-block cluster: every CTA copies its share
// into shared memory and everything after that runs on chip, the CTAs
// exchanging histograms and sums through distributed shared memory.  (Batches
// of bf16 rows and short rows have a kernel of their own further down.)
// Measured (B200, graph of calls): one row of 248320 bf16 22 us, five of 248320
// fp32 30 us, 33 of 32003 fp32 without filters 9.7 us.
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
constexpr int kGroups = 32;       // of 16 bins, a lane each
constexpr int kListCap = 2048;    // entries of the border bin a CTA lists
constexpr int kMaxEntries = 8 * 192 * 1024 / 4;   // fp32 entries that 8 CTAs hold
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

// Weights of one row, round(2^kFix * exp((v - top) / T)), for finite v.  Ten
// fp64 operations, which with the table's reads bound a pass over the row.
constexpr double kMagic = 6755399441055744.0;   // 1.5 * 2^52: adding it rounds to an integer
constexpr double kUnit = 4503599627370496.0;    // 2^52
constexpr double kLog2e = 1.4426950408889634074;
// The table is there 16 times, entry j of copy c at 16 j + c: lane l reads copy
// l mod 16 and no two lanes of a half warp the same bank.  With one copy a read
// took 7 cycles of the pipe and not 2.
constexpr int kCopies = 16;
struct Weights {
    float least;          // 48 binades below the top or lower: no weight
    double c;             // 64 * log2(e) / T
    double k;             // kMagic - top * c, rounded to an integer
    const double *table;  // 2^(j / 64 + kFix), less what that rounding adds; this lane's copy

    // (v - top) / T in units of 1/64 binade: its integer part in the low bits
    __device__ __forceinline__ double scaled(float v) const
    {
        return fma((double)fmaxf(v, least), c, k);
    }

    // First-level bin: 1/16 binade of the weight, the last bin holding
    // everything from 32 binades down.  It never falls as v falls.
    __device__ __forceinline__ int bin(double m) const
    {
        return max(0, min(-__double2loint(m) >> 2, kBins - 1));
    }

    __device__ __forceinline__ int bin(float v) const { return bin(scaled(v)); }

    // 2^(f / 64) - 1 for |f| <= 1/2, by its series to the fourth order, the
    // fifth replaced by its Chebyshev approximation x^5 = (20 h^2 x^3 - 5 h^4 x)
    // / 16 on |x| <= h = ln2 / 128: an error of h^5 / 1920 = 2^-48.5
    __device__ __forceinline__ static double exp_rest(double f)
    {
        constexpr double l = 0.69314718055994530942 / 64.0, h2 = l * l / 4.0;
        constexpr double c1 = l * (1.0 - 5.0 * h2 * h2 / 1920.0), c2 = l * l / 2.0;
        constexpr double c3 = l * l * l * (1.0 / 6.0 + 20.0 * h2 / 1920.0);
        constexpr double c4 = l * l * l * l / 24.0;
        return f * (c1 + f * (c2 + f * (c3 + f * c4)));
    }

    // 2^kFix * the weight, not rounded, of a v that is not below `least`; m = scaled(v)
    __device__ __forceinline__ double exact(float v, double m) const
    {
        const int n = __double2loint(m);
        const double q = exp_rest(fma((double)v, c, k - m));
        const double t = table[(n & 63) * kCopies];
        const double w = fma(t, q, t);
        // times 2^(n / 64) by the exponent field
        return __hiloint2double(__double2hiint(w) + (int)(((uint32_t)n & ~63u) << 14),
                                __double2loint(w));
    }
    __device__ __forceinline__ double exact(float v) const
    {
        return exact(v, fma((double)v, c, k));
    }

    // Weights as the bits of kUnit + weight, which rounds them: the low 52 bits
    // of the sum of up to 255 of those are the sum of the weights.
    __device__ __forceinline__ static u64 raw(double s)
    {
        return (u64)__double_as_longlong(s + kUnit);
    }
    __device__ __forceinline__ static u64 sum_of(u64 raws)
    {
        return raws & 0xFFFFFFFFFFFFFull;
    }

    __device__ __forceinline__ u64 weight(float v, double m) const
    {
        return sum_of(raw(exact(fmaxf(v, least), m)));
    }

    __device__ __forceinline__ u64 operator()(float v) const { return weight(v, scaled(v)); }
};

// The table before a row's own part comes in, by the same threads.
__device__ __forceinline__ void fill_table(double *table)
{
    for (int i = threadIdx.x; i < 64 * kCopies; i += blockDim.x)
        table[i] = exp2((double)(i / kCopies) * (1.0 / 64.0) + kFix);
}

// The weights of a row, by all threads of the CTA.
__device__ __forceinline__ Weights row_weights(float top, float temp, double *table)
{
    // a temperature at which the next lower float has no weight is as good as
    // any below it, and keeps (v - top) / T in range
    const double gap = (double)top - (double)nextafterf(top, -INFINITY);
    const double t = fmax((double)temp, gap * (kLog2e / 48.0));
    Weights w;
    w.c = 64.0 * kLog2e / t;
    w.k = rint(kMagic - (double)top * w.c);
    w.least = fmaxf(__double2float_rd((double)top - 48.0 / kLog2e * t), -FLT_MAX);
    // the top's own rest goes into the table, so that its weight is 1
    const double rest = Weights::exp_rest(-fma((double)top, w.c, w.k - kMagic));
    for (int i = threadIdx.x; i < 64 * kCopies; i += blockDim.x)
        table[i] = fma(table[i], rest, table[i]);
    __syncthreads();
    w.table = table + threadIdx.x % kCopies;
    return w;
}

// The lowest value that passes min-p (the test rises with the value); -inf
// never does.
__device__ __forceinline__ float lowest_kept(float top, float temp, float min_p)
{
    float low = -FLT_MAX;
    if (min_p > 0.f) {
        const double cut = (double)temp * log(fmin((double)min_p, 1.0));
        low = fmaxf(__double2float_rd((double)top + cut), -FLT_MAX);
        for (int i = 0; i < 2 && low > -FLT_MAX; ++i) {
            const float below = nextafterf(low, -INFINITY);
            if ((double)below - (double)top >= cut)
                low = below;
        }
        for (int i = 0; i < 3 && (double)low - (double)top < cut; ++i)
            low = nextafterf(low, INFINITY);
    }
    return low;
}

// ------------------------------------------------------------ shared memory
struct Hist {
    uint32_t lo[kBins], hi[kBins];   // 64-bit sums in two words
    u64 group[kGroups];              // sums of kBins / kGroups bins
};

// A search for a border: the bins of the next histogram are the 2^sh keys
// each from r down to l, and `base` lies above them.
struct Search {
    u64 target, base;
    uint32_t l, r;
    int sh;
    int bin;      // first level: the border's bin, kBins without a border
};

struct Shared {
    double table[64 * kCopies];
    Hist hist[2][2];             // [level parity][masses, counts]
    Search find[2];              // top-p (masses), top-k (counts)
    uint32_t list[kListCap];     // keys of the border bin
    u64 wmass[kMaxWarps];        // kept mass above the cut, per warp segment
    uint32_t wtie[kMaxWarps];    // entries equal to the cut, per warp segment
    uint32_t red[kMaxWarps];
    int listed;
    uint32_t bound[2];           // the border bin's largest and smallest key
    // exchanged with the peers
    uint32_t top_key, first;     // largest key; first index of the maximum
    u64 mass;                    // kept mass above the cut
    uint32_t ties;               // entries equal to the cut
};

__device__ __forceinline__ u64 warp_sum(u64 v)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The same of values below 2^63 in three parts of 21 bits: three reductions of
// the warp side by side, for five rounds of two shuffles.
__device__ __forceinline__ u64 warp_sum63(u64 v)
{
    const uint32_t a = __reduce_add_sync(0xffffffffu, (uint32_t)v & 0x1FFFFFu);
    const uint32_t b = __reduce_add_sync(0xffffffffu, (uint32_t)(v >> 21) & 0x1FFFFFu);
    const uint32_t c = __reduce_add_sync(0xffffffffu, (uint32_t)(v >> 42));
    return a + ((u64)b << 21) + ((u64)c << 42);
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

// Adds w to a bin of this CTA's histogram.  Integer sums: their order does not
// matter; the low words carry into the high ones (a 64-bit shared-memory
// atomic is a compare-and-swap loop, 43 cycles a warp against 9 for the two).
template <bool MASS>
__device__ __forceinline__ void hist_add(Hist &h, int bin, u64 w)
{
    const uint32_t lo = (uint32_t)w;
    if (!MASS) {
        if (lo)
            atomicAdd(&h.lo[bin], lo);
    } else if (w) {
        const uint32_t old = atomicAdd(&h.lo[bin], lo);
        const uint32_t hi = (uint32_t)(w >> 32) + (old + lo < old ? 1u : 0u);
        if (hi)
            atomicAdd(&h.hi[bin], hi);
    }
}

__device__ __forceinline__ void hist_clear(Hist &h)
{
    for (int i = threadIdx.x; i < kBins; i += blockDim.x) {
        h.lo[i] = 0;
        h.hi[i] = 0;
    }
}

// The sums of this CTA's groups of bins, from a complete histogram: a thread
// per group of 16, one after another (few bins, off no critical path wider
// than a barrier).
__device__ __forceinline__ void hist_groups(Hist &h, int thread)
{
    if (thread >= 0 && thread < kGroups) {
        u64 v = 0;
#pragma unroll
        for (int j = 0; j < kBins / kGroups; ++j) {
            // each thread starts at another bank
            const int i = thread * (kBins / kGroups) + ((j + thread) & (kBins / kGroups - 1));
            v += (u64)h.lo[i] + ((u64)h.hi[i] << 32);
        }
        h.group[thread] = v;
    }
}

// The border in the cluster's histogram h, by one warp: the first bin whose
// running sum from `base` reaches the target, with the sum before it in base;
// kBins when none does.  target = 0: ceil(p * (sum of all bins)), at least 1.
// Reads the peers' groups first, then the bins of one group: a quarter of a
// kilobyte per peer and not the four of the whole histogram.
__device__ __forceinline__ int hist_find(const Hist &h, u64 &base, u64 &target, double p, int lane)
{
    const uint32_t n = cluster_size();
    u64 v = 0;
    for (uint32_t c0 = 0; c0 < n; c0 += 8) {
        u64 part[8];
#pragma unroll
        for (uint32_t c = 0; c < 8; ++c)
            part[c] = c0 + c < n ? ld_peer64(&h.group[lane], c0 + c) : 0;
#pragma unroll
        for (uint32_t c = 0; c < 8; ++c)
            v += part[c];
    }
    u64 incl = base + warp_scan(v, lane);
    if (target == 0)
        target = max(1ull, (u64)ceil(p * (double)(__shfl_sync(0xffffffffu, incl, 31) - base)));
    const unsigned over = __ballot_sync(0xffffffffu, incl >= target);
    if (!over)
        return kBins;
    const int g = __ffs(over) - 1;
    base = __shfl_sync(0xffffffffu, incl - v, g);
    // 16 bins, the peers shared between the halves of the warp
    constexpr int kPer = kBins / kGroups;
    const int i = g * kPer + lane % kPer;
    v = 0;
    for (uint32_t c0 = 0; c0 < n; c0 += 8) {
        uint32_t lo[4], hi[4];
#pragma unroll
        for (uint32_t c = 0; c < 4; ++c) {
            const uint32_t peer = c0 + 2 * c + lane / kPer;
            lo[c] = peer < n ? ld_peer(&h.lo[i], peer) : 0;
            hi[c] = peer < n ? ld_peer(&h.hi[i], peer) : 0;
        }
#pragma unroll
        for (uint32_t c = 0; c < 4; ++c)
            v += (u64)lo[c] + ((u64)hi[c] << 32);
    }
    v += __shfl_xor_sync(0xffffffffu, v, kPer);
    if (lane >= kPer)
        v = 0;
    incl = base + warp_scan(v, lane);
    const int b = __ffs(__ballot_sync(0xffffffffu, incl >= target)) - 1;
    base = __shfl_sync(0xffffffffu, incl - v, b);
    return g * kPer + b;
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
    const int tid = threadIdx.x, lane = tid & 31, warp = uniform_warp();
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
    fill_table(s.table);
    for (int i = 0; i < 4; ++i)
        hist_clear(s.hist[i / 2][i % 2]);
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
    const float temp = p.temperature ? __ldcg(p.temperature + row) : 1.f;
    const float top_p = p.top_p ? __ldcg(p.top_p + row) : 1.f;
    const float min_p = p.min_p ? __ldcg(p.min_p + row) : 0.f;
    const int top_k = p.top_k ? __ldcg(p.top_k + row) : 0;
    const float u = __ldcg(p.u + row);

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
            const float a = canonical(value_of(__ldcg(src + i)));
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

    const Weights weight = row_weights(top, temp, s.table);
    const float low = lowest_kept(top, temp, min_p);

    // ---- the cut of top-p and top-k: keep values above it, and the first
    // cut_ties in index order of those equal to it
    const bool use_p = __any_sync(0xffffffffu, top_p < 1.f);
    const bool use_k = __any_sync(0xffffffffu, top_k > 0);
    float cut = -INFINITY;
    u64 cut_ties = 0;
    if (use_p || use_k) {
        // first level: all entries, four a lane and step
        auto first_level = [&](auto with_p, auto with_k) {
            constexpr bool P = decltype(with_p)::value, K = decltype(with_k)::value;
            for (int i = b0 + 4 * lane; i < b1; i += 128) {
                float v[4];
                load4(data, i, v);
                u64 w[4] = {};
                int bin[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const double m = weight.scaled(v[e]);
                    bin[e] = weight.bin(m);
                    if (P)
                        w[e] = v[e] > -INFINITY ? weight.weight(v[e], m) : 0;
                }
                // a warp whose entries fall into one bin (rows of equal
                // values) adds them up first: 32 atomics on one word run one
                // after another
                const bool one = bin[0] == __shfl_sync(0xffffffffu, bin[0], 0) &&
                                 bin[1] == bin[0] && bin[2] == bin[0] && bin[3] == bin[0];
                if (__all_sync(0xffffffffu, one)) {
                    const u64 sum = P ? warp_sum(w[0] + w[1] + w[2] + w[3]) : 0;
                    uint32_t n = 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        n += v[e] > -INFINITY;
                    n = K ? __reduce_add_sync(0xffffffffu, n) : 0;
                    if (lane == 0) {
                        if (P)
                            hist_add<true>(s.hist[0][0], bin[0], sum);
                        if (K)
                            hist_add<false>(s.hist[0][1], bin[0], n);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (P)
                            hist_add<true>(s.hist[0][0], bin[e], w[e]);
                        if (K)
                            hist_add<false>(s.hist[0][1], bin[e], v[e] > -INFINITY);
                    }
                }
            }
        };
        if (use_p && use_k)
            first_level(std::true_type(), std::true_type());
        else if (use_p)
            first_level(std::true_type(), std::false_type());
        else
            first_level(std::false_type(), std::true_type());
        // completes this level's histograms in the cluster
        int level = 0;
        auto exchange = [&](bool do_p, bool do_k) {
            __syncthreads();
            if (do_p)
                hist_groups(s.hist[level & 1][0], tid);
            if (do_k)
                hist_groups(s.hist[level & 1][1], tid - 64);
            cluster_barrier();
        };
        exchange(use_p, use_k);
        // warp 0 looks for top-p's border, warp 1 for top-k's
        if (warp < 2) {
            u64 base = 0, target = warp ? (u64)max(top_k, 0) : 0;
            // no border: the filter is off, or keeps all
            int bin = hist_find(s.hist[0][warp], base, target, (double)top_p, lane);
            if (!(warp ? use_k : use_p))
                bin = kBins;
            if (lane == 0)
                s.find[warp] = Search{target, base, 0, 0, 0, bin};
        }
        __syncthreads();
        // the stricter filter decides; both are followed when their borders
        // fall into one bin
        const int bin = min(s.find[0].bin, s.find[1].bin);
        if (bin < kBins) {
            const bool do_p = s.find[0].bin == bin, do_k = s.find[1].bin == bin;
            // the bin's keys are kl .. kh: a warp for each end
            if (warp < 2) {
                const uint32_t k_min = key_of(-FLT_MAX, T(0)), k_top = key_of(top, T(0));
                // the last key whose bin is at least `bin` (kh), or above it (kl - 1)
                const int least = bin + warp;
                auto yes = [&](uint32_t k) { return weight.bin(key_value(k, T(0))) >= least; };
                uint32_t k = last_key(k_min, k_top, lane, yes);
                if (warp == 1)
                    k = yes(k_min) ? k + 1 : k_min;
                if (lane == 0)
                    s.bound[warp] = k;
            }
            __syncthreads();
            const uint32_t kh = s.bound[0], kl = s.bound[1];
            const float vl = key_value(kl, T(0)), vh = key_value(kh, T(0));
            const int sh0 = max(0, 32 - __clz(kh - kl) - 9);   // bins of 2^sh keys from kh down
            if (tid < 2) {
                s.find[tid].l = kl;
                s.find[tid].r = kh;
                s.find[tid].sh = sh0;
            }
            // second level: histograms of those keys, and a list of them for
            // the levels behind it (when they are too many for the list, those
            // look through the slots again)
            for (int i = b0 + 4 * lane; i < b1; i += 128) {
                float v[4];
                load4(data, i, v);
                bool in[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    in[e] = v[e] >= vl && v[e] <= vh;
                if (!__any_sync(0xffffffffu, in[0] || in[1] || in[2] || in[3]))
                    continue;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const unsigned found = __ballot_sync(0xffffffffu, in[e]);
                    if (!found)
                        continue;
                    const uint32_t k = key_of(v[e], T(0));
                    const int b = in[e] ? (int)((kh - k) >> sh0) : 0;
                    u64 w = in[e] && do_p ? weight(v[e]) : 0;
                    uint32_t n = in[e];
                    const int f = __ffs(found) - 1;
                    const int bf = __shfl_sync(0xffffffffu, b, f);
                    if (__all_sync(0xffffffffu, !in[e] || b == bf)) {   // as above
                        w = do_p ? warp_sum(w) : 0;
                        n = __popc(found);
                        if (lane != f)
                            w = n = 0;
                    }
                    if (do_p)
                        hist_add<true>(s.hist[1][0], b, w);
                    if (do_k)
                        hist_add<false>(s.hist[1][1], b, n);
                    if (sh0 > 0) {
                        int at = 0;
                        if (lane == 0)
                            at = atomicAdd(&s.listed, __popc(found));
                        at = __shfl_sync(0xffffffffu, at, 0) + __popc(found & ((1u << lane) - 1));
                        if (in[e] && at < kListCap)
                            s.list[at] = k;
                    }
                }
            }
            // further levels, until both searches are at one key
            bool open = true;
            while (open) {
                level ^= 1;
                exchange(do_p, do_k);
                hist_clear(s.hist[level ^ 1][0]);   // the peers have read these by now
                hist_clear(s.hist[level ^ 1][1]);
                if (warp < 2 && (warp ? do_k : do_p) && s.find[warp].sh >= 0) {
                    Search f = s.find[warp];
                    const int b = hist_find(s.hist[level][warp], f.base, f.target, 0.0, lane);
                    f.r -= (uint32_t)b << f.sh;
                    f.l = max(f.l, f.r - ((1u << f.sh) - 1));
                    // the next bins, or -1: l = r is the border
                    f.sh = f.l < f.r ? max(0, 32 - __clz(f.r - f.l) - 9) : -1;
                    __syncwarp();
                    if (lane == 0)
                        s.find[warp] = f;
                }
                __syncthreads();
                const Search fp = s.find[0], fk = s.find[1];
                const bool more_p = do_p && fp.sh >= 0, more_k = do_k && fk.sh >= 0;
                open = more_p || more_k;
                if (!open)
                    break;
                const bool listed = s.listed <= kListCap;
                const int entries = listed ? s.listed : used;
                for (int i = tid; i < entries; i += blockDim.x) {
                    const uint32_t k = listed ? s.list[i] : key_of(value_of(data[i]), T(0));
                    if (more_p && k >= fp.l && k <= fp.r)
                        hist_add<true>(s.hist[level ^ 1][0], (int)((fp.r - k) >> fp.sh),
                                       weight(key_value(k, T(0))));
                    if (more_k && k >= fk.l && k <= fk.r)
                        hist_add<false>(s.hist[level ^ 1][1], (int)((fk.r - k) >> fk.sh), 1ull);
                }
            }
            // the stricter cut of the two
            uint32_t cut_key = 0;
            if (do_p) {
                cut_key = s.find[0].r;
                const u64 each = weight(key_value(cut_key, T(0)));
                cut_ties = (s.find[0].target - s.find[0].base + each - 1) / each;
            }
            if (do_k) {
                const u64 ties = s.find[1].target - s.find[1].base;
                const uint32_t key = s.find[1].r;
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
    // (fewer than 256 a lane)
    static_assert(kSmemSlice / 2 + kSlack < 256 * 512, "entries a CTA, at two bytes and 512 threads");
    u64 raws = 0;
    uint32_t tie = 0;
    // four weights side by side, where any of the four is kept
    auto add_kept = [&](const float (&v)[4]) {
        if (fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])) < keep)
            return;
        u64 w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            w[e] = Weights::raw(weight.exact(fmaxf(v[e], weight.least)));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const bool in = v[e] >= keep, eq = v[e] == cut;
            if (in && !eq)
                raws += w[e];
            tie += in && eq;
        }
    };
    for (int i = b0 + 4 * lane; i < b1; i += 128) {
        float v[4];
        load4(data, i, v);
        add_kept(v);
    }
    const u64 mass = warp_sum(Weights::sum_of(raws));
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
            raws = 0;
            tie = 0;
            for (int i = b0 + lane * sub; i < min(b1, b0 + (lane + 1) * sub); i += 4) {
                float v[4];
                load4(data, i, v);
                add_kept(v);
            }
            __syncwarp();
            part = of(Weights::sum_of(raws), tie, ties_before);
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

// --------------------------------------------------- bf16 rows, one CTA a row
// A batch with a row for most SMs has nothing to split, and bf16 has 65536
// values only: a CTA counts how often each occurs (one shared-memory atomic an
// entry, against a weight of some 40 instructions and two atomics), computes
// the weight of every value that occurs once, and finds the cut from the
// products.  A second pass over the row, out of L2, adds the kept weights per
// step of 256 entries, from the end nearer to the token and no further.  The
// integers are those of the kernel above, and so are the tokens.
//
// Measured: 128 rows of 248320, mixed filters, 58 us (clusters: 161 us), of
// which the counting pass takes 21 us (14 us of atomics with their bank
// conflicts), the sums over the counters and the borders 6 us, the second pass
// 2 to 11 us by the row; 8 rows of 5003 12 us.
//
// Counters: word i counts the values of magnitude i, the negative ones in its
// low half and the positive ones in its high half.  A half that overflows (a
// value that occurs more than 65535 times) makes the sum of all halves fall
// short of the number of entries; the row is then counted in 32 bits, the
// negative values first.
constexpr int kTableThreads = 1024;
constexpr int kTableWords = 32768;
constexpr int kTableParts = 2048;   // runs of 32 keys from the top; steps of 256 entries
static_assert((kMaxEntries + 7 + 255) / 256 <= kTableParts, "a sum per step");
static_assert(kTableParts == 2 * kTableThreads, "two sums a thread");
constexpr int kBatches = kTableParts / 128;   // most batches of 128 steps
static_assert(kBatches <= 32, "a lane each");

struct Border {
    int run;             // the run of keys it is in, -1: none
    u64 mass, n;         // sums of the runs above
    u64 target;          // what the search's sum has to reach
    uint32_t key;
    u64 ties;            // entries equal to the key that are kept
    u64 above, equal;    // mass above the key, entries equal to it
};

struct Table {
    uint32_t count[kTableWords];
    u64 mass[kTableParts];       // per run of keys, then per step
    uint32_t n[kTableParts];
    double table[64 * kCopies];
    u64 scan[2][32];             // warps' sums of a scan
    float guess[kBatches];       // mass per batch, roughly
    uint32_t red[2][32];
    Border border[3];            // of top-p, top-k and min-p
    uint32_t first;
};

// Keys of two bf16 in a word, -0 as +0: all bits of a negative value and the
// sign bit of a positive one flipped.
__device__ __forceinline__ uint32_t keys_of(uint32_t w)
{
    uint32_t sign;
    asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(w) : "r"(0u));
    asm("prmt.b32 %0, %1, 0, 0xBB99;" : "=r"(sign) : "r"(w));
    return w ^ (sign | 0x80008000u);
}
// Neither NaN nor -inf.
__device__ __forceinline__ bool key_counts(uint32_t k)
{
    return k - 0x0080u <= 0xFF80u - 0x0080u;
}
// The counter of a key.
__device__ __forceinline__ uint32_t word_of(uint32_t k)
{
    return k >> 15 ? k & 0x7FFFu : 0x7FFFu - k;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b)   // of two bf16 each, NaN least
{
    uint32_t d;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t equal2(uint32_t a, uint32_t b)   // ones where equal
{
    return __heq2_mask(reinterpret_cast<const __nv_bfloat162 &>(a),
                       reinterpret_cast<const __nv_bfloat162 &>(b));
}

// Inclusive sum over the threads before and at this one of v, and of all.
__device__ __forceinline__ u64 block_scan(u64 v, u64 (&sums)[32], int lane, int warp, u64 &all)
{
    u64 incl = warp_scan(v, lane);
    if (lane == 31)
        sums[warp] = incl;
    __syncthreads();
    const u64 w = warp_scan(sums[lane], lane);
    all = __shfl_sync(0xffffffffu, w, 31);
    return incl + (warp ? __shfl_sync(0xffffffffu, w, warp - 1) : 0);
}

__global__ void __launch_bounds__(kTableThreads, 1) sample_table_kernel(const SampleParams p)
{
    extern __shared__ __align__(16) uint8_t dyn[];
    Table &s = *reinterpret_cast<Table *>(dyn);
    const int tid = threadIdx.x, lane = tid & 31, warp = uniform_warp();
    const int row = blockIdx.x;
    const uint16_t *src = static_cast<const uint16_t *>(p.logits) + row * p.ld;
    // vectors of 8 slots at 16-byte boundaries: slot e is entry e - skew
    const int skew = (int)(reinterpret_cast<uintptr_t>(src) & 15u) / 2;
    const int vecs = (skew + p.V + 7) / 8;
    auto load = [&](int i) {
        const int e = 8 * i - skew;
        if (e >= 0 && e + 8 <= p.V)
            return __ldcg(reinterpret_cast<const uint4 *>(src + e));
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int a = e + 2 * j, b = a + 1;
            w[j] = (a >= 0 && a < p.V ? __ldcg(src + a) : 0xFF80u) |
                   (b >= 0 && b < p.V ? (uint32_t)__ldcg(src + b) : 0xFF80u) << 16;
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    };
    // a batch of 128 steps: every warp takes four, all four in flight
    auto for_batch = [&](int batch, auto body) {
        const int i0 = batch * 4 * kTableThreads + warp * 32;
        uint4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = i0 + j * kTableThreads + lane;
            v[j] = make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);
            if (i < vecs)
                v[j] = load(i);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i0 + j * kTableThreads < vecs) {
                const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
                body((i0 + j * kTableThreads) / 32, w);
            }
    };
    auto for_steps = [&](auto body) {
        for (int b = 0; b * 4 * kTableThreads < vecs; ++b)
            for_batch(b, body);
    };
    auto clear = [&] {
        for (int i = tid; i < kTableWords / 4; i += kTableThreads)
            reinterpret_cast<uint4 *>(s.count)[i] = make_uint4(0, 0, 0, 0);
    };
    clear();
    fill_table(s.table);
    for (int i = tid; i < kTableParts; i += kTableThreads) {
        s.mass[i] = 0;
        s.n[i] = 0;
    }
    if (tid < kBatches)
        s.guess[tid] = 0.f;
    if (tid == 0) {
        s.border[0].run = s.border[1].run = -1;
        s.first = 0xFFFFFFFFu;
    }
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    const float temp = p.temperature ? __ldcg(p.temperature + row) : 1.f;
    const float top_p = p.top_p ? __ldcg(p.top_p + row) : 1.f;
    const float min_p = p.min_p ? __ldcg(p.min_p + row) : 0.f;
    const int top_k = p.top_k ? __ldcg(p.top_k + row) : 0;
    const float u = __ldcg(p.u + row);
    const bool greedy = __any_sync(0xffffffffu, !(temp > 0.f));

    // ---- first pass: the largest key, and how often each occurs
    uint32_t top2 = 0xFF80FF80u, entries = 0;
    auto count = [&](const uint32_t (&w)[4]) {
        top2 = max2(top2, max2(max2(w[0], w[1]), max2(w[2], w[3])));
        // a warp whose entries are all equal adds them up first
        if (__all_sync(0xffffffffu, w[0] == __shfl_sync(0xffffffffu, w[0], 0))) {
            const bool one = w[1] == w[0] && w[2] == w[0] && w[3] == w[0] &&
                             w[0] >> 16 == (w[0] & 0xFFFFu);
            if (__all_sync(0xffffffffu, one)) {
                if (w[0] < 0xFF800000u) {
                    entries += 8;
                    if (lane == 0)
                        atomicAdd(&s.count[w[0] >> 16 & 0x7FFFu], w[0] >> 31 ? 256u : 256u << 16);
                }
                return;
            }
        }
        // -inf and the negative NaNs are left out; the counters of the
        // others are not looked at
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t b = j & 1 ? w[j / 2] : w[j / 2] << 16;
            if (b < 0xFF800000u) {
                const uint32_t neg = (uint32_t)((int32_t)b >> 31);
                ++entries;
                atomicAdd(&s.count[b >> 16 & 0x7FFFu], (neg & 1u) | (~neg & 0x10000u));
            }
        }
    };
    // in 32 bits, one sign only
    auto count_wide = [&](uint32_t sign) {
        for_steps([&](int, const uint32_t (&w)[4]) {
            uint32_t k[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                k[j] = keys_of(w[j]);
            const uint32_t k0 = __shfl_sync(0xffffffffu, k[0], 0);
            const bool one = k[0] == k0 && k[1] == k0 && k[2] == k0 && k[3] == k0 &&
                             k0 >> 16 == (k0 & 0xFFFFu);
            const bool all = __all_sync(0xffffffffu, one);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t key = j & 1 ? k[j / 2] >> 16 : k[j / 2] & 0xFFFFu;
                if (key_counts(key) && key >> 15 == sign && (!all || (lane == 0 && j == 0)))
                    atomicAdd(&s.count[word_of(key)], all ? 256u : 1u);
            }
        });
    };
    if (!greedy) {
        // and, for the order of the second pass, a rough mass per batch: the
        // largest weight of every eight entries, in fp32 and relative to the
        // largest of the first 256
        const uint4 v = lane < vecs ? load(lane) : make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u,
                                                               0xFF80FF80u);
        const uint32_t ref2 = max2(max2(v.x, v.y), max2(v.z, v.w));
        const float ref = key_value(
            __reduce_max_sync(0xffffffffu,
                              key_of(fmaxf(__uint_as_float(ref2 << 16),
                                           __uint_as_float(ref2 & 0xFFFF0000u)), 0u)), 0u);
        const float c = (float)kLog2e / temp;
        const float d = fabsf(ref) < INFINITY ? -ref * c : 0.f;
        for (int b = 0; b * 4 * kTableThreads < vecs; ++b) {
            float g = 0.f;
            for_batch(b, [&](int, const uint32_t (&w)[4]) {
                const uint32_t top2 = max2(max2(w[0], w[1]), max2(w[2], w[3]));
                g += exp2_approx(fmaf(fmaxf(__uint_as_float(top2 << 16),
                                            __uint_as_float(top2 & 0xFFFF0000u)), c, d));
                count(w);
            });
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1)
                g += __shfl_xor_sync(0xffffffffu, g, o);
            if (lane == 0)
                atomicAdd(&s.guess[b], g);
        }
    } else {
        for_steps([&](int, const uint32_t (&w)[4]) {
            top2 = max2(top2, max2(max2(w[0], w[1]), max2(w[2], w[3])));
        });
    }
    // 0: nothing but NaN and -inf
    uint32_t top_key = keys_of(top2);
    top_key = max(top_key & 0xFFFFu, top_key >> 16);
    top_key = __reduce_max_sync(0xffffffffu, key_counts(top_key) ? top_key : 0u);
    entries = __reduce_add_sync(0xffffffffu, entries);
    if (lane == 0) {
        s.red[0][warp] = top_key;
        s.red[1][warp] = entries;
    }
    __syncthreads();
    top_key = __reduce_max_sync(0xffffffffu, s.red[0][lane]);
    entries = __reduce_add_sync(0xffffffffu, s.red[1][lane]);

    if (top_key == 0 || greedy) {   // nothing to take, or greedy
        uint32_t first = 0xFFFFFFFFu;
        if (top_key)
            for_steps([&](int step, const uint32_t (&w)[4]) {
#pragma unroll
                for (int j = 7; j >= 0; --j) {
                    const uint32_t k = keys_of(w[j / 2]);
                    if ((j & 1 ? k >> 16 : k & 0xFFFFu) == top_key)
                        first = min(first, (uint32_t)(256 * step + 8 * lane + j - skew));
                }
            });
        first = __reduce_min_sync(0xffffffffu, first);
        if (lane == 0 && first != 0xFFFFFFFFu)
            atomicMin(&s.first, first);
        __syncthreads();
        if (tid == 0) {
            p.tokens[row] = (int)s.first;
            if (p.probs)
                p.probs[row] = top_key ? 1.f : 0.f;
        }
        return;
    }
    // the +inf entries share the mass, with a weight of 1 each
    const bool inf = top_key == 0xFF80u;
    const float top = inf ? 0.f : key_value(top_key, uint16_t(0));
    const uint32_t least_key = inf ? top_key : 0x0080u;
    const Weights weight = row_weights(top, temp, s.table);
    auto key_weight = [&](uint32_t k) { return weight(inf ? 0.f : key_value(k, uint16_t(0))); };
    // the lowest key that min-p keeps: a bound between two bf16 truncates to
    // the one nearer to zero, which a positive bound leaves out; -0 does not occur
    const float low = lowest_kept(top, temp, min_p);
    uint32_t low_key = key_of(low, uint16_t(0));
    low_key += key_value(low_key, uint16_t(0)) < low || low_key == 0x7FFFu;
    low_key = max(least_key, low_key);

    // ---- mass and number of the entries in each run of 32 keys; run r holds
    // the keys from 0xFFFF - 32 r down
    uint32_t sum = 0;
    auto run_of = [](uint32_t k) { return kTableParts - 1 - (int)(k >> 5); };
    // counters of the magnitudes i .. i + 3, eight lanes a run: the negative
    // and the positive values of each in 16 bits, or those of one sign in 32
    auto sum_runs = [&](uint32_t i, const uint4 &words, uint32_t half) {
        if (!__any_sync(0xffffffffu, words.x | words.y | words.z | words.w))
            return;
        const uint32_t c[4] = {words.x, words.y, words.z, words.w};
        u64 mn = 0, mp = 0;
        uint32_t nn = 0, np = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t neg = half == 2 ? c[j] & 0xFFFFu : half == 0 ? c[j] : 0;
            uint32_t pos = half == 2 ? c[j] >> 16 : half == 1 ? c[j] : 0;
            sum += neg + pos;
            const uint32_t kp = 0x8000u + i + j, kn = 0x7FFFu - i - j;
            if (i + j == 0) {   // -0 is +0
                pos += neg;
                neg = 0;
            }
            neg = kn >= least_key ? neg : 0;
            pos = kp >= least_key && kp <= 0xFF80u ? pos : 0;
            const u64 wn = neg * key_weight(kn), wp = pos * key_weight(kp);
            mn += neg ? wn : 0;
            mp += pos ? wp : 0;
            nn += neg;
            np += pos;
        }
#pragma unroll
        for (int o = 4; o >= 1; o >>= 1) {
            mn += __shfl_xor_sync(0xffffffffu, mn, o);
            mp += __shfl_xor_sync(0xffffffffu, mp, o);
            nn += __shfl_xor_sync(0xffffffffu, nn, o);
            np += __shfl_xor_sync(0xffffffffu, np, o);
        }
        if (lane % 8 == 0 && half != 1) {
            s.mass[run_of(0x7FFFu - i)] = mn;
            s.n[run_of(0x7FFFu - i)] = nn;
        }
        if (lane % 8 == 0 && half != 0) {
            s.mass[run_of(0x8000u + i)] = mp;
            s.n[run_of(0x8000u + i)] = np;
        }
    };
    // all counters, 128 a warp and step, so that the values between two powers
    // of two go to one warp and those between the next two to the next
    auto sum_all = [&](uint32_t half) {
        for (int i = 4 * tid; i < kTableWords; i += 4 * kTableThreads)
            sum_runs(i, *reinterpret_cast<const uint4 *>(s.count + i), half);
    };
    sum_all(2);
    sum = __reduce_add_sync(0xffffffffu, sum);
    if (lane == 0)
        s.red[0][warp] = sum;
    __syncthreads();
    const bool wide = __reduce_add_sync(0xffffffffu, s.red[0][lane]) != entries;
    auto recount = [&](uint32_t sign) {
        __syncthreads();
        clear();
        __syncthreads();
        count_wide(sign);
        __syncthreads();
    };
    if (wide) {
        for (int i = tid; i < kTableParts; i += kTableThreads) {
            s.mass[i] = 0;
            s.n[i] = 0;
        }
        recount(0);
        sum_all(0);
        recount(1);
        sum_all(1);
        __syncthreads();
    }

    // ---- the runs in which the borders of top-p, top-k and min-p are
    {
        const u64 m0 = s.mass[2 * tid], m1 = s.mass[2 * tid + 1];
        const u64 n0 = s.n[2 * tid], n1 = s.n[2 * tid + 1];
        u64 all_m, all_n;
        const u64 m = block_scan(m0 + m1, s.scan[0], lane, warp, all_m) - m0 - m1;
        const u64 n = block_scan(n0 + n1, s.scan[1], lane, warp, all_n) - n0 - n1;
        auto found = [&](Border &b, int which, u64 target) {
            b.run = 2 * tid + which;
            b.mass = which ? m + m0 : m;
            b.n = which ? n + n0 : n;
            b.target = target;
        };
        if (top_p < 1.f) {
            const u64 target = max(1ull, (u64)ceil((double)top_p * (double)all_m));
            if (m < target && target <= m + m0 + m1)
                found(s.border[0], m + m0 < target, target);
        }
        if (top_k > 0) {
            const u64 target = (u64)top_k;
            if (n < target && target <= n + n0 + n1)
                found(s.border[1], n + n0 < target, target);
        }
        if (run_of(low_key) >> 1 == tid)
            found(s.border[2], run_of(low_key) & 1, 0);
    }
    __syncthreads();
    // the key in its run: a warp for each border; in 32 bits the positive
    // keys (the upper runs) are there and the negative ones counted again
    auto resolve = [&](int first_run, int last_run) {
        if (warp >= 3 || s.border[warp].run < first_run || s.border[warp].run > last_run)
            return;
        Border &b = s.border[warp];
        const uint32_t k = 0xFFFFu - 32 * b.run - lane;
        uint32_t c = s.count[word_of(k)];
        if (!wide)
            c = k == 0x8000u ? (c >> 16) + (c & 0xFFFFu) : k >> 15 ? c >> 16 : c & 0xFFFFu;
        if (k < least_key || k > 0xFF80u || k == 0x7FFFu)
            c = 0;
        const u64 each = c ? key_weight(k) : 0ull;
        const u64 m = b.mass + warp_scan(c * each, lane);
        const u64 n = b.n + warp_scan(c, lane);
        const bool in = warp == 0 ? m >= b.target : warp == 1 ? n >= b.target : k == low_key;
        if (lane == __ffs(__ballot_sync(0xffffffffu, in)) - 1) {
            b.key = k;
            b.above = m - c * each;
            b.equal = c;
            // what is missing to the target, in whole entries
            b.ties = warp == 0 ? (b.target - b.above + each - 1) / each
                               : warp == 1 ? b.target - (n - c) : c;
        }
    };
    if (!wide) {
        resolve(0, kTableParts - 1);
    } else {
        resolve(0, kTableParts / 2 - 1);
        const bool again = max(max(s.border[0].run, s.border[1].run), s.border[2].run) >=
                           kTableParts / 2;
        if (again) {
            recount(0);
            resolve(kTableParts / 2, kTableParts - 1);
        }
    }
    __syncthreads();
    // the strictest: keep values above the cut, and the first cut_ties in
    // index order of those equal to it
    int strict = 2;
    for (int i = 0; i < 2; ++i)
        if (s.border[i].run >= 0 &&
            (s.border[i].key > s.border[strict].key ||
             (s.border[i].key == s.border[strict].key && s.border[i].ties < s.border[strict].ties)))
            strict = i;
    const float cut = key_value(s.border[strict].key, uint16_t(0));
    const u64 cut_ties = s.border[strict].ties;
    const u64 each = key_weight(s.border[strict].key);
    // kept mass of a part, with the ties before it
    auto of = [&](u64 m, u64 n, u64 before) {
        return m + each * (before >= cut_ties ? 0ull : min(n, cut_ties - before));
    };
    const u64 total = of(s.border[strict].above, s.border[strict].equal, 0);
    const double x = (double)u * (double)total;
    u64 target = total - 1;
    if (x < (double)target)
        target = x > 0.0 ? (u64)x : 0;

    // ---- second pass: kept mass above the cut and ties per step, batches of
    // 128 steps from the nearer end until the target is passed
    // (raw values: NaN is neither above the cut nor equal to it, and -0 is
    // equal to +0 in the comparisons and in the weight)
    const float above = fmaxf(cut, nextafterf(weight.least, -INFINITY));   // below it: no weight
    const uint32_t cut2 = (__float_as_uint(cut) >> 16) * 0x10001u;
    auto kept = [&](const uint32_t (&w)[4], u64 &mass, uint32_t &tie) {
        mass = 0;
        tie = 0;
        const uint32_t top2 = max2(max2(w[0], w[1]), max2(w[2], w[3]));
        if (!__any_sync(0xffffffffu, fmaxf(__uint_as_float(top2 << 16),
                                           __uint_as_float(top2 & 0xFFFF0000u)) >= cut))
            return false;
        u64 raws = 0;
        uint32_t same = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float a = __uint_as_float(w[j] << 16), b = __uint_as_float(w[j] & 0xFFFF0000u);
            const u64 wa = Weights::raw(weight.exact(a)), wb = Weights::raw(weight.exact(b));
            if (a > above)
                raws += wa;
            if (b > above)
                raws += wb;
            same |= equal2(w[j], cut2) & (0x00010001u << j);
        }
        mass = Weights::sum_of(raws);
        tie = __popc(same);
        return true;
    };
    const int batches = (vecs + 4 * kTableThreads - 1) / (4 * kTableThreads);
    bool back;
    {
        // the batch where the guess passes its part of the mass; sums that are
        // not finite, or of entries that the cut leaves out, cost time only
        float g = lane < kBatches ? s.guess[lane] : 0.f;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const float b = __shfl_up_sync(0xffffffffu, g, o);
            g += lane >= o ? b : 0.f;
        }
        const float part = __shfl_sync(0xffffffffu, g, 31) * ((float)target / (float)total);
        const int at = __popc(__ballot_sync(0xffffffffu, g < part));
        back = __any_sync(0xffffffffu, batches - at < at + 1);
    }
    u64 m = back ? s.border[strict].above : 0, n = back ? s.border[strict].equal : 0;
    int batch = back ? batches - 1 : 0;
    while (true) {
        for_batch(batch, [&](int step, const uint32_t (&w)[4]) {
            u64 mass;
            uint32_t tie;
            if (kept(w, mass, tie)) {
                mass = warp_sum63(mass);
                tie = __reduce_add_sync(0xffffffffu, tie);
            }
            if (lane == 0) {
                s.mass[step] = mass;
                s.n[step] = tie;
            }
        });
        __syncthreads();
        // every warp adds the batch up for itself, four steps a lane
        u64 bm = 0;
        uint32_t bn = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int step = batch * 128 + 4 * lane + j;
            if (step * 32 < vecs) {
                bm += s.mass[step];
                bn += s.n[step];
            }
        }
        bm = warp_sum63(bm);
        bn = __reduce_add_sync(0xffffffffu, bn);
        if (back) {
            m -= bm;
            n -= bn;
            if (of(m, n, 0) <= target || batch == 0)
                break;
            --batch;
        } else {
            if (of(m + bm, n + bn, 0) > target || batch == batches - 1)
                break;
            m += bm;
            n += bn;
            ++batch;
        }
    }
    // ---- the step, the lane and the entry where u * (kept mass) falls
    if (warp == 0) {
        u64 run = of(m, n, 0);
        u64 sm[4], sn[4], lane_m = 0, lane_n = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int step = batch * 128 + 4 * lane + j;
            sm[j] = step * 32 < vecs ? s.mass[step] : 0;
            sn[j] = step * 32 < vecs ? s.n[step] : 0;
            lane_m += sm[j];
            lane_n += sn[j];
        }
        u64 ties = n + warp_scan(lane_n, lane) - lane_n;
        u64 part = of(lane_m, lane_n, ties);
        u64 incl = run + warp_scan(part, lane);
        int at = __ffs(__ballot_sync(0xffffffffu, incl > target)) - 1;
        // that lane's step
        run = incl - part;
        int step = batch * 128 + 4 * lane;
#pragma unroll
        for (int j = 0; j < 3; ++j) {
            const u64 mine = of(sm[j], sn[j], ties);
            if (step == batch * 128 + 4 * lane + j && run + mine <= target) {
                run += mine;
                ties += sn[j];
                ++step;
            }
        }
        run = __shfl_sync(0xffffffffu, run, at);
        ties = __shfl_sync(0xffffffffu, ties, at);
        step = __shfl_sync(0xffffffffu, step, at);
        const int i = step * 32 + lane;
        uint4 v = make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);
        if (i < vecs)
            v = load(i);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        u64 mass;
        uint32_t tie;
        kept(w, mass, tie);
        ties += warp_scan(tie, lane) - tie;
        part = of(mass, tie, ties);
        incl = run + warp_scan(part, lane);
        at = __ffs(__ballot_sync(0xffffffffu, incl > target)) - 1;
        // that lane's eight entries, a lane each
        run = __shfl_sync(0xffffffffu, incl - part, at);
        ties = __shfl_sync(0xffffffffu, ties, at);
        uint32_t bits = 0xFF800000u;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t word = __shfl_sync(0xffffffffu, w[j / 2], at);
            if (lane == j)
                bits = j & 1 ? word & 0xFFFF0000u : word << 16;
        }
        const float a = __uint_as_float(bits);
        const unsigned equal = __ballot_sync(0xffffffffu, a == cut);
        const u64 mine = a > above ? weight(a)
                         : a == cut && ties + __popc(equal & ((1u << lane) - 1)) < cut_ties ? each
                                                                                            : 0ull;
        incl = run + warp_scan(mine, lane);
        if (lane == __ffs(__ballot_sync(0xffffffffu, incl > target)) - 1) {
            p.tokens[row] = 8 * (step * 32 + at) + lane - skew;
            if (p.probs)
                p.probs[row] = (float)((double)mine / (double)total);
        }
    }
}

// The kernel's attributes, set once per device.
template <typename T>
cudaError_t prepare_kernel(int dev)
{
    const void *fn = reinterpret_cast<const void *>(&sample_kernel<T>);
    static std::atomic<bool> done[kMaxDeviceCache];
    if (done[dev].load(std::memory_order_acquire))
        return cudaSuccess;
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kSmemSlice + kSlack * (int)sizeof(T));
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess)
        done[dev].store(true, std::memory_order_release);
    return e;
}

// Clusters of 16 CTAs that the device runs at the same time (0 where it takes
// none), asked once per device.
template <typename T>
int wide_clusters_of(int dev)
{
    static std::atomic<int> known[kMaxDeviceCache];   // plus one
    if (dev < 0 || dev >= kMaxDeviceCache)
        return 0;
    int n = known[dev].load(std::memory_order_acquire);
    if (n == 0) {
        int got = 0;
        if (prepare_kernel<T>(dev) == cudaSuccess) {
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = dim3(16);
            cfg.blockDim = dim3(1024);
            cfg.dynamicSmemBytes = (size_t)(kMaxEntries / 16 + kSlack) * sizeof(T);
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 16;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            if (cudaOccupancyMaxActiveClusters(&got, &sample_kernel<T>, &cfg) != cudaSuccess) {
                (void)cudaGetLastError();
                got = 0;
            }
        }
        n = 1 + std::max(0, got);
        known[dev].store(n, std::memory_order_release);
    }
    return n - 1;
}

int wide_clusters(int dev, bool fp32)
{
    return fp32 ? wide_clusters_of<uint32_t>(dev) : wide_clusters_of<uint16_t>(dev);
}

cudaError_t launch_table(const SampleParams &p, cudaStream_t stream)
{
    const void *fn = reinterpret_cast<const void *>(&sample_table_kernel);
    static std::atomic<bool> done[kMaxDeviceCache];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= kMaxDeviceCache)
        return cudaErrorInvalidDevice;
    if (!done[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Table));
        if (e != cudaSuccess)
            return e;
        done[dev].store(true, std::memory_order_release);
    }
    SampleParams q = p;
    void *args[] = {&q};
    return launch_pdl(fn, dim3((unsigned)p.M), dim3(kTableThreads), sizeof(Table), stream, args);
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
    if ((e = prepare_kernel<T>(dev)) != cudaSuccess)
        return e;
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
    return M >= 1 && M <= (1 << 27) && V >= 1 && V <= kMaxEntries;
}

SamplePlan plan_sample(int device, int M, int V, bool fp32, bool filtered)
{
    const int size = fp32 ? 4 : 2;
    SamplePlan pl{};
    const int sms = device_info(device).sms;
    // A row per SM at a time pays off for short rows, which clusters split for
    // little (V = 5003: one row 11.2 us against 12.5, 24 rows 12 against 14), and
    // from a fifth of the SMs on for long ones (V = 128256, top-p: 24 rows 30 us
    // against 35, 64 rows 36 against 55, 148 rows 36 against 106; V = 248320: 24
    // rows 54 against 54).  More rows than SMs queue, where clusters of short
    // rows share SMs (V = 2000: 220 rows 23 us against 14; V = 16384: 28 against
    // 32).  Without top-p and top-k there is no cut to find: many long rows only
    // (V = 128256: 64 rows 36 against 26, 148 rows 36 against 58).
    pl.table = !fp32 && (!filtered ? 3LL * M >= 2 * sms && V >= 65536
                         : M > sms ? V >= 16384
                                   : V <= 16384 || 5LL * M >= sms);
    if (pl.table)
        return pl;
    // a CTA per 4096 entries at least while that leaves SMs idle.  Sixteen CTAs
    // take a GPC, of which a device has one for about 18 SMs
    pl.cluster = 1;
    while (pl.cluster < 8 && ((V > 4096 * pl.cluster && (long long)M * pl.cluster * 2 <= sms) ||
                              (long long)(V + pl.cluster - 1) / pl.cluster * size > 72 * 1024))
        pl.cluster *= 2;
    if (pl.cluster == 8 && V > 8 * 4096 && M <= wide_clusters(device, fp32))
        pl.cluster = 16;
    pl.per = ((V + pl.cluster - 1) / pl.cluster + 7) / 8 * 8;
    // 1024 threads for CTAs that have an SM each, else 512, two CTAs an SM
    // (fp32, mixed filters: 128 rows of 128256 121 us against 190 with 1024, 33
    // rows of 128256 40 against 57; 20 bf16 rows of 128256 39 against 36).
    // Slices of more than half an SM's shared memory leave one CTA on it all the
    // same (128 fp32 rows of 248320: 271 against 253)
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
    if (pl.table)
        return launch_table(p, stream);
    return a.fp32 ? launch_typed<uint32_t>(pl, p, stream) : launch_typed<uint16_t>(pl, p, stream);
}

}  // namespace mxg
