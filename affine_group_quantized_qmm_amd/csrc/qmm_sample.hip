// A token for each row of logits from a given uniform number, after
// temperature, top-k, top-p and min-p.
//
// All filters keep a prefix of one order (falling logit, ties by rising
// index), and the token is where the cumulative kept mass passes u times its
// total. So the operator is a few searches of the form "where does the count
// or the mass of the order cross this value", and none of them needs a sort:
//
//   1. histogram  One pass over the logits. With z = x / T, bin b = rint(8 z)
//                 holds the elements' number and their mass relative to the
//                 bin's centre, e^(z - b/8) = 1 + q with |q| < 0.065, so that a
//                 small polynomial in fp32 gives a weight to 2^-29 and neither
//                 the row's maximum nor a range reduction is needed first.
//                 Weights are integers (2^31 (1 + q)): sums do not depend on
//                 their order. Number and mass share one 64-bit LDS atomic.
//                 Only the 384 bins below the maximum's count: e^-48 of the
//                 largest weight is below 2^-69.
//   2. gather     Cumulative counts and masses over those bins (64-bit floats)
//                 tell which bins each crossing can fall into; the elements
//                 of those bins (tens to hundreds of a vocabulary) are listed.
//   3. finish     Each crossing is resolved inside its bin by narrowing a key
//                 range with 512-way histograms over the list.
//
// Tokens have to be equal to what 64-bit arithmetic gives, whatever the order of
// the sums: the weights' relative errors (below 2^-28, of either sign) shift a
// cumulative sum of n similar tokens by 2^-28 / sqrt(n) of itself, which moves
// a token only if u falls within that of a border.
//
// Rows whose maximum lies outside the histogram's range (|z| of 500, or an
// infinity) are counted again relative to their maximum by the finishing
// workgroup alone, as are rows whose list overflows (thousands of equal
// logits): slower, the same answer.
//
// Each launch reads the logits at most once; a row is cut into slices so that
// few rows still fill the GPU.
#include "qmm_device.hpp"
#include "qmm_kernels.hpp"
#include "qmm_step.hpp"

namespace qmm {
namespace {

constexpr int kScanThreads = 1024;   // histogram and gather
constexpr int kThreads = 512;        // finish
constexpr int kRange = 8192;         // bins of the histogram: z of -512 .. 512
constexpr int kBins = 384;           // bins that count, from the maximum's down
constexpr double kPerUnit = 8.0;     // bins per unit of z
constexpr int kSumBits = 46;         // low field of a packed bin: the sum of q
constexpr float kUnit = 2147483648.0f;   // 2^31: the weight of a bin's centre
constexpr int kMaxSlice = 1 << 17;   // elements of a slice: the packed number has 18 bits, the sum 45 and a sign
constexpr int kMaxSlices = 64;
constexpr int kSliceList = 1024;     // listed elements of a slice
constexpr int kList = 4096;          // listed elements of a row
constexpr double kMagic = 6755399441055744.0;  // 1.5 * 2^52: adding it leaves the nearest integer in the low word

// What a slice leaves behind.
struct SliceHead {
    float top;          // largest logit (-inf: none)
    uint32_t listed;    // elements of the gathered bins, before the cap
    uint32_t pad[2];
};
struct Entry {
    float x;
    uint32_t index;
};
__host__ __device__ constexpr size_t slice_bytes() { return sizeof(SliceHead) + kBins * 8 + kSliceList * sizeof(Entry); }
__device__ __forceinline__ char *slice_at(const SampleArgs &a, int row, int s, int S)
{
    return static_cast<char *>(a.workspace) + ((size_t)row * S + s) * slice_bytes();
}
__device__ __forceinline__ SliceHead *head_of(char *p) { return reinterpret_cast<SliceHead *>(p); }
__device__ __forceinline__ uint64_t *hist_of(char *p) { return reinterpret_cast<uint64_t *>(p + sizeof(SliceHead)); }
__device__ __forceinline__ Entry *list_of(char *p)
{
    return reinterpret_cast<Entry *>(p + sizeof(SliceHead) + kBins * 8);
}

// A row's parameters. T <= 0 (or NaN) asks for the largest logit: the first
// of the order, that is top-k of 1 at any temperature.
struct RowParams {
    double per_unit;   // kPerUnit / T
    double u, top_p, log_min_p;
    int top_k;
};
__device__ __forceinline__ RowParams params_of(const SampleArgs &a, int row)
{
    RowParams p;
    const float t = a.temperature ? a.temperature[row] : 1.f;
    const bool greedy = !(t > 0.f);
    p.per_unit = kPerUnit / (greedy ? 1.0 : (double)t);
    const float u = a.u[row];
    p.u = !(u > 0.f) ? 0.0 : u < 1.f ? (double)u : (double)0x1.fffffep-1f;
    p.top_k = greedy ? 1 : a.top_k ? a.top_k[row] : 0;
    const float tp = a.top_p ? a.top_p[row] : 1.f;
    p.top_p = !(tp < 1.f) ? 1.0 : tp > 0.f ? (double)tp : 0.0;
    const float mp = a.min_p ? a.min_p[row] : 0.f;
    p.log_min_p = !(mp > 0.f) ? -1e300 : mp < 1.f ? log((double)mp) : 0.0;
    return p;
}

// Every kernel has to put an element into the same bin with the same weight:
// these two functions round each operation by itself (the compiler may fuse a
// product and a sum in one place and not in another) and spell out the fused
// ones they want.
//
// The scaled logit 8 z, relative to `ref` (0 as a rule; the row's maximum for
// rows outside the range, where equality stands for infinities too).
template <bool REL>
__device__ __forceinline__ double scaled(float x, double per_unit, float ref)
{
#pragma clang fp contract(off)
    if constexpr (REL)
        return x == ref ? 0.0 : ((double)x - (double)ref) * per_unit;
    else
        return (double)x * per_unit;
}

// Bin and weight (2^31 (1 + q)) of a scaled logit within the range.
struct Binned {
    int bin;
    int q;
};
__device__ __forceinline__ Binned binned(double d)
{
#pragma clang fp contract(off)
    const double t = d + kMagic;
    Binned b;
    b.bin = (int)(uint32_t)__builtin_bit_cast(uint64_t, t);
    const float r = (float)(d - (t - kMagic));  // -1/2 .. 1/2, in bins
    // 2^31 (e^(r/8) - 1) by its series: the first term left out is below 2^-33 of the weight
    constexpr float c1 = kUnit / 8.f, c2 = c1 / 16.f, c3 = c2 / 24.f, c4 = c3 / 32.f, c5 = c4 / 40.f;
    b.q = (int)(r * __builtin_fmaf(r, __builtin_fmaf(r, __builtin_fmaf(r, __builtin_fmaf(r, c5, c4), c3), c2), c1));
    return b;
}

// Whether the largest logit of a slice has a bin, and whether that of a row
// leaves every bin that counts inside the range (false for -inf and NaN).
__device__ __forceinline__ bool has_bin(float top, double per_unit)
{
    const double d = (double)top * per_unit;
    return d < kRange / 2 - 1 && d > 1 - kRange / 2;
}
__device__ __forceinline__ bool in_range(float top, double per_unit)
{
    return has_bin(top, per_unit) && (double)top * per_unit > kBins - kRange / 2;
}

__device__ __forceinline__ uint32_t order_key(float x)
{
    x += 0.f;  // -0 and 0 are equal logits
    const uint32_t b = __builtin_bit_cast(uint32_t, x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k)
{
    return __builtin_bit_cast(float, k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

template <typename T>
__device__ __forceinline__ float to_float(T v) { return (float)v; }

// Calls f(x, index) for the elements [begin, end) of a row, `threads` threads
// together: 16 bytes a load where a unit of 16 bytes lies inside, one by one
// at the ends (rows need not be aligned).
template <typename T, int UNROLL, typename F>
__device__ __forceinline__ void for_elements(const T *row, int begin, int end, int threads, F f)
{
    constexpr int E = 16 / sizeof(T);
    typedef T vec __attribute__((ext_vector_type(E)));
    const T *first = row + begin;
    const int lead = (int)((16 - (reinterpret_cast<uintptr_t>(first) & 15u)) & 15u) / (int)sizeof(T);
    const int body = begin + (lead < end - begin ? lead : end - begin);
    const int units = (end - body) / E;
    const int tail = body + units * E;
    if ((int)threadIdx.x < body - begin)
        f(to_float(row[begin + threadIdx.x]), begin + (int)threadIdx.x);
    if ((int)threadIdx.x < end - tail)
        f(to_float(row[tail + threadIdx.x]), tail + (int)threadIdx.x);
    const vec *p = reinterpret_cast<const vec *>(row + body);
    int i = threadIdx.x;
    for (; i + (UNROLL - 1) * threads < units; i += UNROLL * threads) {
        vec v[UNROLL];
#pragma unroll
        for (int j = 0; j < UNROLL; ++j)
            v[j] = p[i + j * threads];
#pragma unroll
        for (int j = 0; j < UNROLL; ++j)
#pragma unroll
            for (int e = 0; e < E; ++e)
                f(to_float(v[j][e]), body + (i + j * threads) * E + e);
    }
    for (; i < units; i += threads) {
        const vec v = p[i];
#pragma unroll
        for (int e = 0; e < E; ++e)
            f(to_float(v[e]), body + i * E + e);
    }
}

__device__ __forceinline__ void slice_of(int V, int S, int s, int &begin, int &end)
{
    begin = (int)((int64_t)V * s / S);
    end = (int)((int64_t)V * (s + 1) / S);
}

// ---------------------------------------------------------------------------
// 1. Histogram of one slice of one row.
// ---------------------------------------------------------------------------
template <typename T>
__global__ __launch_bounds__(kScanThreads) void sample_histogram_kernel(const SampleArgs a, int S)
{
    __shared__ uint64_t bins[kRange];
    __shared__ float tops[kScanThreads / kWave];
    const int s = blockIdx.x, row = blockIdx.y;
    for (int i = threadIdx.x; i < kRange; i += kScanThreads)
        bins[i] = 0;
    const float t = a.temperature ? a.temperature[row] : 1.f;
    const double per_unit = kPerUnit / (t > 0.f ? (double)t : 1.0);
    int begin, end;
    slice_of(a.V, S, s, begin, end);
    __syncthreads();
    float top = -__builtin_inff();
    for_elements<T, 4>(static_cast<const T *>(a.logits) + row * a.row_stride, begin, end, kScanThreads,
                       [&](float x, int) {
                           top = fmaxf(top, x);
                           const double d = scaled<false>(x, per_unit, 0.f);
                           if (d >= -(kRange / 2) + 1) {  // not NaN, not -inf, not below the range
                               const Binned b = binned(d);
                               // the mask bounds the address of rows above the range, whose bins are not used
                               atomicAdd(reinterpret_cast<unsigned long long *>(&bins[(b.bin + kRange / 2) & (kRange - 1)]),
                                         ((unsigned long long)1 << kSumBits) + (long long)b.q);
                           }
                       });
#pragma unroll
    for (int d = 1; d < kWave; d *= 2)
        top = fmaxf(top, __shfl_xor(top, d));
    if (threadIdx.x % kWave == 0)
        tops[threadIdx.x / kWave] = top;
    __syncthreads();
    top = tops[threadIdx.x % (kScanThreads / kWave)];
#pragma unroll
    for (int d = 1; d < kScanThreads / kWave; d *= 2)
        top = fmaxf(top, __shfl_xor(top, d));
    char *out = slice_at(a, row, s, S);
    if (threadIdx.x == 0)
        head_of(out)->top = top;
    if (threadIdx.x < kBins && has_bin(top, per_unit)) {
        const int b = binned((double)top * per_unit).bin + kRange / 2 - (int)threadIdx.x;
        hist_of(out)[threadIdx.x] = b >= 0 ? bins[b] : 0;
    }
}

// ---------------------------------------------------------------------------
// Cumulative counts and masses over a row's bins, in LDS.
// ---------------------------------------------------------------------------
struct Cumulative {
    uint32_t count[kBins];   // elements of bins 0 .. t (bin 0 holds the maximum)
    double mass[kBins];      // their mass, e^z relative to bin 0's centre
    float top;               // the row's maximum
    uint32_t wave_count[kScanThreads / kWave];
    double wave_mass[kScanThreads / kWave];
};

// Weight of bin t's centre relative to bin 0's, over the weights' unit.
__device__ __forceinline__ double bin_factor(int t) { return exp(-(double)t / kPerUnit) * 0x1p-31; }

// Inclusive sums over the workgroup's threads, in thread order.
template <typename M>
__device__ __forceinline__ void block_sums(uint32_t &c, M &m, uint32_t *wave_c, M *wave_m, int waves)
{
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
        const uint32_t pc = __shfl_up(c, d);
        const M pm = __shfl_up(m, d);
        if (lane >= d) {
            c += pc;
            m += pm;
        }
    }
    if (lane == kWave - 1) {
        wave_c[wave] = c;
        wave_m[wave] = m;
    }
    __syncthreads();
    uint32_t bc = 0;
    M bm = 0;
    for (int w = 0; w < waves; ++w)
        if (w < wave) {
            bc += wave_c[w];
            bm += wave_m[w];
        }
    c += bc;
    m += bm;
    __syncthreads();
}

__device__ __forceinline__ void store_cumulative(Cumulative &cum, uint32_t c, double m, int waves)
{
    block_sums(c, m, cum.wave_count, cum.wave_mass, waves);
    if (threadIdx.x < kBins) {
        cum.count[threadIdx.x] = c;
        cum.mass[threadIdx.x] = m;
    }
    __syncthreads();
}

// Joins the slices' histograms. The order of the sums is fixed: every
// workgroup of a row gets the same numbers. False: the row is out of range
// (or has no logit above -inf); cum.top is set in any case.
__device__ __forceinline__ bool join_slices(const SampleArgs &a, int row, int S, double per_unit, Cumulative &cum,
                                            int waves)
{
    const int lane = threadIdx.x % kWave;
    float top = lane < S ? head_of(slice_at(a, row, lane, S))->top : -__builtin_inff();  // S <= 64
    const int own = has_bin(top, per_unit) ? binned((double)top * per_unit).bin : -(1 << 30);
#pragma unroll
    for (int d = 1; d < kWave; d *= 2)
        top = fmaxf(top, __shfl_xor(top, d));
    if (threadIdx.x == 0)
        cum.top = top;
    const bool fine = in_range(top, per_unit);  // false for -inf
    uint32_t count = 0;
    int64_t sum = 0;
    if (fine) {
        const int bin = binned((double)top * per_unit).bin - (int)threadIdx.x;
        for (int s0 = 0; s0 < S; s0 += 8) {  // eight loads in flight
            uint64_t v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int s = s0 + j, at = __shfl(own, s & (kWave - 1)) - bin;
                v[j] = s < S && threadIdx.x < kBins && at >= 0 && at < kBins
                           ? hist_of(slice_at(a, row, s, S))[at] : 0;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int64_t q = (int64_t)(v[j] << (64 - kSumBits)) >> (64 - kSumBits);
                sum += q;
                count += (uint32_t)((v[j] - (uint64_t)q) >> kSumBits);
            }
        }
    }
    const double mass = threadIdx.x < kBins
                            ? ((double)count * (double)kUnit + (double)sum) * bin_factor(threadIdx.x) : 0.0;
    store_cumulative(cum, count, mass, waves);
    return fine;
}

// First bin whose cumulative mass reaches (or with PAST passes) a value, the
// last bin if none does; by binary search, the same in every thread.
template <bool PAST>
__device__ __forceinline__ int first_mass(const Cumulative &cum, double value)
{
    int lo = 0, hi = kBins - 1;
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        const bool there = PAST ? cum.mass[mid] > value : cum.mass[mid] >= value;
        if (there)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}
// First bin with a cumulative count of at least k; kBins if none.
__device__ __forceinline__ int first_count(const Cumulative &cum, uint32_t k)
{
    int lo = 0, hi = kBins;
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (cum.count[mid] >= k)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}
__device__ __forceinline__ double mass_before(const Cumulative &cum, int t) { return t > 0 ? cum.mass[t - 1] : 0.0; }

// The bins whose elements decide. A crossing's value is only known to lie
// between bounds until the crossing before it is resolved, so it brings a range
// (widened by more than the roundings of the masses).
struct Wanted {
    int k_bin, p_low, p_high, m_bin, r_low, r_high;
    __device__ __forceinline__ bool has(int t) const
    {
        return t == k_bin || (t >= p_low && t <= p_high) || t == m_bin || (t >= r_low && t <= r_high);
    }
    __device__ __forceinline__ int last() const
    {
        int t = k_bin > p_high ? k_bin : p_high;
        t = t > m_bin ? t : m_bin;
        return t > r_high ? t : r_high;
    }
};
// The bin of min-p's border, relative to the maximum's bin; -1: none.
__device__ __forceinline__ int min_p_bin(const RowParams &p, double top_scaled)
{
    const double d = top_scaled + p.log_min_p * kPerUnit;
    if (!(p.log_min_p > -1e299) || top_scaled - d > kBins)
        return -1;
    const int t = binned(top_scaled).bin - binned(d).bin;
    return t < kBins ? t : -1;
}
__device__ __forceinline__ Wanted wanted_bins(const Cumulative &cum, const RowParams &p, double top_scaled)
{
    Wanted w;
    double low = cum.mass[kBins - 1], high = low;
    w.k_bin = -1;
    if (p.top_k > 0) {
        const int t = first_count(cum, p.top_k);
        if (t < kBins) {
            w.k_bin = t;
            low = mass_before(cum, t);
            high = cum.mass[t];
        }
    }
    w.p_low = 0;
    w.p_high = -1;
    if (p.top_p < 1.0) {
        w.p_low = first_mass<false>(cum, p.top_p * low * (1.0 - 1e-12));
        w.p_high = first_mass<false>(cum, p.top_p * high * (1.0 + 1e-12));
        const double l = mass_before(cum, w.p_low), h = cum.mass[w.p_high];
        low = l < low ? l : low;
        high = h < high ? h : high;
    }
    w.m_bin = min_p_bin(p, top_scaled);
    if (w.m_bin >= 0) {
        const double l = mass_before(cum, w.m_bin), h = cum.mass[w.m_bin];
        low = l < low ? l : low;
        high = h < high ? h : high;
    }
    w.r_low = first_mass<true>(cum, p.u * low * (1.0 - 1e-12));
    w.r_high = first_mass<true>(cum, p.u * high * (1.0 + 1e-12));
    return w;
}

// Elements of wanted bins are offered to take(x, index). Most logits lie below
// the last wanted bin; one comparison with a bound that errs on the safe side
// drops them.
template <typename T, typename F>
__device__ __forceinline__ void for_wanted(const T *row, int begin, int end, int threads, double per_unit,
                                           double top_scaled, const Wanted &w, F take)
{
    const int top_bin = binned(top_scaled).bin;
    const double bound = (top_bin - w.last() - 1) / per_unit;
    const float low = bound > -3e38 && bound < 3e38 ? (float)bound - fabsf((float)bound) * 1e-6f : -__builtin_inff();
    for_elements<T, 4>(row, begin, end, threads, [&](float x, int index) {
        if (x >= low) {
            const double d = scaled<false>(x, per_unit, 0.f);
            if (d > top_scaled - kBins - 1 && w.has(top_bin - binned(d).bin))
                take(x, index);
        }
    });
}

// ---------------------------------------------------------------------------
// 2. Gather of one slice (rows cut into several).
// ---------------------------------------------------------------------------
template <typename T>
__global__ __launch_bounds__(kScanThreads) void sample_gather_kernel(const SampleArgs a, int S)
{
    __shared__ Cumulative cum;
    __shared__ uint32_t listed;
    const int s = blockIdx.x, row = blockIdx.y;
    if (threadIdx.x == 0)
        listed = 0;
    const RowParams p = params_of(a, row);
    if (!join_slices(a, row, S, p.per_unit, cum, kScanThreads / kWave))
        return;
    const double top_scaled = (double)cum.top * p.per_unit;
    const Wanted w = wanted_bins(cum, p, top_scaled);
    int begin, end;
    slice_of(a.V, S, s, begin, end);
    char *out = slice_at(a, row, s, S);
    Entry *list = list_of(out);
    for_wanted(static_cast<const T *>(a.logits) + row * a.row_stride, begin, end, kScanThreads, p.per_unit, top_scaled,
               w, [&](float x, int index) {
                   const uint32_t at = atomicAdd(&listed, 1u);
                   if (at < kSliceList)
                       list[at] = Entry{x, (uint32_t)index};
               });
    __syncthreads();
    if (threadIdx.x == 0)
        head_of(out)->listed = listed;
}

// ---------------------------------------------------------------------------
// 3. Finish: one workgroup a row.
// ---------------------------------------------------------------------------
struct Finish {
    Cumulative cum;
    uint32_t bin_count[kThreads];
    unsigned long long bin_sum[kThreads];
    Entry list[kList];
    uint32_t listed;
    uint32_t low_key, high_key, number;      // of the current range
    uint32_t found_bin, found_count, found_total;
    unsigned long long found_sum;
    unsigned long long total_mass;
    uint32_t token;
    uint32_t wave_c[kThreads / kWave];
    long long wave_m[kThreads / kWave];
};

// The elements that a search looks at: those of bin `t` of the row, from the
// list, or from the row itself where the list could not hold them.
template <typename T, bool REL>
struct Source {
    Finish &f;
    const T *row;
    int V;
    bool rescan;
    double per_unit, top_scaled;
    float ref;
    int top_bin;

    template <typename F>
    __device__ __forceinline__ void of_bin(int t, F g) const
    {
        auto offer = [&](float x, uint32_t index) {
            const double d = scaled<REL>(x, per_unit, ref);
            if (d > top_scaled - kBins - 1) {
                const Binned b = binned(d);
                if (top_bin - b.bin == t)
                    g(order_key(x), index, b.q, d);
            }
        };
        if (rescan)
            for_elements<T, 1>(row, 0, V, kThreads, [&](float x, int i) { offer(x, (uint32_t)i); });
        else
            for (uint32_t i = threadIdx.x; i < f.listed; i += kThreads)
                offer(f.list[i].x, f.list[i].index);
    }
};

// Smallest and largest value and number of the elements that pass.
template <typename Each>
__device__ __forceinline__ void range_of(Finish &f, Each each)
{
    if (threadIdx.x == 0) {
        f.low_key = 0xFFFFFFFFu;
        f.high_key = 0;
        f.number = 0;
    }
    __syncthreads();
    uint32_t lo = 0xFFFFFFFFu, hi = 0, n = 0;
    each([&](uint32_t v) {
        lo = v < lo ? v : lo;
        hi = v > hi ? v : hi;
        ++n;
    });
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
        const uint32_t l = __shfl_xor(lo, d), h = __shfl_xor(hi, d);
        lo = l < lo ? l : lo;
        hi = h > hi ? h : hi;
        n += __shfl_xor(n, d);
    }
    if (threadIdx.x % kWave == 0 && n) {
        atomicMin(&f.low_key, lo);
        atomicMax(&f.high_key, hi);
        atomicAdd(&f.number, n);
    }
    __syncthreads();
}

__device__ __forceinline__ int shift_for(uint32_t range)
{
    int s = 0;
    while ((range >> s) >= (uint32_t)kThreads)
        ++s;
    return s;
}

enum class Cross { count, reach, pass };  // count >= c, mass >= value, mass > value

struct Found {
    uint32_t key;            // the crossing element's
    uint32_t nth;            // which of the elements with this key (1, 2, ...)
    uint32_t equal;          // how many there are
    unsigned long long mass; // of the bin's elements up to and with it
};

// Where the elements of bin t, in order, cross a count or a mass (in units of
// the weights). If they do not, the last element.
template <typename S>
__device__ __forceinline__ Found find_in_bin(Finish &f, const S &src, int t, Cross kind, uint32_t count, double value)
{
    uint32_t low = 0, high = 0xFFFFFFFFu, before = 0;
    unsigned long long mass = 0;
    // A value that rounding took to the bin's edge still crosses at the first
    // element (every weight is far above 1/2).
    const double least = kind == Cross::reach ? 0.5 : 0.0;
    value = value > least ? value : least;
    for (;;) {  // every turn narrows [low, high] by a factor of 512 or ends
        range_of(f, [&](auto add) {
            src.of_bin(t, [&](uint32_t key, uint32_t, int, double) {
                if (key >= low && key <= high)
                    add(key);
            });
        });
        low = f.low_key;
        high = f.high_key;
        const uint32_t number = f.number;
        __syncthreads();
        if (number == 0 || low == high) {
            const double d = scaled<S::kRel>(key_value(low), src.per_unit, src.ref);
            const unsigned long long w = (unsigned long long)(2147483648LL + binned(d).q);
            uint32_t j = number;
            if (kind == Cross::count) {
                j = count - before;
            } else {
                const double left = (value - (double)mass) / (double)w;
                const double n = kind == Cross::reach ? ceil(left) : floor(left) + 1.0;
                j = n < 1.0 ? 1u : n < (double)number ? (uint32_t)n : number;
            }
            j = j < 1 ? 1 : j > number ? number : j;
            return Found{low, j, number, mass + j * w};
        }
        // 512 parts of the range, the highest keys first
        const int shift = shift_for(high - low);
        f.bin_count[threadIdx.x] = 0;
        f.bin_sum[threadIdx.x] = 0;
        if (threadIdx.x == 0)
            f.found_bin = 0xFFFFFFFFu;
        __syncthreads();
        src.of_bin(t, [&](uint32_t key, uint32_t, int q, double) {
            if (key >= low && key <= high) {
                const uint32_t part = (high - key) >> shift;
                atomicAdd(&f.bin_count[part], 1u);
                atomicAdd(&f.bin_sum[part], (unsigned long long)(2147483648LL + q));
            }
        });
        __syncthreads();
        const uint32_t mine = f.bin_count[threadIdx.x];
        const long long my_sum = (long long)f.bin_sum[threadIdx.x];
        uint32_t c = mine;
        long long m = my_sum;
        block_sums(c, m, f.wave_c, f.wave_m, kThreads / kWave);
        const unsigned long long upto = mass + (unsigned long long)m, from = upto - (unsigned long long)my_sum;
        bool here;
        if (kind == Cross::count)
            here = before + c >= count && before + c - mine < count;
        else if (kind == Cross::reach)
            here = (double)upto >= value && (double)from < value;
        else
            here = (double)upto > value && (double)from <= value;
        if (mine && here) {
            f.found_bin = threadIdx.x;
            f.found_count = before + c - mine;
            f.found_sum = from;
        }
        __syncthreads();
        if (f.found_bin == 0xFFFFFFFFu && mine && c == number) {  // not crossed (uniform): the last part
            f.found_count = before + c - mine;
            f.found_sum = from;
            f.found_total = threadIdx.x;
        }
        __syncthreads();
        const uint32_t part = f.found_bin != 0xFFFFFFFFu ? f.found_bin : f.found_total;
        before = f.found_count;
        mass = f.found_sum;
        const uint32_t top = high - (part << shift);
        const uint32_t width = (1u << shift) - 1;
        low = top - low > width ? top - width : low;
        high = top;
        __syncthreads();
    }
}

// The index of the nth (from 1, by rising index) element of bin t with this key.
template <typename S>
__device__ __forceinline__ uint32_t nth_index(Finish &f, const S &src, int t, uint32_t key, uint32_t nth)
{
    uint32_t low = 0, high = 0xFFFFFFFFu, before = 0;
    for (;;) {
        range_of(f, [&](auto add) {
            src.of_bin(t, [&](uint32_t k, uint32_t index, int, double) {
                if (k == key && index >= low && index <= high)
                    add(index);
            });
        });
        low = f.low_key;
        high = f.high_key;
        const uint32_t number = f.number;
        __syncthreads();
        if (number == 0 || low == high)
            return low;
        const int shift = shift_for(high - low);
        f.bin_count[threadIdx.x] = 0;
        if (threadIdx.x == 0)
            f.found_bin = 0;
        __syncthreads();
        src.of_bin(t, [&](uint32_t k, uint32_t index, int, double) {
            if (k == key && index >= low && index <= high)
                atomicAdd(&f.bin_count[(index - low) >> shift], 1u);
        });
        __syncthreads();
        const uint32_t mine = f.bin_count[threadIdx.x];
        uint32_t c = mine;
        long long none = 0;
        block_sums(c, none, f.wave_c, f.wave_m, kThreads / kWave);
        if (mine && before + c >= nth && before + c - mine < nth) {
            f.found_bin = threadIdx.x;
            f.found_count = before + c - mine;
        }
        __syncthreads();
        before = f.found_count;
        const uint32_t from = low + (f.found_bin << shift);
        const uint32_t width = (1u << shift) - 1;
        high = high - from > width ? from + width : high;
        low = from;
        __syncthreads();
    }
}

template <typename T, bool REL>
struct RowSource : Source<T, REL> {
    static constexpr bool kRel = REL;
};

// The searches, in the order of the filters.
template <typename T, bool REL>
__device__ __forceinline__ void finish_row(const SampleArgs &a, int row, const RowParams &p, Finish &f, const RowSource<T, REL> &src)
{
    const Cumulative &cum = f.cum;
    double kept = cum.mass[kBins - 1];
    const double all = kept;
    double limit = all;  // mass of the top-k prefix
    if (p.top_k > 0) {
        const int t = first_count(cum, p.top_k);
        if (t < kBins) {
            const Found e = find_in_bin(f, src, t, Cross::count, p.top_k - (t > 0 ? cum.count[t - 1] : 0), 0.0);
            limit = kept = mass_before(cum, t) + (double)e.mass * bin_factor(t);
        }
    }
    if (p.top_p < 1.0) {
        const double target = p.top_p * limit;
        const int t = first_mass<false>(cum, target);
        const Found e = find_in_bin(f, src, t, Cross::reach, 0, (target - mass_before(cum, t)) / bin_factor(t));
        const double m = mass_before(cum, t) + (double)e.mass * bin_factor(t);
        kept = m < kept ? m : kept;
    }
    const int mt = min_p_bin(p, src.top_scaled);
    if (mt >= 0) {
        if (threadIdx.x == 0)
            f.total_mass = 0;
        __syncthreads();
        unsigned long long sum = 0;
        src.of_bin(mt, [&](uint32_t, uint32_t, int q, double d) {
            if ((d - src.top_scaled) / kPerUnit >= p.log_min_p)
                sum += (unsigned long long)(2147483648LL + q);
        });
#pragma unroll
        for (int d = 1; d < kWave; d *= 2)
            sum += __shfl_xor(sum, d);
        if (threadIdx.x % kWave == 0 && sum)
            atomicAdd(&f.total_mass, sum);
        __syncthreads();
        const double m = mass_before(cum, mt) + (double)f.total_mass * bin_factor(mt);
        kept = m < kept ? m : kept;
        __syncthreads();
    }
    const double r = p.u * kept;
    const int t = first_mass<true>(cum, r);
    const Found e = find_in_bin(f, src, t, Cross::pass, 0, (r - mass_before(cum, t)) / bin_factor(t));
    const uint32_t index = nth_index(f, src, t, e.key, e.nth);
    if (threadIdx.x == 0) {
        a.tokens[row] = (int32_t)index;
        if (a.logprobs) {
            // the weight as the sums hold it, so that a token kept alone has share 1
            const int q = binned(scaled<REL>(key_value(e.key), src.per_unit, src.ref)).q;
            const double lp = log((double)(2147483648LL + q) * bin_factor(t) / kept);
            a.logprobs[row] = lp < 0.0 ? (float)lp : 0.f;
        }
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void sample_finish_kernel(const SampleArgs a, int S)
{
    __shared__ Finish f;
    const int row = blockIdx.x;
    const RowParams p = params_of(a, row);
    if (threadIdx.x == 0)
        f.listed = 0;
    const bool fine = join_slices(a, row, S, p.per_unit, f.cum, kThreads / kWave);
    const float top = f.cum.top;
    const T *x = static_cast<const T *>(a.logits) + row * a.row_stride;
    if (top == -__builtin_inff()) {  // no logit above -inf
        if (threadIdx.x == 0) {
            a.tokens[row] = -1;
            if (a.logprobs)
                a.logprobs[row] = -__builtin_inff();
        }
        return;
    }
    if (fine) {
        RowSource<T, false> src{{f, x, a.V, false, p.per_unit, (double)top * p.per_unit, 0.f, 0}};
        src.top_bin = binned(src.top_scaled).bin;
        if (S == 1) {
            const Wanted w = wanted_bins(f.cum, p, src.top_scaled);
            for_wanted(x, 0, a.V, kThreads, p.per_unit, src.top_scaled, w, [&](float v, int index) {
                const uint32_t at = atomicAdd(&f.listed, 1u);
                if (at < kList)
                    f.list[at] = Entry{v, (uint32_t)index};
            });
            __syncthreads();
            src.rescan = f.listed > kList;
        } else {
            const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
            const uint32_t own = lane < S ? head_of(slice_at(a, row, lane, S))->listed : 0;
            uint32_t upto = own;
            bool over = own > kSliceList;
#pragma unroll
            for (int d = 1; d < kWave; d *= 2) {
                const uint32_t v = __shfl_up(upto, d);
                upto += lane >= d ? v : 0;
            }
            const uint32_t total = __shfl(upto, kWave - 1);
            src.rescan = __any(over) || total > kList;
            if (!src.rescan)
                for (int s = wave; s < S; s += kThreads / kWave) {
                    const uint32_t n = __shfl(own, s), to = __shfl(upto, s) - n;
                    const Entry *list = list_of(slice_at(a, row, s, S));
                    for (uint32_t i = lane; i < n; i += kWave)
                        f.list[to + i] = list[i];
                }
            if (threadIdx.x == 0)
                f.listed = total;
            __syncthreads();
        }
        finish_row<T, false>(a, row, p, f, src);
    } else {
        // Counted again, relative to the maximum.
        RowSource<T, true> src{{f, x, a.V, true, p.per_unit, 0.0, top, 0}};
        f.bin_count[threadIdx.x] = 0;
        f.bin_sum[threadIdx.x] = 0;
        __syncthreads();
        for_elements<T, 1>(x, 0, a.V, kThreads, [&](float v, int) {
            const double d = scaled<true>(v, p.per_unit, top);
            if (d > -(kBins - 1)) {
                const Binned b = binned(d);
                atomicAdd(&f.bin_count[-b.bin & (kThreads - 1)], 1u);
                atomicAdd(&f.bin_sum[-b.bin & (kThreads - 1)], (unsigned long long)(long long)b.q);
            }
        });
        __syncthreads();
        const int t = threadIdx.x;
        const uint32_t c = t < kBins ? f.bin_count[t] : 0;
        const double m = t < kBins ? ((double)c * (double)kUnit + (double)(long long)f.bin_sum[t]) * bin_factor(t) : 0.0;
        __syncthreads();
        store_cumulative(f.cum, c, m, kThreads / kWave);
        finish_row<T, true>(a, row, p, f, src);
    }
}

// Slices of a row: enough workgroups to fill the GPU, none with fewer
// elements than its threads load at a time (4 units of 16 bytes of fp32).
int slices_of(int M, int V)
{
    const int least = (V + kMaxSlice - 1) / kMaxSlice;
    int s = device_cu_count() / M;
    const int most = V / (4 * kScanThreads);
    s = s < most ? s : most;
    s = s < kMaxSlices ? s : kMaxSlices;
    return s > least ? s : least > 1 ? least : 1;
}

template <typename T>
hipError_t launch(const SampleArgs &a, hipStream_t stream)
{
    const int S = slices_of(a.M, a.V);
    sample_histogram_kernel<T><<<dim3(S, a.M), kScanThreads, 0, stream>>>(a, S);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && S > 1) {
        sample_gather_kernel<T><<<dim3(S, a.M), kScanThreads, 0, stream>>>(a, S);
        e = hipGetLastError();
    }
    if (e != hipSuccess)
        return e;
    sample_finish_kernel<T><<<dim3(a.M), kThreads, 0, stream>>>(a, S);
    return hipGetLastError();
}

}  // namespace

bool sample_size_supported(int V) { return V >= 1 && V <= kMaxSlice * kMaxSlices; }

size_t sample_workspace_bytes(int M, int V) { return (size_t)M * slices_of(M, V) * slice_bytes(); }

hipError_t launch_sample(const SampleArgs &a, int type, hipStream_t stream)
{
    switch (type) {
    case 0: return launch<_Float16>(a, stream);
    case 1: return launch<__bf16>(a, stream);
    case 2: return launch<float>(a, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace qmm
