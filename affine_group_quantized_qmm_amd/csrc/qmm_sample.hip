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
//                 bin's centre, e^(z - b/8) = 1 + q with |q| < 0.065, so that an
//                 integer and a small polynomial in fp32 give a weight to 2^-30
//                 and neither the row's maximum nor a range reduction is needed first.
//                 Weights are integers (2^31 (1 + q)): sums do not depend on
//                 their order. Number and mass share one 64-bit LDS atomic.
//                 Only the 384 bins below the maximum's count: e^-48 of the
//                 largest weight is below 2^-69.
//   2. gather     Cumulative counts and masses over those bins (64-bit floats)
//                 tell which bins each crossing can fall into; the elements
//                 of those bins (tens to hundreds of a vocabulary) are listed.
//   3. finish     Each crossing is resolved inside its bin: a histogram of 512
//                 parts of the bin's width leaves a few elements (or equal
//                 ones), which are ranked by comparing all pairs.
//
// Tokens have to be equal to what 64-bit arithmetic gives, whatever the order of
// the sums: the weights' relative errors (below 2^-30) move a border between two
// tokens by at most a quarter of the difference of two of them, 2^-31 of the kept
// mass, and a token only if u falls within that.
//
// Rows of bf16 logits take another way, by their values (see there).
//
// Slower, the same answer: rows whose maximum lies outside the histogram's range
// (|z| of 500, or an infinity) are counted again relative to their maximum by the
// finishing workgroup alone; where the wanted bins hold more elements than the
// lists take, the finishing workgroup lists the row again for each search; and
// where one bin does, or more than a thousand elements share a part of it, it
// narrows the search down over the row, some passes each.
// That is what flat rows cost (160000 fp32 logits of standard deviation 1, 0.5
// and 0.25 after temperature, without filters: one row 26, 126 and 255 us, 256 rows
// 120, 557 and 637; with top-p 0.9 one row 54, 393 and 514, 256 rows 170, 963 and 1003).
//
// Else the histogram and the listing read the logits once each; a row is cut into
// slices so that few rows still fill the GPU.
//
// What bounds it. Few rows: two or three launches one after the other, each with
// its code to fetch: one row of 131072 fp32 logits takes 18 to 20 us (histogram 5,
// gather 8, finish 5), 16 rows of 151001 with top-k and top-p 25, 32 rows of 32003
// fp16 logits 24. 256 rows of 131072 fp32 logits take 57 us with top-k 50 and top-p
// 0.9, without top-k 66: two passes over 134 MB (27 each at the rate of a copy), and
// the searches, up to 9 each. With 16-bit logits the histogram still takes 25: a
// CU issues 20 instructions and one LDS atomic for every element.
#include "qmm_device.hpp"
#include "qmm_kernels.hpp"
#include "qmm_step.hpp"

namespace qmm {
namespace {

constexpr int kScanThreads = 1024;   // histogram; finish of rows of one slice, which it scans too
constexpr int kThreads = 512;        // gather; finish of rows cut into slices
constexpr int kRange = 8192;         // bins of the histogram: z of -512 .. 512
constexpr int kBins = 384;           // bins that count, from the maximum's down
constexpr int kSlots = 512;          // of a slice's histogram: bin b lies in slot b mod 512
constexpr double kPerUnit = 8.0;     // bins per unit of z
constexpr int kSumBits = 46;         // low field of a packed bin: the sum of its weights over kLeast
constexpr float kUnit = 2147483648.0f;   // 2^31: the weight of a bin's centre
constexpr uint32_t kLeast = (1u << 31) - (1u << 27);  // what every weight passes (2^31 e^(-1/16) is above it)
constexpr int kMaxSlice = 1 << 17;   // elements of a slice: the packed number has 18 bits, the sum 46
// Rows up to this long are gathered by the workgroup that finishes them: 32000
// logits 17.6 us a call against 20.4 with a launch of its own for the gather,
// 65000 20.9 and 20.5, 131072 24.1 and 20.5 (one row, top-k and top-p).
constexpr int kGatherMin = 1 << 16;
constexpr int kMaxSlices = 64;
constexpr int kSliceList = 1024;     // listed elements of a slice
// Listed elements of a row, as many as the LDS takes: batches of 256 rows of 131072
// fp16 logits with top-p 0.95 take 61 us on average, with lists of 8192 68 (more of
// them have a row that is listed once for each search); in fp32 73 and 82.
constexpr int kList = 11264;
constexpr int kParts = 512;          // parts of a bin
constexpr int kRanked = 1024;        // elements that are ranked by pairs
// A bin of up to this many is ranked as it is (32 rows of 32003 logits with top-k
// 1000 and min-p 24.0 us a call, with 64 24.6; with 192 16 rows of 131072 take 30
// instead of 28).
constexpr int kWhole = 128;
constexpr double kMagic = 25165824.5;  // 1.5 * 2^24: adding it leaves a number in steps of 2^-28 in the low bits; and half a bin

// What a slice leaves behind, and a row (cut into slices).
struct SliceHead {
    float top;          // largest logit (-inf: none)
    uint32_t listed;    // elements of the gathered bins, before the cap
    uint32_t pad[2];
};
struct Entry {
    float x;
    uint32_t index;
};
struct RowSums {
    double mass[kBins];      // mass of bins 0 .. t (bin 0 holds the maximum), e^z relative to bin 0's centre
    uint32_t count[kBins];   // their elements
    float top;               // the row's maximum
    int fine;                // whether it is in the histogram's range
    uint32_t pad[2];
};
__host__ __device__ constexpr size_t slice_bytes() { return sizeof(SliceHead) + kSlots * 8 + kSliceList * sizeof(Entry); }
__host__ __device__ constexpr size_t row_bytes(int S) { return sizeof(RowSums) + S * slice_bytes(); }
static_assert(kParts == 1 << 9, "binned's parts");
static_assert(sizeof(RowSums) % 16 == 0 && slice_bytes() % 16 == 0, "aligned parts");
__device__ __forceinline__ RowSums *sums_of(const SampleArgs &a, int row, int S)
{
    return reinterpret_cast<RowSums *>(static_cast<char *>(a.workspace) + row * row_bytes(S));
}
__device__ __forceinline__ char *slice_at(const SampleArgs &a, int row, int s, int S)
{
    return static_cast<char *>(a.workspace) + row * row_bytes(S) + sizeof(RowSums) + s * slice_bytes();
}
__device__ __forceinline__ SliceHead *head_of(char *p) { return reinterpret_cast<SliceHead *>(p); }
__device__ __forceinline__ uint64_t *hist_of(char *p) { return reinterpret_cast<uint64_t *>(p + sizeof(SliceHead)); }
__device__ __forceinline__ Entry *list_of(char *p)
{
    return reinterpret_cast<Entry *>(p + sizeof(SliceHead) + kSlots * 8);
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

// Bin and weight (2^31 (1 + q) = kLeast + over) of a scaled logit within the range, and the part
// of the bin (0: its upper end) that it lies in.
struct Binned {
    int bin;
    uint32_t over;
    int part;
    __device__ __forceinline__ uint32_t weight() const { return kLeast + over; }
};
// d + 1/2 in steps of 2^-28 bins is an integer (kMagic's last bit is one): its upper bits are the
// bin, the lower 28 (`above` the bin's lower end), over 2^31 and less 1/16, are x = ln(1 + q), and
// so as they stand the first term of 2^31 (e^x - 1). The others, below 2^22, are summed in fp32;
// the first one left out is below 2^-33 of the weight. Together 2^-30 at most, where the whole
// series in fp32 is off by 2^-26.7.
__device__ __forceinline__ Binned binned(double d)
{
#pragma clang fp contract(off)
    const uint64_t u = __builtin_bit_cast(uint64_t, d + kMagic);
    constexpr uint32_t none = (uint32_t)(__builtin_bit_cast(uint64_t, kMagic) >> 28);  // of bin 0
    constexpr uint32_t low = (1u << 28) - 1;
    const uint32_t above = (uint32_t)u & low;
    Binned b;
    b.bin = (int)((uint32_t)(u >> 28) - none);
    b.part = (int)((low - above) >> 19);  // 2^28 / kParts each
    constexpr float c2 = kUnit / 2.f, c3 = kUnit / 6.f, c4 = kUnit / 24.f, c5 = kUnit / 120.f;
    const float x = __builtin_fmaf((float)above, 0x1p-31f, -0x1p-4f);
    const float rest = __builtin_fmaf(x, __builtin_fmaf(x, __builtin_fmaf(x, c5, c4), c3), c2);
    b.over = above + (uint32_t)__builtin_fmaf(x * x, rest, 0.5f);
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

// Elements [begin, end) of a row (which need not be aligned): single ones up
// to `body`, whole units of 16 bytes, single ones from `tail`.
struct Span {
    int body, units, tail;
};
template <typename T>
__device__ __forceinline__ Span span_of_row(const T *row, int begin, int end, int size)
{
    const int E = 16 / size;
    const int lead = (int)((16 - (reinterpret_cast<uintptr_t>(row + begin) & 15u)) & 15u) / size;
    Span s;
    s.body = begin + (lead < end - begin ? lead : end - begin);
    s.units = (end - s.body) / E;
    s.tail = s.body + s.units * E;
    return s;
}

// Calls f(x, index) for the elements [begin, end) of a row, `threads` threads
// together: 16 bytes a load where a unit of 16 bytes lies inside, one by one
// at the ends (rows need not be aligned).
template <typename T, int UNROLL, typename F>
__device__ __forceinline__ void for_elements(const T *row, int begin, int end, int threads, F f)
{
    constexpr int E = 16 / sizeof(T);
    typedef T vec __attribute__((ext_vector_type(E)));
    const Span s = span_of_row(row, begin, end, (int)sizeof(T));
    const int body = s.body, units = s.units, tail = s.tail;
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
                                         ((unsigned long long)1 << kSumBits) + b.over);
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
        const int b = binned((double)top * per_unit).bin - (int)threadIdx.x, at = b + kRange / 2;
        hist_of(out)[b & (kSlots - 1)] = at >= 0 ? bins[at] : 0;
    }
}

// ---------------------------------------------------------------------------
// Cumulative counts and masses over a row's bins.
// ---------------------------------------------------------------------------

// Weight of bin t's centre relative to bin 0's, over the weights' unit:
// e^(-t/8) 2^-31 as powers of e^(-1/8) (a load is shorter than the code of an
// exponential that every launch would have to fetch first).
struct Factors {
    double of[kBins];
    constexpr Factors() : of()
    {
        constexpr double sixteenth[4] = {1.0, 0.88249690258459540286, 0.77880078307140486825, 0.68728927879097219855};
        double half = 0x1p-31;  // e^(-t/2) for t in steps of 4 bins
        for (int t = 0; t < kBins; t += 4) {
            for (int j = 0; j < 4; ++j)
                of[t + j] = half * sixteenth[j];
            half *= 0.60653065971263342360;
        }
    }
};
__device__ const Factors factors{};

// Inclusive sums over the workgroup's threads, in thread order.
template <typename M>
struct WaveSums {
    M mass[kScanThreads / kWave];
    uint32_t count[kScanThreads / kWave];
};
// A 32- or 64-bit value moved between lanes by a DPP control, 0 where no lane gives one.
template <int CTRL, typename V>
__device__ __forceinline__ V moved(V v)
{
    if constexpr (sizeof(V) == 4) {
        return __builtin_bit_cast(V, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
    } else {
        const uint64_t u = __builtin_bit_cast(uint64_t, v);
        const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xF, 0xF, true);
        const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(u >> 32), CTRL, 0xF, 0xF, true);
        return __builtin_bit_cast(V, (uint64_t)hi << 32 | lo);
    }
}
template <typename V>
__device__ __forceinline__ V of_lane(V v, int lane)
{
    if constexpr (sizeof(V) == 4) {
        return __builtin_bit_cast(V, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
    } else {
        const uint64_t u = __builtin_bit_cast(uint64_t, v);
        const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, lane);
        const uint32_t hi = __builtin_amdgcn_readlane((int)(u >> 32), lane);
        return __builtin_bit_cast(V, (uint64_t)hi << 32 | lo);
    }
}
// Inclusive sums over a wave's lanes: shifts within rows of 16, then the rows before.
template <typename V>
__device__ __forceinline__ V wave_sums(V v)
{
    v += moved<0x111>(v);  // row_shr:1
    v += moved<0x112>(v);
    v += moved<0x114>(v);
    v += moved<0x118>(v);
    const V r0 = of_lane(v, 15), r1 = of_lane(v, 31), r2 = of_lane(v, 47);
    const int row = threadIdx.x % kWave / 16;
    const V before = row == 0 ? (V)0 : row == 1 ? r0 : row == 2 ? r0 + r1 : r0 + r1 + r2;
    return v + before;
}
// Their total alone, in the last lane: half as many instructions.
template <int CTRL, int ROWS, typename V>
__device__ __forceinline__ V moved_to_rows(V v)
{
    if constexpr (sizeof(V) == 4) {
        return __builtin_bit_cast(V, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, ROWS, 0xF, false));
    } else {
        const uint64_t u = __builtin_bit_cast(uint64_t, v);
        const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xF, false);
        const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(u >> 32), CTRL, ROWS, 0xF, false);
        return __builtin_bit_cast(V, (uint64_t)hi << 32 | lo);
    }
}
template <typename V>
__device__ __forceinline__ V wave_total(V v)
{
    v += moved<0x111>(v);
    v += moved<0x112>(v);
    v += moved<0x114>(v);
    v += moved<0x118>(v);
    v += moved_to_rows<0x142, 0xA>(v);  // row_bcast:15: a row's sum to the next, for the odd rows
    v += moved_to_rows<0x143, 0xC>(v);  // row_bcast:31: the first half's sum to the second
    return v;
}
template <int THREADS, typename M>
__device__ __forceinline__ void block_sums(uint32_t &c, M &m, WaveSums<M> &w)
{
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    c = wave_sums(c);
    m = wave_sums(m);
    if (lane == kWave - 1) {
        w.count[wave] = c;
        w.mass[wave] = m;
    }
    __syncthreads();
    // the waves before: their sums, in lanes
    constexpr int WAVES = THREADS / kWave;
    const uint32_t wc = wave_sums(lane < WAVES ? w.count[lane % WAVES] : 0u);
    const M wm = wave_sums(lane < WAVES ? w.mass[lane % WAVES] : (M)0);
    const int before = __builtin_amdgcn_readfirstlane(wave) - 1;
    const uint32_t bc = before >= 0 ? of_lane(wc, before) : 0u;
    const M bm = before >= 0 ? of_lane(wm, before) : (M)0;
    c += bc;
    m += bm;
    __syncthreads();
}

template <int THREADS>
__device__ __forceinline__ void store_sums(RowSums &sums, uint32_t c, double m, WaveSums<double> &w)
{
    block_sums<THREADS>(c, m, w);
    if (threadIdx.x < kBins) {
        sums.count[threadIdx.x] = c;
        sums.mass[threadIdx.x] = m;
    }
    __syncthreads();
}

// Joins the slices' histograms, of THREADS / 512 groups of threads each a share
// of them. Everything is loaded at once: which bin a slot holds follows from
// its slice's maximum, and whether the row wants it is seen afterwards. The
// sums are of integers (and the scan's order is fixed): every workgroup of a
// row gets the same numbers.
struct Joined {
    uint32_t count[kSlots];
    uint64_t sum[kSlots];
};
__device__ __forceinline__ void unpack(uint64_t v, uint32_t &count, uint64_t &sum)
{
    sum += v & (((uint64_t)1 << kSumBits) - 1);
    count += (uint32_t)(v >> kSumBits);
}
// Mass of elements whose weights over kLeast have this sum.
__device__ __forceinline__ uint64_t mass_of(uint32_t count, uint64_t sum) { return (uint64_t)count * kLeast + sum; }
template <int THREADS, int AT_ONCE>
__device__ __forceinline__ void join_slices(const SampleArgs &a, int row, int S, double per_unit, RowSums &sums,
                                            WaveSums<double> &w, Joined &joined)
{
    constexpr int GROUPS = THREADS / kSlots;
    const int lane = threadIdx.x % kWave, slot = threadIdx.x % kSlots;
    const int group = __builtin_amdgcn_readfirstlane(threadIdx.x / kSlots);
    const double factor = threadIdx.x < kBins ? factors.of[threadIdx.x] : 0.0;
    float top = lane < S ? head_of(slice_at(a, row, lane, S))->top : -__builtin_inff();  // S <= 64
    uint64_t v[AT_ONCE];
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j) {
        const int s = group + j * GROUPS;
        v[j] = s < S ? hist_of(slice_at(a, row, s, S))[slot] : 0;
    }
    const int own = has_bin(top, per_unit) ? binned((double)top * per_unit).bin : -(1 << 30);
#pragma unroll
    for (int d = 1; d < kWave; d *= 2)
        top = fmaxf(top, __shfl_xor(top, d));
    const bool fine = in_range(top, per_unit);  // false for -inf
    if (threadIdx.x == 0) {
        sums.top = top;
        sums.fine = fine;
    }
    const int top_bin = binned(fine ? (double)top * per_unit : 0.0).bin;
    const int t = (top_bin - slot) & (kSlots - 1);  // the slot's bin, from the maximum's down
    uint32_t count = 0;
    uint64_t sum = 0, packed = 0;
    // Up to this many elements fit the packed fields of one bin (each adds less than 2^28 + 2^23).
    const bool together = a.V <= 250000;
    for (int s0 = 0; fine && s0 < S; s0 += AT_ONCE * GROUPS) {
        if (s0 > 0) {
#pragma unroll
            for (int j = 0; j < AT_ONCE; ++j) {
                const int s = s0 + group + j * GROUPS;
                v[j] = s < S ? hist_of(slice_at(a, row, s, S))[slot] : 0;
            }
        }
#pragma unroll
        for (int j = 0; j < AT_ONCE; ++j) {
            const int s = s0 + group + j * GROUPS;
            // the slice's maximum's bin down to this one
            const int below = __builtin_amdgcn_readlane(own, s & (kWave - 1)) - (top_bin - t);
            v[j] = s < S && (uint32_t)below < (uint32_t)kBins ? v[j] : 0;
            packed += v[j];
        }
        if (!together) {
#pragma unroll
            for (int j = 0; j < AT_ONCE; ++j)
                unpack(v[j], count, sum);
        }
    }
    if (together)
        unpack(packed, count, sum);
    if (group == 0) {
        joined.count[t] = count;
        joined.sum[t] = sum;
    }
    __syncthreads();
    if constexpr (GROUPS == 2) {
        if (group == 1) {
            joined.count[t] += count;
            joined.sum[t] += sum;
        }
        __syncthreads();
    }
    count = threadIdx.x < kBins ? joined.count[threadIdx.x] : 0;
    const double mass = threadIdx.x < kBins ? (double)mass_of(count, joined.sum[threadIdx.x]) * factor : 0.0;
    store_sums<THREADS>(sums, count, mass, w);
}

// The sums in a wave's registers, where a search is a comparison and a count
// of lanes for each 64 bins: the sums rise, so that the first bin to reach a
// value is the number of bins that do not.
struct Search {
    double mass[kBins / kWave];
    uint32_t count[kBins / kWave];
    __device__ __forceinline__ explicit Search(const RowSums &s)
    {
#pragma unroll
        for (int j = 0; j < kBins / kWave; ++j) {
            mass[j] = s.mass[j * kWave + threadIdx.x % kWave];
            count[j] = s.count[j * kWave + threadIdx.x % kWave];
        }
    }
    // First bin whose cumulative mass reaches (or with PAST passes) a value, the
    // last bin if none does.
    template <bool PAST>
    __device__ __forceinline__ int first_mass(double value) const
    {
        int n = 0;
#pragma unroll
        for (int j = 0; j < kBins / kWave; ++j)
            n += __popcll(__ballot(PAST ? mass[j] <= value : mass[j] < value));
        return n < kBins ? n : kBins - 1;
    }
    // First bin with a cumulative count of at least k; kBins if none.
    __device__ __forceinline__ int first_count(uint32_t k) const
    {
        int n = 0;
#pragma unroll
        for (int j = 0; j < kBins / kWave; ++j)
            n += __popcll(__ballot(count[j] < k));
        return n;
    }
};
__device__ __forceinline__ double mass_before(const RowSums &s, int t) { return t > 0 ? s.mass[t - 1] : 0.0; }
__device__ __forceinline__ uint32_t count_before(const RowSums &s, int t) { return t > 0 ? s.count[t - 1] : 0u; }
// The sums of mass are rounded in another order for each bin, so that one may
// rise by a rounding at a bin without elements. A crossing found there lies at the
// end of the last bin with elements, whose last element it is: the value becomes
// one that no sum in the bin reaches. (That bin is listed: wanted ranges are
// wider than roundings.)
__device__ __forceinline__ void leave_empty_bin(const RowSums &s, const Search &find, int &t, double &value)
{
    const uint32_t count = s.count[t];
    if (__builtin_expect(count == count_before(s, t), 0)) {
        t = find.first_count(count);
        value = 1e300;
    }
}

// The bins whose elements decide. A crossing's value is only known to lie
// between bounds until the crossing before it is resolved, so it brings a range
// (widened by more than the roundings of the masses).
struct Wanted {
    int k_bin, p_low, p_high, m_bin, r_low, r_high;
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
__device__ __forceinline__ Wanted wanted_bins(const RowSums &sums, const RowParams &p, double top_scaled)
{
    const Search find(sums);
    Wanted w;
    double low = sums.mass[kBins - 1], high = low;
    w.k_bin = -1;
    if (p.top_k > 0) {
        const int t = find.first_count(p.top_k);
        if (t < kBins) {
            w.k_bin = t;
            low = mass_before(sums, t);
            high = sums.mass[t];
        }
    }
    w.p_low = 0;
    w.p_high = -1;
    if (p.top_p < 1.0) {
        w.p_low = find.first_mass<false>(p.top_p * low * (1.0 - 1e-12));
        w.p_high = find.first_mass<false>(p.top_p * high * (1.0 + 1e-12));
        const double l = mass_before(sums, w.p_low), h = sums.mass[w.p_high];
        low = l < low ? l : low;
        high = h < high ? h : high;
    }
    w.m_bin = min_p_bin(p, top_scaled);
    if (w.m_bin >= 0) {
        const double l = mass_before(sums, w.m_bin), h = sums.mass[w.m_bin];
        low = l < low ? l : low;
        high = h < high ? h : high;
    }
    w.r_low = find.first_mass<true>(p.u * low * (1.0 - 1e-12));
    w.r_high = find.first_mass<true>(p.u * high * (1.0 + 1e-12));
    return w;
}

// Intervals of logits that hold the wanted bins. Their ends are moved outwards
// by more than their roundings (to fp32 at most 4096 bins from zero: 2^-12 of a
// bin); what they let in besides is told apart by its bin later. Overlapping
// ones are one.
struct Intervals {
    float low[4], high[4];
    int number;
};
__device__ __forceinline__ Intervals intervals_of(const Wanted &w, double per_unit, int top_bin)
{
    constexpr double kReach = 0.5 + 0x1p-10;
    const double unit = 1.0 / per_unit;
    Intervals v;
    v.number = 0;
    const int first[4] = {w.k_bin, w.p_low, w.m_bin, w.r_low}, last[4] = {w.k_bin, w.p_high, w.m_bin, w.r_high};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        v.low[k] = __builtin_inff();
        v.high[k] = -__builtin_inff();
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (last[k] < first[k] || last[k] < 0)
            continue;
        // bin t: z of (top_bin - t - 1/2) / 8 .. (top_bin - t + 1/2) / 8
        float l = (float)((top_bin - last[k] - kReach) * unit), h = (float)((top_bin - first[k] + kReach) * unit);
#pragma unroll
        for (int j = 0; j < k; ++j)
            if (v.low[j] <= h && l <= v.high[j]) {  // takes j over
                l = v.low[j] < l ? v.low[j] : l;
                h = v.high[j] > h ? v.high[j] : h;
                v.low[j] = __builtin_inff();
                v.high[j] = -__builtin_inff();
            }
        v.low[k] = l;
        v.high[k] = h;
    }
    // The ones that are left, in front; behind them infinity alone, which no
    // row has whose bins are used.
    float low[4], high[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
        low[k] = high[k] = __builtin_inff();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (!(v.low[k] <= v.high[k]))
            continue;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j == v.number) {
                low[j] = v.low[k];
                high[j] = v.high[k];
            }
        ++v.number;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        v.low[k] = low[k];
        v.high[k] = high[k];
    }
    return v;
}

// Writes the places of the elements [begin, end) of a row that lie in one of N
// intervals to `places` (up to cap of them; *listed counts all). 32 elements
// (16 in fp32) give a lane one word of hits and one place to write to.
template <int N, typename T>
__device__ __forceinline__ void list_places(const T *row, int begin, int end, int threads, const Intervals &v,
                                            uint32_t *listed, uint32_t *places, int cap)
{
    auto hit = [&](float x) {
        // the middle of x and an interval's ends is x inside it (and not for NaN)
        bool h = __builtin_amdgcn_fmed3f(x, v.low[0], v.high[0]) == x;
#pragma unroll
        for (int k = 1; k < N; ++k)
            h |= __builtin_amdgcn_fmed3f(x, v.low[k], v.high[k]) == x;
        return h;
    };
    auto put = [&](uint32_t at, int place) {
        if (at < (uint32_t)cap)
            places[at] = (uint32_t)place;
    };
    constexpr int E = 16 / sizeof(T), UNROLL = 4;
    typedef T vec __attribute__((ext_vector_type(E)));
    const Span s = span_of_row(row, begin, end, (int)sizeof(T));
    const int single = (int)threadIdx.x < s.body - begin ? begin + (int)threadIdx.x : -1;
    if (single >= 0 && hit((float)row[single]))
        put(atomicAdd(listed, 1u), single);
    if ((int)threadIdx.x < end - s.tail && hit((float)row[s.tail + threadIdx.x]))
        put(atomicAdd(listed, 1u), s.tail + (int)threadIdx.x);
    const vec *p = reinterpret_cast<const vec *>(row + s.body);
    const int first = threadIdx.x & ~(kWave - 1);  // whole waves: the places are taken together
    for (int i0 = first; i0 < s.units; i0 += UNROLL * threads) {
        const int i = i0 + (int)threadIdx.x % kWave;
        vec x[UNROLL];
#pragma unroll
        for (int j = 0; j < UNROLL; ++j)
            x[j] = p[i + j * threads < s.units ? i + j * threads : i0];
        uint32_t hits = 0;  // bit E j + e
#pragma unroll
        for (int j = UNROLL - 1; j >= 0; --j) {
            uint32_t h = 0;
#pragma unroll
            for (int e = E - 1; e >= 0; --e)
                h = h + h + (hit((float)x[j][e]) ? 1u : 0u);
            hits = hits << E | (i + j * threads < s.units ? h : 0u);
        }
        if (__any(hits != 0)) {
            // One lane takes places for the whole wave (the same address from
            // 64 lanes would be served one by one).
            const uint32_t mine = __popc(hits), upto = wave_sums(mine), all = of_lane(upto, kWave - 1);
            uint32_t from = 0;
            if (threadIdx.x % kWave == 0)
                from = atomicAdd(listed, all);
            uint32_t at = of_lane(from, 0) + upto - mine;
            while (hits) {
                const int bit = __builtin_ctz(hits);
                hits &= hits - 1;
                put(at++, s.body + (i + bit / E * threads) * E + bit % E);
            }
        }
    }
}

// Lists the elements [begin, end) that lie in wanted bins, and a few others.
template <typename T>
__device__ __forceinline__ void list_wanted(const T *row, int begin, int end, int threads, double per_unit, int top_bin,
                                            const Wanted &w, uint32_t *listed, uint32_t *places, int cap, Entry *list)
{
    const Intervals v = intervals_of(w, per_unit, top_bin);
    if (v.number <= 2)
        list_places<2>(row, begin, end, threads, v, listed, places, cap);
    else
        list_places<4>(row, begin, end, threads, v, listed, places, cap);
    __syncthreads();
    const int n = *listed < (uint32_t)cap ? (int)*listed : cap;
    for (int i = threadIdx.x; i < n; i += threads) {
        const uint32_t place = places[i];
        list[i] = Entry{(float)row[place], place};
    }
}

// ---------------------------------------------------------------------------
// 2. Gather of one slice (rows cut into several).
// ---------------------------------------------------------------------------
template <typename T>
__global__ __launch_bounds__(kThreads) void sample_gather_kernel(const SampleArgs a, int S)
{
    __shared__ RowSums sums;
    __shared__ WaveSums<double> waves;
    __shared__ Joined joined;
    __shared__ uint32_t listed, places[kSliceList];
    const int s = blockIdx.x, row = blockIdx.y;
    if (threadIdx.x == 0)
        listed = 0;
    const RowParams p = params_of(a, row);
    join_slices<kThreads, 32>(a, row, S, p.per_unit, sums, waves, joined);
    if (s == 0) {  // for the finish
        const uint32_t *from = reinterpret_cast<const uint32_t *>(&sums);
        uint32_t *to = reinterpret_cast<uint32_t *>(sums_of(a, row, S));
        for (int i = threadIdx.x; i < (int)(sizeof(RowSums) / 4); i += kThreads)
            to[i] = from[i];
    }
    if (!sums.fine)
        return;
    const double top_scaled = (double)sums.top * p.per_unit;
    const Wanted w = wanted_bins(sums, p, top_scaled);
    int begin, end;
    slice_of(a.V, S, s, begin, end);
    char *out = slice_at(a, row, s, S);
    list_wanted(static_cast<const T *>(a.logits) + row * a.row_stride, begin, end, kThreads, p.per_unit,
                binned(top_scaled).bin, w, &listed, places, kSliceList, list_of(out));
    if (threadIdx.x == 0)
        head_of(out)->listed = listed;
}

// ---------------------------------------------------------------------------
// 3. Finish: one workgroup a row.
// ---------------------------------------------------------------------------
struct alignas(16) Ranked {
    uint64_t place;   // order_key and ~index: greater is earlier in the order, 0 is no element
    uint32_t weight;
};
template <int THREADS>
struct Finish {
    RowSums sums;
    WaveSums<double> waves;
    WaveSums<long long> part_waves;
    uint32_t part_count[kParts];
    unsigned long long part_sum[kParts];
    Entry list[kList];
    union {
        Ranked ranked[kRanked];
        uint32_t places[kList];
        Joined joined;
    };
    double factor[kBins];
    uint32_t listed, chosen;
    uint32_t low_key, high_key, number;      // of the current range
    uint32_t found, found_count, found_last;
    unsigned long long found_sum;
    uint32_t key, nth;                       // the crossing element's
    unsigned long long mass;
};

// The four searches: the k-th element, top-p's last, min-p's last, the token.
enum Query { kTopK, kTopP, kMinP, kToken };

// Whether the elements up to one of weight w, before which there are `before`
// elements of mass `from`, cross.
__device__ __forceinline__ bool crosses(int query, uint32_t before, unsigned long long from, uint32_t number,
                                        unsigned long long w, uint32_t count, double value)
{
    if (query == kTopK)
        return before < count && before + number >= count;
    const double lo = (double)from, hi = (double)(from + w);
    return query == kTopP ? lo < value && hi >= value : lo <= value && hi > value;
}

// Where the listed elements of bin t, in order, cross a count or a mass (in
// units of the weights): f.key, f.nth (its index) and f.mass (of the bin's
// elements up to and with it). If they do not cross, the last element. False
// (for all threads) if more elements than can be ranked share a part of the bin.
template <int THREADS>
__device__ __forceinline__ bool find_listed(Finish<THREADS> &f, int t, int top_bin, double per_unit, int query, uint32_t count,
                                            double value, double top_scaled, double log_min_p)
{
    const uint32_t total = f.sums.count[t] - count_before(f.sums, t);
    int part = -1;
    uint32_t before = 0;
    unsigned long long mass = 0;
    // Each of a thread's elements of bin t, with its part and weight.
    auto each = [&](auto g) {
        for (uint32_t i = threadIdx.x; i < f.listed; i += THREADS) {
            const Entry e = f.list[i];
            const double d = scaled<false>(e.x, per_unit, 0.f);
            const Binned b = binned(d);
            if (d > top_scaled - kBins - 1 && top_bin - b.bin == t)  // not NaN either
                g(e, b.part, b.weight(), d);
        }
    };
    if (threadIdx.x == 0) {
        f.chosen = 0;
        f.found = 0xFFFFFFFFu;
        f.mass = 0;
    }
    if (query == kMinP) {  // the elements that pass the comparison
        __syncthreads();
        unsigned long long sum = 0;
        each([&](const Entry &, int, uint32_t w, double d) {
            sum += (d - top_scaled) / kPerUnit >= log_min_p ? w : 0u;
        });
#pragma unroll
        for (int d = 1; d < kWave; d *= 2)
            sum += __shfl_xor(sum, d);
        if (threadIdx.x % kWave == 0 && sum)
            atomicAdd(&f.mass, sum);
        __syncthreads();
        return true;
    }
    if (total > kWhole) {
        if (threadIdx.x < kParts)
            f.part_sum[threadIdx.x] = 0;
        __syncthreads();
        each([&](const Entry &, int part, uint32_t w, double) {  // packed as in the histogram
            atomicAdd(&f.part_sum[part], ((unsigned long long)1 << kSumBits) + (w - kLeast));
        });
        __syncthreads();
        uint32_t mine = 0;
        uint64_t over = 0;
        if (threadIdx.x < kParts)
            unpack(f.part_sum[threadIdx.x], mine, over);
        const long long my_mass = (long long)mass_of(mine, over);
        uint32_t c = mine;
        long long m = my_mass;
        block_sums<THREADS>(c, m, f.part_waves);
        if (mine && crosses(query, c - mine, (unsigned long long)(m - my_mass), mine, (unsigned long long)my_mass, count,
                            value))
            f.found = threadIdx.x;
        if (mine && c == total)
            f.found_last = threadIdx.x;
        __syncthreads();
        part = (int)(f.found != 0xFFFFFFFFu ? f.found : f.found_last);
        if ((int)threadIdx.x == part) {
            f.found_count = c - mine;
            f.found_sum = (unsigned long long)(m - my_mass);
            f.number = mine;
        }
        __syncthreads();
        before = f.found_count;
        mass = f.found_sum;
        if (f.number > kRanked) {
            __syncthreads();  // all have read f.number, which the caller's next search clears
            return false;
        }
    }
    for (int i = threadIdx.x; i < kRanked; i += THREADS)
        f.ranked[i].place = 0;
    __syncthreads();
    each([&](const Entry &e, int p, uint32_t w, double) {
        if (part < 0 || p == part)
            f.ranked[atomicAdd(&f.chosen, 1u)] = Ranked{(uint64_t)order_key(e.x) << 32 | (uint32_t)~e.index, w};
    });
    __syncthreads();
    // Each element is compared with all, where they are many by several
    // neighbouring lanes (16-bit logits leave hundreds of equal ones: 258 take
    // 7.2 us, by one lane each 13); for a few the lanes' sums would cost more.
    constexpr int AT_ONCE = 4;
    const uint32_t n = f.chosen;
    int lanes = 0;  // their logarithm
    while ((n >> lanes) > 16 && (n << (lanes + 1)) <= (uint32_t)THREADS)
        ++lanes;
    // a turn starts below n, at a multiple of AT_ONCE << lanes, and stays inside
    static_assert(kRanked % (AT_ONCE * kScanThreads / 16) == 0, "kRanked is a multiple of a turn");
    const uint32_t share = threadIdx.x & ((1u << lanes) - 1);
    for (uint32_t i = threadIdx.x >> lanes; i < n; i += (uint32_t)THREADS >> lanes) {
        const Ranked mine = f.ranked[i];
        uint32_t c = 0;
        unsigned long long from = 0;
        for (uint32_t j0 = share; j0 < n; j0 += AT_ONCE << lanes) {
            Ranked e[AT_ONCE];
#pragma unroll
            for (int j = 0; j < AT_ONCE; ++j)
                e[j] = f.ranked[j0 + (j << lanes)];
#pragma unroll
            for (int j = 0; j < AT_ONCE; ++j) {
                const bool earlier = e[j].place > mine.place;
                c += earlier ? 1u : 0u;
                from += earlier ? e[j].weight : 0u;
            }
        }
        for (int d = 1; d < 1 << lanes; d *= 2) {
            c += __shfl_xor(c, d);
            from += __shfl_xor(from, d);
        }
        c += before;
        from += mass;
        const bool last = c + 1 == before + n;
        const bool here = crosses(query, c, from, 1, mine.weight, count, value);
        // not crossed: the last element (its sum is below the value, or the count)
        const bool none = last && (query == kTopK   ? c + 1 < count
                                   : query == kTopP ? (double)(from + mine.weight) < value
                                                    : (double)(from + mine.weight) <= value);
        if (share == 0 && (here || none)) {
            f.key = (uint32_t)(mine.place >> 32);
            f.nth = ~(uint32_t)mine.place;
            f.mass = from + mine.weight;
        }
    }
    __syncthreads();
    return true;
}

// All searches by one wave, without a barrier, of a list of up to 64 elements, one
// a lane (16 rows of 151001 logits with top-k and top-p: 26 us a call, 28 without
// it). Sets f.key and f.nth, the kept mass and the token's bin.
template <int THREADS>
__device__ __forceinline__ void search_few(Finish<THREADS> &f, const RowParams &p, int top_bin, double top_scaled,
                                           double &kept, int &t)
{
    const int lane = threadIdx.x;
    const Search find(f.sums);
    const bool mine = lane < (int)f.listed;
    const Entry e = f.list[mine ? lane : 0];
    const double scale = scaled<false>(e.x, p.per_unit, 0.f);
    const Binned b = binned(scale);
    const int below = mine && scale > top_scaled - kBins - 1 ? top_bin - b.bin : -1;
    const uint64_t place = (uint64_t)order_key(e.x) << 32 | (uint32_t)~e.index;
    const uint32_t weight = b.weight();
    double limit = kept;
#pragma unroll 1
    for (int query = kTopK; query <= kToken; ++query) {
        uint32_t count = 0;
        double value = 0.0;
        if (query == kTopK) {
            t = p.top_k > 0 ? find.first_count(p.top_k) : kBins;
            if (t == kBins)
                continue;
            count = p.top_k - count_before(f.sums, t);
        } else if (query == kMinP) {
            t = min_p_bin(p, top_scaled);
            if (t < 0)
                continue;
        } else {
            if (query == kTopP && !(p.top_p < 1.0))
                continue;
            const double target = query == kTopP ? p.top_p * limit : p.u * kept;
            t = query == kTopP ? find.template first_mass<false>(target) : find.template first_mass<true>(target);
            value = (target - mass_before(f.sums, t)) / f.factor[t];
            const double least = query == kTopP ? 0.5 : 0.0;
            value = value > least ? value : least;
        }
        unsigned long long mass;
        if (query == kMinP) {
            mass = below == t && (scale - top_scaled) / kPerUnit >= p.log_min_p ? weight : 0u;
            mass = of_lane(wave_sums(mass), kWave - 1);
        } else {
            uint64_t bin = __ballot(below == t);
            if (__builtin_expect(bin == 0, 0)) {
                leave_empty_bin(f.sums, find, t, value);
                bin = __ballot(below == t);
            }
            const uint32_t n = __popcll(bin);
            uint32_t c = 0;
            unsigned long long from = 0;
            for (uint64_t left = bin; left; left &= left - 1) {
                const int j = __builtin_ctzll(left);
                const bool earlier = of_lane(place, j) > place;
                const uint32_t other = of_lane(weight, j);
                c += earlier ? 1u : 0u;
                from += earlier ? other : 0u;
            }
            const bool here = crosses(query, c, from, 1, weight, count, value);
            const bool none = c + 1 == n && (query == kTopK   ? n < count
                                             : query == kTopP ? (double)(from + weight) < value
                                                              : (double)(from + weight) <= value);
            const uint64_t found = __ballot(below == t && (here || none));
            const int who = found ? __builtin_ctzll(found) : 0;  // one is, as no bin with a crossing is empty
            mass = of_lane(from + weight, who);
            const uint64_t chosen = of_lane(place, who);
            if (lane == 0) {
                f.key = (uint32_t)(chosen >> 32);
                f.nth = ~(uint32_t)chosen;
            }
        }
        if (query != kToken) {
            const double m = mass_before(f.sums, t) + (double)mass * f.factor[t];
            kept = m < kept ? m : kept;
            if (query == kTopK)
                limit = kept;
        }
    }
}

// Smallest and largest value and number of the elements that pass.
template <int THREADS, typename Each>
__device__ __forceinline__ void range_of(Finish<THREADS> &f, Each each)
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
    while ((range >> s) >= (uint32_t)kParts)
        ++s;
    return s;
}

// The same searches over the row itself, for lists that overflow and rows out of
// the histogram's range: a range of values is narrowed 512-fold a turn, by keys
// for the crossing and then by indexes among equal keys. With `indexes` the
// values are the indexes of the elements whose key is f.key and the crossing is
// the count'th; else they are keys, and f.key, f.nth (which of the equal ones, 1,
// 2, ...) and f.mass are set.
template <typename T, bool REL, int THREADS>
__device__ __forceinline__ void narrow(Finish<THREADS> &f, const T *row, int V, int t, int top_bin, double per_unit, float ref,
                                       double top_scaled, bool indexes, int query, uint32_t count, double value)
{
    const uint32_t key = f.key;
    uint32_t low = 0, high = 0xFFFFFFFFu, before = 0;
    unsigned long long mass = 0;
    // Values to find stand in falling order for keys, in rising order for indexes.
    auto each = [&](auto g) {
        for_elements<T, 1>(row, 0, V, THREADS, [&](float x, int i) {
            const double d = scaled<REL>(x, per_unit, ref);
            if (d > top_scaled - kBins - 1) {
                const Binned b = binned(d);
                const uint32_t k = order_key(x), v = indexes ? ~(uint32_t)i : k;
                if (top_bin - b.bin == t && (!indexes || k == key) && v >= low && v <= high)
                    g(v, b.weight());
            }
        });
    };
    for (;;) {  // every turn narrows [low, high] by a factor of 512 or ends
        range_of(f, [&](auto add) { each([&](uint32_t v, uint32_t) { add(v); }); });
        low = f.low_key;
        high = f.high_key;
        const uint32_t number = f.number;
        __syncthreads();
        if (number == 0 || low == high) {
            if (threadIdx.x == 0) {
                if (indexes) {
                    f.nth = ~low;
                } else {
                    const double d = scaled<REL>(key_value(low), per_unit, ref);
                    const unsigned long long w = binned(d).weight();
                    uint32_t j = number;
                    if (query == kTopK) {
                        j = count - before;
                    } else {
                        const double left = (value - (double)mass) / (double)w;
                        const double n = query == kTopP ? ceil(left) : floor(left) + 1.0;
                        j = n < 1.0 ? 1u : n < (double)number ? (uint32_t)n : number;
                    }
                    j = j < 1 ? 1 : j > number ? number : j;
                    f.key = low;
                    f.nth = j;
                    f.mass = mass + j * w;
                }
            }
            __syncthreads();
            return;
        }
        const int shift = shift_for(high - low);
        if (threadIdx.x < kParts) {
            f.part_count[threadIdx.x] = 0;
            f.part_sum[threadIdx.x] = 0;
        }
        if (threadIdx.x == 0)
            f.found = 0xFFFFFFFFu;
        __syncthreads();
        each([&](uint32_t v, uint32_t w) {
            const uint32_t part = (high - v) >> shift;
            atomicAdd(&f.part_count[part], 1u);
            atomicAdd(&f.part_sum[part], (unsigned long long)w);
        });
        __syncthreads();
        const uint32_t mine = threadIdx.x < kParts ? f.part_count[threadIdx.x] : 0;
        const long long my_mass = threadIdx.x < kParts ? (long long)f.part_sum[threadIdx.x] : 0;
        uint32_t c = mine;
        long long m = my_mass;
        block_sums<THREADS>(c, m, f.part_waves);
        if (mine && crosses(indexes ? (int)kTopK : query, before + c - mine, mass + (unsigned long long)(m - my_mass), mine,
                            (unsigned long long)my_mass, count, value))
            f.found = threadIdx.x;
        if (mine && c == number)
            f.found_last = threadIdx.x;
        __syncthreads();
        const uint32_t part = f.found != 0xFFFFFFFFu ? f.found : f.found_last;
        if (threadIdx.x == part) {
            f.found_count = before + c - mine;
            f.found_sum = mass + (unsigned long long)(m - my_mass);
        }
        __syncthreads();
        before = f.found_count;
        mass = f.found_sum;
        const uint32_t top = high - (part << shift);
        const uint32_t width = (1u << shift) - 1;
        low = top - low > width ? top - width : low;
        high = top;
        __syncthreads();
    }
}

template <typename T, bool REL, int THREADS>
__device__ __forceinline__ void find_in_row(Finish<THREADS> &f, const T *row, int V, int t, int top_bin, double per_unit,
                                            float ref, double top_scaled, int query, uint32_t count, double value,
                                            double log_min_p)
{
    if (query == kMinP) {
        if (threadIdx.x == 0)
            f.mass = 0;
        __syncthreads();
        unsigned long long sum = 0;
        for_elements<T, 1>(row, 0, V, THREADS, [&](float x, int) {
            const double d = scaled<REL>(x, per_unit, ref);
            if (d > top_scaled - kBins - 1) {
                const Binned b = binned(d);
                if (top_bin - b.bin == t && (d - top_scaled) / kPerUnit >= log_min_p)
                    sum += b.weight();
            }
        });
#pragma unroll
        for (int d = 1; d < kWave; d *= 2)
            sum += __shfl_xor(sum, d);
        if (threadIdx.x % kWave == 0 && sum)
            atomicAdd(&f.mass, sum);
        __syncthreads();
        return;
    }
    // First the key, then for the token the index among equal keys.
    for (int pass = 0; pass < (query == kToken ? 2 : 1); ++pass)
        narrow<T, REL, THREADS>(f, row, V, t, top_bin, per_unit, ref, top_scaled, pass == 1, query, pass == 1 ? f.nth : count,
                       value);
}

template <typename T, int THREADS>
__global__ __launch_bounds__(THREADS) void sample_finish_kernel(const SampleArgs a, int S)
{
    __shared__ Finish<THREADS> f;
    const int row = blockIdx.x;
    const RowParams p = params_of(a, row);
    const T *x = static_cast<const T *>(a.logits) + row * a.row_stride;
    if (threadIdx.x == 0)
        f.listed = 0;
    if (threadIdx.x < kBins)
        f.factor[threadIdx.x] = factors.of[threadIdx.x];
    constexpr bool kLists = THREADS == kScanThreads;  // no gather before
    if constexpr (kLists) {
        join_slices<THREADS, 8>(a, row, S, p.per_unit, f.sums, f.waves, f.joined);
    } else {
        const uint32_t *from = reinterpret_cast<const uint32_t *>(sums_of(a, row, S));
        uint32_t *to = reinterpret_cast<uint32_t *>(&f.sums);
        for (int i = threadIdx.x; i < (int)(sizeof(RowSums) / 4); i += THREADS)
            to[i] = from[i];
        __syncthreads();
    }
    const float top = f.sums.top;
    if (top == -__builtin_inff()) {  // no logit above -inf
        if (threadIdx.x == 0) {
            a.tokens[row] = -1;
            if (a.logprobs)
                a.logprobs[row] = -__builtin_inff();
        }
        return;
    }
    const bool fine = f.sums.fine;
    const double top_scaled = fine ? (double)top * p.per_unit : 0.0;
    const int top_bin = binned(top_scaled).bin;
    // Elements of the wanted bins: of all searches at once, from the gather or
    // (one slice) listed below; where these are too many, of one search at a time.
    Wanted w;
    bool listed = fine, one_by_one = false;
    if (fine && kLists) {
        w = wanted_bins(f.sums, p, top_scaled);
        list_wanted(x, 0, a.V, THREADS, p.per_unit, top_bin, w, &f.listed, f.places, kList, f.list);
        __syncthreads();
        one_by_one = f.listed > kList;
        __syncthreads();
    } else if (fine) {
        const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
        const uint32_t own = lane < S ? head_of(slice_at(a, row, lane, S))->listed : 0;
        uint32_t upto = own;
#pragma unroll
        for (int d = 1; d < kWave; d *= 2) {
            const uint32_t v = __shfl_up(upto, d);
            upto += lane >= d ? v : 0;
        }
        const uint32_t total = __shfl(upto, kWave - 1);
        one_by_one = __any(own > kSliceList) || total > kList;
        if (!one_by_one)
            for (int s = wave; s < S; s += THREADS / kWave) {
                const uint32_t n = __shfl(own, s), to = __shfl(upto, s) - n;
                const Entry *list = list_of(slice_at(a, row, s, S));
                for (uint32_t i = lane; i < n; i += kWave)
                    f.list[to + i] = list[i];
            }
        if (threadIdx.x == 0)
            f.listed = total;
        __syncthreads();
    } else {
        // Counted again, relative to the maximum.
        if (threadIdx.x < kParts) {
            f.part_count[threadIdx.x] = 0;
            f.part_sum[threadIdx.x] = 0;
        }
        __syncthreads();
        for_elements<T, 1>(x, 0, a.V, THREADS, [&](float v, int) {
            const double d = scaled<true>(v, p.per_unit, top);
            if (d > -(kBins - 1)) {
                const Binned b = binned(d);
                atomicAdd(&f.part_count[-b.bin & (kParts - 1)], 1u);
                atomicAdd(&f.part_sum[-b.bin & (kParts - 1)], (unsigned long long)b.over);
            }
        });
        __syncthreads();
        const int t = threadIdx.x;
        const uint32_t c = t < kBins ? f.part_count[t] : 0;
        const double m =
            t < kBins ? (double)mass_of(c, f.part_sum[t]) * f.factor[t] : 0.0;
        __syncthreads();
        store_sums<THREADS>(f.sums, c, m, f.waves);
    }

    // The searches, in the order of the filters.
    double kept = f.sums.mass[kBins - 1], limit = kept;  // mass kept so far; of the top-k prefix
    int t = 0;
    bool few = false;
    if (fine && !one_by_one && f.listed <= kWave) {
        if (threadIdx.x >= kWave)
            return;
        search_few(f, p, top_bin, top_scaled, kept, t);
        few = true;
    }
    for (int query = few ? kToken + 1 : kTopK; query <= kToken; ++query) {
        const Search find(f.sums);  // read again: held over the turns, its 18 registers would spill
        uint32_t count = 0;
        double value = 0.0;
        if (query == kTopK) {
            t = p.top_k > 0 ? find.first_count(p.top_k) : kBins;
            if (t == kBins)
                continue;
            count = p.top_k - count_before(f.sums, t);
        } else if (query == kMinP) {
            t = min_p_bin(p, top_scaled);
            if (t < 0)
                continue;
        } else {
            if (query == kTopP && !(p.top_p < 1.0))
                continue;
            const double target = query == kTopP ? p.top_p * limit : p.u * kept;
            t = query == kTopP ? find.first_mass<false>(target) : find.first_mass<true>(target);
            // A value that rounding took to the bin's edge still crosses at the
            // first element (every weight is far above 1/2).
            value = (target - mass_before(f.sums, t)) / f.factor[t];
            const double least = query == kTopP ? 0.5 : 0.0;
            value = value > least ? value : least;
            leave_empty_bin(f.sums, find, t, value);
        }
        if (one_by_one) {
            if (threadIdx.x == 0)
                f.listed = 0;
            __syncthreads();
            w = Wanted{t, 0, -1, -1, 0, -1};
            list_wanted(x, 0, a.V, THREADS, p.per_unit, top_bin, w, &f.listed, f.places, kList, f.list);
            __syncthreads();
            listed = f.listed <= kList;
            __syncthreads();
        }
        bool done = false;
        if (listed)
            done = find_listed(f, t, top_bin, p.per_unit, query, count, value, top_scaled, p.log_min_p);
        if (__builtin_expect(!done, 0)) {
            if (fine)
                find_in_row<T, false, THREADS>(f, x, a.V, t, top_bin, p.per_unit, 0.f, top_scaled, query, count, value, p.log_min_p);
            else
                find_in_row<T, true, THREADS>(f, x, a.V, t, top_bin, p.per_unit, top, top_scaled, query, count, value, p.log_min_p);
        }
        if (query != kToken) {
            const double m = mass_before(f.sums, t) + (double)f.mass * f.factor[t];
            kept = m < kept ? m : kept;
            if (query == kTopK)
                limit = kept;
            __syncthreads();
        }
    }
    if (threadIdx.x == 0) {
        a.tokens[row] = (int32_t)f.nth;
        if (a.logprobs) {
            // the weight as the sums hold it, so that a token kept alone has share 1
            const float v = key_value(f.key);
            const Binned b = binned(fine ? scaled<false>(v, p.per_unit, 0.f) : scaled<true>(v, p.per_unit, top));
            const double lp = log((double)b.weight() * f.factor[t] / kept);
            a.logprobs[row] = lp < 0.0 ? (float)lp : 0.f;
        }
    }
}

// ---------------------------------------------------------------------------
// Rows of bf16 logits: one workgroup a row and no bins. A row has at most
// 65536 different logits, so that their numbers fit the LDS; the filters and the
// token's logit follow from sums over the values in falling order, and one more
// pass finds which of the equal ones the token is. Counting takes 4 instructions
// an element where the histogram of bins takes 20, and nothing is listed: 256
// rows of 131072 logits with top-p take 35 us, by bins 68 (counting 11, at 6 TB/s,
// the values' sums 8, searches 4, the last pass 3 to 8). In fp16, whose values near
// zero lie four times as densely, the sums take more than that saves: the same
// rows 49 us (46 by bins), 32 rows of 32003 with top-k and min-p 31 (24).
// ---------------------------------------------------------------------------
constexpr int kWords = 1 << 15;                // of counts: by magnitude; positive logits in the low half, negative in the high
constexpr int kGroups = 2 * kWords / kWave;    // of 64 values in falling order: positive ones from the largest, then negative ones

constexpr uint32_t kInfinity = 0x7F80;

__device__ __forceinline__ float value_of(uint32_t bits) { return __builtin_bit_cast(float, bits << 16); }

struct Values {
    uint32_t counts[kWords];
    double mass[kGroups];       // of the groups up to and with each
    uint32_t count[kGroups];
    WaveSums<double> waves;
    uint32_t seen[kScanThreads / kWave];
    uint32_t first;             // place of the largest logit in falling order
    uint32_t heavy[2], heavy_count[2], heavies;  // logits of more than 65535 elements, which have no place in `counts`
    uint32_t numbers[2][kWave];
    uint32_t bits, nth, index;  // the token's logit, which of the equal ones, and where it stands
};

// Bits of the logit at a place in falling order (0: the largest), and how many
// elements have it; none for NaN and -inf. -0 counts as 0.
__device__ __forceinline__ uint32_t bits_at(uint32_t place) { return place < kWords ? kWords - 1 - place : place; }
__device__ __forceinline__ uint32_t count_at(const Values &f, uint32_t place, uint32_t heavies)
{
    const uint32_t bits = bits_at(place), word = bits & (kWords - 1);
    const uint32_t w = f.counts[word];
    const bool negative = place >= kWords;
    uint32_t c = negative ? w >> 16 : w & 0xFFFFu;
    if (word == 0)
        c = negative ? 0u : c + (w >> 16);
    for (uint32_t k = 0; k < heavies; ++k) {
        const uint32_t h = f.heavy[k] == 0x8000u ? 0u : f.heavy[k];
        c += h == bits ? f.heavy_count[k] : 0u;
    }
    return word < kInfinity || (word == kInfinity && !negative) ? c : 0u;
}

// Scaled logit relative to the largest one.
__device__ __forceinline__ double below_top(float x, float top, double per_unit, bool fine)
{
    return fine ? (double)x * per_unit - (double)top * per_unit : scaled<true>(x, per_unit, top);
}

// e^(d/8) for d of -384 .. 0, exactly 1 for 0: 2^n times the series of e^r, |r| up to
// ln 2 / 2, whose first term left out is below 2^-41 (a library's exponential,
// good to the last bit, is three times the code).
__device__ __forceinline__ double exp_eighth(double d)
{
    const double n = rint(d * 0.18033688011112042);             // log2(e) / 8
    const double r = __builtin_fma(n, -5.5451774444795623, d) * 0.125;  // 8 ln 2
    double e = 1.0 / 3628800.0;
    constexpr double inverse[10] = {1.0, 1.0, 1.0 / 2, 1.0 / 6, 1.0 / 24, 1.0 / 120, 1.0 / 720, 1.0 / 5040, 1.0 / 40320, 1.0 / 362880};
#pragma unroll
    for (int k = 9; k >= 0; --k)
        e = __builtin_fma(e, r, inverse[k]);
    return __builtin_ldexp(e, (int)n);
}

// The lanes' values of a group: how many elements, and their mass each.
__device__ __forceinline__ void group_at(const Values &f, uint32_t group, uint32_t heavies, float top, double per_unit, bool fine,
                                         uint32_t &count, double &weight)
{
    const uint32_t place = group * kWave + threadIdx.x % kWave;
    count = count_at(f, place, heavies);
    const double d = below_top(value_of(bits_at(place)), top, per_unit, fine);
    if (!(d > 1 - kBins))  // e^-48 of the largest, as above; NaN where infinity times 0 is
        count = 0;
    weight = count ? exp_eighth(d) : 0.0;
}

__device__ __forceinline__ void count_values(Values &f, const uint16_t *bits, int V)
{
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    const Span s = span_of_row(bits, 0, V, 2);
    auto add = [&](uint32_t b) { atomicAdd(&f.counts[b & (kWords - 1)], b & 0x8000u ? 0x10000u : 1u); };
    if ((int)threadIdx.x < s.body)
        add(bits[threadIdx.x]);
    if ((int)threadIdx.x < V - s.tail)
        add(bits[s.tail + threadIdx.x]);
    const u32x4 *p = reinterpret_cast<const u32x4 *>(bits + s.body);
    constexpr int UNROLL = 4;
    for (int i = threadIdx.x; i < s.units; i += UNROLL * kScanThreads) {
        u32x4 v[UNROLL];
#pragma unroll
        for (int j = 0; j < UNROLL; ++j)
            v[j] = p[i + j * kScanThreads < s.units ? i + j * kScanThreads : i];
#pragma unroll
        for (int j = 0; j < UNROLL; ++j)
            if (i + j * kScanThreads < s.units)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    add(v[j][e] & 0xFFFFu);
                    add(v[j][e] >> 16);
                }
    }
}

// For rows with a logit of more than 65535 elements (two at most, see kMostByValues): which
// they are, by their high and then their low bytes, and the counts without them.
__device__ __forceinline__ void count_without_heavy(Values &f, const uint16_t *row, int V)
{
    uint32_t high[2] = {0, 0};
    for (int turn = 0; turn < 3; ++turn) {  // the high bytes; the low ones of up to two high ones
        if (turn > 0 && high[turn - 1] == 0)
            break;
        __syncthreads();
        if (threadIdx.x < 256)
            f.counts[threadIdx.x] = 0;
        __syncthreads();
        const uint32_t of = turn > 0 ? high[turn - 1] - 1 : 0;
        for_elements<uint16_t, 1>(row, 0, V, kScanThreads, [&](float x, int) {
            const uint32_t b = (uint32_t)x;
            if (turn == 0 || b >> 8 == of)
                atomicAdd(&f.counts[turn == 0 ? b >> 8 : b & 255], 1u);
        });
        __syncthreads();
        for (uint32_t b = 0; b < 256; ++b)  // by all threads alike
            if (f.counts[b] > 65535u) {
                if (turn == 0) {
                    high[high[0] ? 1 : 0] = b + 1;
                } else if (threadIdx.x == 0) {
                    f.heavy[f.heavies] = of << 8 | b;
                    f.heavy_count[f.heavies++] = f.counts[b];
                }
            }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kWords; i += kScanThreads)
        f.counts[i] = 0;
    const uint32_t n = f.heavies, h0 = n > 0 ? f.heavy[0] : 0x10000u, h1 = n > 1 ? f.heavy[1] : 0x10000u;
    __syncthreads();
    for_elements<uint16_t, 1>(row, 0, V, kScanThreads, [&](float x, int) {
        const uint32_t b = (uint32_t)x;
        if (b != h0 && b != h1)
            atomicAdd(&f.counts[b & (kWords - 1)], b & 0x8000u ? 0x10000u : 1u);
    });
    __syncthreads();
}

// Which of a word's two elements have the bits looked for: `mask` leaves out the
// sign where they are 0.
__device__ __forceinline__ uint32_t hits_of(uint32_t w, uint32_t mask, uint32_t both)
{
    const uint32_t e = (w & mask) ^ both;
    return ((e & 0xFFFFu) == 0 ? 1u : 0u) + (e < 0x10000u ? 2u : 0u);
}

// Where the nth (1, 2, ...) element of the given bits stands: 4096 units of 16
// bytes at a time, in order, until it is among them (the next ones on their way).
__device__ __forceinline__ void find_nth(Values &f, const uint16_t *row, int V)
{
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    constexpr int WAVES = kScanThreads / kWave, TURN = 4;
    static_assert(TURN * WAVES == kWave, "a wave's lanes look at all numbers of a turn");
    uint32_t nth = f.nth;
    const uint32_t wanted = f.bits, mask = wanted ? 0xFFFFFFFFu : 0x7FFF7FFFu, both = wanted << 16 | wanted;
    const Span s = span_of_row(row, 0, V, 2);
    const u32x4 *p = reinterpret_cast<const u32x4 *>(row + s.body);
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    // Single elements before the units and behind them, fewer than 8: by every wave alike.
    auto single = [&](int begin, int end) {
        const bool hit = begin + lane < end && ((row[begin + lane] & mask) ^ (wanted & mask)) == 0;
        const uint64_t hits = __ballot(hit);
        if (hit && (uint32_t)__popcll(hits & (((uint64_t)2 << lane) - 1)) == nth)
            f.index = begin + lane;
        const uint32_t n = __popcll(hits);
        const bool found = nth <= n;
        nth -= found ? 0 : n;
        return found;
    };
    if (single(0, s.body))
        return;
    u32x4 v[TURN], next[TURN];
    auto load = [&](u32x4 *to, int i) {
#pragma unroll
        for (int j = 0; j < TURN; ++j)
            to[j] = p[i + j * kScanThreads < s.units ? i + j * kScanThreads : 0];
    };
    if (s.units > 0)
        load(next, threadIdx.x);
    int turn = 0;
    for (int i0 = 0; i0 < s.units; i0 += TURN * kScanThreads, turn ^= 1) {
        const int i = i0 + (int)threadIdx.x;
#pragma unroll
        for (int j = 0; j < TURN; ++j)
            v[j] = next[j];
        load(next, i + TURN * kScanThreads);
        uint32_t hits = 0;  // bit 8 j + e
#pragma unroll
        for (int j = 0; j < TURN; ++j) {
            uint32_t h = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                h |= hits_of(v[j][e], mask, both) << 2 * e;
            hits |= (i + j * kScanThreads < s.units ? h : 0u) << 8 * j;
        }
        // a wave's numbers of each quarter (512 at most), two to a word
        const uint32_t n01 = of_lane(wave_sums(__popc(hits & 0xFFu) | __popc(hits & 0xFF00u) << 16), kWave - 1);
        const uint32_t n23 = of_lane(wave_sums(__popc(hits & 0xFF0000u) | __popc(hits >> 24) << 16), kWave - 1);
        if (lane < TURN)
            f.numbers[turn][lane * WAVES + wave] = ((lane & 2 ? n23 : n01) >> (lane & 1 ? 16 : 0)) & 0xFFFFu;
        __syncthreads();
        const uint32_t own = f.numbers[turn][lane], upto = wave_sums(own);
        const uint64_t reached = __ballot(upto >= nth);
        if (reached) {
            const int at = __builtin_ctzll(reached);
            nth -= of_lane(upto - own, at);
            if (wave == at % WAVES) {
                uint32_t h = hits >> 8 * (at / WAVES) & 0xFFu;
                const uint32_t mine = __popc(h), to = wave_sums(mine);
                if (nth > to - mine && nth <= to) {
                    for (uint32_t k = to - mine + 1; k < nth; ++k)
                        h &= h - 1;
                    f.index = s.body + 8 * (i + at / WAVES * kScanThreads) + __builtin_ctz(h);
                }
            }
            return;
        }
        nth -= of_lane(upto, kWave - 1);
    }
    single(s.tail, V);
}

__global__ __launch_bounds__(kScanThreads) void sample_values_kernel(const SampleArgs a)
{
    __shared__ Values f;
    constexpr int WAVES = kScanThreads / kWave;
    const int row = blockIdx.x, lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const uint16_t *x = static_cast<const uint16_t *>(a.logits) + row * a.row_stride;
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    for (int i = threadIdx.x; i < kWords / 4; i += kScanThreads)
        reinterpret_cast<u32x4 *>(f.counts)[i] = u32x4{0, 0, 0, 0};
    if (threadIdx.x == 0) {
        f.heavies = 0;
        f.first = 0xFFFFFFFFu;
    }
    const RowParams p = params_of(a, row);
    __syncthreads();
    count_values(f, x, a.V);
    __syncthreads();
    // Both halves' groups of a word's 64 go to one wave. The sum of all counts
    // tells whether one passed 65535: each time takes 65535 or 65536 off.
    uint32_t sum = 0, used = 0;  // bit j: group wave + 16 j has elements
    for (int j = 0; j < kWords / kWave / WAVES; ++j) {
        const uint32_t w = f.counts[(wave + WAVES * j) * kWave + lane];
        sum += (w & 0xFFFFu) + (w >> 16);
        used |= __any(w != 0) ? 1u << j : 0u;
    }
    sum = of_lane(wave_sums(sum), kWave - 1);
    if (lane == 0)
        f.seen[wave] = sum;
    __syncthreads();
    sum = 0;
    for (int j = 0; j < WAVES; ++j)
        sum += f.seen[j];
    if (__builtin_expect(sum != (uint32_t)a.V, 0)) {
        count_without_heavy(f, x, a.V);
        used = 0xFFFFFFFFu;
    }
    const uint32_t heavies = f.heavies;
    // The largest logit: the first place in falling order that has elements.
    uint32_t first = 0xFFFFFFFFu;
    bool found = false;
    for (uint32_t left = used; left && !found; left &= ~(0x80000000u >> __builtin_clz(left))) {  // positive ones from the largest
        const uint32_t place = kWords - (wave + WAVES * (31 - __builtin_clz(left)) + 1) * kWave + lane;
        first = count_at(f, place, heavies) ? place : first;
        found = __any(first != 0xFFFFFFFFu);
    }
    for (uint32_t left = used; left && !found; left &= left - 1) {  // negative ones from the smallest
        const uint32_t place = kWords + (wave + WAVES * __builtin_ctz(left)) * kWave + lane;
        first = count_at(f, place, heavies) ? place : first;
        found = __any(first != 0xFFFFFFFFu);
    }
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
        const uint32_t o = __shfl_xor(first, d);
        first = o < first ? o : first;
    }
    if (lane == 0)
        atomicMin(&f.first, first);
    for (int i = threadIdx.x; i < kGroups; i += kScanThreads) {
        f.mass[i] = 0.0;
        f.count[i] = 0;
    }
    __syncthreads();
    first = f.first;
    if (first == 0xFFFFFFFFu) {  // no logit above -inf
        if (threadIdx.x == 0) {
            a.tokens[row] = -1;
            if (a.logprobs)
                a.logprobs[row] = -__builtin_inff();
        }
        return;
    }
    const float top = value_of(bits_at(first));
    const bool fine = in_range(top, p.per_unit);
    // Each group's number and mass.
    for (int half = 0; half < 2; ++half)
        for (uint32_t left = used; left; left &= left - 1) {
            const uint32_t words = wave + WAVES * __builtin_ctz(left);
            const uint32_t group = half ? kGroups / 2 + words : kGroups / 2 - 1 - words;
            uint32_t count;
            double weight;
            group_at(f, group, heavies, top, p.per_unit, fine, count, weight);
            if (!__any(count != 0))
                continue;
            const uint32_t c = wave_total(count);
            const double m = wave_total((double)count * weight);
            if (lane == kWave - 1) {
                f.count[group] = c;
                f.mass[group] = m;
            }
        }
    __syncthreads();
    static_assert(kGroups == kScanThreads, "a thread a group");
    uint32_t gc = f.count[threadIdx.x];
    double gm = f.mass[threadIdx.x];
    block_sums<kScanThreads>(gc, gm, f.waves);
    f.count[threadIdx.x] = gc;
    f.mass[threadIdx.x] = gm;
    __syncthreads();

    // The searches, by one wave: the group first (how many lie before the crossing),
    // then the value inside it, then which of its elements.
    double kept = 0.0, weight = 0.0;
    if (wave == 0) {
        kept = f.mass[kGroups - 1];
        double limit = kept;
#pragma unroll 1
        for (int query = kTopK; query <= kToken; ++query) {
            double value = 0.0;
            uint32_t last = 0;  // of min-p: the places that pass
            if (query == kTopK) {
                if (p.top_k <= 0 || f.count[kGroups - 1] < (uint32_t)p.top_k)
                    continue;
            } else if (query == kTopP) {
                if (!(p.top_p < 1.0))
                    continue;
                value = p.top_p * limit;
                value = value > 0.5 ? value : 0.5;  // the first element has mass 1
            } else if (query == kMinP) {
                if (!(p.log_min_p > -1e299))
                    continue;
                for (uint32_t step = kGroups; step; step /= kWave) {  // of 1024, then 16, then 1 place
                    const uint32_t place = last + step * lane;
                    const bool passes = place < 2 * kWords &&
                        (place <= first || below_top(value_of(bits_at(place)), top, p.per_unit, fine) / kPerUnit >= p.log_min_p);
                    const uint64_t no = ~__ballot(passes);
                    const uint32_t n = no ? __builtin_ctzll(no) : kWave;
                    last += step * (n - 1);  // place 0 passes
                    if (step == 16) {
                        const uint32_t at = last + lane;
                        const uint64_t out = ~__ballot(lane < 16 && at < 2 * kWords &&
                            (at <= first || below_top(value_of(bits_at(at)), top, p.per_unit, fine) / kPerUnit >= p.log_min_p));
                        last += __builtin_ctzll(out) - 1;
                        break;
                    }
                }
            } else {
                value = p.u * kept;
            }
            uint32_t group = 0;
            if (query == kMinP) {
                group = last / kWave;
            } else {
                auto below = [&](uint32_t at) {
                    return query == kTopK   ? f.count[at] < (uint32_t)p.top_k
                           : query == kTopP ? f.mass[at] < value
                                            : f.mass[at] <= value;
                };
                constexpr uint32_t BLOCKS = kGroups / kWave;  // of 64 groups, first by their ends
                uint32_t block = __popcll(__ballot(lane < (int)BLOCKS && below(lane % BLOCKS * kWave + kWave - 1)));
                block = block < BLOCKS ? block : BLOCKS - 1;
                group = block * kWave + __popcll(__ballot(below(block * kWave + lane)));
                group = group < (uint32_t)kGroups ? group : kGroups - 1;
                // past a border by a rounding: back to a group with elements
                while (group && f.count[group] == f.count[group - 1])
                    --group;
            }
            const uint32_t count_before = group ? f.count[group - 1] : 0u;
            const double mass_before = group ? f.mass[group - 1] : 0.0;
            uint32_t count;
            double w;
            group_at(f, group, heavies, top, p.per_unit, fine, count, w);
            const double own = (double)count * w, upto = wave_sums(own);
            const uint32_t number = wave_sums(count);
            const uint64_t some = __ballot(count != 0);
            if (query == kMinP) {
                const double m = mass_before + of_lane(upto, last % kWave);
                kept = m < kept ? m : kept;
                continue;
            }
            const uint64_t over = some & __ballot(query == kTopK   ? count_before + number >= (uint32_t)p.top_k
                                                  : query == kTopP ? mass_before + upto >= value
                                                                   : mass_before + upto > value);
            // rounding at the group's end: its last value
            const int who = over ? __builtin_ctzll(over) : some ? 63 - __builtin_clzll(some) : 0;
            const double before = mass_before + (upto - own), left = (value - before) / w;
            uint32_t nth = 0;
            if (query == kTopK) {
                nth = p.top_k - (count_before + number - count);
            } else {
                const double n = query == kTopP ? ceil(left) : floor(left) + 1.0;
                nth = n < 1.0 ? 1u : n < (double)count ? (uint32_t)n : count;
            }
            const double m = of_lane(before + (double)nth * w, who);
            if (query == kToken) {
                weight = of_lane(w, who);
                const uint32_t j = of_lane(nth, who);
                if (lane == 0) {
                    f.bits = bits_at(group * kWave + who);
                    f.nth = j;
                }
            } else {
                kept = m < kept ? m : kept;
                if (query == kTopK)
                    limit = kept;
            }
        }
    }
    __syncthreads();
    find_nth(f, x, a.V);
    __syncthreads();
    if (threadIdx.x == 0) {
        a.tokens[row] = (int32_t)f.index;
        if (a.logprobs) {
            const double lp = log(weight / kept);
            a.logprobs[row] = lp < 0.0 ? (float)lp : 0.f;
        }
    }
}

// Slices of a row: enough workgroups to fill the GPU (64 rows of 131072 logits:
// 32 us a call; with half as many 40, with twice as many 34), none with fewer
// than 8 elements for each thread (one such row: 20.5 us; with 4 or 16 elements
// 21.5, for the slices have to be joined by each workgroup of the gather).
int slices_of(int M, int V)
{
    const int least = (V + kMaxSlice - 1) / kMaxSlice;
    int s = device_cu_count() / M;
    const int most = V / (8 * kScanThreads);
    s = s < most ? s : most;
    s = s < kMaxSlices ? s : kMaxSlices;
    return s > least ? s : least > 1 ? least : 1;
}

// Whether rows of bf16 logits are taken by their values: its fixed 15 us and one
// CU for a row are too much for short rows, and for few long ones (us by bins and
// by values, with top-k 50 and top-p 0.9, then without top-k):
//   8 x 500       15 : 16,  13 : 16       1 x 131072    21 : 27,  27 : 25
//   8 x 4000      15 : 17,  17 : 16       32 x 131072   25 : 31,  37 : 30
//   8 x 16000     19 : 18,  23 : 17       64 x 131072   30 : 33,  46 : 32
//   32 x 65000    23 : 23,  29 : 23       128 x 131072  39 : 33,  75 : 32
//   256 x 32000   26 : 21,  31 : 20       256 x 131072  48 : 36,  59 : 35
//   64 x 152064   32 : 34,  44 : 32       64 x 196607   34 : 39,  45 : 37
//   128 x 152064  43 : 34,  65 : 32       128 x 196607  49 : 39,  73 : 37
//   256 x 152064  59 : 37,  79 : 36       256 x 196607  70 : 43,  99 : 42
// The longest row is the counts': with one element more, three logits could have more
// than 65535 each.
constexpr int kMostByValues = 3 * 65536 - 1;
bool by_values(int M, int V) { return V >= 1 << 13 && V <= (M >= 64 ? kMostByValues : 1 << 16); }

template <typename T>
hipError_t launch(const SampleArgs &a, hipStream_t stream)
{
    if constexpr (__is_same(T, __bf16)) {
        if (by_values(a.M, a.V)) {
            sample_values_kernel<<<dim3(a.M), kScanThreads, 0, stream>>>(a);
            return hipGetLastError();
        }
    }
    const int S = slices_of(a.M, a.V);
    sample_histogram_kernel<T><<<dim3(S, a.M), kScanThreads, 0, stream>>>(a, S);
    hipError_t e = hipGetLastError();
    const bool gather = S > 1 && a.V > kGatherMin;
    if (e == hipSuccess && gather) {
        sample_gather_kernel<T><<<dim3(S, a.M), kThreads, 0, stream>>>(a, S);
        e = hipGetLastError();
    }
    if (e != hipSuccess)
        return e;
    if (gather)
        sample_finish_kernel<T, kThreads><<<dim3(a.M), kThreads, 0, stream>>>(a, S);
    else
        sample_finish_kernel<T, kScanThreads><<<dim3(a.M), kScanThreads, 0, stream>>>(a, S);
    return hipGetLastError();
}

}  // namespace

bool sample_size_supported(int V) { return V >= 1 && V <= kMaxSlice * kMaxSlices; }

size_t sample_workspace_bytes(int M, int V) { return (size_t)M * row_bytes(slices_of(M, V)); }

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
