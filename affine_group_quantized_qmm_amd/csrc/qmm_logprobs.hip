// Log probabilities of given tokens with their ranks, the entropy of each row and
// its most probable tokens, in one read of the logits.
//
//   S = sum_i e^(x_i - m),  T = sum_i e^(x_i - m) (x_i - m),  m = max_i x_i
//   log p_j = x_j - m - log S,   entropy = log S - T / S
//   rank_j = the number of logits in front of x_j (larger, or equal with a lower index)
//
// A workgroup holds a slice of a row in registers. A first walk over the registers gives
// the maxima of 128 groups of elements (a lane of every other wave). Their largest
// is m of the slice, and the n-th largest is a bound that n elements reach, so
// that hardly more than n elements have to be looked at as candidates for the n
// best: 22 for 20 where they lie at random, 89 for 64. The second walk sums, counts,
// and puts the candidates into a list, which is ranked element against element. A row's slices
// meet in a second kernel, which finds the n best of theirs in the same way.
//
// Sums are fp32 within a wave (up to 16 terms a thread, then in pairs) and 64 bits
// from there on, in a fixed order; the list's order is any, but ranks do not
// depend on it. Bound by memory (1021 rows of 151001 fp32: 88 us, 7.0 TB/s,
// and 4.7 us for the second kernel), for bf16 rows with the best wanted by the instructions
// (256 rows of 131072: 29 us, of which 20 are 343 vector instructions a wave, and 5 us), for a
// few rows by two launches (one row of 131072 fp32, 20 best: 7 us and 6 us).
#include "qmm_device.hpp"
#include "qmm_kernels.hpp"
#include "qmm_step.hpp"

namespace qmm {
namespace {

constexpr int kList = 512;  // candidates of a slice; with more, the n best are found one by one

typedef _Float16 half8v __attribute__((ext_vector_type(8)));

// 16 bytes of logits as fp32; NaN counts as -infinity.
template <typename T>
struct Logits;
template <>
struct Logits<float> {
    static constexpr int kVec = 4;
    static constexpr uint32_t kNone = 0xFF800000u;  // -infinity in every place of a word
    static __device__ __forceinline__ void put(u32x4 &v, int i, const float *p) { v[i] = __builtin_bit_cast(uint32_t, *p); }
    static __device__ __forceinline__ float one(const void *p, int64_t i) { return static_cast<const float *>(p)[i]; }
    static __device__ __forceinline__ void unpack(u32x4 v, float (&x)[4])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = __uint_as_float(v[i]);
    }
};
template <>
struct Logits<__bf16> {
    static constexpr int kVec = 8;
    static constexpr uint32_t kNone = 0xFF80FF80u;
    static __device__ __forceinline__ void put(u32x4 &v, int i, const void *p)
    {
        const uint32_t h = *static_cast<const uint16_t *>(p);
        v[i / 2] = i % 2 ? (v[i / 2] & 0xFFFFu) | h << 16 : (v[i / 2] & 0xFFFF0000u) | h;
    }
    static __device__ __forceinline__ float one(const void *p, int64_t i)
    {
        return bf16_bits_to_float(static_cast<const uint16_t *>(p)[i]);
    }
    static __device__ __forceinline__ void unpack(u32x4 v, float (&x)[8])
    {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = __builtin_bit_cast(float, i % 2 ? v[i / 2] & 0xFFFF0000u : v[i / 2] << 16);
    }
};
template <>
struct Logits<_Float16> {
    static constexpr int kVec = 8;
    static constexpr uint32_t kNone = 0xFC00FC00u;
    static __device__ __forceinline__ void put(u32x4 &v, int i, const void *p)
    {
        const uint32_t h = *static_cast<const uint16_t *>(p);
        v[i / 2] = i % 2 ? (v[i / 2] & 0xFFFFu) | h << 16 : (v[i / 2] & 0xFFFF0000u) | h;
    }
    static __device__ __forceinline__ float one(const void *p, int64_t i)
    {
        return half_bits_to_float(static_cast<const uint16_t *>(p)[i]);
    }
    static __device__ __forceinline__ void unpack(u32x4 v, float (&x)[8])
    {
        const half8v h = __builtin_bit_cast(half8v, v);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = (float)h[i];
    }
};

constexpr float kInf = __builtin_inff();

// Numbers in their order as unsigned integers; -0 and +0 are one.
__device__ __forceinline__ uint32_t ordered(float x)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t o)
{
    return __builtin_bit_cast(float, o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
// The fp32 number below x (of -infinity, itself).
__device__ __forceinline__ float below(float x)
{
    if (x == -kInf)
        return x;
    if (x == 0.f)
        return -0x1p-149f;
    const int b = __builtin_bit_cast(int, x);
    return __builtin_bit_cast(float, b > 0 ? b - 1 : b + 1);
}

// What is known of a part of a row.
struct Part {
    float m;        // the largest logit
    uint32_t ahead; // logits in front of the token
    double s, t;    // S and T about m; for m = +infinity the number of such logits, and 0
};
// A part's sums about a larger maximum.
__device__ __forceinline__ void raise(Part &p, float m)
{
    if (p.m == m || p.m == -kInf) {
        p.s = p.m == m ? p.s : 0;
        p.t = p.m == m ? p.t : 0;
        return;
    }
    const double d = (double)p.m - m, f = exp(d);  // below 0, maybe -infinity
    p.t = f > 0 ? f * (p.t + p.s * d) : 0;
    p.s = f > 0 ? p.s * f : 0;
}

constexpr int kGroups = 2 * kWave;

// Largest and smallest of the wave's lanes.
__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
    auto up = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
    v = up(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));   // quad_perm [1,0,3,2]
    v = up(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));   // quad_perm [2,3,0,1]
    v = up(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xF, 0xF, false));  // row_ror:4
    v = up(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xF, 0xF, false));  // row_ror:8
    return up(up(__builtin_amdgcn_readlane(v, 0), __builtin_amdgcn_readlane(v, 16)),
              up(__builtin_amdgcn_readlane(v, 32), __builtin_amdgcn_readlane(v, 48)));
}

// A bound that at least n (up to 128) of the 128 values (two a lane) reach, within
// 2^-10 of their range of the largest such. All of them lie in [lo, hi].
__device__ __forceinline__ uint32_t nth_largest(uint32_t v, uint32_t w, uint32_t lo, uint32_t hi, int n)
{
#pragma unroll 2
    for (int i = 0; i < 10; ++i) {
        const uint32_t mid = lo + (hi - lo + 1) / 2;
        const bool enough = __popcll(__ballot(v >= mid)) + __popcll(__ballot(w >= mid)) >= n;
        lo = enough ? mid : lo;
        hi = enough ? hi : mid - 1;  // (lo <= hi: for mid == lo all reach it)
    }
    return lo;
}

struct Best {
    float x;
    int index;
};
__device__ __forceinline__ bool in_front(Best a, Best b) { return a.x > b.x || (a.x == b.x && a.index < b.index); }

// LDS of a workgroup.
template <int THREADS>
struct Lds {
    uint32_t group_max[kGroups];
    uint32_t bound;
    int listed;
    Best list[kList];
    Best wave_best[THREADS / kWave];
    float s[THREADS / kWave], t[THREADS / kWave];
    uint32_t ahead[THREADS / kWave];
};

// The first n elements in order of those that threads hold, each handed to
// put(rank, best) once; ranks without an element are handed over with index -1.
// collect(add) calls add(has, best) for at least every element that may be among them; element(i, best) gives the i-th of `count` of a thread, false for
// none. Called by all threads, after a barrier that follows the clearing of
// lds.listed.
template <int THREADS, typename Collect, typename Element, typename Put>
__device__ __forceinline__ void first_n(Lds<THREADS> &lds, int n, int count, Collect collect, Element element, Put put)
{
    const int tid = threadIdx.x;
    collect([&](bool has, Best e) {
        if (has && e.x > -kInf) {
            const int at = atomicAdd(&lds.listed, 1);
            if (at < kList)
                lds.list[at] = e;
        }
    });
    __syncthreads();
    const int listed = lds.listed;
    if (listed <= kList) {
        for (int i = tid; i < listed; i += THREADS) {
            const Best mine = lds.list[i];
            int rank = 0;
            for (int j = 0; j < listed; ++j)
                rank += in_front(lds.list[j], mine);
            if (rank < n)
                put(rank, mine);
        }
        for (int r = listed + tid; r < n; r += THREADS)
            put(r, Best{-kInf, -1});
        return;
    }
    // Too many are alike: one after the other, the first behind the last one found.
    Best last{kInf, -1};
    for (int r = 0; r < n; ++r) {
        Best best{-kInf, INT32_MAX};
        for (int i = 0; i < count; ++i) {
            Best e;
            if (element(i, e) && e.x > -kInf && in_front(last, e) && in_front(e, best))
                best = e;
        }
#pragma unroll
        for (int d = 1; d < kWave; d *= 2) {
            const Best other{__shfl_xor(best.x, d), __shfl_xor(best.index, d)};
            if (in_front(other, best))
                best = other;
        }
        __syncthreads();
        if (tid % kWave == 0)
            lds.wave_best[tid / kWave] = best;
        __syncthreads();
        for (int w = 0; w < THREADS / kWave; ++w)
            if (in_front(lds.wave_best[w], best))
                best = lds.wave_best[w];
        if (best.x == -kInf)
            best.index = -1;
        if (tid == 0)
            put(r, best);
        last = best.index < 0 ? Best{-kInf, INT32_MAX} : best;
    }
}

// A row's results.
__device__ __forceinline__ void finish(const LogprobArgs &a, int row, const Part &p, int token, float x)
{
    const double log_s = p.s > 0 ? log(p.s) : 0;
    const bool known = token >= 0 && token < a.V;
    a.logprobs[row] = !known || x == -kInf ? -kInf : p.m == kInf ? (x == kInf ? (float)-log_s : -kInf)
                                                                : (float)((double)x - p.m - log_s);
    if (a.ranks)
        a.ranks[row] = known ? (int)p.ahead : -1;
    if (a.entropy)
        a.entropy[row] = p.s > 0 ? (float)(log_s - p.t / p.s) : 0.f;
}
__device__ __forceinline__ void finish_top(const LogprobArgs &a, int row, const Part &p, int rank, Best e)
{
    const double log_s = p.s > 0 ? log(p.s) : 0;
    const int64_t at = (int64_t)row * a.n + rank;
    a.top_tokens[at] = e.index;
    a.top_logprobs[at] = e.index < 0 ? -kInf : p.m == kInf ? (e.x == kInf ? (float)-log_s : -kInf)
                                                          : (float)((double)e.x - p.m - log_s);
}

template <typename T, int THREADS, int LOADS>
__global__ __launch_bounds__(THREADS) void logprobs_kernel(const LogprobArgs a)
{
    using L = Logits<T>;
    constexpr int kVec = L::kVec, kWaves = THREADS / kWave;
    __shared__ Lds<THREADS> lds;
    const int tid = threadIdx.x, wave = tid / kWave, lane = tid % kWave;
    const int row = blockIdx.x / a.slices, slice = blockIdx.x - row * a.slices;
    const T *logits = static_cast<const T *>(a.logits) + row * a.row_stride;
    // Loads are of whole 16 bytes of memory: where a row begins within one, its
    // element 0 has place `skew` in them.
    const int skew = (int)((a.skew + row * (uint64_t)a.row_stride) % kVec);
    const int token = a.tokens[row];
    const bool known = token >= 0 && token < a.V;
    if (tid < kGroups)
        lds.group_max[tid] = 0;
    if (tid == 0)
        lds.listed = 0;

    float x[LOADS][kVec];
    u32x4 v[LOADS];
    auto first_of = [&](int c) { return ((slice * LOADS + c) * THREADS + tid) * kVec - skew; };
#pragma unroll
    for (int c = 0; c < LOADS; ++c) {
        const int j = first_of(c);
        if (j >= 0 && j + kVec <= a.V) {
            v[c] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(logits + j));
        } else {  // an end of the row: only what is in it
            u32x4 w{L::kNone, L::kNone, L::kNone, L::kNone};
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                if (j + i >= 0 && j + i < a.V)
                    L::put(w, i, logits + (j + i));
            v[c] = w;
        }
    }
    const float x_token = known ? __builtin_fmaxf(L::one(logits, token), -kInf) : -kInf;
    float top[LOADS], most = -kInf;
#pragma unroll
    for (int c = 0; c < LOADS; ++c) {
        L::unpack(v[c], x[c]);
        top[c] = -kInf;  // (a maximum is never NaN)
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            top[c] = __builtin_fmaxf(top[c], x[c][i]);
        most = __builtin_fmaxf(most, top[c]);
    }
    __syncthreads();
    atomicMax(&lds.group_max[tid % kGroups], ordered(most));
    __syncthreads();
    const uint32_t group0 = lds.group_max[lane], group1 = lds.group_max[lane + kWave];
    const uint32_t largest = wave_max(group0 > group1 ? group0 : group1);
    const float m = unordered(largest);
    if (wave == 0 && a.n > 0) {
        const uint32_t least = ~wave_max(~(group0 < group1 ? group0 : group1));
        lds.bound = nth_largest(group0, group1, least, largest, a.n);
    }

    // The second walk.
    float s = 0.f, t = 0.f;
    if (m == kInf) {
#pragma unroll
        for (int c = 0; c < LOADS; ++c)
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                s += x[c][i] == kInf ? 1.f : 0.f;
    } else {
#pragma unroll
        for (int c = 0; c < LOADS; ++c)
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                // (NaN, from NaN or from a difference of infinities, is as far below as any)
                const float d = __builtin_fmaxf(x[c][i] - m, -1e4f);
                const float e = __builtin_amdgcn_exp2f(d * 1.44269504088896340736f);
                s += e;
                t = __builtin_fmaf(e, d, t);
            }
    }
    // Logits in front of the token: larger ones, and up to its own 16 bytes those above
    // the number below it. NaN is above nothing.
    const float thr_behind = known ? x_token : kInf, thr_front = known ? below(x_token) : kInf;
    uint32_t ahead = 0, ahead_lane = 0;
#pragma unroll
    for (int c = 0; c < LOADS; ++c) {
        const int j = first_of(c);
        const float thr = j + kVec <= token ? thr_front : thr_behind;
        if (__any(top[c] > thr)) {  // (seldom for a likely token)
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                ahead += __popcll(__ballot(x[c][i] > thr));
        }
        if (j < token && j + kVec > token) {
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                ahead_lane += j + i >= 0 && j + i < token && x[c][i] == x_token && x_token > -kInf;
        }
        // In front of a token of -infinity (or NaN) are all of lower index.
        if (__builtin_expect(known && x_token == -kInf, 0)) {
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                ahead_lane += j + i >= 0 && j + i < token && !(x[c][i] > -kInf);
        }
    }
    s = wave_sum(s);
    t = wave_sum(t);
    if (__any(ahead_lane != 0)) {
#pragma unroll
        for (int d = 1; d < kWave; d *= 2)
            ahead_lane += __shfl_xor(ahead_lane, d);
    }
    if (lane == 0) {
        lds.s[wave] = s;
        lds.t[wave] = t;
        lds.ahead[wave] = ahead + ahead_lane;
    }
    __syncthreads();
    auto whole = [&] {
        Part p{m, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            p.s += (double)lds.s[w];
            p.t += (double)lds.t[w];
            p.ahead += lds.ahead[w];
        }
        return p;
    };
    if (wave == 0) {
        const Part p = whole();
        if (tid == 0 && a.slices == 1)
            finish(a, row, p, token, x_token);
        else if (tid == 0)
            a.parts[blockIdx.x] = LogprobPart{m, p.ahead, p.s, p.t};
    }
    if (a.n == 0)
        return;
    const float least = unordered(lds.bound);  // (NaN below -infinity: everything reaches it)
    auto collect = [&](auto add) {
#pragma unroll
        for (int c = 0; c < LOADS; ++c) {
            if (!__any(!(top[c] < least)))
                continue;
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                add(!(x[c][i] < least), Best{x[c][i], first_of(c) + i});
        }
    };
    auto element = [&](int i, Best &e) {  // rarely used: any order of registers will do
        float y = -kInf;
        int j = 0;
#pragma unroll
        for (int c = 0; c < LOADS; ++c) {
            if (i / kVec != c)
                continue;
#pragma unroll
            for (int k = 0; k < kVec; ++k)
                y = i % kVec == k ? x[c][k] : y;
            j = first_of(c) + i % kVec;
        }
        e = Best{y, j};
        return true;  // (places outside the row are -infinity)
    };
    first_n<THREADS>(lds, a.n, LOADS * kVec, collect, element, [&](int rank, Best e) {
        if (a.slices == 1)
            finish_top(a, row, whole(), rank, e);
        else
            a.best[(int64_t)blockIdx.x * a.n + rank] = float2{e.x, __builtin_bit_cast(float, e.index)};
    });
}

constexpr int kJoinThreads = 256;
constexpr int kHeld = 6;  // of the slices' best that a thread loads ahead

__global__ __launch_bounds__(kJoinThreads) void logprobs_join_kernel(const LogprobArgs a, int type)
{
    __shared__ Lds<kJoinThreads> lds;
    const int row = blockIdx.x, tid = threadIdx.x, lane = tid % kWave;
    if (tid < kGroups)
        lds.group_max[tid] = 0;
    if (tid == 0)
        lds.listed = 0;
    // All that is needed is on its way before the first of it is used (one row of
    // 131072 fp32 with its 20 best: 6.1 us instead of 8.2).
    const int64_t all = (int64_t)a.slices * a.n;
    const float2 *best = a.best + row * all;
    const float2 none{-kInf, __builtin_bit_cast(float, -1)};
    float2 held[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
        held[i] = none;
        if (i * kJoinThreads + tid < all)
            held[i] = best[i * kJoinThreads + tid];
    }
    const LogprobPart *parts = a.parts + (int64_t)row * a.slices;
    const LogprobPart first = lane < a.slices ? parts[lane] : LogprobPart{-kInf, 0, 0, 0};
    const int token = a.tokens[row];
    float x = -kInf;
    if (token >= 0 && token < a.V) {
        const int64_t at = row * a.row_stride + token;
        x = type == 0 ? Logits<_Float16>::one(a.logits, at) : type == 1 ? Logits<__bf16>::one(a.logits, at)
                                                                         : Logits<float>::one(a.logits, at);
        x = __builtin_fmaxf(x, -kInf);
    }
    // The slices' sums about the row's maximum, lanes pairwise: the same bits in every
    // thread.
    float m = first.m;
    for (int i = lane + kWave; i < a.slices; i += kWave)
        m = __builtin_fmaxf(m, parts[i].m);
#pragma unroll
    for (int d = 1; d < kWave; d *= 2)
        m = __builtin_fmaxf(m, __shfl_xor(m, d));
    Part p{m, 0, 0, 0};
    for (int i = lane; i < a.slices; i += kWave) {  // (every wave sums them all)
        const LogprobPart q = i == lane ? first : parts[i];
        Part about{q.m, q.ahead, q.s, q.t};
        raise(about, m);
        p.s += about.s;
        p.t += about.t;
        p.ahead += q.ahead;
    }
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
        p.s += __shfl_xor(p.s, d);
        p.t += __shfl_xor(p.t, d);
        p.ahead += __shfl_xor(p.ahead, d);
    }
    if (tid == 0)
        finish(a, row, p, token, x);
    if (a.n == 0)
        return;
    auto best_of = [&](float2 v) { return Best{v.x, __builtin_bit_cast(int, v.y)}; };
    auto element = [&](int i, Best &e) {
        const int64_t at = (int64_t)i * kJoinThreads + tid;
        e = best_of(at < all ? best[at] : none);
        return at < all;
    };
    const int count = (int)((all + kJoinThreads - 1) / kJoinThreads);
    auto each = [&](auto use) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            use(best_of(held[i]));
        for (int i = kHeld; i < count; ++i) {
            Best e;
            element(i, e);
            use(e);
        }
    };
    float most = -kInf;
    each([&](Best e) { most = __builtin_fmaxf(most, e.x); });
    __syncthreads();
    atomicMax(&lds.group_max[tid % kGroups], ordered(most));
    __syncthreads();
    const uint32_t group0 = lds.group_max[lane], group1 = lds.group_max[lane + kWave];
    const float least = unordered(nth_largest(group0, group1, ~wave_max(~(group0 < group1 ? group0 : group1)),
                                              wave_max(group0 > group1 ? group0 : group1), a.n));
    auto collect = [&](auto add) { each([&](Best e) { add(!(e.x < least), e); }); };  // (none are -infinity)
    first_n<kJoinThreads>(lds, a.n, count, collect, element, [&](int rank, Best e) { finish_top(a, row, p, rank, e); });
}

// Elements of a slice: 256 threads with 16 each where the rows' slices fill the
// GPU, else 8 each (fp32, 131072 a row: one row with its 20 best 12.9 us with 8, 13.5 with
// 16; 64 rows with 5 best 17.3 and 15.9).
constexpr int kLongThreads = 256, kLongEach = 16, kLong = kLongThreads * kLongEach, kShort = 256 * 8;
int slice_of(int M, int V)
{
    const int64_t slices = (int64_t)M * ((V + kLong - 1) / kLong);
    return slices >= device_cu_count() ? kLong : kShort;
}
template <typename T>
hipError_t launch(const LogprobArgs &a, int slice, int type, hipStream_t stream)
{
    const uint32_t blocks = (uint32_t)a.M * a.slices;
    if (slice == kLong)
        logprobs_kernel<T, kLongThreads, kLongEach / Logits<T>::kVec><<<blocks, kLongThreads, 0, stream>>>(a);
    else
        logprobs_kernel<T, 256, 8 / Logits<T>::kVec><<<blocks, 256, 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.slices == 1)
        return e;
    logprobs_join_kernel<<<(uint32_t)a.M, kJoinThreads, 0, stream>>>(a, type);
    return hipGetLastError();
}

}  // namespace

LogprobPlan logprobs_plan(int M, int V, int n, int skew)
{
    LogprobPlan p;
    p.slices = (V + skew + slice_of(M, V) - 1) / slice_of(M, V);
    p.threads = (int64_t)M * p.slices * (slice_of(M, V) == kLong ? kLongThreads : 256);
    const size_t parts = p.slices == 1 ? 0 : (size_t)M * p.slices;
    p.workspace_bytes = parts * (sizeof(LogprobPart) + sizeof(float2) * n);
    return p;
}

hipError_t launch_logprobs(LogprobArgs a, const LogprobPlan &p, int type, void *workspace, hipStream_t stream)
{
    a.slices = p.slices;
    a.skew = (int)(reinterpret_cast<uintptr_t>(a.logits) % 16) / (type == 2 ? 4 : 2);
    a.parts = static_cast<LogprobPart *>(workspace);
    a.best = reinterpret_cast<float2 *>(a.parts + (p.slices == 1 ? 0 : (size_t)a.M * p.slices));
    const int slice = slice_of(a.M, a.V);
    switch (type) {
    case 0: return launch<_Float16>(a, slice, type, stream);
    case 1: return launch<__bf16>(a, slice, type, stream);
    case 2: return launch<float>(a, slice, type, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace qmm
