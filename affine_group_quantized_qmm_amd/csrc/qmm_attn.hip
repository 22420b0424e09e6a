// Attention of the newest rows of each sequence over the paged key-value
// cache, with an optional sliding window and sink tokens.
//
// For one sequence and one kv head the query rows that read the same keys are
// the (row, head of the group) pairs; they are the 16-wide columns of the
// matrix instructions, up to NT tiles of 16 in a workgroup. A wave walks over
// tiles of 32 tokens:
//
//   S^T = K Q^T      16x16x32 MFMA; K goes from memory straight to the operand
//                    registers (lane = token, 16 bytes of its row)
//   p = 2^(s - m)    a lane holds 8 tokens of one column, so that maximum and
//                    sum stay in the lane; m is raised (and the accumulators
//                    rescaled) only when some score passes it by 2^8, which
//                    bounds p and needs no exchange between lanes per tile
//   O^T += V^T P^T   the 8 tokens that a lane holds after the first product are
//                    the 8 it must supply to the second, so P needs no movement;
//                    V^T comes out of LDS with transposing reads
//
// P is kept as the sum of two 16-bit numbers (a rounding and its remainder):
// rounding p once to bf16 would add an error as large as the output's own
// rounding, and the matrix units have room for the second product.
//
// What bounds it is the stream of K and V: each byte is read once by a
// workgroup, and a wave keeps the whole next tile's K and V loads in flight
// (registers) while it computes. Waves share nothing until the end, where the
// four waves of a workgroup are joined through LDS. When (sequence, kv head)
// pairs are few, the visible length is cut into splits of equal token counts
// whose partials a second kernel joins.
#include "qmm_device.hpp"
#include "qmm_kernels.hpp"
#include "qmm_step.hpp"

namespace qmm {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = kWaves * kWave;
constexpr int kTile = 32;                  // tokens of a tile
constexpr uint32_t kNoRow = 0xFFFFFFFFu;   // token without a row in the cache
constexpr float kRaise = 8.0f;             // a score may pass the running maximum by this (log2)

typedef float float2_t __attribute__((ext_vector_type(2)));
typedef short short4_t __attribute__((ext_vector_type(4)));

template <typename T>
struct Elem;
template <>
struct Elem<_Float16> {
    typedef _Float16 x8 __attribute__((ext_vector_type(8)));
    typedef _Float16 x4 __attribute__((ext_vector_type(4)));
    static constexpr uint32_t exponent = 0x7C00u;
    static __device__ __forceinline__ float4_t mfma(x8 a, x8 b, float4_t c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};
template <>
struct Elem<__bf16> {
    typedef __bf16 x8 __attribute__((ext_vector_type(8)));
    typedef __bf16 x4 __attribute__((ext_vector_type(4)));
    static constexpr uint32_t exponent = 0x7F80u;
    static __device__ __forceinline__ float4_t mfma(x8 a, x8 b, float4_t c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};

// A 32-bit word with its non-finite halves set to zero.
template <typename T>
__device__ __forceinline__ uint32_t finite_halves(uint32_t w)
{
    constexpr uint32_t e = Elem<T>::exponent;
    if ((w & e) == e)
        w &= 0xFFFF0000u;
    if ((w >> 16 & e) == e)
        w &= 0x0000FFFFu;
    return w;
}

// The rows and tiles of (sequence b, column chunk): what a workgroup and the
// join agree on.
struct Span {
    int start, n;        // first row in q, number of rows
    int first_pos;       // position of row 0
    int pmin, pmax;      // positions of the chunk's first and last row
    int sink_tiles, low; // tiles [0, sink_tiles) and from `low` on
    int count;           // tiles in all
};

__device__ __forceinline__ Span span_of(const AttnArgs &a, int b, int x0, int cols)
{
    Span s;
    const int begin = a.row_starts[b], end = a.row_starts[b + 1];
    const bool sound = begin >= 0 && begin <= end && end <= a.T;
    s.start = sound ? begin : 0;
    s.n = sound ? end - begin : 0;
    const int G = a.Hq / a.Hkv;
    const int len = a.context_lens[b] < 0 ? 0 : a.context_lens[b];
    s.first_pos = len - s.n;
    s.sink_tiles = s.low = s.count = 0;
    s.pmin = s.pmax = -1;
    if (x0 >= s.n * G)
        return s;
    const int last = x0 + cols < s.n * G ? x0 + cols : s.n * G;
    s.pmin = s.first_pos + x0 / G;
    s.pmax = s.first_pos + (last - 1) / G;
    // tokens past the table have no page
    const int capacity = a.max_pages * a.page_size;
    const int high = s.pmax + 1 < capacity ? s.pmax + 1 : capacity;
    if (high <= 0)
        return s;
    const int high_tile = (high + kTile - 1) / kTile;
    if (a.window > 0) {
        const int first = s.pmin - a.window + 1;
        s.low = first > 0 ? first / kTile : 0;
        s.low = s.low < high_tile ? s.low : high_tile;
        const int sink_tiles = a.sinks / kTile + (a.sinks % kTile != 0);
        s.sink_tiles = sink_tiles < s.low ? sink_tiles : s.low;
    }
    s.count = s.sink_tiles + high_tile - s.low;
    return s;
}

// Splits that hold tiles of a span (the last split takes whatever is left).
__device__ __forceinline__ int splits_of(const AttnArgs &a, int count)
{
    const int n = (count + a.split_tiles - 1) / a.split_tiles;
    return n < 1 ? 1 : n < a.splits ? n : a.splits;
}

template <typename T, int D, int NT>
__global__ __launch_bounds__(kThreads, (D * NT <= 128 ? 2 : 1)) void attn_kernel(const AttnArgs a)
{
    using E = Elem<T>;
    using x8 = typename E::x8;
    constexpr int KS = D / 32;              // contraction steps of K Q^T
    constexpr int DT = D / 16;              // output tiles along the head
    constexpr int U = D / 8;                // 16-byte units of a cache row
    constexpr int NL = U * kTile / kWave;   // loads of a V tile per lane
    // LDS row of V: 32 bytes past the data shift consecutive rows by 8 banks,
    // so that the 8 rows that a transposing read touches at a time do not collide.
    constexpr int kPitch = 2 * D + 32;
    constexpr int kRegion = kTile * kPitch; // bytes of a wave's V tile
    constexpr int kJoinPitch = D + 4;       // floats of a column in the join
    static_assert(16 * kJoinPitch * 4 <= kRegion, "the join reuses the V tiles");
    static_assert(U * kTile % kWave == 0, "whole loads");
    __shared__ __align__(16) char lds[kWaves * kRegion];
    __shared__ float2_t stats[kWaves][NT * 16];
    // The queries' operands stay in registers (4 a step and column tile) while
    // these are few, else in LDS, where the four waves share them.
    constexpr bool kQueriesInLds = NT * KS > 8;
    __shared__ u32x4 q_lds[kQueriesInLds ? NT * KS * kWave : 1];

    // Block -> (chunk, head, split, sequence): the chunks of one piece of the
    // cache are 8 apart, that is on one XCD, behind one L2.
    const int grp = blockIdx.x / (8 * a.chunks), rem = blockIdx.x % (8 * a.chunks);
    const int chunk = rem / 8;
    int work = grp * 8 + rem % 8;
    if (work >= a.Hkv * a.splits * a.B)
        return;
    const int h = work % a.Hkv;
    work /= a.Hkv;
    const int z = work % a.splits, b = work / a.splits;

    const int G = a.Hq / a.Hkv;
    const int x0 = chunk * 16 * NT;
    const Span span = span_of(a, b, x0, 16 * NT);
    const int pieces = splits_of(a, span.count);
    if (x0 >= span.n * G || z >= pieces)
        return;
    const int begin = z * a.split_tiles;
    const int end = z == pieces - 1 ? span.count : begin + a.split_tiles;

    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    const int c = lane / 16, n = lane % 16;

    // Queries of this lane's columns, and their positions (-1: no such column).
    x8 qf[kQueriesInLds ? 1 : NT][KS];
    int pos[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int x = x0 + t * 16 + n;
        const bool live = x < span.n * G;
        const int r = live ? x / G : 0;
        pos[t] = live ? span.first_pos + r : -1;
        const T *qp = static_cast<const T *>(a.q) + (span.start + r) * a.q_stride +
                      (int64_t)(h * G + (live ? x - r * G : 0)) * D + c * 8;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            if constexpr (!kQueriesInLds)
                qf[t][s] = *reinterpret_cast<const x8 *>(qp + s * 32);
            else if ((t * KS + s) % kWaves == wave)
                q_lds[(t * KS + s) * kWave + lane] = *reinterpret_cast<const u32x4 *>(qp + s * 32);
        }
    }
    if constexpr (kQueriesInLds)
        __syncthreads();

    float4_t acc[NT][DT];
    float m[NT], l[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        m[t] = -__builtin_inff();
        l[t] = 0.f;
#pragma unroll
        for (int d = 0; d < DT; ++d)
            acc[t][d] = float4_t{0.f, 0.f, 0.f, 0.f};
    }

    const int32_t *table = a.block_table + (int64_t)b * a.max_pages;
    const int capacity = a.max_pages * a.page_size;
    const int last_token = span.pmax < capacity ? span.pmax : capacity - 1;
    auto tile_of = [&](int x) { return x < span.sink_tiles ? x : span.low + x - span.sink_tiles; };
    // Token (lane % 32) of a tile: whether some row of the workgroup sees it.
    // The others are not read: their pages may be gone, their values anything.
    auto seen_by_any = [&](int j) {
        return j <= last_token && (a.window == 0 || j > span.pmin - a.window || j < a.sinks);
    };
    auto look_up = [&](int x) -> int {
        if (x >= end)
            return -1;
        const int j = tile_of(x) * kTile + lane % kTile;
        return seen_by_any(j) ? table[divide(j, a.page_magic, a.page_shift)] : -1;
    };
    auto row_of = [&](int page, int x) -> uint32_t {
        if ((uint32_t)page >= (uint32_t)a.num_pages)
            return kNoRow;
        const uint32_t j = tile_of(x) * kTile + lane % kTile;
        const uint32_t off = j - divide(j, a.page_magic, a.page_shift) * a.page_size;
        return ((uint32_t)page * a.Hkv + h) * a.page_size + off;
    };
    // Rows in the cache are below 2^32, byte offsets are not: 64-bit products.
    auto at = [&](const void *cache, uint32_t row) {
        return static_cast<const T *>(cache) + (uint64_t)(row == kNoRow ? 0u : row) * D;
    };

    u32x4 kr[2][KS], vr[NL];
    auto load_k = [&](uint32_t row) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const T *p = at(a.k_cache, __shfl(row, t * 16 + n)) + c * 8;
#pragma unroll
            for (int s = 0; s < KS; ++s)
                kr[t][s] = *reinterpret_cast<const u32x4 *>(p + s * 32);
        }
    };
    auto load_v = [&](uint32_t row) {
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const int unit = i * kWave + lane;
            vr[i] = *reinterpret_cast<const u32x4 *>(at(a.v_cache, __shfl(row, unit / U)) + unit % U * 8);
        }
    };

    char *region = lds + wave * kRegion;
    const char *tr_base = region + (4 * c + n / 4) * kPitch + n % 4 * 8;

    int x = begin + wave;
    int page = look_up(x);
    uint32_t row = row_of(page, x);
    if (x < end) {
        load_k(row);
        page = look_up(x + kWaves);
        load_v(row);
    }
    for (; x < end; x += kWaves) {
        const int j0 = tile_of(x) * kTile;
        const uint32_t present = (uint32_t)__ballot(row != kNoRow);  // bit t: token t has a row
        const uint32_t row_now = row;

        float4_t s[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            s[t][0] = s[t][1] = float4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int q = 0; q < KS; ++q) {
                x8 qv;
                if constexpr (kQueriesInLds)
                    qv = __builtin_bit_cast(x8, q_lds[(t * KS + q) * kWave + lane]);
                else
                    qv = qf[t][q];
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    s[t][k] = E::mfma(__builtin_bit_cast(x8, kr[k][q]), qv, s[t][k]);
            }
        }
        const bool more = x + kWaves < end;
        if (more) {
            row = row_of(page, x + kWaves);
            load_k(row);
            page = look_up(x + 2 * kWaves);
        }

        // V to LDS. In tiles that not every row sees whole, values that could
        // poison a product with p = 0 are kept out: tokens without a row are
        // cleared, non-finite values are cleared here and added back below for
        // the rows that see them.
        const bool partial = present != 0xFFFFFFFFu || j0 + kTile - 1 > span.pmin ||
                             (a.window > 0 && j0 <= span.pmax - a.window && j0 + kTile > a.sinks);
        uint32_t poisoned = 0;  // tokens with non-finite values
        if (partial) {
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                const int token = (i * kWave + lane) / U;
                u32x4 v = vr[i];
                const u32x4 zero{0u, 0u, 0u, 0u};
                if (!(present >> token & 1u))
                    v = zero;
                const u32x4 f{finite_halves<T>(v.x), finite_halves<T>(v.y), finite_halves<T>(v.z),
                              finite_halves<T>(v.w)};
                const bool differs = f.x != v.x || f.y != v.y || f.z != v.z || f.w != v.w;
                poisoned |= differs ? 1u << token : 0u;
                vr[i] = f;
            }
#pragma unroll
            for (int d = 1; d < kWave; d *= 2)
                poisoned |= __shfl_xor(poisoned, d);
        }
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const int unit = i * kWave + lane;
            *reinterpret_cast<u32x4 *>(region + unit / U * kPitch + unit % U * 16) = vr[i];
        }
        if (more)
            load_v(row);

        x8 hi[NT], lo[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float w = s[t][k][i] * a.scale_log2;
                    if (partial) {
                        const int tok = k * 16 + 4 * c + i, j = j0 + tok;
                        const bool sees = j <= pos[t] && (present >> tok & 1u) &&
                                          (a.window == 0 || j > pos[t] - a.window || j < a.sinks);
                        w = sees ? w : -__builtin_inff();
                    }
                    v[4 * k + i] = w;
                }
            const float top = fmaxf(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])),
                                    fmaxf(fmaxf(v[4], v[5]), fmaxf(v[6], v[7])));
            if (__any(top > m[t] + kRaise)) {
                float up = fmaxf(top, __shfl_xor(top, 16));
                up = fmaxf(m[t], fmaxf(up, __shfl_xor(up, 32)));
                const float f = up == -__builtin_inff() ? 1.f : __builtin_amdgcn_exp2f(m[t] - up);
                m[t] = up;
                l[t] *= f;
#pragma unroll
                for (int d = 0; d < DT; ++d)
                    acc[t][d] *= f;
            }
            const float base = m[t] == -__builtin_inff() ? 0.f : m[t];
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float p = __builtin_amdgcn_exp2f(v[i] - base);
                sum += p;
                hi[t][i] = (T)p;
                lo[t][i] = (T)(p - (float)hi[t][i]);
            }
            l[t] += sum;
        }

        wave_lds_sync();
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            typedef __attribute__((address_space(3))) short4_t lds4;
            const short4_t v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(tr_base + d * 32));
            const short4_t v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(tr_base + d * 32 + 16 * kPitch));
            const x8 vt = __builtin_bit_cast(x8, __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                acc[t][d] = E::mfma(vt, hi[t], acc[t][d]);
                acc[t][d] = E::mfma(vt, lo[t], acc[t][d]);
            }
        }
        wave_lds_sync();

        if (poisoned) {  // a token of a partly visible tile holds infinities or NaN
            for (int tok = 0; tok < kTile; ++tok) {
                if (!(poisoned >> tok & 1u))
                    continue;
                const T *vp = at(a.v_cache, __builtin_amdgcn_readlane(row_now, tok)) + 4 * c;
                const int from = tok % 16 / 4 * 16 + n, which = tok / 16 * 4 + tok % 4, j = j0 + tok;
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    float p = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        p = i == which ? (float)hi[t][i] + (float)lo[t][i] : p;
                    p = __shfl(p, from);
                    const bool sees = j <= pos[t] && (a.window == 0 || j > pos[t] - a.window || j < a.sinks);
#pragma unroll
                    for (int d = 0; d < DT; ++d) {
                        const u32x2 raw = *reinterpret_cast<const u32x2 *>(vp + d * 16);
                        const typename E::x4 v4 = __builtin_bit_cast(typename E::x4, raw);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float v = (float)v4[i];
                            const bool odd = !(__builtin_fabsf(v) < __builtin_inff());
                            acc[t][d][i] += odd && sees ? p * v : 0.f;
                        }
                        __builtin_amdgcn_sched_barrier(0);  // rare: few registers rather than loads in flight
                    }
                }
            }
        }
    }

    // Join of the four waves. Every lane of a column has the same m.
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        l[t] += __shfl_xor(l[t], 16);
        l[t] += __shfl_xor(l[t], 32);
        if (c == 0)
            stats[wave][t * 16 + n] = float2_t{m[t], l[t]};
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        float top = -__builtin_inff();
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            top = fmaxf(top, stats[w][t * 16 + n].x);
        const float f = top == -__builtin_inff() ? 1.f : __builtin_amdgcn_exp2f(m[t] - top);
        float *mine = reinterpret_cast<float *>(region) + n * kJoinPitch + 4 * c;
#pragma unroll
        for (int d = 0; d < DT; ++d)
            *reinterpret_cast<float4_t *>(mine + d * 16) = acc[t][d] * f;
        __syncthreads();
        for (int i = threadIdx.x; i < 16 * D / 4; i += kThreads) {
            const int col = i / (D / 4), d = i % (D / 4) * 4;
            const int x = x0 + t * 16 + col;
            if (x >= span.n * G)
                continue;
            float total = 0.f, big = -__builtin_inff();
#pragma unroll
            for (int w = 0; w < kWaves; ++w)
                big = fmaxf(big, stats[w][t * 16 + col].x);
            float4_t o{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const float2_t ml = stats[w][t * 16 + col];
                total += big == -__builtin_inff() ? ml.y : ml.y * __builtin_amdgcn_exp2f(ml.x - big);
                o += *reinterpret_cast<const float4_t *>(reinterpret_cast<const float *>(lds + w * kRegion) +
                                                         col * kJoinPitch + d);
            }
            const int r = x / G;
            const int64_t at_row = (int64_t)(span.start + r) * a.Hq + h * G + (x - r * G);
            if (pieces == 1) {
                const float inv = total == 0.f ? 0.f : 1.f / total;
                typename E::x4 y;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    y[k] = (T)(o[k] * inv);  // the output's one rounding
                *reinterpret_cast<typename E::x4 *>(static_cast<T *>(a.out) + at_row * D + d) = y;
                if (a.lse && d == 0)
                    a.lse[at_row] = total == 0.f ? -__builtin_inff()
                                                 : (big + __builtin_amdgcn_logf(total)) * 0.69314718055994530942f;
            } else {
                *reinterpret_cast<float4_t *>(a.part_acc + (at_row * a.splits + z) * D + d) = o;
                if (d == 0)
                    *reinterpret_cast<float2_t *>(a.part_ml + (at_row * a.splits + z) * 2) = float2_t{big, total};
            }
        }
        __syncthreads();
    }
}

// Join of the splits of one (row, head): sum_z acc_z 2^(m_z - M) over
// sum_z l_z 2^(m_z - M). A workgroup's threads are D/4 values wide and the rest
// of them share the splits, so that their loads are in flight together.
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void attn_join_kernel(const AttnArgs a, int cols)
{
    using E = Elem<T>;
    constexpr int W = D / 4;                // threads of one split's values
    constexpr int P = kThreads / W;         // splits read at a time
    __shared__ float4_t part[P][W];
    __shared__ float sums[P];
    const int head = blockIdx.x % a.Hq, r = blockIdx.x / a.Hq, b = blockIdx.y;
    const int G = a.Hq / a.Hkv;
    const int x = r * G + head % G;
    const Span span = span_of(a, b, x / cols * cols, cols);
    const int pieces = splits_of(a, span.count);
    if (r >= span.n || x >= a.chunks * cols || pieces == 1)
        return;
    const int64_t at_row = (int64_t)(span.start + r) * a.Hq + head;
    const float2_t *ml = reinterpret_cast<const float2_t *>(a.part_ml) + at_row * a.splits;
    float top = -__builtin_inff();
    for (int z = threadIdx.x % kWave; z < pieces; z += kWave)
        top = fmaxf(top, ml[z].x);
#pragma unroll
    for (int d = 1; d < kWave; d *= 2)
        top = fmaxf(top, __shfl_xor(top, d));
    const int d4 = threadIdx.x % W, first = threadIdx.x / W;
    float4_t o{0.f, 0.f, 0.f, 0.f};
    float total = 0.f;
    if (first < P) {
#pragma unroll 4
        for (int z = first; z < pieces; z += P) {
            const float2_t v = ml[z];
            const float f = top == -__builtin_inff() ? 1.f : __builtin_amdgcn_exp2f(v.x - top);
            total += v.y * f;
            o += *reinterpret_cast<const float4_t *>(a.part_acc + (at_row * a.splits + z) * D + d4 * 4) * f;
        }
        part[first][d4] = o;
        if (d4 == 0)
            sums[first] = total;
    }
    __syncthreads();
    if (first == 0) {
        for (int p = 1; p < P; ++p) {
            o += part[p][d4];
            total += sums[p];
        }
        const float inv = total == 0.f ? 0.f : 1.f / total;
        typename E::x4 y;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            y[k] = (T)(o[k] * inv);
        *reinterpret_cast<typename E::x4 *>(static_cast<T *>(a.out) + at_row * D + d4 * 4) = y;
        if (a.lse && d4 == 0)
            a.lse[at_row] = total == 0.f ? -__builtin_inff()
                                         : (top + __builtin_amdgcn_logf(total)) * 0.69314718055994530942f;
    }
}

template <typename T, int D, int NT>
hipError_t launch(const AttnArgs &a, const AttnPlan &p, hipStream_t stream)
{
    const int64_t work = (int64_t)a.Hkv * a.splits * a.B;
    const int64_t blocks = (work + 7) / 8 * 8 * a.chunks;
    attn_kernel<T, D, NT><<<dim3((uint32_t)blocks), kThreads, 0, stream>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1)
        return e;
    const int G = a.Hq / a.Hkv;
    const int rows = a.chunks * 16 * NT / G + 1;  // at least max_rows
    attn_join_kernel<T, D><<<dim3((uint32_t)(a.Hq * rows), a.B), kThreads, 0, stream>>>(a, 16 * NT);
    return hipGetLastError();
}

template <typename T, int D>
hipError_t launch_cols(const AttnArgs &a, const AttnPlan &p, hipStream_t stream)
{
    if (p.col_tiles == 1)
        return launch<T, D, 1>(a, p, stream);
    if (p.col_tiles == 2)
        return launch<T, D, 2>(a, p, stream);
    if constexpr (D <= 128)
        if (p.col_tiles == 4)
            return launch<T, D, 4>(a, p, stream);
    return hipErrorInvalidValue;
}

template <typename T>
hipError_t launch_dim(const AttnArgs &a, const AttnPlan &p, int D, hipStream_t stream)
{
    switch (D) {
    case 64: return launch_cols<T, 64>(a, p, stream);
    case 96: return launch_cols<T, 96>(a, p, stream);
    case 128: return launch_cols<T, 128>(a, p, stream);
    case 192: return launch_cols<T, 192>(a, p, stream);
    case 256: return launch_cols<T, 256>(a, p, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace

bool attn_head_dim_supported(int D) { return D == 64 || D == 96 || D == 128 || D == 192 || D == 256; }

AttnPlan attn_plan(int T, int B, int Hq, int Hkv, int D, int max_rows, int max_context, int window, int sinks)
{
    AttnPlan p;
    const int64_t columns = (int64_t)max_rows * (Hq / Hkv);
    const int most = D <= 128 ? 4 : 2;  // column tiles whose accumulators fit the registers
    p.col_tiles = columns <= 16 ? 1 : columns <= 32 || most == 2 ? 2 : 4;
    p.chunks = (int)((columns + 16 * p.col_tiles - 1) / (16 * p.col_tiles));
    int64_t visible = max_context;
    if (window > 0 && (int64_t)window + max_rows + sinks + 2 * kTile < visible)
        visible = (int64_t)window + max_rows + sinks + 2 * kTile;
    const int64_t tiles = (visible + kTile - 1) / kTile;
    const int64_t base = (int64_t)B * Hkv * p.chunks;
    const int64_t target = 4 * (int64_t)device_cu_count();
    int64_t each = (tiles * base + target - 1) / target;
    each = each < 2 * kWaves ? 2 * kWaves : (each + kWaves - 1) / kWaves * kWaves;
    p.split_tiles = (int)each;
    p.splits = (int)((tiles + each - 1) / each);
    p.splits = p.splits < 1 ? 1 : p.splits;
    p.workspace_bytes = p.splits == 1 ? 0 : (size_t)T * Hq * p.splits * (D + 2) * sizeof(float);
    return p;
}

hipError_t launch_paged_attention(AttnArgs a, const AttnPlan &p, int D, bool bf16, hipStream_t stream)
{
    a.chunks = p.chunks;
    a.splits = p.splits;
    a.split_tiles = p.split_tiles;
    return bf16 ? launch_dim<__bf16>(a, p, D, stream) : launch_dim<_Float16>(a, p, D, stream);
}

}  // namespace qmm
