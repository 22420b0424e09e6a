// Attention of the newest rows of each sequence over a paged cache of 8- or 4-bit
// codes: the same mathematics and layout of a call as over 16-bit rows
// (qmm_attn.hip). A cache row comes in as codes with the (scale, bias) words of
// its groups, and its numbers, fp16, are formed between the registers that a
// tile was loaded to and LDS: one byte permutation, one packed subtraction and one packed
// multiply-add for two values. From there on the products are those of fp16.
#pragma once

#include "qmm_attn.hpp"
#include "qmm_quant.hpp"

namespace qmm {
namespace {

// Four outputs in their type.
__device__ __forceinline__ u32x2 rounded4(const AttnArgs &a, float4_t v)
{
    typedef _Float16 h4 __attribute__((ext_vector_type(4)));
    typedef __bf16 b4 __attribute__((ext_vector_type(4)));
    if (a.io_bf16)
        return __builtin_bit_cast(u32x2, b4{(__bf16)v.x, (__bf16)v.y, (__bf16)v.z, (__bf16)v.w});
    return __builtin_bit_cast(u32x2, h4{(_Float16)v.x, (_Float16)v.y, (_Float16)v.z, (_Float16)v.w});
}

template <int BITS, int D, int NT>
__global__ __launch_bounds__(waves_of(D, NT) * kWave, 2) void attn_codes_kernel(const AttnArgs a)
{
    using T = _Float16;
    using E = Elem<T>;
    using x8 = typename E::x8;
    using x4 = typename E::x4;
    constexpr int kWaves = waves_of(D, NT), kTile = tile_of(D, NT);
    static_assert(kTile <= kAttnMostTile, "the host's limit on token numbers");
    constexpr int KS = D / 32;                  // contraction steps of K Q^T; loads of a lane for K and for V
    constexpr int DT = D / 16;                  // output tiles along the head
    constexpr int DW = (DT + kWaves - 1) / kWaves;  // of one wave: tiles wave, wave + kWaves, ...
    // A lane's share of 16 rows of a cache, as it is loaded: units of codes, each
    // within one group, with their (scale, bias) words.
    constexpr int kCodes = D % 64 == 0 ? 16 : 8;
    typedef uint32_t Unit __attribute__((ext_vector_type(kCodes * BITS / 32)));
    constexpr int U = D / kCodes;               // units of a cache row
    constexpr int kLoads = U / 4;               // units of a lane
    constexpr int kParts = kCodes / 8;          // 16 bytes in LDS for each 8 values
    // LDS row of V: 32 bytes past the data shift consecutive rows by 8 banks,
    // so that the 8 rows that a transposing read touches at a time do not collide.
    constexpr int kPitch = 2 * D + 32;
    constexpr int kColumn = kTile + 8;          // elements of a column of P: 16 bytes of padding for the same reason
    // The queries' operands stay in registers (4 a step and column tile) while
    // these are few, else in LDS, where the waves share them.
    constexpr bool kQueriesInLds = NT * KS > 8;
    // Each wave's 16 rows hold its K tile up to the first barrier of a turn, then V.
    __shared__ __align__(16) char kv_lds[kTile * kPitch];
    __shared__ __align__(16) T p_hi[NT * 16 * kColumn], p_lo[NT * 16 * kColumn];
    __shared__ u32x4 q_lds[kQueriesInLds ? NT * KS * kWave : 1];
    __shared__ float col_max[NT * 16], col_sum[kWaves][NT * 16];
    __shared__ uint32_t query_top[kQueriesInLds ? NT * 16 : 1];  // largest magnitude of a column's queries, as bits
    __shared__ u32x4 bad_tokens[kWaves / 4];  // a word for each wave; after the last tile whether its sums are not all finite
    __shared__ uint32_t rows_lds[kTile];

    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    const int c = lane / 16, n = lane % 16;
    const int G = a.G;
    constexpr int kColumns = 16 * NT;

    Start at_first;
    if (!find_start<kTile, kColumns>(a, at_first))
        return;
    int b = at_first.b, chunk = at_first.chunk, h = at_first.h, tile = at_first.tile, left = at_first.left;
    int item_unit = at_first.item_unit;
    int run_begin = at_first.run_begin, run_end = at_first.run_end, run_len = at_first.run_len;  // of sequence b
    const int w = at_first.w, here = at_first.here;
    const Runs runs = at_first.runs;
    const int tr_offset = (4 * c + n / 4) * kPitch + n % 4 * 8;

    // Infinities and NaN in V of a tile that every row sees whole go through both
    // products as they are, where infinity times a remainder of 0 or below is not
    // infinity. They leave no output of the piece finite: then it is computed once
    // more with every tile treated as partly visible (`careful`), which takes
    // them one by one. Nothing is looked for in the tiles themselves.
    bool careful = false;
    for (;; lds_barrier()) {  // the items of the run
    const int x0 = chunk * kColumns;
    const Span span = span_of<kTile>(a, run_begin, run_end, run_len, x0, kColumns);
    const int count = tiles_of(span);
    const int begin = tile, end = left < count - begin ? begin + left : count;
    if (!a.whole && begin == 0 && threadIdx.x == 0)  // who holds the pieces of the item that begins here
        a.joins[(b * a.chunks + chunk) * a.Hkv + h] =
            int2{w, a.pieces ? w + here - 1 : owner_of(runs, item_unit + count - 1)};

    const int32_t *table = a.block_table + (int64_t)b * a.max_pages;
    const int capacity = a.max_pages * a.page_size;
    const int last_token = span.pmax < capacity ? span.pmax : capacity - 1;
    auto first_of = [&](int x) {
        return (x < span.sink_tiles ? x : span.low + x - span.sink_tiles) * kTile;
    };
    // Token (16 * wave + n) of a tile: whether some row of the workgroup sees
    // it. The others are not read: their pages may be gone, their values anything.
    auto seen_by_any = [&](int j) {
        return j <= last_token && (a.window == 0 || j > span.pmin - a.window || j < a.sinks);
    };
    // Loads are issued without branches around them (past the end they go to the
    // cache's first row): where paths with and without a load meet, the compiler
    // has to wait for all that are in flight.
    // Pages of whole multiples of 16 tokens: the wave's 16 tokens are in one
    // page, their rows one after the other.
    const bool one_page = a.one_page;
    auto look_up = [&](int x) -> int {
        const int j0 = first_of(x) + 16 * wave, j = one_page ? j0 : j0 + n;
        const bool seen = x < end && (one_page ? j0 <= last_token && (a.window == 0 || j0 + 15 > span.pmin - a.window ||
                                                                     j0 < a.sinks)
                                               : seen_by_any(j));
        const int page = table[seen ? divide(j, a.page_magic, a.page_shift) : 0u];
        return seen ? page : -1;
    };
    // The cache row of token 16 * wave + n, and where the wave's rows are one
    // after the other the first of them.
    struct Rows {
        uint32_t mine, first;
    };
    auto rows_of = [&](int page, int x) -> Rows {
        const int j0 = first_of(x) + 16 * wave;
        Rows r{kNoRow, 0u};
        if (one_page) {
            const uint32_t p = __builtin_amdgcn_readfirstlane(page);
            const uint32_t off = j0 - divide(j0, a.page_magic, a.page_shift) * a.page_size;
            if (p < (uint32_t)a.num_pages) {
                r.first = (p * a.Hkv + h) * a.page_size + off;
                r.mine = seen_by_any(j0 + n) ? r.first + n : kNoRow;
            }
        } else if ((uint32_t)page < (uint32_t)a.num_pages) {
            const uint32_t off = j0 + n - divide(j0 + n, a.page_magic, a.page_shift) * a.page_size;
            r.mine = ((uint32_t)page * a.Hkv + h) * a.page_size + off;
        }
        return r;
    };
    // Rows in the cache are below 2^32, byte offsets are not: 64-bit products.
    constexpr int kRowBytes = D * BITS / 8;
    auto at = [&](const void *cache, uint32_t row) {
        return static_cast<const char *>(cache) + (uint64_t)(row == kNoRow ? 0u : row) * kRowBytes;
    };
    auto words_at = [&](const uint32_t *sb, uint32_t row) {
        return sb + ((uint64_t)(row == kNoRow ? 0u : row) << a.words_shift) * (D % 96 == 0 ? 3 : 1);
    };

    // Whole rows of the wave's 16 tokens; to LDS in the same order.
    Unit kr[kLoads], vr[kLoads];
    uint32_t kw[kLoads], vw[kLoads];
    // They are read once: the nontemporal hint gives 6.75 TB/s of such rows
    // instead of 6.05.
    auto load = [&](Unit (&r)[kLoads], uint32_t (&w)[kLoads], const void *cache, const uint32_t *sb, Rows rows) {
        if (one_page) {
            const Unit *p = reinterpret_cast<const Unit *>(static_cast<const char *>(cache) + (uint64_t)rows.first * kRowBytes);
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                r[i] = __builtin_nontemporal_load(p + (i * kWave + lane));
            const uint32_t *s = words_at(sb, rows.first);
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                w[i] = s[(uint32_t)(i * kWave + lane) * kCodes >> a.code_shift];
        } else {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int unit = i * kWave + lane;
                const uint32_t row = __shfl(rows.mine, unit / U);
                const Unit *p = reinterpret_cast<const Unit *>(at(cache, row)) + unit % U;
                r[i] = __builtin_nontemporal_load(p);
                w[i] = words_at(sb, row)[(uint32_t)(unit % U) * kCodes >> a.code_shift];
            }
        }
    };
    // The 16 bytes of LDS that hold 8 values: unit i of the lane, part j.
    auto place = [&](int i, int j) {
        const int unit = i * kWave + lane;
        return reinterpret_cast<u32x4 *>(kv_lds + (16 * wave + unit / U) * kPitch + (unit % U * kParts + j) * 16);
    };
    auto numbers = [&](const Unit (&r)[kLoads], const uint32_t (&w)[kLoads], int i, int j) -> u32x4 {
        if constexpr (BITS == 8)
            return eight_numbers(r[i][2 * j], r[i][2 * j + 1], w[i]);
        else
            return eight_numbers(r[i][j], w[i]);
    };
    auto store = [&](const Unit (&r)[kLoads], const uint32_t (&w)[kLoads]) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
#pragma unroll
            for (int j = 0; j < kParts; ++j)
                *place(i, j) = numbers(r, w, i, j);
    };

    int page = look_up(begin);
    // Queries of column tile t, step q: column n's values 32 q + 8 c ...
    auto query_at = [&](int t, int q) {
        const int x = x0 + t * 16 + n;
        const bool live = x < span.n * G;
        const int r = live ? row_of_column(a, x) : 0, g = live ? x - r * G : 0;
        return static_cast<const uint16_t *>(a.q) + (span.start + r) * a.q_stride + (int64_t)(h * G + g) * D + q * 32 + c * 8;
    };
    // bf16 queries of a quantized cache become fp16: a column's are multiplied by
    // the power of two that brings the largest to 2^14 .. 2^15, which keeps their 8
    // bits down to 2^-28 of it, and its scores are divided by it.
    const bool convert = a.io_bf16;
    auto top_of = [&](u32x4 v) {  // largest magnitude of 8 bf16 values, as an fp32's bits
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t lo = v[k] << 16 & 0x7FFF0000u, hi = v[k] & 0x7FFF0000u;
            top = lo > top ? lo : top;
            top = hi > top ? hi : top;
        }
        return top;
    };
    auto lift_of = [&](uint32_t top) {  // exponent of that power; columns of zeros, or with infinities or NaN, stay
        return top == 0 || top >= 0x7F800000u ? 0 : 15 - __builtin_amdgcn_frexp_expf(__builtin_bit_cast(float, top));
    };
    auto lifted = [&](u32x4 v, int lift) {
        half8_t h;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            h[k] = (_Float16)__builtin_amdgcn_ldexpf(bf16_bits_to_float(v[k / 2] >> 16 * (k % 2) & 0xFFFFu), lift);
        return __builtin_bit_cast(u32x4, h);
    };
    float score_scale[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
        score_scale[t] = a.scale_log2;
    x8 qf[kQueriesInLds ? 1 : NT][KS];
    if constexpr (kQueriesInLds) {
        constexpr int P = (NT * KS + kWaves - 1) / kWaves;
        u32x4 v[P];
#pragma unroll
        for (int i = 0; i < P; ++i) {  // all in flight before the first is stored
            const int piece = i * kWaves + wave < NT * KS ? i * kWaves + wave : wave;
            v[i] = *reinterpret_cast<const u32x4 *>(query_at(piece / KS, piece % KS));
        }
        if (convert) {
            if (threadIdx.x < NT * 16)
                query_top[threadIdx.x] = 0;
            lds_barrier();
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int piece = i * kWaves + wave < NT * KS ? i * kWaves + wave : wave;
                __hip_atomic_fetch_max(&query_top[piece / KS * 16 + n], top_of(v[i]), __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_WORKGROUP);
            }
            lds_barrier();
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int piece = i * kWaves + wave < NT * KS ? i * kWaves + wave : wave;
                v[i] = lifted(v[i], lift_of(query_top[piece / KS * 16 + n]));
            }
#pragma unroll
            for (int t = 0; t < NT; ++t)
                score_scale[t] = __builtin_amdgcn_ldexpf(a.scale_log2, -lift_of(query_top[t * 16 + n]));
        }
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int piece = i * kWaves + wave < NT * KS ? i * kWaves + wave : wave;
            q_lds[piece * kWave + lane] = v[i];
        }
    } else {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int q = 0; q < KS; ++q)
                qf[t][q] = *reinterpret_cast<const x8 *>(query_at(t, q));
        if (convert) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                uint32_t top = 0;
#pragma unroll
                for (int q = 0; q < KS; ++q) {
                    const uint32_t x = top_of(__builtin_bit_cast(u32x4, qf[t][q]));
                    top = x > top ? x : top;
                }
#pragma unroll
                for (int d = 16; d < kWave; d *= 2) {
                    const uint32_t x = __shfl_xor(top, d);
                    top = x > top ? x : top;
                }
                const int lift = lift_of(top);
#pragma unroll
                for (int q = 0; q < KS; ++q)
                    qf[t][q] = __builtin_bit_cast(x8, lifted(__builtin_bit_cast(u32x4, qf[t][q]), lift));
                score_scale[t] = __builtin_amdgcn_ldexpf(a.scale_log2, -lift);
            }
        }
    }
    int pos[NT];  // positions of this lane's columns (-1: no such column)
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int x = x0 + t * 16 + n;
        pos[t] = x < span.n * G ? span.first_pos + row_of_column(a, x) : -1;
    }
    if (threadIdx.x < NT * 16)
        col_max[threadIdx.x] = -__builtin_inff();
    Rows rows = rows_of(page, begin);
    load(kr, kw, a.k_cache, a.k_sb, rows);
    page = look_up(begin + 1);
    load(vr, vw, a.v_cache, a.v_sb, rows);
    lds_barrier();

    float4_t acc[NT][DW];
    float m[NT], l[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        m[t] = -__builtin_inff();
        l[t] = 0.f;
#pragma unroll
        for (int d = 0; d < DW; ++d)
            acc[t][d] = float4_t{0.f, 0.f, 0.f, 0.f};
    }
    for (int x = begin; x < end; ++x) {
        const int j0 = first_of(x) + 16 * wave;  // the wave's first token
        const uint32_t present = (uint32_t)__ballot(rows.mine != kNoRow) & 0xFFFFu;
        const uint32_t row_now = rows.mine;

        store(kr, kw);
        rows = rows_of(page, x + 1);
        load(kr, kw, a.k_cache, a.k_sb, rows);
        page = look_up(x + 2);
        wave_lds_sync();
        float4_t s[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t)
            s[t] = float4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < KS; ++q) {
            const x8 kf = *reinterpret_cast<const x8 *>(kv_lds + (16 * wave + n) * kPitch + q * 64 + c * 16);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                x8 qv;
                if constexpr (kQueriesInLds)
                    qv = __builtin_bit_cast(x8, q_lds[(t * KS + q) * kWave + lane]);
                else
                    qv = qf[t][q];
                s[t] = E::mfma(kf, qv, s[t]);
            }
            if (NT * KS >= 16 && q % 2 == 1)  // not all of the operands in registers at once
                __builtin_amdgcn_sched_barrier(0);
        }

        // Tiles that not every row sees whole: scores that a row does not see
        // are -infinity.
        const bool partial = careful || present != 0xFFFFu || j0 + 15 > span.pmin ||
                             (a.window > 0 && j0 <= span.pmax - a.window && j0 + 16 > a.sinks);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            s[t] *= score_scale[t];
            if (partial) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = j0 + 4 * c + i;
                    const bool sees = j <= pos[t] && (present >> (4 * c + i) & 1u) &&
                                      (a.window == 0 || j > pos[t] - a.window || j < a.sinks);
                    s[t][i] = sees ? s[t][i] : -__builtin_inff();
                }
            }
            const float top = fmaxf(fmaxf(s[t][0], s[t][1]), fmaxf(s[t][2], s[t][3]));
            if (top > m[t] + E::kRaise)
                __hip_atomic_fetch_max(&col_max[t * 16 + n], top, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        }
        lds_barrier();  // the columns' maxima are in

#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const float up = col_max[t * 16 + n];
            if (__any(up > m[t])) {
                const float f = up > m[t] ? __builtin_amdgcn_exp2f(m[t] - up) : 1.f;
                m[t] = up;
                l[t] *= f;
#pragma unroll
                for (int d = 0; d < DW; ++d)
                    acc[t][d] *= f;
            }
            const float base = m[t] == -__builtin_inff() ? 0.f : m[t] - E::kLift;
            x4 hi, lo;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float p = __builtin_amdgcn_exp2f(s[t][i] - base);
                l[t] += p;
                hi[i] = (T)p;
                lo[i] = (T)(p - (float)hi[i]);
            }
            const int to = (t * 16 + n) * kColumn + 16 * wave + 4 * c;
            *reinterpret_cast<x4 *>(&p_hi[to]) = hi;
            *reinterpret_cast<x4 *>(&p_lo[to]) = lo;
        }
        // V to LDS. In partly visible tiles, values that could poison a product
        // with p = 0 are kept out: tokens without a row are cleared, non-finite
        // values are cleared here and added back below for the rows that see them.
        uint32_t bad = 0;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            u32x4 v[kParts];
#pragma unroll
            for (int j = 0; j < kParts; ++j)
                v[j] = numbers(vr, vw, i, j);
            if (partial) {
                typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
                const int token = (i * kWave + lane) / U;
                const bool there = present >> token & 1u;
                u16x2 largest{0, 0};  // of the magnitudes' bits: an exponent of all ones is above every finite one
#pragma unroll
                for (int k = 0; k < 4 * kParts; ++k) {
                    v[k / 4][k % 4] = there ? v[k / 4][k % 4] : 0u;
                    largest = __builtin_elementwise_max(largest, __builtin_bit_cast(u16x2, v[k / 4][k % 4] & 0x7FFF7FFFu));
                }
                const bool odd = largest.x >= E::exponent || largest.y >= E::exponent;
                if (__builtin_expect(__any(odd), 0)) {
#pragma unroll
                    for (int k = 0; k < 4 * kParts; ++k)
                        v[k / 4][k % 4] = finite_halves<T>(v[k / 4][k % 4]);
                    uint32_t here_bad = odd ? 1u << token : 0u;
#pragma unroll
                    for (int d = 1; d < kWave; d *= 2)
                        here_bad |= __shfl_xor(here_bad, d);
                    bad |= here_bad;
                }
            }
#pragma unroll
            for (int j = 0; j < kParts; ++j)
                *place(i, j) = v[j];
            if constexpr (NT >= 3)  // not all of the numbers in registers at once
                __builtin_amdgcn_sched_barrier(0);
        }
        if (lane < 16) {
            rows_lds[16 * wave + lane] = row_now;
            reinterpret_cast<uint32_t *>(bad_tokens)[wave] = bad;
        }
        load(vr, vw, a.v_cache, a.v_sb, rows);
        lds_barrier();  // P and V are in

        // Step q takes tokens 4c .. 4c+3 of waves 2q and 2q+1.
#pragma unroll
        for (int q = 0; q < kWaves / 2; ++q) {
            x8 vt[DW];
#pragma unroll
            for (int d = 0; d < DW; ++d) {
                const int dt = wave + kWaves * d;
                if (DT % kWaves != 0 && dt >= DT)
                    break;
                typedef __attribute__((address_space(3))) short4_t lds4;
                const char *p = kv_lds + tr_offset + 32 * q * kPitch + dt * 32;
                const short4_t v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)p);
                const short4_t v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)(p + 16 * kPitch));
                vt[d] = __builtin_bit_cast(x8, __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7));
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int from = (t * 16 + n) * kColumn + 32 * q + 4 * c;
                const x8 hi = __builtin_shufflevector(*reinterpret_cast<const x4 *>(&p_hi[from]),
                                                      *reinterpret_cast<const x4 *>(&p_hi[from + 16]), 0, 1, 2, 3, 4, 5, 6, 7);
                const x8 lo = __builtin_shufflevector(*reinterpret_cast<const x4 *>(&p_lo[from]),
                                                      *reinterpret_cast<const x4 *>(&p_lo[from + 16]), 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
                for (int d = 0; d < DW; ++d) {
                    if (DT % kWaves != 0 && wave + kWaves * d >= DT)
                        break;
                    acc[t][d] = E::mfma(vt[d], hi, acc[t][d]);
                    acc[t][d] = E::mfma(vt[d], lo, acc[t][d]);
                }
                if constexpr (NT >= 3)  // not all of the operands in registers at once
                    __builtin_amdgcn_sched_barrier(0);
            }
        }

        u32x4 any_bad = bad_tokens[0];
        if constexpr (kWaves == 8)
            any_bad |= bad_tokens[1];
        const uint32_t some = __builtin_amdgcn_readfirstlane(any_bad.x | any_bad.y | any_bad.z | any_bad.w);
        for (int v = 0; __builtin_expect(some != 0, 0) && v < kWaves; ++v) {
            uint32_t left = __builtin_amdgcn_readfirstlane(reinterpret_cast<const uint32_t *>(bad_tokens)[v]);
            while (left) {  // a token of a partly visible tile holds infinities or NaN
                const int tok = 16 * v + __builtin_ctz(left);
                left &= left - 1;
                const int j = first_of(x) + tok;
                const char *vp = at(a.v_cache, rows_lds[tok]);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const int from = (t * 16 + n) * kColumn + tok;
                    // a weight that was too small for its type is not zero
                    const float p = (float)p_hi[from] + (float)p_lo[from] + 0x1p-126f;
                    const bool sees = j <= pos[t] && (a.window == 0 || j > pos[t] - a.window || j < a.sinks);
#pragma unroll
                    for (int d = 0; d < DW; ++d) {
                        const int dt = wave + kWaves * d;
                        if (DT % kWaves != 0 && dt >= DT)
                            break;
                        const int first = dt * 16 + 4 * c;  // of 4 codes
                        uint32_t bytes;
                        if constexpr (BITS == 8) {
                            bytes = *reinterpret_cast<const uint32_t *>(vp + first);
                        } else {
                            const uint32_t w = *reinterpret_cast<const uint16_t *>(vp + first / 2);
                            bytes = (w & 15) | (w & 0xF0) << 4 | (w & 0xF00) << 8 | (w & 0xF000) << 12;
                        }
                        const half2_t sb = __builtin_bit_cast(half2_t, words_at(a.v_sb, rows_lds[tok])[first >> a.code_shift]);
                        const x4 v4 = __builtin_bit_cast(x4, code_numbers(bytes, half2_t{sb.x, sb.x}, half2_t{sb.y, sb.y}));
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float f = (float)v4[i];
                            const bool odd = !(__builtin_fabsf(f) < __builtin_inff());
                            acc[t][d][i] += odd && sees ? p * f : 0.f;
                        }
                        __builtin_amdgcn_sched_barrier(0);  // rare: few registers rather than loads in flight
                    }
                }
            }
        }
        lds_barrier();  // every wave is past V and P
    }

    // Sums of the columns over the lanes and waves that share them.
    float zero = 0.f;  // NaN if some sum is not finite
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        l[t] += __shfl_xor(l[t], 16);
        l[t] += __shfl_xor(l[t], 32);
        if (c == 0)
            col_sum[wave][t * 16 + n] = l[t];
#pragma unroll
        for (int d = 0; d < DW; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                zero = __builtin_fmaf(acc[t][d][i], 0.f, zero);
    }
    const uint32_t odd = __any(zero != 0.f);
    if (lane == 0)
        reinterpret_cast<uint32_t *>(bad_tokens)[wave] = odd;
    lds_barrier();
    u32x4 any_odd = bad_tokens[0];
    if constexpr (kWaves == 8)
        any_odd |= bad_tokens[1];
    if (!careful && __builtin_amdgcn_readfirstlane(any_odd.x | any_odd.y | any_odd.z | any_odd.w)) {
        careful = true;
        continue;
    }
    careful = false;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int x = x0 + t * 16 + n;
        if (x >= span.n * G)
            continue;
        float total = 0.f;
#pragma unroll
        for (int v = 0; v < kWaves; ++v)
            total += col_sum[v][t * 16 + n];
        const int r = row_of_column(a, x);
        const int64_t at_row = (int64_t)(span.start + r) * a.Hq + h * G + (x - r * G);
        const bool first = wave == 0 && c == 0;
        if (begin == 0 && end == count) {
            const float inv = total == 0.f ? 0.f : 1.f / total;
            uint16_t *to = static_cast<uint16_t *>(a.out) + at_row * D + wave * 16 + 4 * c;
#pragma unroll
            for (int d = 0; d < DW; ++d) {
                const u32x2 y = rounded4(a, acc[t][d] * inv);  // the output's one rounding
                if (DT % kWaves == 0 || wave + kWaves * d < DT)
                    *reinterpret_cast<u32x2 *>(to + kWaves * d * 16) = y;
            }
            if (first && a.lse)
                a.lse[at_row] = total == 0.f ? -__builtin_inff()
                                             : (m[t] + __builtin_amdgcn_logf(total * E::kUnlift)) * 0.69314718055994530942f;
        } else {
            const int64_t part = (int64_t)slot_of(w, begin == 0) * kColumns + t * 16 + n;
            float *to = a.part_acc + part * D + wave * 16 + 4 * c;
#pragma unroll
            for (int d = 0; d < DW; ++d)
                if (DT % kWaves == 0 || wave + kWaves * d < DT)
                    *reinterpret_cast<float4_t *>(to + kWaves * d * 16) = acc[t][d];
            if (first)
                *reinterpret_cast<float2_t *>(a.part_ml + part * 2) = float2_t{m[t], total};
        }
    }

    left -= end - begin;
    if (left <= 0)
        return;
    tile = 0;
    item_unit += count;
    if (++h == a.Hkv) {  // the next item that exists (there is one: the run is not done)
        h = 0;
        ++chunk;
        while (chunk == a.chunks || chunk * kColumns >= span_of<kTile>(a, run_begin, run_end, run_len, 0, kColumns).n * G) {
            chunk = 0;
            if (++b >= a.B)
                return;
            run_begin = a.row_starts[b];
            run_end = a.row_starts[b + 1];
            run_len = a.context_lens[b];
        }
    }
    }
}

template <int BITS, int D, int NT>
hipError_t launch(const AttnArgs &a, const AttnPlan &p, hipStream_t stream)
{
    attn_codes_kernel<BITS, D, NT><<<dim3((uint32_t)p.blocks), waves_of(D, NT) * kWave, 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.whole)
        return e;
    const dim3 joins((uint32_t)p.items, p.join_columns);
    if (a.io_bf16)
        attn_join_kernel<Elem<_Float16>, __bf16, D><<<joins, p.join_threads, 0, stream>>>(a, 16 * NT);
    else
        attn_join_kernel<Elem<_Float16>, _Float16, D><<<joins, p.join_threads, 0, stream>>>(a, 16 * NT);
    return hipGetLastError();
}

template <int BITS, int D>
hipError_t launch_cols(const AttnArgs &a, const AttnPlan &p, hipStream_t stream)
{
    switch (p.col_tiles) {
    case 1: return launch<BITS, D, 1>(a, p, stream);
    case 2: return launch<BITS, D, 2>(a, p, stream);
    case 3: return launch<BITS, D, 3>(a, p, stream);
    case 4:
        if constexpr (most_col_tiles(D, true) >= 4)
            return launch<BITS, D, 4>(a, p, stream);
        return hipErrorInvalidValue;
    case 6:
        if constexpr (most_col_tiles(D, true) >= 6)
            return launch<BITS, D, 6>(a, p, stream);
        return hipErrorInvalidValue;
    default: return hipErrorInvalidValue;
    }
}

template <int BITS>
hipError_t launch_dim(const AttnArgs &a, const AttnPlan &p, int D, hipStream_t stream)
{
    switch (D) {
    case 64: return launch_cols<BITS, 64>(a, p, stream);
    case 96: return launch_cols<BITS, 96>(a, p, stream);
    case 128: return launch_cols<BITS, 128>(a, p, stream);
    case 192: return launch_cols<BITS, 192>(a, p, stream);
    case 256: return launch_cols<BITS, 256>(a, p, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace
}  // namespace qmm
