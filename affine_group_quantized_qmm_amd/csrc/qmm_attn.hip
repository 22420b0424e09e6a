// Attention of the newest rows of each sequence over the paged key-value
// cache, with an optional sliding window and sink tokens.
//
// For one sequence and one kv head the query rows that read the same keys are
// the (row, head of the group) pairs; they are the 16-wide columns of the
// matrix instructions, up to NT tiles of 16 in a workgroup. A wave holds 16
// tokens at a time:
//
//   S^T = K Q^T      16x16x32 MFMA, tokens by columns
//   p = 2^(s - m)    a lane holds 4 tokens of one column; the columns' running
//                    maxima m are in LDS and are raised (and the accumulators
//                    rescaled) only when some score passes them by kRaise, which
//                    bounds p and leaves nothing to exchange in most turns
//   O^T += V^T P^T   over 32 tokens: the 4 + 4 that one lane group wrote of two
//                    waves; V^T comes out of LDS with transposing reads
//
// P is kept as the sum of two 16-bit numbers (a rounding and its remainder):
// rounding p once to bf16 would add an error as large as the output's own
// rounding, and the matrix units have room for the second product. In fp16 all of
// p is scaled by 2^15 (kLift), for the numbers below 2^-14 lose bits there: a
// first token with a large score and a small value, and a long tail of small
// weights that makes up the output, are ordinary.
//
// A tile is 16 tokens for each wave of a workgroup. Each wave multiplies its own
// 16 tokens with all columns; the columns' maxima meet in LDS, P and V lie there
// for the second product, which the waves split along the head (D / waves
// values each), so that the accumulators of up to 96 columns fit and a piece of
// the cache is read once by one workgroup. K and V come in whole rows with the
// nontemporal hint, straight past the barriers into registers: the next tile's
// are in flight while this one is computed.
//
// What bounds it is that stream: 6.6 TB/s of 1.61 GB (64 sequences of 4k to 8k
// tokens, 8 heads of 128) where a kernel that does nothing but read such pages
// reaches 6.75; a fixed 10 to 12 us (the plan, the first pages, the join)
// where there is little to read.
//
// How a call is laid out: (sequence, kv head) pairs are too few or too unequal
// to fill the GPU as they are, and their lengths are known on the GPU alone.
// Every workgroup sums up the lengths and finds its own equal share (see
// "How they are dealt out" below); a second kernel joins pieces of one item.
#include "qmm_device.hpp"
#include "qmm_kernels.hpp"
#include "qmm_step.hpp"

namespace qmm {
namespace {

constexpr int kJoinThreads = 1024;
// Waves of a workgroup; each has 16 tokens of a tile. A turn of a wave is some
// thousand instructions one after the other, which only another wave of the
// same SIMD can hide. Heads of 192 and 256, whose registers and LDS leave room
// for one workgroup on a CU, take two waves a SIMD (131071 tokens of 4 heads of
// 256: 92 us against 98 with four waves; 8 sequences of 8 rows 41 against 60);
// narrower ones get them from a second workgroup (64 sequences, 8 heads of 128:
// 250 us with two of four waves, 252 with one of eight; 32 sequences of 1000
// tokens 27.9 against 31.4, 256 of 600 85 against 111).
// So do the most columns (6 tiles of heads of 128), whose accumulators would
// spill with four.
constexpr int waves_of(int D, int NT) { return D >= 192 || (D == 128 && NT == 6) ? 8 : 4; }
constexpr int tile_of(int D, int NT) { return 16 * waves_of(D, NT); }
constexpr uint32_t kNoRow = 0xFFFFFFFFu;   // token without a row in the cache

typedef float float2_t __attribute__((ext_vector_type(2)));
typedef short short4_t __attribute__((ext_vector_type(4)));

// A type's matrix instructions and how its weights are scaled: p = 2^(s - m +
// kLift), where a score may pass the running maximum m by kRaise (both log2);
// kUnlift is 2^-kLift.
template <typename T>
struct Elem;
template <>
struct Elem<_Float16> {
    typedef _Float16 x8 __attribute__((ext_vector_type(8)));
    typedef _Float16 x4 __attribute__((ext_vector_type(4)));
    static constexpr uint32_t exponent = 0x7C00u;
    // p is at most 2^15.5, below the type's largest, and 2^15 at the maximum: the
    // second part's steps of 2^-24 then hold a weight to 2^-40 of the largest one.
    static constexpr float kLift = 15.0f, kUnlift = 0x1p-15f, kRaise = 0.5f;
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
    static constexpr float kLift = 0.0f, kUnlift = 1.0f, kRaise = 8.0f;  // fp32's range: no floor to keep away from
    static __device__ __forceinline__ float4_t mfma(x8 a, x8 b, float4_t c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};

template <int CTRL>
__device__ __forceinline__ int dpp_or_zero(int v)
{
    return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, true);
}
// Inclusive sums over the lanes of a wave: within rows of 16 by shifts, then
// the rows before.
__device__ __forceinline__ int wave_scan(int v)
{
    v += dpp_or_zero<0x111>(v);  // row_shr:1
    v += dpp_or_zero<0x112>(v);
    v += dpp_or_zero<0x114>(v);
    v += dpp_or_zero<0x118>(v);
    const int r0 = __builtin_amdgcn_readlane(v, 15), r1 = __builtin_amdgcn_readlane(v, 31),
              r2 = __builtin_amdgcn_readlane(v, 47);
    const int row = threadIdx.x % kWave / 16;
    return v + (row > 0 ? r0 : 0) + (row > 1 ? r1 : 0) + (row > 2 ? r2 : 0);
}

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

__device__ __forceinline__ int row_of_column(const AttnArgs &a, int x)
{
    return divide(x, a.group_magic, a.group_shift);
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

template <int TILE>
__device__ __forceinline__ Span span_of(const AttnArgs &a, int begin, int end, int len, int x0, int cols)
{
    Span s;
    const bool sound = begin >= 0 && begin <= end && end <= a.T;
    s.start = sound ? begin : 0;
    s.n = sound ? end - begin : 0;
    const int G = a.G;
    len = len < 0 ? 0 : len;
    s.first_pos = len - s.n;
    s.sink_tiles = s.low = s.count = 0;
    s.pmin = s.pmax = -1;
    if (x0 >= s.n * G)
        return s;
    const int last = x0 + cols < s.n * G ? x0 + cols : s.n * G;
    s.pmin = s.first_pos + row_of_column(a, x0);
    s.pmax = s.first_pos + row_of_column(a, last - 1);
    // tokens past the table have no page
    const int capacity = a.max_pages * a.page_size;
    const int high = s.pmax + 1 < capacity ? s.pmax + 1 : capacity;
    if (high <= 0)
        return s;
    const int high_tile = (high + TILE - 1) / TILE;
    if (a.window > 0) {
        const int first = s.pmin - a.window + 1;
        s.low = first > 0 ? first / TILE : 0;
        s.low = s.low < high_tile ? s.low : high_tile;
        const int sink_tiles = a.sinks / TILE + (a.sinks % TILE != 0);
        s.sink_tiles = sink_tiles < s.low ? sink_tiles : s.low;
    }
    s.count = s.sink_tiles + high_tile - s.low;
    return s;
}

template <int TILE>
__device__ __forceinline__ Span span_of(const AttnArgs &a, int b, int x0, int cols)
{
    return span_of<TILE>(a, a.row_starts[b], a.row_starts[b + 1], a.context_lens[b], x0, cols);
}

// An item is one kv head of one column chunk of one sequence; its tiles are
// at least one, so that rows that see nothing are written too. Items are
// numbered by sequence, chunk and head. How they are dealt out:
//   whole    one workgroup an item; no join.
//   pieces   (few items) each item in equal pieces of at most `size` tiles, one
//            a workgroup, with the smallest size that gives at most as many
//            pieces as workgroups.
//   runs     (about as many items as workgroups) the tiles of all items one after
//            the other, in equal runs: a run may hold the end of one item and
//            the beginning of another, and no workgroup has more than its share
//            whatever the lengths are.
__device__ __forceinline__ int tiles_of(const Span &s) { return s.count > 1 ? s.count : 1; }

// Run w takes `each` tiles, one more for the first `more` runs.
struct Runs {
    int each, more;
};
__device__ __forceinline__ int first_tile(Runs r, int w) { return w * r.each + (w < r.more ? w : r.more); }
__device__ __forceinline__ int owner_of(Runs r, int tile)
{
    const int longer = r.more * (r.each + 1);
    return tile < longer ? (uint32_t)tile / (uint32_t)(r.each + 1)
                         : r.more + (uint32_t)(tile - longer) / (uint32_t)r.each;
}

// A run's partial results: of an item that it begins (but does not finish), and
// of one that it does not begin (its first).
__device__ __forceinline__ int slot_of(int w, bool begins) { return 2 * w + (begins ? 1 : 0); }

// What a barrier has to order here is LDS only: loads of the next tile stay in
// flight across it.
__device__ __forceinline__ void lds_barrier()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

template <typename T, int D, int NT>
__global__ __launch_bounds__(waves_of(D, NT) * kWave, 2) void attn_kernel(const AttnArgs a)
{
    using E = Elem<T>;
    using x8 = typename E::x8;
    using x4 = typename E::x4;
    constexpr int kWaves = waves_of(D, NT), kTile = tile_of(D, NT);
    static_assert(kTile <= kAttnMostTile, "the host's limit on token numbers");
    constexpr int KS = D / 32;                  // contraction steps of K Q^T; loads of a lane for K and for V
    constexpr int DT = D / 16;                  // output tiles along the head
    constexpr int DW = (DT + kWaves - 1) / kWaves;  // of one wave: tiles wave, wave + kWaves, ...
    constexpr int U = D / 8;                    // 16-byte units of a cache row
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
    __shared__ u32x4 bad_tokens[kWaves / 4];  // a word for each wave; after the last tile whether its sums are not all finite
    __shared__ uint32_t rows_lds[kTile];

    const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
    const int c = lane / 16, n = lane % 16;
    const int G = a.G;
    constexpr int kColumns = 16 * NT;

    // Where the run starts: (sequence, chunk, head, tile), and its length.
    int b, chunk, h, tile = 0, w = 0, left, item_unit = 0, here = 1;
    int run_begin, run_end, run_len;  // of sequence b
    Runs runs{1, 0};
    if (a.whole) {
        // One item a workgroup; the chunks of a head are 8 apart, that is on one
        // XCD, behind one L2.
        const int grp = blockIdx.x / (8 * a.chunks), rem = blockIdx.x % (8 * a.chunks);
        chunk = rem / 8;
        const int item = grp * 8 + rem % 8;
        h = item % a.Hkv;
        b = item / a.Hkv;
        if (b >= a.B)
            return;
        run_begin = a.row_starts[b];
        run_end = a.row_starts[b + 1];
        run_len = a.context_lens[b];
        const Span s = span_of<kTile>(a, run_begin, run_end, run_len, chunk * kColumns, kColumns);
        if (chunk * kColumns >= s.n * G)
            return;
        left = tiles_of(s);
    } else {
        w = blockIdx.x;
        // Sequences are shared out to the lanes in order; the waves do the same.
        // The host has checked that the sum of tiles has 31 bits. Up to 64
        // sequences of one chunk stay in the lanes' registers.
        const bool small = a.B <= kWave && a.chunks == 1;
        const int each = (a.B + kWave - 1) / kWave;
        const int b0 = lane * each, b1 = b0 + each < a.B ? b0 + each : a.B;
        int lane_begin = 0, lane_end = 0, lane_len = 0, lane_tiles = 0;
        if (__builtin_expect(small, 1)) {
            if (lane < a.B) {
                lane_begin = a.row_starts[lane];
                lane_end = a.row_starts[lane + 1];
                lane_len = a.context_lens[lane];
            }
            const Span s = span_of<kTile>(a, lane_begin, lane_end, lane_len, 0, kColumns);
            lane_tiles = s.n > 0 ? tiles_of(s) : 0;
        }
        // Tiles of this lane's items, or pieces of `size` tiles.
        auto sum_of = [&](int size) {
            int sum = 0;
            if (__builtin_expect(small, 1))
                sum = size == 1 ? lane_tiles : (uint32_t)(lane_tiles + size - 1) / (uint32_t)size;
            else
                for (int i = b0; i < b1; ++i)
                    for (int k = 0; k < a.chunks; ++k) {
                        const Span s = span_of<kTile>(a, i, k * kColumns, kColumns);
                        if (k * kColumns >= s.n * G)
                            break;
                        sum += size == 1 ? tiles_of(s) : (uint32_t)(tiles_of(s) + size - 1) / (uint32_t)size;
                    }
            return sum * a.Hkv;
        };
        int mine = sum_of(1), upto = wave_scan(mine), size = 1, from = w;
        int units = __builtin_amdgcn_readlane(upto, kWave - 1);  // runs are dealt in tiles, pieces one by one
        left = 1;
        if (a.pieces) {
            size = (units + a.groups - 1) / (uint32_t)a.groups;
            for (;;) {  // ends: with a size of the longest item every item is one piece
                size = size > 1 ? size : 1;
                mine = sum_of(size);
                upto = wave_scan(mine);
                units = __builtin_amdgcn_readlane(upto, kWave - 1);
                if (units <= a.groups)
                    break;
                size += (size + 7) / 8;
            }
            if (w >= units)
                return;
        } else {
            const uint32_t groups = units < a.groups ? units : a.groups;
            if (w >= (int)groups)
                return;
            runs.each = units / groups;
            runs.more = units - runs.each * groups;
            from = first_tile(runs, w);
            left = first_tile(runs, w + 1) - from;
        }
        // The lane whose share holds the run's first unit, then the item in it.
        const int in = __builtin_ctzll(__ballot(from < upto));
        int at = __builtin_amdgcn_readlane(upto - mine, in);
        b = in * each;
        chunk = 0;
        int count;
        if (__builtin_expect(small, 1)) {
            count = __builtin_amdgcn_readlane(lane_tiles, in);
            here = (uint32_t)(count + size - 1) / (uint32_t)size;
            run_begin = __builtin_amdgcn_readlane(lane_begin, in);
            run_end = __builtin_amdgcn_readlane(lane_end, in);
            run_len = __builtin_amdgcn_readlane(lane_len, in);
        } else {
            for (;;) {
                if (b >= a.B)
                    return;  // not reached: the sums above found the unit
                const Span s = span_of<kTile>(a, b, chunk * kColumns, kColumns);
                if (chunk == a.chunks || chunk * kColumns >= s.n * G) {
                    chunk = 0;
                    ++b;
                    continue;
                }
                count = tiles_of(s);
                here = (uint32_t)(count + size - 1) / (uint32_t)size;
                if (from < at + here * a.Hkv)
                    break;
                at += here * a.Hkv;
                ++chunk;
            }
            run_begin = a.row_starts[b];
            run_end = a.row_starts[b + 1];
            run_len = a.context_lens[b];
        }
        h = (uint32_t)(from - at) / (uint32_t)here;
        item_unit = at + h * here;
        tile = from - item_unit;
        if (a.pieces) {  // piece `tile` of `here` equal ones
            const int q = (uint32_t)count / (uint32_t)here, more = count - q * here, piece = tile;
            tile = first_tile(Runs{q, more}, piece);
            left = first_tile(Runs{q, more}, piece + 1) - tile;
        }
    }
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
    auto at = [&](const void *cache, uint32_t row) {
        return static_cast<const T *>(cache) + (uint64_t)(row == kNoRow ? 0u : row) * D;
    };

    // Whole rows of the wave's 16 tokens; to LDS in the same order.
    u32x4 kr[KS], vr[KS];
    // They are read once: the nontemporal hint gives 6.75 TB/s of such rows
    // instead of 6.05.
    auto load = [&](u32x4 (&r)[KS], const void *cache, Rows rows) {
        if (one_page) {
            const u32x4 *p = reinterpret_cast<const u32x4 *>(static_cast<const T *>(cache) + (uint64_t)rows.first * D);
#pragma unroll
            for (int i = 0; i < KS; ++i)
                r[i] = __builtin_nontemporal_load(p + (i * kWave + lane));
        } else {
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                const int unit = i * kWave + lane;
                const u32x4 *p = reinterpret_cast<const u32x4 *>(at(cache, __shfl(rows.mine, unit / U)) + unit % U * 8);
                r[i] = __builtin_nontemporal_load(p);
            }
        }
    };
    auto store = [&](const u32x4 (&r)[KS]) {
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            const int unit = i * kWave + lane;
            *reinterpret_cast<u32x4 *>(kv_lds + (16 * wave + unit / U) * kPitch + unit % U * 16) = r[i];
        }
    };

    int page = look_up(begin);
    // Queries of column tile t, step q: column n's values 32 q + 8 c ...
    auto query_at = [&](int t, int q) {
        const int x = x0 + t * 16 + n;
        const bool live = x < span.n * G;
        const int r = live ? row_of_column(a, x) : 0, g = live ? x - r * G : 0;
        return static_cast<const T *>(a.q) + (span.start + r) * a.q_stride + (int64_t)(h * G + g) * D + q * 32 + c * 8;
    };
    x8 qf[kQueriesInLds ? 1 : NT][KS];
    if constexpr (kQueriesInLds) {
        constexpr int P = (NT * KS + kWaves - 1) / kWaves;
        u32x4 v[P];
#pragma unroll
        for (int i = 0; i < P; ++i) {  // all in flight before the first is stored
            const int piece = i * kWaves + wave < NT * KS ? i * kWaves + wave : wave;
            v[i] = *reinterpret_cast<const u32x4 *>(query_at(piece / KS, piece % KS));
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
    load(kr, a.k_cache, rows);
    page = look_up(begin + 1);
    load(vr, a.v_cache, rows);
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

        store(kr);
        rows = rows_of(page, x + 1);
        load(kr, a.k_cache, rows);
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
            s[t] *= a.scale_log2;
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
        if (partial) {
            typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
            u16x2 largest{0, 0};  // of the magnitudes' bits: an exponent of all ones is above every finite one
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                const bool there = present >> ((i * kWave + lane) / U) & 1u;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    vr[i][k] = there ? vr[i][k] : 0u;
                    largest = __builtin_elementwise_max(largest, __builtin_bit_cast(u16x2, vr[i][k] & 0x7FFF7FFFu));
                }
            }
            if (__builtin_expect(__any(largest.x >= E::exponent || largest.y >= E::exponent), 0)) {
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                    bool differs = false;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t f = finite_halves<T>(vr[i][k]);
                        differs |= f != vr[i][k];
                        vr[i][k] = f;
                    }
                    bad |= differs ? 1u << (i * kWave + lane) / U : 0u;
                }
#pragma unroll
                for (int d = 1; d < kWave; d *= 2)
                    bad |= __shfl_xor(bad, d);
            }
        }
        store(vr);
        if (lane < 16) {
            rows_lds[16 * wave + lane] = row_now;
            reinterpret_cast<uint32_t *>(bad_tokens)[wave] = bad;
        }
        load(vr, a.v_cache, rows);
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
                const T *vp = at(a.v_cache, rows_lds[tok]) + 4 * c;
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
                        const u32x2 raw = *reinterpret_cast<const u32x2 *>(vp + dt * 16);
                        const x4 v4 = __builtin_bit_cast(x4, raw);
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
            T *to = static_cast<T *>(a.out) + at_row * D + wave * 16 + 4 * c;
#pragma unroll
            for (int d = 0; d < DW; ++d) {
                x4 y;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    y[i] = (T)(acc[t][d][i] * inv);  // the output's one rounding
                if (DT % kWaves == 0 || wave + kWaves * d < DT)
                    *reinterpret_cast<x4 *>(to + kWaves * d * 16) = y;
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

// Join of the pieces of an item that several runs share:
// sum_z acc_z 2^(m_z - M) over sum_z l_z 2^(m_z - M) for each column. A
// workgroup's threads are D/4 values wide and the rest of them share the
// pieces, so that their loads are in flight together.
template <typename T, int D>
__global__ __launch_bounds__(kJoinThreads) void attn_join_kernel(const AttnArgs a, int columns)
{
    using E = Elem<T>;
    constexpr int W = D / 4;                // threads of one piece's values
    const int P = blockDim.x / W;           // pieces read at a time
    __shared__ float4_t part[kJoinThreads / W][W];
    __shared__ float sums[kJoinThreads / W];
    const int G = a.G;
    const int h = blockIdx.x % a.Hkv, k = blockIdx.x / a.Hkv % a.chunks, b = blockIdx.x / a.Hkv / a.chunks;
    const int x0 = k * columns;
    const int begin = a.row_starts[b], end = a.row_starts[b + 1];
    const int2 join = a.joins[blockIdx.x];  // of items that exist
    const int rows = begin >= 0 && begin <= end && end <= a.T ? end - begin : 0;
    const int live = x0 + columns < rows * G ? columns : rows * G - x0;
    if (live <= 0 || join.x == join.y)
        return;
    const int pieces = join.y - join.x + 1;
    auto slot = [&](int z) { return (int64_t)slot_of(join.x + z, z == 0) * columns; };
    for (int col = blockIdx.y; col < live; col += gridDim.y) {
        const int x = x0 + col, r = row_of_column(a, x);
        const int64_t at_row = (int64_t)(begin + r) * a.Hq + h * G + (x - r * G);
        const float2_t *ml = reinterpret_cast<const float2_t *>(a.part_ml) + col;
        float top = -__builtin_inff();
        for (int z = threadIdx.x % kWave; z < pieces; z += kWave)
            top = fmaxf(top, ml[slot(z)].x);
#pragma unroll
        for (int d = 1; d < kWave; d *= 2)
            top = fmaxf(top, __shfl_xor(top, d));
        const int d4 = threadIdx.x % W, first = threadIdx.x / W;
        float4_t o{0.f, 0.f, 0.f, 0.f};
        float total = 0.f;
        if (first < P) {
#pragma unroll 8
            for (int z = first; z < pieces; z += P) {
                const float2_t v = ml[slot(z)];
                const float f = top == -__builtin_inff() ? 1.f : __builtin_amdgcn_exp2f(v.x - top);
                total += v.y * f;
                o += *reinterpret_cast<const float4_t *>(a.part_acc + (slot(z) + col) * D + d4 * 4) * f;
            }
            part[first][d4] = o;
            if (d4 == 0)
                sums[first] = total;
        }
        __syncthreads();
        if (first == 0) {
            for (int p = 1; p < P && p < pieces; ++p) {
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
                                             : (top + __builtin_amdgcn_logf(total * E::kUnlift)) * 0.69314718055994530942f;
        }
        __syncthreads();
    }
}

template <typename T, int D, int NT>
hipError_t launch(const AttnArgs &a, const AttnPlan &p, hipStream_t stream)
{
    attn_kernel<T, D, NT><<<dim3((uint32_t)p.blocks), waves_of(D, NT) * kWave, 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.whole)
        return e;
    attn_join_kernel<T, D><<<dim3((uint32_t)p.items, p.join_columns), p.join_threads, 0, stream>>>(a, 16 * NT);
    return hipGetLastError();
}

// Column tiles that a workgroup takes at most: with more, the accumulators
// (D / 16 registers a tile) and the queries in LDS would leave room for one
// workgroup on a CU instead of two.
constexpr int most_col_tiles(int D) { return D == 64 || D == 128 ? 6 : D == 96 ? 4 : 3; }

template <typename T, int D>
hipError_t launch_cols(const AttnArgs &a, const AttnPlan &p, hipStream_t stream)
{
    switch (p.col_tiles) {
    case 1: return launch<T, D, 1>(a, p, stream);
    case 2: return launch<T, D, 2>(a, p, stream);
    case 3: return launch<T, D, 3>(a, p, stream);
    case 4:
        if constexpr (most_col_tiles(D) >= 4)
            return launch<T, D, 4>(a, p, stream);
        return hipErrorInvalidValue;
    case 6:
        if constexpr (most_col_tiles(D) >= 6)
            return launch<T, D, 6>(a, p, stream);
        return hipErrorInvalidValue;
    default: return hipErrorInvalidValue;
    }
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

AttnPlan attn_plan(int B, int Hq, int Hkv, int D, int max_rows, int max_context, int window, int sinks,
                   int page_size, int max_pages)
{
    AttnPlan p;
    const int64_t columns = (int64_t)max_rows * (Hq / Hkv);
    const int64_t col_tiles = (columns + 15) / 16;
    const int64_t chunks = (col_tiles + most_col_tiles(D) - 1) / most_col_tiles(D);
    p.col_tiles = (int)((col_tiles + chunks - 1) / chunks);
    p.col_tiles += p.col_tiles == 5;
    p.chunks = (int)((col_tiles + p.col_tiles - 1) / p.col_tiles);
    const int kTile = tile_of(D, p.col_tiles);
    int64_t visible = max_context;
    if (window > 0 && (int64_t)window + max_rows + sinks + 2 * kTile < visible)
        visible = (int64_t)window + max_rows + sinks + 2 * kTile;
    const int64_t tiles = visible > kTile ? (visible + kTile - 1) / kTile : 1;
    const int64_t items = (int64_t)B * Hkv * p.chunks;
    // Workgroups of a full GPU: as many as keep 48 to 64 KB of K and V in flight
    // on a CU (a workgroup has a tile of each). More only add plans, partial
    // results and joins: 131071 tokens take 96 us with one on a CU and 111 with
    // two, heads of 64 with a window 24.3, 23.8 and 24.3 with two, three and four.
    const int per_cu = waves_of(D, p.col_tiles) == 8 ? 1 : D >= 96 ? 2 : 3;
    const int64_t full = (int64_t)per_cu * device_cu_count();
    // The runs count tiles in 31 bits, up to the block table's end.
    const int64_t most_tiles = items * ((int64_t)max_pages * page_size / kTile + 1);
    // Whole items where a join costs more than it saves: up to 256 tokens (24
    // heads over 4 of 128, 150 to 190 tokens: 7.5 us against 10.7; 500 tokens of
    // heads of 256 18 against 12 in pieces), up to 1024 with two items or more
    // for each workgroup (256 sequences, 8 heads of 128, 600 tokens: 84 us against
    // 93; 4000 tokens 515 against 499), and where they are eight (512 sequences of
    // 600 tokens: 159 against 176).
    p.whole = visible <= 256 || items >= (visible <= 1024 ? 2 : 8) * full || most_tiles > INT32_MAX;
    const int64_t groups = items * tiles < full ? items * tiles : full;
    p.groups = (int)groups;
    p.items = items;
    p.blocks = p.whole ? ((int64_t)B * Hkv + 7) / 8 * 8 * p.chunks : p.groups;
    // Pieces where items have four or more (16 sequences of 4000 tokens, 8 heads
    // of 128: 42 us against 45 in runs), runs where few of unequal length share
    // the GPU (32 sequences: 74 against 80 in pieces).
    // Workgroups of the join for each item: one for each column while the items
    // have many pieces, else one for a few columns; and their threads (one
    // sequence of 4000 tokens: 13.3 us with 1024, 13.8 with 256; 64 sequences of
    // 600 36 with 1024, 31 with 256).
    const int live = (int)(columns < 16 * p.col_tiles ? columns : 16 * p.col_tiles);
    p.pieces = items * 4 <= groups;
    p.join_columns = p.pieces ? live : (live + 3) / 4;
    p.join_threads = items * 16 <= groups ? kJoinThreads : 256;
    p.join_bytes = p.whole ? 0 : (items * sizeof(int2) + 15) / 16 * 16;
    p.workspace_bytes =
        p.whole ? 0 : p.join_bytes + (size_t)p.groups * 2 * 16 * p.col_tiles * (D + 2) * sizeof(float);
    return p;
}

hipError_t launch_paged_attention(AttnArgs a, const AttnPlan &p, int D, bool bf16, void *workspace, hipStream_t stream)
{
    a.chunks = p.chunks;
    a.groups = p.groups;
    a.whole = p.whole;
    a.pieces = p.pieces;
    a.one_page = a.page_size % 16 == 0;
    a.G = a.Hq / a.Hkv;
    const MagicDiv g = magic_div(a.G);
    a.group_magic = g.magic;
    a.group_shift = g.shift;
    if (!p.whole) {
        const size_t columns = (size_t)p.groups * 2 * 16 * p.col_tiles;
        a.joins = static_cast<int2 *>(workspace);
        a.part_acc = reinterpret_cast<float *>(static_cast<char *>(workspace) + p.join_bytes);
        a.part_ml = a.part_acc + columns * D;
    }
    return bf16 ? launch_dim<__bf16>(a, p, D, stream) : launch_dim<_Float16>(a, p, D, stream);
}

}  // namespace qmm
