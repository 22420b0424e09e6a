// Norms of queries and keys per head, rotation by position, and the append of
// keys and values to the paged cache, in one pass over the projections'
// outputs.
//
//   n_d = x_d * rsqrt(mean_d x_d^2 + eps) * (weight_offset + w_d)
//   pair (i, j): (n_i cos a - n_j sin a, n_j cos a + n_i sin a), a = pos * f_i
//
// Every value is read once and written once with about ten operations in
// between, so the pass is bound by memory, or for a few rows by the launch.
// A head's D values are cut into units of 8 that hold whole rotation pairs:
// in the half-split order unit u < R/8 takes values 4u..4u+3 and
// R/2+4u..R/2+4u+3, so that a pair never leaves its lane and no value crosses
// lanes except in the sum of squares. L = 8, 16 or 32 neighbouring lanes hold
// one head (the smallest that covers D/8 units) and a thread keeps its unit
// while it walks over heads, so that the four angles are computed once per
// row and thread.
//
// 8192 rows (24 query and 4 + 4 key and value heads of 256, fp32 in, bf16 out:
// 403 MB) take 76 us, 5.3 TB/s where a copy of 1 GiB reaches 5.0; 123 rows of 64
// heads of 128 take 3.9 us, one row 3.0, which is a launch with its cold code.
#include "qmm_device.hpp"
#include "qmm_kernels.hpp"
#include "qmm_step.hpp"

namespace qmm {
namespace {

constexpr int kThreads = 256;

typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));

template <typename T>
struct Load4;
template <>
struct Load4<float> {
    static __device__ __forceinline__ float4_t at(const float *p) { return *reinterpret_cast<const float4_t *>(p); }
};
template <>
struct Load4<_Float16> {
    typedef _Float16 h4 __attribute__((ext_vector_type(4)));
    static __device__ __forceinline__ float4_t at(const _Float16 *p)
    {
        const h4 v = *reinterpret_cast<const h4 *>(p);
        return float4_t{(float)v.x, (float)v.y, (float)v.z, (float)v.w};
    }
};
template <>
struct Load4<__bf16> {
    static __device__ __forceinline__ float4_t at(const __bf16 *p)
    {
        const u16x4 v = *reinterpret_cast<const u16x4 *>(p);
        return float4_t{bf16_bits_to_float(v.x), bf16_bits_to_float(v.y), bf16_bits_to_float(v.z),
                        bf16_bits_to_float(v.w)};
    }
};

// The one rounding of the pass: fp32 to the 16-bit output type, to nearest even.
template <typename T>
__device__ __forceinline__ void store4(T *p, float4_t v)
{
    typedef T t4 __attribute__((ext_vector_type(4)));
    *reinterpret_cast<t4 *>(p) = t4{(T)v.x, (T)v.y, (T)v.z, (T)v.w};
}

// Sum over the L lanes of a head (L consecutive lanes, aligned).
template <int L>
__device__ __forceinline__ float head_sum(float v)
{
    v += dpp_f32<0xB1>(v);       // quad_perm [1,0,3,2]
    v += dpp_f32<0x4E>(v);       // quad_perm [2,3,0,1]
    v += dpp_f32<0x141>(v);      // row_half_mirror: the other quad of 8 lanes
    if constexpr (L >= 16)
        v += dpp_f32<0x140>(v);  // row_mirror: the other half of 16 lanes
    if constexpr (L >= 32)
        v += __shfl_xor(v, 16);
    return v;
}

template <int L, typename TIN, typename TOUT, bool INTER>
__global__ __launch_bounds__(kThreads) void qk_norm_rope_kernel(const RopeArgs a)
{
    constexpr int HP = kThreads / L;  // heads that a workgroup handles at a time
    const int row = blockIdx.x;
    const int u = threadIdx.x % L;
    const int heads = a.Hq + 2 * a.Hkv;
    const int step = HP * gridDim.y;
    int h = blockIdx.y * HP + threadIdx.x / L;
    const bool in_head = u < a.D / 8, rotated = u < a.R / 8;
    const int d0 = INTER || !rotated ? 8 * u : 4 * u;
    const int d1 = INTER || !rotated ? 8 * u + 4 : a.R / 2 + 4 * u;

    auto source = [&](int head) -> const TIN * {
        if (head < a.Hq)
            return static_cast<const TIN *>(a.q) + row * a.q_stride + (int64_t)head * a.D;
        if (head < a.Hq + a.Hkv)
            return static_cast<const TIN *>(a.k) + row * a.k_stride + (int64_t)(head - a.Hq) * a.D;
        return static_cast<const TIN *>(a.v) + row * a.v_stride + (int64_t)(head - a.Hq - a.Hkv) * a.D;
    };
    float4_t x0{0.f, 0.f, 0.f, 0.f}, x1{0.f, 0.f, 0.f, 0.f};
    if (h < heads && in_head) {  // ahead of the angles, whose arithmetic hides it
        const TIN *s = source(h);
        x0 = Load4<TIN>::at(s + d0);
        x1 = Load4<TIN>::at(s + d1);
    }

    // Four angles, in turns: the product in 64 bits (position 262143 times a
    // frequency of 1 would keep only 5 fraction bits of a radian's 2^-24 in
    // 32), brought to [-1/2, 1/2] before it is rounded to 32.
    float cosine[4] = {1.f, 1.f, 1.f, 1.f}, sine[4] = {0.f, 0.f, 0.f, 0.f};
    if (rotated) {
        const double pos = (double)a.positions[row] * 0.15915494309189533577;  // 1 / (2 pi)
        const float4_t f = *reinterpret_cast<const float4_t *>(a.inv_freq + 4 * u);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const double t = pos * (double)f[j];
            sincospif(2.0f * (float)(t - rint(t)), &sine[j], &cosine[j]);
        }
    }
    // Where this row's key and value go; -1: nowhere.
    const int slot = a.slots[row];
    const bool kept = slot >= 0 && slot < a.slot_count;
    const uint32_t page = kept ? divide(slot, a.page_magic, a.page_shift) : 0;
    const uint32_t offset = kept ? slot - page * a.page_size : 0;

    for (; h < heads; h += step) {
        const bool more = h + step < heads && in_head;
        float4_t n0{0.f, 0.f, 0.f, 0.f}, n1{0.f, 0.f, 0.f, 0.f};
        if (more) {  // the next head's values are on their way during this one's arithmetic
            const TIN *s = source(h + step);
            n0 = Load4<TIN>::at(s + d0);
            n1 = Load4<TIN>::at(s + d1);
        }
        const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hkv;
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            ss += x0[j] * x0[j] + x1[j] * x1[j];
        const float r = rsqrtf(head_sum<L>(ss) * (1.0f / (float)a.D) + a.eps);
        if (in_head) {
            float4_t y0 = x0, y1 = x1;
            if (!is_v) {
                const float *w = is_q ? a.q_weight : a.k_weight;
                const float4_t w0 = *reinterpret_cast<const float4_t *>(w + d0);
                const float4_t w1 = *reinterpret_cast<const float4_t *>(w + d1);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x0[j] = x0[j] * r * (a.weight_offset + w0[j]);
                    x1[j] = x1[j] * r * (a.weight_offset + w1[j]);
                }
                y0 = x0;
                y1 = x1;
                if (rotated && INTER) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        y0[2 * j] = x0[2 * j] * cosine[j] - x0[2 * j + 1] * sine[j];
                        y0[2 * j + 1] = x0[2 * j + 1] * cosine[j] + x0[2 * j] * sine[j];
                        y1[2 * j] = x1[2 * j] * cosine[2 + j] - x1[2 * j + 1] * sine[2 + j];
                        y1[2 * j + 1] = x1[2 * j + 1] * cosine[2 + j] + x1[2 * j] * sine[2 + j];
                    }
                } else if (rotated) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        y0[j] = x0[j] * cosine[j] - x1[j] * sine[j];
                        y1[j] = x1[j] * cosine[j] + x0[j] * sine[j];
                    }
                }
            }
            if (is_q) {
                TOUT *o = static_cast<TOUT *>(a.q_out) + ((int64_t)row * a.Hq + h) * a.D;
                store4(o + d0, y0);
                store4(o + d1, y1);
            } else if (kept) {
                const int hk = h - a.Hq - (is_v ? a.Hkv : 0);
                TOUT *o = static_cast<TOUT *>(is_v ? a.v_cache : a.k_cache) +
                          (((int64_t)page * a.Hkv + hk) * a.page_size + offset) * a.D;
                store4(o + d0, y0);
                store4(o + d1, y1);
            }
        }
        x0 = n0;
        x1 = n1;
    }
}

template <int L, typename TIN, typename TOUT>
hipError_t launch(const RopeArgs &a, bool interleaved, hipStream_t stream)
{
    // Passes of a workgroup over a row's heads: with enough rows to fill the
    // GPU one workgroup takes a whole row and computes its angles once; with
    // fewer rows the heads are spread over workgroups (1024 rows of 32 heads of
    // 256: 10.7 us with four workgroups a CU wanted, 11.1 with 8, 12.0 with 16;
    // 256 rows 5.0, with two 5.2).
    constexpr int HP = kThreads / L;
    const int passes = (a.Hq + 2 * a.Hkv + HP - 1) / HP;
    const int want = (4 * device_cu_count() + a.M - 1) / a.M;  // workgroups per row that fill the GPU
    const dim3 grid(a.M, want < passes ? want : passes);
    if (interleaved)
        qk_norm_rope_kernel<L, TIN, TOUT, true><<<grid, kThreads, 0, stream>>>(a);
    else
        qk_norm_rope_kernel<L, TIN, TOUT, false><<<grid, kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

template <typename TIN, typename TOUT>
hipError_t launch_lanes(const RopeArgs &a, bool interleaved, hipStream_t stream)
{
    if (a.D <= 64)
        return launch<8, TIN, TOUT>(a, interleaved, stream);
    if (a.D <= 128)
        return launch<16, TIN, TOUT>(a, interleaved, stream);
    return launch<32, TIN, TOUT>(a, interleaved, stream);
}

template <typename TIN>
hipError_t launch_out(const RopeArgs &a, bool bf16_out, bool interleaved, hipStream_t stream)
{
    return bf16_out ? launch_lanes<TIN, __bf16>(a, interleaved, stream)
                    : launch_lanes<TIN, _Float16>(a, interleaved, stream);
}

}  // namespace

hipError_t launch_qk_norm_rope(const RopeArgs &a, int in_type, bool bf16_out, bool interleaved, hipStream_t stream)
{
    switch (in_type) {
    case 0: return launch_out<_Float16>(a, bf16_out, interleaved, stream);
    case 1: return launch_out<__bf16>(a, bf16_out, interleaved, stream);
    case 2: return launch_out<float>(a, bf16_out, interleaved, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace qmm
