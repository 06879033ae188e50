// quantize_int8.hip -- bf16 rows to int8 with one f32 scale a row.
//
// m = max(max|x|, 127 2^-126), scale = m / 127, q = round_to_nearest_even(127 x / m).
// For bf16 x that quotient is decided exactly: 127 x is exact in f32 and m has 8
// bits, so 127 x / m either is a half integer, which a correctly rounded f32
// quotient keeps, or is 2^-9 away from one at least.  A row with an infinity or a NaN
// gets the scale NaN and zeros: its products are NaN.
#include "experts_internal.h"

namespace ep {
namespace {

constexpr int kWaves = kBlock / kWave;
constexpr float kLeastTop = 127.0f * 0x1p-126f;       // scales stay normal numbers

__device__ __forceinline__ float top16(const u32x4 (&v)[2]) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t p = v[i / 4][i % 4];
        // as integers, since a NaN is above infinity
        const uint32_t lo = p << 16 & 0x7FFFFFFFu, hi = p & 0x7FFF0000u;
        const uint32_t a = __float_as_uint(m);
        m = __uint_as_float(lo > hi ? (lo > a ? lo : a) : (hi > a ? hi : a));
    }
    return m;
}

// 127 x / m to the nearest integer.  Both are first scaled by the power of two that
// brings m to [2, 4): exact, but for x so small that q is 0, and 127 x stays in
// range.  With r the rounded 1 / m, t = 127 x r is two steps off the quotient at most,
// and t + (127 x - t m) r, both fused, is the quotient correctly rounded.  Adding 1.5
// 2^23 leaves the nearest integer, ties to even, in the low bits.
struct Quotient {
    float by, m, r;
    __device__ __forceinline__ explicit Quotient(float top) {
        const float p = pow2(128 - int(__float_as_uint(top) >> 23));
        by = 127.0f * p;
        m = top * p;
        r = 1.0f / m;
    }
    __device__ __forceinline__ uint32_t nearest(float x) const {
        const float y = x * by, t = y * r;
        return __float_as_uint(__builtin_fmaf(__builtin_fmaf(-t, m, y), r, t) + 0x1.8p23f);
    }
};

// The row that a workgroup quantises: of x, or, with first and past, of the rows
// [*first, *past) clamped to [0, S).  pos: to the k rows pos[t][j] instead of row t,
// those outside [0, T k) skipped.
__global__ __launch_bounds__(kBlock) void quantize_rows_int8_kernel(
    const uint16_t* __restrict__ x, int T, int H, int k, const int32_t* __restrict__ pos,
    const int32_t* __restrict__ first, const int32_t* __restrict__ past, int8_t* __restrict__ q,
    float* __restrict__ scale)
{
    __shared__ uint32_t part[kWaves];
    const int64_t S = int64_t(T) * k;
    for (int t = blockIdx.x; t < T; t += gridDim.x) {
        if (first && (t < *first || t >= *past)) continue;
        const uint16_t* const row = x + int64_t(t) * H;
        uint32_t m = 0;
        for (int c = threadIdx.x * 16; c < H; c += kBlock * 16) {
            const u32x4 v[2] = {load16(row + c), load16(row + c + 8)};
            const uint32_t n = __float_as_uint(top16(v));
            m = m > n ? m : n;
        }
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
            const uint32_t n = uint32_t(__shfl_xor(int(m), d, kWave));
            m = m > n ? m : n;
        }
        __syncthreads();
        if (lane_id() == 0) part[threadIdx.x / kWave] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kWaves; ++i) m = m > part[i] ? m : part[i];
        const bool finite = m < 0x7F800000u;
        const float top = fmaxf(__uint_as_float(finite ? m : 0u), kLeastTop);
        const Quotient quotient(top);
        for (int j = 0; j < k; ++j) {
            const int64_t to = pos ? pos[int64_t(t) * k + j] : t;
            if (to < 0 || to >= S) continue;
            for (int c = threadIdx.x * 16; c < H; c += kBlock * 16) {
                const u32x4 v[2] = {load16(row + c), load16(row + c + 8)};
                u32x4 o;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t b = 0;
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        const uint32_t u = v[i / 2][i % 2 * 2 + d / 2];
                        const float f = d & 1 ? bf16_hi(u) : bf16_lo(u);
                        b |= (quotient.nearest(f) & 255) << (8 * d);
                    }
                    o[i] = finite ? b : 0u;
                }
                store16(q + to * H + c, o);
            }
            if (threadIdx.x == 0)
                scale[to] = finite ? top / 127.0f : __uint_as_float(0x7FC00000u);
        }
    }
}

}  // namespace

hipError_t launch_quantize_rows_int8(const uint16_t* x, int T, int H, int k, const int32_t* pos,
                                     const int32_t* first, const int32_t* past, int8_t* q,
                                     float* scale, hipStream_t s)
{
    const uint32_t grid = uint32_t(T) < kMaxGrid ? uint32_t(T) : kMaxGrid;
    EP_LAUNCH(quantize_rows_int8_kernel, dim3(grid), dim3(kBlock), 0, s, x, T, H, k, pos, first, past,
              q, scale);
    return hipGetLastError();
}

}  // namespace ep
