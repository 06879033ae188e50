// quantize_int8.hip -- bf16 rows to int8 with one f32 scale a row.
//
// m = max(max|x|, 127 2^-126), scale = m / 127, q = round_to_nearest_even(127 x / m).
// For bf16 x that quotient is decided exactly: 127 x is exact in f32, and with X, M <
// 2^8 the mantissas as integers and 2^d the ratio of their units, 127 x / m = 127 X / (M
// 2^d) is |254 X - h M 2^d| / (M 2^(d+1)) away from a half integer h / 2: it is one, which a
// correctly rounded f32 quotient keeps, or 1 / (254 X) of itself away at least, more than
// 2^-16, where such a quotient is off by 2^-24 of itself.  A row with an infinity or a NaN
// gets the scale NaN and zeros: its products are NaN.
//
// Bytes bound it, 2 H read and (H + 4) written for each copy of a row: a row is read once
// and kept in registers from its maximum to its values, by one wave up to 2048 values
// and by four up to 8192.  MI355X, H = 7168: 4096 tokens to 8 rows each 49 us, 6.0 TB/s
// (by a workgroup a row that reads it twice 88); 32768 rows to one 125 us, 5.6 TB/s,
// reads and writes mixed, where a copy reaches 5.0.  One division a row.
#include "experts_internal.h"

namespace ep {
namespace {

constexpr int kWavesPerBlock = kBlock / kWave;
constexpr int kLaneValues = 16;                       // two 16-byte loads, one 16-byte store
constexpr int kWaveValues = kWave * kLaneValues;      // 1024
constexpr float kLeastTop = 127.0f * 0x1p-126f;       // scales stay normal numbers

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// The largest magnitude as an integer (where NaN lies above infinity), bf16's bits.
struct Top {
    u16x2 m = {0, 0};
    __device__ __forceinline__ void add(u32x4 v) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, v[i] & 0x7FFF7FFFu));
    }
    __device__ __forceinline__ uint32_t of_wave() const {
        uint32_t t = m[0] > m[1] ? m[0] : m[1];
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
            const uint32_t o = uint32_t(__shfl_xor(int(t), d, kWave));
            t = t > o ? t : o;
        }
        return t;
    }
};

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

// 32 bytes of bf16 to 16 integers; `keep` 0 makes them zeros.
__device__ __forceinline__ u32x4 quantize16(const u32x4 (&v)[2], const Quotient& quotient, uint32_t keep) {
    u32x4 q;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t p = v[i / 2][(i % 2) * 2], r = v[i / 2][(i % 2) * 2 + 1];
        // the low bytes of two, then of four
        const uint32_t lo = __builtin_amdgcn_perm(quotient.nearest(bf16_hi(p)),
                                                  quotient.nearest(bf16_lo(p)), 0x0C0C0400u);
        const uint32_t hi = __builtin_amdgcn_perm(quotient.nearest(bf16_hi(r)),
                                                  quotient.nearest(bf16_lo(r)), 0x0C0C0400u);
        q[i] = __builtin_amdgcn_perm(hi, lo, 0x05040100u) & keep;
    }
    return q;
}

// WAVES waves take a row of up to U * 1024 * WAVES values, which stay in registers
// between its maximum and its quantising (U = 0: any length, read twice, the second
// time from the caches).  first, past: only the rows [*first, *past).  pos: to the k
// rows pos[t][j] instead of row t, those outside [0, S) skipped.
template <int WAVES, int U>
__global__ __launch_bounds__(kBlock) void quantize_rows_int8_kernel(
    const uint16_t* __restrict__ x, int T, int H, int k, const int32_t* __restrict__ pos,
    const int32_t* __restrict__ first, const int32_t* __restrict__ past, int8_t* __restrict__ q,
    float* __restrict__ scale, uint32_t S)
{
    constexpr int kRows = kWavesPerBlock / WAVES, kStep = WAVES * kWaveValues;
    __shared__ uint32_t part[2][kWavesPerBlock];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = lane_id();
    const int c0 = (wave % WAVES) * kWaveValues + lane * kLaneValues;
    int begin = 0, end = T;
    if (first) {
        begin = *first > 0 ? *first : 0;
        end = *past < T ? *past : T;
    }
    int turn = 0;
    // 64 bits: a grid past the last row
    for (int64_t t0 = begin + int64_t(blockIdx.x) * kRows; t0 < end;
         t0 += int64_t(gridDim.x) * kRows, turn ^= 1) {
        const int t = int(t0) + wave / WAVES;
        if (WAVES == 1 && t >= end) break;
        const uint16_t* const row = x + int64_t(t) * H;
        Top top;
        u32x4 v[U ? U : 1][2];
        if (U) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + u * kStep;
                v[u][0] = v[u][1] = u32x4{0, 0, 0, 0};
                if (c < H) {
                    v[u][0] = load16(row + c);
                    v[u][1] = load16(row + c + 8);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                top.add(v[u][0]);
                top.add(v[u][1]);
            }
        } else {
            for (int c = c0; c < H; c += kStep) {
                top.add(load16(row + c));
                top.add(load16(row + c + 8));
            }
        }
        uint32_t m = top.of_wave();
        if (WAVES > 1) {
            if (lane == 0) part[turn][wave] = m;      // the next row's go to the other set
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kWavesPerBlock; ++i) m = m > part[turn][i] ? m : part[turn][i];
        }
        m = uint32_t(__builtin_amdgcn_readfirstlane(int(m)));
        const bool finite = m < 0x7F80u;
        const float most = fmaxf(__uint_as_float(finite ? m << 16 : 0u), kLeastTop);
        const Quotient quotient(most);
        const uint32_t keep = finite ? 0xFFFFFFFFu : 0u;
        const float unit = finite ? most / 127.0f : __uint_as_float(0x7FC00000u);
        if (U) {
            u32x4 out[U ? U : 1];
#pragma unroll
            for (int u = 0; u < U; ++u) out[u] = quantize16(v[u], quotient, keep);
            for (int j = 0; j < k; ++j) {
                const uint32_t to = pos ? uint32_t(pos[int64_t(t) * k + j]) : uint32_t(t);
                if (to >= S) continue;
                const __amdgpu_buffer_rsrc_t r = buffer_rsrc(q + int64_t(to) * H, H);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (c0 + u * kStep < H) store16_coherent(r, c0 + u * kStep, out[u]);
                if (lane == 0 && wave % WAVES == 0) scale[to] = unit;
            }
        } else {
            for (int c = c0; c < H; c += kStep) {
                const u32x4 w[2] = {load16(row + c), load16(row + c + 8)};
                const u32x4 out = quantize16(w, quotient, keep);
                for (int j = 0; j < k; ++j) {
                    const uint32_t to = pos ? uint32_t(pos[int64_t(t) * k + j]) : uint32_t(t);
                    if (to < S) store16_nt(q + int64_t(to) * H + c, out);
                }
            }
            if (lane == 0 && wave == 0)
                for (int j = 0; j < k; ++j) {
                    const uint32_t to = pos ? uint32_t(pos[int64_t(t) * k + j]) : uint32_t(t);
                    if (to < S) scale[to] = unit;
                }
        }
    }
}

template <int WAVES, int U>
hipError_t launch(const uint16_t* x, int T, int H, int k, const int32_t* pos, const int32_t* first,
                  const int32_t* past, int8_t* q, float* scale, hipStream_t s)
{
    constexpr int kRows = kWavesPerBlock / WAVES;
    const uint32_t blocks = (uint32_t(T) + kRows - 1) / kRows;
    const uint32_t grid = blocks < kMaxGrid ? blocks : kMaxGrid;
    EP_LAUNCH((quantize_rows_int8_kernel<WAVES, U>), dim3(grid), dim3(kBlock), 0, s, x, T, H, k, pos,
              first, past, q, scale, uint32_t(T) * uint32_t(k));
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_rows_int8(const uint16_t* x, int T, int H, int k, const int32_t* pos,
                                     const int32_t* first, const int32_t* past, int8_t* q,
                                     float* scale, hipStream_t s)
{
    if (H <= 2 * kWaveValues) return launch<1, 2>(x, T, H, k, pos, first, past, q, scale, s);
    if (H <= 8 * kWaveValues) return launch<4, 2>(x, T, H, k, pos, first, past, q, scale, s);
    return launch<4, 0>(x, T, H, k, pos, first, past, q, scale, s);
}

}  // namespace ep
