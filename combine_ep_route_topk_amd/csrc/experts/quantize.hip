// quantize.hip -- bf16 rows and weight matrices to e4m3 with one power-of-two
// scale per block of 128 (rows) or 128 x 128 (weights).
//
// q = round_to_nearest_even(x / s), s the least power of two with
// max|x| / s <= 448 over the block.  Reading is one pass: a block's 128 values
// sit in 8 lanes of one wave, its maximum takes three lane exchanges, and the
// quantised values go straight to the rows' final places -- for ep_dispatch_fp8
// to each of the token's k rows of the expert-contiguous buffer.  HBM-bound, for
// a dispatch most of it writes: 4096 tokens of 7168 to 8 rows each in 48 us on MI355X,
// 6.1 TB/s; 128 tokens in 4 us, one round of latency; 32768 rows as they are in 128 us,
// 5.5 TB/s.
#include "experts_internal.h"

namespace ep {
namespace {

constexpr int kWavesPerBlock = kBlock / kWave;
constexpr int kLaneValues = 16;                       // two 16-byte loads, one 16-byte store
constexpr int kWaveValues = kWave * kLaneValues;      // 1024: eight scale blocks

template <int CTRL>
__device__ __forceinline__ float dpp_max(float v) {
    const int o = __builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true);
    return fmaxf(v, __int_as_float(o));
}
// Maximum over each group of 8 neighbouring lanes: xor 1, xor 2, mirror.
__device__ __forceinline__ float max8(float v) {
    v = dpp_max<0xB1>(v);
    v = dpp_max<0x4E>(v);
    return dpp_max<0x141>(v);
}

__device__ __forceinline__ u32x4 quantize16(const u32x4 (&v)[2], float inv) {
    u32x4 q;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t p = v[i / 2][(i % 2) * 2], r = v[i / 2][(i % 2) * 2 + 1];
        q[i] = pack_e4m3x4(bf16_lo(p) * inv, bf16_hi(p) * inv, bf16_lo(r) * inv, bf16_hi(r) * inv);
    }
    return q;
}

__device__ __forceinline__ float amax16(const u32x4 (&v)[2]) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t p = v[i / 4][i % 4];
        m = max_finite(max_finite(m, bf16_lo(p)), bf16_hi(p));
    }
    return m;
}

// One wave per (row, segment of U * 1024 values).  pos == nullptr: row t of q;
// otherwise its k rows pos[t][j], those outside [0, S) skipped.
template <int U>
__global__ __launch_bounds__(kBlock) void quantize_rows_kernel(
    const uint16_t* __restrict__ x, int T, int H, int k, const int32_t* __restrict__ pos,
    uint8_t* __restrict__ q, uint8_t* __restrict__ scale, uint32_t segs, uint32_t items,
    uint32_t S)
{
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int lane = lane_id(), nb = scale_blocks(H);
    for (uint32_t b = blockIdx.x; b < items; b += gridDim.x) {
        const uint32_t group = b / segs;
        const int seg = int(b - group * segs);
        const int t = int(group) * kWavesPerBlock + wave;
        if (t >= T) continue;
        const int c0 = seg * U * kWaveValues + lane * kLaneValues;
        u32x4 v[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int c = c0 + u * kWaveValues;
            v[u][0] = v[u][1] = u32x4{0, 0, 0, 0};
            if (c < H) {
                const uint16_t* p = x + int64_t(t) * H + c;
                v[u][0] = load16(p);
                v[u][1] = load16(p + 8);
            }
        }
        u32x4 out[U];
        int byte[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int e = scale_exponent(max8(amax16(v[u])));
            byte[u] = e + 127;
            out[u] = quantize16(v[u], pow2(-e));
        }
        for (int j = 0; j < k; ++j) {
            const uint32_t p = pos ? uint32_t(pos[int64_t(t) * k + j]) : uint32_t(t);
            if (p >= S) continue;
            const __amdgpu_buffer_rsrc_t row = buffer_rsrc(q + int64_t(p) * H, H);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + u * kWaveValues;
                if (c < H) {
                    store16_coherent(row, c, out[u]);
                    if (lane % 8 == 0)
                        scale[int64_t(p) * nb + c / kScaleBlock] = uint8_t(byte[u]);
                }
            }
        }
    }
}

template <int U>
hipError_t launch_rows(const uint16_t* x, int T, int H, int k, const int32_t* pos, uint8_t* q,
                       uint8_t* scale, uint32_t cap, hipStream_t s)
{
    const uint32_t segs = uint32_t((H + U * kWaveValues - 1) / (U * kWaveValues));
    const uint64_t all = uint64_t((T + kWavesPerBlock - 1) / kWavesPerBlock) * segs;
    const uint32_t items = uint32_t(all);
    const uint32_t rounds = (items + cap - 1) / cap;
    const uint32_t grid = (items + rounds - 1) / rounds;
    EP_LAUNCH((quantize_rows_kernel<U>), dim3(grid), dim3(kBlock), 0, s, x, T, H, k, pos, q, scale,
              segs, items, uint32_t(T) * uint32_t(k));
    return hipGetLastError();
}

// One workgroup per 128 x 128 block: 16-value runs, 8 to a row, 4 to a thread.
// The transposed copy goes through LDS (rows padded to 132 bytes).  A block's rows
// are 256 bytes read and 128 written, and a workgroup waits for its maximum before it
// writes: 8 experts x 4096 x 7168 in 132 us on MI355X, 5.4 TB/s; with the transposed
// copy 178 us, 5.3 TB/s.
__global__ __launch_bounds__(kBlock) void quantize_weight_kernel(
    const uint16_t* __restrict__ w, int N, int K, uint8_t* __restrict__ q,
    uint8_t* __restrict__ scale, uint8_t* __restrict__ q_t, uint8_t* __restrict__ scale_t)
{
    constexpr int kPitch = kScaleBlock + 4;
    __shared__ float part[kWavesPerBlock];
    __shared__ __attribute__((aligned(16))) uint8_t tile[kScaleBlock * kPitch];
    const int kb = blockIdx.x, nb = blockIdx.y, e = blockIdx.z;
    const int KB = scale_blocks(K), NB = scale_blocks(N);
    const int64_t base = int64_t(e) * N * K;
    u32x4 v[4][2];
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int run = i * kBlock + int(threadIdx.x);
        const int n = nb * kScaleBlock + run / 8, c = kb * kScaleBlock + run % 8 * kLaneValues;
        v[i][0] = v[i][1] = u32x4{0, 0, 0, 0};
        if (n < N && c < K) {
            const uint16_t* p = w + base + int64_t(n) * K + c;
            v[i][0] = load16(p);
            v[i][1] = load16(p + 8);
        }
        m = fmaxf(m, amax16(v[i]));
    }
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) m = fmaxf(m, __shfl_xor(m, d, kWave));
    if (lane_id() == 0) part[threadIdx.x / kWave] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWavesPerBlock; ++i) m = fmaxf(m, part[i]);
    const int ex = scale_exponent(m);
    const float inv = pow2(-ex);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int run = i * kBlock + int(threadIdx.x);
        const int r = run / 8, cc = run % 8 * kLaneValues;
        const int n = nb * kScaleBlock + r, c = kb * kScaleBlock + cc;
        const u32x4 o = quantize16(v[i], inv);
        if (n < N && c < K) store16(q + base + int64_t(n) * K + c, o);
        if (q_t) {
#pragma unroll
            for (int d = 0; d < 4; ++d)
                *reinterpret_cast<uint32_t*>(tile + r * kPitch + cc + d * 4) = o[d];
        }
    }
    if (threadIdx.x == 0) {
        scale[(int64_t(e) * NB + nb) * KB + kb] = uint8_t(ex + 127);
        if (q_t) scale_t[(int64_t(e) * KB + kb) * NB + nb] = uint8_t(ex + 127);
    }
    if (!q_t) return;
    __syncthreads();
    for (int i = 0; i < 4; ++i) {
        const int run = i * kBlock + int(threadIdx.x);
        const int c = run / 8, r0 = run % 8 * kLaneValues;      // transposed: row c, columns r0..
        if (kb * kScaleBlock + c >= K || nb * kScaleBlock + r0 >= N) continue;
        u32x4 o;
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            uint32_t p = 0;
#pragma unroll
            for (int b = 0; b < 4; ++b)
                p |= uint32_t(tile[(r0 + d * 4 + b) * kPitch + c]) << (8 * b);
            o[d] = p;
        }
        store16(q_t + base + int64_t(kb * kScaleBlock + c) * N + nb * kScaleBlock + r0, o);
    }
}

}  // namespace

hipError_t launch_quantize_rows(const uint16_t* x, int T, int H, int k, const int32_t* pos,
                                uint8_t* q, uint8_t* scale, hipStream_t s)
{
    if (small_scatter(T, H, k)) return launch_rows<1>(x, T, H, k, pos, q, scale, kMaxGrid, s);
    return launch_rows<4>(x, T, H, k, pos, q, scale, kMaxGrid, s);
}

hipError_t launch_quantize_weight(const uint16_t* w, int E, int N, int K, uint8_t* q,
                                  uint8_t* scale, uint8_t* q_t, uint8_t* scale_t, hipStream_t s)
{
    EP_LAUNCH(quantize_weight_kernel, dim3(scale_blocks(K), scale_blocks(N), E), dim3(kBlock), 0, s,
              w, N, K, q, scale, q_t, scale_t);
    return hipGetLastError();
}

}  // namespace ep
