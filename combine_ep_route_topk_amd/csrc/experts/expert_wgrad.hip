// expert_wgrad.hip -- gradients of the experts' weights from bf16 rows.
//
// For expert e with rows [b, n):  dW[e][i][j] = sum_{s in [b, n)} dy[s][i] x[s][j]
// in f32, stored or added.  The summed axis is the slow one of both operands:
// tiles of kRows rows are staged as they lie in memory (direct loads into LDS)
// and the matrix instruction's operands -- eight summed values of one column --
// come from LDS through its transposing 16-bit read.  A lane ends up with four
// neighbouring j of one i: 16-byte stores.  Rows past the segment lie outside
// the load descriptors and read as zero.
#include "experts_internal.h"

namespace ep {
namespace {

typedef short s16x8 __attribute__((ext_vector_type(8)));

constexpr int kRows = 32;                   // summed rows per step: one matrix instruction

struct WgradArgs {
    const uint16_t* dy;
    const uint16_t* x;
    const int32_t* offsets;
    int S, N, K, E, accumulate;
    float* dw;
};


template <int TN, int TK, int WN, int WK>
__global__ __launch_bounds__(WN* WK* kWave) void expert_wgrad_kernel(WgradArgs p)
{
    constexpr int kWaves = WN * WK;
    constexpr int FN = TN / WN / 16, FK = TK / WK / 16;
    constexpr int kStage = kRows * (TN + TK) * 2;
    constexpr int kVecN = TN / 8, kVecK = TK / 8;         // 16-byte vectors of a row
    constexpr int kLoadsN = kRows * kVecN / kWave / kWaves, kLoadsK = kRows * kVecK / kWave / kWaves;
    static_assert(kLoadsN * kWave * kWaves == kRows * kVecN, "whole loads");
    static_assert(kLoadsK * kWave * kWaves == kRows * kVecK, "whole loads");
    __shared__ __attribute__((aligned(128))) uint8_t lds[2 * kStage];

    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wn = wave % WN, wk = wave / WN;
    const int N = p.N, K = p.K;
    const int nt = (N + TN - 1) / TN, kt = (K + TK - 1) / TK;
    const int per_expert = nt * kt;
    const int e = int(blockIdx.x) / per_expert;
    const int in = int(blockIdx.x) - e * per_expert;
    const int n0 = in % nt * TN, k0 = in / nt * TK;
    int begin, end;
    segment_of(p.offsets, e, p.S, begin, end);
    begin = __builtin_amdgcn_readfirstlane(begin);
    end = __builtin_amdgcn_readfirstlane(end);
    const int rows = end - begin, steps = (rows + kRows - 1) / kRows;

    uint32_t noff[kLoadsN], koff[kLoadsK];
#pragma unroll
    for (int i = 0; i < kLoadsN; ++i) {
        const int v = (i * kWaves + wave) * kWave + lane, r = v / kVecN, c = n0 + v % kVecN * 8;
        noff[i] = c < N ? uint32_t(r) * uint32_t(N) * 2u + uint32_t(c) * 2u : kOutside;
    }
#pragma unroll
    for (int i = 0; i < kLoadsK; ++i) {
        const int v = (i * kWaves + wave) * kWave + lane, r = v / kVecK, c = k0 + v % kVecK * 8;
        koff[i] = c < K ? uint32_t(r) * uint32_t(K) * 2u + uint32_t(c) * 2u : kOutside;
    }
    auto issue = [&](int step) {
        uint8_t* st = lds + (step & 1) * kStage;
        const int64_t r0 = begin + int64_t(step) * kRows;
        const int left = end - int(r0) < kRows ? end - int(r0) : kRows;
        const __amdgpu_buffer_rsrc_t nr =
            buffer_rsrc(const_cast<uint16_t*>(p.dy) + r0 * N, int64_t(left) * N * 2);
        const __amdgpu_buffer_rsrc_t kr =
            buffer_rsrc(const_cast<uint16_t*>(p.x) + r0 * K, int64_t(left) * K * 2);
#pragma unroll
        for (int i = 0; i < kLoadsN; ++i)
            load16_to_lds(nr, st + (i * kWaves + wave) * 1024, noff[i]);
#pragma unroll
        for (int i = 0; i < kLoadsK; ++i)
            load16_to_lds(kr, st + kRows * TN * 2 + (i * kWaves + wave) * 1024, koff[i]);
    };

    f32x4 acc[FK][FN];
#pragma unroll
    for (int i = 0; i < FK; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

    // 16 columns from `col` on, all kRows rows: lane group g takes rows 8 g ..
    const int g = lane / 16, l = lane % 16;
    auto fragment = [&](uint8_t* base, int C, int col) {
        uint8_t* a = base + ((g * 8 + l / 4) * C + col + l % 4 * 4) * 2;
        const s16x4 lo = read_transposed(a);
        const s16x4 hi = read_transposed(a + 4 * C * 2);
        const s16x8 v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        return __builtin_bit_cast(bf16x8, v);
    };

    if (steps) issue(0);
    for (int s = 0; s < steps; ++s) {
        wait_own_stores();      // this wave's loads into LDS have landed
        __syncthreads();
        if (s + 1 < steps) issue(s + 1);
        uint8_t* st = lds + (s & 1) * kStage;
        bf16x8 dy[FN];
#pragma unroll
        for (int j = 0; j < FN; ++j) dy[j] = fragment(st, TN, (wn * FN + j) * 16);
#pragma unroll
        for (int i = 0; i < FK; ++i) {
            const bf16x8 x = fragment(st + kRows * TN * 2, TK, (wk * FK + i) * 16);
#pragma unroll
            for (int j = 0; j < FN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, dy[j], acc[i][j], 0, 0, 0);
        }
    }

    float* out = p.dw + int64_t(e) * N * K;
#pragma unroll
    for (int j = 0; j < FN; ++j) {
        const int n = n0 + (wn * FN + j) * 16 + l;
        if (n >= N) continue;
#pragma unroll
        for (int i = 0; i < FK; ++i) {
            const int k = k0 + (wk * FK + i) * 16 + g * 4;
            if (k >= K) continue;
            f32x4* d = reinterpret_cast<f32x4*>(out + int64_t(n) * K + k);
            f32x4 v = acc[i][j];
            if (p.accumulate) {
                const f32x4 o = *d;
#pragma unroll
                for (int c = 0; c < 4; ++c) v[c] += o[c];
            }
            *d = v;
        }
    }
}

template <int TN, int TK, int WN, int WK>
hipError_t launch(const WgradArgs& p, hipStream_t s)
{
    const int64_t grid = int64_t((p.N + TN - 1) / TN) * ((p.K + TK - 1) / TK) * p.E;
    if (grid * WN * WK * kWave >= (int64_t(1) << 31)) return hipErrorInvalidConfiguration;
    EP_LAUNCH((expert_wgrad_kernel<TN, TK, WN, WK>), dim3(uint32_t(grid)), dim3(WN * WK * kWave), 0,
              s, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_expert_wgrad(const uint16_t* grad_y, const uint16_t* x, const int32_t* offsets,
                               int S, int N, int K, int E, int accumulate, float* grad_w,
                               hipStream_t s)
{
    const WgradArgs p{grad_y, x, offsets, S, N, K, E, accumulate, grad_w};
    return launch<256, 256, 4, 2>(p, s);
}

}  // namespace ep
