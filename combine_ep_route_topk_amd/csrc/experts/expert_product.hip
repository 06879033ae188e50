// expert_product.hip -- grouped products of bf16 and of 8-bit integers over
// expert segments, with the gated activation for an epilogue.
//
// For a row s of expert e:
//   bf16:  y[s][n] = sum_k a[s][k] W[e][n][k]            (f32 sums, rounded once)
//          y[s][n] = sum_k a[s][k] W[e][k][n]            (transposed)
//   int8:  y[s][n] = as[s] (ws[e][n] sum_k a[s][k] W[e][n][k])   (integer sums)
//   gated: g and u so from the rows [0, I) and [I, 2I) of W, h = silu(g) u in f32,
//          rounded once to bf16.
// A tile of 64 rows x 64 weight rows a workgroup, 128 bytes of k a step.
#include "expert_tiles.h"

namespace ep {
namespace {

struct ProductArgs {
    const uint8_t* a;
    const float* a_scale;
    const uint8_t* w;
    const float* w_scale;
    const int32_t* offsets;
    int S, N, K, E;      // N: rows of one expert's weights (2 I when gated)
    int max_tiles;       // row tiles that S rows in E segments can make
    uint16_t* y;         // plain: [S][N]; gated: gate_up [S][N] or NULL
    uint16_t* h;         // gated: [S][N/2]
};

struct Bf16 {
    typedef f32x4 Acc;
    static constexpr int kBytes = 2;
    static __device__ __forceinline__ Acc mfma(u32x4 w, u32x4 x, Acc c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w),
                                                       __builtin_bit_cast(bf16x8, x), c, 0, 0, 0);
    }
};
struct Int8 {
    typedef i32x4 Acc;
    static constexpr int kBytes = 1;
    static __device__ __forceinline__ Acc mfma(u32x4 w, u32x4 x, Acc c) {
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, w),
                                                     __builtin_bit_cast(i32x4, x), c, 0, 0, 0);
    }
};

template <class T, bool TRANS, bool GATED>
__global__ __launch_bounds__(256) void expert_product_kernel(ProductArgs p)
{
    constexpr int kTile = 64, kPitch = 128 + 16, kParts = GATED ? 2 : 1;
    __shared__ __attribute__((aligned(16))) uint8_t xs[kTile * kPitch];
    __shared__ __attribute__((aligned(16))) uint8_t ws[kParts * kTile * kPitch];
    const int lane = lane_id(), l = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int rows_n = GATED ? p.N / 2 : p.N, row_bytes = p.K * T::kBytes;
    const GemmTile tile = GemmTiles(p, kTile, (rows_n + kTile - 1) / kTile).at(p, kTile, 0);
    const RowTile t = tile.rows;
    if (t.expert < 0) return;
    const int rows = t.end - t.row0 < kTile ? t.end - t.row0 : kTile;
    const int first = tile.n * kTile;
    const int left = rows_n - first < kTile ? rows_n - first : kTile;

    typename T::Acc acc[kParts][4];
#pragma unroll
    for (int i = 0; i < kParts; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = typename T::Acc{0, 0, 0, 0};
    for (int k0 = 0; k0 < row_bytes; k0 += 128) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = (i * 256 + int(threadIdx.x)) / 8, c = threadIdx.x % 8 * 16;
            u32x4 v = {0, 0, 0, 0};
            if (r < rows && k0 + c < row_bytes)
                v = load16(p.a + int64_t(t.row0 + r) * row_bytes + k0 + c);
            store16(xs + r * kPitch + c, v);
            if (TRANS) {                        // 64 rows of k x 64 columns
                const int k = k0 / 2 + r, n = first + c / 2;
                v = u32x4{0, 0, 0, 0};
                if (k < p.K && n < p.N) v = load16(p.w + ((int64_t(t.expert) * p.K + k) * p.N + n) * 2);
#pragma unroll
                for (int d = 0; d < 8; ++d)
                    *reinterpret_cast<uint16_t*>(ws + (c / 2 + d) * kPitch + r * 2) =
                        uint16_t(v[d / 2] >> (d % 2 * 16));
            } else {
#pragma unroll
                for (int q = 0; q < kParts; ++q) {
                    v = u32x4{0, 0, 0, 0};
                    if (r < left && k0 + c < row_bytes)
                        v = load16(p.w + (int64_t(t.expert) * p.N + q * rows_n + first + r) * row_bytes +
                                   k0 + c);
                    store16(ws + (q * kTile + r) * kPitch + c, v);
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            u32x4 w[kParts];
#pragma unroll
            for (int q = 0; q < kParts; ++q)
                w[q] = load16(ws + (q * kTile + wave * 16 + l) * kPitch + c * 64 + g * 16);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const u32x4 x = load16(xs + (j * 16 + l) * kPitch + c * 64 + g * 16);
#pragma unroll
                for (int q = 0; q < kParts; ++q) acc[q][j] = T::mfma(w[q], x, acc[q][j]);
            }
        }
    }
    // lane: token 16 j + l, weight rows 16 wave + 4 g + 0..3
    const int n = first + wave * 16 + g * 4;
    if (n >= rows_n) return;
    f32x4 scale[kParts];
#pragma unroll
    for (int q = 0; q < kParts; ++q) {
        scale[q] = f32x4{1, 1, 1, 1};
        if (T::kBytes == 1)
            scale[q] = *reinterpret_cast<const f32x4*>(p.w_scale + int64_t(t.expert) * p.N +
                                                       q * rows_n + n);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int m = j * 16 + l;
        if (m >= rows) continue;
        const float token = T::kBytes == 1 ? p.a_scale[t.row0 + m] : 1.0f;
        f32x4 v[kParts];
#pragma unroll
        for (int q = 0; q < kParts; ++q)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                v[q][c] = T::kBytes == 1 ? float(acc[q][j][c]) * scale[q][c] * token
                                         : float(acc[q][j][c]);
#pragma unroll
        for (int q = 0; q < kParts; ++q)
            if (p.y)
                *reinterpret_cast<u32x2*>(p.y + int64_t(t.row0 + m) * p.N + q * rows_n + n) =
                    u32x2{pack_bf16x2(v[q][0], v[q][1]), pack_bf16x2(v[q][2], v[q][3])};
        if (GATED) {
            float h[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) h[c] = v[0][c] * sigmoid(v[0][c]) * v[kParts - 1][c];
            *reinterpret_cast<u32x2*>(p.h + int64_t(t.row0 + m) * rows_n + n) =
                u32x2{pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3])};
        }
    }
}

template <class T, bool TRANS, bool GATED>
hipError_t launch(ProductArgs p, hipStream_t s)
{
    ProductArgs tiles = p;
    tiles.N = GATED ? p.N / 2 : p.N;
    const uint32_t grid = gemm_tiles(tiles, 64, 64);
    p.max_tiles = tiles.max_tiles;
    if (!grid || uint64_t(grid) * 256 >= (uint64_t(1) << 31)) return hipErrorInvalidConfiguration;
    EP_LAUNCH((expert_product_kernel<T, TRANS, GATED>), dim3(grid), dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_expert_gemm_bf16(const uint16_t* a, const uint16_t* w, const int32_t* offsets,
                                   int S, int N, int K, int E, bool transposed, uint16_t* y,
                                   hipStream_t s)
{
    const ProductArgs p{reinterpret_cast<const uint8_t*>(a), nullptr,
                        reinterpret_cast<const uint8_t*>(w), nullptr, offsets, S, N, K, E, 0, y,
                        nullptr};
    return transposed ? launch<Bf16, true, false>(p, s) : launch<Bf16, false, false>(p, s);
}

hipError_t launch_expert_swiglu_bf16(const uint16_t* a, const uint16_t* w13, const int32_t* offsets,
                                     int S, int I, int K, int E, uint16_t* h, uint16_t* gate_up,
                                     hipStream_t s)
{
    return launch<Bf16, false, true>(
        ProductArgs{reinterpret_cast<const uint8_t*>(a), nullptr,
                    reinterpret_cast<const uint8_t*>(w13), nullptr, offsets, S, 2 * I, K, E, 0,
                    gate_up, h}, s);
}

hipError_t launch_expert_gemm_int8(const int8_t* a, const float* a_scale, const int8_t* w,
                                   const float* w_scale, const int32_t* offsets, int S, int N, int K,
                                   int E, uint16_t* y, hipStream_t s)
{
    return launch<Int8, false, false>(
        ProductArgs{reinterpret_cast<const uint8_t*>(a), a_scale, reinterpret_cast<const uint8_t*>(w),
                    w_scale, offsets, S, N, K, E, 0, y, nullptr}, s);
}

hipError_t launch_expert_swiglu_int8(const int8_t* a, const float* a_scale, const int8_t* w13,
                                     const float* w13_scale, const int32_t* offsets, int S, int I,
                                     int K, int E, uint16_t* h, hipStream_t s)
{
    return launch<Int8, false, true>(
        ProductArgs{reinterpret_cast<const uint8_t*>(a), a_scale,
                    reinterpret_cast<const uint8_t*>(w13), w13_scale, offsets, S, 2 * I, K, E, 0,
                    nullptr, h}, s);
}

}  // namespace ep
