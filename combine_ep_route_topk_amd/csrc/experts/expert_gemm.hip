// expert_gemm.hip -- grouped block-scaled FP8 products over expert segments.
//
// For a row s of expert e:  y[s][n] = sum_b 2^(as[s][b] + ws[n/128][b] - 254)
//                                     sum_{k in block b} a[s][k] w[e][n][k].
// The scales are powers of two for blocks of 128 along k, so the matrix
// instruction (16 x 16 outputs, 128 of k) takes both as operands and the f32
// accumulators never leave the matrix core's registers: no multiply-add per
// block on the vector ALU.  The weights are its row operand: a lane then holds
// four neighbouring n of one token.
#include "expert_gemm_large.h"

namespace ep {
namespace {

constexpr int kBK = kScaleBlock;          // bytes of k per step = one scale block

// LDS image of a tile: rows of 128 bytes in eight 16-byte chunks, chunk c of
// row r at slot c ^ (r / 2 % 8): 16 lanes reading the same chunk of 16
// consecutive rows touch all 64 banks once.
__device__ __forceinline__ int chunk_slot(int r, int c) { return c ^ ((r >> 1) & 7); }

// Weight row (within the expert) of row r of a tile.  Gated: groups of 16
// rows alternate between gate and up, so one wave holds both of each output.
template <int TN, bool GATED>
__device__ __forceinline__ int weight_row(int tile_n, int r, int N) {
    if (!GATED) return tile_n * TN + r;
    const int g = r >> 4;
    return tile_n * (TN / 2) + (g >> 1) * 16 + (r & 15) + (g & 1) * (N / 2);
}

template <int TN, int TM, int WN, int WM, bool GATED>
__global__ __launch_bounds__(WN* WM* kWave) void expert_gemm_kernel(GemmArgs p)
{
    constexpr int kWaves = WN * WM;
    constexpr int FN = TN / WN / 16, FM = TM / WM / 16;
    constexpr int kLoadsW = TN / 8 / kWaves, kLoadsX = TM / 8 / kWaves;
    static_assert(kLoadsW * 8 * kWaves == TN && kLoadsX * 8 * kWaves == TM, "whole loads");
    static_assert(!GATED || TN == 2 * kScaleBlock, "a gated tile makes one scale block");
    constexpr int kStage = (TN + TM) * kBK;
    __shared__ __attribute__((aligned(128))) uint8_t lds[2 * kStage];

    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wn = wave % WN, wm = wave / WN;
    const int N = p.N, K = p.K, KB = scale_blocks(K);

    const GemmTile tile = GemmTiles(p, TM, GATED ? N / 256 : (N + TN - 1) / TN).at(p, TM, 0);
    const RowTile t = tile.rows;
    const int tile_n = tile.n;
    if (t.expert < 0) return;
    const int rows = t.end - t.row0 < TM ? t.end - t.row0 : TM;

    const uint8_t* wbase = p.w + int64_t(t.expert) * N * K;
    const uint8_t* xbase = p.a + int64_t(t.row0) * K;
    const int wrows = GATED ? N : (N - tile_n * TN < TN ? N - tile_n * TN : TN);
    if (!GATED) wbase += int64_t(tile_n) * TN * K;
    const int64_t wbytes = int64_t(wrows) * K, xbytes = int64_t(rows) * K;

    // ---- this lane's source offsets (row and chunk), one per load
    uint32_t woff[kLoadsW], xoff[kLoadsX];
    const int lrow = lane / 8, lslot = lane % 8;
    int chunk[2];       // chunk of even and odd instructions' rows: rows advance by 8 * kWaves
    chunk[0] = chunk_slot(lrow + wave * 8, lslot);
    static_assert(kWaves % 2 == 0, "rows of one lane's loads differ by multiples of 16");
    const uint32_t cb = uint32_t(chunk[0]) * 16;
#pragma unroll
    for (int i = 0; i < kLoadsW; ++i) {
        const int r = (i * kWaves + wave) * 8 + lrow;
        const int g = GATED ? weight_row<TN, true>(tile_n, r, N) : r;
        woff[i] = uint32_t(g) * uint32_t(K) + cb;
    }
#pragma unroll
    for (int i = 0; i < kLoadsX; ++i)
        xoff[i] = uint32_t((i * kWaves + wave) * 8 + lrow) * uint32_t(K) + cb;

    const int steps = KB;
    auto issue = [&](int step) {
        uint8_t* st = lds + (step & 1) * kStage;
        const int k0 = step * kBK;
        const __amdgpu_buffer_rsrc_t wr = buffer_rsrc(const_cast<uint8_t*>(wbase) + k0, wbytes - k0);
        const __amdgpu_buffer_rsrc_t xr = buffer_rsrc(const_cast<uint8_t*>(xbase) + k0, xbytes - k0);
        const bool out = int(cb) >= K - k0;
#pragma unroll
        for (int i = 0; i < kLoadsW; ++i)
            load16_to_lds(wr, st + (i * kWaves + wave) * 1024, out ? kOutside : woff[i]);
#pragma unroll
        for (int i = 0; i < kLoadsX; ++i)
            load16_to_lds(xr, st + TN * kBK + (i * kWaves + wave) * 1024,
                          out ? kOutside : xoff[i]);
    };

    // ---- scales: one weight block per wave (gated: gate's and up's)
    const int NB = scale_blocks(N);
    const uint8_t* wsb = p.w_scale + int64_t(t.expert) * NB * KB;
    const uint8_t* wsc[FN];
#pragma unroll
    for (int i = 0; i < FN; ++i) {
        int n = GATED ? weight_row<TN, true>(tile_n, (wn * FN + i) * 16, N)
                      : tile_n * TN + (wn * FN + i) * 16;
        n = n < N ? n : N - 1;
        wsc[i] = wsb + int64_t(n / kScaleBlock) * KB;
    }
    const uint8_t* xsc[FM];
#pragma unroll
    for (int j = 0; j < FM; ++j) {
        const int m = (wm * FM + j) * 16 + lane % 16;
        xsc[j] = p.a_scale + int64_t(t.row0 + (m < rows ? m : rows - 1)) * KB;
    }

    f32x4 acc[FN][FM];
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

    const int frow = lane % 16, g = lane / 16;
    auto fragment = [&](const uint8_t* base, int row) {
        const uint8_t* r = base + row * kBK;
        const u32x4 lo = load16(r + chunk_slot(row, 2 * g) * 16);
        const u32x4 hi = load16(r + chunk_slot(row, 2 * g + 1) * 16);
        return i32x8{int(lo[0]), int(lo[1]), int(lo[2]), int(lo[3]),
                     int(hi[0]), int(hi[1]), int(hi[2]), int(hi[3])};
    };

    // the scales of a step are loaded one step ahead, before the tiles' loads
    int ws[FN], xs[FM], ws_next[FN], xs_next[FM];
    auto load_scales = [&](int step) {
#pragma unroll
        for (int i = 0; i < FN; ++i) ws_next[i] = wsc[i][step];
#pragma unroll
        for (int j = 0; j < FM; ++j) xs_next[j] = xsc[j][step];
    };

    load_scales(0);
    issue(0);
    for (int s = 0; s < steps; ++s) {
        wait_own_stores();      // this wave's loads into LDS have landed
        __syncthreads();
#pragma unroll
        for (int i = 0; i < FN; ++i) ws[i] = ws_next[i];
#pragma unroll
        for (int j = 0; j < FM; ++j) xs[j] = xs_next[j];
        if (s + 1 < steps) {
            load_scales(s + 1);
            issue(s + 1);
        }
        const uint8_t* st = lds + (s & 1) * kStage;
        i32x8 x[FM];
#pragma unroll
        for (int j = 0; j < FM; ++j) x[j] = fragment(st + TN * kBK, (wm * FM + j) * 16 + frow);
#pragma unroll
        for (int i = 0; i < FN; ++i) {
            const i32x8 w = fragment(st, (wn * FN + i) * 16 + frow);
#pragma unroll
            for (int j = 0; j < FM; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    w, x[j], acc[i][j], 0, 0, 0, ws[i], 0, xs[j]);
        }
    }

    // ---- epilogue
    if constexpr (!GATED) {
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            const int m = (wm * FM + j) * 16 + frow;
            if (m >= rows) continue;
            uint16_t* row = p.y + int64_t(t.row0 + m) * N;
#pragma unroll
            for (int i = 0; i < FN; ++i) {
                const int n = tile_n * TN + (wn * FN + i) * 16 + g * 4;
                if (n >= N) continue;
                const u32x2 v = {pack_bf16x2(acc[i][j][0], acc[i][j][1]),
                                 pack_bf16x2(acc[i][j][2], acc[i][j][3])};
                *reinterpret_cast<u32x2*>(row + n) = v;
            }
        }
    } else {
        __shared__ float part[WN][TM];
        const int I = N / 2;
        f32x4 hv[FN / 2][FM];
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            const int m = (wm * FM + j) * 16 + frow;
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < FN / 2; ++i) {
                const f32x4 gate = acc[2 * i][j], up = acc[2 * i + 1][j];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float v = gate[c] * sigmoid(gate[c]) * up[c];
                    hv[i][j][c] = v;
                    top = max_finite(top, v);
                }
                if (p.y && m < rows) {
                    uint16_t* row = p.y + int64_t(t.row0 + m) * N + tile_n * kScaleBlock +
                                    (wn * FN / 2 + i) * 16 + g * 4;
                    *reinterpret_cast<u32x2*>(row) = u32x2{pack_bf16x2(gate[0], gate[1]),
                                                           pack_bf16x2(gate[2], gate[3])};
                    *reinterpret_cast<u32x2*>(row + I) = u32x2{pack_bf16x2(up[0], up[1]),
                                                               pack_bf16x2(up[2], up[3])};
                }
            }
            top = fmaxf(top, __shfl_xor(top, 16, kWave));
            top = fmaxf(top, __shfl_xor(top, 32, kWave));
            if (g == 0) part[wn][m] = top;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            const int m = (wm * FM + j) * 16 + frow;
            float top = part[0][m];
#pragma unroll
            for (int q = 1; q < WN; ++q) top = fmaxf(top, part[q][m]);
            if (m >= rows) continue;
            const int e = scale_exponent(top);
            const float inv = pow2(-e);
            uint8_t* row = p.h + int64_t(t.row0 + m) * I + tile_n * kScaleBlock + wn * (FN / 2) * 16 +
                           g * 4;
#pragma unroll
            for (int i = 0; i < FN / 2; ++i) {
                const f32x4 v = hv[i][j];
                *reinterpret_cast<uint32_t*>(row + i * 16) =
                    pack_e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
            }
            if (g == 0 && wn == 0)
                p.h_scale[int64_t(t.row0 + m) * (I / kScaleBlock) + tile_n] = uint8_t(e + 127);
        }
    }
}

// Grid for tiles of TM rows and nt n tiles (a multiple of 8, for the XCDs), or
// 0 when a launch cannot hold it; sets p.max_tiles.
uint32_t gemm_grid(GemmArgs& p, int TM, int64_t nt, int threads)
{
    const int64_t mt = p.S / TM + (p.E < p.S ? p.E : p.S);
    p.max_tiles = int(mt);
    const int64_t grid = (mt * nt + 7) / 8 * 8;
    return grid * threads < (int64_t(1) << 31) ? uint32_t(grid) : 0;
}

template <int TN, int TM, int WN, int WM, bool GATED>
hipError_t launch(GemmArgs p, hipStream_t s)
{
    const uint32_t grid = gemm_grid(p, TM, GATED ? p.N / 256 : (p.N + TN - 1) / TN, WN * WM * kWave);
    if (!grid) return hipErrorInvalidConfiguration;
    EP_LAUNCH((expert_gemm_kernel<TN, TM, WN, WM, GATED>), dim3(grid), dim3(WN * WM * kWave), 0, s,
              p);
    return hipGetLastError();
}

template <bool GATED>
hipError_t launch_large(GemmArgs p, hipStream_t s)
{
    // one workgroup a CU (it takes all of the LDS), each with its share of tiles
    uint32_t grid =
        gemm_grid(p, kLargeTile, GATED ? p.N / 256 : (p.N + kLargeTile - 1) / kLargeTile, 1);
    if (!grid) return hipErrorInvalidConfiguration;
    const uint32_t cus = device_cu_count() / 8 * 8;
    grid = grid < cus || cus == 0 ? grid : cus;
    EP_LAUNCH((expert_gemm_large_kernel<GATED>), dim3(grid), dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_expert_gemm(const uint8_t* a, const uint8_t* a_scale, const uint8_t* w,
                              const uint8_t* w_scale, const int32_t* offsets, int S, int N, int K,
                              int E, uint16_t* y, hipStream_t s)
{
    const GemmArgs p{a, a_scale, w, w_scale, offsets, S, N, K, E, 0, y, nullptr, nullptr};
    if (S >= 64 * E) return launch_large<false>(p, s);
    return launch<128, 32, 4, 1, false>(p, s);
}

hipError_t launch_expert_swiglu(const uint8_t* a, const uint8_t* a_scale, const uint8_t* w13,
                                const uint8_t* w13_scale, const int32_t* offsets, int S, int I,
                                int K, int E, uint8_t* h, uint8_t* h_scale, uint16_t* gate_up,
                                hipStream_t s)
{
    const GemmArgs p{a, a_scale, w13, w13_scale, offsets, S, 2 * I, K, E, 0, gate_up, h, h_scale};
    if (S >= 64 * E) return launch_large<true>(p, s);
    return launch<256, 32, 4, 1, true>(p, s);
}

}  // namespace ep
