// expert_gemm.hip -- grouped block-scaled FP8 products over expert segments.
//
// For a row s of expert e:  y[s][n] = sum_b 2^(as[s][b] + ws[n/128][b] - 254)
//                                     sum_{k in block b} a[s][k] w[e][n][k].
// The scales are powers of two for blocks of 128 along k, so the matrix
// instruction takes them as operands and the f32 accumulators never leave the
// matrix core's registers: no multiply-add per block on the vector ALU.  The
// weights are its row operand: a lane then holds four neighbouring n of one
// token.  (The unit adds eight neighbouring products at a time, each cut towards zero
// at 2^-13 of the largest one's power of two, and goes on in f32: results of values
// with an ordinary spread are 1.6e-5 of their terms' magnitude off the exact sum, for
// one block as for many; of h some 0.16% of the values then round to their e4m3
// neighbour.  Products of bf16, summed in f32, keep them, but take 64 us instead of 52
// gated, 8 experts x 4096 x 7168, 32 rows each.)
//
// Segments of many rows are bound by matrix work and take the kernel of
// expert_gemm_large.h; the one here is for few rows, where the weights' bytes
// bound it.  (Times of a step are those before and after it; the present ones stand
// with the rules in expert_choice.h.)
#include "expert_choice.h"
#include "expert_gemm_large.h"

namespace ep {
namespace {

// A workgroup makes ROWS weight rows a wave (gated: 16 gate rows and their 16 up
// rows; eight waves make one scale block) x up to TM tokens.  Each wave brings its
// own rows, and its share of the tokens that all waves use, through LDS by direct
// loads kDepth - 1 steps of 128 k ahead, counted by one wait a step, since loads
// return in order.  (Straight into registers in the matrix instruction's order,
// neighbouring lanes are rows apart and every lane of a load is a request of its
// own: 8 experts x 4096 x 7168, eight rows each, 65 us instead of 44.)
template <int TM, int WAVES, int ROWS, bool GATED, bool NT>
__global__ __launch_bounds__(WAVES* kWave) void expert_gemm_stream_kernel(GemmArgs p)
{
    constexpr int kDepth = 3, kBK = kScaleBlock, TN = ROWS * WAVES, NF = ROWS / 16;
    // every wave loads whole 1 KB pieces of the tokens (rows past TM are zeros)
    constexpr int kXRows = TM > 8 * WAVES ? TM : 8 * WAVES;
    constexpr int FM = TM / 16, kXLoads = kXRows / 8 / WAVES, kWStage = ROWS * kBK;
    constexpr int kXStage = kXRows * kBK;
    static_assert(!GATED || (TN == 256 && ROWS == 32), "a gated tile makes one scale block");
    constexpr int kOps = ROWS / 8 + kXLoads;               // loads of one step
    constexpr int kPitch = 68;                      // 64 scale bytes of a token, padded
    __shared__ __attribute__((aligned(256)))
    uint8_t lds[kDepth * (WAVES * kWStage + kXStage) + TM * kPitch];
    uint8_t* const xstage = lds + kDepth * WAVES * kWStage;
    uint8_t* const scales = xstage + kDepth * kXStage;

    const int lane = lane_id(), l = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int N = p.N, K = p.K, KB = scale_blocks(K), NB = scale_blocks(N);
    const GemmTile tile = GemmTiles(p, TM, GATED ? N / 256 : (N + TN - 1) / TN).at(p, TM, 0);
    const RowTile t = tile.rows;
    if (t.expert < 0) return;
    const int rows = t.end - t.row0 < TM ? t.end - t.row0 : TM;
    const int used = (rows + 15) / 16;              // column tiles that hold tokens
    uint8_t* const wstage = lds + wave * kDepth * kWStage;

    // LDS rows of 128 bytes, chunk c of row r at c ^ r / 2 % 8; a load instruction
    // fills 8 rows
    const int lrow = lane / 8, wchunk[2] = {(lane & 7) ^ (lane >> 4), (lane & 7) ^ (4 + (lane >> 4))};
    const int64_t first = int64_t(tile.n) * (GATED ? TN / 2 : TN);
    const int64_t wrows = GATED ? N - first : (N - first < TN ? N - first : TN);
    const __amdgpu_buffer_rsrc_t wr = buffer_rsrc(
        const_cast<uint8_t*>(p.w) + (int64_t(t.expert) * N + first) * K, wrows * K);
    const uint32_t woff = uint32_t((GATED ? wave * 16 : wave * ROWS) + lrow) * uint32_t(K);
    const uint32_t whalf = uint32_t(GATED ? N / 2 : 16) * uint32_t(K);     // to the second fragment
    int block = GATED ? tile.n : (int(first) + wave * ROWS) / kScaleBlock;
    block = block < NB ? block : NB - 1;
    const uint8_t* const wsc = p.w_scale + (int64_t(t.expert) * NB + block) * KB;

    const __amdgpu_buffer_rsrc_t xr =
        buffer_rsrc(const_cast<uint8_t*>(p.a) + int64_t(t.row0) * K, int64_t(rows) * K);
    const int xchunk = wchunk[wave & 1];
    const uint32_t xoff = uint32_t(wave * 8 + lrow) * uint32_t(K);
    const __amdgpu_buffer_rsrc_t xsr =
        buffer_rsrc(const_cast<uint8_t*>(p.a_scale) + int64_t(t.row0) * KB, int64_t(rows) * KB);

    // Steps go round from one that differs between the weights' tiles: all of them at
    // the same k of rows 4096 bytes apart would keep to a few memory channels (64
    // experts x 1024 x 4096, four rows each: 69 us, 47).
    const int turn = (t.expert * 5 + tile.n * 3) % KB;
    auto block_of = [&](int step) {
        const int s = step + turn;
        return s < KB ? s : s - KB;
    };
    // Scale bytes of 64 steps: the weights' one in each lane, the tokens' in LDS (a
    // row's are neighbours: a lane each, where a load for each step would touch a
    // line for each token).
    int ws[GATED ? 2 : 1];
    auto load_scales = [&](int step, auto&& meanwhile) {
        const int b = block_of(step + lane < KB ? step + lane : 0);
#pragma unroll
        for (int i = 0; i < (GATED ? 2 : 1); ++i) ws[i] = wsc[int64_t(i) * (NB / 2) * KB + b];
        int v[TM / WAVES];
#pragma unroll
        for (int i = 0; i < TM / WAVES; ++i)
            v[i] = __builtin_amdgcn_raw_buffer_load_b8(xsr, (wave * (TM / WAVES) + i) * KB + b, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
        meanwhile();
#pragma unroll
        for (int i = 0; i < TM / WAVES; ++i)
            scales[(wave * (TM / WAVES) + i) * kPitch + lane] = uint8_t(v[i]);
    };
    auto load = [&](int step, int d) {
        const int k = step < KB ? block_of(step) * kBK : K;
#pragma unroll
        for (int i = 0; i < ROWS / 8; ++i) {
            const int kc = k + wchunk[i & 1] * 16;
            const uint32_t row = (i & 1) * 8 * uint32_t(K) + (i >> 1) * whalf;
            load16_to_lds<NT>(wr, wstage + d * kWStage + i * 1024,
                          kc < K ? woff + row + uint32_t(kc) : kOutside);
        }
#pragma unroll
        for (int i = 0; i < kXLoads; ++i) {
            const int kc = k + xchunk * 16;
            load16_to_lds<false>(xr, xstage + d * kXStage + (i * WAVES + wave) * 1024,
                          kc < K ? xoff + uint32_t(i * WAVES * 8) * uint32_t(K) + uint32_t(kc)
                                 : kOutside);
        }
        __builtin_amdgcn_sched_barrier(0);
    };

    f32x4 acc[NF][FM];
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    // lane: row r, chunks g and 4 + g
    auto fragment = [&](const uint8_t* stage, int r) {
        const u32x4 lo = load16(stage + r * kBK + ((g ^ ((r >> 1) & 7)) * 16));
        const u32x4 hi = load16(stage + r * kBK + (((4 + g) ^ ((r >> 1) & 7)) * 16));
        return i32x8{int(lo[0]), int(lo[1]), int(lo[2]), int(lo[3]),
                     int(hi[0]), int(hi[1]), int(hi[2]), int(hi[3])};
    };

    load_scales(0, [&] {
#pragma unroll
        for (int d = 0; d < kDepth - 1; ++d) load(d, d);
    });
    for (int s0 = 0; s0 < KB; s0 += kDepth) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {                // past the last step: zeros
            // step s0 + d has landed for every wave, the step before has been read
            wait_and_barrier<(kDepth - 2) * kOps>();
            __builtin_amdgcn_sched_barrier(0);
            const int s = s0 + d;
            if ((s & 63) == 0 && s > 0 && s < KB) {
                load_scales(s, [] {});
                __syncthreads();
            }
            load(s + kDepth - 1, (d + kDepth - 1) % kDepth);
            int wscale[2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                wscale[i] = __builtin_amdgcn_readlane(ws[GATED ? i : 0], s & 63);
            const uint8_t* const ws_now = wstage + d * kWStage;
            const i32x8 w0 = fragment(ws_now, l), w1 = fragment(ws_now, ROWS - 16 + l);
#pragma unroll
            for (int j = 0; j < FM; ++j) {
                if (j >= used) break;
                const int r = j * 16 + l;
                const i32x8 x = fragment(xstage + d * kXStage, r);
                const int scale = scales[r * kPitch + (s & 63)];
                acc[0][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    w0, x, acc[0][j], 0, 0, 0, wscale[0], 0, scale);
                if (NF > 1) acc[NF - 1][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    w1, x, acc[NF - 1][j], 0, 0, 0, wscale[1], 0, scale);
            }
        }
    }
    wait_and_barrier<0>();          // every stage has been read, no load is on its way

    if constexpr (!GATED) {
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            const int m = j * 16 + l;
            if (m >= rows) continue;
            uint16_t* row = p.y + int64_t(t.row0 + m) * N;
#pragma unroll
            for (int i = 0; i < NF; ++i) {
                const int n = int(first) + wave * ROWS + i * 16 + g * 4;
                if (n >= N) continue;
                *reinterpret_cast<u32x2*>(row + n) =
                    u32x2{pack_bf16x2(acc[i][j][0], acc[i][j][1]),
                          pack_bf16x2(acc[i][j][2], acc[i][j][3])};
            }
        }
    } else {
        float* const part = reinterpret_cast<float*>(lds);        // [WAVES][TM]
        const int I = N / 2;
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            const int m = j * 16 + l;
            const f32x4 gate = acc[0][j], up = acc[NF - 1][j];
            if (p.y && m < rows) {
                uint16_t* row = p.y + int64_t(t.row0 + m) * N + int(first) + wave * 16 + g * 4;
                *reinterpret_cast<u32x2*>(row) = u32x2{pack_bf16x2(gate[0], gate[1]),
                                                       pack_bf16x2(gate[2], gate[3])};
                *reinterpret_cast<u32x2*>(row + I) = u32x2{pack_bf16x2(up[0], up[1]),
                                                           pack_bf16x2(up[2], up[3])};
            }
            float top = 0.0f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float v = gate[c] * sigmoid(gate[c]) * up[c];
                acc[0][j][c] = v;
                top = max_finite(top, v);
            }
            top = fmaxf(top, __shfl_xor(top, 16, kWave));
            top = fmaxf(top, __shfl_xor(top, 32, kWave));
            if (g == 0) part[wave * TM + m] = top;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < FM; ++j) {
            const int m = j * 16 + l;
            float top = part[m];
#pragma unroll
            for (int q = 1; q < WAVES; ++q) top = fmaxf(top, part[q * TM + m]);
            if (m >= rows) continue;
            const int e = scale_exponent(top);
            const float inv = pow2(-e);
            const f32x4 v = acc[0][j];
            *reinterpret_cast<uint32_t*>(p.h + int64_t(t.row0 + m) * I + int(first) + wave * 16 +
                                         g * 4) =
                pack_e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
            if (g == 0 && wave == 0)
                p.h_scale[int64_t(t.row0 + m) * (I / kScaleBlock) + tile.n] = uint8_t(e + 127);
        }
    }
}

template <int TM, int WAVES, int ROWS, bool GATED>
hipError_t launch_stream(GemmArgs p, hipStream_t s)
{
    const uint32_t grid = gemm_tiles(p, TM, ROWS * WAVES);
    if (!grid || uint64_t(grid) * WAVES * kWave >= (uint64_t(1) << 31))
        return hipErrorInvalidConfiguration;
    const dim3 block(WAVES * kWave);
    if (int64_t(p.E) * p.N * p.K > kStreamBytes)
        EP_LAUNCH((expert_gemm_stream_kernel<TM, WAVES, ROWS, GATED, true>), dim3(grid), block, 0, s, p);
    else
        EP_LAUNCH((expert_gemm_stream_kernel<TM, WAVES, ROWS, GATED, false>), dim3(grid), block, 0, s, p);
    return hipGetLastError();
}

template <bool GATED>
hipError_t launch_large(GemmArgs p, hipStream_t s)
{
    // one workgroup a CU (it takes all of the LDS), each with its share of tiles
    uint32_t grid = gemm_tiles(p, kLargeTile, kLargeTile);
    if (!grid) return hipErrorInvalidConfiguration;
    const uint32_t cus = device_cu_count() / 8 * 8;
    grid = grid < cus || cus == 0 ? grid : cus;
    if (GATED && p.y)
        EP_LAUNCH((expert_gemm_large_kernel<GATED, GATED>), dim3(grid), dim3(256), 0, s, p);
    else
        EP_LAUNCH((expert_gemm_large_kernel<GATED, false>), dim3(grid), dim3(256), 0, s, p);
    return hipGetLastError();
}

template <bool GATED>
hipError_t launch(const GemmArgs& p, hipStream_t s)
{
    const GemmKernel kernel = choose_gemm(p.S, p.N, p.E, GATED, device_cu_count());
    switch (kernel) {
        case kGemmLarge: return launch_large<GATED>(p, s);
        case kGemm128x256: return launch_stream<128, 8, 32, GATED>(p, s);
        case kGemm64x256: return launch_stream<64, 8, 32, GATED>(p, s);
        case kGemm32x256: return launch_stream<32, 8, 32, GATED>(p, s);
        default: break;
    }
    if constexpr (!GATED) {
        switch (kernel) {
            case kGemm128x128: return launch_stream<128, 4, 32, false>(p, s);
            case kGemm64x128: return launch_stream<64, 4, 32, false>(p, s);
            case kGemm32x64: return launch_stream<32, 4, 16, false>(p, s);
            default: break;
        }
    }
    return hipErrorInvalidConfiguration;
}

}  // namespace

hipError_t launch_expert_gemm(const uint8_t* a, const uint8_t* a_scale, const uint8_t* w,
                              const uint8_t* w_scale, const int32_t* offsets, int S, int N, int K,
                              int E, uint16_t* y, hipStream_t s)
{
    return launch<false>(
        GemmArgs{a, a_scale, w, w_scale, offsets, S, N, K, E, 0, y, nullptr, nullptr}, s);
}

hipError_t launch_expert_swiglu(const uint8_t* a, const uint8_t* a_scale, const uint8_t* w13,
                                const uint8_t* w13_scale, const int32_t* offsets, int S, int I,
                                int K, int E, uint8_t* h, uint8_t* h_scale, uint16_t* gate_up,
                                hipStream_t s)
{
    return launch<true>(GemmArgs{a, a_scale, w13, w13_scale, offsets, S, 2 * I, K, E, 0, gate_up, h,
                                 h_scale}, s);
}

}  // namespace ep
