// moe_tokens.hip -- the whole mixture-of-experts layer for up to 64 tokens, in
// two launches:
//   h[t][j] = w[t][j] silu(G) * U,  [G; U] = W13[e] x[t],  e = idx[t][j]
//   out[t]  = sum_j W2[e] h[t][j]
//
// Bound by the bytes of the picked experts' weights: each is read once,
// whatever the number of tokens that picked it, by streaming 16 rows at a time
// straight into registers as the matrix instruction's row operand, with the
// tokens as its columns.  8-bit weights become bf16 times their block's power
// of two on the way (exact); h is kept as two bf16 halves (16 bits of
// mantissa), so that no step rounds to fewer bits than the products need.
//
// First launch: one workgroup per (pick, 16 outputs of I); the first pick of
// an expert works for all tokens that picked it, the others leave at once.
// Its waves split H and join in LDS.  Second launch: one workgroup per 16
// outputs of H; its waves split the picked experts and join in LDS in a fixed
// order -- no atomics, the same result on every call.
#include "experts_internal.h"

namespace ep {
namespace {

constexpr int kUpWaves = 4;       // first launch: waves that split H
constexpr int kDownWaves = 8;     // second launch: waves that split the experts
constexpr int kStep = 128;        // k values per step: 32 of one row in each lane

struct MoeArgs {
    const uint16_t* x;
    const int32_t* idx;
    const float* topk_w;
    int T, H, I, E, k;
    const uint8_t* w13;
    const uint8_t* s13;
    const uint8_t* w2;
    const uint8_t* s2;
    uint16_t* out;
    uint16_t* h_hi;      // [T*k][I]
    uint16_t* h_lo;      // [T*k][I]
    int32_t* pick_of;    // [T*k][64]: for an expert's first pick p, the pick of
                         //            token t that carries h, or -1; [p][0] = -2:
                         //            p is no expert's first pick
};

// 32 consecutive k values of one row: 32 bytes (e4m3) or 64 (bf16).
template <bool FP8>
struct Run {
    u32x4 v[FP8 ? 2 : 4];
};

// Loads the 32 values at column c of a row of n (n % 16 == 0); zeros past it.
template <bool FP8>
__device__ __forceinline__ Run<FP8> load_run(const uint8_t* __restrict__ row, int c, int n) {
    Run<FP8> r;
    constexpr int kVec = FP8 ? 16 : 8;       // values per 16-byte vector
#pragma unroll
    for (int i = 0; i < (FP8 ? 2 : 4); ++i) {
        r.v[i] = u32x4{0, 0, 0, 0};
        if (c + i * kVec < n) r.v[i] = load16_nt(row + (c + i * kVec) * (FP8 ? 1 : 2));
    }
    return r;
}

// Values 8 i .. 8 i + 7 of a run as a bf16 operand, times the block's scale.
template <bool FP8>
__device__ __forceinline__ bf16x8 run_operand(const Run<FP8>& r, int i, float scale) {
    if constexpr (FP8) {
        u32x4 o;
#pragma unroll
        for (int d = 0; d < 2; ++d) {
            const uint32_t v = r.v[i / 2][(i % 2) * 2 + d];
            o[2 * d] = __builtin_bit_cast(
                uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, scale, false));
            o[2 * d + 1] = __builtin_bit_cast(
                uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, scale, true));
        }
        return __builtin_bit_cast(bf16x8, o);
    } else {
        return __builtin_bit_cast(bf16x8, r.v[i]);
    }
}

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// ---------------------------------------------------------------- gate and up
template <bool FP8, int CT>
__device__ __forceinline__ void up_body(const MoeArgs& p, int e, int n0, int m,
                                        const uint8_t* token_of, float* weight_of,
                                        const int* pick_of, f32x4* red)
{
    const int lane = lane_id(), l = lane % 16, g = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int H = p.H, I = p.I, HB = scale_blocks(H);
    constexpr int kBytes = FP8 ? 1 : 2;
    const uint8_t* gate = p.w13 + (int64_t(e) * 2 * I + n0 + l) * H * kBytes;
    const uint8_t* up = gate + int64_t(I) * H * kBytes;
    const uint8_t* gs = nullptr;
    const uint8_t* us = nullptr;
    if (FP8) {
        gs = p.s13 + (int64_t(e) * scale_blocks(2 * I) + n0 / kScaleBlock) * HB;
        us = gs + int64_t(I / kScaleBlock) * HB;
    }
    const uint16_t* xr[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) {
        const int col = c * 16 + l;
        xr[c] = p.x + int64_t(token_of[col < m ? col : 0]) * H;
    }
    f32x4 ag[CT], au[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) ag[c] = au[c] = f32x4{0, 0, 0, 0};

    const int steps = (H + kStep - 1) / kStep;
    const int per = (steps + kUpWaves - 1) / kUpWaves;
    const int first = wave * per, last = first + per < steps ? first + per : steps;
    // weights run kAhead steps ahead of their use
    constexpr int kAhead = FP8 ? 4 : 2;
    Run<FP8> bg[kAhead], bu[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
        const int c = (first + a) * kStep + g * 32;
        bg[a] = load_run<FP8>(gate, c, first + a < last ? H : 0);
        bu[a] = load_run<FP8>(up, c, first + a < last ? H : 0);
    }
    for (int s0 = first; s0 < last; s0 += kAhead) {
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            const int s = s0 + a;
            if (s >= last) break;
            const int c = s * kStep + g * 32;
            const Run<FP8> wg = bg[a], wu = bu[a];
            const int next = s + kAhead;
            bg[a] = load_run<FP8>(gate, next * kStep + g * 32, next < last ? H : 0);
            bu[a] = load_run<FP8>(up, next * kStep + g * 32, next < last ? H : 0);
            const float sg = FP8 ? pow2(int(gs[s]) - 127) : 1.0f;
            const float su = FP8 ? pow2(int(us[s]) - 127) : 1.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bf16x8 a_g = run_operand<FP8>(wg, i, sg);
                const bf16x8 a_u = run_operand<FP8>(wu, i, su);
#pragma unroll
                for (int t = 0; t < CT; ++t) {
                    u32x4 xv = {0, 0, 0, 0};
                    if (c + i * 8 < H) xv = load16(xr[t] + c + i * 8);
                    const bf16x8 b = __builtin_bit_cast(bf16x8, xv);
                    ag[t] = mfma(a_g, b, ag[t]);
                    au[t] = mfma(a_u, b, au[t]);
                }
            }
        }
    }
    // join the waves' parts of H: wave w sums column tiles w, w + kUpWaves, ..
#pragma unroll
    for (int t = 0; t < CT; ++t) {
        red[((wave * CT + t) * 2 + 0) * kWave + lane] = ag[t];
        red[((wave * CT + t) * 2 + 1) * kWave + lane] = au[t];
    }
    __syncthreads();
    for (int t = wave; t < CT; t += kUpWaves) {
        f32x4 sg = red[(t * 2 + 0) * kWave + lane], su = red[(t * 2 + 1) * kWave + lane];
#pragma unroll
        for (int w = 1; w < kUpWaves; ++w) {
            const f32x4 vg = red[((w * CT + t) * 2 + 0) * kWave + lane];
            const f32x4 vu = red[((w * CT + t) * 2 + 1) * kWave + lane];
#pragma unroll
            for (int c = 0; c < 4; ++c) { sg[c] += vg[c]; su[c] += vu[c]; }
        }
        const int col = t * 16 + l;
        if (col >= m) continue;
        const float w = weight_of[col];
        float hi[4], lo[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float h = w * (sg[c] * sigmoid(sg[c]) * su[c]);
            hi[c] = bf16_lo(pack_bf16x2(h, 0.0f));
            lo[c] = h - hi[c];
        }
        const int64_t at = int64_t(pick_of[col]) * I + n0 + g * 4;
        *reinterpret_cast<u32x2*>(p.h_hi + at) =
            u32x2{pack_bf16x2(hi[0], hi[1]), pack_bf16x2(hi[2], hi[3])};
        *reinterpret_cast<u32x2*>(p.h_lo + at) =
            u32x2{pack_bf16x2(lo[0], lo[1]), pack_bf16x2(lo[2], lo[3])};
    }
}

template <bool FP8>
__global__ __launch_bounds__(kUpWaves* kWave) void moe_up_kernel(MoeArgs p)
{
    __shared__ uint8_t token_of[kMoeMaxTokens];
    __shared__ float weight_of[kMoeMaxTokens];
    __shared__ int pick_of[kMoeMaxTokens];
    __shared__ f32x4 red[kUpWaves * 4 * 2 * kWave];
    const int pick = blockIdx.y, chunk = blockIdx.x;
    const int lane = lane_id();
    const int e = p.idx[pick];
    // lane t looks for e among token t's picks: the first pick that has it
    // carries the row, with the weights of all that have it (each counted once)
    int mine = -1;
    float w = 0.0f;
    if (lane < p.T && unsigned(e) < unsigned(p.E)) {
        for (int j = 0; j < p.k; ++j) {
            if (p.idx[lane * p.k + j] != e) continue;
            if (mine < 0) mine = lane * p.k + j;
            w += p.topk_w[lane * p.k + j];
        }
    }
    const uint64_t has = ballot(mine >= 0);
    const bool leads = has && __builtin_amdgcn_readlane(mine, __builtin_ctzll(has)) == pick;
    if (!leads) {
        if (chunk == 0 && threadIdx.x == 0) p.pick_of[int64_t(pick) * kMoeMaxTokens] = -2;
        return;
    }
    if (threadIdx.x < kWave) {
        if (chunk == 0) p.pick_of[int64_t(pick) * kMoeMaxTokens + lane] = mine;
        if (mine >= 0) {
            const int c = popc64(has & lanes_below());
            token_of[c] = uint8_t(lane);
            weight_of[c] = w;
            pick_of[c] = mine;
        }
    }
    __syncthreads();
    const int m = popc64(has), n0 = chunk * 16;
    if (m <= 16) up_body<FP8, 1>(p, e, n0, m, token_of, weight_of, pick_of, red);
    else if (m <= 32) up_body<FP8, 2>(p, e, n0, m, token_of, weight_of, pick_of, red);
    else up_body<FP8, 4>(p, e, n0, m, token_of, weight_of, pick_of, red);
}

// ---------------------------------------------------------------- down
// CT column tiles of 16 tokens.
template <bool FP8, int CT>
__global__ __launch_bounds__(kDownWaves* kWave) void moe_down_kernel(MoeArgs p)
{
    __shared__ int leaders[kMoeMaxTokens * kMaxK];
    __shared__ int count;
    __shared__ f32x4 red[kDownWaves * CT * kWave];
    const int lane = lane_id(), l = lane % 16, g = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int H = p.H, I = p.I, IB = scale_blocks(I), n0 = int(blockIdx.x) * 16;
    constexpr int kBytes = FP8 ? 1 : 2;
    if (wave == 0) {
        int n = 0;
        for (int base = 0; base < p.T * p.k; base += kWave) {
            const int q = base + lane;
            const bool lead = q < p.T * p.k && p.pick_of[int64_t(q) * kMoeMaxTokens] != -2;
            const uint64_t b = ballot(lead);
            if (lead) leaders[n + popc64(b & lanes_below())] = q;
            n += popc64(b);
        }
        if (lane == 0) count = n;
    }
    __syncthreads();
    const int units = __builtin_amdgcn_readfirstlane(count);

    f32x4 acc[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) acc[c] = f32x4{0, 0, 0, 0};
    const int steps = (I + kStep - 1) / kStep;
    for (int u = wave; u < units; u += kDownWaves) {
        const int lead = __builtin_amdgcn_readfirstlane(leaders[u]);
        const int e = p.idx[lead];
        const uint8_t* row = p.w2 + (int64_t(e) * H + n0 + l) * I * kBytes;
        const uint8_t* sc = FP8 ? p.s2 + (int64_t(e) * scale_blocks(H) + n0 / kScaleBlock) * IB
                                : nullptr;
        int from[CT];
        uint64_t any[CT];
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            const int t = c * 16 + l;
            from[c] = t < p.T ? p.pick_of[int64_t(lead) * kMoeMaxTokens + t] : -1;
            any[c] = ballot(from[c] >= 0);
        }
        // an expert's part is summed apart and added for its own tokens only: a
        // NaN or infinite weight reaches no token that did not pick it
        f32x4 part[CT];
#pragma unroll
        for (int c = 0; c < CT; ++c) part[c] = f32x4{0, 0, 0, 0};
        constexpr int kAhead = FP8 ? 4 : 2;
        Run<FP8> b[kAhead];
#pragma unroll
        for (int a = 0; a < kAhead; ++a)
            b[a] = load_run<FP8>(row, a * kStep + g * 32, a < steps ? I : 0);
        for (int s0 = 0; s0 < steps; s0 += kAhead) {
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                const int s = s0 + a;
                if (s >= steps) break;
                const int c0 = s * kStep + g * 32;
                const Run<FP8> w = b[a];
                const int next = s + kAhead;
                b[a] = load_run<FP8>(row, next * kStep + g * 32, next < steps ? I : 0);
                const float scale = FP8 ? pow2(int(sc[s]) - 127) : 1.0f;
                bf16x8 op[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) op[i] = run_operand<FP8>(w, i, scale);
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    if (!any[c]) continue;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        u32x4 hi = {0, 0, 0, 0}, lo = {0, 0, 0, 0};
                        if (from[c] >= 0 && c0 + i * 8 < I) {
                            const int64_t at = int64_t(from[c]) * I + c0 + i * 8;
                            hi = load16(p.h_hi + at);
                            lo = load16(p.h_lo + at);
                        }
                        part[c] = mfma(op[i], __builtin_bit_cast(bf16x8, hi), part[c]);
                        part[c] = mfma(op[i], __builtin_bit_cast(bf16x8, lo), part[c]);
                    }
                }
            }
        }
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[c][i] += from[c] >= 0 ? part[c][i] : 0.0f;
    }
#pragma unroll
    for (int c = 0; c < CT; ++c) red[(wave * CT + c) * kWave + lane] = acc[c];
    __syncthreads();
    for (int c = wave; c < CT; c += kDownWaves) {
        f32x4 s = red[c * kWave + lane];
#pragma unroll
        for (int w = 1; w < kDownWaves; ++w) {
            const f32x4 v = red[(w * CT + c) * kWave + lane];
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i] += v[i];
        }
        const int t = c * 16 + l;
        if (t < p.T)
            *reinterpret_cast<u32x2*>(p.out + int64_t(t) * H + n0 + g * 4) =
                u32x2{pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3])};
    }
}

template <bool FP8>
hipError_t launch(const MoeArgs& p, hipStream_t s)
{
    EP_LAUNCH((moe_up_kernel<FP8>), dim3(uint32_t(p.I / 16), uint32_t(p.T * p.k)),
              dim3(kUpWaves * kWave), 0, s, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const dim3 grid(uint32_t(p.H / 16)), block(kDownWaves * kWave);
    if (p.T <= 16) EP_LAUNCH((moe_down_kernel<FP8, 1>), grid, block, 0, s, p);
    else if (p.T <= 32) EP_LAUNCH((moe_down_kernel<FP8, 2>), grid, block, 0, s, p);
    else EP_LAUNCH((moe_down_kernel<FP8, 4>), grid, block, 0, s, p);
    return hipGetLastError();
}

}  // namespace

size_t moe_tokens_workspace(int T, int k, int I)
{
    const size_t picks = size_t(T) * k;
    return 2 * align256(picks * I * 2) + align256(picks * kMoeMaxTokens * sizeof(int32_t));
}

hipError_t launch_moe_tokens(const uint16_t* x, const int32_t* idx, const float* topk_w, int T,
                             int H, int I, int E, int k, const void* w13, const uint8_t* w13_scale,
                             const void* w2, const uint8_t* w2_scale, uint16_t* out, void* ws,
                             hipStream_t s)
{
    char* base = static_cast<char*>(ws);
    const size_t half = align256(size_t(T) * k * I * 2);
    const MoeArgs p{x, idx, topk_w, T, H, I, E, k,
                    static_cast<const uint8_t*>(w13), w13_scale,
                    static_cast<const uint8_t*>(w2), w2_scale, out,
                    reinterpret_cast<uint16_t*>(base), reinterpret_cast<uint16_t*>(base + half),
                    reinterpret_cast<int32_t*>(base + 2 * half)};
    return w13_scale ? launch<true>(p, s) : launch<false>(p, s);
}

}  // namespace ep
