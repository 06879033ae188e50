// moe_tokens.hip -- the whole mixture-of-experts layer for up to 64 tokens, in
// two launches:
//   h[t][j] = w[t][j] silu(G) * U,  [G; U] = W13[e] x[t],  e = idx[t][j]
//   out[t]  = sum_j W2[e] h[t][j]
//
// Bound by the bytes of the picked experts' weights: each is read once for up to 32
// (first launch) or 8 (second) tokens that picked it, 16 rows at a time as the
// matrix instruction's row operand, with the tokens as its columns.  8-bit weights
// become bf16 times their block's power of two on the way (exact for 2^-117 to
// 2^119); h is kept as two bf16 halves (16 bits of mantissa), two columns of the
// second launch's product, so that no step rounds to fewer bits than the products
// need.
//
// First launch: one workgroup per (picked expert, 16 outputs of I), which finds
// its expert from the picks alone.  Its waves split H and join in LDS.  Second
// launch: one workgroup per 16 outputs of H; its waves take the picked experts in
// turn, each adding to sums of its own in LDS, which are joined in a fixed order
// -- the same result on every call.
//
// Weights and activations go through LDS by direct loads, each wave's own stages, a
// few steps of 128 k ahead: loads return in order, so one counted wait a step covers
// them, and no wave waits for another.  Weights that are read once go past the
// caches when there are many (one token 58 us instead of 64, 32 tokens 613 instead
// of 664).
#include "experts_internal.h"

namespace ep {
namespace {

constexpr int kUpWaves = 4;       // first launch: waves that split H
constexpr int kStep = 128;        // k values per step: 32 of one row in each lane
constexpr float kBf16Max = 0x1.fep127f;

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
    uint16_t* h;         // [2][T*k][I]: high halves, then low ones
    int32_t* units;      // [kHead + n * kUnit]: n, the number of experts picked; then for
                         //   each (in the order of their ids) the expert, the number m
                         //   of its tokens, and their picks that carry h
};
constexpr int kHead = 8, kUnit = 2 + kMoeMaxTokens;
constexpr int kMaxWords = kMaxE / 32;

// 16 rows of weights x 128 k in LDS, as they lie in memory: rows of 128 bytes
// (e4m3) or 256 (bf16) in chunks of 16, chunk c of row r at c ^ swizzle(r), so that
// 16 rows' reads of one chunk touch every bank once.  A load instruction fills 1 KB
// of neighbouring chunks: its lanes' requests join to whole lines.  (Loaded
// straight into registers in the matrix instruction's order, neighbouring lanes are
// rows apart and every lane is a request of its own: one token 68 us, 32 tokens
// 673.)
template <bool FP8>
struct Rows {
    static constexpr int kRow = FP8 ? 128 : 256, kBytes = 16 * kRow, kLoads = kBytes / 1024;
    static constexpr int kPerLoad = 1024 / kRow;                 // rows of one load
    __device__ __forceinline__ static int64_t bytes(int n) { return int64_t(16) * n * (FP8 ? 1 : 2); }
    __device__ __forceinline__ static int swizzle(int r) { return FP8 ? (r >> 1) & 7 : r & 15; }
    // r: the 16 rows of n values; zeros from k value n on
    template <bool NT>
    __device__ __forceinline__ static void load(__amdgpu_buffer_rsrc_t r, uint8_t* to, int step,
                                                int n, int width, int lane) {
        constexpr int kChunks = kRow / 16;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int row = i * kPerLoad + lane / kChunks;
            const int k = step * kStep + ((lane % kChunks) ^ swizzle(row)) * (FP8 ? 16 : 8);
            load16_to_lds<NT>(r, to + i * 1024,
                                  k < n ? (uint32_t(row) * uint32_t(width) + uint32_t(k)) * (FP8 ? 1u : 2u)
                                    : kOutside);
        }
    }
    // Operands of the four matrix instructions of a step, times the block's scale:
    // row l, and of instruction i the eight values from k = 32 g + 8 i (e4m3) or
    // 32 i + 8 g on.
    __device__ __forceinline__ static void operands(const uint8_t* from, int lane, float scale,
                                                    bf16x8 (&o)[4]) {
        const int l = lane & 15, g = lane >> 4;
        const uint8_t* row = from + l * kRow;
        if constexpr (FP8) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const u32x4 v = load16(row + (((2 * g + c) ^ swizzle(l)) * 16));
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    u32x4 b;
#pragma unroll
                    for (int d = 0; d < 2; ++d) {
                        const uint32_t q = v[2 * h + d];
                        b[2 * d] = __builtin_bit_cast(
                            uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q, scale, false));
                        b[2 * d + 1] = __builtin_bit_cast(
                            uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q, scale, true));
                    }
                    o[2 * c + h] = __builtin_bit_cast(bf16x8, b);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[i] = __builtin_bit_cast(bf16x8, load16(row + (((4 * i + g) ^ swizzle(l)) * 16)));
        }
    }
};
template <bool FP8>
__device__ __forceinline__ constexpr int operand_k(int i, int g) {
    return FP8 ? g * 32 + i * 8 : i * 32 + g * 8;
}

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Waits until at most VM vector-memory operations of this wave and none of its
// LDS reads are outstanding.
template <int VM>
__device__ __forceinline__ void wait_loads() {
    static_assert(VM < 64, "the counter's range");
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt((VM & 15) | (7 << 4) | ((VM >> 4) << 14));
    __builtin_amdgcn_sched_barrier(0);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// C columns (rows of activations) x 128 k of bf16 in LDS: 256 bytes a column, its
// chunk c of 16 bytes at c ^ column % 16, so that 16 columns' reads of one chunk
// touch every bank once.  A load instruction fills four columns.
template <int C>
struct Columns {
    static constexpr int kLoads = C / 4, kBytes = C * 256, kTiles = (C + 15) / 16;
    uint32_t at[kLoads];      // byte offset of the lane's column in the source
    int chunk[kLoads];        // the lane's chunk

    // row_of(c): the source row of column c
    template <class F>
    __device__ __forceinline__ void init(int lane, uint32_t row_bytes, F row_of) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int c = i * 4 + lane / 16;
            at[i] = uint32_t(row_of(c)) * row_bytes;
            chunk[i] = (lane & 15) ^ (c & 15);
        }
    }
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint8_t* to, int step, int n) const {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int k = step * kStep + chunk[i] * 8;
            load16_to_lds<false>(r, to + i * 1024, k < n ? at[i] + uint32_t(k) * 2u : kOutside);
        }
    }
    // operand i (of 4) of column tile t: the lane's column l (fewer than 16: again
    // from the first)
    template <bool FP8>
    __device__ __forceinline__ static bf16x8 operand(const uint8_t* from, int t, int i, int lane) {
        const int c = C < 16 ? (lane & (C - 1)) : t * 16 + (lane & 15), g = lane >> 4;
        return __builtin_bit_cast(bf16x8, load16(from + c * 256 + ((operand_k<FP8>(i, g) / 8 ^ (c & 15)) * 16)));
    }
};

// Scale bytes of 64 steps, one in each lane.
struct Scales {
    const uint8_t* from;
    int count, value;
    __device__ __forceinline__ void fill(int step) {
        const int s = (step & ~63) + lane_id();
        value = from[s < count ? s : count - 1];
    }
    __device__ __forceinline__ float at(int step) const {
        return pow2(__builtin_amdgcn_readlane(value, step & 63) - 127);
    }
};

// ---------------------------------------------------------------- gate and up
// Bytes of one wave's stages: gate rows, up rows, and C columns of activations.
template <bool FP8, int C>
constexpr int up_stage() { return 2 * Rows<FP8>::kBytes + Columns<C>::kBytes; }
// As many as leave room for two workgroups a CU.
constexpr int up_stages(bool fp8, int C) { return C <= 4 ? (fp8 ? 3 : 2) : C <= 16 && fp8 ? 2 : 1; }
template <bool FP8, bool FEW>
constexpr int up_bytes() {
    int most = up_stage<FP8, 4>() * up_stages(FP8, 4);
    if (!FEW) {
        const int a = up_stage<FP8, 16>() * up_stages(FP8, 16);
        const int b = up_stage<FP8, 32>() * up_stages(FP8, 32);
        most = a > most ? a : most;
        most = b > most ? b : most;
    }
    return most;
}

// Columns first .. first + C - 1 of the unit's m tokens.
template <bool FP8, int C, bool NT, int BYTES>
__device__ __forceinline__ void up_body(const MoeArgs& p, int e, int n0, int m, int first_col,
                                        const uint8_t* token_of, const float* weight_of,
                                        const int* pick_of, uint8_t* lds)
{
    using X = Columns<C>;
    using W = Rows<FP8>;
    constexpr int CT = X::kTiles, kStages = up_stages(FP8, C), kStage = up_stage<FP8, C>();
    static_assert(kStages * kStage <= BYTES, "stages");
    constexpr int kOps = 2 * W::kLoads + X::kLoads;
    const int lane = lane_id(), l = lane % 16, g = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int H = p.H, I = p.I, HB = scale_blocks(H);
    constexpr int kBytes = FP8 ? 1 : 2;
    uint8_t* const gate = const_cast<uint8_t*>(p.w13) + (int64_t(e) * 2 * I + n0) * H * kBytes;
    const __amdgpu_buffer_rsrc_t gr = buffer_rsrc(gate, W::bytes(H));
    const __amdgpu_buffer_rsrc_t ur = buffer_rsrc(gate + int64_t(I) * H * kBytes, W::bytes(H));
    const __amdgpu_buffer_rsrc_t xr = buffer_rsrc(const_cast<uint16_t*>(p.x), int64_t(p.T) * H * 2);
    X x;
    x.init(lane, uint32_t(H) * 2u, [&](int c) {
        return token_of[first_col + c < m ? first_col + c : 0];
    });

    const int steps = (H + kStep - 1) / kStep, per = (steps + kUpWaves - 1) / kUpWaves;
    const int first = wave * per, last = first + per < steps ? first + per : steps;
    Scales sg{nullptr, HB, 0}, su{nullptr, HB, 0};
    if (FP8) {
        sg.from = p.s13 + (int64_t(e) * scale_blocks(2 * I) + n0 / kScaleBlock) * HB;
        su.from = sg.from + int64_t(I / kScaleBlock) * HB;
    }
    f32x4 ag[CT], au[CT];
#pragma unroll
    for (int t = 0; t < CT; ++t) ag[t] = au[t] = f32x4{0, 0, 0, 0};

    uint8_t* const stages = lds + wave * BYTES;
    auto load = [&](int s, int a) {
        const int n = s < last ? H : 0;
        uint8_t* const to = stages + a * kStage;
        W::template load<NT>(gr, to, s, n, H, lane);
        W::template load<NT>(ur, to + W::kBytes, s, n, H, lane);
        x.load(xr, to + 2 * W::kBytes, s, n);
        __builtin_amdgcn_sched_barrier(0);
    };
    if (first < last) {
        if (FP8) {
            sg.fill(first);
            su.fill(first);
        }
#pragma unroll
        for (int a = 0; a < kStages; ++a) load(first + a, a);
        for (int s0 = first; s0 < last; s0 += kStages) {
#pragma unroll
            for (int a = 0; a < kStages; ++a) {       // past the last step: zeros
                const int s = s0 + a;
                if (FP8 && (s & 63) == 0 && s != first) {
                    sg.fill(s);
                    su.fill(s);
                    wait_loads<0>();      // here, or every step would wait for everything
                }
                wait_loads<(kStages - 1) * kOps>();
                const float fg = FP8 ? sg.at(s) : 1.0f, fu = FP8 ? su.at(s) : 1.0f;
                const uint8_t* const from = stages + a * kStage;
                bf16x8 a_g[4], a_u[4];
                W::operands(from, lane, fg, a_g);
                W::operands(from + W::kBytes, lane, fu, a_u);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
#pragma unroll
                    for (int t = 0; t < CT; ++t) {
                        const bf16x8 b =
                            X::template operand<FP8>(from + 2 * W::kBytes, t, i, lane);
                        ag[t] = mfma(a_g[i], b, ag[t]);
                        au[t] = mfma(a_u[i], b, au[t]);
                    }
                }
                wait_loads<(kStages - 1) * kOps>();   // the stage has been read
                load(s + kStages, a);
            }
        }
    }
    // join the waves' parts of H: wave w sums column tiles w, w + kUpWaves, ..
    wait_loads<0>();
    __syncthreads();
    f32x4* const red = reinterpret_cast<f32x4*>(lds);
#pragma unroll
    for (int t = 0; t < CT; ++t) {
        red[((wave * CT + t) * 2 + 0) * kWave + lane] = ag[t];
        red[((wave * CT + t) * 2 + 1) * kWave + lane] = au[t];
    }
    __syncthreads();
    for (int t = wave; t < CT; t += kUpWaves) {
        f32x4 vg = red[(t * 2 + 0) * kWave + lane], vu = red[(t * 2 + 1) * kWave + lane];
#pragma unroll
        for (int w = 1; w < kUpWaves; ++w) {
            const f32x4 og = red[((w * CT + t) * 2 + 0) * kWave + lane];
            const f32x4 ou = red[((w * CT + t) * 2 + 1) * kWave + lane];
#pragma unroll
            for (int c = 0; c < 4; ++c) { vg[c] += og[c]; vu[c] += ou[c]; }
        }
        const int in = t * 16 + l, col = first_col + in;
        if (in >= C || col >= m) continue;
        const float w = weight_of[col];
        float hi[4], lo[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const float h = w * (vg[c] * sigmoid(vg[c]) * vu[c]);
            // h that rounds past bf16's largest value keeps that as its high half and
            // the rest as its low one; an infinite h has no rest (inf - inf is NaN).
            const bool finite = fabsf(h) < __builtin_inff();
            hi[c] = bf16_lo(pack_bf16x2(h, 0.0f));
            if (finite) hi[c] = fminf(fmaxf(hi[c], -kBf16Max), kBf16Max);
            lo[c] = finite ? h - hi[c] : 0.0f;
        }
        const int64_t at = int64_t(pick_of[col]) * I + n0 + g * 4;
        *reinterpret_cast<u32x2*>(p.h + at) =
            u32x2{pack_bf16x2(hi[0], hi[1]), pack_bf16x2(hi[2], hi[3])};
        *reinterpret_cast<u32x2*>(p.h + int64_t(p.T) * p.k * I + at) =
            u32x2{pack_bf16x2(lo[0], lo[1]), pack_bf16x2(lo[2], lo[3])};
    }
    __syncthreads();
}

// One token: pick u's expert, or -1 when an earlier pick has it already or it is
// none.  mine: the lane's pick; same: the picks that have it.
__device__ __forceinline__ int only_pick(const MoeArgs& p, int u, int& mine, uint64_t& same) {
    const int lane = lane_id();
    mine = p.idx[lane < p.k ? lane : p.k - 1];
    if (lane >= p.k) mine = -1;
    const int e = __builtin_amdgcn_readlane(mine, u);
    same = ballot(mine == e);
    return unsigned(e) < unsigned(p.E) && __builtin_ctzll(same) == u ? e : -1;
}

// FEW: at most four tokens.
template <bool FP8, bool FEW, bool NT>
__global__ __launch_bounds__(kUpWaves* kWave) void moe_up_kernel(MoeArgs p)
{
    // One array for all: with several, the compiler tells them apart and waits for
    // every load into LDS before any read of the same one.
    constexpr int kBytes = up_bytes<FP8, FEW>(), kStageBytes = kUpWaves * kBytes;
    constexpr int kLists = kMoeMaxTokens * 9, kWords = kMaxWords * 4;
    __shared__ __attribute__((aligned(256)))
    uint8_t lds[kStageBytes + kUpWaves * (kLists + kWords)];
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    // lists and picked experts: each wave's own, so that none waits here
    float* const weight_of =
        reinterpret_cast<float*>(lds + kStageBytes + wave * (kLists + kWords));
    int* const pick_of = reinterpret_cast<int*>(weight_of + kMoeMaxTokens);
    uint32_t* const words = reinterpret_cast<uint32_t*>(pick_of + kMoeMaxTokens);
    uint8_t* const token_of = reinterpret_cast<uint8_t*>(words + kMaxWords);

    const int u = blockIdx.y, chunk = blockIdx.x;
    if (FEW && p.T == 1) {      // one user's token: the shortest way to the weights
        int mine;
        uint64_t same;
        const float wl = p.topk_w[lane < p.k ? lane : p.k - 1];
        const int e = only_pick(p, u, mine, same);
        if (e < 0) return;
        float w = 0.0f;
        for (; same; same &= same - 1)
            w += __int_as_float(
                __builtin_amdgcn_readlane(__float_as_int(wl), __builtin_ctzll(same)));
        if (lane == 0) {
            token_of[0] = 0;
            weight_of[0] = w;
            pick_of[0] = u;
        }
        __builtin_amdgcn_wave_barrier();
        up_body<FP8, 4, NT, kBytes>(p, e, chunk * 16, 1, 0, token_of, weight_of, pick_of, lds);
        return;
    }

    // lane t: the picks of token t, eight at a time, the first eight kept
    const bool token = lane < p.T;
    const int32_t* const picks = p.idx + (token ? lane : 0) * p.k;
    const float* const weights = p.topk_w + (token ? lane : 0) * p.k;
    int id[8];
    float wj[8];
    auto read = [&](int j0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int at = j0 + j < p.k ? j0 + j : p.k - 1;
            id[j] = picks[at];
            wj[j] = weights[at];
            if (!token || j0 + j >= p.k) id[j] = -1;
        }
    };
    read(0);
    if (lane < kMaxWords) words[lane] = 0;
    __builtin_amdgcn_wave_barrier();
    for (int j0 = 0;;) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (unsigned(id[j]) < unsigned(p.E)) atomicOr(words + id[j] / 32, 1u << (id[j] & 31));
        j0 += 8;
        if (j0 >= p.k) break;
        read(j0);
    }
    __builtin_amdgcn_wave_barrier();
    // the u-th expert picked, in the order of their ids
    const uint32_t word = lane < kMaxWords ? words[lane] : 0;
    const int upto = wave_inclusive_sum(__popc(word));
    const int n = __builtin_amdgcn_readlane(upto, kWave - 1);
    if (u == 0 && chunk == 0 && threadIdx.x == 0) p.units[0] = n;
    if (u >= n) return;
    const int at = __builtin_ctzll(ballot(upto > u));
    uint32_t bits = __builtin_amdgcn_readlane(word, at);
    for (int skip = u - (__builtin_amdgcn_readlane(upto, at) - __popc(bits)); skip > 0; --skip)
        bits &= bits - 1;
    const int e = at * 32 + __builtin_ctz(bits);
    // its tokens: the first pick that has it carries the row, with the weights of
    // all that have it (each counted once)
    int mine = -1;
    float w = 0.0f;
    if (p.k > 8) read(0);
    for (int j0 = 0;;) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (id[j] != e) continue;
            if (mine < 0) mine = lane * p.k + j0 + j;
            w += wj[j];
        }
        j0 += 8;
        if (j0 >= p.k) break;
        read(j0);
    }
    const uint64_t has = ballot(mine >= 0);
    const int m = popc64(has), n0 = chunk * 16;
    if (mine >= 0) {
        const int c = popc64(has & lanes_below());
        token_of[c] = uint8_t(lane);
        weight_of[c] = w;
        pick_of[c] = mine;
        if (chunk == 0 && wave == 0) {
            int32_t* const unit = p.units + kHead + int64_t(u) * kUnit;
            if (c == 0) {
                unit[0] = e;
                unit[1] = m;
            }
            unit[2 + c] = mine;
        }
    }
    __builtin_amdgcn_wave_barrier();
    if (m <= 4) {
        up_body<FP8, 4, NT, kBytes>(p, e, n0, m, 0, token_of, weight_of, pick_of, lds);
    } else if constexpr (!FEW) {
        if (m <= 16) {
            up_body<FP8, 16, NT, kBytes>(p, e, n0, m, 0, token_of, weight_of, pick_of, lds);
        } else {
            for (int c = 0; c < m; c += 32)
                up_body<FP8, 32, false, kBytes>(p, e, n0, m, c, token_of, weight_of, pick_of, lds);
        }
    }
}

// ---------------------------------------------------------------- down
// A wave's expert, tokens first .. first + C / 2 - 1 of its m, into
// sums[token][16].  The C columns are the tokens' high halves, then their low ones;
// a token's two columns are added at the end.  With one token its pick is `only`.
template <bool FP8, int C, bool NT, int STAGES>
__device__ __forceinline__ void down_body(const MoeArgs& p, int e, int n0, int m, int first,
                                          int only, const int32_t* picks, uint8_t* stage,
                                          f32x4* sums)
{
    using X = Columns<C>;
    using W = Rows<FP8>;
    constexpr int kOps = W::kLoads + X::kLoads, kStage = W::kBytes + X::kBytes, kHalf = C / 2;
    const int lane = lane_id(), l = lane % 16, g = lane / 16;
    const int H = p.H, I = p.I, IB = scale_blocks(I);
    const __amdgpu_buffer_rsrc_t wr = buffer_rsrc(
        const_cast<uint8_t*>(p.w2) + (int64_t(e) * H + n0) * I * (FP8 ? 1 : 2), W::bytes(I));
    // the low halves follow the high ones in memory, T * k rows on
    const int64_t picks_all = int64_t(p.T) * p.k;
    const __amdgpu_buffer_rsrc_t hr = buffer_rsrc(p.h, 2 * picks_all * I * 2);
    X x;
    x.init(lane, uint32_t(I) * 2u, [&](int c) {
        const int t = first + c % kHalf;
        const int pick = m == 1 ? only : picks[t < m ? t : 0];
        return pick + (c < kHalf ? 0 : int(picks_all));
    });
    const int steps = (I + kStep - 1) / kStep;
    Scales sc{nullptr, IB, 0};
    if (FP8) {
        sc.from = p.s2 + (int64_t(e) * scale_blocks(H) + n0 / kScaleBlock) * IB;
        sc.fill(0);
    }
    auto load = [&](int s, int a) {
        const int n = s < steps ? I : 0;
        W::template load<NT>(wr, stage + a * kStage, s, n, I, lane);
        x.load(hr, stage + a * kStage + W::kBytes, s, n);
        __builtin_amdgcn_sched_barrier(0);
    };
    f32x4 part = {0, 0, 0, 0};
#pragma unroll
    for (int a = 0; a < STAGES; ++a) load(a, a);
    for (int s0 = 0; s0 < steps; s0 += STAGES) {
#pragma unroll
        for (int a = 0; a < STAGES; ++a) {            // past the last step: zeros
            const int s = s0 + a;
            if (FP8 && (s & 63) == 0 && s) {
                sc.fill(s);
                wait_loads<0>();          // here, or every step would wait for everything
            }
            wait_loads<(STAGES - 1) * kOps>();
            const uint8_t* const from = stage + a * kStage;
            bf16x8 op[4];
            W::operands(from, lane, FP8 ? sc.at(s) : 1.0f, op);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                part = mfma(op[i], X::template operand<FP8>(from + W::kBytes, 0, i, lane), part);
            wait_loads<(STAGES - 1) * kOps>();        // the stage has been read
            load(s + STAGES, a);
        }
    }
    wait_loads<0>();
#pragma unroll
    for (int c = 0; c < 4; ++c) part[c] += __shfl(part[c], lane + kHalf, kWave);
    // the sums of this expert's own tokens only: a NaN or infinite weight
    // reaches no token that did not pick it
    if (l < kHalf && first + l < m) {
        f32x4* const to = sums + ((m == 1 ? only : picks[first + l]) / p.k) * 4 + g;
        f32x4 v = *to;
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] += part[c];
        *to = v;
    }
    __builtin_amdgcn_wave_barrier();
}

// Stages of C columns, and the bytes of one wave's: two workgroups a CU and more.
constexpr int down_stages(bool fp8, int C) { return C <= 4 ? (fp8 ? 3 : 2) : C <= 8 ? (fp8 ? 3 : 2)
                                                                                : (fp8 ? 2 : 1); }
template <bool FP8, int C>
constexpr int down_stage_bytes() {
    return (Rows<FP8>::kBytes + Columns<C>::kBytes) * down_stages(FP8, C);
}
template <bool FP8, int TMAX>
constexpr int down_bytes() {
    if (TMAX == 1) return down_stage_bytes<FP8, 4>();
    const int a = down_stage_bytes<FP8, 8>(), b = down_stage_bytes<FP8, 16>();
    return a > b ? a : b;
}

// TMAX tokens at most.
template <bool FP8, int TMAX, int WAVES, bool NT>
__global__ __launch_bounds__(WAVES* kWave) void moe_down_kernel(MoeArgs p)
{
    constexpr int kSums = TMAX * 4, kDownBytes = down_bytes<FP8, TMAX>();      // a wave's
    // stages, then the waves' sums (one array: see the first launch)
    __shared__ __attribute__((aligned(256))) uint8_t lds[WAVES * (kDownBytes + kSums * 16)];
    f32x4* const sums = reinterpret_cast<f32x4*>(lds + WAVES * kDownBytes);
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int H = p.H, n0 = int(blockIdx.x) * 16;
    const int n = TMAX == 1 ? p.k : p.units[0];
    for (int i = lane; i < kSums; i += kWave) sums[wave * kSums + i] = f32x4{0, 0, 0, 0};
    __builtin_amdgcn_wave_barrier();
    for (int u = wave; u < n; u += WAVES) {
        uint8_t* const stage = lds + wave * kDownBytes;
        f32x4* const to = sums + wave * kSums;
        if constexpr (TMAX == 1) {
            int mine;
            uint64_t same;
            const int e = only_pick(p, u, mine, same);
            if (e >= 0)
                down_body<FP8, 4, NT, down_stages(FP8, 4)>(p, e, n0, 1, 0, u, nullptr, stage, to);
        } else {
            const int32_t* unit = p.units + kHead + int64_t(u) * kUnit;
            const int e = unit[0], m = unit[1], only = unit[2];
            if (m <= 4) {
                down_body<FP8, 8, NT, down_stages(FP8, 8)>(p, e, n0, m, 0, only, unit + 2, stage, to);
            } else {
                for (int c = 0; c < m; c += 8)
                    down_body<FP8, 16, false, down_stages(FP8, 16)>(p, e, n0, m, c, only,
                                                                    unit + 2, stage, to);
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.T * 4; i += WAVES * kWave) {
        f32x4 s = sums[i];
#pragma unroll
        for (int w = 1; w < WAVES; ++w)
#pragma unroll
            for (int c = 0; c < 4; ++c) s[c] += sums[w * kSums + i][c];
        *reinterpret_cast<u32x2*>(p.out + int64_t(i / 4) * H + n0 + i % 4 * 4) =
            u32x2{pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3])};
    }
}

template <bool FP8, bool NT>
hipError_t launch(const MoeArgs& p, hipStream_t s)
{
    const int picks = p.T * p.k;
    const dim3 up(uint32_t(p.I / 16), uint32_t(picks < p.E ? picks : p.E)), block(kUpWaves * kWave);
    if (p.T <= 4) EP_LAUNCH((moe_up_kernel<FP8, true, NT>), up, block, 0, s, p);
    else EP_LAUNCH((moe_up_kernel<FP8, false, NT>), up, block, 0, s, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    // sums in LDS for as few tokens as will do: more workgroups a CU
    const dim3 down(uint32_t(p.H / 16));
    if (p.T == 1)
        EP_LAUNCH((moe_down_kernel<FP8, 1, 8, NT>), down, dim3(8 * kWave), 0, s, p);
    else if (p.T <= 32)
        EP_LAUNCH((moe_down_kernel<FP8, 32, 4, NT>), down, dim3(4 * kWave), 0, s, p);
    else
        EP_LAUNCH((moe_down_kernel<FP8, kMoeMaxTokens, 4, NT>), down, dim3(4 * kWave), 0, s, p);
    return hipGetLastError();
}

}  // namespace

size_t moe_tokens_workspace(int T, int k, int I)
{
    const size_t picks = size_t(T) * k;
    return align256(2 * picks * I * 2) + align256((kHead + picks * kUnit) * sizeof(int32_t));
}

hipError_t launch_moe_tokens(const uint16_t* x, const int32_t* idx, const float* topk_w, int T,
                             int H, int I, int E, int k, const void* w13, const uint8_t* w13_scale,
                             const void* w2, const uint8_t* w2_scale, uint16_t* out, void* ws,
                             hipStream_t s)
{
    char* base = static_cast<char*>(ws);
    const size_t h_bytes = align256(2 * size_t(T) * k * I * 2);
    const MoeArgs p{x, idx, topk_w, T, H, I, E, k,
                    static_cast<const uint8_t*>(w13), w13_scale,
                    static_cast<const uint8_t*>(w2), w2_scale, out,
                    reinterpret_cast<uint16_t*>(base),
                    reinterpret_cast<int32_t*>(base + h_bytes)};
    const bool large = int64_t(E) * 3 * I * H * (w13_scale ? 1 : 2) > kStreamBytes;
    if (w13_scale) return large ? launch<true, true>(p, s) : launch<true, false>(p, s);
    return large ? launch<false, true>(p, s) : launch<false, false>(p, s);
}

}  // namespace ep
