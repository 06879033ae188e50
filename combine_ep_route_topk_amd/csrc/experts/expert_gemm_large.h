// expert_gemm_large.h -- the grouped product's kernel for segments of many rows.
//
// A persistent workgroup of four waves makes 256 weight rows x 256 tokens at a
// time; each wave 128 x 128 with 32 x 32 x 64 matrix instructions, its 256
// accumulators and two sets of operands (8 fragments each) filling the 512
// registers that one wave per SIMD may use.  Why this tile: a step of 128 k
// costs a CU 2048 cycles of matrix work against 128 KB of LDS reads + 64 KB of
// writes at 128 bytes a cycle, 1536 cycles; eight waves of 128 x 64 would read
// 192 KB, and the sum fill all of it.
//
// k moves through all 160 KB of LDS: three stages of 128 bytes of k for the
// weights, two for the tokens.  Half a step works on fragments already in
// registers; between its 16 matrix instructions it reads the next half's from
// LDS and issues 8 of the step's 16 loads, the weights' in the first half (into
// the stage that the step before left), the tokens' in the second (into the one
// that this step has just left): one barrier a step.  The stream runs on across
// tiles, so that the first loads of a tile and the stores of the one before it
// hide behind matrix work.
//
// Measured on MI355X, 8 experts, sustained: 32768 rows x 7168 x 4096 in 802 to 840
// us, 32768 x 4096 x 7168 in 765 to 811 (2.3 to 2.5 PFLOP/s; a library product of
// one matrix of that size 656 to 692 and 611), the same gated 744 to 753, with the
// gate and up values kept 837.  The steps
// before, at the first size: eight waves of 128 x 64 on two stages 1062; four
// waves, 64 bytes of k on four stages, all loads of a step at once 990 (rows of 64
// bytes ask the L2 for half lines); whole lines on two stages with one load after
// each matrix instruction 954 (all at once 964: the wave stalls behind its own
// loads); five stages 865; persistent 830; whole-line stores 815.  What bounds it
// now: power (the clock falls to about 1.9 GHz; register-only matrix work on random
// data reaches 3.8 PFLOP/s), and that loads and stores complete in order: a tile's
// third step waits for the last tile's stores.
#pragma once

#include "expert_tiles.h"

namespace ep {
namespace {

struct GemmArgs {
    const uint8_t* a;
    const uint8_t* a_scale;
    const uint8_t* w;
    const uint8_t* w_scale;
    const int32_t* offsets;
    int S, N, K, E;      // N: rows of one expert's weights (2 I when gated)
    int max_tiles;       // row tiles that S rows in E segments can make
    uint16_t* y;         // plain: [S][N]; gated: gate_up [S][N] or NULL
    uint8_t* h;          // gated: [S][N/2]
    uint8_t* h_scale;    // gated: [S][N/256]
};

constexpr int kLargeTile = 256;

// SAVE: gated, and gate_up is wanted.
template <bool GATED, bool SAVE>
__global__ __launch_bounds__(256, 1) void expert_gemm_large_kernel(GemmArgs p)
{
    constexpr int kTile = kLargeTile, kBK = kScaleBlock;
    constexpr int kStage = kTile * kBK;                  // 32 KB of one operand
    constexpr int kLoads = kStage / 16 / 256;            // 8 of 16 bytes a thread
    // three stages of the weights, then two of the tokens
    __shared__ __attribute__((aligned(256))) uint8_t lds[5 * kStage];

    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wn = wave & 1, wm = wave >> 1;
    const int N = p.N, K = p.K, KB = scale_blocks(K);
    const GemmTiles tiles(p, kTile, GATED ? N / 256 : (N + kTile - 1) / kTile);

    // What a tile's loads need: its operands from the tile's first row on.
    struct Base {
        const uint8_t* w;
        const uint8_t* x;
        int64_t wbytes, xbytes;      // 0: no tile
    };
    auto base_of = [&](const GemmTile& t) {
        if (t.rows.expert < 0) return Base{p.w, p.a, 0, 0};
        const int left = t.rows.end - t.rows.row0;
        const int64_t first = int64_t(t.n) * (GATED ? kTile / 2 : kTile);     // weight row
        const int64_t wrows = GATED ? N - first : (N - first < kTile ? N - first : kTile);
        return Base{p.w + (int64_t(t.rows.expert) * N + first) * K, p.a + int64_t(t.rows.row0) * K,
                    wrows * K, int64_t(left < kTile ? left : kTile) * K};
    };

    // LDS image: rows of 128 bytes, chunk c of 16 at slot c ^ (row / 2 % 8): the
    // 16 lanes that read one chunk of 16 rows touch every bank once.  A load
    // instruction fills 8 rows; its lanes fetch the chunks that belong there.
    const int lchunk = (lane & 7) ^ (((wave & 1) * 4 + (lane >> 4)) & 7);
    const uint32_t off0 = uint32_t(wave * 8 + lane / 8) * uint32_t(K) + lchunk * 16;
    // load i of the weights: rows 32 i on; gated: the groups of 32 rows alternate
    // between gate and up
    auto weight_group = [&](int i) {
        return uint32_t(GATED ? (i >> 1) * 32 + (i & 1) * (N / 2) : i * 32) * uint32_t(K);
    };
    auto token_group = [&](int i) { return uint32_t(i * 32) * uint32_t(K); };
    const int steps = (KB + 1) & ~1;      // even: an odd count's last step is all zeros
    // One operand's loads of one step; past the end they store zeros.
    struct Source {
        __amdgpu_buffer_rsrc_t r;
        uint32_t off;
        uint8_t* to;
    };
    auto source = [&](const uint8_t* base, int64_t bytes, int s, uint8_t* to) {
        const int k0 = s * kBK;
        const int left = K - k0;
        int off = off0;
        hide(off);          // or every load's offset would take a register of its own
        return Source{buffer_rsrc(const_cast<uint8_t*>(base) + k0, bytes > k0 ? bytes - k0 : 0),
                      uint32_t(off) | (lchunk * 16 >= left ? kOutside : 0), to + wave * 1024};
    };
    auto issue = [&](const Source& c, bool weights, int i) {
        load16_to_lds<false>(c.r, c.to + i * 4096, c.off + (weights ? weight_group(i) : token_group(i)));
    };

    // scale bytes of one 128-block: the wave's 128 weight rows share one (gated:
    // gate and up one each); one for each of the lane's four tokens
    const int NB = scale_blocks(N);
    const int lt = lane & 31, lk = lane >> 5;
    const uint32_t soff = uint32_t(wm * 128 + lt) * uint32_t(KB);
    struct ScaleBase {
        const uint8_t* w;
        const uint8_t* x;
        int xbytes;
    };
    auto scales_of = [&](const GemmTile& t) {
        if (t.rows.expert < 0) return ScaleBase{p.w_scale, p.a_scale, 0};
        int block = GATED ? t.n : (t.n * kTile + wn * 128) / kScaleBlock;
        block = block < NB ? block : NB - 1;
        const int left = t.rows.end - t.rows.row0;
        return ScaleBase{p.w_scale + (int64_t(t.rows.expert) * NB + block) * KB,
                         p.a_scale + int64_t(t.rows.row0) * KB, (left < kTile ? left : kTile) * KB};
    };
    struct Scales {
        int w[2], x[4];
    };
    auto load_scales = [&](const ScaleBase& from, int b, Scales& c) {
        b = b < KB ? b : KB - 1;
        c.w[0] = from.w[b];
        c.w[1] = GATED ? from.w[int64_t(NB / 2) * KB + b] : c.w[0];
        const __amdgpu_buffer_rsrc_t r =
            buffer_rsrc(const_cast<uint8_t*>(from.x) + b, from.xbytes > b ? from.xbytes - b : 0);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            c.x[j] = __builtin_amdgcn_raw_buffer_load_b8(r, int(soff + uint32_t(j * 32 * KB)), 0, 0);
    };

    // fragments: 32 rows x 64 k (half a step), lane: row lt, k 32 lk ..
    int foff[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int c = 0; c < 2; ++c)
            foff[h][c] = lt * kBK + (((4 * h + 2 * lk + c) ^ ((lt >> 1) & 7)) * 16);
    f32x16 acc[4][4];
    struct Half {
        u32x4 w[4][2], x[4][2];
    };
    // read n of 16 of a half step's fragments, first those that it uses first
    auto read = [&](const uint8_t* wl, const uint8_t* xl, int h, Half& f, int n) {
        const int c = n & 1, i = n >> 1;
        if (i == 0) f.w[0][c] = load16(wl + foff[h][c]);
        else if (i < 5) f.x[i - 1][c] = load16(xl + (i - 1) * 32 * kBK + foff[h][c]);
        else f.w[i - 4][c] = load16(wl + (i - 4) * 32 * kBK + foff[h][c]);
    };
    auto operand = [&](const u32x4 (&v)[2]) {
        return i32x8{int(v[0][0]), int(v[0][1]), int(v[0][2]), int(v[0][3]),
                     int(v[1][0]), int(v[1][1]), int(v[1][2]), int(v[1][3])};
    };
    // Half a step: 16 matrix instructions on `f`, and between them the reads of
    // the next half (half h of stages wl and xl) and eight loads.  The empty asm
    // holds each matrix instruction in its place: the compiler would gather them
    // otherwise, and run out of registers.
    auto multiply = [&](const Half& f, const Scales& c, const uint8_t* wl, const uint8_t* xl, int h,
                        Half& next, const Source& src, bool weights) {
#pragma unroll
        for (int n = 0; n < 16; ++n) {
            const int i = n / 4, j = n % 4;
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                operand(f.w[i]), operand(f.x[j]), acc[i][j], 0, 0, 0, c.w[i & 1], 0, c.x[j]);
            pin(acc[i][j]);
            read(wl, xl, h, next, n);
            if (n & 1) issue(src, weights, n / 2);
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    uint8_t* const xstage = lds + 3 * kStage;
    Scales sa, sb;
    Half f0, f1;
    GemmTile t = tiles.at(p, kTile, 0);
    if (t.rows.expert < 0) return;
    Base cur = base_of(t);
    ScaleBase scur = scales_of(t);
    load_scales(scur, 0, sa);
    auto issue_all = [&](const Source& c, bool weights) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) issue(c, weights, i);
    };
    issue_all(source(cur.w, cur.wbytes, 0, lds), true);
    issue_all(source(cur.x, cur.xbytes, 0, xstage), false);
    issue_all(source(cur.w, cur.wbytes, 1, lds + kStage), true);
    issue_all(source(cur.x, cur.xbytes, 1, xstage + kStage), false);
    wait_and_barrier<2 * kLoads>();
    const uint8_t* const wfrag = lds + wn * 128 * kBK;
    const uint8_t* const xfrag = xstage + wm * 128 * kBK;
#pragma unroll
    for (int n = 0; n < 16; ++n) read(wfrag, xfrag, 0, f0, n);
    int wslot = 0;                                       // the weights' stage of this step

    // The tiles' steps follow each other without a gap: the last two steps of a
    // tile load the first two of the next one, whose first fragments are in
    // registers when the epilogue ends.
    for (int turn = 1;; ++turn) {
        const GemmTile tnext = tiles.at(p, kTile, turn);
        const Base next = base_of(tnext);
        const ScaleBase snext = scales_of(tnext);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int c = 0; c < 16; ++c) acc[i][j][c] = 0.0f;

        // One step: its first half is in registers, its scales are in c; the
        // next step's scales go to d.
        auto step = [&](int s, const Scales& c, Scales& d) {
            const int wnext = wslot == 2 ? 0 : wslot + 1, wlast = wslot == 0 ? 2 : wslot - 1;
            const bool over = s + 2 >= steps;
            const int s2 = over ? s + 2 - steps : s + 2;
            if (s + 1 < steps) load_scales(scur, s + 1, d);
            else load_scales(snext, 0, d);
            __builtin_amdgcn_sched_barrier(0);
            // the weights' stage that step s - 1 left takes step s + 2
            multiply(f0, c, wfrag + wslot * kStage, xfrag + (s & 1) * kStage, 1, f1,
                     source(over ? next.w : cur.w, over ? next.wbytes : cur.wbytes, s2,
                            lds + wlast * kStage), true);
            // Every wave has left this step's stages, and the next step's have
            // landed: newer than those are this half's 8 loads, and in a tile's
            // first step also the last tile's stores, 32 (gated: 8) at least.
            if (s == 0 && turn > 1) wait_and_barrier<kLoads + (GATED ? 8 : 32)>();
            else wait_and_barrier<kLoads>();
            __builtin_amdgcn_sched_barrier(0);
            multiply(f1, c, wfrag + wnext * kStage, xfrag + ((s + 1) & 1) * kStage, 0, f0,
                     source(over ? next.x : cur.x, over ? next.xbytes : cur.xbytes, s2,
                            xstage + (s & 1) * kStage), false);
            wslot = wnext;
        };
        for (int s = 0; s < steps; s += 2) {
            step(s, sa, sb);
            step(s + 1, sb, sa);
        }
        __builtin_amdgcn_sched_barrier(0);

        // ---- epilogue: lane has tokens wm 128 + 32 j + lt, weight rows
        // 32 i + 8 q + 4 lk + 0..3 (register 4 q + 0..3).  Every store is issued
        // whatever the tile's edges (the descriptor drops what lies outside), so
        // that their number is known above.
        int el = lane;
        hide(el);                // keeps the addresses below out of the main loop's registers
        const int lane = el, lt = lane & 31, lk = lane >> 5;
        const int row0 = t.rows.row0;
        const int rows = t.rows.end - row0 < kTile ? t.rows.end - row0 : kTile;
        // 16 bf16 of two neighbouring q to one 16-byte store a lane
        auto pack_pair = [&](const f32x16& v, int q) {
            const auto lo = __builtin_amdgcn_permlane32_swap(
                pack_bf16x2(v[4 * q], v[4 * q + 1]), pack_bf16x2(v[4 * q + 4], v[4 * q + 5]), false,
                false);
            const auto hi = __builtin_amdgcn_permlane32_swap(
                pack_bf16x2(v[4 * q + 2], v[4 * q + 3]), pack_bf16x2(v[4 * q + 6], v[4 * q + 7]),
                false, false);
            return u32x4{lo[0], hi[0], lo[1], hi[1]};
        };
        const __amdgpu_buffer_rsrc_t yr = buffer_rsrc(
            GATED && !SAVE ? p.y : p.y + int64_t(row0) * N,
            GATED && !SAVE ? 0 : int64_t(rows) * N * 2);
        // the weights' stage that the last step left is free until the next step
        // loads into it
        uint8_t* const scratch = lds + (wslot == 0 ? 2 : wslot - 1) * kStage;
        if constexpr (!GATED) {
            // 32 tokens x 128 weight rows at a time through 8 KB of the wave's own,
            // so that stores write whole lines, and past the caches, where tokens
            // and weights are read again (32-byte parts of lines straight from
            // registers: 32768 rows x 7168 x 4096 830 us, so 815): rows of 256
            // bytes, chunk c of 16 of row r at c ^ r % 16
            uint8_t* const mine = scratch + wave * 8192;
            const int srow = lane / 16, sn = t.n * kTile + wn * 128 + lane % 16 * 8;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int q = 0; q < 4; q += 2)
                        *reinterpret_cast<u32x4*>(
                            mine + lt * 256 + (((i * 4 + q + lk) ^ (lt & 15)) * 16)) =
                            pack_pair(acc[i][j], q);
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int r = k * 4 + srow, m = wm * 128 + j * 32 + r;
                    const u32x4 v = load16(mine + r * 256 + (((lane & 15) ^ (r & 15)) * 16));
                    __builtin_amdgcn_raw_buffer_store_b128(
                        v, yr,
                        int(sn < N ? (uint32_t(m) * uint32_t(N) + uint32_t(sn)) * 2u : kOutside), 0,
                        2);
                }
                __builtin_amdgcn_wave_barrier();
            }
            __syncthreads();        // the scratch is read before the next loads into it
        } else {
            // the waves' maxima [2][256], then the tile's 256 x 128 bytes on their way
            // to whole-line stores
            float* part = reinterpret_cast<float*>(scratch);
            const int I = N / 2;
            if constexpr (SAVE) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int q = 0; q < 4; q += 2) {
                            const int m = wm * 128 + j * 32 + lt;
                            const int n = t.n * kScaleBlock + wn * 64 + (i >> 1) * 32 + (i & 1) * I +
                                          8 * (q + lk);
                            __builtin_amdgcn_raw_buffer_store_b128(
                                pack_pair(acc[i][j], q), yr,
                                int((uint32_t(m) * uint32_t(N) + uint32_t(n)) * 2u), 0, 0);
                            __builtin_amdgcn_sched_barrier(0);
                        }
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) pin(acc[i][j]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int m = wm * 128 + j * 32 + lt;
                float top = 0.0f;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const float g = acc[2 * i][j][c];
                        const float v = g * sigmoid(g) * acc[2 * i + 1][j][c];
                        acc[2 * i][j][c] = v;
                        top = max_finite(top, v);
                    }
                    pin(acc[2 * i][j]);
                    __builtin_amdgcn_sched_barrier(0);
                }
                top = fmaxf(top, __shfl_xor(top, 32, kWave));
                if (lk == 0) part[wn * 256 + m] = top;
            }
            __syncthreads();
            int ex[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int m = wm * 128 + j * 32 + lt;
                ex[j] = scale_exponent(fmaxf(part[m], part[256 + m]));
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int m = wm * 128 + j * 32 + lt;
                const float inv = pow2(-ex[j]);
                __builtin_amdgcn_sched_barrier(0);
                // rows of 128 bytes in words, word c of row m at c ^ m % 32
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const f32x16& v = acc[2 * i][j];
                        const int c = wn * 16 + i * 8 + q * 2 + lk;
                        *reinterpret_cast<uint32_t*>(scratch + m * 128 + ((c ^ (m & 31)) * 4)) =
                            pack_e4m3x4(v[4 * q] * inv, v[4 * q + 1] * inv, v[4 * q + 2] * inv,
                                        v[4 * q + 3] * inv);
                    }
                if (lk == 0 && wn == 0 && m < rows)
                    p.h_scale[int64_t(row0 + m) * (I / kScaleBlock) + t.n] = uint8_t(ex[j] + 127);
            }
            __syncthreads();
            const __amdgpu_buffer_rsrc_t hr =
                buffer_rsrc(p.h + int64_t(row0) * I, int64_t(rows) * I);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int m = k * 32 + wave * 8 + lane / 8, c = lane % 8 * 4;
                u32x4 v;
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    v[d] = *reinterpret_cast<const uint32_t*>(scratch + m * 128 +
                                                              (((c + d) ^ (m & 31)) * 4));
                __builtin_amdgcn_raw_buffer_store_b128(
                    v, hr, int(uint32_t(m) * uint32_t(I) + t.n * kScaleBlock + c * 4), 0, 0);
            }
            __syncthreads();        // the scratch is read before the next loads into it
        }
        if (tnext.rows.expert < 0) break;
        t = tnext;
        cur = next;
        scur = snext;
        if constexpr (GATED) {
            // read again rather than held through the epilogue, whose registers
            // would spill, each reload a wait for every load and store (23 us a tile)
#pragma unroll
            for (int n = 0; n < 16; ++n) read(wfrag + wslot * kStage, xfrag, 0, f0, n);
        }
    }
    wait_and_barrier<0>();          // no load into LDS outlives the workgroup
}

}  // namespace
}  // namespace ep
