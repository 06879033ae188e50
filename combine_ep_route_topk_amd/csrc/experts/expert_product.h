// expert_product.h -- the grouped product's kernel for operands without block
// scales: bf16, and 8-bit integers.
//
// For a row s of expert e:
//   bf16:  y[s][n] = sum_k a[s][k] W[e][n][k]            (f32 sums, rounded once)
//          y[s][n] = sum_k a[s][k] W[e][k][n]            (transposed)
//   int8:  y[s][n] = as[s] (ws[e][n] sum_k a[s][k] W[e][n][k])   (integer sums)
//   gated: g and u so from the rows [0, I) and [I, 2I) of W, h = silu(g) u in f32,
//          rounded once to bf16.
//
// A persistent workgroup of four waves, WN of them along the weight rows, makes TN =
// 32 FN WN weight rows x TM = 32 FM (4 / WN) tokens at a time with 32 x 32 matrix
// instructions of 16 bytes of k a lane; the weights are the row operand, so a lane
// holds four neighbouring n of one token.  A step is 128 bytes of k of every row:
// whole lines from memory.  Its loads go straight into LDS, STAGES of the weights and
// one less of the tokens, the stream running on across tiles, so that a tile's first
// loads and the stores of the one before it hide behind matrix work (with more than 64
// experts the search for the next segment waits for both: expert_tiles.h).  A step's four
// quarters work on fragments in registers while the next quarter's are read.
// Before the last quarter all waves meet: this step's stages have been read, the
// next step's have landed.  The weights of step s + STAGES - 1 are asked for in the
// first half of step s, into the stage that step s - 1 left; the tokens of it in the
// last quarter, into the stage that s itself has just left.
//
// Many rows (MI355X, 32768 of them, 8 experts, random values): bf16 x 7168 x 4096
// transposed 1470 to 1560 us, gated x 7168 x 2048 1530, x 2048 x 7168 795, 1.2 to 1.3
// PFLOP/s, where the library's dense products reach 1.25 to 1.5; int8 gated 797, down 434,
// 2.2 to 2.4 PFLOP/s (library 2.3 and 2.0).  Power bounds both: matrix instructions alone,
// from registers, reach 1.6 to 1.7 PFLOP/s on such bf16 values (2.4 on zeros) and 3.3 on
// int8; in bf16 the matrix unit is busy 77% of the time at 1.6 GHz.  Without its stores
// 3 to 6% faster, with all loads from L2 6 to 8%.  Accumulators of 32 x 32 rather than
// 16 x 16 (1.72 against 1.62 from registers) for the same reason: half the operand reads.
// int8 with a short k (2048: 235 us for 16384 rows x 7168, 52% busy) also pays for its
// epilogue, 3 us a tile that nothing else on its CU hides: the accumulators take the
// registers of a second workgroup.
// Few rows: the weights' bytes.  8 x 4096 x 7168 bf16, 64 rows 74 us, 6.4 TB/s; int8, 256
// uneven rows 45 us, 5.3 TB/s (launch, segments and the first loads, 5 us, are the same
// of half as many bytes); one row each 69 and 37, 6.8 and 6.4 TB/s.
// The steps there, the decode, ragged, training and int8 prefill sizes of the kernel as it
// was first (us, 64 x 8 x 4096 x 7168 / 1000 rows x 16 x 4096 x 2816 transposed / 32768 x 8 x 7168
// x 4096 transposed / int8 16384 x 8 x 7168 x 2048): 207 / 192 / 8849 / 513; now 74 / 51 /
// 1480 / 235.  A stage more (128 x 64, 128 x 128, 256 x 64), or whole steps in registers: within
// 3%.
#pragma once

#include "expert_choice.h"
#include "expert_tiles.h"

namespace ep {
namespace {

typedef short s16x8 __attribute__((ext_vector_type(8)));

struct ProductArgs {
    const uint8_t* a;
    const float* a_scale;
    const uint8_t* w;
    const float* w_scale;
    const int32_t* offsets;
    int S, N, K, E;      // N: columns of y, half the weights' rows when gated
    int max_tiles;       // row tiles that S rows in E segments can make
    uint16_t* y;         // plain: [S][N]; gated: gate_up [S][2N], if wanted
    uint16_t* h;         // gated: [S][N]
};

struct Bf16 {
    typedef f32x16 Acc;
    typedef f32x4 Quad;
    static constexpr int kBytes = 2;
    static constexpr bool kScaled = false;
    static __device__ __forceinline__ Acc mfma(u32x4 w, u32x4 x, Acc c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, w),
                                                       __builtin_bit_cast(bf16x8, x), c, 0, 0, 0);
    }
};
struct Int8 {
    typedef i32x16 Acc;
    typedef i32x4 Quad;
    static constexpr int kBytes = 1;
    static constexpr bool kScaled = true;
    static __device__ __forceinline__ Acc mfma(u32x4 w, u32x4 x, Acc c) {
        return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, w),
                                                     __builtin_bit_cast(i32x4, x), c, 0, 0, 0);
    }
};

enum ProductKind { kPlain, kTransposed, kGated, kGatedSaved };

template <class T_, ProductKind KIND_, int FN_, int FM_, int WN_, int STAGES_, bool TURN_, bool NT_>
struct ProductShape {
    typedef T_ T;
    static constexpr ProductKind KIND = KIND_;
    static constexpr int FN = FN_, FM = FM_, WN = WN_, STAGES = STAGES_;
    static constexpr bool TURN = TURN_;          // every tile of weights starts at another k
    static constexpr bool NT = NT_;              // the weights past the caches
    static constexpr bool TRANS = KIND == kTransposed, GATED = KIND >= kGated;
    static constexpr int TN = 32 * FN * WN, TM = 32 * FM * (4 / WN);
    static constexpr int kColumns = GATED ? TN / 2 : TN;      // of y or h
    static constexpr int kLds = (STAGES * TN + (STAGES - 1) * TM) * 128;
    // stores of one tile that every wave issues
    static constexpr int kStores = (KIND == kGated ? 1 : KIND == kGatedSaved ? 3 : 2) * FN * FM;
    static constexpr bool kStoreNt = TN == 256 && TM == 256;
    static_assert(!GATED || FN % 2 == 0, "gate and up rows alternate");
    static_assert(!TRANS || TN >= 128, "a row of a transposed stage has four units at least");
};

// What was found in the segments: their row tiles of the shape's size, and of up to 64
// experts the one of each lane.
struct Segments {
    int row_tiles, begin, end;
};

// What the workgroup has of a part of the tiles, in shape P.
template <class P>
__device__ __forceinline__ void product_tiles(const ProductArgs& p, const Segments& segments,
                                              const GemmShare& share, uint8_t* lds)
{
    typedef typename P::T T;
    constexpr int FN = P::FN, FM = P::FM, TN = P::TN, TM = P::TM, STAGES = P::STAGES;
    constexpr bool TRANS = P::TRANS, GATED = P::GATED;
    constexpr int kBK = 128;                             // bytes of k a step
    constexpr int kWStage = TN * kBK, kXStage = TM * kBK;
    constexpr int kWLoads = TN / 32, kXLoads = TM / 32;  // of 16 bytes a thread
    constexpr int kStepLoads = kWLoads + kXLoads;
    uint8_t* const xlds = lds + STAGES * kWStage;

    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wn = wave % P::WN, wm = wave / P::WN;
    const int N = p.N, row_bytes = p.K * T::kBytes;
    const int blocks = (row_bytes + kBK - 1) / kBK;
    const GemmTiles tiles(TM << share.halved, (N + P::kColumns - 1) / P::kColumns, segments.row_tiles,
                          segments.begin, segments.end);

    // LDS image of rows of 128 bytes: chunk c of 16 at slot c ^ (row / 2 % 8), so that
    // the 16 lanes that read one chunk of 16 rows touch every bank once.  A load
    // instruction fills 8 rows; its lanes fetch the chunks that belong there.
    const int lchunk = (lane & 7) ^ (((wave & 1) * 4 + (lane >> 4)) & 7);
    const uint32_t off0 = uint32_t(wave * 8 + lane / 8) * uint32_t(row_bytes) + lchunk * 16;
    // Transposed weights: 64 rows of k of TN columns, in units of 64 bytes, unit u of
    // row r at u ^ r % 4: a transposing read takes 8 rows x 64 bytes, rows 0..3 and
    // 8..11 of 16, which then touch every bank twice, the least that 512 bytes can.
    constexpr int kLanesPerRow = TN / 8, kRowsPerLoad = kWave / kLanesPerRow;
    const int trow = wave * kRowsPerLoad + lane / kLanesPerRow;
    const int tchunk = (lane & 3) | ((((lane % kLanesPerRow) >> 2) ^ (trow & 3)) << 2);

    // Where the stream of loads is: a tile, its next block of k, and how many blocks are
    // left (none: zeros).
    struct Cursor {
        const uint8_t* w;
        const uint8_t* x;
        int wbytes, xbytes;      // 0: no tile; transposed weights: of a row of k
        int k, left;
        uint32_t woff;           // transposed
    };
    auto start = [&](const GemmTile& t) {
        const bool some = t.rows.expert >= 0;
        const int rows = t.rows.end - t.rows.row0, first = t.n * P::kColumns;
        const int cols = N - first < P::kColumns ? N - first : P::kColumns;
        Cursor c;
        c.x = p.a + (some ? int64_t(t.rows.row0) * row_bytes : 0);
        c.xbytes = some ? (rows < TM ? rows : TM) * row_bytes : 0;
        const int64_t row = int64_t(some ? t.rows.expert : 0) * (TRANS ? p.K : GATED ? 2 * N : N);
        c.w = p.w + (TRANS ? row * N * 2 : (row + (some ? first : 0)) * row_bytes);
        c.wbytes = !some ? 0 : TRANS ? N * 2 : cols * row_bytes;
        c.k = P::TURN && some ? (t.rows.expert * 5 + t.n * 3) % blocks : 0;
        c.left = blocks;
        const int n = first + tchunk * 8;
        c.woff = n < N ? (uint32_t(trow) * uint32_t(N) + uint32_t(n)) * 2u : kOutside;
        return c;
    };
    auto advance = [&](Cursor& c) {
        ++c.k;
        --c.left;
        if (P::TURN && c.k == blocks) c.k = 0;
    };
    struct Source {
        __amdgpu_buffer_rsrc_t r, up;      // up: gated
        uint32_t off, group;
    };
    // Rows from block k on.  A lane's chunk of the last block may lie behind the row's end.
    const int chunk_end = row_bytes - lchunk * 16;
    auto rows_source = [&](const Cursor& c, const uint8_t* base, const uint8_t* up, int bytes) {
        const int k0 = c.k * kBK;
        const int use = c.left > 0 && bytes > k0 ? bytes - k0 : 0;
        int off = off0;
        hide(off);          // or every load's offset would take a register of its own
        return Source{buffer_rsrc(const_cast<uint8_t*>(base) + k0, use),
                      buffer_rsrc(const_cast<uint8_t*>(up) + k0, use),
                      k0 < chunk_end ? uint32_t(off) : kOutside, uint32_t(row_bytes) * 32u};
    };
    auto weights_source = [&](const Cursor& c) {
        if (!TRANS)
            return rows_source(c, c.w, GATED ? c.w + int64_t(N) * row_bytes : c.w, c.wbytes);
        const int k0 = c.k * (kBK / 2);
        const int rows = p.K - k0 < kBK / 2 ? p.K - k0 : kBK / 2;
        int off = int(c.woff);
        hide(off);
        const __amdgpu_buffer_rsrc_t r = buffer_rsrc(
            const_cast<uint8_t*>(c.w) + int64_t(k0) * N * 2, c.left > 0 ? rows * c.wbytes : 0);
        return Source{r, r, uint32_t(off), uint32_t(N) * uint32_t(kRowsPerLoad * 8)};
    };
    auto tokens_source = [&](const Cursor& c) { return rows_source(c, c.x, c.x, c.xbytes); };
    // load i of the weights: rows 32 i on, or gated groups of 32 rows that alternate
    // between gate and up
    auto issue_w = [&](const Source& c, uint8_t* to, int i) {
        uint8_t* const at = to + i * 4096 + wave * 1024;
        if (GATED) load16_to_lds<P::NT>(i & 1 ? c.up : c.r, at, c.off + uint32_t(i >> 1) * c.group);
        else load16_to_lds<P::NT>(c.r, at, c.off + uint32_t(i) * c.group);
    };
    auto issue_x = [&](const Source& c, uint8_t* to, int i) {
        load16_to_lds<false>(c.r, to + i * 4096 + wave * 1024, c.off + uint32_t(i) * c.group);
    };

    // Fragments of a quarter: 32 rows x 32 bytes of k, lane: row lt, the half lk.
    const int lt = lane & 31, lk = lane >> 5, g = lane >> 4, l = lane & 15;
    int foff[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) foff[q] = lt * kBK + (((2 * q + lk) ^ ((lt >> 1) & 7)) * 16);
    const int woff = TRANS ? 0 : wn * FN * 32 * kBK, xoff = wm * FM * 32 * kBK;
    // transposed: two transposing reads of rows 16 q + 8 lk .. + 3 and the four after them
    int toff[FN];
#pragma unroll
    for (int i = 0; i < FN; ++i)
        toff[i] = (lk * 8 + (l >> 2)) * (TN * 2) + ((wn * FN + i) ^ (l >> 2)) * 64 + (g & 1) * 32 +
                  (l & 3) * 8;
    struct Quarter {
        u32x4 w[FN], x[FM];
    };
    constexpr int kWReads = TRANS ? 2 * FN : FN, kReads = kWReads + FM;
    auto read = [&](uint8_t* ws, uint8_t* xs, int q, Quarter& f, int n) {
        // the first weights, the tokens, the other weights: as they are used
        constexpr int kFirst = TRANS ? 2 : 1;
        if (n >= kFirst && n < kFirst + FM) {
            f.x[n - kFirst] = load16(xs + xoff + (n - kFirst) * 32 * kBK + foff[q]);
            return;
        }
        const int m = n < kFirst ? n : n - FM;
        if (TRANS) {
            const s16x4 v = read_transposed(ws + toff[m / 2] + (q * 16 + m % 2 * 4) * (TN * 2));
            const u32x2 b = __builtin_bit_cast(u32x2, v);
            f.w[m / 2][m % 2 * 2] = b[0];
            f.w[m / 2][m % 2 * 2 + 1] = b[1];
        } else {
            f.w[m] = load16(ws + woff + m * 32 * kBK + foff[q]);
        }
    };
    constexpr int kSlots = FN * FM;
    typename T::Acc acc[FN][FM];
    // FN x FM matrix instructions on `f` (half: the first half, -1, or the second, 1), in
    // the first half the reads of the next quarter (quarter q of stages ws and xs), and
    // throughout the loads [first, last) of `src` into `to`.
    // Each matrix instruction is held in its place: the compiler would gather them
    // otherwise, and run out of registers.  The stages are named restrict: it would
    // wait for every load into LDS before a transposing read otherwise.
    auto multiply = [&](const Quarter& f, uint8_t* __restrict__ ws, uint8_t* __restrict__ xs, int q,
                        Quarter& next, const Source& src, uint8_t* __restrict__ to, bool weights,
                        int first, int last, int half) {
        constexpr int kEarly = (kSlots + 1) / 2;
#pragma unroll
        for (int n = half > 0 ? kSlots / 2 : 0; n < (half < 0 ? kSlots / 2 : kSlots); ++n) {
            const int i = n / FM, j = n % FM;
            acc[i][j] = T::mfma(f.w[i], f.x[j], acc[i][j]);
            pin(acc[i][j]);
#pragma unroll
            for (int r = n * kReads / kEarly; r < (n + 1) * kReads / kEarly && r < kReads; ++r)
                read(ws, xs, q, next, r);
#pragma unroll
            for (int r = first + n * (last - first) / kSlots;
                 r < first + (n + 1) * (last - first) / kSlots; ++r) {
                if (weights) issue_w(src, to, r);
                else issue_x(src, to, r);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    GemmTile t = tiles.at(p, TM, 0, share);
    if (t.rows.expert < 0) return;
    // a tile's loads reach into the next one only
    const int steps = blocks > STAGES - 1 ? blocks : STAGES - 1;
    Cursor cursor = start(t);
#pragma unroll
    for (int d = 0; d < STAGES - 1; ++d) {
        const Source w = weights_source(cursor), x = tokens_source(cursor);
#pragma unroll
        for (int i = 0; i < kWLoads; ++i) issue_w(w, lds + d * kWStage, i);
#pragma unroll
        for (int i = 0; i < kXLoads; ++i) issue_x(x, xlds + d * kXStage, i);
        advance(cursor);
    }
    wait_and_barrier<(STAGES - 2) * kStepLoads>();
    Quarter f0, f1;
#pragma unroll
    for (int n = 0; n < kReads; ++n) read(lds, xlds, 0, f0, n);
    int wslot = 0, xslot = 0;                            // the stages of this step

    for (int turn = 1;; ++turn) {
        const GemmTile tnext = tiles.at(p, TM, turn, share);
        if (steps == STAGES - 1) cursor = start(tnext);
        Source w = weights_source(cursor);
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < FM; ++j)
#pragma unroll
                for (int c = 0; c < 16; ++c) acc[i][j][c] = 0;
        for (int s = 0; s < steps; ++s) {
            const int wnext = wslot == STAGES - 1 ? 0 : wslot + 1;
            const int wlast = wslot == 0 ? STAGES - 1 : wslot - 1;
            const int xnext = xslot == STAGES - 2 ? 0 : xslot + 1;
            uint8_t* const ws = lds + wslot * kWStage;
            uint8_t* const xs = xlds + xslot * kXStage;
            uint8_t* const to = lds + wlast * kWStage;
            multiply(f0, ws, xs, 1, f1, w, to, true, 0, kWLoads / 2, 0);
            multiply(f1, ws, xs, 2, f0, w, to, true, kWLoads / 2, kWLoads, 0);
            // what the next loads need is worked out between matrix instructions: ahead of
            // a quarter it would leave the matrix unit idle
            multiply(f0, ws, xs, 3, f1, w, to, true, 0, 0, -1);
            const Source x = tokens_source(cursor);
            advance(cursor);
            __builtin_amdgcn_sched_barrier(0);
            multiply(f0, ws, xs, 3, f1, w, to, true, 0, 0, 1);
            // newer than the next step's loads: those of STAGES - 3 steps, this step's
            // weights, and in a tile's first step the last tile's stores
            constexpr int kNewer = (STAGES - 3) * kStepLoads + kWLoads;
            constexpr int kAfterStores = kNewer + P::kStores < 63 ? kNewer + P::kStores : 63;
            if (s == 0 && turn > 1) wait_and_barrier<kAfterStores>();
            else wait_and_barrier<kNewer>();
            __builtin_amdgcn_sched_barrier(0);
            uint8_t* const wsn = lds + wnext * kWStage;
            uint8_t* const xsn = xlds + xnext * kXStage;
            multiply(f1, wsn, xsn, 0, f0, x, xs, false, 0, kXLoads, -1);
            // the last STAGES - 1 steps of a tile load the first ones of the next
            if (s + STAGES == steps) cursor = start(tnext);
            w = weights_source(cursor);
            __builtin_amdgcn_sched_barrier(0);
            multiply(f1, wsn, xsn, 0, f0, x, xs, false, 0, kXLoads, 1);
            wslot = wnext;
            xslot = xnext;
        }
        __builtin_amdgcn_sched_barrier(0);

        // ---- epilogue: lane has tokens 32 j + lt of the wave's, weight rows 32 i + 8 q
        // + 4 lk + 0..3 (register 4 q + 0..3).  32 tokens x NF fragments at a time go
        // through LDS of the wave's own (the weights' stage that the last step left), so
        // that stores write whole pieces of rows.  Every store is issued whatever the
        // tile's edges (the descriptor drops what lies outside), so that their number is
        // known above.
        int el = lane;
        hide(el);                // keeps the addresses below out of the main loop's registers
        const int lane = el, lt = lane & 31, lk = lane >> 5;
        const int rows = t.rows.end - t.rows.row0 < TM ? t.rows.end - t.rows.row0 : TM;
        const int64_t row0 = t.rows.row0;
        uint8_t* const scratch = lds + (wslot == 0 ? STAGES - 1 : wslot - 1) * kWStage;
        constexpr int kPut = GATED ? FN / 2 : FN;
        uint8_t* const mine = scratch + wave * (kPut * 2048);
        const int col0 = t.n * P::kColumns + wn * kPut * 32;      // of the wave
        auto put = [&](auto&& get, const __amdgpu_buffer_rsrc_t& r, int width, int at, int j) {
            constexpr int kShift = kPut == 4 ? 0 : kPut == 2 ? 1 : 2, kMask = 4 * kPut - 1;
#pragma unroll
            for (int i = 0; i < kPut; ++i)
#pragma unroll
                for (int q = 0; q < 4; q += 2) {
                    float v[8];
#pragma unroll
                    for (int c = 0; c < 8; ++c) v[c] = get(i, 4 * q + c);
                    const auto lo = __builtin_amdgcn_permlane32_swap(
                        pack_bf16x2(v[0], v[1]), pack_bf16x2(v[4], v[5]), false, false);
                    const auto hi = __builtin_amdgcn_permlane32_swap(
                        pack_bf16x2(v[2], v[3]), pack_bf16x2(v[6], v[7]), false, false);
                    *reinterpret_cast<u32x4*>(
                        mine + lt * (64 * kPut) +
                        (((i * 4 + q + lk) ^ ((lt >> kShift) & kMask)) * 16)) =
                        u32x4{lo[0], hi[0], lo[1], hi[1]};
                }
            __builtin_amdgcn_wave_barrier();
            constexpr int kRows = 16 / kPut;
#pragma unroll
            for (int k = 0; k < 2 * kPut; ++k) {
                const int row = k * kRows + lane / (4 * kPut), c = lane % (4 * kPut);
                const u32x4 v = load16(mine + row * (64 * kPut) + ((c ^ ((row >> kShift) & kMask)) * 16));
                const int m = (wm * FM + j) * 32 + row, n = col0 + c * 8;
                __builtin_amdgcn_raw_buffer_store_b128(
                    v, r, int(n < N ? (uint32_t(m) * uint32_t(width) + uint32_t(at + n)) * 2u : kOutside), 0,
                    P::kStoreNt ? 2 : 0);
            }
            __builtin_amdgcn_wave_barrier();
        };
        // int8: the channels' scales and the tokens'
        f32x4 wscale[T::kScaled ? FN : 1][4];
        float token[FM];
        if constexpr (T::kScaled) {
            const int64_t expert = t.rows.expert;
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int n = col0 + (GATED ? i >> 1 : i) * 32 + 8 * q + 4 * lk;
                    const int64_t at = expert * (GATED ? 2 * N : N) + (GATED && (i & 1) ? N : 0);
                    wscale[i][q] = f32x4{0, 0, 0, 0};
                    if (n < N) wscale[i][q] = *reinterpret_cast<const f32x4*>(p.w_scale + at + n);
                }
#pragma unroll
            for (int j = 0; j < FM; ++j) {
                const int m = (wm * FM + j) * 32 + lt;
                token[j] = m < rows ? p.a_scale[row0 + m] : 0.0f;
            }
        }
        auto value = [&](int i, int j, int c) {
            if constexpr (T::kScaled) return float(acc[i][j][c]) * wscale[i][c / 4][c % 4] * token[j];
            else return float(acc[i][j][c]);
        };
        // The accumulators stay where they are until their turn: all at once they would
        // take registers that spill.
        auto take = [&](int j) {
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < FN; ++i) pin(acc[i][j]);
        };
        if constexpr (!GATED) {
            const __amdgpu_buffer_rsrc_t r = buffer_rsrc(p.y + row0 * N, int64_t(rows) * N * 2);
#pragma unroll
            for (int j = 0; j < FM; ++j) {
                take(j);
                put([&](int i, int c) { return value(i, j, c); }, r, N, 0, j);
            }
        } else {
            const __amdgpu_buffer_rsrc_t hr = buffer_rsrc(p.h + row0 * N, int64_t(rows) * N * 2);
#pragma unroll
            for (int j = 0; j < FM; ++j) {
                take(j);
                if constexpr (P::KIND == kGatedSaved) {
                    const __amdgpu_buffer_rsrc_t yr =
                        buffer_rsrc(p.y + row0 * 2 * N, int64_t(rows) * N * 4);
                    put([&](int i, int c) { return value(2 * i, j, c); }, yr, 2 * N, 0, j);
                    put([&](int i, int c) { return value(2 * i + 1, j, c); }, yr, 2 * N, N, j);
                }
                put([&](int i, int c) {
                    const float gate = value(2 * i, j, c);
                    return gate * sigmoid(gate) * value(2 * i + 1, j, c);
                }, hr, N, 0, j);
            }
        }
        if (tnext.rows.expert < 0) break;
        wait_and_barrier<63>();     // the scratch has been read before the next loads into it
        t = tnext;
    }
    wait_and_barrier<0>();          // no load into LDS outlives the workgroup
}

// Sum over the wave by row moves: the shuffles of wave_inclusive_sum would have the
// compiler keep their addresses, and spill them, for the tiles' own.
template <int CTRL, int ROWS>
__device__ __forceinline__ int add_moved(int v) {
    return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ int wave_sum(int v) {
    v = add_moved<0x111, 0xF>(v);       // from 1, 2, 4 and 8 lanes below in a row of 16
    v = add_moved<0x112, 0xF>(v);
    v = add_moved<0x114, 0xF>(v);
    v = add_moved<0x118, 0xF>(v);
    v = add_moved<0x142, 0xA>(v);       // a row's last lane to the odd row above it
    v = add_moved<0x143, 0xC>(v);       // the lower half's to the upper half
    return __builtin_amdgcn_readlane(v, kWave - 1);
}

// Which shape: by the row tiles that the segments make of each size, counted here, since
// sizes do not tell how the rows fall on the experts (choose_product_tile).  One
// workgroup a CU.  whole_lines: the weights' rows begin on lines and are more than the
// caches keep.
template <class T, ProductKind KIND>
__global__ __launch_bounds__(256, 1) void expert_product_kernel(ProductArgs p, int whole_lines)
{
    __shared__ __attribute__((aligned(256))) uint8_t lds[160 * 1024];
    int used = 0, tiles[3] = {0, 0, 0};            // of 64, 128 and 256 rows
    Segments found = {0, 0, 0};
    for (int e = int(threadIdx.x) % kWave; e < p.E; e += kWave) {
        segment_of(p.offsets, e, p.S, found.begin, found.end);
        const int rows = found.end - found.begin;
        used += rows > 0;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            tiles[i] += (rows + (64 << i) - 1) >> (6 + i);
            tiles[i] = tiles[i] < (1 << 24) ? tiles[i] : (1 << 24);      // 64 lanes stay below 2^31
        }
    }
    used = wave_sum(used);
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        // segments that do not overlap cannot pass the limit; others are cut there
        const int limit = (p.S >> (6 + i)) + (p.E < p.S ? p.E : p.S);
        tiles[i] = wave_sum(tiles[i]);
        tiles[i] = tiles[i] < limit ? tiles[i] : limit;
    }
    const int blocks = (p.K * T::kBytes + 127) / 128;
    int kernel = choose_product_tile(tiles[0], tiles[1], tiles[2], p.N, blocks, KIND >= kGated,
                                     int(gridDim.x));
    const int tokens = product_tile(kernel).tokens;
    found.row_tiles = tokens == 64 ? tiles[0] : tokens == 128 ? tiles[1] : tiles[2];
    bool past = product_past_caches(found.row_tiles, used, whole_lines != 0);
    GemmShare share = kWholeShare;
    if (kernel == kProduct256x256) {
        // whole rounds, then the last one in pieces
        constexpr int kColumns = KIND >= kGated ? 128 : 256;
        const int all = (found.row_tiles * ((p.N + kColumns - 1) / kColumns) + 7) / 8;
        const int slots = int(gridDim.x / 8), rest = all % slots;
        const int halved = rest && all > slots ? product_tail(rest, slots) : 0;
        if (halved) share.last = all - rest;
        if (past) product_tiles<ProductShape<T, KIND, 4, 4, 2, 3, true, true>>(p, found, share, lds);
        else product_tiles<ProductShape<T, KIND, 4, 4, 2, 3, false, false>>(p, found, share, lds);
        if (!halved) return;
        kernel = halved == 2 ? kProduct256x64 : kProduct256x128;
        past = false;                    // the pieces of a tile read the same weights
        share = {all - rest, all, halved};
    }
    switch (kernel) {
        case kProduct256x128:
            if (past) product_tiles<ProductShape<T, KIND, 4, 2, 2, 3, true, true>>(p, found, share, lds);
            else product_tiles<ProductShape<T, KIND, 4, 2, 2, 3, true, false>>(p, found, share, lds);
            break;
        case kProduct128x128:
            if (past) product_tiles<ProductShape<T, KIND, 2, 2, 2, 4, true, true>>(p, found, kWholeShare, lds);
            else product_tiles<ProductShape<T, KIND, 2, 2, 2, 4, true, false>>(p, found, kWholeShare, lds);
            break;
        case kProduct256x64:
            if (past) product_tiles<ProductShape<T, KIND, 2, 2, 4, 3, true, true>>(p, found, share, lds);
            else product_tiles<ProductShape<T, KIND, 2, 2, 4, 3, true, false>>(p, found, share, lds);
            break;
        default:
            if (past) product_tiles<ProductShape<T, KIND, 2, 1, 2, 4, true, true>>(p, found, kWholeShare, lds);
            else product_tiles<ProductShape<T, KIND, 2, 1, 2, 4, true, false>>(p, found, kWholeShare, lds);
    }
}

template <class T, ProductKind KIND>
hipError_t launch_product(const ProductArgs& p, hipStream_t s)
{
    const int64_t row_bytes = int64_t(p.K) * T::kBytes;
    const int64_t line_bytes = KIND == kTransposed ? int64_t(p.N) * T::kBytes : row_bytes;
    const bool whole = product_whole_lines(p.N, row_bytes, p.E, KIND >= kGated, line_bytes);
    if (product_most_tiles(p.S, p.N, p.E, KIND >= kGated) >= kProductMostTiles)
        return hipErrorInvalidConfiguration;
    const uint32_t cus = device_cu_count() / 8 * 8;
    EP_LAUNCH((expert_product_kernel<T, KIND>), dim3(cus ? cus : 8), dim3(256), 0, s, p, int(whole));
    return hipGetLastError();
}

// ------------------------------------------------------------- few tiles
// Few rows against few weight rows: tiles of 32 FN weight rows (gated, FN = 1: 16 of
// the gate and their 16 up rows) x 32 FM tokens, and the four waves of a workgroup
// share k instead: wave v takes the blocks v, v + 4, .. of 128 bytes, through stages
// of its own, without a barrier.  Their sums meet in LDS, in the waves' order; wave v
// finishes the rows 8 v .. 8 v + 7 of each 32.
// Bound by the latency of a few steps in a row: 1 x 4096 x 7168 of 8 rows (bf16, 59 MB)
// 17 us, 3.5 TB/s, where the persistent 128 x 64 tile takes 46; 4 x 2048 x 4096 of 40 rows
// 19 (28), 1 x 512 x 512 of 8 rows 3.5 (5), of which a launch is 2.  Eight waves with two
// stages each, for four with three: within 3%.
template <class T_, ProductKind KIND_, int FN_, int FM_, int STAGES_>
struct NarrowShape {
    typedef T_ T;
    static constexpr ProductKind KIND = KIND_;
    static constexpr int FN = FN_, FM = FM_, STAGES = STAGES_;
    static constexpr bool TRANS = KIND == kTransposed, GATED = KIND >= kGated;
    static constexpr int TN = 32 * FN, TM = 32 * FM;
    static constexpr int kColumns = GATED ? TN / 2 : TN;
    static constexpr int kLds = 4 * STAGES * (TN + TM) * 128;
    static constexpr int kOccupancy = kLds > 80 * 1024 ? 1 : 2;
    static constexpr bool kHalves = GATED && FN == 1;     // gate and up share a fragment
    static_assert(!GATED || FN <= 2, "gate rows, then their up rows");
    static_assert(FN <= 2, "a row of a transposed stage is a line at most");
    static_assert(4 * FN * FM * 4096 <= kLds, "the waves' sums");
};

template <class P>
__global__ __launch_bounds__(256, P::kOccupancy) void expert_narrow_kernel(ProductArgs p)
{
    typedef typename P::T T;
    constexpr int FN = P::FN, FM = P::FM, STAGES = P::STAGES;
    constexpr bool TRANS = P::TRANS, GATED = P::GATED;
    constexpr int kBK = 128, kStage = (P::TN + P::TM) * kBK, kLoads = 4 * (FN + FM);
    __shared__ __attribute__((aligned(256))) uint8_t lds[P::kLds];

    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int N = p.N, row_bytes = p.K * T::kBytes;
    const int blocks = (row_bytes + kBK - 1) / kBK;
    const GemmTile tile = GemmTiles(p, P::TM, (N + P::kColumns - 1) / P::kColumns).at(p, P::TM, 0);
    const RowTile t = tile.rows;
    if (t.expert < 0) return;
    const int rows = t.end - t.row0 < P::TM ? t.end - t.row0 : P::TM;
    const int col0 = tile.n * P::kColumns;
    const int cols = N - col0 < P::kColumns ? N - col0 : P::kColumns;
    // every tile starts at another block of k: rows a power of two apart would keep
    // to a few memory channels
    // (tiles of half a line stay together)
    const int turn = (t.expert * 5 + (TRANS && FN == 1 ? tile.n / 2 : tile.n) * 3) % blocks;
    uint8_t* const mine = lds + wave * STAGES * kStage;

    const __amdgpu_buffer_rsrc_t xr =
        buffer_rsrc(const_cast<uint8_t*>(p.a) + int64_t(t.row0) * row_bytes, int64_t(rows) * row_bytes);
    const uint8_t* const w0 =
        TRANS ? p.w + int64_t(t.expert) * p.K * N * 2
              : p.w + (int64_t(t.expert) * (GATED ? 2 * N : N) + col0) * row_bytes;
    const __amdgpu_buffer_rsrc_t wr =
        buffer_rsrc(const_cast<uint8_t*>(w0), TRANS ? 0 : int64_t(cols) * row_bytes);
    const __amdgpu_buffer_rsrc_t ur = buffer_rsrc(
        const_cast<uint8_t*>(w0) + (GATED ? int64_t(N) * row_bytes : 0), int64_t(cols) * row_bytes);

    // Rows of 128 bytes: load i fills rows 8 i .. 8 i + 7, chunk c of row r at c ^ r /
    // 2 % 8; transposed weights are 64 rows of k of a line (FN = 2), unit u (64 bytes) of
    // row r at u ^ r / 2 % 2, or half of one.
    const int lrow = lane / 8;
    auto load = [&](int step, uint8_t* to) {
        const bool some = step < blocks;
        int b = step + turn;
        b = b < blocks ? b : b - blocks;
        const int k0 = some ? b * kBK : row_bytes;
#pragma unroll
        for (int i = 0; i < 4 * FN; ++i) {
            if (TRANS) {
                const int row = FN == 2 ? i * 8 + lrow : i * 16 + lane / 4;
                const int chunk =
                    (lane & 3) | (FN == 2 ? (((lane & 7) >> 2) ^ (row >> 1 & 1)) << 2 : 0);
                const int left = p.K - k0 / 2, n = col0 + chunk * 8;
                const __amdgpu_buffer_rsrc_t r = buffer_rsrc(
                    const_cast<uint8_t*>(w0) + int64_t(some ? k0 / 2 : 0) * N * 2,
                    int64_t(!some ? 0 : left < 64 ? left : 64) * N * 2);
                load16_to_lds<false>(r, to + i * 1024,
                                    n < N ? (uint32_t(row) * uint32_t(N) + uint32_t(n)) * 2u : kOutside);
            } else {
                // gated: the gate rows, then their up rows
                const int kc = k0 + ((lane & 7) ^ ((i & 1) * 4 + (lane >> 4))) * 16;
                const int row = (GATED ? i % (2 * FN) : i) * 8 + lrow;
                load16_to_lds<false>(GATED && i >= 2 * FN ? ur : wr, to + i * 1024,
                                    kc < row_bytes ? uint32_t(row) * uint32_t(row_bytes) + uint32_t(kc)
                                                   : kOutside);
            }
        }
#pragma unroll
        for (int i = 0; i < 4 * FM; ++i) {
            const int kc = k0 + ((lane & 7) ^ ((i & 1) * 4 + (lane >> 4))) * 16;
            load16_to_lds<false>(xr, to + P::TN * kBK + i * 1024,
                                 kc < row_bytes ? uint32_t(i * 8 + lrow) * uint32_t(row_bytes) + uint32_t(kc)
                                                : kOutside);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    const int lt = lane & 31, lk = lane >> 5, g = lane >> 4, l = lane & 15;
    auto rows_fragment = [&](const uint8_t* from, int q) {
        return load16(from + lt * kBK + (((2 * q + lk) ^ ((lt >> 1) & 7)) * 16));
    };
    auto weights_fragment = [&](uint8_t* __restrict__ from, int i, int q) {
        if (!TRANS) return rows_fragment(from + i * 32 * kBK, q);
        u32x4 v;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int row = q * 16 + lk * 8 + c * 4 + (l >> 2);
            const u32x2 b = __builtin_bit_cast(
                u32x2, read_transposed(from + row * (64 * FN) + (FN == 2 ? (i ^ (row >> 1 & 1)) * 64 : 0) +
                                       (g & 1) * 32 + (l & 3) * 8));
            v[2 * c] = b[0];
            v[2 * c + 1] = b[1];
        }
        return v;
    };

    typename T::Acc acc[FN][FM];
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j)
#pragma unroll
            for (int c = 0; c < 16; ++c) acc[i][j][c] = 0;
    auto multiply = [&](uint8_t* __restrict__ from) {
        u32x4 w[FN][4], x[FM][4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
#pragma unroll
            for (int i = 0; i < FN; ++i) w[i][q] = weights_fragment(from, i, q);
#pragma unroll
            for (int j = 0; j < FM; ++j) x[j][q] = rows_fragment(from + (P::TN + j * 32) * kBK, q);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int i = 0; i < FN; ++i)
#pragma unroll
                for (int j = 0; j < FM; ++j) acc[i][j] = T::mfma(w[i][q], x[j][q], acc[i][j]);
    };
#pragma unroll
    for (int d = 0; d < STAGES - 1; ++d) load(wave + 4 * d, mine + d * kStage);
    const int count = (blocks - wave + 3) / 4;       // of this wave; may be 0
    for (int s0 = 0; s0 < count; s0 += STAGES) {
#pragma unroll
        for (int d = 0; d < STAGES; ++d) {            // past the last block: zeros
            // step s0 + d has landed, the step before has been read
            wait_loads<(STAGES - 2) * kLoads>();
            load(wave + 4 * (s0 + d + STAGES - 1), mine + (d + STAGES - 1) % STAGES * kStage);
            multiply(mine + d * kStage);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    wait_and_barrier<0>();          // no load is on its way, every stage has been read

    // the waves' sums: 4 values of a lane for each fragment and q, [wave][fragment][q][lane]
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<typename T::Quad*>(lds + (((wave * FN + i) * FM + j) * 4 + q) * 1024 +
                                                     lane * 16) =
                    typename T::Quad{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                                     acc[i][j][4 * q + 3]};
    __syncthreads();
    // lane: token 32 j + lt, weight rows 32 i + 8 wave + 4 lk + 0..3
    const int n = col0 + wave * 8 + lk * 4;           // of fragment 0
    auto store = [&](uint16_t* to, f32x4 v) {
        *reinterpret_cast<u32x2*>(to) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    };
#pragma unroll
    for (int j = 0; j < FM; ++j) {
        const int m = j * 32 + lt;
        if (m >= rows) continue;
        const int64_t row = t.row0 + m;
        const float token = T::kScaled ? p.a_scale[row] : 1.0f;
        // rows q of fragment i; channel: of y, or of [g; u]
        auto value = [&](int i, int q, int channel) {
            typename T::Quad sum;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const auto part = *reinterpret_cast<const typename T::Quad*>(
                    lds + (((k * FN + i) * FM + j) * 4 + q) * 1024 + lane * 16);
                if (k == 0) sum = part;
                else
#pragma unroll
                    for (int c = 0; c < 4; ++c) sum[c] += part[c];
            }
            f32x4 v;
            if constexpr (T::kScaled) {
                const f32x4 scale = *reinterpret_cast<const f32x4*>(
                    p.w_scale + int64_t(t.expert) * (GATED ? 2 * N : N) + channel);
#pragma unroll
                for (int c = 0; c < 4; ++c) v[c] = float(sum[c]) * scale[c] * token;
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c) v[c] = sum[c];
            }
            return v;
        };
        if constexpr (!GATED) {
#pragma unroll
            for (int i = 0; i < FN; ++i)
                if (n + i * 32 < N) store(p.y + row * N + n + i * 32, value(i, wave, n + i * 32));
        } else {
            if (n >= N || (P::kHalves && wave >= 2)) continue;
            const f32x4 gate = value(0, wave, n);
            const f32x4 up = P::kHalves ? value(0, wave + 2, N + n) : value(FN - 1, wave, N + n);
            if constexpr (P::KIND == kGatedSaved) {
                store(p.y + row * 2 * N + n, gate);
                store(p.y + row * 2 * N + N + n, up);
            }
            f32x4 h;
#pragma unroll
            for (int c = 0; c < 4; ++c) h[c] = gate[c] * sigmoid(gate[c]) * up[c];
            store(p.h + row * N + n, h);
        }
    }
}

template <class P>
hipError_t launch_narrow(ProductArgs p, hipStream_t s)
{
    const uint32_t grid = gemm_tiles(p, P::TM, P::kColumns);
    if (!grid || uint64_t(grid) * 256 >= (uint64_t(1) << 31)) return hipErrorInvalidConfiguration;
    EP_LAUNCH((expert_narrow_kernel<P>), dim3(grid), dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace
}  // namespace ep
