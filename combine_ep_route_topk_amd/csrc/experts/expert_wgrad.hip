// expert_wgrad.hip -- gradients of the experts' weights from bf16 rows.
//
// For expert e with rows [b, n):  dW[e][i][j] = sum_{s in [b, n)} dy[s][i] x[s][j]
// in f32, stored or added.  The summed axis is the slow one of both operands:
// rows are staged as they lie in memory (direct loads into LDS) and the matrix
// instruction's operands -- eight summed values of one column -- come from LDS
// through its transposing 16-bit read.  x is the row operand: a lane ends up
// with four neighbouring j of one i, 16-byte stores.  Rows past the segment lie
// outside the load descriptors and read as zero.
#include "expert_choice.h"
#include "experts_internal.h"

namespace ep {
namespace {

typedef short s16x8 __attribute__((ext_vector_type(8)));

struct WgradArgs {
    const uint16_t* dy;
    const uint16_t* x;
    const int32_t* offsets;
    int S, N, K, E;
    float* dw;
};

__device__ __forceinline__ bf16x8 join(s16x4 lo, s16x4 hi) {
    return __builtin_bit_cast(
        bf16x8, s16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
}

// The fragments of A x 32 j that a wave holds of 32 i (lane: column i = lane % 32,
// rows j in registers) to rows i of 32 j in memory, or added to what is there:
// through `buf`, 4 KB of LDS of the wave's own for each of two fragments, so that
// every store writes eight whole 128-byte lines (straight from registers a lane
// pair writes 32 bytes of a line: 16 experts x 2816 x 4096 from 128 rows each
// 230 us, through LDS 163).  Rows of 128 bytes, chunk c of row r at c ^ r % 8.
// All A fragments' old values are asked for at once.  A store is issued whatever
// the tile's edges (the descriptor drops what lies outside).
//
// NT: past the caches, so that a large output does not push the operands, which
// every tile of an expert reads again, out of L2 (128 rows each: 133 us instead of
// 197; an output that fits, 8 x 1024 x 1024: 33, 28).
template <bool ACC, bool NT, int A>
__device__ __forceinline__ void put_fragments(__amdgpu_buffer_rsrc_t r, uint8_t* buf, int lane,
                                              const f32x16 (&v)[A], int i0, int j0, int K) {
    const int lt = lane & 31, lk = lane >> 5, row = lane / 8;
    auto at = [&](int a, int k) {
        const int i = i0 + k * 8 + row, j = j0 + a * 32 + lane % 8 * 4;
        return j < K ? (uint32_t(i) * uint32_t(K) + uint32_t(j)) * 4u : kOutside;
    };
    f32x4 old[ACC ? A : 1][4];
    if (ACC) {
#pragma unroll
        for (int a = 0; a < A; ++a)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                old[a][k] = __builtin_bit_cast(
                    f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, int(at(a, k)), 0, NT ? 2 : 0));
        __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int a = 0; a < A; ++a) {
        uint8_t* const to = buf + (a & 1) * 4096;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            *reinterpret_cast<f32x4*>(to + lt * 128 + (((2 * q + lk) ^ (lt & 7)) * 16)) =
                f32x4{v[a][4 * q], v[a][4 * q + 1], v[a][4 * q + 2], v[a][4 * q + 3]};
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            f32x4 o = *reinterpret_cast<const f32x4*>(to + (k * 8 + row) * 128 +
                                                      (((lane & 7) ^ row) * 16));
            if (ACC)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[c] += old[a][k][c];
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, o), r, int(at(a, k)), 0,
                                                   NT ? 2 : 0);
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// ------------------------------------------------------------- large tiles
// A persistent workgroup of four waves makes 256 i x 256 j at a time, each wave
// 128 x 128 with 32 x 32 x 16 matrix instructions (the tile and the reasons of
// the grouped 8-bit product: 2048 cycles of matrix work for each 64 rows
// against 1536 of LDS).  64 rows are a step; its 512-byte row parts go through
// three stages of dy and two of x, all 160 KB of LDS.  A quarter step works on
// fragments in registers and reads the next quarter's.  Before the last quarter
// all waves meet: this step's stages have been read, the next step's have
// landed.  The stream runs on across tiles.
//
// Measured on MI355X, 8 experts x 4096 x 7168, 4096 rows each: 1492 to 1565 us (1.26
// PFLOP/s; a library product of one matrix of that size with the same transposed
// operands 1974 to 2035, with both turned beforehand 1530 to 1600), added to what is
// there 1600 to 1608 (0.94 GB more are read); eight waves of 128 x 64 on two stages,
// without the units' exchange, 3721 us, all of it LDS bank conflicts.
//
// LDS image of a stage: rows of 512 bytes in units of 64, unit u of row r at
// u ^ r % 4: a transposing read takes 8 rows x 64 bytes, rows 0..3 and 8..11 of
// 16, which then touch every bank twice, the least that 512 bytes can.
constexpr int kTile = kWgradTile, kRows = 64;
constexpr int kStage = kRows * kTile * 2;            // 32 KB of one operand
constexpr int kLoads = kStage / 16 / 256;            // 8 of 16 bytes a thread

struct WgradTile {
    int expert, i0, j0, begin, end;      // expert -1: none
};

template <bool ACC>
__global__ __launch_bounds__(256, 1) void expert_wgrad_large_kernel(WgradArgs p)
{
    __shared__ __attribute__((aligned(256))) uint8_t lds[5 * kStage];
    uint8_t* const xstage = lds + 3 * kStage;

    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wi = wave & 1, wj = wave >> 1;
    const int N = p.N, K = p.K;
    const int nt = (N + kTile - 1) / kTile, kt = (K + kTile - 1) / kTile;
    const int total = nt * kt * p.E;

    // Tiles in blocks of as many as an XCD runs at once, given to the XCDs in
    // turn (experts differ in rows, so a contiguous share each would not do);
    // within an expert, 8 j tiles x all i tiles, j fastest.
    const int slots = int(gridDim.x / 8);
    auto tile_at = [&](int turn) {
        WgradTile t{-1, 0, 0, 0, 0};
        const int id = (turn * 8 + int(blockIdx.x % 8)) * slots + int(blockIdx.x / 8);
        if (id >= total) return t;
        t.expert = id / (nt * kt);
        const int in = id - t.expert * nt * kt;
        const int group = in / (8 * nt), size = kt - group * 8 < 8 ? kt - group * 8 : 8;
        const int rest = in - group * 8 * nt;
        t.j0 = (group * 8 + rest % size) * kTile;
        t.i0 = rest / size * kTile;
        int b, n;
        segment_of(p.offsets, t.expert, p.S, b, n);
        t.begin = __builtin_amdgcn_readfirstlane(b);
        t.end = __builtin_amdgcn_readfirstlane(n);
        return t;
    };
    const int turns = (total + int(gridDim.x) - 1) / int(gridDim.x);
    auto output = [&](const WgradTile& t) {
        const int rows = N - t.i0 < kTile ? N - t.i0 : kTile;
        return buffer_rsrc(p.dw + (int64_t(t.expert) * N + t.i0) * K, int64_t(rows) * K * 4);
    };
    // tiles without rows: zeros, apart from the stream
    if (!ACC) {
        for (int turn = 0; turn < turns; ++turn) {
            const WgradTile t = tile_at(turn);
            if (t.expert < 0 || t.end > t.begin) continue;
            const __amdgpu_buffer_rsrc_t r = output(t);
            for (int v = threadIdx.x; v < kTile * kTile / 4; v += 256) {
                const int i = v / (kTile / 4), j = t.j0 + v % (kTile / 4) * 4;
                __builtin_amdgcn_raw_buffer_store_b128(
                    u32x4{0, 0, 0, 0}, r,
                    int(j < K ? (uint32_t(i) * uint32_t(K) + uint32_t(j)) * 4u : kOutside), 0, 2);
            }
        }
    }
    int turn = 0;
    auto next_tile = [&]() {       // the next tile with rows
        WgradTile t{-1, 0, 0, 0, 0};
        while (turn < turns) {
            t = tile_at(turn++);
            if (t.expert < 0 || t.end > t.begin) break;
            t.expert = -1;
        }
        return t;
    };
    auto steps_of = [](const WgradTile& t) {     // even: an odd count's last step is zeros
        return ((t.end - t.begin + kRows - 1) / kRows + 1) & ~1;
    };

    // One operand's loads of one step: a load instruction fills two rows; its
    // lanes fetch the chunks that belong there.
    const int chunk = (lane & 3) | ((((lane >> 2) & 7) ^ ((wave & 1) * 2 + (lane >> 5))) << 2);
    const int lrow = wave * 2 + lane / 32;
    struct Source {
        __amdgpu_buffer_rsrc_t r;
        uint32_t off, group;
    };
    auto source = [&](const uint16_t* base, int width, const WgradTile& t, int c0, int s) {
        const int64_t row = t.begin + int64_t(s) * kRows;
        const int64_t left = t.end - row;
        int c = c0 + chunk * 8;
        hide(c);          // or every load's offset would take a register of its own
        const uint32_t off = (uint32_t(lrow) * uint32_t(width) + uint32_t(c)) * 2u;
        const int64_t use = left <= 0 ? 0 : left < kRows ? left : kRows;
        return Source{buffer_rsrc(const_cast<uint16_t*>(base) + (use ? row * width : 0),
                                  use * width * 2),
                      c < width ? off : kOutside, uint32_t(width) * 16u};
    };
    auto issue = [&](const Source& c, uint8_t* to, int i) {
        load16_to_lds<false>(c.r, to + wave * 1024 + i * 4096, c.off + uint32_t(i) * c.group);
    };

    // Fragment f of 32 columns, quarter q: two transposing reads of rows
    // 16 q + 8 (lane / 32) .. + 3 and the four after them.
    const int g = lane >> 4, l = lane & 15;
    int foff[4];
#pragma unroll
    for (int f = 0; f < 4; ++f)
        foff[f] = ((g >> 1) * 8 + (l >> 2)) * 512 + (f ^ (l >> 2)) * 64 + (g & 1) * 32 + (l & 3) * 8;
    struct Quarter {
        s16x4 y[4][2], x[4][2];
    };
    auto read = [&](uint8_t* ys, uint8_t* xs, int q, Quarter& f, int n) {
        const int c = n & 1, i = n >> 1;
        const int at = q * 16 * 512 + c * 4 * 512;
        if (i == 0) f.x[0][c] = read_transposed(xs + foff[0] + at);
        else if (i < 5) f.y[i - 1][c] = read_transposed(ys + foff[i - 1] + at);
        else f.x[i - 4][c] = read_transposed(xs + foff[i - 4] + at);
    };
    f32x16 acc[4][4];      // [i fragment][j fragment]
    // 16 matrix instructions, between them the reads of the next quarter and
    // `loads` of eight loads from `first` on into `to`.  The stages are named
    // restrict: the compiler would wait for every load into LDS before a
    // transposing read otherwise.
    auto multiply = [&](const Quarter& f, uint8_t* __restrict__ ys, uint8_t* __restrict__ xs, int q,
                        Quarter& next, const Source& src, uint8_t* __restrict__ to, int first,
                        int loads) {
#pragma unroll
        for (int n = 0; n < 16; ++n) {
            const int a = n / 4, b = n % 4;
            acc[b][a] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                join(f.x[a][0], f.x[a][1]), join(f.y[b][0], f.y[b][1]), acc[b][a], 0, 0, 0);
            pin(acc[b][a]);
            read(ys, xs, q, next, n);
            if (loads && n % (16 / loads) == 16 / loads - 1) issue(src, to, first + n / (16 / loads));
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    WgradTile t = next_tile();
    if (t.expert < 0) return;
    int steps = steps_of(t);
    {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const Source y = source(p.dy, N, t, t.i0, k), x = source(p.x, K, t, t.j0, k);
#pragma unroll
            for (int i = 0; i < kLoads; ++i) issue(y, lds + k * kStage, i);
#pragma unroll
            for (int i = 0; i < kLoads; ++i) issue(x, xstage + k * kStage, i);
        }
    }
    wait_and_barrier<2 * kLoads>();
    uint8_t* const yfrag = lds + wi * 256;
    uint8_t* const xfrag = xstage + wj * 256;
    Quarter f0, f1;
#pragma unroll
    for (int n = 0; n < 16; ++n) read(yfrag, xfrag, 0, f0, n);
    int yslot = 0;
    bool stored = false;
    for (;;) {
        const WgradTile tnext = next_tile();
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
                for (int c = 0; c < 16; ++c) acc[a][b][c] = 0.0f;
        for (int s = 0; s < steps; ++s) {
            const int ynext = yslot == 2 ? 0 : yslot + 1, ylast = yslot == 0 ? 2 : yslot - 1;
            const bool over = s + 2 >= steps;
            const int s2 = over ? s + 2 - steps : s + 2;
            const WgradTile& from = over ? tnext : t;
            uint8_t* const ys = yfrag + yslot * kStage;
            uint8_t* const xs = xfrag + (s & 1) * kStage;
            // dy's stage that step s - 1 left takes step s + 2
            const Source ysrc = source(p.dy, N, from, from.i0, s2);
            uint8_t* const yto = lds + ylast * kStage;
            multiply(f0, ys, xs, 1, f1, ysrc, yto, 0, 4);
            multiply(f1, ys, xs, 2, f0, ysrc, yto, 4, 4);
            multiply(f0, ys, xs, 3, f1, ysrc, yto, 0, 0);
            // newer than the next step's loads: dy's 8, and in a tile's first
            // step the 64 stores of the last tile
            if (s == 0 && stored) wait_and_barrier<63>();
            else wait_and_barrier<kLoads>();
            __builtin_amdgcn_sched_barrier(0);
            const Source xsrc = source(p.x, K, from, from.j0, s2);
            multiply(f1, yfrag + ynext * kStage, xfrag + ((s + 1) & 1) * kStage, 0, f0, xsrc,
                     xstage + (s & 1) * kStage, 0, 8);
            yslot = ynext;
        }
        __builtin_amdgcn_sched_barrier(0);
        // the stage of dy that the last step left is free until the next step
        // loads into it
        int el = lane;
        hide(el);          // keeps the addresses out of the main loop's registers
        uint8_t* const buf = lds + (yslot == 0 ? 2 : yslot - 1) * kStage + wave * 8192;
        const __amdgpu_buffer_rsrc_t r = output(t);
#pragma unroll
        for (int b = 0; b < 4; ++b)
            put_fragments<ACC, true>(r, buf, el, acc[b], wi * 128 + b * 32, t.j0 + wj * 128, K);
        __syncthreads();
        if (tnext.expert < 0) break;
        t = tnext;
        steps = steps_of(t);
        stored = !ACC;
    }
    wait_and_barrier<0>();          // no load into LDS outlives the workgroup
}

// ------------------------------------------------------------- small tiles
// 128 i x 128 j, four waves of 64 x 64, steps of 32 rows on three stages (48 KB:
// three workgroups a CU, one's stores behind another's loads).  Bound by what it
// writes: 16 experts x 2816 x 4096 from 2000 ragged rows in 128 us, 6.0 TB/s (added
// to what is there, 128 rows each, 244 us, 6.1 TB/s both ways); tiles of a row of the
// output run together (column by column: 64 rows each 149 us, 133).  With few tiles
// each expert's rows are split over `parts` workgroups a tile, whose sums go to
// a workspace [part][E][N][K] and are joined in order by a second launch.
constexpr int kSmallTile = kWgradSmallTile, kSmallRows = 32;
constexpr int kSmallStage = 2 * kSmallRows * kSmallTile * 2;      // dy, then x: 16 KB

template <bool ACC, bool NT>
__global__ __launch_bounds__(256) void expert_wgrad_small_kernel(WgradArgs p, int parts)
{
    constexpr int kStages = 3, kOperand = kSmallStage / 2, kPer = kOperand / 16 / 256;   // 2 loads
    __shared__ __attribute__((aligned(256))) uint8_t lds[kStages * kSmallStage];
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wi = wave & 1, wj = wave >> 1;
    const int N = p.N, K = p.K;
    const int nt = (N + kSmallTile - 1) / kSmallTile, kt = (K + kSmallTile - 1) / kSmallTile;
    const int part = int(blockIdx.x) % parts, tile = int(blockIdx.x) / parts;
    const int e = tile / (nt * kt), in = tile - e * nt * kt;
    const int i0 = in / kt * kSmallTile, j0 = in % kt * kSmallTile;
    int b0, n0;
    segment_of(p.offsets, e, p.S, b0, n0);
    int begin = __builtin_amdgcn_readfirstlane(b0), end = __builtin_amdgcn_readfirstlane(n0);
    if (ACC && end == begin) return;
    if (parts > 1) {      // whole steps to each part
        const int all = (end - begin + kSmallRows - 1) / kSmallRows;
        const int per = (all + parts - 1) / parts * kSmallRows;
        const int64_t from = begin + int64_t(part) * per;
        begin = from < end ? int(from) : end;
        end = end - begin < per ? end : begin + per;
    }
    const int steps = (end - begin + kSmallRows - 1) / kSmallRows;

    // a load instruction fills four rows of 256 bytes in units of 64, unit u of
    // row r at u ^ r % 4
    const int lrow = lane / 16, chunk = (lane & 3) | ((((lane >> 2) & 3) ^ (lrow & 3)) << 2);
    auto issue = [&](int s) {
        uint8_t* st = lds + s % kStages * kSmallStage;
        const int64_t row = begin + int64_t(s) * kSmallRows;
        const int64_t left = end - row, use = left <= 0 ? 0 : left < kSmallRows ? left : kSmallRows;
        const __amdgpu_buffer_rsrc_t yr =
            buffer_rsrc(const_cast<uint16_t*>(p.dy) + (use ? row * N : 0), use * N * 2);
        const __amdgpu_buffer_rsrc_t xr =
            buffer_rsrc(const_cast<uint16_t*>(p.x) + (use ? row * K : 0), use * K * 2);
        const int i = i0 + chunk * 8, j = j0 + chunk * 8;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const uint32_t r = (k * 4 + wave) * 4 + lrow;
            load16_to_lds<false>(yr, st + (k * 4 + wave) * 1024,
                          i < N ? (r * uint32_t(N) + uint32_t(i)) * 2u : kOutside);
        }
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const uint32_t r = (k * 4 + wave) * 4 + lrow;
            load16_to_lds<false>(xr, st + kOperand + (k * 4 + wave) * 1024,
                          j < K ? (r * uint32_t(K) + uint32_t(j)) * 2u : kOutside);
        }
    };
    const int g = lane >> 4, l = lane & 15;
    const int frow = ((g >> 1) * 8 + (l >> 2)) * 256 + (g & 1) * 32 + (l & 3) * 8;
    f32x16 acc[2][2];
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int c = 0; c < 16; ++c) acc[a][b][c] = 0.0f;
    auto multiply = [&](uint8_t* __restrict__ ys, uint8_t* __restrict__ xs) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            bf16x8 y[2], x[2];
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                uint8_t* a = ys + q * 16 * 256 + frow + (((wi * 2 + f) ^ (l >> 2)) * 64);
                uint8_t* b = xs + q * 16 * 256 + frow + (((wj * 2 + f) ^ (l >> 2)) * 64);
                y[f] = join(read_transposed(a), read_transposed(a + 4 * 256));
                x[f] = join(read_transposed(b), read_transposed(b + 4 * 256));
            }
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
                for (int b = 0; b < 2; ++b)
                    acc[b][a] =
                        __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[a], y[b], acc[b][a], 0, 0, 0);
        }
    };
    issue(0);
    issue(1);
    for (int s = 0; s < steps; ++s) {
        wait_and_barrier<2 * kPer>();        // step s has landed, step s - 1 has been read
        issue(s + 2);                        // past the end: zeros
        uint8_t* st = lds + s % kStages * kSmallStage;
        multiply(st, st + kOperand);
    }
    wait_and_barrier<0>();          // every stage has been read, no load is on its way
    const int rows = N - i0 < kSmallTile ? N - i0 : kSmallTile;
    const __amdgpu_buffer_rsrc_t r =
        buffer_rsrc(p.dw + ((int64_t(part) * p.E + e) * N + i0) * K, int64_t(rows) * K * 4);
#pragma unroll
    for (int b = 0; b < 2; ++b)
        put_fragments<ACC, NT>(r, lds + wave * 8192, lane, acc[b], wi * 64 + b * 32, j0 + wj * 64, K);
}

hipError_t launch_large(const WgradArgs& p, int64_t tiles, bool accumulate, hipStream_t s)
{
    // one workgroup a CU (it takes all of the LDS), each with its share of tiles
    const int64_t most = (tiles + 7) / 8 * 8;
    const int64_t cus = device_cu_count() / 8 * 8;
    const dim3 grid(uint32_t(most < cus || cus == 0 ? most : cus));
    if (accumulate) EP_LAUNCH((expert_wgrad_large_kernel<true>), grid, dim3(256), 0, s, p);
    else EP_LAUNCH((expert_wgrad_large_kernel<false>), grid, dim3(256), 0, s, p);
    return hipGetLastError();
}

template <bool ACC>
__global__ __launch_bounds__(256) void join_parts_kernel(const float* __restrict__ sums, int parts,
                                                         int64_t vecs, float* __restrict__ dw)
{
    for (int64_t v = int64_t(blockIdx.x) * 256 + threadIdx.x; v < vecs;
         v += int64_t(gridDim.x) * 256) {
        f32x4 o = {0, 0, 0, 0};
        if (ACC) o = reinterpret_cast<const f32x4*>(dw)[v];
        f32x4 t = reinterpret_cast<const f32x4*>(sums)[v];
        for (int q = 1; q < parts; ++q) {
            const f32x4 u = reinterpret_cast<const f32x4*>(sums)[q * vecs + v];
#pragma unroll
            for (int c = 0; c < 4; ++c) t[c] += u[c];
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) o[c] = ACC ? o[c] + t[c] : t[c];
        reinterpret_cast<f32x4*>(dw)[v] = o;
    }
}

hipError_t launch_small(WgradArgs p, int parts, bool accumulate, float* sums, hipStream_t s)
{
    const int64_t tiles = int64_t((p.N + kSmallTile - 1) / kSmallTile) *
                          ((p.K + kSmallTile - 1) / kSmallTile) * p.E;
    if (tiles * parts * 256 >= (int64_t(1) << 31)) return hipErrorInvalidConfiguration;
    const dim3 grid{uint32_t(tiles * parts)};
    float* const dw = p.dw;
    if (parts > 1) p.dw = sums;
    const bool nt = parts == 1 && int64_t(p.E) * p.N * p.K >= int64_t(16) << 20;   // 64 MB
    if (accumulate && parts == 1) {
        if (nt) EP_LAUNCH((expert_wgrad_small_kernel<true, true>), grid, dim3(256), 0, s, p, parts);
        else EP_LAUNCH((expert_wgrad_small_kernel<true, false>), grid, dim3(256), 0, s, p, parts);
    } else {
        if (nt) EP_LAUNCH((expert_wgrad_small_kernel<false, true>), grid, dim3(256), 0, s, p, parts);
        else EP_LAUNCH((expert_wgrad_small_kernel<false, false>), grid, dim3(256), 0, s, p, parts);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || parts == 1) return e;
    const int64_t vecs = int64_t(p.E) * p.N * p.K / 4, want = (vecs + 255) / 256;
    const dim3 join(uint32_t(want < 4096 ? want : 4096));
    if (accumulate) EP_LAUNCH((join_parts_kernel<true>), join, dim3(256), 0, s, sums, parts, vecs, dw);
    else EP_LAUNCH((join_parts_kernel<false>), join, dim3(256), 0, s, sums, parts, vecs, dw);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_expert_wgrad(const uint16_t* grad_y, const uint16_t* x, const int32_t* offsets,
                               int S, int N, int K, int E, int accumulate, float* grad_w,
                               float* sums, hipStream_t s)
{
    const WgradArgs p{grad_y, x, offsets, S, N, K, E, grad_w};
    if (wgrad_tiles(N, K, E, kSmallTile) >= (int64_t(1) << 30)) return hipErrorInvalidConfiguration;
    if (wgrad_large(S, N, K, E))
        return launch_large(p, wgrad_tiles(N, K, E, kTile), accumulate != 0, s);
    return launch_small(p, sums ? wgrad_parts(S, N, K, E) : 1, accumulate != 0, sums, s);
}

}  // namespace ep
