// expert_choice.h -- which kernel a grouped product or a weight gradient takes.
// Rules on sizes (and, for the bf16 and int8 products' tiles, on how the rows fall on the
// experts), in a header of their own so that a test can ask which kernel its sizes reach.
#pragma once

#include <math.h>
#include <stdint.h>

#if defined(__HIPCC__)
#include <hip/hip_runtime.h>
#define EP_BOTH __host__ __device__ inline
#else
#define EP_BOTH inline
#endif

namespace ep {

// Weights that one call reads once, of more than this, are read past the caches:
// until their next use the rest of a model will have gone through the 256 MB that
// the memory side keeps.  Streaming weights on MI355X, cached / past the caches: 235
// MB (8 experts x 4096 x 7168, 32 rows each) 43 / 39 us, 940 MB 159 / 145; 33 MB
// that the last call left there 11 / 15.
constexpr int64_t kStreamBytes = int64_t(64) << 20;

// ------------------------------------------------------------- grouped products
// The persistent 256 x 256 kernel, or the kernel for few rows with tiles of so
// many tokens x weight rows.
enum GemmKernel {
    kGemmLarge,
    kGemm128x256,
    kGemm64x256,
    kGemm32x256,
    kGemm128x128,
    kGemm64x128,
    kGemm32x64,
};

// Which kernel, by the rows an expert has on average and the workgroups that a
// tile would make.  Measured on MI355X with weights that come from memory, even rows,
// us for 64 / 128 tokens x 256 weight rows / the large kernel:
//   8 experts x 4096 x 7168, rows each   48: 53 / 55 / 74    96: 53 / 64 / 75
//                                       160: 98 / 83 / 79   192: 101 / 83 / 82
//   16 x 2816 x 4096                     48: 34 / 35 / 51   128: 59 / 45 / 55   160: 87 / 87 / 56
//   1 x 4096 x 4096                    1024: 26 / 38 / 46  2048: 52 / 41 / 47
//   4 x 2048 x 4096                     256: 28 / 40 / 50   512: 28 / 40 / 50
//   32 x 2816 x 4096                    128: 98 / 91 / 113  256: 167 / 131 / 126
// With few rows the weights are read at the rate of the busiest CU, so as near to
// one workgroup each as can be; us for 256 / 128 / 64 weight rows a workgroup:
//   16 experts x 2816 x 4096, 30 rows each  32 / 38 / 33
//   8 x 4096 x 7168, 32 rows                51 / 39 / 39
//   2 x 4096 x 7168, 8 rows                 42 / 29 / 24
//   32 x 4096 x 7168, 16 rows              145 / 143 / 145
// With 256 weight rows (gated always), 64 / 32 tokens a workgroup, gated:
//   8 x 4096 x 7168, 48 rows 54 / 49, 96 rows 52 / 92;  1 x 4096 x 7168, 64 rows 48 /
//   42;  4 x 1024 x 2048, 300 rows 16 / 13;  16 x 2816 x 4096, 30 rows 32 / 32, 45 rows
//   34 / 52;  32 x 4096 x 4096, 48 rows 89 / 116
// One workgroup a CU has room for 128 rows: where the 32 rows are an average, of 94
// to 12, 45 us instead of 62; of 64 rows at most in all there is nothing to hold
// (8 rows over 64 experts x 4096 x 7168: 37.6, with 64 36.7).
// At most S experts have rows.  All of them counted / those, 7168 values of k: 8 rows
// over 64 experts x 2048 29.9 / 25.9, 8 over 16 x 4096 46.5 / 36.1, 3 over 8 x 4096
// 30.7 / 24.6, 1 over 64 x 4096 27.2 / 23.0.
// Sizes alone do not say how even the rows are, and the rule is not the best one
// everywhere: 8 x 4096 x 7168, 96 even rows take 53 us where 128 x 128 takes 47; 4 x
// 2048 x 4096, 256 even rows 30 where 64 x 128 takes 20; 1 x 4096 x 4096, 2048 rows 47
// where 128 x 256 takes 41.
// N: rows of one expert's weights (2 I when gated).
inline GemmKernel choose_gemm(int64_t S, int64_t N, int64_t E, bool gated, int64_t cus)
{
    const int64_t used = S < E ? S : E;         // experts that can have rows
    auto tiles = [&](int64_t tm, int64_t tn) {
        const int64_t mt = (S + tm - 1) / tm;
        return (mt > used ? mt : used) * ((N + tn - 1) / tn);
    };
    if (S >= 160 * E && tiles(256, 256) >= 112) return kGemmLarge;
    if (S > 48 * E && tiles(128, 256) > 128) return kGemm128x256;
    if (!gated) {
        const int64_t wide = tiles(64, 256);
        if (wide > cus || wide * 3 < cus * 2) {
            if (tiles(32, 64) <= cus) return kGemm32x64;
            if (S > 64 && tiles(128, 128) <= cus) return kGemm128x128;
            return kGemm64x128;
        }
    }
    // a last, partly filled tile for every other expert
    const int64_t few = (S / 32 + used / 2) * ((N + 255) / 256);
    return few <= cus ? kGemm32x256 : kGemm64x256;
}

// ------------------------------------------------------------- bf16 and int8 products
// Tiles of so many weight rows x tokens: persistent ones of the kernel whose waves
// split the tile, and narrow ones of the kernel whose waves share k; those of 32 x 32 with
// three stages, or with two and two workgroups a CU.
enum ProductKernel {
    kProduct256x256,
    kProduct256x128,
    kProduct128x128,
    kProduct256x64,
    kProduct128x64,
    kNarrow64x64,
    kNarrow32x32,
    kNarrow32x32Paired,
    kProductKernels,
};
constexpr int kProductTiles = kNarrow64x64;      // the persistent ones come first
constexpr float kLookUs = 1.0f;                  // and look at the segments before

// What a tile takes on MI355X, us: `tile`, and `step` for each 128 bytes of k.  Fitted to 4970
// measured sizes (1 to 64 experts of 1 to 2500 rows on average, even, as even picks
// fall or by a Zipf law, 64 to 8192 weight rows, 128 to 8192 values of k, bf16 either way
// round, gated and int8, weights from memory), before last rounds in pieces and 256 x 256 tiles
// past the caches were there.  Of 12751 other such sizes, on the kernels as they are: what is
// chosen by them takes 1.5% longer than the best on average, 14% at the 97th percentile,
// 1.7 times as long at the worst; with the row tiles estimated from sizes, and not counted
// in the segments, 2.2%, 18% and 2.4 times.  What the best of the others takes without one of
// them, on average and at the worst: 256 x 256 2.0% and 59%, 256 x 128 0.7% and 38%, 128 x 128
// 0.8% and 48%, 256 x 64 0.5% and 23%, 128 x 64 1.4% and 36%, narrow 64 x 64 1.4% and 64%, 32 x
// 32 2.7% and 63%, paired 2.2% and 46%.  With 128 and 256 experts, 12 sizes, the best or
// within 4% of it.
// For instance, us (bf16, weights from memory; narrow 32 x 32 with three stages / paired):
//                                          256x256 256x128 128x128 256x64 128x64   32x32
//   8 experts x 4096 x 7168, 8 rows each      122      98      71      93     70   86 / 81
//   16 x 2816 x 4096, 64                        80      63      85      62     77
//   16 x 2816 x 4096, 128                       85      68      98     107
//   8 x 4096 x 7168, 500                       186     219     291
//   1 x 4096 x 4096, 1024                       76      55      41      47
//   4 x 2048 x 4096, 40                                 52      33      49     31   23 / 18
//   1 x 4096 x 7168, 8                                          49      80     45   17 / 23
//   1 x 512 x 512, 8                                                              3.8 / 3.5
struct ProductTile {
    int weights, tokens, groups;     // groups: workgroups a CU
    float step, tile;
};
EP_BOTH ProductTile product_tile(int kernel)
{
    constexpr ProductTile tiles[kProductKernels] = {
        {256, 256, 1, 1.11f, 4.6f}, {256, 128, 1, 0.83f, 2.05f}, {128, 128, 1, 0.46f, 2.3f},
        {256, 64, 1, 0.725f, 1.4f}, {128, 64, 1, 0.40f, 1.0f},   {64, 64, 1, 0.39f, 2.05f},
        {32, 32, 1, 0.355f, 2.5f},  {32, 32, 2, 0.395f, 1.8f},
    };
    return tiles[kernel];
}
// The same for all tiles, on so many CUs at once.
EP_BOTH float product_us(int kernel, float tiles, int blocks, int cus)
{
    const ProductTile t = product_tile(kernel);
    tiles = tiles < 1e9f ? tiles : 1e9f;         // an integer holds them
    float rounds = tiles / float(cus * t.groups);
    if (kernel < kProductTiles) {
        // each XCD has an eighth of the tiles, and its workgroups take them in turn
        const int share = (int(tiles) + 7) / 8, slots = cus / 8;
        rounds = float((share + slots - 1) / slots);
    } else if (rounds < 1.0f) {
        rounds = 1.0f;
    }
    return rounds * (t.tile + float(blocks) * t.step);
}

// The persistent tile for segments that make so many row tiles of 64, 128 and 256
// rows, n tiles of `weights` (gated: half as many columns) each.
EP_BOTH int choose_product_tile(int tiles64, int tiles128, int tiles256, int N, int blocks, bool gated,
                                int cus)
{
    int best = 0;
    float least = 0.0f;
    for (int k = 0; k < kProductTiles; ++k) {
        const ProductTile t = product_tile(k);
        const int columns = gated ? t.weights / 2 : t.weights;
        const int rows = t.tokens == 64 ? tiles64 : t.tokens == 128 ? tiles128 : tiles256;
        const float us = product_us(k, float(rows) * float((N + columns - 1) / columns), blocks, cus);
        if (k == 0 || us < least) {
            least = us;
            best = k;
        }
    }
    return best;
}

// The last, partly filled round of 256 x 256 tiles, `rest` of them for `slots` CUs: how often
// their rows are halved, as long as one round of the pieces holds them (256 x 128 and 256 x 64,
// a workgroup that has a piece through in two thirds of the time).  us whole / in pieces:
// 8 experts x 4096 x 7168, 500 rows each as picks fall 292 / 248; 2 x 7168 (gated) x 1408, 718
// rows 69 / 63; 16 x 2816 x 1408, 1433 rows by a Zipf law 190 / 174; int8 8 x 2048 x 4096, 1431
// rows 102 / 97; no size took longer in pieces.  Counted in the estimates above it
// would take 256 x 256 where 256 x 128 is faster (8 x 2048 (gated) x 4096, 598 rows 148 / 164).
EP_BOTH int product_tail(int rest, int slots)
{
    return rest * 4 <= slots ? 2 : rest * 2 <= slots ? 1 : 0;
}

// Whether such a tile reads the weights past the caches: where each of them is read once.
// Past / through the caches, weights from memory: 0.89 to 0.96 with 64 MB and more, 0.87 to 0.98
// with less (but 33 MB that the last call left there would take 15 us instead of 11); with
// more rows than a tile holds 1.0 to 1.2; with rows of k that do not begin on lines 1.0 to
// 1.15.  256 x 256, where this also gives every tile of weights a turn of k: 0.73 to 0.88 at
// sizes that are powers of two (16 experts x 4096 x 4096, 256 rows 144 / 123 us; 64 x 2048 x
// 2048, 220 rows 166 / 121), 0.98 on average at any.
EP_BOTH bool product_past_caches(int row_tiles, int used, bool whole_lines)
{
    return whole_lines && row_tiles <= used;
}

// Whether a call takes the persistent kernel, which looks at the segments itself, or a
// narrow one.  The host knows sizes only: rows on as many experts as even picks fall on,
// spread evenly between 0.4 and 1.6 of the average, and their square root more or less.
// N: columns of the result; row_bytes: of a row of k; gated: 2 N weight rows.
inline int choose_product(int64_t S, int64_t N, int64_t row_bytes, int64_t E, bool gated, int64_t cus)
{
    const double used = fmax(double(E) * (1.0 - pow(1.0 - 1.0 / double(E), double(S))), 1.0);
    const double rows = double(S) / used;
    const int blocks = int((row_bytes + 127) / 128);
    auto upto = [](double x) {               // integral of ceil from 0
        return x <= 0.0 ? 0.0 : floor(x) * (floor(x) + 1.0) / 2.0 + ceil(x) * (x - floor(x));
    };
    int best = 0;
    float least = 0.0f;
    for (int k = 0; k < kProductKernels; ++k) {
        const ProductTile t = product_tile(k);
        const int64_t columns = gated ? t.weights / 2 : t.weights;
        const double high = (1.6 * rows + sqrt(rows)) / t.tokens;
        const double low = fmax((0.4 * rows - sqrt(rows)) / t.tokens, 0.0);
        double each = used == 1.0 ? ceil(rows / t.tokens) : (upto(high) - upto(low)) / (high - low);
        if (each < 1.0) each = 1.0;
        const double tiles = ceil(fmin(used * each, double(S)) * double((N + columns - 1) / columns));
        const float us = product_us(k, float(tiles), blocks, int(cus > 8 ? cus : 8)) +
                         (k < kProductTiles ? kLookUs : 0.0f);
        if (k == 0 || us < least) {
            least = us;
            best = k < kProductTiles ? 0 : k;
        }
    }
    return best;
}

// The most tiles that a call can make, of the smallest persistent shape.  Their numbers are kept in
// 32 bits: sizes that can make 2^30 are refused (their y or h would take 8 TB and more).
inline int64_t product_most_tiles(int64_t S, int64_t N, int64_t E, bool gated)
{
    const int64_t columns = gated ? 64 : 128;
    return (S / 64 + (E < S ? E : S)) * ((N + columns - 1) / columns);
}
constexpr int64_t kProductMostTiles = int64_t(1) << 30;

// Whether the weights' rows begin on lines and are more than the caches keep until the
// next call.
inline bool product_whole_lines(int64_t N, int64_t row_bytes, int64_t E, bool gated, int64_t line_bytes)
{
    return (gated ? 2 : 1) * E * N * row_bytes > kStreamBytes && line_bytes % 128 == 0;
}

// ------------------------------------------------------------- weight gradients
constexpr int kWgradTile = 256, kWgradSmallTile = 128;

inline int64_t wgrad_tiles(int N, int K, int E, int tile)
{
    return int64_t((N + tile - 1) / tile) * ((K + tile - 1) / tile) * E;
}

// Large tiles want a whole round of them and rows enough to hide their stores
// (16 experts x 2816 x 4096, large / small tiles: 128 rows each 134 / 122 us, 176
// rows 150 / 139, 256 rows 155 / 163; 8 experts x 1024 x 1024, half a round: 256 rows
// 14.5 / 13.0, but 4096 rows 85 / 100).
inline bool wgrad_large(int S, int N, int K, int E)
{
    return wgrad_tiles(N, K, E, kWgradTile) >= 256 && S >= int64_t(192) * E;
}

// Parts that an expert's rows are split into: 1, unless there are few small
// tiles (up to 192, towards 768 workgroups) and rows for several parts of 128.
// 32768 rows, 256 x 512 (8 tiles): 390 us whole, 35 in 64 parts; 4 experts of 4096
// rows, 512 x 512 (64 tiles): 52, 27 in 12; 8 of 4096, 512 x 1024 (256): 57, 69 in 3.
// From sizes alone, so that a workspace's size holds on every device.
inline int wgrad_parts(int S, int N, int K, int E)
{
    if (wgrad_large(S, N, K, E)) return 1;
    const int64_t tiles = wgrad_tiles(N, K, E, kWgradSmallTile);
    if (tiles > 192) return 1;
    const int64_t most = 768 / tiles, rows = S / (int64_t(128) * E);
    const int64_t parts = most < rows ? most : rows;
    return parts < 2 ? 1 : parts > 64 ? 64 : int(parts);
}

}  // namespace ep
