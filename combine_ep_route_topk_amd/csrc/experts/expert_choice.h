// expert_choice.h -- which kernel a grouped product or a weight gradient takes.
// Host rules on sizes alone, in a header of their own so that a test can ask
// which kernel its sizes reach.
#pragma once

#include <stdint.h>

namespace ep {

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
