// experts_internal.h -- launchers and device helpers of the expert operators:
// FP8 quantisation, grouped products over expert segments, their gradients,
// and the whole layer for a few tokens.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../ep_device.h"
#include "../ep_internal.h"
#include "expert_choice.h"

namespace ep {

// Values that share one scale: along a row of activations, and on both axes
// of a weight matrix.
constexpr int kScaleBlock = 128;
__host__ __device__ constexpr int scale_blocks(int n) { return (n + kScaleBlock - 1) / kScaleBlock; }

// Largest batch of the few-token layer.
constexpr int kMoeMaxTokens = 64;

// ----------------------------------------------------------------- launchers
hipError_t launch_quantize_rows(const uint16_t* x, int T, int H, int k, const int32_t* pos,
                                uint8_t* q, uint8_t* scale, hipStream_t s);
hipError_t launch_quantize_weight(const uint16_t* w, int E, int N, int K, uint8_t* q,
                                  uint8_t* scale, uint8_t* q_t, uint8_t* scale_t, hipStream_t s);
hipError_t launch_expert_gemm(const uint8_t* a, const uint8_t* a_scale, const uint8_t* w,
                              const uint8_t* w_scale, const int32_t* offsets, int S, int N, int K,
                              int E, uint16_t* y, hipStream_t s);
hipError_t launch_expert_swiglu(const uint8_t* a, const uint8_t* a_scale, const uint8_t* w13,
                                const uint8_t* w13_scale, const int32_t* offsets, int S, int I,
                                int K, int E, uint8_t* h, uint8_t* h_scale, uint16_t* gate_up,
                                hipStream_t s);
hipError_t launch_expert_wgrad(const uint16_t* grad_y, const uint16_t* x, const int32_t* offsets,
                               int S, int N, int K, int E, int accumulate, float* grad_w,
                               float* sums, hipStream_t s);
hipError_t launch_swiglu_grad(const uint16_t* grad_h, const uint16_t* gate_up, int S, int I,
                              uint16_t* grad_gate_up, uint16_t* h, hipStream_t s);
size_t moe_tokens_workspace(int T, int k, int I);
hipError_t launch_moe_tokens(const uint16_t* x, const int32_t* idx, const float* topk_w, int T,
                             int H, int I, int E, int k, const void* w13, const uint8_t* w13_scale,
                             const void* w2, const uint8_t* w2_scale, uint16_t* out, void* ws,
                             hipStream_t s);

hipError_t launch_expert_gemm_bf16(const uint16_t* a, const uint16_t* w, const int32_t* offsets,
                                   int S, int N, int K, int E, bool transposed, uint16_t* y,
                                   hipStream_t s);
hipError_t launch_expert_swiglu_bf16(const uint16_t* a, const uint16_t* w13, const int32_t* offsets,
                                     int S, int I, int K, int E, uint16_t* h, uint16_t* gate_up,
                                     hipStream_t s);
// `first` and `past` (both or neither): only the rows [*first, *past).
hipError_t launch_quantize_rows_int8(const uint16_t* x, int T, int H, int k, const int32_t* pos,
                                     const int32_t* first, const int32_t* past, int8_t* q,
                                     float* scale, hipStream_t s);
hipError_t launch_expert_gemm_int8(const int8_t* a, const float* a_scale, const int8_t* w,
                                   const float* w_scale, const int32_t* offsets, int S, int N, int K,
                                   int E, uint16_t* y, hipStream_t s);
hipError_t launch_expert_swiglu_int8(const int8_t* a, const float* a_scale, const int8_t* w13,
                                     const float* w13_scale, const int32_t* offsets, int S, int I,
                                     int K, int E, uint16_t* h, hipStream_t s);

// ----------------------------------------------------------------- device
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// The scale byte of a block whose largest magnitude is amax (finite, >= 0):
// the least power of two s with amax / s <= 448, e4m3's largest value.  With
// amax = f 2^e, 1 <= f < 2 and 448 = 1.75 * 2^8: s = 2^(e-8), or 2^(e-7) when
// f > 1.75; at least 2^-126; 1 for a block of zeros.  Since s is a power of
// two, x / s and q * s are exact and quantising rounds once.
__device__ __forceinline__ int scale_exponent(float amax) {
    const uint32_t b = __float_as_uint(amax);
    const int e = int(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u);
    return b == 0 ? 0 : (e < -126 ? -126 : e);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }

// Four f32 -> four e4m3 bytes (nearest even; a non-finite value becomes NaN).
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true));
}

__device__ __forceinline__ float max_finite(float m, float v) {
    v = fabsf(v);
    return v < __builtin_inff() ? fmaxf(m, v) : m;      // NaN and infinity leave m
}

// sigmoid(g): exp(-g) overflowing to infinity gives 0, its limit.
__device__ __forceinline__ float sigmoid(float g) {
    return __builtin_amdgcn_rcpf(1.0f + __expf(-g));
}

// ----------------------------------------------------------------- LDS
// 16 bytes per lane from offset `off` of the descriptor straight into LDS at
// `to` (wave-uniform) + 16 * lane; an offset past the descriptor stores zeros.
// NT: past the caches.
template <bool NT>
__device__ __forceinline__ void load16_to_lds(__amdgpu_buffer_rsrc_t r, uint8_t* to, uint32_t off) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)(to), 16,
                                             int(off), 0, 0, NT ? 2 : 0);
}
constexpr uint32_t kOutside = 0x80000000u;   // past every descriptor used here

// Transposing read: the 16 lanes of a group read 4 rows x 16 columns of 16-bit
// values (lane i its four at row i / 4, columns 4 (i % 4) ..); lane i receives
// column i's four.
typedef short s16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ s16x4 read_transposed(uint8_t* p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) s16x4*)(p));
}

// ----------------------------------------------------------------- order
// Waits until at most VM of this wave's vector-memory operations and none of
// its LDS reads are outstanding, then for the workgroup.
template <int VM>
__device__ __forceinline__ void wait_and_barrier() {
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt((VM & 15) | (7 << 4) | ((VM >> 4) << 14));
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// The wait alone, for loads into LDS of the wave's own.
template <int VM>
__device__ __forceinline__ void wait_loads() {
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt((VM & 15) | (7 << 4) | (15 << 8) | ((VM >> 4) << 14));
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_sched_barrier(0);
}

// Keeps a matrix instruction's result, and so the instruction, in its place.
template <class V>
__device__ __forceinline__ void pin(V& v) {
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("" : "+a"(v));
#endif
}

// Makes a value look new, so that nothing computed from it is moved before.
__device__ __forceinline__ void hide(int& v) {
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("" : "+v"(v));
#endif
}

// ----------------------------------------------------------------- segments
// Expert e's rows as clamped to the buffer: [begin, end) within [0, S], end
// not before begin, so that no offsets reach outside the row buffers.
__device__ __forceinline__ void segment_of(const int32_t* __restrict__ offsets, int e, int S,
                                           int& begin, int& end) {
    const int b = offsets[e], n = offsets[e + 1];
    begin = b < 0 ? 0 : (b > S ? S : b);
    end = n > S ? S : (n < begin ? begin : n);
}

struct RowTile {
    int expert;      // -1: past the last tile
    int row0, end;   // first row of the tile, end of the expert's rows
};

// Tile `index` of the experts' segments cut into tiles of TM rows, expert
// after expert (index < 2^30).  The whole wave takes part: lane i holds expert
// base + i.
__device__ __forceinline__ RowTile find_row_tile(const int32_t* __restrict__ offsets, int E, int S,
                                                 int TM, int index) {
    int seen = 0;
    for (int base = 0; base < E; base += kWave) {
        const int e = base + lane_id();
        int b = 0, n = 0;
        if (e < E) segment_of(offsets, e, S, b, n);
        int tiles = (n - b + TM - 1) / TM;
        tiles = tiles < (1 << 24) ? tiles : (1 << 24);
        const int upto = seen + wave_inclusive_sum(tiles);
        const uint64_t past = ballot(upto > index);
        if (past) {
            const int l = __builtin_ctzll(past);
            RowTile t;
            t.expert = base + l;
            const int first = __builtin_amdgcn_readlane(upto - tiles, l);
            t.row0 = __builtin_amdgcn_readlane(b, l) + (index - first) * TM;
            t.end = __builtin_amdgcn_readlane(n, l);
            return t;
        }
        seen = __builtin_amdgcn_readlane(upto, kWave - 1);
    }
    return RowTile{-1, 0, 0};
}

// Number of row tiles of all segments; at most `most`, which segments that do
// not overlap cannot pass (others, from offsets that decrease, are cut there).
__device__ __forceinline__ int count_row_tiles(const int32_t* __restrict__ offsets, int E, int S,
                                               int TM, int most) {
    int tiles = 0;
    for (int e = lane_id(); e < E; e += kWave) {
        int b, n;
        segment_of(offsets, e, S, b, n);
        tiles += (n - b + TM - 1) / TM;
        tiles = tiles < (1 << 24) ? tiles : (1 << 24);      // 64 lanes stay below 2^31
    }
    tiles = __builtin_amdgcn_readlane(wave_inclusive_sum(tiles), kWave - 1);
    return tiles < most ? tiles : most;
}

}  // namespace ep
