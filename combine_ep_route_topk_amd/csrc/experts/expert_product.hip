// expert_product.hip -- grouped products of bf16 and of 8-bit integers over expert
// segments: which shape of expert_product.h's kernel a call takes.
#include "expert_choice.h"
#include "expert_product.h"

namespace ep {
namespace {

// Tiles whose k starts at another block for each tile of weights: rows a power of two
// apart would keep to a few memory channels (16 experts x 2816 x 4096 of bf16, 128 rows
// each, 256 x 128 tiles: 78 us instead of 88, past the caches 67).  The 256 x 256 tiles,
// bound by matrix work, share more through L2 without (500 rows, 8 x 4096 x 7168: 186, 200).
template <class T, ProductKind KIND, int FN, int FM, int WN, int STAGES>
hipError_t launch_turning(const ProductArgs& p, hipStream_t s)
{
    typedef ProductShape<T, KIND, FN, FM, WN, STAGES, true, false> Cached;
    typedef ProductShape<T, KIND, FN, FM, WN, STAGES, true, true> Past;
    const int64_t row_bytes = int64_t(p.K) * T::kBytes;
    const int64_t line_bytes = KIND == kTransposed ? int64_t(p.N) * T::kBytes : row_bytes;
    if (product_past_caches(p.S, p.N, row_bytes, p.E, KIND >= kGated, line_bytes, Cached::TM))
        return launch_product<Past>(p, s);
    return launch_product<Cached>(p, s);
}

template <class T, ProductKind KIND>
hipError_t launch(const ProductArgs& p, hipStream_t s)
{
    switch (choose_product(p.S, p.N, int64_t(p.K) * T::kBytes, p.E, KIND >= kGated, device_cu_count())) {
        case kProduct256x256: return launch_product<ProductShape<T, KIND, 4, 4, 2, 3, false, false>>(p, s);
        case kProduct256x128: return launch_turning<T, KIND, 4, 2, 2, 3>(p, s);
        case kProduct128x128: return launch_turning<T, KIND, 2, 2, 2, 3>(p, s);
        case kProduct256x64: return launch_turning<T, KIND, 2, 2, 4, 3>(p, s);
        case kProduct128x64: return launch_turning<T, KIND, 2, 1, 2, 4>(p, s);
        case kNarrow64x64: return launch_narrow<NarrowShape<T, KIND, 2, 2, 2>>(p, s);
        case kNarrow32x64: return launch_narrow<NarrowShape<T, KIND, 1, 2, 3>>(p, s);
        case kNarrow32x32: return launch_narrow<NarrowShape<T, KIND, 1, 1, 3>>(p, s);
        default: return hipErrorInvalidConfiguration;
    }
}

}  // namespace

hipError_t launch_expert_gemm_bf16(const uint16_t* a, const uint16_t* w, const int32_t* offsets,
                                   int S, int N, int K, int E, bool transposed, uint16_t* y,
                                   hipStream_t s)
{
    const ProductArgs p{reinterpret_cast<const uint8_t*>(a), nullptr,
                        reinterpret_cast<const uint8_t*>(w), nullptr, offsets, S, N, K, E, 0, y,
                        nullptr};
    return transposed ? launch<Bf16, kTransposed>(p, s) : launch<Bf16, kPlain>(p, s);
}

hipError_t launch_expert_swiglu_bf16(const uint16_t* a, const uint16_t* w13, const int32_t* offsets,
                                     int S, int I, int K, int E, uint16_t* h, uint16_t* gate_up,
                                     hipStream_t s)
{
    const ProductArgs p{reinterpret_cast<const uint8_t*>(a), nullptr,
                        reinterpret_cast<const uint8_t*>(w13), nullptr, offsets, S, I, K, E, 0,
                        gate_up, h};
    return gate_up ? launch<Bf16, kGatedSaved>(p, s) : launch<Bf16, kGated>(p, s);
}

hipError_t launch_expert_gemm_int8(const int8_t* a, const float* a_scale, const int8_t* w,
                                   const float* w_scale, const int32_t* offsets, int S, int N, int K,
                                   int E, uint16_t* y, hipStream_t s)
{
    return launch<Int8, kPlain>(
        ProductArgs{reinterpret_cast<const uint8_t*>(a), a_scale, reinterpret_cast<const uint8_t*>(w),
                    w_scale, offsets, S, N, K, E, 0, y, nullptr}, s);
}

hipError_t launch_expert_swiglu_int8(const int8_t* a, const float* a_scale, const int8_t* w13,
                                     const float* w13_scale, const int32_t* offsets, int S, int I,
                                     int K, int E, uint16_t* h, hipStream_t s)
{
    return launch<Int8, kGated>(
        ProductArgs{reinterpret_cast<const uint8_t*>(a), a_scale,
                    reinterpret_cast<const uint8_t*>(w13), w13_scale, offsets, S, I, K, E, 0, nullptr,
                    h}, s);
}

}  // namespace ep
