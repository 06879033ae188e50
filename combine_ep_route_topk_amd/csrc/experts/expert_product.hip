// expert_product.hip -- grouped products of bf16 and of 8-bit integers over expert
// segments: which shape of expert_product.h's kernel a call takes.
#include "expert_choice.h"
#include "expert_product.h"

namespace ep {
namespace {

template <class T, ProductKind KIND>
hipError_t launch(const ProductArgs& p, hipStream_t s)
{
    switch (choose_product(p.S, p.N, int64_t(p.K) * T::kBytes, p.E, KIND >= kGated, device_cu_count())) {
        case kNarrow64x64: return launch_narrow<NarrowShape<T, KIND, 2, 2, 2>>(p, s);
        case kNarrow32x32: return launch_narrow<NarrowShape<T, KIND, 1, 1, 3>>(p, s);
        case kNarrow32x32Paired: return launch_narrow<NarrowShape<T, KIND, 1, 1, 2>>(p, s);
        default: return launch_product<T, KIND>(p, s);
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
