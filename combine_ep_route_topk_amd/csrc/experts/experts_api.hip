// experts_api.hip -- the extern "C" entry points of the expert operators
// (include/ep_route_topk.h): argument validation, then kernel launches.
#include "../ep_api.h"
#include "expert_choice.h"
#include "experts_internal.h"

namespace {

using ep::fail;
using ep::launched;
using ep::ok;
using ep::TimingScope;

// S rows of E segments against weights [E][N][K]; rows of `step` values.
ep_status check_expert_sizes(const char* fn, int32_t S, int32_t N, int32_t K, int32_t E,
                             int32_t step, const char* n_name, const char* k_name)
{
    if (S < 0) return fail(EP_ERR_INVALID_ARG, "%s: S=%d must be >= 0", fn, S);
    if (S >= (1 << 30)) return fail(EP_ERR_UNSUPPORTED, "%s: S=%d must be < 2^30", fn, S);
    if (E < 1) return fail(EP_ERR_INVALID_ARG, "%s: E=%d must be >= 1", fn, E);
    if (E > ep::kMaxE) return fail(EP_ERR_UNSUPPORTED, "%s: E=%d exceeds %d", fn, E, ep::kMaxE);
    if (N < step || N % step != 0)
        return fail(EP_ERR_INVALID_ARG, "%s: %s=%d must be a positive multiple of %d", fn, n_name, N,
                    step);
    if (K < step || K % step != 0)
        return fail(EP_ERR_INVALID_ARG, "%s: %s=%d must be a positive multiple of %d", fn, k_name, K,
                    step);
    if (N > (1 << 17) || K > (1 << 17))
        return fail(EP_ERR_UNSUPPORTED, "%s: %s=%d and %s=%d must not exceed 2^17", fn, n_name, N,
                    k_name, K);
    return EP_OK;
}

#define EP_REQUIRE_ALIGNED(fn, p, a)                                                     \
    do {                                                                                 \
        if ((p) && !::ep::aligned((p), (a)))                                             \
            return ::ep::fail(EP_ERR_INVALID_ARG, "%s: %s is not %d-byte aligned", fn, #p, \
                              int(a));                                                   \
    } while (0)

ep_status check_quantize(const char* fn, int32_t T, int32_t H, int32_t k)
{
    if (k < 1) return fail(EP_ERR_INVALID_ARG, "%s: k=%d must be >= 1", fn, k);
    if (k > ep::kMaxK) return fail(EP_ERR_UNSUPPORTED, "%s: k=%d exceeds %d", fn, k, ep::kMaxK);
    if (H < 16 || H % 16 != 0)
        return fail(EP_ERR_INVALID_ARG, "%s: H=%d must be a positive multiple of 16", fn, H);
    if (H > (1 << 20)) return fail(EP_ERR_UNSUPPORTED, "%s: H=%d exceeds 2^20", fn, H);
    if (int64_t(T) * k >= (int64_t(1) << 30))
        return fail(EP_ERR_UNSUPPORTED, "%s: T*k=%lld must be < 2^30", fn, (long long)T * k);
    if (int64_t(T) * H >= (int64_t(1) << 40))
        return fail(EP_ERR_UNSUPPORTED, "%s: T*H=%lld must be < 2^40", fn, (long long)T * H);
    return EP_OK;
}

// A sum of K products of two 8-bit integers stays below 2^31.
ep_status check_int8_sum(const char* fn, int32_t K)
{
    if (K >= (1 << 17))
        return fail(EP_ERR_UNSUPPORTED, "%s: K=%d must be < 2^17 in 8-bit integers", fn, K);
    return EP_OK;
}

}  // namespace

extern "C" {

ep_status ep_quantize_fp8(const uint16_t* x, int32_t S, int32_t H, uint8_t* q, uint8_t* scale,
                          void* stream)
{
    const char* fn = "ep_quantize_fp8";
    TimingScope timing_scope;
    if (S < 0) return fail(EP_ERR_INVALID_ARG, "%s: S=%d must be >= 0", fn, S);
    EP_TRY(check_quantize(fn, S, H, 1));
    if (S == 0) return ok();
    EP_REQUIRE_PTR(fn, x, 16);
    EP_REQUIRE_PTR(fn, q, 16);
    EP_REQUIRE_PTR(fn, scale, 1);
    return launched(ep::launch_quantize_rows(x, S, H, 1, nullptr, q, scale,
                                             static_cast<hipStream_t>(stream)),
                    fn);
}

ep_status ep_dispatch_fp8(const uint16_t* x, int32_t T, int32_t H, int32_t k, const int32_t* pos,
                          uint8_t* send, uint8_t* scale, void* stream)
{
    const char* fn = "ep_dispatch_fp8";
    TimingScope timing_scope;
    if (T < 1) return fail(EP_ERR_INVALID_ARG, "%s: T=%d must be >= 1", fn, T);
    EP_TRY(check_quantize(fn, T, H, k));
    EP_REQUIRE_PTR(fn, x, 16);
    EP_REQUIRE_PTR(fn, pos, 4);
    EP_REQUIRE_PTR(fn, send, 16);
    EP_REQUIRE_PTR(fn, scale, 1);
    return launched(ep::launch_quantize_rows(x, T, H, k, pos, send, scale,
                                             static_cast<hipStream_t>(stream)),
                    fn);
}

ep_status ep_quantize_weight_fp8(const uint16_t* w, int32_t E, int32_t N, int32_t K, uint8_t* q,
                                 uint8_t* scale, uint8_t* q_t, uint8_t* scale_t, void* stream)
{
    const char* fn = "ep_quantize_weight_fp8";
    TimingScope timing_scope;
    EP_TRY(check_expert_sizes(fn, 0, N, K, E, 16, "N", "K"));
    EP_REQUIRE_PTR(fn, w, 16);
    EP_REQUIRE_PTR(fn, q, 16);
    EP_REQUIRE_PTR(fn, scale, 1);
    if ((q_t == nullptr) != (scale_t == nullptr))
        return fail(EP_ERR_INVALID_ARG, "%s: q_t and scale_t go together", fn);
    EP_REQUIRE_ALIGNED(fn, q_t, 16);
    return launched(ep::launch_quantize_weight(w, E, N, K, q, scale, q_t, scale_t,
                                               static_cast<hipStream_t>(stream)),
                    fn);
}

ep_status ep_expert_gemm_fp8(const uint8_t* a, const uint8_t* a_scale, const uint8_t* w,
                             const uint8_t* w_scale, const int32_t* expert_offsets, int32_t S,
                             int32_t N, int32_t K, int32_t E, uint16_t* y, void* stream)
{
    const char* fn = "ep_expert_gemm_fp8";
    TimingScope timing_scope;
    EP_TRY(check_expert_sizes(fn, S, N, K, E, 16, "N", "K"));
    if (S == 0) return ok();
    EP_REQUIRE_PTR(fn, a, 16);
    EP_REQUIRE_PTR(fn, a_scale, 1);
    EP_REQUIRE_PTR(fn, w, 16);
    EP_REQUIRE_PTR(fn, w_scale, 1);
    EP_REQUIRE_PTR(fn, expert_offsets, 4);
    EP_REQUIRE_PTR(fn, y, 16);
    return launched(ep::launch_expert_gemm(a, a_scale, w, w_scale, expert_offsets, S, N, K, E, y,
                                           static_cast<hipStream_t>(stream)),
                    fn);
}

ep_status ep_expert_swiglu_fp8(const uint8_t* a, const uint8_t* a_scale, const uint8_t* w13,
                               const uint8_t* w13_scale, const int32_t* expert_offsets, int32_t S,
                               int32_t I, int32_t K, int32_t E, uint8_t* h, uint8_t* h_scale,
                               uint16_t* gate_up, void* stream)
{
    const char* fn = "ep_expert_swiglu_fp8";
    TimingScope timing_scope;
    EP_TRY(check_expert_sizes(fn, S, I, K, E, 16, "I", "K"));
    if (I % ep::kScaleBlock != 0)
        return fail(EP_ERR_INVALID_ARG, "%s: I=%d must be a multiple of %d", fn, I,
                    ep::kScaleBlock);
    if (int64_t(I) * 2 * K >= (int64_t(1) << 31))
        return fail(EP_ERR_UNSUPPORTED, "%s: 2*I*K=%lld must be < 2^31", fn, (long long)I * 2 * K);
    if (S == 0) return ok();
    EP_REQUIRE_PTR(fn, a, 16);
    EP_REQUIRE_PTR(fn, a_scale, 1);
    EP_REQUIRE_PTR(fn, w13, 16);
    EP_REQUIRE_PTR(fn, w13_scale, 1);
    EP_REQUIRE_PTR(fn, expert_offsets, 4);
    EP_REQUIRE_PTR(fn, h, 16);
    EP_REQUIRE_PTR(fn, h_scale, 1);
    EP_REQUIRE_ALIGNED(fn, gate_up, 16);
    return launched(ep::launch_expert_swiglu(a, a_scale, w13, w13_scale, expert_offsets, S, I, K, E,
                                             h, h_scale, gate_up, static_cast<hipStream_t>(stream)),
                    fn);
}

size_t ep_expert_wgrad_workspace_bytes(int32_t S, int32_t N, int32_t K, int32_t E)
{
    if (S < 1 || N < 8 || K < 8 || E < 1) return 0;
    const int parts = ep::wgrad_parts(S, N, K, E);
    return parts > 1 ? size_t(parts) * E * N * K * sizeof(float) : 0;
}

ep_status ep_expert_wgrad(const uint16_t* grad_y, const uint16_t* x, const int32_t* expert_offsets,
                          int32_t S, int32_t N, int32_t K, int32_t E, int32_t accumulate,
                          float* grad_w, void* workspace, size_t workspace_bytes, void* stream)
{
    const char* fn = "ep_expert_wgrad";
    TimingScope timing_scope;
    EP_TRY(check_expert_sizes(fn, S, N, K, E, 8, "N", "K"));
    if (S > 0) {
        EP_REQUIRE_PTR(fn, grad_y, 16);
        EP_REQUIRE_PTR(fn, x, 16);
    }
    EP_REQUIRE_PTR(fn, expert_offsets, 4);
    EP_REQUIRE_PTR(fn, grad_w, 16);
    const size_t need = ep_expert_wgrad_workspace_bytes(S, N, K, E);
    if (workspace) {
        EP_REQUIRE_ALIGNED(fn, workspace, 256);
        if (workspace_bytes < need)
            return fail(EP_ERR_WORKSPACE, "%s: workspace has %zu bytes, needs %zu", fn,
                        workspace_bytes, need);
    }
    return launched(ep::launch_expert_wgrad(grad_y, x, expert_offsets, S, N, K, E,
                                            accumulate ? 1 : 0, grad_w,
                                            need ? static_cast<float*>(workspace) : nullptr,
                                            static_cast<hipStream_t>(stream)),
                    fn);
}

ep_status ep_swiglu_grad(const uint16_t* grad_h, const uint16_t* gate_up, int32_t S, int32_t I,
                         uint16_t* grad_gate_up, uint16_t* h, void* stream)
{
    const char* fn = "ep_swiglu_grad";
    TimingScope timing_scope;
    EP_TRY(check_expert_sizes(fn, S, I, I, 1, 8, "I", "I"));
    if (S == 0) return ok();
    EP_REQUIRE_PTR(fn, grad_h, 16);
    EP_REQUIRE_PTR(fn, gate_up, 16);
    EP_REQUIRE_PTR(fn, grad_gate_up, 16);
    EP_REQUIRE_ALIGNED(fn, h, 16);
    return launched(ep::launch_swiglu_grad(grad_h, gate_up, S, I, grad_gate_up, h,
                                           static_cast<hipStream_t>(stream)),
                    fn);
}

ep_status ep_expert_gemm_bf16(const uint16_t* a, const uint16_t* w, const int32_t* expert_offsets,
                              int32_t S, int32_t N, int32_t K, int32_t E, int32_t transposed,
                              uint16_t* y, void* stream)
{
    const char* fn = "ep_expert_gemm_bf16";
    TimingScope timing_scope;
    EP_TRY(check_expert_sizes(fn, S, N, K, E, 8, "N", "K"));
    if (S == 0) return ok();
    EP_REQUIRE_PTR(fn, a, 16);
    EP_REQUIRE_PTR(fn, w, 16);
    EP_REQUIRE_PTR(fn, expert_offsets, 4);
    EP_REQUIRE_PTR(fn, y, 16);
    return launched(ep::launch_expert_gemm_bf16(a, w, expert_offsets, S, N, K, E, transposed != 0, y,
                                                static_cast<hipStream_t>(stream)),
                    fn);
}

ep_status ep_expert_swiglu_bf16(const uint16_t* a, const uint16_t* w13, const int32_t* expert_offsets,
                                int32_t S, int32_t I, int32_t K, int32_t E, uint16_t* h,
                                uint16_t* gate_up, void* stream)
{
    const char* fn = "ep_expert_swiglu_bf16";
    TimingScope timing_scope;
    EP_TRY(check_expert_sizes(fn, S, I, K, E, 8, "I", "K"));
    if (S == 0) return ok();
    EP_REQUIRE_PTR(fn, a, 16);
    EP_REQUIRE_PTR(fn, w13, 16);
    EP_REQUIRE_PTR(fn, expert_offsets, 4);
    EP_REQUIRE_PTR(fn, h, 16);
    EP_REQUIRE_ALIGNED(fn, gate_up, 16);
    return launched(ep::launch_expert_swiglu_bf16(a, w13, expert_offsets, S, I, K, E, h, gate_up,
                                                  static_cast<hipStream_t>(stream)),
                    fn);
}

ep_status ep_quantize_int8(const uint16_t* x, int32_t S, int32_t H, int8_t* q, float* scale,
                           void* stream)
{
    const char* fn = "ep_quantize_int8";
    TimingScope timing_scope;
    if (S < 0) return fail(EP_ERR_INVALID_ARG, "%s: S=%d must be >= 0", fn, S);
    EP_TRY(check_quantize(fn, S, H, 1));
    if (S == 0) return ok();
    EP_REQUIRE_PTR(fn, x, 16);
    EP_REQUIRE_PTR(fn, q, 16);
    EP_REQUIRE_PTR(fn, scale, 4);
    return launched(ep::launch_quantize_rows_int8(x, S, H, 1, nullptr, nullptr, nullptr, q, scale,
                                                  static_cast<hipStream_t>(stream)),
                    fn);
}

ep_status ep_dispatch_int8(const uint16_t* x, int32_t T, int32_t H, int32_t k, const int32_t* pos,
                           int8_t* send, float* scale, void* stream)
{
    const char* fn = "ep_dispatch_int8";
    TimingScope timing_scope;
    if (T < 1) return fail(EP_ERR_INVALID_ARG, "%s: T=%d must be >= 1", fn, T);
    EP_TRY(check_quantize(fn, T, H, k));
    EP_REQUIRE_PTR(fn, x, 16);
    EP_REQUIRE_PTR(fn, pos, 4);
    EP_REQUIRE_PTR(fn, send, 16);
    EP_REQUIRE_PTR(fn, scale, 4);
    return launched(ep::launch_quantize_rows_int8(x, T, H, k, pos, nullptr, nullptr, send, scale,
                                                  static_cast<hipStream_t>(stream)),
                    fn);
}

ep_status ep_expert_gemm_int8(const int8_t* a, const float* a_scale, const int8_t* w,
                              const float* w_scale, const int32_t* expert_offsets, int32_t S,
                              int32_t N, int32_t K, int32_t E, uint16_t* y, void* stream)
{
    const char* fn = "ep_expert_gemm_int8";
    TimingScope timing_scope;
    EP_TRY(check_expert_sizes(fn, S, N, K, E, 16, "N", "K"));
    EP_TRY(check_int8_sum(fn, K));
    if (S == 0) return ok();
    EP_REQUIRE_PTR(fn, a, 16);
    EP_REQUIRE_PTR(fn, a_scale, 4);
    EP_REQUIRE_PTR(fn, w, 16);
    EP_REQUIRE_PTR(fn, w_scale, 16);
    EP_REQUIRE_PTR(fn, expert_offsets, 4);
    EP_REQUIRE_PTR(fn, y, 16);
    return launched(ep::launch_expert_gemm_int8(a, a_scale, w, w_scale, expert_offsets, S, N, K, E, y,
                                                static_cast<hipStream_t>(stream)),
                    fn);
}

size_t ep_expert_swiglu_int8_workspace_bytes(int32_t S, int32_t I)
{
    return S < 1 || I < 1 ? 0 : size_t(S) * I * sizeof(uint16_t);
}

ep_status ep_expert_swiglu_int8(const int8_t* a, const float* a_scale, const int8_t* w13,
                                const float* w13_scale, const int32_t* expert_offsets, int32_t S,
                                int32_t I, int32_t K, int32_t E, int8_t* h, float* h_scale,
                                void* workspace, size_t workspace_bytes, void* stream)
{
    const char* fn = "ep_expert_swiglu_int8";
    TimingScope timing_scope;
    EP_TRY(check_expert_sizes(fn, S, I, K, E, 16, "I", "K"));
    EP_TRY(check_int8_sum(fn, K));
    if (S == 0) return ok();
    EP_REQUIRE_PTR(fn, a, 16);
    EP_REQUIRE_PTR(fn, a_scale, 4);
    EP_REQUIRE_PTR(fn, w13, 16);
    EP_REQUIRE_PTR(fn, w13_scale, 16);
    EP_REQUIRE_PTR(fn, expert_offsets, 4);
    EP_REQUIRE_PTR(fn, h, 16);
    EP_REQUIRE_PTR(fn, h_scale, 4);
    EP_REQUIRE_PTR(fn, workspace, 256);
    const size_t need = ep_expert_swiglu_int8_workspace_bytes(S, I);
    if (workspace_bytes < need)
        return fail(EP_ERR_WORKSPACE, "%s: workspace has %zu bytes, needs %zu", fn, workspace_bytes,
                    need);
    uint16_t* const rows = static_cast<uint16_t*>(workspace);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e = ep::launch_expert_swiglu_int8(a, a_scale, w13, w13_scale, expert_offsets, S, I, K, E,
                                                 rows, s);
    if (e == hipSuccess)
        e = ep::launch_quantize_rows_int8(rows, S, I, 1, nullptr, expert_offsets, expert_offsets + E, h,
                                          h_scale, s);
    return launched(e, fn);
}

size_t ep_moe_tokens_workspace_bytes(int32_t T, int32_t k, int32_t I)
{
    if (T < 1 || T > ep::kMoeMaxTokens || k < 1 || k > ep::kMaxK || I < 1) return 0;
    return ep::moe_tokens_workspace(T, k, I);
}

ep_status ep_moe_tokens(const uint16_t* x, const int32_t* topk_idx, const float* topk_w, int32_t T,
                        int32_t H, int32_t I, int32_t E, int32_t k, const void* w13,
                        const uint8_t* w13_scale, const void* w2, const uint8_t* w2_scale,
                        uint16_t* out, void* workspace, size_t workspace_bytes, void* stream)
{
    const char* fn = "ep_moe_tokens";
    TimingScope timing_scope;
    if (T < 1) return fail(EP_ERR_INVALID_ARG, "%s: T=%d must be >= 1", fn, T);
    if (T > ep::kMoeMaxTokens)
        return fail(EP_ERR_UNSUPPORTED,
                    "%s: T=%d exceeds %d (route, dispatch and the expert products take more)", fn, T,
                    ep::kMoeMaxTokens);
    EP_TRY(check_expert_sizes(fn, T, I, H, E, 16, "I", "H"));
    if (k < 1 || k > E) return fail(EP_ERR_INVALID_ARG, "%s: k=%d must be in [1, E=%d]", fn, k, E);
    if (k > ep::kMaxK) return fail(EP_ERR_UNSUPPORTED, "%s: k=%d exceeds %d", fn, k, ep::kMaxK);
    if ((w13_scale == nullptr) != (w2_scale == nullptr))
        return fail(EP_ERR_INVALID_ARG, "%s: w13_scale and w2_scale go together", fn);
    if (w13_scale && I % ep::kScaleBlock != 0)
        return fail(EP_ERR_INVALID_ARG, "%s: I=%d must be a multiple of %d with 8-bit weights", fn,
                    I, ep::kScaleBlock);
    EP_REQUIRE_PTR(fn, x, 16);
    EP_REQUIRE_PTR(fn, topk_idx, 4);
    EP_REQUIRE_PTR(fn, topk_w, 4);
    EP_REQUIRE_PTR(fn, w13, 16);
    EP_REQUIRE_PTR(fn, w2, 16);
    EP_REQUIRE_PTR(fn, out, 16);
    EP_REQUIRE_PTR(fn, workspace, 256);
    const size_t need = ep::moe_tokens_workspace(T, k, I);
    if (workspace_bytes < need)
        return fail(EP_ERR_WORKSPACE, "%s: workspace has %zu bytes, needs %zu", fn, workspace_bytes,
                    need);
    return launched(ep::launch_moe_tokens(x, topk_idx, topk_w, T, H, I, E, k, w13, w13_scale, w2,
                                          w2_scale, out, workspace,
                                          static_cast<hipStream_t>(stream)),
                    fn);
}

}  // extern "C"
