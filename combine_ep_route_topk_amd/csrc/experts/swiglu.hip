// swiglu.hip -- the gradient of the gated activation h = silu(g) * u.
//
// With sig = 1 / (1 + exp(-g)) and silu = g sig:
//   dg = dh u (sig + silu (1 - sig)),   du = dh silu,   h = silu u.
// One pass: 3 I values read and 3 I written for each row (h is what the
// second weight's gradient needs, and recomputing it here costs no extra
// read).  All arithmetic is f32; each output rounds once.
//
// HBM-bound, nothing is used twice: loads and stores past the caches, one 16-byte
// piece a thread.  32768 rows of 2048 on MI355X: 130 us, 6.2 TB/s (with a grid of
// 16 workgroups a CU that goes round: 142; through the caches besides: 152).
#include "experts_internal.h"

namespace ep {
namespace {

__global__ __launch_bounds__(kBlock) void swiglu_grad_kernel(
    const uint16_t* __restrict__ grad_h, const uint16_t* __restrict__ gate_up, int64_t vecs,
    int I, int rowvecs, uint16_t* __restrict__ grad_gate_up, uint16_t* __restrict__ h)
{
    for (int64_t i = int64_t(blockIdx.x) * kBlock + threadIdx.x; i < vecs;
         i += int64_t(gridDim.x) * kBlock) {
        const int64_t row = i / rowvecs;
        const int c = int(i - row * rowvecs) * 8;
        const int64_t at = row * 2 * I + c;
        const u32x4 g = load16_nt(gate_up + at), u = load16_nt(gate_up + at + I);
        const u32x4 d = load16_nt(grad_h + row * I + c);
        u32x4 dg, du, o;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            float a[2], b[2], hh[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const float gv = q ? bf16_hi(g[p]) : bf16_lo(g[p]);
                const float uv = q ? bf16_hi(u[p]) : bf16_lo(u[p]);
                const float dv = q ? bf16_hi(d[p]) : bf16_lo(d[p]);
                const float sig = sigmoid(gv), silu = gv * sig;
                a[q] = dv * uv * (sig + silu * (1.0f - sig));
                b[q] = dv * silu;
                hh[q] = silu * uv;
            }
            dg[p] = pack_bf16x2(a[0], a[1]);
            du[p] = pack_bf16x2(b[0], b[1]);
            o[p] = pack_bf16x2(hh[0], hh[1]);
        }
        store16_nt(grad_gate_up + at, dg);
        store16_nt(grad_gate_up + at + I, du);
        if (h) store16_nt(h + row * I + c, o);
    }
}

}  // namespace

hipError_t launch_swiglu_grad(const uint16_t* grad_h, const uint16_t* gate_up, int S, int I,
                              uint16_t* grad_gate_up, uint16_t* h, hipStream_t s)
{
    const int64_t vecs = int64_t(S) * (I / 8);
    const int64_t want = (vecs + kBlock - 1) / kBlock;
    const uint32_t grid = want < (1 << 20) ? uint32_t(want) : 1u << 20;
    EP_LAUNCH(swiglu_grad_kernel, dim3(grid), dim3(kBlock), 0, s, grad_h, gate_up, vecs, I, I / 8,
              grad_gate_up, h);
    return hipGetLastError();
}

}  // namespace ep
