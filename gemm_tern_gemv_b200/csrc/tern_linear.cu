// Fused linear layer y = act(W x + b) (+ residual), gated or not, on packed ternary weights.
#include "tern_layer.cuh"

namespace tern {
namespace {

constexpr int kTok = 4;  // rows of x per warp

// One warp per output feature (and its gate partner): lanes stride over K, fp32 accumulation.
__global__ void __launch_bounds__(128) linear_kernel(tern_matrix W, const uint16_t* __restrict__ x, int64_t m,
                                                     uint16_t* y, Epilogue e) {
  const int lane = threadIdx.x & 31;
  const int64_t nout = e.gated ? W.n / 2 : W.n;
  const int64_t o = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (o >= nout) return;
  const uint8_t* codes = static_cast<const uint8_t*>(W.codes);
  for (int64_t m0 = (int64_t)blockIdx.y * kTok; m0 < m; m0 += (int64_t)gridDim.y * kTok) {
    const int nt = (int)(m - m0 < kTok ? m - m0 : kTok);
    float acc[2][kTok] = {};
    for (int h = 0; h < (e.gated ? 2 : 1); h++) {
      const int64_t n = o + h * nout;
      for (int64_t k = lane; k < W.k; k += 32) {
        const float w = decode_t(W.layout, codes + n * W.code_row_stride, k) * h2f(W.scales[n * W.scale_row_stride + k / kGroup]);
        for (int i = 0; i < nt; i++) acc[h][i] = fmaf(w, h2f(x[(m0 + i) * W.k + k]), acc[h][i]);
      }
      for (int i = 0; i < kTok; i++)
        for (int s = 16; s; s >>= 1) acc[h][i] += __shfl_xor_sync(0xffffffffu, acc[h][i], s);
    }
    if (lane >= nt) continue;
    float z[2];
    for (int h = 0; h < 2; h++) {
      z[h] = acc[h][0];
      for (int i = 1; i < kTok; i++)
        if (lane == i) z[h] = acc[h][i];
    }
    const int64_t t = m0 + lane;
    if (e.bias) {
      z[0] += h2f(e.bias[o]);
      if (e.gated) z[1] += h2f(e.bias[o + nout]);
    }
    if (e.preact) {
      e.preact[t * W.n + o] = f2h(z[0]);
      if (e.gated) e.preact[t * W.n + o + nout] = f2h(z[1]);
    }
    float v = act_fwd(e.act, z[0]);
    if (e.gated) v *= z[1];
    if (e.residual) v += h2f(e.residual[t * nout + o]);
    y[t * nout + o] = f2h(v);
  }
}

}  // namespace

cudaError_t launch_linear(const tern_matrix& W, const uint16_t* x, int64_t m, uint16_t* y, const Epilogue& e,
                          uint32_t flags, uint32_t* status, cudaStream_t st) {
  (void)flags;
  (void)status;
  const int64_t nout = e.gated ? W.n / 2 : W.n;
  const dim3 grid((unsigned)((nout + 3) / 4), (unsigned)std::min<int64_t>((m + kTok - 1) / kTok, 65535));
  linear_kernel<<<grid, 128, 0, st>>>(W, x, m, y, e);
  return cudaGetLastError();
}

}  // namespace tern
