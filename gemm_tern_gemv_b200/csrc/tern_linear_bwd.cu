// Backward of the fused linear layer: dz = dy * act'(z), db = sum over rows of dz, dx = dz W.
#include "tern_layer.cuh"

namespace tern {
namespace {

// One thread per output feature walks the rows: dz rounded to fp16, db summed unrounded in fp32.
__global__ void __launch_bounds__(128) dz_kernel(const uint16_t* __restrict__ dy, const uint16_t* __restrict__ z,
                                                 int64_t m, int64_t n, int act, int gated, uint16_t* dz, float* db) {
  const int64_t nout = gated ? n / 2 : n;
  const int64_t o = (int64_t)blockIdx.x * 128 + threadIdx.x;
  if (o >= nout) return;
  double s0 = 0., s1 = 0.;
  for (int64_t t = 0; t < m; t++) {
    const float d = h2f(dy[t * nout + o]);
    const float a = z ? h2f(z[t * n + o]) : 0.f;
    if (gated) {
      const float u = h2f(z[t * n + o + nout]);
      const float g0 = d * u * act_bwd(act, a), g1 = d * act_fwd(act, a);
      s0 += g0;
      s1 += g1;
      dz[t * n + o] = f2h(g0);
      dz[t * n + o + nout] = f2h(g1);
    } else {
      const float g0 = d * act_bwd(act, a);
      s0 += g0;
      if (dz) dz[t * n + o] = f2h(g0);
    }
  }
  if (db) {
    db[o] = (float)s0;
    if (gated) db[o + nout] = (float)s1;
  }
}

// One thread per column k and row of dz.
__global__ void __launch_bounds__(128) dx_kernel(tern_matrix W, const uint16_t* __restrict__ dz, int64_t m, uint16_t* dx) {
  const int64_t k = (int64_t)blockIdx.x * 128 + threadIdx.x;
  const uint8_t* codes = static_cast<const uint8_t*>(W.codes);
  for (int64_t t = blockIdx.y; t < m; t += gridDim.y) {
    float acc = 0.f;
    for (int64_t n = 0; n < W.n; n++)
      acc = fmaf(h2f(dz[t * W.n + n]) * h2f(W.scales[n * W.scale_row_stride + blockIdx.x]),
                 decode_t(W.layout, codes + n * W.code_row_stride, k), acc);
    dx[t * W.k + k] = f2h(acc);
  }
}

}  // namespace

cudaError_t launch_linear_backward(const tern_matrix& W, const uint16_t* dy, const uint16_t* z, int64_t m, int act,
                                   int gated, uint16_t* dx, uint16_t* dz, float* db, uint32_t* status, cudaStream_t st) {
  (void)status;
  const int64_t nout = gated ? W.n / 2 : W.n;
  if (dz || db) {
    dz_kernel<<<(unsigned)((nout + 127) / 128), 128, 0, st>>>(dy, z, m, W.n, act, gated, dz, db);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (!dx) return cudaSuccess;
  const dim3 grid((unsigned)(W.k / kGroup), (unsigned)std::min<int64_t>(m, 65535));
  dx_kernel<<<grid, 128, 0, st>>>(W, dz ? dz : dy, m, dx);
  return cudaGetLastError();
}

}  // namespace tern
