// Fused linear layer y = act(W x + b) (+ residual), gated or not, on packed ternary weights.
//
// Few rows of x (see few_rows): linear_rows_kernel, the register core of tern_rows.cuh. One CTA per SM
// owns a run of 16-row tiles (gated: 8 gate rows and their 8 up rows, so that both halves of an output meet
// in one thread); its warps cut K, their partial sums meet in shared memory in warp order, and the epilogue
// runs on the fp32 sums.
// More rows: the tensor-core kernel of tern_layer_gemm.cu.
#include "tern_rows.cuh"

namespace tern {
namespace {

__device__ __forceinline__ void epilogue(const Epilogue& e, int64_t n, int64_t nout, int64_t t, int64_t o, float z0, float z1,
                                         uint16_t* y) {
  if (e.bias) {
    z0 += h2f(e.bias[o]);
    if (e.gated) z1 += h2f(e.bias[o + nout]);
  }
  if (e.preact) {
    e.preact[t * n + o] = f2h(z0);
    if (e.gated) e.preact[t * n + o + nout] = f2h(z1);
  }
  float v = act_fwd(e.act, z0);
  if (e.gated) v *= z1;
  if (e.residual) v += h2f(e.residual[t * nout + o]);
  y[t * nout + o] = f2h(v);
}

struct RowsParams {
  rows::Mat mat;
  rows::Map map;
  rows::Split split;
  const uint16_t* x;
  uint16_t* y;
  Epilogue e;
  int64_t n, nout;
  int tiles, tokens, early;
  int each, extra;  // tiles of a CTA; `extra` of the CTAs have one more
};

template <int L, class P>
__global__ void __launch_bounds__(rows::kThreads, 1) linear_rows_kernel(const __grid_constant__ RowsParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  sm100::griddep_launch_dependents();
  if (!p.early) sm100::griddep_wait();
  const int b = (int)blockIdx.x, ctas = (int)gridDim.x;
  const int t0 = rows::first_tile(b, ctas, p.each, p.extra), t1 = rows::first_tile(b + 1, ctas, p.each, p.extra);
  const rows::HalfRows xs{p.x, p.mat.K, nullptr};
  P prod;
  prod.run(smem, p.split, p.mat, p.map, t0, t1, xs, p.tokens, [&] { if (p.early) sm100::griddep_wait(); },
           [&](int tile, int r, int t, float z0, float z1) {
             epilogue(p.e, p.n, p.nout, t, (int64_t)tile * p.map.step + r, z0, z1, p.y);
           });
}

constexpr size_t kRoom = 227 * 1024;  // shared memory of a CTA

template <int L, class P>
cudaError_t launch_rows(RowsParams& p, cudaStream_t st) {
  const int step = p.e.gated ? P::kTileRows / 2 : P::kTileRows;
  p.map.step = step;
  p.map.ahead = p.e.gated ? 0 : step / 2;
  p.tiles = (int)((p.nout + step - 1) / step);
  const int grid = std::min(p.tiles, sm_count());
  p.each = p.tiles / grid;
  p.extra = p.tiles % grid;
  if (!P::plan((p.tiles + grid - 1) / grid, p.mat.units, kRoom, &p.split)) return cudaErrorInvalidValue;
  const size_t smem = P::smem_bytes(p.split);
  const cudaError_t err = allow_smem(reinterpret_cast<const void*>(&linear_rows_kernel<L, P>), kRoom);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(rows::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, linear_rows_kernel<L, P>, p);
}

// Int8 digits for one row of x, fp16 column tiles of 8 rows (4 with two slots per unit) for more. The digits take
// longer to build than a row's fp16 operands, for few tiles longer than they save; us with int8 and with fp16:
//   one row, n x k:    24576 x 4096   12288 x 4096   4096 x 12288   1000 x 2176   512 x 17408
//     Q2                13.2 / 13.9     9.5 / 9.9     12.3 / 13.1     4.3 / 3.9    13.2 / 11.1
//     base-3            17.2 / 18.6    12.1 / 12.6    17.9 / 17.1     4.6 / 4.2    15.9 / 14.1
//     binary            10.2 / 15.6     7.5 / 10.6     9.9 / 13.4     4.1 / 4.7     9.6 / 10.6
//   two rows, Q2        14.7 / 14.2    11.2 / 10.2    17.2 / 13.5     5.0 / 4.0    18.6 / 11.3
//     base-3            23.1 / 18.8    16.4 / 12.8    26.7 / 17.4     6.1 / 4.3    28.7 / 14.3
//     binary            13.2 / 15.9     9.8 / 10.9    15.3 / 14.0     5.3 / 4.9    16.5 / 11.4
template <int L>
cudaError_t pick_rows(RowsParams& p, cudaStream_t st) {
  const int64_t tiles = (p.n + 15) / 16, sms = sm_count();  // 16 packed rows to a tile, gated or not
  if (p.tokens == 1 && tiles > (L == TERN_Q1_0_G128 ? 0 : L == TERN_Q2_0_G128 ? sms : 4 * sms))
    return launch_rows<L, rows::Product<L, rows::kInt8, 1>>(p, st);
  if constexpr (L == TERN_Q1_0_G128)
    if (p.tokens == 2 && tiles > 4 * sms) return launch_rows<L, rows::Product<L, rows::kInt8, 2>>(p, st);
  const int nt = (p.tokens + rows::Geo<L, rows::kFp16>::kTok - 1) / rows::Geo<L, rows::kFp16>::kTok;
  if (nt == 1) return launch_rows<L, rows::Product<L, rows::kFp16, 1>>(p, st);
  if (nt == 2) return launch_rows<L, rows::Product<L, rows::kFp16, 2>>(p, st);
  return launch_rows<L, rows::Product<L, rows::kFp16, 4>>(p, st);
}

// Rows of x that the register core takes. Operands of nine rows and more stay in shared memory up to k = 1920 (base-3:
// four column tiles, half of them zeros), 4096 (binary, the same) and 4608 (Q2, two tiles); longer rows take them in
// passes, built again for every few tiles of a CTA. us on this core and on the tensor cores of the other kernel:
//                   4096 x 4096   4096 x 5120   24576 x 5120   4096 x 12288   5120 x 17408
//   Q2       9 rows    8.5 / 16.8   12.1 / 18.1   28.4 / 47.6    20.1 / 27.2    33.9 / 34.1
//           16         9.4 / 16.9   13.3 / 18.1   31.0 / 47.8    22.8 / 27.4    38.1 / 34.3
//   base-3   9        16.7 / 18.6   19.6 / 20.2   48.1 / 57.9    42.1 / 31.5    66.5 / 40.2
//           16        17.7 / 18.7   20.8 / 20.4   50.9 / 58.0    45.0 / 31.7    70.7 / 40.4
//   binary   9        11.4 / 15.5   17.7 / 16.9   43.2 / 43.8    31.1 / 25.8    53.9 / 32.1
//           16        13.2 / 15.7   20.6 / 17.2   47.3 / 43.9    37.3 / 25.9    63.1 / 32.4
bool few_rows(const tern_matrix& W, int64_t m) {
  return m <= 8 || (m <= 16 && (W.layout == TERN_Q2_0_G128 || W.k <= (W.layout == TERN_T3_5PB_G128 ? 5120 : 4096)));
}

}  // namespace

cudaError_t launch_linear(const tern_matrix& W, const uint16_t* x, int64_t m, uint16_t* y, const Epilogue& e,
                          uint32_t flags, uint32_t* status, cudaStream_t st) {
  const int64_t nout = e.gated ? W.n / 2 : W.n;
  if (few_rows(W, m)) {
    RowsParams p{};
    p.mat = rows::Mat{static_cast<const uint8_t*>(W.codes), W.scales, W.code_row_stride, W.scale_row_stride, (int)W.k,
                      (int)row_bytes(W.layout, W.k), (int)(W.k / kGroup), (int)((row_bytes(W.layout, W.k) + 31) / 32)};
    p.map = rows::Map{0, e.gated ? nout : 0, (int)nout, 0, 0};
    p.x = x;
    p.y = y;
    p.e = e;
    p.n = W.n;
    p.nout = nout;
    p.tokens = (int)m;
    p.early = (flags & TERN_GEMV_STATIC_WEIGHTS) ? 1 : 0;
    switch (W.layout) {
      case TERN_Q2_0_G128: return pick_rows<TERN_Q2_0_G128>(p, st);
      case TERN_T3_5PB_G128: return pick_rows<TERN_T3_5PB_G128>(p, st);
      default: return pick_rows<TERN_Q1_0_G128>(p, st);
    }
  }
  return launch_layer_gemm(W, x, m, y, e, status, st);
}

}  // namespace tern
