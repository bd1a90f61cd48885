// Backward of the fused linear layer: dz = dy * act'(z), dbias = sum over rows of dz, dx = dz W.
//
// dz and dbias come from one pass (dz_kernel), bound by HBM: dy and z are read once, dz is written once (2048 x 24576
// gated: 252 MB in 52 us, 4.8 TB/s; the activations' arithmetic is most of the rest).
// A CTA takes 16 x VEC columns and a slice of the rows, a half-warp every sixteenth of them, a lane VEC columns
// (16 bytes where rows are aligned to that). Column sums stay in fp32 registers, are joined over the warps
// through shared memory and over the row slices through the cluster's shared memory, always in the same
// order. dx is the transposed product of tern_layer_gemm.cu on the rounded dz.
#include "sm100.cuh"
#include "tern_layer.cuh"

namespace tern {
namespace {

constexpr int kPerSm = 4, kWarps = 8, kLanes = 16, kRowsAtOnce = kWarps * 32 / kLanes;

struct DzParams {
  const uint16_t *dy, *z;
  uint16_t* dz;
  float* db;
  int64_t m, n, nout, dz_stride;
  int act, gated, identity;
};

template <int VEC> struct Halves { uint16_t v[VEC]; };
template <int VEC>
__device__ __forceinline__ Halves<VEC> load_halves(const uint16_t* p) {
  Halves<VEC> h;
  if constexpr (VEC == 8) {
    const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
    *reinterpret_cast<uint4*>(h.v) = u;
  } else {
    h.v[0] = __ldcs(p);
  }
  return h;
}
template <int VEC>
__device__ __forceinline__ void store_halves(uint16_t* p, const Halves<VEC>& h) {
  if constexpr (VEC == 8) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(h.v);
  else p[0] = h.v[0];
}

__device__ __forceinline__ uint32_t cluster_rank_y() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float ld_peer(const float* local, uint32_t rank) {
  uint32_t remote;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"((uint32_t)__cvta_generic_to_shared(local)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote) : "memory");
  return v;
}

template <int VEC>
__device__ __forceinline__ void dz_rows(const DzParams& p, int act, int64_t c, int64_t t0, int64_t t1, float (&s0)[VEC], float (&s1)[VEC]) {
#pragma unroll 1
  for (int64_t t = t0; t < t1; t += kRowsAtOnce) {
    const Halves<VEC> d = load_halves<VEC>(p.dy + t * p.nout + c);
    Halves<VEC> a{}, u{}, o0, o1;
    if (!p.identity) a = load_halves<VEC>(p.z + t * p.n + c);
    if (p.gated) u = load_halves<VEC>(p.z + t * p.n + p.nout + c);
#pragma unroll
    for (int i = 0; i < VEC; i++) {
      const float g = h2f(d.v[i]), za = h2f(a.v[i]);
      float f, df;
      act_both(act, za, &f, &df);
      const float x0 = (p.gated ? g * h2f(u.v[i]) : g) * df, x1 = g * f;
      s0[i] += x0;
      s1[i] += x1;
      o0.v[i] = f2h(x0);
      o1.v[i] = f2h(x1);
    }
    if (p.dz) {
      store_halves<VEC>(p.dz + t * p.dz_stride + c, o0);
      if (p.gated) store_halves<VEC>(p.dz + t * p.dz_stride + p.nout + c, o1);
    }
  }
}

template <int VEC>
__global__ void __launch_bounds__(kWarps * 32, kPerSm) dz_kernel(const __grid_constant__ DzParams p) {
  constexpr int kCols = kLanes * VEC;
  __shared__ float sums[2][kRowsAtOnce][kCols];
  sm100::griddep_launch_dependents();
  sm100::griddep_wait();
  const int lane = threadIdx.x % kLanes, sub = threadIdx.x / kLanes;
  const int64_t c = (int64_t)blockIdx.x * kCols + lane * VEC;
  const int64_t r0 = p.m * blockIdx.y / gridDim.y, r1 = p.m * (blockIdx.y + 1) / gridDim.y;
  float s0[VEC] = {}, s1[VEC] = {};
  if (c < p.nout)
    with_act(p.act, [&](auto act) { dz_rows<VEC>(p, act.value, c, r0 + sub, r1, s0, s1); });
  if (!p.db) return;  // the same for every CTA of the cluster
#pragma unroll
  for (int i = 0; i < VEC; i++) {
    sums[0][sub][lane * VEC + i] = s0[i];
    sums[1][sub][lane * VEC + i] = s1[i];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * kCols; i += kWarps * 32) {
    float s = 0.f;
    for (int w = 0; w < kRowsAtOnce; w++) s += sums[i / kCols][w][i % kCols];
    sums[i / kCols][0][i % kCols] = s;  // only this thread reads and writes column i's sums
  }
  cluster_sync_all();
  const uint32_t slices = gridDim.y;
  for (int i = threadIdx.x + kWarps * 32 * (int)cluster_rank_y(); i < (p.gated ? 2 : 1) * kCols; i += kWarps * 32 * (int)slices) {
    const int64_t j = (int64_t)blockIdx.x * kCols + i % kCols;
    if (j >= p.nout) continue;
    float s = 0.f;
    for (uint32_t r = 0; r < slices; r++) s += ld_peer(&sums[i / kCols][0][i % kCols], r);
    p.db[j + (i / kCols) * p.nout] = s;
  }
  cluster_sync_all();  // no CTA leaves while another may still read its sums
}

template <int VEC>
cudaError_t launch_dz(const DzParams& p, cudaStream_t st) {
  const int64_t cols = kLanes * VEC;
  cudaLaunchConfig_t cfg{};
  const int64_t blocks = (p.nout + cols - 1) / cols;
  // as many slices of the rows (1, 2, 4 or 8 to a cluster) as still run at the same time: 2048 x 24576 gated takes 60 us
  // with 8, 52 with 4; 65 with 6, which leave SMs of the GPCs over
  int slices = p.m >= 64 ? 8 : p.m >= 16 ? 2 : 1;
  while (slices > 1 && blocks * slices > kPerSm * sm_count()) slices /= 2;
  cfg.gridDim = dim3((unsigned)blocks, (unsigned)slices);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = cfg.gridDim.y;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, dz_kernel<VEC>, p);
}

}  // namespace

cudaError_t launch_linear_backward(const tern_matrix& W, const uint16_t* dy, const uint16_t* z, int64_t m, int act,
                                   int gated, uint16_t* dx, uint16_t* dz, int64_t dz_stride, float* db, uint32_t* status,
                                   cudaStream_t st) {
  DzParams p{dy, z, dz, db, m, W.n, gated ? W.n / 2 : W.n, dz_stride, act, gated, act == TERN_ACT_NONE && !gated};
  if (dz || db) {
    // 16-byte loads where every row of every operand starts on 16 bytes
    const bool wide = p.nout % 8 == 0 && p.dz_stride % 8 == 0 &&
                      ((reinterpret_cast<uintptr_t>(dy) | reinterpret_cast<uintptr_t>(z) | reinterpret_cast<uintptr_t>(dz)) & 15u) == 0;
    const cudaError_t e = wide ? launch_dz<8>(p, st) : launch_dz<1>(p, st);
    if (e != cudaSuccess) return e;
  }
  if (!dx) return cudaSuccess;
  return dz ? launch_layer_gemm_t(W, dz, dz_stride, m, dx, status, st) : launch_layer_gemm_t(W, dy, W.n, m, dx, status, st);
}

}  // namespace tern
