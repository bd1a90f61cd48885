// Mixture-of-experts layer for a few tokens on packed ternary experts:
//   p = softmax(R x), the top_k experts of each token (ties to the lower index), optionally renormalised;
//   y[t] = sum_j p[t][j] D_e (act(G_e x) * U_e x) (+ residual), e = ids[t][j].
#include "tern_layer.cuh"

namespace tern {
namespace {

__device__ __forceinline__ float warp_sum(float v) {
  for (int s = 16; s; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}

// One block per token: logits, softmax statistics and the top_k selection on fp64 logits (products of
// fp16 values are exact in fp32; experts next to one another at the border keep their order).
__global__ void __launch_bounds__(256) route_kernel(MoeParams p) {
  __shared__ double prob[kMoeMaxExperts];
  const int t = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int e = warp; e < p.experts; e += 8) {
    double s = 0.;
    for (int k = lane; k < p.d; k += 32) s += (double)(h2f(p.x[(int64_t)t * p.d + k]) * h2f(p.router[(int64_t)e * p.d + k]));
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) prob[e] = s;
  }
  __syncthreads();
  if (threadIdx.x) return;
  double mx = -INFINITY;
  float sum = 0.f;
  for (int e = 0; e < p.experts; e++) mx = fmax(mx, prob[e]);
  for (int e = 0; e < p.experts; e++) sum += expf((float)(prob[e] - mx));
  float chosen = 0.f;
  uint32_t used[kMoeMaxExperts / 32] = {};
  for (int j = 0; j < p.top_k; j++) {
    int best = -1;
    for (int e = 0; e < p.experts; e++)
      if (!(used[e >> 5] >> (e & 31) & 1) && (best < 0 || prob[e] > prob[best] || (prob[best] != prob[best] && prob[e] == prob[e])))
        best = e;
    used[best >> 5] |= 1u << (best & 31);
    const float w = expf((float)(prob[best] - mx)) / sum;
    chosen += w;
    p.ids[t * p.top_k + j] = best;
    p.weights[t * p.top_k + j] = w;
  }
  if (p.renormalize)
    for (int j = 0; j < p.top_k; j++) p.weights[t * p.top_k + j] /= chosen;
}

__global__ void __launch_bounds__(128) moe_up_kernel(tern_matrix G, MoeParams p) {
  const int lane = threadIdx.x & 31;
  const int o = blockIdx.x * 4 + (threadIdx.x >> 5), pair = blockIdx.y;
  const int t = pair / p.top_k, e = p.ids[pair];
  const uint8_t* codes = static_cast<const uint8_t*>(G.codes);
  float z[2] = {};
  for (int h = 0; h < 2; h++) {
    const int64_t n = (int64_t)e * 2 * p.f + o + (int64_t)h * p.f;
    for (int k = lane; k < p.d; k += 32)
      z[h] = fmaf(decode_t(G.layout, codes + n * G.code_row_stride, k) * h2f(G.scales[n * G.scale_row_stride + k / kGroup]),
                  h2f(p.x[(int64_t)t * p.d + k]), z[h]);
    z[h] = warp_sum(z[h]);
  }
  if (lane == 0) p.h[(int64_t)pair * p.f + o] = act_fwd(p.act, z[0]) * z[1];
}

__global__ void __launch_bounds__(128) moe_down_kernel(tern_matrix D, MoeParams p) {
  const int lane = threadIdx.x & 31;
  const int o = blockIdx.x * 4 + (threadIdx.x >> 5), t = blockIdx.y;
  const uint8_t* codes = static_cast<const uint8_t*>(D.codes);
  float y = 0.f;
  for (int j = 0; j < p.top_k; j++) {
    const int pair = t * p.top_k + j;
    const int64_t n = (int64_t)p.ids[pair] * p.d + o;
    float z = 0.f;
    for (int k = lane; k < p.f; k += 32)
      z = fmaf(decode_t(D.layout, codes + n * D.code_row_stride, k) * h2f(D.scales[n * D.scale_row_stride + k / kGroup]),
               p.h[(int64_t)pair * p.f + k], z);
    y = fmaf(p.weights[pair], warp_sum(z), y);
  }
  if (lane) return;
  if (p.residual) y += h2f(p.residual[(int64_t)t * p.d + o]);
  p.y[(int64_t)t * p.d + o] = f2h(y);
}

}  // namespace

MoePlan moe_plan(int64_t tokens, int64_t d, int64_t f, int experts, int top_k) {
  (void)d;
  (void)experts;
  MoePlan w{};
  size_t o = 0;
  auto take = [&](size_t bytes) { const size_t at = o; o += (bytes + 255) / 256 * 256; return at; };
  w.ids = take((size_t)tokens * top_k * 4);
  w.weights = take((size_t)tokens * top_k * 4);
  w.h = take((size_t)tokens * top_k * f * 4);
  w.bytes = o;
  return w;
}

cudaError_t launch_moe(const tern_matrix& G, const tern_matrix& D, MoeParams p, const MoePlan& w, void* workspace,
                       cudaStream_t st) {
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (!p.ids) p.ids = reinterpret_cast<int32_t*>(ws + w.ids);
  if (!p.weights) p.weights = reinterpret_cast<float*>(ws + w.weights);
  p.h = reinterpret_cast<float*>(ws + w.h);
  route_kernel<<<p.tokens, 256, 0, st>>>(p);
  moe_up_kernel<<<dim3(p.f / 4, p.tokens * p.top_k), 128, 0, st>>>(G, p);
  moe_down_kernel<<<dim3(p.d / 4, p.tokens), 128, 0, st>>>(D, p);
  return cudaGetLastError();
}

}  // namespace tern
