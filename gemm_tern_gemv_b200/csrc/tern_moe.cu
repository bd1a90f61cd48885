// Mixture-of-experts layer for a few tokens on packed ternary experts:
//   p = softmax(R x), the top_k experts of each token (ties to the lower index), optionally renormalised;
//   y[t] = sum_j p[t][j] D_e (act(G_e x[t]) * U_e x[t]) (+ residual), e = ids[t][j].
//
// Bound by the packed weights of the experts in use, read once from HBM (and by latency for one token). Three
// launches, each started while the one before ends (programmatic dependent launch):
//   route  a cluster of eight CTAs for one to four tokens: each computes the logits of every eighth expert,
//          the first collects them through the cluster's shared memory and picks.
//   up     the (token, expert) pairs are sorted by expert; the 8-output tiles (gate and up rows) of all experts
//          in use form one list that is dealt evenly to one CTA per SM. The products are those of
//          tern_rows.cuh: int8 digits for one or two tokens of an expert, fp16 for more. h = act(g) u in fp32.
//   down   the same over 16-row tiles of the down matrices, with h brought into fp16's range by a power of two
//          per pair. Sums of a pair go to the workspace; whoever finishes a 16-column strip of y last (a counter
//          per strip) adds its pairs up in the order of j, so the result does not depend on who that was.
#include "tern_rows.cuh"

namespace tern {
namespace {

constexpr int kRouteCtas = 8, kRouteThreads = 256;
constexpr int kMaxPairs = TERN_MOE_MAX_TOKENS * TERN_MOE_MAX_TOP_K;

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void store_first(double* local, double v) {  // into the first CTA's copy of *local
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(remote) : "r"(sm100::smem_u32(local)));
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(remote), "d"(v) : "memory");
}

// Whether logit a of expert ia goes before logit b of ib: larger first, ties to the lower index, NaN last.
__device__ __forceinline__ bool before(double a, int ia, double b, int ib) {
  const bool na = a != a, nb = b != b;
  if (na != nb) return nb;
  if (!na && a != b) return a > b;
  return ia < ib;
}

// e^d with d's rounding to fp32 made good: e^(hi + lo) = e^hi (1 + lo).
__device__ __forceinline__ float exp_exact(double d) {
  const float hi = (float)d;
  const float e = expf(hi);
  return hi > -INFINITY ? fmaf(e, (float)(d - (double)hi), e) : e;
}

// Logits in fp64 (products of fp16 values are exact in fp32), so that experts next to one another at the
// border keep their order.
template <int TOK>
__global__ void __cluster_dims__(kRouteCtas, 1, 1) __launch_bounds__(kRouteThreads) route_kernel(const __grid_constant__ MoeParams p) {
  __shared__ double logit[TOK][kMoeMaxExperts];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t0 = (int)(blockIdx.x / kRouteCtas) * TOK;
  const int rank = (int)cluster_rank();
  sm100::griddep_launch_dependents();
  sm100::griddep_wait();
  for (int i = (int)(blockIdx.x * kRouteThreads + threadIdx.x); i < p.tokens * p.top_k + p.d / 16; i += (int)gridDim.x * kRouteThreads)
    p.clear[i] = 0;  // largest |h| of each pair, then the strips' counters
  for (int e = rank + kRouteCtas * warp; e < p.experts; e += kRouteCtas * (kRouteThreads / 32)) {
    double s[TOK] = {};
    const uint4* w = reinterpret_cast<const uint4*>(p.router + (int64_t)e * p.d);
#pragma unroll 2
    for (int v = lane; v < p.d / 8; v += 32) {
      const uint4 a = __ldg(w + v);
      const uint32_t av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int i = 0; i < TOK; i++) {
        if (t0 + i >= p.tokens) break;
        const uint4 b = *(reinterpret_cast<const uint4*>(p.x + (int64_t)(t0 + i) * p.d) + v);
        const uint32_t bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int q = 0; q < 4; q++) {
          const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&av[q])), y = __half22float2(*reinterpret_cast<const __half2*>(&bv[q]));
          s[i] += (double)(x.x * y.x);
          s[i] += (double)(x.y * y.y);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < TOK; i++) {
      for (int o = 16; o; o >>= 1) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
      if (lane == 0) store_first(&logit[i][e], s[i]);
    }
  }
  cluster_sync();
  if (rank || warp >= TOK || t0 + warp >= p.tokens) return;
  // one warp per token: lane l holds the logits of experts l, l + 32, ...
  const int t = t0 + warp;
  constexpr int kPer = kMoeMaxExperts / 32;
  double l[kPer];
  double mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < kPer; i++) {
    l[i] = lane + 32 * i < p.experts ? logit[warp][lane + 32 * i] : -INFINITY;
    mx = fmax(mx, l[i]);
  }
  for (int o = 16; o; o >>= 1) mx = fmax(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; i++)
    if (lane + 32 * i < p.experts) sum += exp_exact(l[i] - mx);
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  uint32_t used = 0;  // bit i: expert lane + 32 i is taken
  float chosen = 0.f, mine = 0.f;
  for (int j = 0; j < p.top_k; j++) {
    double best = 0.;
    int be = kMoeMaxExperts + lane;  // none
    bool has = false;
#pragma unroll
    for (int i = 0; i < kPer; i++) {
      const int e = lane + 32 * i;
      if (e < p.experts && !(used >> i & 1) && (!has || before(l[i], e, best, be))) {
        best = l[i];
        be = e;
        has = true;
      }
    }
    for (int o = 16; o; o >>= 1) {
      const double ob = __shfl_xor_sync(0xffffffffu, best, o);
      const int oe = __shfl_xor_sync(0xffffffffu, be, o);
      const bool oh = oe < kMoeMaxExperts;
      if (oh && (be >= kMoeMaxExperts || before(ob, oe, best, be))) {
        best = ob;
        be = oe;
      }
    }
    if ((be & 31) == lane) used |= 1u << (be >> 5);
    const float w = exp_exact(best - mx) / sum;
    chosen += w;
    if (lane == j) {
      mine = w;
      p.ids[t * p.top_k + j] = be;
    }
  }
  if (lane < p.top_k) p.weights[t * p.top_k + lane] = p.renormalize ? mine / chosen : mine;
}

// ---- the experts ------------------------------------------------------------------------------------------
// Columns of a chunk: pairs of one expert that go through its weights together.
template <int L> constexpr int chunk() { return 2 * rows::Geo<L, rows::kFp16>::kTok; }
constexpr int kPlans = 8;  // cuts for up to 1, 2, 3, 4, 6, 8, 16 and any number of tiles
__host__ __device__ constexpr int plan_tiles(int i) { return i < 4 ? i + 1 : i == 4 ? 6 : i == 5 ? 8 : i == 6 ? 16 : 32; }
enum Variant { kOne8, kTwo8, kOne16, kTwo16, kVariants };  // int8 with one or two column tiles, fp16 likewise
struct Plans {
  rows::Split split[kVariants][kPlans];
};

struct Lists {
  int segments, tiles;             // chunks of pairs; 16-row tiles of all of them
  uint16_t pair[kMaxPairs];        // pairs sorted by expert
  uint16_t seg_expert[kMaxPairs], seg_first[kMaxPairs];
  uint8_t seg_count[kMaxPairs];
  uint16_t expert[kMaxPairs];      // of each pair, in the pairs' own order
  int count[kMoeMaxExperts], first[kMoeMaxExperts];
  int index[16];                   // rows of the activations of the current segment
  float mul[16];                   // and their powers of two
  int last[64];                    // strips that this CTA finished
};

// Sorts the pairs by expert (in the pairs' order within an expert) and cuts them into segments.
__device__ void build_lists(const MoeParams& p, Lists& s, int cols, int tiles_per_segment) {
  const int tid = threadIdx.x, lane = tid & 31, pairs = p.tokens * p.top_k;
  for (int i = tid; i < pairs; i += rows::kThreads) s.expert[i] = (uint16_t)p.ids[i];
  for (int i = tid; i < kMoeMaxExperts; i += rows::kThreads) s.count[i] = 0;
  __syncthreads();
  if (tid < 32) {
    for (int i0 = 0; i0 < pairs; i0 += 32) {
      const int i = i0 + lane, e = i < pairs ? (int)s.expert[i] : kMoeMaxExperts + lane;
      const uint32_t same = __match_any_sync(0xffffffffu, e);
      if (i < pairs) {
        const int base = s.count[e];
        s.pair[i] = (uint16_t)(base + __popc(same & ((1u << lane) - 1u)));  // its place among the expert's pairs
        __syncwarp(__activemask());
        if (lane == __ffs(same) - 1) s.count[e] = base + __popc(same);
      }
      __syncwarp();
    }
    int before = 0, segs = 0;
    for (int e0 = 0; e0 < kMoeMaxExperts; e0 += 32) {
      const int n = s.count[e0 + lane], g = (n + cols - 1) / cols;
      int a = n, b = g;
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) {
          a += x;
          b += y;
        }
      }
      s.first[e0 + lane] = before + a - n;
      for (int i = 0, at = segs + b - g; i < g; i++, at++) {
        s.seg_expert[at] = (uint16_t)(e0 + lane);
        s.seg_first[at] = (uint16_t)(before + a - n + i * cols);
        s.seg_count[at] = (uint8_t)min(cols, n - i * cols);
      }
      before += __shfl_sync(0xffffffffu, a, 31);
      segs += __shfl_sync(0xffffffffu, b, 31);
    }
    if (lane == 0) {
      s.segments = segs;
      s.tiles = segs * tiles_per_segment;
    }
  }
  __syncthreads();
  // every pair to its place: read the places first, they share the array
  uint16_t at[kMaxPairs / rows::kThreads];
#pragma unroll
  for (int c = 0; c < kMaxPairs / rows::kThreads; c++) {
    const int i = tid + c * rows::kThreads;
    at[c] = i < pairs ? (uint16_t)(s.first[s.expert[i]] + s.pair[i]) : (uint16_t)0;
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < kMaxPairs / rows::kThreads; c++) {
    const int i = tid + c * rows::kThreads;
    if (i < pairs) s.pair[at[c]] = (uint16_t)i;
  }
  __syncthreads();
}

struct ExpertParams {
  MoeParams p;
  rows::Mat mat;
  Plans plans;
};

// Tiles [a, b) of segment g in one form of the product. Out of line: inlined side by side, the forms would
// share their registers.
template <int L, bool UP, int MODE, int NT>
__device__ __noinline__ void run_form(uint8_t* smem, const ExpertParams* q, const Lists* s, int form, int g, int a, int b) {
  const MoeParams& p = q->p;
  int plan = 0;
  while (plan < kPlans - 1 && plan_tiles(plan) < b - a) plan++;
  const uint16_t* pair = s->pair + s->seg_first[g];
  const int n = s->seg_count[g];
  const auto none = [] {};
  rows::Product<L, MODE, NT> prod;
  if constexpr (UP) {
    const int64_t first = (int64_t)s->seg_expert[g] * 2 * p.f;
    prod.run(smem, q->plans.split[form][plan], q->mat, rows::Map{first, first + p.f, p.f, 8, 0}, a, b, rows::HalfRows{p.x, p.d, s->index},
             n, none, [&](int tile, int r, int c, float gate, float up) {
               const float h = act_fwd(p.act, gate) * up;
               const int pr = pair[c];
               p.h[(int64_t)pr * p.f + tile * 8 + r] = h;
               // largest |h| of the pair, as bits: order does not matter to a maximum. NaN counts as the largest.
               atomicMax(p.clear + pr, __float_as_uint(h) & 0x7fffffffu);
             });
  } else {
    const int64_t first = (int64_t)s->seg_expert[g] * p.d;
    prod.run(smem, q->plans.split[form][plan], q->mat, rows::Map{first, first, p.d, 16, 8}, a, b,
             rows::FloatRows{p.h, p.f, s->index, s->mul}, n, none, [&](int tile, int r, int c, float z, float) {
               p.z[(int64_t)pair[c] * p.d + tile * 16 + r] = MODE == rows::kFp16 ? z / s->mul[c] : z;
             });
  }
}

template <int L, bool UP>
__device__ __forceinline__ void run_segment(uint8_t* smem, const ExpertParams* q, const Lists* s, int g, int a, int b) {
  constexpr int k8 = rows::Geo<L, rows::kInt8>::kTok, k16 = rows::Geo<L, rows::kFp16>::kTok;
  const int n = s->seg_count[g];
  if (n <= k8) run_form<L, UP, rows::kInt8, 1>(smem, q, s, kOne8, g, a, b);
  else if (n <= 2) run_form<L, UP, rows::kInt8, k8 < 2 ? 2 : 1>(smem, q, s, kTwo8, g, a, b);
  else if (n <= k16) run_form<L, UP, rows::kFp16, 1>(smem, q, s, kOne16, g, a, b);
  else run_form<L, UP, rows::kFp16, 2>(smem, q, s, kTwo16, g, a, b);
}

template <int L>
__global__ void __launch_bounds__(rows::kThreads, 1) moe_up_kernel(const __grid_constant__ ExpertParams q) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Lists s;
  const MoeParams& p = q.p;
  sm100::griddep_launch_dependents();
  sm100::griddep_wait();
  const int per = p.f / 8;  // tiles of a segment
  build_lists(p, s, chunk<L>(), per);
  const int t1 = (int)((int64_t)(blockIdx.x + 1) * s.tiles / gridDim.x);
  for (int t = (int)((int64_t)blockIdx.x * s.tiles / gridDim.x); t < t1;) {
    const int g = t / per, a = t % per, b = min(per, a + t1 - t), n = s.seg_count[g];
    const uint16_t* pair = s.pair + s.seg_first[g];
    if ((int)threadIdx.x < n) s.index[threadIdx.x] = pair[threadIdx.x] / p.top_k;
    __syncthreads();
    run_segment<L, true>(smem, &q, &s, g, a, b);
    __syncthreads();
    t += b - a;
  }
}

template <int L>
__global__ void __launch_bounds__(rows::kThreads, 1) moe_down_kernel(const __grid_constant__ ExpertParams q) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Lists s;
  const MoeParams& p = q.p;
  sm100::griddep_launch_dependents();
  sm100::griddep_wait();
  const int per = p.d / 16, tid = threadIdx.x;
  build_lists(p, s, chunk<L>(), per);
  uint32_t* counter = p.clear + p.tokens * p.top_k;
  const int t1 = (int)((int64_t)(blockIdx.x + 1) * s.tiles / gridDim.x);
  for (int t = (int)((int64_t)blockIdx.x * s.tiles / gridDim.x); t < t1;) {
    const int g = t / per, a = t % per, b = min(min(per, a + t1 - t), a + 64), n = s.seg_count[g];
    const uint16_t* pair = s.pair + s.seg_first[g];
    if (tid < n) {
      const int pr = pair[tid];
      const uint32_t top = p.clear[pr];
      s.index[tid] = pr;
      // the fp16 form takes h times a power of two that brings the pair's largest to [2^14, 2^15)
      s.mul[tid] = top == 0 || top >= 0x7f800000u ? 1.f : rows::exp2i(min(100, 15 - rows::exponent(top)));
    }
    __syncthreads();
    run_segment<L, false>(smem, &q, &s, g, a, b);
    // strips that now have the sums of every segment
    __syncthreads();
    if (tid < b - a) {
      __threadfence();
      s.last[tid] = atomicAdd(counter + a + tid, 1u) == (uint32_t)s.segments - 1u;
      __threadfence();
    }
    __syncthreads();
    for (int i = tid; i < (b - a) * 16 * p.tokens; i += rows::kThreads) {
      const int r = i % 16, tl = i / 16 % (b - a), tok = i / (16 * (b - a));
      if (!s.last[tl]) continue;
      const int o = (a + tl) * 16 + r;
      float y = 0.f;
      for (int j = 0; j < p.top_k; j++) y = fmaf(p.weights[tok * p.top_k + j], __ldcg(p.z + (int64_t)(tok * p.top_k + j) * p.d + o), y);
      const int64_t at = (int64_t)tok * p.d + o;
      if (p.residual) y += h2f(p.residual[at]);
      p.y[at] = f2h(y);
    }
    __syncthreads();
    t += b - a;
  }
}

constexpr size_t kRoom = 227 * 1024 - (sizeof(Lists) + 1023) / 1024 * 1024 - 1024;  // dynamic shared memory

template <int L, int MODE, int NT>
bool plan_variant(int units, rows::Split* out, size_t* smem) {
  using P = rows::Product<L, MODE, NT>;
  for (int i = 0; i < kPlans; i++) {
    if (!rows::plan_split<P>(plan_tiles(i), units, kRoom, out + i)) return false;
    *smem = std::max(*smem, P::smem_bytes(out[i]));
  }
  return true;
}

cudaError_t launch(const void* kern, int grid, int threads, size_t smem, cudaStream_t st, void* arg) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[] = {arg};
  return cudaLaunchKernelExC(&cfg, kern, args);
}

template <int L, bool UP>
cudaError_t launch_experts(const tern_matrix& W, const MoeParams& p, cudaStream_t st) {
  ExpertParams q;
  q.p = p;
  q.mat = rows::Mat{static_cast<const uint8_t*>(W.codes), W.scales, W.code_row_stride, W.scale_row_stride, (int)W.k,
                    (int)row_bytes(W.layout, W.k), (int)(W.k / kGroup), (int)((row_bytes(W.layout, W.k) + 31) / 32)};
  size_t smem = 0;
  const bool ok = plan_variant<L, rows::kInt8, 1>(q.mat.units, q.plans.split[kOne8], &smem) &&
                  plan_variant<L, rows::kInt8, L == TERN_Q2_0_G128 ? 1 : 2>(q.mat.units, q.plans.split[kTwo8], &smem) &&
                  plan_variant<L, rows::kFp16, 1>(q.mat.units, q.plans.split[kOne16], &smem) &&
                  plan_variant<L, rows::kFp16, 2>(q.mat.units, q.plans.split[kTwo16], &smem);
  if (!ok) return cudaErrorInvalidValue;
  const void* kern = UP ? reinterpret_cast<const void*>(&moe_up_kernel<L>) : reinterpret_cast<const void*>(&moe_down_kernel<L>);
  const cudaError_t e = allow_smem(kern, kRoom);
  if (e != cudaSuccess) return e;
  return launch(kern, sm_count(), rows::kThreads, smem, st, &q);
}

template <bool UP>
cudaError_t dispatch(const tern_matrix& W, const MoeParams& p, cudaStream_t st) {
  switch (W.layout) {
    case TERN_Q2_0_G128: return launch_experts<TERN_Q2_0_G128, UP>(W, p, st);
    case TERN_T3_5PB_G128: return launch_experts<TERN_T3_5PB_G128, UP>(W, p, st);
    default: return launch_experts<TERN_Q1_0_G128, UP>(W, p, st);
  }
}

}  // namespace

MoePlan moe_plan(int64_t tokens, int64_t d, int64_t f, int top_k) {
  MoePlan w{};
  const size_t pairs = (size_t)tokens * top_k;
  size_t o = 0;
  auto take = [&](size_t bytes) { const size_t at = o; o += (bytes + 255) / 256 * 256; return at; };
  w.ids = take(pairs * 4);
  w.weights = take(pairs * 4);
  w.clear = take((pairs + d / 16) * 4);
  w.h = take(pairs * f * 4);
  w.z = take(pairs * d * 4);
  w.bytes = o;
  return w;
}

cudaError_t launch_moe(const tern_matrix& G, const tern_matrix& D, MoeParams p, const MoePlan& w, void* workspace,
                       cudaStream_t st) {
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (!p.ids) p.ids = reinterpret_cast<int32_t*>(ws + w.ids);
  if (!p.weights) p.weights = reinterpret_cast<float*>(ws + w.weights);
  p.clear = reinterpret_cast<uint32_t*>(ws + w.clear);
  p.h = reinterpret_cast<float*>(ws + w.h);
  p.z = reinterpret_cast<float*>(ws + w.z);
  const int tok = p.tokens > 32 ? 4 : p.tokens > 16 ? 2 : 1;
  const void* route = tok == 4   ? reinterpret_cast<const void*>(&route_kernel<4>)
                      : tok == 2 ? reinterpret_cast<const void*>(&route_kernel<2>)
                                 : reinterpret_cast<const void*>(&route_kernel<1>);
  cudaError_t e = launch(route, (p.tokens + tok - 1) / tok * kRouteCtas, kRouteThreads, 0, st, &p);
  if (e != cudaSuccess) return e;
  e = dispatch<true>(G, p, st);
  if (e != cudaSuccess) return e;
  return dispatch<false>(D, p, st);
}

}  // namespace tern
