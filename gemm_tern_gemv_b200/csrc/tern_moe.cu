// Mixture-of-experts layer for a few tokens on packed ternary experts:
//   p = softmax(R x), the top_k experts of each token (ties to the lower index), optionally renormalised;
//   y[t] = sum_j p[t][j] D_e (act(G_e x[t]) * U_e x[t]) (+ residual), e = ids[t][j].
//
// The least is to read the packed weights of the experts in use once. What it takes is decoding: a segment of an
// expert's pairs goes through the expert's weights as one product, so two segments decode them twice. 16 tokens,
// 128 base-3 experts of 2048 x 768: 94 us (route 11, up 43, down 33, combine 3); 64 tokens, 8 Q2 experts of 4096 x
// 12288: 298 us (up 170, down 115), where up keeps shared memory 58 % busy, the tensor pipe 38 and issue 49; one
// token, 8 of 64 Q2 experts of 2048 x 1024: 31 us, about as long as the launches take the host.
// Four launches, each started while the one before ends (programmatic dependent launch):
//   route  a cluster of eight CTAs for one to four tokens: each computes the logits of every eighth expert,
//          the first collects them through the cluster's shared memory and picks.
//   up     the (token, expert) pairs are sorted by expert; the 8-output tiles (gate and up rows) of all experts
//          in use form one list that is dealt evenly to one CTA per SM. The products are those of
//          tern_rows.cuh. h = act(g) u in fp32.
//   down   the same over 16-row tiles of the down matrices and over slices of K where f is long. Sums of a pair and
//          slice go to the workspace. What h loses: the int8 form takes it as integers, off by 2^-27 of the largest
//          of its slot; the fp16 form rounds it to fp16, brought into range by a power of two per pair (2^-11 of
//          itself). Two fp16 terms for each h would keep 22 bits, for twice the MMAs and operand reads of a kernel
//          that shared memory already holds up; one is what a layer with fp16 activations between its products has.
//   combine  adds a token's pairs up, in the order of j and of the slices.
#include "tern_rows.cuh"

namespace tern {
namespace {

constexpr int kRouteCtas = 8, kRouteThreads = 256, kCombineThreads = 128;
constexpr int kMaxPairs = TERN_MOE_MAX_TOKENS * TERN_MOE_MAX_TOP_K;

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void store_first(double* local, double v) {  // into the first CTA's copy of *local
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(remote) : "r"(sm100::smem_u32(local)));
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(remote), "d"(v) : "memory");
}

// 64-bit key whose unsigned order is that of the doubles, -0 as 0, any NaN below everything (and above 0 = none).
__device__ __forceinline__ uint64_t order_key(double v) {
  if (v != v) return 1;
  const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
  return b >> 63 ? ~b : b | 1ull << 63;
}

// e^d with d's rounding to fp32 made good: e^(hi + lo) = e^hi (1 + lo).
__device__ __forceinline__ float exp_exact(double d) {
  const float hi = (float)d;
  const float e = expf(hi);
  return hi > -INFINITY ? fmaf(e, (float)(d - (double)hi), e) : e;
}

// Logits in fp64 (products of fp16 values are exact in fp32), so that experts next to one another at the
// border keep their order.
// Where there are fewer experts than warps in a cluster, 2, 4 or 8 warps share an expert's dot product.
template <int TOK>
__global__ void __cluster_dims__(kRouteCtas, 1, 1) __launch_bounds__(kRouteThreads) route_kernel(const __grid_constant__ MoeParams p) {
  __shared__ double logit[TOK][kMoeMaxExperts];
  constexpr int kWarps = kRouteCtas * kRouteThreads / 32;
  const int parts = p.experts * 8 <= kWarps ? 8 : p.experts * 4 <= kWarps ? 4 : p.experts * 2 <= kWarps ? 2 : 1;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t0 = (int)(blockIdx.x / kRouteCtas) * TOK;
  const int rank = (int)cluster_rank();
  sm100::griddep_launch_dependents();
  cluster_arrive();
  sm100::griddep_wait();
  bool met = false;  // the first CTA is known to run, so that its shared memory may be written
  for (int i = (int)(blockIdx.x * kRouteThreads + threadIdx.x); i < p.tokens * p.top_k; i += (int)gridDim.x * kRouteThreads)
    p.clear[i] = 0;  // largest |h| of each pair
  for (int i = rank + kRouteCtas * warp; i < p.experts * parts; i += kWarps) {
    const int e = i / parts, v0 = p.d / 8 * (i % parts) / parts, v1 = p.d / 8 * (i % parts + 1) / parts;
    double s[TOK][4] = {};  // four sums each: fp64 additions take long one after the other
    const uint4* w = reinterpret_cast<const uint4*>(p.router + (int64_t)e * p.d);
#pragma unroll 4
    for (int v = v0 + lane; v < v1; v += 32) {
      const uint4 a = __ldg(w + v);
      const uint32_t av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int k = 0; k < TOK; k++) {
        if (t0 + k >= p.tokens) break;
        const uint4 b = *(reinterpret_cast<const uint4*>(p.x + (int64_t)(t0 + k) * p.d) + v);
        const uint32_t bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int q = 0; q < 4; q++) {
          const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&av[q])), y = __half22float2(*reinterpret_cast<const __half2*>(&bv[q]));
          s[k][q] += (double)(x.x * y.x);
          s[k][q] += (double)(x.y * y.y);
        }
      }
    }
    if (!met) cluster_wait();
    met = true;
#pragma unroll
    for (int k = 0; k < TOK; k++) {
      double v = (s[k][0] + s[k][1]) + (s[k][2] + s[k][3]);
      for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == 0) store_first(&logit[k][i], v);
    }
  }
  if (!met) cluster_wait();
  cluster_arrive();
  cluster_wait();
  if (rank || warp >= TOK || t0 + warp >= p.tokens) return;
  if (parts > 1) {  // the parts' sums in their order; at most 64 of them, read before any is overwritten
    double v = 0.;
    if (lane < p.experts)
      for (int i = 0; i < parts; i++) v += logit[warp][lane * parts + i];
    __syncwarp();
    if (lane < p.experts) logit[warp][lane] = v;
    __syncwarp();
  }
  // One warp per token; lane l holds the logits of experts l, l + 32, ... as 64-bit keys whose unsigned order
  // is the logits' (NaN last). Each pick is three warp reductions: high word, low word, lowest index.
  const int t = t0 + warp;
  uint64_t key[kMoeMaxExperts / 32];
#pragma unroll
  for (int i = 0; i < kMoeMaxExperts / 32; i++) key[i] = lane + 32 * i < p.experts ? order_key(logit[warp][lane + 32 * i]) : 0;
  int mine = 0;  // lane j: pick j
  for (int j = 0; j < p.top_k; j++) {
    uint64_t best = key[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < kMoeMaxExperts / 32; i++)
      if (key[i] > best) {
        best = key[i];
        at = i;
      }
    const uint32_t hi = (uint32_t)(best >> 32), top = __reduce_max_sync(0xffffffffu, hi);
    const uint32_t low = __reduce_max_sync(0xffffffffu, hi == top ? (uint32_t)best : 0u);
    const uint32_t e = __reduce_min_sync(0xffffffffu, hi == top && (uint32_t)best == low ? (uint32_t)(lane + 32 * at) : 0xffffu);
    if ((e & 31) == lane)
#pragma unroll
      for (int i = 0; i < kMoeMaxExperts / 32; i++)
        if (i == (int)(e >> 5)) key[i] = 0;
    if (lane == j) mine = (int)e;
  }
  const double mx = logit[warp][__shfl_sync(0xffffffffu, mine, 0)];
  float sum = 0.f;
  for (int e = lane; e < p.experts; e += 32) sum += exp_exact(logit[warp][e] - mx);
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float w = lane < p.top_k ? exp_exact(logit[warp][mine] - mx) / sum : 0.f;
  float chosen = w;
  for (int o = 8; o; o >>= 1) chosen += __shfl_xor_sync(0xffffffffu, chosen, o);
  if (lane >= p.top_k) return;
  p.ids[t * p.top_k + lane] = mine;
  p.weights[t * p.top_k + lane] = p.renormalize ? w / chosen : w;
}

// ---- the experts ------------------------------------------------------------------------------------------
// The form of a product (gate/up or down) is the same for all experts of a call (side by side in one kernel the forms would
// share their registers): int8 digits or fp16 column tiles, see with_form. P::kRows pairs of an expert go through
// its weights together.
constexpr int kPlans = 9;  // cuts for up to 1, 2, 3, 4, 6, 8, 16, 32 and any number of tiles
__host__ __device__ constexpr int plan_tiles(int i) { return i < 4 ? i + 1 : i == 4 ? 6 : i == 5 ? 8 : i == 6 ? 16 : i == 7 ? 32 : 128; }

constexpr int kMaxRows = 16;  // pairs that go through an expert's weights together, at most

struct Lists {
  int segments, tiles;             // chunks of pairs; row tiles of all of them
  uint16_t pair[kMaxPairs];        // pairs sorted by expert
  uint16_t unsorted[kMaxPairs];
  uint16_t seg_expert[kMaxPairs], seg_first[kMaxPairs];
  uint8_t seg_count[kMaxPairs];
  int count[kMoeMaxExperts], first[kMoeMaxExperts];
  uint32_t total[kMoeMaxExperts / 32];
  int index[kMaxRows];             // rows of the activations of the current segment
  float mul[kMaxRows];             // and their powers of two
  uint32_t top[kMaxRows];          // largest |h| of each in this CTA
};

// Sorts the pairs by expert, in their own order within it (every CTA has to cut the same segments), and cuts
// them into segments of at most `cols`.
__device__ __forceinline__ void build_lists(const MoeParams& p, Lists& s, int cols, int tiles_per_segment) {
  constexpr int kPer = kMaxPairs / rows::kThreads, kWarps = kMoeMaxExperts / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, pairs = p.tokens * p.top_k;
  int e[kPer], place[kPer];
  if (tid < kMoeMaxExperts) s.count[tid] = 0;
#pragma unroll
  for (int c = 0; c < kPer; c++) e[c] = tid + c * rows::kThreads < pairs ? p.ids[tid + c * rows::kThreads] : -1;
  __syncthreads();
#pragma unroll
  for (int c = 0; c < kPer; c++)
    if (e[c] >= 0) place[c] = atomicAdd(&s.count[e[c]], 1);
  __syncthreads();
  // prefix sums over the experts: pairs in the low, segments in the high half of a word
  uint32_t n = 0, g = 0, sum = 0;
  if (tid < kMoeMaxExperts) {
    n = (uint32_t)s.count[tid];
    g = (n + cols - 1) / cols;
    sum = n | g << 16;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    if (lane == 31) s.total[warp] = sum;
  }
  __syncthreads();
  if (tid < kMoeMaxExperts) {
    uint32_t all = 0, base = 0;
#pragma unroll
    for (int w = 0; w < kWarps; w++) {
      const uint32_t v = s.total[w];
      if (w < warp) base += v;
      all += v;
    }
    const uint32_t at = base + sum - (n | g << 16);
    s.first[tid] = (int)(at & 0xffff);
    for (uint32_t i = 0; i < g; i++) {
      s.seg_expert[(at >> 16) + i] = (uint16_t)tid;
      s.seg_first[(at >> 16) + i] = (uint16_t)((at & 0xffff) + i * cols);
      s.seg_count[(at >> 16) + i] = (uint8_t)min((uint32_t)cols, n - i * cols);
    }
    if (tid == 0) {
      s.segments = (int)(all >> 16);
      s.tiles = (int)(all >> 16) * tiles_per_segment;
    }
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < kPer; c++)
    if (e[c] >= 0) s.unsorted[s.first[e[c]] + place[c]] = (uint16_t)(tid + c * rows::kThreads);
  __syncthreads();
#pragma unroll
  for (int c = 0; c < kPer; c++) {
    if (e[c] < 0) continue;
    const int me = tid + c * rows::kThreads, first = s.first[e[c]], of = s.count[e[c]];
    int rank = 0;
#pragma unroll 4
    for (int i = 0; i < of; i++) rank += s.unsorted[first + i] < me;
    s.pair[first + rank] = (uint16_t)me;
  }
  __syncthreads();
}

struct ExpertParams {
  MoeParams p;
  rows::Mat mat;
  rows::Split split[kPlans];
  int slices, slice_blocks;  // down: K cut into this many runs of blocks
};
// Blocks [b0, b0 + n) of K as a matrix of its own.
template <int L>
__device__ __forceinline__ rows::Mat slice_of(const rows::Mat& m, int b0, int n) {
  constexpr int kBlockK = rows::kBlk * rows::Lay<L>::kUnitK, kGroups = kBlockK / kGroup;
  rows::Mat s = m;
  s.codes += b0 * 128;
  s.scales += b0 * kGroups;
  s.K = min(m.K - b0 * kBlockK, n * kBlockK);
  s.row_bytes = min(m.row_bytes - b0 * 128, n * 128);
  s.groups = min(m.groups - b0 * kGroups, n * kGroups);
  s.units = min(m.units - b0 * rows::kBlk, n * rows::kBlk);
  return s;
}
__device__ __forceinline__ int first_tile(int tiles, int b) {
  const int ctas = (int)gridDim.x, each = tiles / ctas;
  return rows::first_tile(b, ctas, each, tiles - each * ctas);
}
__device__ __forceinline__ const rows::Split& split_for(const ExpertParams& q, int tiles) {
  int i = 0;
  while (i < kPlans - 1 && plan_tiles(i) < tiles) i++;
  return q.split[i];
}

template <int L, class P>
__global__ void __launch_bounds__(rows::kThreads, 1) moe_up_kernel(const __grid_constant__ ExpertParams q) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Lists s;
  const MoeParams& p = q.p;
  constexpr int kStep = P::kTileRows / 2;
  static_assert(P::kRows <= kMaxRows);
  sm100::griddep_launch_dependents();
  sm100::griddep_wait();
  const int per = p.f / kStep;  // tiles of a segment
  build_lists(p, s, P::kRows, per);
  const int t1 = first_tile(s.tiles, (int)blockIdx.x + 1);
#pragma unroll 1
  for (int t = first_tile(s.tiles, (int)blockIdx.x); t < t1;) {
    const int g = t / per, a = t % per, b = min(per, a + t1 - t), n = s.seg_count[g];
    const uint16_t* pair = s.pair + s.seg_first[g];
    if ((int)threadIdx.x < n) {
      s.index[threadIdx.x] = pair[threadIdx.x] / p.top_k;
      s.top[threadIdx.x] = 0;
    }
    __syncthreads();
    const int64_t first = (int64_t)s.seg_expert[g] * 2 * p.f;
    P prod;
    prod.run(smem, split_for(q, b - a), q.mat, rows::Map{first, first + p.f, p.f, kStep, 0}, a, b, rows::HalfRows{p.x, p.d, s.index},
             n, [] {}, [&](int tile, int r, int c, float gate, float up) {
               const float h = act_fwd(p.act, gate) * up;
               p.h[(int64_t)pair[c] * p.f + tile * kStep + r] = h;
               // largest finite |h| of the pair, as bits: order does not matter to a maximum
               const uint32_t bits = __float_as_uint(h) & 0x7fffffffu;
               if (p.scaled && bits < 0x7f800000u) atomicMax(s.top + c, bits);
             });
    __syncthreads();
    if (p.scaled && (int)threadIdx.x < n) atomicMax(p.clear + pair[threadIdx.x], s.top[threadIdx.x]);
    __syncthreads();
    t += b - a;
  }
}

template <int L, class P>
__global__ void __launch_bounds__(rows::kThreads, 1) moe_down_kernel(const __grid_constant__ ExpertParams q) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Lists s;
  const MoeParams& p = q.p;
  constexpr int kStep = P::kTileRows;
  static_assert(P::kRows <= kMaxRows);
  sm100::griddep_launch_dependents();
  sm100::griddep_wait();
  const int per = p.d / kStep, tid = threadIdx.x;
  build_lists(p, s, P::kRows, per * q.slices);
  const int t1 = first_tile(s.tiles, (int)blockIdx.x + 1);
#pragma unroll 1
  for (int t = first_tile(s.tiles, (int)blockIdx.x); t < t1;) {
    const int g = t / per / q.slices, sl = t / per % q.slices;  // segment and slice of K
    const int a = t % per, b = min(per, a + t1 - t), n = s.seg_count[g];
    const uint16_t* pair = s.pair + s.seg_first[g];
    if (tid < n) {
      const int pr = pair[tid];
      s.index[tid] = pr;
      if (P::kMode == rows::kFp16) {
        // the fp16 form takes h times a power of two that brings the pair's largest finite one to [2^14, 2^15)
        const uint32_t top = p.clear[pr];
        s.mul[tid] = top == 0 ? 1.f : rows::exp2i(min(100, 15 - rows::exponent(top)));
      }
    }
    __syncthreads();
    const int64_t first = (int64_t)s.seg_expert[g] * p.d;
    P prod;
    float* zs = p.z + (int64_t)sl * p.tokens * p.top_k * p.d;
    prod.run(smem, split_for(q, b - a), slice_of<L>(q.mat, sl * q.slice_blocks, q.slice_blocks),
             rows::Map{first, first, p.d, kStep, kStep / 2}, a, b,
             rows::FloatRows{p.h + sl * q.slice_blocks * rows::kBlk * rows::Lay<L>::kUnitK, p.f, s.index, s.mul}, n, [] {},
             [&](int tile, int r, int c, float z, float) {
               zs[(int64_t)pair[c] * p.d + tile * kStep + r] = P::kMode == rows::kFp16 ? z / s.mul[c] : z;
             });
    __syncthreads();
    t += b - a;
  }
}

// y = sum_j p_j (sum over the slices of z_j) (+ residual), four outputs a thread. (The last CTA at a strip of
// outputs adding them up inside the down kernel left that to the few CTAs that the last segment is dealt to:
// at 64 tokens, 8 experts of 4096 x 12288 the down kernel took 430 us so, against 144 and 5 for this one.)
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const __grid_constant__ MoeParams p) {
  const int per = p.d / 4, i = (int)(blockIdx.x * kCombineThreads + threadIdx.x);
  sm100::griddep_launch_dependents();
  sm100::griddep_wait();
  if (i >= p.tokens * per) return;
  const int tok = i / per, pairs = p.tokens * p.top_k;
  const int64_t at = (int64_t)tok * p.d + (i - tok * per) * 4;
  float y[4] = {};
  const float4* z = reinterpret_cast<const float4*>(p.z + (int64_t)tok * p.top_k * p.d) + (i - tok * per);
#pragma unroll 4
  for (int j = 0; j < p.top_k; j++) {
    const float w = __ldcg(p.weights + tok * p.top_k + j);
    float4 v = __ldcg(z + (int64_t)j * per);
    for (int s = 1; s < p.slices; s++) {
      const float4 u = __ldcg(z + ((int64_t)s * pairs + j) * per);
      v.x += u.x;
      v.y += u.y;
      v.z += u.z;
      v.w += u.w;
    }
    y[0] = fmaf(w, v.x, y[0]);
    y[1] = fmaf(w, v.y, y[1]);
    y[2] = fmaf(w, v.z, y[2]);
    y[3] = fmaf(w, v.w, y[3]);
  }
#pragma unroll
  for (int k = 0; k < 4; k++) p.y[at + k] = f2h(p.residual ? y[k] + h2f(p.residual[at + k]) : y[k]);
}

constexpr size_t kRoom = 227 * 1024 - (sizeof(Lists) + 1023) / 1024 * 1024 - 1024;  // dynamic shared memory

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

// Blocks of each of s slices: an even number, since a base-3 block's scales are 10 bytes and are copied by words.
int slice_blocks(int blocks, int s) { return s == 1 ? blocks : ((blocks + s - 1) / s + 1) / 2 * 2; }

template <int L, bool UP, class P>
cudaError_t launch_form(const tern_matrix& W, const MoeParams& p, cudaStream_t st) {
  ExpertParams q;
  q.p = p;
  q.mat = rows::Mat{static_cast<const uint8_t*>(W.codes), W.scales, W.code_row_stride, W.scale_row_stride, (int)W.k,
                    (int)row_bytes(W.layout, W.k), (int)(W.k / kGroup), (int)((row_bytes(W.layout, W.k) + 31) / 32)};
  size_t smem = 0;
  const int blocks = (q.mat.units + rows::kBlk - 1) / rows::kBlk;
  q.slices = UP ? 1 : p.slices;
  q.slice_blocks = slice_blocks(blocks, q.slices);
  for (int i = 0; i < kPlans; i++) {
    if (!P::plan(plan_tiles(i), std::min(q.mat.units, q.slice_blocks * rows::kBlk), kRoom, q.split + i)) return cudaErrorInvalidValue;
    smem = std::max(smem, P::smem_bytes(q.split[i]));
  }
  const void* kern = UP ? reinterpret_cast<const void*>(&moe_up_kernel<L, P>) : reinterpret_cast<const void*>(&moe_down_kernel<L, P>);
  const cudaError_t e = allow_smem(kern, kRoom);
  if (e != cudaSuccess) return e;
  return launch(kern, sm_count(), rows::kThreads, smem, st, &q);
}

// f(form) with the form of the product that a call takes: int8 digits for few pairs per expert (on average), else
// fp16 column tiles. The int8 form decodes faster, but an expert of more than P::kRows pairs (Q2 two, else one) takes
// it again for the next; 64 experts of 2048 x 1024, 8 chosen, us with int8 and with fp16:
//   pairs per expert   1/2        3/4        1          2
//   Q2                 45 / 47    49 / 52    55 / 57    70 / 67
//   base-3             56 / 58    66 / 67    76 / 73   116 / 87     (128 experts of 2048 x 768: 70 / 73, 86 / 84, 101 / 93)
//   binary             42 / 57    48 / 62    52 / 69    72 / 82
// Two column tiles where an expert's pairs often need
// them; eight experts of 4096 x 12288, 2 chosen, us with one and with two:
//   pairs per expert   4            8            16
//   Q2                 153 / 206    193 / 218    302 / 297
//   base-3             245 / 238    387 / 342    680 / 529
//   binary             212 / 199    343 / 276    591 / 448
template <class P> struct Form { using type = P; };
template <int L, class F>
auto with_form(int tokens, int top_k, int experts, F f) {
  const int pairs = tokens * top_k;
  const int few = L == TERN_Q1_0_G128 ? 2 * experts : L == TERN_Q2_0_G128 ? experts : experts / 2;
  if (tokens == 1 || pairs <= few) return f(Form<rows::Product<L, rows::kInt8, 1>>{});
  if (pairs < (L == TERN_Q2_0_G128 ? 14 : 4) * experts) return f(Form<rows::Product<L, rows::kFp16, 1>>{});
  return f(Form<rows::Product<L, rows::kFp16, 2>>{});
}

template <int L, bool UP>
cudaError_t launch_experts(const tern_matrix& W, const MoeParams& p, cudaStream_t st) {
  return with_form<L>(p.tokens, p.top_k, p.experts, [&](auto form) { return launch_form<L, UP, typename decltype(form)::type>(W, p, st); });
}

// Slices of K for the down products: the fewest (up to eight) whose operands stay in shared memory while a CTA
// goes down the rows. (Passes over K inside a CTA build them again for every few tiles: 8 experts of
// 4096 x 12288 at 64 tokens took 333 us so, 144 with three slices.) A slice is not empty.
template <int L>
int down_slices(int64_t f, int tokens, int top_k, int experts) {
  const int units = (int)((row_bytes(L, f) + 31) / 32), blocks = (units + rows::kBlk - 1) / rows::kBlk;
  return with_form<L>(tokens, top_k, experts, [&](auto form) {
    using P = typename decltype(form)::type;
    int s = 1;
    for (; s < 8; s++) {
      const int n = slice_blocks(blocks, s);
      rows::Split split;
      if (P::plan(128, std::min(units, n * rows::kBlk), kRoom, &split) && split.pass >= n) break;
    }
    const int n = slice_blocks(blocks, s);
    return (blocks + n - 1) / n;
  });
}

template <int L>
bool takes_fp16(const MoeParams& p) {
  return with_form<L>(p.tokens, p.top_k, p.experts, [](auto form) { return decltype(form)::type::kMode == rows::kFp16; });
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

MoePlan moe_plan(int32_t down_layout, int64_t tokens, int64_t d, int64_t f, int experts, int top_k) {
  MoePlan w{};
  w.slices = down_layout == TERN_Q2_0_G128     ? down_slices<TERN_Q2_0_G128>(f, (int)tokens, top_k, experts)
             : down_layout == TERN_T3_5PB_G128 ? down_slices<TERN_T3_5PB_G128>(f, (int)tokens, top_k, experts)
                                               : down_slices<TERN_Q1_0_G128>(f, (int)tokens, top_k, experts);
  const size_t pairs = (size_t)tokens * top_k;
  size_t o = 0;
  auto take = [&](size_t bytes) { const size_t at = o; o += (bytes + 255) / 256 * 256; return at; };
  w.ids = take(pairs * 4);
  w.weights = take(pairs * 4);
  w.clear = take(pairs * 4);
  w.h = take(pairs * f * 4);
  w.z = take(w.slices * pairs * d * 4);
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
  p.slices = w.slices;
  // (the layouts, and with them the forms of the two products, may differ)
  p.scaled = D.layout == TERN_Q2_0_G128     ? takes_fp16<TERN_Q2_0_G128>(p)
             : D.layout == TERN_T3_5PB_G128 ? takes_fp16<TERN_T3_5PB_G128>(p)
                                            : takes_fp16<TERN_Q1_0_G128>(p);
  const int tok = p.tokens > 32 ? 4 : p.tokens > 16 ? 2 : 1;
  const void* route = tok == 4   ? reinterpret_cast<const void*>(&route_kernel<4>)
                      : tok == 2 ? reinterpret_cast<const void*>(&route_kernel<2>)
                                 : reinterpret_cast<const void*>(&route_kernel<1>);
  cudaError_t e = launch(route, (p.tokens + tok - 1) / tok * kRouteCtas, kRouteThreads, 0, st, &p);
  if (e != cudaSuccess) return e;
  e = dispatch<true>(G, p, st);
  if (e != cudaSuccess) return e;
  e = dispatch<false>(D, p, st);
  if (e != cudaSuccess) return e;
  return launch(reinterpret_cast<const void*>(&combine_kernel), (p.tokens * (p.d / 4) + kCombineThreads - 1) / kCombineThreads, kCombineThreads, 0, st, &p);
}

}  // namespace tern
