// Many-row products of the layer operators on tcgen05 tensor cores, weights decoded into tensor memory:
//     forward     z[t][n]  = sum_k x[t][k]  s[n][k/128] t[n][k]     (tern_linear)
//     transposed  dx[t][k] = sum_n dz[t][n] s[n][k/128] t[n][k]     (tern_linear_backward)
//
// A pair of CTAs computes tiles of 256 weight rows (forward) or weight columns (transposed), 128 in each, by
// `bn` rows of x, 64 terms of the sum at a time. In D = A B^T the decoded weights are A (cta_group::2,
// M = 256), the activations B.
//   * What bounds it. Per 64 terms the MMAs take bn / 256 x 512 cycles. With one CTA a tile, B would be
//     written to shared memory by TMA and read by the MMAs at 128 bytes a cycle in all, which is all that
//     shared memory gives, and would cross from L2 at 64 bytes a cycle and SM, more than L2 gives (a version
//     of this kernel without pairs stopped at 0.9 PFLOP/s there). As a pair each CTA brings half of B. And
//     A does not go through shared memory at all, it lives in tensor memory: decoder warps turn codes into
//     fp16 2 s t (binary: s t) in registers, exactly, and store them with tcgen05.st; 32 columns hold 64 terms.
//   * Tensor memory: two accumulators of up to 192 columns, so that the epilogue of a tile runs beside the
//     MMAs of the next, and a ring of 4 to 8 A stages of 32 columns in what they leave.
//   * Warps: 0 and 2 TMA, 1 MMA, 4-11 epilogue (two for each 32 rows of A, every other 16 columns each), 12 on
//     decode (three sets of four; a set takes every third stage, which hides the latencies between a stage's
//     arrival and its decoded weights').
//   * bn is chosen by the host so that the tiles fill whole waves of CTAs. Where there are few tiles, two to four
//     pairs in a cluster take a part of a tile's sum each and exchange the accumulators through each other's
//     shared memory, in a fixed order.
//   * Transposed: A's rows are the columns of the packed rows, whose group is one scale per packed row.
//     ldmatrix.trans hands a lane 16-bit pieces of two adjacent rows; each field of theirs is a finished
//     pair of A, and the 16x128b store shape has rows by lane / 4 and columns by lane % 4 as ldmatrix has.
//   * Base-3 bytes go through a table of five 2-bit fields each and become words of Q2's form first.
// Every wait is bounded in wall time; on expiry the CTA raises its abort flag, ORs TERN_DEVICE_TIMEOUT into
// the caller's status word, lets copies and MMAs in flight end, frees tensor memory and exits.
#include <cuda.h>

#include "sm100.cuh"
#include "tern_layer.cuh"

namespace tern {
namespace {

using namespace sm100;

constexpr int BM = 128;      // rows of A per tile
constexpr int BK = 64;       // terms per stage (one 128-byte swizzle row of fp16)
constexpr int kMaxBN = 192;  // rows of x per tile (of a pair of CTAs)
constexpr int kMaxSplits = 4;  // pairs that may share a tile's sum (a cluster of 8 CTAs)
constexpr int STAGES = 8;    // TMA ring
constexpr int ASTAGES = 8;   // A ring in tensor memory, at most: what the accumulators leave of it
// 24 warps: the forward epilogue has more to do, the transposed decoding
constexpr int kThreads = 768, kMaxSets = 4;
constexpr int kEpiBarrier = 1, kSetBarrier = 2;  // named barriers: the epilogue's, and one for each decoder set
constexpr int epi_warps(bool trans) { return trans ? 4 : 8; }
constexpr int decoder_sets(bool trans) { return (kThreads / 32 - 4 - epi_warps(trans)) / 4; }
constexpr uint32_t kTmemCols = 512;  // accumulators at 0 and bn, the A ring from 2 bn on
// Limit of a wait. The epilogue's wait covers a whole sum: that much more for each 64 terms of it (they take about 0.3 us).
constexpr uint64_t kWaitNs = 1000000000ull, kBlockNs = 1000;

constexpr int X_BYTES = kMaxBN / 2 * BK * 2;  // a CTA's half of the tile's rows of x
constexpr int P_BYTES = BM * 32;  // codes of a stage: forward 128 rows x 16 or 32 bytes, transposed 64 x 16, 32 or 48
constexpr int OFF_P = STAGES * X_BYTES;
constexpr int OFF_Q = OFF_P + STAGES * P_BYTES;  // transposed base-3: two tiles of each set in Q2's form [64][32]
constexpr int OFF_LUT = OFF_Q + 2 * kMaxSets * 64 * 32;
constexpr int kBigTiles = 16;  // tiles that decoders may be ahead of the epilogue, and more
constexpr int OFF_BIG = OFF_LUT + 256 * 32 * 4;
constexpr int OFF_BAR = OFF_BIG + kBigTiles * BM;
constexpr int NUM_BARS = 2 * STAGES + 2 * ASTAGES + 4 + 1;
constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;  // + slack to align the base to 1024

struct Params {
  int64_t m;             // rows of x
  int64_t n;             // packed rows
  int64_t k;             // weights of a packed row
  int64_t nout;          // outputs of a row: n, n / 2 (gated) or k (transposed)
  int terms;             // length of the sum: k or n
  int bn, rtiles, mtiles;
  int splits;            // pairs of CTAs that share a tile's sum, up to kMaxSplits; if more than one, a pair has one tile
  const uint16_t* x;
  int64_t xstride;
  const uint8_t* codes;
  int64_t cstride;
  const uint16_t* scales;
  int64_t sstride;
  uint16_t* y;
  Epilogue e;
  uint32_t* status;
};

// ---- tensor memory stores and A operands from it -----------------------------------------------------
__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
      "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]),
      "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// 16 rows x 32 columns: r[2i] is (row lane / 4, column 4 i + lane % 4), r[2i + 1] the same 8 rows below.
__device__ __forceinline__ void tmem_st_16x128b_x8(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void mma_f16_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(tmem_d), "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// ---- pairs of CTAs ------------------------------------------------------------------------------------
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)), "r"(ncols) : "memory");
}
__device__ __forceinline__ void tmem_relinquish_pair() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// Arrives on `bar` of both CTAs (of cluster ranks first and first + 1) once every MMA issued before has completed.
__device__ __forceinline__ void commit_both(uint64_t* bar, int first) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
               ::"r"(smem_u32(bar)), "h"((uint16_t)(3 << first)) : "memory");
}
__device__ __forceinline__ void commit_own(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// Address of `local` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t in_cta(const void* local, int rank) {
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(local)), "r"(rank));
  return remote;
}
// Arrives on the copy of `bar` of the pair's first CTA.
__device__ __forceinline__ void arrive_first(uint64_t* bar, int first) {
  const uint32_t remote = in_cta(bar, first);
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(remote) : "memory");
}
// Waits on a barrier that both CTAs arrive on.
__device__ __forceinline__ bool try_wait_pair(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool wait_pair(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t* status) {
  return mbar_wait_bounded(bar, parity, abort, status, TERN_DEVICE_TIMEOUT, kWaitNs) && try_wait_pair(bar, parity);
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// Named barrier of `threads` threads; true if `fine` is true in all of them.
__device__ __forceinline__ bool bar_all(int id, int threads, bool fine) {
  uint32_t r = fine;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %0, 0;\n\tbar.red.and.pred q, %1, %2, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
               : "+r"(r) : "r"(id), "r"(threads) : "memory");
  return r != 0;
}

// ---- decoding ------------------------------------------------------------------------------------------
// Scales from 2^15 on (kBigScale, as fp16 bits): 2 s does not fit fp16. The epilogue leaves out the outputs they
// belong to; finish_big computes them term by term instead.
constexpr uint32_t kBigScale = 0x7800;

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&v);
}
// 16 two's-complement fields of a word -> eight fp16 pairs 2 s t (s2: s in both halves). A field in the top
// bits of a half's high byte is +-2.0 or 0: shifted copies of the word hold field f of every byte there, one
// permute takes the bytes of two adjacent weights from two of them, one mask leaves the fields.
__device__ __forceinline__ void pairs_q2(uint32_t w, uint32_t s2, uint32_t* o) {
  const uint32_t v[4] = {w << 6, w << 4, w << 2, w};  // field f of every byte at its top
#pragma unroll
  for (int j = 0; j < 8; j++)  // weights 2j and 2j + 1: fields f, f + 1 of byte j / 2
    o[j] = hmul2(__byte_perm(v[2 * (j & 1)], v[2 * (j & 1) + 1], (j >> 1) << 4 | (4 + (j >> 1)) << 12) & 0xC000C000u, s2);
}
// The same with a multiplication for the permute and the shifts, where base-3's table needs the ALU: it brings
// the two fields of a pair, masked first, to bits 14..15 and 30..31.
__device__ __forceinline__ void pairs_mul(uint32_t w, uint32_t s2, uint32_t* o) {
#pragma unroll
  for (int j = 0; j < 8; j++) {
    const int jj = j & 3, a = 14 - 4 * jj;
    const uint32_t x = (j < 4 ? w : w >> 16) & (0xFu << (4 * jj));
    o[j] = hmul2((x * ((1u << a) + (1u << (a + 14)))) & 0xC000C000u, s2);
  }
}
// 32 sign bits -> sixteen fp16 pairs s t: the bit of a weight at the top of a half, flipped into the sign of s.
__device__ __forceinline__ void pairs_q1(uint32_t w, uint32_t s2, uint32_t* o) {
  uint32_t v[8];  // bit f of every byte at its top
#pragma unroll
  for (int f = 0; f < 8; f++) v[f] = w << (7 - f);
#pragma unroll
  for (int j = 0; j < 16; j++)
    o[j] = (~__byte_perm(v[2 * (j & 3)], v[2 * (j & 3) + 1], (j >> 2) << 4 | (4 + (j >> 2)) << 12) & 0x80008000u) ^ s2;
}
// 64 trits as four words of 16 two's-complement fields. Trit 64 q starts at digit (64 q) mod 5 of byte
// (64 q) / 5, which is 0, 12, 9, 6 or 3 past a 16-byte boundary for q mod 5 = V = 0 .. 4: u and v are the 32
// bytes from that boundary on. lut: this lane's column of the table (32 copies, so that no two lanes of a warp
// meet in a bank).
template <int V>
__device__ __forceinline__ void t3_words_v(const uint4& u, const uint4& v, const uint32_t* lut, uint32_t (&w)[4]) {
  constexpr int kOff = (64 * V / 5) % 16, R0 = (64 * V) % 5, NB = (R0 + 63) / 5 + 1;
  const uint32_t b[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
  w[0] = w[1] = w[2] = w[3] = 0;
#pragma unroll
  for (int j = 0; j < NB; j++) {
    const uint32_t f = lut[__byte_perm(b[(kOff + j) >> 2], 0u, 0x4440 + ((kOff + j) & 3)) * 32u];
    const int at = 10 * j - 2 * R0;  // bit of the byte's first field
    if (at < 0) {
      w[0] |= f >> -at;
    } else {
      w[at >> 5] |= f << (at & 31);
      if ((at & 31) > 22 && (at >> 5) < 3) w[(at >> 5) + 1] |= f >> (32 - (at & 31));
    }
  }
}
__device__ __forceinline__ void t3_words(int v5, const uint8_t* p, const uint32_t* lut, uint32_t (&w)[4]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p), v = *reinterpret_cast<const uint4*>(p + 16);
  switch (v5) {
    case 0: t3_words_v<0>(u, v, lut, w); break;
    case 1: t3_words_v<1>(u, v, lut, w); break;
    case 2: t3_words_v<2>(u, v, lut, w); break;
    case 3: t3_words_v<3>(u, v, lut, w); break;
    default: t3_words_v<4>(u, v, lut, w); break;
  }
}

// ---- epilogue --------------------------------------------------------------------------------------------
// 16 rows of x from t0 on of output j: this lane writes the first `lim`. r arrives from tensor memory.
template <int ACT>
__device__ __forceinline__ void finish(const Params& p, uint32_t (&r)[16], float half, float bias, int64_t t0, int64_t j, int lim) {
  uint16_t rv[16];
  if (p.e.residual) {
    const uint16_t* res = p.e.residual + t0 * p.nout + j;
#pragma unroll
    for (int i = 0; i < 16; i++, res += p.nout)
      if (i < lim) rv[i] = *res;
  }
  if (p.e.preact) {
    uint16_t* z = p.e.preact + t0 * p.n + j;
#pragma unroll
    for (int i = 0; i < 16; i++, z += p.n)
      if (i < lim) *z = f2h(fmaf(__uint_as_float(r[i]), half, bias));
  }
  uint16_t* y = p.y + t0 * p.nout + j;
#pragma unroll
  for (int i = 0; i < 16; i++, y += p.nout) {
    float v = act_fwd(ACT, fmaf(__uint_as_float(r[i]), half, bias));
    if (p.e.residual) v += h2f(rv[i]);
    if (i < lim) *y = f2h(v);
  }
}
// Lanes l and l + 16 hold the gate and the up sums of one output; of two rows of x the lower lane finishes
// the first, the upper one (`up`) the second.
template <int ACT>
__device__ __forceinline__ void finish_gated(const Params& p, uint32_t (&r)[16], float half, float bias, int64_t t0, int64_t j, int lim, bool up) {
  const int own = up ? 1 : 0;
  uint16_t rv[8];
  if (p.e.residual) {
    const uint16_t* res = p.e.residual + (t0 + own) * p.nout + j;
#pragma unroll
    for (int i = 0; i < 8; i++, res += 2 * p.nout)
      if (2 * i + own < lim) rv[i] = *res;
  }
  if (p.e.preact) {
    uint16_t* z = p.e.preact + t0 * p.n + j + (up ? p.nout : 0);
#pragma unroll
    for (int i = 0; i < 16; i++, z += p.n)
      if (i < lim) *z = f2h(fmaf(__uint_as_float(r[i]), half, bias));
  }
  uint16_t* y = p.y + (t0 + own) * p.nout + j;
#pragma unroll
  for (int i = 0; i < 8; i++, y += 2 * p.nout) {
    const float z0 = fmaf(__uint_as_float(r[2 * i]), half, bias), z1 = fmaf(__uint_as_float(r[2 * i + 1]), half, bias);
    const float got = __shfl_xor_sync(0xffffffffu, up ? z0 : z1, 16);
    float v = act_fwd(ACT, up ? got : z0) * (up ? z1 : got);
    if (p.e.residual) v += h2f(rv[i]);
    if (2 * i + own < lim) *y = f2h(v);
  }
}

template <int LAYOUT, bool TRANS>
__device__ __forceinline__ void write_outputs(const Params& p, uint32_t (&r)[16], float bias, int64_t t0, int64_t j, int lim, bool up) {
  constexpr float half = LAYOUT == TERN_Q1_0_G128 ? 1.f : 0.5f;  // the accumulators hold 2 s t x (binary: s t x)
  if constexpr (TRANS) {
    uint16_t* y = p.y + t0 * p.nout + j;
#pragma unroll
    for (int i = 0; i < 16; i++, y += p.nout)
      if (i < lim) *y = f2h(__uint_as_float(r[i]) * half);
  } else {
    with_act(p.e.act, [&](auto act) {
      if (p.e.gated) finish_gated<act.value>(p, r, half, bias, t0, j, lim, up);
      else finish<act.value>(p, r, half, bias, t0, j, lim);
    });
  }
}
// Row of A, as an output of the tile (gated: of the gate or the up half), that `lane` of the warps at `quad` holds.
template <int LAYOUT, bool TRANS>
__device__ __forceinline__ int output_of(int quad, int lane, bool gated) {
  if (!TRANS) return gated ? quad * 16 + (lane & 15) : quad * 32 + lane;
  if (LAYOUT == TERN_Q1_0_G128) return 16 * (lane & 7) + 4 * quad + (lane >> 3);
  return 64 * (quad >> 1) + 8 * (lane & 7) + 4 * (quad & 1) + (lane >> 3);
}

// The outputs that the epilogue left out, in all tiles of this CTA. Runs when the pipeline is done and tensor memory is
// free: it may take longer than any wait allows, and nothing waits for it. A warp takes 32 outputs by 16 rows of x.
template <int LAYOUT, bool TRANS>
__device__ __noinline__ void finish_big(const Params p, int rank, int slice, int pair, int pairs, int tiles) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const bool gated = !TRANS && p.e.gated, up = gated && lane >= 16;
  const auto is_big = [](uint16_t s) { return (s & 0x7fffu) >= kBigScale; };
  for (int tile = pair; tile < tiles; tile += pairs) {
    const int64_t r0 = (int64_t)(tile / p.mtiles * 2 + rank) * (gated ? 64 : BM), m0 = (int64_t)(tile % p.mtiles) * p.bn;
    const int cols = (int)(p.m - m0 < p.bn ? p.m - m0 : p.bn);
    for (int item = warp; 16 * (item >> 2) < cols; item += kThreads / 32) {
      const int quad = item & 3, c0 = 16 * (item >> 2);
      if ((item >> 2) % p.splits != slice) continue;
      const int64_t j = r0 + output_of<LAYOUT, TRANS>(quad, lane, gated), row = j + (up ? p.nout : 0), t0 = m0 + c0;
      const bool in = j < p.nout;
      bool hit = false;
      if (TRANS) {
        if (r0 < p.nout)
          for (int64_t n = lane; n < p.n && !hit; n += 32) hit = is_big(p.scales[n * p.sstride + r0 / kGroup]);
        hit = __any_sync(0xffffffffu, hit);
      } else {
        for (int64_t g = 0; in && !hit && g < p.k / kGroup; g++) hit = is_big(p.scales[row * p.sstride + g]);
        if (gated) hit |= __shfl_xor_sync(0xffffffffu, hit, 16);
      }
      const int lim = in && hit ? cols - c0 : 0;
      if (!__any_sync(0xffffffffu, lim > 0)) continue;
      float z[16] = {};
      if (lim > 0) {
#pragma unroll 1
        for (int64_t q = 0; q < p.terms; q++) {
          const int64_t n = TRANS ? q : row, k = TRANS ? j : q;
          const float w = h2f(p.scales[n * p.sstride + k / kGroup]) * decode_t(LAYOUT, p.codes + n * p.cstride, k);
          const uint16_t* x = p.x + t0 * p.xstride + q;
#pragma unroll
          for (int i = 0; i < 16; i++, x += p.xstride)
            if (i < lim) z[i] = fmaf(w, h2f(*x), z[i]);
        }
      }
      __syncwarp();
      uint32_t r[16];
#pragma unroll
      for (int i = 0; i < 16; i++) r[i] = __float_as_uint(2.f * z[i]);  // the accumulators' unit
      write_outputs<LAYOUT, TRANS>(p, r, !TRANS && p.e.bias && in ? h2f(p.e.bias[row]) : 0.f, t0, j, lim, up);
    }
  }
}

// ---- the kernel ------------------------------------------------------------------------------------------
template <int LAYOUT, bool TRANS>
__global__ void __launch_bounds__(kThreads, 1)
layer_gemm_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_w, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr int kEpi = epi_warps(TRANS), SETS = decoder_sets(TRANS), kFirstDecoder = 4 + kEpi;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + OFF_BAR);  // TMA -> decoders, MMA
  uint64_t* empty = full + STAGES;                               // MMA -> TMA
  uint64_t* dfull = empty + STAGES;                              // decoders -> MMA
  uint64_t* dempty = dfull + ASTAGES;                            // MMA -> decoders
  uint64_t* tfull = dempty + ASTAGES;                            // MMA -> epilogue (2)
  uint64_t* tempty = tfull + 2;                                  // epilogue -> MMA (2)
  uint64_t* drain = tempty + 2;                                  // MMA completion on abort
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_MISC + 4);
  uint32_t* lut = reinterpret_cast<uint32_t*>(smem + OFF_LUT);
  volatile int* left_out = reinterpret_cast<volatile int*>(smem + OFF_MISC + 8);  // the epilogue left outputs to finish_big
  // per tile (in turn) and row of A: a scale of kBigScale or more was met (transposed: row 0 for the whole tile)
  volatile uint8_t* big = smem + OFF_BIG;

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  // the CTA's place in its pair, the pair's first CTA in the cluster, and the pair's slice of the sum; a cluster is
  // `splits` pairs, `pair` and `pairs` count clusters
  const int rank = (int)cluster_rank() & 1, first = (int)cluster_rank() - rank, slice = first / 2;
  const int pair = (int)blockIdx.x / (2 * p.splits), pairs = (int)gridDim.x / (2 * p.splits);
  const int tiles = (p.rtiles + 1) / 2 * p.mtiles;  // of pairs
  const int all_blocks = (p.terms + BK - 1) / BK;
  const int first_kb = all_blocks * slice / p.splits, kblocks = all_blocks * (slice + 1) / p.splits - first_kb;
  const uint32_t a_col = 2 * p.bn, a_stages = min((kTmemCols - a_col) / 32, (uint32_t)ASTAGES);
  const bool gated = !TRANS && p.e.gated;
  const int step = gated ? 64 : BM;  // outputs of a tile

  griddep_launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; i++) { mbar_init(full + i, 2); mbar_init(empty + i, 1); }
    for (int i = 0; i < ASTAGES; i++) { mbar_init(dfull + i, 8); mbar_init(dempty + i, 1); }
    for (int i = 0; i < 2; i++) { mbar_init(tfull + i, 1); mbar_init(tempty + i, 2 * kEpi); }
    mbar_init(drain, 1);
    *abort_flag = 0;
    *left_out = 0;
    fence_mbar_init();
  }
  for (int i = threadIdx.x; i < kBigTiles * BM; i += kThreads) big[i] = 0;
  if (warp == 0 && lane == 0) { prefetch_tmap(&tmap_x); prefetch_tmap(&tmap_w); }
  if (LAYOUT == TERN_T3_5PB_G128) {
    // a thread computes one entry and stores a third of its copies, a warp's in different banks at a time
    const int v = threadIdx.x % 256;
    uint32_t f = 0, r = (uint32_t)v;
    if (v < 243) {
#pragma unroll
      for (int d = 0; d < 5; d++) { f |= ((r % 3u + 3u) & 3u) << (2 * d); r /= 3u; }  // c - 1 as two bits
    }  // an invalid byte reads as five t = 0
    for (int i = threadIdx.x / 256; i < 32; i += kThreads / 256) lut[v * 32 + ((v + i) & 31)] = f;
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_holder, kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers are ready before either arrives on the other's
  tc_fence_after();
  griddep_wait();  // from here on operands are read and results written
  const uint32_t tmem = __reduce_or_sync(0xffffffffu, *tmem_holder);  // the same in all lanes, in a uniform register

  if (warp == 0 || warp == 2) {
    // ------------------------------------------------------------------ TMA producers
    // Warp 0 brings the rows of x, warp 2 the codes. As in the MMA warp the whole warp runs the loop and one
    // elected lane issues (one lane's loop with both took 600 cycles a stage, more than the MMAs).
    constexpr int P_ROW = TRANS ? (LAYOUT == TERN_Q1_0_G128 ? 16 : LAYOUT == TERN_Q2_0_G128 ? 32 : 48)
                                : (LAYOUT == TERN_T3_5PB_G128 ? 32 : 16);
    const uint32_t bytes = warp == 0 ? (uint32_t)p.bn / 2 * BK * 2 : (TRANS ? BK : BM) * P_ROW;
    uint32_t ph = 1;
    int s = 0, sent = 0;
    bool dead = false;
    for (int tile = pair; tile < tiles; tile += pairs) {
      const int r0 = (tile / p.mtiles * 2 + rank) * step, m0 = (tile % p.mtiles) * p.bn + rank * (p.bn / 2);
      for (int kb = first_kb; kb < first_kb + kblocks; kb++) {
        if (!dead) dead = !mbar_wait_bounded(empty + s, ph, abort_flag, p.status, TERN_DEVICE_TIMEOUT, kWaitNs);
        dead = __any_sync(0xffffffffu, dead);
        if (elect_one() && !dead) {
          mbar_arrive_expect_tx(full + s, bytes);
          if (warp == 0) {
            tma_load_2d(smem + s * X_BYTES, &tmap_x, full + s, kb * BK, m0);
          } else {
            uint8_t* dst = smem + OFF_P + s * P_BYTES;
            if (TRANS) {  // columns r0 .. r0 + 127 of rows kb * 64 ..
              const int px = LAYOUT == TERN_Q2_0_G128 ? r0 / 4 : LAYOUT == TERN_Q1_0_G128 ? r0 / 8 : (r0 / 5) & ~15;
              tma_load_2d(dst, &tmap_w, full + s, px, kb * BK);
            } else {
              const int px = LAYOUT == TERN_Q2_0_G128 ? kb * (BK / 4) : LAYOUT == TERN_Q1_0_G128 ? (kb * (BK / 8)) & ~15 : ((kb * BK) / 5) & ~15;
              tma_load_2d(dst, &tmap_w, full + s, px, r0);
              if (gated) tma_load_2d(dst + 64 * P_ROW, &tmap_w, full + s, px, (int)p.nout + r0);
            }
          }
        }
        __syncwarp();
        if (!dead) sent++;
        if (++s == STAGES) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    // copies in flight must land before the CTA's shared memory goes away. (Otherwise the decoders have waited
    // for them all.) A stage's barrier completes only if both warps sent theirs, so this wait is bounded too.
    if (dead && lane == 0) {
      const uint64_t t0 = globaltimer_ns();
      for (int i = sent > STAGES ? sent - STAGES : 0; i < sent; i++)
        while (!mbar_try_wait(full + i % STAGES, (uint32_t)(i / STAGES) & 1u) && globaltimer_ns() - t0 < kWaitNs / 4) {
        }
    }
  } else if (warp == 1 && rank == 0) {
    // ------------------------------------------------------------------ MMA issuer
    // The whole warp runs the loop, without leaving it early, and one elected lane issues: so the operands
    // stay in uniform registers. (Where the loop can be left on a wait's verdict, or is run by one lane, every
    // MMA takes about 100 cycles whatever its N; as it is, N / 2 + 11.)
    const uint32_t idesc = idesc_f16_f32(2 * BM, p.bn);
    uint32_t lt = 0, dph = 0;
    int s = 0, d = 0;
    bool dead = false, issued = false, ready = false;
    for (int tile = pair; tile < tiles; tile += pairs, lt++) {
      const uint32_t acc = lt & 1u;
      if (!dead) dead = !mbar_wait_bounded(tempty + acc, ((lt >> 1) & 1u) ^ 1u, abort_flag, p.status, TERN_DEVICE_TIMEOUT, kWaitNs);
      const uint32_t tmem_d = tmem + acc * p.bn;
      for (int kb = 0; kb < kblocks; kb++) {
        // both CTAs' decoders arrive after their A is stored, and after they saw their stage's copies land
        if (!dead && !ready) dead = !wait_pair(dfull + d, dph, abort_flag, p.status);
        dead = __any_sync(0xffffffffu, dead);
        tc_fence_after();
        const uint64_t bdesc = smem_desc_sw128(smem_u32(smem + s * X_BYTES));
        const uint32_t a = tmem + a_col + d * 32;
        if (elect_one() && !dead) {
#pragma unroll
          for (int kk = 0; kk < BK / 16; kk++) mma_f16_ts(tmem_d, a + 8 * kk, bdesc + 2 * kk, idesc, (kb | kk) != 0);
          commit_both(empty + s, first);
          commit_both(dempty + d, first);
          if (kb == kblocks - 1) commit_both(tfull + acc, first);
          issued = true;
        }
        __syncwarp();
        if (++s == STAGES) s = 0;
        if (++d == (int)a_stages) {
          d = 0;
          dph ^= 1u;
        }
        ready = try_wait_pair(dfull + d, dph);  // looked at while the MMAs run
      }
    }
    if (dead && issued) {  // (in the lane that issued) the MMAs must end before tensor memory is freed
      commit_own(drain);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(drain, 0) && globaltimer_ns() - t0 < kWaitNs / 4) {
      }
    }
    __syncwarp();
  } else if (warp >= 4 && warp < kFirstDecoder) {
    // ------------------------------------------------------------------ epilogue
    const int quad = warp & 3;
    const bool up = gated && lane >= 16;
    const int o = output_of<LAYOUT, TRANS>(quad, lane, gated);
    const uint64_t sum_ns = kWaitNs + (uint64_t)kblocks * kBlockNs;
    uint32_t lt = 0;
    for (int tile = pair; tile < tiles; tile += pairs, lt++) {
      const int64_t j = (int64_t)(tile / p.mtiles * 2 + rank) * step + o;  // output column
      const int64_t m0 = (int64_t)(tile % p.mtiles) * p.bn;
      const bool in = j < p.nout;
      const float bias = !TRANS && p.e.bias && in ? h2f(p.e.bias[j + (up ? p.nout : 0)]) : 0.f;
      const uint32_t acc = lt & 1u;
      // the warps leave together, and have all read the tile's flags before any of them is cleared
      const bool fine = mbar_wait_bounded(tfull + acc, (lt >> 1) & 1u, abort_flag, p.status, TERN_DEVICE_TIMEOUT, sum_ns);
      volatile uint8_t* flag = big + (lt % kBigTiles) * BM + (TRANS ? 0 : quad * 32 + lane);
      const uint32_t taddr = tmem + acc * p.bn + ((uint32_t)(quad * 32) << 16);
      const int cols = (int)(p.m - m0 < p.bn ? p.m - m0 : p.bn);  // rows of x in this tile
      bool again = LAYOUT != TERN_Q1_0_G128 && fine && *flag;
      const bool go = bar_all(kEpiBarrier, kEpi * 32, fine);
      if (p.splits > 1) {
        // 16 columns at a time belong to the pairs in turn: what the others have of them comes to their owner
        __syncwarp();
        cluster_sync();  // the stages' memory is no longer in use anywhere in the cluster
        if (go) {
          tc_fence_after();
          float* in = reinterpret_cast<float*>(smem) + quad * 32 + lane;
#pragma unroll 1
          for (int c = (warp >> 2) - 1; 16 * c < cols; c += kEpi / 4) {
            const int owner = c % p.splits;
            if (owner == slice) continue;
            uint32_t r[16];
            tmem_ld_32x32b_x16(taddr + 16 * c, r);
            const uint32_t to = in_cta(in + ((c / p.splits) * (p.splits - 1) + slice - (slice > owner)) * 16 * BM, 2 * owner + rank);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; i++) asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(to + i * BM * 4), "r"(r[i]) : "memory");
          }
          if (again)
            for (int i = 0; i < p.splits; i++)
              asm volatile("st.shared::cluster.u8 [%0], %1;" ::"r"(in_cta(const_cast<uint8_t*>(flag), 2 * i + rank)), "r"(1) : "memory");
        }
        __syncwarp();
        cluster_sync();
        again = LAYOUT != TERN_Q1_0_G128 && *flag;
      }
      if (!go) break;
      if (again && p.splits == 1) *flag = 0;
      if (again) *left_out = 1;
      if (LAYOUT != TERN_Q1_0_G128 && gated) again |= __shfl_xor_sync(0xffffffffu, again, 16);
      tc_fence_after();
#pragma unroll 1
      for (int c0 = 16 * (slice + p.splits * ((warp >> 2) - 1)); c0 < cols; c0 += 4 * kEpi * p.splits) {
        uint32_t r[16];
        tmem_ld_32x32b_x16(taddr + c0, r);
        const int lim = in && !again ? cols - c0 : 0;  // rows of x that this lane writes
        const int64_t t0 = m0 + c0;
        tmem_ld_wait();
        for (int i = 1; i < p.splits; i++) {
          const float* in = reinterpret_cast<const float*>(smem) + ((c0 / 16 / p.splits) * (p.splits - 1) + i - 1) * 16 * BM + quad * 32 + lane;
#pragma unroll
          for (int q = 0; q < 16; q++) r[q] = __float_as_uint(__uint_as_float(r[q]) + in[q * BM]);
        }
        write_outputs<LAYOUT, TRANS>(p, r, bias, t0, j, lim, up);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_first(tempty + acc, first);
    }
  } else if (warp >= kFirstDecoder) {
    // ------------------------------------------------------------------ decoders
    const int quad = warp & 3, set = (warp - kFirstDecoder) >> 2, st = threadIdx.x & 127;
    const uint32_t a_lane = tmem + a_col + ((uint32_t)(quad * 32) << 16);
    // stage and A slot of the set's next block, with the parities to wait for
    int s = set % STAGES, d = set % (int)a_stages, kb = set, flip = 0;
    uint32_t fph = 0, eph = 1;
    uint32_t lt = 0;
    bool ok = true;
    for (int tile = pair; tile < tiles && ok; tile += pairs, lt++) {
      const int r0 = (tile / p.mtiles * 2 + rank) * step;
      // forward: this lane's row of A is packed row `row`, at row `src` of the stage's codes
      const int src = gated ? (lane >> 4) * 64 + quad * 16 + (lane & 15) : quad * 32 + lane;
      const int64_t row = gated ? (int64_t)r0 + (src & 63) + (src >= 64 ? p.nout : 0) : (int64_t)r0 + src;
      const uint16_t* srow = p.scales + (row < p.n ? row : p.n - 1) * p.sstride;
      // forward: the lane's own row's scale; transposed: those of packed rows 2 lane and 2 lane + 1 of the
      // block as a pair
      auto fetch = [&](int kb) -> uint32_t {
        if (kb >= kblocks || (TRANS && r0 >= p.k)) return 0;  // (the second CTA's columns may lie past the matrix)
        kb += first_kb;
        if (!TRANS) return __ldg(srow + (kb * BK) / kGroup);
        const int64_t n = (int64_t)kb * BK + 2 * lane;
        const uint16_t* q = p.scales + n * p.sstride + r0 / kGroup;
        return (n < p.n ? (uint32_t)__ldg(q) : 0u) | (n + 1 < p.n ? (uint32_t)__ldg(q + p.sstride) << 16 : 0u);
      };
      uint32_t sc = fetch(kb);
      for (; kb < kblocks; kb += SETS) {
        const uint32_t cur = sc;
        const bool f0 = mbar_try_wait(full + s, fph), e0 = mbar_try_wait(dempty + d, eph);
        sc = fetch(kb + SETS);
        bool fine = f0 || mbar_wait_bounded(full + s, fph, abort_flag, p.status, TERN_DEVICE_TIMEOUT, kWaitNs);
        fine = fine && (e0 || mbar_wait_bounded(dempty + d, eph, abort_flag, p.status, TERN_DEVICE_TIMEOUT, kWaitNs));
        const uint8_t* P = smem + OFF_P + s * P_BYTES;
        if constexpr (!TRANS) {
          if (!__all_sync(0xffffffffu, fine)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if ((cur & 0x7fff) >= kBigScale && LAYOUT != TERN_Q1_0_G128) big[(lt % kBigTiles) * BM + quad * 32 + lane] = 1;
          const uint32_t s2 = cur | cur << 16;
          uint32_t o[32];
          if constexpr (LAYOUT == TERN_Q1_0_G128) {
            const uint2 w = *reinterpret_cast<const uint2*>(P + src * 16 + 8 * ((first_kb + kb) & 1));
            pairs_q1(w.x, s2, o);
            pairs_q1(w.y, s2, o + 16);
          } else {
            uint32_t w[4];
            if (LAYOUT == TERN_Q2_0_G128) {
              const uint4 u = *reinterpret_cast<const uint4*>(P + src * 16);
              w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
            } else {
              t3_words((first_kb + kb) % 5, P + src * 32, lut + lane, w);
            }
#pragma unroll
            for (int j = 0; j < 4; j++) {
              if (LAYOUT == TERN_Q2_0_G128) pairs_q2(w[j], s2, o + 8 * j);
              else pairs_mul(w[j], s2, o + 8 * j);
            }
          }
          tmem_st_32x32b_x32(a_lane + d * 32, o);
        } else {
          const uint32_t Q = smem_u32(smem + OFF_Q + (set * 2 + flip) * 64 * 32);
          if (LAYOUT == TERN_T3_5PB_G128) {
            // the set's four warps write the block in Q2's form for one another, into two buffers in turn: who
            // has passed this block's barrier has done with the buffer of the block before
            if (fine) {
              const int t0 = r0 + (st & 64);  // two warps take the first 64 columns of the 64 rows, two the others
              uint32_t w[4];
              t3_words((t0 / 64) % 5, P + (st & 63) * 48 + (((t0 / 5) & ~15) - ((r0 / 5) & ~15)), lut + lane, w);
              *reinterpret_cast<uint4*>(smem + OFF_Q + (set * 2 + flip) * 64 * 32 + (st & 63) * 32 + (st & 64 ? 16 : 0)) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            }
            fine = bar_all(kSetBarrier + set, 128, fine);  // the four warps leave together
          }
          if (!__all_sync(0xffffffffu, fine)) {
            ok = false;
            break;
          }
          if (LAYOUT != TERN_Q1_0_G128 && ((cur & 0x7fff) >= kBigScale || ((cur >> 16) & 0x7fff) >= kBigScale)) big[(lt % kBigTiles) * BM] = 1;
          tc_fence_after();
          // columns of 16 bits of the codes: Q2 eight fields (two column groups of 16 bytes), binary 16 bits
          const int group = LAYOUT == TERN_Q1_0_G128 ? 0 : quad >> 1;
          const uint32_t base = LAYOUT == TERN_T3_5PB_G128 ? Q : smem_u32(P);
          constexpr int pitch = LAYOUT == TERN_Q1_0_G128 ? 16 : 32;
          uint32_t R[8], sp[8];
#pragma unroll
          for (int h = 0; h < 2; h++) {
            uint32_t v[4];
            ldmatrix_x4_trans(base + (uint32_t)((32 * h + lane) * pitch + 16 * group), v);
#pragma unroll
            for (int q = 0; q < 4; q++) R[4 * h + q] = v[q];
          }
#pragma unroll
          for (int q = 0; q < 8; q++) sp[q] = __shfl_sync(0xffffffffu, cur, 4 * q + (lane & 3));
          const int f0 = LAYOUT == TERN_Q1_0_G128 ? 4 * quad : 4 * (quad & 1);  // the warp's first field
          const uint32_t up_mul = LAYOUT == TERN_Q1_0_G128 ? 1u << (12 - f0) : 1u << (8 - 2 * f0);
#pragma unroll
          for (int half = 0; half < 2; half++) {
            uint32_t o[16];
#pragma unroll
            for (int q = 0; q < 8; q++) {
#pragma unroll
              for (int b = 0; b < 2; b++) {
                const int f = 2 * half + b;  // field f0 + f of both halves of R[q]
                if (LAYOUT == TERN_Q1_0_G128) {
                  const uint32_t x = R[q] & (0x00010001u << f0 << f);  // bit f0 + f -> bit 15
                  o[2 * q + b] = (~(x * (up_mul << (3 - f))) & 0x80008000u) ^ sp[q];
                } else {
                  const uint32_t x = R[q] & (0x00030003u << (2 * f0) << (2 * f));  // field -> bits 14..15
                  o[2 * q + b] = hmul2(x * (up_mul << (6 - 2 * f)), sp[q]);
                }
              }
            }
            tmem_st_16x128b_x8(a_lane + ((uint32_t)(16 * half) << 16) + d * 32, o);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_first(dfull + d, first);
        flip ^= 1;
        s += SETS;
        if (s >= STAGES) {
          s -= STAGES;
          fph ^= 1u;
        }
        for (d += SETS; d >= (int)a_stages; d -= (int)a_stages) eph ^= 1u;
      }
      kb -= kblocks;
    }
  }

  if (p.splits > 1 && !(warp >= 4 && warp < kFirstDecoder)) {  // with the epilogue's warps: see there
    __syncwarp();
    cluster_sync();
    cluster_sync();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no CTA leaves while another may still arrive on its barriers or read its operands
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
  if (LAYOUT != TERN_Q1_0_G128 && *left_out && !*abort_flag) finish_big<LAYOUT, TRANS>(p, rank, slice, pair, pairs, tiles);
}

cudaLaunchConfig_t config(int clusters, int splits, cudaStream_t st, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(clusters * 2 * splits));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)(2 * splits);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

// Clusters of 2 x `splits` CTAs that run at the same time. The GPCs have different numbers of SMs, so this is less
// than SMs / CTAs (74, 33, 22 and 15 for 1 to 4). Asked for once: other devices of a machine may differ a little,
// which costs them time only.
template <int LAYOUT, bool TRANS>
int clusters_at_once(int splits) {
  struct Counts {
    int of[kMaxSplits + 1] = {};
    Counts() {
      const void* kern = reinterpret_cast<const void*>(&layer_gemm_kernel<LAYOUT, TRANS>);
      if (allow_smem(kern, SMEM_BYTES) != cudaSuccess) return;
      for (int i = 1; i <= kMaxSplits; i++) {
        cudaLaunchAttribute attr[2];
        cudaLaunchConfig_t cfg = config(1, i, nullptr, attr);
        cfg.numAttrs = 1;  // the cluster
        if (cudaOccupancyMaxActiveClusters(&of[i], kern, &cfg) != cudaSuccess) {
          of[i] = 0;
          (void)cudaGetLastError();
        }
      }
    }
  };
  static const Counts counts;
  return counts.of[splits];
}

// Rows of x per tile, the multiple of 32 up to kMaxBN, and pairs to a tile that make the waves of tiles cheapest.
// 64 terms of a tile cost four MMAs of bn / 2 + 11 cycles, and no less than what the warps of an SM need to decode
// them and to finish the tile before (about 480 cycles, measured at bn = 128 and 160). Two to four pairs share a
// tile's sum where all tiles run at once then; bringing the sums together costs about kJoin cycles. (4096 x 12288
// Q2 with 64 rows, 16 tiles: 58 us with one pair each, 30 with three.)
template <int LAYOUT, bool TRANS>
void pick_tiles(Params& p) {
  constexpr int kJoin = 2500;
  const int64_t blocks = (p.terms + BK - 1) / BK;
  double cost = -1;
  for (int bn = 32; bn <= kMaxBN; bn += 32) {
    if (bn > 32 && bn - 32 >= p.m) break;
    const int64_t tiles = ((int64_t)p.rtiles + 1) / 2 * ((p.m + bn - 1) / bn), waves = (tiles + sm_count() / 2 - 1) / (sm_count() / 2);
    for (int splits = 1; splits <= kMaxSplits; splits++) {
      if (splits > 1 && (tiles > (int64_t)clusters_at_once<LAYOUT, TRANS>(splits) || splits > blocks)) break;
      const double c = (double)waves * ((blocks + splits - 1) / splits) * std::max(2 * bn + 44, 480) + (splits > 1 ? kJoin : 0);
      if (cost < 0 || c < cost) {
        cost = c;
        p.bn = bn;
        p.splits = splits;
      }
    }
  }
}

template <int LAYOUT, bool TRANS>
cudaError_t launch_t(const tern_matrix& W, const uint16_t* x, int64_t xstride, Params& p, cudaStream_t st) {
  CUtensorMap mx, mw;
  p.x = x;
  p.xstride = xstride;
  pick_tiles<LAYOUT, TRANS>(p);
  const int64_t mt = (p.m + p.bn - 1) / p.bn;
  if (mt * p.rtiles > (int64_t)INT32_MAX) return cudaErrorInvalidValue;
  p.mtiles = (int)mt;
  if (!tmap_2d_new(&mx, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, x, (uint64_t)p.terms, (uint64_t)p.m, (uint64_t)xstride * 2, BK,
                   (uint32_t)p.bn / 2, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  // codes as bytes [n][row data]: reads past them give zero
  const uint64_t data = LAYOUT == TERN_Q2_0_G128 ? W.k / 4 : LAYOUT == TERN_Q1_0_G128 ? W.k / 8 : (W.k + 4) / 5;
  const uint32_t width = TRANS ? (LAYOUT == TERN_Q1_0_G128 ? 16 : LAYOUT == TERN_Q2_0_G128 ? 32 : 48)
                               : (LAYOUT == TERN_T3_5PB_G128 ? 32 : 16);
  if (!tmap_2d_new(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, W.codes, data, (uint64_t)W.n, (uint64_t)W.code_row_stride, width,
                   TRANS || p.e.gated ? 64 : BM, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  const void* kern = reinterpret_cast<const void*>(&layer_gemm_kernel<LAYOUT, TRANS>);
  const cudaError_t e = allow_smem(kern, SMEM_BYTES);
  if (e != cudaSuccess) return e;
  const int64_t tiles = ((int64_t)p.rtiles + 1) / 2 * p.mtiles;
  const int64_t clusters = p.splits > 1 ? tiles : std::min<int64_t>(tiles, sm_count() / 2);
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = config((int)clusters, p.splits, st, attr);
  return cudaLaunchKernelEx(&cfg, &layer_gemm_kernel<LAYOUT, TRANS>, mx, mw, (const Params)p);
}

template <bool TRANS>
cudaError_t dispatch(const tern_matrix& W, const uint16_t* x, int64_t xstride, Params& p, cudaStream_t st) {
  switch (W.layout) {
    case TERN_Q2_0_G128: return launch_t<TERN_Q2_0_G128, TRANS>(W, x, xstride, p, st);
    case TERN_T3_5PB_G128: return launch_t<TERN_T3_5PB_G128, TRANS>(W, x, xstride, p, st);
    default: return launch_t<TERN_Q1_0_G128, TRANS>(W, x, xstride, p, st);
  }
}

Params common(const tern_matrix& W, int64_t m, uint32_t* status) {
  Params p{};
  p.m = m;
  p.n = W.n;
  p.k = W.k;
  p.codes = static_cast<const uint8_t*>(W.codes);
  p.cstride = W.code_row_stride;
  p.scales = W.scales;
  p.sstride = W.scale_row_stride;
  p.status = status;
  return p;
}

}  // namespace

cudaError_t launch_layer_gemm(const tern_matrix& W, const uint16_t* x, int64_t m, uint16_t* y, const Epilogue& e,
                              uint32_t* status, cudaStream_t st) {
  Params p = common(W, m, status);
  p.nout = e.gated ? W.n / 2 : W.n;
  p.terms = (int)W.k;
  p.y = y;
  p.e = e;
  const int step = e.gated ? 64 : BM;
  p.rtiles = (int)((p.nout + step - 1) / step);
  return dispatch<false>(W, x, W.k, p, st);
}

cudaError_t launch_layer_gemm_t(const tern_matrix& W, const uint16_t* dz, int64_t dz_stride, int64_t m, uint16_t* dx,
                                uint32_t* status, cudaStream_t st) {
  Params p = common(W, m, status);
  p.nout = W.k;
  p.terms = (int)W.n;
  p.y = dx;
  p.rtiles = (int)(W.k / BM);
  return dispatch<true>(W, dz, dz_stride, p, st);
}

}  // namespace tern
