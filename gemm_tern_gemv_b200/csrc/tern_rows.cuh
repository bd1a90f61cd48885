// The few-rows product core of the layer operators: y[t][o] = sum_k w[o][k] x[t][k] for a handful of
// rows t of x, on mma.sync, weights read once from global memory straight into registers.
//
// A row of packed codes is cut into units of 32 bytes (128 weights of Q2_0_g128, 160 of base-3, 256 of
// binary); a warp takes 16 output rows and one unit at a time, each lane 8 bytes of rows g and g + 8
// (g = lane / 4). A unit lies in one 128-weight group (Q2) or two (slots 0 and 1 of base-3 and binary).
// Two forms of the product:
//   int8 (1-2 rows of x per tile of 8 MMA columns): activations become exact integers. Per unit, slot
//     and row of x, X = round(x 2^S) with S from the largest |x| of the slot, written as four balanced
//     base-256 digits; the columns are (row of x, or slot) x (digit), and the epilogue joins them. The
//     codes become u8 operands with one LOP3 per four weights and no shift to a common place:
//       Q2      (word ^ 0xAA..) & 0x03.. (or 0x0C..) is c = t + 2 (or 4 c): the sign bit flipped turns a
//               two's-complement field into an offset one; the high nibble is shifted down once. B holds
//               X (or X / 4), and the accumulators start at -2 sum of what B holds.
//       binary  word & (0x01.. << j) is 2^j b (t = 2 b - 1), B holds X / 2^j, start -sum X / 2.
//       base-3  quotients q_j = floor(v / 3^j): c_j = q_j - 3 q_{j+1}, so B holds X_j - 3 X_{j-1} and the
//               accumulators start at -sum X; q_{j+1} = (85 q_j + 80) >> 8 for every q_j <= 242.
//     All of that is exact in int32; an activation is off by at most 2^-27 of the largest of its slot.
//   fp16 (up to 8 rows per tile; 4 with two slots): x itself is the B operand, the codes become +-2 / 0 by
//     one multiply and one mask per two weights, fp32 accumulators restart at every unit.
// Either way each unit's sums take their group scale in fp32. The activation operands of a CTA are built
// once in shared memory, in the order the MMA lanes read them.
#pragma once

#include "sm100.cuh"
#include "tern_layer.cuh"
#include "tern_t3.cuh"

namespace tern {
namespace rows {

constexpr int kMaxWarps = 16, kThreads = kMaxWarps * 32;

template <int L> struct Lay;
template <> struct Lay<TERN_Q2_0_G128> { static constexpr int kUnitK = 128, kSlots = 1, kMma8 = 4, kMma16 = 8; };
template <> struct Lay<TERN_T3_5PB_G128> { static constexpr int kUnitK = 160, kSlots = 2, kMma8 = 5, kMma16 = 10; };
template <> struct Lay<TERN_Q1_0_G128> { static constexpr int kUnitK = 256, kSlots = 2, kMma8 = 8, kMma16 = 16; };

enum Mode { kInt8 = 0, kFp16 = 1 };

// Geometry of one column tile's activation operands: kEnt 16-byte entries per pair of MMAs, kPairs pairs.
template <int L, int MODE> struct Geo {
  using T = Lay<L>;
  static constexpr int kTok = (MODE == kInt8 ? 2 : 8) / T::kSlots;  // rows of x per column tile
  static constexpr int kMma = MODE == kInt8 ? T::kMma8 : T::kMma16;
  static constexpr int kPairs = (kMma + 1) / 2;
  // Q2: (row of x, digit) or row of x, by q; base-3: every lane; binary: only the lanes of a k's own slot
  static constexpr int kEnt = L == TERN_Q1_0_G128 ? 16 : 32;
  static constexpr int kTileBytes = kPairs * kEnt * 16 + (MODE == kInt8 ? 64 : 0);  // + starts and scales
};

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
// 16 bytes when pred is set, zeros otherwise.
__device__ __forceinline__ uint4 lds128_if(uint32_t a, bool pred) {
  uint4 v = make_uint4(0, 0, 0, 0);
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t@p ld.shared.v4.u32 {%0,%1,%2,%3}, [%5];\n\t}"
               : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
               : "r"((uint32_t)pred), "r"(a));
  return v;
}
__device__ __forceinline__ void mma_u8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
               : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 8 bytes of codes when pred is set (v keeps its value otherwise). Weights are read once: no place in L1.
__device__ __forceinline__ void ldg_codes(uint2& v, const uint8_t* p, bool pred) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %3, 0;\n\t@p ld.global.nc.L1::no_allocate.L2::256B.v2.u32 {%0,%1}, [%2];\n\t}"
      : "+r"(v.x), "+r"(v.y)
      : "l"(p), "r"((uint32_t)pred));
}

// Balanced base-256 digits of X (|X| <= 2^30): byte p of the result is d_p in [-128, 127], X = sum d_p 2^(8p).
__device__ __forceinline__ uint32_t digits(int X) { return ((uint32_t)X + 0x00808080u) ^ 0x00808080u; }
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
// Smallest E with |x| < 2^E for a finite positive fp32 value given by its bits (subnormals count as 2^-126).
__device__ __forceinline__ int exponent(uint32_t abs_bits) { return (int)(abs_bits >> 23) - 126; }

// Rows of x as the core reads them: fp16 rows, or fp32 rows of expert activations. load() gives NE
// consecutive activations as floats, load16() N (a multiple of 8) as fp16 bits; both are zero from K on.
// K is a multiple of 8 and so are load16's k0 and, unless NE is 5, load's k0 of NE; rows are 16-byte aligned.
struct HalfRows {
  const uint16_t* base;
  int64_t stride;
  const int* index;  // row t of the product is row index[t] of base (null: t)
  __device__ __forceinline__ const uint16_t* row(int t) const { return base + (int64_t)(index ? index[t] : t) * stride; }
  __device__ __forceinline__ float at(int t, int k) const { return h2f(row(t)[k]); }
  template <int NE> __device__ __forceinline__ void load(int t, int k0, int K, float (&v)[NE]) const {
    const uint16_t* r = row(t);
    if constexpr (NE == 4) {
      if (k0 < K) {
        const uint2 u = *reinterpret_cast<const uint2*>(r + k0);
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x)), b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
        v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
      }
    } else {
#pragma unroll
      for (int e = 0; e < NE; e++)
        if (k0 + e < K) v[e] = h2f(r[k0 + e]);
    }
  }
  template <int N> __device__ __forceinline__ void load16(int t, int k0, int K, uint32_t (&v)[N / 2]) const {
    const uint16_t* r = row(t);
#pragma unroll
    for (int c = 0; c < N / 8; c++) {
      uint4 u = make_uint4(0, 0, 0, 0);
      if (k0 + 8 * c < K) u = *reinterpret_cast<const uint4*>(r + k0 + 8 * c);
      v[4 * c] = u.x; v[4 * c + 1] = u.y; v[4 * c + 2] = u.z; v[4 * c + 3] = u.w;
    }
  }
};
struct FloatRows {
  const float* base;
  int64_t stride;
  const int* index;
  const float* mul;  // load16 gives v * mul[t]: a power of two that brings the row into fp16's range
  __device__ __forceinline__ const float* row(int t) const { return base + (int64_t)index[t] * stride; }
  __device__ __forceinline__ float at(int t, int k) const { return row(t)[k]; }
  template <int NE> __device__ __forceinline__ void load(int t, int k0, int K, float (&v)[NE]) const {
    const float* r = row(t);
    if constexpr (NE == 4) {
      if (k0 < K) {
        const float4 u = *reinterpret_cast<const float4*>(r + k0);
        v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < NE; e++)
        if (k0 + e < K) v[e] = r[k0 + e];
    }
  }
  template <int N> __device__ __forceinline__ void load16(int t, int k0, int K, uint32_t (&v)[N / 2]) const {
    const float* r = row(t);
    const float m = mul[t];
#pragma unroll
    for (int c = 0; c < N / 4; c++) {
      float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k0 + 4 * c < K) u = *reinterpret_cast<const float4*>(r + k0 + 4 * c);
      const __half2 a = __floats2half2_rn(u.x * m, u.y * m), b = __floats2half2_rn(u.z * m, u.w * m);
      v[2 * c] = *reinterpret_cast<const uint32_t*>(&a);
      v[2 * c + 1] = *reinterpret_cast<const uint32_t*>(&b);
    }
  }
};

// ---- building the activation operands -----------------------------------------------------------------
// int8 form of one (unit u, row t of x), the tok-th of its column tile. scr: 32 x 8 words of this warp;
// frag: the column tile's entries, then one 16-byte record for each q: accumulator starts of columns 2 q
// and 2 q + 1 (binary: their sum to be added to twice the accumulators) and the scale 2^-S (x 2^16 for
// digits 2 and 3). Non-finite activations count as zero here (the caller adds them apart) and set *odd.
template <int L, class X>
__device__ __forceinline__ void build_int8(const X& xs, int t, int tok, int u, int K, uint32_t* scr, uint4* frag, int* odd) {
  using T = Lay<L>;
  using G = Geo<L, kInt8>;
  const int lane = threadIdx.x & 31;
  constexpr int NE = T::kUnitK / 32;  // activations of this lane: the weights of byte `lane` of the unit
  constexpr bool two_in_a_byte = L == TERN_T3_5PB_G128;  // a byte may hold weights of both slots
  float xv[NE];
#pragma unroll
  for (int e = 0; e < NE; e++) xv[e] = 0.f;
  xs.template load<NE>(t, u * T::kUnitK + lane * NE, K, xv);
  // first weight of the unit that belongs to slot 1
  const int edge = T::kSlots == 1 ? T::kUnitK : (L == TERN_Q1_0_G128 ? 128 : 128 - (u * 160) % 128);
  uint32_t mx[2] = {0, 0};
  bool bad = false;
#pragma unroll
  for (int e = 0; e < NE; e++) {
    uint32_t b = __float_as_uint(xv[e]) & 0x7fffffffu;
    if (b >= 0x7f800000u) {
      bad = true;
      b = 0;
      xv[e] = 0.f;
    }
    const int s = (lane * NE + e < edge) ? 0 : 1;
    mx[0] = max(mx[0], s ? 0u : b);
    mx[1] = max(mx[1], s ? b : 0u);
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) *odd = 1;
  constexpr int kTop = L == TERN_T3_5PB_G128 ? 28 : 30;  // base-3 operands add up to four activations
  int S[2] = {0, 0};
#pragma unroll
  for (int s = 0; s < T::kSlots; s++) {
    mx[s] = __reduce_max_sync(0xffffffffu, mx[s]);
    S[s] = mx[s] ? min(100, kTop - exponent(mx[s])) : 0;
  }
  const int w = lane >> 2, pl = lane & 3;  // the word and the digit that this lane gathers
  const uint32_t sel = (uint32_t)pl | ((uint32_t)(pl + 4) << 4);
  auto plane = [&](const uint32_t* d4) {  // digit pl of four consecutive scratch words
    const uint4 d = *reinterpret_cast<const uint4*>(d4);
    return __byte_perm(__byte_perm(d.x, d.y, sel), __byte_perm(d.z, d.w, sel), 0x5410);
  };
#pragma unroll
  for (int s = 0; s < (two_in_a_byte ? 2 : 1); s++) {
    const int Ss = L == TERN_Q1_0_G128 ? S[lane >> 4] : S[s];
    if constexpr (two_in_a_byte) {
      int xi[5], sum = 0;
#pragma unroll
      for (int e = 0; e < 5; e++) {
        xi[e] = ((lane * 5 + e < edge) == (s == 0)) ? __float2int_rn(xv[e] * exp2i(Ss)) : 0;
        sum += xi[e];
      }
#pragma unroll
      for (int e = 0; e < 5; e++) scr[e * 32 + lane] = digits(xi[e] - (e ? 3 * xi[e - 1] : 0));
      scr[5 * 32 + lane] = digits(sum);  // |sum| <= 5 2^28: its digits fit too
    } else {
#pragma unroll
      for (int e = 0; e < NE; e++) {
        const int sh = L == TERN_Q2_0_G128 ? 2 * (e & 1) : (e & 3);  // the code operand is 2^sh times c (or b)
        scr[e * 32 + lane] = digits(__float2int_rn(xv[e] * exp2i(Ss - sh)));
      }
    }
    __syncwarp();
    const int sl = L == TERN_Q1_0_G128 ? 0 : (two_in_a_byte ? s : tok);
    const int ent = sl * 16 + (w >> 1) * 4 + pl;
    int sum = 0;
#pragma unroll
    for (int e = 0; e < NE; e++) {
      const uint32_t r = plane(scr + e * 32 + 4 * w);
      reinterpret_cast<uint32_t*>(frag + (e >> 1) * G::kEnt + ent)[(e & 1) * 2 + (w & 1)] = r;
      if (L == TERN_Q2_0_G128) sum = __dp4a((int)r, (e & 1) ? 0x04040404 : 0x01010101, sum);
      if (L == TERN_Q1_0_G128) sum = __dp4a((int)r, 0x01010101 << (e & 3), sum);
    }
    if (two_in_a_byte) sum = __dp4a((int)plane(scr + 5 * 32 + 4 * w), 0x01010101, 0);
    // over the words of the slot: all eight, or for binary the four of each half
    sum += __shfl_xor_sync(0xffffffffu, sum, 4);
    sum += __shfl_xor_sync(0xffffffffu, sum, 8);
    if (L != TERN_Q1_0_G128) sum += __shfl_xor_sync(0xffffffffu, sum, 16);
    const int start = L == TERN_Q2_0_G128 ? -2 * sum : -sum;
    const int next = __shfl_down_sync(0xffffffffu, start, 1);
    const int half = L == TERN_Q1_0_G128 ? lane >> 4 : (two_in_a_byte ? s : tok);
    if ((lane & (L == TERN_Q1_0_G128 ? 12 : 28)) == 0 && (pl & 1) == 0)
      frag[G::kPairs * G::kEnt + half * 2 + (pl >> 1)] =
          make_uint4((uint32_t)(L == TERN_Q1_0_G128 ? start + 256 * next : start), (uint32_t)next,
                     __float_as_uint(exp2i((pl ? 16 : 0) - Ss)), 0u);
    __syncwarp();
  }
}

// fp16 form of one (unit, column tile): lane (g, q) writes the operand words of column g.
template <int L, class X>
__device__ __forceinline__ void build_fp16(const X& xs, int t0, int tokens, int u, int K, uint4* frag) {
  using G = Geo<L, kFp16>;
  const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int tok = L == TERN_Q2_0_G128 ? g : (g & 3);
  if (t0 + tok >= tokens) return;
  if constexpr (L == TERN_T3_5PB_G128) {
    uint32_t v[20];
    const int k0 = 160 * u + 40 * q;
    xs.template load16<40>(t0 + tok, k0, K, v);
    const int edge = ((160 * u) / kGroup + 1) * kGroup - k0;  // first of the lane's weights in slot 1
    auto h = [&](int e) -> uint32_t {
      return ((e < edge) == (g < 4)) ? ((e & 1) ? v[e >> 1] >> 16 : v[e >> 1] & 0xffffu) : 0u;
    };
    // word b of the lane, register r = 5 h + i: digit 4 - i of bytes h and h + 2
    auto reg = [&](int b, int r) { const int e = 20 * b + 5 * (r / 5) + 4 - r % 5; return h(e) | (h(e + 10) << 16); };
#pragma unroll
    for (int p = 0; p < 5; p++) frag[p * 32 + lane] = make_uint4(reg(0, 2 * p), reg(1, 2 * p), reg(0, 2 * p + 1), reg(1, 2 * p + 1));
  } else if constexpr (L == TERN_Q2_0_G128) {
    uint32_t v[16];
    xs.template load16<32>(t0 + tok, 128 * u + 32 * q, K, v);
#pragma unroll
    for (int p = 0; p < 4; p++)  // register i: fields i and i + 8 of a word
      frag[p * 32 + lane] = make_uint4(__byte_perm(v[p], v[p + 4], 0x5410), __byte_perm(v[8 + p], v[12 + p], 0x5410),
                                       __byte_perm(v[p], v[p + 4], 0x7632), __byte_perm(v[8 + p], v[12 + p], 0x7632));
  } else {
    if ((g >> 2) != (q >> 1)) return;
    uint32_t v[32];
    xs.template load16<64>(t0 + tok, 256 * u + 64 * q, K, v);
#pragma unroll
    for (int p = 0; p < 8; p++)  // register i: bits i and i + 16 of a word
      frag[p * G::kEnt + q * 4 + tok] =
          make_uint4(__byte_perm(v[p], v[p + 8], 0x5410), __byte_perm(v[16 + p], v[24 + p], 0x5410),
                     __byte_perm(v[p], v[p + 8], 0x7632), __byte_perm(v[16 + p], v[24 + p], 0x7632));
  }
}

// ---- the product --------------------------------------------------------------------------------------
struct Mat {
  const uint8_t* codes;
  const uint16_t* scales;
  int64_t cstride, sstride;
  int K, row_bytes, groups, units;
};
// Rows of a 16-row tile: tile t holds, as rows 0-7, first + min(t step + r, limit - 1) and, as rows 8-15,
// second + min(t step + ahead + r, limit - 1): 16 rows in turn, or 8 gate rows and their 8 up rows.
struct Map {
  int64_t first, second;
  int limit, step, ahead;
};
// How a CTA cuts its work: warps = wk (along K) x tg (tiles); `pass` blocks of K and `batch` tiles at a time.
struct Split {
  int wk, tg, pass, batch;
};

// A block is four units, 128 bytes of a row: what a warp requests and works off at a time. Its addresses
// are one base and constant offsets, and a lane's scales of a row come in one or two loads.
constexpr int kBlk = 4;

// Code operands a0 .. a3 of each int8 MMA from 8 bytes of rows g (a) and g + 8 (b). k85, kc80: 85 and 80 in
// both halves, opaque to the compiler so that the base-3 steps stay multiplications.
template <int L>
__device__ __forceinline__ void operands8(uint2 a, uint2 b, uint32_t k85, uint32_t kc80, uint32_t (&F)[4][Geo<L, kInt8>::kPairs * 2]) {
  const uint32_t w[4] = {a.x, b.x, a.y, b.y};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    if constexpr (L == TERN_Q2_0_G128) {
      const uint32_t z = w[i] >> 4;
      F[i][0] = (w[i] ^ 0xAAAAAAAAu) & 0x03030303u;
      F[i][1] = (w[i] ^ 0xAAAAAAAAu) & 0x0C0C0C0Cu;
      F[i][2] = (z ^ 0xAAAAAAAAu) & 0x03030303u;
      F[i][3] = (z ^ 0xAAAAAAAAu) & 0x0C0C0C0Cu;
    } else if constexpr (L == TERN_Q1_0_G128) {
      const uint32_t z = w[i] >> 4;
#pragma unroll
      for (int j = 0; j < 4; j++) {
        F[i][j] = w[i] & (0x01010101u << j);
        F[i][4 + j] = z & (0x01010101u << j);
      }
    } else {
      uint32_t E = w[i] & 0x00FF00FFu, O = __byte_perm(w[i], 0u, 0x4341);
      F[i][0] = w[i];
#pragma unroll
      for (int j = 1; j <= 4; j++) {
        E = E * k85 + kc80;
        O = O * k85 + kc80;
        F[i][j] = __byte_perm(E, O, 0x7351);
        if (j < 4) {
          E = __byte_perm(E, 0u, 0x4341);
          O = __byte_perm(O, 0u, 0x4341);
        }
      }
      F[i][5] = 0;
    }
  }
}

template <int L, int MODE, int NT>
struct Product {
  using T = Lay<L>;
  using G = Geo<L, MODE>;
  static constexpr int kRows = NT * G::kTok;             // rows of x
  static constexpr int kDepth = 2;                       // blocks requested ahead by a warp
  static constexpr int kUnitBytes = NT * G::kTileBytes;  // activation operands of one unit
  static constexpr int kAcc = MODE == kInt8 ? 2 : 4;
  static constexpr int kTileRows = 16, kMode = MODE;
  static bool plan(int tiles, int units, size_t room, Split* out);

  // shared memory: operands [pass], partial sums [batch][wk][16][kRows], scratch [warps][256 words], flags
  static __host__ __device__ size_t part_bytes(const Split& s) { return (size_t)s.batch * s.wk * 16 * kRows * 4; }
  static __host__ __device__ size_t smem_bytes(const Split& s) {
    return (size_t)s.pass * kBlk * kUnitBytes + part_bytes(s) + (MODE == kInt8 ? kMaxWarps * 1024 : 0) + 64;
  }

  uint2 wa[kDepth][kBlk], wb[kDepth][kBlk];
  // group scales of the block's units: Q2 four groups; binary eight (the lane's slot picks); base-3 the
  // lane's four
  uint4 sa[kDepth], sb[kDepth];
  // load cursor: codes (at the lane's bytes) and scales of the lane's two rows, tile, block
  const uint8_t *pa, *pb;
  const uint16_t *ga, *gb;
  int lt, lb;
  uint32_t k85, kc80;  // opaque to the compiler, so that the base-3 steps stay multiplications

  __device__ __forceinline__ void set_rows(const Mat& M, const Map& R) {
    const int g = (threadIdx.x & 31) >> 2, q = threadIdx.x & 3;
    const int64_t o = (int64_t)lt * R.step + g;
    const int64_t a = R.first + min(o, (int64_t)R.limit - 1), b = R.second + min(o + R.ahead, (int64_t)R.limit - 1);
    pa = M.codes + a * M.cstride + 8 * q;
    pb = M.codes + b * M.cstride + 8 * q;
    ga = M.scales + a * M.sstride;
    gb = M.scales + b * M.sstride;
  }
  __device__ __forceinline__ void request_scales(const Mat& M, int d) {
    if constexpr (L == TERN_T3_5PB_G128) {  // a block of 640 weights starts at group 5 lb; unit j meets groups j, j + 1 of it
      const int g0 = 5 * lb + ((threadIdx.x & 3) >> 1);
      uint16_t u[4], v[4];
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const int g = min(g0 + j, M.groups - 1);
        u[j] = __ldg(ga + g);
        v[j] = __ldg(gb + g);
      }
      sa[d] = make_uint4(u[0], u[1], u[2], u[3]);
      sb[d] = make_uint4(v[0], v[1], v[2], v[3]);
    } else {  // rows of scales are 16-byte aligned and a multiple of 16 bytes
      constexpr int n = L == TERN_Q2_0_G128 ? 4 : 8;  // groups of a block
      if constexpr (n == 4) {
        const uint2 u = __ldg(reinterpret_cast<const uint2*>(ga + 4 * lb)), v = __ldg(reinterpret_cast<const uint2*>(gb + 4 * lb));
        sa[d] = make_uint4(u.x, u.y, 0, 0);
        sb[d] = make_uint4(v.x, v.y, 0, 0);
      } else {
        sa[d] = __ldg(reinterpret_cast<const uint4*>(ga + 8 * lb));
        sb[d] = __ldg(reinterpret_cast<const uint4*>(gb + 8 * lb));
      }
      const int have = M.groups - n * lb;
      if (have < n) {  // what lies past the row's last group counts as 0
        auto keep = [&](uint32_t w, int i) { return 2 * i >= have ? 0u : (2 * i + 1 >= have ? w & 0xffffu : w); };
        sa[d] = make_uint4(keep(sa[d].x, 0), keep(sa[d].y, 1), keep(sa[d].z, 2), keep(sa[d].w, 3));
        sb[d] = make_uint4(keep(sb[d].x, 0), keep(sb[d].y, 1), keep(sb[d].z, 2), keep(sb[d].w, 3));
      }
    }
  }
  // Unit j of the block at the cursor. The row may end inside the block (a base-3 or binary row inside a
  // unit): what lies past it is not read, its operands are zero and any codes will do.
  __device__ __forceinline__ void request_unit(const Mat& M, int d, int j, bool on) {
    const int off = lb * 128 + j * 32;
    const bool in = on && off + 8 * (int)(threadIdx.x & 3) < M.row_bytes;
    ldg_codes(wa[d][j], pa + off, in);
    ldg_codes(wb[d][j], pb + off, in);
  }
  __device__ __forceinline__ float scale(const uint4& s, int j) const {
    if constexpr (L == TERN_Q2_0_G128) {
      const uint32_t w = j < 2 ? s.x : s.y;
      return h2f((uint16_t)((j & 1) ? w >> 16 : w & 0xffffu));
    } else if constexpr (L == TERN_Q1_0_G128) {
      const uint32_t w = j == 0 ? s.x : (j == 1 ? s.y : (j == 2 ? s.z : s.w));
      return h2f((uint16_t)((threadIdx.x & 2) ? w >> 16 : w & 0xffffu));
    } else {
      return h2f((uint16_t)(j == 0 ? s.x : (j == 1 ? s.y : (j == 2 ? s.z : s.w))));
    }
  }

  // One unit: codes and scales of rows g (a) and g + 8 (b) times the operands at base + ent[.] (this lane's
  // entries; starts and scales at hd) into acc.
  __device__ __forceinline__ void unit(uint2 a, uint2 b, float s0, float s1, uint32_t base, uint32_t hd, const uint32_t (&ent)[NT],
                                       float (&acc)[NT][kAcc]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    if constexpr (MODE == kInt8) {
      int c[NT][4];
      float sc[NT];
      int add[NT];
#pragma unroll
      for (int n = 0; n < NT; n++) {
        const uint4 r = lds128(hd + (uint32_t)(n * G::kTileBytes));
        if (L == TERN_Q1_0_G128) {
          add[n] = (int)r.x;
          c[n][0] = c[n][1] = c[n][2] = c[n][3] = 0;
        } else {
          c[n][0] = c[n][2] = (int)r.x;
          c[n][1] = c[n][3] = (int)r.y;
        }
        sc[n] = __uint_as_float(r.z);
      }
      uint32_t F[4][G::kPairs * 2];
      operands8<L>(a, b, k85, kc80, F);
#pragma unroll
      for (int p = 0; p < G::kPairs; p++)
#pragma unroll
        for (int n = 0; n < NT; n++) {
          // binary: the columns of the other slot are zero
          const uint32_t at = base + ent[n] + (uint32_t)(n * G::kTileBytes + p * G::kEnt * 16);
          const uint4 f = L == TERN_Q1_0_G128 ? lds128_if(at, (g >> 2) == (q >> 1)) : lds128(at);
          mma_u8(c[n], F[0][2 * p], F[1][2 * p], F[2][2 * p], F[3][2 * p], f.x, f.y);
          if (2 * p + 1 < G::kMma) mma_u8(c[n], F[0][2 * p + 1], F[1][2 * p + 1], F[2][2 * p + 1], F[3][2 * p + 1], f.z, f.w);
        }
#pragma unroll
      for (int n = 0; n < NT; n++) {
        int v0 = c[n][0] + 256 * c[n][1], v1 = c[n][2] + 256 * c[n][3];
        if (L == TERN_Q1_0_G128) {  // t = 2 b - 1
          v0 = 2 * v0 + add[n];
          v1 = 2 * v1 + add[n];
        }
        acc[n][0] = fmaf(s0 * sc[n], (float)v0, acc[n][0]);
        acc[n][1] = fmaf(s1 * sc[n], (float)v1, acc[n][1]);
      }
    } else {
      const uint32_t w[4] = {a.x, b.x, a.y, b.y};
      float c[NT][4];
#pragma unroll
      for (int n = 0; n < NT; n++) c[n][0] = c[n][1] = c[n][2] = c[n][3] = 0.f;
      uint32_t O[4][L == TERN_T3_5PB_G128 ? 10 : 1];
      if constexpr (L == TERN_T3_5PB_G128) {
#pragma unroll
        for (int i = 0; i < 4; i++) dec_t3_word(w[i], 0x00820082u + 0xC000C000u, O[i]);
      }
      auto A = [&](int i, int r) -> uint32_t {  // register r of word i: fp16 2 t
        if constexpr (L == TERN_Q2_0_G128) return (r < 7 ? w[i] << (14 - 2 * r) : w[i]) & 0xC000C000u;
        else if constexpr (L == TERN_Q1_0_G128) return ((w[i] << (15 - r)) & 0x80008000u) ^ 0xC000C000u;
        else return O[i][r];
      };
#pragma unroll
      for (int p = 0; p < G::kPairs; p++) {
        const uint32_t a00 = A(0, 2 * p), a01 = A(1, 2 * p), a02 = A(2, 2 * p), a03 = A(3, 2 * p);
        const uint32_t a10 = A(0, 2 * p + 1), a11 = A(1, 2 * p + 1), a12 = A(2, 2 * p + 1), a13 = A(3, 2 * p + 1);
#pragma unroll
        for (int n = 0; n < NT; n++) {
          const uint32_t at = base + ent[n] + (uint32_t)(n * G::kTileBytes + p * G::kEnt * 16);
          const uint4 f = L == TERN_Q1_0_G128 ? lds128_if(at, (g >> 2) == (q >> 1)) : lds128(at);
          mma_f16(c[n], a00, a01, a02, a03, f.x, f.y);
          mma_f16(c[n], a10, a11, a12, a13, f.z, f.w);
        }
      }
#pragma unroll
      for (int n = 0; n < NT; n++) {
        acc[n][0] = fmaf(s0, c[n][0], acc[n][0]);
        acc[n][1] = fmaf(s0, c[n][1], acc[n][1]);
        acc[n][2] = fmaf(s1, c[n][2], acc[n][2]);
        acc[n][3] = fmaf(s1, c[n][3], acc[n][3]);
      }
    }
  }

  // Partial sums of a finished tile: the lanes that share rows are summed, then one float per (row, row
  // of x) goes to `out` ([16][kRows]); `more` adds to what an earlier pass over K left there.
  __device__ __forceinline__ void store_part(float* out, bool more, float (&acc)[NT][kAcc]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; n++) {
      if constexpr (MODE == kInt8) {
        float v0 = acc[n][0], v1 = acc[n][1];
        v0 += __shfl_xor_sync(0xffffffffu, v0, 1);
        v1 += __shfl_xor_sync(0xffffffffu, v1, 1);
        if (T::kSlots == 2) {
          v0 += __shfl_xor_sync(0xffffffffu, v0, 2);
          v1 += __shfl_xor_sync(0xffffffffu, v1, 2);
        }
        if (T::kSlots == 2 ? q == 0 : (q & 1) == 0) {
          const int t = n * G::kTok + (T::kSlots == 2 ? 0 : q >> 1);
          float *x = out + g * kRows + t, *y = out + (g + 8) * kRows + t;
          *x = more ? *x + v0 : v0;
          *y = more ? *y + v1 : v1;
        }
        acc[n][0] = acc[n][1] = 0.f;
      } else {
#pragma unroll
        for (int i = 0; i < 4; i++) {
          float v = acc[n][i] * 0.5f;  // the codes' operand is 2 t
          if (T::kSlots == 2) v += __shfl_xor_sync(0xffffffffu, v, 2);
          if (T::kSlots == 1 || q < 2) {
            float* x = out + (g + 8 * (i >> 1)) * kRows + n * G::kTok + 2 * q + (i & 1);
            *x = more ? *x + v : v;
          }
          acc[n][i] = 0.f;
        }
      }
    }
  }

  // Tiles [t0, t1) of M's rows by R times rows [0, tokens) of xs. For every output row and row of x
  // fin(tile, r, t, z, -) gets the sum of tile row r, or with R.ahead == 0 (gate and up rows)
  // fin(tile, r, t, z_gate, z_up) for r < 8. All threads of the CTA call this together; `first` is called
  // once the first weights are requested, before xs is read.
  template <class X, class First, class Fin>
  __device__ __forceinline__ void run(uint8_t* smem, const Split& s, const Mat& M, const Map& R, int t0, int t1, const X& xs,
                                      int tokens, First first, Fin fin) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, q = lane & 3;
    uint8_t* frag = smem;
    float* part = reinterpret_cast<float*>(smem + (size_t)s.pass * kBlk * kUnitBytes);
    uint32_t* scr = reinterpret_cast<uint32_t*>(smem + (size_t)s.pass * kBlk * kUnitBytes + part_bytes(s)) + warp * 256;
    int* odd = reinterpret_cast<int*>(smem + smem_bytes(s) - 64);  // rows of x with a non-finite activation
    const int kg = warp % s.wk, tg = warp / s.wk;
    const int blocks = (M.units + kBlk - 1) / kBlk;
    k85 = 85u;
    kc80 = 0x00500050u;
    asm volatile("" : "+r"(k85), "+r"(kc80));
    // This lane's entry of a column tile's operands: column g, k by q. Columns of absent rows of x read
    // those of a present one (their sums are never looked at).
    uint32_t ent[NT];
#pragma unroll
    for (int n = 0; n < NT; n++) {
      const int here = tokens - n * G::kTok;  // rows of x in this column tile (0 or less: none)
      int e;
      if (MODE == kInt8) {
        e = q * 4 + (g & 3) + (L == TERN_T3_5PB_G128 || (L == TERN_Q2_0_G128 && here > 1) ? (g >> 2) * 16 : 0);
      } else if (L == TERN_Q2_0_G128) {
        e = (g < here ? g : 0) * 4 + q;
      } else {
        const int tok = (g & 3) < here ? g & 3 : 0;
        e = L == TERN_Q1_0_G128 ? q * 4 + tok : ((g & 4) + tok) * 4 + q;
      }
      ent[n] = (uint32_t)e * 16u;
    }
    const uint32_t base0 = sm100::smem_u32(frag);
    const uint32_t hd0 = base0 + (uint32_t)(G::kPairs * G::kEnt * 16 + q * 16);
    const int64_t step_c = (int64_t)R.step * M.cstride, step_s = (int64_t)R.step * M.sstride;
    const int whole = R.limit / R.step;  // tiles that are not cut short
    bool fresh = true;
    if (tid < 16) odd[tid] = 0;
    for (int b0 = t0; b0 < t1; b0 += s.batch) {
      const int b1 = min(t1, b0 + s.batch);
      int ta = b0, tb = b0;
      if (tg < s.tg) {
        ta = b0 + (b1 - b0) * tg / s.tg;
        tb = b0 + (b1 - b0) * (tg + 1) / s.tg;
      }
      for (int p0 = 0; p0 < blocks; p0 += s.pass) {
        const int p1 = min(blocks, p0 + s.pass);
        const int lo = p0 + (p1 - p0) * kg / s.wk, hi = p0 + (p1 - p0) * (kg + 1) / s.wk;  // the warp's blocks
        int left = (tb - ta) * (hi - lo);  // blocks still to be requested
        lt = ta;
        lb = lo;
        const int total = left;
        if (left > 0) set_rows(M, R);
        auto advance = [&]() {
          --left;
          if (++lb == hi) {
            lb = lo;
            ++lt;
            if (lt >= whole) {
              set_rows(M, R);  // the last tile may be cut short
            } else {
              pa += step_c; pb += step_c;
              ga += step_s; gb += step_s;
            }
          }
        };
#pragma unroll
        for (int d = 0; d < kDepth; d++)
          if (left > 0) {
            request_scales(M, d);
#pragma unroll
            for (int j = 0; j < kBlk; j++) {
              wa[d][j] = wb[d][j] = make_uint2(0, 0);
              request_unit(M, d, j, true);
            }
            advance();
          }
        if (fresh) first();
        if (fresh || s.pass < blocks) {
          __syncthreads();  // the operands of the pass before are no longer read (and the flags are clear)
          const int u0 = p0 * kBlk, nu = min(M.units, p1 * kBlk) - u0;
          for (uint32_t i = (uint32_t)nu * kUnitBytes + tid * 16; i < (uint32_t)(p1 * kBlk - u0) * kUnitBytes; i += kThreads * 16)
            *reinterpret_cast<uint4*>(frag + i) = make_uint4(0, 0, 0, 0);  // units past the row's end
          if constexpr (MODE == kInt8) {
            for (int i = warp; i < nu * tokens; i += kMaxWarps) {
              const int u = i / tokens, t = i % tokens;
              build_int8<L>(xs, t, t % G::kTok, u0 + u, M.K, scr,
                            reinterpret_cast<uint4*>(frag + (size_t)u * kUnitBytes + (t / G::kTok) * G::kTileBytes), odd + t);
            }
          } else {
            for (int i = warp; i < nu * NT; i += kMaxWarps) {
              const int u = i / NT, n = i % NT;
              build_fp16<L>(xs, n * G::kTok, tokens, u0 + u, M.K,
                            reinterpret_cast<uint4*>(frag + (size_t)u * kUnitBytes + n * G::kTileBytes));
            }
          }
          __syncthreads();
        }
        fresh = false;
        if (total > 0) {
          float acc[NT][kAcc] = {};
          int cb = lo;
          float* out = part + (size_t)((ta - b0) * s.wk + kg) * 16 * kRows;
          for (int i = total; i > 0;) {
#pragma unroll
            for (int d = 0; d < kDepth; d++) {
              if (i <= 0) break;
              const uint4 s0 = sa[d], s1 = sb[d];
              const bool ml = left > 0;
              if (ml) request_scales(M, d);
              const uint32_t fo = (uint32_t)((cb - p0) * kBlk * kUnitBytes);
#pragma unroll
              for (int j = 0; j < kBlk; j++) {
                const uint2 a = wa[d][j], b = wb[d][j];
                request_unit(M, d, j, ml);
                unit(a, b, scale(s0, j), scale(s1, j), base0 + fo + j * kUnitBytes, hd0 + fo + j * kUnitBytes, ent, acc);
              }
              if (ml) advance();
              --i;
              if (++cb == hi) {
                store_part(out, p0 > 0, acc);
                cb = lo;
                out += s.wk * 16 * kRows;
              }
            }
          }
        }
      }
      __syncthreads();
      // the wk partial sums of each output, in order
      const bool pairs = R.ahead == 0;
      const int rows = pairs ? 8 : 16;
      const int outs = (b1 - b0) * rows * tokens;
      for (int i = tid; i < outs; i += kThreads) {
        const int r = i % rows, t = (i / rows) % tokens, tl = i / (rows * tokens);
        const int64_t o = (int64_t)(b0 + tl) * R.step + r;
        if (o >= R.limit) continue;
        const float* x = part + (size_t)tl * s.wk * 16 * kRows + r * kRows + t;
        float z0 = 0.f, z1 = 0.f;
#pragma unroll 4
        for (int w = 0; w < s.wk; w++) {
          z0 += x[w * 16 * kRows];
          if (pairs) z1 += x[(w * 16 + 8) * kRows];
        }
        if (MODE == kInt8 && odd[t]) {  // infinities and NaN of x, which the integers leave out
          const int64_t ra = R.first + o, rb = R.second + o;
          for (int k = 0; k < M.K; k++) {
            const float v = xs.at(t, k);
            if (fabsf(v) <= 3.402823466e38f) continue;
            z0 = fmaf(h2f(M.scales[ra * M.sstride + k / kGroup]) * decode_t(L, M.codes + ra * M.cstride, k), v, z0);
            if (pairs) z1 = fmaf(h2f(M.scales[rb * M.sstride + k / kGroup]) * decode_t(L, M.codes + rb * M.cstride, k), v, z1);
          }
        }
        fin(b0 + tl, r, t, z0, z1);
      }
      if (b1 < t1) __syncthreads();
    }
  }
};

// ---- one or two rows of x ---------------------------------------------------------------------------------
// The same product for NTOK = 1 or 2 rows of x in the int8 form, with the activation operands in registers.
// An MMA's 16 A rows are here 8 output rows x the two 32-byte halves of a 64-byte unit, and its 8 columns
// the halves x the four digits; a half's rows only use its own columns (the others' results are dropped, the
// tensor pipe has the time). So eight neighbouring lanes read 64 consecutive bytes of a row (half as many
// lines a load as in Product), a warp keeps the operands of its C units of K in registers and runs down the
// rows, and nothing but the codes and scales is loaded on the way: about 45 instructions per 512 bytes of
// Q2, where Product has over 100 and shared-memory loads among them.
// C: units (64 bytes) of a warp at most; D: tiles requested ahead.
template <int L, int NTOK, int C, int D>
struct Narrow {
  using T = Lay<L>;
  using G = Geo<L, kInt8>;
  static constexpr int kRows = NTOK, kS = T::kSlots, kTiles = (NTOK + G::kTok - 1) / G::kTok;
  static constexpr int kUnitBytes = 2 * kTiles * G::kTileBytes;  // operands of a 64-byte unit
  static constexpr int kBlocksPerWarp = C;                       // for plan_split: a "block" is a 64-byte unit here
  static constexpr int kTileRows = 8, kMode = kInt8;
  static bool plan(int tiles, int units, size_t room, Split* out);

  static __host__ __device__ size_t part_bytes(const Split& s) { return (size_t)s.batch * s.wk * 8 * kRows * 4; }
  static __host__ __device__ size_t smem_bytes(const Split& s) {
    return (size_t)s.pass * kUnitBytes + part_bytes(s) + kMaxWarps * 1024 + 64;
  }

  uint2 wa[D][C], wb[D][C];
  uint32_t sa[D][C], sb[D][C];  // scales of the lane's half: one (Q2) or both slots
  uint4 bop[C][NTOK][kS][G::kPairs];
  int st[C][NTOK][kS][2];       // accumulator starts (binary: [0] is what twice the accumulators need added)
  float sc[C][NTOK][kS];
  const uint8_t *pa, *pb;
  const uint16_t *ga, *gb;
  int lt;

  __device__ __forceinline__ void set_rows(const Mat& M, const Map& R, int ua) {
    const int lane = threadIdx.x & 31, r = lane >> 3, h = (lane >> 2) & 1, q = lane & 3;
    const int64_t o = (int64_t)lt * R.step + r;
    const int64_t a = R.first + min(o, (int64_t)R.limit - 1), b = R.second + min(o + R.ahead, (int64_t)R.limit - 1);
    pa = M.codes + a * M.cstride + 64 * ua + 32 * h + 8 * q;
    pb = M.codes + b * M.cstride + 64 * ua + 32 * h + 8 * q;
    ga = M.scales + a * M.sstride;
    gb = M.scales + b * M.sstride;
  }
  // Tile at the cursor into ring slot d. in: bit c, whether the lane's bytes of unit c exist, bit 16 + c,
  // whether its half of the unit does; g0, g1: groups.
  __device__ __forceinline__ void request(int d, uint32_t in, const int (&g0)[C], const int (&g1)[C]) {
#pragma unroll
    for (int c = 0; c < C; c++) {
      const bool on = in >> c & 1;
      ldg_codes(wa[d][c], pa + 64 * c, on);
      ldg_codes(wb[d][c], pb + 64 * c, on);
      if (in >> (16 + c) & 1) {
        if constexpr (kS == 1) {
          sa[d][c] = __ldg(ga + g0[c]);
          sb[d][c] = __ldg(gb + g0[c]);
        } else {
          sa[d][c] = __ldg(ga + g0[c]) | (uint32_t)__ldg(ga + g1[c]) << 16;
          sb[d][c] = __ldg(gb + g0[c]) | (uint32_t)__ldg(gb + g1[c]) << 16;
        }
      }
    }
  }

  // As Product::run: fin(tile, r, t, z, -) for tile row r of 8, or with R.ahead == 0 fin(tile, r, t, gate, up), r < 4.
  template <class X, class First, class Fin>
  __device__ __forceinline__ void run(uint8_t* smem, const Split& s, const Mat& M, const Map& R, int t0, int t1, const X& xs,
                                      int tokens, First first, Fin fin) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, q = lane & 3, h = g & 1;
    uint8_t* frag = smem;
    float* part = reinterpret_cast<float*>(smem + (size_t)s.pass * kUnitBytes);
    uint32_t* scr = reinterpret_cast<uint32_t*>(smem + (size_t)s.pass * kUnitBytes + part_bytes(s)) + warp * 256;
    int* odd = reinterpret_cast<int*>(smem + smem_bytes(s) - 64);
    const int kg = warp % s.wk, tg = warp / s.wk;
    const int units = (M.units + 1) / 2;  // of 64 bytes
    const bool mine = (q >> 1) == h;      // this lane's columns belong to its rows' half
    uint32_t k85 = 85u, kc80 = 0x00500050u;
    asm volatile("" : "+r"(k85), "+r"(kc80));
    const int64_t step_c = (int64_t)R.step * M.cstride, step_s = (int64_t)R.step * M.sstride;
    const int whole = R.limit / R.step;  // tiles that are not cut short
    bool fresh = true;
    if (tid < 16) odd[tid] = 0;
    for (int b0 = t0; b0 < t1; b0 += s.batch) {
      const int b1 = min(t1, b0 + s.batch);
      int ta = b0, tb = b0;
      if (tg < s.tg) {
        ta = b0 + (b1 - b0) * tg / s.tg;
        tb = b0 + (b1 - b0) * (tg + 1) / s.tg;
      }
      for (int p0 = 0; p0 < units; p0 += s.pass) {
        const int p1 = min(units, p0 + s.pass);
        const int ua = p0 + (p1 - p0) * kg / s.wk, ub = p0 + (p1 - p0) * (kg + 1) / s.wk;
        const int total = ua < ub ? tb - ta : 0;  // tiles
        uint32_t in = 0;
        int g0[C], g1[C];
#pragma unroll
        for (int c = 0; c < C; c++) {
          const int v = 2 * (ua + c) + h;  // the lane's 32-byte unit
          // (a lane past the end of a row's last half unit still holds results of that unit, and needs its scale)
          if (ua + c < ub && 32 * v + 8 * q < M.row_bytes) in |= 1u << c;
          if (ua + c < ub && v < M.units) in |= 1u << (16 + c);
          const int gr = L == TERN_Q2_0_G128 ? v : (L == TERN_T3_5PB_G128 ? (5 * v) >> 2 : 2 * v);
          g0[c] = min(gr, M.groups - 1);
          g1[c] = min(gr + 1, M.groups - 1);  // (past the row's end its operands are zero)
        }
        int left = total;
        lt = ta;
        auto advance = [&]() {
          --left;
          ++lt;
          if (lt >= whole) {
            set_rows(M, R, ua);  // the last tile may be cut short
          } else {
            pa += step_c; pb += step_c;
            ga += step_s; gb += step_s;
          }
        };
        if (total > 0) set_rows(M, R, ua);
#pragma unroll
        for (int d = 0; d < D; d++) {
#pragma unroll
          for (int c = 0; c < C; c++) {
            wa[d][c] = wb[d][c] = make_uint2(0, 0);
            sa[d][c] = sb[d][c] = 0;
          }
          if (left > 0) {
            request(d, in, g0, g1);
            advance();
          }
        }
        if (fresh) first();
        if (fresh || s.pass < units) {
          __syncthreads();  // the operands of the pass before have been taken (and the flags are clear)
          const int v0 = 2 * p0, nv = min(M.units, 2 * p1) - v0;
          for (uint32_t i = (uint32_t)nv * (kUnitBytes / 2) + tid * 16; i < (uint32_t)(2 * p1 - v0) * (kUnitBytes / 2); i += kThreads * 16)
            *reinterpret_cast<uint4*>(frag + i) = make_uint4(0, 0, 0, 0);  // a half past the row's end
          for (int i = warp; i < nv * NTOK; i += kMaxWarps) {
            const int v = i / NTOK, t = i % NTOK;
            if (t < tokens)
              build_int8<L>(xs, t, t % G::kTok, v0 + v, M.K, scr,
                            reinterpret_cast<uint4*>(frag + (size_t)v * (kUnitBytes / 2) + (t / G::kTok) * G::kTileBytes), odd + t);
          }
          __syncthreads();
          // this lane's operands: column (half g / 4, digit g % 4), k by q; starts and scales of columns 2q, 2q + 1
          const uint32_t base = sm100::smem_u32(frag);
#pragma unroll
          for (int c = 0; c < C; c++)
#pragma unroll
            for (int t = 0; t < NTOK; t++)
#pragma unroll
              for (int l = 0; l < kS; l++) {
                const bool on = ua + c < ub && t < tokens;
                const uint32_t tile = (uint32_t)((t / G::kTok) * G::kTileBytes);
                const uint32_t ub_ = base + (uint32_t)(2 * (ua + c - p0) + (g >> 2)) * (kUnitBytes / 2) + tile;
                const int ent = L == TERN_Q1_0_G128 ? q * 4 + (g & 3) : (L == TERN_Q2_0_G128 ? t : l) * 16 + q * 4 + (g & 3);
#pragma unroll
                for (int p = 0; p < G::kPairs; p++)
                  bop[c][t][l][p] = lds128_if(ub_ + (uint32_t)((p * G::kEnt + ent) * 16), on && (L != TERN_Q1_0_G128 || l == (q >> 1)));
                const uint32_t hd = base + (uint32_t)(2 * (ua + c - p0) + (q >> 1)) * (kUnitBytes / 2) + tile + G::kPairs * G::kEnt * 16;
                const uint4 r = lds128_if(hd + (uint32_t)(((L == TERN_Q2_0_G128 ? t : l) * 2 + (q & 1)) * 16), on);
                st[c][t][l][0] = (int)r.x;
                st[c][t][l][1] = (int)r.y;
                sc[c][t][l] = __uint_as_float(r.z);
              }
        }
        fresh = false;
        float* out = part + (size_t)((ta - b0) * s.wk + kg) * 8 * kRows;
        for (int i = 0; i < total;) {
#pragma unroll
          for (int d = 0; d < D; d++) {
            if (i >= total) break;
            float acc[NTOK][2] = {};
            uint2 xa[C], xb[C];
            uint32_t ya[C], yb[C];
#pragma unroll
            for (int c = 0; c < C; c++) {
              xa[c] = wa[d][c]; xb[c] = wb[d][c];
              ya[c] = sa[d][c]; yb[c] = sb[d][c];
            }
            if (left > 0) {
              request(d, in, g0, g1);
              advance();
            }
#pragma unroll
            for (int c = 0; c < C; c++) {
              uint32_t F[4][G::kPairs * 2];
              operands8<L>(xa[c], xb[c], k85, kc80, F);
#pragma unroll
              for (int t = 0; t < NTOK; t++)
#pragma unroll
                for (int l = 0; l < kS; l++) {
                  int e[4];
                  e[0] = e[2] = L == TERN_Q1_0_G128 ? 0 : st[c][t][l][0];
                  e[1] = e[3] = L == TERN_Q1_0_G128 ? 0 : st[c][t][l][1];
#pragma unroll
                  for (int p = 0; p < G::kPairs; p++) {
                    const uint4& f = bop[c][t][l][p];
                    mma_u8(e, F[0][2 * p], F[1][2 * p], F[2][2 * p], F[3][2 * p], f.x, f.y);
                    if (2 * p + 1 < G::kMma) mma_u8(e, F[0][2 * p + 1], F[1][2 * p + 1], F[2][2 * p + 1], F[3][2 * p + 1], f.z, f.w);
                  }
                  int v0 = e[0] + 256 * e[1], v1 = e[2] + 256 * e[3];
                  if (L == TERN_Q1_0_G128) {  // t = 2 b - 1
                    v0 = 2 * v0 + st[c][t][l][0];
                    v1 = 2 * v1 + st[c][t][l][0];
                  }
                  const float s0 = h2f((uint16_t)(l ? ya[c] >> 16 : ya[c] & 0xffffu)), s1 = h2f((uint16_t)(l ? yb[c] >> 16 : yb[c] & 0xffffu));
                  acc[t][0] = fmaf(s0 * sc[c][t][l], (float)v0, acc[t][0]);
                  acc[t][1] = fmaf(s1 * sc[c][t][l], (float)v1, acc[t][1]);
                }
            }
            // a row's sums are in four lanes: digits 0-1 and 2-3 of the half in lanes 8 r, 8 r + 1, of the other
            // half in lanes 8 r + 6, 8 r + 7; the lanes between hold other columns' results
#pragma unroll
            for (int t = 0; t < NTOK; t++) {
              float v0 = mine ? acc[t][0] : 0.f, v1 = mine ? acc[t][1] : 0.f;
              v0 += __shfl_xor_sync(0xffffffffu, v0, 1);
              v1 += __shfl_xor_sync(0xffffffffu, v1, 1);
              v0 += __shfl_xor_sync(0xffffffffu, v0, 6);
              v1 += __shfl_xor_sync(0xffffffffu, v1, 6);
              if ((lane & 7) == 0) {
                float *x = out + (lane >> 3) * kRows + t, *y = x + 4 * kRows;
                *x = p0 > 0 ? *x + v0 : v0;
                *y = p0 > 0 ? *y + v1 : v1;
              }
            }
            out += s.wk * 8 * kRows;
            i++;
          }
        }
      }
      __syncthreads();
      const bool pairs = R.ahead == 0;
      const int rows = pairs ? 4 : 8;
      for (int i = tid; i < (b1 - b0) * rows * tokens; i += kThreads) {
        const int r = i % rows, t = tokens == 1 ? 0 : (i / rows) % tokens, tl = i / (rows * tokens);
        const int64_t o = (int64_t)(b0 + tl) * R.step + r;
        if (o >= R.limit) continue;
        const float* x = part + (size_t)tl * s.wk * 8 * kRows + r * kRows + t;
        float z0 = 0.f, z1 = 0.f;
#pragma unroll
        for (int w = 0; w < kMaxWarps; w++)
          if (w < s.wk) {
            z0 += x[w * 8 * kRows];
            if (pairs) z1 += x[(w * 8 + 4) * kRows];
          }
        if (odd[t]) {
          const int64_t ra = R.first + o, rb = R.second + o;
          for (int k = 0; k < M.K; k++) {
            const float v = xs.at(t, k);
            if (fabsf(v) <= 3.402823466e38f) continue;
            z0 = fmaf(h2f(M.scales[ra * M.sstride + k / kGroup]) * decode_t(L, M.codes + ra * M.cstride, k), v, z0);
            if (pairs) z1 = fmaf(h2f(M.scales[rb * M.sstride + k / kGroup]) * decode_t(L, M.codes + rb * M.cstride, k), v, z1);
          }
        }
        fin(b0 + tl, r, t, z0, z1);
      }
      if (b1 < t1) __syncthreads();
    }
  }
};

// The cut for a Narrow product: wk warps along K with at most C units each, tg tile groups, so that the
// busiest warp has the least to do; a tile's end counts as two thirds of a unit.
template <class P>
inline bool plan_narrow(int tiles, int units32, size_t room, Split* out) {
  Split best{};
  double best_cost = -1;
  const int units = (units32 + 1) / 2;
  for (int wk = std::min(units, kMaxWarps); wk >= 1; wk--) {
    Split s{wk, std::max(1, std::min(kMaxWarps / wk, tiles)), 0, 0};
    const size_t tile_bytes = (size_t)wk * 8 * P::kRows * 4, fixed = P::smem_bytes(Split{wk, 1, 0, 0});
    s.batch = std::min<int>(tiles, std::max<int>(s.tg, (int)std::min<size_t>(room / 4 / tile_bytes, 256)));
    const int most = (int)std::min<size_t>((size_t)wk * P::kBlocksPerWarp, (room - fixed - s.batch * tile_bytes) / P::kUnitBytes);
    if (fixed + s.batch * tile_bytes > room || most < wk) continue;  // (the first pass gives every warp a unit)
    const int passes = (units + most - 1) / most;
    s.pass = std::max(wk, (units + passes - 1) / passes);
    const int batches = (tiles + s.batch - 1) / s.batch;
    const double per_group = (double)((s.batch + s.tg - 1) / s.tg);
    const double work = per_group * ((s.pass + wk - 1) / wk + 0.67);
    const double cost = (double)batches * passes * (work + 1.0) + (passes > 1 ? 0.5 * batches * units : 0.0);
    if (best_cost < 0 || cost < best_cost) {
      best_cost = cost;
      best = s;
    }
  }
  *out = best;
  return best_cost >= 0;
}

// The cut for `tiles` tiles per CTA, `units` units of K and kRows rows of x within `room` bytes of shared
// memory: as many blocks as fit beside the partial sums of a few tiles; then wk x tg warps so that the
// busiest warp has the least to do, a tile's end counted as half a block. False when not even one block
// fits (never within the limits of the callers).
template <class P>
inline bool plan_split(int tiles, int units, size_t room, Split* out) {
  Split best{};
  double best_cost = -1;
  const int blocks = (units + kBlk - 1) / kBlk;
  for (int wk = std::min(blocks, kMaxWarps); wk >= 1; wk--) {
    Split s{wk, std::max(1, std::min(kMaxWarps / wk, tiles)), 0, 0};
    const size_t tile_bytes = (size_t)wk * 16 * P::kRows * 4, fixed = P::smem_bytes(Split{wk, 1, 0, 0});
    const size_t block_bytes = (size_t)kBlk * P::kUnitBytes;
    // up to a quarter of the room for partial sums, but one tile for each tile group at least
    s.batch = std::min<int>(tiles, std::max<int>(s.tg, (int)std::min<size_t>(room / 4 / tile_bytes, 64)));
    if (fixed + s.batch * tile_bytes + wk * block_bytes > room) continue;  // a block for each warp along K
    s.pass = (int)std::min<size_t>(blocks, (room - fixed - s.batch * tile_bytes) / block_bytes);
    // balanced passes; the first one gives every chunk a block, so every partial sum is written
    const int passes = (blocks + s.pass - 1) / s.pass;
    s.pass = std::max(wk, (blocks + passes - 1) / passes);
    const int batches = (tiles + s.batch - 1) / s.batch;
    const double per_group = (double)((s.batch + s.tg - 1) / s.tg);  // tiles of a tile group in a batch
    const double work = per_group * ((s.pass + wk - 1) / wk + 0.5);
    double cost = (double)batches * passes * (work + 1.0) + (passes > 1 ? 0.5 * batches * blocks : 0.0);
    // warps side by side along K read a row's bytes together; far fewer than 1 KB of it at a time cost DRAM its
    // open pages (16 warps on 16 tiles of their own: a third of the rate)
    const int together = std::min(blocks, 8);
    if (wk < together) cost *= 0.5 + 0.5 * together / wk;
    if (best_cost < 0 || cost < best_cost) {
      best_cost = cost;
      best = s;
    }
  }
  *out = best;
  return best_cost >= 0;
}

template <int L, int MODE, int NT>
bool Product<L, MODE, NT>::plan(int tiles, int units, size_t room, Split* out) { return plan_split<Product>(tiles, units, room, out); }
template <int L, int NTOK, int C, int D>
bool Narrow<L, NTOK, C, D>::plan(int tiles, int units, size_t room, Split* out) { return plan_narrow<Narrow>(tiles, units, room, out); }

// Units of a warp and tiles ahead that fit the registers.
template <int L, int NTOK>
#ifdef VC
using NarrowFor = Narrow<L, NTOK, VC, VD>;
#else
using NarrowFor = Narrow<L, NTOK, L == TERN_Q2_0_G128 ? (NTOK == 1 ? 4 : 2) : L == TERN_T3_5PB_G128 && NTOK == 1 ? 2 : 1,
                         L == TERN_Q2_0_G128 ? (NTOK == 1 ? 2 : 3) : L == TERN_T3_5PB_G128 && NTOK == 1 ? 2 : 4>;
#endif

}  // namespace rows
}  // namespace tern
