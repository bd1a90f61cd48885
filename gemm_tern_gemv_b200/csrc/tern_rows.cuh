// The few-rows product core of the layer operators: y[t][o] = sum_k w[o][k] x[t][k] for a handful of
// rows t of x, on mma.sync, weights read once from global memory.
//
// A row of packed codes is cut into units of 32 bytes (128 weights of Q2_0_g128, 160 of base-3, 256 of
// binary); a warp takes 16 output rows and one unit at a time, each lane 8 bytes of rows g and g + 8
// (g = lane / 4). Four units, 128 bytes of a row, are a block: what a warp copies ahead into its own ring in
// shared memory (cp.async, four whole lines an instruction; the copies need no registers and no barrier
// but the warp's own). A unit lies in one 128-weight group (Q2) or two (slots 0 and 1 of base-3 and binary).
// Two forms of the product:
//   int8 (one row of x, two rows of 8 MMA columns at most): activations become exact integers. Per unit, slot
//     and row of x, X = round(x 2^S) with S from the largest |x| of the slot, written as four balanced
//     base-256 digits; the columns are (row of x, or slot) x (digit), and the epilogue joins them. The
//     codes become u8 operands with one LOP3 per four weights and no shift to a common place:
//       Q2      (word ^ 0xAA..) & 0x03.. (or 0x0C..) is c = t + 2 (or 4 c): the sign bit flipped turns a
//               two's-complement field into an offset one; the high nibble is shifted down once. B holds
//               X (or X / 4), and the accumulators start at -2 sum of what B holds.
//       binary  word & (0x01.. << j) is 2^j b (t = 2 b - 1), B holds X / 2^j, start -sum X / 2.
//       base-3  quotients q_j = floor(v / 3^j): c_j = q_j - 3 q_{j+1}, so B holds X_j - 3 X_{j-1} and the
//               accumulators start at -sum X; q_{j+1} = (85 q_j + 80) >> 8 for every q_j <= 242.
//     All of that is exact in int32; an activation is off by at most 2^-27 of the largest of its slot. For binary, whose
//     weights are never zero, that is less than the error of the sum in fp32. Where they can be zero an output may depend on
//     the small activations alone, so what the rounding takes from the caller's is added afterwards (of fp16 activations
//     it takes nothing unless a slot holds one of 16 or more beside one 2^17 times smaller): up to kMaxLost of them from
//     a list, more by add_lost. 24576 x 4096 Q2, one row, 12.8 us without
//     one, 14.7 with one such unit, 16.0 with one of 1500 in every unit beside N(0, 1), 93 where every activation is rounded
//     (base-3 17.0, 19.3, 20.9, 172). The experts' own h keep the rounding.
//   fp16 (up to 8 rows per tile; 4 with two slots): x itself is the B operand, the codes become +-2 / 0 by
//     one multiply and one mask per two weights, fp32 accumulators restart at every unit.
// Either way each unit's sums take their group scale in fp32. The activation operands of a CTA are built
// once in shared memory, in the order the MMA lanes read them.
//
// What bounds it: for small matrices the way in (entry and first requests about 2000 cycles, operands 2500 a row of
// 4096) and out; 4096 x 4096 Q2, one row, 6.1 us. For large ones latency, with the four warps a scheduler that the
// registers leave: at 24576 x 4096 and one row issue slots are 44 % busy with Q2 (49 % base-3), the shared-memory pipe
// 36 % (34 %), DRAM 21 % (13 %). Of 8.8 warp cycles an instruction 1.9 go to waiting for copies, 1.9 to fixed latencies, 0.9 to
// shared memory, 0.8 to barriers; base-3 spends 1.9 of 8.0 at barriers, where its 10 or 11 tiles x 7 blocks leave warps
// idle. A unit of 16 rows takes a warp 95 (Q2, int8), 129 (Q2, fp16, one column tile) or 171 (base-3, int8)
// instructions; 13.1 us Q2 = 2.1 TB/s, 17.2 base-3, 10.2 binary; 26.9 Q2 at 16 rows. With two column tiles and more the
// operands' reads from shared memory (512 bytes for two MMAs) come close to its limit. Why copies run through shared
// memory: with loads into registers a warp has too few bytes in flight (25 us there), and 128-byte pieces of a row keep
// DRAM's pages open.
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
// The first of a chain, on accumulators that start at c0 and c1 in both rows.
__device__ __forceinline__ void mma_u8_first(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1, int c0, int c1) {
  asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%10,%11};\n"
               : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(c0), "r"(c1));
}
__device__ __forceinline__ void mma_f16_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
               : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
// Copies of B bytes into shared memory; of `have` bytes at src only those are read, the rest arrives as zeros.
template <int B>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, int have) {
  if constexpr (B == 16) asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(have) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(B), "r"(have) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Balanced base-256 digits of X (|X| <= 2^30): byte p of the result is d_p in [-128, 127], X = sum d_p 2^(8p).
__device__ __forceinline__ uint32_t digits(int X) { return ((uint32_t)X + 0x00808080u) ^ 0x00808080u; }
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
// Smallest E with |x| < 2^E for a finite positive fp32 value given by its bits (subnormals count as 2^-126).
__device__ __forceinline__ int exponent(uint32_t abs_bits) { return (int)(abs_bits >> 23) - 126; }

// Rows of x as the core reads them: fp16 rows, or fp32 rows of expert activations. load() gives NE
// consecutive activations as floats, load16() N (a multiple of 8) as fp16 bits; both are zero from K on.
// K is a multiple of 8 and so are load16's k0 and, unless NE is 5, load's k0 of NE; rows are 16-byte aligned.
struct HalfRows {
  static constexpr bool kExact = true;  // the int8 form has to make its rounding good
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
  static constexpr bool kExact = false;
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
// First weight of unit u that belongs to slot 1.
template <int L>
__device__ __forceinline__ int slot_edge(int u) {
  return Lay<L>::kSlots == 1 ? Lay<L>::kUnitK : (L == TERN_Q1_0_G128 ? 128 : 128 - (u * 160) % 128);
}
// Exponents S of the slots of a unit, from the largest finite |x|: the integers are round(x 2^(S - sh)), sh by code_shift.
// xv: this lane's activations, those of the weights of byte `lane`; non-finite ones become zero (true if there was one).
template <int L>
__device__ __forceinline__ bool slot_exponents(float (&xv)[Lay<L>::kUnitK / 32], int edge, int (&S)[2]) {
  constexpr int NE = Lay<L>::kUnitK / 32;
  const int lane = threadIdx.x & 31;
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
  constexpr int kTop = L == TERN_T3_5PB_G128 ? 28 : 30;  // base-3 operands add up to four activations
  S[0] = S[1] = 0;
#pragma unroll
  for (int s = 0; s < Lay<L>::kSlots; s++) {
    mx[s] = __reduce_max_sync(0xffffffffu, mx[s]);
    S[s] = mx[s] ? min(100, kTop - exponent(mx[s])) : 0;
  }
  return bad;
}
// The code operand of weight e of a byte is 2^sh times c (or b).
template <int L> __device__ __forceinline__ constexpr int code_shift(int e) {
  return L == TERN_Q2_0_G128 ? 2 * (e & 1) : L == TERN_Q1_0_G128 ? (e & 3) : 0;
}

// What the int8 form's rounding takes from fp16 activations, multiples of 2^-24 below 2^-12: in a list while it fits. The
// list's order changes from run to run, so its sums are taken in integers.
constexpr int kMaxLost = 256;
struct Lost {
  uint32_t marks[32];     // bit u mod 1024: an activation of unit u was rounded
  int count;              // rounded activations, those past the list's end among them
  int pad[3];
  uint2 list[kMaxLost];   // k | row of x << 31, what is missing times 2^24
};

// int8 form of one unit u of row t of x, the tok-th of its column tile. xv: this lane's activations. scr: 32 x 8 words of this warp;
// frag: the column tile's entries, then one 16-byte record for each q: accumulator starts of columns 2 q
// and 2 q + 1 (binary: their sum to be added to twice the accumulators) and the scale 2^-S (x 2^16 for
// digits 2 and 3). Non-finite activations count as zero here (the caller adds them apart) and set *odd. lost (EXACT)
// receives what rounding takes, its list only if `list`.
template <int L, bool EXACT>
__device__ __forceinline__ void build_int8(float (&xv)[Lay<L>::kUnitK / 32], int t, int tok, int u, uint32_t* scr, uint4* frag, int* odd, Lost* lost, bool list) {
  using T = Lay<L>;
  using G = Geo<L, kInt8>;
  const int lane = threadIdx.x & 31;
  constexpr int NE = T::kUnitK / 32;  // activations of this lane: the weights of byte `lane` of the unit
  constexpr bool two_in_a_byte = L == TERN_T3_5PB_G128;  // a byte may hold weights of both slots
  const int edge = slot_edge<L>(u);
  int S[2];
  if (__any_sync(0xffffffffu, slot_exponents<L>(xv, edge, S)) && lane == 0) *odd = 1;
  // every fp16 activation is a multiple of 2^-24
  const bool coarse = EXACT && min(S[0], T::kSlots == 2 ? S[1] : S[0]) < 24 + code_shift<L>(1);
  bool rounded = false;
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
        const float v = ((lane * 5 + e < edge) == (s == 0)) ? xv[e] * exp2i(Ss) : 0.f;
        xi[e] = __float2int_rn(v);
        if (coarse) rounded |= rintf(v) != v;
        sum += xi[e];
      }
#pragma unroll
      for (int e = 0; e < 5; e++) scr[e * 32 + lane] = digits(xi[e] - (e ? 3 * xi[e - 1] : 0));
      scr[5 * 32 + lane] = digits(sum);  // |sum| <= 5 2^28: its digits fit too
    } else {
#pragma unroll
      for (int e = 0; e < NE; e++) {
        const float v = xv[e] * exp2i(Ss - code_shift<L>(e));
        if (coarse) rounded |= rintf(v) != v;
        scr[e * 32 + lane] = digits(__float2int_rn(v));
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
  if (coarse && __any_sync(0xffffffffu, rounded)) {
    if (lane == 0) atomicOr(lost->marks + (u >> 5 & 31), 1u << (u & 31));
#pragma unroll 1
    for (int e = 0; list && e < NE; e++) {
      float x = xv[0];
#pragma unroll
      for (int i = 1; i < NE; i++) x = e == i ? xv[i] : x;
      const int Se = S[lane * NE + e < edge ? 0 : 1] - code_shift<L>(e);
      const float v = x * exp2i(Se), d = v - rintf(v);
      if (d == 0.f) continue;
      const int i = atomicAdd(&lost->count, 1);
      if (i < kMaxLost) lost->list[i] = make_uint2((uint32_t)(u * T::kUnitK + lane * NE + e) | (uint32_t)t << 31, (uint32_t)__float2int_rn(d * exp2i(24 - Se)));
    }
  }
}

// fp16 form of one (unit, column tile from row t0 of x on): lane (g, q) loads and writes the operand words of
// column g.
template <int L> constexpr int kLaneWords = Lay<L>::kUnitK / 8;  // pairs of activations a lane takes
template <int L, class X>
__device__ __forceinline__ void load_fp16(const X& xs, int t0, int tokens, int u, int K, uint32_t (&v)[kLaneWords<L>]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int tok = t0 + (L == TERN_Q2_0_G128 ? g : (g & 3));
  if (tok < tokens && (L != TERN_Q1_0_G128 || (g >> 2) == (q >> 1))) xs.template load16<2 * kLaneWords<L>>(tok, Lay<L>::kUnitK * u + 2 * kLaneWords<L> * q, K, v);
}
template <int L>
__device__ __forceinline__ void store_fp16(const uint32_t (&v)[kLaneWords<L>], int t0, int tokens, int u, uint4* frag) {
  using G = Geo<L, kFp16>;
  const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int tok = L == TERN_Q2_0_G128 ? g : (g & 3);
  if (t0 + tok >= tokens) return;
  if constexpr (L == TERN_T3_5PB_G128) {
    const int k0 = 160 * u + 40 * q;
    const int edge = ((160 * u) / kGroup + 1) * kGroup - k0;  // first of the lane's weights in slot 1
    auto h = [&](int e) -> uint32_t {
      return ((e < edge) == (g < 4)) ? ((e & 1) ? v[e >> 1] >> 16 : v[e >> 1] & 0xffffu) : 0u;
    };
    // word b of the lane, register r = 5 h + i: digit 4 - i of bytes h and h + 2
    auto reg = [&](int b, int r) { const int e = 20 * b + 5 * (r / 5) + 4 - r % 5; return h(e) | (h(e + 10) << 16); };
#pragma unroll
    for (int p = 0; p < 5; p++) frag[p * 32 + lane] = make_uint4(reg(0, 2 * p), reg(1, 2 * p), reg(0, 2 * p + 1), reg(1, 2 * p + 1));
  } else if constexpr (L == TERN_Q2_0_G128) {
#pragma unroll
    for (int p = 0; p < 4; p++)  // register i: fields i and i + 8 of a word
      frag[p * 32 + lane] = make_uint4(__byte_perm(v[p], v[p + 4], 0x5410), __byte_perm(v[8 + p], v[12 + p], 0x5410),
                                       __byte_perm(v[p], v[p + 4], 0x7632), __byte_perm(v[8 + p], v[12 + p], 0x7632));
  } else {
    if ((g >> 2) != (q >> 1)) return;
#pragma unroll
    for (int p = 0; p < 8; p++)  // register i: bits i and i + 16 of a word
      frag[p * G::kEnt + q * 4 + tok] =
          make_uint4(__byte_perm(v[p], v[p + 8], 0x5410), __byte_perm(v[16 + p], v[24 + p], 0x5410),
                     __byte_perm(v[p], v[p + 8], 0x7632), __byte_perm(v[16 + p], v[24 + p], 0x7632));
  }
}

// a / c for a < 2^20 by the reciprocal of c; the half keeps the result off the edges.
__device__ __forceinline__ int part_of(int a, float inv) { return (int)(((float)a + 0.5f) * inv); }
// First tile of CTA b where each of `ctas` has `each` and `extra` of them, evenly spread, one more. (All of these
// side by side crowd their GPCs: a 4096 x 12288 down product of two experts took 20.5 us so, 16 spread.)
__device__ __forceinline__ int first_tile(int b, int ctas, int each, int extra) {
  return b * each + part_of(b * extra, __fdividef(1.f, (float)ctas));
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

// A block is four units, 128 bytes of a row: what a warp copies and works off at a time.
constexpr int kBlk = 4;

// Code operands a0 .. a3 of each int8 MMA from 8 bytes of rows g (a) and g + 8 (b). kx, ky are constants opaque
// to the compiler: base-3's 85 and 80 in both halves, so that its steps stay multiplications; Q2's 0xAA..,
// so that flipping and masking are one three-input operation.
template <int L>
__device__ __forceinline__ void operands8(uint2 a, uint2 b, uint32_t kx, uint32_t ky, uint32_t (&F)[4][Geo<L, kInt8>::kPairs * 2]) {
  const uint32_t w[4] = {a.x, b.x, a.y, b.y};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    if constexpr (L == TERN_Q2_0_G128) {
      const uint32_t z = w[i] >> 4;
      F[i][0] = (w[i] ^ kx) & 0x03030303u;
      F[i][1] = (w[i] ^ kx) & 0x0C0C0C0Cu;
      F[i][2] = (z ^ kx) & 0x03030303u;
      F[i][3] = (z ^ kx) & 0x0C0C0C0Cu;
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
        E = E * kx + ky;
        O = O * kx + ky;
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
  static constexpr int kDepth = MODE == kInt8 ? 3 : 2;   // blocks in a warp's ring
  static constexpr int kUnitBytes = NT * G::kTileBytes;  // activation operands of one unit
  static constexpr int kAcc = MODE == kInt8 ? 2 : 4;
  static constexpr int kTileRows = 16, kMode = MODE;
  // scales of a block and row: Q2 four groups, binary eight; base-3 five, copied as the four words from the
  // 4-byte boundary below the first on
  static constexpr int kScaleBytes = L == TERN_Q2_0_G128 ? 8 : 16;
  static constexpr int kStage = 16 * 128 + 16 * kScaleBytes;  // [16][128] codes, [16][kScaleBytes] scales
  static constexpr int kFlags = 64 + (MODE == kInt8 && L != TERN_Q1_0_G128 ? (int)sizeof(Lost) : 0);  // bytes: `odd`, `lost`
  static bool plan(int tiles, int units, size_t room, Split* out);

  // shared memory: operands [pass], partial sums [batch][wk][16][kRows], flags, scratch of the int8 operands'
  // building, rings
  static __host__ __device__ size_t part_bytes(const Split& s) { return (size_t)s.batch * s.wk * 16 * kRows * 4; }
  static __host__ __device__ size_t smem_bytes(const Split& s) {
    return (size_t)s.pass * kBlk * kUnitBytes + part_bytes(s) + (MODE == kInt8 ? kMaxWarps * 1024 : 0) + kMaxWarps * kDepth * kStage + kFlags + 128;
  }

  // copy cursor: this lane's four rows (lane / 8 + 4 i) of the tile's codes at its 16-byte piece of the block,
  // and its row of scales; tile, block
  const uint8_t* pc[4];
  const uint16_t* ps;
  int lt, lb;
  uint32_t kx, ky;  // see operands8
  int carry;        // base-3, int8: all ones above bit 16 in lanes of the low digits

  __device__ __forceinline__ void set_rows(const Mat& M, const Map& R) {
    const int lane = threadIdx.x & 31;
    const int64_t o = (int64_t)lt * R.step, first = R.first + o, second = R.second + o;
    const int last = (int)min((int64_t)R.limit - 1 - o, (int64_t)64);  // rows of the tile that are there, less one
    const uint8_t* c = M.codes + 16 * (lane & 7);
    const uint8_t *a = c + first * M.cstride, *b = c + second * M.cstride;
#pragma unroll
    for (int i = 0; i < 2; i++) {
      pc[i] = a + min((lane >> 3) + 4 * i, last) * M.cstride;
      pc[i + 2] = b + min((lane >> 3) + 4 * i + R.ahead, last) * M.cstride;
    }
    const int r = L == TERN_T3_5PB_G128 ? lane >> 1 : lane & 15;
    ps = M.scales + (r < 8 ? first + min(r, last) : second + min(r - 8 + R.ahead, last)) * M.sstride;
  }
  // The block at the cursor into the ring stage at `stage`. Piece c of a row lies at (c / 2 ^ row % 4) * 32 +
  // c % 2 * 16, so that the four rows a half-warp reads 32 bytes of are in different banks.
  __device__ __forceinline__ void request(const Mat& M, uint32_t stage) {
    const int lane = threadIdx.x & 31, c = lane & 7;
    const int off = lb * 128, have = min(max(M.row_bytes - off - 16 * c, 0), 16);
    const uint32_t dst = stage + (lane >> 3) * 128 + (((c >> 1) ^ (lane >> 3)) * 32) + (c & 1) * 16;
#pragma unroll
    for (int i = 0; i < 4; i++) copy_async<16>(dst + i * 512, pc[i] + off, have);
    const uint32_t ds = stage + 16 * 128;
    if constexpr (L == TERN_T3_5PB_G128) {
      // groups 5 lb .. 5 lb + 4 of a row, two words a lane
      const int w = ((10 * lb) & ~3) + 8 * (lane & 1), left = 2 * M.groups - w;
#pragma unroll
      for (int i = 0; i < 2; i++)
        copy_async<4>(ds + (lane >> 1) * 16 + 8 * (lane & 1) + 4 * i, reinterpret_cast<const uint8_t*>(ps) + w + 4 * i, min(max(left - 4 * i, 0), 4));
    } else {
      const int left = 2 * M.groups - kScaleBytes * lb;
      if (lane < 16) copy_async<kScaleBytes>(ds + lane * kScaleBytes, reinterpret_cast<const uint8_t*>(ps) + kScaleBytes * lb, min(max(left, 0), kScaleBytes));
    }
  }

  // One unit: codes and scales of rows g (a) and g + 8 (b) times the operands at base + ent[.] (this lane's
  // entries; starts and scales at hd) into acc.
  __device__ __forceinline__ void unit(uint2 a, uint2 b, float s0, float s1, uint32_t base, uint32_t hd, const uint32_t (&ent)[NT],
                                       float (&acc)[NT][kAcc]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    if constexpr (MODE == kInt8) {
      int c[NT][4];
      uint4 st[NT];  // accumulator starts (binary: what twice the accumulators need added) and 2^-S
#pragma unroll
      for (int n = 0; n < NT; n++) st[n] = lds128(hd + (uint32_t)(n * G::kTileBytes));
      uint32_t F[4][G::kPairs * 2];
      operands8<L>(a, b, kx, ky, F);
#pragma unroll
      for (int p = 0; p < G::kPairs; p++)
#pragma unroll
        for (int n = 0; n < NT; n++) {
          // binary: the columns of the other slot are zero
          const uint32_t at = base + ent[n] + (uint32_t)(n * G::kTileBytes + p * G::kEnt * 16);
          const uint4 f = L == TERN_Q1_0_G128 ? lds128_if(at, (g >> 2) == (q >> 1)) : lds128(at);
          if (p == 0) mma_u8_first(c[n], F[0][0], F[1][0], F[2][0], F[3][0], f.x, f.y, L == TERN_Q1_0_G128 ? 0 : (int)st[n].x, L == TERN_Q1_0_G128 ? 0 : (int)st[n].y);
          else mma_u8(c[n], F[0][2 * p], F[1][2 * p], F[2][2 * p], F[3][2 * p], f.x, f.y);
          if (2 * p + 1 < G::kMma) mma_u8(c[n], F[0][2 * p + 1], F[1][2 * p + 1], F[2][2 * p + 1], F[3][2 * p + 1], f.z, f.w);
        }
#pragma unroll
      for (int n = 0; n < NT; n++) {
        int v0 = c[n][0] + 256 * c[n][1], v1 = c[n][2] + 256 * c[n][3];
        if (L == TERN_Q1_0_G128) {  // t = 2 b - 1
          v0 = 2 * v0 + (int)st[n].x;
          v1 = 2 * v1 + (int)st[n].x;
        }
        if (L == TERN_T3_5PB_G128) {
          // The digits of X_j - 3 X_{j-1} carry: what weights of zero leave is zero only in both lanes of a sum together, and
          // 2^16 more in one of them than the sum may be. So the carry goes over.
          const int o0 = (v0 + 0x8000) & carry, o1 = (v1 + 0x8000) & carry;
          v0 += (__shfl_xor_sync(0xffffffffu, o0, 1) >> 16) - o0;
          v1 += (__shfl_xor_sync(0xffffffffu, o1, 1) >> 16) - o1;
        }
        const float sc = __uint_as_float(st[n].z);
        acc[n][0] = fmaf(s0 * sc, (float)v0, acc[n][0]);
        acc[n][1] = fmaf(s1 * sc, (float)v1, acc[n][1]);
      }
    } else {
      const uint32_t w[4] = {a.x, b.x, a.y, b.y};
      float c[NT][4];
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
          if (p == 0) mma_f16_first(c[n], a00, a01, a02, a03, f.x, f.y);
          else mma_f16(c[n], a00, a01, a02, a03, f.x, f.y);
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

  // Adds the list's terms to the first partial sums of tiles [b0, b1), eight lanes for each output row. Scales and what is
  // missing are multiples of 2^-24, below 2^16 and 2^-12, so 256 terms fit 64 bits. (A scale that is not finite has made
  // the sum infinite or NaN already.)
  static __device__ __forceinline__ void add_listed(const uint2* list, int n, float* part, int wk, const Mat& M, const Map& R, int b0,
                                                    int b1, int tokens) {
    const int sub = threadIdx.x & 7;
    for (int i = threadIdx.x >> 3; i < (b1 - b0) * 16; i += kThreads / 8) {  // (a tile is four warps' rows: all lanes go on)
      const int tl = i >> 4, r = i & 15;
      const int64_t o = (int64_t)(b0 + tl) * R.step, last = min((int64_t)R.limit - 1 - o, (int64_t)64);
      const int64_t row = r < 8 ? R.first + o + min((int64_t)r, last) : R.second + o + min((int64_t)(r - 8 + R.ahead), last);
      const uint8_t* codes = M.codes + row * M.cstride;
      const uint16_t* scales = M.scales + row * M.sstride;
      int64_t z[kRows] = {};
#pragma unroll 4
      for (int j = sub; j < n; j += 8) {
        const uint2 e = list[j];
        const int k = (int)(e.x & 0x7fffffffu);
        const float w = h2f(scales[k / kGroup]) * decode_t(L, codes, k);
        const int64_t term = fabsf(w) <= 65504.f ? (int64_t)__float2ll_rn(w * 16777216.f) * (int)e.y : 0;
#pragma unroll
        for (int t = 0; t < kRows; t++) z[t] += (int)(e.x >> 31) == t ? term : 0;
      }
#pragma unroll
      for (int t = 0; t < kRows; t++) {
#pragma unroll
        for (int d = 4; d; d >>= 1) z[t] += __shfl_xor_sync(0xffffffffu, z[t], d);
        if (sub == 0 && t < tokens) part[(size_t)tl * wk * 16 * kRows + r * kRows + t] += (float)((double)z[t] * (1. / 281474976710656.));
      }
    }
  }

  // Adds what the integers leave out of the activations in the units marked in `lost` to the first partial sums of tiles
  // [b0, b1): a warp takes four rows of a tile, a lane its byte of each unit. Units of an equal mark add zeros.
  template <class X>
  static __device__ __forceinline__ void add_lost(const uint32_t* lost, float* part, int wk, const Mat& M, const Map& R, int b0, int b1,
                                               const X& xs, int tokens) {
    constexpr int NE = T::kUnitK / 32;
    const int lane = threadIdx.x & 31;
    const uint32_t marks = lost[lane];
    for (int item = threadIdx.x >> 5; item < (b1 - b0) * 4; item += kMaxWarps) {
      const int tl = item >> 2, r0 = 4 * (item & 3);
      const int64_t o = (int64_t)(b0 + tl) * R.step, last = min((int64_t)R.limit - 1 - o, (int64_t)64);
      const int64_t base = (r0 < 8 ? R.first : R.second) + o;
      const int at = r0 < 8 ? r0 : r0 - 8 + R.ahead;
      for (int c = 0; c < M.units; c += 1024)
        for (int w = 0; w < 32; w++)
          for (uint32_t bits = __shfl_sync(0xffffffffu, marks, w); bits; bits &= bits - 1) {
            const int u = c + 32 * w + __ffs(bits) - 1;
            if (u >= M.units) break;
            const int edge = slot_edge<L>(u), byte = 32 * u + lane, g = u * T::kUnitK / kGroup;
            for (int t = 0; t < tokens; t++) {
              float xv[NE] = {};
              xs.template load<NE>(t, u * T::kUnitK + lane * NE, M.K, xv);
              int S[2];
              slot_exponents<L>(xv, edge, S);
#pragma unroll
              for (int e = 0; e < NE; e++) {
                const int Ss = S[lane * NE + e < edge ? 0 : 1] - code_shift<L>(e);
                const float v = xv[e] * exp2i(Ss);
                xv[e] = (v - rintf(v)) * exp2i(-Ss);
              }
#pragma unroll
              for (int i = 0; i < 4; i++) {
                const int64_t row = base + min((int64_t)(at + i), last);
                const uint16_t* s = M.scales + row * M.sstride;
                const float s0 = h2f(s[g]), s1 = h2f(s[min(g + 1, M.groups - 1)]);
                int code = byte < M.row_bytes ? M.codes[row * M.cstride + byte] : 0;
                float z = 0.f;
#pragma unroll
                for (int e = 0; e < NE; e++) {
                  int c3 = (code & 1) - (code & 2);
                  if constexpr (L == TERN_T3_5PB_G128) {
                    const int q = code / 3;
                    c3 = code - 3 * q - 1;
                    code = q;
                  } else {
                    code >>= 2;
                  }
                  // (a scale that is not finite does not meet activations that are whole)
                  if (xv[e] != 0.f) z = fmaf((lane * NE + e < edge ? s0 : s1) * (float)c3, xv[e], z);
                }
#pragma unroll
                for (int d = 16; d; d >>= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
                if (lane == 0) part[(size_t)tl * wk * 16 * kRows + (r0 + i) * kRows + t] += z;
              }
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
    uint8_t* tail = smem + (size_t)s.pass * kBlk * kUnitBytes + part_bytes(s);
    int* odd = reinterpret_cast<int*>(tail);  // rows of x with a non-finite activation
    Lost* lost = reinterpret_cast<Lost*>(tail + 64);  // int8, but for binary
    uint32_t* scr = reinterpret_cast<uint32_t*>(tail + kFlags) + warp * 256;
    const uint32_t ring = ((sm100::smem_u32(tail) + kFlags + (MODE == kInt8 ? kMaxWarps * 1024 : 0) + 127) & ~127u) + warp * (kDepth * kStage);
    const int blocks = (M.units + kBlk - 1) / kBlk;
    const int wk = min(s.wk, blocks);  // (M may be shorter than what was planned for)
    const float inv_wk = __fdividef(1.f, (float)wk), inv_tg = __fdividef(1.f, (float)s.tg);
    const int tg = part_of(warp, inv_wk), kg = warp - tg * wk;
    kx = L == TERN_Q2_0_G128 ? 0xAAAAAAAAu : 85u;
    ky = 0x00500050u;
    carry = q & 1 ? 0 : ~0xffff;
    asm volatile("" : "+r"(kx), "+r"(ky));
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
    const uint32_t lane_c = (uint32_t)(g * 128 + (g & 3) * 32 + 8 * q);  // unit 0 of row g in a stage
    bool fresh = true;
    constexpr bool kLost = MODE == kInt8 && L != TERN_Q1_0_G128 && X::kExact;
    if (tid < 16) odd[tid] = 0;
    if (kLost && tid < 32) lost->marks[tid] = 0;
    if (kLost && tid == 0) lost->count = 0;
    for (int b0 = t0; b0 < t1; b0 += s.batch) {
      const int b1 = min(t1, b0 + s.batch);
      int ta = b0, tb = b0;
      if (tg < s.tg) {
        ta = b0 + part_of((b1 - b0) * tg, inv_tg);
        tb = b0 + part_of((b1 - b0) * (tg + 1), inv_tg);
      }
      for (int p0 = 0; p0 < blocks; p0 += s.pass) {
        const int p1 = min(blocks, p0 + s.pass);
        const int lo = p0 + part_of((p1 - p0) * kg, inv_wk), hi = p0 + part_of((p1 - p0) * (kg + 1), inv_wk);  // the warp's blocks
        int left = (tb - ta) * (hi - lo);  // blocks still to be copied
        const int total = left;
        lt = ta;
        lb = lo;
        auto next = [&](uint32_t stage) {  // requests a block, or nothing; one group of copies either way
          if (left > 0) {
            request(M, stage);
            --left;
            if (++lb == hi) {
              lb = lo;
              ++lt;
              if (lt >= whole) {
                set_rows(M, R);  // the last tile may be cut short
              } else {
#pragma unroll
                for (int i = 0; i < 4; i++) pc[i] += step_c;
                ps += step_s;
              }
            }
          }
          copy_commit();
        };
        if (left > 0) set_rows(M, R);
#pragma unroll 1
        for (int d = 0; d < kDepth; d++) next(ring + d * kStage);
        if (fresh) first();
        if (fresh || s.pass < blocks) {
          __syncthreads();  // the operands of the pass before are no longer read (and the flags are clear)
          const int u0 = p0 * kBlk, nu = min(M.units, p1 * kBlk) - u0;
          // (row or column tile, unit) pairs dealt to the warps, the next pair's activations under way meanwhile
          const int all = (MODE == kInt8 ? tokens : NT) * nu;
          if constexpr (MODE == kInt8) {
            constexpr int NE = T::kUnitK / 32;
            float ahead[NE];
            auto fetch = [&](int i) {
#pragma unroll
              for (int e = 0; e < NE; e++) ahead[e] = 0.f;
              if (i < all) xs.template load<NE>(kRows == 1 || i < nu ? 0 : 1, (u0 + (i < nu ? i : i - nu)) * T::kUnitK + lane * NE, M.K, ahead);
            };
            static_assert(kRows <= 2, "");
            fetch(warp);
#pragma unroll 1
            for (int i = warp; i < all; i += kMaxWarps) {
              float xv[NE];
#pragma unroll
              for (int e = 0; e < NE; e++) xv[e] = ahead[e];
              fetch(i + kMaxWarps);
              const int t = kRows == 1 || i < nu ? 0 : 1, u = i < nu ? i : i - nu;
              build_int8<L, kLost>(xv, t, t % G::kTok, u0 + u, scr, reinterpret_cast<uint4*>(frag + (size_t)u * kUnitBytes + (t / G::kTok) * G::kTileBytes),
                            odd + t, lost, b0 == t0);
            }
          } else {
            uint32_t ahead[kLaneWords<L>] = {};
            auto split = [&](int i, int& n, int& u) {
              n = 0;
              u = i;
#pragma unroll
              for (int j = 1; j < NT; j++)
                if (u >= nu) {
                  u -= nu;
                  n++;
                }
            };
            int n, u;
            split(warp, n, u);
            if (warp < all) load_fp16<L>(xs, n * G::kTok, tokens, u0 + u, M.K, ahead);
#pragma unroll 1
            for (int i = warp; i < all; i += kMaxWarps) {
              uint32_t v[kLaneWords<L>];
#pragma unroll
              for (int e = 0; e < kLaneWords<L>; e++) v[e] = ahead[e];
              const int n0 = n, v0 = u;
              split(i + kMaxWarps, n, u);
              if (i + kMaxWarps < all) load_fp16<L>(xs, n * G::kTok, tokens, u0 + u, M.K, ahead);
              store_fp16<L>(v, n0 * G::kTok, tokens, u0 + v0, reinterpret_cast<uint4*>(frag + (size_t)v0 * kUnitBytes + n0 * G::kTileBytes));
            }
          }
          __syncthreads();
        }
        fresh = false;
        float acc[NT][kAcc] = {};
        int cb = lo;
        uint32_t stage = ring;
        float* out = part + (size_t)((ta - b0) * wk + kg) * 16 * kRows;
#pragma unroll 1
        for (int i = 0; i < total; i++) {
          copy_wait<kDepth - 1>();
          __syncwarp();
          const uint32_t fo = (uint32_t)((cb - p0) * kBlk * kUnitBytes);
          uint32_t sa[kBlk], sb[kBlk];  // scales of rows g and g + 8, as fp16 bits
          const uint32_t sc = stage + 16 * 128 + g * kScaleBytes;
          if constexpr (L == TERN_Q2_0_G128) {
            const uint2 a = lds64(sc), b = lds64(sc + 8 * kScaleBytes);
            sa[0] = a.x & 0xffff; sa[1] = a.x >> 16; sa[2] = a.y & 0xffff; sa[3] = a.y >> 16;
            sb[0] = b.x & 0xffff; sb[1] = b.x >> 16; sb[2] = b.y & 0xffff; sb[3] = b.y >> 16;
          } else {
            const uint32_t at = sc + (L == TERN_Q1_0_G128 ? (q & 2) : ((10 * cb) & 3) + (q & 2));  // by the lane's slot
#pragma unroll
            for (int j = 0; j < kBlk; j++) {
              sa[j] = lds_u16(at + (L == TERN_Q1_0_G128 ? 4 : 2) * j);
              sb[j] = lds_u16(at + (L == TERN_Q1_0_G128 ? 4 : 2) * j + 8 * kScaleBytes);
            }
          }
          uint2 a[kBlk], b[kBlk];
#pragma unroll
          for (int j = 0; j < kBlk; j++) {
            const uint32_t at = (stage + lane_c) ^ (32u * j);
            a[j] = lds64(at);
            b[j] = lds64(at + 8 * 128);
          }
          __syncwarp();  // every lane has read the stage
          const int have = M.units - cb * kBlk;
          next(stage);
          stage = stage == ring + (kDepth - 1) * kStage ? ring : stage + kStage;
#pragma unroll
          for (int j = 0; j < kBlk; j++) {
            if (j >= have) break;  // the row ends inside the block
            unit(a[j], b[j], h2f((uint16_t)sa[j]), h2f((uint16_t)sb[j]), base0 + fo + j * kUnitBytes, hd0 + fo + j * kUnitBytes, ent, acc);
          }
          if (++cb == hi) {
            store_part(out, p0 > 0, acc);
            cb = lo;
            out += wk * 16 * kRows;
          }
        }
        copy_wait<0>();
      }
      __syncthreads();
      if constexpr (kLost) {
        if (lost->count) {
          if (lost->count > kMaxLost) add_lost(lost->marks, part, wk, M, R, b0, b1, xs, tokens);
          else add_listed(lost->list, lost->count, part, wk, M, R, b0, b1, tokens);
          __syncthreads();
        }
      }
      // the wk partial sums of each output, in order
      const bool pairs = R.ahead == 0;
      const int rows = pairs ? 8 : 16, shift = pairs ? 3 : 4;
      for (int i = tid; i < (b1 - b0) * rows * tokens; i += kThreads) {
        const int r = i & (rows - 1), tt = i >> shift, t = tokens == 1 ? 0 : tt % tokens, tl = tokens == 1 ? tt : tt / tokens;
        const int64_t o = (int64_t)(b0 + tl) * R.step + r;
        if (o >= R.limit) continue;
        const float* x = part + (size_t)tl * wk * 16 * kRows + r * kRows + t;
        float z0 = 0.f, z1 = 0.f;
#pragma unroll 4
        for (int w = 0; w < wk; w++) {
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

// The cut for `tiles` tiles per CTA, `units` units of K and kRows rows of x within `room` bytes of shared
// memory: as many blocks as fit beside the partial sums of a few tiles; then wk x tg warps so that the
// busiest warp has the least to do, a tile's end counted as 0.3 of a block. False when not even one block
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
    // batches of one, two, four, ... tiles for each group, up to a quarter of the room for partial sums
    for (int each = 1; each == 1 || (s.batch < tiles && s.batch < 64 && (size_t)s.batch * tile_bytes < room / 4); each *= 2) {
      s.batch = std::min(tiles, each * s.tg);
      if (fixed + s.batch * tile_bytes + wk * block_bytes > room) break;  // a block for each warp along K
      s.pass = (int)std::min<size_t>(blocks, (room - fixed - s.batch * tile_bytes) / block_bytes);
      // balanced passes; the first one gives every chunk a block, so every partial sum is written
      const int passes = (blocks + s.pass - 1) / s.pass;
      s.pass = std::max(wk, (blocks + passes - 1) / passes);
      const int batches = (tiles + s.batch - 1) / s.batch;
      const double work = (double)((s.batch + s.tg - 1) / s.tg) * ((s.pass + wk - 1) / wk + 0.3);
      double cost = (double)batches * passes * (work + 1.0) + (passes > 1 ? 0.5 * batches * blocks : 0.0);
      // warps side by side along K read a row's bytes together; much less than 512 of them at a time cost DRAM
      // its open pages (24576 x 4096 Q2, one row: 13.6 us with 4, 8 or 16 warps along K, 14.2 with 2)
      const int together = std::min(blocks, 4);
      if (wk < together) cost *= 0.9 + 0.1 * together / wk;
      if (best_cost < 0 || cost < best_cost) {
        best_cost = cost;
        best = s;
      }
    }
  }
  *out = best;
  return best_cost >= 0;
}

template <int L, int MODE, int NT>
bool Product<L, MODE, NT>::plan(int tiles, int units, size_t room, Split* out) { return plan_split<Product>(tiles, units, room, out); }

}  // namespace rows
}  // namespace tern
