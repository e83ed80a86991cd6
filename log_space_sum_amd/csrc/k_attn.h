// k_attn.h -- what the softmax attention's kernels share: how a type is
// multiplied, tiles in LDS and their fragments, where rows lie.
//
// Every product runs on the 32 x 32 x 16 matrix instruction.  Its operands: a
// lane holds 8 consecutive elements of the contracted dimension, from 8 h, of row
// (column) l of 32, with l = lane % 32, h = lane / 32; its result: a lane holds
// column l and of the rows 8 (r / 4) + 4 h + r % 4, r = 0 .. 15.  So a result's
// registers are the next product's operand where the contraction takes the
// elements in that order on both sides: the other operand is read from LDS by the
// transposing read, four rows of one column at a time, from rows 4 h and 8 + 4 h of
// every 16.  Scores and weights never pass through LDS.
//
// Precision.  16-bit tensors are multiplied as they are.  What a kernel computes
// and multiplies again (the weights P, the gradients dS of the scores) is split into
// planes, each the rounding of what the planes before it leave: three of bfloat16 (24 bits), or
// two of float16 (22 bits, and none below 2^-39 of a sum's largest: its numbers end at 2^-24, and the
// largest is held near 2^14).  One plane, the usual choice, would add an error as
// large as the output's own rounding; with these, outputs are what float32 arithmetic
// gives, rounded once.  float32 tensors are split into three bfloat16 planes
// too, and products of planes p, q with p + q <= 2 are summed (24 bits).
#pragma once
#include <type_traits>

#include "pc_ops.h"
#include "pc_ring.h"

namespace pc {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;

typedef uint4 frag;     // 8 elements of 16 bits

constexpr float LOG2E = 1.44269504088896341f, LN2 = 0.693147180559945309f;

// ---- types -------------------------------------------------------------------
// IN: planes of a tensor's values, W: planes of computed ones.  BIAS: the forward's
// weights, at most 1, are held as 2^BIAS times themselves (float16: its small numbers have few bits).
struct Bf16Planes {
  static __device__ __forceinline__ f32x16 mma(frag a, frag b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t pack(float x, float y) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x, y}, bf16x2));
  }
  // x less the low (high) value of a pair, in one instruction: a dot product with (-1, 0) or (0, -1).  The other value is
  // finite where x is: both were rounded from one split's values.  (The constant goes through a register: as an
  // inline constant the instruction would take the other half.)
  static __device__ __forceinline__ float less(float x, uint32_t u, uint32_t one) {
    asm("" : "+s"(one));
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, u), __builtin_bit_cast(bf16x2, one), x, false);
  }
  static __device__ __forceinline__ float less_low(float x, uint32_t u) { return less(x, u, 0x0000bf80u); }
  static __device__ __forceinline__ float less_high(float x, uint32_t u) { return less(x, u, 0xbf800000u); }
};
template <typename T>
struct Num;
template <>
struct Num<bf16> : Bf16Planes {
  static constexpr int IN = 1, W = 3, BIAS = 0;
};
template <>
struct Num<float> : Bf16Planes {
  static constexpr int IN = 3, W = 3, BIAS = 0;
};
template <>
struct Num<f16> {
  static constexpr int IN = 1, W = 2, BIAS = 14;
  static __device__ __forceinline__ f32x16 mma(frag a, frag b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t pack(float x, float y) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x, y}, f16x2));
  }
  // (one mixed instruction; the compiler takes a conversion and a subtraction)
  static __device__ __forceinline__ float less_low(float x, uint32_t u) {
    float r;
    asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel_hi:[1,0,0]" : "=v"(r) : "v"(u), "v"(x));
    return r;
  }
  static __device__ __forceinline__ float less_high(float x, uint32_t u) {
    float r;
    asm("v_fma_mix_f32 %0, %1, -1.0, %2 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "=v"(r) : "v"(u), "v"(x));
    return r;
  }
};

// The planes of 8 values.
template <typename N, int P>
__device__ __forceinline__ void planes_of(const float (&v)[8], frag (&out)[P]) {
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = v[e];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      w[e] = N::pack(x[2 * e], x[2 * e + 1]);
      if (p + 1 < P) {
        x[2 * e] = N::less_low(x[2 * e], w[e]);
        x[2 * e + 1] = N::less_high(x[2 * e + 1], w[e]);
      }
    }
    out[p] = frag{w[0], w[1], w[2], w[3]};
  }
}

// c + a b over all planes that count, the small ones first.
template <typename N, int PA, int PB>
__device__ __forceinline__ f32x16 mma_planes(const frag (&a)[PA], const frag (&b)[PB], f32x16 c) {
  constexpr int TOP = (PA > PB ? PA : PB) - 1;
#pragma unroll
  for (int s = TOP; s >= 0; --s)
#pragma unroll
    for (int p = 0; p < PA; ++p)
      if (s - p >= 0 && s - p < PB) c = N::mma(a[p], b[s - p], c);
  return c;
}

// ---- rows in memory -------------------------------------------------------------
// 8 elements of a row as they lie there.
template <typename T>
struct Unit {
  T v[8];
};
// A row's address that went between lanes as a number.
template <typename T>
__device__ __forceinline__ const T* global_row(uint64_t at) {
  return (const T*)(const __attribute__((address_space(1))) T*)at;
}
// Elements d .. d + 7 of a row of `dim`, with the row's first ones in the place of those behind it.  UNITS: dim is a multiple
// of 8.  Enough for a tile: what is behind the row meets zeros in a contraction, or makes results that are not stored; if it
// is not finite, nor are sums that are, and the tile is done again carefully.
template <bool UNITS, typename T>
__device__ __forceinline__ Unit<T> load_unit(const T* row, int d, int dim) {
  Unit<T> u;
  if constexpr (UNITS) {
    __builtin_memcpy(&u, row + (d < dim ? d : 0), sizeof(u));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) u.v[e] = row[d + e < dim ? d + e : 0];
  }
  return u;
}
// The same with zeros behind the row: a wave's own operands.  By masks whose value the compiler cannot see: it would
// branch around each load's zeros, and wait for the load there (13 ragged streams x 6 heads x 48, 80 float32 over a cache: 31 us for 26).
template <bool UNITS, typename T>
__device__ __forceinline__ Unit<T> load_own(const T* row, int d, int dim) {
  using Bits = std::conditional_t<sizeof(T) == 2, uint16_t, uint32_t>;
  Unit<T> u = load_unit<UNITS>(row, d, dim);
  if constexpr (UNITS) {
    uint32_t mask = d < dim ? ~0u : 0u, x[sizeof(u) / 4];
    asm("" : "+v"(mask));
    __builtin_memcpy(x, &u, sizeof(u));
#pragma unroll
    for (uint32_t& w : x) w &= mask;
    __builtin_memcpy(&u, x, sizeof(u));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      uint32_t mask = d + e < dim ? ~0u : 0u;
      asm("" : "+v"(mask));
      u.v[e] = __builtin_bit_cast(T, (Bits)(__builtin_bit_cast(Bits, u.v[e]) & (Bits)mask));
    }
  }
  return u;
}
template <typename T>
__device__ __forceinline__ void frags_of(const Unit<T>& u, frag (&out)[Num<T>::IN]) {
  if constexpr (Num<T>::IN == 1) {
    __builtin_memcpy(&out[0], &u, sizeof(frag));
  } else {
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = u.v[e];
    planes_of<Num<T>>(x, out);
  }
}

// ---- tiles in LDS ------------------------------------------------------------------
// A tile of rows of D (32, 64, 96 or 128) elements, in planes, read by rows and by columns.
// Rows of P = 64 or 128 elements are not padded; their 16-byte chunks are exchanged, chunk c of row r lying
// at c ^ turn(r), so that both reads meet every bank once: of 16 consecutive rows one
// chunk each, and of four rows (from a multiple of four) four chunks each.  (Rows padded by 16 bytes: the
// column reads meet half of the banks twice, 16384 tokens x 16 heads x 128 bfloat16 1.94 ms.)
template <typename T, int ROWS, int D>
struct Tile {
  static constexpr int P = D <= 64 ? 64 : 128;
  static constexpr int PLANE = ROWS * P;
  alignas(16) uint16_t at[Num<T>::IN * PLANE];

  static __device__ __forceinline__ int turn(int r) {
    return P == 128 ? (r & 3) << 2 | (r >> 2 & 3) : (r >> 1 & 1) << 2 | (r >> 2 & 3);
  }
  // d: a multiple of 8
  __device__ __forceinline__ void put(int row, int d, const Unit<T>& u) {
    frag f[Num<T>::IN];
    frags_of(u, f);
#pragma unroll
    for (int p = 0; p < Num<T>::IN; ++p) *(frag*)(at + p * PLANE + row * P + (d ^ turn(row) * 8)) = f[p];
  }
  // Units first, first + STEP, .. of the tile (STEP threads take the units of whole rows): row and element of the first
  // and u are apart, which keeps the addresses few.
  template <int STEP, int U>
  __device__ __forceinline__ void put_all(int first, const Unit<T> (&x)[U]) {
    constexpr int PER_ROW = P / 8, ROWS_STEP = STEP / PER_ROW;
    static_assert(STEP % PER_ROW == 0 && (ROWS_STEP & (ROWS_STEP - 1)) == 0, "turn(a + b) = turn(a) ^ turn(b) where no bit is in both");
    const int row = first / PER_ROW, at0 = row * P + (first % PER_ROW ^ turn(row)) * 8;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      frag f[Num<T>::IN];
      frags_of(x[u], f);
#pragma unroll
      for (int p = 0; p < Num<T>::IN; ++p)
        *(frag*)(at + p * PLANE + (at0 ^ turn(u * ROWS_STEP) * 8) + u * ROWS_STEP * P) = f[p];
    }
  }
  // Rows row0 + l (row0 a multiple of 32), elements 16 step + 8 h ..: the operand whose rows are the tile's.
  __device__ __forceinline__ void rows(int row0, int step, int lane, frag (&out)[Num<T>::IN]) const {
    const int l = lane & 31, x = (turn(l) ^ (lane >> 5)) * 8;
#pragma unroll
    for (int p = 0; p < Num<T>::IN; ++p) out[p] = *(const frag*)(at + p * PLANE + row0 * P + l * P + (x ^ 16 * step));
  }
  // Columns d0 + l (d0 a multiple of 32) of rows row0 + 4 h .. + 3 and row0 + 8 + 4 h .. + 3 (row0 a multiple of 16): the
  // operand that is contracted with a result's registers.
  __device__ __forceinline__ void cols(int row0, int d0, int lane, frag (&out)[Num<T>::IN]) const {
    const int l16 = lane & 15, r = 4 * (lane >> 5) + (l16 >> 2);
    const int c = 16 * ((lane >> 4) & 1) + 8 * (l16 >> 1 & 1);
    const int x = (c ^ turn(r) * 8) + 4 * (l16 & 1), y = (c ^ turn(r + 8) * 8) + 4 * (l16 & 1);
#pragma unroll
    for (int p = 0; p < Num<T>::IN; ++p) {
      const uint16_t* p0 = at + p * PLANE + row0 * P + r * P;
      const uint2 a = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(p0 + (x ^ d0))));
      const uint2 b = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(p0 + 8 * P + (y ^ d0))));
      out[p] = frag{a.x, a.y, b.x, b.y};
    }
  }
};

// Direct loads of a tile (16-bit types, rows of D elements, 16-byte aligned): unit u of NT threads is the LDS chunk
// u * NT + thread; which chunk of which row that holds is the row's turn, the same for all of a thread's units, which
// lie STEP rows apart.
template <int D, int NT = 256>
struct DirectUnit {
  static constexpr int P = D <= 64 ? 64 : 128, STEP = NT / (P / 8);
  int row, chunk;    // of the first unit
  __device__ __forceinline__ DirectUnit(int tid) {
    row = tid / (P / 8);
    chunk = (tid % (P / 8)) ^ Tile<bf16, 64, D>::turn(row);
  }
  // The unit's byte of a row of `dim` elements.  Chunks behind it hold the first one: they meet zeros in a contraction,
  // or results that are not stored.
  __device__ __forceinline__ int byte(int dim) const { return 8 * chunk < dim ? 16 * chunk : 0; }
};
static_assert(DirectUnit<128>::STEP % 16 == 0 && DirectUnit<64>::STEP % 16 == 0, "turns repeat every 16 rows");
__device__ __forceinline__ uint32_t lds_byte(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}
// As lds_load16, from an address of each lane's own.
__device__ __forceinline__ void lds_load16_at(const void* p, uint32_t to) {
  const uint32_t m0 = (uint32_t)__builtin_amdgcn_readfirstlane((int)to);
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(p), "s"(m0) : "memory", "m0");
}
// Waits for this wave's direct loads; a barrier behind it makes them everybody's.
__device__ __forceinline__ void direct_wait() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(WaitVmLgkm<0>::imm);
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// ---- lanes ------------------------------------------------------------------------
// The same lane's value of the other half of the wave, in one of two results.
__device__ __forceinline__ void both_halves(float x, float& lo, float& hi) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  lo = __uint_as_float(r[0]);
  hi = __uint_as_float(r[1]);
}
__device__ __forceinline__ float max_halves(float x) {
  float a, b;
  both_halves(x, a, b);
  return fmaxf(a, b);
}
__device__ __forceinline__ float add_halves(float x) {
  float a, b;
  both_halves(x, a, b);
  return a + b;
}
// Row 8 (r / 4) + 4 h + r % 4 of a result's register r.
__device__ __forceinline__ int row_of(int r, int h) { return 8 * (r >> 2) + 4 * h + (r & 3); }
// x, or -inf where `off`, inside a rare branch: the compiler would rather take the masks' instructions of every
// tile, a quarter of its vector instructions.  Results are always assigned, s[r] = masked(s[r], off), never by
// `if (off) s[r] = ..`: where `off` had a load behind ||, hipcc 7.2 left such an assignment to a result of 16 registers out
// (the branch's body was empty, and the register that held -inf was overwritten by the copy of the others).
__device__ __forceinline__ float masked(float x, bool off, float to = -INFINITY) {
  float y = off ? to : x;
  asm volatile("" : "+v"(y));
  return y;
}
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// The thread's number, from which nothing is computed before this place: the registers of a workgroup's loop over
// tiles are full, and values made in front of it would be spilled, to be waited for behind loads in flight.
__device__ __forceinline__ int thread_here() {
  int t = threadIdx.x;
  asm volatile("" : "+v"(t));
  return t;
}

// Four values side by side in memory, where they exist (`have` of them).
template <typename T>
__device__ __forceinline__ void store4(T* to, const float (&x)[4], int have) {
  if (have >= 4) {
    T t[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) t[e] = from_f32<T>(x[e]);
    __builtin_memcpy(to, t, sizeof(t));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < have) to[e] = from_f32<T>(x[e]);
  }
}

// Whether a tensor's rows can be loaded to LDS directly: 16-byte aligned, a tile's offsets in 32 bits.
inline bool direct_rows(const void* p, int64_t ts, int64_t hs) {
  return ((uintptr_t)p | (uintptr_t)(ts * 2) | (uintptr_t)(hs * 2)) % 16 == 0 && ts < (1 << 23);
}
// How a call meets the kernels: the width D of tiles and results, and whether dims are multiples of 8 (and 16-bit
// rows can be loaded to LDS directly), or any.
enum FitMode { ANY, UNITS };
struct Fit {
  int D;
  FitMode mode;
};
template <typename T>
Fit fit_of(const AttnArgs& a, bool cache, bool rows = false) {
  const int big = a.dk > a.dv ? a.dk : a.dv;
  bool units = a.dk % 8 == 0 && a.dv % 8 == 0;
  if (sizeof(T) == 2) {
    units = units && direct_rows(a.k.p, a.k.ts, a.k.hs) && direct_rows(a.v.p, a.v.ts, a.v.hs);
    if (rows) units = units && direct_rows(a.q.p, a.q.ts, a.q.hs) && direct_rows(a.d_o.p, a.d_o.ts, a.d_o.hs);
    if (cache)
      for (const AttnCache* c : {&a.pages.k, &a.pages.v})
        units = units && direct_rows(c->p, c->token_stride, c->head_stride) && c->page_stride % 8 == 0 && c->page_stride < (1LL << 31);
  }
  const int step = units ? 32 : 64;
  return {(big + step - 1) / step * step, units ? UNITS : ANY};
}
// f(D, mode) as constants.
template <typename F>
void by_fit(const Fit& fit, F&& f) {
  using Units = std::integral_constant<FitMode, UNITS>;
  using Any = std::integral_constant<FitMode, ANY>;
  if (fit.mode == UNITS) {
    if (fit.D == 32) f(std::integral_constant<int, 32>{}, Units{});
    else if (fit.D == 64) f(std::integral_constant<int, 64>{}, Units{});
    else if (fit.D == 96) f(std::integral_constant<int, 96>{}, Units{});
    else f(std::integral_constant<int, 128>{}, Units{});
  } else {
    if (fit.D == 64) f(std::integral_constant<int, 64>{}, Any{});
    else f(std::integral_constant<int, 128>{}, Any{});
  }
}

// What block b of a grid is: parts are the slowest index.  (Blocks go to the eight parts of the card in turn, and a
// part's work depends on its place: beside the heads they would leave some of those idle, 2 x 4000 x 16 (4) heads x 128
// bfloat16 in two parts 527 us for 267.)
struct Block {
  int kvh, split;
  int64_t slot;
};
__device__ __forceinline__ Block block_of(int64_t b, int kv_heads, int64_t slots) {
  const int64_t x = b / kv_heads, split = x / slots;
  return {(int)(b - x * kv_heads), (int)split, x - split * slots};
}

// ---- sequences -----------------------------------------------------------------------
// A sequence's rows are its tokens times the heads that share a key / value head,
// row = token * group + head.  Rows are taken in tiles of B; sequence i has the
// slots from floor(cu[i] group / B) + i, one more than it can need at most, so a
// launch of floor(tokens group / B) + seqs slots holds every tile whatever the
// lengths are, and a slot's sequence is found by search (64 at a time).  Without cu:
// one sequence, or of `seqs` sequences one token each.
struct SeqTile {
  int seq;             // -1: none
  int64_t t0, len, tile;
};
__device__ __forceinline__ int64_t seq_start(const int32_t* cu, int i, int64_t tokens) {
  return min(max((int64_t)cu[i], (int64_t)0), tokens);
}
__device__ __forceinline__ SeqTile find_tile(const int32_t* cu, int seqs, int64_t tokens, int group, int B, int64_t slot) {
  if (!cu) {       // one sequence, or one token of each
    if (seqs <= 1) return {0, 0, tokens, slot};
    const int64_t per = (group + B - 1) / B, i = slot / per;
    return i < seqs ? SeqTile{(int)i, i, 1, slot - i * per} : SeqTile{-1, 0, 0, 0};
  }
  const int lane = threadIdx.x & 63;
  int lo = 0, n = seqs;
  while (true) {
    const int step = (n + 63) >> 6, i = lo + lane * step;
    const bool ok = lane * step < n && seq_start(cu, i, tokens) * group / B + i <= slot;
    const int c = __popcll(__ballot(ok));
    if (c == 0) return {-1, 0, 0, 0};
    lo += (c - 1) * step;
    n = min(step, n - (c - 1) * step);
    if (step == 1) break;
  }
  lo = __builtin_amdgcn_readfirstlane(lo);
  const int64_t t0 = seq_start(cu, lo, tokens), t1 = max(seq_start(cu, lo + 1, tokens), t0);
  // (where the offsets fall, the search can end at a sequence that starts behind the slot)
  const int64_t tile = slot - (t0 * group / B + lo);
  return {tile < 0 ? -1 : lo, t0, t1 - t0, tile};
}

// The sequence of token t (which lies in one): its first token and length.
__device__ __forceinline__ SeqTile find_token(const int32_t* cu, int seqs, int64_t tokens, int64_t t) {
  if (!cu) return {0, 0, tokens, 0};
  int lo = 0, hi = seqs;           // cu[lo] <= t < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (seq_start(cu, mid, tokens) <= t) lo = mid;
    else hi = mid;
  }
  const int64_t t0 = seq_start(cu, lo, tokens);
  return {lo, t0, max(seq_start(cu, lo + 1, tokens) - t0, (int64_t)0), 0};
}

}  // namespace pc
