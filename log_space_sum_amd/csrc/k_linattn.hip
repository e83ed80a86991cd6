// k_linattn.hip -- linear attention with a decay for each head.
//
//   S_t = l S_{t-1} + k_t v_t^T,   o_t = scale q_t^T S_t,   l = exp(log_decay[head])
//
// and its gradients, with the adjoint state D_t = l D_{t+1} + scale q_t do_t^T:
//
//   dq_t = scale S_t do_t,   dk_t = D_t v_t,   dv_t = D_t^T k_t,
//   dS_0 = l D_1,  D_{T+1} = the given gradient of the final state / l
//
// All four are one walk: a state [da, dc] is carried along the tokens, b_t c_t^T
// joins it, and a_t is contracted with it (forward: a, b, c = q, k, v; dq: do,
// v, k on the transposed state; dv: k, q, do and dk: v, do, q, from the end).
// The walk goes in chunks of C tokens.  Inside a chunk, with i, j the tokens
// and n their number,
//
//   o_i = l^{i+off} a_i^T S + sum_{j <= i} l^{i-j} (a_i . b_j) c_j,
//   S  <- l^n S + sum_j l^{n-off-j} b_j c_j^T
//
// are matrix products.  A workgroup of four or eight waves walks one (sequence,
// head); each wave carries 16 columns of the state in its registers for the
// whole walk, in the accumulator layout, in which four consecutive rows lie in one
// lane: with the contraction's order permuted alike on both sides, the same
// registers are the operand of the next product, so the state never passes
// through LDS.  Only the [C, C] products a_i . b_j do (one tile a wave).
//
// Long sequences are cut into segments (a rule on the number of heads and
// sequences, see mix_segments) that walk side by side: one pass makes each
// segment's own state, a scan joins them, and the walk starts from there.
//
// What bounds it: at dim 128 the matrix instructions (busy 36% of the time), the
// vector instructions that split planes (52%) and LDS (51%) share a walk, at 2.6
// TB/s of the tokens' bytes; at dim 64 and below, or with few tokens, the chain
// of chunks.  16384 tokens x 32 heads x 128 bfloat16 (541 MB): segments' states
// 87 us, scan 13, walk 210 when profiled, 262 us together unprofiled.  Measured
// and not taken: waves of 32 columns (the same, 12% slower for float32), the
// state's update before the inside products' barrier (the same at dim 64, 5%
// slower at 128; these with two planes), tiles with exchanged chunks instead of padding (half of the
// bank conflicts, but registers past the limit of two workgroups: the same).
//
// Precision: bfloat16 tensors are multiplied in bfloat16 with float32 sums.
// What is not exact in bfloat16, the decay-weighted l^{n-off-j} c_j, the carried
// state and the inside products (a_i . b_j) l^{i-j}, is split into three
// bfloat16 planes (24 bits), so state and output keep float32 accuracy however
// long the walk.  (Two planes of the state and of the inside products are 6 to 8%
// faster, 252 against 268 us for 16384 x 32 heads x 128, but leave 2^-17 of every
// term: after rounding, outputs 9e-5 off the rounded definition's, 2e-5 with three.)
// float32 and float16 tensors run on the float32 matrix instruction throughout
// (float16's range cannot hold the state or its planes).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "pc_ops.h"

namespace pc {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;

// l^m for m >= 0 (l = 0, that is log_decay -inf, gives 1 at m = 0).
__device__ __forceinline__ float decay_pow(float g, float m) { return m == 0.0f ? 1.0f : expf(g * m); }

// ---- the two compute types -------------------------------------------------
// A "quad" is four consecutive elements of the contracted dimension held by a
// lane: of a 16-wide block, lanes 16 g .. 16 g + 15 hold elements 4 g .. 4 g + 3
// of their row.  mma() multiplies two blocks (32 elements).
template <typename CT>
struct Ops;

template <>
struct Ops<bf16> {
  static constexpr int C = 64;       // tokens of a chunk
  static constexpr int EV = 8;       // elements of a staged unit
  // row padding of the tiles read by rows, and by columns (16 lanes' 4 rows of 32 bytes lie in different banks then);
  // b's tile is read by both in a walk (there the first measured 3% faster)
  static constexpr int PAD = 8, CPAD = 16;
  // planes of the weighted c, of the state in the output's product, and of the inside products
  static constexpr int CPLANES = 3, SPLANES = 3, PPLANES = 3;
  typedef uint2 quad;
  static __device__ __forceinline__ f32x4 mma(quad a0, quad a1, quad b0, quad b1, f32x4 acc) {
    const uint4 a = {a0.x, a0.y, a1.x, a1.y}, b = {b0.x, b0.y, b1.x, b1.y};
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
  }
  static __device__ __forceinline__ quad row(const bf16* p) { return *(const quad*)p; }
  // Tiles read by rows alone are stored so that a lane's two quads of a 32-wide
  // block lie side by side: one 16-byte read.  at(): the place of element j.
  static __device__ __forceinline__ int at(int j) { return (j & ~31) + 8 * ((j >> 2) & 3) + 4 * ((j >> 4) & 1) + (j & 3); }
  static __device__ __forceinline__ void row2(const bf16* r, int block, int g, quad& x, quad& y) {
    const uint4 v = *(const uint4*)(r + 32 * block + 8 * g);
    x = quad{v.x, v.y};
    y = quad{v.z, v.w};
  }
  // Four rows of one column: the 16 lanes of a group hand in 4 x 16 elements,
  // each four consecutive ones, and get back a column each.
  static __device__ __forceinline__ quad col(const bf16* tile, int stride) {
    const int l = threadIdx.x & 63;
    const bf16* p = tile + (4 * (l >> 4) + ((l & 15) >> 2)) * stride + 4 * (l & 3);
    return __builtin_bit_cast(quad, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(p)));
  }
  static __device__ __forceinline__ uint32_t pack(float x, float y) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{x, y}, bf16x2));   // one instruction
  }
  static __device__ __forceinline__ quad round(f32x4 v) { return quad{pack(v[0], v[1]), pack(v[2], v[3])}; }
  static __device__ __forceinline__ f32x4 wide(quad q) {
    return f32x4{__uint_as_float(q.x << 16), __uint_as_float(q.x & 0xffff0000u), __uint_as_float(q.y << 16),
                 __uint_as_float(q.y & 0xffff0000u)};
  }
};

template <>
struct Ops<float> {
  static constexpr int C = 32;
  static constexpr int EV = 4;
  static constexpr int PAD = 4, CPAD = 4;
  static constexpr int CPLANES = 1, SPLANES = 1, PPLANES = 1;
  typedef f32x4 quad;
  static __device__ __forceinline__ f32x4 mma(quad a0, quad a1, quad b0, quad b1, f32x4 acc) {
#pragma unroll
    for (int e = 0; e < 4; ++e) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a0[e], b0[e], acc, 0, 0, 0);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a1[e], b1[e], acc, 0, 0, 0);
    return acc;
  }
  static __device__ __forceinline__ quad row(const float* p) { return *(const quad*)p; }
  static __device__ __forceinline__ int at(int j) { return j; }
  static __device__ __forceinline__ void row2(const float* r, int block, int g, quad& x, quad& y) {
    x = row(r + 32 * block + 4 * g);
    y = row(r + 32 * block + 16 + 4 * g);
  }
  static __device__ __forceinline__ quad col(const float* tile, int stride) {
    const int l = threadIdx.x & 63;
    const float* p = tile + 4 * (l >> 4) * stride + (l & 15);
    return quad{p[0], p[stride], p[2 * stride], p[3 * stride]};
  }
  static __device__ __forceinline__ quad round(f32x4 v) { return v; }
  static __device__ __forceinline__ f32x4 wide(quad q) { return q; }
};

// The planes of four values: planes[0] the rounding, each further one the
// rounding of what is left.
template <typename CT, int P>
__device__ __forceinline__ void split(f32x4 v, typename Ops<CT>::quad (&planes)[P]) {
#pragma unroll
  for (int p = 0; p < P; ++p) {
    planes[p] = Ops<CT>::round(v);
    if (p + 1 < P) v -= Ops<CT>::wide(planes[p]);
  }
}

// How the dims meet the tiles and units: FULL both are tile sizes, UNITS both
// are whole units, ANY neither.
enum Fit { FULL, UNITS, ANY };

// EV elements of a row as loaded, from an address that exists also where the
// row has fewer than `have` (the others are cleared when they are staged).
template <typename IO, int EV>
struct Unit {
  IO v[EV];
};
template <Fit F, typename IO, int EV>
__device__ __forceinline__ Unit<IO, EV> load_unit(const char* base, uint32_t offset, int d, int dim) {
  Unit<IO, EV> u;
  const IO* p = (const IO*)(base + offset);
  if constexpr (F == FULL) {
    __builtin_memcpy(&u, p + d, sizeof(u));
  } else if constexpr (F == UNITS) {
    __builtin_memcpy(&u, p + (d < dim ? d : 0), sizeof(u));
  } else {
#pragma unroll
    for (int e = 0; e < EV; ++e) u.v[e] = p[min(d + e, dim - 1)];
  }
  return u;
}
template <Fit F, typename IO, int EV>
__device__ __forceinline__ void clear(Unit<IO, EV>& u, bool row, int d, int dim) {
  if (!row || (F == UNITS && d >= dim)) u = Unit<IO, EV>{};
  if constexpr (F == ANY) {
#pragma unroll
    for (int e = 0; e < EV; ++e)
      if (d + e >= dim) u.v[e] = IO{};
  }
}

// Whether a unit holds a value that is not finite (an exponent of ones).
template <int EV>
__device__ __forceinline__ bool not_finite(const Unit<bf16, EV>& u) {
  uint32_t w[EV / 2], r = 0;
  __builtin_memcpy(w, &u, sizeof(w));
#pragma unroll
  for (int e = 0; e < EV / 2; ++e) r |= (w[e] & 0x7f807f80u) + 0x00800080u;   // carries into a half's top bit
  return (r & 0x80008000u) != 0;
}
template <int EV>
__device__ __forceinline__ bool not_finite(const Unit<f16, EV>& u) {
  uint32_t w[EV / 2], r = 0;
  __builtin_memcpy(w, &u, sizeof(w));
#pragma unroll
  for (int e = 0; e < EV / 2; ++e) r |= (w[e] & 0x7c007c00u) + 0x04000400u;
  return (r & 0x80008000u) != 0;
}
template <int EV>
__device__ __forceinline__ bool not_finite(const Unit<float, EV>& u) {
  uint32_t r = 0;
#pragma unroll
  for (int e = 0; e < EV; ++e) r |= (__float_as_uint(u.v[e]) & 0x7f800000u) + 0x00800000u;
  return (r & 0x80000000u) != 0;
}

template <typename CT, typename IO, int EV>
__device__ __forceinline__ void stage(CT* dst, const Unit<IO, EV>& u) {
  if constexpr (std::is_same_v<CT, IO>) {
    __builtin_memcpy(__builtin_assume_aligned(dst, 16), &u, sizeof(u));
  } else {
    f32x4 w;
#pragma unroll
    for (int e = 0; e < EV; ++e) w[e] = to_f32(u.v[e]);
    *(f32x4*)dst = w;
  }
}

// The same into a tile read by rows (elements at Ops::at).
template <typename CT, typename IO, int EV>
__device__ __forceinline__ void stage_rows(CT* row, int d, const Unit<IO, EV>& u) {
  if constexpr (std::is_same_v<CT, bf16>) {
    static_assert(EV == 8, "two quads");
    CT* p = row + Ops<CT>::at(d);
    __builtin_memcpy(__builtin_assume_aligned(p, 8), &u, 8);
    __builtin_memcpy(__builtin_assume_aligned(p + 8, 8), (const char*)&u + 8, 8);   // the next quad's place
  } else {
    stage<CT, IO, EV>(row + d, u);
  }
}

// ---- the walk ---------------------------------------------------------------
// DKB: 16-blocks of the contracted dimension (even); NW: waves, each with 16
// output columns.  WALK false: only the state, from zero, of every segment but
// a sequence's last, into `seg`.
template <typename IO, typename CT, int DKB, int NW, Fit F, bool WALK>
__global__ __launch_bounds__(64 * NW, F != FULL ? 2 : NW == 8 ? 4 : 3) void mix_walk(MixMany many) {
  const MixArgs& m = many.w[blockIdx.z / many.seqs];
  using O = Ops<CT>;
  using quad = typename O::quad;
  constexpr int C = O::C, CB = C / 16, EV = O::EV, NT = 64 * NW;
  constexpr int DA = 16 * DKB, DC = 16 * NW;
  constexpr int LA = DA + O::PAD, LB = DA + (WALK ? O::PAD : O::CPAD), LC = DC + O::CPAD;
  // A plane of the inside products: of every 32 rows the columns up to their
  // last, so that three planes leave room for a third workgroup at dim 64 and a
  // second at 128 (all columns: 57 and 80 KB; the first 70 instead of 63 us for
  // a ragged forward of 24 x 1500 x 16 heads).
  constexpr int SPZ = 512 * CB / 2 * (CB / 2 + 1) + 16 * CB * O::PAD;
  auto sp_row = [](int i) { return 512 * (i >> 5) * ((i >> 5) + 1) + 32 * (i >> 5) * O::PAD + (i & 31) * (32 * ((i >> 5) + 1) + O::PAD); };
  constexpr int UA = C * DA / EV / NT, UC = C * DC / EV / NT;   // staged units of a thread
  static_assert(UA * NT * EV == C * DA && UC * NT * EV == C * DC, "whole units");
  constexpr int CP = O::CPLANES, SP = O::SPLANES, PP = O::PPLANES;
  constexpr int PAIRS = CB * (CB + 1) / 2, MINE = (PAIRS + NW - 1) / NW;
  __shared__ __align__(16) CT sa[WALK ? C * LA : 8];
  __shared__ __align__(16) CT sb[C * LB];
  __shared__ __align__(16) CT sc[C * LC];
  __shared__ __align__(16) CT sp[WALK ? PP * SPZ : 8];
  // weights: of a token's part in the state (for the chunk's size), of the
  // inside products at distance d = i - j (at C - 1 - d; 0 behind C - 1), and
  // of the state in token i's output
  __shared__ __align__(16) float swt[C], sdec[C + 16], siw[C];
  __shared__ int sbad[2];

  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, g = lane >> 4, l16 = lane & 15;
  const int head = blockIdx.x, seq = blockIdx.z % many.seqs;
  int sgm = blockIdx.y;
  int64_t t0 = 0, t1 = m.tokens;
  if (m.cu) {
    t0 = min(max((int64_t)m.cu[seq], (int64_t)0), m.tokens);
    t1 = min(max((int64_t)m.cu[seq + 1], t0), m.tokens);
  }
  const int64_t len = t1 - t0;
  const int64_t live = min(max((len + m.seglen - 1) / m.seglen, (int64_t)1), (int64_t)m.nsegs);
  if (sgm >= live || (!WALK && sgm == live - 1)) return;
  const int64_t pos0 = (int64_t)sgm * m.seglen, pos1 = sgm == live - 1 ? len : pos0 + m.seglen;

  const float gam = m.log_decay[head];
  const IO* pa = (const IO*)m.a.p + (int64_t)(head / m.a.div) * m.a.hs;
  const IO* pb = (const IO*)m.b.p + (int64_t)(head / m.b.div) * m.b.hs;
  const IO* pc = (const IO*)m.c.p + (int64_t)(head / m.c.div) * m.c.hs;
  const int da = F == FULL ? DA : m.da, dc = F == FULL ? DC : m.dc;
  const int64_t elems = (int64_t)da * dc;
  const int col = wave * 16 + l16;         // this lane's column of the state
  const bool wave_on = F == FULL || wave * 16 < dc;

  // the carried state: lane l16 of group g holds rows 16 kb + 4 g + r of its column
  f32x4 st[DKB];
  {
    const float* from = nullptr;
    if (WALK) from = live > 1 ? m.seg + ((seg_slot(m.packed, m.nsegs, m.seglen, seq, t0) + sgm) * m.heads + head) * elems
                              : (m.init ? m.init + ((int64_t)seq * m.heads + head) * elems : nullptr);
#pragma unroll
    for (int kb = 0; kb < DKB; ++kb) {
      const int row = 16 * kb + 4 * g;
      st[kb] = f32x4{};
      if (!from) continue;
      if (m.st_r == 1 && (F == FULL || (row + 4 <= da && col < dc))) {
        __builtin_memcpy(&st[kb], from + row + (int64_t)col * m.st_c, 16);   // transposed: a lane's rows lie side by side
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (F == FULL || (row + r < da && col < dc)) st[kb][r] = from[(row + r) * m.st_r + col * m.st_c];
      }
    }
  }
  if constexpr (WALK) {
    for (int e = tid; e < C + 16; e += NT) sdec[e] = e < C ? m.pscale * decay_pow(gam, (float)(C - 1 - e)) : 0.0f;
    for (int e = tid; e < C; e += NT) siw[e] = m.oscale * decay_pow(gam, (float)(e + m.off));
    // the products' tiles right of the diagonal that a 32-wide step reads: always 0
    for (int e = tid; e < PP * C * 16; e += NT) {
      const int i = (e >> 4) % C, ib = i >> 4;
      if ((ib & 1) == 0) sp[e / (C * 16) * SPZ + sp_row(i) + O::at(16 * (ib + 1) + (e & 15))] = CT{};
    }
  }

  // Rows pos .. pos + n - 1 (n >= 1); a row behind them loads one of them.
  // The base is uniform, a lane's offset 32 bits wide.
  Unit<IO, EV> ra[WALK ? UA : 1], rb[UA], rc[UC];
  const uint32_t a_row = (uint32_t)(m.a.ts * sizeof(IO)), b_row = (uint32_t)(m.b.ts * sizeof(IO)),
                 c_row = (uint32_t)(m.c.ts * sizeof(IO));
  auto fetch = [&](int64_t pos, int n) {
    const int64_t first = m.rev ? t1 - pos - n : t0 + pos;
    const char *qa = (const char*)(pa + first * m.a.ts), *qb = (const char*)(pb + first * m.b.ts),
               *qc = (const char*)(pc + first * m.c.ts);
#pragma unroll
    for (int u = 0; u < UA; ++u) {
      const int id = u * NT + tid, i = min(id / (DA / EV), n - 1), d = id % (DA / EV) * EV;
      const uint32_t r = (uint32_t)(m.rev ? n - 1 - i : i);
      if constexpr (WALK) ra[u] = load_unit<F, IO, EV>(qa, r * a_row, d, da);
      rb[u] = load_unit<F, IO, EV>(qb, r * b_row, d, da);
    }
#pragma unroll
    for (int u = 0; u < UC; ++u) {
      const int id = u * NT + tid, i = min(id / (DC / EV), n - 1), d = id % (DC / EV) * EV;
      const uint32_t r = (uint32_t)(m.rev ? n - 1 - i : i);
      rc[u] = load_unit<F, IO, EV>(qc, r * c_row, d, dc);
    }
  };

  if (tid < 2) sbad[tid] = 0;
  __syncthreads();
  int turn = 0;
  float ln = 1.0f;
  int wn = -1;             // the chunk size that ln and swt are of
  int64_t single = pos0;   // tokens before this position go one by one
  int64_t pos = pos0;
  if (pos < pos1) fetch(pos, (int)min((int64_t)C, pos1 - pos));
  while (pos < pos1) {
    int n = pos < single ? 1 : (int)min((int64_t)C, pos1 - pos);
    auto clear_tail = [&] {
      if (F == FULL && n == C) return;
#pragma unroll
      for (int u = 0; u < UA; ++u) {
        const int id = u * NT + tid, i = id / (DA / EV), d = id % (DA / EV) * EV;
        if constexpr (WALK) clear<F>(ra[u], i < n, d, da);
        clear<F>(rb[u], i < n, d, da);
      }
#pragma unroll
      for (int u = 0; u < UC; ++u) {
        const int id = u * NT + tid, i = id / (DC / EV), d = id % (DC / EV) * EV;
        clear<F>(rc[u], i < n, d, dc);
      }
    };
    clear_tail();
    // A value that is not finite would reach the tokens before it in the chunk
    // through a zero product: such a chunk is walked token by token.
    bool bad = false;
    if (n > 1) {
#pragma unroll
      for (int u = 0; u < UC; ++u) bad |= not_finite(rc[u]);
    }
    if (bad) sbad[turn] = 1;
    __syncthreads();               // (also: every wave is done with the last chunk's tiles)
    const bool any = sbad[turn] != 0;
    turn ^= 1;
    if (tid == 0) sbad[turn] = 0;  // the next chunk's, written behind the next barrier
    if (any) {
      single = pos + n;
      n = 1;
      fetch(pos, n);
      clear_tail();
    }
#pragma unroll
    for (int u = 0; u < UA; ++u) {
      const int id = u * NT + tid, i = id / (DA / EV), d = id % (DA / EV) * EV;
      if constexpr (WALK) stage_rows<CT, IO, EV>(sa + i * LA, d, ra[u]);
      stage<CT, IO, EV>(sb + i * LB + d, rb[u]);
    }
#pragma unroll
    for (int u = 0; u < UC; ++u) {
      const int id = u * NT + tid;
      stage<CT, IO, EV>(sc + id / (DC / EV) * LC + id % (DC / EV) * EV, rc[u]);
    }
    if (n != wn) {
      wn = n;
      ln = decay_pow(gam, (float)n);
      if (tid < C) swt[tid] = tid < n ? m.wscale * decay_pow(gam, (float)(n - m.off - tid)) : 0.0f;
    }
    __syncthreads();
    const int64_t next = pos + n;
    // The next chunk's rows, in flight over this chunk (with eight waves, whose
    // registers are fewer, over its second half).  Behind the last chunk: its
    // last row again, since under a condition the loads would wait for each
    // other.
    constexpr bool EARLY = NW == 4 || !WALK;
    auto fetch_next = [&] {
      fetch(min(next, pos1 - 1), next < single ? 1 : (int)min((int64_t)C, max(pos1 - next, (int64_t)1)));
    };
    if (EARLY) fetch_next();
    f32x4 o[WALK ? CB : 1];
    if constexpr (WALK) {
      // inside products b_j . a_i, transposed: a lane holds four j of one i
#pragma unroll
      for (int k = 0; k < MINE; ++k) {
        int ib = 0, jb = wave + NW * k;
        while (jb > ib) jb -= ++ib;   // pair number -> (ib, jb), jb <= ib
        if (wave + NW * k < PAIRS) {
          f32x4 acc = {};
          const CT* rj = sb + (16 * jb + l16) * LB + 4 * g;
          const CT* ri = sa + (16 * ib + l16) * LA;
#pragma unroll
          for (int kb = 0; kb < DKB; kb += 2) {
            quad a0, a1;
            O::row2(ri, kb / 2, g, a0, a1);
            acc = O::mma(O::row(rj + 16 * kb), O::row(rj + 16 * kb + 16), a0, a1, acc);
          }
          const float* dec = sdec + C - 1 - 16 * (ib - jb) - l16 + 4 * g;
          const int ahead = ib == jb ? l16 - 4 * g : C;   // elements behind it are later tokens
          f32x4 w = {dec[0], dec[1], dec[2], dec[3]};
          w *= acc;
#pragma unroll
          for (int r = 0; r < 4; ++r) w[r] = r > ahead ? 0.0f : w[r];
          quad pl[PP];
          split<CT, PP>(w, pl);
#pragma unroll
          for (int p = 0; p < PP; ++p) *(quad*)(sp + p * SPZ + sp_row(16 * ib + l16) + O::at(16 * jb + 4 * g)) = pl[p];
        }
      }
      // the state's part of the output
#pragma unroll
      for (int ib = 0; ib < CB; ++ib) o[ib] = f32x4{};
      if (wave_on) {
#pragma unroll
        for (int kb = 0; kb < DKB; kb += 2) {
          quad s0[SP], s1[SP];
          split<CT, SP>(st[kb], s0);
          split<CT, SP>(st[kb + 1], s1);
          quad a0[CB], a1[CB];
#pragma unroll
          for (int ib = 0; ib < CB; ++ib) {
            O::row2(sa + (16 * ib + l16) * LA, kb / 2, g, a0[ib], a1[ib]);
          }
#pragma unroll
          for (int p = SP - 1; p >= 0; --p)
#pragma unroll
            for (int ib = 0; ib < CB; ++ib) o[ib] = O::mma(s0[p], s1[p], a0[ib], a1[ib], o[ib]);
        }
#pragma unroll
        for (int ib = 0; ib < CB; ++ib) o[ib] *= siw[16 * ib + l16];
      }
      __syncthreads();
    }
    if (!EARLY) fetch_next();
    if (wave_on) {
#pragma unroll
      for (int kb = 0; kb < DKB; ++kb) st[kb] *= ln;
#pragma unroll
      for (int b = 0; b < CB; b += 2) {
        quad w0[CP], w1[CP];
        const quad c0 = O::col(sc + 16 * b * LC + wave * 16, LC);
        const quad c1 = O::col(sc + (16 * b + 16) * LC + wave * 16, LC);
        split<CT, CP>(O::wide(c0) * *(const f32x4*)(swt + 16 * b + 4 * g), w0);
        split<CT, CP>(O::wide(c1) * *(const f32x4*)(swt + 16 * b + 16 + 4 * g), w1);
        if constexpr (WALK) {
#pragma unroll
          for (int p = PP - 1; p >= 0; --p)
#pragma unroll
            for (int ib = b; ib < CB; ++ib) {
              quad p0, p1;
              O::row2(sp + p * SPZ + sp_row(16 * ib + l16), b / 2, g, p0, p1);
              o[ib] = O::mma(c0, c1, p0, p1, o[ib]);
            }
        }
        // (four blocks of rows side by side: no product waits for the one before it)
        constexpr int KG = 2;
#pragma unroll
        for (int k0 = 0; k0 < DKB; k0 += KG) {
          quad b0[KG], b1[KG];
#pragma unroll
          for (int k = 0; k < KG; ++k) {
            b0[k] = O::col(sb + 16 * b * LB + 16 * (k0 + k), LB);
            b1[k] = O::col(sb + (16 * b + 16) * LB + 16 * (k0 + k), LB);
          }
#pragma unroll
          for (int p = CP - 1; p >= 0; --p)
#pragma unroll
            for (int k = 0; k < KG; ++k) st[k0 + k] = O::mma(b0[k], b1[k], w0[p], w1[p], st[k0 + k]);
        }
      }
      if constexpr (WALK) {
        // transposed outputs: a lane holds four columns of one token
        const int oc = wave * 16 + 4 * g, have = dc - oc;
        const int64_t base = (m.rev ? t1 - pos - n : t0 + pos) * m.o_ts + (int64_t)head * m.o_hs;
#pragma unroll
        for (int ib = 0; ib < CB; ++ib) {
          const int i = 16 * ib + l16;
          if (i >= n || (F != FULL && have <= 0)) continue;
          const uint32_t at = (uint32_t)(m.rev ? n - 1 - i : i) * (uint32_t)m.o_ts + oc;
          if (m.out_f32) {
            float* q = (float*)m.out + base + at;
            if (F == FULL || have >= 4) {
              __builtin_memcpy(q, &o[ib], 16);
            } else {
              for (int r = 0; r < have; ++r) q[r] = o[ib][r];
            }
          } else {
            IO* q = (IO*)m.out + base + at;
            IO w[4];
            if constexpr (std::is_same_v<IO, bf16>) {
              const uint2 two = O::round(o[ib]);
              __builtin_memcpy(w, &two, 8);
            } else {
#pragma unroll
              for (int r = 0; r < 4; ++r) w[r] = from_f32<IO>(o[ib][r]);
            }
            if (F == FULL || have >= 4) {
              __builtin_memcpy(q, w, sizeof(w));
            } else {
              for (int r = 0; r < have; ++r) q[r] = w[r];
            }
          }
        }
      }
    }
    pos = next;
  }

  float* to = nullptr;
  if (!WALK) to = m.seg + ((seg_slot(m.packed, m.nsegs, m.seglen, seq, t0) + sgm) * m.heads + head) * elems;
  else if (m.fin && sgm == live - 1) to = m.fin + ((int64_t)seq * m.heads + head) * elems;
  if (!to) return;
#pragma unroll
  for (int kb = 0; kb < DKB; ++kb)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * kb + 4 * g + r;
      if (F == FULL || (row < da && col < dc)) to[row * m.st_r + col * m.st_c] = st[kb][r];
    }
}

// The states at the segments' starts from the segments' own states, in place
// (bound by the states' bytes: 16 segments x 32 heads x 128 x 128, 13 us or 5 TB/s):
// start_0 = init, start_{s+1} = l^seglen start_s + own_s.
// EV elements a thread; four segments' loads in flight.  A sequence of one
// segment walks from its given state.
template <int EV>
__global__ __launch_bounds__(256) void mix_scan(MixScanArgs m0, MixScanArgs m1) {
  const MixScanArgs& m = (int)blockIdx.z < m0.seqs ? m0 : m1;
  const int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * EV;
  const int head = blockIdx.y, seq = blockIdx.z % m0.seqs;
  if (e >= m.elems) return;
  int64_t t0 = 0, t1 = m.tokens;
  if (m.cu) {
    t0 = min(max((int64_t)m.cu[seq], (int64_t)0), m.tokens);
    t1 = min(max((int64_t)m.cu[seq + 1], t0), m.tokens);
  }
  const int live = (int)min(max((t1 - t0 + m.seglen - 1) / m.seglen, (int64_t)1), (int64_t)m.nsegs);
  if (live == 1) return;
  const float ls = decay_pow(m.log_decay[head], (float)m.seglen);
  float* p = m.seg + (seg_slot(m.packed, m.nsegs, m.seglen, seq, t0) * m.heads + head) * m.elems + e;
  const int64_t step = (int64_t)m.heads * m.elems;
  struct Some {
    float v[EV];
  } run = {}, own[4];
  if (m.init) __builtin_memcpy(&run, m.init + ((int64_t)seq * m.heads + head) * m.elems + e, sizeof(run));
  // (the last segment's own state is not needed, nor made: its place is loaded and not used)
  for (int s0 = 0; s0 < live; s0 += 4) {
#pragma unroll
    for (int k = 0; k < 4; ++k) __builtin_memcpy(&own[k], p + min(s0 + k, live - 1) * step, sizeof(run));
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (s0 + k >= live) break;
      __builtin_memcpy(p + (s0 + k) * step, &run, sizeof(run));
#pragma unroll
      for (int v = 0; v < EV; ++v) run.v[v] = run.v[v] * ls + own[k].v[v];
    }
  }
}

// Gradients of shared key / value heads (bound by the partial sums' bytes): the sum over the heads that share one,
// in their order.  Only tokens of the sequences are written.  (A launch takes fewer than 2^32 threads: past
// MIX_SUM_BLOCKS blocks each takes several pieces.)
constexpr int64_t MIX_SUM_BLOCKS = 1 << 22;
template <typename IO>
__global__ __launch_bounds__(256) void mix_sum(MixSumArgs m0, MixSumArgs m1) {
  const MixSumArgs& m = blockIdx.y ? m1 : m0;
  const int per = m.kv_heads * m.dim;
  int64_t t0 = 0, t1 = m.tokens;
  if (m.cu) {
    t0 = min(max((int64_t)m.cu[0], (int64_t)0), m.tokens);
    t1 = min(max((int64_t)m.cu[m.seqs], t0), m.tokens);
  }
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < (t1 - t0) * per; e += (int64_t)gridDim.x * 256) {
    const int64_t t = t0 + e / per;
    const int h = (int)(e % per) / m.dim, d = (int)(e % per) % m.dim;
    const float* p = m.part + (t * m.kv_heads + h) * (int64_t)m.group * m.dim + d;
    float s = 0.0f;
    for (int k = 0; k < m.group; ++k) s += p[(int64_t)k * m.dim];
    ((IO*)m.out)[t * m.o_ts + (int64_t)h * m.o_hs + d] = from_f32<IO>(s);
  }
}

// ---- single tokens ----------------------------------------------------------
// One workgroup per (row, head): the state is read, updated, written and
// contracted with q in one pass; bound by the state's bytes (256 rows x 32
// heads x 128 x 128: 207 us, 5.2 TB/s, the rate of a copy).  CV columns a
// thread, the rows dealt out over the workgroup's row groups, whose partial
// outputs are added in a fixed order.  Rows that name the same slot are
// successive tokens of that state: the first of them does them all, in order.
constexpr int MIX_STEP_ROWS = 32768;   // rows of a launch's second dimension; more go along the third
template <typename IO, int CV>
__global__ __launch_bounds__(256) void mix_step(MixStepArgs m) {
  const int64_t at = (int64_t)blockIdx.z * MIX_STEP_ROWS + blockIdx.y;
  if (at >= m.batch) return;
  const int head = blockIdx.x, first = (int)at, tid = threadIdx.x;
  const int kv = head / m.group;
  const int slot = m.slot ? m.slot[first] : first;
  if (slot < 0 || slot >= m.slots) return;
  if (m.slot) {
    bool seen = false;
    for (int b = tid; b < first; b += 256) seen |= m.slot[b] == slot;
    if (__syncthreads_or(seen)) return;
  }
  __shared__ float sq[MIX_MAX_DIM], sk[MIX_MAX_DIM], sv[MIX_MAX_DIM];
  __shared__ float part[256 * CV];
  const int across = (m.dv + CV - 1) / CV;          // threads of a row
  int lanes = 1;
  while (lanes < across) lanes *= 2;
  const int groups = 256 / lanes, grp = tid / lanes, col = tid % lanes * CV;
  const bool on = col < m.dv;
  const float lam = expf(m.log_decay[head]);
  float* s = m.state + ((int64_t)slot * m.heads + head) * m.dk * m.dv + col;
  int row = first;
  for (;;) {
    if (tid < m.dk) {
      sq[tid] = m.scale * to_f32(((const IO*)m.q)[(int64_t)row * m.q_ts + (int64_t)head * m.q_hs + tid]);
      sk[tid] = to_f32(((const IO*)m.k)[(int64_t)row * m.k_ts + (int64_t)kv * m.k_hs + tid]);
    } else if (tid >= 128 && tid - 128 < m.dv) {
      sv[tid - 128] = to_f32(((const IO*)m.v)[(int64_t)row * m.v_ts + (int64_t)kv * m.v_hs + tid - 128]);
    }
    float o[CV];
#pragma unroll
    for (int c = 0; c < CV; ++c) o[c] = 0.0f;
    __syncthreads();
    if (on) {
      float v[CV];
#pragma unroll
      for (int c = 0; c < CV; ++c) v[c] = col + c < m.dv ? sv[col + c] : 0.0f;
#pragma unroll 4
      for (int r = grp; r < m.dk; r += groups) {
        float x[CV];
        float* p = s + (int64_t)r * m.dv;
        if (CV == 4) __builtin_memcpy(x, p, 4 * CV);
        else x[0] = p[0];
#pragma unroll
        for (int c = 0; c < CV; ++c) {
          x[c] = lam * x[c] + sk[r] * v[c];
          o[c] += sq[r] * x[c];
        }
        if (CV == 4) __builtin_memcpy(p, x, 4 * CV);
        else p[0] = x[0];
      }
    }
#pragma unroll
    for (int c = 0; c < CV; ++c) part[tid * CV + c] = o[c];
    __syncthreads();
    if (tid < m.dv) {
      float t = 0.0f;
      for (int k = 0; k < groups; ++k) t += part[k * lanes * CV + tid];
      ((IO*)m.o)[(int64_t)row * m.o_ts + (int64_t)head * m.o_hs + tid] = from_f32<IO>(t);
    }
    if (!m.slot) return;
    // the next row of this slot
    __shared__ int nextrow;
    if (tid == 0) nextrow = m.batch;
    __syncthreads();
    for (int b = row + 1 + tid; b < m.batch; b += 256)
      if (m.slot[b] == slot) {
        atomicMin(&nextrow, b);
        break;
      }
    __syncthreads();
    row = nextrow;
    if (row >= m.batch) return;
    __syncthreads();
  }
}

template <typename IO, typename CT, bool WALK, int DKB, int NW>
void walk_fit(const MixMany& a, dim3 grid, hipStream_t s) {
  constexpr int EV = Ops<CT>::EV;
  const int da = a.w[0].da, dc = a.w[0].dc;
  if (da == 16 * DKB && dc == 16 * NW) launch_kernel(mix_walk<IO, CT, DKB, NW, FULL, WALK>, grid, dim3(64 * NW), 0, s, a);
  else if (da % EV == 0 && dc % EV == 0) launch_kernel(mix_walk<IO, CT, DKB, NW, UNITS, WALK>, grid, dim3(64 * NW), 0, s, a);
  else launch_kernel(mix_walk<IO, CT, DKB, NW, ANY, WALK>, grid, dim3(64 * NW), 0, s, a);
}
template <typename IO, typename CT, bool WALK, int DKB>
void walk_waves(const MixMany& a, dim3 grid, hipStream_t s) {
  if (a.w[0].dc <= 64) walk_fit<IO, CT, WALK, DKB, 4>(a, grid, s);
  else walk_fit<IO, CT, WALK, DKB, 8>(a, grid, s);
}
template <typename IO, typename CT, bool WALK>
void walk(const MixMany& a, hipStream_t s) {
  const MixArgs& w = a.w[0];
  const dim3 grid((unsigned)w.heads, (unsigned)(WALK ? w.nsegs : w.nsegs - 1), (unsigned)(a.seqs * a.n));
  if (w.da <= 32 && w.dc <= 64) walk_fit<IO, CT, WALK, 2, 4>(a, grid, s);
  else if (w.da <= 64) walk_waves<IO, CT, WALK, 4>(a, grid, s);
  else if (w.da <= 96 && w.dc <= 64) walk_fit<IO, CT, WALK, 6, 4>(a, grid, s);
  else walk_waves<IO, CT, WALK, 8>(a, grid, s);
}
template <bool WALK>
void walk_type(const MixArgs* a, int n, int dtype, hipStream_t s) {
  MixMany many{};
  for (int k = 0; k < n; ++k) {   // as many in one launch as have one shape and fit the grid
    many.w[many.n++] = a[k];
    many.seqs = a[k].seqs;
    if (k + 1 < n && a[k + 1].da == a[k].da && a[k + 1].dc == a[k].dc && (int64_t)(many.n + 1) * a[k].seqs <= 65535) continue;
    if (dtype == PC_DTYPE_BF16) walk<bf16, bf16, WALK>(many, s);
    else if (dtype == PC_DTYPE_F16) walk<f16, float, WALK>(many, s);
    else walk<float, float, WALK>(many, s);
    many = MixMany{};
  }
}

}  // namespace

void launch_mix_walk(const MixArgs* a, int n, int dtype, hipStream_t s) { walk_type<true>(a, n, dtype, s); }
void launch_mix_states(const MixArgs* a, int n, int dtype, hipStream_t s) { walk_type<false>(a, n, dtype, s); }

void launch_mix_scan(const MixScanArgs* a, int n, hipStream_t s) {
  const bool both = n == 2 && 2 * (int64_t)a[0].seqs <= 65535;
  for (int k = 0; k < n; k += both ? 2 : 1) {
    const int ev = a[k].elems % 4 == 0 ? 4 : 1;
    const dim3 grid((unsigned)((a[k].elems / ev + 255) / 256), (unsigned)a[k].heads, (unsigned)(a[k].seqs * (both ? 2 : 1)));
    if (ev == 4) launch_kernel(mix_scan<4>, grid, dim3(256), 0, s, a[k], a[both ? 1 : k]);
    else launch_kernel(mix_scan<1>, grid, dim3(256), 0, s, a[k], a[both ? 1 : k]);
  }
}

void launch_mix_sum(const MixSumArgs& a, const MixSumArgs& b, int dtype, hipStream_t s) {
  const int64_t n = a.tokens * a.kv_heads * std::max(a.dim, b.dim);
  const dim3 grid((unsigned)std::min<int64_t>((n + 255) / 256, MIX_SUM_BLOCKS), 2);
  if (dtype == PC_DTYPE_F32) launch_kernel(mix_sum<float>, grid, dim3(256), 0, s, a, b);
  else if (dtype == PC_DTYPE_F16) launch_kernel(mix_sum<f16>, grid, dim3(256), 0, s, a, b);
  else launch_kernel(mix_sum<bf16>, grid, dim3(256), 0, s, a, b);
}

void launch_mix_step(const MixStepArgs& a, int dtype, hipStream_t s) {
  const dim3 grid((unsigned)a.heads, (unsigned)std::min(a.batch, MIX_STEP_ROWS),
                  (unsigned)((a.batch + (int64_t)MIX_STEP_ROWS - 1) / MIX_STEP_ROWS));
  // rows of four columns can be loaded as vectors when none is cut
  const bool four = a.dv % 4 == 0;
#define PC_MIX_STEP(T)                                                          \
  if (four) launch_kernel(mix_step<T, 4>, grid, dim3(256), 0, s, a);            \
  else launch_kernel(mix_step<T, 1>, grid, dim3(256), 0, s, a);
  if (dtype == PC_DTYPE_F32) {
    PC_MIX_STEP(float)
  } else if (dtype == PC_DTYPE_F16) {
    PC_MIX_STEP(f16)
  } else {
    PC_MIX_STEP(bf16)
  }
#undef PC_MIX_STEP
}

}  // namespace pc
