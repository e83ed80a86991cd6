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
// are matrix products.  A workgroup of four waves walks one (sequence, head);
// each wave carries dc / 4 columns of the state in its registers for the whole
// walk, in the accumulator layout, in which four consecutive rows lie in one
// lane: with the contraction's order permuted alike on both sides, the same
// registers are the operand of the next product, so the state never passes
// through LDS.  Only the [C, C] products a_i . b_j do (one tile a wave).
//
// Long sequences are cut into segments (a rule on the number of heads and
// sequences, see mix_segments) that walk side by side: one pass makes each
// segment's own state, a scan joins them, and the walk starts from there.
//
// Precision: bfloat16 tensors are multiplied in bfloat16 with float32 sums.
// The decay weights are not exact in bfloat16: l^{n-off-j} c_j is split into
// three bfloat16 planes, so the state keeps float32 accuracy however long the
// walk; in the output's products the carried state and the inside products
// (a_i . b_j) l^{i-j} are split into two (2^-17 of a value is left out, far
// below the output's own rounding; one plane would add 2^-9 of every term).  float32 and float16 tensors run on the
// float32 matrix instruction throughout (float16's range cannot hold the
// state or its planes).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "pc_ops.h"

namespace pc {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
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
  static constexpr int PAD = 8;
  static constexpr int CPLANES = 3;  // planes of the weighted c, and of the state in the output's product
  static constexpr int SPLANES = 2;
  static constexpr int PPLANES = 2;  // of the inside products
  typedef uint2 quad;
  static __device__ __forceinline__ f32x4 mma(quad a0, quad a1, quad b0, quad b1, f32x4 acc) {
    const uint4 a = {a0.x, a0.y, a1.x, a1.y}, b = {b0.x, b0.y, b1.x, b1.y};
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
  }
  static __device__ __forceinline__ quad row(const bf16* p) { return *(const quad*)p; }
  // Four rows of one column: the 16 lanes of a group hand in 4 x 16 elements,
  // each four consecutive ones, and get back a column each.
  static __device__ __forceinline__ quad col(const bf16* tile, int stride) {
    const int l = threadIdx.x & 63;
    const bf16* p = tile + (4 * (l >> 4) + ((l & 15) >> 2)) * stride + 4 * (l & 3);
    return __builtin_bit_cast(quad, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(p)));
  }
  static __device__ __forceinline__ uint32_t pack(float x, float y) {
    return (uint32_t)bf16_bits(x) | ((uint32_t)bf16_bits(y) << 16);
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
  static constexpr int PAD = 4;
  static constexpr int CPLANES = 1;
  static constexpr int SPLANES = 1;
  static constexpr int PPLANES = 1;
  typedef f32x4 quad;
  static __device__ __forceinline__ f32x4 mma(quad a0, quad a1, quad b0, quad b1, f32x4 acc) {
#pragma unroll
    for (int e = 0; e < 4; ++e) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a0[e], b0[e], acc, 0, 0, 0);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a1[e], b1[e], acc, 0, 0, 0);
    return acc;
  }
  static __device__ __forceinline__ quad row(const float* p) { return *(const quad*)p; }
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

// EV elements of a row, of which `have` exist (the others are 0), as loaded.
template <typename IO, int EV>
struct Unit {
  IO v[EV];
};
template <typename IO, int EV>
__device__ __forceinline__ Unit<IO, EV> load_unit(const IO* p, int have) {
  Unit<IO, EV> u;
  if (have >= EV) {
    __builtin_memcpy(&u, p, sizeof(u));
  } else {
#pragma unroll
    for (int e = 0; e < EV; ++e) u.v[e] = e < have ? p[e] : IO{};
  }
  return u;
}
__device__ __forceinline__ bool not_finite(bf16 x) { return (x.u & 0x7f80) == 0x7f80; }
__device__ __forceinline__ bool not_finite(f16 x) { return (__builtin_bit_cast(uint16_t, x) & 0x7c00) == 0x7c00; }
__device__ __forceinline__ bool not_finite(float x) { return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u; }

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

// ---- the walk ---------------------------------------------------------------
// DKB: 16-blocks of the contracted dimension (even), NB: 16-blocks of output
// columns a wave carries.  WALK false: only the state, from zero, of every
// segment but a sequence's last, into `seg`.
template <typename IO, typename CT, int DKB, int NB, bool WALK>
__global__ __launch_bounds__(256, 2) void mix_walk(MixArgs m) {
  using O = Ops<CT>;
  using quad = typename O::quad;
  constexpr int C = O::C, CB = C / 16, EV = O::EV;
  constexpr int DA = 16 * DKB, DC = 64 * NB;
  constexpr int LA = DA + O::PAD, LC = DC + O::PAD, LP = C + O::PAD;
  constexpr int UA = C * DA / EV / 256, UC = C * DC / EV / 256;   // staged units of a thread
  constexpr int CP = O::CPLANES, SP = O::SPLANES, PP = O::PPLANES;
  __shared__ __align__(16) CT sa[WALK ? C * LA : 8];
  __shared__ __align__(16) CT sb[C * LA];
  __shared__ __align__(16) CT sc[C * LC];
  __shared__ __align__(16) CT sp[WALK ? PP * C * LP : 8];

  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, g = lane >> 4, l16 = lane & 15;
  const int head = blockIdx.x, seq = blockIdx.z;
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
  const int64_t elems = (int64_t)m.da * m.dc;
  const int col0 = wave * 16 * NB + l16;   // this lane's column of block 0
  const bool wave_on = wave * 16 * NB < m.dc;

  // the carried state: lane l16 of group g holds rows 16 kb + 4 g + r of column col0 + 16 nb
  f32x4 st[DKB][NB];
  {
    const float* from = nullptr;
    if (WALK) from = m.nsegs > 1 ? m.seg + (((int64_t)seq * m.nsegs + sgm) * m.heads + head) * elems
                                 : (m.init ? m.init + ((int64_t)seq * m.heads + head) * elems : nullptr);
#pragma unroll
    for (int kb = 0; kb < DKB; ++kb)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * kb + 4 * g + r, col = col0 + 16 * nb;
          st[kb][nb][r] = from && row < m.da && col < m.dc ? from[(int64_t)row * m.st_r + (int64_t)col * m.st_c] : 0.0f;
        }
  }

  // constants of the chunk: the masked decays of this wave's tiles of the
  // inside products, and the output's weight of the state for its tokens
  constexpr int PAIRS = CB * (CB + 1) / 2, MINE = (PAIRS + 3) / 4;
  float md[WALK ? MINE : 1][4], iw[WALK ? CB : 1];
  if constexpr (WALK) {
#pragma unroll
    for (int k = 0; k < MINE; ++k) {
      int ib = 0, jb = wave + 4 * k;
      while (jb > ib) jb -= ++ib;   // pair number -> (ib, jb), jb <= ib
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int d = 16 * (ib - jb) + l16 - 4 * g - r;
        md[k][r] = d >= 0 ? m.pscale * decay_pow(gam, (float)d) : 0.0f;
      }
    }
#pragma unroll
    for (int ib = 0; ib < CB; ++ib) iw[ib] = m.oscale * decay_pow(gam, (float)(16 * ib + l16 + m.off));
    // the products' tiles right of the diagonal that a 32-wide step reads: always 0
    for (int e = tid; e < PP * C * 16; e += 256) {
      const int i = e >> 4, ib = (i % C) >> 4;
      if ((ib & 1) == 0) sp[i * LP + 16 * (ib + 1) + (e & 15)] = CT{};
    }
  }

  Unit<IO, EV> ra[WALK ? UA : 1], rb[UA], rc[UC];
  auto fetch = [&](int64_t pos, int n) {
#pragma unroll
    for (int u = 0; u < UA; ++u) {
      const int id = u * 256 + tid, i = id / (DA / EV), d = id % (DA / EV) * EV;
      const int64_t t = m.rev ? t1 - 1 - pos - i : t0 + pos + i;
      const int have = i < n ? m.da - d : 0;
      if constexpr (WALK) ra[u] = load_unit<IO, EV>(pa + t * m.a.ts + d, have);
      rb[u] = load_unit<IO, EV>(pb + t * m.b.ts + d, have);
    }
#pragma unroll
    for (int u = 0; u < UC; ++u) {
      const int id = u * 256 + tid, i = id / (DC / EV), d = id % (DC / EV) * EV;
      const int64_t t = m.rev ? t1 - 1 - pos - i : t0 + pos + i;
      rc[u] = load_unit<IO, EV>(pc + t * m.c.ts + d, i < n ? m.dc - d : 0);
    }
  };

  float wc[CB][4];      // weights of a token's part in the state
  float ln = 1.0f;
  int wn = -1;          // the chunk size they are of
  int64_t single = pos0;   // tokens before this position go one by one
  int64_t pos = pos0;
  if (pos < pos1) fetch(pos, (int)min((int64_t)C, pos1 - pos));
  while (pos < pos1) {
    int n = pos < single ? 1 : (int)min((int64_t)C, pos1 - pos);
    // A value that is not finite would reach the tokens before it in the chunk
    // through a zero product: such a chunk is walked token by token.
    bool bad = false;
    if (n > 1) {
#pragma unroll
      for (int u = 0; u < UC; ++u)
#pragma unroll
        for (int e = 0; e < EV; ++e) bad |= not_finite(rc[u].v[e]);
    }
    if (__syncthreads_or(bad)) {   // (also: every wave is done with the last chunk's tiles)
      single = pos + n;
      n = 1;
      fetch(pos, n);
    }
#pragma unroll
    for (int u = 0; u < UA; ++u) {
      const int id = u * 256 + tid, at = id / (DA / EV) * LA + id % (DA / EV) * EV;
      if constexpr (WALK) stage<CT, IO, EV>(sa + at, ra[u]);
      stage<CT, IO, EV>(sb + at, rb[u]);
    }
#pragma unroll
    for (int u = 0; u < UC; ++u) {
      const int id = u * 256 + tid;
      stage<CT, IO, EV>(sc + id / (DC / EV) * LC + id % (DC / EV) * EV, rc[u]);
    }
    __syncthreads();
    const int64_t next = pos + n;
    if (next < pos1) fetch(next, next < single ? 1 : (int)min((int64_t)C, pos1 - next));
    if (n != wn) {
      wn = n;
      ln = decay_pow(gam, (float)n);
#pragma unroll
      for (int b = 0; b < CB; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = 16 * b + 4 * g + e;
          wc[b][e] = j < n ? m.wscale * decay_pow(gam, (float)(n - m.off - j)) : 0.0f;
        }
    }
    f32x4 o[WALK ? CB : 1][NB];
    if constexpr (WALK) {
      // inside products b_j . a_i, transposed: a lane holds four j of one i
#pragma unroll
      for (int k = 0; k < MINE; ++k) {
        int ib = 0, jb = wave + 4 * k;
        while (jb > ib) jb -= ++ib;
        if (wave + 4 * k < PAIRS) {
          f32x4 acc = {};
          const CT* rj = sb + (16 * jb + l16) * LA + 4 * g;
          const CT* ri = sa + (16 * ib + l16) * LA + 4 * g;
#pragma unroll
          for (int kb = 0; kb < DKB; kb += 2)
            acc = O::mma(O::row(rj + 16 * kb), O::row(rj + 16 * kb + 16), O::row(ri + 16 * kb), O::row(ri + 16 * kb + 16), acc);
          f32x4 w;
#pragma unroll
          for (int r = 0; r < 4; ++r) w[r] = md[k][r] == 0.0f && (ib == jb && 4 * g + r > l16) ? 0.0f : acc[r] * md[k][r];
          quad pl[PP];
          split<CT, PP>(w, pl);
#pragma unroll
          for (int p = 0; p < PP; ++p) *(quad*)(sp + (p * C + 16 * ib + l16) * LP + 16 * jb + 4 * g) = pl[p];
        }
      }
      // the state's part of the output
#pragma unroll
      for (int ib = 0; ib < CB; ++ib)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) o[ib][nb] = f32x4{};
      if (wave_on) {
#pragma unroll
        for (int kb = 0; kb < DKB; kb += 2) {
          quad s0[NB][SP], s1[NB][SP];
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            split<CT, SP>(st[kb][nb], s0[nb]);
            split<CT, SP>(st[kb + 1][nb], s1[nb]);
          }
#pragma unroll
          for (int ib = 0; ib < CB; ++ib) {
            const CT* ri = sa + (16 * ib + l16) * LA + 16 * kb + 4 * g;
            const quad a0 = O::row(ri), a1 = O::row(ri + 16);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int p = SP - 1; p >= 0; --p) o[ib][nb] = O::mma(s0[nb][p], s1[nb][p], a0, a1, o[ib][nb]);
          }
        }
#pragma unroll
        for (int ib = 0; ib < CB; ++ib)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) o[ib][nb] *= iw[ib];
      }
      __syncthreads();
    }
    if (wave_on) {
#pragma unroll
      for (int kb = 0; kb < DKB; ++kb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) st[kb][nb] *= ln;
#pragma unroll
      for (int b = 0; b < CB; b += 2) {
        quad c0[NB], c1[NB], w0[NB][CP], w1[NB][CP];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          c0[nb] = O::col(sc + 16 * b * LC + wave * 16 * NB + 16 * nb, LC);
          c1[nb] = O::col(sc + (16 * b + 16) * LC + wave * 16 * NB + 16 * nb, LC);
          split<CT, CP>(O::wide(c0[nb]) * f32x4{wc[b][0], wc[b][1], wc[b][2], wc[b][3]}, w0[nb]);
          split<CT, CP>(O::wide(c1[nb]) * f32x4{wc[b + 1][0], wc[b + 1][1], wc[b + 1][2], wc[b + 1][3]}, w1[nb]);
        }
        if constexpr (WALK) {
#pragma unroll
          for (int ib = b; ib < CB; ++ib) {
#pragma unroll
            for (int p = PP - 1; p >= 0; --p) {
              const CT* ri = sp + (p * C + 16 * ib + l16) * LP + 16 * b + 4 * g;
              const quad p0 = O::row(ri), p1 = O::row(ri + 16);
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) o[ib][nb] = O::mma(c0[nb], c1[nb], p0, p1, o[ib][nb]);
            }
          }
        }
#pragma unroll
        for (int kb = 0; kb < DKB; ++kb) {
          const quad b0 = O::col(sb + 16 * b * LA + 16 * kb, LA), b1 = O::col(sb + (16 * b + 16) * LA + 16 * kb, LA);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int p = CP - 1; p >= 0; --p) st[kb][nb] = O::mma(b0, b1, w0[nb][p], w1[nb][p], st[kb][nb]);
        }
      }
      if constexpr (WALK) {
        // transposed outputs: a lane holds four columns of one token
#pragma unroll
        for (int ib = 0; ib < CB; ++ib) {
          const int i = 16 * ib + l16;
          if (i >= n) continue;
          const int64_t t = m.rev ? t1 - 1 - pos - i : t0 + pos + i;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const int col = wave * 16 * NB + 16 * nb + 4 * g, have = m.dc - col;
            if (have <= 0) continue;
            const int64_t at = t * m.o_ts + (int64_t)head * m.o_hs + col;
            if (m.out_f32) {
              float* q = (float*)m.out + at;
              if (have >= 4) {
                __builtin_memcpy(q, &o[ib][nb], 16);
              } else {
                for (int r = 0; r < have; ++r) q[r] = o[ib][nb][r];
              }
            } else {
              IO* q = (IO*)m.out + at;
              IO w[4];
#pragma unroll
              for (int r = 0; r < 4; ++r) w[r] = from_f32<IO>(o[ib][nb][r]);
              if (have >= 4) {
                __builtin_memcpy(q, w, sizeof(w));
              } else {
                for (int r = 0; r < have; ++r) q[r] = w[r];
              }
            }
          }
        }
      }
    }
    pos = next;
  }

  float* to = nullptr;
  if (!WALK) to = m.seg + (((int64_t)seq * m.nsegs + sgm) * m.heads + head) * elems;
  else if (m.fin && sgm == live - 1) to = m.fin + ((int64_t)seq * m.heads + head) * elems;
  if (!to) return;
#pragma unroll
  for (int kb = 0; kb < DKB; ++kb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * kb + 4 * g + r, col = col0 + 16 * nb;
        if (row < m.da && col < m.dc) to[(int64_t)row * m.st_r + (int64_t)col * m.st_c] = st[kb][nb][r];
      }
}

// The states at the segments' starts from the segments' own states, in place:
// start_0 = init, start_{s+1} = l^seglen start_s + own_s.
__global__ __launch_bounds__(256) void mix_scan(MixScanArgs m) {
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int head = blockIdx.y, seq = blockIdx.z;
  if (e >= m.elems) return;
  int64_t t0 = 0, t1 = m.tokens;
  if (m.cu) {
    t0 = min(max((int64_t)m.cu[seq], (int64_t)0), m.tokens);
    t1 = min(max((int64_t)m.cu[seq + 1], t0), m.tokens);
  }
  const int live = (int)min(max((t1 - t0 + m.seglen - 1) / m.seglen, (int64_t)1), (int64_t)m.nsegs);
  const float ls = decay_pow(m.log_decay[head], (float)m.seglen);
  float* p = m.seg + ((int64_t)seq * m.nsegs * m.heads + head) * m.elems + e;
  const int64_t step = (int64_t)m.heads * m.elems;
  float run = m.init ? m.init[((int64_t)seq * m.heads + head) * m.elems + e] : 0.0f;
  for (int s = 0; s < live; ++s) {
    const float own = s + 1 < live ? p[s * step] : 0.0f;
    p[s * step] = run;
    run = run * ls + own;
  }
}

// Gradients of shared key / value heads: the sum over the heads that share one,
// in their order.  Only tokens of the sequences are written.
template <typename IO>
__global__ __launch_bounds__(256) void mix_sum(MixSumArgs m) {
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int per = m.kv_heads * m.dim;
  const int64_t t = e / per;
  const int h = (int)(e % per) / m.dim, d = (int)(e % per) % m.dim;
  int64_t t0 = 0, t1 = m.tokens;
  if (m.cu) {
    t0 = min(max((int64_t)m.cu[0], (int64_t)0), m.tokens);
    t1 = min(max((int64_t)m.cu[m.seqs], t0), m.tokens);
  }
  if (t < t0 || t >= t1) return;
  const float* p = m.part + (t * m.kv_heads + h) * (int64_t)m.group * m.dim + d;
  float s = 0.0f;
  for (int k = 0; k < m.group; ++k) s += p[(int64_t)k * m.dim];
  ((IO*)m.out)[t * m.o_ts + (int64_t)h * m.o_hs + d] = from_f32<IO>(s);
}

// ---- single tokens ----------------------------------------------------------
// One workgroup per (row, head): the state is read, updated, written and
// contracted with q in one pass; bound by the state's bytes.  CV columns a
// thread, the rows dealt out over the workgroup's row groups, whose partial
// outputs are added in a fixed order.  Rows that name the same slot are
// successive tokens of that state: the first of them does them all, in order.
template <typename IO, int CV>
__global__ __launch_bounds__(256) void mix_step(MixStepArgs m) {
  const int head = blockIdx.x % m.heads, first = blockIdx.x / m.heads, tid = threadIdx.x;
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

template <typename IO, typename CT, bool WALK, int DKB>
void walk_nb(const MixArgs& a, dim3 grid, hipStream_t s) {
  if (a.dc <= 64) launch_kernel(mix_walk<IO, CT, DKB, 1, WALK>, grid, dim3(256), 0, s, a);
  else launch_kernel(mix_walk<IO, CT, DKB, 2, WALK>, grid, dim3(256), 0, s, a);
}
template <typename IO, typename CT, bool WALK>
void walk(const MixArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)a.heads, (unsigned)(WALK ? a.nsegs : a.nsegs - 1), (unsigned)a.seqs);
  if (a.da <= 32) walk_nb<IO, CT, WALK, 2>(a, grid, s);
  else if (a.da <= 64) walk_nb<IO, CT, WALK, 4>(a, grid, s);
  else walk_nb<IO, CT, WALK, 8>(a, grid, s);
}
template <bool WALK>
void walk_type(const MixArgs& a, int dtype, hipStream_t s) {
  if (dtype == PC_DTYPE_BF16) walk<bf16, bf16, WALK>(a, s);
  else if (dtype == PC_DTYPE_F16) walk<f16, float, WALK>(a, s);
  else walk<float, float, WALK>(a, s);
}

}  // namespace

void launch_mix_walk(const MixArgs& a, int dtype, hipStream_t s) { walk_type<true>(a, dtype, s); }
void launch_mix_states(const MixArgs& a, int dtype, hipStream_t s) { walk_type<false>(a, dtype, s); }

void launch_mix_scan(const MixScanArgs& a, hipStream_t s) {
  launch_kernel(mix_scan, dim3((unsigned)((a.elems + 255) / 256), (unsigned)a.heads, (unsigned)a.seqs), dim3(256), 0, s, a);
}

void launch_mix_sum(const MixSumArgs& a, int dtype, hipStream_t s) {
  const int64_t n = a.tokens * a.kv_heads * a.dim;
  const dim3 grid((unsigned)((n + 255) / 256));
  if (dtype == PC_DTYPE_F32) launch_kernel(mix_sum<float>, grid, dim3(256), 0, s, a);
  else if (dtype == PC_DTYPE_F16) launch_kernel(mix_sum<f16>, grid, dim3(256), 0, s, a);
  else launch_kernel(mix_sum<bf16>, grid, dim3(256), 0, s, a);
}

void launch_mix_step(const MixStepArgs& a, int dtype, hipStream_t s) {
  const dim3 grid((unsigned)a.heads * (unsigned)a.batch);
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
