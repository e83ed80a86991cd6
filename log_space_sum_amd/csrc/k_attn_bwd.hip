// k_attn_bwd.hip -- the gradients of causal softmax attention, from its outputs o and lse.
//
//   P_ij = exp(scale q_i . k_j - lse_i),  delta_i = do_i . o_i,  dS_ij = P_ij (do_i . v_j - delta_i)
//   dq_i = scale sum_j dS_ij k_j,   dk_j = scale sum_i dS_ij q_i,   dv_j = sum_i P_ij do_i
//
// Two kernels: the first keeps 32 rows of q, do and dq a wave and goes along the
// keys, as the forward does; in the second pairs of waves keep 32 keys of k, v, dk and dv and
// go along the rows of every head that shares them.  Scores are computed in both,
// so that no sum is shared: no atomics, the same bits at every run, and the sums over sharing
// heads stay in registers.  The first leaves delta for the second.  Few long sequences are cut, along the keys and along
// the rows; a third kernel sums the parts.
//
// What bounds it: matrix instructions.  Of bfloat16 the first kernel takes S, dP and three planes of dS, 5 products' work, the
// second S twice, dP and three planes each of P and dS, 9: 8 x 2048 x 16 heads x 128 in 0.98 ms are 0.98 PFLOP/s of them (a large
// library product: 1.39); float16, two planes, 11: 0.93 ms; float32, 6 for each, 48: 3.63 ms, 0.9 PFLOP/s.  Small ones are chains of tiles.
#include <algorithm>

#include "k_attn.h"

namespace pc {
namespace {

// float16 planes of dS and, for dv, of P: a lane's column (a row of dq, a key of dk
// or dv) is held as a power of two times itself that keeps its largest element so
// far below 2^15, moved as the maximum of a softmax is.  bfloat16's range needs none.
// (P at a fixed 2^14 would lose all bits of weights below 2^-39: keys that no row
// looks at, whose dv is an ordinary number again under scaled losses.)
template <typename T>
struct Scale {
  static constexpr bool ON = std::is_same_v<T, f16>;
  float by = ON ? 0x1p126f : 1.0f;
  template <int DB>
  __device__ __forceinline__ void move(f32x16& ds, f32x16 (&acc)[DB]) {
    if constexpr (ON) {
      float top = 0.0f;
#pragma unroll
      for (int r = 0; r < 16; ++r) top = fmaxf(top, fabsf(ds[r]));
      top = max_halves(top);
      if (__any(top * by > 32768.0f)) {
        float to = by;
        if (top * by > 32768.0f)      // 2^(14 - exponent)
          to = __uint_as_float(min(max(127 + 14 + 127 - (int)(__float_as_uint(top) >> 23), 1), 253) << 23);
        const float f = to / by;
        by = to;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int r = 0; r < 16; ++r) acc[d][r] *= f;
      }
#pragma unroll
      for (int r = 0; r < 16; ++r) ds[r] *= by;
    }
  }
};

template <int DB>
__device__ __forceinline__ bool any_not_finite(const f32x16 (&x)[DB]) {
  float bad = 0.0f;
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int r = 0; r < 16; ++r) bad = fmaf(x[d][r], 0.0f, bad);
  return !(bad == 0.0f);
}

// Keys (of dq) or rows (of dk and dv) from .. to - 1 of a part, between `first` and `end`.
struct Part {
  int from, to;
};
__device__ __forceinline__ Part part_of(const AttnArgs& a, int split, int first, int end) {
  if (a.nsplit == 1) return {first, end};
  const int64_t lo = (int64_t)split * a.part_len, hi = split + 1 < a.nsplit ? lo + a.part_len : (int64_t)end;
  return {(int)min(max(lo, (int64_t)first), (int64_t)end), (int)min(hi, (int64_t)end)};
}

template <typename T>
__device__ __forceinline__ float dot(const T* a, const T* b, int n) {
  float s = 0.0f;
  for (int d = 0; d < n; ++d) s = fmaf(to_f32(a[d]), to_f32(b[d]), s);
  return s;
}

// ---- a block of 32 by 32 (16-bit types) ---------------------------------------------
// s = A x^T and, with BOTH, dp = B y^T for 32 rows of two tiles and a wave's own operands.  The rows of A are
// all asked for before they are used, those of B meanwhile; a single product goes in two chains.
template <typename T, int D, bool UNIT, bool BOTH, typename TileT>
__device__ __forceinline__ void block_products(const TileT& ta, const TileT& tb, int r0, int lane, const frag (&x)[D / 16][1],
                                               const frag (&y)[BOTH ? D / 16 : 1][1], f32x16& s, f32x16& dp) {
  using N = Num<T>;
  constexpr int DS = D / 16;
  frag fa[DS][1], fb[BOTH ? DS : 1][1];
#pragma unroll
  for (int st = 0; st < DS; ++st)
    ta.rows(r0, st, lane, fa[st]);
  if (UNIT) __builtin_amdgcn_sched_barrier(0);
  s = dp = f32x16{};
#pragma unroll
  for (int st = 0; st < DS; ++st) {
    if constexpr (BOTH) {
      tb.rows(r0, st, lane, fb[st]);
      s = N::mma(fa[st][0], x[st][0], s);
      if (UNIT) __builtin_amdgcn_sched_barrier(0);
    } else {
      if (st & 1) dp = N::mma(fa[st][0], x[st][0], dp);
      else s = N::mma(fa[st][0], x[st][0], s);
    }
  }
  if constexpr (BOTH) {
#pragma unroll
    for (int st = 0; st < DS; ++st)
      dp = N::mma(fb[st][0], y[st][0], dp);
  } else {
    s += dp;
  }
}
// acc += A^T x for 32 rows of a tile and a result x of them; the second 16 rows' values are read and planes made
// between the first's matrix instructions.
template <typename T, int D, bool UNIT, typename TileT>
__device__ __forceinline__ void block_add(const TileT& ta, int r0, int lane, const f32x16& x, f32x16 (&acc)[D / 32]) {
  using N = Num<T>;
  constexpr int W = N::W, DB = D / 32;
  frag w[2][W], f[2][DB][1];
  auto ready = [&](int st) {
#pragma unroll
    for (int d = 0; d < DB; ++d)
      ta.cols(r0 + 16 * st, 32 * d, lane, f[st][d]);
    float p[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) p[e] = x[8 * st + e];
    planes_of<N>(p, w[st]);
  };
  ready(0);
  if (UNIT) __builtin_amdgcn_sched_barrier(0);
  ready(1);
#pragma unroll
  for (int st = 0; st < 2; ++st)
#pragma unroll
    for (int p = W - 1; p >= 0; --p)
#pragma unroll
      for (int d = 0; d < DB; ++d)
        acc[d] = N::mma(f[st][d][0], w[st][p], acc[d]);
  if (UNIT) {
    __builtin_amdgcn_sched_group_barrier(0x100, 2 * DB, 0);
#pragma unroll
    for (int k = 0; k < W * DB; ++k) {
      __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x2, 3, 0);
    }
  }
}

// ---- dq -------------------------------------------------------------------------
template <typename T, int D>
struct DqShape {
  static constexpr int IN = Num<T>::IN, BK = IN == 3 ? 32 : 64, BUFS = IN == 3 ? 1 : 2;
  struct Lds {
    Tile<T, BK, D> k[BUFS], v[BUFS];
  };
};

// A row after the other in float32, for a tile whose results are not finite (see careful_rows of the forward).
template <typename T>
__device__ __attribute__((noinline)) void careful_dq(AttnArgs a, int64_t t0, int64_t first, int count, int kvh, int split, Part part) {
  const int lane = threadIdx.x & 63;
  const T *k0 = (const T*)a.k.p + t0 * a.k.ts + kvh * a.k.hs, *v0 = (const T*)a.v.p + t0 * a.v.ts + kvh * a.v.hs;
  for (int r = threadIdx.x >> 6; r < count; r += 4) {
    const int64_t i = (first + r) / a.group, t = t0 + i, h = (int64_t)kvh * a.group + (first + r) % a.group;
    const T *q = (const T*)a.q.p + t * a.q.ts + h * a.q.hs, *go = (const T*)a.d_o.p + t * a.d_o.ts + h * a.d_o.hs;
    const T* o = (const T*)a.out.p + t * a.out.ts + h * a.out.hs;
    const float lse = a.lse[t * a.kv_heads * a.group + h], delta = dot(go, o, a.dv);
    float acc[2] = {0.0f, 0.0f};
    const int64_t last = min(i, (int64_t)part.to - 1);
    for (int64_t j0 = part.from; j0 <= last; j0 += 64) {
      const int64_t j = min(j0 + lane, last);
      const float p = exp2_fast((dot(q, k0 + j * a.k.ts, a.dk) * a.scale - lse) * LOG2E);
      const float ds = p * (dot(go, v0 + j * a.v.ts, a.dv) - delta);
      for (int x = 0; x < min((int64_t)64, last - j0 + 1); ++x) {
        const float w = __shfl(ds, x);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (lane + 64 * e < a.dk) acc[e] = fmaf(w, to_f32(k0[(j0 + x) * a.k.ts + lane + 64 * e]), acc[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (lane + 64 * e < a.dk) {
        if (a.nsplit > 1) a.part[(((int64_t)split * a.tokens + t) * a.kv_heads * a.group + h) * a.dk + lane + 64 * e] = acc[e] * a.scale;
        else ((T*)a.dq)[t * a.dq_ts + h * a.dq_hs + lane + 64 * e] = from_f32<T>(acc[e] * a.scale);
      }
  }
}

template <typename T, int D, FitMode MODE>
__global__ __launch_bounds__(256, Num<T>::IN == 3 || MODE == ANY ? 1 : 2) void attn_dq(AttnArgs a, int64_t slots) {
  using N = Num<T>;
  using S = DqShape<T, D>;
  constexpr int IN = N::IN, W = N::W, BK = S::BK, KB = BK / 32, BUFS = S::BUFS, DS = D / 16, DB = D / 32;
  constexpr int PER_ROW = Tile<T, 32, D>::P / 8, U = BK * PER_ROW / 256;
  constexpr bool UNIT = MODE == UNITS, DIRECT = IN == 1 && UNIT;
  __shared__ typename S::Lds lds;
  const int heads = a.kv_heads * a.group, dk = a.dk, dv = a.dv;
  const float c = a.scale * LOG2E;
  for (int64_t b = blockIdx.x; b < slots * a.nsplit * a.kv_heads; b += gridDim.x) {
    const auto [kvh, split, slot] = block_of(b, a.kv_heads, slots);
    const SeqTile at = find_tile(a.cu, a.seqs, a.tokens, a.group, ATTN_ROWS, slots - 1 - slot);
    const int64_t first = at.tile * ATTN_ROWS, rows_all = at.len * a.group;
    if (at.seq < 0 || first >= rows_all) continue;
    const int tid = thread_here(), wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, h = lane >> 5;
    const int64_t tf = first / a.group;
    const int rem = (int)(first - tf * a.group), count = (int)min((int64_t)ATTN_ROWS, rows_all - first);
    auto token_of = [&](int i) { return (int)((uint32_t)(rem + i) / (uint32_t)a.group); };
    const int wave_first = 32 * wave, mine = min(wave_first + (lane & 31), count - 1);
    const bool wave_on = wave_first < count;
    const int tl = token_of(mine), hl = rem + mine - tl * a.group;      // this lane's token and head in the tile
    const int last = (int)tf + tl, first_last = (int)tf + token_of(min(wave_first, count - 1)),
              last_last = (int)tf + token_of(min(wave_first + 31, count - 1)), end = (int)tf + token_of(count - 1) + 1;
    const int64_t t = at.t0 + tf + tl, head = (int64_t)kvh * a.group + hl;
    const Part part = part_of(a, split, 0, end);
    if (part.from >= part.to) continue;
    const float lse2 = a.lse[t * heads + head] * LOG2E;
    frag q[DS][IN], go[DS][IN];
    float delta = 0.0f;
    {
      const T *pq = (const T*)a.q.p + t * a.q.ts + head * a.q.hs, *pg = (const T*)a.d_o.p + t * a.d_o.ts + head * a.d_o.hs;
      const T* po = (const T*)a.out.p + t * a.out.ts + head * a.out.hs;
#pragma unroll
      for (int s = 0; s < DS; ++s) {
        frags_of(load_own<UNIT>(pq, 16 * s + 8 * h, dk), q[s]);
        const Unit<T> g = load_own<UNIT>(pg, 16 * s + 8 * h, dv), o = load_own<UNIT>(po, 16 * s + 8 * h, dv);
#pragma unroll
        for (int e = 0; e < 8; ++e) delta = fmaf(to_f32(g.v[e]), to_f32(o.v[e]), delta);
        frags_of(g, go[s]);
      }
      delta = add_halves(delta);
      if (split == 0 && h == 0 && wave_first + lane < count) a.delta[t * heads + head] = delta;
    }
    f32x16 acc[DB];
#pragma unroll
    for (int d = 0; d < DB; ++d) acc[d] = f32x16{};
    Scale<T> scale;

    const T *k0 = (const T*)a.k.p + at.t0 * a.k.ts + kvh * a.k.hs, *v0 = (const T*)a.v.p + at.t0 * a.v.ts + kvh * a.v.hs;
    const DirectUnit<D> unit(tid);
    const int kbyte = unit.byte(dk), vbyte = unit.byte(dv);
    const uint32_t ok = (uint32_t)(unit.row * (int)a.k.ts * 2 + kbyte), ov = (uint32_t)(unit.row * (int)a.v.ts * 2 + vbyte);
    auto load = [&](int x, int key) {
      const uint32_t kb = lds_byte(lds.k[x].at) + wave * 1024, vb = lds_byte(lds.v[x].at) + wave * 1024;
      const T *kr = k0 + key * a.k.ts, *vr = v0 + key * a.v.ts;
      if (key + BK <= end) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          lds_load16(kr + u * unit.STEP * a.k.ts, ok, kb + u * 4096);
          lds_load16(vr + u * unit.STEP * a.v.ts, ov, vb + u * 4096);
        }
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int row = min(unit.row + u * unit.STEP, end - 1 - key);
          lds_load16(kr, (uint32_t)(row * (int)a.k.ts * 2 + kbyte), kb + u * 4096);
          lds_load16(vr, (uint32_t)(row * (int)a.v.ts * 2 + vbyte), vb + u * 4096);
        }
      }
    };
    Unit<T> rk[DIRECT ? 1 : U], rv[DIRECT ? 1 : U];
    auto fetch = [&](int key) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int id = u * 256 + tid, j = min(key + id / PER_ROW, end - 1), d = id % PER_ROW * 8;
        rk[u] = load_unit<UNIT>(k0 + j * a.k.ts, d, dk);
        rv[u] = load_unit<UNIT>(v0 + j * a.v.ts, d, dv);
      }
    };
    auto stage = [&](int x) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int id = u * 256 + tid;
        lds.k[x].put(id / PER_ROW, id % PER_ROW * 8, rk[u]);
        lds.v[x].put(id / PER_ROW, id % PER_ROW * 8, rv[u]);
      }
    };
    auto compute = [&](int x, int key) {
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        f32x16 s = f32x16{}, dp = f32x16{};
        if constexpr (IN == 1) {
          block_products<T, D, UNIT, true>(lds.k[x], lds.v[x], 32 * kb, lane, q, go, s, dp);
        } else {
#pragma unroll
        for (int st = 0; st < DS; ++st) {
          frag f[IN];
          if (32 * (st / 2) < dk) {
            lds.k[x].rows(32 * kb, st, lane, f);
            s = mma_planes<N>(f, q[st], s);
          }
          if (32 * (st / 2) < dv) {
            lds.v[x].rows(32 * kb, st, lane, f);
            dp = mma_planes<N>(f, go[st], dp);
          }
        }
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) s[r] = exp2_fast(fmaf(s[r], c, -lse2));
        if (key + 32 * kb + 31 > first_last) {
#pragma unroll
          for (int r = 0; r < 16; ++r) s[r] = masked(s[r], key + 32 * kb + row_of(r, h) > last, 0.0f);
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) s[r] *= dp[r] - delta;
        scale.move(s, acc);
        if constexpr (IN == 1) {
          block_add<T, D, UNIT>(lds.k[x], 32 * kb, lane, s, acc);
          continue;
        }
#pragma unroll
        for (int st = 0; st < 2; ++st) {
          float p[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) p[e] = s[8 * st + e];
          frag w[W];
          planes_of<N>(p, w);
#pragma unroll
          for (int d = 0; d < DB; ++d) {
            if (32 * d >= dk) continue;
            frag f[IN];
            lds.k[x].cols(32 * kb + 16 * st, 32 * d, lane, f);
            acc[d] = mma_planes<N>(f, w, acc[d]);
          }
        }
      }
    };
    __syncthreads();
    if constexpr (DIRECT) {
      load(0, part.from);
      direct_wait();
      __syncthreads();
      int x = 0;
      for (int key = part.from; key < part.to; key += BK, x ^= 1) {
        if (key + BK < part.to) load(x ^ 1, key + BK);
        if (wave_on && key <= last_last) compute(x, key);
        direct_wait();
        __syncthreads();
      }
    } else if constexpr (BUFS == 2) {
      fetch(part.from);
      stage(0);
      __syncthreads();
      int x = 0;
      for (int key = part.from; key < part.to; key += BK, x ^= 1) {
        const bool more = key + BK < part.to;
        if (more) fetch(key + BK);
        if (wave_on && key <= last_last) compute(x, key);
        if (more) stage(x ^ 1);
        __syncthreads();
      }
    } else {
      fetch(part.from);
      for (int key = part.from; key < part.to; key += BK) {
        stage(0);
        __syncthreads();
        if (key + BK < part.to) fetch(key + BK);
        if (wave_on && key <= last_last) compute(0, key);
        __syncthreads();
      }
    }
    const bool store = wave_first + (lane & 31) < count;
    if (__syncthreads_or(store && any_not_finite(acc))) {
      careful_dq<T>(a, at.t0, first, count, kvh, split, part);
      continue;
    }
    if (!store) continue;
    const float f = a.scale / scale.by;
    float* sum = a.nsplit > 1 ? a.part + (((int64_t)split * a.tokens + t) * heads + head) * dk : nullptr;
    T* to = (T*)a.dq + t * a.dq_ts + head * a.dq_hs;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int e = 32 * d + 8 * r + 4 * h;
        const float x[4] = {acc[d][4 * r] * f, acc[d][4 * r + 1] * f, acc[d][4 * r + 2] * f, acc[d][4 * r + 3] * f};
        if (sum) store4<float>(sum + e, x, dk - e);
        else store4<T>(to + e, x, dk - e);
      }
  }
}

// ---- dk, dv ---------------------------------------------------------------------
template <typename T>
__device__ __attribute__((noinline)) void careful_dkv(AttnArgs a, int64_t t0, int64_t first, int count, int kvh, int nwaves, int split, Part part) {
  const int lane = threadIdx.x & 63, heads = a.kv_heads * a.group;
  for (int r = threadIdx.x >> 6; r < count; r += nwaves) {
    const int64_t j = first + r;
    const T *k = (const T*)a.k.p + (t0 + j) * a.k.ts + kvh * a.k.hs, *v = (const T*)a.v.p + (t0 + j) * a.v.ts + kvh * a.v.hs;
    float dk[2] = {0.0f, 0.0f}, dv[2] = {0.0f, 0.0f};
    for (int64_t h = (int64_t)kvh * a.group; h < (int64_t)(kvh + 1) * a.group; ++h)
      for (int64_t i0 = max(j, (int64_t)part.from); i0 < part.to; i0 += 64) {
        const int64_t t = t0 + min(i0 + lane, (int64_t)part.to - 1);
        const float p = exp2_fast((dot((const T*)a.q.p + t * a.q.ts + h * a.q.hs, k, a.dk) * a.scale - a.lse[t * heads + h]) * LOG2E);
        const float ds = p * (dot((const T*)a.d_o.p + t * a.d_o.ts + h * a.d_o.hs, v, a.dv) - a.delta[t * heads + h]);
        for (int x = 0; x < min((int64_t)64, part.to - i0); ++x) {
          const float wp = __shfl(p, x), ws = __shfl(ds, x);
          const T *q = (const T*)a.q.p + (t0 + i0 + x) * a.q.ts + h * a.q.hs, *go = (const T*)a.d_o.p + (t0 + i0 + x) * a.d_o.ts + h * a.d_o.hs;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int d = lane + 64 * e;
            if (d < a.dk) dk[e] = fmaf(ws, to_f32(q[d]), dk[e]);
            if (d < a.dv) dv[e] = fmaf(wp, to_f32(go[d]), dv[e]);
          }
        }
      }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int d = lane + 64 * e;
      if (a.nsplit > 1) {
        const int64_t at = ((int64_t)split * a.tokens + t0 + j) * a.kv_heads + kvh;
        if (d < a.dk) a.part_k[at * a.dk + d] = dk[e] * a.scale;
        if (d < a.dv) a.part_v[at * a.dv + d] = dv[e];
        continue;
      }
      if (d < a.dk) ((T*)a.dk_)[(t0 + j) * a.dk_ts + kvh * a.dk_hs + d] = from_f32<T>(dk[e] * a.scale);
      if (d < a.dv) ((T*)a.dv_)[(t0 + j) * a.dv_ts + kvh * a.dv_hs + d] = from_f32<T>(dv[e]);
    }
  }
}

// A pair of waves shares 32 keys, the first makes their dv (from S and P), the second their dk (from S, dP and
// dS), so that either fits the registers of two waves a SIMD.  S is made twice (9 products' work for 8).
constexpr int PAIRS = 2;
template <typename T, int D>
struct PairShape {
  static constexpr bool F32 = Num<T>::IN == 3;
  static constexpr int BR = F32 ? 32 : 64, KEYS = 32 * PAIRS, NT = 128 * PAIRS;
  struct Lds {
    Tile<T, BR, D> q[2], go[2];
    alignas(16) float lse2[2][BR];
    alignas(16) float delta[2][BR];
    int bad;
  };
};

// One wave's part of a tile of keys: DK: dk, else dv, of its 32.
template <typename T, int D, FitMode MODE, bool DK>
__device__ __forceinline__ void pair_tile(typename PairShape<T, D>::Lds& lds, const AttnArgs& a, const SeqTile& at, int kvh, int split) {
  using N = Num<T>;
  using S = PairShape<T, D>;
  constexpr bool UNIT = MODE == UNITS, DIRECT = UNIT && !S::F32;
  constexpr int IN = N::IN, W = N::W, BR = S::BR, DS = D / 16, DB = D / 32, NT = S::NT;
  constexpr int PER_ROW = Tile<T, 32, D>::P / 8, U = BR * PER_ROW / NT;
  const int tid = thread_here(), wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, h = lane >> 5;
  const int heads = a.kv_heads * a.group, dk = a.dk, dv = a.dv;
  const float c = a.scale * LOG2E;
  const DirectUnit<D, NT> unit(tid);
  const int qbyte = unit.byte(dk), gbyte = unit.byte(dv);
  const uint32_t oq = (uint32_t)(unit.row * (int)a.q.ts * 2 + qbyte), og = (uint32_t)(unit.row * (int)a.d_o.ts * 2 + gbyte);
  const int len = (int)at.len, first = (int)(at.tile * S::KEYS), count = min(S::KEYS, len - first), block = 32 * (wave % PAIRS);
  const Part part = part_of(a, split, first, len);
  if (part.from >= part.to) return;     // (every wave)
  const int key = first + min(block + (lane & 31), count - 1), wave_key = first + block;
  const bool wave_on = block < count;
  frag k[DS][IN], v[DK ? DS : 1][IN];
  {
    const T *pk = (const T*)a.k.p + (at.t0 + key) * a.k.ts + kvh * a.k.hs, *pv = (const T*)a.v.p + (at.t0 + key) * a.v.ts + kvh * a.v.hs;
#pragma unroll
    for (int s = 0; s < DS; ++s) {
      frags_of(load_own<UNIT>(pk, 16 * s + 8 * h, dk), k[s]);
      if constexpr (DK) frags_of(load_own<UNIT>(pv, 16 * s + 8 * h, dv), v[s]);
    }
  }
  f32x16 acc[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d) acc[d] = f32x16{};
  Scale<T> scale;

  Unit<T> rq[DIRECT ? 1 : U], rg[DIRECT ? 1 : U];
  float rs = 0.0f;
  auto fetch = [&](int x, int head, int row) {
    const T *q0 = (const T*)a.q.p + (at.t0 + row) * a.q.ts + head * a.q.hs, *g0 = (const T*)a.d_o.p + (at.t0 + row) * a.d_o.ts + head * a.d_o.hs;
    if constexpr (DIRECT) {
      const uint32_t qb = lds_byte(lds.q[x].at) + wave * 1024, gb = lds_byte(lds.go[x].at) + wave * 1024;
      if (row + BR <= len) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          lds_load16(q0 + u * unit.STEP * a.q.ts, oq, qb + u * NT * 16);
          lds_load16(g0 + u * unit.STEP * a.d_o.ts, og, gb + u * NT * 16);
        }
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int r = min(unit.row + u * unit.STEP, len - 1 - row);
          lds_load16(q0, (uint32_t)(r * (int)a.q.ts * 2 + qbyte), qb + u * NT * 16);
          lds_load16(g0, (uint32_t)(r * (int)a.d_o.ts * 2 + gbyte), gb + u * NT * 16);
        }
      }
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int id = u * NT + tid, d = id % PER_ROW * 8;
        const int64_t r = min(id / PER_ROW, len - 1 - row);
        rq[u] = load_unit<UNIT>(q0 + r * a.q.ts, d, dk);
        rg[u] = load_unit<UNIT>(g0 + r * a.d_o.ts, d, dv);
      }
    }
    if (tid < 2 * BR) {
      const int64_t i = (at.t0 + min(row + (tid & (BR - 1)), len - 1)) * heads + head;
      rs = tid < BR ? a.lse[i] * LOG2E : a.delta[i];
    }
  };
  auto stage = [&](int x) {
    if constexpr (!DIRECT) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int id = u * NT + tid;
        lds.q[x].put(id / PER_ROW, id % PER_ROW * 8, rq[u]);
        lds.go[x].put(id / PER_ROW, id % PER_ROW * 8, rg[u]);
      }
    }
    if (tid < BR) lds.lse2[x][tid] = rs;
    else if (tid < 2 * BR) lds.delta[x][tid - BR] = rs;
  };
  auto compute = [&](int x, int row, int r0) {
    f32x16 s, dp;
    if constexpr (IN == 1) {
      block_products<T, D, UNIT, DK>(lds.q[x], lds.go[x], r0, lane, k, v, s, dp);
    } else {
      s = dp = f32x16{};
#pragma unroll
      for (int st = 0; st < DS; ++st) {
        frag f[IN];
        if (32 * (st / 2) < dk) {
          lds.q[x].rows(r0, st, lane, f);
          s = mma_planes<N>(f, k[st], s);
        }
        if constexpr (DK)
          if (32 * (st / 2) < dv) {
            lds.go[x].rows(r0, st, lane, f);
            dp = mma_planes<N>(f, v[st], dp);
          }
      }
    }
#pragma unroll
    for (int r4 = 0; r4 < 4; ++r4) {
      const f32x4 l4 = *(const f32x4*)&lds.lse2[x][r0 + 8 * r4 + 4 * h];
#pragma unroll
      for (int e = 0; e < 4; ++e) s[4 * r4 + e] = exp2_fast(fmaf(s[4 * r4 + e], c, -l4[e]));
    }
    if (row < wave_key + 31 || row + 32 > len) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int i = row + row_of(r, h);
        s[r] = masked(s[r], i < key || i >= len, 0.0f);
      }
    }
    if constexpr (DK) {
#pragma unroll
      for (int r4 = 0; r4 < 4; ++r4) {
        const f32x4 d4 = *(const f32x4*)&lds.delta[x][r0 + 8 * r4 + 4 * h];
#pragma unroll
        for (int e = 0; e < 4; ++e) s[4 * r4 + e] *= dp[4 * r4 + e] - d4[e];
      }
    }
    scale.move(s, acc);
    const auto& by = DK ? lds.q[x] : lds.go[x];
    if constexpr (IN == 1) {
      block_add<T, D, UNIT>(by, r0, lane, s, acc);
    } else {
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        float p[8];
        frag w[W];
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = s[8 * st + e];
        planes_of<N>(p, w);
#pragma unroll
        for (int d = 0; d < DB; ++d) {
          if (32 * d >= (DK ? dk : dv)) continue;
          frag f[IN];
          by.cols(r0 + 16 * st, 32 * d, lane, f);
          acc[d] = mma_planes<N>(f, w, acc[d]);
        }
      }
    }
  };
  const int h0 = kvh * a.group, h1 = h0 + a.group;      // rows from the tile's first key on attend it
  __syncthreads();
  if (tid == 0) lds.bad = 0;
  int head = h0, row = part.from, x = 0;
  fetch(0, head, row);
  stage(0);
  direct_wait();
  __syncthreads();
  while (head < h1) {
    int nh = head, nr = row + BR;
    if (nr >= part.to) {
      nr = part.from;
      ++nh;
    }
    if (nh < h1) fetch(x ^ 1, nh, nr);
#pragma unroll 1
    for (int r0 = 0; r0 < BR; r0 += 32)
      if (wave_on && row + r0 + 31 >= wave_key && row + r0 < part.to) compute(x, row + r0, r0);
    if (nh < h1) stage(x ^ 1);
    direct_wait();
    __syncthreads();
    x ^= 1;
    head = nh;
    row = nr;
  }
  const bool store = block + (lane & 31) < count;
  if (store && any_not_finite(acc)) lds.bad = 1;
  __syncthreads();
  if (lds.bad) {
    if (!DK) careful_dkv<T>(a, at.t0, first, count, kvh, PAIRS, split, part);
    return;
  }
  if (!store) return;
  const float f = (DK ? a.scale : 1.0f) / scale.by;
  const int dim = DK ? dk : dv;
  const int64_t sum = ((int64_t)split * a.tokens + at.t0 + key) * a.kv_heads + kvh;
  float* parts = a.nsplit == 1 ? nullptr : DK ? a.part_k + sum * dk : a.part_v + sum * dv;
  T* to = DK ? (T*)a.dk_ + (at.t0 + key) * a.dk_ts + kvh * a.dk_hs : (T*)a.dv_ + (at.t0 + key) * a.dv_ts + kvh * a.dv_hs;
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int e = 32 * d + 8 * r + 4 * h;
      const float y[4] = {acc[d][4 * r] * f, acc[d][4 * r + 1] * f, acc[d][4 * r + 2] * f, acc[d][4 * r + 3] * f};
      if (parts) store4<float>(parts + e, y, dim - e);
      else store4<T>(to + e, y, dim - e);
    }
}

template <typename T, int D, FitMode MODE>
__global__ __launch_bounds__(128 * PAIRS, MODE == ANY || (PairShape<T, D>::F32 && D > 64) ? 1 : 2) void attn_dkv(AttnArgs a, int64_t slots) {
  __shared__ typename PairShape<T, D>::Lds lds;
  for (int64_t b = blockIdx.x; b < slots * a.nsplit * a.kv_heads; b += gridDim.x) {
    const auto [kvh, split, slot] = block_of(b, a.kv_heads, slots);
    const SeqTile at = find_tile(a.cu, a.seqs, a.tokens, 1, PairShape<T, D>::KEYS, slot);
    if (at.seq < 0 || at.tile * PairShape<T, D>::KEYS >= at.len) continue;
    // (both parts pass the same barriers)
    if (__builtin_amdgcn_readfirstlane(threadIdx.x >> 6) >= PAIRS) pair_tile<T, D, MODE, true>(lds, a, at, kvh, split);
    else pair_tile<T, D, MODE, false>(lds, a, at, kvh, split);
  }
}

template <typename T>
void bwd(const AttnArgs& a, hipStream_t s) {
  auto grid = [&](int64_t slots) { return dim3((uint32_t)std::min<int64_t>(slots * a.nsplit * a.kv_heads, 1 << 22)); };
  by_fit(fit_of<T>(a, false, true), [&](auto d, auto mode) {
    constexpr int D = decltype(d)::value;
    constexpr FitMode MODE = decltype(mode)::value;
    const int64_t rows = a.tokens * a.group / ATTN_ROWS + a.seqs;
    launch_kernel(attn_dq<T, D, MODE>, grid(rows), dim3(256), 0, s, a, rows);
    const int64_t keys = a.tokens / PairShape<T, D>::KEYS + a.seqs;
    launch_kernel(attn_dkv<T, D, MODE>, grid(keys), dim3(PairShape<T, D>::NT), 0, s, a, keys);
  });
}

// Sums over the parts: a wave takes a token's heads of dq, dk and dv in turn.  Token i of its sequence has parts of
// dq up to its own position, and of dk and dv from there on.
template <typename T>
__global__ __launch_bounds__(256) void attn_sum(AttnArgs a) {
  const int lane = threadIdx.x & 63, heads = a.kv_heads * a.group, all = heads + 2 * a.kv_heads;
  const int64_t t0 = a.cu ? seq_start(a.cu, 0, a.tokens) : 0, t1 = a.cu ? seq_start(a.cu, a.seqs, a.tokens) : a.tokens;
  for (int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); i < a.tokens * all; i += (int64_t)gridDim.x * 4) {
    const int64_t t = i / all;
    int h = (int)(i - t * all);
    if (t < t0 || t >= t1) continue;
    const SeqTile seq = find_token(a.cu, a.seqs, a.tokens, t);
    const int64_t at = t - seq.t0;
    const int mine = (int)min(at / a.part_len, (int64_t)a.nsplit - 1), last = (int)min((seq.len - 1) / a.part_len, (int64_t)a.nsplit - 1);
    auto sum = [&](const float* part, int n, int dim, int from, int to, void* out, int64_t ts, int64_t hs) {
      const int64_t step = a.tokens * n * dim;
      const float* p = part + (t * n + h) * dim;
      for (int d = lane; d < dim; d += 64) {
        float x = 0.0f;
        for (int s = from; s <= to; s += 4) {      // (in the parts' order, four in flight)
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = p[min(s + e, to) * step + d];
#pragma unroll
          for (int e = 0; e < 4; ++e) x += s + e <= to ? v[e] : 0.0f;
        }
        ((T*)out)[t * ts + h * hs + d] = from_f32<T>(x);
      }
    };
    if (h < heads) sum(a.part, heads, a.dk, 0, mine, a.dq, a.dq_ts, a.dq_hs);
    else if ((h -= heads) < a.kv_heads) sum(a.part_k, a.kv_heads, a.dk, mine, last, a.dk_, a.dk_ts, a.dk_hs);
    else {
      h -= a.kv_heads;
      sum(a.part_v, a.kv_heads, a.dv, mine, last, a.dv_, a.dv_ts, a.dv_hs);
    }
  }
}

}  // namespace

void launch_attn_sum(const AttnArgs& a, int dtype, hipStream_t s) {
  const int64_t rows = a.tokens * (a.kv_heads * (a.group + 2));
  const dim3 grid((uint32_t)std::min<int64_t>((rows + 3) / 4, 1 << 22));
  if (dtype == PC_DTYPE_BF16) launch_kernel(attn_sum<bf16>, grid, dim3(256), 0, s, a);
  else if (dtype == PC_DTYPE_F16) launch_kernel(attn_sum<f16>, grid, dim3(256), 0, s, a);
  else launch_kernel(attn_sum<float>, grid, dim3(256), 0, s, a);
}

void launch_attn_bwd(const AttnArgs& a, int dtype, hipStream_t s) {
  if (dtype == PC_DTYPE_BF16) bwd<bf16>(a, s);
  else if (dtype == PC_DTYPE_F16) bwd<f16>(a, s);
  else bwd<float>(a, s);
}

}  // namespace pc
