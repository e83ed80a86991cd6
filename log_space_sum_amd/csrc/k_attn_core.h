// k_attn_core.h -- attention of a tile of rows over a range of keys: the loop of
// the forward kernels (whole sequences: k_attn_fwd.hip; a cache in pages: k_attn_cached.hip).
#pragma once
#include "k_attn.h"

namespace pc {

// Where the keys and values of one (sequence, shared head) lie.  Position j of a
// sequence is, with `past` of them in the cache: page table[j / page] row j % page
// below `past`, the new token j - past from there on.
template <typename T, bool PAGED>
struct Keys {
  const T *k, *v;            // the new tokens' first row
  int64_t k_ts, v_ts;
  int past, total;           // positions: in the cache, all
  const T *kc, *vc;          // the cache, at the head
  const int32_t* table;      // the sequence's
  int64_t k_page, k_row, v_page, v_row;     // strides in the cache
  int num_pages, page_size;
  uint32_t magic, shift;     // j / page_size = j magic >> shift

  // Page and row of cached position j; false where the table names no page.
  __device__ __forceinline__ bool place(int j, int64_t& page, int& row) const {
    const int i = (int)(((uint64_t)(uint32_t)j * magic) >> shift);
    row = j - i * page_size;
    const int p = table[i];
    page = p;
    return (uint32_t)p < (uint32_t)num_pages;
  }
  // Rows of position j (any other where j is behind the last, or in no page: false then).
  __device__ __forceinline__ bool find(int j, const T*& kr, const T*& vr) const {
    j = min(j, total - 1);
    if constexpr (PAGED) {
      if (j < past) {
        int64_t page;
        int row;
        if (place(j, page, row)) {
          kr = kc + page * k_page + (int64_t)row * k_row;
          vr = vc + page * v_page + (int64_t)row * v_row;
          return true;
        }
        kr = k;
        vr = v;
        return false;
      }
      j -= past;
    }
    kr = k + (int64_t)j * k_ts;
    vr = v + (int64_t)j * v_ts;
    return true;
  }
  // The same in two steps, so that a tile's pages are looked up a tile ahead: where position j lies, and the rows of a
  // place.  Nothing is made of the page in the first, which would wait for it.
  struct Place {
    int page, row;         // row < 0: the new token -1 - row
  };
  __device__ __forceinline__ Place locate(int j) const {
    j = min(j, total - 1);
    const int i = (int)(((uint64_t)(uint32_t)j * magic) >> shift);
    Place at{0, past - 1 - j};
    if (j < past) at = {table[i], j - i * page_size};
    return at;
  }
  __device__ __forceinline__ bool none(Place at) const { return at.row >= 0 && (uint32_t)at.page >= (uint32_t)num_pages; }
  // The rows of keys and values; of a place in no page any.
  __device__ __forceinline__ const T* key_row(Place at) const { return row_of(at, kc, k_page, k_row, k, k_ts); }
  __device__ __forceinline__ const T* value_row(Place at) const { return row_of(at, vc, v_page, v_row, v, v_ts); }
  __device__ __forceinline__ const T* row_of(Place at, const T* cache, int64_t page, int64_t row, const T* fresh, int64_t ts) const {
    const bool cached = at.row >= 0 && !none(at);
    return (cached ? cache : fresh) + (cached ? at.page : 0) * page + (at.row < 0 ? -1 - at.row : cached ? at.row : 0) * (cached ? row : ts);
  }
  __device__ __forceinline__ bool there(int j) const {
    if constexpr (!PAGED) return true;
    int64_t page;
    int row;
    return j >= past || place(j, page, row);
  }
};

// The tile's rows: row i of it is token (rem + i) / group behind the tile's first, head
// (rem + i) % group of those that share.
template <typename T>
struct Rows {
  const T* q;                // the tile's first token, the first of the sharing heads
  int64_t q_ts, q_hs;
  int group, rem, count;
  int first;                 // position of the tile's first token

  __device__ __forceinline__ int token(int i) const { return (int)((uint32_t)(rem + i) / (uint32_t)group); }
  __device__ __forceinline__ int head(int i) const { return rem + i - token(i) * group; }
  __device__ __forceinline__ const T* row(int i) const { return q + token(i) * q_ts + head(i) * q_hs; }
  // the last position that row i attends
  __device__ __forceinline__ int last(int i) const { return first + token(i); }
};

// Results of a tile of rows: outputs, or what a split over the keys leaves to be joined.
struct RowOut {
  void* o;                   // as Rows::q
  int64_t o_ts, o_hs;
  float* lse;                // [tokens, heads] at the tile's first token and the first sharing head, nullable
  int heads;
  float* part;               // [tokens, heads, dv] of this split, at the same place, nullable: final
  float2* stat;              // [tokens, heads] (m, l): the weights are 2^(score - m), l is their sum
};
__device__ __forceinline__ void put_stat(const RowOut& out, int t, int h, float m, float l) {
  const int64_t at = (int64_t)t * out.heads + h;
  if (out.part) out.stat[at] = float2{m, l};
  else if (out.lse) out.lse[at] = (m + __log2f(l)) * LN2;
}

// A part without keys of these rows.
template <typename T>
__device__ __forceinline__ void no_keys(const Rows<T>& rows, const RowOut& out) {
  for (int i = threadIdx.x; i < rows.count; i += 256)
    out.stat[(int64_t)rows.token(i) * out.heads + rows.head(i)] = float2{-INFINITY, 0.0f};
}

// One row after the other in plain float32: the path of a tile whose results are not
// finite, since there a weight of 0 met an infinity or a NaN that the row may not
// attend, or planes of infinities gave NaN.  Waves take rows in turn.
template <typename T, bool PAGED>
__device__ __attribute__((noinline)) void careful_rows(Keys<T, PAGED> keys, Rows<T> rows, RowOut out, int dk, int dv,
                                                       float c, int key0, int key1, int nwaves) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int r = wave; r < rows.count; r += nwaves) {
    const T* q = rows.row(r);
    const int last = min(rows.last(r), key1 - 1), t = rows.token(r), h = rows.head(r);
    auto score = [&](int j) {
      const T *kr, *vr;
      if (j > last || !keys.find(j, kr, vr)) return -INFINITY;
      float s = 0.0f;
      for (int d = 0; d < dk; ++d) s = fmaf(to_f32(q[d]), to_f32(kr[d]), s);
      return s * c;
    };
    float m = -INFINITY;
    for (int j = key0 + lane; j <= last; j += 64) m = fmaxf(m, score(j));
    for (int x = 32; x; x >>= 1) m = fmaxf(m, __shfl_xor(m, x));
    const float shift = (float)Num<T>::BIAS - (m == -INFINITY ? 0.0f : m);
    float l = 0.0f, acc[2] = {0.0f, 0.0f};
    for (int j0 = key0; j0 <= last; j0 += 64) {
      const float s = score(j0 + lane);
      const bool on = j0 + lane <= last && keys.there(j0 + lane);
      const float p = on ? exp2_fast(s + shift) : 0.0f;
      l += p;
      for (int i = 0; i < min(64, last - j0 + 1); ++i) {
        const T *kr, *v;
        const float w = __shfl(p, i);
        if (!__shfl((int)on, i)) continue;
        keys.find(j0 + i, kr, v);
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (lane + 64 * e < dv) acc[e] = fmaf(w, to_f32(v[lane + 64 * e]), acc[e]);
      }
    }
    for (int x = 32; x; x >>= 1) l += __shfl_xor(l, x);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int d = lane + 64 * e;
      if (d >= dv) continue;
      if (out.part) out.part[((int64_t)t * out.heads + h) * dv + d] = acc[e];
      else ((T*)out.o)[t * out.o_ts + h * out.o_hs + d] = from_f32<T>(acc[e] / l);
    }
    if (lane == 0) put_stat(out, t, h, m == -INFINITY ? m : -shift, l);
  }
}

// A row's running maximum m (of scores before the factor c) and the shift in its weights 2^(c score + shift), which
// is kept as rounded: sums at an older maximum are carried on by the difference of the shifts exactly as they were used.
// Returns the factor of what was summed so far.
__device__ __forceinline__ float move_maximum(float& m, float& shift, float top, float c, float bias) {
  const float was = m, used = shift;
  m = fmaxf(m, top);
  shift = bias - (m == -INFINITY ? 0.0f : m * c);
  return was == -INFINITY ? 0.0f : exp2_fast(shift - used);
}

// The loop of a workgroup of four waves, each with 32 of the tile's 128 rows,
// over keys key0 .. key1 - 1 (key0 a multiple of the key tile) that are staged in
// LDS for all of them.
//
// Transposed, S^T = K Q^T, a lane holds one row's scores: its maximum and sum take
// one exchange of the wave's halves, and the weights are the operand of O^T = V^T P^T
// as they stand.
template <typename T, int D>
struct FwdShape {
  static constexpr int IN = Num<T>::IN, BK = IN == 3 ? 32 : 64, BUFS = IN == 3 ? 1 : 2;
  struct Lds {
    Tile<T, BK, D> k[BUFS], v[BUFS];
    int absent[BUFS];        // the first key of the last tile in this buffer that has a key in no page
  };
};

template <typename T, int D, FitMode MODE, bool PAGED>
__device__ __forceinline__ void attend_tile(typename FwdShape<T, D>::Lds& lds, const Keys<T, PAGED> keys, const Rows<T> rows,
                                            const RowOut out, int dk_, int dv_, float c, bool negative, int key0, int key1) {
  using N = Num<T>;
  using S = FwdShape<T, D>;
  constexpr int IN = N::IN, W = N::W, BK = S::BK, KB = BK / 32, BUFS = S::BUFS, DS = D / 16, DB = D / 32;
  constexpr int NT = 256, PER_ROW = Tile<T, 32, D>::P / 8, U = BK * PER_ROW / NT;
  constexpr bool UNIT = MODE == UNITS, DIRECT = IN == 1 && UNIT;
  const int dk = dk_, dv = dv_;
  const int tid = thread_here(), wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, h = lane >> 5;
  const int wave_first = 32 * wave, end = rows.count;
  const bool wave_on = wave_first < end;
  const int mine = min(wave_first + (lane & 31), end - 1);     // rows behind the last are that one again, and not stored
  const int last = rows.last(mine);
  // the last keys of the wave's first and last row
  const int first_last = rows.last(min(wave_first, end - 1)), last_last = rows.last(min(wave_first + 31, end - 1));

  frag q[DS][IN];
  {
    const T* p = rows.row(mine);
#pragma unroll
    for (int s = 0; s < DS; ++s) {
      frags_of(load_own<UNIT>(p, 16 * s + 8 * h, dk), q[s]);
      if (negative) {
#pragma unroll
        for (int i = 0; i < IN; ++i) {
          q[s][i].x ^= 0x80008000u;
          q[s][i].y ^= 0x80008000u;
          q[s][i].z ^= 0x80008000u;
          q[s][i].w ^= 0x80008000u;
        }
      }
    }
  }
  f32x16 o[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d) o[d] = f32x16{};
  float m = -INFINITY, shift = (float)N::BIAS, l = 0.0f;

  Unit<T> rk[DIRECT ? 1 : U], rv[DIRECT ? 1 : U];
  const DirectUnit<D> unit(tid);
  const int kbyte = unit.byte(dk), vbyte = unit.byte(dv);
  const uint32_t ok = (uint32_t)(unit.row * (int)keys.k_ts * 2 + kbyte), ov = (uint32_t)(unit.row * (int)keys.v_ts * 2 + vbyte);
  typename Keys<T, PAGED>::Place next{};
  if (DIRECT && PAGED && key0 < key1) next = keys.locate(key0 + lane);
  static_assert(!(DIRECT && PAGED) || BK == 64, "a lane a key");
  const int in_cache = keys.num_pages > 0 ? keys.past : 0;     // positions whose rows may be any page's
  auto load = [&](int b, int key) {
    const uint32_t kb = lds_byte(lds.k[b].at) + wave * 1024, vb = lds_byte(lds.v[b].at) + wave * 1024;
    if constexpr (PAGED) {
      uint64_t kr, vr;       // rows of position key + lane
      if (key + BK <= in_cache) {
        // (all in the cache, strides of 32 bits: a quarter of the general form's instructions, of which a tile has
        // as many as its matrix instructions leave room for; four chunks of 512 behind 8192 562 us, 575 without.  A key
        // in no page takes page 0, which a cache without pages does not have.)
        const uint32_t page = keys.none(next) ? 0u : (uint32_t)next.page, row = (uint32_t)next.row;
        kr = (uint64_t)keys.kc + (uint64_t)page * (uint32_t)(2 * keys.k_page) + (uint64_t)row * (uint32_t)(2 * keys.k_row);
        vr = (uint64_t)keys.vc + (uint64_t)page * (uint32_t)(2 * keys.v_page) + (uint64_t)row * (uint32_t)(2 * keys.v_row);
      } else {
        kr = (uint64_t)keys.key_row(next);
        vr = (uint64_t)keys.value_row(next);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = unit.row + u * unit.STEP;
        lds_load16_at((const char*)__shfl(kr, r) + kbyte, kb + u * 4096);
        lds_load16_at((const char*)__shfl(vr, r) + vbyte, vb + u * 4096);
      }
      if (keys.none(next)) lds.absent[b] = key;
      if (key + BK < key1) next = keys.locate(key + BK + lane);
    } else {
      const T *kr = keys.k + (int64_t)key * keys.k_ts, *vr = keys.v + (int64_t)key * keys.v_ts;
      if (key + BK <= keys.total) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          lds_load16(kr + u * unit.STEP * keys.k_ts, ok, kb + u * 4096);
          lds_load16(vr + u * unit.STEP * keys.v_ts, ov, vb + u * 4096);
        }
      } else {       // rows behind the last are that one again
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int row = min(unit.row + u * unit.STEP, keys.total - 1 - key);
          lds_load16(kr, (uint32_t)(row * (int)keys.k_ts * 2 + kbyte), kb + u * 4096);
          lds_load16(vr, (uint32_t)(row * (int)keys.v_ts * 2 + vbyte), vb + u * 4096);
        }
      }
    }
  };
  bool absent = false;
  auto fetch = [&](int key) {
    absent = false;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int id = u * NT + tid, row = id / PER_ROW, d = id % PER_ROW * 8;
      const T *kr, *vr;
      absent |= !keys.find(key + row, kr, vr);
      rk[u] = load_unit<UNIT>(kr, d, dk);
      rv[u] = load_unit<UNIT>(vr, d, dv);
    }
  };
  auto stage = [&](int b, int key) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int id = u * NT + tid, row = id / PER_ROW, d = id % PER_ROW * 8;
      lds.k[b].put(row, d, rk[u]);
      lds.v[b].put(row, d, rv[u]);
    }
    if (PAGED && absent) lds.absent[b] = key;
  };
  auto compute = [&](int b, int key) {
    f32x16 s[KB];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) s[kb] = f32x16{};
#pragma unroll
    for (int st = 0; st < DS; ++st) {
      if (IN == 3 && 32 * (st / 2) >= dk) continue;
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        frag a[IN];
        lds.k[b].rows(32 * kb, st, lane, a);
        s[kb] = mma_planes<N>(a, q[st], s[kb]);
      }
    }
    if (key + BK - 1 > first_last) {
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          s[kb][r] = masked(s[kb][r], key + 32 * kb + row_of(r, h) > last);
    }
    if (PAGED && lds.absent[b] == key) {
      const uint64_t gone = __ballot(lane < BK && !keys.there(key + lane));
#pragma unroll
      for (int kb = 0; kb < KB; ++kb)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          s[kb][r] = masked(s[kb][r], gone >> (32 * kb + row_of(r, h)) & 1);
    }
    float top = s[0][0];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int r = 0; r < 16; ++r) top = fmaxf(top, s[kb][r]);
    top = max_halves(top);
    if (__any(!(top <= m))) {
      const float f = move_maximum(m, shift, top, c, (float)N::BIAS);
      l *= f;
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[d][r] *= f;
    }
    if constexpr (IN == 1) {
      // 16 keys a step; the next step's weights are made and its values read between this one's matrix instructions
      constexpr int STEPS = 2 * KB;
      auto weights = [&](int step, frag (&w)[W]) {
        float p[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          p[e] = exp2_fast(fmaf(s[step >> 1][8 * (step & 1) + e], c, shift));
          l += p[e];
        }
        planes_of<N>(p, w);
      };
      auto values = [&](int step, frag (&a)[DB][IN]) {
#pragma unroll
        for (int d = 0; d < DB; ++d)
          lds.v[b].cols(16 * step, 32 * d, lane, a[d]);
      };
      frag w[W], a[DB][IN];
      values(0, a);
      weights(0, w);
#pragma unroll
      for (int step = 0; step < STEPS; ++step) {
        frag wn[W], an[DB][IN];
        if (step + 1 < STEPS) {
          values(step + 1, an);
          weights(step + 1, wn);
        }
#pragma unroll
        for (int p = W - 1; p >= 0; --p)
#pragma unroll
          for (int d = 0; d < DB; ++d)
            o[d] = N::mma(a[d][0], w[p], o[d]);
        if (step + 1 < STEPS) {
          __builtin_amdgcn_sched_group_barrier(0x100, 2 * DB, 0);
#pragma unroll
          for (int i = 0; i < W * DB; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x2 | 0x400, (24 + 16 * W + W * DB - 1) / (W * DB), 0);
          }
        }
        if (step + 1 < STEPS) {
#pragma unroll
          for (int p = 0; p < W; ++p) w[p] = wn[p];
#pragma unroll
          for (int d = 0; d < DB; ++d) a[d][0] = an[d][0];
        }
      }
      return;
    }
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        float p[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          p[e] = exp2_fast(fmaf(s[kb][8 * st + e], c, shift));
          l += p[e];
        }
        frag w[W];
        planes_of<N>(p, w);
#pragma unroll
        for (int d = 0; d < DB; ++d) {
          if (32 * d >= dv) continue;
          frag a[IN];
          lds.v[b].cols(32 * kb + 16 * st, 32 * d, lane, a);
          o[d] = mma_planes<N>(a, w, o[d]);
        }
      }
  };

  __syncthreads();                 // the last tile's readers are done
  if (PAGED && tid < BUFS) lds.absent[tid] = -1;
  if constexpr (DIRECT) {
    if (PAGED) __syncthreads();
    if (key0 < key1) load(0, key0);
    direct_wait();
    __syncthreads();
    int b = 0;
    for (int key = key0; key < key1; key += BK, b ^= 1) {
      if (key + BK < key1) load(b ^ 1, key + BK);
      if (wave_on && key <= last_last) compute(b, key);
      direct_wait();
      __syncthreads();
    }
  } else if constexpr (BUFS == 2) {
    if (key0 < key1) fetch(key0);
    if (PAGED) __syncthreads();
    if (key0 < key1) stage(0, key0);
    __syncthreads();
    int b = 0;
    for (int key = key0; key < key1; key += BK, b ^= 1) {
      const bool more = key + BK < key1;
      if (more) fetch(key + BK);
      if (wave_on && key <= last_last) compute(b, key);
      if (more) stage(b ^ 1, key + BK);
      __syncthreads();
    }
  } else {
    if (key0 < key1) fetch(key0);
    if (PAGED) __syncthreads();
    for (int key = key0; key < key1; key += BK) {
      stage(0, key);
      __syncthreads();
      if (key + BK < key1) fetch(key + BK);
      if (wave_on && key <= last_last) compute(0, key);
      __syncthreads();
    }
  }

  l = add_halves(l);
  const bool store = wave_first + (lane & 31) < end;
  float bad = l * 0.0f;
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int r = 0; r < 16; ++r) bad = fmaf(o[d][r], 0.0f, bad);
  if (__syncthreads_or(store && !(bad == 0.0f))) {
    careful_rows<T, PAGED>(keys, rows, out, dk, dv, negative ? -c : c, key0, key1, 4);
    return;
  }
  if (!store) return;
  const int t = rows.token(mine), head = rows.head(mine);
  if (h == 0) put_stat(out, t, head, m == -INFINITY ? m : -shift, l);
  const float inv = out.part ? 1.0f : 1.0f / l;
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int at = 32 * d + 8 * r + 4 * h;
      const float x[4] = {o[d][4 * r] * inv, o[d][4 * r + 1] * inv, o[d][4 * r + 2] * inv, o[d][4 * r + 3] * inv};
      if (out.part) store4<float>(out.part + ((int64_t)t * out.heads + head) * dv + at, x, dv - at);
      else store4<T>((T*)out.o + t * out.o_ts + head * out.o_hs + at, x, dv - at);
    }
}

}  // namespace pc
