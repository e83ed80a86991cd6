// k_attn_cached.hip -- softmax attention of new tokens over a cache in pages, which they join.
//
// Two forms.  Many rows (new tokens times the heads that share a key / value head): the loop
// of whole sequences, with keys found through the page table.  Few rows: the four
// waves of a workgroup share up to 32 rows and take key tiles of their own in turn, so that a
// single token has as many loads in flight as a long one; their results are
// joined in LDS.  Long caches are cut into parts of a fixed number of keys, so streams of
// different lengths give workgroups of equal work; a second kernel joins the parts.
//
// What bounds it.  Few rows: memory; 64 streams of up to 8192 tokens x 32 (8) heads x 128 bfloat16, a token each, take 235 us
// (3.7 TB/s; a sum over a tensor reads 4.0).  Many: matrix instructions, as whole sequences; four chunks of 512 behind 8192 x 32 (8)
// heads x 128 bfloat16 562 us, 1.01 PFLOP/s of its four products' work.  One token behind 1000 x 16 (4) heads x 64: 9.5 us and 3.5
// for joining, the chain of sequence, page, rows, two tiles, exchange.
//
// The new keys and values are read from their tensors, not from the cache, so storing
// them needs no launch in front: the workgroup of a token's first row does it.
#include <algorithm>

#include "k_attn_core.h"

namespace pc {
namespace {

// What a workgroup works on; count 0: nothing.
template <typename T>
struct Work {
  Keys<T, true> keys;
  Rows<T> rows;
  RowOut out;
  int key0, key1;
};
template <typename T>
__device__ __forceinline__ Work<T> find_work(const AttnArgs& a, int64_t slot, int kvh, int split, int tile) {
  Work<T> w;
  w.rows.count = 0;
  const SeqTile at = find_tile(a.cu, a.seqs, a.tokens, a.group, tile, slot);
  const int64_t first = at.tile * tile, rows_all = at.len * a.group;
  if (at.seq < 0 || first >= rows_all) return w;
  const int heads = a.kv_heads * a.group;
  const int64_t tf = first / a.group, t = at.t0 + tf;
  const int past = min(max(a.pages.past[at.seq], 0), a.pages.max_pages * a.pages.page_size);
  w.rows.q = (const T*)a.q.p + t * a.q.ts + (int64_t)kvh * a.group * a.q.hs;
  w.rows.q_ts = a.q.ts;
  w.rows.q_hs = a.q.hs;
  w.rows.group = a.group;
  w.rows.rem = (int)(first - tf * a.group);
  w.rows.count = (int)min((int64_t)tile, rows_all - first);
  w.rows.first = past + (int)tf;
  w.keys.k = (const T*)a.k.p + at.t0 * a.k.ts + kvh * a.k.hs;
  w.keys.v = (const T*)a.v.p + at.t0 * a.v.ts + kvh * a.v.hs;
  w.keys.k_ts = a.k.ts;
  w.keys.v_ts = a.v.ts;
  w.keys.past = past;
  w.keys.total = past + (int)at.len;
  w.keys.kc = (const T*)a.pages.k.p + kvh * a.pages.k.head_stride;
  w.keys.vc = (const T*)a.pages.v.p + kvh * a.pages.v.head_stride;
  w.keys.table = a.pages.table + at.seq * a.pages.table_stride;
  w.keys.k_page = a.pages.k.page_stride;
  w.keys.k_row = a.pages.k.token_stride;
  w.keys.v_page = a.pages.v.page_stride;
  w.keys.v_row = a.pages.v.token_stride;
  w.keys.num_pages = a.pages.num_pages;
  w.keys.page_size = a.pages.page_size;
  w.keys.magic = a.pages.magic;
  w.keys.shift = a.pages.shift;
  w.out = RowOut{};
  w.out.o = (T*)a.o + t * a.o_ts + (int64_t)kvh * a.group * a.o_hs;
  w.out.o_ts = a.o_ts;
  w.out.o_hs = a.o_hs;
  w.out.heads = heads;
  if (a.nsplit > 1) {
    const int64_t place = ((int64_t)split * a.tokens + t) * heads + kvh * a.group;
    w.out.part = a.part + place * a.dv;
    w.out.stat = a.stat + place;
  }
  const int end = w.rows.last(w.rows.count - 1) + 1;
  w.key0 = a.nsplit > 1 ? (int)min((int64_t)split * a.part_len, (int64_t)end) : 0;
  w.key1 = a.nsplit > 1 && split + 1 < a.nsplit ? (int)min((int64_t)(split + 1) * a.part_len, (int64_t)end) : end;
  return w;
}

// The tile's tokens join the cache (a token on two tiles is the first one's).
template <typename T>
__device__ __forceinline__ void join_cache(const AttnArgs& a, const Work<T>& w, int kvh) {
  const int past_tile = w.rows.first - w.keys.past;       // the tile's first token among the new ones
  const int t0 = w.rows.rem ? 1 : 0, n = w.rows.token(w.rows.count - 1) + 1 - t0;
  if (n <= 0) return;
  const int cap = a.pages.max_pages * a.pages.page_size;
  auto copy = [&](const T* from, int64_t ts, const AttnCache& c, int dim) {
    for (int e = threadIdx.x; e < n * dim; e += 256) {
      const int i = (int)((uint32_t)e / (uint32_t)dim), d = e - i * dim, t = past_tile + t0 + i, pos = w.keys.past + t;
      int64_t page;
      int row;
      if (pos < cap && w.keys.place(pos, page, row))
        ((T*)c.p)[page * c.page_stride + (int64_t)row * c.token_stride + kvh * c.head_stride + d] = from[(int64_t)t * ts + d];
    }
  };
  copy(w.keys.k, a.k.ts, a.pages.k, a.dk);
  copy(w.keys.v, a.v.ts, a.pages.v, a.dv);
}

template <typename T, int D, FitMode MODE>
__global__ __launch_bounds__(256, (Num<T>::IN == 3 || MODE == ANY) && D > 64 ? 1 : 2) void attn_cached_many(AttnArgs a, int64_t slots) {
  __shared__ typename FwdShape<T, D>::Lds lds;
  const int64_t per = (int64_t)a.kv_heads * a.nsplit;
  for (int64_t b = blockIdx.x; b < slots * per; b += gridDim.x) {
    const int kvh = (int)(b % a.kv_heads), split = (int)(b / a.kv_heads % a.nsplit);
    const int64_t slot = b / per;
    const Work<T> w = find_work<T>(a, slots - 1 - slot, kvh, split, ATTN_ROWS);
    if (w.rows.count == 0) continue;
    if (w.key0 >= w.key1) no_keys(w.rows, w.out);
    else
      attend_tile<T, D, MODE, true>(lds, w.keys, w.rows, w.out, a.dk, a.dv, fabsf(a.scale) * LOG2E, a.scale < 0.0f, w.key0, w.key1);
    if (split == 0) join_cache(a, w, kvh);
  }
}

template <typename T, int D>
struct FewShape {
  struct Lds {
    union {
      Tile<T, 32, D> own[4];          // each wave's: keys, then values
      alignas(16) float acc[4][32][D + 4];
    };
    float2 stat[4][32];
  };
};

__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}
template <typename T, int D, FitMode MODE>
__global__ __launch_bounds__(256, Num<T>::IN == 3 || (MODE == ANY && D > 64) ? 1 : 2) void attn_cached_few(AttnArgs a, int64_t slots) {
  using N = Num<T>;
  constexpr bool UNIT = MODE == UNITS;
  constexpr int IN = N::IN, W = N::W, DS = D / 16, DB = D / 32, PER_ROW = Tile<T, 32, D>::P / 8, U = 32 * PER_ROW / 64;
  __shared__ typename FewShape<T, D>::Lds lds;
  const int64_t per = (int64_t)a.kv_heads * a.nsplit;
  const int dk = a.dk, dv = a.dv;
  const float c = fabsf(a.scale) * LOG2E;
  for (int64_t b = blockIdx.x; b < slots * per; b += gridDim.x) {
    // parts, which are alike here, lie side by side (as the slowest index: 64 streams of up to 8192 252 us for 235)
    const int kvh = (int)(b % a.kv_heads), split = (int)(b / a.kv_heads % a.nsplit);
    const int64_t slot = b / per;
    const Work<T> w = find_work<T>(a, slot, kvh, split, ATTN_FEW_ROWS);
    if (w.rows.count == 0) continue;
    if (w.key0 >= w.key1) {
      no_keys(w.rows, w.out);
      continue;
    }
    const int tid = thread_here(), wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, h = lane >> 5;
    const int mine = min(lane & 31, w.rows.count - 1), last = w.rows.last(mine), first_last = w.rows.last(0);
    frag q[DS][IN];
    {
      const T* p = w.rows.row(mine);
#pragma unroll
      for (int s = 0; s < DS; ++s) {
        frags_of(load_own<UNIT>(p, 16 * s + 8 * h, dk), q[s]);
        if (a.scale < 0.0f) {
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

    // Rows are read whole, 16 lanes a row of 128, and go through the wave's part of LDS (a lane with its own key's
    // row would touch each line four times).  The next tile's rows are in flight over a whole tile, its pages looked up a
    // tile before that.  A lane knows where one row lies: of the tile's keys, or (lanes from 32 on) of its values.
    Unit<T> rk[U], rv[U];
    uint32_t absent = 0;     // keys of the tile in no page
    typename Keys<T, true>::Place place{};
    uint64_t row_at = 0;
    auto fetch_keys = [&] {
      const uint64_t keys_at = (uint64_t)w.keys.key_row(place), values_at = (uint64_t)w.keys.value_row(place);
      row_at = h ? values_at : keys_at;
      absent = (uint32_t)__ballot(w.keys.none(place));
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int id = u * 64 + lane;
        rk[u] = load_unit<UNIT>(global_row<T>(__shfl(row_at, id / PER_ROW)), id % PER_ROW * 8, dk);
      }
    };
    auto fetch_values = [&](int key) {
      // (asked for in front of the values, which need not be there when it is used)
      if (key + 128 < w.key1) place = w.keys.locate(key + 128 + (lane & 31));
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int id = u * 64 + lane;
        rv[u] = load_unit<UNIT>(global_row<T>(__shfl(row_at, 32 + id / PER_ROW)), id % PER_ROW * 8, dv);
      }
    };
    auto put = [&](const Unit<T>(&x)[U]) {
      lds.own[wave].template put_all<64>(lane, x);
      wave_fence();
    };
    __syncthreads();          // the last work's readers are done
    int key = w.key0 + 32 * wave;
    // (also a wave without a tile, of the last row: with a branch, the rows of q would be waited for as the last loads)
    place = w.keys.locate(key + (lane & 31));
    fetch_keys();
    fetch_values(key);
    for (bool more = key < w.key1; more; key += 128) {
      const uint32_t gone = absent;
      f32x16 s;
      auto scores = [&] {
        int here = lane;     // (addresses are made again: held over the loop, they would cost a load in flight)
        asm volatile("" : "+v"(here));
        s = f32x16{};
#pragma unroll
        for (int st = 0; st < DS; ++st) {
          if (IN == 3 && 32 * (st / 2) >= dk) continue;
          frag f[IN];
          lds.own[wave].rows(0, st, here, f);
          s = mma_planes<N>(f, q[st], s);
        }
        wave_fence();
      };
      more = key + 128 < w.key1;
      put(rk);
      // (two copies: with a branch at either fetch, the keys would be waited for as if no values came behind them)
      if (more) {
        fetch_keys();
        scores();
        put(rv);
        fetch_values(key + 128);
      } else {
        scores();
        put(rv);
      }
      if (key + 31 > first_last || gone) {
#pragma unroll
        for (int r = 0; r < 16; ++r)
          s[r] = masked(s[r], key + row_of(r, h) > last || (gone >> row_of(r, h) & 1));
      }
      float top = s[0];
#pragma unroll
      for (int r = 1; r < 16; ++r) top = fmaxf(top, s[r]);
      top = max_halves(top);
      if (__any(!(top <= m))) {
        const float f = move_maximum(m, shift, top, c, (float)N::BIAS);
        l *= f;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int r = 0; r < 16; ++r) o[d][r] *= f;
      }
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        float p[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          p[e] = exp2_fast(fmaf(s[8 * st + e], c, shift));
          l += p[e];
        }
        frag x[W];
        planes_of<N>(p, x);
#pragma unroll
        for (int d = 0; d < DB; ++d) {
          frag f[IN];
          lds.own[wave].cols(16 * st, 32 * d, lane, f);
          o[d] = mma_planes<N>(f, x, o[d]);
        }
      }
      wave_fence();
    }
    l = add_halves(l);
    __syncthreads();
    if (h == 0) lds.stat[wave][lane] = float2{m == -INFINITY ? m : -shift, l};
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        *(f32x4*)&lds.acc[wave][lane & 31][32 * d + 8 * r + 4 * h] = f32x4{o[d][4 * r], o[d][4 * r + 1], o[d][4 * r + 2], o[d][4 * r + 3]};
    __syncthreads();
    // eight threads a row join the waves'
    const int row = tid >> 3;
    float top = -INFINITY, sum = 0.0f, f[4], x[D / 32][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) top = fmaxf(top, lds.stat[i][row].x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = lds.stat[i][row].x == -INFINITY ? 0.0f : exp2_fast(lds.stat[i][row].x - top);
      sum += f[i] * lds.stat[i][row].y;
    }
    float bad = sum * 0.0f;
#pragma unroll
    for (int e = 0; e < D / 32; ++e) {
      f32x4 v = f32x4{};
#pragma unroll
      for (int i = 0; i < 4; ++i) v += f[i] * *(const f32x4*)&lds.acc[i][row][4 * (tid & 7) + 32 * e];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        x[e][r] = v[r];
        bad = fmaf(v[r], 0.0f, bad);
      }
    }
    const bool store = row < w.rows.count;
    if (__syncthreads_or(store && !(bad == 0.0f))) {
      careful_rows<T, true>(w.keys, w.rows, w.out, dk, dv, a.scale * LOG2E, w.key0, w.key1, 4);
    } else if (store) {
      const int t = w.rows.token(row), head = w.rows.head(row);
      if ((tid & 7) == 0) put_stat(w.out, t, head, top, sum);
      const float inv = w.out.part ? 1.0f : 1.0f / sum;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) {
        const int d = 4 * (tid & 7) + 32 * e;
#pragma unroll
        for (int r = 0; r < 4; ++r) x[e][r] *= inv;
        if (w.out.part) store4<float>(w.out.part + ((int64_t)t * w.out.heads + head) * dv + d, x[e], dv - d);
        else store4<T>((T*)w.out.o + t * w.out.o_ts + head * w.out.o_hs + d, x[e], dv - d);
      }
    }
    // (behind the results: in front, its loads would be waited for before the first keys')
    if (split == 0) join_cache(a, w, kvh);
  }
}

// Joins the parts of a row: a wave each.
template <typename T>
__global__ __launch_bounds__(256) void attn_join(AttnArgs a) {
  const int heads = a.kv_heads * a.group, lane = threadIdx.x & 63;
  const int64_t n = a.tokens * heads;
  const int64_t t0 = a.cu ? seq_start(a.cu, 0, a.tokens) : 0, t1 = a.cu ? seq_start(a.cu, a.seqs, a.tokens) : a.tokens;
  for (int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); i < n; i += (int64_t)gridDim.x * 4) {
    const int64_t t = i / heads;
    const int h = (int)(i - t * heads);
    if (t < t0 || t >= t1) continue;
    // a lane a part
    const float2 st = lane < a.nsplit ? a.stat[lane * n + i] : float2{-INFINITY, 0.0f};
    const bool on = !(st.x == -INFINITY && st.y == 0.0f);
    const uint64_t active = __ballot(on);
    float top = st.x;
    for (int x = 32; x; x >>= 1) top = fmaxf(top, __shfl_xor(top, x));
    const float f = on ? exp2_fast(st.x - top) : 0.0f;
    float l = f * st.y, acc[2] = {0.0f, 0.0f};
    for (int x = 32; x; x >>= 1) l += __shfl_xor(l, x);
    // four parts in flight; a part without keys has nothing written
    for (int s0 = 0; s0 < a.nsplit; s0 += 4) {
      float v[4][2];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        v[x][0] = v[x][1] = 0.0f;
        if (!(active >> (s0 + x) & 1)) continue;
        const float* p = a.part + ((s0 + x) * n + i) * a.dv;
#pragma unroll
        for (int e = 0; e < 2; ++e) v[x][e] = p[min(lane + 64 * e, a.dv - 1)];
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float w = __shfl(f, s0 + x);
        if (!(active >> (s0 + x) & 1)) continue;
#pragma unroll
        for (int e = 0; e < 2; ++e) acc[e] = fmaf(w, v[x][e], acc[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (lane + 64 * e < a.dv) ((T*)a.o)[t * a.o_ts + h * a.o_hs + lane + 64 * e] = from_f32<T>(acc[e] / l);
    if (a.lse && lane == 0) a.lse[i] = (top + __log2f(l)) * LN2;
  }
}

template <typename T>
void cached(const AttnArgs& a, bool few, hipStream_t s) {
  const int64_t slots = a.tokens * a.group / (few ? ATTN_FEW_ROWS : ATTN_ROWS) + a.seqs;
  const dim3 grid((uint32_t)std::min<int64_t>(slots * a.kv_heads * a.nsplit, 1 << 23));
  by_fit(fit_of<T>(a, true), [&](auto d, auto mode) {
    constexpr int D = decltype(d)::value;
    constexpr FitMode MODE = decltype(mode)::value;
    if (!few) launch_kernel(attn_cached_many<T, D, MODE>, grid, dim3(256), 0, s, a, slots);
    else launch_kernel(attn_cached_few<T, D, MODE>, grid, dim3(256), 0, s, a, slots);
  });
}

}  // namespace

void launch_attn_cached(const AttnArgs& a, int dtype, bool few, hipStream_t s) {
  if (dtype == PC_DTYPE_BF16) cached<bf16>(a, few, s);
  else if (dtype == PC_DTYPE_F16) cached<f16>(a, few, s);
  else cached<float>(a, few, s);
}

void launch_attn_join(const AttnArgs& a, int dtype, hipStream_t s) {
  const int64_t rows = a.tokens * a.kv_heads * a.group;
  const dim3 grid((uint32_t)std::min<int64_t>((rows + 3) / 4, 1 << 22));
  if (dtype == PC_DTYPE_BF16) launch_kernel(attn_join<bf16>, grid, dim3(256), 0, s, a);
  else if (dtype == PC_DTYPE_F16) launch_kernel(attn_join<f16>, grid, dim3(256), 0, s, a);
  else launch_kernel(attn_join<float>, grid, dim3(256), 0, s, a);
}

}  // namespace pc
