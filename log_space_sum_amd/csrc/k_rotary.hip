// k_rotary.hip -- norm of query and key heads with the rotation by position, in one pass.
//
//   n = x / sqrt(mean(x^2) + eps),   g = n w,   (y_a, y_b) = magnitude (g_a cos - g_b sin, g_b cos + g_a sin)
//
// for the pairs (a, b) of the head's first `part` elements, angle = position freq; the others are g.  Backward:
//
//   h = R^T dy,   dw = sum h n,   dx = (h w - n mean(h w n)) / sqrt(mean(x^2) + eps)
//
// (without norm: y = R x, dx = R^T dy).  Everything of a head is read once and written once.
//
// A head's row is taken by 4 .. 32 lanes with four pairs each, several rows a
// wave.  A wave stays with a token and goes through its heads, so that a pair's
// angle is made once for all of them: position freq is taken in 64 bits, in turns,
// and its whole part left out, so positions of millions lose nothing.
//
// What bounds it: memory.  16384 tokens x 32 (8) heads x 128 bfloat16 take 70 us forward (4.8 TB/s; a copy 5.0); x 16 (16) heads
// backward 84 us (4.8 TB/s), 88 with the weights' gradients: each workgroup's sums, then theirs in a fixed order.
#include <algorithm>

#include "k_attn.h"

namespace pc {
namespace {

// A lane's four pairs: x[2 i], x[2 i + 1] are pair i's.
struct Pairs {
  float x[8];
};

// Where a lane's pairs lie in a row.
struct Place {
  int p0, half, part, dim;     // first pair; pairs turned; elements turned; all
  bool pairs;
  __device__ __forceinline__ bool split(int p) const { return !pairs && p < half; }
  __device__ __forceinline__ int a(int p) const { return split(p) ? p : 2 * p; }
  __device__ __forceinline__ int b(int p) const { return split(p) ? p + half : 2 * p + 1; }
};

// VEC: a lane's pairs are all turned or all not, and all there or none.
template <bool VEC, typename T>
__device__ __forceinline__ Pairs load_pairs(const T* row, const Place& at) {
  Pairs v;
  if constexpr (VEC) {
    const bool on = 2 * at.p0 < at.dim, split = at.split(at.p0);
    T a[4], b[4];
    const int p0 = on ? at.p0 : 0;
    const bool s0 = on && split;
    __builtin_memcpy(a, row + (s0 ? p0 : 2 * p0), sizeof(a));
    __builtin_memcpy(b, row + (s0 ? p0 + at.half : 2 * p0 + 4), sizeof(b));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // split: pair i is (a[i], b[i]); else the eight lie in order
      const float u = to_f32(a[i]), w = to_f32(b[i]);
      v.x[i] = on ? u : 0.0f;
      v.x[4 + i] = on ? w : 0.0f;
    }
    if (split) {
      const Pairs t = v;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v.x[2 * i] = t.x[i];
        v.x[2 * i + 1] = t.x[4 + i];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int p = at.p0 + i, a = at.a(p), b = at.b(p);
      v.x[2 * i] = a < at.dim ? to_f32(row[a]) : 0.0f;
      v.x[2 * i + 1] = b < at.dim ? to_f32(row[b]) : 0.0f;
    }
  }
  return v;
}
template <bool VEC, typename T>
__device__ __forceinline__ void store_pairs(T* row, const Place& at, const Pairs& v) {
  if constexpr (VEC) {
    if (2 * at.p0 >= at.dim) return;
    const bool split = at.split(at.p0);
    T a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = from_f32<T>(split ? v.x[2 * i] : v.x[i]);
      b[i] = from_f32<T>(split ? v.x[2 * i + 1] : v.x[4 + i]);
    }
    __builtin_memcpy(row + (split ? at.p0 : 2 * at.p0), a, sizeof(a));
    __builtin_memcpy(row + (split ? at.p0 + at.half : 2 * at.p0 + 4), b, sizeof(b));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int p = at.p0 + i, a = at.a(p), b = at.b(p);
      if (a < at.dim) row[a] = from_f32<T>(v.x[2 * i]);
      if (b < at.dim) row[b] = from_f32<T>(v.x[2 * i + 1]);
    }
  }
}

// cos and sin (times the magnitude) of a lane's pairs at a position; those that are not turned: 1 and 0.
struct Angles {
  float c[4], s[4];
  __device__ __forceinline__ void at(int position, const double (&turns)[4], const Place& pl, float magnitude) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const double t = (double)position * turns[i];
      float sn, cs;
      sincospif((float)(2.0 * (t - rint(t))), &sn, &cs);
      const bool on = pl.p0 + i < pl.half;
      c[i] = on ? cs * magnitude : 1.0f;
      s[i] = on ? sn * magnitude : 0.0f;
    }
  }
  __device__ __forceinline__ void turn(Pairs& v, float way) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = v.x[2 * i], b = v.x[2 * i + 1], t = way * s[i];
      v.x[2 * i] = fmaf(a, c[i], -(b * t));
      v.x[2 * i + 1] = fmaf(b, c[i], a * t);
    }
  }
};

template <int LANES>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int d = LANES / 2; d; d >>= 1) x += __shfl_xor(x, d);
  return x;
}
__device__ __forceinline__ void turns_of(const RotaryArgs& a, const Place& at, double (&turns)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) turns[i] = at.p0 + i < at.half ? a.freq[at.p0 + i] * 0.15915494309189533577 : 0.0;
}
template <bool VEC>
__device__ __forceinline__ Pairs weights_of(const float* w, const Place& at) {
  if (w) return load_pairs<VEC, float>(w, at);
  Pairs v;
#pragma unroll
  for (int e = 0; e < 8; ++e) v.x[e] = 1.0f;
  return v;
}

// `share`: waves that share a token's heads.
template <typename T, int LANES, bool VEC, bool NORM>
__global__ __launch_bounds__(256) void rotary_fwd(RotaryArgs a, int share) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, sub = lane / LANES;
  constexpr int ROWS = 64 / LANES;
  const Place at{lane % LANES * 4, a.part / 2, a.part, a.dim, a.pairs != 0};
  double turns[4];
  turns_of(a, at, turns);
  Pairs qw, kw;
  if constexpr (NORM) {
    qw = weights_of<VEC>(a.qw, at);
    kw = weights_of<VEC>(a.kw, at);
  }
  const float inv = 1.0f / (float)a.dim;
  const int64_t step = (int64_t)gridDim.x * 4 / share;
  for (int64_t t = ((int64_t)blockIdx.x * 4 + wave) / share; t < a.tokens; t += step) {
    Angles g;
    g.at(a.positions[t], turns, at, a.magnitude);
    auto heads = [&](const AttnTensor& x, void* y, int64_t y_ts, int64_t y_hs, int n, const Pairs& w) {
      const T* from = (const T*)x.p + t * x.ts;
      T* to = (T*)y + t * y_ts;
      // (every lane of a wave stays in the loop: rows are summed over lanes)
      for (int r0 = wave % share * ROWS; r0 < n; r0 += share * ROWS) {
        const int r = r0 + sub;
        Pairs v = load_pairs<VEC>(from + (int64_t)min(r, n - 1) * x.hs, at);
        if constexpr (NORM) {
          float ss = 0.0f;
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = fmaf(v.x[e], v.x[e], ss);
          const float rms = rsqrtf(fmaf(row_sum<LANES>(ss), inv, a.eps));
#pragma unroll
          for (int e = 0; e < 8; ++e) v.x[e] *= rms * w.x[e];
        }
        g.turn(v, 1.0f);
        if (r < n) store_pairs<VEC>(to + (int64_t)r * y_hs, at, v);
      }
    };
    heads(a.q, a.qo, a.qo_ts, a.qo_hs, a.heads, qw);
    heads(a.k, a.ko, a.ko_ts, a.ko_hs, a.kv_heads, kw);
  }
}

template <typename T, int LANES, bool VEC, bool NORM>
__global__ __launch_bounds__(256) void rotary_bwd(RotaryArgs a, int share) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, sub = lane / LANES;
  constexpr int ROWS = 64 / LANES;
  const Place at{lane % LANES * 4, a.part / 2, a.part, a.dim, a.pairs != 0};
  double turns[4];
  turns_of(a, at, turns);
  Pairs qw, kw, qs{}, ks{};
  if constexpr (NORM) {
    qw = weights_of<VEC>(a.qw, at);
    kw = weights_of<VEC>(a.kw, at);
  }
  const float inv = 1.0f / (float)a.dim;
  const int64_t step = (int64_t)gridDim.x * 4 / share;
  for (int64_t t = ((int64_t)blockIdx.x * 4 + wave) / share; t < a.tokens; t += step) {
    Angles g;
    g.at(a.positions[t], turns, at, a.magnitude);
    auto heads = [&](const AttnTensor& dy, const AttnTensor& x, void* y, int64_t y_ts, int64_t y_hs, int n, const Pairs& w, Pairs& sum) {
      const T *from = (const T*)dy.p + t * dy.ts, *in = NORM ? (const T*)x.p + t * x.ts : nullptr;
      T* to = (T*)y + t * y_ts;
      for (int r0 = wave % share * ROWS; r0 < n; r0 += share * ROWS) {
        const int r = r0 + sub, row = min(r, n - 1);
        Pairs v = load_pairs<VEC>(from + (int64_t)row * dy.hs, at);
        if constexpr (NORM) {
          Pairs u = load_pairs<VEC>(in + (int64_t)row * x.hs, at);
          g.turn(v, -1.0f);
          float ss = 0.0f;
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = fmaf(u.x[e], u.x[e], ss);
          const float rms = rsqrtf(fmaf(row_sum<LANES>(ss), inv, a.eps));
          float hn = 0.0f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            u.x[e] *= rms;
            if (r < n) sum.x[e] = fmaf(v.x[e], u.x[e], sum.x[e]);
            v.x[e] *= w.x[e];
            hn = fmaf(v.x[e], u.x[e], hn);
          }
          hn = row_sum<LANES>(hn) * inv;
#pragma unroll
          for (int e = 0; e < 8; ++e) v.x[e] = rms * fmaf(-u.x[e], hn, v.x[e]);
        } else {
          g.turn(v, -1.0f);
        }
        if (r < n) store_pairs<VEC>(to + (int64_t)r * y_hs, at, v);
      }
    };
    heads(a.dq, a.q, a.qo, a.qo_ts, a.qo_hs, a.heads, qw, qs);
    heads(a.dk, a.k, a.ko, a.ko_ts, a.ko_hs, a.kv_heads, kw, ks);
  }
  if constexpr (NORM) {
    if (!a.part_sums) return;
    // the block's sums, in the order of its waves and of a wave's rows
    __shared__ float sums[2][4][2 * 4 * LANES];
    for (int x = 0; x < 2; ++x) {
      Pairs& s = x ? ks : qs;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
#pragma unroll
        for (int d = LANES; d < 64; d <<= 1) s.x[e] += __shfl_xor(s.x[e], d);
        if (sub == 0) {
          const int p = at.p0 + e / 2, i = e & 1 ? at.b(p) : at.a(p);
          if (i < at.dim) sums[x][wave][i] = s.x[e];
        }
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.dim; i += 256) {
      const int x = i >= a.dim, d = i - x * a.dim;
      a.part_sums[(int64_t)blockIdx.x * 2 * a.dim + i] = (sums[x][0][d] + sums[x][1][d]) + (sums[x][2][d] + sums[x][3][d]);
    }
  }
}

// dweight = sum of the blocks' parts in a fixed order: a workgroup for four of the 2 dim sums, 64 threads each, eight
// parts in flight (16 sums with 16 threads each, a part after the other: 10 us for 1024 parts of 256).
__global__ __launch_bounds__(256) void rotary_weights(RotaryArgs a) {
  const int i = blockIdx.x * 4 + (threadIdx.x & 3), y = threadIdx.x >> 2;
  __shared__ float s[4][4];
  float v = 0.0f;
  if (i < 2 * a.dim)
    for (int p = y; p < a.parts; p += 512) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = a.part_sums[(int64_t)min(p + 64 * e, a.parts - 1) * 2 * a.dim + i];
#pragma unroll
      for (int e = 0; e < 8; ++e) v += p + 64 * e < a.parts ? x[e] : 0.0f;
    }
  for (int x = 4; x < 64; x *= 2) v += __shfl_xor(v, x);
  if ((threadIdx.x & 63) < 4) s[threadIdx.x >> 6][threadIdx.x & 3] = v;
  __syncthreads();
  if (threadIdx.x >= 4 || i >= 2 * a.dim) return;
  v = s[0][threadIdx.x] + s[1][threadIdx.x] + s[2][threadIdx.x] + s[3][threadIdx.x];
  float* to = i < a.dim ? a.dqw : a.dkw;
  if (to) to[i < a.dim ? i : i - a.dim] = v;
}

// Waves that share a token: as many as there are rows for while tokens are few
// (doubled below 2048 waves, so fewer than 4096: sixteen a compute unit).
int share_of(const RotaryArgs& a, int lanes) {
  const int rows = (std::max(a.heads, a.kv_heads) * lanes + 63) / 64;
  int s = 1;
  while (s < 4 && s < rows && a.tokens * s < 2048) s *= 2;
  return s;
}
template <typename T, int LANES, bool VEC, bool NORM>
void launch(const RotaryArgs& a, bool backward, hipStream_t s) {
  const int share = share_of(a, LANES);
  const int64_t blocks = (a.tokens * share + 3) / 4;
  if (backward) launch_kernel(rotary_bwd<T, LANES, VEC, NORM>, dim3(a.parts), dim3(256), 0, s, a, share);
  else launch_kernel(rotary_fwd<T, LANES, VEC, NORM>, dim3((uint32_t)std::min<int64_t>(blocks, 1 << 20)), dim3(256), 0, s, a, share);
}
template <typename T, int LANES>
void pick(const RotaryArgs& a, bool backward, hipStream_t s) {
  const bool vec = a.part % 8 == 0 && a.dim % 8 == 0;
  if (vec) {
    if (a.norm) launch<T, LANES, true, true>(a, backward, s);
    else launch<T, LANES, true, false>(a, backward, s);
  } else {
    if (a.norm) launch<T, LANES, false, true>(a, backward, s);
    else launch<T, LANES, false, false>(a, backward, s);
  }
}
template <typename T>
void by_dim(const RotaryArgs& a, bool backward, hipStream_t s) {
  if (a.dim <= 32) pick<T, 4>(a, backward, s);
  else if (a.dim <= 64) pick<T, 8>(a, backward, s);
  else if (a.dim <= 128) pick<T, 16>(a, backward, s);
  else pick<T, 32>(a, backward, s);
}
void launch_any(const RotaryArgs& a, int dtype, bool backward, hipStream_t s) {
  if (dtype == PC_DTYPE_BF16) by_dim<bf16>(a, backward, s);
  else if (dtype == PC_DTYPE_F16) by_dim<f16>(a, backward, s);
  else by_dim<float>(a, backward, s);
}

}  // namespace

// Blocks of the backward pass: each leaves one partial sum of the weights' gradients.
int rotary_parts(int64_t tokens) {
  return (int)std::max<int64_t>(1, std::min<int64_t>(tokens, 1024));
}
void launch_rotary_fwd(const RotaryArgs& a, int dtype, hipStream_t s) { launch_any(a, dtype, false, s); }
void launch_rotary_bwd(const RotaryArgs& a, int dtype, hipStream_t s) {
  if (a.tokens > 0) launch_any(a, dtype, true, s);
  if (!a.norm || !(a.dqw || a.dkw)) return;
  RotaryArgs b = a;
  if (a.tokens == 0) b.parts = 0;
  launch_kernel(rotary_weights, dim3((2 * a.dim + 3) / 4), dim3(256), 0, s, b);
}

}  // namespace pc
