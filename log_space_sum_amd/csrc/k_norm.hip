// k_norm.hip -- layer norm over the last dimension, forward and backward.
//
//   mean = sum x / n,  rstd = 1 / sqrt(sum (x - mean)^2 / n + eps),
//   y = (x - mean) rstd w + b
//   n = (x - mean) rstd,  g = dy w,
//   dx = rstd (g - mean(g) - n mean(g n)),  dw = sum_rows dy n,  db = sum_rows dy
//
// Both passes are bound by memory (forward: 9001 x 1001 float16, 36 MB, 11.6 us;
// backward: 16384 x 4096 bfloat16, 403 MB, 90 us or 4.5 TB/s, with its sum
// kernel 5 us of it): a row is read once into registers (16-byte
// loads, also from rows whose start is not aligned), its two sums are taken
// there, the variance from the centred values, and the result is written from
// the same registers.  A row belongs to TPR threads: few for short rows, so a
// wave holds several, up to 1024 for the longest (see shape_of).  The backward's weight
// gradient is summed per thread over the rows that its group walks, in a fixed
// order, and a second kernel adds the groups' partial sums: no atomics, the
// same bits at every run.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "pc_ops.h"

namespace pc {
namespace {

template <typename T>
struct Vec {
  static constexpr int N = 16 / sizeof(T);
  T v[N];
};

// 16 bytes from an address that only T's own alignment is known of (one
// instruction: gfx950 loads and stores unaligned vectors; through a 128-bit
// value, since an array would be taken apart into elements).
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
template <typename T>
__device__ __forceinline__ Vec<T> load_vec(const T* p) {
  u32x4 r;
  __builtin_memcpy(&r, p, 16);
  return __builtin_bit_cast(Vec<T>, r);
}
template <typename T>
__device__ __forceinline__ void store_vec(T* p, const Vec<T>& v) {
  const u32x4 r = __builtin_bit_cast(u32x4, v);
  __builtin_memcpy(p, &r, 16);
}

template <typename T>
__device__ __forceinline__ Vec<T> load_part(const T* p, int have) {   // elements behind `have` are 0
  u32x4 r;
  if (have >= Vec<T>::N) {
    __builtin_memcpy(&r, p, 16);
  } else {
    Vec<T> t = {};
#pragma unroll
    for (int e = 0; e < Vec<T>::N; ++e)
      if (e < have) t.v[e] = p[e];
    r = __builtin_bit_cast(u32x4, t);
  }
  return __builtin_bit_cast(Vec<T>, r);
}

// Sum over the TPR threads of a row's group, the same value in every thread.
// Within a wave by shuffles; across waves through `red` (two slots used in
// turn, so one barrier per sum is enough).
template <int TPR>
__device__ __forceinline__ float row_sum(float x, float* red, int& slot) {
#pragma unroll
  for (int d = 1; d < (TPR < 64 ? TPR : 64); d <<= 1) x += __shfl_xor(x, d, 64);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    float* r = red + slot * W;
    if ((threadIdx.x & 63) == 0) r[threadIdx.x >> 6] = x;
    __syncthreads();
    x = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) x += r[w];
    slot ^= 1;
  }
  return x;
}

// Threads of a block: groups of TPR, one row each.
template <int TPR>
constexpr int block_of() { return TPR > 64 ? TPR : 256; }

template <typename T, int TPR, int R>
__global__ __launch_bounds__(block_of<TPR>()) void norm_fwd(NormArgs a) {
  constexpr int V = Vec<T>::N, BLK = block_of<TPR>(), G = BLK / TPR;
  __shared__ float red[2 * (BLK / 64)];
  int slot = 0;
  const int lane = threadIdx.x % TPR;
  const float count = (float)a.cols;
  // every group of a block runs the same number of rounds: the sums of wide rows hold barriers
  for (int64_t r0 = (int64_t)blockIdx.x * G; r0 < a.rows; r0 += (int64_t)gridDim.x * G) {
    const int64_t row = r0 + threadIdx.x / TPR;
    const bool on = row < a.rows;
    const T* x = (const T*)a.x + (on ? row : 0) * a.x_stride;
    float v[R][V];
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int c = (i * TPR + lane) * V;
      Vec<T> u = {};
      if (c < a.cols) u = load_part(x + c, a.cols - c);
#pragma unroll
      for (int e = 0; e < V; ++e) s += v[i][e] = to_f32(u.v[e]);
    }
    const float mean = row_sum<TPR>(s, red, slot) / count;
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int c = (i * TPR + lane) * V + e;
        v[i][e] = c < a.cols ? v[i][e] - mean : 0.0f;
        q += v[i][e] * v[i][e];
      }
    const float rstd = 1.0f / sqrtf(row_sum<TPR>(q, red, slot) / count + a.eps);
    if (!on) continue;
    if (lane == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    T* y = (T*)a.y + row * a.y_stride;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int c = (i * TPR + lane) * V;
      if (c >= a.cols) continue;
      const int have = a.cols - c;
      float w[V], b[V];
#pragma unroll
      for (int e = 0; e < V; e += 4) {
        Vec<float> t;
        if (a.weight) t = load_part(a.weight + c + e, have - e);
#pragma unroll
        for (int k = 0; k < 4; ++k) w[e + k] = a.weight ? t.v[k] : 1.0f;
        if (a.bias) t = load_part(a.bias + c + e, have - e);
#pragma unroll
        for (int k = 0; k < 4; ++k) b[e + k] = a.bias ? t.v[k] : 0.0f;
      }
      Vec<T> o;
#pragma unroll
      for (int e = 0; e < V; ++e) o.v[e] = from_f32<T>(v[i][e] * rstd * w[e] + b[e]);
      if (have >= V) {
        store_vec(y + c, o);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (e < have) y[c + e] = o.v[e];
      }
    }
  }
}

// Two sums at once.
template <int TPR>
__device__ __forceinline__ void row_sums(float& x, float& y, float* red, int& slot) {
#pragma unroll
  for (int d = 1; d < (TPR < 64 ? TPR : 64); d <<= 1) {
    x += __shfl_xor(x, d, 64);
    y += __shfl_xor(y, d, 64);
  }
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    float* r = red + slot * 2 * W;
    if ((threadIdx.x & 63) == 0) {
      r[threadIdx.x >> 6] = x;
      r[W + (threadIdx.x >> 6)] = y;
    }
    __syncthreads();
    x = y = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      x += r[w];
      y += r[W + w];
    }
    slot ^= 1;
  }
}

template <typename T, int TPR, int R>
__global__ __launch_bounds__(block_of<TPR>()) void norm_bwd(NormArgs a) {
  constexpr int V = Vec<T>::N, BLK = block_of<TPR>(), G = BLK / TPR;
  __shared__ float red[4 * (BLK / 64)];
  int slot = 0;
  const int lane = threadIdx.x % TPR, group = threadIdx.x / TPR;
  const float inv = 1.0f / (float)a.cols;
  float w[R][V], dw[R][V], db[R][V];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int c = (i * TPR + lane) * V + e;
      w[i][e] = c < a.cols ? (a.weight ? a.weight[c] : 1.0f) : 0.0f;
      dw[i][e] = db[i][e] = 0.0f;
    }
  Vec<T> ux[R], ud[R];
  float mean, rstd;
  // a row behind the last loads the last one's values: the loads need no condition
  auto fetch = [&](int64_t r0) {
    const int64_t row = min(r0 + group, a.rows - 1);
    const T* x = (const T*)a.x + row * a.x_stride;
    const T* dy = (const T*)a.dy + row * a.dy_stride;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int c = (i * TPR + lane) * V;
      ux[i] = ud[i] = Vec<T>{};
      if (c < a.cols) {
        ux[i] = load_part(x + c, a.cols - c);
        ud[i] = load_part(dy + c, a.cols - c);
      }
    }
    mean = a.mean[row];
    rstd = a.rstd[row];
  };
  const int64_t step = (int64_t)gridDim.x * G;
  fetch((int64_t)blockIdx.x * G);
  for (int64_t r0 = (int64_t)blockIdx.x * G; r0 < a.rows; r0 += step) {
    const int64_t row = r0 + group;
    const bool on = row < a.rows;
    const float rs = rstd;
    float n[R][V], g[R][V], s = 0.0f, t = 0.0f;
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const bool in = on && (i * TPR + lane) * V + e < a.cols;
        const float d = on ? to_f32(ud[i].v[e]) : 0.0f;
        n[i][e] = in ? (to_f32(ux[i].v[e]) - mean) * rs : 0.0f;
        g[i][e] = d * w[i][e];
        dw[i][e] += d * n[i][e];
        db[i][e] += d;
        s += g[i][e];
        t += g[i][e] * n[i][e];
      }
    fetch(r0 + step);   // the next row, in flight over the sums and the store
    row_sums<TPR>(s, t, red, slot);
    const float mg = s * inv, mgn = t * inv;
    if (!on) continue;
    T* dx = (T*)a.y + row * a.y_stride;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int c = (i * TPR + lane) * V;
      if (c >= a.cols) continue;
      Vec<T> o;
#pragma unroll
      for (int e = 0; e < V; ++e) o.v[e] = from_f32<T>(rs * (g[i][e] - mg - n[i][e] * mgn));
      if (a.cols - c >= V) {
        store_vec(dx + c, o);
      } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (e < a.cols - c) dx[c + e] = o.v[e];
      }
    }
  }
  if (!a.part) return;
  float* pw = a.part + ((int64_t)blockIdx.x * G + group) * 2 * a.cols;
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int c = (i * TPR + lane) * V + e;
      if (c < a.cols) {
        pw[c] = dw[i][e];
        pw[a.cols + c] = db[i][e];
      }
    }
}

// Sums the partial sums (512 of 2 x 4096: 5 us; 1024 of them, 18 us) of the
// 2 cols columns: 32 columns a block, every eighth
// partial row a thread (eight loads in flight), joined in a fixed order.
__global__ __launch_bounds__(256) void norm_bwd_sum(NormArgs a) {
  __shared__ float red[8][33];
  const int col = threadIdx.x & 31, part = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + col, n = 2 * a.cols;
  float s = 0.0f;
  if (c < n) {
#pragma unroll 8
    for (int p = part; p < a.parts; p += 8) s += a.part[(int64_t)p * n + c];
  }
  red[part][col] = s;
  __syncthreads();
  if (part == 0 && c < n) {
    s = 0.0f;
#pragma unroll
    for (int p = 0; p < 8; ++p) s += red[p][col];
    float* out = c < a.cols ? a.dweight : a.dbias;
    if (out) out[c < a.cols ? c : c - a.cols] = s;
  }
}

struct Shape {
  int tpr, r;
};
// Threads of a row and vectors of a thread.  One vector a thread where latency
// counts (few rows) and in the backward, which holds five values for each
// element (two vectors a thread: 137 instead of 103 us for 16384 x 4096 bf16).
// The forward of many rows: a wave as far as four vectors a thread go, since
// its sums need no barrier.
Shape shape_of(int64_t rows, int cols, int vec, bool backward) {
  const int nv = (cols + vec - 1) / vec;
  for (int tpr : {8, 16, 32, 64})
    if (nv <= tpr) return {tpr, 1};
  if (!backward && rows >= 2048) {
    if (nv <= 128) return {64, 2};
    if (nv <= 256) return {64, 4};
  }
  for (int tpr : {128, 256, 512, 1024})
    if (nv <= tpr) return {tpr, 1};
  return nv <= 2048 ? Shape{1024, 2} : Shape{1024, 4};
}

template <typename T, typename F>
void dispatch(int64_t rows, int cols, bool backward, F&& f) {
  const Shape s = shape_of(rows, cols, Vec<T>::N, backward);
#define PC_NORM_CASE(TPR, R)                                                \
  if (s.tpr == TPR && s.r == R) {                                           \
    f(std::integral_constant<int, TPR>{}, std::integral_constant<int, R>{}); \
    return;                                                                 \
  }
  PC_NORM_CASE(8, 1)
  PC_NORM_CASE(16, 1)
  PC_NORM_CASE(32, 1)
  PC_NORM_CASE(64, 1)
  PC_NORM_CASE(64, 2)
  PC_NORM_CASE(64, 4)
  PC_NORM_CASE(128, 1)
  PC_NORM_CASE(256, 1)
  PC_NORM_CASE(512, 1)
  PC_NORM_CASE(1024, 1)
  PC_NORM_CASE(1024, 2)
  PC_NORM_CASE(1024, 4)
#undef PC_NORM_CASE
}

template <typename T>
void fwd(const NormArgs& a, hipStream_t s) {
  dispatch<T>(a.rows, a.cols, false, [&](auto tpr, auto r) {
    constexpr int TPR = decltype(tpr)::value, BLK = block_of<TPR>(), G = BLK / TPR;
    const int64_t need = (a.rows + G - 1) / G;
    launch_kernel(norm_fwd<T, TPR, decltype(r)::value>, dim3((unsigned)std::min<int64_t>(need, 1 << 20)), dim3(BLK), 0, s, a);
  });
}

template <typename T>
void bwd(const NormArgs& a, hipStream_t s) {
  dispatch<T>(a.rows, a.cols, true, [&](auto tpr, auto r) {
    constexpr int TPR = decltype(tpr)::value, BLK = block_of<TPR>(), G = BLK / TPR;
    NormArgs b = a;
    const int64_t need = (a.rows + G - 1) / G;
    int64_t grid = std::min<int64_t>(need, std::max(1, norm_parts(a.rows, a.cols) / G));
    if (!a.dweight && !a.dbias) {
      b.part = nullptr;
      grid = std::min<int64_t>(need, 4096);
    }
    b.parts = (int)(grid * G);
    if (grid > 0) launch_kernel(norm_bwd<T, TPR, decltype(r)::value>, dim3((unsigned)grid), dim3(BLK), 0, s, b);
    if (a.dweight || a.dbias) launch_kernel(norm_bwd_sum, dim3((unsigned)((2 * a.cols + 31) / 32)), dim3(256), 0, s, b);
  });
}

}  // namespace

// Most partial sums of the weight gradient: enough row groups to fill the card,
// at most 17 MB of them (or 512).  From about 1000 columns up, where that is a
// small part of the traffic, the sums cost little (16384 x 4096 bfloat16: 5 of 90
// us); narrower rows pay for them (16384 x 256: 71 us, 12 without the gradients
// of the parameters, 17 MB of sums to 25 MB of tensors).
int norm_parts(int64_t rows, int cols) {
  if (rows <= 0) return 0;
  const int64_t by_size = std::max<int64_t>(512, (int64_t)(1 << 21) / std::max(1, cols));
  return (int)std::min<int64_t>(std::min<int64_t>(by_size, 8192), (rows + 31) / 32 * 32);
}

void launch_norm_fwd(const NormArgs& a, int dtype, hipStream_t s) {
  if (dtype == PC_DTYPE_F32) fwd<float>(a, s);
  else if (dtype == PC_DTYPE_F16) fwd<f16>(a, s);
  else fwd<bf16>(a, s);
}
void launch_norm_bwd(const NormArgs& a, int dtype, hipStream_t s) {
  if (dtype == PC_DTYPE_F32) bwd<float>(a, s);
  else if (dtype == PC_DTYPE_F16) bwd<f16>(a, s);
  else bwd<bf16>(a, s);
}

}  // namespace pc
