// k_orth.hip -- the orthogonalised update: Newton-Schulz steps
//   X <- a X + (b A + c A^2) X,  A = X X^T,  from X = G / (|G| + eps),  X [m, n], m <= n.
//
// Two ways, by the smaller dimension m:
//
// m <= 64 (LowRank factors and their like, many and thin): X after all steps
// is Q X_0 with Q a polynomial in A_0, so the steps run on m x m matrices,
//   M = a I + b A + c A^2,   Q <- Q M,   A <- A M^2,
// and the matrix itself is read twice and written once.  Squaring the matrix
// costs half of the digits, so A, M and Q are held in 64 bits (one workgroup
// a matrix, on the float64 matrix instruction).  Bound by latency: 64 matrices of
// 1024 x 16 float32 take 13.7 us, of which the steps, a chain of 17 products in one
// wave, are about four.  The last product Q X_0 is taken in 64 bits as well, since
// its terms cancel where G has no singular value: Q is the product of the a's there
// (in float32: 1.1 us less, but 5e-5 of the result for a rank 1 matrix after five
// steps, 4e-4 after six, and no result where Q / |G| leaves float32's range).
// This holds for few steps.  Where G has a small or no singular value, A's
// rounding leaves an eigenvalue of about -1e-16 there, which every step multiplies
// by up to a^2 (16 steps of the usual a = 3.4: past 1, and then without bound).
// Past a growth of Q of ORTH_GROWTH the steps therefore run on a factor X' with
// X' X'^T = A_0 + d I (Cholesky), X' <- M X', and A = X' X'^T is formed afresh in
// every step: it has no negative eigenvalue beyond its rounding, which is not
// carried on.  d, above the rounding of A_0, keeps the factorisation definite and
// |X'| >= |X| in every direction, so Q X_0 stays within the steps' bounds, and Q
// below top / sqrt(d), which 64 bits hold (rank 1 and 4 matrices after 32 steps:
// 1e-8 of the result).
//
// Larger m: three products a step on the float16 matrix instruction.  An
// operand is split into two float16 planes of a value scaled by a power of two
// (hi + lo: 22 bits; the spectra are bounded, so the scales are known before
// the call), and hi hi + hi lo + lo hi are summed in float32: the accuracy of
// float32 steps at three times the cost of a 16-bit product.  So it is for
// every type: one plane of A's operands alone would put 4e-4 of the result on
// top of a bfloat16 result's own rounding (1.7e-3).  The symmetric products (A,
// A^2) compute the tiles on and above the diagonal only.  Bound by the matrix
// instructions: at 4096 x 4096 B X runs at 1.06 PFLOP/s of float16 products
// (390 us for three of 137 GFLOP; a library product reaches 1.08), A and A^2 at
// 0.95 (with the tiles left over).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "pc_ops.h"
#include "pc_ring.h"

namespace pc {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef double f64x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// X[i][p] of a matrix: i along m, p along n
template <typename IO>
__device__ __forceinline__ int64_t at_x(const OrthIo& io, int64_t row_stride, int64_t i, int64_t p) {
  return io.tall ? p * row_stride + i : i * row_stride + p;
}

// ---------------------------------------------------------------------------
// m <= 64: one workgroup a matrix
// ---------------------------------------------------------------------------

// C = A B of symmetric commuting [16 MB]^2 matrices in LDS (row stride LD):
// the part on and above the diagonal, mirrored by store().
template <int MB, int LD, int W, typename F>
__device__ __forceinline__ void small_product(const double* A, const double* B, F&& store) {
  constexpr int T = MB * (MB + 1) / 2, MINE = (T + W - 1) / W;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, g = lane >> 4, l16 = lane & 15;
  f64x4 acc[MINE];
#pragma unroll
  for (int k = 0; k < MINE; ++k) {
    int jb = 0, ib = wave + W * k;
    if (ib >= T) continue;
    while (ib > jb) ib -= ++jb;
    acc[k] = f64x4{0.0, 0.0, 0.0, 0.0};
#pragma unroll
    for (int q = 0; q < 4 * MB; ++q)
      acc[k] = __builtin_amdgcn_mfma_f64_16x16x4f64(A[(16 * ib + l16) * LD + 4 * q + g], B[(16 * jb + l16) * LD + 4 * q + g],
                                                    acc[k], 0, 0, 0);
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < MINE; ++k) {
    int jb = 0, ib = wave + W * k;
    if (ib >= T) continue;
    while (ib > jb) ib -= ++jb;
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (16 * ib + g + 4 * r <= 16 * jb + l16) store(16 * ib + g + 4 * r, 16 * jb + l16, acc[k][r]);
  }
  __syncthreads();
}

// The same of one block of 16: a lane's four results, rows g + 4 r of column
// l16, are by the symmetry also its operand's four values, columns 4 q + g of
// row l16.  No matrix leaves its registers.  (Two sums: a float64 matrix
// instruction waits long for the one before it.)
__device__ __forceinline__ f64x4 product16(f64x4 a, f64x4 b) {
  f64x4 c = {0.0, 0.0, 0.0, 0.0}, d = c;
  c = __builtin_amdgcn_mfma_f64_16x16x4f64(a[0], b[0], c, 0, 0, 0);
  d = __builtin_amdgcn_mfma_f64_16x16x4f64(a[1], b[1], d, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f64_16x16x4f64(a[2], b[2], c, 0, 0, 0);
  d = __builtin_amdgcn_mfma_f64_16x16x4f64(a[3], b[3], d, 0, 0, 0);
  return c + d;
}

// Four consecutive p of row i (zeros behind m and n; the loads need no
// condition), p0 + 4 g ... for lane group g.
template <typename IO>
__device__ __forceinline__ f32x4 load_p(const IO* x, const OrthIo& io, int i, int p) {
  const bool row = i < io.m;
  const int64_t ii = row ? i : 0;
  f32x4 v;
  if (!io.tall && p + 4 <= io.n) {
    IO u[4];
    __builtin_memcpy(u, x + ii * io.g_row + p, sizeof(u));
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = row ? to_f32(u[e]) : 0.0f;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float t = to_f32(x[at_x<IO>(io, io.g_row, ii, min(p + e, io.n - 1))]);
      v[e] = row && p + e < io.n ? t : 0.0f;
    }
  }
  return v;
}
// Four consecutive i of column p.
template <typename IO>
__device__ __forceinline__ f32x4 load_i(const IO* x, const OrthIo& io, int i, int p) {
  const int64_t pp = min(p, io.n - 1);
  f32x4 v;
  if (io.tall && i + 4 <= io.m) {
    IO u[4];
    __builtin_memcpy(u, x + pp * io.g_row + i, sizeof(u));
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = p < io.n ? to_f32(u[e]) : 0.0f;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float t = to_f32(x[at_x<IO>(io, io.g_row, min(i + e, io.m - 1), pp)]);
      v[e] = i + e < io.m && p < io.n ? t : 0.0f;
    }
  }
  return v;
}

// C = M B of [16 MB]^2 matrices in LDS, M symmetric; C may be B.
template <int MB, int LD, int W>
__device__ __forceinline__ void small_multiply(const double* M, const double* B, double* C) {
  constexpr int T = MB * MB, MINE = (T + W - 1) / W;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, g = lane >> 4, l16 = lane & 15;
  f64x4 acc[MINE];
#pragma unroll
  for (int k = 0; k < MINE; ++k) {
    const int t = wave + W * k, ib = t / MB, jb = t % MB;
    acc[k] = f64x4{0.0, 0.0, 0.0, 0.0};
    if (t >= T) continue;
#pragma unroll
    for (int q = 0; q < 4 * MB; ++q)
      acc[k] = __builtin_amdgcn_mfma_f64_16x16x4f64(M[(16 * ib + l16) * LD + 4 * q + g], B[(4 * q + g) * LD + 16 * jb + l16],
                                                    acc[k], 0, 0, 0);
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < MINE; ++k) {
    const int t = wave + W * k, ib = t / MB, jb = t % MB;
    if (t >= T) continue;
#pragma unroll
    for (int r = 0; r < 4; ++r) C[(16 * ib + g + 4 * r) * LD + 16 * jb + l16] = acc[k][r];
  }
  __syncthreads();
}

// L with L L^T = S of a [D, D] matrix in LDS, column by column; S is used up.
// A pivot below `least` (S is definite up to rounding) is taken as that.
template <int D, int LD, int NT>
__device__ __forceinline__ void small_cholesky(double* S, double* L, double least) {
  for (int k = 0; k < D; ++k) {
    double pivot = S[k * LD + k];
    pivot = pivot < least ? least : pivot;   // (NaN stays)
    const double r = 1.0 / sqrt(pivot);
    if ((int)threadIdx.x < D) {
      const int i = threadIdx.x;
      L[i * LD + k] = i < k ? 0.0 : (i == k ? pivot : S[i * LD + k]) * r;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < D * D; e += NT) {
      const int i = e / D, j = e % D;
      if (i > k && j > k) S[i * LD + j] -= L[i * LD + k] * L[j * LD + k];
    }
    __syncthreads();
  }
}

// LONG: many steps, on a factor of A (see the top).
template <typename IO, int MB, int NT, bool LONG>
__global__ __launch_bounds__(NT) void orth_small(OrthIo io, OrthPoly poly) {
  constexpr int D = 16 * MB, LD = D + 2, W = NT / 64, T = MB * (MB + 1) / 2;
  // the waves' parts of the Gram matrix, then the matrices of the steps
  constexpr int PARTS = W < 4 ? W : (T * W * 256 > 4 * D * LD ? 4 : W);
  constexpr int POOL = PARTS * T * 256 > 4 * D * LD ? PARTS * T * 256 : 4 * D * LD;
  __shared__ double pool[POOL];
  __shared__ double s_inv;
  double *sA = pool, *sM = pool + D * LD, *sQ = pool + 2 * D * LD, *sT = pool + 3 * D * LD;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, g = lane >> 4, l16 = lane & 15;
  const IO* x = (const IO*)io.g + (int64_t)blockIdx.x * io.g_batch;
  const int m = io.m, n = io.n;

  // A = G G^T in 64 bits: every wave its share of p, four consecutive p a lane
  f64x4 acc[T];
#pragma unroll
  for (int t = 0; t < T; ++t) acc[t] = f64x4{0.0, 0.0, 0.0, 0.0};
  for (int p0 = wave * 16; p0 < n; p0 += W * 16) {
    f32x4 v[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) v[b] = load_p<IO>(x, io, 16 * b + l16, p0 + 4 * g);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      int t = 0;
#pragma unroll
      for (int jb = 0; jb < MB; ++jb)
#pragma unroll
        for (int ib = 0; ib <= jb; ++ib, ++t)
          acc[t] = __builtin_amdgcn_mfma_f64_16x16x4f64((double)v[ib][e], (double)v[jb][e], acc[t], 0, 0, 0);
    }
  }
  // the waves' parts, added in a fixed order
  for (int round = 0; round < W; round += PARTS) {
    if (wave >= round && wave < round + PARTS) {
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          double* s = pool + ((wave - round) * T + t) * 256 + r * 64 + lane;
          *s = round ? *s + acc[t][r] : acc[t][r];
        }
    }
    __syncthreads();
  }
  double own[(T * 256 + NT - 1) / NT];
#pragma unroll
  for (int k = 0; k < (T * 256 + NT - 1) / NT; ++k) {
    const int e = k * NT + tid;
    own[k] = 0.0;
    if (e < T * 256)
#pragma unroll
      for (int w = 0; w < PARTS; ++w) own[k] += pool[w * T * 256 + e];
  }
  __syncthreads();

  if constexpr (MB == 1 && !LONG) {
    // one wave takes all steps in its registers
#pragma unroll
    for (int k = 0; k < (256 + NT - 1) / NT; ++k)
      if (k * NT + tid < 256) pool[k * NT + tid] = own[k];
    __syncthreads();
    if (wave == 0) {
      f64x4 A, Q = {0.0, 0.0, 0.0, 0.0};
      double tr = 0.0;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        A[r] = pool[r * 64 + lane];
        if (g + 4 * r == l16) tr += A[r];
      }
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) tr += __shfl_xor(tr, d, 64);
      const double inv = 1.0 / (sqrt(tr) + (double)io.eps);
      A *= inv * inv;
      for (int s = 0; s < poly.steps; ++s) {
        const double a = poly.c[s][0], b = poly.c[s][1], c = poly.c[s][2];
        f64x4 M = b * A + c * product16(A, A);
#pragma unroll
        for (int r = 0; r < 4; ++r) M[r] += g + 4 * r == l16 ? a : 0.0;
        Q = s ? product16(Q, M) : M;
        if (s + 1 < poly.steps) A = product16(product16(A, M), M);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) sQ[l16 * LD + g + 4 * r] = Q[r] * inv;
    }
    __syncthreads();
  } else {
    for (int e = tid; e < D * LD; e += NT) sA[e] = 0.0;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < (T * 256 + NT - 1) / NT; ++k) {
      const int e = k * NT + tid;
      if (e >= T * 256) continue;
      int jb = 0, ib = e >> 8;
      while (ib > jb) ib -= ++jb;
      const int i = 16 * ib + ((e & 63) >> 4) + 4 * ((e >> 6) & 3), j = 16 * jb + (e & 15);
      if (i <= j) sA[i * LD + j] = sA[j * LD + i] = own[k];
    }
    __syncthreads();
    if (wave == 0) {
      double tr = 0.0;
      for (int i = lane; i < m; i += 64) tr += sA[i * LD + i];
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) tr += __shfl_xor(tr, d, 64);
      if (lane == 0) s_inv = 1.0 / (sqrt(tr) + (double)io.eps);
    }
    __syncthreads();
    const double inv = s_inv;
    for (int e = tid; e < D * D; e += NT)
      sA[e / D * LD + e % D] = sA[e / D * LD + e % D] * (inv * inv) + (LONG && e / D == e % D ? poly.shift : 0.0);
    __syncthreads();
    double* sX = sT;   // LONG: the factor
    if constexpr (LONG) small_cholesky<D, LD, NT>(sA, sX, 0.25 * poly.shift);
    for (int s = 0; s < poly.steps; ++s) {
      const double a = poly.c[s][0], b = poly.c[s][1], c = poly.c[s][2];
      if constexpr (LONG)
        small_product<MB, LD, W>(sX, sX, [&](int i, int j, double v) { sA[i * LD + j] = sA[j * LD + i] = v; });
      small_product<MB, LD, W>(sA, sA, [&](int i, int j, double v) {
        const double u = (i == j ? a : 0.0) + b * sA[i * LD + j] + c * v;
        sM[i * LD + j] = sM[j * LD + i] = u;
        if (s == 0) sQ[i * LD + j] = sQ[j * LD + i] = u;
      });
      if constexpr (LONG) {
        if (s > 0) small_multiply<MB, LD, W>(sM, sQ, sQ);
        if (s + 1 < poly.steps) small_multiply<MB, LD, W>(sM, sX, sX);
        continue;
      }
      if (s > 0) small_product<MB, LD, W>(sQ, sM, [&](int i, int j, double v) { sQ[i * LD + j] = sQ[j * LD + i] = v; });
      if (s + 1 < poly.steps) {
        small_product<MB, LD, W>(sA, sM, [&](int i, int j, double v) { sT[i * LD + j] = sT[j * LD + i] = v; });
        small_product<MB, LD, W>(sT, sM, [&](int i, int j, double v) { sA[i * LD + j] = sA[j * LD + i] = v; });
      }
    }
    for (int e = tid; e < D * D; e += NT) sQ[e / D * LD + e % D] *= inv;
    __syncthreads();
  }

  // out = (Q / |G|) G, in 64 bits: where G has no singular value Q is the product
  // of the a's, and its terms cancel
  double q[MB][MB][4];   // [block of i][block of k][e]: Q[16 ib + l16][16 kb + 4 g + e] / |G|
#pragma unroll
  for (int ib = 0; ib < MB; ++ib)
#pragma unroll
    for (int kb = 0; kb < MB; ++kb)
#pragma unroll
      for (int e = 0; e < 4; ++e) q[ib][kb][e] = sQ[(16 * ib + l16) * LD + 16 * kb + 4 * g + e];
  IO* y = (IO*)io.out + (int64_t)blockIdx.x * io.o_batch;
  // 16 columns p a wave; the operands are exchanged where the tensor's rows run
  // along i, so that 16 lanes always write consecutive elements
  auto columns = [&](auto tall) {
    constexpr bool TALL = decltype(tall)::value;
#pragma unroll 2
    for (int p0 = wave * 16; p0 < n; p0 += W * 16) {
      f32x4 v[MB];
#pragma unroll
      for (int kb = 0; kb < MB; ++kb) v[kb] = load_i<IO>(x, io, 16 * kb + 4 * g, p0 + l16);
#pragma unroll
      for (int ib = 0; ib < MB; ++ib) {
        f64x4 o = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
        for (int kb = 0; kb < MB; ++kb)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            o = TALL ? __builtin_amdgcn_mfma_f64_16x16x4f64((double)v[kb][e], q[ib][kb][e], o, 0, 0, 0)
                     : __builtin_amdgcn_mfma_f64_16x16x4f64(q[ib][kb][e], (double)v[kb][e], o, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int i = 16 * ib + (TALL ? l16 : g + 4 * r), p = p0 + (TALL ? g + 4 * r : l16);
          if (i < m && p < n) y[TALL ? (int64_t)p * io.o_row + i : (int64_t)i * io.o_row + p] = from_f32<IO>((float)o[r]);
        }
      }
    }
  };
  if (io.tall) columns(std::true_type{});
  else columns(std::false_type{});
}

// ---------------------------------------------------------------------------
// larger m: norm, planes, products
// ---------------------------------------------------------------------------

// Partial sums of the squares, in 64 bits (bound by G's bytes and the launch:
// 4096 x 4096 bfloat16 14 us); grid (ORTH_NORM_BLOCKS, batch).
template <typename IO>
__global__ __launch_bounds__(256) void orth_norm(OrthIo io, double* part) {
  __shared__ double red[4];
  const int rows = io.tall ? io.n : io.m, cols = io.tall ? io.m : io.n;
  const IO* x = (const IO*)io.g + (int64_t)blockIdx.y * io.g_batch;
  double s = 0.0;
  const int across = (cols + 2047) / 2048;   // spans of 2048 columns, eight of them a thread
  for (int64_t u = blockIdx.x; u < (int64_t)rows * across; u += ORTH_NORM_BLOCKS) {
    const IO* p = x + u / across * io.g_row;
    const int c = (int)(u % across) * 2048 + threadIdx.x * 8;
    float v[8];
    if (c + 8 <= cols) {
      IO w[8];
      __builtin_memcpy(w, p + c, sizeof(w));
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = to_f32(w[k]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = c + k < cols ? to_f32(p[c + k]) : 0.0f;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) s += (double)v[k] * (double)v[k];
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) part[(int64_t)blockIdx.y * ORTH_NORM_BLOCKS + blockIdx.x] = red[0] + red[1] + red[2] + red[3];
}

// A value's planes.  The value is rounded to float32 first, for both: the
// compiler may fuse the product behind v with one of its conversions and not with
// the other, and where v then lies halfway the low plane belongs to another high
// one (off by 2^-11 in one element of some thousands: 7e-6 of the result).
__device__ __forceinline__ void planes_of(float v, uint16_t& hi, uint16_t& lo) {
  asm volatile("" : "+v"(v));
  const f16 h = (f16)v;
  hi = __builtin_bit_cast(uint16_t, h);
  lo = __builtin_bit_cast(uint16_t, (f16)(v - (float)h));
}
__device__ __forceinline__ float f16_value(uint16_t u) { return (float)__builtin_bit_cast(f16, u); }

// The planes of X = scale G / (|G| + eps) and of its transpose, pads 0; one
// 32 x 32 tile a block, grid (np / 32, mp / 32, batch).  Such a tile of a panel
// is one run of 2 KB: half of the threads write X's, 16 bytes of a plane each,
// half its transpose's.  Bound by the planes' bytes (4096 x 4096 bfloat16: 33 MB
// read, 134 MB written, 40 us).
template <typename IO>
__global__ __launch_bounds__(256) void orth_split(OrthIo io, const double* part, float scale, int mp, int np, OrthMat x,
                                                  OrthMat xt) {
  __shared__ float tile[32][33];
  __shared__ float s_mant;   // scale / (|G| + eps) = s_mant 2^s_exp: of a tiny matrix it is past float32
  __shared__ int s_exp;
  const int p0 = blockIdx.x * 32, i0 = blockIdx.y * 32;
  const int64_t b = blockIdx.z;
  if (threadIdx.x < 64) {
    double s = 0.0;
#pragma unroll
    for (int k = 0; k < ORTH_NORM_BLOCKS / 64; ++k) s += part[b * ORTH_NORM_BLOCKS + 64 * k + threadIdx.x];
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d, 64);
    if (threadIdx.x == 0) {
      int e;
      s_mant = (float)frexp((double)scale / (sqrt(s) + (double)io.eps), &e);
      s_exp = e;
    }
  }
  const IO* g = (const IO*)io.g + b * io.g_batch;
  const int c = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < 4; ++k) {   // rows of the tensor: along i or, tall, along p
    const int r = (threadIdx.x >> 5) + 8 * k;
    const int i = i0 + (io.tall ? c : r), p = p0 + (io.tall ? r : c);
    const float v = i < io.m && p < io.n ? to_f32(g[at_x<IO>(io, io.g_row, i, p)]) : 0.0f;
    tile[i - i0][p - p0] = v;
  }
  __syncthreads();
  const float mant = s_mant;
  const int ex = s_exp;
  const bool turned = threadIdx.x >= 128;
  const int row = (threadIdx.x & 127) >> 2, k8 = (threadIdx.x & 3) * 8;
  uint16_t hi[8], lo[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) planes_of(ldexpf(turned ? tile[k8 + e][row] : tile[row][k8 + e], ex) * mant, hi[e], lo[e]);
  const OrthMat& to = turned ? xt : x;
  uint16_t* at = to.p + b * to.batch + (turned ? panel(p0 + row, i0 + k8, np) : panel(i0 + row, p0 + k8, mp));
  __builtin_memcpy(__builtin_assume_aligned(at, 16), hi, 16);
  __builtin_memcpy(__builtin_assume_aligned(at + to.plane, 16), lo, 16);
}

// Row and column of a tile: on and above the diagonal, column after column, or
// row after row.
template <bool SYM>
__device__ __forceinline__ void place(int tile, int nt, int& ti, int& tj) {
  if constexpr (SYM) {
    tj = (int)((sqrtf(8.0f * (float)tile + 1.0f) - 1.0f) * 0.5f);
    while ((tj + 1) * (tj + 2) / 2 <= tile) ++tj;
    while (tj * (tj + 1) / 2 > tile) --tj;
    ti = tile - tj * (tj + 1) / 2;
  } else {
    ti = tile / nt;
    tj = tile % nt;
  }
}

// Between a wave's writes to its own LDS and its lanes' reads of each other's
// (and back): LDS takes a wave's operations in their order, so only the
// compiler, for which differently typed accesses are independent, has to keep it.
__device__ __forceinline__ void wave_fence() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_wave_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// What is done with a wave's WT x WT piece of a product, at row row_w and column
// col_w: scaled, the other terms added, rounded and written.  A lane holds rows
// 8 (r / 4) + 4 hf + r % 4 of column l32 of every 32 x 32 block.  Panels go
// through `mine`, a piece of LDS of the wave's own, one plane at a time:
// 32-column blocks of WT rows of 64 bytes, which are whole kilobytes of the
// panel in memory.
template <int EPI, int NF, typename IO>
__device__ __forceinline__ void finish(const OrthGemmArgs& a, f32x16 (&acc)[NF][NF], int row_w, int col_w, bool off_diagonal,
                                       int64_t z, char* mine) {
  constexpr int WT = 32 * NF;
  constexpr bool SYM = EPI == ORTH_GRAM || EPI == ORTH_POLY;
  const int lane = threadIdx.x & 63, l32 = lane & 31, hf = lane >> 5;
  constexpr int LINES = WT * WT * 2 / 1024, PER = WT / 16;   // kilobytes, and those of a block
  auto line = [&](const OrthMat& t, int rows, int r0, int k0, int n) {   // a lane's 16 bytes of kilobyte n
    return t.p + z * t.batch + panel(r0 + n % PER * 16 + (lane >> 2), k0 + n / PER * 32 + (lane & 3) * 8, rows);
  };
#pragma unroll
  for (int i = 0; i < NF; ++i)
#pragma unroll
    for (int j = 0; j < NF; ++j) acc[i][j] *= a.sacc;
  if constexpr (EPI == ORTH_POLY) {   // b A + a I
    for (int p = 0; p < 2; ++p) {
      uint4 in[LINES];
#pragma unroll
      for (int n = 0; n < LINES; ++n) in[n] = *(const uint4*)(line(a.old, a.M, row_w, col_w, n) + p * a.old.plane);
#pragma unroll
      for (int n = 0; n < LINES; ++n) *(uint4*)(mine + n * 1024 + lane * 16) = in[n];
      wave_fence();
#pragma unroll
      for (int i = 0; i < NF; ++i)
#pragma unroll
        for (int j = 0; j < NF; ++j)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            acc[i][j][r] += a.sold * f16_value(*(const uint16_t*)(mine + ((j * WT + 32 * i + 8 * (r >> 2) + 4 * hf + (r & 3)) * 32 + l32) * 2));
      wave_fence();
    }
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
      for (int j = 0; j < NF; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (row_w + 32 * i + 8 * (r >> 2) + 4 * hf + (r & 3) == col_w + 32 * j + l32) acc[i][j][r] += a.diag;
  }
  if constexpr (EPI == ORTH_OUT) {
    const OrthIo& io = a.io;
    IO* y = (IO*)io.out + z * io.o_batch;
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
      for (int j = 0; j < NF; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int row = row_w + 32 * i + 8 * (r >> 2) + 4 * hf + (r & 3), col = col_w + 32 * j + l32;
          if (row < io.m && col < io.n) y[at_x<IO>(io, io.o_row, row, col)] = from_f32<IO>(acc[i][j][r]);
        }
    return;
  }
  const bool mirror = !SYM || off_diagonal;
  const OrthMat& turned = SYM ? a.c : a.ct;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    // one float32 value for all of a plane's conversions (see planes_of)
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
      for (int j = 0; j < NF; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          float v = acc[i][j][r];
          asm volatile("" : "+v"(v));
          acc[i][j][r] = v;
        }
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
      for (int j = 0; j < NF; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          *(f16*)(mine + ((j * WT + 32 * i + 8 * (r >> 2) + 4 * hf + (r & 3)) * 32 + l32) * 2) = (f16)acc[i][j][r];
    wave_fence();
#pragma unroll
    for (int n = 0; n < LINES; ++n)
      *(uint4*)(line(a.c, a.M, row_w, col_w, n) + p * a.c.plane) = *(const uint4*)(mine + n * 1024 + lane * 16);
    wave_fence();
    if (mirror) {
#pragma unroll
      for (int i = 0; i < NF; ++i)
#pragma unroll
        for (int j = 0; j < NF; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            f16 h[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) h[r] = (f16)acc[i][j][4 * q + r];
            __builtin_memcpy(__builtin_assume_aligned(mine + ((i * WT + 32 * j + l32) * 32 + 8 * q + 4 * hf) * 2, 8), h, 8);
          }
      wave_fence();
#pragma unroll
      for (int n = 0; n < LINES; ++n)
        *(uint4*)(line(turned, a.N, col_w, row_w, n) + p * turned.plane) = *(const uint4*)(mine + n * 1024 + lane * 16);
      wave_fence();
    }
    // what the plane leaves
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
      for (int j = 0; j < NF; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] -= (float)(f16)acc[i][j][r];
  }
}

// C = A B^T on TILE x TILE tiles, four waves of half of that, K in slices of 32
// through an LDS ring of ST stages of KS slices.  TILE 128, or 64 where tiles of
// 128 would leave compute units without one (3 x 333 x 1000, A: 25 us in tiles
// of 128, 13 in tiles of 64, 11 split along K).  Three products of the operands'
// planes.  Slot s of a row's four 16-byte chunks holds chunk s ^ ((row >> 2) & 3),
// so the 16 rows a wave reads at a time lie in different banks.
template <int EPI, int TILE, int ST, bool PART, typename IO>
__global__ __launch_bounds__(256, 2) void orth_gemm(OrthGemmArgs a) {
  constexpr int PL = 2;              // planes of an operand
  constexpr int SLICE = TILE * 64;   // bytes of an operand plane's slice
  constexpr int WT = TILE / 2, NF = WT / 32, LR = TILE / 4;   // a wave's rows, its 32-row blocks, the rows it loads
  constexpr int STAGE = 2 * PL * SLICE;
  constexpr int KS = TILE == 64 ? 2 : 1;   // slices of a round (K is padded to four)
  constexpr bool SYM = EPI == ORTH_GRAM || EPI == ORTH_POLY;
  __shared__ __align__(16) char lds[ST * KS * STAGE];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int64_t z = blockIdx.z;
  int ti, tj;
  // PART: the tiles from a.full on, each in a.split parts along K, whose sums go
  // to a.parts and are joined by orth_join.
  const int tile = PART ? a.full + (int)blockIdx.x / a.split : (int)blockIdx.x;
  place<SYM>(tile, a.N / TILE, ti, tj);
  const int row0 = ti * TILE, col0 = tj * TILE;
  const uint16_t* pa = a.a.p + z * a.a.batch;
  const uint16_t* pb = a.b.p + z * a.b.batch;

  // 1 KB (16 rows of 64 bytes) an instruction: wave w loads rows LR w .. LR w + LR - 1
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;
  const uint32_t src = (uint32_t)((lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 4) & 3)) * 16));
  auto issue_slice = [&](int stage, int kb) {
#pragma unroll
    for (int op = 0; op < 2; ++op) {
      const uint16_t* base = op ? pb : pa;
      const int R = op ? a.N : a.M, r0 = op ? col0 : row0;
      const int64_t plane = op ? a.b.plane : a.a.plane;
#pragma unroll
      for (int p = 0; p < PL; ++p)
#pragma unroll
        for (int h = 0; h < LR / 16; ++h) {
          const uint16_t* from = base + p * plane + ((int64_t)kb * R + r0 + LR * wave + 16 * h) * 32;
          lds_load16(from, src, lds0 + stage * STAGE + (op * PL + p) * SLICE + (LR * wave + 16 * h) * 64);
        }
    }
  };
  f32x16 acc[NF][NF] = {};
  const int wr = (wave >> 1) * WT, wc = (wave & 1) * WT, l32 = lane & 31, hf = lane >> 5;
  int k0 = 0, nk = a.K / 32;   // the slices of this workgroup
  if constexpr (PART) {
    const int all = nk, part = (int)blockIdx.x % a.split;
    k0 = (int)((int64_t)(all / 4) * part / a.split) * 4;   // fours of slices: whole rounds
    nk = (int)((int64_t)(all / 4) * (part + 1) / a.split) * 4 - k0;
  }
  // Loads of a wave in a round; rounds behind the last load its slices again, so
  // that the count of loads in flight is the same in every round.
  constexpr int LOADS = 2 * PL * (LR / 16) * KS;
  const int rounds = nk / KS;
  auto issue = [&](int stage, int round) {
#pragma unroll
    for (int k = 0; k < KS; ++k) issue_slice(stage * KS + k, k0 + min(round, rounds - 1) * KS + k);
  };
  for (int s = 0; s < ST - 1; ++s) issue(s, s);
  int cur = 0, fill = ST - 1;
  f32x16 cross[NF == 1 ? 1 : NF][NF == 1 ? 1 : NF] = {};   // of the small planes, where one block a wave would wait for itself
  for (int rd = 0; rd < rounds; ++rd) {
    __builtin_amdgcn_s_waitcnt(WaitVmLgkm<LOADS * (ST - 2)>::imm);
    ring_barrier();   // the round's slices are there, and every wave is done with the stage that is filled next
    issue(fill, rd + ST - 1);
    const char* st0 = lds + cur * (KS * STAGE);
    cur = cur + 1 == ST ? 0 : cur + 1;
    fill = fill + 1 == ST ? 0 : fill + 1;
#pragma unroll
    for (int k = 0; k < 2 * KS; ++k) {
      const char* st = st0 + (k >> 1) * STAGE;
      const int ch = 2 * (k & 1) + hf;
      f16x8 fa[PL][NF], fb[PL][NF];
#pragma unroll
      for (int p = 0; p < PL; ++p)
#pragma unroll
        for (int t = 0; t < NF; ++t) {
          const int ra = wr + 32 * t + l32, rb = wc + 32 * t + l32;
          fa[p][t] = *(const f16x8*)(st + p * SLICE + ra * 64 + ((ch ^ ((ra >> 2) & 3)) * 16));
          fb[p][t] = *(const f16x8*)(st + (PL + p) * SLICE + rb * 64 + ((ch ^ ((rb >> 2) & 3)) * 16));
        }
#pragma unroll
      for (int i = 0; i < NF; ++i)
#pragma unroll
        for (int j = 0; j < NF; ++j) {
          f32x16& x = NF == 1 ? cross[0][0] : acc[i][j];
          x = __builtin_amdgcn_mfma_f32_32x32x16_f16(fa[1][i], fb[0][j], x, 0, 0, 0);
          x = __builtin_amdgcn_mfma_f32_32x32x16_f16(fa[0][i], fb[1][j], x, 0, 0, 0);
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fa[0][i], fb[0][j], acc[i][j], 0, 0, 0);
        }
    }
  }
  if constexpr (NF == 1) acc[0][0] += cross[0][0];
  __builtin_amdgcn_s_waitcnt(WaitVmLgkm<0>::imm);   // no load may reach LDS after the workgroup's end
  if constexpr (PART) {   // [tile, part][wave][16 registers of four][lane]
    float* to = a.parts + ((z * gridDim.x + blockIdx.x) * 4 + wave) * (NF * NF * 1024) + lane * 4;
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
      for (int j = 0; j < NF; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *(f32x4*)(to + ((i * NF + j) * 4 + q) * 256) =
              f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
  } else {
    ring_barrier();   // every wave is done with the ring
    finish<EPI, NF, IO>(a, acc, row0 + wr, col0 + wc, ti != tj, z, lds + wave * (WT * WT * 2));
  }
}

// The tiles that were split along K: one wave a quarter, its parts added in
// their order (16 tiles in 8 parts: 10 us, bound by latency).
template <int EPI, int TILE, typename IO>
__global__ __launch_bounds__(64) void orth_join(OrthGemmArgs a) {
  constexpr int NF = TILE / 64, WT = TILE / 2;
  constexpr bool SYM = EPI == ORTH_GRAM || EPI == ORTH_POLY;
  __shared__ __align__(16) char lds[WT * WT * 2];
  const int wave = blockIdx.x & 3, tile = blockIdx.x >> 2;
  const int64_t z = blockIdx.z;
  int ti, tj;
  place<SYM>(a.full + tile, a.N / TILE, ti, tj);
  f32x16 acc[NF][NF] = {};
  for (int p = 0; p < a.split; ++p) {
    const float* from = a.parts + (((z * (gridDim.x >> 2) + tile) * a.split + p) * 4 + wave) * (NF * NF * 1024) + threadIdx.x * 4;
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
      for (int j = 0; j < NF; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const f32x4 v = *(const f32x4*)(from + ((i * NF + j) * 4 + q) * 256);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][j][4 * q + r] += v[r];
        }
  }
  finish<EPI, NF, IO>(a, acc, ti * TILE + (wave >> 1) * WT, tj * TILE + (wave & 1) * WT, ti != tj, z, lds);
}

template <typename IO>
void small(const OrthIo& io, const OrthPoly& p, hipStream_t s) {
  const dim3 grid((unsigned)io.batch);
#define PC_ORTH_SMALL(MB, NT)                                                            \
  if (p.shift > 0.0) launch_kernel(orth_small<IO, MB, NT, true>, grid, dim3(NT), 0, s, io, p); \
  else launch_kernel(orth_small<IO, MB, NT, false>, grid, dim3(NT), 0, s, io, p);
  if (io.m <= 16) {
    PC_ORTH_SMALL(1, 1024)
  } else if (io.m <= 32) {
    PC_ORTH_SMALL(2, 512)
  } else {
    PC_ORTH_SMALL(4, 512)
  }
#undef PC_ORTH_SMALL
}

template <int EPI, typename IO>
void gemm(const OrthGemmArgs& a, hipStream_t s) {
  const bool sym = EPI == ORTH_GRAM || EPI == ORTH_POLY;
  auto grid = [&](int tile) {
    const unsigned mt = (unsigned)(a.M / tile), nt = (unsigned)(a.N / tile);
    return dim3(sym ? mt * (mt + 1) / 2 : mt * nt, 1, (unsigned)a.io.batch);
  };
  OrthGemmArgs b = a;
  dim3 g = grid(128);
  if ((int64_t)g.x * g.z < 256) {
    // Tiles of 64.  Few of them with a long K are bound by a compute unit's
    // loads in flight: they are split along K, so that more units load.
    g = grid(64);
    const int64_t tiles = (int64_t)g.x * g.z;
    b.full = 0;
    b.split = a.parts ? (int)std::min<int64_t>({4, ORTH_FEW_PARTS / tiles, a.K / 32 / 8}) : 1;
    if (b.split > 1) {
      const dim3 parts(g.x * (unsigned)b.split, 1, g.z), quarters(g.x * 4, 1, g.z);
      launch_kernel(orth_gemm<EPI, 64, 2, true, IO>, parts, dim3(256), 0, s, b);
      launch_kernel(orth_join<EPI, 64, IO>, quarters, dim3(64), 0, s, b);
    } else {
      launch_kernel(orth_gemm<EPI, 64, 2, false, IO>, g, dim3(256), 0, s, b);
    }
    return;
  }
  // Whole rounds of one workgroup a compute unit take whole tiles; the tiles
  // left over, which would take another round for a few of them (528 tiles of a
  // symmetric 4096: 16), are split along K into up to 8 parts each, of 8 slices
  // or more.
  const int rest = (int)(g.x % 256);
  b.full = (int)g.x - rest;
  b.split = a.parts && g.z == 1 && rest ? std::max(1, std::min({ORTH_PARTS / rest, 8, a.K / 32 / 8})) : 1;
  if (b.split > 1) g.x = (unsigned)b.full;
  launch_kernel(orth_gemm<EPI, 128, 2, false, IO>, g, dim3(256), 0, s, b);
  if (b.split > 1) {
    launch_kernel(orth_gemm<EPI, 128, 2, true, IO>, dim3((unsigned)(rest * b.split)), dim3(256), 0, s, b);
    launch_kernel(orth_join<EPI, 128, IO>, dim3((unsigned)rest * 4), dim3(64), 0, s, b);
  }
}
}  // namespace

#define PC_ORTH_TYPES(f)                    \
  if (dtype == PC_DTYPE_F32) {              \
    f(float)                                \
  } else if (dtype == PC_DTYPE_F16) {       \
    f(f16)                                  \
  } else {                                  \
    f(bf16)                                 \
  }

void launch_orth_small(const OrthIo& io, const OrthPoly& p, int dtype, hipStream_t s) {
#define F(T) small<T>(io, p, s);
  PC_ORTH_TYPES(F)
#undef F
}

void launch_orth_norm(const OrthIo& io, int dtype, double* part, hipStream_t s) {
  const dim3 grid(ORTH_NORM_BLOCKS, (unsigned)io.batch);
#define F(T) launch_kernel(orth_norm<T>, grid, dim3(256), 0, s, io, part);
  PC_ORTH_TYPES(F)
#undef F
}

void launch_orth_split(const OrthIo& io, int dtype, const double* part, float scale, int mp, int np, const OrthMat& x,
                       const OrthMat& xt, hipStream_t s) {
  const dim3 grid((unsigned)(np / 32), (unsigned)(mp / 32), (unsigned)io.batch);
#define F(T) launch_kernel(orth_split<T>, grid, dim3(256), 0, s, io, part, scale, mp, np, x, xt);
  PC_ORTH_TYPES(F)
#undef F
}

void launch_orth_gemm(const OrthGemmArgs& a, int epi, int dtype, hipStream_t s) {
  if (epi == ORTH_GRAM) gemm<ORTH_GRAM, float>(a, s);
  else if (epi == ORTH_POLY) gemm<ORTH_POLY, float>(a, s);
  else if (epi == ORTH_APPLY) gemm<ORTH_APPLY, float>(a, s);
  else {
#define F(T) gemm<ORTH_OUT, T>(a, s);
    PC_ORTH_TYPES(F)
#undef F
  }
}

}  // namespace pc
