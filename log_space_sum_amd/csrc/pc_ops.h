// pc_ops.h -- argument blocks and launchers of the sequence-network operators
// (layer norm, linear attention with decay, orthogonalised update).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/pc.h"
#include "pc_device.h"
#include "pc_launch.h"

namespace pc {

// ---- element types ---------------------------------------------------------
// bfloat16 as its 16 bits; conversions round to nearest even and keep NaN.
struct bf16 {
  uint16_t u;
};
typedef _Float16 f16;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(f16 x) { return (float)x; }
__device__ __forceinline__ float to_f32(bf16 x) { return __uint_as_float((uint32_t)x.u << 16); }
__device__ __forceinline__ uint16_t bf16_bits(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }
template <typename T>
__device__ __forceinline__ T from_f32(float f);
template <>
__device__ __forceinline__ float from_f32<float>(float f) { return f; }
template <>
__device__ __forceinline__ f16 from_f32<f16>(float f) { return (f16)f; }
template <>
__device__ __forceinline__ bf16 from_f32<bf16>(float f) { return bf16{bf16_bits(f)}; }

// ---- layer norm ------------------------------------------------------------
struct NormArgs {
  int64_t rows;
  int32_t cols;
  const void* x;
  int64_t x_stride;
  const void* dy;       // backward
  int64_t dy_stride;
  const float* weight;  // nullable: 1
  const float* bias;    // nullable: 0
  float eps;
  void* y;              // forward: y; backward: dx
  int64_t y_stride;
  float* mean;
  float* rstd;
  float* part;          // backward: [parts][2][cols] partial sums of dweight, dbias
  int32_t parts;
  float* dweight;
  float* dbias;
};
constexpr int NORM_MAX_COLS = 16384;
int norm_parts(int64_t rows, int cols);
void launch_norm_fwd(const NormArgs& a, int dtype, hipStream_t s);
void launch_norm_bwd(const NormArgs& a, int dtype, hipStream_t s);

// ---- linear attention with a decay for each head ---------------------------
// One walk along the sequences (see k_linattn.hip): tensors a (contracted with
// the state), b and c (which make the state), the output, and the states.
struct MixTensor {
  const void* p;
  int64_t ts, hs;       // token and head strides (elements)
  int32_t div;          // heads that share one of the tensor's: head h reads h / div
};
struct MixArgs {
  int32_t seqs, heads, da, dc;
  int64_t tokens;
  const int32_t* cu;    // [seqs + 1], null: one sequence of all tokens
  const float* log_decay;
  MixTensor a, b, c;
  void* out;
  int64_t o_ts, o_hs;
  int32_t out_f32;      // the output is a float32 partial, whatever the tensors' type
  int32_t rev;          // tokens from the sequence's end to its start
  int32_t off;          // 1: the carried state is decayed before a token joins it, 0: after
  float pscale, wscale, oscale;   // factors of the inside products, of a token's part in the state, of the state's output
  const float* init;    // [seqs, heads, da x dc], nullable: 0
  float* fin;           // the states after the last token, nullable
  int32_t st_r, st_c;   // strides of a state's row (da) and column (dc)
  float* seg;           // [slots, heads, da x dc] states at the segments' starts, when nsegs > 1 (see seg_slot)
  int32_t nsegs, packed;
  int64_t seglen;
};
// Walks of one shape (da, dc), sequences and segments that a launch takes side
// by side: the backward's three, or its two passes over the segments.
struct MixMany {
  MixArgs w[3];
  int32_t n, seqs;
};
struct MixScanArgs {
  int32_t seqs, heads, nsegs, packed, elems;
  int64_t tokens, seglen;
  const int32_t* cu;
  const float* log_decay;
  const float* init;
  float* seg;
};
// Where the states of a sequence's segments lie, of its first: in a row for
// every sequence, or packed by the sequences' first tokens t0.  Only sequences of
// more than one segment have any; such a one of n tokens has ceil(n / seglen)
// <= floor(2 n / seglen) of them, so the next one's begin behind its last.
__host__ __device__ inline int64_t seg_slot(int packed, int nsegs, int64_t seglen, int64_t seq, int64_t t0) {
  return packed ? 2 * t0 / seglen : seq * nsegs;
}
struct MixSumArgs {     // out[t, h] = sum of the group's heads of part[t, h * group ..], of the sequences' tokens
  int64_t tokens;
  int32_t seqs, kv_heads, group, dim;
  const int32_t* cu;
  const float* part;    // [tokens, kv_heads * group, dim]
  void* out;
  int64_t o_ts, o_hs;
};
struct MixStepArgs {
  int32_t batch, heads, group, dk, dv, slots;
  const void *q, *k, *v;
  int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs;
  const float* log_decay;
  float scale;
  float* state;         // [slots, heads, dk, dv]
  const int32_t* slot;  // [batch], null: row b uses slot b
  void* o;
  int64_t o_ts, o_hs;
};
constexpr int MIX_MAX_DIM = 128;
constexpr int64_t MIX_MAX_STRIDE = 1 << 23;   // elements from a token to the next: 64 rows within 2^31 bytes
void launch_mix_walk(const MixArgs* a, int n, int dtype, hipStream_t s);    // outputs (and final states)
void launch_mix_states(const MixArgs* a, int n, int dtype, hipStream_t s);  // each segment's own state into seg
void launch_mix_scan(const MixScanArgs* a, int n, hipStream_t s);           // seg: own states -> states at the starts
void launch_mix_sum(const MixSumArgs& a, const MixSumArgs& b, int dtype, hipStream_t s);
void launch_mix_step(const MixStepArgs& a, int dtype, hipStream_t s);

// ---- orthogonalised update ---------------------------------------------------
// m <= n: the smaller and the larger dimension of the matrices; tall: the rows
// are the larger one.  X [m, n] is the matrix or its transpose.
struct OrthIo {
  int64_t batch;
  int32_t m, n, tall;
  const void* g;
  int64_t g_batch, g_row;
  void* out;
  int64_t o_batch, o_row;
  float eps;
};
constexpr int ORTH_SMALL = 64;       // all steps on m x m matrices, in 64 bits, up to this m
constexpr int ORTH_MAX_STEPS = 32;
constexpr double ORTH_GROWTH = 2048.0;   // of Q, up to which its steps run on A itself
struct OrthPoly {
  int32_t steps;
  float c[ORTH_MAX_STEPS][3];
  double shift;                      // past that growth: added to A's diagonal; else 0
};
constexpr int ORTH_TILE = 128;       // rows and columns of the operands are padded to it
constexpr int ORTH_NORM_BLOCKS = 512; // partial sums of a matrix's norm
// Operands of the products: float16 planes (hi, lo) of scaled values in
// K-blocked panels, one after the other for the matrices of the batch.
struct OrthMat {
  uint16_t* p;
  int64_t plane;        // elements from the hi to the lo plane
  int64_t batch;        // elements from one matrix to the next
};
constexpr int ORTH_PARTS = 512;       // partial tiles (128) of a product's last round
constexpr int ORTH_FEW_PARTS = 256;   // partial tiles (64) of a product with few tiles
enum OrthEpi { ORTH_GRAM, ORTH_POLY, ORTH_APPLY, ORTH_OUT };
struct OrthGemmArgs {
  int32_t M, N, K;      // padded; C [M, N] = A [M, K] B [N, K]^T
  OrthMat a, b;
  OrthMat old;          // POLY: added to the product (panels of [M, N])
  OrthMat c, ct;        // the result's panels and its transpose's (GRAM / POLY: c alone, both halves)
  float sacc, sold;     // result = sacc acc (POLY: + sold old)
  float diag;           // POLY: + diag I
  float* parts;         // room for ORTH_PARTS or ORTH_FEW_PARTS tiles' partial sums, nullable
  int32_t full, split;  // set at the launch: tiles taken whole, parts of each tile behind them
  OrthIo io;            // OUT
};
void launch_orth_small(const OrthIo& io, const OrthPoly& p, int dtype, hipStream_t s);
void launch_orth_norm(const OrthIo& io, int dtype, double* part, hipStream_t s);
void launch_orth_split(const OrthIo& io, int dtype, const double* part, float scale, int mp, int np, const OrthMat& x,
                       const OrthMat& xt, hipStream_t s);
void launch_orth_gemm(const OrthGemmArgs& a, int epi, int dtype, hipStream_t s);

}  // namespace pc
