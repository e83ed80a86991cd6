// pc_ops_api.hip -- the C ABI of the sequence-network operators: argument
// checks, the linear attention's split into segments, and the launch lists.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <exception>
#include <string>

#include "pc_ops.h"
#include "pc_runtime.h"

using namespace pc;

namespace {

template <typename F>
int guarded(F&& f) {
  try {
    f();
    return PC_OK;
  } catch (const Error& e) {
    return set_error(e.code, e.msg);
  } catch (const std::exception& e) {
    return set_error(PC_ERR_INVALID_ARG, e.what());
  }
}

void need(bool ok, const std::string& what) {
  if (!ok) fail(PC_ERR_INVALID_ARG, what);
}

void check_device(int device) {
  if (device < 0) fail(PC_ERR_NO_DEVICE, "device " + std::to_string(device));
}

void check_dtype(int dtype) {
  if (dtype != PC_DTYPE_F32 && dtype != PC_DTYPE_BF16 && dtype != PC_DTYPE_F16)
    fail(PC_ERR_UNSUPPORTED, "unknown dtype " + std::to_string(dtype));
}

void check_ws(const void* ws, size_t have, size_t want) {
  if (want == 0) return;
  if (!ws || have < want)
    fail(PC_ERR_WORKSPACE, "workspace of " + std::to_string(ws ? have : 0) + " bytes, needs " + std::to_string(want));
  need((uintptr_t)ws % 16 == 0, "workspace not aligned to 16 bytes");
}

// ---- layer norm --------------------------------------------------------------

void check_norm(int64_t rows, int32_t cols) {
  need(rows >= 0 && rows <= INT_MAX, "rows must be in [0, 2^31)");
  need(cols >= 1, "cols must be at least 1");
  if (cols > NORM_MAX_COLS)
    fail(PC_ERR_UNSUPPORTED, std::to_string(cols) + " columns (at most " + std::to_string(NORM_MAX_COLS) + ")");
}

size_t norm_ws(int64_t rows, int32_t cols) { return (size_t)norm_parts(rows, cols) * 2 * cols * sizeof(float); }

// ---- linear attention ----------------------------------------------------------

void check_mix(const pc_linear_attention* d) {
  need(d, "null descriptor");
  check_dtype(d->dtype);
  need(d->heads >= 1 && d->kv_heads >= 1 && d->heads % d->kv_heads == 0, "kv_heads must divide heads");
  need(d->heads <= 65535, "more than 65535 heads");
  need(d->dim_k >= 1 && d->dim_v >= 1, "dim_k and dim_v must be at least 1");
  if (d->dim_k > MIX_MAX_DIM || d->dim_v > MIX_MAX_DIM)
    fail(PC_ERR_UNSUPPORTED, "dim_k " + std::to_string(d->dim_k) + ", dim_v " + std::to_string(d->dim_v) + " (at most " +
                                 std::to_string(MIX_MAX_DIM) + ")");
  need(d->num_tokens >= 0 && d->num_tokens <= INT_MAX, "num_tokens must be in [0, 2^31)");
}

void check_seqs(const pc_linear_attention* d) {
  check_mix(d);
  need(d->num_seqs >= 0, "num_seqs must be at least 0");
  if (d->num_seqs > 65535) fail(PC_ERR_UNSUPPORTED, std::to_string(d->num_seqs) + " sequences (at most 65535)");
  need(d->max_seqlen >= 0, "max_seqlen must be at least 0");
}

void check_call(const pc_linear_attention* d) {
  check_seqs(d);
  need(d->cu_seqlens || d->num_seqs == 1, "without cu_seqlens num_seqs is 1");
  need(d->log_decay, "null log_decay");
  need(std::isfinite(d->scale) && d->scale != 0.0f, "scale must be finite and not 0");
}

template <typename D>
void check_heads(const D* d, const pc_heads& t, const char* what, bool chunks = true) {
  need(t.data || d->num_tokens == 0, std::string("null ") + what);
  need(t.token_stride >= 0 && t.head_stride >= 0, std::string("negative stride of ") + what);
  // a chunk's rows are addressed with 32-bit byte offsets
  if (chunks && d->num_tokens > 1 && t.token_stride > MIX_MAX_STRIDE)
    fail(PC_ERR_UNSUPPORTED, std::string("token stride of ") + what + " above " + std::to_string(MIX_MAX_STRIDE));
}
// an output's elements must be distinct
template <typename D>
void check_out(const D* d, const pc_heads& t, int heads, int dim, const char* what, bool chunks = true) {
  check_heads(d, t, what, chunks);
  const int64_t ts = t.token_stride, hs = t.head_stride;
  const bool tokens_outside = (heads == 1 || hs >= dim) && (d->num_tokens <= 1 || ts >= (heads - 1) * hs + dim);
  const bool heads_outside = (d->num_tokens <= 1 || ts >= dim) && (heads == 1 || hs >= (d->num_tokens - 1) * ts + dim);
  need(tokens_outside || heads_outside, std::string("elements of ") + what + " overlap");
}

// Segments of the longest sequence.  One walk of a (sequence, head) is a chain
// of chunks (about 3 us each when little else runs), so where sequences and
// heads are too few to fill the card the sequences are cut.  A cut costs a
// second reading of b and c, two more launches, and a state for each segment
// and head that is written and read twice:
//  - up to five chunks are not cut (one sequence of 300 x 4 heads x 64: 18 us
//    whole, 20 in three; 16 of 200 x 8 heads: 18 and 24),
//  - a segment has two chunks or more, and tokens enough that their own bytes
//    are as many as the state's (two sequences of 4000 x 8 heads x 128: 53 us in
//    segments of 256 tokens, 58 in segments of 128),
//  - the scan goes through the segments one after the other, so their number is
//    at most of the order of the root of the chunks' number.
// Ragged batches are counted as full sequences of the same number of tokens.
struct Split {
  int nsegs;
  int64_t len;
};
Split mix_segments(const pc_linear_attention* d) {
  const int64_t longest = std::max<int64_t>(1, std::min(d->max_seqlen, d->num_tokens));
  const int64_t chunk = d->dtype == PC_DTYPE_BF16 ? 64 : 32, chunks = (longest + chunk - 1) / chunk;
  if (chunks <= 5) return {1, chunks * chunk};
  const int64_t full = std::min<int64_t>(d->num_seqs, (d->num_tokens + longest - 1) / longest);
  const int64_t walks = std::max<int64_t>(1, full * d->heads);
  // walks aimed at: two workgroups a compute unit at dim 128, four of the smallest
  // at 64 and below (of bfloat16 at dim 64 three fit, of dims between 64 and 128
  // one or two: there some walks take a second round)
  const int64_t room = std::max(d->dim_k, d->dim_v) > 64 ? 512 : 1024;
  const double mean = 2.0 * d->dim_k * d->dim_v / (d->dim_k + d->dim_v);
  const int64_t least = std::max(2 * chunk, (int64_t)(3.2 * mean / (d->dtype == PC_DTYPE_F32 ? 4 : 2)));
  const int64_t n = std::max<int64_t>(1, std::min({(room + walks - 1) / walks, (longest + least - 1) / least,
                                                   (int64_t)std::sqrt(32.0 * (double)chunks)}));
  const int64_t len = ((longest + n - 1) / n + chunk - 1) / chunk * chunk;
  return {(int)((longest + len - 1) / len), len};
}

// The states' slots (see seg_slot): packed where that takes fewer, as with many
// sequences of which few can have a second segment (4096 of 512 tokens whose
// longest is not given, 16 heads x 128: 65 slots instead of 131072 = 137 GB).
struct Slots {
  int64_t n;
  bool packed;
};
Slots mix_slots(const pc_linear_attention* d, const Split& sp) {
  if (sp.nsegs <= 1) return {0, false};
  const int64_t rows = (int64_t)d->num_seqs * sp.nsegs, packed = 2 * d->num_tokens / sp.len + 1;
  return {std::min(rows, packed), packed < rows};
}

struct MixWs {
  size_t seg_f = 0, seg_r = 0, dk = 0, dv = 0, total = 0;
};
MixWs mix_ws(const pc_linear_attention* d, bool backward) {
  MixWs w;
  const Split sp = mix_segments(d);
  const size_t states = (size_t)mix_slots(d, sp).n * d->heads * d->dim_k * d->dim_v * sizeof(float);
  auto take = [&](size_t bytes) {
    const size_t at = w.total;
    w.total += (bytes + 255) / 256 * 256;
    return at;
  };
  w.seg_f = take(states);
  if (backward) {
    w.seg_r = take(states);
    if (d->heads != d->kv_heads) {
      w.dk = take((size_t)d->num_tokens * d->heads * d->dim_k * sizeof(float));
      w.dv = take((size_t)d->num_tokens * d->heads * d->dim_v * sizeof(float));
    }
  }
  return w;
}

MixTensor tensor(const pc_heads& t, int div) { return {t.data, t.token_stride, t.head_stride, div}; }

MixArgs mix_base(const pc_linear_attention* d, const Split& sp) {
  MixArgs a{};
  a.seqs = d->num_seqs;
  a.heads = d->heads;
  a.tokens = d->num_tokens;
  a.cu = d->cu_seqlens;
  a.log_decay = d->log_decay;
  a.pscale = d->scale;
  a.nsegs = sp.nsegs;
  a.packed = mix_slots(d, sp).packed;
  a.seglen = sp.len;
  return a;
}

// The states at the segments' starts (nothing to do for one segment) of n walks
// of the shape (dim_k, dim_v), from the states in a[k].init.
void mix_starts(const pc_linear_attention* d, const MixArgs* a, int n, hipStream_t s) {
  if (a[0].nsegs <= 1) return;
  launch_mix_states(a, n, d->dtype, s);
  check_launch();
  MixScanArgs c[2]{};
  for (int k = 0; k < n; ++k) {
    c[k].seqs = a[k].seqs;
    c[k].heads = a[k].heads;
    c[k].nsegs = a[k].nsegs;
    c[k].packed = a[k].packed;
    c[k].elems = d->dim_k * d->dim_v;
    c[k].tokens = a[k].tokens;
    c[k].seglen = a[k].seglen;
    c[k].cu = a[k].cu;
    c[k].log_decay = a[k].log_decay;
    c[k].init = a[k].init;
    c[k].seg = a[k].seg;
  }
  launch_mix_scan(c, n, s);
  check_launch();
}

// ---- softmax attention -----------------------------------------------------------

void check_attn_sizes(const pc_attention* d) {
  need(d, "null descriptor");
  check_dtype(d->dtype);
  need(d->heads >= 1 && d->kv_heads >= 1 && d->heads % d->kv_heads == 0, "kv_heads must divide heads");
  need(d->heads <= 65535, "more than 65535 heads");
  need(d->dim_k >= 1 && d->dim_v >= 1, "dim_k and dim_v must be at least 1");
  if (d->dim_k > ATTN_MAX_DIM || d->dim_v > ATTN_MAX_DIM)
    fail(PC_ERR_UNSUPPORTED, "dim_k " + std::to_string(d->dim_k) + ", dim_v " + std::to_string(d->dim_v) + " (at most " +
                                 std::to_string(ATTN_MAX_DIM) + ")");
  need(d->num_tokens >= 0 && d->num_tokens <= 1 << 30, "num_tokens must be in [0, 2^30]");
  need(d->num_seqs >= 0 && d->num_seqs <= 1 << 24, "num_seqs must be in [0, 2^24]");
  need(d->max_seqlen >= 0 && d->max_length >= 0, "max_seqlen and max_length must be at least 0");
}

void check_attn(const pc_attention* d, bool cached = false) {
  check_attn_sizes(d);
  if (cached) need(d->cu_seqlens || d->num_seqs == 1 || d->num_seqs == d->num_tokens, "without cu_seqlens num_seqs is 1 or num_tokens");
  else need(d->cu_seqlens || d->num_seqs == 1, "without cu_seqlens num_seqs is 1");
  need(std::isfinite(d->scale) && d->scale != 0.0f, "scale must be finite and not 0");
  check_heads(d, d->q, "q", false);
  check_heads(d, d->k, "k", false);
  check_heads(d, d->v, "v", false);
}

AttnTensor attn_tensor(const pc_heads& t) { return {t.data, t.token_stride, t.head_stride}; }

AttnArgs attn_base(const pc_attention* d) {
  AttnArgs a{};
  a.seqs = d->num_seqs;
  a.kv_heads = d->kv_heads;
  a.group = d->heads / d->kv_heads;
  a.dk = d->dim_k;
  a.dv = d->dim_v;
  a.tokens = d->num_tokens;
  a.cu = d->cu_seqlens;
  a.scale = d->scale;
  a.q = attn_tensor(d->q);
  a.k = attn_tensor(d->k);
  a.v = attn_tensor(d->v);
  a.o = d->o.data;
  a.o_ts = d->o.token_stride;
  a.o_hs = d->o.head_stride;
  a.lse = d->lse;
  a.nsplit = 1;
  return a;
}

// Parts of whole sequences' keys (and, for dk and dv, rows), where rows, heads and
// sequences are too few to fill the card: a tile of 128 rows is a chain of key
// tiles, 1 to 5 us each.  A part costs its results, written and read once in float32, and a launch that joins them, so
// tiles (`works`) are cut up to a number, to get `aim` of them, not into less than `least`, and no call of up to
// `whole` keys.  Measured, heads x dims bfloat16 unless said, cut and not:
//   forward: 128 works (2048 x 8 (2) x 64, four parts) 37, 50 us, float32 62, 117; 256 works (4 x 1000 x 8 (2) x 128) 57, 44;
//     300 keys (8 (2) x 64) 18, 15; 700 (three parts) 18, 21, float32 27, 45
//   backward: aims of 512, 1024: 128 works 113, 99, float32 258, 211; 256 works 174, 161; 1000 works (2 x 4000 x 16 (4) x
//     128) 1223 whole, 1328; least 256, 128: 700 keys 58, 44, float32 7 ragged of up to 900
//     x 6 (3) x 48, 80 133, 143
struct AttnSplit {
  int nsplit, part_len;
};
AttnSplit attn_split(const pc_attention* d, bool backward) {
  const int64_t group = d->heads / d->kv_heads, tokens = std::max<int64_t>(1, d->num_tokens);
  const int64_t longest = std::max<int64_t>(1, std::min(d->max_seqlen, tokens));
  const int64_t full = std::min<int64_t>(std::max(1, d->num_seqs), (tokens + longest - 1) / longest);
  const int64_t works = full * ((longest * group + ATTN_ROWS - 1) / ATTN_ROWS) * d->kv_heads;
  const int64_t most = backward ? 768 : 128, aim = backward ? 1024 : 512, least = backward && d->dtype != PC_DTYPE_F32 ? 128 : 256;
  const int64_t whole = backward ? 0 : d->dtype == PC_DTYPE_F32 ? 256 : 512;
  if (works > most || longest <= whole) return {1, (int)std::min<int64_t>(longest, INT_MAX)};
  int64_t len = std::max<int64_t>(least, (longest * works + aim - 1) / aim);
  len = round_up(std::max(len, (longest + ATTN_MAX_SPLIT - 1) / ATTN_MAX_SPLIT), 128);
  return {(int)((longest + len - 1) / len), (int)std::min<int64_t>(len, INT_MAX)};
}
struct AttnWs {
  size_t part = 0, stat = 0, part_k = 0, part_v = 0, delta = 0, total = 0;
};
AttnWs attn_ws(const pc_attention* d, bool backward) {
  AttnWs w;
  auto take = [&](size_t bytes) {
    const size_t at = w.total;
    w.total += (bytes + 255) / 256 * 256;
    return at;
  };
  const size_t n = attn_split(d, backward).nsplit, tokens = (size_t)d->num_tokens;
  if (backward) w.delta = take(tokens * d->heads * sizeof(float));
  if (n > 1) {
    w.part = take(n * tokens * d->heads * (backward ? d->dim_k : d->dim_v) * sizeof(float));
    if (!backward) w.stat = take(n * tokens * d->heads * sizeof(float2));
    else {
      w.part_k = take(n * tokens * d->kv_heads * d->dim_k * sizeof(float));
      w.part_v = take(n * tokens * d->kv_heads * d->dim_v * sizeof(float));
    }
  }
  return w;
}

void check_pages(const pc_attention* d) {
  check_attn_sizes(d);
  need(d->page_size >= 1, "page_size must be at least 1");
  need(d->num_pages >= 0 && d->max_pages >= 0, "num_pages and max_pages must be at least 0");
  need((int64_t)d->max_pages * d->page_size + d->num_tokens <= INT_MAX - (1 << 16), "2^31 positions or more");
}

// How new tokens meet a cache.  Rows are the new tokens of a sequence times the
// heads that share a key / value head.
struct CachedPlan {
  bool few;              // few rows: tiles of 32 that all waves share
  int nsplit, part_len;
  size_t part, stat, total;
};
CachedPlan cached_plan(const pc_attention* d) {
  CachedPlan p{};
  const int64_t group = d->heads / d->kv_heads, tokens = std::max<int64_t>(1, d->num_tokens);
  const int64_t rows = std::max<int64_t>(1, std::min(d->max_seqlen, tokens)) * group;
  const int64_t full = std::min<int64_t>(std::max(1, d->num_seqs), (tokens * group + rows - 1) / rows);
  // Two tiles of 32 rows read the keys twice, but each key tile is one wave's: faster for few streams and heads (64 rows of
  // 4 streams x 2 heads x 64 behind 3000 19 us, as one tile of 128 22; 12 streams 25.5, 25; 32 44, 40; 16 x 8 x 128 111, 90; float32 4 streams 21, 33; 16 53, 39).
  p.few = rows <= ATTN_FEW_ROWS || (rows <= 2 * ATTN_FEW_ROWS && full * d->kv_heads <= 24);
  const int64_t tile = p.few ? ATTN_FEW_ROWS : ATTN_ROWS;
  const int64_t works = std::min<int64_t>(std::max<int64_t>(1, full * ((rows + tile - 1) / tile) * d->kv_heads), INT_MAX);
  const int64_t longest = std::max<int64_t>(1, std::min<int64_t>(d->max_length, (int64_t)d->max_pages * d->page_size + tokens));
  // Few rows: many parts, that streams of different lengths fill the card (64 streams of up to 8192 x 32 (8) heads x 128: 235 us with
  // 8192 workgroups, 240 with 4096, 248 with 2048).  Many: two workgroups a CU (four chunks of 512 behind 8192 563 us; with 1024
  // of half the length 591; 16 chunks of 64 behind 4000 187, 210, with 256 258).
  const int64_t aim = p.few ? 8192 : 512;
  // Short ones whole: a launch that joins parts costs 4 us (a token of 8 heads x 64 bfloat16 behind 500: 15 us whole, 18.5 in
  // parts; x 128 17.6, 18.9; behind 1000 18.4, 18.6 and 24, 19; float32 behind 500 19.6, 18.5).
  const int64_t whole = !p.few ? 0 : d->dtype == PC_DTYPE_F32 ? 256 : 512;
  int64_t len = longest <= whole ? whole : std::max<int64_t>(256, (longest * works + aim - 1) / aim);
  len = round_up(std::max(len, (longest + ATTN_MAX_SPLIT - 1) / ATTN_MAX_SPLIT), 128);
  p.nsplit = (int)((longest + len - 1) / len);
  p.part_len = (int)std::min<int64_t>(len, INT_MAX);
  if (p.nsplit > 1) {
    const size_t all = (size_t)p.nsplit * d->num_tokens * d->heads;
    p.stat = (size_t)round_up((int64_t)(all * d->dim_v * sizeof(float)), 256);
    p.total = p.stat + all * sizeof(float2);
  }
  return p;
}

// ---- heads' norm and rotation ------------------------------------------------------

void check_rotary(const pc_rotary* d) {
  need(d, "null descriptor");
  check_dtype(d->dtype);
  need(d->num_tokens >= 0 && d->num_tokens <= INT_MAX, "num_tokens must be in [0, 2^31)");
  need(d->heads >= 0 && d->kv_heads >= 0 && d->heads <= 65535 && d->kv_heads <= 65535, "heads must be in [0, 65535]");
  need(d->dim >= 1, "dim must be at least 1");
  if (d->dim > ROTARY_MAX_DIM)
    fail(PC_ERR_UNSUPPORTED, "dim " + std::to_string(d->dim) + " (at most " + std::to_string(ROTARY_MAX_DIM) + ")");
  need(d->rotary_dim >= 0 && d->rotary_dim % 2 == 0 && d->rotary_dim <= d->dim, "rotary_dim must be even and at most dim");
}

RotaryArgs rotary_base(const pc_rotary* d) {
  check_rotary(d);
  need(d->interleaved == 0 || d->interleaved == 1, "interleaved must be 0 or 1");
  need(d->norm == 0 || d->norm == 1, "norm must be 0 or 1");
  need(std::isfinite(d->magnitude), "magnitude must be finite");
  need(!d->norm || (std::isfinite(d->eps) && d->eps >= 0.0f), "eps must be finite and at least 0");
  need(d->num_tokens == 0 || d->positions, "null positions");
  need(d->rotary_dim == 0 || d->freq, "null freq");
  RotaryArgs a{};
  a.tokens = d->num_tokens;
  a.heads = d->heads;
  a.kv_heads = d->kv_heads;
  a.dim = d->dim;
  a.part = d->rotary_dim;
  a.pairs = d->interleaved;
  a.norm = d->norm;
  a.eps = d->eps;
  a.magnitude = d->magnitude;
  a.positions = d->positions;
  a.freq = d->freq;
  a.qw = d->q_weight;
  a.kw = d->k_weight;
  return a;
}

// An output that is an input has its strides.
void check_place(const pc_rotary* d, const pc_heads& out, const pc_heads& in, int heads, const char* what) {
  need(out.data != in.data || ((d->num_tokens <= 1 || out.token_stride == in.token_stride) && (heads <= 1 || out.head_stride == in.head_stride)),
       std::string(what) + " is its input at other strides");
}

// ---- orthogonalised update -----------------------------------------------------

struct OrthPlan {
  int m, n, mp, np;
  bool small;
  OrthMat x[2], xt[2], a, b;
  size_t part, parts, total;
  bool split;
};
OrthPlan orth_plan(int64_t batch, int32_t rows, int32_t cols, void* ws) {
  OrthPlan p{};
  p.m = std::min(rows, cols);
  p.n = std::max(rows, cols);
  p.small = p.m <= ORTH_SMALL;
  if (p.small || batch == 0) return p;
  p.mp = (int)round_up(p.m, ORTH_TILE);
  p.np = (int)round_up(p.n, ORTH_TILE);
  auto mat = [&](int64_t rows_, int64_t cols_) {
    OrthMat o{};
    o.plane = batch * rows_ * cols_;
    o.batch = rows_ * cols_;
    o.p = (uint16_t*)((char*)ws + p.total);
    p.total += (size_t)round_up(2 * o.plane * (int64_t)sizeof(uint16_t), 256);
    return o;
  };
  for (int k = 0; k < 2; ++k) {
    p.x[k] = mat(p.mp, p.np);
    p.xt[k] = mat(p.np, p.mp);
  }
  p.a = mat(p.mp, p.mp);
  p.b = mat(p.mp, p.mp);
  p.part = p.total;
  p.total += (size_t)batch * ORTH_NORM_BLOCKS * sizeof(double);
  // partial sums of split tiles: of a last round of tiles of 128 (one matrix), or of few tiles of 64
  const int64_t t128 = (int64_t)(p.mp / 128) * (p.np / 128) * batch, s64 = (int64_t)(p.mp / 64) * (p.mp / 64 + 1) / 2 * batch;
  const size_t parts = batch == 1 && t128 >= 256 ? (size_t)ORTH_PARTS * 128 * 128 * sizeof(float)
                       : 2 * s64 <= ORTH_FEW_PARTS ? (size_t)ORTH_FEW_PARTS * 64 * 64 * sizeof(float) : 0;
  p.split = parts > 0;
  p.parts = (size_t)round_up((int64_t)p.total, 256);
  if (p.split) p.total = p.parts + parts;
  return p;
}

void check_orth(int dtype, int64_t batch, int32_t rows, int32_t cols) {
  check_dtype(dtype);
  need(batch >= 0, "batch must be at least 0");
  need(rows >= 1 && cols >= 1, "rows and cols must be at least 1");
  if (batch > 65535) fail(PC_ERR_UNSUPPORTED, std::to_string(batch) + " matrices (at most 65535)");
  if (rows > 32768 || cols > 32768)
    fail(PC_ERR_UNSUPPORTED, std::to_string(rows) + " x " + std::to_string(cols) + " matrices (at most 32768)");
}

// Bounds of the singular values at every step and of the step's polynomials
// b t + c t^2 and a + b t + c t^2 (t the squared singular value), where they start in [0, 1]: the
// largest magnitudes at the interval's ends and the extrema inside it.  What
// goes into the next step's interval is widened by 2^-20, as far as a step's
// rounding (two float16 planes, 2^-22) can carry a value: triples tuned for their
// own interval rise steeply behind its end, so a wider margin would compound
// into a growth that is none.  The 2% are room in the scales alone.
struct OrthBounds {
  double x[ORTH_MAX_STEPS + 1], p[ORTH_MAX_STEPS];
};
OrthBounds orth_bounds(int steps, const float* coef) {
  OrthBounds o;
  double top = 1.0;
  for (int s = 0; s < steps; ++s) {
    const double a = coef[3 * s], b = coef[3 * s + 1], c = coef[3 * s + 2], tmax = top * top;
    o.x[s] = 1.02 * top;
    double next = 0.0, poly = 0.0;
    auto at = [&](double t) {
      if (!(t >= 0.0 && t <= tmax)) return;
      poly = std::max({poly, std::fabs(t * (b + c * t)), std::fabs(a + t * (b + c * t))});
      next = std::max(next, std::fabs(std::sqrt(t) * (a + t * (b + c * t))));
    };
    at(0.0);
    at(tmax);
    if (c != 0.0) {
      at(-b / (2.0 * c));                                 // of the polynomial
      const double d = 9.0 * b * b - 20.0 * a * c;        // of a x + b x^3 + c x^5: a + 3 b t + 5 c t^2 = 0
      if (d >= 0.0) {
        at((-3.0 * b + std::sqrt(d)) / (10.0 * c));
        at((-3.0 * b - std::sqrt(d)) / (10.0 * c));
      }
    } else if (b != 0.0) {
      at(-a / (3.0 * b));
    }
    o.p[s] = 1.02 * poly;
    top = (1.0 + std::ldexp(1.0, -20)) * next;
    if (!(top <= 1024.0)) fail(PC_ERR_INVALID_ARG, "coefficients of step " + std::to_string(s) + " let the matrix grow past 1024");
  }
  o.x[steps] = 1.02 * top;
  return o;
}
// The shift of A's diagonal that the steps on m x m matrices need, 0 where
// Q grows little (64 x 1024 x 16 float32: six steps on A 14.4 us, seven on the
// factor 25; 64 x 1024 x 64: 115 and 184).  `noise` follows the size of an eigenvalue of A that should be 0: the
// rounding of sums of n products (waves of n / 8 or fewer), multiplied by a^2 and
// joined by two products' rounding in every step.
double orth_shift(int m, int n, int steps, const float* coef, const OrthBounds& o) {
  const double half = std::ldexp(1.0, -53), gram = (n / 8.0 + 16.0) * half;
  double growth = 1.0, noise = gram;
  bool few = true;
  for (int s = 0; s < steps; ++s) {
    few = few && noise <= std::ldexp(1.0, -16);
    const double a = std::max(1.0, std::fabs((double)coef[3 * s])), am = o.x[s] * o.p[s];
    growth *= a;
    noise = noise * a * a + 2.0 * m * half * am * am;
  }
  return few && growth <= ORTH_GROWTH ? 0.0 : 4.0 * (gram + m * half);
}
// The power of two that scales values up to `top` into float16's upper range.
float orth_scale(double top) { return (float)std::ldexp(1.0, std::min(30, 14 - (int)std::ceil(std::log2(std::max(top, 1e-6))))); }

}  // namespace

extern "C" {

int pc_layer_norm_forward(int device, int dtype, int64_t rows, int32_t cols, const void* x, int64_t x_stride,
                          const float* weight, const float* bias, float eps, void* y, int64_t y_stride,
                          float* mean, float* rstd, void* stream) {
  return guarded([&] {
    check_device(device);
    check_dtype(dtype);
    check_norm(rows, cols);
    need(std::isfinite(eps) && eps >= 0.0f, "eps must be finite and at least 0");
    if (rows == 0) return;
    need(x && y, "null x or y");
    need(x_stride >= cols || (x_stride >= 0 && rows == 1), "x_stride below cols");
    need(y_stride >= cols || (y_stride >= 0 && rows == 1), "y_stride below cols");
    need(y != x || y_stride == x_stride || rows == 1, "y is x at another stride");
    DeviceGuard dg(device);
    NormArgs a{};
    a.rows = rows;
    a.cols = cols;
    a.x = x;
    a.x_stride = x_stride;
    a.weight = weight;
    a.bias = bias;
    a.eps = eps;
    a.y = y;
    a.y_stride = y_stride;
    a.mean = mean;
    a.rstd = rstd;
    launch_norm_fwd(a, dtype, (hipStream_t)stream);
    check_launch();
  });
}

int pc_layer_norm_workspace_bytes(int64_t rows, int32_t cols, size_t* bytes) {
  return guarded([&] {
    need(bytes, "null bytes");
    check_norm(rows, cols);
    *bytes = norm_ws(rows, cols);
  });
}

int pc_layer_norm_backward(int device, int dtype, int64_t rows, int32_t cols, const void* dy, int64_t dy_stride,
                           const void* x, int64_t x_stride, const float* weight, const float* mean, const float* rstd,
                           void* dx, int64_t dx_stride, float* dweight, float* dbias,
                           void* ws, size_t ws_bytes, void* stream) {
  return guarded([&] {
    check_device(device);
    check_dtype(dtype);
    check_norm(rows, cols);
    need(rows == 0 || (dy && x && mean && rstd && dx), "null dy, x, mean, rstd or dx");
    for (int64_t st : {dy_stride, x_stride, dx_stride}) need(st >= cols || (st >= 0 && rows <= 1), "a row stride is below cols");
    need(rows <= 1 || ((dx != dy || dx_stride == dy_stride) && (dx != x || dx_stride == x_stride)), "dx is dy or x at another stride");
    const bool params = dweight || dbias;
    if (rows == 0 && !params) return;
    if (params) check_ws(ws, ws_bytes, norm_ws(rows, cols));
    DeviceGuard dg(device);
    NormArgs a{};
    a.rows = rows;
    a.cols = cols;
    a.x = x;
    a.x_stride = x_stride;
    a.dy = dy;
    a.dy_stride = dy_stride;
    a.weight = weight;
    a.y = dx;
    a.y_stride = dx_stride;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.part = params ? (float*)ws : nullptr;
    a.dweight = dweight;
    a.dbias = dbias;
    launch_norm_bwd(a, dtype, (hipStream_t)stream);
    check_launch();
  });
}

int pc_linear_attention_workspace_bytes(const pc_linear_attention* d, int backward, size_t* bytes) {
  return guarded([&] {
    need(bytes, "null bytes");
    check_seqs(d);
    *bytes = mix_ws(d, backward != 0).total;
  });
}

int pc_linear_attention_forward(int device, const pc_linear_attention* d, void* ws, size_t ws_bytes, void* stream) {
  return guarded([&] {
    check_device(device);
    check_call(d);
    check_heads(d, d->q, "q");
    check_heads(d, d->k, "k");
    check_heads(d, d->v, "v");
    check_out(d, d->o, d->heads, d->dim_v, "o");
    const MixWs w = mix_ws(d, false);
    check_ws(ws, ws_bytes, w.total);
    if (d->num_seqs == 0) return;
    DeviceGuard dg(device);
    const hipStream_t s = (hipStream_t)stream;
    const int group = d->heads / d->kv_heads;
    MixArgs a = mix_base(d, mix_segments(d));
    a.da = d->dim_k;
    a.dc = d->dim_v;
    a.st_r = d->dim_v;
    a.st_c = 1;
    a.a = tensor(d->q, 1);
    a.b = tensor(d->k, group);
    a.c = tensor(d->v, group);
    a.out = d->o.data;
    a.o_ts = d->o.token_stride;
    a.o_hs = d->o.head_stride;
    a.off = 1;
    a.wscale = 1.0f;
    a.oscale = d->scale;
    a.init = d->state_in;
    a.fin = d->state_out;
    a.seg = (float*)((char*)ws + w.seg_f);
    mix_starts(d, &a, 1, s);
    launch_mix_walk(&a, 1, d->dtype, s);
    check_launch();
  });
}

int pc_linear_attention_backward(int device, const pc_linear_attention* d, void* ws, size_t ws_bytes, void* stream) {
  return guarded([&] {
    check_device(device);
    check_call(d);
    check_heads(d, d->q, "q");
    check_heads(d, d->k, "k");
    check_heads(d, d->v, "v");
    check_heads(d, d->d_o, "d_o");
    check_out(d, d->d_q, d->heads, d->dim_k, "d_q");
    check_out(d, d->d_k, d->kv_heads, d->dim_k, "d_k");
    check_out(d, d->d_v, d->kv_heads, d->dim_v, "d_v");
    const MixWs w = mix_ws(d, true);
    check_ws(ws, ws_bytes, w.total);
    if (d->num_seqs == 0) return;
    DeviceGuard dg(device);
    const hipStream_t s = (hipStream_t)stream;
    const int group = d->heads / d->kv_heads, dk = d->dim_k, dv = d->dim_v;
    char* base = (char*)ws;
    const MixTensor q = tensor(d->q, 1), k = tensor(d->k, group), v = tensor(d->v, group), go = tensor(d->d_o, 1);
    // the walk that makes the forward's states (used for them alone), and dq,
    // contracted with the state's columns
    MixArgs f = mix_base(d, mix_segments(d));
    f.off = 1;
    f.wscale = 1.0f;
    f.init = d->state_in;
    f.seg = (float*)(base + w.seg_f);
    MixArgs q_walk = f;
    f.da = dk;
    f.dc = dv;
    f.st_r = dv;
    f.st_c = 1;
    f.b = k;
    f.c = v;
    q_walk.da = dv;
    q_walk.dc = dk;
    q_walk.st_r = 1;
    q_walk.st_c = dv;
    q_walk.a = go;
    q_walk.b = v;
    q_walk.c = k;
    q_walk.oscale = d->scale;
    q_walk.out = d->d_q.data;
    q_walk.o_ts = d->d_q.token_stride;
    q_walk.o_hs = d->d_q.head_stride;
    // dv and dk from the adjoint states, from the sequences' ends.  The carried
    // state is the one already decayed onto the token before (off 0), so it
    // starts as the given gradient and ends as the gradient of state_in; scale
    // belongs to a token's part in it.
    MixArgs v_walk = mix_base(d, mix_segments(d));
    v_walk.rev = 1;
    v_walk.off = 0;
    v_walk.wscale = d->scale;
    v_walk.oscale = 1.0f;
    v_walk.init = d->dstate_out;
    v_walk.seg = (float*)(base + w.seg_r);
    MixArgs k_walk = v_walk;
    v_walk.da = dk;
    v_walk.dc = dv;
    v_walk.st_r = dv;
    v_walk.st_c = 1;
    v_walk.a = k;
    v_walk.b = q;
    v_walk.c = go;
    v_walk.fin = d->dstate_in;
    k_walk.da = dv;
    k_walk.dc = dk;
    k_walk.st_r = 1;
    k_walk.st_c = dv;
    k_walk.a = v;
    k_walk.b = go;
    k_walk.c = q;
    auto target = [&](MixArgs& a, const pc_heads& to, size_t part, int dim) {
      if (group == 1) {
        a.out = to.data;
        a.o_ts = to.token_stride;
        a.o_hs = to.head_stride;
      } else {
        a.out = base + part;
        a.o_ts = (int64_t)d->heads * dim;
        a.o_hs = dim;
        a.out_f32 = 1;
      }
    };
    target(k_walk, d->d_k, w.dk, dk);
    target(v_walk, d->d_v, w.dv, dv);
    const MixArgs starts[2] = {f, v_walk};
    mix_starts(d, starts, 2, s);
    // dv's walk apart where it overwrites the states that dk's walk starts from
    const MixArgs walks[3] = {q_walk, k_walk, v_walk};
    const bool apart = d->dstate_in && d->dstate_in == d->dstate_out;
    launch_mix_walk(walks, apart ? 2 : 3, d->dtype, s);
    check_launch();
    if (apart) {
      launch_mix_walk(walks + 2, 1, d->dtype, s);
      check_launch();
    }
    if (group > 1 && d->num_tokens > 0) {
      auto sum = [&](const pc_heads& to, size_t part, int dim) {
        MixSumArgs m{};
        m.tokens = d->num_tokens;
        m.seqs = d->num_seqs;
        m.kv_heads = d->kv_heads;
        m.group = group;
        m.dim = dim;
        m.cu = d->cu_seqlens;
        m.part = (const float*)(base + part);
        m.out = to.data;
        m.o_ts = to.token_stride;
        m.o_hs = to.head_stride;
        return m;
      };
      launch_mix_sum(sum(d->d_k, w.dk, dk), sum(d->d_v, w.dv, dv), d->dtype, s);
      check_launch();
    }
  });
}

int pc_linear_attention_step(int device, const pc_linear_attention* d, void* stream) {
  return guarded([&] {
    check_device(device);
    check_mix(d);
    need(d->log_decay, "null log_decay");
    need(std::isfinite(d->scale) && d->scale != 0.0f, "scale must be finite and not 0");
    check_heads(d, d->q, "q", false);
    check_heads(d, d->k, "k", false);
    check_heads(d, d->v, "v", false);
    check_out(d, d->o, d->heads, d->dim_v, "o", false);
    need(d->num_slots >= 0 && d->num_slots <= INT_MAX, "num_slots must be in [0, 2^31)");
    need(d->slots || d->num_slots >= d->num_tokens, "fewer slots than rows");
    need((int64_t)d->heads * d->num_tokens <= INT_MAX, "more than 2^31 rows times heads");
    if (d->num_tokens == 0 || d->num_slots == 0) return;
    need(d->state, "null state");
    DeviceGuard dg(device);
    MixStepArgs a{};
    a.batch = (int)d->num_tokens;
    a.heads = d->heads;
    a.group = d->heads / d->kv_heads;
    a.dk = d->dim_k;
    a.dv = d->dim_v;
    a.slots = (int)d->num_slots;
    a.q = d->q.data;
    a.k = d->k.data;
    a.v = d->v.data;
    a.q_ts = d->q.token_stride;
    a.q_hs = d->q.head_stride;
    a.k_ts = d->k.token_stride;
    a.k_hs = d->k.head_stride;
    a.v_ts = d->v.token_stride;
    a.v_hs = d->v.head_stride;
    a.log_decay = d->log_decay;
    a.scale = d->scale;
    a.state = d->state;
    a.slot = d->slots;
    a.o = d->o.data;
    a.o_ts = d->o.token_stride;
    a.o_hs = d->o.head_stride;
    launch_mix_step(a, d->dtype, (hipStream_t)stream);
    check_launch();
  });
}

int pc_attention_workspace_bytes(const pc_attention* d, int backward, size_t* bytes) {
  return guarded([&] {
    need(bytes, "null bytes");
    check_attn_sizes(d);
    *bytes = attn_ws(d, backward != 0).total;
  });
}

int pc_attention_forward(int device, const pc_attention* d, void* ws, size_t ws_bytes, void* stream) {
  return guarded([&] {
    check_device(device);
    check_attn(d);
    check_out(d, d->o, d->heads, d->dim_v, "o", false);
    const AttnWs w = attn_ws(d, false);
    if (ws) check_ws(ws, ws_bytes, w.total);
    if (d->num_seqs == 0 || d->num_tokens == 0) return;
    AttnArgs a = attn_base(d);
    if (ws) {       // (without a workspace the keys are not cut)
      const AttnSplit sp = attn_split(d, false);
      a.nsplit = sp.nsplit;
      a.part_len = sp.part_len;
      a.part = (float*)((char*)ws + w.part);
      a.stat = (float2*)((char*)ws + w.stat);
    }
    DeviceGuard dg(device);
    launch_attn_fwd(a, d->dtype, (hipStream_t)stream);
    check_launch();
    if (a.nsplit > 1) {
      launch_attn_join(a, d->dtype, (hipStream_t)stream);
      check_launch();
    }
  });
}

int pc_attention_backward(int device, const pc_attention* d, void* ws, size_t ws_bytes, void* stream) {
  return guarded([&] {
    check_device(device);
    check_attn(d);
    check_heads(d, d->o, "o", false);
    check_heads(d, d->d_o, "d_o", false);
    need(d->lse || d->num_tokens == 0, "null lse");
    check_out(d, d->d_q, d->heads, d->dim_k, "d_q", false);
    check_out(d, d->d_k, d->kv_heads, d->dim_k, "d_k", false);
    check_out(d, d->d_v, d->kv_heads, d->dim_v, "d_v", false);
    const AttnWs w = attn_ws(d, true);
    check_ws(ws, ws_bytes, w.total);
    if (d->num_seqs == 0 || d->num_tokens == 0) return;
    DeviceGuard dg(device);
    AttnArgs a = attn_base(d);
    const AttnSplit sp = attn_split(d, true);
    a.nsplit = sp.nsplit;
    a.part_len = sp.part_len;
    a.part = (float*)((char*)ws + w.part);
    a.part_k = (float*)((char*)ws + w.part_k);
    a.part_v = (float*)((char*)ws + w.part_v);
    a.out = attn_tensor(d->o);
    a.d_o = attn_tensor(d->d_o);
    a.dq = d->d_q.data;
    a.dq_ts = d->d_q.token_stride;
    a.dq_hs = d->d_q.head_stride;
    a.dk_ = d->d_k.data;
    a.dk_ts = d->d_k.token_stride;
    a.dk_hs = d->d_k.head_stride;
    a.dv_ = d->d_v.data;
    a.dv_ts = d->d_v.token_stride;
    a.dv_hs = d->d_v.head_stride;
    a.delta = (float*)((char*)ws + w.delta);
    launch_attn_bwd(a, d->dtype, (hipStream_t)stream);
    check_launch();
    if (a.nsplit > 1) {
      launch_attn_sum(a, d->dtype, (hipStream_t)stream);
      check_launch();
    }
  });
}

int pc_attention_cached_workspace_bytes(const pc_attention* d, size_t* bytes) {
  return guarded([&] {
    need(bytes, "null bytes");
    check_pages(d);
    *bytes = cached_plan(d).total;
  });
}

int pc_attention_cached(int device, const pc_attention* d, void* ws, size_t ws_bytes, void* stream) {
  return guarded([&] {
    check_device(device);
    check_pages(d);
    check_attn(d, true);
    check_out(d, d->o, d->heads, d->dim_v, "o", false);
    auto cache = [&](const pc_pages& c, int dim, const char* what) {
      need(c.data || d->num_pages == 0, std::string("null ") + what);
      need(c.page_stride >= 0 && c.token_stride >= 0 && c.head_stride >= 0, std::string("negative stride of ") + what);
      // two of the three dimensions inside the third, in any order: elements are distinct
      struct Dim {
        int64_t n, stride;
      } x[3] = {{d->num_pages, c.page_stride}, {d->page_size, c.token_stride}, {d->kv_heads, c.head_stride}};
      std::sort(x, x + 3, [](const Dim& p, const Dim& q) { return p.stride < q.stride; });
      int64_t span = dim;
      for (const Dim& y : x) {
        if (y.n <= 1) continue;
        need(y.stride >= span, std::string("elements of ") + what + " overlap");
        span += (y.n - 1) * y.stride;
      }
      return AttnCache{c.data, c.page_stride, c.token_stride, c.head_stride};
    };
    const CachedPlan p = cached_plan(d);
    AttnArgs a = attn_base(d);
    a.lse = nullptr;
    a.pages.k = cache(d->k_cache, d->dim_k, "k_cache");
    a.pages.v = cache(d->v_cache, d->dim_v, "v_cache");
    need(d->cached || d->num_seqs == 0, "null cached");
    need(d->page_table || d->max_pages == 0 || d->num_seqs == 0, "null page_table");
    need(d->page_table_stride >= d->max_pages || d->num_seqs <= 1, "page_table_stride below max_pages");
    check_ws(ws, ws_bytes, p.total);
    if (d->num_seqs == 0 || d->num_tokens == 0) return;
    a.pages.table = d->page_table;
    a.pages.table_stride = d->page_table_stride;
    a.pages.past = d->cached;
    a.pages.num_pages = d->num_pages;
    a.pages.page_size = d->page_size;
    a.pages.max_pages = d->max_pages;
    // j / page_size for j < 2^31: s = ceil(log2 page_size), ceil(2^(31 + s) / page_size) fits 32 bits
    int s = 0;
    while ((int64_t)1 << s < d->page_size) ++s;
    a.pages.shift = 31 + s;
    a.pages.magic = (uint32_t)((((uint64_t)1 << (31 + s)) + d->page_size - 1) / d->page_size);
    a.nsplit = p.nsplit;
    a.part_len = p.part_len;
    a.part = (float*)ws;
    a.stat = (float2*)((char*)ws + p.stat);
    DeviceGuard dg(device);
    launch_attn_cached(a, d->dtype, p.few, (hipStream_t)stream);
    check_launch();
    if (p.nsplit > 1) {
      launch_attn_join(a, d->dtype, (hipStream_t)stream);
      check_launch();
    }
  });
}

int pc_rotary_frequencies(int32_t rotary_dim, double base, int scaling, double factor, double original, double low, double high,
                          double* freq) {
  return guarded([&] {
    need(rotary_dim >= 0 && rotary_dim % 2 == 0, "rotary_dim must be even and at least 0");
    need(freq || rotary_dim == 0, "null freq");
    need(std::isfinite(base) && base > 0.0, "base must be finite and above 0");
    need(scaling >= PC_ROTARY_PLAIN && scaling <= PC_ROTARY_PARTS, "unknown scaling");
    need(scaling == PC_ROTARY_PLAIN || (std::isfinite(factor) && factor > 0.0), "factor must be finite and above 0");
    if (scaling == PC_ROTARY_PARTS)
      need(std::isfinite(original) && original > 0.0 && std::isfinite(low) && std::isfinite(high) && low < high,
           "original must be above 0 and low below high");
    if (scaling == PC_ROTARY_BASE) {
      need(rotary_dim != 2, "scaling of the base needs two pairs");
      base *= std::pow(factor, (double)rotary_dim / std::max(1, rotary_dim - 2));
    }
    for (int i = 0; i < rotary_dim / 2; ++i) {
      double f = std::pow(base, -2.0 * i / rotary_dim);
      if (scaling == PC_ROTARY_LINEAR) f /= factor;
      if (scaling == PC_ROTARY_PARTS) {
        const double turns = original * f / 6.283185307179586477, keep = std::min(1.0, std::max(0.0, (turns - low) / (high - low)));
        f *= keep + (1.0 - keep) / factor;
      }
      freq[i] = f;
    }
  });
}

int pc_rotary_workspace_bytes(const pc_rotary* d, size_t* bytes) {
  return guarded([&] {
    need(bytes, "null bytes");
    check_rotary(d);
    *bytes = (size_t)rotary_parts(d->num_tokens) * 2 * d->dim * sizeof(float);
  });
}

int pc_rotary_forward(int device, const pc_rotary* d, void* stream) {
  return guarded([&] {
    check_device(device);
    RotaryArgs a = rotary_base(d);
    auto side = [&](const pc_heads& y, const pc_heads& x, int heads, const char* n0, const char* n1) {
      if (!heads) return;
      check_heads(d, x, n1, false);
      check_out(d, y, heads, d->dim, n0, false);
      check_place(d, y, x, heads, n0);
    };
    side(d->q_out, d->q, d->heads, "q_out", "q");
    side(d->k_out, d->k, d->kv_heads, "k_out", "k");
    if (d->num_tokens == 0 || d->heads + d->kv_heads == 0) return;
    a.q = attn_tensor(d->q);
    a.k = attn_tensor(d->k);
    a.qo = d->q_out.data;
    a.qo_ts = d->q_out.token_stride;
    a.qo_hs = d->q_out.head_stride;
    a.ko = d->k_out.data;
    a.ko_ts = d->k_out.token_stride;
    a.ko_hs = d->k_out.head_stride;
    DeviceGuard dg(device);
    launch_rotary_fwd(a, d->dtype, (hipStream_t)stream);
    check_launch();
  });
}

int pc_rotary_backward(int device, const pc_rotary* d, void* ws, size_t ws_bytes, void* stream) {
  return guarded([&] {
    check_device(device);
    RotaryArgs a = rotary_base(d);
    auto side = [&](const pc_heads& dy, const pc_heads& dx, const pc_heads& x, int heads, const char* n0, const char* n1, const char* n2) {
      if (!heads) return;
      check_heads(d, dy, n0, false);
      check_out(d, dx, heads, d->dim, n1, false);
      check_place(d, dx, dy, heads, n1);
      if (!d->norm) return;
      check_heads(d, x, n2, false);
      check_place(d, dx, x, heads, n1);
    };
    side(d->d_q_out, d->d_q, d->q, d->heads, "d_q_out", "d_q", "q");
    side(d->d_k_out, d->d_k, d->k, d->kv_heads, "d_k_out", "d_k", "k");
    const bool weights = d->norm && (d->d_q_weight || d->d_k_weight);
    a.parts = rotary_parts(d->num_tokens);
    if (weights) check_ws(ws, ws_bytes, (size_t)a.parts * 2 * d->dim * sizeof(float));
    if ((d->num_tokens == 0 || d->heads + d->kv_heads == 0) && !weights) return;
    a.q = attn_tensor(d->q);
    a.k = attn_tensor(d->k);
    a.dq = attn_tensor(d->d_q_out);
    a.dk = attn_tensor(d->d_k_out);
    a.qo = d->d_q.data;
    a.qo_ts = d->d_q.token_stride;
    a.qo_hs = d->d_q.head_stride;
    a.ko = d->d_k.data;
    a.ko_ts = d->d_k.token_stride;
    a.ko_hs = d->d_k.head_stride;
    a.dqw = d->d_q_weight;
    a.dkw = d->d_k_weight;
    a.part_sums = weights ? (float*)ws : nullptr;
    DeviceGuard dg(device);
    launch_rotary_bwd(a, d->dtype, (hipStream_t)stream);
    check_launch();
  });
}

int pc_orthogonalize_workspace_bytes(int dtype, int64_t batch, int32_t rows, int32_t cols, size_t* bytes) {
  return guarded([&] {
    need(bytes, "null bytes");
    check_orth(dtype, batch, rows, cols);
    *bytes = orth_plan(batch, rows, cols, nullptr).total;
  });
}

int pc_orthogonalize(int device, int dtype, int64_t batch, int32_t rows, int32_t cols, const void* g, int64_t g_batch,
                     int64_t g_row, void* out, int64_t out_batch, int64_t out_row, int32_t steps,
                     const float* coefficients, float eps, void* ws, size_t ws_bytes, void* stream) {
  return guarded([&] {
    check_device(device);
    check_orth(dtype, batch, rows, cols);
    need(steps >= 1 && steps <= ORTH_MAX_STEPS, "steps must be in [1, " + std::to_string(ORTH_MAX_STEPS) + "]");
    need(coefficients, "null coefficients");
    need(std::isfinite(eps) && eps >= 0.0f, "eps must be finite and at least 0");
    OrthPoly poly{};
    poly.steps = steps;
    for (int k = 0; k < 3 * steps; ++k) {
      need(std::isfinite(coefficients[k]), "a coefficient is not finite");
      poly.c[k / 3][k % 3] = coefficients[k];
    }
    const OrthBounds bound = orth_bounds(steps, coefficients);
    need(batch == 0 || (g && out), "null matrices");
    need(g_row >= cols || (g_row >= 0 && rows == 1), "g_row below cols");
    need(out_row >= cols || (out_row >= 0 && rows == 1), "out_row below cols");
    const int64_t span = (rows - 1) * out_row + cols;
    need(g_batch >= 0, "g_batch is negative");
    need(batch <= 1 || out_batch >= span || (out_batch >= cols && out_row >= (batch - 1) * out_batch + cols),
         "the matrices of out overlap");
    need(out != g || batch == 0 || ((rows == 1 || out_row == g_row) && (batch == 1 || out_batch == g_batch)),
         "out is g at other strides");
    OrthPlan p = orth_plan(batch, rows, cols, ws);
    check_ws(ws, ws_bytes, p.total);
    if (batch == 0) return;
    DeviceGuard dg(device);
    const hipStream_t s = (hipStream_t)stream;
    OrthIo io{};
    io.batch = batch;
    io.m = p.m;
    io.n = p.n;
    io.tall = rows > cols;
    io.g = g;
    io.g_batch = g_batch;
    io.g_row = g_row;
    io.out = out;
    io.o_batch = out_batch;
    io.o_row = out_row;
    io.eps = eps;
    if (p.small) {
      poly.shift = orth_shift(p.m, p.n, steps, coefficients, bound);
      launch_orth_small(io, poly, dtype, s);
      check_launch();
      return;
    }
    double* part = (double*)((char*)ws + p.part);
    launch_orth_norm(io, dtype, part, s);
    check_launch();
    float sx = orth_scale(bound.x[0]);
    launch_orth_split(io, dtype, part, sx, p.mp, p.np, p.x[0], p.xt[0], s);
    check_launch();
    for (int k = 0; k < steps; ++k) {
      const float *c = coefficients + 3 * k;
      const OrthMat &x = p.x[k & 1], &xt = p.xt[k & 1];
      const float sa = orth_scale(bound.x[k] * bound.x[k]), sb = orth_scale(bound.p[k]);
      const float sn = k + 1 < steps ? orth_scale(bound.x[k + 1]) : 1.0f;
      OrthGemmArgs a{};
      a.io = io;
      a.parts = p.split ? (float*)((char*)ws + p.parts) : nullptr;
      // A = X X^T
      a.M = a.N = p.mp;
      a.K = p.np;
      a.a = a.b = x;
      a.c = p.a;
      a.sacc = sa / (sx * sx);
      launch_orth_gemm(a, ORTH_GRAM, dtype, s);
      check_launch();
      // B = a I + b A + c A^2, then X <- B X
      a.K = p.mp;
      a.a = a.b = a.old = p.a;
      a.c = p.b;
      a.sacc = sb * c[2] / (sa * sa);
      a.sold = sb * c[1] / sa;
      a.diag = sb * c[0];
      launch_orth_gemm(a, ORTH_POLY, dtype, s);
      check_launch();
      a.N = p.np;
      a.a = p.b;
      a.b = xt;
      a.c = p.x[(k + 1) & 1];
      a.ct = p.xt[(k + 1) & 1];
      a.sacc = sn / (sb * sx);
      launch_orth_gemm(a, k + 1 < steps ? ORTH_APPLY : ORTH_OUT, dtype, s);
      check_launch();
      sx = sn;
    }
  });
}

}  // extern "C"
