// k_attn_fwd.hip -- causal softmax attention over whole packed sequences.
//
//   o_i = sum_{j <= i} p_ij v_j / sum_{j <= i} p_ij,   p_ij = exp(scale q_i . k_j - m_i),   lse_i = m_i + log sum p_ij
//
// one pass over the keys with a running maximum and sum; see k_attn_core.h for the loop.  Few long sequences are cut
// along the keys; attn_join (k_attn_cached.hip) joins the parts.
//
// What bounds it: matrix instructions.  Of 16-bit tensors a tile takes the scores and a product for each plane of the
// weights (bfloat16 4 products' work in all, float16 3): 16384 tokens x 16 heads x 128 bfloat16 in 1.83 ms are 1.20 PFLOP/s of
// them (a large library product: 1.39); float32, 6 for each, 8 x 2048 x 16 heads x 128 in 0.90 ms, 0.92 PFLOP/s; 24 ragged
// sequences of up to 1500 x 16 heads x 64 float16 74 us.
#include <algorithm>

#include "k_attn_core.h"

namespace pc {
namespace {

template <typename T, int D, FitMode MODE>
__global__ __launch_bounds__(256, 2) void attn_fwd(AttnArgs a, int64_t slots) {
  __shared__ typename FwdShape<T, D>::Lds lds;
  const int heads = a.kv_heads * a.group;
  for (int64_t b = blockIdx.x; b < slots * a.nsplit * a.kv_heads; b += gridDim.x) {
    const auto [kvh, split, slot] = block_of(b, a.kv_heads, slots);
    // the last tiles, which have the most keys, first
    const SeqTile at = find_tile(a.cu, a.seqs, a.tokens, a.group, ATTN_ROWS, slots - 1 - slot);
    const int64_t first = at.tile * ATTN_ROWS, rows_all = at.len * a.group;
    if (at.seq < 0 || first >= rows_all) continue;
    const int64_t tf = first / a.group, t = at.t0 + tf;
    Rows<T> rows;
    rows.q = (const T*)a.q.p + t * a.q.ts + (int64_t)kvh * a.group * a.q.hs;
    rows.q_ts = a.q.ts;
    rows.q_hs = a.q.hs;
    rows.group = a.group;
    rows.rem = (int)(first - tf * a.group);
    rows.count = (int)min((int64_t)ATTN_ROWS, rows_all - first);
    rows.first = (int)tf;
    Keys<T, false> keys{};
    keys.k = (const T*)a.k.p + at.t0 * a.k.ts + kvh * a.k.hs;
    keys.v = (const T*)a.v.p + at.t0 * a.v.ts + kvh * a.v.hs;
    keys.k_ts = a.k.ts;
    keys.v_ts = a.v.ts;
    keys.total = (int)at.len;
    RowOut out{};
    out.o = (T*)a.o + t * a.o_ts + (int64_t)kvh * a.group * a.o_hs;
    out.o_ts = a.o_ts;
    out.o_hs = a.o_hs;
    out.heads = heads;
    out.lse = a.lse ? a.lse + t * heads + kvh * a.group : nullptr;
    const int end = rows.last(rows.count - 1) + 1;
    int key0 = 0, key1 = end;
    if (a.nsplit > 1) {
      const int64_t place = ((int64_t)split * a.tokens + t) * heads + kvh * a.group;
      out.part = a.part + place * a.dv;
      out.stat = a.stat + place;
      key0 = (int)min((int64_t)split * a.part_len, (int64_t)end);
      if (split + 1 < a.nsplit) key1 = (int)min((int64_t)(split + 1) * a.part_len, (int64_t)end);
    }
    if (key0 >= key1) no_keys(rows, out);
    else
      attend_tile<T, D, MODE, false>(lds, keys, rows, out, a.dk, a.dv, fabsf(a.scale) * LOG2E, a.scale < 0.0f, key0, key1);
  }
}

template <typename T>
void fwd(const AttnArgs& a, hipStream_t s) {
  const int64_t slots = a.tokens * a.group / ATTN_ROWS + a.seqs;
  const dim3 grid((uint32_t)std::min<int64_t>(slots * a.nsplit * a.kv_heads, 1 << 23));
  by_fit(fit_of<T>(a, false), [&](auto d, auto mode) {
    launch_kernel(attn_fwd<T, decltype(d)::value, decltype(mode)::value>, grid, dim3(256), 0, s, a, slots);
  });
}

}  // namespace

void launch_attn_fwd(const AttnArgs& a, int dtype, hipStream_t s) {
  if (dtype == PC_DTYPE_BF16) fwd<bf16>(a, s);
  else if (dtype == PC_DTYPE_F16) fwd<f16>(a, s);
  else fwd<float>(a, s);
}

}  // namespace pc
