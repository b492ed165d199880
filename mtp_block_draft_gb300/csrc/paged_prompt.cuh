// Attention of many rows over a paged cache: what its kernels share.
//
// Work. The queries of one kv head of a sequence (rows x query heads of the group, a row's heads
// side by side) are cut into tiles; a tile and a kv head are a unit. A tile's rows see an interval
// of positions each, so its keys are those from the smallest `lo` to the largest `hi`, and a block
// of keys that lies between the largest `lo` and the smallest `hi` needs no mask. The sequences'
// row counts are only known on the device: the grid has room for n_rows group / tile + n_seqs tiles,
// and a CTA finds its own in the row starts. Tiles are taken from the last to the first: of a
// sequence's rows the later ones see more. When the units are too few for the GPU, a unit's keys
// are split into `splits` ranges of the same number of blocks, whose (max, sum, O) a second
// kernel joins in order.
#pragma once

#include "paged.cuh"

namespace dmtp {

struct PagedPrompt {
  PageMap m;
  const void *k, *v;
  const float *ks, *vs;
  dmtp_paged_prompt a;
  unsigned* err;
  int group, tile, splits;
  int box;              // rows of a TMA box (0: rows are copied one by one)
  float scale2;         // scale log2(e)
  float capl, cap_inv;  // cap log2(e) (0: scores are not capped), and 1 / that
  float* part_o;        // [units][splits][tile][head_dim]
  float2* part_ml;      // [units][splits][tile] (max in base 2, sum)
};

struct PromptPlan {
  bool tc;
  int tile, tiles, splits;  // queries of a tile; tiles at most
  size_t part_o, part_ml, bytes;
};
cudaError_t paged_prompt_tc(const PagedPrompt& p, const PromptPlan& pl, Rows f, bool mod, cudaStream_t st);
cudaError_t paged_prompt_tc_scaled(const PagedPrompt& p, const PromptPlan& pl, Rows f, bool mod, cudaStream_t st);
cudaError_t paged_prompt_simt(const PagedPrompt& p, const PromptPlan& pl, int dtype, Rows f, cudaStream_t st);

// A tile: `count` queries from query q0 on of sequence b, whose rows are row0 .. row0 + n - 1 of the
// call and its last `n` of len positions.
struct PromptTile {
  int b, row0, n, len, q0, count;
};
__device__ __forceinline__ int2 prompt_rows(const PagedPrompt& p, int s) {  // first row, number of rows
  const int a = min(max(__ldg(p.a.row_start + s), 0), p.a.n_rows);
  return make_int2(a, min(max(__ldg(p.a.row_start + s + 1), a), p.a.n_rows) - a);
}
// Tile `t` of all from the end; false: there is none. Every warp finds it for itself; all lanes call.
__device__ __forceinline__ bool prompt_tile(const PagedPrompt& p, int t, PromptTile& w) {
  const int lane = threadIdx.x & 31, S = p.m.n_seqs;
  int before = 0;  // tiles of the sequences after these 32
  for (int s1 = S; s1 > 0; s1 -= 32) {
    const int s = s1 - 1 - lane;
    int2 rows = make_int2(0, 0);
    if (s >= 0) rows = prompt_rows(p, s);
    const int nq = rows.y * p.group, tiles = (nq + p.tile - 1) / p.tile;
    int inc = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    const unsigned past = __ballot_sync(0xffffffffu, before + inc > t);
    if (past) {
      const int l = __ffs(past) - 1;
      const int in = t - (before + __shfl_sync(0xffffffffu, inc - tiles, l));
      w.b = s1 - 1 - l;
      w.row0 = __shfl_sync(0xffffffffu, rows.x, l);
      w.n = __shfl_sync(0xffffffffu, rows.y, l);
      const int n = __ldg(p.a.kv_len + w.b), all = w.n * p.group;
      w.len = n < 0 ? 0 : n > p.m.reach ? p.m.reach : n;
      w.q0 = ((all + p.tile - 1) / p.tile - 1 - in) * p.tile;
      w.count = min(p.tile, all - w.q0);
      return true;
    }
    before += __shfl_sync(0xffffffffu, inc, 31);
  }
  return false;
}
// What only the device sees of the arguments, reported by one warp of the grid.
__device__ __forceinline__ void prompt_report(const PagedPrompt& p) {
  for (int s = threadIdx.x; s < p.m.n_seqs; s += 32) {
    const int a = __ldg(p.a.row_start + s), b = __ldg(p.a.row_start + s + 1);
    if (a < 0 || b < a || b > p.a.n_rows) set_err(p.err, DMTP_OPS_ERR_ROWS);
    if (__ldg(p.a.kv_len + s) > p.m.reach) set_err(p.err, DMTP_OPS_ERR_POS);
  }
}
// Positions [lo, hi) that query t of a tile sees (empty: lo >= hi), its row's own, and its head in
// the group.
struct PromptQuery {
  int lo, hi, pos, row, head;
};
__device__ __forceinline__ PromptQuery prompt_query(const PagedPrompt& p, const PromptTile& w, int t) {
  PromptQuery q;
  const int i = (w.q0 + t) / p.group;
  q.head = w.q0 + t - i * p.group;
  q.row = w.row0 + i;
  q.pos = w.len - w.n + i;
  q.lo = p.a.first ? max(__ldg(p.a.first + q.row), 0) : 0;
  if (p.a.window > 0 && q.pos >= p.a.window) q.lo = max(q.lo, q.pos - p.a.window + 1);
  q.hi = min(p.a.end ? __ldg(p.a.end + q.row) : q.pos + 1, w.len);
  return q;
}

// Eight columns of a cached row as fp32: of row `line` of a page, times s (rows with scales).
template <typename T, Rows F>
__device__ __forceinline__ void load8(const PagedPrompt& p, const void* base, int64_t page, int64_t line, int c, float s,
                                      float (&f)[8]) {
  const int hd = p.m.head_dim;
  if constexpr (F == kRaw) {
    Raw<T> r;
    const T* src = (const T*)base + page * p.m.page_stride + line * hd + c;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) r.u[i] = __ldg(reinterpret_cast<const uint4*>(src) + i);
    values(r, f);
  } else if constexpr (F == kE4M3) {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>((const uint8_t*)base + page * p.m.page_stride + line * hd + c));
    const float4 a = e4m3x4_to_f4(u.x), b = e4m3x4_to_f4(u.y);
    f[0] = a.x * s, f[1] = a.y * s, f[2] = a.z * s, f[3] = a.w * s;
    f[4] = b.x * s, f[5] = b.y * s, f[6] = b.z * s, f[7] = b.w * s;
  } else {
    const uint8_t* pg = (const uint8_t*)base + page * p.m.page_stride;
    e2m1x8_to_f8(__ldg(reinterpret_cast<const uint32_t*>(pg + line * (hd / 2) + c / 2)), f);
    const float b = h2_to_f2(e4m3x2_to_h2(__ldg(pg + e2m1_blocks(p.m) + line * (hd / 16) + c / 16))).x;
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = f[e] * b * s;
  }
}

}  // namespace dmtp
