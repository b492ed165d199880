// Attention over a paged cache: what its kernels share - the arguments, how the key tiles
// of all sequences are dealt out to the CTAs, and the partial results.
//
// Work. Sequence b's positions [first_b, len_b) that a row can see (first_b rounded down) are n_b tiles of TK keys. A unit is
// one (sequence, kv head, chunk of at most QN queries); a sequence has U = n_kv_heads x
// chunks of them. All units' tiles laid end to end (T in all) are dealt to the G CTAs in
// equal contiguous ranges (G at most T), CTA c taking tiles [c T / G, (c + 1) T / G): every CTA streams
// the same number of tiles whatever the lengths, which only the device knows, and the grid
// is fixed, so a call can be captured. A CTA's part of one unit is a piece. A piece that is
// a whole unit writes its output rows; any other leaves (max, sum, O) in the workspace, in
// slot 0 of its CTA if an earlier CTA began the unit, else in slot 1 (the unit is then the
// CTA's last), and the merge kernel joins a unit's pieces in order.
#pragma once

#include "paged.cuh"

namespace dmtp {

struct PagedAttn {
  PageMap m;
  const void *k, *v;
  const float *ks, *vs;
  dmtp_paged_query a;
  unsigned* err;
  int group, nq, qn, chunks, units;  // queries per kv head; of a unit; units of a sequence
  float* part_o;                     // [G][2][qn][head_dim]
  float2* part_ml;                   // [G][2][qn] (max in base 2, sum)
  int* prefix;                       // [n_seqs + 1] tiles before sequence b
  float scale2;                      // scale log2(e)
};

// Length of sequence b inside the table's reach.
__device__ __forceinline__ int seq_len(const PagedAttn& p, int b) {
  const int n = __ldg(p.a.kv_len + b);
  return n < 0 ? 0 : n > p.m.reach ? p.m.reach : n;
}
// First position of sequence b's tiles: that any row sees, down to a whole 64.
__device__ __forceinline__ int seq_first(const PagedAttn& p, int len) {
  if (p.a.window <= 0) return 0;
  const int f = len - p.a.rows + 1 - p.a.window;
  return f > 0 ? f & ~63 : 0;
}
template <int TK>
__device__ __forceinline__ int seq_tiles(const PagedAttn& p, int len) {
  return (len - seq_first(p, len) + TK - 1) / TK;
}

// CTAs that take tiles: with fewer tiles than CTAs, as many as there are tiles, so that
// every one of them has a piece of each unit it lies in.
__device__ __forceinline__ int busy_ctas(long long total, int G) {
  return total < G ? (int)total : G;
}

struct Walk {
  long long total;  // T
  int pos, end;     // this CTA's tiles
  int b, base;      // the sequence of tile pos, tiles before it
};

// This CTA's range and where it starts, by all THREADS threads of the CTA. `sh`: THREADS / 32
// + 4 ints of shared memory. CTA 0 also leaves the prefix sums for the merge kernel.
template <int TK, int THREADS>
__device__ __forceinline__ Walk deal(const PagedAttn& p, int* sh) {
  constexpr int W = THREADS / 32;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, n = p.m.n_seqs;
  Walk w;
  int sum = 0;
  for (int b = threadIdx.x; b < n; b += THREADS) sum += seq_tiles<TK>(p, seq_len(p, b));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) sh[wid] = sum;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) total += sh[i];
  w.total = (long long)total * p.units;
  const int G = busy_ctas(w.total, gridDim.x), c = min((int)blockIdx.x, G);
  w.pos = G ? (int)(w.total * c / G) : 0;
  w.end = G ? (int)(w.total * min(c + 1, G) / G) : 0;
  w.b = 0;
  w.base = 0;
  int before = 0;  // tiles of one unit before this round of sequences
  for (int b0 = 0; b0 < n; b0 += THREADS) {
    const int b = b0 + threadIdx.x;
    const int len = b < n ? seq_len(p, b) : 0;
    if (blockIdx.x == 0 && b < n && __ldg(p.a.kv_len + b) > p.m.reach) set_err(p.err, DMTP_OPS_ERR_POS);
    const int t = b < n ? seq_tiles<TK>(p, len) : 0;
    int inc = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    __syncthreads();  // sh of the total (or the last round) has been read
    if (lane == 31) sh[wid] = inc;
    __syncthreads();
    int off = before, all = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if (i < wid) off += sh[i];
      all += sh[i];
    }
    const int lo = (off + inc - t) * p.units, hi = (off + inc) * p.units;
    if (blockIdx.x == 0 && b < n) {
      p.prefix[b] = lo;
      if (b == n - 1) p.prefix[n] = hi;
    }
    if (t > 0 && w.pos >= lo && w.pos < hi) {
      sh[W] = b;
      sh[W + 1] = lo;
    }
    before += all;
  }
  __syncthreads();
  if (w.pos < w.end) {
    w.b = sh[W];
    w.base = sh[W + 1];
  }
  return w;
}

// Output row of query t of a unit: query head and row.
__device__ __forceinline__ void query_of(const PagedAttn& p, int unit, int t, int* head, int* row) {
  const int kvh = unit / p.chunks, qi = (unit - kvh * p.chunks) * p.qn + t;
  *row = qi / p.group;
  *head = kvh * p.group + (qi - *row * p.group);
}
__device__ __forceinline__ int queries_of(const PagedAttn& p, int unit) {
  const int left = p.nq - (unit % p.chunks) * p.qn;
  return left < p.qn ? left : p.qn;
}

// Which kernel takes a call: the tensor cores (paged_attn_tc.cu) or the CUDA cores
// (paged_attn_simt.cu), with tiles of 64 or 128 keys.
struct PagedPlan {
  bool tc;
  int qn, chunks, grid;
  size_t part_o, part_ml, prefix, bytes;  // workspace offsets
};
cudaError_t paged_attn_tc(const PagedAttn& p, const PagedPlan& pl, bool e8, cudaStream_t st);
cudaError_t paged_attn_simt(const PagedAttn& p, const PagedPlan& pl, int dtype, bool e8, cudaStream_t st);
int paged_tc_grid(int head_dim, bool e8, int qn);
int paged_simt_grid(int head_dim, int dtype, bool e8);

}  // namespace dmtp
