// Attention over a paged cache: what its kernels share - the arguments, how the key tiles
// of all sequences are dealt out to the CTAs, and the partial results.
//
// Work. Sequence b's positions [first_b, len_b) that a row can see (first_b rounded down) are
// n_b tiles of 64 keys. A unit is one (sequence, kv head, chunk of at most QN queries); a
// sequence has U = n_kv_heads x chunks of them.
//
// Whole units (short tables, see kWholeReach): CTA c takes unit c, and
// one launch is all; nothing about the lengths has to be known before.
//
// Split units: all units' tiles laid end to end (T in all) are dealt to the G CTAs (G at most
// T) in contiguous ranges of T / G tiles, the first T % G of them one more: every CTA streams
// the same number of tiles whatever the lengths, which only the device knows, and the grid is
// fixed, so a call can be captured. A CTA's part of one unit is a piece. A piece that is a whole
// unit writes its output rows; any other leaves (max, sum, O) in the workspace, in slot 0 of its
// CTA if an earlier CTA began the unit, else in slot 1 (the unit is then the CTA's last). The CTA
// that begins a unit notes which CTAs have its pieces, and the merge kernel joins them in order.
// Sequences without a tile get their zeros from CTA b % G.
#pragma once

#include "paged.cuh"

namespace dmtp {

// Units are not split when the table reaches no further than kWholeReach positions, or, with
// kWholeUnits units to keep the SMs busy, kWholeReachMany. Measured in a captured graph (us,
// split / whole; 4 kv heads of 128, 32 query heads, bf16): one sequence of 256 positions
// 7.8 / 6.8, of 512 7.9 / 9.7, of 1024 8.1 / 14.8; 32 sequences (128 units) of 512 15.1 / 11.6,
// of 1024 19.3 / 19.1, of 2048 28.6 / 33.7.
constexpr int kWholeReach = 256, kWholeReachMany = 1024, kWholeUnits = 64;

struct PagedNote {
  int first, last;  // the CTAs of a unit's pieces; last < 0: nothing to join
};

struct PagedAttn {
  PageMap m;
  const void *k, *v;
  const float *ks, *vs;
  dmtp_paged_query a;
  unsigned* err;
  int group, nq, qn, chunks, units;  // queries per kv head; of a unit; units of a sequence
  float* part_o;                     // [G][2][qn][head_dim]
  float2* part_ml;                   // [G][2][qn] (max in base 2, sum)
  PagedNote* note;                   // [n_seqs units]; null: whole units
  float scale2;                      // scale log2(e)
};

// Length of sequence b inside the table's reach.
__device__ __forceinline__ int seq_len(const PagedAttn& p, int b) {
  const int n = __ldg(p.a.kv_len + b);
  return n < 0 ? 0 : n > p.m.reach ? p.m.reach : n;
}
// First position that any row of a sequence sees. The pages before it are not looked up: with a
// window a user may have taken them back.
__device__ __forceinline__ int seq_low(const PagedAttn& p, int len) {
  return p.a.window <= 0 ? 0 : max(0, len - p.a.rows + 1 - p.a.window);
}
// First position of its tiles: that, down to a whole 64.
__device__ __forceinline__ int seq_first(const PagedAttn& p, int len) { return seq_low(p, len) & ~63; }
__device__ __forceinline__ int seq_tiles(const PagedAttn& p, int len) {
  return (len - seq_first(p, len) + 63) / 64;
}

// The tiles of a CTA in order: [pos, end) of all, pos lying in tile t of a unit of sequence b.
struct Tiles {
  int pos, end, b, unit, t, n, len, first;
  __device__ __forceinline__ void seq(const PagedAttn& p) {
    len = seq_len(p, b);
    first = seq_first(p, len);
    n = (len - first + 63) / 64;
  }
  __device__ __forceinline__ void skip(const PagedAttn& p, int tiles) {  // to the next unit at most
    pos += tiles;
    t += tiles;
    if (t == n && pos < end) {
      t = 0;
      if (++unit == p.units) {
        unit = 0;
        do {
          ++b;
          seq(p);
        } while (n == 0);
      }
    }
  }
};
struct Deal {
  int each, more;  // tiles of a CTA, and how many CTAs have one more
  __device__ __forceinline__ int begin(int c) const { return c * each + min(c, more); }
  __device__ __forceinline__ int owner(int tile) const {
    const int big = more * (each + 1);
    return tile < big ? tile / (each + 1) : more + (tile - big) / each;
  }
};

// This CTA's tiles. Every warp finds them for itself. Also zeros the output of sequences that
// have none, and reports lengths past the table's reach. All threads call it.
template <typename T>
__device__ __forceinline__ Tiles my_tiles(const PagedAttn& p, Deal& d, int threads) {
  const int lane = threadIdx.x & 31, n = p.m.n_seqs, G = gridDim.x, c = blockIdx.x;
  Tiles w;
  d.each = 1;
  d.more = 0;
  int zero_b, zero_step;  // sequences to look at
  if (!p.note) {
    w.b = c / p.units;
    w.unit = c - w.b * p.units;
    w.t = 0;
    w.seq(p);
    w.pos = 0;
    w.end = w.n;
    zero_b = w.unit == 0 ? w.b : n;
    zero_step = n;
  } else {
    int total = 0;
    for (int b = lane; b < n; b += 32) total += seq_tiles(p, seq_len(p, b));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    total *= p.units;
    const int busy = min(total, G);
    d.each = busy ? total / busy : 1;
    d.more = busy ? total - d.each * busy : 0;
    w.pos = c < busy ? d.begin(c) : 0;
    w.end = c < busy ? d.begin(c + 1) : 0;
    w.b = w.unit = w.t = w.n = w.len = w.first = 0;
    if (w.pos < w.end) {
      int before = 0;  // tiles of the sequences before these 32
      for (int b0 = 0; b0 < n; b0 += 32) {
        const int t = b0 + lane < n ? seq_tiles(p, seq_len(p, b0 + lane)) * p.units : 0;
        int inc = t;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += v;
        }
        const unsigned past = __ballot_sync(0xffffffffu, before + inc > w.pos);
        if (past) {
          const int l = __ffs(past) - 1;
          w.b = b0 + l;
          const int in = w.pos - (before + __shfl_sync(0xffffffffu, inc - t, l));
          w.seq(p);
          w.unit = in / w.n;
          w.t = in - w.unit * w.n;
          break;
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
      }
    }
    zero_b = c;
    zero_step = G;
  }
  for (int b = zero_b; b < n; b += zero_step) {
    const int raw = __ldg(p.a.kv_len + b);
    if (raw > p.m.reach && threadIdx.x == 0) set_err(p.err, DMTP_OPS_ERR_POS);
    if (raw > 0) continue;
    const int hd = p.m.head_dim;
    if (p.note)
      for (int i = threadIdx.x; i < p.units; i += threads) p.note[b * p.units + i] = PagedNote{0, -1};
    for (int i = threadIdx.x; i < p.a.rows * p.a.n_heads * hd; i += threads) {
      const int rh = i / hd, row = rh / p.a.n_heads;
      ((T*)p.a.out)[(int64_t)b * p.a.o_seq + (int64_t)row * p.a.o_row +
                    (int64_t)(rh - row * p.a.n_heads) * p.a.o_head + (i - rh * hd)] = from_f32<T>(0.f);
    }
  }
  return w;
}
// The note of the unit that begins at w, by one thread of the CTA that begins it.
__device__ __forceinline__ void leave_note(const PagedAttn& p, const Deal& d, const Tiles& w) {
  if (!p.note) return;
  const int last = d.owner(w.pos + w.n - 1), first = blockIdx.x;
  p.note[w.b * p.units + w.unit] = PagedNote{first, last == first ? -1 : last};
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
// (paged_attn_simt.cu), with tiles of 64 keys.
struct PagedPlan {
  bool tc, whole;
  int qn, chunks, grid;
  size_t part_o, part_ml, note, bytes;  // workspace offsets
};
cudaError_t paged_attn_tc(const PagedAttn& p, const PagedPlan& pl, bool e8, cudaStream_t st);
cudaError_t paged_attn_simt(const PagedAttn& p, const PagedPlan& pl, int dtype, bool e8, cudaStream_t st);
int paged_tc_grid(int head_dim, bool e8, int qn);
int paged_simt_grid(int head_dim);

}  // namespace dmtp
