// dmtp_paged_attention: argument checks, the plan (which kernel, how many CTAs, the
// workspace) and the merge of split units.
#include "paged_attn.cuh"

using namespace dmtp;

namespace {

// The merge of split units (paged_attn.cuh): with M the largest of the pieces' maxima,
// out = sum_c 2^(m_c - M) O_c / sum_c 2^(m_c - M) l_c. A CTA of 16 warps takes a unit's queries
// PER at a time: each with 16 / PER warps that take turns on the pieces, whose sums are then added
// in order. It is all latency (the pieces lie in L2), so a warp asks for its first pieces' rows
// together with their maxima; its launch overlaps the end of the kernel before it. On its own it
// takes 6.6 us for 128 units of 8 queries in about 4 pieces each, 12 us for 64 queries.
template <typename T, int PER>
__global__ void __launch_bounds__(512) k_paged_merge(const PagedAttn p, int units) {
  constexpr int WQ = 16 / PER, AHEAD = 4;
  __shared__ __align__(16) float part[16][DMTP_OPS_MAX_HEAD_DIM];
  pdl_wait();
  const int hd = p.m.head_dim, lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int turn = wid % WQ, t = blockIdx.y * PER + wid / WQ;
  for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const PagedNote note = p.note[unit];
    if (note.last < 0) continue;
    const int b = unit / p.units, u = unit - b * p.units;
    const int c0 = note.first, c1 = note.last;
    const bool live = t < queries_of(p, u);
    float M = -INFINITY, L = 0.f;
    auto at = [&](int c) { return (c * 2 + (c == c0)) * p.qn + t; };
    for (int d0 = 0; d0 < hd; d0 += 128) {
      const int d = d0 + 4 * lane;
      float4 ahead[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int c = c0 + turn + i * WQ;
        ahead[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (live && c <= c1 && d < hd) ahead[i] = *reinterpret_cast<const float4*>(p.part_o + (int64_t)at(c) * hd + d);
      }
      if (d0 == 0 && live) {
#pragma unroll 2
        for (int c = c0 + lane; c <= c1; c += 32) {
          const float2 ml = p.part_ml[at(c)];
          const float n = fmaxf(M, ml.x), ref = n == -INFINITY ? 0.f : n;
          L = L * ex2(M - ref) + ml.y * ex2(ml.x - ref);
          M = n;
        }
        const float n = warp_max(M), ref = n == -INFINITY ? 0.f : n;
        L = warp_sum(L * ex2(M - ref));
        M = ref;
      }
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      auto add = [&](int c, float4 v) {
        const float w = ex2(p.part_ml[at(c)].x - M);
        o = make_float4(fmaf(w, v.x, o.x), fmaf(w, v.y, o.y), fmaf(w, v.z, o.z), fmaf(w, v.w, o.w));
      };
      if (live && d < hd) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
          if (c0 + turn + i * WQ <= c1) add(c0 + turn + i * WQ, ahead[i]);
#pragma unroll 4
        for (int c = c0 + turn + AHEAD * WQ; c <= c1; c += WQ)
          add(c, *reinterpret_cast<const float4*>(p.part_o + (int64_t)at(c) * hd + d));
        *reinterpret_cast<float4*>(&part[wid][d]) = o;
      }
      __syncthreads();
      if (turn == 0 && live && d < hd) {
#pragma unroll
        for (int i = 1; i < WQ; ++i) {
          const float4 v = *reinterpret_cast<const float4*>(&part[wid + i][d]);
          o = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
        }
        int head, row;
        query_of(p, u, t, &head, &row);
        T* out = (T*)p.a.out + (int64_t)b * p.a.o_seq + (int64_t)row * p.a.o_row + (int64_t)head * p.a.o_head;
        const float inv = L != 0.f ? 1.f / L : 0.f;
        store_act4(out + d, 0, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
      }
      __syncthreads();  // part is free again
    }
  }
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

int check_query(const dmtp_paged_kv* c, const dmtp_paged_query* a) {
  const int e = check_cache(c);
  if (e) return e;
  if (!a || a->rows < 1 || a->rows > DMTP_OPS_MAX_ROWS || a->n_heads < 1 || a->n_heads > 4096 ||
      a->n_heads % c->n_kv_heads || a->window < 0)
    return DMTP_EINVAL;
  return DMTP_OK;
}

int plan(const dmtp_paged_kv* c, const dmtp_paged_query* a, PagedPlan* pl) {
  const int nq = a->rows * (a->n_heads / c->n_kv_heads), hd = c->head_dim;
  pl->tc = c->dtype == 1 && (hd == 64 || hd == 128);
  if (pl->tc) {
    pl->qn = nq <= 8 ? 8 : nq <= 16 ? 16 : nq <= 32 ? 32 : 64;
    pl->grid = paged_tc_grid(hd, c->e4m3 != 0, pl->qn);
  } else {
    pl->qn = 8;
    pl->grid = paged_simt_grid(hd);
  }
  pl->chunks = (nq + pl->qn - 1) / pl->qn;
  const int64_t reach = (int64_t)c->max_blocks * c->page_size;
  const int64_t units = (int64_t)c->n_seqs * c->n_kv_heads * pl->chunks;
  if ((reach + 63) / 64 * units >= (1ll << 31)) return DMTP_EINVAL;
  pl->whole = reach <= (units >= kWholeUnits ? kWholeReachMany : kWholeReach);
  if (pl->whole) {
    pl->grid = (int)units;
    pl->part_o = pl->part_ml = pl->note = pl->bytes = 0;
    return DMTP_OK;
  }
  const size_t parts = (size_t)pl->grid * 2 * pl->qn;
  pl->part_o = 0;
  pl->part_ml = up256(parts * hd * 4);
  pl->note = pl->part_ml + up256(parts * 8);
  pl->bytes = pl->note + up256((size_t)units * sizeof(PagedNote));
  return DMTP_OK;
}

}  // namespace

extern "C" int dmtp_paged_attention_workspace(const dmtp_paged_kv* c, const dmtp_paged_query* a,
                                              size_t* bytes) {
  const int e = check_query(c, a);
  if (e) return e;
  if (!bytes) return DMTP_EINVAL;
  PagedPlan pl;
  const int r = plan(c, a, &pl);
  if (r) return r;
  *bytes = pl.bytes;
  return DMTP_OK;
}

extern "C" int dmtp_paged_attention(const dmtp_paged_kv* c, const dmtp_paged_query* a, void* workspace,
                                    size_t ws_bytes, uint32_t* err, void* stream) {
  const int e = check_query(c, a);
  if (e) return e;
  const int es = c->dtype ? 2 : 4, hd = c->head_dim;
  if (!a->q || !a->out || !a->kv_len) return DMTP_EINVAL;
  if (!aligned_to(a->q, 16) || !aligned_to(a->out, 16) || !aligned_to(a->kv_len, 4) ||
      !aligned_to(workspace, 256) || (err && !aligned_to(err, 4)))
    return DMTP_EINVAL;
  const int64_t strides[6] = {a->q_seq, a->q_row, a->q_head, a->o_seq, a->o_row, a->o_head};
  for (int64_t s : strides)
    if (s < 0 || !mult(s * es, 16)) return DMTP_EINVAL;
  // (output rows of one address)
  if (a->o_head < hd || (a->rows > 1 && a->o_row < hd) || (c->n_seqs > 1 && a->o_seq < hd)) return DMTP_EINVAL;
  if (!(a->scale >= -1e30f && a->scale <= 1e30f)) return DMTP_EINVAL;
  PagedPlan pl;
  const int r = plan(c, a, &pl);
  if (r) return r;
  if (pl.bytes && !workspace) return DMTP_EINVAL;
  if (ws_bytes < pl.bytes) return DMTP_ENOMEM;
  if (cudaPeekAtLastError() != cudaSuccess) return DMTP_ECUDA;
  PagedAttn p;
  p.m = page_map(*c);
  p.k = c->k;
  p.v = c->v;
  p.ks = c->k_scale;
  p.vs = c->v_scale;
  p.a = *a;
  if (p.a.window >= p.m.reach) p.a.window = 0;  // every position lies inside it
  p.err = err;
  p.group = a->n_heads / c->n_kv_heads;
  p.nq = a->rows * p.group;
  p.qn = pl.qn;
  p.chunks = pl.chunks;
  p.units = c->n_kv_heads * pl.chunks;
  p.part_o = (float*)((char*)workspace + pl.part_o);
  p.part_ml = (float2*)((char*)workspace + pl.part_ml);
  p.note = pl.whole ? nullptr : (PagedNote*)((char*)workspace + pl.note);
  p.scale2 = a->scale * 1.4426950408889634f;
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t le = pl.tc ? paged_attn_tc(p, pl, c->e4m3 != 0, st)
                         : paged_attn_simt(p, pl, c->dtype, c->e4m3 != 0, st);
  if (le == cudaSuccess && !pl.whole) {
    const int nq = p.nq < pl.qn ? p.nq : pl.qn, units = p.units * c->n_seqs;
    // A CTA's 16 warps go by the pieces that a unit has on average, and one more: all to one query
    // while that leaves two CTAs an SM at most. The whole attention with 1 / 4 / 8 / 16 queries a
    // CTA, us: 15 pieces x 32 units of 8 queries 18.5 / 18.9 / 19.5 / 19.5; 58 x 8 of 64 40.7 / 39.8
    // / 41.7 / 43.1; 115 x 4 of 64 39.3 / 41.5 / 44.6 / 49.1; 10 x 32 of 32 32.0 / 26.3 / 26.8 /
    // 27.4; 4 x 128 of 8 35.9 / 30.5 / 30.7 / 30.9, of 64 118 / 76.6 / 68.9 / 65.8.
    const int pieces = pl.grid / units + 1;
    const int per = pieces > 12 && units * nq <= 304 ? 1 : pieces > 6 ? 4 : nq > 8 ? 16 : 8;
    const dim3 grid(units < 1216 ? units : 1216, (nq + per - 1) / per);
    auto k = c->dtype ? (per == 1   ? k_paged_merge<bf16, 1>
                         : per == 4 ? k_paged_merge<bf16, 4>
                         : per == 8 ? k_paged_merge<bf16, 8>
                                    : k_paged_merge<bf16, 16>)
                      : (per == 1   ? k_paged_merge<float, 1>
                         : per == 4 ? k_paged_merge<float, 4>
                         : per == 8 ? k_paged_merge<float, 8>
                                    : k_paged_merge<float, 16>);
    le = launch_op(k, grid, 512, 0, st, true, 1, p, units);
  }
  return le == cudaSuccess ? DMTP_OK : (cudaGetLastError(), DMTP_ECUDA);
}
