// dmtp_paged_attention: argument checks, the plan (which kernel, how many CTAs, the
// workspace) and the merge of split units.
#include "paged_attn.cuh"

using namespace dmtp;

namespace {

// The merge of the unit that CTA blockIdx.x began and did not end (paged_attn.cuh): with M the
// largest of the pieces' maxima, out = sum_c 2^(m_c - M) O_c / sum_c 2^(m_c - M) l_c. A CTA takes
// PER queries: four of them, one a warp, or one, with every fourth piece a warp's and the four
// sums added in order. It is all latency (the pieces lie in L2), so their rows are asked for
// eight at a time.
template <typename T, int PER>
__global__ void __launch_bounds__(128) k_paged_merge(const PagedAttn p) {
  __shared__ __align__(16) float part[3][DMTP_OPS_MAX_HEAD_DIM];
  pdl_wait();
  const int c0 = blockIdx.x, hd = p.m.head_dim, lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const PagedNote note = p.note[c0];
  if (note.b < 0) return;
  const int t = PER == 4 ? blockIdx.y * 4 + wid : blockIdx.y;
  if (t >= queries_of(p, note.unit)) return;
  const int c1 = note.last;
  float M = -INFINITY, L = 0.f;
  for (int c = c0 + lane; c <= c1; c += 32)
    M = fmaxf(M, p.part_ml[(c * 2 + (c == c0)) * p.qn + t].x);
  M = warp_max(M);
  const float ref = M == -INFINITY ? 0.f : M;
  for (int c = c0 + lane; c <= c1; c += 32) {
    const float2 ml = p.part_ml[(c * 2 + (c == c0)) * p.qn + t];
    L += ml.y * ex2(ml.x - ref);
  }
  L = warp_sum(L);
  const float inv = L != 0.f ? 1.f / L : 0.f;
  int head, row;
  query_of(p, note.unit, t, &head, &row);
  T* out = (T*)p.a.out + (int64_t)note.b * p.a.o_seq + (int64_t)row * p.a.o_row + (int64_t)head * p.a.o_head;
  for (int d = 4 * lane; d < (hd + 127) / 128 * 128; d += 128) {
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (d < hd) {
#pragma unroll 8
      for (int c = c0 + (PER == 4 ? 0 : wid); c <= c1; c += (PER == 4 ? 1 : 4)) {
        const int at = (c * 2 + (c == c0)) * p.qn + t;
        const float w = ex2(p.part_ml[at].x - ref);
        const float4 v = *reinterpret_cast<const float4*>(p.part_o + (int64_t)at * hd + d);
        o = make_float4(fmaf(w, v.x, o.x), fmaf(w, v.y, o.y), fmaf(w, v.z, o.z), fmaf(w, v.w, o.w));
      }
    }
    if (PER == 1) {
      if (wid && d < hd) *reinterpret_cast<float4*>(&part[wid - 1][d]) = o;
      __syncthreads();
      if (wid) continue;
      if (d < hd) {
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          const float4 v = *reinterpret_cast<const float4*>(&part[i][d]);
          o = make_float4(o.x + v.x, o.y + v.y, o.z + v.z, o.w + v.w);
        }
      }
    }
    if (d < hd) store_act4(out + d, 0, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
  }
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

int check_query(const dmtp_paged_kv* c, const dmtp_paged_query* a) {
  const int e = check_cache(c);
  if (e) return e;
  if (!a || a->rows < 1 || a->rows > DMTP_OPS_MAX_ROWS || a->n_heads < 1 || a->n_heads > 4096 ||
      a->n_heads % c->n_kv_heads || a->window < 0 || c->n_seqs > 65535)
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
    pl->grid = paged_simt_grid(hd, c->dtype, c->e4m3 != 0);
  }
  pl->chunks = (nq + pl->qn - 1) / pl->qn;
  const int64_t reach = (int64_t)c->max_blocks * c->page_size;
  const int64_t units = (int64_t)c->n_seqs * c->n_kv_heads * pl->chunks;
  if ((reach + 63) / 64 * units >= (1ll << 31)) return DMTP_EINVAL;
  pl->whole = reach <= kWholeReach;
  if (pl->whole) {
    pl->grid = (int)units;
    pl->part_o = pl->part_ml = pl->note = pl->bytes = 0;
    return DMTP_OK;
  }
  const size_t parts = (size_t)pl->grid * 2 * pl->qn;
  pl->part_o = 0;
  pl->part_ml = up256(parts * hd * 4);
  pl->note = pl->part_ml + up256(parts * 8);
  pl->bytes = pl->note + up256((size_t)pl->grid * sizeof(PagedNote));
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
  if (a->o_head < hd || !(a->scale > -3.4e38f && a->scale < 3.4e38f)) return DMTP_EINVAL;
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
    const int nq = p.nq < pl.qn ? p.nq : pl.qn;
    const bool four = nq > 8;
    const dim3 grid(pl.grid, four ? (nq + 3) / 4 : nq);
    auto k = c->dtype ? (four ? k_paged_merge<bf16, 4> : k_paged_merge<bf16, 1>)
                      : (four ? k_paged_merge<float, 4> : k_paged_merge<float, 1>);
    le = launch_op(k, grid, 128, 0, st, true, 1, p);
  }
  return le == cudaSuccess ? DMTP_OK : (cudaGetLastError(), DMTP_ECUDA);
}
