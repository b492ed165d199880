// dmtp_paged_prompt_attention: argument checks, the plan and the merge of split units.
#include "paged_attn.cuh"
#include "paged_prompt.cuh"

using namespace dmtp;

namespace {

// out = sum_z 2^(m_z - M) O_z / sum_z 2^(m_z - M) l_z over the ranges of a unit, in order. A warp
// takes a query.
template <typename T>
__global__ void __launch_bounds__(256) k_prompt_merge(const PagedPrompt p) {
  pdl_wait();
  PromptTile w;
  if (!prompt_tile(p, blockIdx.x, w)) return;
  const int lane = threadIdx.x & 31, hd = p.m.head_dim, kvh = blockIdx.y;
  const int64_t unit = (int64_t)blockIdx.x * gridDim.y + kvh;
  for (int t = blockIdx.z * 8 + (threadIdx.x >> 5); t < w.count; t += gridDim.z * 8) {
    const int64_t at = unit * p.splits * p.tile + t;
    float M = -INFINITY;
    for (int z = 0; z < p.splits; ++z) M = fmaxf(M, p.part_ml[at + (int64_t)z * p.tile].x);
    const float ref = M == -INFINITY ? 0.f : M;
    float L = 0.f;
    for (int z = 0; z < p.splits; ++z) {
      const float2 ml = p.part_ml[at + (int64_t)z * p.tile];
      L += ml.y * ex2(ml.x - ref);
    }
    const float inv = L != 0.f ? 1.f / L : 0.f;
    const int i = (w.q0 + t) / p.group, head = kvh * p.group + (w.q0 + t - i * p.group);
    T* out = (T*)p.a.out + (int64_t)(w.row0 + i) * p.a.o_row + (int64_t)head * p.a.o_head;
    for (int d = 4 * lane; d < hd; d += 128) {
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int z = 0; z < p.splits; ++z) {
        const float f = ex2(p.part_ml[at + (int64_t)z * p.tile].x - ref);
        const float4 v = *reinterpret_cast<const float4*>(p.part_o + (at + (int64_t)z * p.tile) * hd + d);
        o = make_float4(fmaf(f, v.x, o.x), fmaf(f, v.y, o.y), fmaf(f, v.z, o.z), fmaf(f, v.w, o.w));
      }
      store_act4(out + d, 0, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
    }
  }
}

size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

int check_prompt(const dmtp_paged_kv* c, const dmtp_paged_prompt* a) {
  const int e = check_cache(c);
  if (e) return e;
  if (!a || a->n_rows < 0 || a->n_rows > (1 << 24) || a->n_heads < 1 || a->n_heads > 4096 ||
      a->n_heads % c->n_kv_heads || (int64_t)a->n_rows * a->n_heads >= (1ll << 31) - 65536)
    return DMTP_EINVAL;
  return DMTP_OK;
}

int plan(const dmtp_paged_kv* c, const dmtp_paged_prompt* a, PromptPlan* pl) {
  const int64_t nq = (int64_t)a->n_rows * (a->n_heads / c->n_kv_heads);
  pl->tc = c->dtype == 1 && c->head_dim <= 128;
  pl->tile = pl->tc ? 256 : 64;
  const int64_t tiles = nq / pl->tile + (c->n_seqs < a->n_rows ? c->n_seqs : a->n_rows);
  const int64_t units = tiles * c->n_kv_heads, reach = (int64_t)c->max_blocks * c->page_size;
  if (tiles >= (1ll << 31)) return DMTP_EINVAL;
  pl->tiles = (int)tiles;
  // Few units: their keys are split so that all together fill the SMs once (the CUDA-core kernel's two
  // CTAs an SM), into ranges of 512 positions of the table's reach at least. 32 / 4 heads of 128, us, whole /
  // split: 8 rows over 32768 bf16 positions 267 / 42, 64 rows 299 / 51, over 2048 33 / 26, 256 rows over
  // 2048 38 / 31, 4 x 16 rows over 4096 53 / 26; fp32, 64 rows over 16384 2635 / 505 (469 now). Ranges of 256: 512
  // rows over nothing 27.5 instead of 20.3, 64 rows over 2048 24.4 instead of 25.8.
  int64_t s = units ? (pl->tc ? 152 : 304) / units : 1;
  const int64_t most = reach / 512;
  s = s > most ? most : s;
  pl->splits = s < 1 ? 1 : s > 64 ? 64 : (int)s;
  pl->part_o = pl->part_ml = pl->bytes = 0;
  if (pl->splits > 1) {
    const size_t parts = (size_t)units * pl->splits * pl->tile;
    pl->part_ml = up256(parts * c->head_dim * 4);
    pl->bytes = pl->part_ml + up256(parts * 8);
  }
  return DMTP_OK;
}

}  // namespace

extern "C" int dmtp_paged_prompt_workspace(const dmtp_paged_kv* c, const dmtp_paged_prompt* a, size_t* bytes) {
  const int e = check_prompt(c, a);
  if (e) return e;
  if (!bytes) return DMTP_EINVAL;
  PromptPlan pl;
  const int r = plan(c, a, &pl);
  if (r) return r;
  *bytes = pl.bytes;
  return DMTP_OK;
}

extern "C" int dmtp_paged_prompt_attention(const dmtp_paged_kv* c, const dmtp_paged_prompt* a, void* workspace,
                                           size_t ws_bytes, uint32_t* err, void* stream) {
  const int e = check_prompt(c, a);
  if (e) return e;
  const int es = c->dtype ? 2 : 4, hd = c->head_dim;
  if (a->window < 0 || !(a->scale >= -1e30f && a->scale <= 1e30f) || !scores_ok(a->scores)) return DMTP_EINVAL;
  if (a->n_rows == 0) return DMTP_OK;
  if (!a->q || !a->out || !a->row_start || !a->kv_len) return DMTP_EINVAL;
  if (!aligned_to(a->q, 16) || !aligned_to(a->out, 16) || !aligned_to(a->row_start, 4) || !aligned_to(a->kv_len, 4) ||
      !aligned_to(a->first, 4) || !aligned_to(a->end, 4) || !aligned_to(workspace, 256) || (err && !aligned_to(err, 4)))
    return DMTP_EINVAL;
  const int64_t strides[4] = {a->q_row, a->q_head, a->o_row, a->o_head};
  for (int64_t s : strides)
    if (s < 0 || !mult(s * es, 16)) return DMTP_EINVAL;
  if (a->o_head < hd || (a->n_rows > 1 && a->o_row < hd)) return DMTP_EINVAL;  // (output rows of one address)
  PromptPlan pl;
  const int r = plan(c, a, &pl);
  if (r) return r;
  if (pl.bytes && !workspace) return DMTP_EINVAL;
  if (ws_bytes < pl.bytes) return DMTP_ENOMEM;
  if (cudaPeekAtLastError() != cudaSuccess) return DMTP_ECUDA;
  PagedPrompt p;
  p.m = page_map(*c);
  p.k = c->k;
  p.v = c->v;
  p.ks = c->k_scale;
  p.vs = c->v_scale;
  p.a = *a;
  if (p.a.window >= p.m.reach) p.a.window = 0;  // every position lies inside it
  p.err = err;
  p.group = a->n_heads / c->n_kv_heads;
  p.tile = pl.tile;
  p.splits = pl.splits;
  p.scale2 = a->scale * 1.4426950408889634f;
  p.capl = a->scores.cap * 1.4426950408889634f;
  p.cap_inv = p.capl > 0.f ? 1.f / p.capl : 0.f;
  p.part_o = (float*)((char*)workspace + pl.part_o);
  p.part_ml = (float2*)((char*)workspace + pl.part_ml);
  cudaStream_t st = (cudaStream_t)stream;
  const bool mod = p.capl > 0.f || a->scores.slopes;
  cudaError_t le = pl.tc ? paged_prompt_tc(p, pl, rows_of(*c), mod, st) : paged_prompt_simt(p, pl, c->dtype, rows_of(*c), st);
  if (le == cudaSuccess && pl.splits > 1) {
    const dim3 grid(pl.tiles, c->n_kv_heads, pl.tile / 8);
    le = launch_op(c->dtype ? k_prompt_merge<bf16> : k_prompt_merge<float>, grid, 256, 0, st, true, 1, p);
  }
  return le == cudaSuccess ? DMTP_OK : (cudaGetLastError(), DMTP_ECUDA);
}
