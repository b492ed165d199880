// dmtp_paged_write and dmtp_paged_read: rows into and out of the pages of a K/V cache.
//
// Write. A group of lanes takes one head of one row: lane i holds eight values of each half
// of the head (the rotate-half partners sit in one thread), rotates them, and, for an E4M3
// cache, the group reduces the row's largest magnitude and stores bytes and scale. The
// bytes moved are the rows once in and once out; nothing else is read but the positions.
// 8188 rows of 32 + 2 x 4 heads of 128 into bf16 pages take 31.8 us (167 MB, 0.78 of the copy
// rate, two thirds of the issue slots used); 32 rows into E4M3 pages 3.0 us, which is latency.
//
// Angles. Position p turns pair i by p f_i turns, f_i = theta^(-2i/hd) / 2 pi < 1. The host
// forms f_i in double and passes f_i 2^64 as an integer; p times that, modulo 2^64, is the angle's
// fraction of a turn in fixed point, which loses nothing more at far positions and needs none of
// the GPU's slow double arithmetic. What is left is f_i's own error: its power is off by
// (ln(theta) 2i/hd + 4) 2^-53 of itself at most, in turns less than 2^-53, so p 2^-53 at
// position p. The fraction goes to the sine as a 24-bit value and a first-order correction for the rest.
#include <math.h>

#include <cuda_fp16.h>

#include "paged.cuh"

namespace {

struct Turns {
  unsigned long long f[DMTP_OPS_MAX_HEAD_DIM / 2];
};

__device__ __forceinline__ float2 cos_sin_turns(unsigned long long frac) {
  const int hi = (int)(frac >> 32);                       // signed: [-1/2, 1/2) turns
  const float xh = __int2float_rn(hi);
  const long long rest = (long long)(frac - ((unsigned long long)(long long)xh << 32));
  const float d = __ll2float_rn(rest) * 3.4061215800304e-19f;  // 2 pi 2^-64
  float s, c;
  sincospif(xh * 4.656612873077393e-10f, &s, &c);          // 2 * 2^-32 half turns
  return make_float2(fmaf(-s, d, c), fmaf(c, d, s));
}

struct WriteArgs {
  PageMap m;
  void *k, *v;
  float *ks, *vs;
  dmtp_paged_rows r;
  unsigned* err;
  int lanes, group;  // lanes that hold values; lanes of a group (a power of two >= lanes)
  bool wide;         // rows allow 16-byte accesses
};

__device__ __forceinline__ uint2 e4m3_row8(const float (&f)[8], float inv) {
  return make_uint2(e4m3_row4(make_float4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv)),
                    e4m3_row4(make_float4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv)));
}

// A CTA takes ROWS rows: their pages and angles are found together, behind the first heads'
// loads, and a group asks for its next head before it works on the one it has.
template <typename T, bool E8, int ROWS>
__global__ void __launch_bounds__(256) k_paged_write(const WriteArgs a, const Turns turns) {
  __shared__ __align__(16) float cs[ROWS][2][DMTP_OPS_MAX_HEAD_DIM / 2];
  __shared__ int s_page[ROWS], s_off[ROWS], s_pos[ROWS];
  const int row0 = blockIdx.x * ROWS, hd = a.m.head_dim, half = hd >> 1;
  const bool rot = a.r.rope_theta > 0.f;
  const int nq = a.r.q ? a.r.n_heads : 0, hkv = a.m.n_kv_heads, items = nq + 2 * hkv;
  const int rows = min(ROWS, a.r.n_rows - row0), all = rows * items;
  const int gl = threadIdx.x & (a.group - 1), ng = blockDim.x / a.group;
  const bool on = gl < a.lanes;
  // a group's loop count is the CTA's: the shuffles below see every lane
  const int step = gridDim.y * ng, mine = threadIdx.x / a.group;
  Raw<T> x, y;
  auto ask = [&](int it) {
    if (on && it < all) {
      const int r = ROWS == 1 ? 0 : it / items, i = it - r * items;
      const int64_t row = row0 + r;
      const T* src = i < nq         ? (const T*)a.r.q + row * a.r.q_row + (int64_t)i * a.r.q_head
                     : i < nq + hkv ? (const T*)a.r.k + row * a.r.k_row + (int64_t)(i - nq) * a.r.k_head
                                    : (const T*)a.r.v + row * a.r.v_row + (int64_t)(i - nq - hkv) * a.r.v_head;
      fetch(src + 8 * gl, a.wide, x);
      fetch(src + half + 8 * gl, a.wide, y);
    }
  };
  ask(blockIdx.y * ng + mine);
  if (threadIdx.x < ROWS) {
    int page = -1, off = 0, pos = 0;
    if ((int)threadIdx.x < rows) {
      const int seq = __ldg(a.r.seq + row0 + threadIdx.x);
      pos = __ldg(a.r.pos + row0 + threadIdx.x);
      if (seq >= a.m.n_seqs)
        set_err(a.err, DMTP_OPS_ERR_SEQ);
      else if (seq >= 0 && (unsigned)pos >= (unsigned)a.m.reach)
        set_err(a.err, DMTP_OPS_ERR_POS);
      else if (seq >= 0)
        page = page_of(a.m, seq, pos, off, a.err);
    }
    s_page[threadIdx.x] = page;
    s_off[threadIdx.x] = off;
    s_pos[threadIdx.x] = pos;
  }
  if (ROWS > 1) __syncthreads();
  if (rot) {
    for (int i = threadIdx.x; i < rows * half; i += blockDim.x) {
      const int r = ROWS == 1 ? 0 : i / half, h = i - r * half;
      // (of a single row every thread reads the position for itself: no barrier before)
      const int pos = ROWS == 1 ? __ldg(a.r.pos + row0) : s_pos[r];
      const float2 t = cos_sin_turns((unsigned long long)(unsigned)pos * turns.f[h]);
      cs[r][0][h] = t.x;
      cs[r][1][h] = t.y;
    }
  }
  __syncthreads();
  for (int it0 = blockIdx.y * ng; it0 < all; it0 += step) {
    const int it = it0 + mine;
    float f[8], g[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = g[e] = 0.f;
    const int r = ROWS == 1 ? 0 : it / items, i = it - r * items;
    const int page = it < all ? s_page[r] : -1;
    const bool live = on && page >= 0, isq = i < nq, isv = i >= nq + hkv;
    if (live) {
      values(x, f);
      values(y, g);
    }
    ask(it + step);
    if (rot && live && !isv) {
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        const float4 c = *reinterpret_cast<const float4*>(&cs[r][0][8 * gl + e]);
        const float4 s = *reinterpret_cast<const float4*>(&cs[r][1][8 * gl + e]);
        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float p = f[e + j], q = g[e + j];
          f[e + j] = p * cc[j] - q * ss[j];
          g[e + j] = q * cc[j] + p * ss[j];
        }
      }
    }
    if (live && isq) {
      T* dst = (T*)a.r.q_out + (int64_t)(row0 + r) * a.r.qo_row + (int64_t)i * a.r.qo_head;
      store8(dst + 8 * gl, a.wide, f);
      store8(dst + half + 8 * gl, a.wide, g);
    }
    float amax = 0.f;
    if (E8) {
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fmaxf(finite_abs(f[e]), finite_abs(g[e])));
      for (int o = a.group >> 1; o > 0; o >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    }
    if (live && !isq) {
      const int64_t line = (int64_t)(i - nq - (isv ? hkv : 0)) * a.m.page_size + s_off[r];
      const int64_t at = (int64_t)page * a.m.page_stride + line * hd;
      if (E8) {
        const int e = e4m3_exponent(amax);
        const float inv = pow2f(-e);  // |e| <= 126: a normal number, the scaling is exact
        uint8_t* dst = (uint8_t*)(isv ? a.v : a.k) + at;
        *reinterpret_cast<uint2*>(dst + 8 * gl) = e4m3_row8(f, inv);
        *reinterpret_cast<uint2*>(dst + half + 8 * gl) = e4m3_row8(g, inv);
        if (gl == 0) (isv ? a.vs : a.ks)[(int64_t)page * a.m.scale_stride + line] = pow2f(e);
      } else {
        T* dst = (T*)(isv ? a.v : a.k) + at;
        store8(dst + 8 * gl, true, f);
        store8(dst + half + 8 * gl, true, g);
      }
    }
  }
}

struct ReadArgs {
  PageMap m;
  const void *k, *v;
  const float *ks, *vs;
  const int32_t *seq, *pos;
  void *ko, *vo;
  int n_rows, lanes, group;
  unsigned* err;
};

// A group of lanes copies kHeads heads of one row, 16 bytes of the cache a lane and head (of an
// E4M3 cache 8, so that a bf16 row is written in whole lines): the chain position -> page -> row
// is walked once for all of them, and their loads are in flight together. 8 prefixes of 4096 rows of
// 2 x 2 heads of 128, E4M3 to bf16, take 11.5 us (51 MB, 0.65 of the copy rate): 2048 CTAs, 1.7
// waves, each behind that chain of loads. 37 rows take 2.5 us.
constexpr int kHeads = 4;
template <typename T, bool E8>
__global__ void __launch_bounds__(256) k_paged_read(const ReadArgs a) {
  constexpr int E = E8 ? 8 : 16 / (int)sizeof(T);  // values of a lane
  const int hd = a.m.head_dim, hkv = a.m.n_kv_heads;
  const int gl = threadIdx.x & (a.group - 1), ng = blockDim.x / a.group;
  const int64_t row = (int64_t)blockIdx.x * ng + threadIdx.x / a.group;
  const int h0 = blockIdx.y * kHeads;  // of the k and v heads
  if (gl >= a.lanes || row >= a.n_rows) return;
  const int seq = __ldg(a.seq + row), pos = __ldg(a.pos + row);
  if (seq < 0) return;
  if (seq >= a.m.n_seqs || (unsigned)pos >= (unsigned)a.m.reach) {
    if (gl == 0) set_err(a.err, seq >= a.m.n_seqs ? DMTP_OPS_ERR_SEQ : DMTP_OPS_ERR_POS);
    return;
  }
  int off;
  const int page = page_of(a.m, seq, pos, off, gl == 0 ? a.err : nullptr);
  if (page < 0) return;
  uint4 u[kHeads];
  float s[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int h2 = h0 + i;
    if (h2 < 2 * hkv) {
      const bool isv = h2 >= hkv;
      const int64_t line = (int64_t)(isv ? h2 - hkv : h2) * a.m.page_size + off;
      const int64_t at = ((int64_t)page * a.m.page_stride + line * hd) * (E8 ? 1 : (int)sizeof(T)) + (E8 ? 8 : 16) * gl;
      const char* src = (const char*)(isv ? a.v : a.k) + at;
      if (E8) {
        const uint2 w = __ldcs(reinterpret_cast<const uint2*>(src));
        u[i] = make_uint4(w.x, w.y, 0, 0);
      } else {
        u[i] = __ldcs(reinterpret_cast<const uint4*>(src));
      }
      if (E8) s[i] = __ldg((isv ? a.vs : a.ks) + (int64_t)page * a.m.scale_stride + line);
    }
  }
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int h2 = h0 + i;
    if (h2 < 2 * hkv) {
      const bool isv = h2 >= hkv;
      T* dst = (T*)(isv ? a.vo : a.ko) + (row * hkv + (isv ? h2 - hkv : h2)) * hd + E * gl;
      if (E8) {
        const float4 x = e4m3x4_to_f4(u[i].x), y = e4m3x4_to_f4(u[i].y);
        const float f[8] = {x.x * s[i], x.y * s[i], x.z * s[i], x.w * s[i],
                            y.x * s[i], y.y * s[i], y.z * s[i], y.w * s[i]};
        store8(dst, true, f);
      } else {
        *reinterpret_cast<uint4*>(dst) = u[i];
      }
    }
  }
}

int group_of(int lanes) {
  int g = 1;
  while (g < lanes) g <<= 1;
  return g;
}

}  // namespace

namespace dmtp {

int check_cache(const dmtp_paged_kv* c) {
  if (!c || !c->k || !c->v || !c->table) return DMTP_EINVAL;
  if ((c->dtype != 0 && c->dtype != 1) || (c->e4m3 != 0 && c->e4m3 != 1)) return DMTP_EINVAL;
  if (c->e4m3 && (!c->k_scale || !c->v_scale)) return DMTP_EINVAL;
  if (c->head_dim < 16 || c->head_dim > DMTP_OPS_MAX_HEAD_DIM || c->head_dim % 16) return DMTP_EINVAL;
  if (c->n_pages < 1 || c->n_kv_heads < 1 || c->n_kv_heads > 4096 || c->n_seqs < 1 || c->max_blocks < 1)
    return DMTP_EINVAL;
  if (c->page_size < 1 || c->page_size > 65536) return DMTP_EINVAL;
  if ((int64_t)c->max_blocks * c->page_size >= (1ll << 31) - 65536) return DMTP_EINVAL;
  const int64_t lines = (int64_t)c->n_kv_heads * c->page_size;
  const int es = c->e4m3 ? 1 : c->dtype ? 2 : 4;
  if (c->page_stride < lines * c->head_dim || !mult(c->page_stride * es, 16)) return DMTP_EINVAL;
  if (c->e4m3 && c->scale_stride < lines) return DMTP_EINVAL;
  if (c->table_stride < c->max_blocks) return DMTP_EINVAL;
  if (!aligned_to(c->k, 16) || !aligned_to(c->v, 16)) return DMTP_EINVAL;
  if (c->e4m3 && (!aligned_to(c->k_scale, 4) || !aligned_to(c->v_scale, 4))) return DMTP_EINVAL;
  if (!aligned_to(c->table, 4)) return DMTP_EINVAL;
  return DMTP_OK;
}

}  // namespace dmtp

using namespace dmtp;

namespace {
// theta^(-2i/hd) / (2 pi) * 2^64 for a head's pairs; a thread that keeps calling with
// one base and head size forms them once.
const Turns& turns_of(float theta, int hd) {
  static thread_local Turns t;
  static thread_local float t_theta = 0.f;
  static thread_local int t_hd = 0;
  if (theta != t_theta || hd != t_hd) {
    for (int i = 0; i < hd / 2; ++i) {
      const double f = pow((double)theta, -2.0 * i / hd) * 0.15915494309189533577;
      t.f[i] = f >= 1.0 ? 0 : (unsigned long long)ldexp(f, 64);
    }
    t_theta = theta;
    t_hd = hd;
  }
  return t;
}
bool row_ok(const void* p, int64_t row, int64_t head, int es, int hd, int heads) {
  return p && aligned_to(p, 4 * es) && mult(row, 4) && mult(head, 4) && head >= hd && row >= 0 &&
         heads >= 1;
}
}  // namespace

extern "C" int dmtp_paged_write(const dmtp_paged_kv* c, const dmtp_paged_rows* r, uint32_t* err,
                                void* stream) {
  int e = check_cache(c);
  if (e) return e;
  if (!r || r->n_rows < 0) return DMTP_EINVAL;
  if (r->n_rows == 0) return DMTP_OK;
  const int es = c->dtype ? 2 : 4, hd = c->head_dim;
  if (!row_ok(r->k, r->k_row, r->k_head, es, hd, 1) || !row_ok(r->v, r->v_row, r->v_head, es, hd, 1) ||
      !r->seq || !r->pos || !aligned_to(r->seq, 4) || !aligned_to(r->pos, 4))
    return DMTP_EINVAL;
  if (r->q && (r->n_heads < 1 || r->n_heads > 4096 ||
               !row_ok(r->q, r->q_row, r->q_head, es, hd, r->n_heads) ||
               !row_ok(r->q_out, r->qo_row, r->qo_head, es, hd, r->n_heads) ||
               (r->n_rows > 1 && r->qo_row < hd)))  // rows of one address
    return DMTP_EINVAL;
  // theta >= 1: every pair's rate is at most one radian per position, below one turn
  if (!(r->rope_theta == 0.f || (r->rope_theta >= 1.f && r->rope_theta <= 3.4e38f))) return DMTP_EINVAL;
  if (err && !aligned_to(err, 4)) return DMTP_EINVAL;
  if (cudaPeekAtLastError() != cudaSuccess) return DMTP_ECUDA;
  WriteArgs a;
  a.m = page_map(*c);
  a.k = c->k;
  a.v = c->v;
  a.ks = c->k_scale;
  a.vs = c->v_scale;
  a.r = *r;
  a.err = err;
  a.lanes = hd / 16;
  a.group = group_of(a.lanes);
  a.wide = true;
  const int64_t strides[] = {r->k_row, r->k_head, r->v_row, r->v_head,
                             r->q ? r->q_row : 0, r->q ? r->q_head : 0, r->q ? r->qo_row : 0, r->q ? r->qo_head : 0};
  for (int64_t x : strides) a.wide = a.wide && mult(x * es, 16);
  for (const void* p : {r->k, r->v, r->q, (const void*)r->q_out}) a.wide = a.wide && aligned_to(p, 16);
  // Few rows: one a CTA, its heads spread over CTAs, one a group, so that a row's chain of loads
  // is walked once. More: four rows a CTA, whose pages and angles are found together, spread over
  // CTAs while there are fewer than four an SM. Rows of 40 heads of 128, us, few / many: 32 into
  // bf16 pages 3.1 / 3.3 (not spread 5.1), 256 3.5 / 4.3, 512 5.0 / 5.0, 768 6.5 / 5.7, 1024 7.7 /
  // 6.7, 2047 14.7 / 10.3; into E4M3 pages 256 4.0 / 4.7, 512 5.7 / 5.7, 768 7.4 / 6.3; of 144
  // heads 64 3.5 / 3.8, 307 7.2 / 6.9, 600 12.3 / 10.3.
  const int items = (r->q ? r->n_heads : 0) + 2 * c->n_kv_heads, ng = 256 / a.group;
  const int blocks = (items + ng - 1) / ng;
  const bool few = (int64_t)r->n_rows * blocks <= 608;
  const int quads = (r->n_rows - 1) / 4 + 1, spread = quads < 608 ? 608 / quads : 1, rounds = (4 * items + ng - 1) / ng;
  const dim3 grid(few ? r->n_rows : quads, few ? blocks : spread < rounds ? spread : rounds);
  const Turns* t = r->rope_theta > 0.f ? &turns_of(r->rope_theta, hd) : nullptr;
  static const Turns none = {};
  auto k = few ? (c->dtype ? (c->e4m3 ? k_paged_write<bf16, true, 1> : k_paged_write<bf16, false, 1>)
                           : (c->e4m3 ? k_paged_write<float, true, 1> : k_paged_write<float, false, 1>))
               : (c->dtype ? (c->e4m3 ? k_paged_write<bf16, true, 4> : k_paged_write<bf16, false, 4>)
                           : (c->e4m3 ? k_paged_write<float, true, 4> : k_paged_write<float, false, 4>));
  return launch_op(k, grid, 256, 0, (cudaStream_t)stream, false, 1, a, t ? *t : none) == cudaSuccess
             ? DMTP_OK
             : (cudaGetLastError(), DMTP_ECUDA);
}

extern "C" int dmtp_paged_read(const dmtp_paged_kv* c, const int32_t* seq, const int32_t* pos,
                               int n_rows, void* k_out, void* v_out, uint32_t* err, void* stream) {
  int e = check_cache(c);
  if (e) return e;
  if (n_rows < 0) return DMTP_EINVAL;
  if (n_rows == 0) return DMTP_OK;
  if (!seq || !pos || !k_out || !v_out || !aligned_to(seq, 4) || !aligned_to(pos, 4) ||
      !aligned_to(k_out, 16) || !aligned_to(v_out, 16) || (err && !aligned_to(err, 4)))
    return DMTP_EINVAL;
  if (cudaPeekAtLastError() != cudaSuccess) return DMTP_ECUDA;
  ReadArgs a;
  a.m = page_map(*c);
  a.k = c->k;
  a.v = c->v;
  a.ks = c->k_scale;
  a.vs = c->v_scale;
  a.seq = seq;
  a.pos = pos;
  a.ko = k_out;
  a.vo = v_out;
  a.n_rows = n_rows;
  a.lanes = c->head_dim / (c->e4m3 || c->dtype ? 8 : 4);
  a.group = group_of(a.lanes);
  a.err = err;
  const int ng = 256 / a.group, heads = (2 * c->n_kv_heads + kHeads - 1) / kHeads;
  const dim3 grid((unsigned)((n_rows + (int64_t)ng - 1) / ng), heads);
  auto k = c->dtype ? (c->e4m3 ? k_paged_read<bf16, true> : k_paged_read<bf16, false>)
                    : (c->e4m3 ? k_paged_read<float, true> : k_paged_read<float, false>);
  return launch_op(k, grid, 256, 0, (cudaStream_t)stream, false, 1, a) == cudaSuccess
             ? DMTP_OK
             : (cudaGetLastError(), DMTP_ECUDA);
}
