// dmtp_paged_write and dmtp_paged_read: rows into and out of the pages of a K/V cache.
//
// Write. A group of lanes takes one head of one row: lane i holds four values of each half
// of the head (the rotate-half partners sit in one thread), rotates them, and, for an E4M3
// cache, the group reduces the row's largest magnitude and stores bytes and scale. The
// bytes moved are the rows once in and once out; nothing else is read but the positions.
//
// Angles. Position p turns pair i by p f_i turns, f_i = theta^(-2i/hd) / 2 pi < 1. The host
// forms f_i in double and passes round(f_i 2^64); p times that, modulo 2^64, is the angle's
// fraction of a turn in fixed point, with no loss at far positions (error p 2^-55 from
// f_i's own 53 bits) and without the GPU's slow double arithmetic. The fraction
// goes to the sine as a 24-bit value and a first-order correction for the rest.
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
};

template <typename T>
__device__ __forceinline__ void store4(T* p, float4 v) {
  store_act4(p, 0, v);
}

template <typename T, bool E8>
__global__ void __launch_bounds__(256) k_paged_write(const WriteArgs a, const Turns turns) {
  __shared__ float2 cs[DMTP_OPS_MAX_HEAD_DIM / 2];
  const int row = blockIdx.x, hd = a.m.head_dim, half = hd >> 1;
  const int seq = __ldg(a.r.seq + row), pos = __ldg(a.r.pos + row);
  if (seq < 0) return;
  if (seq >= a.m.n_seqs || (unsigned)pos >= (unsigned)a.m.reach) {
    if (threadIdx.x == 0)
      set_err(a.err, seq >= a.m.n_seqs ? DMTP_OPS_ERR_SEQ : DMTP_OPS_ERR_POS);
    return;
  }
  int off;
  const int page = page_of(a.m, seq, pos, off, threadIdx.x == 0 ? a.err : nullptr);
  if (page < 0) return;
  const bool rot = a.r.rope_theta > 0.f;
  if (rot) {
    for (int i = threadIdx.x; i < half; i += blockDim.x)
      cs[i] = cos_sin_turns((unsigned long long)(unsigned)pos * turns.f[i]);
    __syncthreads();
  }
  const int nq = a.r.q ? a.r.n_heads : 0, hkv = a.m.n_kv_heads, items = nq + 2 * hkv;
  const int gl = threadIdx.x & (a.group - 1), ng = blockDim.x / a.group;
  const bool on = gl < a.lanes;
  // a group's loop count is the warp's: the shuffles below see every lane
  const int first = blockIdx.y * ng, step = gridDim.y * ng;
  for (int it0 = first; it0 < items; it0 += step) {
    const int it = it0 + (int)threadIdx.x / a.group;
    const bool live = on && it < items;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
    const bool isq = it < nq;
    const int h = isq ? it : it - nq < hkv ? it - nq : it - nq - hkv;
    const bool isv = it >= nq + hkv;
    if (live) {
      const T* src = isq   ? (const T*)a.r.q + (int64_t)row * a.r.q_row + (int64_t)h * a.r.q_head
                     : isv ? (const T*)a.r.v + (int64_t)row * a.r.v_row + (int64_t)h * a.r.v_head
                           : (const T*)a.r.k + (int64_t)row * a.r.k_row + (int64_t)h * a.r.k_head;
      x = load4(src + 4 * gl);
      y = load4(src + half + 4 * gl);
      if (rot && !isv) {
        const float2 t0 = cs[4 * gl], t1 = cs[4 * gl + 1], t2 = cs[4 * gl + 2], t3 = cs[4 * gl + 3];
        const float4 u = x;
        x = make_float4(u.x * t0.x - y.x * t0.y, u.y * t1.x - y.y * t1.y, u.z * t2.x - y.z * t2.y,
                        u.w * t3.x - y.w * t3.y);
        y = make_float4(y.x * t0.x + u.x * t0.y, y.y * t1.x + u.y * t1.y, y.z * t2.x + u.z * t2.y,
                        y.w * t3.x + u.w * t3.y);
      }
    }
    if (live && isq) {
      T* dst = (T*)a.r.q_out + (int64_t)row * a.r.qo_row + (int64_t)h * a.r.qo_head;
      store4(dst + 4 * gl, x);
      store4(dst + half + 4 * gl, y);
    }
    float amax = 0.f;
    if (E8) {
      amax = fmaxf(fmaxf(fmaxf(finite_abs(x.x), finite_abs(x.y)), fmaxf(finite_abs(x.z), finite_abs(x.w))),
                   fmaxf(fmaxf(finite_abs(y.x), finite_abs(y.y)), fmaxf(finite_abs(y.z), finite_abs(y.w))));
      for (int o = a.group >> 1; o > 0; o >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    }
    if (live && !isq) {
      const int64_t line = (int64_t)h * a.m.page_size + off;
      const int64_t at = (int64_t)page * a.m.page_stride + line * hd;
      if (E8) {
        const int e = e4m3_exponent(amax);
        const float inv = pow2f(-e);  // |e| <= 126: a normal number, the scaling is exact
        uint8_t* dst = (uint8_t*)(isv ? a.v : a.k) + at;
        *reinterpret_cast<uint32_t*>(dst + 4 * gl) =
            e4m3_row4(make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
        *reinterpret_cast<uint32_t*>(dst + half + 4 * gl) =
            e4m3_row4(make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
        if (gl == 0) (isv ? a.vs : a.ks)[(int64_t)page * a.m.scale_stride + line] = pow2f(e);
      } else {
        T* dst = (T*)(isv ? a.v : a.k) + at;
        store4(dst + 4 * gl, x);
        store4(dst + half + 4 * gl, y);
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

// A group of lanes copies one head's row, eight values a lane.
template <typename T, bool E8>
__global__ void __launch_bounds__(256) k_paged_read(const ReadArgs a) {
  const int hd = a.m.head_dim, hkv = a.m.n_kv_heads;
  const int gl = threadIdx.x & (a.group - 1), ng = blockDim.x / a.group;
  const int64_t it = (int64_t)blockIdx.x * ng + threadIdx.x / a.group;
  if (gl >= a.lanes || it >= (int64_t)a.n_rows * 2 * hkv) return;
  const int row = (int)(it / (2 * hkv)), h2 = (int)(it - (int64_t)row * 2 * hkv);
  const bool isv = h2 >= hkv;
  const int h = isv ? h2 - hkv : h2;
  const int seq = __ldg(a.seq + row), pos = __ldg(a.pos + row);
  if (seq < 0) return;
  if (seq >= a.m.n_seqs || (unsigned)pos >= (unsigned)a.m.reach) {
    if (gl == 0) set_err(a.err, seq >= a.m.n_seqs ? DMTP_OPS_ERR_SEQ : DMTP_OPS_ERR_POS);
    return;
  }
  int off;
  const int page = page_of(a.m, seq, pos, off, gl == 0 ? a.err : nullptr);
  if (page < 0) return;
  const int64_t line = (int64_t)h * a.m.page_size + off;
  const int64_t at = (int64_t)page * a.m.page_stride + line * hd + 8 * gl;
  T* dst = (T*)(isv ? a.vo : a.ko) + ((int64_t)row * hkv + h) * hd + 8 * gl;
  if (E8) {
    const uint2 u = __ldcs(reinterpret_cast<const uint2*>((const uint8_t*)(isv ? a.v : a.k) + at));
    const float s = __ldg((isv ? a.vs : a.ks) + (int64_t)page * a.m.scale_stride + line);
    const float4 x = e4m3x4_to_f4(u.x), y = e4m3x4_to_f4(u.y);
    store4(dst, make_float4(x.x * s, x.y * s, x.z * s, x.w * s));
    store4(dst + 4, make_float4(y.x * s, y.y * s, y.z * s, y.w * s));
  } else {
    const uint4* src = reinterpret_cast<const uint4*>((const T*)(isv ? a.v : a.k) + at);
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(dst)[i] = __ldcs(src + i);
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
// round(theta^(-2i/hd) / (2 pi) * 2^64) for a head's pairs; a thread that keeps calling with
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
               !row_ok(r->q_out, r->qo_row, r->qo_head, es, hd, r->n_heads)))
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
  a.lanes = hd / 8;
  a.group = group_of(a.lanes);
  const int items = (r->q ? r->n_heads : 0) + 2 * c->n_kv_heads, ng = 256 / a.group;
  const int blocks = (items + ng - 1) / ng;
  const dim3 grid(r->n_rows, r->n_rows < 304 ? (blocks < 65535 ? blocks : 65535) : 1);
  const Turns* t = r->rope_theta > 0.f ? &turns_of(r->rope_theta, hd) : nullptr;
  static const Turns none = {};
  auto k = c->dtype ? (c->e4m3 ? k_paged_write<bf16, true> : k_paged_write<bf16, false>)
                    : (c->e4m3 ? k_paged_write<float, true> : k_paged_write<float, false>);
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
  a.lanes = c->head_dim / 8;
  a.group = group_of(a.lanes);
  a.err = err;
  const int ng = 256 / a.group;
  const int64_t blocks = ((int64_t)n_rows * 2 * c->n_kv_heads + ng - 1) / ng;
  if (blocks > 0x7fffffff) return DMTP_EINVAL;
  auto k = c->dtype ? (c->e4m3 ? k_paged_read<bf16, true> : k_paged_read<bf16, false>)
                    : (c->e4m3 ? k_paged_read<float, true> : k_paged_read<float, false>);
  return launch_op(k, dim3((unsigned)blocks), 256, 0, (cudaStream_t)stream, false, 1, a) == cudaSuccess
             ? DMTP_OK
             : (cudaGetLastError(), DMTP_ECUDA);
}
