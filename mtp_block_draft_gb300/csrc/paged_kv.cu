// dmtp_paged_write and dmtp_paged_read: rows into and out of the pages of a K/V cache.
//
// Write. A group of lanes takes one head of one row: lane i holds eight values of each half
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
  bool wide;         // rows allow 16-byte accesses
};

// Eight consecutive values; `wide`: at a 16-byte boundary (else fp32 at one, bf16 at 8 bytes).
__device__ __forceinline__ void load8(const float* p, bool wide, float (&f)[8]) {
  const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p + 4));
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}
__device__ __forceinline__ void load8(const bf16* p, bool wide, float (&f)[8]) {
  uint4 u;
  if (wide) {
    u = __ldcs(reinterpret_cast<const uint4*>(p));
  } else {
    const uint2 a = __ldcs(reinterpret_cast<const uint2*>(p)), b = __ldcs(reinterpret_cast<const uint2*>(p + 4));
    u = make_uint4(a.x, a.y, b.x, b.y);
  }
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8(float* p, bool wide, const float (&f)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void store8(bf16* p, bool wide, const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  if (wide) {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2*>(p + 4) = make_uint2(w[2], w[3]);
  }
}
__device__ __forceinline__ uint2 e4m3_row8(const float (&f)[8], float inv) {
  return make_uint2(e4m3_row4(make_float4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv)),
                    e4m3_row4(make_float4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv)));
}

// UN: heads that a group has in flight at once.
template <typename T, bool E8, int UN>
__global__ void __launch_bounds__(256) k_paged_write(const WriteArgs a, const Turns turns) {
  __shared__ __align__(16) float cs[2][DMTP_OPS_MAX_HEAD_DIM / 2];
  const int row = blockIdx.x, hd = a.m.head_dim, half = hd >> 1;
  const bool rot = a.r.rope_theta > 0.f;
  const int nq = a.r.q ? a.r.n_heads : 0, hkv = a.m.n_kv_heads, items = nq + 2 * hkv;
  const int gl = threadIdx.x & (a.group - 1), ng = blockDim.x / a.group;
  const bool on = gl < a.lanes;
  // a group's loop count is the CTA's: the shuffles and the barrier below see every thread
  const int step = gridDim.y * ng;
  const int seq = __ldg(a.r.seq + row), pos = __ldg(a.r.pos + row);
  int page = -1, off = 0;
  bool angles = false;
  for (int it0 = blockIdx.y * ng; it0 < items; it0 += step * UN) {
    float x[UN][8], y[UN][8];
#pragma unroll
    for (int n = 0; n < UN; ++n) {
      const int it = it0 + n * step + (int)threadIdx.x / a.group;
      const bool isq = it < nq, isv = it >= nq + hkv;
      const int h = isq ? it : it - nq - (isv ? hkv : 0);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[n][i] = y[n][i] = 0.f;
      if (on && it < items) {
        const T* src = isq   ? (const T*)a.r.q + (int64_t)row * a.r.q_row + (int64_t)h * a.r.q_head
                       : isv ? (const T*)a.r.v + (int64_t)row * a.r.v_row + (int64_t)h * a.r.v_head
                             : (const T*)a.r.k + (int64_t)row * a.r.k_row + (int64_t)h * a.r.k_head;
        load8(src + 8 * gl, a.wide, x[n]);
        load8(src + half + 8 * gl, a.wide, y[n]);
      }
    }
    if (!angles) {  // the page and the angles, while the rows are on their way
      if (seq < 0) return;
      if (seq >= a.m.n_seqs || (unsigned)pos >= (unsigned)a.m.reach) {
        if (threadIdx.x == 0)
          set_err(a.err, seq >= a.m.n_seqs ? DMTP_OPS_ERR_SEQ : DMTP_OPS_ERR_POS);
        return;
      }
      page = page_of(a.m, seq, pos, off, threadIdx.x == 0 ? a.err : nullptr);
      if (page < 0) return;
      if (rot) {
        for (int i = threadIdx.x; i < half; i += blockDim.x) {
          const float2 t = cos_sin_turns((unsigned long long)(unsigned)pos * turns.f[i]);
          cs[0][i] = t.x;
          cs[1][i] = t.y;
        }
        __syncthreads();
      }
      angles = true;
    }
#pragma unroll
    for (int n = 0; n < UN; ++n) {
      const int it = it0 + n * step + (int)threadIdx.x / a.group;
      const bool live = on && it < items, isq = it < nq, isv = it >= nq + hkv;
      const int h = isq ? it : it - nq - (isv ? hkv : 0);
      if (rot && live && !isv) {
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          const float4 c = *reinterpret_cast<const float4*>(&cs[0][8 * gl + i]);
          const float4 s = *reinterpret_cast<const float4*>(&cs[1][8 * gl + i]);
          const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float p = x[n][i + e], q = y[n][i + e];
            x[n][i + e] = p * cc[e] - q * ss[e];
            y[n][i + e] = q * cc[e] + p * ss[e];
          }
        }
      }
      if (live && isq) {
        T* dst = (T*)a.r.q_out + (int64_t)row * a.r.qo_row + (int64_t)h * a.r.qo_head;
        store8(dst + 8 * gl, a.wide, x[n]);
        store8(dst + half + 8 * gl, a.wide, y[n]);
      }
      float amax = 0.f;
      if (E8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fmaxf(finite_abs(x[n][i]), finite_abs(y[n][i])));
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
          *reinterpret_cast<uint2*>(dst + 8 * gl) = e4m3_row8(x[n], inv);
          *reinterpret_cast<uint2*>(dst + half + 8 * gl) = e4m3_row8(y[n], inv);
          if (gl == 0) (isv ? a.vs : a.ks)[(int64_t)page * a.m.scale_stride + line] = pow2f(e);
        } else {
          T* dst = (T*)(isv ? a.v : a.k) + at;
          store8(dst + 8 * gl, true, x[n]);
          store8(dst + half + 8 * gl, true, y[n]);
        }
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

// A group of lanes copies kHeads heads of one row, 16 bytes of the cache a lane and head: the
// chain position -> page -> row is walked once for all of them, and their loads are in flight
// together.
constexpr int kHeads = 4;
template <typename T, bool E8>
__global__ void __launch_bounds__(256) k_paged_read(const ReadArgs a) {
  constexpr int E = E8 ? 16 : 16 / (int)sizeof(T);  // values of a lane
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
      const int64_t at = ((int64_t)page * a.m.page_stride + line * hd) * (E8 ? 1 : (int)sizeof(T)) + 16 * gl;
      u[i] = __ldcs(reinterpret_cast<const uint4*>((const char*)(isv ? a.v : a.k) + at));
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
        const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
        for (int p = 0; p < 4; p += 2) {
          const float4 x = e4m3x4_to_f4(w[p]), y = e4m3x4_to_f4(w[p + 1]);
          const float f[8] = {x.x * s[i], x.y * s[i], x.z * s[i], x.w * s[i],
                              y.x * s[i], y.y * s[i], y.z * s[i], y.w * s[i]};
          store8(dst + 4 * p, true, f);
        }
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
  a.lanes = hd / 16;
  a.group = group_of(a.lanes);
  a.wide = true;
  const int64_t strides[] = {r->k_row, r->k_head, r->v_row, r->v_head,
                             r->q ? r->q_row : 0, r->q ? r->q_head : 0, r->q ? r->qo_row : 0, r->q ? r->qo_head : 0};
  for (int64_t x : strides) a.wide = a.wide && mult(x * es, 16);
  for (const void* p : {r->k, r->v, r->q, (const void*)r->q_out}) a.wide = a.wide && aligned_to(p, 16);
  // few rows: their heads spread over CTAs, one a group; many: a row's heads in one CTA
  const int items = (r->q ? r->n_heads : 0) + 2 * c->n_kv_heads, ng = 256 / a.group;
  const int blocks = (items + ng - 1) / ng;
  const bool few = r->n_rows < 304;
  const dim3 grid(r->n_rows, few ? (blocks < 65535 ? blocks : 65535) : 1);
  const Turns* t = r->rope_theta > 0.f ? &turns_of(r->rope_theta, hd) : nullptr;
  static const Turns none = {};
  auto k = few ? (c->dtype ? (c->e4m3 ? k_paged_write<bf16, true, 1> : k_paged_write<bf16, false, 1>)
                           : (c->e4m3 ? k_paged_write<float, true, 1> : k_paged_write<float, false, 1>))
               : (c->dtype ? (c->e4m3 ? k_paged_write<bf16, true, 2> : k_paged_write<bf16, false, 2>)
                           : (c->e4m3 ? k_paged_write<float, true, 2> : k_paged_write<float, false, 2>));
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
  a.lanes = c->head_dim * (c->e4m3 ? 1 : c->dtype ? 2 : 4) / 16;
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
