// Shared by the operators of a decode step over a paged cache (include/dmtp_ops.h):
// device-side page lookups, E4M3 row helpers, row loads, and the launch helpers.
#pragma once

#include <cuda_fp16.h>

#include "../../include/dmtp_ops.h"
#include "common.cuh"
#include "ops.h"

namespace dmtp {

// How a cache's rows are stored: values of its dtype, or with scales.
enum Rows { kRaw, kE4M3, kE2M1 };
inline Rows rows_of(const dmtp_paged_kv& c) { return c.e4m3 == DMTP_OPS_E2M1 ? kE2M1 : c.e4m3 ? kE4M3 : kRaw; }

// ---- host -----------------------------------------------------------------------------
// Launch on `st`; `after`: a kernel of the same call precedes it and it calls pdl_wait()
// before touching what that one writes, so its launch may overlap the other's end.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_op(void (*k)(KArgs...), dim3 grid, dim3 block, size_t smem,
                             cudaStream_t st, bool after, unsigned cluster, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  unsigned n = 0;
  if (cluster > 1) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = cluster;
    at[n].val.clusterDim.y = 1;
    at[n].val.clusterDim.z = 1;
    ++n;
  }
  if (after && pdl_enabled()) {
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = at;
  cfg.numAttrs = n;
  pdl_fence();  // the round's own launches do not overlap an operator's
  return cudaLaunchKernelEx(&cfg, k, static_cast<KArgs>(args)...);
}
// Raise a kernel's dynamic shared memory limit once per device (`done`: one bit a device).
inline bool smem_limit(const void* k, int bytes, unsigned long long* done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  if (__atomic_load_n(done, __ATOMIC_ACQUIRE) >> dev & 1) return true;
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  __atomic_fetch_or(done, 1ull << dev, __ATOMIC_RELEASE);
  return true;
}
inline bool mult(int64_t v, int64_t of) { return v % of == 0; }
// The checks of dmtp_ops.h that every call makes of its cache.
int check_cache(const dmtp_paged_kv* c);
// dmtp_paged_read of a cache of E2M1 rows, its arguments checked.
cudaError_t read_e2m1(const dmtp_paged_kv* c, const int32_t* seq, const int32_t* pos, int n_rows, void* k_out,
                      void* v_out, uint32_t* err, cudaStream_t st);

}  // namespace dmtp

// ---- device ---------------------------------------------------------------------------
struct PageMap {
  const int32_t* table;
  int64_t page_stride, scale_stride, table_stride;
  int n_pages, page_size, n_kv_heads, head_dim, n_seqs, reach;  // reach: max_blocks page_size
  uint32_t div_mul;
  int div_shift;  // pos / page_size = pos div_mul >> div_shift
};
inline PageMap page_map(const dmtp_paged_kv& c) {
  // with 2^s >= page_size and m = ceil(2^(31 + s) / page_size), m page_size exceeds 2^(31 + s)
  // by less than 2^s, so pos m >> (31 + s) is exact for pos < 2^31
  int s = 0;
  while ((1 << s) < c.page_size) ++s;
  const uint64_t m = ((1ull << (31 + s)) + c.page_size - 1) / c.page_size;
  return PageMap{c.table,      c.page_stride, c.scale_stride, c.table_stride,
                 c.n_pages,    c.page_size,   c.n_kv_heads,   c.head_dim,
                 c.n_seqs,     c.max_blocks * c.page_size,    (uint32_t)m, 31 + s};
}
// Page and row in it (off) of position pos of sequence seq (pos already inside the table's
// reach); -1 and the page bit of the error word for a page that is none.
__device__ __forceinline__ int page_of(const PageMap& m, int seq, int pos, int& off, unsigned* err) {
  const int q = (int)((unsigned long long)(unsigned)pos * m.div_mul >> m.div_shift);
  off = pos - q * m.page_size;
  const int p = __ldg(m.table + (int64_t)seq * m.table_stride + q);
  if ((unsigned)p < (unsigned)m.n_pages) return p;
  set_err(err, DMTP_OPS_ERR_PAGE);
  return -1;
}

// E4M3 rows: exponent of the power-of-two scale of a row whose largest finite magnitude is
// amax. 448 = 1.75 * 2^8, so amax = f * 2^E (1 <= f < 2) takes E - 8, or E - 7 for
// f > 1.75; below 2^-126 the scale stops at the smallest normal number.
__device__ __forceinline__ int e4m3_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  if (u == 0) return 0;
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < -126 ? -126 : e;
}
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// |x| for a row's maximum: NaN and infinities do not count.
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.f;
}
// Four values as E4M3 bytes; a NaN or infinity becomes the E4M3 NaN (the conversion alone
// would saturate an infinity).
__device__ __forceinline__ uint32_t e4m3_row4(float4 v) {
  uint32_t r = e4m3x4(v);
  if (!(fabsf(v.x) <= 448.f)) r |= 0x7fu;
  if (!(fabsf(v.y) <= 448.f)) r |= 0x7f00u;
  if (!(fabsf(v.z) <= 448.f)) r |= 0x7f0000u;
  if (!(fabsf(v.w) <= 448.f)) r |= 0x7f000000u;
  return r;
}
// Two E4M3 bytes (low: first) as exact halves.
__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint32_t two) {
  uint32_t h;
  asm("{.reg .b16 a;\n\tcvt.u16.u32 a, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;}" : "=r"(h) : "r"(two));
  return h;
}
__device__ __forceinline__ float2 h2_to_f2(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ float4 e4m3x4_to_f4(uint32_t u) {
  const float2 a = h2_to_f2(e4m3x2_to_h2(u & 0xffffu)), b = h2_to_f2(e4m3x2_to_h2(u >> 16));
  return make_float4(a.x, a.y, b.x, b.y);
}

// E2M1 rows: the row's scale, as above (2688 = 6 * 448 = 1.3125 * 2^11).
__device__ __forceinline__ int e2m1_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  if (u == 0) return 0;
  const int e = (int)(u >> 23) - 127 - 11 + ((u & 0x7fffffu) > 0x280000u ? 1 : 0);
  return e < -126 ? -126 : e;
}
// Byte of a page at which the block scales begin.
__device__ __forceinline__ int64_t e2m1_blocks(const PageMap& m) {
  return (int64_t)m.n_kv_heads * m.page_size * (m.head_dim / 2);
}
__device__ __forceinline__ uint32_t e4m3_byte(float x) {
  return __nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
}
// Eight values (larger ones saturate) as E2M1, the first in the lowest bits.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}
// Eight E2M1 values as pairs of exact halves, in order.
__device__ __forceinline__ void e2m1x8_to_h2(uint32_t u, uint32_t (&h)[4]) {
  asm("{.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(u));
}
__device__ __forceinline__ void e2m1x8_to_f8(uint32_t u, float (&f)[8]) {
  uint32_t h[4];
  e2m1x8_to_h2(u, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = h2_to_f2(h[i]);
    f[2 * i] = x.x;
    f[2 * i + 1] = x.y;
  }
}

// Eight consecutive values as they lie in memory; `wide`: at a 16-byte boundary (else fp32 at
// one, bf16 at 8 bytes).
template <typename T>
struct Raw {
  uint4 u[sizeof(T) / 2];
};
__device__ __forceinline__ void fetch(const float* p, bool, Raw<float>& r) {
  r.u[0] = __ldcs(reinterpret_cast<const uint4*>(p));
  r.u[1] = __ldcs(reinterpret_cast<const uint4*>(p + 4));
}
__device__ __forceinline__ void fetch(const bf16* p, bool wide, Raw<bf16>& r) {
  if (wide) {
    r.u[0] = __ldcs(reinterpret_cast<const uint4*>(p));
  } else {
    const uint2 a = __ldcs(reinterpret_cast<const uint2*>(p)), b = __ldcs(reinterpret_cast<const uint2*>(p + 4));
    r.u[0] = make_uint4(a.x, a.y, b.x, b.y);
  }
}
__device__ __forceinline__ void values(const Raw<float>& r, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f[4 * i] = __uint_as_float(r.u[i].x);
    f[4 * i + 1] = __uint_as_float(r.u[i].y);
    f[4 * i + 2] = __uint_as_float(r.u[i].z);
    f[4 * i + 3] = __uint_as_float(r.u[i].w);
  }
}
__device__ __forceinline__ void values(const Raw<bf16>& r, float (&f)[8]) {
  const uint32_t w[4] = {r.u[0].x, r.u[0].y, r.u[0].z, r.u[0].w};
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
// 16-byte asynchronous copy global -> shared; bytes = 0 writes zeros instead.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
// The same of 16 bytes that are there, with an L2 policy.
__device__ __forceinline__ void cp_async16_hint(uint32_t dst, const void* src, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(policy)
               : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two floats in one register pair: Blackwell's packed single-precision instructions, which halve
// the issue slots of a pair of operations.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack(f32x2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 both(float a) { return pack(a, a); }
// tanh(y) to about 3e-7 of its value: near 0 y + y^3 P(y^2), P fitted to the least largest
// relative error (4e-9) on |y| <= kTanhNear; further out 1 - 2 / (1 + e^2y), whose error of 2e-7 is no
// longer large beside it.
constexpr float kTanhNear = 0.625f, kTanh3 = -0.3333328068256378f, kTanh5 = 0.13331441581249237f,
                kTanh7 = -0.05373971536755562f, kTanh9 = 0.0206390842795372f, kTanh11 = -0.005704984068870544f;
__device__ __forceinline__ float soft_tanh(float y) {
  const float t = y * y;
  const float p = fmaf(t, fmaf(t, fmaf(t, fmaf(t, kTanh11, kTanh9), kTanh7), kTanh5), kTanh3);
  const float near = fmaf(y * t, p, y);
  const float far = fmaf(-2.f, rcp(1.f + ex2(y * 2.8853900817779268f)), 1.f);
  return fabsf(y) <= kTanhNear ? near : far;
}
// The same of two values near 0, t = y^2.
__device__ __forceinline__ f32x2 tanh_near(f32x2 y, f32x2 t) {
  f32x2 p = fma2(t, both(kTanh11), both(kTanh9));
  p = fma2(t, p, both(kTanh7));
  p = fma2(t, p, both(kTanh5));
  p = fma2(t, p, both(kTanh3));
  return fma2(mul2(y, t), p, y);
}
