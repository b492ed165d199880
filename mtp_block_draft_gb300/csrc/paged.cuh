// Shared by the operators of a decode step over a paged cache (include/dmtp_ops.h):
// device-side page lookups, E4M3 row helpers, row loads, and the launch helpers.
#pragma once

#include "../../include/dmtp_ops.h"
#include "common.cuh"
#include "ops.h"

namespace dmtp {

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
