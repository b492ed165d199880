// dmtp_add_rmsnorm_e4m3: residual addition, RMS norm and E4M3 rows in one pass.
//
// One CTA per row; the row stays in registers between the sum of squares, the row maximum
// and the conversion, so each input is read once and each output written once:
// d (2 tx + ty + 1) bytes a row, which is what bounds it (a few operations a byte).
//
// The sum of squares is kept as a pair of floats (each square with its rounding error, each
// addition with its own), and 1/rms is corrected once in that precision: the factor is the
// correctly rounded one in all but about one row in 10^6, whatever the thread count, so a
// row's E4M3 values do not depend on how the sum was split.
#include "paged.cuh"

namespace {

struct F2 {  // hi + lo
  float hi, lo;
};
__device__ __forceinline__ F2 two_sum(float a, float b) {
  const float s = a + b, t = s - a;
  return F2{s, (a - (s - t)) + (b - t)};
}
__device__ __forceinline__ F2 add(F2 a, F2 b) {
  F2 s = two_sum(a.hi, b.hi);
  return F2{s.hi, s.lo + (a.lo + b.lo)};
}
__device__ __forceinline__ void add_square(F2& a, float x) {
  const float p = x * x, e = fmaf(x, x, -p);
  const F2 s = two_sum(a.hi, p);
  a.hi = s.hi;
  a.lo += s.lo + e;
}
__device__ __forceinline__ float4 gain4(const void* p, int dt, int i) {
  return dt ? load4((const bf16*)p + i) : load4((const float*)p + i);
}

template <typename TX, typename TY, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS) k_add_rmsnorm_e4m3(const dmtp_norm_args a) {
  __shared__ float2 red2[THREADS / 32];
  __shared__ float red[THREADS / 32];
  const int d4 = a.d >> 2, lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int64_t row = blockIdx.x;
  const TX* x = (const TX*)a.x + row * a.x_row;
  float4 v[NV];
  F2 ss = {0.f, 0.f};
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = threadIdx.x + k * THREADS;
    v[k] = i < d4 ? load4(x + 4 * i) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  if (a.y) {
    const TY* y = (const TY*)a.y + row * a.y_row;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = threadIdx.x + k * THREADS;
      if (i < d4) {
        const float4 w = load4(y + 4 * i);
        v[k] = make_float4(v[k].x + w.x, v[k].y + w.y, v[k].z + w.z, v[k].w + w.w);
      }
    }
  }
  if (a.x_out) {
    TX* xo = (TX*)a.x_out + row * a.xo_row;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = threadIdx.x + k * THREADS;
      if (i < d4) store_act4(xo + 4 * i, 0, v[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    add_square(ss, v[k].x);
    add_square(ss, v[k].y);
    add_square(ss, v[k].z);
    add_square(ss, v[k].w);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    ss = add(ss, F2{__shfl_xor_sync(0xffffffffu, ss.hi, o), __shfl_xor_sync(0xffffffffu, ss.lo, o)});
  if (lane == 0) red2[wid] = make_float2(ss.hi, ss.lo);
  __syncthreads();
  ss = F2{red2[0].x, red2[0].y};
#pragma unroll
  for (int w = 1; w < THREADS / 32; ++w) ss = add(ss, F2{red2[w].x, red2[w].y});
  // mean + eps as a pair: q = S / d, then the division's remainder
  const float n = (float)a.d, q0 = ss.hi / n;
  F2 ms = two_sum(q0, a.eps);
  ms.lo += (fmaf(-q0, n, ss.hi) + ss.lo) / n;
  // r ~ 1 / sqrt(ms), one Newton step on the pair: r + r (1 - ms r^2) / 2
  const float r0 = rsqrtf(ms.hi);
  const float rr = r0 * r0, rl = fmaf(r0, r0, -rr);
  const float p = ms.hi * rr;
  const float res = (1.f - p) - (fmaf(ms.hi, rr, -p) + ms.hi * rl + ms.lo * rr);
  // a sum that overflowed, or no non-zero element and eps 0: the plain value
  const float r = fabsf(res) < 0.25f ? fmaf(0.5f * r0, res, r0) : rsqrtf(ss.hi / n + a.eps);
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = threadIdx.x + k * THREADS;
    if (i < d4) {
      const float4 g = gain4(a.gain, a.gain_dtype, 4 * i);
      v[k] = make_float4(v[k].x * r * g.x, v[k].y * r * g.y, v[k].z * r * g.z, v[k].w * r * g.w);
      amax = fmaxf(amax, fmaxf(fmaxf(finite_abs(v[k].x), finite_abs(v[k].y)),
                               fmaxf(finite_abs(v[k].z), finite_abs(v[k].w))));
    }
  }
  amax = warp_max(amax);
  if (lane == 0) red[wid] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) amax = fmaxf(amax, red[w]);
  const int e = e4m3_exponent(amax);
  const float inv = pow2f(-e);
  uint8_t* q = (uint8_t*)a.q + row * a.q_row;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int i = threadIdx.x + k * THREADS;
    if (i < d4)
      *reinterpret_cast<uint32_t*>(q + 4 * i) = e4m3_row4(
          make_float4(v[k].x * inv, v[k].y * inv, v[k].z * inv, v[k].w * inv));
  }
  if (threadIdx.x == 0) a.scale[row] = pow2f(e);
}

template <typename TX, typename TY>
cudaError_t launch(const dmtp_norm_args& a, cudaStream_t st) {
  using dmtp::launch_op;
  const int d4 = a.d / 4;
#define DMTP_NORM(NV_, TH_) \
  return launch_op(k_add_rmsnorm_e4m3<TX, TY, NV_, TH_>, a.rows, TH_, 0, st, false, 1, a)
  if (d4 <= 128) DMTP_NORM(1, 128);
  if (d4 <= 256) DMTP_NORM(2, 128);
  if (d4 <= 512) DMTP_NORM(2, 256);
  if (d4 <= 1024) DMTP_NORM(4, 256);
  if (d4 <= 2048) DMTP_NORM(4, 512);
  DMTP_NORM(8, 512);
#undef DMTP_NORM
}

}  // namespace

extern "C" int dmtp_add_rmsnorm_e4m3(const dmtp_norm_args* a, void* stream) {
  if (!a || a->rows < 0) return DMTP_EINVAL;
  if (a->rows == 0) return DMTP_OK;
  if (a->d < 8 || a->d > DMTP_OPS_MAX_NORM_D || a->d % 8) return DMTP_EINVAL;
  if (a->x_dtype < 0 || a->x_dtype > 1 || a->y_dtype < 0 || a->y_dtype > 1 || a->gain_dtype < 0 ||
      a->gain_dtype > 1)
    return DMTP_EINVAL;
  if (!a->x || !a->gain || !a->q || !a->scale || (a->y && !a->x_out)) return DMTP_EINVAL;
  if (!aligned_to(a->x, 16) || !aligned_to(a->gain, 16) || !aligned_to(a->q, 8) ||
      !aligned_to(a->scale, 4) || (a->y && !aligned_to(a->y, 16)) ||
      (a->x_out && !aligned_to(a->x_out, 16)))
    return DMTP_EINVAL;
  const int64_t d = a->d;
  if (a->x_row < d || a->x_row % 8 || a->q_row < d || a->q_row % 8 ||
      (a->y && (a->y_row < d || a->y_row % 8)) || (a->x_out && (a->xo_row < d || a->xo_row % 8)))
    return DMTP_EINVAL;
  if (!(a->eps >= 0.f && a->eps <= 3.4e38f)) return DMTP_EINVAL;
  if (cudaPeekAtLastError() != cudaSuccess) return DMTP_ECUDA;
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = a->x_dtype ? (a->y_dtype ? launch<bf16, bf16>(*a, st) : launch<bf16, float>(*a, st))
                                   : (a->y_dtype ? launch<float, bf16>(*a, st) : launch<float, float>(*a, st));
  return e == cudaSuccess ? DMTP_OK : (cudaGetLastError(), DMTP_ECUDA);
}
