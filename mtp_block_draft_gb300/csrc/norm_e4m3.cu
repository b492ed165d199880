// dmtp_add_rmsnorm_e4m3: residual addition, RMS norm and E4M3 rows in one pass.
//
// One CTA at a row; the row stays in registers between the sum of squares, the row maximum
// and the conversion, so each input is read once and each output written once:
// d (2 tx + ty + 1) bytes a row, which is what bounds it (a few operations a byte).
//
// The sum of squares carries its rounding errors along (about 2^-30 of it is lost), and 1/rms is
// corrected once in that precision: the factor is the correctly rounded one but for the last
// bit of about one row in a hundred, so a row's E4M3 values hardly depend on how the sum was
// split. Sixteen values a thread, so that what every thread does once per row (the reductions,
// the factor) stays below what it does per value
// (with few rows eight, see launch()).
//
// 8188 rows of 2048 bf16 take 22.9 us (117 MB, 0.75 of the copy rate; 70% of the issue slots used),
// 32 rows of fp32 2.6 us, which is latency.
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
// hi += x^2, the part of it that the sum's rounding loses carried over to the next one.
__device__ __forceinline__ void add_squares(f32x2& hi, f32x2& carry, f32x2 x, f32x2 minus) {
  const f32x2 y = fma2(x, x, carry), s = add2(hi, y);
  carry = fma2(fma2(hi, minus, s), minus, y);  // y - (s - hi)
  hi = s;
}
// CTAs of an SM: what the registers of a row and the next one allow. Measured on 8188 rows of
// 2048 bf16 values: 512, 768, 1024, 1280, 1536 threads an SM 28.0, 24.5, 22.7, 26.4, 30.0 us.
template <typename TX, typename TY, int NV, int THREADS>
constexpr int ctas_of() {
  return NV == 4 ? 1 : THREADS > 384 ? (sizeof(TX) + sizeof(TY) <= 4 ? 2 : 1) : (sizeof(TX) + sizeof(TY) <= 4 ? 1024 : 768) / THREADS;
}

// NV: eights of a thread. A CTA takes every gridDim.x-th row and asks for the next one's values
// before it works on the one it has, so the reductions' barriers do not leave the memory idle.
template <typename TX, typename TY, int NV, int THREADS>
__global__ void __launch_bounds__(THREADS, ctas_of<TX, TY, NV, THREADS>()) k_add_rmsnorm_e4m3(const dmtp_norm_args a) {
  __shared__ float2 red2[2][THREADS / 32];
  __shared__ uint32_t red[2][THREADS / 32];
  const int d8 = a.d >> 3, lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  Raw<TX> rx[NV];
  Raw<TY> ry[NV];
  auto ask = [&](int64_t row) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = threadIdx.x + k * THREADS;
      if (i < d8) {
        fetch((const TX*)a.x + row * a.x_row + 8 * i, true, rx[k]);
        if (a.y) fetch((const TY*)a.y + row * a.y_row + 8 * i, true, ry[k]);
      }
    }
  };
  ask(blockIdx.x);
  const float rn = 1.f / (float)a.d;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    float v[NV][8];
    const f32x2 minus = pack(-1.f, -1.f);
    f32x2 hi2 = 0ull, lo2 = 0ull;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = threadIdx.x + k * THREADS;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[k][e] = 0.f;
      if (i < d8) {
        values(rx[k], v[k]);
        if (a.y) {
          float w[8];
          values(ry[k], w);
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const float2 s = unpack(add2(pack(v[k][e], v[k][e + 1]), pack(w[e], w[e + 1])));
            v[k][e] = s.x;
            v[k][e + 1] = s.y;
          }
        }
      }
    }
    if (row + gridDim.x < a.rows) ask(row + gridDim.x);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = threadIdx.x + k * THREADS;
      if (a.x_out && i < d8) store8((TX*)a.x_out + row * a.xo_row + 8 * i, true, v[k]);
#pragma unroll
      for (int e = 0; e < 8; e += 2) add_squares(hi2, lo2, pack(v[k][e], v[k][e + 1]), minus);
    }
    const float2 h2 = unpack(hi2), l2 = unpack(lo2);
    F2 ss = add(F2{h2.x, l2.x}, F2{h2.y, l2.y});
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      ss = add(ss, F2{__shfl_xor_sync(0xffffffffu, ss.hi, o), __shfl_xor_sync(0xffffffffu, ss.lo, o)});
    if (THREADS > 32) {
      if (lane == 0) red2[turn][wid] = make_float2(ss.hi, ss.lo);
      __syncthreads();
      const float2 part = red2[turn][lane % (THREADS / 32)];
      ss = F2{part.x, part.y};
#pragma unroll
      for (int o = THREADS / 64; o > 0; o >>= 1)
        ss = add(ss, F2{__shfl_xor_sync(0xffffffffu, ss.hi, o), __shfl_xor_sync(0xffffffffu, ss.lo, o)});
    }
    if (!(ss.hi <= 3.402823466e38f)) {
      // an infinity or NaN (or squares past fp32): what the sum carries along, infinity less infinity,
      // made it a NaN if anything came after. The plain sum tells the two apart: next to an
      // infinity finite values become 0, next to a NaN all are NaN.
      float plain = 0.f;
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) plain = fmaf(v[k][e], v[k][e], plain);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) plain += __shfl_xor_sync(0xffffffffu, plain, o);
      if (THREADS > 32) {
        __syncthreads();
        if (lane == 0) red2[turn][wid].x = plain;
        __syncthreads();
        plain = 0.f;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) plain += red2[turn][w].x;
      }
      ss = F2{plain, 0.f};
    }
    // mean + eps as a pair: S / d by the reciprocal, then the quotient's remainder
    const float n = (float)a.d, q0 = ss.hi * rn;
    F2 ms = two_sum(q0, a.eps);
    ms.lo += (fmaf(-q0, n, ss.hi) + ss.lo) * rn;
    // r ~ 1 / sqrt(ms), one Newton step on the pair: r + r (1 - ms r^2) / 2
    const float r0 = rsqrtf(ms.hi);
    const float rr = r0 * r0, rl = fmaf(r0, r0, -rr);
    const float p = ms.hi * rr;
    const float res = (1.f - p) - (fmaf(ms.hi, rr, -p) + ms.hi * rl + ms.lo * rr);
    // an infinite sum, or no non-zero element and eps 0: the plain value
    const float r = fabsf(res) < 0.25f ? fmaf(0.5f * r0, res, r0) : rsqrtf(ss.hi / n + a.eps);
    const f32x2 r2 = pack(r, r);
    uint32_t top = 0;  // largest magnitude, as bits: an infinity or NaN is above every number
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = threadIdx.x + k * THREADS;
      if (i < d8) {
        float g[8];
        if (a.gain_dtype)
          values(Raw<bf16>{__ldg((const uint4*)a.gain + i)}, g);
        else
          values(Raw<float>{__ldg((const uint4*)a.gain + 2 * i), __ldg((const uint4*)a.gain + 2 * i + 1)}, g);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float2 h = unpack(mul2(mul2(pack(v[k][e], v[k][e + 1]), r2), pack(g[e], g[e + 1])));
          v[k][e] = h.x;
          v[k][e + 1] = h.y;
          top = max(top, max(__float_as_uint(h.x) & 0x7fffffffu, __float_as_uint(h.y) & 0x7fffffffu));
        }
      }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (THREADS > 32) {
      if (lane == 0) red[turn][wid] = top;
      __syncthreads();
      top = __reduce_max_sync(0xffffffffu, red[turn][lane % (THREADS / 32)]);
    }
    const bool odd = top >= 0x7f800000u;
    if (odd) {  // the scale goes by the finite values
      uint32_t t = 0;
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (threadIdx.x + k * THREADS < d8) t = max(t, __float_as_uint(finite_abs(v[k][e])));
      t = __reduce_max_sync(0xffffffffu, t);
      __syncthreads();
      if (lane == 0) red[turn][wid] = t;
      __syncthreads();
      top = 0;
#pragma unroll
      for (int w = 0; w < THREADS / 32; ++w) top = max(top, red[turn][w]);
    }
    const int e = e4m3_exponent(__uint_as_float(top));
    const float inv = pow2f(-e);
    uint8_t* q = (uint8_t*)a.q + row * a.q_row;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = threadIdx.x + k * THREADS;
      const float (&f)[8] = v[k];
      const float4 lo = make_float4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
      const float4 hi = make_float4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv);
      if (i < d8)
        *reinterpret_cast<uint2*>(q + 8 * i) =
            odd ? make_uint2(e4m3_row4(lo), e4m3_row4(hi)) : make_uint2(e4m3x4(lo), e4m3x4(hi));
    }
    if (threadIdx.x == 0) a.scale[row] = pow2f(e);
  }
}

template <typename TX, typename TY>
cudaError_t launch(const dmtp_norm_args& a, cudaStream_t st) {
  using dmtp::launch_op;
  const int d8 = a.d / 8;
  auto grid = [&](int ctas) { return a.rows < 152 * ctas ? a.rows : 152 * ctas; };
#define DMTP_NORM(NV_, TH_) \
  return launch_op(k_add_rmsnorm_e4m3<TX, TY, NV_, TH_>, grid(ctas_of<TX, TY, NV_, TH_>()), TH_, 0, st, false, 1, a)
  // A CTA an SM and less: eight values a thread, the row's latency counts. More: sixteen. us, eight /
  // sixteen: 64 rows of 2048 bf16 2.5 / 2.8, 152 2.6 / 3.0, 608 3.7 / 3.4, 8188 25.3 / 23.1; of 4096
  // fp32, 64 rows 3.1 / 3.3, 152 3.15 / 3.3, 304 4.7 / 4.2, 8188 77.7 / 69.3; of 8192 bf16, 32 rows
  // 4.9 (with 1024 threads) / 3.5.
  if (a.rows <= 152) {
    if (d8 > 32 && d8 <= 64) DMTP_NORM(1, 64);
    if (d8 > 64 && d8 <= 128) DMTP_NORM(1, 128);
    if (d8 > 128 && d8 <= 256) DMTP_NORM(1, 256);
    if (d8 > 256 && d8 <= 512) DMTP_NORM(1, 512);
  }
  if (d8 <= 32) DMTP_NORM(1, 32);
  if (d8 <= 64) DMTP_NORM(2, 32);
  if (d8 <= 128) DMTP_NORM(2, 64);
  if (d8 <= 256) DMTP_NORM(2, 128);
  if (d8 <= 512) DMTP_NORM(2, 256);
  if (d8 <= 1024) DMTP_NORM(2, 512);
  DMTP_NORM(4, 512);
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
