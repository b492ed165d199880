// Attention of many rows over a paged cache on the CUDA cores: fp32 rows, and bf16 rows that the
// tensor-core kernel does not take.
//
// A CTA of 256 threads has a tile of 64 queries and goes through the keys 64 (heads over 128
// columns: 32) at a time, Q, K and V as fp32 in shared memory. A thread has 4 queries: of the
// scores with 4 keys, of the output with a sixteenth of the columns: per four columns and key pair of
// loads 64 fused operations, two an instruction (sums over even and odd columns, two columns of the
// output), so the fp32 pipes bound it: 64 fp32 rows of 32 / 4 heads of 128 over 16384 positions 469 us
// (one an instruction 505), 2048 rows 1.08 ms, 32 TFLOP/s with what the causal blocks waste. (16384
// bf16 rows, which the tensor cores take, took 66 ms here.)
#include <type_traits>

#include "paged_prompt.cuh"

using namespace dmtp;

namespace {

constexpr int kThreads = 256, kTile = 64;

template <int HDM>
struct Shape {
  static constexpr int TK = HDM > 128 ? 32 : 64, KJ = TK / 16, CJ = HDM / 64;
  static __host__ __device__ constexpr int pitch(int hd) { return hd + 4; }
  static constexpr int kP = TK + 4;
  // floats of K's place, which the weights take after it
  static __host__ __device__ constexpr int keys(int hd) {
    return TK * pitch(hd) > kTile * kP ? TK * pitch(hd) : kTile * kP;
  }
  static __host__ __device__ constexpr int smem(int hd) {
    return (kTile + TK) * pitch(hd) * 4 + keys(hd) * 4 + TK * 16;
  }
};

template <typename T, Rows F, int HDM>
__global__ void __launch_bounds__(kThreads, HDM > 128 ? 1 : 2) k_prompt_simt(const PagedPrompt p) {
  using Sh = Shape<HDM>;
  constexpr int TK = Sh::TK, KJ = Sh::KJ, CJ = Sh::CJ, PP = Sh::kP;
  extern __shared__ __align__(16) float smem[];
  __shared__ int s_lo[kThreads / 32], s_hi[kThreads / 32];
  pdl_trigger();
  if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x < 32) prompt_report(p);
  PromptTile w;
  if (!prompt_tile(p, blockIdx.x, w)) return;
  const int hd = p.m.head_dim, pitch = Sh::pitch(hd), kvh = blockIdx.y, tid = threadIdx.x;
  const int tx = tid & 15, ty = tid >> 4;
  float *sQ = smem, *sK = sQ + kTile * pitch, *sV = sK + Sh::keys(hd);
  float* sP = sK;  // the weights, once the scores are done with K
  int64_t* s_line = (int64_t*)(sV + TK * pitch);  // a key's page (-1: it is not there)
  int* s_in = (int*)(s_line + TK);                // and its row in the page
  // the queries
  for (int i = tid; i < kTile * (hd / 8); i += kThreads) {
    const int t = i / (hd / 8), c = (i - t * (hd / 8)) * 8;
    float f[8] = {};
    if (t < w.count) {
      const int r = (w.q0 + t) / p.group, head = kvh * p.group + (w.q0 + t - r * p.group);
      const T* src = (const T*)p.a.q + (int64_t)(w.row0 + r) * p.a.q_row + (int64_t)head * p.a.q_head + c;
      Raw<T> raw;
#pragma unroll
      for (int x = 0; x < (int)(sizeof(T) / 2); ++x) raw.u[x] = __ldg(reinterpret_cast<const uint4*>(src) + x);
      values(raw, f);
    }
    *reinterpret_cast<float4*>(sQ + t * pitch + c) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(sQ + t * pitch + c + 4) = make_float4(f[4], f[5], f[6], f[7]);
  }
  int lo[4], hi[4], pos[4], least = 0x7fffffff, most = 0;
  float slope[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lo[i] = hi[i] = pos[i] = 0;
    slope[i] = 0.f;
    if (4 * ty + i < w.count) {
      const PromptQuery q = prompt_query(p, w, 4 * ty + i);
      lo[i] = q.lo;
      hi[i] = q.hi;
      pos[i] = q.pos;
      if (p.a.scores.slopes) slope[i] = __ldg(p.a.scores.slopes + kvh * p.group + q.head) * 1.4426950408889634f;
      if (q.lo < q.hi) {
        least = min(least, q.lo);
        most = max(most, q.hi);
      }
    }
  }
  least = __reduce_min_sync(0xffffffffu, least);
  most = __reduce_max_sync(0xffffffffu, most);
  if ((tid & 31) == 0) {
    s_lo[tid >> 5] = least;
    s_hi[tid >> 5] = most;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    least = min(least, s_lo[i]);
    most = max(most, s_hi[i]);
  }
  const int j_first = least < most ? least / TK : 0, tiles = least < most ? (most + TK - 1) / TK - j_first : 0;
  const int t0 = (int)((int64_t)tiles * blockIdx.z / p.splits), t1 = (int)((int64_t)tiles * (blockIdx.z + 1) / p.splits);

  f32x2 o[4][CJ][2];  // two columns each
  float m[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < CJ; ++c) o[i][c][0] = o[i][c][1] = 0ull;
  }
  for (int t = t0; t < t1; ++t) {
    const int j0 = (j_first + t) * TK;
    if (tid < TK) {
      const int j = j0 + tid;
      int off = 0, page = -1;
      if (j >= least && j < most) page = page_of(p.m, w.b, j, off, p.err);
      s_line[tid] = page;
      s_in[tid] = off;
    }
    __syncthreads();
    bool odd = false;  // a value that is not finite
    for (int i = tid; i < TK * (hd / 8); i += kThreads) {
      const int r = i / (hd / 8), c = (i - r * (hd / 8)) * 8;
      float a[8] = {}, b[8] = {};
      const int64_t page = s_line[r];
      if (page >= 0) {
        const int64_t line = (int64_t)kvh * p.m.page_size + s_in[r];
        const float fk = F == kRaw ? 1.f : __ldg(p.ks + page * p.m.scale_stride + line);
        const float fv = F == kRaw ? 1.f : __ldg(p.vs + page * p.m.scale_stride + line);
        load8<T, F>(p, p.k, page, line, c, fk, a);
        load8<T, F>(p, p.v, page, line, c, fv, b);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) odd = odd || !(fabsf(b[e]) <= 3.402823466e38f);
      *reinterpret_cast<float4*>(sK + r * pitch + c) = make_float4(a[0], a[1], a[2], a[3]);
      *reinterpret_cast<float4*>(sK + r * pitch + c + 4) = make_float4(a[4], a[5], a[6], a[7]);
      *reinterpret_cast<float4*>(sV + r * pitch + c) = make_float4(b[0], b[1], b[2], b[3]);
      *reinterpret_cast<float4*>(sV + r * pitch + c + 4) = make_float4(b[4], b[5], b[6], b[7]);
    }
    odd = __syncthreads_or(odd);
    float s[4][KJ];
    {
      f32x2 s2[4][KJ];  // the sums over even and over odd columns
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < KJ; ++j) s2[i][j] = 0ull;
#pragma unroll 2
      for (int d = 0; d < hd; d += 4) {
        ulonglong2 a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const ulonglong2*>(sQ + (4 * ty + i) * pitch + d);
#pragma unroll
        for (int j = 0; j < KJ; ++j) {
          const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(sK + (tx + 16 * j) * pitch + d);
#pragma unroll
          for (int i = 0; i < 4; ++i) s2[i][j] = fma2(a[i].y, b.y, fma2(a[i].x, b.x, s2[i][j]));
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < KJ; ++j) {
          const float2 x = unpack(s2[i][j]);
          s[i][j] = x.x + x.y;
        }
    }
    __syncthreads();  // K has been read: its place takes the weights
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < KJ; ++j) {
        const int key = tx + 16 * j, at = j0 + key;
        float x = s[i][j] * p.scale2;
        if (p.capl > 0.f) x = p.capl * soft_tanh(x * p.cap_inv);
        x = fmaf(-slope[i], (float)abs(pos[i] - at), x);
        const bool seen = at >= lo[i] && at < hi[i] && s_line[key] >= 0;
        s[i][j] = seen ? x : -INFINITY;
        top = fmaxf(top, s[i][j]);
      }
#pragma unroll
      for (int k = 1; k < 16; k <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
      const float n = fmaxf(m[i], top), ref = n == -INFINITY ? 0.f : n, fix = ex2(m[i] - ref);
      m[i] = n;
      l[i] *= fix;
#pragma unroll
      for (int c = 0; c < CJ; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e) o[i][c][e] = mul2(o[i][c][e], both(fix));
#pragma unroll
      for (int j = 0; j < KJ; ++j) {
        const float x = ex2(s[i][j] - ref);
        l[i] += x;
        sP[(4 * ty + i) * PP + tx + 16 * j] = x;
      }
    }
    __syncthreads();
    if (!odd) {
#pragma unroll 2
      for (int k = 0; k < TK; k += 4) {
        float x[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 v = *reinterpret_cast<const float4*>(sP + (4 * ty + i) * PP + k);
          x[i][0] = v.x, x[i][1] = v.y, x[i][2] = v.z, x[i][3] = v.w;
        }
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
          for (int c = 0; c < CJ; ++c) {
            const int d = 64 * c + 4 * tx;
            if (d >= hd) break;
            const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(sV + (k + y) * pitch + d);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              o[i][c][0] = fma2(both(x[i][y]), v.x, o[i][c][0]);
              o[i][c][1] = fma2(both(x[i][y]), v.y, o[i][c][1]);
            }
          }
      }
    } else {  // a weight of zero leaves a value that is not finite out
#pragma unroll 1
      for (int k = 0; k < TK; ++k)
#pragma unroll
        for (int c = 0; c < CJ; ++c) {
          const int d = 64 * c + 4 * tx;
          if (d >= hd) break;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x = sP[(4 * ty + i) * PP + k];
            if (x != 0.f) {
              const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(sV + k * pitch + d);
              o[i][c][0] = fma2(both(x), v.x, o[i][c][0]);
              o[i][c][1] = fma2(both(x), v.y, o[i][c][1]);
            }
          }
        }
    }
    __syncthreads();  // the tiles are free again
  }
  const int64_t part = (((int64_t)blockIdx.x * gridDim.y + kvh) * p.splits + blockIdx.z) * kTile;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int k = 1; k < 16; k <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], k);
    const int t = 4 * ty + i;
    if (t >= w.count) continue;
    if (p.splits > 1) {
      if (tx == 0) p.part_ml[part + t] = make_float2(m[i], l[i]);
#pragma unroll
      for (int c = 0; c < CJ; ++c)
        if (64 * c + 4 * tx < hd)
          *reinterpret_cast<ulonglong2*>(p.part_o + (part + t) * hd + 64 * c + 4 * tx) = make_ulonglong2(o[i][c][0], o[i][c][1]);
      continue;
    }
    const int r = (w.q0 + t) / p.group, head = kvh * p.group + (w.q0 + t - r * p.group);
    T* out = (T*)p.a.out + (int64_t)(w.row0 + r) * p.a.o_row + (int64_t)head * p.a.o_head;
    const float inv = l[i] != 0.f ? 1.f / l[i] : 0.f;
#pragma unroll
    for (int c = 0; c < CJ; ++c)
      if (64 * c + 4 * tx < hd) {
        const float2 x = unpack(mul2(o[i][c][0], both(inv))), y = unpack(mul2(o[i][c][1], both(inv)));
        store_act4(out + 64 * c + 4 * tx, 0, make_float4(x.x, x.y, y.x, y.y));
      }
  }
}

template <typename T, Rows F, int HDM>
cudaError_t launch_m(const PagedPrompt& p, const PromptPlan& pl, cudaStream_t st) {
  static unsigned long long done = 0;
  auto k = k_prompt_simt<T, F, HDM>;
  if (!smem_limit((const void*)k, Shape<HDM>::smem(HDM), &done)) return cudaErrorInvalidValue;
  const dim3 grid(pl.tiles, p.m.n_kv_heads, pl.splits);
  return launch_op(k, grid, kThreads, Shape<HDM>::smem(p.m.head_dim), st, false, 1, p);
}
template <typename T, Rows F>
cudaError_t launch_t(const PagedPrompt& p, const PromptPlan& pl, cudaStream_t st) {
  const int hd = p.m.head_dim;
  return hd <= 64 ? launch_m<T, F, 64>(p, pl, st) : hd <= 128 ? launch_m<T, F, 128>(p, pl, st) : launch_m<T, F, 256>(p, pl, st);
}

}  // namespace

namespace dmtp {

cudaError_t paged_prompt_simt(const PagedPrompt& p, const PromptPlan& pl, int dtype, Rows f, cudaStream_t st) {
  if (f == kE2M1) return dtype ? launch_t<bf16, kE2M1>(p, pl, st) : launch_t<float, kE2M1>(p, pl, st);
  if (f == kE4M3) return dtype ? launch_t<bf16, kE4M3>(p, pl, st) : launch_t<float, kE4M3>(p, pl, st);
  return dtype ? launch_t<bf16, kRaw>(p, pl, st) : launch_t<float, kRaw>(p, pl, st);
}

}  // namespace dmtp
