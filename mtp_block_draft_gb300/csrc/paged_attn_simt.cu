// Attention over a paged cache on the CUDA cores: fp32 rows, and bf16 rows of head sizes
// that the tensor-core kernel does not take.
//
// A unit is 8 queries (rows x query heads) of one kv head. A tile of 64 keys is staged in
// shared memory as it is stored (16-byte asynchronous copies, a row's page looked up by one
// thread). Each of the CTA's two warps takes 32 keys: scores with a lane per key (the K row
// read from shared memory once for all 8 queries, the queries broadcast), one maximum and
// sum per query over the warp, then O += P V with a lane per column. All arithmetic is fp32.
//
// One stage and several CTAs per SM: while one CTA computes, the others' copies are in flight.
#include <cuda_fp16.h>

#include "paged_attn.cuh"

using namespace dmtp;

namespace {

constexpr int kTK = 64, kThreads = 64, kQ = 8;

// Row pitch in shared memory: 16-byte steps of consecutive rows must fall into different
// banks, so the pitch is an odd number of 16-byte steps.
__host__ __device__ constexpr int pitch_of(int row_bytes) {
  return (row_bytes / 16) % 2 ? row_bytes : row_bytes + 16;
}
__host__ __device__ inline int smem_of(int hd, int es) {
  return 2 * kTK * pitch_of(hd * es)  // K, V
         + kQ * hd * 4                // queries
         + 2 * kQ * 32 * 4            // P of each warp
         + kQ * hd * 4                // joining the warps
         + 2 * kTK * 4                // scales
         + kTK * 8 + kQ * 8;          // row offsets, warps' statistics
}

template <typename S> struct Chunk;  // values of a 16-byte step
template <> struct Chunk<float> {
  static constexpr int E = 4;
  __device__ static void get(uint4 u, float* f) {
    f[0] = __uint_as_float(u.x), f[1] = __uint_as_float(u.y), f[2] = __uint_as_float(u.z), f[3] = __uint_as_float(u.w);
  }
};
template <> struct Chunk<bf16> {
  static constexpr int E = 8;
  __device__ static void get(uint4 u, float* f) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <> struct Chunk<uint8_t> {
  static constexpr int E = 16;
  __device__ static void get(uint4 u, float* f) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = e4m3x4_to_f4(w[i]);
      f[4 * i] = v.x, f[4 * i + 1] = v.y, f[4 * i + 2] = v.z, f[4 * i + 3] = v.w;
    }
  }
};
__device__ __forceinline__ float one(const float* p) { return *p; }
__device__ __forceinline__ float one(const bf16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float one(const uint8_t* p) { return h2_to_f2(e4m3x2_to_h2(*p)).x; }

// O += P V over a warp's 32 keys: lane has columns lane + 32 i.
template <typename S, int NI, bool GUARD>
__device__ __forceinline__ void add_pv(const float* sP, const unsigned char* sV, int pitch, int lane,
                                       int hd, float (&o)[kQ][NI]) {
  for (int k4 = 0; k4 < 32; k4 += 4) {
    float4 pq[kQ];
#pragma unroll
    for (int q = 0; q < kQ; ++q) pq[q] = *reinterpret_cast<const float4*>(sP + q * 32 + k4);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      const S* vr = (const S*)(sV + (k4 + kk) * pitch);
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int d = lane + 32 * i;
        const float x = d < hd ? one(vr + d) : 0.f;
#pragma unroll
        for (int q = 0; q < kQ; ++q) {
          const float pw = kk == 0 ? pq[q].x : kk == 1 ? pq[q].y : kk == 2 ? pq[q].z : pq[q].w;
          const float r = fmaf(pw, x, o[q][i]);
          o[q][i] = GUARD && pw == 0.f ? o[q][i] : r;
        }
      }
    }
  }
}

// T: type of q and out; S: stored type (uint8_t: E4M3); NI: columns of a lane.
template <typename T, typename S, int NI>
__global__ void __launch_bounds__(kThreads) k_paged_attn_simt(const PagedAttn p) {
  extern __shared__ __align__(16) unsigned char smem[];
  pdl_trigger();
  const int hd = p.m.head_dim, rb = hd * (int)sizeof(S), pitch = pitch_of(rb), ch = rb / 16;
  unsigned char* sK = smem;
  unsigned char* sV = sK + kTK * pitch;
  float* sQ = (float*)(sV + kTK * pitch);
  float* sO = sQ + kQ * hd;
  float* sP = sO + kQ * hd;
  float* sS = sP + 2 * kQ * 32;
  int64_t* sRow = (int64_t*)(sS + 2 * kTK);
  float2* sML = (float2*)(sRow + kTK);
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  Deal deal;
  Tiles w = my_tiles<T>(p, deal, kThreads);

  while (w.pos < w.end) {
    const int len = w.len, first = w.first, n = w.n, unit = w.unit, t0 = w.t;
    const int t1 = min(n, t0 + w.end - w.pos);
    const int kvh = unit / p.chunks, nq = queries_of(p, unit);
    for (int i = tid; i < kQ * hd; i += kThreads) {
      const int t = i / hd, d = i - t * hd;
      float x = 0.f;
      if (t < nq) {
        int head, row;
        query_of(p, unit, t, &head, &row);
        x = to_f32(((const T*)p.a.q)[(int64_t)w.b * p.a.q_seq + (int64_t)row * p.a.q_row +
                                     (int64_t)head * p.a.q_head + d]);
      }
      sQ[i] = x;
    }
    float m[kQ], l[kQ], o[kQ][NI];
    int top[kQ];  // last position that a query's row sees
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
      m[q] = -INFINITY;
      l[q] = 0.f;
      int head, row;
      query_of(p, unit, q, &head, &row);
      top[q] = q < nq ? len - p.a.rows + row : -1;
#pragma unroll
      for (int i = 0; i < NI; ++i) o[q][i] = 0.f;
    }
    for (int t = t0; t < t1; ++t) {
      const int j0 = first + t * kTK;
      __syncthreads();  // the last tile has been used
      {
        const int j = j0 + tid;
        int64_t at = -1, line = 0;
        if (j < len && j >= seq_low(p, len)) {
          int off;
          const int page = page_of(p.m, w.b, j, off, p.err);
          line = (int64_t)kvh * p.m.page_size + off;
          if (page >= 0) {
            at = (int64_t)page * p.m.page_stride + line * hd;
            line += (int64_t)page * p.m.scale_stride;
          }
        }
        sRow[tid] = at;
        if (sizeof(S) == 1) {
          sS[tid] = at >= 0 ? p.ks[line] : 0.f;
          sS[kTK + tid] = at >= 0 ? p.vs[line] : 0.f;
        }
      }
      __syncthreads();
      for (int i = tid; i < kTK * ch; i += kThreads) {
        const int r = i / ch, c = i - r * ch;
        const int64_t at = sRow[r];
        const int bytes = at >= 0 ? 16 : 0;
        const int64_t src = (at >= 0 ? at * (int)sizeof(S) + c * 16 : 0);
        cp_async16(smem_u32(sK + r * pitch + c * 16), (const char*)p.k + src, bytes);
        cp_async16(smem_u32(sV + r * pitch + c * 16), (const char*)p.v + src, bytes);
      }
      cp_async_commit();
      cp_async_wait<0>();
      __syncthreads();
      const int key = wid * 32 + lane, j = j0 + key;
      float s[kQ];
#pragma unroll
      for (int q = 0; q < kQ; ++q) s[q] = 0.f;
      constexpr int E = Chunk<S>::E;
      for (int c = 0; c < ch; ++c) {
        float f[E];
        Chunk<S>::get(*reinterpret_cast<const uint4*>(sK + key * pitch + c * 16), f);
#pragma unroll
        for (int q = 0; q < kQ; ++q)
#pragma unroll
          for (int i = 0; i < E; i += 4) {
            const float4 x = *reinterpret_cast<const float4*>(sQ + q * hd + c * E + i);
            s[q] = fmaf(x.x, f[i], fmaf(x.y, f[i + 1], fmaf(x.z, f[i + 2], fmaf(x.w, f[i + 3], s[q]))));
          }
      }
      const bool there = sRow[key] >= 0;
      const float f = sizeof(S) == 1 ? sS[key] * p.scale2 : p.scale2;
      const float vs = sizeof(S) == 1 ? sS[kTK + key] : 1.f;
#pragma unroll
      for (int q = 0; q < kQ; ++q) {
        const bool seen = there && j <= top[q] && (p.a.window <= 0 || j > top[q] - p.a.window);
        const float x = seen ? s[q] * f : -INFINITY;
        const float mn = fmaxf(m[q], warp_max(x));
        const float ref = mn == -INFINITY ? 0.f : mn;
        const float pw = seen ? ex2(x - ref) : 0.f, fix = ex2(m[q] - ref);
        l[q] = fmaf(l[q], fix, pw);
        m[q] = mn;
#pragma unroll
        for (int i = 0; i < NI; ++i) o[q][i] *= fix;
        sP[(wid * kQ + q) * 32 + lane] = pw * vs;
      }
      __syncwarp();
      // A position that only some of the rows see may hold an infinity or a NaN, which a
      // weight of zero would turn into a NaN: those tiles leave zero weights out.
      const bool edge = j0 + kTK > len - p.a.rows || (p.a.window > 0 && j0 < len - p.a.window);
      if (edge)
        add_pv<S, NI, true>(sP + wid * kQ * 32, sV + wid * 32 * pitch, pitch, lane, hd, o);
      else
        add_pv<S, NI, false>(sP + wid * kQ * 32, sV + wid * 32 * pitch, pitch, lane, hd, o);
      __syncwarp();
    }
    // join the two warps: warp 1 leaves its state, warp 0 adds it and writes
    if (wid == 1) {
#pragma unroll
      for (int q = 0; q < kQ; ++q) {
        const float lq = warp_sum(l[q]);
        if (lane == 0) sML[q] = make_float2(m[q], lq);
#pragma unroll
        for (int i = 0; i < NI; ++i)
          if (lane + 32 * i < hd) sO[q * hd + lane + 32 * i] = o[q][i];
      }
    }
    __syncthreads();
    if (wid == 0) {
      const bool whole = t0 == 0 && t1 == n;
#pragma unroll
      for (int q = 0; q < kQ; ++q) {
        const float lq = warp_sum(l[q]);
        const float2 other = sML[q];
        const float M = fmaxf(m[q], other.x), ref = M == -INFINITY ? 0.f : M;
        const float fa = ex2(m[q] - ref), fb = ex2(other.x - ref);
        const float L = lq * fa + other.y * fb;
        if (q < nq) {
          int head, row;
          query_of(p, unit, q, &head, &row);
          T* out = (T*)p.a.out + (int64_t)w.b * p.a.o_seq + (int64_t)row * p.a.o_row + (int64_t)head * p.a.o_head;
          const int at = ((int)blockIdx.x * 2 + (t0 == 0)) * p.qn + q;
          const float inv = L != 0.f ? 1.f / L : 0.f;
#pragma unroll
          for (int i = 0; i < NI; ++i) {
            const int d = lane + 32 * i;
            if (d < hd) {
              const float x = o[q][i] * fa + sO[q * hd + d] * fb;
              if (whole)
                out[d] = from_f32<T>(x * inv);
              else
                p.part_o[(int64_t)at * hd + d] = x;
            }
          }
          if (!whole && lane == 0) p.part_ml[at] = make_float2(M, L);
        }
      }
    }
    if (t0 == 0 && tid == 0) leave_note(p, deal, w);
    w.skip(p, t1 - t0);
    __syncthreads();
  }
}

template <typename T, typename S, int NI>
cudaError_t launch_ni(const PagedAttn& p, int grid, cudaStream_t st) {
  static unsigned long long done = 0;
  auto k = k_paged_attn_simt<T, S, NI>;
  if (!smem_limit((const void*)k, smem_of(NI * 32, sizeof(S)), &done)) return cudaErrorInvalidValue;
  return launch_op(k, grid, kThreads, smem_of(p.m.head_dim, sizeof(S)), st, false, 1, p);
}
template <typename T, typename S>
cudaError_t launch_t(const PagedAttn& p, int grid, cudaStream_t st) {
  const int hd = p.m.head_dim;
  if (hd <= 32) return launch_ni<T, S, 1>(p, grid, st);
  if (hd <= 64) return launch_ni<T, S, 2>(p, grid, st);
  if (hd <= 96) return launch_ni<T, S, 3>(p, grid, st);
  if (hd <= 128) return launch_ni<T, S, 4>(p, grid, st);
  return launch_ni<T, S, 8>(p, grid, st);
}

}  // namespace

namespace dmtp {

int paged_simt_grid(int head_dim, int dtype, bool e8) {
  // CTAs of an SM by shared memory (227 KB, 1 KB of it each CTA's own), at most 8
  const int per = 227 * 1024 / (smem_of(head_dim, e8 ? 1 : dtype ? 2 : 4) + 1024);
  return 152 * (per < 1 ? 1 : per > 8 ? 8 : per);
}

cudaError_t paged_attn_simt(const PagedAttn& p, const PagedPlan& pl, int dtype, bool e8, cudaStream_t st) {
  if (e8) return dtype ? launch_t<bf16, uint8_t>(p, pl.grid, st) : launch_t<float, uint8_t>(p, pl.grid, st);
  return dtype ? launch_t<bf16, bf16>(p, pl.grid, st) : launch_t<float, float>(p, pl.grid, st);
}

}  // namespace dmtp
