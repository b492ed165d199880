// Attention over a paged cache on the CUDA cores: fp32 rows, and bf16 rows of head sizes
// that the tensor-core kernel does not take.
//
// A unit is 8 queries (rows x query heads) of one kv head. A CTA's four warps take 16 keys each of
// a tile of 64, four at a time: a lane has four columns (hd > 128: twice four) of the four K rows
// and of the eight queries, so the rows come by copies of whole lines into a ring of the warp's
// own, and a lane reads back only what it brought. The 32 products (4 keys x 8 queries) are summed
// over the lanes so that each lane ends up with one of them: 31 exchanges instead of 160. Then one
// exponential a lane serves all of them, and O += P V runs on the same columns with the weights
// broadcast from shared memory. Heads of 64 or 32 columns leave lanes over: half or a quarter of
// the warp takes a row, and the warp eight or sixteen keys at a time. All arithmetic is fp32, two
// queries an instruction.
//
// What bounds it is issue: about 175 instructions a key row and 8 queries (61% of the issue slots
// at three CTAs an SM), of which 64 are the products. 32 sequences of 512 to 4096 positions, 4 kv
// heads of 128, 8 queries each: fp32 74.6 us (0.60 of the copy rate), 64 queries (eight passes over
// the rows, seven of them from L2) 512 us; bf16 heads of 96 74 us, of 32 34 us; 2 kv heads of 256
// 130 us. With a lane per key and the rows staged for the CTA, one stage at a time, those took 147,
// 954, 70, 33 and 220 us. Bf16 heads of 128 take 92 us and with 64 queries 520 us that way, on the
// tensor cores 30 and 72: they are left to those.
#include <cuda_fp16.h>

#include "paged_attn.cuh"

using namespace dmtp;

namespace {

constexpr int kThreads = 128, kWarps = 4, kQ = 8;

template <typename S, int C, int H>
struct Shape {
  static constexpr int VB = 4 * (int)sizeof(S);              // bytes of a lane's four columns
  static constexpr int kRows = 2 * 4 * C * 32 * VB;          // a stage: four H rows of K and of V,
  static constexpr int kStage = kRows + 32 * H + 16;         // their scales, and which are there
  static constexpr int NST = kRows > 4096 ? 3 : 16384 / kRows > 8 ? 8 : 16384 / kRows;
  static constexpr int CTAS = C == 1 ? 3 : 2;                // registers: 168 or 255 a thread
  static __host__ __device__ int smem(int hd) {
    return kWarps * NST * kStage + kWarps * 32 * H * 4 + kQ * hd * 4 + kWarps * kQ * 8;
  }
};

__device__ __forceinline__ void get4(const float* p, float (&f)[4]) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
}
__device__ __forceinline__ void get4(const bf16* p, float (&f)[4]) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  f[0] = __uint_as_float(u.x << 16), f[1] = __uint_as_float(u.x & 0xffff0000u);
  f[2] = __uint_as_float(u.y << 16), f[3] = __uint_as_float(u.y & 0xffff0000u);
}
__device__ __forceinline__ void get4(const uint8_t* p, float (&f)[4]) {
  const float4 v = e4m3x4_to_f4(*reinterpret_cast<const uint32_t*>(p));
  f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
}
template <int VB>
__device__ __forceinline__ void copy(uint32_t dst, const void* src, int bytes) {
  if (VB == 16)
    cp_async16(dst, src, bytes);
  else if (VB == 8)
    cp_async8(dst, src, bytes);
  else
    cp_async4(dst, src, bytes);
}
// Lane n of a group of 32 / H gets v[n H + x], x < H, summed over the group, as v[x].
template <int H>
__device__ __forceinline__ void sum_to_lane(float (&v)[32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o >= H; o >>= 1) {
    const bool up = lane & o / H;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float keep = up ? v[i + o] : v[i], give = up ? v[i] : v[i + o];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o / H);
    }
  }
}

// T: type of q and out; S: stored type (uint8_t: E4M3); C: fours of columns of a lane; H: rows that a
// warp takes side by side.
template <typename T, typename S, int C, int H>
__global__ void __launch_bounds__(kThreads, Shape<S, C, H>::CTAS) k_paged_attn_simt(const PagedAttn p) {
  using Sh = Shape<S, C, H>;
  constexpr int VB = Sh::VB, NST = Sh::NST, LPR = 32 / H, KG = 4 * H;  // lanes of a row, keys of a group
  constexpr bool E8 = sizeof(S) == 1;
  extern __shared__ __align__(16) unsigned char smem[];
  pdl_trigger();
  const int hd = p.m.head_dim, tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int part = lane / LPR, lcol = lane % LPR * 4;  // which of the rows side by side, first column
  float* sP = (float*)(smem + kWarps * NST * Sh::kStage) + wid * 32 * H;
  float* sO = (float*)(smem + kWarps * NST * Sh::kStage) + kWarps * 32 * H;
  float2* sML = (float2*)(sO + kQ * hd);
  unsigned char* ring = smem + wid * NST * Sh::kStage;
  Deal deal;
  Tiles cons = my_tiles<T>(p, deal, kThreads);
  if (cons.pos >= cons.end) return;
  bool col[C];  // this lane's columns are some of the head's
#pragma unroll
  for (int c = 0; c < C; ++c) {
    col[c] = c * 128 + lcol < hd;
    if (!col[c])  // never copied: zeros
      for (int i = 0; i < NST * 8; ++i) {
        unsigned char* at = ring + (i >> 3) * Sh::kStage + (((i & 7) * C + c) * 32 + lane) * VB;
#pragma unroll
        for (int x = 0; x < VB; x += 4) *reinterpret_cast<uint32_t*>(at + x) = 0u;
      }
  }

  // ---- copies: groups of KG keys of the warp's 16 of every tile ----
  // Lane i (and i + 16) finds the row of key i, a tile ahead of its use: its first element in the
  // cache, or -1, and its scale's place.
  Tiles ahead = cons;
  int left = cons.end - cons.pos, stage_in = 0, group_in = 0;
  int64_t row = -1, next_row = -1, line = 0, next_line = 0;
  auto look_up = [&]() {
    next_row = -1;
    const int j = ahead.first + ahead.t * 64 + wid * 16 + (lane & 15);
    if (ahead.pos < ahead.end && j < ahead.len && j >= seq_low(p, ahead.len)) {
      int off;
      const int page = page_of(p.m, ahead.b, j, off, p.err);
      if (page >= 0) {
        const int64_t in_page = (int64_t)(ahead.unit / p.chunks) * p.m.page_size + off;
        next_row = (int64_t)page * p.m.page_stride + in_page * hd;
        next_line = (int64_t)page * p.m.scale_stride + in_page;
      }
    }
  };
  look_up();
  auto produce = [&]() {
    if (left > 0) {
      if (group_in == 0) {
        row = next_row;
        line = next_line;
        ahead.skip(p, 1);
        look_up();
      }
      unsigned char* st = ring + stage_in * Sh::kStage;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t at = __shfl_sync(0xffffffffu, row, group_in * KG + part * 4 + k);
        const int bytes = at < 0 ? 0 : VB;  // (a row that is not there is not read: zeros)
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (col[c]) {
            const int64_t src = at < 0 ? 0 : (at + c * 128 + lcol) * (int)sizeof(S);
            copy<VB>(smem_u32(st + ((k * C + c) * 32 + lane) * VB), (const char*)p.k + src, bytes);
            copy<VB>(smem_u32(st + (((4 + k) * C + c) * 32 + lane) * VB), (const char*)p.v + src, bytes);
          }
      }
      const bool there = __shfl_sync(0xffffffffu, row, group_in * KG + lane % KG) >= 0;
      if (E8) {
        const int64_t at = __shfl_sync(0xffffffffu, line, group_in * KG + lane % KG);
        if (lane < 2 * KG)
          cp_async4(smem_u32(st + Sh::kRows + lane * 4), (lane < KG ? p.ks : p.vs) + (there ? at : 0), there ? 4 : 0);
      }
      const unsigned ok = __ballot_sync(0xffffffffu, there) & ((1u << KG) - 1);
      if (lane == 0) *reinterpret_cast<uint32_t*>(st + Sh::kRows + 8 * KG) = ok;
      if (++group_in == 16 / KG) {
        group_in = 0;
        --left;
      }
    }
    cp_async_commit();
    stage_in = stage_in + 1 == NST ? 0 : stage_in + 1;
  };
  for (int i = 0; i < NST - 1; ++i) produce();

  int stage = 0;
  // of the scores, this lane's: H queries from my_q on of one key
  constexpr int QL = 8 / H;  // lanes of a key
  const int my_q = lane % QL * H, my_key = lane / QL;
  while (cons.pos < cons.end) {
    // ---- one piece: tiles t0..t1 of a unit ----
    const int t0 = cons.t, t1 = min(cons.n, t0 + cons.end - cons.pos);
    const int nq = queries_of(p, cons.unit);
    f32x2 q2[kQ / 2][C][4], o2[kQ / 2][C][4];  // queries 2 i and 2 i + 1 side by side
#pragma unroll
    for (int i = 0; i < kQ / 2; ++i)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float x[2][4] = {};
#pragma unroll
        for (int y = 0; y < 2; ++y)
          if (2 * i + y < nq && col[c]) {
            int head, r;
            query_of(p, cons.unit, 2 * i + y, &head, &r);
            get4((const T*)p.a.q + (int64_t)cons.b * p.a.q_seq + (int64_t)r * p.a.q_row + (int64_t)head * p.a.q_head +
                     c * 128 + lcol, x[y]);
          }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          q2[i][c][e] = pack(x[0][e], x[1][e]);
          o2[i][c][e] = 0ull;
        }
      }
    float m[H], l[H];
    int top[H];  // last position that a query of this lane's sees
#pragma unroll
    for (int x = 0; x < H; ++x) {
      m[x] = -INFINITY;
      l[x] = 0.f;
      top[x] = -1;
      if (my_q + x < nq) {
        int head, r;
        query_of(p, cons.unit, my_q + x, &head, &r);
        top[x] = cons.len - p.a.rows + r;
      }
    }
    for (int g = 16 / KG * t0; g < 16 / KG * t1; ++g) {
      cp_async_wait<NST - 2>();
      __syncwarp();  // this stage is here; the one before has been used
      produce();
      const unsigned char* st = ring + stage * Sh::kStage;
      stage = stage + 1 == NST ? 0 : stage + 1;
      const unsigned ok = *reinterpret_cast<const uint32_t*>(st + Sh::kRows + 8 * KG);
      if (!ok) continue;
      const int j0 = cons.first + g / (16 / KG) * 64 + wid * 16 + g % (16 / KG) * KG;
      float v[32];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        f32x2 s[kQ / 2];
#pragma unroll
        for (int c = 0; c < C; ++c) {
          float f[4];
          get4((const S*)(st + ((k * C + c) * 32 + lane) * VB), f);
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int i = 0; i < kQ / 2; ++i)
              s[i] = c + e ? fma2(q2[i][c][e], both(f[e]), s[i]) : mul2(q2[i][c][e], both(f[e]));
        }
#pragma unroll
        for (int i = 0; i < kQ / 2; ++i) {
          const float2 x = unpack(s[i]);
          v[8 * k + 2 * i] = x.x;
          v[8 * k + 2 * i + 1] = x.y;
        }
      }
      const float* scales = (const float*)(st + Sh::kRows);
      sum_to_lane<H>(v);
      const float by = E8 ? scales[my_key] * p.scale2 : p.scale2;
      const int j = j0 + my_key;
      float x[H];
      bool seen[H], rise = false;
#pragma unroll
      for (int y = 0; y < H; ++y) {
        seen[y] = (ok >> my_key & 1) && j <= top[y] && (p.a.window <= 0 || j > top[y] - p.a.window);
        x[y] = seen[y] ? v[y] * by : -INFINITY;
        rise = rise || x[y] > m[y] + 8.f;
      }
      // the maximum moves only when a score passes it by 2^8: few groups rescale what they have
      if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
        for (int y = 0; y < H; ++y) {
          float mx = x[y];
#pragma unroll
          for (int o = QL; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          mx = fmaxf(m[y], mx);
          const float fix = mx == -INFINITY ? 1.f : ex2(m[y] - mx);
          m[y] = mx;
          l[y] *= fix;
          if (lane < QL) sP[my_q + y] = fix;
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kQ / 2; ++i) {
          const f32x2 fix = *reinterpret_cast<const f32x2*>(sP + 2 * i);
#pragma unroll
          for (int c = 0; c < C; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) o2[i][c][e] = mul2(o2[i][c][e], fix);
        }
        __syncwarp();
      }
      const float vs = E8 ? scales[KG + my_key] : 1.f;
#pragma unroll
      for (int y = 0; y < H; ++y) {
        const float w = seen[y] ? ex2(x[y] - (m[y] == -INFINITY ? 0.f : m[y])) : 0.f;
        l[y] += w;
        sP[8 * my_key + my_q + y] = E8 ? w * vs : w;
      }
      __syncwarp();
      const float* sW = sP + 32 * part;
      // A position that only some of the rows see may hold an infinity or a NaN, which a
      // weight of zero would turn into a NaN: those groups leave zero weights out.
      const bool edge = j0 + KG - 1 > cons.len - p.a.rows || (p.a.window > 0 && j0 < cons.len - p.a.window);
      bool odd = false;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const ulonglong2 wa = *reinterpret_cast<const ulonglong2*>(sW + 8 * k), wb = *reinterpret_cast<const ulonglong2*>(sW + 8 * k + 4);
        const f32x2 w2[kQ / 2] = {wa.x, wa.y, wb.x, wb.y};
#pragma unroll
        for (int c = 0; c < C; ++c) {
          float f[4];
          get4((const S*)(st + (((4 + k) * C + c) * 32 + lane) * VB), f);
          if (edge) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const bool is = !(fabsf(f[e]) <= 3.402823466e38f);
              odd = odd || is;
              f[e] = is ? 0.f : f[e];
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int i = 0; i < kQ / 2; ++i) o2[i][c][e] = fma2(w2[i], both(f[e]), o2[i][c][e]);
        }
      }
      if (odd) {  // those values, to the queries that see them
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll 1
          for (int k = 0; k < 4; ++k) {
            float f[4];
            get4((const S*)(st + (((4 + k) * C + c) * 32 + lane) * VB), f);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
              for (int i = 0; i < kQ / 2; ++i) {
                const float a = sW[8 * k + 2 * i], b = sW[8 * k + 2 * i + 1];
                const bool is = !(fabsf(f[e]) <= 3.402823466e38f);
                o2[i][c][e] = add2(o2[i][c][e], pack(is && a != 0.f ? a * f[e] : 0.f, is && b != 0.f ? b * f[e] : 0.f));
              }
          }
      }
    }

    // ---- join the warps in order, and write ----
#pragma unroll
    for (int y = 0; y < H; ++y) {
#pragma unroll
      for (int o = QL; o < 32; o <<= 1) l[y] += __shfl_xor_sync(0xffffffffu, l[y], o);
      if (lane < QL) sML[wid * kQ + my_q + y] = make_float2(m[y], l[y]);
    }
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1)  // the rows side by side have the same columns
#pragma unroll
      for (int i = 0; i < kQ / 2; ++i)
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            o2[i][c][e] = add2(o2[i][c][e], __shfl_xor_sync(0xffffffffu, o2[i][c][e], o));
    __syncthreads();
    float f[kQ];
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
      float M = -INFINITY;
#pragma unroll
      for (int x = 0; x < kWarps; ++x) M = fmaxf(M, sML[x * kQ + q].x);
      f[q] = M == -INFINITY ? 0.f : ex2(sML[wid * kQ + q].x - M);
    }
#pragma unroll 1
    for (int turn = 0; turn < kWarps; ++turn) {
      if (turn == wid) {
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (col[c] && part == 0) {
#pragma unroll
            for (int i = 0; i < kQ / 2; ++i)
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                float4* at = reinterpret_cast<float4*>(sO + (2 * i + y) * hd + c * 128 + lcol);
                float4 was = turn ? *at : make_float4(0.f, 0.f, 0.f, 0.f);
                const float2 a = unpack(o2[i][c][0]), b = unpack(o2[i][c][1]), d = unpack(o2[i][c][2]), e = unpack(o2[i][c][3]);
                was.x = fmaf(y ? a.y : a.x, f[2 * i + y], was.x);
                was.y = fmaf(y ? b.y : b.x, f[2 * i + y], was.y);
                was.z = fmaf(y ? d.y : d.x, f[2 * i + y], was.z);
                was.w = fmaf(y ? e.y : e.x, f[2 * i + y], was.w);
                *at = was;
              }
          }
      }
      __syncthreads();
    }
    const bool whole = t0 == 0 && t1 == cons.n;
    const int slot = ((int)blockIdx.x * 2 + (t0 == 0)) * p.qn, fours = hd / 4;
    for (int i = tid; i < nq * fours; i += kThreads) {
      const int q = i / fours, d = (i - q * fours) * 4;
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int x = 0; x < kWarps; ++x) M = fmaxf(M, sML[x * kQ + q].x);
#pragma unroll
      for (int x = 0; x < kWarps; ++x) {
        const float2 ml = sML[x * kQ + q];
        L += M == -INFINITY ? 0.f : ml.y * ex2(ml.x - M);
      }
      const float4 v = *reinterpret_cast<const float4*>(sO + q * hd + d);
      if (whole) {
        int head, r;
        query_of(p, cons.unit, q, &head, &r);
        T* out = (T*)p.a.out + (int64_t)cons.b * p.a.o_seq + (int64_t)r * p.a.o_row + (int64_t)head * p.a.o_head;
        const float inv = L != 0.f ? 1.f / L : 0.f;
        store_act4(out + d, 0, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
      } else {
        *reinterpret_cast<float4*>(p.part_o + (int64_t)(slot + q) * hd + d) = v;
        if (d == 0) p.part_ml[slot + q] = make_float2(M, L);
      }
    }
    if (t0 == 0 && tid == 0) leave_note(p, deal, cons);
    cons.skip(p, t1 - t0);
    __syncthreads();  // sO and sML are free again
  }
  cp_async_wait<0>();
}

template <typename T, typename S, int C, int H>
cudaError_t launch_c(const PagedAttn& p, int grid, cudaStream_t st) {
  static unsigned long long done = 0;
  auto k = k_paged_attn_simt<T, S, C, H>;
  if (!smem_limit((const void*)k, Shape<S, C, H>::smem(C * 128 / H), &done)) return cudaErrorInvalidValue;
  return launch_op(k, grid, kThreads, Shape<S, C, H>::smem(p.m.head_dim), st, false, 1, p);
}
template <typename T, typename S>
cudaError_t launch_t(const PagedAttn& p, int grid, cudaStream_t st) {
  const int hd = p.m.head_dim;
  return hd <= 32   ? launch_c<T, S, 1, 4>(p, grid, st)
         : hd <= 64 ? launch_c<T, S, 1, 2>(p, grid, st)
         : hd <= 128 ? launch_c<T, S, 1, 1>(p, grid, st)
                     : launch_c<T, S, 2, 1>(p, grid, st);
}

}  // namespace

namespace dmtp {

int paged_simt_grid(int head_dim) { return 152 * (head_dim <= 128 ? 3 : 2); }

cudaError_t paged_attn_simt(const PagedAttn& p, const PagedPlan& pl, int dtype, bool e8, cudaStream_t st) {
  if (e8) return dtype ? launch_t<bf16, uint8_t>(p, pl.grid, st) : launch_t<float, uint8_t>(p, pl.grid, st);
  return dtype ? launch_t<bf16, bf16>(p, pl.grid, st) : launch_t<float, float>(p, pl.grid, st);
}

}  // namespace dmtp
