// Attention over a paged cache on the tensor cores: bf16 rows of head size 64 or 128, the
// cache in bf16 or E4M3.
//
// One pass over the cached rows bounds it: each byte of K and V feeds at most 64 queries of
// its kv head (rows x query heads), a few hundred operations. So the CTA (four warps, two
// CTAs an SM) keeps a ring of 64-key tiles in flight by 16-byte asynchronous copies, one
// page lookup per row (made a tile ahead, so no copy waits for the table), and the warps
// work on the 16-bit fragments with m16n8k16 products, which need no staging beyond the tile
// itself and no rows padded to 128 (the tcgen05 form wants M >= 64 of its 128 lanes, mostly
// empty at 1 to 16 queries, and the E4M3 rows would have to be converted through shared
// memory).
//
//   QN queries  warps         a warp's share of a tile
//   8, 16       4 key groups  16 keys x 16 queries
//   32          4 key groups  16 keys x 32 queries
//   64          2 x 2         32 keys x 32 queries
//
// Scores S = Q K^T (fp32 accumulators), weights 2^(S - m) with a running maximum m per row
// that moves only when a score passes it by 2^8 (so most tiles skip the rescaling), and
// O += P V with P as the A operand straight from the registers of S. bf16 caches: P as a
// bf16 pair (16 bits of each weight), two products a fragment. E4M3 caches: rows become fp16
// exactly, the queries too after a power-of-two scale per row, and P carries the value
// row's scale: with v = 2^e c and weight w, m follows log2(w 2^e) and P = w 2^(e - m), so
// what is rounded to fp16 is the row's contribution relative to the largest one; the sum of
// weights undoes the exponent in fp32.
#include <cuda_fp16.h>

#include "paged_attn.cuh"

using namespace dmtp;

namespace {

constexpr int kTK = 64, kThreads = 128;

template <int HD, bool E8, int QN>
struct Shape {
  static constexpr int MW = QN <= 16 ? 1 : 2;     // 16-query tiles of a warp
  static constexpr int QG = QN == 64 ? 2 : 1;     // query groups of warps
  static constexpr int KS = 4 / QG;               // key groups of warps
  static constexpr int QR = 16 * MW * QG;         // query rows of the CTA's tiles
  static constexpr int RB = HD * (E8 ? 1 : 2);    // bytes of a cached row
  static constexpr int kStage = 2 * kTK * RB + (E8 ? 2 * kTK * 4 : 0);
  static constexpr int kPitch = HD + (E8 ? 16 : 8);  // floats of a joined row: no conflicts
  // joined rows; the queries of MW = 2 lie there while the tiles run (QR * HD * 2 bytes)
  static constexpr int kJoin = QR * kPitch * 4 + KS * QR * 8;
  static constexpr int kMisc = 8 * 4 * 4 + 64;    // valid rows of each stage, the walk
  static constexpr int kRoom = 113 * 1024 - kJoin - kMisc;  // two CTAs an SM
  static constexpr int NST = kRoom / kStage > 8 ? 8 : kRoom / kStage;
  static constexpr int kSmem = NST * kStage + kJoin + kMisc;
  static_assert(NST >= 2, "a ring of two tiles at least");
};

// Byte of 16-byte step c of row r in a tile: the steps of eight consecutive rows that
// ldmatrix reads together lie in different banks.
template <int RB>
__device__ __forceinline__ int tile_at(int r, int c) {
  return r * RB + ((RB >= 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4);
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// The halves of a pair that are infinite or NaN, cleared.
template <bool F16>
__device__ __forceinline__ uint32_t finite_pair(uint32_t u) {
  const uint32_t e = F16 ? 0x7c00u : 0x7f80u;
  if ((u & e) == e) u &= 0xffff0000u;
  if ((u >> 16 & e) == e) u &= 0x0000ffffu;
  return u;
}

// The tiles of a CTA's range in order.
struct Tiles {
  int pos, end, b, unit, t, n, len, first;
  __device__ __forceinline__ void seq(const PagedAttn& p) {
    len = seq_len(p, b);
    first = seq_first(p, len);
    n = (len - first + kTK - 1) / kTK;
  }
  __device__ __forceinline__ void start(const PagedAttn& p, const Walk& w) {
    pos = w.pos;
    end = w.end;
    b = w.b;
    unit = t = n = len = first = 0;
    if (pos < end) {
      seq(p);
      unit = (pos - w.base) / n;
      t = pos - w.base - unit * n;
    }
  }
  __device__ __forceinline__ void skip(const PagedAttn& p, int tiles) {  // to the next unit at most
    pos += tiles;
    t += tiles;
    if (t == n && pos < end) {
      t = 0;
      if (++unit == p.units) {
        unit = 0;
        do {
          ++b;
          seq(p);
        } while (n == 0);
      }
    }
  }
};

template <int HD, bool E8, int QN>
__global__ void __launch_bounds__(kThreads, 2) k_paged_attn_tc(const PagedAttn p) {
  using S = Shape<HD, E8, QN>;
  constexpr int MW = S::MW, QG = S::QG, KS = S::KS, QR = S::QR, RB = S::RB, NST = S::NST;
  constexpr int KK = HD / 16;             // products along the head
  constexpr bool kHalf = QN <= 8;         // rows 8..15 of the tile hold no query
  extern __shared__ __align__(128) unsigned char smem[];
  float* sO = (float*)(smem + NST * S::kStage);
  float2* sML = (float2*)(sO + QR * S::kPitch);
  uint4* sQ = (uint4*)sO;
  uint32_t* sOk = (uint32_t*)(sML + KS * QR);
  int* sWalk = (int*)(sOk + 8 * 4);
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, g = lane >> 2, tq = lane & 3;
  const int qg = wid % QG, ks = wid / QG;
  pdl_trigger();
  const Walk w = deal<kTK, kThreads>(p, sWalk);
  if (w.pos >= w.end) return;
  Tiles cons, prod;
  cons.start(p, w);
  prod = cons;

  // ---- copies: warp w brings rows 16 w .. 16 w + 15 of every tile ----
  constexpr int CPR = RB / 16, RPI = 32 / CPR, NI = 16 / RPI;
  int row_page = -1;  // page of this lane's row (lanes 0..15) of the next tile to bring
  auto look_up = [&]() {
    const int j = prod.first + prod.t * kTK + wid * 16 + lane;
    row_page = -1;
    if (prod.pos < prod.end && lane < 16 && j < prod.len) row_page = page_of(p.m, prod.b, j, p.err);
  };
  int stage_in = 0;
  auto produce = [&]() {
    if (prod.pos < prod.end) {
      unsigned char* st = smem + stage_in * S::kStage;
      const int kvh = prod.unit / p.chunks;
      const int j = prod.first + prod.t * kTK + wid * 16 + lane;
      const int line = kvh * p.m.page_size + (unsigned)j % (unsigned)p.m.page_size;
      const int64_t at = row_page < 0 ? -1 : (int64_t)row_page * p.m.page_stride + (int64_t)line * HD;
      const unsigned ok = __ballot_sync(0xffffffffu, row_page >= 0) & 0xffffu;
      if (lane == 0) sOk[stage_in * 4 + wid] = ok;
      if (E8 && lane < 16) {
        const int64_t sat = row_page < 0 ? 0 : (int64_t)row_page * p.m.scale_stride + line;
        const uint32_t d = smem_u32(st + 2 * kTK * RB) + (wid * 16 + lane) * 4;
        cp_async4(d, p.ks + sat, row_page < 0 ? 0 : 4);
        cp_async4(d + kTK * 4, p.vs + sat, row_page < 0 ? 0 : 4);
      }
      const uint32_t dst = smem_u32(st);
      const int rin = lane / CPR, c = lane % CPR;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int r = i * RPI + rin;
        const int64_t a = __shfl_sync(0xffffffffu, at, r);
        const int64_t src = a < 0 ? 0 : a * (E8 ? 1 : 2) + c * 16;
        const uint32_t d = dst + tile_at<RB>(wid * 16 + r, c);
        cp_async16(d, (const char*)p.k + src, a < 0 ? 0 : 16);
        cp_async16(d + kTK * RB, (const char*)p.v + src, a < 0 ? 0 : 16);
      }
      prod.skip(p, 1);
      look_up();
    }
    cp_async_commit();
    stage_in = stage_in + 1 == NST ? 0 : stage_in + 1;
  };
  look_up();
  for (int i = 0; i < NST - 1; ++i) produce();

  int stage = 0;
  while (cons.pos < cons.end) {
    // ---- one piece: tiles t0..t1 of a unit ----
    const int t0 = cons.t, t1 = min(cons.n, t0 + cons.end - cons.pos);
    const int nq = queries_of(p, cons.unit);
    uint32_t qf[MW == 1 ? KK : 1][4];
    float rowf[MW][2], m[MW][2], l[MW][2], o[MW][HD / 8][4];
    int top[MW][2];
#pragma unroll
    for (int mw = 0; mw < MW; ++mw) {
      const bf16* qp[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int t = (qg * MW + mw) * 16 + g + 8 * h;
        m[mw][h] = -INFINITY;
        l[mw][h] = 0.f;
        rowf[mw][h] = p.scale2;
        top[mw][h] = -1;
        qp[h] = nullptr;
        if (t < nq) {
          int head, row;
          query_of(p, cons.unit, t, &head, &row);
          top[mw][h] = cons.len - p.a.rows + row;
          qp[h] = (const bf16*)p.a.q + (int64_t)cons.b * p.a.q_seq + (int64_t)row * p.a.q_row + (int64_t)head * p.a.q_head;
        }
      }
      // A fragments: bf16 rows in the products' own order; for an E4M3 cache a thread holds
      // four consecutive columns, as the bytes of K come
      uint32_t f[KK][4];
#pragma unroll
      for (int k = 0; k < KK; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          f[k][h] = f[k][2 + h] = 0;
          if (qp[h]) {
            if (E8) {
              const uint2 u = *reinterpret_cast<const uint2*>(qp[h] + 16 * k + 4 * tq);
              f[k][h] = u.x;
              f[k][2 + h] = u.y;
            } else {
              f[k][h] = *reinterpret_cast<const uint32_t*>(qp[h] + 16 * k + 2 * tq);
              f[k][2 + h] = *reinterpret_cast<const uint32_t*>(qp[h] + 16 * k + 8 + 2 * tq);
            }
          }
        }
      if (E8) {  // bf16 -> fp16, the row's largest magnitude brought into [2^12, 2^13)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t big = 0;
#pragma unroll
          for (int k = 0; k < KK; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t u = f[k][h + 2 * i];
              const uint32_t a = u << 16 & 0x7fff0000u, b = u & 0x7fff0000u;
              if (a < 0x7f800000u) big = max(big, a);
              if (b < 0x7f800000u) big = max(big, b);
            }
          big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
          big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
          // 2^(12 - floor(log2 big)), kept inside the normal range
          const int e = big ? min(max(12 - ((int)(big >> 23) - 127), -126), 126) : 0;
          const float up = pow2f(e);
          rowf[mw][h] = p.scale2 * pow2f(-e);
#pragma unroll
          for (int k = 0; k < KK; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t u = f[k][h + 2 * i];
              f[k][h + 2 * i] = pack_f16(__uint_as_float(u << 16) * up, __uint_as_float(u & 0xffff0000u) * up);
            }
        }
      }
      if (MW == 1) {
#pragma unroll
        for (int k = 0; k < KK; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) qf[MW == 1 ? k : 0][i] = f[k][i];
      } else if (ks == 0) {
#pragma unroll
        for (int k = 0; k < KK; ++k)
          sQ[((qg * MW + mw) * KK + k) * 32 + lane] = make_uint4(f[k][0], f[k][1], f[k][2], f[k][3]);
      }
#pragma unroll
      for (int i = 0; i < HD / 8; ++i) o[mw][i][0] = o[mw][i][1] = o[mw][i][2] = o[mw][i][3] = 0.f;
    }

    for (int t = t0; t < t1; ++t) {
      cp_async_wait<NST - 2>();
      __syncthreads();  // this tile is here for all warps; the one before has been used
      produce();
      const unsigned char* st = smem + stage * S::kStage;
      const uint32_t sK = smem_u32(st), sV = sK + kTK * RB;
      const float* sS = (const float*)(st + 2 * kTK * RB);
      const int j0 = cons.first + t * kTK;
#pragma unroll 1
      for (int sub = ks; sub < 4; sub += KS) {
        const int r0 = sub * 16;  // first key of the subtile in the tile
        const unsigned ok = sOk[stage * 4 + sub];
        // S = Q K^T: two 8-key blocks
        float s[MW][2][4];
#pragma unroll
        for (int mw = 0; mw < MW; ++mw)
#pragma unroll
          for (int i = 0; i < 2; ++i) s[mw][i][0] = s[mw][i][1] = s[mw][i][2] = s[mw][i][3] = 0.f;
        {
          const int mi = lane >> 3, r = r0 + (lane & 7) + 8 * (mi >> 1);
          if (E8) {
#pragma unroll
            for (int k2 = 0; k2 < KK; k2 += 2) {
              uint32_t kr[4];  // keys 0-7: columns 16 k2.., 16 k2 + 16..; keys 8-15 likewise
              ldsm4(kr, sK + tile_at<RB>(r, k2 + (mi & 1)));
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint32_t a0 = e4m3x2_to_h2(kr[i] & 0xffffu), a1 = e4m3x2_to_h2(kr[i] >> 16);
                const uint32_t b0 = e4m3x2_to_h2(kr[2 + i] & 0xffffu), b1 = e4m3x2_to_h2(kr[2 + i] >> 16);
#pragma unroll
                for (int mw = 0; mw < MW; ++mw) {
                  uint32_t q[4];
                  if (MW == 1) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) q[x] = qf[MW == 1 ? k2 + i : 0][x];
                  } else {
                    const uint4 u = sQ[((qg * MW + mw) * KK + k2 + i) * 32 + lane];
                    q[0] = u.x, q[1] = u.y, q[2] = u.z, q[3] = u.w;
                  }
                  mma16816<true>(s[mw][0], q, a0, a1);
                  mma16816<true>(s[mw][1], q, b0, b1);
                }
              }
            }
          } else {
#pragma unroll
            for (int k = 0; k < KK; ++k) {
              uint32_t kr[4];
              ldsm4(kr, sK + tile_at<RB>(r, 2 * k + (mi & 1)));
#pragma unroll
              for (int mw = 0; mw < MW; ++mw) {
                uint32_t q[4];
                if (MW == 1) {
#pragma unroll
                  for (int x = 0; x < 4; ++x) q[x] = qf[MW == 1 ? k : 0][x];
                } else {
                  const uint4 u = sQ[((qg * MW + mw) * KK + k) * 32 + lane];
                  q[0] = u.x, q[1] = u.y, q[2] = u.z, q[3] = u.w;
                }
                mma16816<false>(s[mw][0], q, kr[0], kr[1]);
                mma16816<false>(s[mw][1], q, kr[2], kr[3]);
              }
            }
          }
        }
        // the thread's four keys: 2 tq, 2 tq + 1 of each block
        float kf[2][2], ve[2][2], vm[2][2], vi[2][2];
        if (E8) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int key = r0 + 8 * i + 2 * tq + x;
              kf[i][x] = sS[key];
              const uint32_t u = __float_as_uint(sS[kTK + key]);  // 2^(u >> 23 - 127) times [1, 2)
              ve[i][x] = __uint_as_float(0x4b000000u | u >> 23) - 8388735.f;
              vm[i][x] = __uint_as_float(0x3f800000u | (u & 0x7fffffu));
              vi[i][x] = pow2f(127 - (int)(u >> 23));
            }
        }
        const int jb = j0 + r0;
        const bool edge = ok != 0xffffu || jb + 15 > cons.len - p.a.rows ||
                          (p.a.window > 0 && jb < cons.len - p.a.window);
        uint32_t pa[MW][4], pl[MW][4];
#pragma unroll
        for (int mw = 0; mw < MW; ++mw) {
          float x[2][2][2];  // [row half][block][key]
          bool rise = false;
#pragma unroll
          for (int h = 0; h < (kHalf ? 1 : 2); ++h) {
            float mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                float v = s[mw][i][2 * h + y] * rowf[mw][h];
                if (E8) v = fmaf(v, kf[i][y], ve[i][y]);
                if (edge) {
                  const int key = 8 * i + 2 * tq + y, j = jb + key;
                  const bool seen = (ok >> key & 1) && j <= top[mw][h] &&
                                    (p.a.window <= 0 || j > top[mw][h] - p.a.window);
                  v = seen ? v : -INFINITY;
                }
                x[h][i][y] = v;
                mx = fmaxf(mx, v);
              }
            rise = rise || mx > m[mw][h] + 8.f;
          }
          if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
            for (int h = 0; h < (kHalf ? 1 : 2); ++h) {
              float mx = fmaxf(fmaxf(x[h][0][0], x[h][0][1]), fmaxf(x[h][1][0], x[h][1][1]));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
              if (mx > m[mw][h] + 8.f) {
                const float fix = ex2(m[mw][h] - mx);  // 0 for the first
                m[mw][h] = mx;
                l[mw][h] *= fix;
#pragma unroll
                for (int i = 0; i < HD / 8; ++i) {
                  o[mw][i][2 * h] *= fix;
                  o[mw][i][2 * h + 1] *= fix;
                }
              }
            }
          }
#pragma unroll
          for (int h = 0; h < (kHalf ? 1 : 2); ++h) {
            const float ref = m[mw][h] == -INFINITY ? 0.f : m[mw][h];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float w0 = ex2(x[h][i][0] - ref), w1 = ex2(x[h][i][1] - ref);
              if (E8) {
                l[mw][h] = fmaf(w0, vi[i][0], fmaf(w1, vi[i][1], l[mw][h]));
                pa[mw][2 * i + h] = pack_f16(w0 * vm[i][0], w1 * vm[i][1]);
              } else {
                l[mw][h] += w0 + w1;
                const uint32_t hi = pack_bf16(w0, w1);
                pa[mw][2 * i + h] = hi;
                pl[mw][2 * i + h] = pack_bf16(w0 - __uint_as_float(hi << 16), w1 - __uint_as_float(hi & 0xffff0000u));
              }
            }
          }
          if (kHalf) pa[mw][1] = pa[mw][3] = pl[mw][1] = pl[mw][3] = 0;
        }
        // O += P V
        const int mi = lane >> 3, vr = r0 + (lane & 7) + 8 * (mi & 1);
        bool odd = false;  // an infinity or NaN among values that not every row sees
#pragma unroll
        for (int c = 0; c < CPR; c += 2) {
          uint32_t v[4];  // two 16-byte steps of keys 0-7 and 8-15
          ldsm4_t(v, sV + tile_at<RB>(vr, c + (mi >> 1)));
          if (E8) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              // bytes (key, key + 1) of columns 2g, 2g + 1
              const uint32_t lo = __byte_perm(v[2 * i], 0, 0x3120), hi = __byte_perm(v[2 * i + 1], 0, 0x3120);
              uint32_t e0 = e4m3x2_to_h2(lo & 0xffffu), e1 = e4m3x2_to_h2(hi & 0xffffu);
              uint32_t d0 = e4m3x2_to_h2(lo >> 16), d1 = e4m3x2_to_h2(hi >> 16);
              if (edge) {
                const uint32_t a = e0, b = e1, cc = d0, d = d1;
                e0 = finite_pair<true>(e0), e1 = finite_pair<true>(e1);
                d0 = finite_pair<true>(d0), d1 = finite_pair<true>(d1);
                odd = odd || a != e0 || b != e1 || cc != d0 || d != d1;
              }
#pragma unroll
              for (int mw = 0; mw < MW; ++mw) {
                mma16816<true>(o[mw][2 * (c + i)], pa[mw], e0, e1);
                mma16816<true>(o[mw][2 * (c + i) + 1], pa[mw], d0, d1);
              }
            }
          } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t b0 = v[2 * i], b1 = v[2 * i + 1];
              if (edge) {
                const uint32_t a = b0, b = b1;
                b0 = finite_pair<false>(b0), b1 = finite_pair<false>(b1);
                odd = odd || a != b0 || b != b1;
              }
#pragma unroll
              for (int mw = 0; mw < MW; ++mw) {
                mma16816<false>(o[mw][c + i], pa[mw], b0, b1);
                mma16816<false>(o[mw][c + i], pl[mw], b0, b1);
              }
            }
          }
        }
        if (edge && __any_sync(0xffffffffu, odd)) {
          // give those values to the rows that do see them: weights by shuffle from the lane
          // that holds them, values from shared memory
#pragma unroll 1
          for (int key = 0; key < 16; ++key) {
            const int from = (lane & ~3) | (key & 7) >> 1;
#pragma unroll
            for (int mw = 0; mw < MW; ++mw)
#pragma unroll
              for (int h = 0; h < (kHalf ? 1 : 2); ++h) {
                const uint32_t a = __shfl_sync(0xffffffffu, pa[mw][h], from);
                const uint32_t b = __shfl_sync(0xffffffffu, pa[mw][2 + h], from);
                const uint32_t u = key < 8 ? a : b;
                const uint32_t bits = key & 1 ? u >> 16 : u & 0xffffu;
                const float wgt = E8 ? h2_to_f2(bits).x : __uint_as_float(bits << 16);
                if (wgt != 0.f) {
                  const unsigned char* row = st + kTK * RB;
#pragma unroll
                  for (int i = 0; i < HD / 8; ++i)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                      const int d = E8 ? 16 * (i >> 1) + 4 * tq + 2 * y + (i & 1) : 8 * i + 2 * tq + y;
                      const int byte = d * (E8 ? 1 : 2);
                      const unsigned char* at = row + tile_at<RB>(r0 + key, byte >> 4) + (byte & 15);
                      const float val = E8 ? h2_to_f2(e4m3x2_to_h2(*at)).x : __bfloat162float(*(const bf16*)at);
                      if (!(fabsf(val) <= 3.402823466e38f)) o[mw][i][2 * h + y] = fmaf(wgt, val, o[mw][i][2 * h + y]);
                    }
                }
              }
          }
        }
      }
      stage = stage + 1 == NST ? 0 : stage + 1;
    }

    // ---- join the key groups in order, and write ----
#pragma unroll
    for (int mw = 0; mw < MW; ++mw)
#pragma unroll
      for (int h = 0; h < (kHalf ? 1 : 2); ++h) {
        l[mw][h] += __shfl_xor_sync(0xffffffffu, l[mw][h], 1);
        l[mw][h] += __shfl_xor_sync(0xffffffffu, l[mw][h], 2);
        if (tq == 0) sML[ks * QR + (qg * MW + mw) * 16 + g + 8 * h] = make_float2(m[mw][h], l[mw][h]);
      }
    __syncthreads();
#pragma unroll
    for (int mw = 0; mw < MW; ++mw)
#pragma unroll
      for (int h = 0; h < (kHalf ? 1 : 2); ++h) {
        const int q = (qg * MW + mw) * 16 + g + 8 * h;
        float M = -INFINITY;
#pragma unroll
        for (int i = 0; i < KS; ++i) M = fmaxf(M, sML[i * QR + q].x);
        const float f = M == -INFINITY ? 0.f : ex2(m[mw][h] - M);
#pragma unroll
        for (int i = 0; i < HD / 8; ++i) {
          o[mw][i][2 * h] *= f;
          o[mw][i][2 * h + 1] *= f;
        }
      }
#pragma unroll
    for (int turn = 0; turn < KS; ++turn) {
      if (turn == ks) {
#pragma unroll
        for (int mw = 0; mw < MW; ++mw)
#pragma unroll
          for (int h = 0; h < (kHalf ? 1 : 2); ++h) {
            float* row = sO + ((qg * MW + mw) * 16 + g + 8 * h) * S::kPitch;
            if (E8) {
#pragma unroll
              for (int c = 0; c < HD / 16; ++c) {
                float4* at = reinterpret_cast<float4*>(row + 16 * c + 4 * tq);
                float4 v = make_float4(o[mw][2 * c][2 * h], o[mw][2 * c + 1][2 * h], o[mw][2 * c][2 * h + 1],
                                       o[mw][2 * c + 1][2 * h + 1]);
                if (turn) {
                  const float4 was = *at;
                  v = make_float4(v.x + was.x, v.y + was.y, v.z + was.z, v.w + was.w);
                }
                *at = v;
              }
            } else {
#pragma unroll
              for (int i = 0; i < HD / 8; ++i) {
                float2* at = reinterpret_cast<float2*>(row + 8 * i + 2 * tq);
                float2 v = make_float2(o[mw][i][2 * h], o[mw][i][2 * h + 1]);
                if (turn) {
                  const float2 was = *at;
                  v = make_float2(v.x + was.x, v.y + was.y);
                }
                *at = v;
              }
            }
          }
      }
      __syncthreads();
    }
    const bool whole = t0 == 0 && t1 == cons.n;
    const int slot = ((int)blockIdx.x * 2 + (t0 == 0)) * p.qn;
    for (int i = tid; i < nq * (HD / 4); i += kThreads) {
      const int q = i / (HD / 4), d = (i - q * (HD / 4)) * 4;
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int x = 0; x < KS; ++x) M = fmaxf(M, sML[x * QR + q].x);
#pragma unroll
      for (int x = 0; x < KS; ++x) {
        const float2 ml = sML[x * QR + q];
        L += M == -INFINITY ? 0.f : ml.y * ex2(ml.x - M);
      }
      const float4 v = *reinterpret_cast<const float4*>(sO + q * S::kPitch + d);
      if (whole) {
        int head, row;
        query_of(p, cons.unit, q, &head, &row);
        const float inv = L != 0.f ? 1.f / L : 0.f;
        bf16* out = (bf16*)p.a.out + (int64_t)cons.b * p.a.o_seq + (int64_t)row * p.a.o_row + (int64_t)head * p.a.o_head;
        store_act4(out + d, 0, make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv));
      } else {
        *reinterpret_cast<float4*>(p.part_o + (int64_t)(slot + q) * HD + d) = v;
        if (d == 0) p.part_ml[slot + q] = make_float2(M, L);
      }
    }
    cons.skip(p, t1 - t0);
    __syncthreads();  // sO (and sQ) and sML are free again
  }
  cp_async_wait<0>();
}

template <int HD, bool E8, int QN>
cudaError_t launch_qn(const PagedAttn& p, int grid, cudaStream_t st) {
  using S = Shape<HD, E8, QN>;
  static unsigned long long done = 0;
  auto k = k_paged_attn_tc<HD, E8, QN>;
  if (!smem_limit((const void*)k, S::kSmem, &done)) return cudaErrorInvalidValue;
  return launch_op(k, grid, kThreads, S::kSmem, st, false, 1, p);
}
template <int HD, bool E8>
cudaError_t launch_hd(const PagedAttn& p, int grid, cudaStream_t st) {
  switch (p.qn) {
    case 8: return launch_qn<HD, E8, 8>(p, grid, st);
    case 16: return launch_qn<HD, E8, 16>(p, grid, st);
    case 32: return launch_qn<HD, E8, 32>(p, grid, st);
    default: return launch_qn<HD, E8, 64>(p, grid, st);
  }
}

}  // namespace

namespace dmtp {

cudaError_t paged_attn_tc(const PagedAttn& p, const PagedPlan& pl, bool e8, cudaStream_t st) {
  if (p.m.head_dim == 64) return e8 ? launch_hd<64, true>(p, pl.grid, st) : launch_hd<64, false>(p, pl.grid, st);
  return e8 ? launch_hd<128, true>(p, pl.grid, st) : launch_hd<128, false>(p, pl.grid, st);
}

}  // namespace dmtp
