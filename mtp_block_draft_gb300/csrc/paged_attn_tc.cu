// Attention over a paged cache on the tensor cores: bf16 rows of head size 64 or 128, the
// cache in bf16 or E4M3.
//
// One pass over the cached rows bounds it: each byte of K and V feeds at most 64 queries of
// its kv head (rows x query heads), a few hundred operations. So the warps keep rings of
// 16-key blocks in flight by 16-byte asynchronous copies (the pages of the next 32 blocks in one
// read of the table) and work on 16-bit fragments with m16n8k16 products that need no staging
// beyond the block itself. Keys are the M side and queries the N
// side of both products (S^T = K Q^T, O^T = V^T P^T), so 8 queries fill an instruction. (The
// tcgen05 form wants 128 rows of keys and one thread to start each product of the whole CTA;
// a block would wait for its neighbours, and E4M3 rows would go through shared memory twice: built
// for 64 queries, one CTA of eight warps an SM, it took 96 us where this takes 66.)
//
//   QN queries    teams             a team's ring
//   8, 16         4 of one warp     16 keys a stage, no barrier but the warp's own
//   32            2 of two warps    32 keys a stage
//   64            one of four       64 keys a stage
//
// The smallest QN that holds a kv head's queries (of more than 64, chunks of 64). 32 sequences of
// 512 to 4096 positions, 4 kv heads of 128, us with QN 8 / 16 / 32 / 64: 8 queries in bf16 30.4 /
// 33.4 / 39.8 / 59.3, in E4M3 23.2 / 29.6 / 37.8 / 55.8; 16 42.5 / 35.8 / 41.6 / 61.0, 34.8 / 31.2 /
// 39.8 / 57.8; 32 68.5 / 53.0 / 44.5 / 64.3, 58.5 / 48.2 / 41.8 / 59.5; 64 121 / 93.3 / 78.5 / 71.6,
// 104 / 86.0 / 72.3 / 65.9 (E4M3 before its stages were looked through for rows of zeros: 1% more now).
//
// Times (us in a captured graph, the merge included): 32 sequences of 512 to 4096 bf16 positions,
// 8 queries a kv head, 30.3 (151 MB, 0.74 of the copy rate; with longer contexts each further byte
// costs what a copy would, 8 us do not grow); 4 sequences of 32768 in E4M3 31.2 (0.65, issue 50%);
// 64 queries in E4M3 66.4: dependent instructions of 12 warps an SM (issue 47%, tensor pipe 29%).
//
// A warp has at most 16 queries: with 32 (and half the conversions of E4M3 rows) only two CTAs fit
// an SM, and 32 sequences of 512 to 4096 E4M3 positions x 64 queries took 78 us instead of 65.
//
// Weights 2^(s - m) use a running maximum m per query that moves only when a score passes it
// by 2^8 (so most blocks skip the rescaling). bf16 caches: P as a bf16 pair (16 bits of each
// weight), two products a fragment. E4M3 caches: rows become fp16 exactly, the queries too
// after a power-of-two scale per query (but elements below 2^-29 of the query's largest, which
// keep 2^-37 of that), and P carries the value row's scale: with v = 2^e c
// and weight w, m follows log2(w 2^e) and P = w 2^(e - m), so what is rounded to fp16 is the
// row's contribution relative to the largest one; the sum of weights undoes the exponent in
// fp32. A weight's 11 bits stand against the 4 of a cached value; with fp16 pairs, as bf16 caches
// have them, 64 queries would take 73.9 us instead of 66.4, 32 48.6 instead of 42.3, 8 24.4
// instead of 23.5. (e stops at -60, and rows of zeros do not set m, see below.)
#include <cuda_fp16.h>

#include "paged_attn.cuh"

using namespace dmtp;

namespace {

constexpr int kThreads = 128;

template <int HD, bool E8, int QN>
struct Shape {
  static constexpr int NT = QN == 8 ? 1 : 2;        // 8-query blocks of a warp
  static constexpr int QG = QN / (8 * NT);          // warps of a team
  static constexpr int KS = 4 / QG;                 // teams
  static constexpr int RB = HD * (E8 ? 1 : 2);      // bytes of a cached row
  static constexpr int NSUB = 4 / KS;               // 16-key blocks of a team in a tile
  static constexpr int kBlock = 2 * 16 * RB + (E8 ? 128 : 0);
  static constexpr int kStage = NSUB * kBlock;      // of a team
  static constexpr int kPitch = HD + 4;             // floats of a joined row: no conflicts
  static constexpr int kJoin = QN * kPitch * 4 + KS * QN * 8;
  static constexpr int kMisc = KS * 8 * NSUB * 4;   // valid rows of the blocks
  // CTAs of an SM: registers (128 threads x 128 or 168) and a ring of two stages at least
  static constexpr int CTAS = HD == 64 ? 4 : QN == 8 ? (E8 ? 4 : 3) : E8 || QN == 16 ? 3 : 2;
  static constexpr int kRoom = 228 * 1024 / CTAS - 1024 - kJoin - kMisc;
  static constexpr int NST = kRoom / (KS * kStage) > 8 ? 8 : kRoom / (KS * kStage);
  static constexpr int kSmem = NST * KS * kStage + kJoin + kMisc;
  static_assert(NST >= 2, "a ring of two stages at least");
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
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
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

__device__ __forceinline__ uint32_t transpose8(uint32_t u) {  // an 8 x 8 block of 16-bit values
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(u));
  return r;
}
// Four E4M3 bytes as two pairs of halves.
__device__ __forceinline__ void e4m3_pairs(uint32_t u, uint32_t& lo, uint32_t& hi) {
  asm("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;}"
      : "=r"(lo), "=r"(hi) : "r"(u));
}
template <int QG>
__device__ __forceinline__ void team_sync(int team) {
  if (QG == 1)
    __syncwarp();
  else if (QG == 4)
    __syncthreads();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(32 * QG) : "memory");
}

// What a warp keeps of a piece: per 8-query block, queries 2 tq and 2 tq + 1.
template <int HD, int NT>
struct State {
  float o[NT][HD / 16][4];  // O^T: [16 columns of the head] x [8 queries]
  float m[NT][2], l[NT][2], rowf[NT][2];
  int top[NT][2];           // last position that the query sees
};

// The value rows of an E4M3 block that are all zeros, as bits. A lane looks at half a row.
template <int RB>
__device__ __forceinline__ unsigned zero_rows(const unsigned char* blk) {
  const int lane = threadIdx.x & 31;
  const uint4* half = reinterpret_cast<const uint4*>(blk + 16 * RB + (lane & 15) * RB + (lane >> 4) * (RB / 2));
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < RB / 32; ++i) bits |= half[i].x | half[i].y | half[i].z | half[i].w;
  const unsigned some = __ballot_sync(0xffffffffu, (bits & 0x7f7f7f7fu) != 0);
  return ~(some | some >> 16) & 0xffffu;
}

// One 16-key block: jb its first position, `ok` its rows that hold a position of the sequence.
// EDGE: some row is not seen by every query. `zeros` (if ZEROS): its value rows that are all zeros.
template <int HD, bool E8, int NT, bool EDGE, bool ZEROS = false>
__device__ __forceinline__ void block(const PagedAttn& p, State<HD, NT>& z,
                                      const uint32_t (&qf)[NT][HD / 16][2], const unsigned char* blk, int jb, unsigned ok,
                                      unsigned zeros = 0) {
  constexpr int RB = HD * (E8 ? 1 : 2), KK = HD / 16;
  const int lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3, mi = lane >> 3;
  const uint32_t sK = smem_u32(blk), sV = sK + 16 * RB;
  const float* sS = (const float*)(blk + 32 * RB);
  // (two accumulators a score: half as long a chain of dependent products)
  float s[NT][4], s1[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) s[n][i] = s1[n][i] = 0.f;
  {  // A fragments of K: rows (keys) 0-7 and 8-15 of two 16-byte steps. A row's steps are
     // permuted by exclusive or, so step k2 is the first one's address with k2's bits flipped.
    const uint32_t a0 = sK + tile_at<RB>((lane & 7) + 8 * (mi & 1), mi >> 1);
#pragma unroll
    for (int k2 = 0; k2 < KK; k2 += 2) {
      uint32_t a[2][4];
      if (E8) {  // a step holds the 16 columns of one product
        uint32_t kr[4];
        ldsm4(kr, a0 ^ (k2 << 4));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          e4m3_pairs(kr[2 * i], a[i][0], a[i][2]);
          e4m3_pairs(kr[2 * i + 1], a[i][1], a[i][3]);
        }
      } else {
        ldsm4(a[0], a0 ^ (2 * k2 << 4));
        ldsm4(a[1], a0 ^ (2 * k2 + 2 << 4));
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma16816<E8>(s[n], a[0], qf[n][k2][0], qf[n][k2][1]);
        mma16816<E8>(s1[n], a[1], qf[n][k2 + 1][0], qf[n][k2 + 1][1]);
      }
    }
  }
  // the thread's keys g and g + 8
  float kf[2], ve[2], vm[2], vi[2];
  if (E8) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      kf[h] = sS[g + 8 * h];
      // 2^ve vm, ve its exponent but at least -60: rows of smaller ones neither lose their weight
      // in the sum (2^-86 of the largest is the least that counts) nor make it overflow
      const float vs = sS[16 + g + 8 * h];
      const bool zero = ZEROS && (zeros >> (g + 8 * h) & 1);
      const uint32_t u = zero ? 67u : max(__float_as_uint(vs) >> 23, 67u);
      ve[h] = __uint_as_float(0x4b000000u | u) - 8388735.f;
      vi[h] = pow2f(127 - (int)u);
      vm[h] = zero ? 0.f : vs * vi[h];
    }
  }
  uint32_t pk[NT][2], pb[NT][2], lb[NT][2];
  bool rise = false;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v = (s[n][2 * h + y] + s1[n][2 * h + y]) * z.rowf[n][y];
        if (E8) v = fmaf(v, kf[h], ve[h]);
        if (EDGE) {
          const int key = g + 8 * h, j = jb + key;
          const bool seen = (ok >> key & 1) && j <= z.top[n][y] &&
                            (p.a.window <= 0 || j > z.top[n][y] - p.a.window);
          v = seen ? v : -INFINITY;
        }
        s[n][2 * h + y] = v;
        rise = rise || v > z.m[n][y] + 8.f;
      }
  if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float mx = fmaxf(s[n][y], s[n][2 + y]);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        if (mx > z.m[n][y] + 8.f) {
          const float fix = ex2(z.m[n][y] - mx);  // 0 for the first
          z.m[n][y] = mx;
          z.l[n][y] *= fix;
#pragma unroll
          for (int i = 0; i < KK; ++i) {
            z.o[n][i][y] *= fix;
            z.o[n][i][2 + y] *= fix;
          }
        }
      }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const float r0 = z.m[n][0] == -INFINITY ? 0.f : z.m[n][0], r1 = z.m[n][1] == -INFINITY ? 0.f : z.m[n][1];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float w0 = ex2(s[n][2 * h] - r0), w1 = ex2(s[n][2 * h + 1] - r1);
      if (E8) {
        z.l[n][0] = fmaf(w0, vi[h], z.l[n][0]);
        z.l[n][1] = fmaf(w1, vi[h], z.l[n][1]);
        pk[n][h] = pack_f16(w0 * vm[h], w1 * vm[h]);
      } else {
        z.l[n][0] += w0;
        z.l[n][1] += w1;
        pk[n][h] = pack_bf16(w0, w1);
        lb[n][h] = transpose8(pack_bf16(w0 - __uint_as_float(pk[n][h] << 16),
                                        w1 - __uint_as_float(pk[n][h] & 0xffff0000u)));
      }
      pb[n][h] = transpose8(pk[n][h]);
    }
  }
  // O^T += V^T P^T: A fragments of V^T, columns of the head as rows
  bool odd = false;  // an infinity or NaN among values that not every query sees
  {
    if (E8) {
      const uint32_t v0 = sV + tile_at<RB>((lane & 7) + 8 * (mi & 1), mi >> 1);
#pragma unroll
      for (int c = 0; c < KK; c += 2) {
        uint32_t v[4];  // step c: keys 0-7, 8-15; step c + 1 likewise
        ldsm4_t(v, v0 ^ (c << 4));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          // bytes of keys 2 tq, 2 tq + 1 by column: rows g hold columns 2 g, rows g + 8 2 g + 1
          uint32_t a[4];
          e4m3_pairs(__byte_perm(v[2 * i], 0, 0x3120), a[0], a[1]);
          e4m3_pairs(__byte_perm(v[2 * i + 1], 0, 0x3120), a[2], a[3]);
          if (EDGE) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint32_t f = finite_pair<true>(a[x]);
              odd = odd || f != a[x];
              a[x] = f;
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16816<true>(z.o[n][c + i], a, pb[n][0], pb[n][1]);
        }
      }
    } else {
      const uint32_t v0 = sV + tile_at<RB>((lane & 7) + 8 * (mi >> 1), mi & 1);
#pragma unroll
      for (int i = 0; i < KK; ++i) {
        uint32_t a[4];  // keys 0-7: columns 0-7, 8-15 of the block; keys 8-15 likewise
        ldsm4_t(a, v0 ^ (2 * i << 4));
        if (EDGE) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint32_t f = finite_pair<false>(a[x]);
            odd = odd || f != a[x];
            a[x] = f;
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma16816<false>(z.o[n][i], a, pb[n][0], pb[n][1]);
          mma16816<false>(z.o[n][i], a, lb[n][0], lb[n][1]);
        }
      }
    }
  }
  if (EDGE && __any_sync(0xffffffffu, odd)) {
    // give those values to the queries that do see them: weights by shuffle from the lane
    // that holds them, values from shared memory
    const unsigned char* vrow = blk + 16 * RB;
#pragma unroll 1
    for (int key = 0; key < 16; ++key) {
      const int from = (key & 7) * 4 + tq;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint32_t lo = __shfl_sync(0xffffffffu, pk[n][0], from), hi = __shfl_sync(0xffffffffu, pk[n][1], from);
        const uint32_t u = key < 8 ? lo : hi;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const uint32_t bits = y ? u >> 16 : u & 0xffffu;
          const float w = E8 ? h2_to_f2(bits).x : __uint_as_float(bits << 16);
          if (w != 0.f) {
#pragma unroll
            for (int i = 0; i < KK; ++i)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int d = E8 ? 16 * i + 2 * g + h : 16 * i + g + 8 * h;
                const int byte = d * (E8 ? 1 : 2);
                const unsigned char* at = vrow + tile_at<RB>(key, byte >> 4) + (byte & 15);
                const float val = E8 ? h2_to_f2(e4m3x2_to_h2(*at)).x : __bfloat162float(*(const bf16*)at);
                if (!(fabsf(val) <= 3.402823466e38f)) z.o[n][i][2 * h + y] = fmaf(w, val, z.o[n][i][2 * h + y]);
              }
          }
        }
      }
    }
  }
}

template <int HD, bool E8, int QN>
__global__ void __launch_bounds__(kThreads, Shape<HD, E8, QN>::CTAS) k_paged_attn_tc(const PagedAttn p) {
  using S = Shape<HD, E8, QN>;
  constexpr int NT = S::NT, QG = S::QG, KS = S::KS, RB = S::RB, NST = S::NST, NSUB = S::NSUB;
  constexpr int KK = HD / 16;
  extern __shared__ __align__(128) unsigned char smem[];
  float* sO = (float*)(smem + NST * KS * S::kStage);
  float2* sML = (float2*)(sO + QN * S::kPitch);
  uint32_t* sOk = (uint32_t*)(sML + KS * QN);
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, g = lane >> 2, tq = lane & 3;
  const int team = wid / QG, qg = wid % QG;
  unsigned char* ring = smem + team * NST * S::kStage;
  sOk += team * 8 * NSUB;
  pdl_trigger();
  Deal deal;
  Tiles cons = my_tiles<bf16>(p, deal, kThreads);
  if (cons.pos >= cons.end) return;
  Tiles prod = cons;

  // ---- copies: a team brings the blocks team + KS i of every tile ----
  constexpr int CPR = RB / 16, RPI = 32 * QG / CPR, NI = RPI < 16 ? 16 / RPI : 1;  // rows of one copy of the team
  const bool copies = RPI <= 16 || (qg * 32 + lane) / CPR < 16;  // (a team may be larger than a block)
  const bool paged16 = p.m.page_size % 16 == 0;  // a block lies in one page
  // Cached rows pass through L2 once: the tables, lengths and partial results should outlive them
  // there. (With several chunks of queries it makes no difference: 129.3 us, kept like the rest 130.5.)
  const uint64_t stream = policy_evict_first();
  // Pages of this team's blocks, 32 of them at a time: lane i holds the block of tile
  // win_t + i / NSUB, number i % NSUB, of sequence win_b. One table read serves them all.
  int win_b = -1, win_t = 0, win_page = -1, win_off = 0;
  auto look_up = [&]() {  // the window holds the next tile to bring
    if (prod.pos >= prod.end || (prod.b == win_b && prod.t >= win_t && prod.t < win_t + 32 / NSUB)) return;
    win_b = prod.b;
    win_t = prod.t;
    const int j = prod.first + (win_t + lane / NSUB) * 64 + (team + KS * (lane % NSUB)) * 16;
    win_page = -1;
    // (no further than this CTA's tiles: pages that others read are theirs to report)
    if (paged16 && j < prod.len && j + 15 >= seq_low(p, prod.len) && lane / NSUB < prod.end - prod.pos)
      win_page = page_of(p.m, prod.b, j, win_off, p.err);
  };
  int stage_in = 0;
  auto produce = [&]() {
    if (prod.pos < prod.end) {
      const int kvh = prod.unit / p.chunks;
      const int tl = qg * 32 + lane, rin = tl / CPR, c = tl % CPR;
#pragma unroll
      for (int i = 0; i < NSUB; ++i) {
        unsigned char* blk = ring + stage_in * S::kStage + i * S::kBlock;
        const uint32_t dst = smem_u32(blk);
        const int jb = prod.first + prod.t * 64 + (team + KS * i) * 16;
        int rows = min(16, prod.len - jb);
        unsigned ok;
        if (paged16) {
          const int src_lane = (prod.t - win_t) * NSUB + i;
          const int page = __shfl_sync(0xffffffffu, win_page, src_lane);
          const int off = __shfl_sync(0xffffffffu, win_off, src_lane);
          if (page < 0) rows = 0;
          ok = rows >= 16 ? 0xffffu : rows > 0 ? (1u << rows) - 1 : 0u;
          const int64_t line = (int64_t)kvh * p.m.page_size + (rows > 0 ? off : 0);
          const int64_t pg = rows > 0 ? page : 0;
          const int64_t at = (pg * p.m.page_stride + line * HD) * (E8 ? 1 : 2) + tl * 16;
          const char *ka = (const char*)p.k + at, *va = (const char*)p.v + at;
          const int64_t sat = pg * p.m.scale_stride + line + (lane & 15);
          if (rows >= 16) {
#pragma unroll
            for (int x = 0; x < NI; ++x) {
              if (!copies) break;
              const uint32_t d = dst + tile_at<RB>(x * RPI + rin, c);
              cp_async16_hint(d, ka + x * (512 * QG), stream);
              cp_async16_hint(d + 16 * RB, va + x * (512 * QG), stream);
            }
            if (E8 && qg == 0) cp_async4(dst + 32 * RB + lane * 4, (lane < 16 ? p.ks : p.vs) + sat, 4);
          } else {
            // (a row that is not there is not read: its address is that of one that is)
#pragma unroll
            for (int x = 0; x < NI; ++x) {
              if (!copies) break;
              const int r = x * RPI + rin, bytes = r < rows ? 16 : 0;
              const uint32_t d = dst + tile_at<RB>(r, c);
              cp_async16(d, bytes ? ka + x * (512 * QG) : (const char*)p.k, bytes);
              cp_async16(d + 16 * RB, bytes ? va + x * (512 * QG) : (const char*)p.v, bytes);
            }
            if (E8 && qg == 0) {
              const float* src = (lane < 16 ? p.ks : p.vs);
              const bool there = (lane & 15) < rows;
              cp_async4(dst + 32 * RB + lane * 4, there ? src + sat : src, there ? 4 : 0);
            }
          }
        } else {
          const int j = jb + (lane & 15);
          int64_t at = -1;
          int64_t sat = 0;
          if (j < prod.len && j >= seq_low(p, prod.len)) {
            int o;
            const int pg = page_of(p.m, prod.b, j, o, p.err);
            const int64_t line = (int64_t)kvh * p.m.page_size + o;
            if (pg >= 0) {
              at = ((int64_t)pg * p.m.page_stride + line * HD) * (E8 ? 1 : 2);
              sat = (int64_t)pg * p.m.scale_stride + line;
            }
          }
          ok = __ballot_sync(0xffffffffu, at >= 0) & 0xffffu;
#pragma unroll
          for (int x = 0; x < NI; ++x) {
            const int r = x * RPI + rin;
            const int64_t a = __shfl_sync(0xffffffffu, at, r & 15);
            if (!copies) break;
            const int bytes = a < 0 ? 0 : 16;
            const int64_t src = a < 0 ? 0 : a + c * 16;
            const uint32_t d = dst + tile_at<RB>(r, c);
            cp_async16(d, (const char*)p.k + src, bytes);
            cp_async16(d + 16 * RB, (const char*)p.v + src, bytes);
          }
          if (E8 && qg == 0)
            cp_async4(dst + 32 * RB + lane * 4, (lane < 16 ? p.ks : p.vs) + sat, at < 0 ? 0 : 4);
        }
        if (lane == 0 && qg == 0) sOk[stage_in * NSUB + i] = ok;
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
    State<HD, NT> z;
    // B fragments of Q^T: query g, columns 2 tq.. in the products' order, or, as the bytes of
    // an E4M3 K come, four consecutive ones
    uint32_t qf[NT][KK][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int t = (qg * NT + n) * 8 + g;
      int head, row;
      query_of(p, cons.unit, t, &head, &row);
      const bf16* qp = (const bf16*)p.a.q + (int64_t)cons.b * p.a.q_seq + (int64_t)row * p.a.q_row + (int64_t)head * p.a.q_head;
#pragma unroll
      for (int k = 0; k < KK; ++k) {
        qf[n][k][0] = qf[n][k][1] = 0;
        if (t < nq) {
          if (E8) {
            const uint2 u = *reinterpret_cast<const uint2*>(qp + 16 * k + 4 * tq);
            qf[n][k][0] = u.x;
            qf[n][k][1] = u.y;
          } else {
            qf[n][k][0] = *reinterpret_cast<const uint32_t*>(qp + 16 * k + 2 * tq);
            qf[n][k][1] = *reinterpret_cast<const uint32_t*>(qp + 16 * k + 8 + 2 * tq);
          }
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int q0 = (qg * NT + n) * 8;
      int head, row;
      float down = p.scale2;
      if (E8) {  // bf16 -> fp16, the query's largest magnitude brought into [2^12, 2^13)
        uint32_t big = 0;
#pragma unroll
        for (int k = 0; k < KK; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t a = qf[n][k][i] << 16 & 0x7fff0000u, b = qf[n][k][i] & 0x7fff0000u;
            if (a < 0x7f800000u) big = max(big, a);
            if (b < 0x7f800000u) big = max(big, b);
          }
        big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
        // 2^(12 - floor(log2 big)), kept inside the normal range
        const int e = big ? min(max(12 - ((int)(big >> 23) - 127), -126), 126) : 0;
        const float up = pow2f(e);
        down *= pow2f(-e);
#pragma unroll
        for (int k = 0; k < KK; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            qf[n][k][i] = pack_f16(__uint_as_float(qf[n][k][i] << 16) * up,
                                   __uint_as_float(qf[n][k][i] & 0xffff0000u) * up);
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        z.rowf[n][y] = __shfl_sync(0xffffffffu, down, (2 * tq + y) * 4);
        z.m[n][y] = -INFINITY;
        z.l[n][y] = 0.f;
        z.top[n][y] = -1;
        if (q0 + 2 * tq + y < nq) {
          query_of(p, cons.unit, q0 + 2 * tq + y, &head, &row);
          z.top[n][y] = cons.len - p.a.rows + row;
        }
      }
#pragma unroll
      for (int i = 0; i < KK; ++i) z.o[n][i][0] = z.o[n][i][1] = z.o[n][i][2] = z.o[n][i][3] = 0.f;
    }

    for (int t = t0; t < t1; ++t) {
      cp_async_wait<NST - 2>();
      team_sync<QG>(team);  // this stage is here; the one before has been used
      produce();
      // A value row of zeros adds nothing to the output, so its scale (1, as rows are written) must
      // not set the maximum that the others' weights are rounded against: with values of 1e-6
      // beside it they would all round to 0. Stages with a scale of 1 or more are looked through,
      // and such a row counts with the least exponent. (64 queries 65.4 -> 66.4 us, 8 23.2 -> 23.4;
      // looking where the maximum rises, whatever the scale, 68.4 and 24.0.)
      bool ones = false;
      if (E8) {
        const unsigned char* at = ring + stage * S::kStage + 32 * RB + 64;  // the first block's v scales
#pragma unroll
        for (int i = 0; i < (NSUB + 1) / 2; ++i) {
          const int sub = min(2 * i + (lane >> 4), NSUB - 1);
          ones = ones || reinterpret_cast<const float*>(at + sub * S::kBlock)[lane & 15] >= 1.f;
        }
        ones = __any_sync(0xffffffffu, ones);
      }
#pragma unroll 1
      for (int i = 0; i < NSUB; ++i) {
        const unsigned char* blk = ring + stage * S::kStage + i * S::kBlock;
        const unsigned ok = sOk[stage * NSUB + i];
        const int jb = cons.first + t * 64 + (team + KS * i) * 16;
        const unsigned zeros = E8 && ones ? zero_rows<RB>(blk) & ok : 0u;
        if (E8 && zeros)
          block<HD, E8, NT, true, true>(p, z, qf, blk, jb, ok, zeros);
        else if (ok == 0xffffu && jb + 15 <= cons.len - p.a.rows && (p.a.window <= 0 || jb >= cons.len - p.a.window))
          block<HD, E8, NT, false>(p, z, qf, blk, jb, ok);
        else if (ok)
          block<HD, E8, NT, true>(p, z, qf, blk, jb, ok);
      }
      stage = stage + 1 == NST ? 0 : stage + 1;
    }

    // ---- join the teams in order, and write ----
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float l = z.l[n][y];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        if (g == 0) sML[team * QN + (qg * NT + n) * 8 + 2 * tq + y] = make_float2(z.m[n][y], l);
      }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int q = (qg * NT + n) * 8 + 2 * tq + y;
        float M = -INFINITY;
#pragma unroll
        for (int i = 0; i < KS; ++i) M = fmaxf(M, sML[i * QN + q].x);
        const float f = M == -INFINITY ? 0.f : ex2(z.m[n][y] - M);
#pragma unroll
        for (int i = 0; i < KK; ++i) {
          z.o[n][i][y] *= f;
          z.o[n][i][2 + y] *= f;
        }
      }
#pragma unroll
    for (int turn = 0; turn < KS; ++turn) {
      if (turn == team) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            float* row = sO + ((qg * NT + n) * 8 + 2 * tq + y) * S::kPitch;
#pragma unroll
            for (int i = 0; i < KK; ++i) {
              const float a = z.o[n][i][y], b = z.o[n][i][2 + y];
              if (E8) {
                float2* at = reinterpret_cast<float2*>(row + 16 * i + 2 * g);
                const float2 was = turn ? *at : make_float2(0.f, 0.f);
                *at = make_float2(a + was.x, b + was.y);
              } else {
                float* at = row + 16 * i + g;
                at[0] = turn ? at[0] + a : a;
                at[8] = turn ? at[8] + b : b;
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
      for (int x = 0; x < KS; ++x) M = fmaxf(M, sML[x * QN + q].x);
#pragma unroll
      for (int x = 0; x < KS; ++x) {
        const float2 ml = sML[x * QN + q];
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
    if (t0 == 0 && tid == 0) leave_note(p, deal, cons);
    cons.skip(p, t1 - t0);
    __syncthreads();  // sO and sML are free again
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

int paged_tc_grid(int head_dim, bool e8, int qn) {
#define DMTP_CTAS(HD_, E8_)                                                           \
  (qn == 8 ? Shape<HD_, E8_, 8>::CTAS : qn == 16 ? Shape<HD_, E8_, 16>::CTAS          \
                                      : qn == 32 ? Shape<HD_, E8_, 32>::CTAS : Shape<HD_, E8_, 64>::CTAS)
  return 152 * (head_dim == 64 ? (e8 ? DMTP_CTAS(64, true) : DMTP_CTAS(64, false))
                               : (e8 ? DMTP_CTAS(128, true) : DMTP_CTAS(128, false)));
#undef DMTP_CTAS
}

cudaError_t paged_attn_tc(const PagedAttn& p, const PagedPlan& pl, bool e8, cudaStream_t st) {
  if (p.m.head_dim == 64) return e8 ? launch_hd<64, true>(p, pl.grid, st) : launch_hd<64, false>(p, pl.grid, st);
  return e8 ? launch_hd<128, true>(p, pl.grid, st) : launch_hd<128, false>(p, pl.grid, st);
}

}  // namespace dmtp
