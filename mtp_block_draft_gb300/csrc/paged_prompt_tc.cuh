// Attention of many rows over a paged cache on the 5th-generation tensor cores: bf16 rows of head
// sizes up to 128.
//
// A CTA has a unit: 256 queries of one kv head as two halves of 128, and goes through its keys 128 at a
// time. Per block of keys and half
//   S = Q K^T   tcgen05, M = 128 queries, N = 128 keys; Q and K from shared memory
//   softmax     a warpgroup, a thread a query: P = 2^(s - m) as bf16 over S's place in TMEM
//   O += P V    tcgen05, A = P from TMEM, B = V as its rows lie (keys by columns, MN-major)
// S and O of both halves fill TMEM's 512 columns; while one half's softmax runs, the tensor cores
// work for the other. The reference m of a query moves only when a score passes it by 2^8, so that O
// is hardly ever rescaled. A thread holds the 128 scores of its query and block in registers, which
// the softmax's warps get from the others (184 and 72 a thread; 128 for all spilled, and a second
// reading from TMEM instead took 3.06 ms where this takes 1.47). The products of a block begin with the
// weights of its first 64 keys. One warp, uniform, starts them all: as one thread of a diverged warp it
// needed 4200 cycles for the 32 products of a block, which take 2048.
//
// Keys and values come into a ring of shared-memory slots:
//   bf16, whole boxes of a page (page sizes that 128 divides or that divide 128, heads of 64 or 128)
//     by TMA, a box a lane, outside the tensor where a page is not looked up (zeros);
//   other bf16 rows, and V at a sequence's end (its rows past the end may be anything) row by row by
//     16-byte copies (a prompt of 16384 rows 3.07 ms so, 1.46 by TMA);
//   E4M3 and E2M1 rows as they lie, by bulk copies of the same boxes, three ahead, which six warps
//     turn into bf16 (over 16384 4-bit positions 465 us; through registers, for other pages, 548).
//
// What bounds it: 16384 rows of 32 / 4 heads of 128, causal: 1.47 ms, 1490 TFLOP/s, 0.87 of what cuBLAS
// sustains at the power limit; a block of keys costs about 3000 cycles where its products take 2048,
// the chain of one half's softmax (1400), products (1024) and barriers. With a bias 2.06 ms, capped
// 2.57: packed fp32 instructions take two cycles a warp, and those of two warps an SM quarter add up.
// 4-bit rows without a bias 277 us (bf16 209): the conversions. Short prompts pay about 5 us a unit
// for its queries, first block and output (4 prompts of 1021 to 2047 rows, uncapped: 160 us, 0.34 of
// the burst rate).
//
// A row may see any interval of positions: a block that not every query of a warp sees whole is
// masked there. In such a block a weight is 0 where a value may be infinite or NaN, and the tensor
// cores' 0 * inf would reach rows that do not see it: the loader looks through those blocks' values,
// and a unit with one that is not finite, or with a page that is none, is computed again row by row.
#pragma once

#include "paged_prompt.cuh"

using namespace dmtp;

namespace {

constexpr int kTile = 256, kKeys = 128, kLoaders = 224;

template <int HD, Rows F>
struct Shape {
  static constexpr int kThreads = 512;                       // softmax 256, loaders 224, products
  // registers of a softmax thread and of the others: together what 512 threads are launched with
  static constexpr int kMine = F == kRaw ? 184 : 168, kOther = F == kRaw ? 72 : 88;
  static_assert(256 * (kMine + kOther) <= 65536, "registers");
  static constexpr uint32_t kSlot = kKeys * HD * 2;          // 128 rows of K or V
  static constexpr int NS = F == kRaw ? (HD == 64 ? 8 : 5) : HD == 64 ? 6 : F == kE2M1 ? 4 : 3;
  // E4M3 and E2M1 rows as they lie, on their way: values, block scales, the rows' scales
  static constexpr uint32_t kValues = F == kRaw ? 0 : kKeys * (F == kE4M3 ? HD : HD / 2);
  static constexpr uint32_t kBlocks = F == kE2M1 ? kKeys * HD / 16 : 0;
  static constexpr uint32_t kStage = F == kRaw ? 0 : kValues + kBlocks + kKeys * 4;
  static constexpr int ST = F == kRaw ? 0 : 3;
  static constexpr uint32_t kQ = 2 * 128 * HD * 2;
  static constexpr uint32_t kHead = 512 + 2 * kKeys * 6;     // barriers, rows of two blocks
  static constexpr uint32_t kSmem = kHead + 1024 + kQ + NS * kSlot + ST * kStage;
  static_assert(kSmem <= 232448, "shared memory");
};

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// byte offset of the 16-byte chunk c (0..7) of row r inside a 128-byte-swizzled block
__device__ __forceinline__ uint32_t sw128(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }
// D[tmem] (+)= A[tmem] B[smem], bf16, fp32 accumulate.
__device__ __forceinline__ void umma_bf16_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// V as its rows lie: 64 columns (128 bytes) of 8 keys are a swizzled kilobyte, the next 8 keys
// follow, the next 64 columns are kKeys rows further.
__device__ __forceinline__ uint64_t umma_desc_mn(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(kKeys * 128 >> 4) << 16;  // leading byte offset: along the columns
  d |= (uint64_t)(1024 >> 4) << 32;         // stride byte offset: along the keys
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
// 32 columns of this warp's 32 lanes, without a wait.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[4][32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[c][i]));  // no use moves above the wait
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// `bytes` bytes (a multiple of 16, both addresses too) from global to shared memory.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(bar)
               : "memory");
}
// 4-D tiled TMA load (x = inner coordinate); what lies outside the tensor becomes zeros.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* tm, int x, int y, int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"((uint64_t)tm), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}
template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ bool odd_pair(uint32_t u) {  // an infinity or NaN among two bf16
  return (u & 0x7f80u) == 0x7f80u || (u & 0x7f800000u) == 0x7f800000u;
}
// Output columns d .. d + 3 of query t of a tile: final, or a part of a split unit.
__device__ __forceinline__ bf16* out_row(const PagedPrompt& p, const PromptTile& w, int kvh, int t) {
  const int r = (w.q0 + t) / p.group, head = kvh * p.group + (w.q0 + t - r * p.group);
  return (bf16*)p.a.out + (int64_t)(w.row0 + r) * p.a.o_row + (int64_t)head * p.a.o_head;
}

// The queries of a unit over the positions [j_lo, j_hi), row by row on the CUDA cores: a warp takes a
// query, a lane a key of 32 and then eight columns. Called by the 8 warps of the softmax.
template <Rows F>
__device__ __noinline__ void row_by_row(const PagedPrompt& p, const PromptTile& w, int kvh, int j_lo, int j_hi,
                                        int64_t part) {
  const int lane = threadIdx.x & 31, hd = p.m.head_dim;
  for (int t = threadIdx.x >> 5; t < w.count; t += 8) {
    const PromptQuery q = prompt_query(p, w, t);
    const int head = kvh * p.group + q.head;
    const bf16* src = (const bf16*)p.a.q + (int64_t)q.row * p.a.q_row + (int64_t)head * p.a.q_head;
    const float slope = p.a.scores.slopes ? __ldg(p.a.scores.slopes + head) * 1.4426950408889634f : 0.f;
    float m = -INFINITY, l = 0.f, o[8] = {};
    const int last = min(q.hi, j_hi);
    for (int j0 = max(q.lo, j_lo); j0 < last; j0 += 32) {
      const int j = j0 + lane;
      int page = -1, off = 0;
      if (j < last) page = page_of(p.m, w.b, j, off, p.err);
      const int64_t line = (int64_t)kvh * p.m.page_size + off;
      float x = -INFINITY;
      if (page >= 0) {
        const float s = F == kRaw ? 1.f : __ldg(p.ks + (int64_t)page * p.m.scale_stride + line);
        x = 0.f;
        for (int c = 0; c < hd; c += 8) {
          float k[8], a[8];
          load8<bf16, F>(p, p.k, page, line, c, s, k);
          Raw<bf16> raw;
          raw.u[0] = __ldg(reinterpret_cast<const uint4*>(src + c));
          values(raw, a);
#pragma unroll
          for (int e = 0; e < 8; ++e) x = fmaf(a[e], k[e], x);
        }
        x *= p.scale2;
        if (p.capl > 0.f) x = p.capl * soft_tanh(x * p.cap_inv);
        x = fmaf(-slope, (float)abs(q.pos - j), x);
      }
      const float n = fmaxf(m, warp_max(x)), ref = n == -INFINITY ? 0.f : n, fix = ex2(m - ref);
      m = n;
      const float weight = ex2(x - ref);
      l = l * fix + weight;
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] *= fix;
      for (int k = 0; k < 32; ++k) {
        const float a = __shfl_sync(0xffffffffu, weight, k);
        const int pg = __shfl_sync(0xffffffffu, page, k);
        const int64_t ln = __shfl_sync(0xffffffffu, line, k);
        if (a != 0.f && pg >= 0 && 8 * lane < hd) {
          float v[8];
          load8<bf16, F>(p, p.v, pg, ln, 8 * lane, F == kRaw ? 1.f : __ldg(p.vs + (int64_t)pg * p.m.scale_stride + ln), v);
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = fmaf(a, v[e], o[e]);
        }
      }
    }
    l = warp_sum(l);
    if (8 * lane < hd) {
      if (p.splits > 1) {
        float* to = p.part_o + (part + t) * hd + 8 * lane;
        *reinterpret_cast<float4*>(to) = make_float4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<float4*>(to + 4) = make_float4(o[4], o[5], o[6], o[7]);
      } else {
        const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] *= inv;
        store8(out_row(p, w, kvh, t) + 8 * lane, true, o);
      }
    }
    if (p.splits > 1 && lane == 0) p.part_ml[part + t] = make_float2(m, l);
  }
}

// The largest of a block's scores.
__device__ __forceinline__ float top_of(const uint32_t (&r)[4][32], float (&tops)[4]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    tops[c] = fmaxf(__uint_as_float(r[c][0]), __uint_as_float(r[c][1]));
#pragma unroll
    for (int e = 2; e < 32; e += 2) tops[c] = max3(tops[c], __uint_as_float(r[c][e]), __uint_as_float(r[c][e + 1]));
  }
  return max3(fmaxf(tops[0], tops[1]), tops[2], tops[3]);
}
// What a thread of the softmax knows of its query.
struct Query {
  int lo, hi, pos;
  float slope, m, l;
};
// Where the query does not see one of the 32 keys from j on: minus infinity.
__device__ __forceinline__ void mask32(const Query& q, uint32_t (&r)[32], int j) {
  const int from = q.lo - j;
  const unsigned n = q.hi > q.lo ? q.hi - q.lo : 0;
#pragma unroll
  for (int e = 0; e < 32; ++e) r[e] = (unsigned)(e - from) < n ? r[e] : 0xff800000u;
}
// Capped and biased scores of 32 keys from j on, in base 2, less `ref`. `behind`: none of them is past a
// query's own position, in the whole warp. Two packed instructions take the time of four others here,
// so the cap's polynomial has the cap and the scale in its coefficients: cap tanh(s by) is
// s (a0 + a1 s^2 + ..), 6 of them a pair.
struct Cap {
  float near, a[5];  // |s| up to `near` takes the polynomial (tanh(y) / y to 2e-8 for |y| <= 1/2)
};
__device__ __forceinline__ Cap cap_of(const PagedPrompt& p, float scale) {
  const float by = scale * p.cap_inv, t = by * by;
  Cap c;
  c.near = 0.5f / by;
  c.a[0] = p.capl * by;
  c.a[1] = c.a[0] * t * -0.333331435918808f;
  c.a[2] = c.a[0] * (t * t) * 0.13325878977775574f;
  c.a[3] = c.a[0] * (t * t * t) * -0.05304549261927605f;
  c.a[4] = c.a[0] * (t * t * t * t) * 0.01724148541688919f;
  return c;
}
__device__ __forceinline__ void scores32(const PagedPrompt& p, const Query& q, const Cap& cap, float scale, float ref,
                                         uint32_t (&r)[32], int j, bool behind) {
  auto at = [&](int e) { return pack(__uint_as_float(r[e]), __uint_as_float(r[e + 1])); };
  auto put = [&](int e, f32x2 v) {
    const float2 x = unpack(v);
    r[e] = __float_as_uint(x.x);
    r[e + 1] = __float_as_uint(x.y);
  };
  if (p.capl > 0.f) {
    const float less = p.a.scores.slopes ? 0.f : -ref;
    float most = 0.f;
#pragma unroll
    for (int e = 0; e < 32; e += 2) most = max3(most, fabsf(__uint_as_float(r[e])), fabsf(__uint_as_float(r[e + 1])));
    // (a NaN is no maximum, and comes through either form; a scale that leaves no polynomial has none)
    if (__all_sync(0xffffffffu, most <= cap.near && cap.a[4] != 0.f)) {
#pragma unroll
      for (int e = 0; e < 32; e += 2) {
        const f32x2 x = at(e), t = mul2(x, x);
        f32x2 v = fma2(t, both(cap.a[4]), both(cap.a[3]));
        v = fma2(t, v, both(cap.a[2]));
        v = fma2(t, v, both(cap.a[1]));
        v = fma2(t, v, both(cap.a[0]));
        put(e, fma2(x, v, both(less)));
      }
    } else {
      const float by = scale * p.cap_inv;
#pragma unroll
      for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(fmaf(p.capl, soft_tanh(__uint_as_float(r[e]) * by), less));
    }
    if (!p.a.scores.slopes) return;
    scale = 1.f;
  }
  const float d = (float)(q.pos - j);
  if (behind) {
    const f32x2 by = both(scale);
    const float base = fmaf(-q.slope, d, -ref);
#pragma unroll
    for (int e = 0; e < 32; e += 2)
      put(e, fma2(at(e), by, pack(fmaf(q.slope, (float)e, base), fmaf(q.slope, (float)(e + 1), base))));
  } else {
#pragma unroll
    for (int e = 0; e < 32; ++e)
      r[e] = __float_as_uint(fmaf(-q.slope, fabsf(d - (float)e), __uint_as_float(r[e]) * scale) - ref);
  }
}

template <int HD, Rows F, bool MOD>
__global__ void __launch_bounds__(Shape<HD, F>::kThreads, 1)
    k_prompt_tc(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const PagedPrompt p) {
  using Sh = Shape<HD, F>;
  constexpr int NS = Sh::NS;
  extern __shared__ __align__(1024) unsigned char smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, kvh = blockIdx.y, hd = p.m.head_dim;
  if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0 && warp == 0) prompt_report(p);
  PromptTile w;
  if (!prompt_tile(p, blockIdx.x, w)) {
    pdl_trigger();
    return;
  }
  uint64_t* full = (uint64_t*)smem;  // [NS] a slot's rows are there
  uint64_t* empty = full + NS;       // [NS] the products have read it
  uint64_t* s_full = empty + NS;     // [2] a half's scores
  uint64_t* p_full = s_full + 2;     // [2][2] its weights of the block's first 64 keys, of the others
  uint64_t* o_full = p_full + 4;     // [2] its last product
  uint64_t* st_full = o_full + 2;    // [ST] rows as they lie are there
  uint64_t* st_empty = st_full + Sh::ST;  // [ST] and have been turned into bf16
  uint32_t* tmem_slot = (uint32_t*)(st_empty + Sh::ST);
  int* s_span = (int*)(tmem_slot + 1);  // [4] least lo, largest hi; largest lo, least hi (what every query sees)
  int* s_odd = s_span + 4;              // the unit has to be computed row by row
  int* s_page = (int*)(smem + 512);                // [2][kKeys] of the blocks in turn: a row's page (-1: it
  uint16_t* s_off = (uint16_t*)(s_page + 2 * kKeys);  // is not there) and which row of that it is
  unsigned char* sQ = smem + Sh::kHead;
  sQ += (1024 - (smem_u32(sQ) & 1023)) & 1023;
  unsigned char* ring = sQ + Sh::kQ;
  unsigned char* stages = ring + NS * Sh::kSlot;
  const bool bulk = F != kRaw && p.box;  // one warp brings the rows, the other loaders convert them
  const int fillers = bulk ? kLoaders - 32 : kLoaders;
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(smem_u32(full + i), fillers);
      mbar_init(smem_u32(empty + i), 1);
    }
    for (int i = 0; i < Sh::ST; ++i) {
      mbar_init(smem_u32(st_full + i), 1);
      mbar_init(smem_u32(st_empty + i), fillers);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(s_full + i), 1);
      mbar_init(smem_u32(p_full + 2 * i), 128);
      mbar_init(smem_u32(p_full + 2 * i + 1), 128);
      mbar_init(smem_u32(o_full + i), 1);
    }
    fence_mbar_init();
    s_span[0] = s_span[3] = 0x7fffffff;
    s_span[1] = s_span[2] = 0;
    *s_odd = 0;
  }
  if (warp == 12) tmem_alloc(smem_u32(tmem_slot), 512);
  __syncthreads();
  pdl_trigger();
  // ---- the queries: their spans, and their rows as an operand of two halves ----
  Query q;
  q.lo = q.hi = q.pos = 0;
  q.slope = q.l = 0.f;
  q.m = -INFINITY;
  if (warp < 8) {
    int least = 0x7fffffff, most = 0, late = 0, early = 0x7fffffff;
    if (tid < w.count) {
      const PromptQuery x = prompt_query(p, w, tid);
      q.lo = x.lo;
      q.hi = x.hi;
      q.pos = x.pos;
      if (MOD && p.a.scores.slopes) q.slope = __ldg(p.a.scores.slopes + kvh * p.group + x.head) * 1.4426950408889634f;
      late = x.lo < x.hi ? x.lo : 0x7fffffff;  // (a row that sees nothing: no block is seen whole)
      early = x.hi;
      if (x.lo < x.hi) {
        least = x.lo;
        most = x.hi;
      }
    }
    least = __reduce_min_sync(0xffffffffu, least);
    most = __reduce_max_sync(0xffffffffu, most);
    late = __reduce_max_sync(0xffffffffu, late);
    early = __reduce_min_sync(0xffffffffu, early);
    if (lane == 0) {
      atomicMin(s_span, least);
      atomicMax(s_span + 1, most);
      atomicMax(s_span + 2, late);
      atomicMin(s_span + 3, early);
    }
  }
  {
    const uint32_t flip = p.scale2 < 0.f ? 0x80008000u : 0u;  // (the softmax takes |scale|)
    const int cpr = hd / 8;
    for (int i = tid; i < kTile * cpr; i += Sh::kThreads) {
      const int t = i / cpr, c = i - t * cpr;
      uint4 u = make_uint4(0, 0, 0, 0);
      if (t < w.count) {
        const int r = (w.q0 + t) / p.group, head = kvh * p.group + (w.q0 + t - r * p.group);
        u = __ldg(reinterpret_cast<const uint4*>((const bf16*)p.a.q + (int64_t)(w.row0 + r) * p.a.q_row +
                                                 (int64_t)head * p.a.q_head) + c);
      }
      u = make_uint4(u.x ^ flip, u.y ^ flip, u.z ^ flip, u.w ^ flip);
      *reinterpret_cast<uint4*>(sQ + (t >> 7) * (128 * HD * 2) + (c >> 3) * 16384 + sw128(t & 127, c & 7)) = u;
    }
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int least = s_span[0], most = s_span[1], late = s_span[2], early = s_span[3];
  const int j_first = least < most ? least / kKeys : 0;
  const int blocks = least < most ? (most + kKeys - 1) / kKeys - j_first : 0;
  const int t0 = (int)((int64_t)blocks * blockIdx.z / p.splits), nt = (int)((int64_t)blocks * (blockIdx.z + 1) / p.splits) - t0;
  const int j_begin = (j_first + t0) * kKeys;
  // First position of block t. With a bias the nearest scores are the largest: from the last block to
  // the first the reference seldom moves (a prompt of 16384 rows 2.06 ms; the other way O was rescaled in
  // most blocks of the steeper heads, 2.48). Without, the masked blocks come better at the end (1.47
  // and 1.52).
  auto block = [&](int t) { return j_begin + (MOD ? nt - 1 - t : t) * kKeys; };
  bool ok = true;

  // all of a CTA's threads, from their different branches
  auto meet = [&]() {
    __syncwarp();
    asm volatile("bar.sync 2, 512;" ::: "memory");
  };

  // (each branch is left only for the end: the registers that a thread has differ)
  if (warp >= 8) {
    fewer_registers<Sh::kOther>();
    if (warp != 12) {
      // ---------------- loaders ----------------
      const int lt = tid - (warp < 12 ? 256 : 288);
      bool odd = false;
      int2 next = make_int2(-1, 0);
      auto look_up = [&](int t) {  // this thread's row of block t
        const int j = block(t) + lt;
        next = make_int2(-1, 0);
        if (lt < kKeys && j >= least && j < most) {
          next.x = page_of(p.m, w.b, j, next.y, p.err);
          odd = odd || next.x < 0;
        }
      };
      // The rows of block t for all loaders; those of the next are looked up meanwhile. (A thread whose
      // wait gave up still takes part, and does nothing else.)
      auto publish = [&](int t) {
        if (lt < kKeys) {
          s_page[(t & 1) * kKeys + lt] = next.x;
          s_off[(t & 1) * kKeys + lt] = (uint16_t)next.y;
        }
        __syncwarp();
        asm volatile("bar.sync 1, %0;" ::"n"(kLoaders) : "memory");
        if (t + 1 < nt) look_up(t + 1);
      };
      auto whole = [&](int t) {  // every query sees all of block t
        const int j = block(t);
        return j >= late && j + kKeys <= early;
      };
      if (!bulk) look_up(0);
      if constexpr (F == kRaw) {
        constexpr int CPR = HD / 8, N = (kKeys * CPR + kLoaders - 1) / kLoaders;  // 16-byte chunks of a row
        for (int n = 0; n < 2 * nt; ++n) {
          const int slot = n % NS, t = n >> 1;
          const bool isv = n & 1;
          if (!isv) publish(t);
          if (ok) ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(empty + slot), ((n / NS) & 1) ^ 1, p.err));
          const int j = block(t);
          const uint32_t to = smem_u32(ring + slot * Sh::kSlot), bar = smem_u32(full + slot);
          const bf16* base = (const bf16*)(isv ? p.v : p.k) + (int64_t)kvh * p.m.page_size * hd;
          const bool look = isv && !whole(t);
          // row `from` r up to r + p.box - 1 that some query sees, if there is one
          auto seen_row = [&](int r) { return min(max(least - j, r), r + p.box - 1); };
          if (ok && p.box && (!isv || j + kKeys <= w.len)) {
            // a box of p.box rows and 64 columns a lane; what no query sees of the sequence comes along.
            // (V rows behind its end may be anything, and become zeros: that block is copied row by row.)
            if (warp == 13) {
              if (lane == 0) mbar_expect_tx(bar, Sh::kSlot);
              __syncwarp();
              for (int i = lane; i < kKeys / p.box * (HD / 64); i += 32) {
                const int r = i / (HD / 64) * p.box, x = i % (HD / 64), rr = seen_row(r);
                const int page = s_page[(t & 1) * kKeys + rr];
                tma_load_4d(to + x * 16384 + r * 128, isv ? &tm_v : &tm_k, 64 * x,
                            page < 0 ? 0 : s_off[(t & 1) * kKeys + rr] - (rr - r), kvh, page < 0 ? p.m.n_pages : page, bar);
              }
              if (lane != 0) mbar_arrive(bar);
            } else {
              mbar_arrive(bar);
            }
            if (look) {  // values that not every query sees
#pragma unroll 5
              for (int i = 0; i < N; ++i) {
                const int x = lt + i * kLoaders, r = x / CPR, c = x % CPR;
                const int rr = seen_row(r & -p.box), page = r < kKeys ? s_page[(t & 1) * kKeys + rr] : -1;
                if (page >= 0) {
                  const uint4 u = __ldg(reinterpret_cast<const uint4*>(
                      base + 8 * c + (int64_t)page * p.m.page_stride + ((int)s_off[(t & 1) * kKeys + rr] + r - rr) * hd));
                  odd = odd || odd_pair(u.x) || odd_pair(u.y) || odd_pair(u.z) || odd_pair(u.w);
                }
              }
            }
          } else if (ok) {
#pragma unroll 5
            for (int i = 0; i < N; ++i) {
              const int x = lt + i * kLoaders, r = x / CPR, c = x % CPR;
              if (r < kKeys && 8 * c < hd) {
                const int page = s_page[(t & 1) * kKeys + r];
                const bf16* src = base + 8 * c;
                if (page >= 0) src += (int64_t)page * p.m.page_stride + (int)s_off[(t & 1) * kKeys + r] * hd;
                cp_async16(to + (c >> 3) * 16384 + sw128(r, c & 7), src, page < 0 ? 0 : 16);
                if (look && page >= 0) {  // values that not every query sees
                  const uint4 u = __ldg(reinterpret_cast<const uint4*>(src));
                  odd = odd || odd_pair(u.x) || odd_pair(u.y) || odd_pair(u.z) || odd_pair(u.w);
                }
              }
            }
            // (arrives when this thread's copies have; the thread that starts the products orders them
            // before those)
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
          }
        }
        cp_async_commit();
        cp_async_wait<0>();
        if (!ok) {  // the copies on their way end before the CTA does
          for (int i = 0; i < NS; ++i)
            if (i < 2 * nt) mbar_wait_for(smem_u32(full + i), 0, p.err, 1000000), mbar_wait_for(smem_u32(full + i), 1, p.err, 1000000);
        }
      } else {
        // 16 columns of a row at a time: their bytes, the block's scale and the row's are asked for
        // while the slot before is filled, and become bf16 on their way into theirs
        constexpr int CPR = HD / 16, N = (kKeys * CPR + kLoaders - 1) / kLoaders;
        const int64_t blk = F == kE2M1 ? e2m1_blocks(p.m) : 0;
        struct Raws {
          uint4 u[N];
          float s[N];
          uint32_t there;
        };
        auto ask = [&](int n, Raws& z) {
          const bool isv = n & 1;
          const unsigned char* base = (const unsigned char*)(isv ? p.v : p.k);
          const float* scales = isv ? p.vs : p.ks;
#pragma unroll
          for (int i = 0; i < N; ++i) {
            // (without branches, so that the loads go out together: of a row that is not there those of
            // page 0 are read and dropped)
            const int x = lt + i * kLoaders, r = min(x / CPR, kKeys - 1), c = min(x % CPR, hd / 16 - 1);
            const int page = s_page[(n >> 1 & 1) * kKeys + r], pg0 = max(page, 0);
            const int64_t line = (int64_t)kvh * p.m.page_size + s_off[(n >> 1 & 1) * kKeys + r];
            const unsigned char* pg = base + (int64_t)pg0 * p.m.page_stride;
            z.s[i] = __ldg(scales + (int64_t)pg0 * p.m.scale_stride + line);
            if (F == kE4M3) {
              z.u[i] = __ldg(reinterpret_cast<const uint4*>(pg + line * hd) + c);
            } else {
              const uint2 v = __ldg(reinterpret_cast<const uint2*>(pg + line * (hd / 2)) + c);
              z.u[i] = make_uint4(v.x, v.y, __ldg(pg + blk + line * (hd / 16) + c), 0);
            }
            z.there = i ? z.there : 0u;
            z.there |= (page >= 0 ? 1u : 0u) << i;
          }
        };
        // a block of 16 columns as bf16; u: its bytes (E2M1: and in z the block's scale), s: the row's scale
        auto convert = [&](uint4 u, float s, bool there, uint32_t (&x)[8]) {
          float f[16];
          if (F == kE4M3) {
            const uint32_t y[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float4 v = e4m3x4_to_f4(y[e]);
              f[4 * e] = v.x * s, f[4 * e + 1] = v.y * s, f[4 * e + 2] = v.z * s, f[4 * e + 3] = v.w * s;
            }
          } else {
            const f32x2 b = both(h2_to_f2(e4m3x2_to_h2(u.z)).x * s);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float v[8];
              e2m1x8_to_f8(h ? u.y : u.x, v);
#pragma unroll
              for (int e = 0; e < 8; e += 2) {
                const float2 y = unpack(mul2(pack(v[e], v[e + 1]), b));
                f[8 * h + e] = y.x, f[8 * h + e + 1] = y.y;
              }
            }
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = pack_bf16(f[2 * e], f[2 * e + 1]);
          if (!there) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = 0u;
          }
        };
        auto put = [&](unsigned char* to, int r, int c, const uint32_t (&x)[8]) {
          *reinterpret_cast<uint4*>(to + (c >> 2) * 16384 + sw128(r, 2 * c & 7)) = make_uint4(x[0], x[1], x[2], x[3]);
          *reinterpret_cast<uint4*>(to + (c >> 2) * 16384 + sw128(r, (2 * c + 1) & 7)) = make_uint4(x[4], x[5], x[6], x[7]);
        };
        auto fill = [&](int n, const Raws& z) {
          const int slot = n % NS;
          if (ok) ok = mbar_wait(smem_u32(empty + slot), ((n / NS) & 1) ^ 1, p.err);
          if (!ok) return;
          unsigned char* to = ring + slot * Sh::kSlot;
          const bool look = (n & 1) && !whole(n >> 1);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const int y = lt + i * kLoaders, r = y / CPR, c = y % CPR;
            if (r >= kKeys || 16 * c >= hd) continue;
            uint32_t x[8];
            convert(z.u[i], z.s[i], z.there >> i & 1, x);
            if (look) {
#pragma unroll
              for (int e = 0; e < 8; ++e) odd = odd || odd_pair(x[e]);
            }
            put(to, r, c, x);
          }
          fence_proxy_async_smem();
          mbar_arrive(smem_u32(full + slot));
        };
        if (bulk && warp == 13) {
          // rows of a page lie side by side: a lane has a box of p.box rows
          int page = -1, off = 0, page1 = -1, off1 = 0;
          auto box_of = [&](int t, int& pg, int& o) {
            const int j = block(t) + lane * p.box;
            pg = -1;
            if (lane < kKeys / p.box && j + p.box > least && j < most) {
              pg = page_of(p.m, w.b, j, o, p.err);
              odd = odd || pg < 0;
            }
          };
          if (nt > 0) box_of(0, page1, off1);
          int n = 0;
          for (; n < 2 * nt; ++n) {
            const int st = n % Sh::ST;
            const bool isv = n & 1;
            if (!isv) {
              page = page1;
              off = off1;
              if (n / 2 + 1 < nt) box_of(n / 2 + 1, page1, off1);
            }
            ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(st_empty + st), ((n / Sh::ST) & 1) ^ 1, p.err));
            if (!ok) break;
            const uint32_t bar = smem_u32(st_full + st), to = smem_u32(stages + st * Sh::kStage);
            const int boxes = __popc(__ballot_sync(0xffffffffu, page >= 0));
            if (lane == 0) mbar_expect_tx(bar, boxes * p.box * (Sh::kStage / kKeys));
            __syncwarp();
            if (page >= 0) {
              const int64_t line = (int64_t)kvh * p.m.page_size + off;
              const unsigned char* pg = (const unsigned char*)(isv ? p.v : p.k) + (int64_t)page * p.m.page_stride;
              const int r = lane * p.box;
              constexpr int VB = Sh::kValues / kKeys, BB = HD / 16;
              bulk_load(to + r * VB, pg + line * VB, p.box * VB, bar);
              if (F == kE2M1) bulk_load(to + Sh::kValues + r * BB, pg + blk + line * BB, p.box * BB, bar);
              bulk_load(to + Sh::kValues + Sh::kBlocks + r * 4, (isv ? p.vs : p.ks) + (int64_t)page * p.m.scale_stride + line,
                        p.box * 4, bar);
            }
          }
          if (!ok) {  // the copies on their way end before the CTA does
            for (int i = max(0, n - Sh::ST); i < n; ++i)
              mbar_wait_for(smem_u32(st_full + i % Sh::ST), (i / Sh::ST) & 1, p.err, 1000000);
          }
        } else if (bulk) {
          constexpr int kFill = kLoaders - 32, M = (kKeys * CPR + kFill - 1) / kFill;
          const int ft = warp < 12 ? lt : lt - 32;
          for (int n = 0; n < 2 * nt; ++n) {
            const int st = n % Sh::ST, slot = n % NS, t = n >> 1, j = block(t);
            if (ok) ok = mbar_wait(smem_u32(st_full + st), (n / Sh::ST) & 1, p.err);
            if (ok) ok = mbar_wait(smem_u32(empty + slot), ((n / NS) & 1) ^ 1, p.err);
            if (!ok) break;
            const unsigned char* from = stages + st * Sh::kStage;
            unsigned char* to = ring + slot * Sh::kSlot;
            const bool look = (n & 1) && !whole(t);
#pragma unroll
            for (int i = 0; i < M; ++i) {
              const int y = ft + i * kFill, r = y / CPR, c = y % CPR;
              if (r >= kKeys) break;
              uint4 u;
              if (F == kE4M3) {
                u = *reinterpret_cast<const uint4*>(from + r * HD + 16 * c);
              } else {
                const uint2 v = *reinterpret_cast<const uint2*>(from + r * (HD / 2) + 8 * c);
                u = make_uint4(v.x, v.y, from[Sh::kValues + r * CPR + c], 0);
              }
              uint32_t x[8];
              convert(u, reinterpret_cast<const float*>(from + Sh::kValues + Sh::kBlocks)[r], j + r >= least && j + r < most, x);
              if (look) {
#pragma unroll
                for (int e = 0; e < 8; ++e) odd = odd || odd_pair(x[e]);
              }
              put(to, r, c, x);
            }
            mbar_arrive(smem_u32(st_empty + st));
            fence_proxy_async_smem();
            mbar_arrive(smem_u32(full + slot));
          }
        } else {
        Raws a, b;  // of K, of V
        if (nt > 0) {
          publish(0);
          ask(0, a);
        }
        for (int t = 0; t < nt; ++t) {
          ask(2 * t + 1, b);
          fill(2 * t, a);
          if (t + 1 < nt) {
            publish(t + 1);
            ask(2 * t + 2, a);
          }
          fill(2 * t + 1, b);
        }
        }
      }
      if (odd) *s_odd = 1;
    } else {
    // ---------------- the products ----------------
    // (the whole warp goes through this, so that addresses and descriptors are uniform; one thread
    // starts the products and commits them)
    if (nt > 0) {
      const bool leader = elect_one();
      const int halves = w.count > 128 ? 2 : 1;
      const uint32_t id_s = umma_idesc_bf16(128, kKeys);
      const uint32_t id_o = umma_idesc_bf16(128, hd) | 1u << 16;  // B is MN-major
      const int ks = hd / 16;
      const uint64_t d_q = umma_desc_sw128(smem_u32(sQ)), d_k = umma_desc_sw128(smem_u32(ring)),
                     d_v = umma_desc_mn(smem_u32(ring));
      auto scores = [&](int h, int t) {  // S of half h over block t
        const uint64_t q0 = d_q + h * (128 * HD * 2 >> 4), k0 = d_k + (2 * t % NS) * (Sh::kSlot >> 4);
        if (leader) {
#pragma unroll
          for (int i = 0; i < HD / 16; ++i) {
            const uint32_t at = ((i >> 2) * 16384 + (i & 3) * 32) >> 4;
            if (i < ks) umma_bf16(tmem + h * 128, q0 + at, k0 + at, id_s, i ? 1u : 0u);
          }
          umma_commit(smem_u32(s_full + h));
        }
      };
      auto wait = [&](uint64_t* bar, int parity) { return __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity, p.err)); };
      auto wait_slot = [&](int n) {
        const bool here = wait(full + n % NS, (n / NS) & 1);
        fence_proxy_async_smem();  // the loaders' writes before the products' reads
        tc_fence_after();
        return here;
      };
      ok = wait_slot(0);
      if (ok) {
        scores(0, 0);
        if (halves > 1) scores(1, 0);
        if (leader) umma_commit(smem_u32(empty));
      }
      for (int t = 0; t < nt && ok; ++t) {
        const int nv = 2 * t + 1;
        ok = wait_slot(nv);
        const uint64_t v0 = d_v + (nv % NS) * (Sh::kSlot >> 4);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h >= halves) break;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (ok) ok = wait(p_full + 2 * h + x, t & 1);
            if (!ok) break;
            tc_fence_after();
            if (leader) {
#pragma unroll
              for (int i = 4 * x; i < 4 * x + 4; ++i)
                umma_bf16_ta(tmem + 256 + h * HD, tmem + h * 128 + 8 * i, v0 + i * (2048 >> 4), id_o, (t | i) ? 1u : 0u);
            }
          }
          if (!ok) break;
          const bool last = h + 1 == halves;
          if (last && leader) umma_commit(smem_u32(empty + nv % NS));
          if (t + 1 < nt) {
            if (h == 0) ok = wait_slot(2 * t + 2);
            if (!ok) break;
            scores(h, t + 1);
            if (last && leader) umma_commit(smem_u32(empty + (2 * t + 2) % NS));
          } else if (leader) {
            umma_commit(smem_u32(o_full + h));
          }
        }
      }
      if (!ok) {  // what was issued ends before TMEM is freed
        if (leader) umma_commit(smem_u32(o_full));
        mbar_wait(smem_u32(o_full), 0, p.err);
      }
    }
    __syncwarp();
    }
    meet();
    meet();
    if (warp == 12) {
      tc_fence_after();
      tmem_dealloc(tmem, 512);
    }
  } else {
    more_registers<Sh::kMine>();
    // ---------------- softmax: warps 0-3 of half 0, 4-7 of half 1 ----------------
    const int h = warp >> 2;
    const float scale = fmaxf(fabsf(p.scale2), 1.17549435e-38f);  // (of 0: masked scores stay minus infinity)
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + h * 128 + lanes, tO = tmem + 256 + h * HD + lanes;
    // what every query of the warp sees needs no mask
    const bool mine = tid < w.count;
    const int from = __reduce_max_sync(0xffffffffu, mine ? (q.lo < q.hi ? q.lo : 0x7fffffff) : 0);
    const int to = __reduce_min_sync(0xffffffffu, mine ? q.hi : 0x7fffffff);
    // scores that a cap keeps within 2^+-60 need no reference but 0
    const bool fixed = MOD && p.capl > 0.f && p.capl <= 60.f && !p.a.scores.slopes;
    if (fixed) q.m = 0.f;
    Cap cap = {};
    if (MOD) cap = cap_of(p, scale);
    const int nearest = __reduce_min_sync(0xffffffffu, mine ? q.pos : 0x7fffffff);
    const bool used = h == 0 || w.count > 128;  // (of a short tile there is no second half)
    for (int t = 0; t < nt && used; ++t) {
      const int j = block(t);
      ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(s_full + h), t & 1, p.err));
      if (!ok) break;
      tc_fence_after();
      const bool edge = j < from || j + kKeys > to, behind = j + kKeys - 1 <= nearest;
      uint32_t r[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, r[c]);
      tmem_wait_ld(r);
      float tops[4], fix = 1.f;
      bool rises = false;
      if constexpr (MOD) {
        // the scores come relative to the reference of the blocks before
        const float was = q.m == -INFINITY ? 0.f : q.m;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          scores32(p, q, cap, scale, was, r[c], j + 32 * c, behind);
          if (edge) mask32(q, r[c], j + 32 * c);
        }
        if (!fixed) {
          const float top = top_of(r, tops);
          const bool up = q.m == -INFINITY ? top > -INFINITY : top > 8.f;
          rises = __any_sync(0xffffffffu, up);
          if (rises) {
            const float by = up ? top : 0.f;
            fix = !up ? 1.f : q.m == -INFINITY ? 0.f : ex2(-by);
            if (up) q.m = was + by;
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int e = 0; e < 32; ++e) r[c][e] = __float_as_uint(__uint_as_float(r[c][e]) - by);
          }
        }
      } else {
        if (edge) {
#pragma unroll
          for (int c = 0; c < 4; ++c) mask32(q, r[c], j + 32 * c);
        }
        const float top = top_of(r, tops) * scale;
        const bool up = q.m == -INFINITY ? top > -INFINITY : top > q.m + 8.f;
        rises = __any_sync(0xffffffffu, up);
        if (rises) {
          fix = up ? ex2(q.m - top) : 1.f;  // (0 for the first)
          if (up) q.m = top;
        }
      }
      if (rises) {
        q.l *= fix;
        if (t > 0) {
#pragma unroll 1
          for (int c = 0; c < hd; c += 16) {
            float v[16];
            uint32_t o[16];
            tmem_ld16(tO + c, v);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(v[e] * fix);
            tmem_st16(tO + c, o);
          }
        }
      }
      const float ref = q.m == -INFINITY ? 0.f : q.m;
      const f32x2 by = both(scale), less = both(-ref);
      f32x2 sum[2] = {both(0.f), both(0.f)};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t w16[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const f32x2 s2 = pack(__uint_as_float(r[c][e]), __uint_as_float(r[c][e + 1]));
          const float2 x = unpack(MOD ? s2 : fma2(s2, by, less));
          const float a = ex2(x.x), b = ex2(x.y);
          sum[e / 2 & 1] = add2(sum[e / 2 & 1], pack(a, b));
          w16[e / 2] = pack_bf16(a, b);
        }
        tmem_st16(tS + 16 * c, w16);
        if (c & 1) {
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(smem_u32(p_full + 2 * h + c / 2));
        }
      }
      const float2 two = unpack(add2(sum[0], sum[1]));
      q.l += two.x + two.y;
    }
    if (ok && nt > 0 && used) ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(o_full + h), 0, p.err));
    tc_fence_after();
    meet();  // the loaders have seen all values
    const int64_t part = (((int64_t)blockIdx.x * gridDim.y + kvh) * p.splits + blockIdx.z) * kTile;
    if (*s_odd) {
      row_by_row<F>(p, w, kvh, j_begin, j_begin + nt * kKeys, part);
    } else if (ok) {
      const float inv = p.splits > 1 ? 1.f : q.l != 0.f ? 1.f / q.l : 0.f;
      bf16* out = tid < w.count ? out_row(p, w, kvh, tid) : nullptr;
      for (int c = 0; c < hd; c += 16) {
        float v[16];
        if (nt > 0 && used) {
          tmem_ld16(tO + c, v);
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = 0.f;
        }
        if (tid < w.count) {
          if (q.l == 0.f) {  // (a row that sees nothing)
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = 0.f;
          }
          if (p.splits > 1) {
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              *reinterpret_cast<float4*>(p.part_o + (part + tid) * hd + c + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
          } else {
#pragma unroll
            for (int e = 0; e < 16; e += 8) {
              float x[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) x[i] = v[e + i] * inv;
              store8(out + c + e, true, x);
            }
          }
        }
      }
      if (p.splits > 1 && tid < w.count) p.part_ml[part + tid] = make_float2(q.m, q.l);
    }
    tc_fence_before();
    meet();
  }
}

// Tensor maps of the pages, [n_pages][n_kv_heads][page_size][head_dim], with boxes of `box` rows.
bool page_maps(const PagedPrompt& p, int box, CUtensorMap (&tm)[2]) {
  const uint64_t row = (uint64_t)p.m.head_dim * 2, page = (uint64_t)p.m.page_stride * 2;
  if (page >= 1ull << 40) return false;
  for (int i = 0; i < 2; ++i)
    if (tc_make_tmap4s(&tm[i], i ? p.v : p.k, p.m.head_dim, p.m.page_size, p.m.n_kv_heads, p.m.n_pages, row,
                       row * p.m.page_size, page, box))
      return false;
  return true;
}

template <int HD, Rows F, bool MOD>
cudaError_t launch_hd(const PagedPrompt& p, const PromptPlan& pl, cudaStream_t st) {
  using Sh = Shape<HD, F>;
  static unsigned long long done = 0;
  auto k = k_prompt_tc<HD, F, MOD>;
  if (!smem_limit((const void*)k, Sh::kSmem, &done)) return cudaErrorInvalidValue;
  const dim3 grid(pl.tiles, p.m.n_kv_heads, pl.splits);
  // Whole boxes of a page make up a block of keys: those come by TMA. (Other page sizes and heads row by row.)
  PagedPrompt a = p;
  CUtensorMap tm[2] = {};
  a.box = 0;
  if (p.m.head_dim == HD) {
    const int ps = p.m.page_size;
    const int box = ps % kKeys == 0 ? kKeys : ps >= 8 && kKeys % ps == 0 ? ps : 0;
    if (F == kRaw)
      a.box = box && page_maps(p, box, tm) ? box : 0;
    else if (aligned_to(p.ks, 16) && aligned_to(p.vs, 16) && mult(p.m.scale_stride, 4))
      a.box = box;
  }
  return launch_op(k, grid, Sh::kThreads, Sh::kSmem, st, false, 1, tm[0], tm[1], a);
}
template <Rows F>
cudaError_t launch_rows(const PagedPrompt& p, const PromptPlan& pl, bool mod, cudaStream_t st) {
  if (p.m.head_dim <= 64) return mod ? launch_hd<64, F, true>(p, pl, st) : launch_hd<64, F, false>(p, pl, st);
  return mod ? launch_hd<128, F, true>(p, pl, st) : launch_hd<128, F, false>(p, pl, st);
}

}  // namespace
