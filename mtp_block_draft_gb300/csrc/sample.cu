// dmtp_sample_rows: temperature, top-k, top-p and min-p sampling from one given uniform
// number per row.
//
// A row's CTAs (one, or a cluster) each hold a slice of it in shared memory, so the logits are read
// from HBM once and every later step runs on chip; a thread owns consecutive ids. Counts, weights
// and histograms are reduced over the cluster through distributed shared memory. (Many rows of a
// large vocabulary are streamed instead, k_sample_stream.) What bounds it is issue: a handful of
// instructions a logit for each pass, and about fifty for a weight; of one row, the barriers. One
// row of 151936 with top_k and top_p takes 20.0 us, 256 rows with top_p 253 us (155 MB: 23 us).
//
// Weights. 2^y with y = (l - max) log2(e) / T as an integer in 2^-44 steps of the largest, so
// that sums are exact and associative: no result depends on how a row was split. The exponent
// is formed as a pair of floats (the difference, the factor and their product with their
// rounding errors); 2^y = 2^n 2^(j/256) 2^r with a table of 2^(j/256) in 62-bit fixed point and
// 2^r - 1 as a series to r^4 (|r| < 2^-9, the next term is 2^-54). The error of a weight is
// about 2^-39 of it and a step.
//
// Filters. The cut is a logit and, among its ties, how many of the lowest ids stay. Logits fall
// into bins of 1/32 octave of weight; the bin in which the count from above reaches top_k is
// then split by the logits' bits (keys) until all of a bin stays or one key is left. For top_p the bins' counts
// give the cut's neighbourhood (their weights, taken at the bins' centres, are off by at most
// 1.1%); one pass then sums every weight exactly - all, those above the neighbourhood, and by
// finer bins inside it - and the bin that the goal falls into is split likewise. A goal outside
// the neighbourhood only costs another pass. The same pass leaves each thread's kept weight
// above the neighbourhood, so the pick needs no second one.
#include <math.h>

#include "paged.cuh"
#include "sample_keys.h"

namespace {

constexpr float kMasked = -INFINITY;  // what a logit that is never kept becomes

// 2^(2^-i), i = 1..8, in 62-bit fixed point: 2^(j/256) is the product of those of j's bits.
__constant__ const unsigned long long kRoots[8] = {
    0x5a827999fcef3242ull, 0x4c1bf828c6dc54b8ull, 0x45cae0f1f545eb73ull, 0x42d561b3e6243d8aull,
    0x4166c34c5615d0ecull, 0x40b268f9de0183baull, 0x4058f6a7ecccd5b6ull, 0x402c6be96af2fb58ull};
__device__ __forceinline__ unsigned long long exp2_256th(int j) {
  unsigned long long t = 1ull << 62;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (j >> (7 - i) & 1) t = __umul64hi(t, kRoots[i]) << 2;
  return t;
}

struct RowsArgs {
  dmtp_sample_args a;
  int slice;  // logits of a CTA
  bool vec;   // rows allow 16-byte loads
};

__device__ __forceinline__ float clean(float l) {  // NaN: masked; +infinity: the largest number
  return fminf(fmaxf(l, kMasked), 3.402823466e38f);
}
// floor(f t) of 0 <= f < 1 (up: the next integer if that is not exact): the whole product,
// 24 by 64 bits, so that a border that f t meets exactly is met here too.
__device__ __forceinline__ unsigned long long part_of(float f, unsigned long long t, bool up) {
  const uint32_t b = __float_as_uint(f), x = b >> 23;
  const unsigned long long m = x ? (b & 0x7fffffu) | 0x800000u : b & 0x7fffffu;
  const int e = x ? 150 - (int)x : 149;  // f = m 2^-e, e >= 24
  const unsigned long long hi = __umul64hi(m, t), lo = m * t;
  unsigned long long r, rest;
  if (e < 64) {
    r = (hi << (64 - e)) | (lo >> e);
    rest = lo << (64 - e);
  } else if (e < 128) {
    r = hi >> (e - 64);
    rest = lo | (e > 64 ? hi << (128 - e) : 0ull);
  } else {
    r = 0;
    rest = hi | lo;
  }
  return r + (up && rest ? 1 : 0);
}

constexpr int kShift = 44;  // weight 1 is 2^44: 2^18 of them stay below 2^63
constexpr int kBins = 2048, kFine = kBins / 4;  // (a fine bin has four words)

struct Weigh {
  float top, chi, clo, cb;
  const unsigned long long* table;

  // Bin of 1/32 octave below the largest logit (the nearest, so bin i is centred at 2^(-i/32));
  // decreasing in l, the last one takes the rest.
  __device__ __forceinline__ int bin(float l) const {
    const float x = fminf((top - l) * cb, (float)(kBins - 1));
    return (int)(__float_as_uint(x + 8388608.f) & (kBins - 1));
  }
  // The weight from the exponent's whole and 256th part (jt, in the low bits of a sum with
  // 1.5 2^15), and 2^r - 1 in steps of 2^-31 (a) and 2^-40 (b), kept likewise. Steps of 2^-44,
  // rounded down: 2^18 of them lose 2^-27 of the largest weight at most.
  __device__ __forceinline__ unsigned long long scaled(float hi, float jt, float a, float b) const {
    const int j = __float_as_int(jt) - 0x47400000;
    const int q = __float_as_int(a) * 512 + __float_as_int(b) - (int)(0x3bc00000u * 512u + 0x37400000u);
    const unsigned long long t62 = table[j & 255];
    const unsigned long long w = t62 + (unsigned long long)((long long)(int)(t62 >> 32) * q >> 8);
    return hi > -45.f ? w >> (62 - kShift - (j >> 8)) : 0ull;  // (below: under half a step, or masked)
  }
  // The weights of two logits.
  __device__ __forceinline__ void two(float2 l, unsigned long long& wx, unsigned long long& wy) const {
    const f32x2 one = both(-1.f), x = pack(l.x, l.y), c = both(chi), nc = both(-chi), ntop = both(-top);
    const f32x2 d = add2(x, ntop), t = fma2(x, one, d);           // l - top and what it lost, e
    const f32x2 e = add2(fma2(fma2(t, one, d), one, x), fma2(t, one, ntop));
    const f32x2 hi = mul2(d, c);                                  // the exponent, hi + lo; nlo = -lo
    const f32x2 nlo = fma2(e, nc, fma2(d, both(-clo), fma2(d, nc, hi)));
    // (adding 1.5 2^k rounds to steps of 2^(k - 23) and leaves the step count in the low bits)
    const f32x2 jt = add2(hi, both(49152.f));
    const f32x2 s = fma2(add2(jt, both(-49152.f)), one, hi);      // exact, |s| <= 2^-9
    const f32x2 h = mul2(s, both(0.693147182464599609f));         // (s + lo) ln 2 = h - g so far
    f32x2 g = fma2(s, both(-0.693147182464599609f), h);
    g = fma2(s, both(1.90465429995776804525e-09f), fma2(nlo, both(0.693147182464599609f), g));
    const f32x2 r = fma2(nlo, one, s);
    g = fma2(mul2(r, r), fma2(r, fma2(r, both(-9.618129107628477e-3f), both(-5.550410866482158e-2f)),
                              both(-0.24022650695910072f)), g);   // 2^(s + lo) - 1 = h - g
    const f32x2 a = add2(h, both(5.859375e-3f));                  // 1.5 2^-8 (|h| < 2^-9): steps of 2^-31
    const f32x2 b = add2(fma2(g, one, fma2(add2(a, both(-5.859375e-3f)), one, h)), both(1.1444091796875e-5f));
    const float2 h2 = unpack(hi), j2 = unpack(jt), a2 = unpack(a), b2 = unpack(b);  // b: 1.5 2^-17
    wx = scaled(h2.x, j2.x, a2.x, b2.x);
    wy = scaled(h2.y, j2.y, a2.y, b2.y);
  }
  __device__ __forceinline__ unsigned long long operator()(float l) const {
    unsigned long long wx, wy;
    two(make_float2(l, l), wx, wy);
    return wx;
  }
};

template <int THREADS>
struct Shared {
  static constexpr int kWarps = THREADS / 32;
  alignas(16) uint32_t hist[kBins];
  union {  // of the cluster, by sum_hist() or sum_fine()
    uint32_t all[kBins];
    unsigned long long fine[kFine][2];  // weight, count
  };
  unsigned long long slot[2][16][2];  // one pair of each CTA of the cluster, twice
  unsigned long long warp[kWarps][2];
  unsigned long long found[4];
  static constexpr int kSlots = 4096 / THREADS;
  uint8_t list[kSlots][THREADS];      // where a thread's ids in the neighbourhood are
  uint32_t edge[5];  // keys: top-k's bin, min_p's cut, top-p's neighbourhood
  int bins[2];
  unsigned long long table[256];
};

template <int THREADS, typename S>
struct Cluster {
  static constexpr int kWarps = THREADS / 32;
  S* s;
  unsigned rank, size;
  int phase;

  __device__ __forceinline__ void sync() const {
    if (size > 1)
      cluster_sync_all();
    else
      __syncthreads();
  }
  // sync() in two halves: what stands between them does not wait for the others
  __device__ __forceinline__ void arrive() const {
    if (size > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  }
  __device__ __forceinline__ void wait() const {
    if (size > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  }
  // Leave (a, b) of this CTA in every CTA's slots (thread t < size sends to CTA t) and wait:
  // afterwards slot[p][r] holds CTA r's pair. Call with a, b valid in threads 0..size-1.
  __device__ __forceinline__ int exchange(unsigned long long a, unsigned long long b) {
    const int p = phase;
    phase ^= 1;
    if (threadIdx.x < size) {
      const uint32_t to = smem_in_rank(smem_u32(&s->slot[p][rank][0]), threadIdx.x);
      asm volatile("st.shared::cluster.v2.u64 [%0], {%1, %2};" ::"r"(to), "l"(a), "l"(b) : "memory");
    }
    sync();
    return p;
  }
  // Sums of (a, b) over the CTA, valid in the first warp.
  __device__ __forceinline__ void cta_sum(unsigned long long& a, unsigned long long& b) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s->warp[threadIdx.x >> 5][0] = a, s->warp[threadIdx.x >> 5][1] = b;
    __syncthreads();
    if (threadIdx.x < 32) {
      a = b = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) a += s->warp[w][0], b += s->warp[w][1];
    }
  }
  // Sums of (a, b) over all threads of the cluster.
  __device__ __forceinline__ void sum(unsigned long long& a, unsigned long long& b) {
    cta_sum(a, b);
    const int p = exchange(a, b);
    a = b = 0;
    for (unsigned r = 0; r < size; ++r) a += s->slot[p][r][0], b += s->slot[p][r][1];
  }
  __device__ __forceinline__ uint32_t cta_max(uint32_t a) {
    a = __reduce_max_sync(0xffffffffu, a);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s->warp[threadIdx.x >> 5][0] = a;
    __syncthreads();
    a = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) a = ::max(a, (uint32_t)s->warp[w][0]);
    return a;
  }
  __device__ __forceinline__ uint32_t max(uint32_t a) {
    const int p = exchange(cta_max(a), 0);
    a = 0;
    for (unsigned r = 0; r < size; ++r) a = ::max(a, (uint32_t)s->slot[p][r][0]);
    return a;
  }
  // Sum the cluster's histograms: every CTA gets the whole of it in `all`, and its own is
  // cleared (a barrier of the CTA must come before the next one is begun).
  __device__ __forceinline__ void sum_hist() {
    sync();
    const int per = kBins / (int)size;
    for (int i = threadIdx.x; i < per; i += THREADS) {
      const int at = (int)rank * per + i;
      uint32_t n = 0;
      for (unsigned r = 0; r < size; ++r) {
        uint32_t v;
        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(smem_in_rank(smem_u32(&s->hist[at]), r)) : "memory");
        n += v;
      }
      for (unsigned r = 0; r < size; ++r)
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(smem_in_rank(smem_u32(&s->all[at]), r)), "r"(n) : "memory");
    }
    sync();
    for (int i = threadIdx.x; i < kBins; i += THREADS) s->hist[i] = 0;
  }
  // The same of histograms filled by add_fine(): every CTA gets the cluster's count and weight of
  // each fine bin in `fine`.
  __device__ __forceinline__ void sum_fine() {
    sync();
    const int per = kFine / (int)size;
    for (int i = threadIdx.x; i < per; i += THREADS) {
      const int at = (int)rank * per + i;
      uint32_t n = 0;
      unsigned long long w = 0;
      for (unsigned r = 0; r < size; ++r) {
        uint32_t c, x, y, z;
        asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(c), "=r"(x), "=r"(y), "=r"(z) : "r"(smem_in_rank(smem_u32(&s->hist[4 * at]), r)) : "memory");
        n += c;
        w += (unsigned long long)x + ((unsigned long long)y << 15) + ((unsigned long long)z << 30);
      }
      for (unsigned r = 0; r < size; ++r)
        asm volatile("st.shared::cluster.v2.u64 [%0], {%1, %2};" ::"r"(smem_in_rank(smem_u32(&s->fine[at][0]), r)),
                     "l"(w), "l"((unsigned long long)n) : "memory");
    }
    sync();
    for (int i = threadIdx.x; i < kBins; i += THREADS) s->hist[i] = 0;
  }
  // Exclusive sum over the CTA's threads, and the total; all threads call it.
  __device__ __forceinline__ unsigned long long scan(unsigned long long v, unsigned long long& total) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    unsigned long long inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    __syncthreads();
    if (lane == 31) s->warp[wid][0] = inc;
    __syncthreads();
    unsigned long long before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < wid) before += s->warp[w][0];
      total += s->warp[w][0];
    }
    return before + inc - v;
  }
  // The bin of `all` (counts, the largest logits first) in which the running count reaches
  // want, 1 <= want <= the total, the count before it and its own. All threads call it.
  __device__ __forceinline__ void find_count(unsigned long long want, int& bin, unsigned long long& before,
                                             unsigned long long& own) {
    constexpr int E = kBins / THREADS;
    unsigned long long n = 0, total;
#pragma unroll
    for (int e = 0; e < E; ++e) n += s->all[threadIdx.x * E + e];
    unsigned long long at = scan(n, total);
    if (at < want && want <= at + n) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const unsigned long long c = s->all[threadIdx.x * E + e];
        if (at < want && want <= at + c) s->found[0] = threadIdx.x * E + e, s->found[1] = at, s->found[2] = c;
        at += c;
      }
    }
    __syncthreads();
    bin = (int)s->found[0];
    before = s->found[1];
    own = s->found[2];
  }
  // The neighbourhood of top-p's cut: the bins (of `all`, bin `first` centred at the largest
  // weight, no more than last_n of last_bin and none after it) at which the running weight is
  // about top_p of all, into s->bins. All threads call it.
  __device__ __forceinline__ void neighbours(float top_p, int last_bin, unsigned long long last_n, float first) {
    constexpr int N = kBins / THREADS;
    float m[N], sum = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const int i = threadIdx.x * N + e;
      const unsigned long long c = s->all[i];
      m[e] = i < last_bin ? (float)c : i == last_bin ? (float)(c < last_n ? c : last_n) : 0.f;
      m[e] *= ex2(((first - (float)i)) * 0.03125f);
      sum += m[e];
    }
    if (threadIdx.x == 0) s->bins[0] = s->bins[1] = last_bin;
    unsigned long long total;  // in 2^-24
    const unsigned long long at = scan((unsigned long long)(sum * 16777216.f), total);
    // a weight taken at its bin's centre is off by 1.1% at most, 0.6% in the mean square, and the
    // errors of the many weights of a flat row average out
    const float p = fmaxf(top_p, 0.f) * (float)total;
    const float wide = fminf(0.023f, 0.0005f + 0.025f * rsqrtf((float)total * 5.9604645e-8f));
    float run = (float)at;
    int lo_b = kBins, hi_b = kBins;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      run += m[e] * 16777216.f;
      if (run >= p * (1.f - wide)) lo_b = min(lo_b, (int)threadIdx.x * N + e);
      if (run >= p * (1.f + wide)) hi_b = min(hi_b, (int)threadIdx.x * N + e);
    }
    if (lo_b <= last_bin) atomicMin(&s->bins[0], lo_b);
    if (hi_b <= last_bin) atomicMin(&s->bins[1], hi_b);
    __syncthreads();
  }
  // 2^-44 weights as three 15-bit parts and a count in bins of the histogram: 32-bit sums hold
  // the 2^17 logits that a CTA has at most (of the cluster's 2^18 they would not).
  __device__ __forceinline__ void add_fine(int i, unsigned long long w) {
    uint32_t* h = &s->hist[4 * i];
    atomicAdd(h, 1u);
    atomicAdd(h + 1, (uint32_t)w & 0x7fffu);
    atomicAdd(h + 2, (uint32_t)(w >> 15) & 0x7fffu);
    atomicAdd(h + 3, (uint32_t)(w >> 30));
  }
};

// The smallest key <= top of which yes(logit) holds (it holds of top, and of every key above
// one of which it holds); one warp searches 32 places at a time.
template <typename F>
__device__ __forceinline__ uint32_t first_key(uint32_t top, F yes) {
  uint32_t lo = kMaskedKey, hi = top;
  const int lane = threadIdx.x & 31;
  while (hi - lo > 1) {
    const uint32_t x = lo + (uint32_t)((unsigned long long)(hi - lo) * (lane + 1) / 33);
    const unsigned b = __ballot_sync(0xffffffffu, x > lo && yes(logit_of(x)));
    const int f = b ? __ffs(b) - 1 : 32;
    const uint32_t nh = __shfl_sync(0xffffffffu, x, f & 31), nl = __shfl_sync(0xffffffffu, x, (f + 31) & 31);
    if (f < 32) hi = nh;
    if (f > 0) lo = nl;
  }
  return hi;
}

template <typename T, int THREADS>
__global__ void __launch_bounds__(THREADS) k_sample_rows(const RowsArgs sa) {
  extern __shared__ __align__(16) unsigned char smem[];
  using Sh = Shared<THREADS>;
  Sh& sh = *reinterpret_cast<Sh*>(smem);
  float* vals = reinterpret_cast<float*>(smem + (sizeof(Sh) + 15) / 16 * 16);
  const dmtp_sample_args& a = sa.a;
  unsigned size;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(size));
  Cluster<THREADS, Sh> cl{&sh, cluster_rank(), size, 0};
  const int row = blockIdx.x / size, tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int V = a.vocab, slice = sa.slice, E = slice / THREADS;
  const int base = (int)cl.rank * slice;
  const int mine = V > base ? min(slice, V - base) : 0;
  const T* lg = (const T*)a.logits + (int64_t)row * a.ld + base;
  float best = kMasked;
  if (sa.vec) {
    constexpr int X = 16 / sizeof(T);
#pragma unroll 4
    for (int i = tid * X; i < slice; i += THREADS * X) {
      float f[X];
      if (i + X <= mine) {
        const uint4 u = __ldcs(reinterpret_cast<const uint4*>(lg + i));
        const T* t = reinterpret_cast<const T*>(&u);
#pragma unroll
        for (int e = 0; e < X; ++e) f[e] = clean(to_f32(t[e]));
      } else {
#pragma unroll
        for (int e = 0; e < X; ++e) f[e] = i + e < mine ? clean(to_f32(lg[i + e])) : kMasked;
      }
#pragma unroll
      for (int e = 0; e < X; e += 4)
        *reinterpret_cast<float4*>(vals + i + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
#pragma unroll
      for (int e = 0; e < X; ++e) best = fmaxf(best, f[e]);
    }
  } else {
#pragma unroll 4
    for (int i = tid; i < slice; i += THREADS) {
      const float f = i < mine ? clean(to_f32(lg[i])) : kMasked;
      vals[i] = f;
      best = fmaxf(best, f);
    }
  }
  for (int i = tid; i < 256; i += THREADS) sh.table[i] = exp2_256th(i);
  for (int i = tid; i < kBins; i += THREADS) sh.hist[i] = 0;
  const float temp = a.temperature ? __ldg(a.temperature + row) : 1.f;
  const int k = a.top_k ? __ldg(a.top_k + row) : 0;
  const float top_p = a.top_p ? __ldg(a.top_p + row) : 1.f;
  const float min_p = a.min_p ? __ldg(a.min_p + row) : 0.f;
  const float u = __ldg(a.u + row);
  cl.sync();  // every CTA of the cluster runs before one writes another's memory
  const uint32_t top = cl.max(key_of(best));
  const bool none = top == kMaskedKey;
  if (none || !(temp > 0.f)) {
    uint32_t id = 0;  // of the largest logit, the lowest: 2^32 - 1 - id is maximal
    const float t = logit_of(top);
    for (int i = tid; i < mine; i += THREADS)
      if (vals[i] == t && !none) id = max(id, 0xffffffffu - (unsigned)(base + i));
    id = cl.max(id);
    if (cl.rank == 0 && tid == 0) {
      a.ids[row] = none ? -1 : (int)(0xffffffffu - id);
      if (a.kept) a.kept[row] = none ? 0 : 1;
    }
    cl.sync();  // no CTA leaves while another may still write its slots
    return;
  }
  Weigh W;
  W.top = logit_of(top);
  W.table = sh.table;
  // c = log2(e) / T as a pair
  const float tt = fminf(fmaxf(temp, 1e-30f), 1e30f);
  W.chi = 1.44269502162933349609f / tt;
  W.clo = (fmaf(-W.chi, tt, 1.44269502162933349609f) + 1.92596299112661746887e-08f) / tt;
  W.cb = W.chi * 32.f;
  const float2* own = reinterpret_cast<const float2*>(vals + tid * E);  // this thread's ids, E even
  const bool by_p = top_p < 1.f;
  // the smallest logit that stays, as a key; `ties` of its ids stay, all of them unless `partial`
  uint32_t cut = kLowestKey;
  unsigned long long ties = 0;
  bool partial = false;
  bool by_k = false;

  if (k > 0 || by_p) {
    // the two end bins, where flat rows and masked logits crowd, are counted by thread
    uint32_t ends[2] = {0, 0};
#pragma unroll 2
    for (int i = 0; i < E / 2; ++i) {
      const float2 xy = own[i];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float x = e ? xy.y : xy.x;
        const int b = W.bin(x);
        if (b > 0 && b < kBins - 1)
          atomicAdd(&sh.hist[b], 1u);
        else if (b == 0)
          ++ends[0];
        else
          ends[1] += x > kMasked;
      }
    }
    ends[0] = __reduce_add_sync(0xffffffffu, ends[0]);
    ends[1] = __reduce_add_sync(0xffffffffu, ends[1]);
    if (lane == 0 && ends[0]) atomicAdd(&sh.hist[0], ends[0]);
    if (lane == 1 && ends[1]) atomicAdd(&sh.hist[kBins - 1], ends[1]);
    cl.sum_hist();
    unsigned long long n = 0, nvalid, before, cnt, want = k;
    for (int i = tid; i < kBins; i += THREADS) n += sh.all[i];
    cl.scan(n, nvalid);
    by_k = k > 0 && (unsigned long long)k < nvalid;
    int last_bin = kBins - 1;           // the last bin that top-k leaves
    unsigned long long last_n = ~0ull;  // and how many of its logits
    if (by_k) {
      cl.find_count(want, last_bin, before, cnt);
      want -= before;
      last_n = want;
    }
    if (by_p) cl.neighbours(top_p, last_bin, last_n, 0.f);
    if (by_k) {
      if (wid < 2) {
        const int b = wid ? last_bin - 1 : last_bin;
        const uint32_t f = b < 0 ? top + 1 : first_key(top, [&](float x) { return W.bin(x) <= b; });
        if (lane == 0) sh.edge[wid] = wid ? f - 1 : f;
      }
      __syncthreads();
      uint32_t lo = sh.edge[0], hi = sh.edge[1];
      while (want != cnt && lo != hi) {
        const int shift = range_shift(lo, hi, 11);
        const float lf = logit_of(lo), hf = logit_of(hi);
        for (int i = 0; i < E / 2; ++i) {
          const float2 x = own[i];
          if (x.x >= lf && x.x <= hf) atomicAdd(&sh.hist[hi - key_of(x.x) >> shift], 1u);
          if (x.y >= lf && x.y <= hf) atomicAdd(&sh.hist[hi - key_of(x.y) >> shift], 1u);
        }
        cl.sum_hist();
        int f;
        cl.find_count(want, f, before, cnt);
        want -= before;
        take_bin(lo, hi, shift, (uint32_t)f);
      }
      cut = lo;
      partial = want != cnt;
      ties = want;
    }
  }
  const unsigned long long tie_mass = partial ? ties * W(logit_of(cut)) : 0ull;
  // min_p as a key
  uint32_t min_key = 0;
  if (min_p > 0.f && wid == 0) {
    const unsigned long long least = min_p < 1.f ? part_of(min_p, 1ull << kShift, true) : 1ull << kShift;
    const uint32_t f = first_key(top, [&](float x) { return W(x) >= least; });
    if (lane == 0) sh.edge[2] = f;
  }

  unsigned long long mass = 0;  // of this thread's kept logits, so far of those above `from`
  uint32_t cnt = 0, from = 0xffffffffu;
  int listed = -1;              // >= 0: the others are in this thread's list, so many
  if (by_p) {
    {
      if (wid < 2) {
        const int b = wid ? sh.bins[0] - 1 : sh.bins[1];
        const uint32_t f = b < 0 ? top + 1 : first_key(top, [&](float x) { return W.bin(x) <= b; });
        if (lane == 0) sh.edge[3 + wid] = wid ? f - 1 : f;  // (others may still read top-k's)
      }
      __syncthreads();
    }
    if (min_p > 0.f) min_key = sh.edge[2];
    const uint32_t least_key = partial ? cut + 1 : cut;  // below it, only the cut's own ties
    uint32_t lo = max(sh.edge[3], least_key), hi = max(sh.edge[4], lo);
    // every weight once: all, above the neighbourhood, and inside it by finer bins
    unsigned long long sum = 0, above = 0;
    int shift = range_shift(lo, hi, 9);
    from = hi;
    listed = 0;
    {
      const float lf = logit_of(lo), hf = logit_of(hi), cf = logit_of(least_key);
      const bool deep = min_key > hi + 1;  // min_p cuts above the neighbourhood
      const float mf = logit_of(deep ? min_key : hi + 1);
#pragma unroll 2
      for (int i = 0; i < E / 2; ++i) {
        const float2 xy = own[i];
        if (by_k && !(fmaxf(xy.x, xy.y) >= cf)) continue;
        unsigned long long w2[2];
        W.two(xy, w2[0], w2[1]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float x = e ? xy.y : xy.x;
          const unsigned long long w = by_k && !(x >= cf) ? 0ull : w2[e];
          sum += w;
          if (x >= mf) mass += w, ++cnt;
          if (deep && x > hf) above += w;
          if (x >= lf && x <= hf) {
            if (listed < Sh::kSlots) sh.list[listed][tid] = (uint8_t)(2 * i + e);
            ++listed;
          }
        }
      }
      if (!deep) above = mass;
      if (listed <= Sh::kSlots) {
        for (int i = 0; i < listed; ++i) {
          const float x = vals[tid * E + sh.list[i][tid]];
          cl.add_fine(hi - key_of(x) >> shift, W(x));
        }
      } else {
        for (int i = 0; i < E; ++i) {
          const float x = vals[tid * E + i];
          if (x >= lf && x <= hf) cl.add_fine(hi - key_of(x) >> shift, W(x));
        }
      }
    }
    cl.sum(sum, above);
    sum += tie_mass;
    unsigned long long goal = part_of(fmaxf(top_p, 0.f), sum, true);
    goal = goal ? goal : 1ull;
    // the first logit from above at which the running weight reaches the goal
    bool moved = false;  // out of the neighbourhood
    while (true) {
      cl.sum_fine();
      constexpr int FE = kFine / THREADS > 1 ? kFine / THREADS : 1;
      unsigned long long m[FE], mine_m = 0, total;
#pragma unroll
      for (int e = 0; e < FE; ++e) {
        const int i = tid * FE + e;
        m[e] = i < kFine ? sh.fine[i][0] : 0ull;
        mine_m += m[e];
      }
      unsigned long long at = above + cl.scan(mine_m, total);
#pragma unroll
      for (int e = 0; e < FE; ++e) {
        if (at < goal && goal <= at + m[e])
          sh.found[0] = tid * FE + e, sh.found[1] = at, sh.found[2] = sh.fine[tid * FE + e][1], sh.found[3] = m[e];
        at += m[e];
      }
      __syncthreads();
      if (above >= goal) {  // the goal lies above this range
        lo = hi + 1;
        hi = top;
        above = 0;
        moved = true;
      } else if (above + total < goal) {  // or below it
        above += total;
        if (lo <= least_key) {  // only the cut's own ties are left
          const unsigned long long wc = W(logit_of(cut));
          const unsigned long long need = wc ? (goal - above + wc - 1) / wc : ties;
          ties = need < ties ? need : ties;
          break;
        }
        hi = lo - 1;
        lo = least_key;
        moved = true;
      } else {
        const int f = (int)sh.found[0];
        above = sh.found[1];
        take_bin(lo, hi, shift, (uint32_t)f);
        const unsigned long long c = sh.found[2];
        if (c == 1 || lo == hi) {
          const unsigned long long wl = c == 1 ? 0ull : sh.found[3] / c;
          const unsigned long long need = c == 1 ? 1ull : (goal - above + wl - 1) / wl;
          partial = need < c;
          ties = need;
          cut = lo;
          break;
        }
      }
      shift = range_shift(lo, hi, 9);
      __syncthreads();  // found has been read, the histogram cleared
      const float lf = logit_of(lo), hf = logit_of(hi);
      if (!moved && listed <= Sh::kSlots) {
        for (int i = 0; i < listed; ++i) {
          const float x = vals[tid * E + sh.list[i][tid]];
          if (x >= lf && x <= hf) cl.add_fine(hi - key_of(x) >> shift, W(x));
        }
      } else {
        for (int i = 0; i < E / 2; ++i) {
          const float2 xy = own[i];
          if (xy.x >= lf && xy.x <= hf) cl.add_fine(hi - key_of(xy.x) >> shift, W(xy.x));
          if (xy.y >= lf && xy.y <= hf) cl.add_fine(hi - key_of(xy.y) >> shift, W(xy.y));
        }
      }
    }
    if (moved) {  // the cut came out elsewhere: count again
      from = 0xffffffffu;
      mass = 0;
      cnt = 0;
    }
    if (moved || partial || listed > Sh::kSlots) listed = -1;
  } else if (min_p > 0.f) {
    __syncthreads();
    min_key = sh.edge[2];
  }
  if (min_key > cut) {  // min_p cuts deeper
    cut = min_key;
    partial = false;
  }

  // ranks of the cut's ties in order of id
  const float cf = logit_of(cut), ff = logit_of(min(from, top));
  unsigned long long rank = 0;
  if (partial) {
    unsigned long long n = 0, total;
    for (int i = 0; i < E; ++i) n += vals[tid * E + i] == cf;
    rank = cl.scan(n, total);
    const int p = cl.exchange(total, 0);
    for (unsigned r = 0; r < cl.rank; ++r) rank += sh.slot[p][r][0];
  }
  if (listed >= 0) {
    for (int i = 0; i < listed; ++i) {
      const float x = vals[tid * E + sh.list[i][tid]];
      if (x >= cf) mass += W(x), ++cnt;
    }
  } else if (cut <= from) {
    unsigned long long r = rank;
#pragma unroll 1
    for (int i = 0; i < E / 2; ++i) {
      const float2 xy = own[i];
      if (!(fmaxf(xy.x, xy.y) >= cf)) continue;
      unsigned long long w2[2];
      W.two(xy, w2[0], w2[1]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float x = e ? xy.y : xy.x;
        if (!(x >= cf && x <= ff)) continue;
        if (partial && x == cf && r++ >= ties) continue;
        mass += w2[e];
        ++cnt;
      }
    }
  }
  // the pick: the thread whose ids hold it, then its ids by a warp
  unsigned long long total, kept, in_cta, n_cta;
  unsigned long long before = cl.scan(mass, in_cta);
  cl.scan(cnt, n_cta);
  {
    const int p = cl.exchange(in_cta, n_cta);
    total = kept = 0;
    for (unsigned r = 0; r < size; ++r) {
      if (r < cl.rank) before += sh.slot[p][r][0];
      total += sh.slot[p][r][0];
      kept += sh.slot[p][r][1];
    }
  }
  const unsigned long long goal = u >= 1.f ? total - 1 : u > 0.f ? part_of(u, total, false) : 0ull;
  if (cl.rank == 0 && tid == 0 && a.kept) a.kept[row] = (int)kept;
  const unsigned holder = __ballot_sync(0xffffffffu, goal >= before && goal < before + mass);
  if (holder) {
    const int t = __ffs(holder) - 1;
    unsigned long long run = __shfl_sync(0xffffffffu, before, t), r = __shfl_sync(0xffffffffu, rank, t);
    const int first = (tid - lane + t) * E;
    for (int i0 = 0; i0 < E; i0 += 32) {
      const int i = i0 + lane;
      const float x = i < E ? vals[first + i] : kMasked;
      const unsigned tie = __ballot_sync(0xffffffffu, x == cf);
      const unsigned long long my = r + __popc(tie & ((1u << lane) - 1));
      r += __popc(tie);
      const unsigned long long w = x >= cf && !(partial && x == cf && my >= ties) ? W(x) : 0ull;
      unsigned long long inc = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, run + inc > goal);
      if (hit) {
        if (lane == __ffs(hit) - 1) a.ids[row] = base + first + i;
        break;
      }
      run += __shfl_sync(0xffffffffu, inc, 31);
    }
  }
  cl.sync();
}

// ---- many rows ------------------------------------------------------------------------
// With more rows than the GPU holds at once, what every thread does once per row counts as much
// as what it does per logit, so a row gets only two CTAs of 512 threads, and the logits, too many
// for their shared memory, are read again from L2 (the rows in flight fit it) for the second
// pass. Warps take segments of 1024 consecutive ids, whose kept weights the pick searches.
// The bins of the first pass hang on the largest of the row's first logits (256 bins above it, 8
// octaves of weight; a row whose later logits are higher still is counted again: of 256 rows of
// normal logits of spread 3 238 at T = 0.3, 282 us instead of 228, and 18 at T = 1, 281 / 264).
// Rows of 151936 in a captured graph, us, clusters of eight / this: top_k 50 with top_p 0.9, 96
// rows 82 / 106, 128 rows 109 / 110, 256 rows 204 / 195; top_p 0.9 alone 114 / 142, 150 / 144,
// 282 / 262.
constexpr int kManyRows = 128, kManyVocab = 100352;  // (two CTAs hold a row of as many)
constexpr int kStream = 512, kSegment = 1024, kAhead = 256;

struct StreamShared {
  static constexpr int kWarps = kStream / 32, kSlots = 16;
  alignas(16) uint32_t hist[kBins];
  union {  // of the cluster, by sum_hist() or sum_fine()
    uint32_t all[kBins];
    unsigned long long fine[kFine][2];  // weight, count
  };
  unsigned long long slot[2][16][2];
  unsigned long long warp[kWarps][2];
  unsigned long long found[4];
  unsigned long long table[256];
  unsigned long long seg[DMTP_OPS_MAX_SAMPLE_VOCAB / 2 / kSegment];  // kept weight of a segment
  uint32_t seg_n[DMTP_OPS_MAX_SAMPLE_VOCAB / 2 / kSegment];          // ties of the cut in it
  uint8_t list[kSlots][kStream];  // a thread's logits in the neighbourhood: where, and which
  float value[kSlots][kStream];
  uint32_t edge[5];  // keys: top-k's bin, min_p's cut, top-p's neighbourhood
  int bins[2];
};

template <typename T>
__global__ void __launch_bounds__(kStream, 2) k_sample_stream(const RowsArgs sa) {
  using Sh = StreamShared;
  constexpr int X = 16 / sizeof(T), J = 32 / X;  // ids of a load, loads of a thread and segment
  extern __shared__ __align__(16) unsigned char smem[];
  Sh& sh = *reinterpret_cast<Sh*>(smem);
  const dmtp_sample_args& a = sa.a;
  unsigned size;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(size));
  Cluster<kStream, Sh> cl{&sh, cluster_rank(), size, 0};
  cl.arrive();
  const int row = blockIdx.x / size, tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int base = (int)cl.rank * sa.slice, end = min(a.vocab, base + sa.slice);
  const int segs = end > base ? (end - base + kSegment - 1) / kSegment : 0;
  const T* lg = (const T*)a.logits + (int64_t)row * a.ld;
  // X logits from id on (masked past `end`)
  auto load = [&](int id, float (&f)[X]) {
    if (sa.vec && id + X <= end) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(lg + id));
      const T* t = reinterpret_cast<const T*>(&u);
#pragma unroll
      for (int e = 0; e < X; ++e) f[e] = clean(to_f32(t[e]));
    } else {
#pragma unroll
      for (int e = 0; e < X; ++e) f[e] = id + e < end ? clean(to_f32(__ldg(lg + id + e))) : kMasked;
    }
  };
  auto id_of = [&](int seg, int j) { return base + seg * kSegment + j * (32 * X) + lane * X; };
  const float temp = a.temperature ? __ldg(a.temperature + row) : 1.f;
  const int k = a.top_k ? __ldg(a.top_k + row) : 0;
  const float top_p = a.top_p ? __ldg(a.top_p + row) : 1.f;
  const float min_p = a.min_p ? __ldg(a.min_p + row) : 0.f;
  const float u = __ldg(a.u + row);
  const bool greedy = !(temp > 0.f), by_p = top_p < 1.f, binned = !greedy && (k > 0 || by_p);
  for (int i = tid; i < 256; i += kStream) sh.table[i] = exp2_256th(i);
  for (int i = tid; i < kBins; i += kStream) sh.hist[i] = 0;
  for (int i = tid; i < segs; i += kStream) sh.seg[i] = 0, sh.seg_n[i] = 0;
  Weigh W;
  W.table = sh.table;
  const float tt = fminf(fmaxf(temp, 1e-30f), 1e30f);
  W.chi = 1.44269502162933349609f / tt;
  W.clo = (fmaf(-W.chi, tt, 1.44269502162933349609f) + 1.92596299112661746887e-08f) / tt;
  W.cb = W.chi * 32.f;

  // the first pass: the largest logit and, for the filters, the bins
  float from_l = kMasked;  // what the bins hang on: both CTAs look at the same logits
  if (binned) {
    float best = kMasked;
    for (int i = tid; i < min(a.vocab, 2 * kStream); i += kStream) best = fmaxf(best, clean(to_f32(__ldg(lg + i))));
    from_l = logit_of(cl.cta_max(key_of(best)));
  }
  int ahead = kAhead;
  const float cb = W.cb;
  // Bin of a logit: (from_l - l) cb to the nearest, `ahead` bins later.
  auto bin_of = [&](float l) {
    const float y = fmaxf((l - from_l) * cb, -4096.f);  // (masked: 4096)
    return ahead - (__float_as_int(fminf(y, 4096.f) + 12582912.f) - 0x4b400000);
  };
  uint32_t top = 0;
  unsigned long long nvalid = 0;
  cl.wait();  // every CTA of the cluster runs before one writes another's memory
  while (true) {
    float best = kMasked;
    uint32_t last = 0;
    const bool use = binned && from_l > kMasked;
    __syncthreads();  // the histogram is clear
    for (int s = wid; s < segs; s += Sh::kWarps) {
#pragma unroll 2
      for (int j = 0; j < J; ++j) {
        float f[X];
        load(id_of(s, j), f);
#pragma unroll
        for (int e = 0; e < X; ++e) {
          best = fmaxf(best, f[e]);
          if (use) {
            const int b = max(bin_of(f[e]), 0);
            if (b < kBins - 1)
              atomicAdd(&sh.hist[b], 1u);
            else
              last += f[e] > kMasked;
          }
        }
      }
    }
    const uint32_t my_top = cl.cta_max(key_of(best));
    unsigned long long l64 = last, pad = 0;
    cl.cta_sum(l64, pad);
    const int p = cl.exchange(my_top, l64);
    top = 0;
    unsigned long long lasts = 0;
    for (unsigned r = 0; r < size; ++r) {
      top = max(top, (uint32_t)sh.slot[p][r][0]);
      lasts += sh.slot[p][r][1];
    }
    nvalid = lasts;  // and the bins' counts, below
    if (!binned || top == kMaskedKey) break;
    if (use && bin_of(logit_of(top)) >= 0) break;
    // the first logits were far below the largest, or masked: hang the bins on that one
    from_l = logit_of(top);
    ahead = 0;
    cl.sync();
    for (int i = tid; i < kBins; i += kStream) sh.hist[i] = 0;
  }
  W.top = logit_of(top);
  const bool none = top == kMaskedKey;
  if (none || greedy) {
    uint32_t id = 0;  // of the largest logit, the lowest: 2^32 - 1 - id is maximal
    if (!none)
      for (int s = wid; s < segs; s += Sh::kWarps)
        for (int j = 0; j < J; ++j) {
          float f[X];
          load(id_of(s, j), f);
#pragma unroll
          for (int e = 0; e < X; ++e)
            if (f[e] == W.top) id = max(id, 0xffffffffu - (unsigned)(id_of(s, j) + e));
        }
    id = cl.cta_max(id);
    const int p = cl.exchange(id, 0);
    id = 0;
    for (unsigned r = 0; r < size; ++r) id = max(id, (uint32_t)sh.slot[p][r][0]);
    if (cl.rank == 0 && tid == 0) {
      a.ids[row] = none ? -1 : (int)(0xffffffffu - id);
      if (a.kept) a.kept[row] = none ? 0 : 1;
    }
    cl.sync();  // no CTA leaves while another may still write its slots
    return;
  }
  // the smallest logit that stays, as a key; `ties` of its ids stay, all of them unless `partial`
  uint32_t cut = kLowestKey;
  unsigned long long ties = 0;
  bool partial = false, by_k = false;
  // The smallest key of bins 0..b, top + 1 if none is that high. One warp.
  auto bin_edge = [&](int b) {
    auto in = [&](float x) { return bin_of(x) <= b; };
    return b >= kBins - 1 ? kLowestKey : b >= 0 && in(W.top) ? first_key(top, in) : top + 1;
  };
  // every logit in [lo, hi]
  auto each_in = [&](uint32_t lo, uint32_t hi, auto&& f) {
    const float lf = logit_of(lo), hf = logit_of(hi);
    for (int s = wid; s < segs; s += Sh::kWarps)
#pragma unroll 2
      for (int j = 0; j < J; ++j) {
        float x[X];
        load(id_of(s, j), x);
#pragma unroll
        for (int e = 0; e < X; ++e)
          if (x[e] >= lf && x[e] <= hf) f(x[e]);
      }
  };

  if (binned) {
    constexpr int N = kBins / kStream;
    cl.sum_hist();
    unsigned long long n = 0, total, before, cnt, want = k;
#pragma unroll
    for (int e = 0; e < N; ++e) n += tid * N + e < kBins - 1 ? sh.all[tid * N + e] : 0u;
    cl.scan(n, total);
    if (tid == 0) sh.all[kBins - 1] = (uint32_t)nvalid;  // the last bin was counted by thread
    nvalid += total;
    __syncthreads();
    by_k = k > 0 && (unsigned long long)k < nvalid;
    int last_bin = kBins - 1;           // the last bin that top-k leaves
    unsigned long long last_n = ~0ull;  // and how many of its logits
    if (by_k) {
      cl.find_count(want, last_bin, before, cnt);
      want -= before;
      last_n = want;
    }
    if (by_p) cl.neighbours(top_p, last_bin, last_n, (float)bin_of(W.top));
    if (by_k) {
      if (wid < 2) {
        const uint32_t f = bin_edge(wid ? last_bin - 1 : last_bin);
        if (lane == 0) sh.edge[wid] = wid ? f - 1 : f;
      }
      __syncthreads();
      uint32_t lo = sh.edge[0], hi = sh.edge[1];
      while (want != cnt && lo != hi) {
        const int shift = range_shift(lo, hi, 11);
        each_in(lo, hi, [&](float x) { atomicAdd(&sh.hist[hi - key_of(x) >> shift], 1u); });
        cl.sum_hist();
        int f;
        cl.find_count(want, f, before, cnt);
        want -= before;
        take_bin(lo, hi, shift, (uint32_t)f);
      }
      cut = lo;
      partial = want != cnt;
      ties = want;
    }
  }
  const unsigned long long tie_mass = partial ? ties * W(logit_of(cut)) : 0ull;
  const uint32_t least_key = partial ? cut + 1 : cut;  // below it, only the cut's own ties
  // the neighbourhood's ends and min_p as keys
  if (wid < 2 && by_p) {
    const uint32_t f = bin_edge(wid ? sh.bins[0] - 1 : sh.bins[1]);
    if (lane == 0) sh.edge[3 + wid] = wid ? f - 1 : f;  // (others may still read top-k's)
  }
  if (wid == 2 && min_p > 0.f) {
    const unsigned long long least = min_p < 1.f ? part_of(min_p, 1ull << kShift, true) : 1ull << kShift;
    const uint32_t f = first_key(top, [&](float x) { return W(x) >= least; });
    if (lane == 0) sh.edge[2] = f;
  }
  __syncthreads();
  const uint32_t min_key = min_p > 0.f ? sh.edge[2] : 0u;

  // The weights of a segment's logits, by pairs: f(weight, logit, code).
  auto weights = [&](int s, int step, float floor_l, auto&& f) {
#pragma unroll 2
    for (int j = 0; j < J; ++j) {
      float x[X];
      load(id_of(s, j), x);
#pragma unroll
      for (int e = 0; e < X; e += 2) {
        if (!(fmaxf(x[e], x[e + 1]) >= floor_l)) continue;
        unsigned long long w0, w1;
        W.two(make_float2(x[e], x[e + 1]), w0, w1);
        f(w0, x[e], step * 32 + j * X + e);
        f(w1, x[e + 1], step * 32 + j * X + e + 1);
      }
    }
  };
  // Add a thread's kept weight to its warp's segment.
  auto add_segment = [&](int s, unsigned long long m) {
    const uint32_t lo = __reduce_add_sync(0xffffffffu, (uint32_t)m & 0xffffffu);
    const uint32_t mid = __reduce_add_sync(0xffffffffu, (uint32_t)(m >> 24) & 0xffffffu);
    const uint32_t hi = __reduce_add_sync(0xffffffffu, (uint32_t)(m >> 48));
    if (lane == 0) sh.seg[s] += (unsigned long long)lo + ((unsigned long long)mid << 24) + ((unsigned long long)hi << 48);
  };

  uint32_t cnt = 0, from = 0xffffffffu;  // kept logits, so far those above `from`
  int listed = -1;                       // >= 0: the others are in this thread's list, so many
  if (by_p) {
    uint32_t lo = max(sh.edge[3], least_key), hi = max(sh.edge[4], lo);
    // every weight once: all, above the neighbourhood, and a list of the neighbourhood
    unsigned long long sum = 0, above = 0;
    int shift = range_shift(lo, hi, 9);
    from = hi;
    listed = 0;
    {
      const float lf = logit_of(lo), hf = logit_of(hi), cf = by_k ? logit_of(least_key) : kMasked;
      const bool deep = min_key > hi + 1;  // min_p cuts above the neighbourhood
      const float mf = logit_of(deep ? min_key : hi + 1);
      int step = 0;
      for (int s = wid; s < segs; s += Sh::kWarps, ++step) {
        unsigned long long mass = 0;
        weights(s, step, cf, [&](unsigned long long w, float x, int code) {
          if (by_k && !(x >= cf)) w = 0;
          sum += w;
          const bool over = x >= mf;
          if (over) mass += w, ++cnt;
          if (deep && x > hf) above += w;
          if (x >= lf && !over && x <= hf) {
            if (listed < Sh::kSlots) sh.list[listed][tid] = (uint8_t)code, sh.value[listed][tid] = x;
            ++listed;
          }
        });
        if (!deep) above += mass;
        add_segment(s, mass);
      }
    }
    // the first logit from above at which the running weight reaches the goal: finer bins
    bool moved = false;  // out of the neighbourhood
    unsigned long long goal = 0;
    while (true) {
      if (!moved && listed <= Sh::kSlots) {
        const float lf = logit_of(lo), hf = logit_of(hi);
        for (int i = 0; i < listed; ++i) {
          const float x = sh.value[i][tid];
          if (x >= lf && x <= hf) cl.add_fine(hi - key_of(x) >> shift, W(x));
        }
      }
      // (a thread whose list overflowed, or a range outside: over its logits again; the loads of
      // a warp stay together)
      if (__any_sync(0xffffffffu, moved || listed > Sh::kSlots)) {
        const bool mine = moved || listed > Sh::kSlots;
        each_in(lo, hi, [&](float x) {
          if (mine) cl.add_fine(hi - key_of(x) >> shift, W(x));
        });
      }
      if (!goal) {  // the first time, with the sums
        cl.cta_sum(sum, above);
        const int p = cl.exchange(sum, above);
        sum = tie_mass;
        above = 0;
        for (unsigned r = 0; r < size; ++r) sum += sh.slot[p][r][0], above += sh.slot[p][r][1];
        goal = part_of(fmaxf(top_p, 0.f), sum, true);
        goal = goal ? goal : 1ull;
      }
      cl.sum_fine();
      static_assert(kFine == kStream, "a fine bin a thread");
      const unsigned long long m = sh.fine[tid][0];
      unsigned long long total;
      const unsigned long long at = above + cl.scan(m, total);
      if (at < goal && goal <= at + m) sh.found[0] = tid, sh.found[1] = at, sh.found[2] = sh.fine[tid][1], sh.found[3] = m;
      __syncthreads();
      if (above >= goal) {  // the goal lies above this range
        lo = hi + 1;
        hi = top;
        above = 0;
        moved = true;
      } else if (above + total < goal) {  // or below it
        above += total;
        if (lo <= least_key) {  // only the cut's own ties are left
          const unsigned long long wc = W(logit_of(cut));
          const unsigned long long need = wc ? (goal - above + wc - 1) / wc : ties;
          ties = need < ties ? need : ties;
          break;
        }
        hi = lo - 1;
        lo = least_key;
        moved = true;
      } else {
        const int f = (int)sh.found[0];
        above = sh.found[1];
        take_bin(lo, hi, shift, (uint32_t)f);
        const unsigned long long n = sh.found[2];
        if (n == 1 || lo == hi) {
          const unsigned long long wl = n == 1 ? 0ull : sh.found[3] / n;
          const unsigned long long need = n == 1 ? 1ull : (goal - above + wl - 1) / wl;
          partial = need < n;
          ties = need;
          cut = lo;
          break;
        }
      }
      shift = range_shift(lo, hi, 9);
      __syncthreads();  // found has been read
    }
    if (moved) {  // the cut came out elsewhere: count again
      from = 0xffffffffu;
      cnt = 0;
      for (int i = tid; i < segs; i += kStream) sh.seg[i] = 0;
      __syncthreads();
      listed = -1;
    }
  }
  if (min_key > cut) {  // min_p cuts deeper
    cut = min_key;
    partial = false;
  }

  // what the neighbourhood keeps (of the cut itself only if all its ties stay)
  const float cf = logit_of(cut), ff = logit_of(min(from, top));
  const bool again = listed < 0 || listed > Sh::kSlots;
  if (!again)
    for (int i = 0; i < listed; ++i) {
      const int code = sh.list[i][tid];
      const float x = sh.value[i][tid];
      if (x > cf || (x == cf && !partial)) {
        atomicAdd(&sh.seg[(code >> 5) * Sh::kWarps + wid], W(x));
        ++cnt;
      }
    }
  if (__any_sync(0xffffffffu, again) && cut <= from) {
    int step = 0;
    for (int s = wid; s < segs; s += Sh::kWarps, ++step) {
      unsigned long long mass = 0;
      weights(s, step, cf, [&](unsigned long long w, float x, int) {
        if (again && x <= ff && (x > cf || (x == cf && !partial))) mass += w, ++cnt;
      });
      add_segment(s, mass);
    }
  }
  // the cut's ties, lowest ids first
  const unsigned long long wc = partial ? W(cf) : 0ull;
  if (partial) {
    for (int s = wid; s < segs; s += Sh::kWarps) {
      uint32_t n = 0;
      for (int j = 0; j < J; ++j) {
        float x[X];
        load(id_of(s, j), x);
#pragma unroll
        for (int e = 0; e < X; ++e) n += x[e] == cf;
      }
      n = __reduce_add_sync(0xffffffffu, n);
      if (lane == 0) sh.seg_n[s] = n;
    }
  }
  __syncthreads();
  // the pick: the segment that holds it (of `segs` <= 512, one a thread), then its ids
  unsigned long long rank = 0, total, kept, in_cta, n_cta = cnt, pad = 0, tie_n = 0;
  const uint32_t my_ties = partial && tid < segs ? sh.seg_n[tid] : 0u;
  if (partial) {
    rank = cl.scan(my_ties, tie_n);
    const int p = cl.exchange(tie_n, 0);
    for (unsigned r = 0; r < cl.rank; ++r) rank += sh.slot[p][r][0];
    tie_n = rank < ties ? min((unsigned long long)my_ties, ties - rank) : 0ull;
    n_cta += tie_n;
  }
  const unsigned long long mass = (tid < segs ? sh.seg[tid] : 0ull) + tie_n * wc;
  unsigned long long before = cl.scan(mass, in_cta);
  cl.cta_sum(n_cta, pad);
  {
    const int p = cl.exchange(in_cta, n_cta);
    total = kept = 0;
    for (unsigned r = 0; r < size; ++r) {
      if (r < cl.rank) before += sh.slot[p][r][0];
      total += sh.slot[p][r][0];
      kept += sh.slot[p][r][1];
    }
  }
  const unsigned long long goal = u >= 1.f ? total - 1 : u > 0.f ? part_of(u, total, false) : 0ull;
  if (cl.rank == 0 && tid == 0 && a.kept) a.kept[row] = (int)kept;
  if (tid == 0) sh.found[3] = ~0ull;
  __syncthreads();
  if (goal >= before && goal < before + mass) sh.found[3] = tid, sh.found[0] = before, sh.found[1] = rank;
  __syncthreads();
  if (sh.found[3] != ~0ull) {  // two ids a thread
    const int s = (int)sh.found[3], id = base + s * kSegment + 2 * tid;
    float x[2];
    unsigned long long w[2], t0, all;
#pragma unroll
    for (int e = 0; e < 2; ++e) x[e] = id + e < end ? clean(to_f32(__ldg(lg + id + e))) : kMasked;
    W.two(make_float2(x[0], x[1]), w[0], w[1]);
    const unsigned long long run = sh.found[0], r0 = sh.found[1];
    t0 = r0 + cl.scan(partial ? (x[0] == cf) + (x[1] == cf) : 0, all);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (!(x[e] >= cf) || (partial && x[e] == cf && t0 >= ties)) w[e] = 0;
      t0 += partial && x[e] == cf;
    }
    const unsigned long long at = run + cl.scan(w[0] + w[1], all);
    if (goal >= at && goal < at + w[0]) a.ids[row] = id;
    if (goal >= at + w[0] && goal < at + w[0] + w[1]) a.ids[row] = id + 1;
  }
  cl.sync();
}

}  // namespace

using namespace dmtp;

namespace {

template <typename T, int THREADS>
cudaError_t launch(const dmtp_sample_args& a, cudaStream_t st) {
  static unsigned long long done = 0;
  auto k = k_sample_rows<T, THREADS>;
  constexpr int kFixed = (sizeof(Shared<THREADS>) + 15) / 16 * 16;
  // A thread's ids: an odd number of pairs, so that the threads' pairs lie in different banks
  auto pairs_of = [](int n) {
    const int p = (n + 2 * THREADS - 1) / (2 * THREADS);
    return p + 1 - p % 2;
  };
  auto bytes_of = [&](unsigned c) { return kFixed + 2 * pairs_of((a.vocab + (int)c - 1) / (int)c) * THREADS * 4; };
  constexpr int kMost = 227 * 1024;  // the largest slice: a CTA of its own on an SM
  if (!smem_limit((const void*)k, kMost, &done)) return cudaErrorInvalidValue;
  // CTAs of a row. One while a pass over the row is short; else as many as leave each an SM of its
  // own, up to 8 (the barriers of a cluster cost more where it shares its SMs: above 8 rows only
  // if the row is long), and if the slices do not fit that way, 8 that share the SMs.
  // Rows of top_k 50 and top_p 0.9, us with 1 / 2 / 4 / 8 CTAs:
  //            1 row                      16 rows                    64 rows
  //   8192     16.5 / 17.2 / 16.4 / 15.9  17.4 / 18.6 / 17.9 / 19.6  17.8 / 18.9 / 22.3 / 40.5
  //   32768    21.9 / 19.4 / 17.2 / 16.4  24.9 / 22.2 / 19.6 / 21.8  25.2 / 22.8 / 24.8 / 44.2
  //   100000      - / 30.2 / 23.2 / 20.1     - / 32.0 / 24.8 / 22.8     - / 35.0 / 48.4 / 50.2
  //   151936      -      - / 24.4 / 19.8     -      - / 28.8 / 23.8     -      - / 61.7 / 57.4
  // 32 rows of 32768 22.3 with 2, 20.1 with 4, of 100000 25.0 with 4, 26.4 with 8; 127 rows of
  // 32768 25.7 / 28.8 / 45.8 / 83.4; 256 rows of 32768 51.5 / 53.2 / 85.8 / 161 (streamed 73.7), of
  // 100000 130.9 with 2 (streamed 153.8).
  unsigned cluster = a.vocab <= 8192 ? 1 : a.rows <= 8 || a.vocab > 65536 ? 8 : 4;
  while (cluster > 1 && (unsigned)a.rows * cluster > 152 && bytes_of(cluster / 2) <= kMost) cluster /= 2;
  if (bytes_of(2) > kMost && (unsigned)a.rows * cluster > 152) cluster = 8;
  RowsArgs s;
  s.a = a;
  s.slice = (bytes_of(cluster) - kFixed) / 4;
  const int es = sizeof(T);
  s.vec = aligned_to(a.logits, 16) && mult(a.ld * es, 16);
  return launch_op(k, (unsigned)a.rows * cluster, THREADS, (size_t)bytes_of(cluster), st, false, cluster, s);
}
template <typename T>
cudaError_t launch_stream(const dmtp_sample_args& a, cudaStream_t st) {
  static unsigned long long done = 0;
  auto k = k_sample_stream<T>;
  if (!smem_limit((const void*)k, sizeof(StreamShared), &done)) return cudaErrorInvalidValue;
  RowsArgs s;
  s.a = a;
  s.slice = ((a.vocab + 1) / 2 + kSegment - 1) / kSegment * kSegment;
  s.vec = aligned_to(a.logits, 16) && mult(a.ld * (int)sizeof(T), 16);
  return launch_op(k, (unsigned)a.rows * 2, kStream, sizeof(StreamShared), st, false, 2, s);
}
template <typename T>
cudaError_t launch_t(const dmtp_sample_args& a, cudaStream_t st) {
  if (a.rows >= kManyRows && a.vocab > kManyVocab) return launch_stream<T>(a, st);
  return launch<T, 512>(a, st);
}

}  // namespace

extern "C" int dmtp_sample_rows(const dmtp_sample_args* a, void* stream) {
  if (!a || a->rows < 0) return DMTP_EINVAL;
  if (a->rows == 0) return DMTP_OK;
  if (!a->logits || !a->u || !a->ids || (a->dtype != 0 && a->dtype != 1) || a->vocab < 1 ||
      a->vocab > DMTP_OPS_MAX_SAMPLE_VOCAB || a->ld < a->vocab || a->rows > (1 << 24))
    return DMTP_EINVAL;
  if (!aligned_to(a->logits, a->dtype ? 2 : 4)) return DMTP_EINVAL;
  const void* words[] = {a->u, a->temperature, a->top_k, a->top_p, a->min_p, a->ids, a->kept};
  for (const void* p : words)
    if (!aligned_to(p, 4)) return DMTP_EINVAL;
  if (cudaPeekAtLastError() != cudaSuccess) return DMTP_ECUDA;
  const cudaError_t e = a->dtype ? launch_t<bf16>(*a, (cudaStream_t)stream) : launch_t<float>(*a, (cudaStream_t)stream);
  return e == cudaSuccess ? DMTP_OK : (cudaGetLastError(), DMTP_ECUDA);
}
