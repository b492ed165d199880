// dmtp_sample_rows: temperature, top-k, top-p and min-p sampling from one given uniform
// number per row.
//
// A cluster of CTAs takes a row: each holds a slice of it in shared memory, as keys whose
// unsigned order is the logits' order, so the logits are read from HBM once and every later
// step runs on chip. Counts and weights are reduced over the cluster through distributed
// shared memory.
//
// Weights. 2^y with y = (l - max) log2(e) / T as a 64-bit integer, so that sums are exact
// and associative: no result depends on how a row was split. The exponent is formed as a
// pair of floats (the difference, the factor and their product with their rounding errors);
// 2^y = 2^n 2^(j/256) e^z with a table of 2^(j/256) in 62-bit fixed point and
// e^z - 1 = z + z^2/2 + z^3/6 + z^4/24 (|z| < 0.00136, next term 4e-17). The scale is
// chosen per row so that the row's sum stays below 2^62; the relative error of a weight is
// about 2^-40.
//
// Filters. The cut is a key and the number of its ties that stay (lowest ids first): the
// largest key whose count from above reaches top_k, then the largest whose weight from above
// reaches top_p of the kept weight, found a bit at a time.
#include <math.h>

#include "paged.cuh"

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr uint32_t kNone = 0u;            // key of a logit that is never kept

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
  int slice;  // keys of a CTA, a multiple of kThreads
  bool vec;   // rows allow 16-byte loads
};

__device__ __forceinline__ uint32_t key_of(float l) {
  l += 0.f;  // -0 ties with +0
  const uint32_t u = __float_as_uint(l);
  if (!(l > -INFINITY)) return kNone;  // NaN, -infinity
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
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

struct Weigh {
  float top, chi, clo;
  int shift;  // weight 1 is 2^shift
  const unsigned long long* table;

  // y = (l - max) c as a pair of floats
  __device__ __forceinline__ void exponent(float l, float& hi, float& lo) const {
    const float d = l - top, t = d - l;
    const float e = (l - (d - t)) + (-top - t);
    hi = d * chi;
    lo = fmaf(d, chi, -hi) + fmaf(d, clo, e * chi);
  }
  __device__ __forceinline__ float rough(uint32_t key) const {
    const float l = logit_of(key);
    const float y = (l - top) * chi;
    return l == top ? 1.f : y > -64.f ? ex2(y) : 0.f;
  }
  __device__ __forceinline__ unsigned long long operator()(uint32_t key) const {
    const float l = logit_of(key);
    if (l == top) return 1ull << shift;
    float hi, lo;
    exponent(l, hi, lo);
    if (!(hi > -64.f)) return 0ull;
    const int j = __float2int_rn(hi * 256.f);  // |j| < 2^14
    const float r = fmaf((float)j, -0.00390625f, hi);  // exact
    // z = (r + lo) ln 2
    const float zh = r * 0.693147182464599609f;
    const float zl = fmaf(r, 0.693147182464599609f, -zh) + fmaf(r, -1.90465429995776804525e-09f, lo * 0.693147182464599609f);
    const float z2 = zh * zh;
    const float p = zl + z2 * fmaf(zh, fmaf(zh, 0.0416666679f, 0.166666672f), 0.5f);
    const int g = __float2int_rn(zh * 1099511627776.f) + __float2int_rn(p * 1099511627776.f);  // 2^40
    const unsigned long long t = table[j & 255];
    const long long w = (long long)t + (((long long)(t >> 32) * g) >> 8);  // 62 bits: Q30 Q40 2^-8
    const int down = 62 - shift - (j >> 8);
    if (down > 63) return 0ull;
    return down > 0 ? ((unsigned long long)w + (1ull << (down - 1))) >> down : (unsigned long long)w;
  }
};

struct Shared {
  unsigned long long slot[2][16][2];  // one (count, weight) of each CTA of the cluster, twice
  unsigned long long warp[kWarps][2];
  unsigned long long total[2];
  int pick;
};

struct Cluster {
  Shared* s;
  unsigned rank, size;
  int phase;

  __device__ __forceinline__ void sync() const {
    if (size > 1)
      cluster_sync_all();
    else
      __syncthreads();
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
  // Sums of (a, b) over all threads of the cluster.
  __device__ __forceinline__ void sum(unsigned long long& a, unsigned long long& b) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s->warp[threadIdx.x >> 5][0] = a, s->warp[threadIdx.x >> 5][1] = b;
    __syncthreads();
    a = b = 0;
    if (threadIdx.x < 32) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) a += s->warp[w][0], b += s->warp[w][1];
    }
    const int p = exchange(a, b);
    a = b = 0;
    for (unsigned r = 0; r < size; ++r) a += s->slot[p][r][0], b += s->slot[p][r][1];
  }
  __device__ __forceinline__ unsigned long long max(unsigned long long a) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long v = __shfl_xor_sync(0xffffffffu, a, o);
      a = a > v ? a : v;
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s->warp[threadIdx.x >> 5][0] = a;
    __syncthreads();
    if (threadIdx.x < 32) {
#pragma unroll
      for (int w = 0; w < kWarps; ++w) a = a > s->warp[w][0] ? a : s->warp[w][0];
    }
    const int p = exchange(a, 0);
    a = 0;
    for (unsigned r = 0; r < size; ++r) a = a > s->slot[p][r][0] ? a : s->slot[p][r][0];
    return a;
  }
  // Exclusive sums, in order of warps and CTAs, of one pair per warp (valid in lane 0 of each
  // warp); also the totals.
  __device__ __forceinline__ void scan(unsigned long long a, unsigned long long b,
                                       unsigned long long& before_a, unsigned long long& before_b,
                                       unsigned long long& all_a, unsigned long long& all_b) {
    const int wid = threadIdx.x >> 5;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s->warp[wid][0] = a, s->warp[wid][1] = b;
    __syncthreads();
    unsigned long long ta = 0, tb = 0;
    before_a = before_b = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w == wid) before_a = ta, before_b = tb;
      ta += s->warp[w][0];
      tb += s->warp[w][1];
    }
    const int p = exchange(ta, tb);
    all_a = all_b = 0;
    for (unsigned r = 0; r < size; ++r) {
      if (r < rank) before_a += s->slot[p][r][0], before_b += s->slot[p][r][1];
      all_a += s->slot[p][r][0];
      all_b += s->slot[p][r][1];
    }
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads) k_sample_rows(const RowsArgs sa) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ Shared sh;
  __shared__ unsigned long long table[256];
  const dmtp_sample_args& a = sa.a;
  unsigned size;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(size));
  Cluster cl{&sh, cluster_rank(), size, 0};
  const int row = blockIdx.x / size, tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int V = a.vocab, slice = sa.slice;
  const int base = (int)cl.rank * slice;
  const int mine = V > base ? min(slice, V - base) : 0;
  const T* lg = (const T*)a.logits + (int64_t)row * a.ld + base;
  if (tid < 256) table[tid] = exp2_256th(tid);
  uint32_t best = 0;
  if (sa.vec) {
    constexpr int E = 16 / sizeof(T);
    for (int i = tid * E; i < slice; i += kThreads * E) {
      uint32_t k[E];
      if (i + E <= mine) {
        const uint4 u = __ldcs(reinterpret_cast<const uint4*>(lg + i));
        const T* t = reinterpret_cast<const T*>(&u);
#pragma unroll
        for (int e = 0; e < E; ++e) k[e] = key_of(to_f32(t[e]));
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) k[e] = i + e < mine ? key_of(to_f32(lg[i + e])) : kNone;
      }
#pragma unroll
      for (int e = 0; e < E; e += 4)
        *reinterpret_cast<uint4*>(keys + i + e) = make_uint4(k[e], k[e + 1], k[e + 2], k[e + 3]);
#pragma unroll
      for (int e = 0; e < E; ++e) best = max(best, k[e]);
    }
  } else {
    for (int i = tid; i < slice; i += kThreads) {
      const uint32_t k = i < mine ? key_of(to_f32(lg[i])) : kNone;
      keys[i] = k;
      best = max(best, k);
    }
  }
  cl.sync();  // every CTA of the cluster runs before one writes another's memory
  const uint32_t top = (uint32_t)cl.max(best);
  const float temp = a.temperature ? __ldg(a.temperature + row) : 1.f;
  const int k = a.top_k ? __ldg(a.top_k + row) : 0;
  const float top_p = a.top_p ? __ldg(a.top_p + row) : 1.f;
  const float min_p = a.min_p ? __ldg(a.min_p + row) : 0.f;
  const bool greedy = !(temp > 0.f);
  if (top == kNone || greedy) {
    unsigned long long id = 0;  // of the largest logit, the lowest: 2^32 - 1 - id is maximal
    for (int i = tid; i < mine; i += kThreads)
      if (keys[i] == top && top != kNone) id = max(id, (unsigned long long)(0xffffffffu - (unsigned)(base + i)));
    id = cl.max(id);
    if (cl.rank == 0 && tid == 0) {
      a.ids[row] = top == kNone ? -1 : (int)(0xffffffffu - (unsigned)id);
      if (a.kept) a.kept[row] = top == kNone ? 0 : 1;
    }
    cl.sync();  // no CTA leaves while another may still write its slots
    return;
  }
  Weigh W;
  W.top = logit_of(top);
  W.table = table;
  // c = log2(e) / T as a pair
  W.chi = 1.44269502162933349609f / temp;
  W.clo = (fmaf(-W.chi, temp, 1.44269502162933349609f) + 1.92596299112661746887e-08f) / temp;
  float rough = 0.f;
  unsigned long long nvalid = 0, none = 0;
  for (int i = tid; i < mine; i += kThreads) {
    const uint32_t x = keys[i];
    if (x != kNone) rough += W.rough(x), ++nvalid;
  }
  {  // the row's weight in 2^-20 steps, only to choose the scale
    unsigned long long r = (unsigned long long)(rough * 1048576.f) + 1;
    cl.sum(nvalid, r);
    W.shift = 61 - (64 - __clzll((long long)(r + (r >> 8) + (1ull << 12))) - 20);
  }
  // top-k: the largest key that at least k keys reach, and how many of its ties stay
  uint32_t cut = 1;  // the smallest key that stays
  unsigned long long ties = ~0ull;
  if (k > 0 && (unsigned long long)k < nvalid) {
    cut = 0;
    for (uint32_t bit = 0x80000000u; bit; bit >>= 1) {
      const uint32_t c = cut | bit;
      unsigned long long n = 0;
      none = 0;
      for (int i = tid; i < mine; i += kThreads) n += keys[i] >= c;
      cl.sum(n, none);
      if (n >= (unsigned long long)k) cut = c;
    }
    unsigned long long above = 0;
    none = 0;
    for (int i = tid; i < mine; i += kThreads) above += keys[i] > cut;
    cl.sum(above, none);
    ties = (unsigned long long)k - above;
  }
  if (top_p < 1.f) {
    unsigned long long eq = 0, mass = 0;
    for (int i = tid; i < mine; i += kThreads) {
      const uint32_t x = keys[i];
      if (x > cut) mass += W(x);
      eq += x == cut;
    }
    cl.sum(eq, mass);
    const unsigned long long cut_w = W(cut), cut_n = eq < ties ? eq : ties;
    mass += cut_n * cut_w;
    unsigned long long goal = part_of(fmaxf(top_p, 0.f), mass, true);
    goal = goal ? goal : 1ull;
    uint32_t t = 0;
    for (uint32_t bit = 0x80000000u; bit; bit >>= 1) {
      const uint32_t c = t | bit;
      unsigned long long m = 0;
      none = 0;
      for (int i = tid; i < mine; i += kThreads) {
        const uint32_t x = keys[i];
        if (x >= c && x > cut) m += W(x);
      }
      cl.sum(none, m);
      if (c <= cut) m += cut_n * cut_w;
      if (m >= goal) t = c;
    }
    // the first ties of key t that bring the weight above it to the goal
    unsigned long long above = 0;
    none = 0;
    for (int i = tid; i < mine; i += kThreads) {
      const uint32_t x = keys[i];
      if (x > t && x > cut) above += W(x);
    }
    cl.sum(none, above);
    const unsigned long long wt = W(t);
    const unsigned long long need = wt ? (goal - above + wt - 1) / wt : ~0ull;
    ties = t == cut ? (need < ties ? need : ties) : need;
    cut = t;
  }
  unsigned long long least = 0;
  if (min_p > 0.f) least = min_p < 1.f ? part_of(min_p, 1ull << W.shift, true) : 1ull << W.shift;
  // ranks of the ties of the cut in order of id, by warps that hold consecutive ids
  const int ws = slice / kWarps, w0 = wid * ws;
  unsigned long long eq = 0;
  for (int i = lane; i < ws; i += 32) eq += __popc(__ballot_sync(0xffffffffu, keys[w0 + i] == cut));
  unsigned long long rank0, zero, all, zero2;
  cl.scan(eq, 0, rank0, zero, all, zero2);
  unsigned long long mass = 0, cnt = 0, r = rank0;
  for (int i = lane; i < ws; i += 32) {
    const uint32_t x = keys[w0 + i];
    const unsigned tie = __ballot_sync(0xffffffffu, x == cut);
    const unsigned long long my = r + __popc(tie & ((1u << lane) - 1));
    r += __popc(tie);
    if (x > cut || (x == cut && my < ties)) {
      const unsigned long long w = W(x);
      if (w >= least) mass += w, ++cnt;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    mass += __shfl_xor_sync(0xffffffffu, mass, o);
    cnt += __shfl_xor_sync(0xffffffffu, cnt, o);
  }
  unsigned long long mass0, cnt0, total, kept;
  cl.scan(mass, cnt, mass0, cnt0, total, kept);
  const float u = __ldg(a.u + row);
  const unsigned long long goal = u >= 1.f ? total - 1 : u > 0.f ? part_of(u, total, false) : 0ull;
  if (cl.rank == 0 && tid == 0 && a.kept) a.kept[row] = (int)kept;
  if (goal >= mass0 && goal < mass0 + mass) {  // this warp holds the pick
    unsigned long long run = mass0;
    r = rank0;
    for (int i = lane; i < ws; i += 32) {
      const uint32_t x = keys[w0 + i];
      const unsigned tie = __ballot_sync(0xffffffffu, x == cut);
      const unsigned long long my = r + __popc(tie & ((1u << lane) - 1));
      r += __popc(tie);
      unsigned long long w = 0;
      if (x > cut || (x == cut && my < ties)) {
        w = W(x);
        if (w < least) w = 0;
      }
      unsigned long long inc = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long v = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += v;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, run + inc > goal);
      if (hit) {
        if (lane == __ffs(hit) - 1) a.ids[row] = base + w0 + i;
        break;
      }
      run += __shfl_sync(0xffffffffu, inc, 31);
    }
  }
  cl.sync();
}

}  // namespace

using namespace dmtp;

namespace {

template <typename T>
cudaError_t launch(const RowsArgs& s, unsigned cluster, cudaStream_t st) {
  static unsigned long long done = 0;
  auto k = k_sample_rows<T>;
  const int most = (DMTP_OPS_MAX_SAMPLE_VOCAB / 8) * 4;
  if (!smem_limit((const void*)k, most, &done)) return cudaErrorInvalidValue;
  return launch_op(k, (unsigned)s.a.rows * cluster, kThreads, (size_t)s.slice * 4, st, false, cluster, s);
}

}  // namespace

extern "C" int dmtp_sample_rows(const dmtp_sample_args* a, void* stream) {
  if (!a || a->rows < 0) return DMTP_EINVAL;
  if (a->rows == 0) return DMTP_OK;
  if (!a->logits || !a->u || !a->ids || (a->dtype != 0 && a->dtype != 1) || a->vocab < 1 ||
      a->vocab > DMTP_OPS_MAX_SAMPLE_VOCAB || a->ld < a->vocab || a->rows > (1 << 24))
    return DMTP_EINVAL;
  const int es = a->dtype ? 2 : 4;
  if (!aligned_to(a->logits, es)) return DMTP_EINVAL;
  const void* words[] = {a->u, a->temperature, a->top_k, a->top_p, a->min_p, a->ids, a->kept};
  for (const void* p : words)
    if (!aligned_to(p, 4)) return DMTP_EINVAL;
  if (cudaPeekAtLastError() != cudaSuccess) return DMTP_ECUDA;
  RowsArgs s;
  s.a = *a;
  const unsigned cluster = a->vocab > 8192 ? 8 : a->vocab > 2048 ? 2 : 1;
  const int per = (a->vocab + (int)cluster - 1) / (int)cluster;
  s.slice = (per + kThreads - 1) / kThreads * kThreads;
  s.vec = aligned_to(a->logits, 16) && mult(a->ld * es, 16);
  const cudaError_t e = a->dtype ? launch<bf16>(s, cluster, (cudaStream_t)stream)
                                 : launch<float>(s, cluster, (cudaStream_t)stream);
  return e == cudaSuccess ? DMTP_OK : (cudaGetLastError(), DMTP_ECUDA);
}
