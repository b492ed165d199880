// dmtp_paged_write_rope, and E2M1 rows into and out of the pages of a K/V cache.
//
// Write. A group of lanes takes one head of one row, a lane two chunks of eight columns of it: side by
// side, or (PAIR) where rotate-half pairs meet eight of each half of what is rotated. A block of an E2M1
// row is then two neighbours' business; where the half is no whole number of blocks, chunks stay
// side by side and the partners are read once more. The bytes moved are the rows
// once in and once out: 8188 rows of 32 + 2 x 4 heads of 128, half of each rotated, into E4M3 pages
// take 37 us (160 MB, 0.63 of the copy rate; with partners read twice 44), whole heads into bf16 pages 36
// (interleaved 39; k_paged_write, which knows its pairs beforehand, 32), 32 rows 3.8 us, which is
// latency; 4096 rows into E2M1 pages and back 29 us (89 MB in two launches). Issue bounds the many-row
// form, of 4-bit rows two rounded quotients a value.
#include <math.h>
#include <string.h>

#include <cuda_fp16.h>

#include "paged.cuh"
#include "paged_rope.cuh"

using namespace dmtp;

namespace {

struct RopeArgs {
  PageMap m;
  void *k, *v;
  float *ks, *vs;
  dmtp_paged_rows r;
  unsigned* err;
  int lanes, group;  // lanes that hold values; lanes of a group (a power of two >= lanes)
  int rot;           // columns that are rotated
  bool wide, inter;  // rows allow 16-byte accesses; interleaved pairs
  float amp;
};

// A CTA takes ROWS rows (see k_paged_write).
template <typename T, Rows F, int ROWS, bool PAIR>
__global__ void __launch_bounds__(256) k_paged_write_rope(const RopeArgs a, const Turns turns) {
  __shared__ __align__(16) float cs[ROWS][2][DMTP_OPS_MAX_HEAD_DIM / 2];
  __shared__ int s_page[ROWS], s_off[ROWS], s_pos[ROWS];
  const int row0 = blockIdx.x * ROWS, hd = a.m.head_dim, half = a.rot >> 1;
  const int nq = a.r.q ? a.r.n_heads : 0, hkv = a.m.n_kv_heads, items = nq + 2 * hkv;
  const int rows = min(ROWS, a.r.n_rows - row0), all = rows * items;
  const int gl = threadIdx.x & (a.group - 1), ng = blockDim.x / a.group;
  const bool on = gl < a.lanes;
  // a group's loop count is the CTA's: the shuffles below see every lane
  const int step = gridDim.y * ng, mine = threadIdx.x / a.group;
  const bool pair = PAIR && 16 * gl < a.rot;
  const int col[2] = {pair ? 8 * gl : 16 * gl, pair ? half + 8 * gl : 16 * gl + 8};
  Raw<T> x[2], y[2];  // this lane's columns, and their partners
  auto ask = [&](int it) {
    if (on && it < all) {
      const int r = ROWS == 1 ? 0 : it / items, i = it - r * items;
      const int64_t row = row0 + r;
      const T* src = i < nq         ? (const T*)a.r.q + row * a.r.q_row + (int64_t)i * a.r.q_head
                     : i < nq + hkv ? (const T*)a.r.k + row * a.r.k_row + (int64_t)(i - nq) * a.r.k_head
                                    : (const T*)a.r.v + row * a.r.v_row + (int64_t)(i - nq - hkv) * a.r.v_head;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = col[h];
        fetch(src + c, a.wide, x[h]);
        if (!PAIR && !a.inter && c < a.rot && i < nq + hkv) fetch(src + (c < half ? c + half : c - half), a.wide, y[h]);
      }
    }
  };
  ask(blockIdx.y * ng + mine);
  if (threadIdx.x < ROWS) {
    int page = -1, off = 0, pos = 0;
    if ((int)threadIdx.x < rows) {
      const int seq = __ldg(a.r.seq + row0 + threadIdx.x);
      pos = __ldg(a.r.pos + row0 + threadIdx.x);
      if (seq >= a.m.n_seqs)
        set_err(a.err, DMTP_OPS_ERR_SEQ);
      else if (seq >= 0 && (unsigned)pos >= (unsigned)a.m.reach)
        set_err(a.err, DMTP_OPS_ERR_POS);
      else if (seq >= 0)
        page = page_of(a.m, seq, pos, off, a.err);
    }
    s_page[threadIdx.x] = page;
    s_off[threadIdx.x] = off;
    s_pos[threadIdx.x] = pos;
  }
  if (ROWS > 1) __syncthreads();
  for (int i = threadIdx.x; i < rows * half; i += blockDim.x) {
    const int r = ROWS == 1 ? 0 : i / half, h = i - r * half;
    // (of a single row every thread reads the position for itself: no barrier before)
    const int pos = ROWS == 1 ? __ldg(a.r.pos + row0) : s_pos[r];
    const float2 t = cos_sin_turns((unsigned long long)(unsigned)pos * turns.f[h]);
    cs[r][0][h] = t.x * a.amp;
    cs[r][1][h] = t.y * a.amp;
  }
  __syncthreads();
  for (int it0 = blockIdx.y * ng; it0 < all; it0 += step) {
    const int it = it0 + mine;
    float f[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) f[e] = 0.f;
    const int r = ROWS == 1 ? 0 : it / items, i = it - r * items;
    const int page = it < all ? s_page[r] : -1;
    const bool live = on && page >= 0, isq = i < nq, isv = i >= nq + hkv;
    if (pair && live) {
      float v[8], w[8];
      values(x[0], v);
      values(x[1], w);
      if (!isv) {
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          const float4 co = *reinterpret_cast<const float4*>(&cs[r][0][8 * gl + e]);
          const float4 si = *reinterpret_cast<const float4*>(&cs[r][1][8 * gl + e]);
          const float cc[4] = {co.x, co.y, co.z, co.w}, ss[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float p = v[e + j], q = w[e + j];
            v[e + j] = p * cc[j] - q * ss[j];
            w[e + j] = q * cc[j] + p * ss[j];
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        f[e] = v[e];
        f[8 + e] = w[e];
      }
    } else if (live) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = col[h];
        float v[8];
        values(x[h], v);
        if (!pair && c < a.rot && !isv) {
          if (a.inter) {
            const float4 co = *reinterpret_cast<const float4*>(&cs[r][0][c / 2]);
            const float4 si = *reinterpret_cast<const float4*>(&cs[r][1][c / 2]);
            const float cc[4] = {co.x, co.y, co.z, co.w}, ss[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float p = v[2 * j], q = v[2 * j + 1];
              v[2 * j] = p * cc[j] - q * ss[j];
              v[2 * j + 1] = q * cc[j] + p * ss[j];
            }
          } else {
            float w[8];
            values(y[h], w);
            const bool low = c < half;
            const int at = low ? c : c - half;
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
              const float4 co = *reinterpret_cast<const float4*>(&cs[r][0][at + e]);
              const float4 si = *reinterpret_cast<const float4*>(&cs[r][1][at + e]);
              const float cc[4] = {co.x, co.y, co.z, co.w}, ss[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) v[e + j] = v[e + j] * cc[j] + w[e + j] * (low ? -ss[j] : ss[j]);
            }
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) f[8 * h + e] = v[e];
      }
    }
    __syncwarp();  // q_out may be q: no lane writes before its partners have read
    ask(it + step);
    if (live && isq) {
      T* dst = (T*)a.r.q_out + (int64_t)(row0 + r) * a.r.qo_row + (int64_t)i * a.r.qo_head;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = f[8 * h + e];
        store8(dst + col[h], a.wide, v);
      }
    }
    float block[2] = {0.f, 0.f}, amax = 0.f;  // of the blocks that the chunks lie in
    bool odd[2] = {false, false};
    if (F != kRaw) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float m = fabsf(f[e]);
        const bool fine = m <= 3.402823466e38f;
        odd[e / 8] = odd[e / 8] || !fine;
        block[e / 8] = fmaxf(block[e / 8], fine ? m : 0.f);
      }
      amax = fmaxf(block[0], block[1]);
      if (F == kE2M1) {
        const float both = amax;
        const bool any = odd[0] || odd[1];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (PAIR) {  // (every lane takes part)
            const float other = __shfl_xor_sync(0xffffffffu, block[h], 1);
            const bool theirs = __shfl_xor_sync(0xffffffffu, (int)odd[h], 1);
            block[h] = pair ? fmaxf(block[h], other) : both;
            odd[h] = pair ? odd[h] || theirs : any;
          } else {
            block[h] = both;
            odd[h] = any;
          }
        }
      }
      for (int o = a.group >> 1; o > 0; o >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    }
    if (live && !isq) {
      const int64_t line = (int64_t)(i - nq - (isv ? hkv : 0)) * a.m.page_size + s_off[r];
      const int64_t at = (int64_t)page * a.m.page_stride;
      if (F == kE2M1) {
        const int e = e2m1_exponent(amax);
        const float inv = pow2f(-e);
        uint8_t* pg = (uint8_t*)(isv ? a.v : a.k) + at;
        uint32_t b[2], w[2] = {0u, 0u};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h && !pair) {
            b[1] = b[0];
          } else {
            b[h] = e4m3_byte(__fdiv_rn(block[h] * inv, 6.f));
            if (odd[h]) b[h] = 0x7fu;
          }
          const float bf = h2_to_f2(e4m3x2_to_h2(b[h])).x;
          if (bf > 0.f) {  // (no NaN)
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __fdiv_rn(f[8 * h + j] * inv, bf);
            w[h] = e2m1x8(v);
          }
        }
        if (pair) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            *reinterpret_cast<uint32_t*>(pg + line * (hd / 2) + col[h] / 2) = w[h];
            if (gl % 2 == 0) pg[e2m1_blocks(a.m) + line * (hd / 16) + col[h] / 16] = (uint8_t)b[h];
          }
        } else {
          *reinterpret_cast<uint2*>(pg + line * (hd / 2) + 8 * gl) = make_uint2(w[0], w[1]);
          pg[e2m1_blocks(a.m) + line * (hd / 16) + gl] = (uint8_t)b[0];
        }
        if (gl == 0) (isv ? a.vs : a.ks)[(int64_t)page * a.m.scale_stride + line] = pow2f(e);
      } else if (F == kE4M3) {
        const int e = e4m3_exponent(amax);
        const float inv = pow2f(-e);  // |e| <= 126: a normal number, the scaling is exact
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[j] = e4m3_row4(make_float4(f[4 * j] * inv, f[4 * j + 1] * inv, f[4 * j + 2] * inv, f[4 * j + 3] * inv));
        uint8_t* dst = (uint8_t*)(isv ? a.v : a.k) + at + line * hd;
        *reinterpret_cast<uint2*>(dst + col[0]) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2*>(dst + col[1]) = make_uint2(w[2], w[3]);
        if (gl == 0) (isv ? a.vs : a.ks)[(int64_t)page * a.m.scale_stride + line] = pow2f(e);
      } else {
        T* dst = (T*)(isv ? a.v : a.k) + at + line * hd;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = f[8 * h + e];
          store8(dst + col[h], true, v);
        }
      }
    }
  }
}

struct ReadArgs {
  PageMap m;
  const uint8_t *k, *v;
  const float *ks, *vs;
  const int32_t *seq, *pos;
  void *ko, *vo;
  int n_rows, lanes, group;
  unsigned* err;
};

// A group of lanes copies kHeads heads of one row, a block of 16 columns a lane and head (see
// k_paged_read).
constexpr int kHeads = 4;
template <typename T>
__global__ void __launch_bounds__(256) k_paged_read_e2m1(const ReadArgs a) {
  const int hd = a.m.head_dim, hkv = a.m.n_kv_heads;
  const int gl = threadIdx.x & (a.group - 1), ng = blockDim.x / a.group;
  const int64_t row = (int64_t)blockIdx.x * ng + threadIdx.x / a.group;
  const int h0 = blockIdx.y * kHeads;  // of the k and v heads
  if (gl >= a.lanes || row >= a.n_rows) return;
  const int seq = __ldg(a.seq + row), pos = __ldg(a.pos + row);
  if (seq < 0) return;
  if (seq >= a.m.n_seqs || (unsigned)pos >= (unsigned)a.m.reach) {
    if (gl == 0) set_err(a.err, seq >= a.m.n_seqs ? DMTP_OPS_ERR_SEQ : DMTP_OPS_ERR_POS);
    return;
  }
  int off;
  const int page = page_of(a.m, seq, pos, off, gl == 0 ? a.err : nullptr);
  if (page < 0) return;
  uint2 u[kHeads];
  uint32_t b[kHeads];
  float s[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int h2 = h0 + i;
    if (h2 < 2 * hkv) {
      const bool isv = h2 >= hkv;
      const int64_t line = (int64_t)(isv ? h2 - hkv : h2) * a.m.page_size + off;
      const uint8_t* pg = (isv ? a.v : a.k) + (int64_t)page * a.m.page_stride;
      u[i] = __ldcs(reinterpret_cast<const uint2*>(pg + line * (hd / 2) + 8 * gl));
      b[i] = __ldg(pg + e2m1_blocks(a.m) + line * (hd / 16) + gl);
      s[i] = __ldg((isv ? a.vs : a.ks) + (int64_t)page * a.m.scale_stride + line);
    }
  }
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int h2 = h0 + i;
    if (h2 < 2 * hkv) {
      const bool isv = h2 >= hkv;
      T* dst = (T*)(isv ? a.vo : a.ko) + (row * hkv + (isv ? h2 - hkv : h2)) * hd + 16 * gl;
      const float bf = h2_to_f2(e4m3x2_to_h2(b[i])).x;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float f[8];
        e2m1x8_to_f8(h ? u[i].y : u[i].x, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = f[e] * bf * s[i];
        store8(dst + 8 * h, true, f);
      }
    }
  }
}

int group_of(int lanes) {
  int g = 1;
  while (g < lanes) g <<= 1;
  return g;
}
bool row_ok(const void* p, int64_t row, int64_t head, int es, int hd, int heads) {
  return p && aligned_to(p, 4 * es) && mult(row, 4) && mult(head, 4) && head >= hd && row >= 0 &&
         heads >= 1;
}
bool finite(double x) { return x - x == 0.0; }
int check_rope(const dmtp_rope& p, int hd) {
  if (p.dims < 16 || p.dims > hd || p.dims % 16 || (p.interleaved != 0 && p.interleaved != 1)) return DMTP_EINVAL;
  if (p.scaling < DMTP_ROPE_PLAIN || p.scaling > DMTP_ROPE_RAMP) return DMTP_EINVAL;
  // theta, factor >= 1: every pair's rate is at most one radian per position, below one turn
  if (!(p.theta >= 1.0 && finite(p.theta) && finite(p.amplitude))) return DMTP_EINVAL;
  if (p.scaling != DMTP_ROPE_PLAIN && !(p.factor >= 1.0 && finite(p.factor))) return DMTP_EINVAL;
  if (p.scaling == DMTP_ROPE_TURNS || p.scaling == DMTP_ROPE_RAMP) {
    if (!(p.low > 0.0 && p.high > p.low && finite(p.high) && p.orig_len > 0.0 && finite(p.orig_len))) return DMTP_EINVAL;
    if (p.scaling == DMTP_ROPE_RAMP && !(p.theta > 1.0)) return DMTP_EINVAL;
  }
  return DMTP_OK;
}
// f_i / (2 pi) * 2^64 of a head's pairs; a thread that keeps calling with one rotation forms them
// once.
const Turns& turns_of(const dmtp_rope& p) {
  static thread_local Turns t;
  static thread_local dmtp_rope last = {};
  if (memcmp(&p, &last, sizeof p)) {
    const double two_pi = 6.283185307179586477;
    double lo = 0, hi = 0;
    if (p.scaling == DMTP_ROPE_RAMP) {
      const double per = p.dims / (2.0 * log(p.theta));
      lo = fmin(fmax(floor(per * log(p.orig_len / (two_pi * p.high))), 0.0), p.dims - 1.0);
      hi = fmin(fmax(ceil(per * log(p.orig_len / (two_pi * p.low))), 0.0), p.dims - 1.0);
    }
    for (int i = 0; i < p.dims / 2; ++i) {
      const double g = pow(p.theta, -2.0 * i / p.dims);
      double f = g;
      if (p.scaling == DMTP_ROPE_LINEAR) f = g / p.factor;
      if (p.scaling == DMTP_ROPE_TURNS || p.scaling == DMTP_ROPE_RAMP) {
        const double w = p.scaling == DMTP_ROPE_TURNS
                             ? fmin(fmax((p.orig_len * g / two_pi - p.low) / (p.high - p.low), 0.0), 1.0)
                             : 1.0 - fmin(fmax((i - lo) / fmax(hi - lo, 0.001), 0.0), 1.0);
        f = w * g + (1.0 - w) * (g / p.factor);
      }
      t.f[i] = (unsigned long long)ldexp(f * 0.15915494309189533577, 64);
    }
    last = p;
  }
  return t;
}

template <typename T, bool PAIR>
auto write_kernel(Rows f, bool few) {
  return few ? (f == kE2M1   ? k_paged_write_rope<T, kE2M1, 1, PAIR>
                : f == kE4M3 ? k_paged_write_rope<T, kE4M3, 1, PAIR>
                             : k_paged_write_rope<T, kRaw, 1, PAIR>)
             : (f == kE2M1   ? k_paged_write_rope<T, kE2M1, 4, PAIR>
                : f == kE4M3 ? k_paged_write_rope<T, kE4M3, 4, PAIR>
                             : k_paged_write_rope<T, kRaw, 4, PAIR>);
}

}  // namespace

extern "C" int dmtp_paged_write_rope(const dmtp_paged_kv* c, const dmtp_paged_rows* r, const dmtp_rope* rope,
                                     uint32_t* err, void* stream) {
  int e = check_cache(c);
  if (e) return e;
  if (!r || r->n_rows < 0) return DMTP_EINVAL;
  const int es = c->dtype ? 2 : 4, hd = c->head_dim;
  dmtp_rope p = {};
  if (rope) {
    p = *rope;
    if (r->rope_theta != 0.f) return DMTP_EINVAL;
    const int bad = check_rope(p, hd);
    if (bad) return bad;
  } else {
    if (c->e4m3 != DMTP_OPS_E2M1) return dmtp_paged_write(c, r, err, stream);
    if (!(r->rope_theta == 0.f || (r->rope_theta >= 1.f && r->rope_theta <= 3.4e38f))) return DMTP_EINVAL;
    p.theta = r->rope_theta;
    p.dims = r->rope_theta > 0.f ? hd : 0;
    p.amplitude = 1.f;
  }
  if (r->n_rows == 0) return DMTP_OK;
  if (!row_ok(r->k, r->k_row, r->k_head, es, hd, 1) || !row_ok(r->v, r->v_row, r->v_head, es, hd, 1) ||
      !r->seq || !r->pos || !aligned_to(r->seq, 4) || !aligned_to(r->pos, 4))
    return DMTP_EINVAL;
  if (r->q && (r->n_heads < 1 || r->n_heads > 4096 ||
               !row_ok(r->q, r->q_row, r->q_head, es, hd, r->n_heads) ||
               !row_ok(r->q_out, r->qo_row, r->qo_head, es, hd, r->n_heads) ||
               (r->n_rows > 1 && r->qo_row < hd)))  // rows of one address
    return DMTP_EINVAL;
  if (err && !aligned_to(err, 4)) return DMTP_EINVAL;
  if (cudaPeekAtLastError() != cudaSuccess) return DMTP_ECUDA;
  RopeArgs a;
  a.m = page_map(*c);
  a.k = c->k;
  a.v = c->v;
  a.ks = c->k_scale;
  a.vs = c->v_scale;
  a.r = *r;
  a.err = err;
  a.lanes = hd / 16;
  a.group = group_of(a.lanes);
  a.rot = p.dims;
  a.inter = p.interleaved != 0;
  a.amp = p.amplitude;
  a.wide = true;
  const int64_t strides[] = {r->k_row, r->k_head, r->v_row, r->v_head,
                             r->q ? r->q_row : 0, r->q ? r->q_head : 0, r->q ? r->qo_row : 0, r->q ? r->qo_head : 0};
  for (int64_t x : strides) a.wide = a.wide && mult(x * es, 16);
  for (const void* x : {r->k, r->v, r->q, (const void*)r->q_out}) a.wide = a.wide && aligned_to(x, 16);
  // (as dmtp_paged_write)
  const int items = (r->q ? r->n_heads : 0) + 2 * c->n_kv_heads, ng = 256 / a.group;
  const int blocks = (items + ng - 1) / ng;
  const bool few = (int64_t)r->n_rows * blocks <= 608;
  const int quads = (r->n_rows - 1) / 4 + 1, spread = quads < 608 ? 608 / quads : 1, rounds = (4 * items + ng - 1) / ng;
  const dim3 grid(few ? r->n_rows : quads, few ? blocks : spread < rounds ? spread : rounds);
  static const Turns none = {};
  const Turns& t = p.dims ? turns_of(p) : none;
  const bool pair = a.rot && !a.inter && (c->e4m3 != DMTP_OPS_E2M1 || a.rot % 32 == 0);
  auto k = c->dtype ? (pair ? write_kernel<bf16, true>(rows_of(*c), few) : write_kernel<bf16, false>(rows_of(*c), few))
                    : (pair ? write_kernel<float, true>(rows_of(*c), few) : write_kernel<float, false>(rows_of(*c), few));
  return launch_op(k, grid, 256, 0, (cudaStream_t)stream, false, 1, a, t) == cudaSuccess
             ? DMTP_OK
             : (cudaGetLastError(), DMTP_ECUDA);
}

namespace dmtp {

cudaError_t read_e2m1(const dmtp_paged_kv* c, const int32_t* seq, const int32_t* pos, int n_rows, void* k_out,
                      void* v_out, uint32_t* err, cudaStream_t st) {
  ReadArgs a;
  a.m = page_map(*c);
  a.k = (const uint8_t*)c->k;
  a.v = (const uint8_t*)c->v;
  a.ks = c->k_scale;
  a.vs = c->v_scale;
  a.seq = seq;
  a.pos = pos;
  a.ko = k_out;
  a.vo = v_out;
  a.n_rows = n_rows;
  a.lanes = c->head_dim / 16;
  a.group = group_of(a.lanes);
  a.err = err;
  const int ng = 256 / a.group, heads = (2 * c->n_kv_heads + kHeads - 1) / kHeads;
  const dim3 grid((unsigned)((n_rows + (int64_t)ng - 1) / ng), heads);
  return launch_op(c->dtype ? k_paged_read_e2m1<bf16> : k_paged_read_e2m1<float>, grid, 256, 0, st, false, 1, a);
}

}  // namespace dmtp
