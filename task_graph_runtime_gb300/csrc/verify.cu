// Verification of drafted tokens against the model's logits with given
// random numbers (mpk_verify_drafts).
//
// With p = softmax(logits / T) after row i and q what draft i + 1 was drawn
// from, draft d is accepted when u q(d) < p(d); the first refused one is
// replaced by a sample of max(p - q, 0) (normalised), and when all are
// accepted one token more is sampled from the last row's p: the tokens are
// distributed as samples of p alone.  A sample of weights w is
// argmax_v w_v / e_v with the given e_v ~ Exp(1): P(v wins) = w_v / sum w,
// so w needs no normalisation and no running sum over the vocabulary, and
// the answer does not depend on the order of one (an inverse CDF's does).
//
// verify_stats: maximum and sum of exponentials of every row and the drafted
// token's logit; greedy rows (T <= 0) the index of the maximum.  A row is cut
// into slices so that few rows still fill the GPU (joining them in a cluster
// of CTAs took half as long again as leaving them to the second pass).
// verify_sample: every CTA of a sequence joins its rows' slices (a warp a
// row; in fp32: the FP64 units are few, and 64-bit sums here cost 10 us a
// launch), finds the first refused draft and races its slice of that one row;
// slices meet in one 64-bit atomic maximum of
// (value, lowest index), whose result does not depend on their order.  Most
// values of a slice cannot win: bounds from fast functions decide that, and
// only the few above a warp's best lower bound are worked out exactly.
// Bound by HBM: each row of logits leaves it once, the row that is sampled
// from once more with its draft and noise rows.  Measured: 64 sequences of 5
// rows of 151936, 48 us for the first pass (5.1 TB/s) and 21 for the second;
// one sequence of 4 rows of 32000 9.2 us, all latency.
#include <cmath>

#include "serve_dev.cuh"

namespace mpk {
namespace {

// A row of logits, its slices joined.
struct VerifyRow {
  float z;                     // sum of e^((x - m) / T)
  float m;                     // maximum
  int best;                    // its lowest index (greedy rows), or -1
};

constexpr int kNT = 256;
constexpr int kMaxOut = 128;     // rows of a sequence
// log2(e) rounded to fp32, and the rest of it
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLog2eLow = (float)(1.4426950408889634074 - (double)kLog2e);

__device__ __forceinline__ float ex2a(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// NaN logits count as -inf: they can be neither accepted nor sampled.
__device__ __forceinline__ float clean(float x) { return fmaxf(x, -INFINITY); }

// (m, z) joined with (m2, z2); equal maxima (infinite ones too) add up.
__device__ __forceinline__ void join(float& m, float& z, float m2, float z2,
                                     float c) {
  const float M = fmaxf(m, m2);
  z = z * (m == M ? 1.f : ex2a((m - M) * c)) +
      z2 * (m2 == M ? 1.f : ex2a((m2 - M) * c));
  m = M;
}

struct RowInfo {
  int b, first, n;     // sequence, its first row, its rows
};
__device__ __forceinline__ RowInfo rows_of(const VerifyArgs& a, int b) {
  RowInfo r;
  r.b = b;
  r.first = sv_row(a.q_start, a.tokens_per_seq, a.n_tokens, b);
  r.n = max(sv_row(a.q_start, a.tokens_per_seq, a.n_tokens, b + 1) - r.first,
            0);
  return r;
}

// T of sequence b: 0 or less (or NaN) is greedy.  Others are kept where
// log2(e) / T is neither 0 nor infinite, whose products with an infinite or
// zero difference of logits would be NaN.
__device__ __forceinline__ float temperature(const VerifyArgs& a, int b) {
  const float T = a.temperature ? __ldg(a.temperature + b) : 1.f;
  return T > 0.f ? fminf(fmaxf(T, 1e-30f), 1e30f) : T;
}

__global__ void __launch_bounds__(kNT, 5)
    verify_stats(const __grid_constant__ VerifyArgs a) {
  sv_grid_wait();
  sv_grid_launch();
  const int tid = threadIdx.x;
  {
    // the words of the second pass start at zero
    const int64_t i =
        ((int64_t)(blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x +
         blockIdx.x) * kNT + tid;
    const int64_t all = (int64_t)gridDim.x * gridDim.y * gridDim.z * kNT;
    for (int64_t b = i; b < a.batch; b += all) {
      a.race[b] = 0ull;
      a.arrived[b] = 0u;
    }
  }
  const int row = blockIdx.y;
  if (row >= a.n_tokens) return;
  const float* x = blockIdx.z ? a.draft + row * a.draft_stride
                              : a.logits + row * a.logits_stride;
  // vectors of four on 16-byte boundaries: vector v holds values
  // [4 v - o, 4 v - o + 4)
  const int o = (int)(((uintptr_t)x >> 2) & 3);
  const int nv = (a.vocab + o + 3) / 4;
  const int v0 = (int)((int64_t)nv * blockIdx.x / gridDim.x);
  const int v1 = (int)((int64_t)nv * (blockIdx.x + 1) / gridDim.x);
  constexpr int U = 4;
  float4 w[U], next[U];
  auto fetch = [&](int v, float4 (&w)[U]) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int vi = v + i * kNT, k = 4 * vi - o;
      w[i] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (vi >= v1) continue;
      if (k >= 0 && k + 4 <= a.vocab) {
        w[i] = __ldg(reinterpret_cast<const float4*>(x + k));
      } else {
        if (k >= 0) w[i].x = x[k];
        if (k + 1 >= 0 && k + 1 < a.vocab) w[i].y = x[k + 1];
        if (k + 2 >= 0 && k + 2 < a.vocab) w[i].z = x[k + 2];
        if (k + 3 < a.vocab) w[i].w = x[k + 3];
      }
    }
  };
  fetch(v0 + tid, w);  // on the way while the sequence is looked up
  const int b = sv_seq_of_warp(a.q_start, a.tokens_per_seq, a.batch, row);
  if (b < 0) return;
  const float T = temperature(a, b);
  const bool greedy = !(T > 0.f);
  const RowInfo ri = rows_of(a, b);
  const bool judges = row < ri.first + ri.n - 1;   // a draft comes after it
  // drafts' rows: none after the last draft, and a greedy sequence does not
  // ask for their distribution
  if (blockIdx.z == 1 && (!judges || greedy)) return;
  const float c = greedy ? 1.f : kLog2e / T;
  float m = -INFINITY, z = 0.f;
  int best = 0x7fffffff;
  for (int v = v0 + tid; v < v1; v += U * kNT) {
    if (v != v0 + tid)
#pragma unroll
      for (int i = 0; i < U; ++i) w[i] = next[i];
    fetch(v + U * kNT, next);
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      w[i].x = clean(w[i].x);
      w[i].y = clean(w[i].y);
      w[i].z = clean(w[i].z);
      w[i].w = clean(w[i].w);
      top = fmaxf(top, fmaxf(fmaxf(w[i].x, w[i].y), fmaxf(w[i].z, w[i].w)));
    }
    if (greedy) {
      if (top > m) {
        m = top;
        // the lowest index that holds the maximum
#pragma unroll
        for (int i = U - 1; i >= 0; --i) {
          const int k = 4 * (v + i * kNT) - o;
          if (w[i].w == top) best = k + 3;
          if (w[i].z == top) best = k + 2;
          if (w[i].y == top) best = k + 1;
          if (w[i].x == top) best = k;
        }
      }
      continue;
    }
    if (top > m) {
      z = m == -INFINITY ? 0.f : z * ex2a((m - top) * c);
      m = top;
    }
    if (m == -INFINITY) continue;
    if (m == INFINITY) {
#pragma unroll
      for (int i = 0; i < U; ++i)
        z += (float)((w[i].x == m) + (w[i].y == m) + (w[i].z == m) +
                     (w[i].w == m));
      continue;
    }
#pragma unroll
    for (int i = 0; i < U; ++i)
      z += (ex2a((w[i].x - m) * c) + ex2a((w[i].y - m) * c)) +
           (ex2a((w[i].z - m) * c) + ex2a((w[i].w - m) * c));
  }
  __shared__ float sm[kNT / 32], sz[kNT / 32];
  __shared__ int sb[kNT / 32];
  auto fold = [&](float m2, float z2, int b2) {
    if (greedy) {
      if (m2 > m || (m2 == m && b2 < best)) {
        m = m2;
        best = b2;
      }
    } else {
      join(m, z, m2, z2, c);
    }
  };
#pragma unroll
  for (int s = 16; s > 0; s >>= 1)
    fold(__shfl_xor_sync(0xffffffffu, m, s), __shfl_xor_sync(0xffffffffu, z, s),
         __shfl_xor_sync(0xffffffffu, best, s));
  if ((tid & 31) == 0) {
    sm[tid >> 5] = m;
    sz[tid >> 5] = z;
    sb[tid >> 5] = best;
  }
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kNT / 32; ++w) fold(sm[w], sz[w], sb[w]);
    const int64_t at =
        ((int64_t)blockIdx.z * a.n_tokens + row) * gridDim.x + blockIdx.x;
    a.part[at] = make_float4(m, z, __int_as_float(best), 0.f);
  }
}

// e^((x - m) / T) with c = log2(e) / T as ch + cl.  The difference keeps its
// rounding error (d + e = x - m exactly), the exponent is split into a whole
// and a fraction f in [-1/2, 1/2], and 2^f is its power series to the 7th
// term (the next is below 6e-9): the result is good to about 1e-7 of itself
// for any x, where one product in 32 bits would lose 2^-24 of an exponent as
// large as 40.  Two candidates of a race that lie closer than that have equal
// chances in all but name.
__device__ __forceinline__ float weight(float x, float m, float ch, float cl) {
  if (x == m) return 1.f;
  const float d = x - m;
  if (!(d * ch > -126.f)) return 0.f;
  const float t = d - x;
  const float e = (x - (d - t)) - (m + t);
  const float n = rintf(d * ch);
  float f = fmaf(d, ch, -n);
  f = fmaf(d, cl, f);
  f = fmaf(e, ch, f);
  float y = 1.5252733804e-5f;
  y = fmaf(y, f, 1.5403530394e-4f);
  y = fmaf(y, f, 1.3333558146e-3f);
  y = fmaf(y, f, 9.6181291076e-3f);
  y = fmaf(y, f, 5.5504108665e-2f);
  y = fmaf(y, f, 2.4022650696e-1f);
  y = fmaf(y, f, 6.9314718056e-1f);
  y = fmaf(y, f, 1.0f);
  return y * __int_as_float(((int)n + 127) << 23);
}

__device__ __forceinline__ unsigned long long race_key(float v, int i) {
  return ((unsigned long long)__float_as_uint(v) << 32) |
         (0xffffffffu - (uint32_t)i);
}

// Bounds of the weights leave room for fast functions: an exponent off by
// 126 x 2^-22 at most, ex2 and a reciprocal good to 2^-22.
constexpr float kUp = 1.f + 0x1p-14f, kDown = 1.f - 0x1p-14f;

// What a slice needs to know of the row that is sampled from.
struct Race {
  const float *x, *y, *e;      // logits, draft (or null), noise
  float m, iz, mq, izq;        // the rows' maxima and reciprocal sums
  float ch, cl;                // log2(e) / T in two parts
  int skip;                    // token whose weight is 0 (or -1)
  bool dlog;
};
__device__ __forceinline__ unsigned long long race_exact(const Race& r, int v,
                                                         bool residual) {
  const float p = weight(clean(r.x[v]), r.m, r.ch, r.cl) * r.iz;
  float w = p;
  if (residual && r.y) {
    const float y = r.y[v];
    w = p - (!r.dlog ? y
             : r.mq == -INFINITY
                 ? 0.f
                 : weight(clean(y), r.mq, r.ch, r.cl) * r.izq);
  } else if (residual && v == r.skip) {
    w = 0.f;
  }
  const float s = w / r.e[v];
  return w > 0.f && s >= 0.f ? race_key(s, v) : 0ull;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// e^((x - m) / T) roughly (1 where x is m, which may be infinite)
__device__ __forceinline__ float rough(float x, float m, float c) {
  return x == m ? 1.f : ex2a((x - m) * c);
}

// The whole row, weight p alone: for a residual that is nowhere positive (p
// and q agree to the last bit), a rare case left to one CTA.
__device__ __noinline__ unsigned long long race_plain(const Race& r,
                                                      int vocab) {
  __shared__ unsigned long long s_k[kNT / 32];
  unsigned long long k = 0;
  for (int v = threadIdx.x; v < vocab; v += kNT)
    k = max(k, race_exact(r, v, false));
#pragma unroll
  for (int s = 16; s > 0; s >>= 1)
    k = max(k, __shfl_xor_sync(0xffffffffu, k, s));
  if ((threadIdx.x & 31) == 0) s_k[threadIdx.x >> 5] = k;
  __syncthreads();
  for (int w = 0; w < kNT / 32; ++w) k = max(k, s_k[w]);
  return k;
}

// KIND: 0 weights p, 1 p - q with probabilities q, 2 p - q with logits q,
// 3 p without one token.  VEC: the rows lie on the same 16-byte phase.
template <int KIND, bool VEC>
__device__ __forceinline__ unsigned long long race_slice(const Race& r,
                                                         int vocab,
                                                         int* s_floor) {
  const int tid = threadIdx.x;
  constexpr bool Q = KIND == 1 || KIND == 2;
  constexpr int U = 4;                 // vectors of four a turn
  const int o = VEC ? (int)(((uintptr_t)r.x >> 2) & 3) : 0;
  const int nv = (vocab + o + 3) / 4;
  const int v0 = (int)((int64_t)nv * blockIdx.x / gridDim.x);
  const int v1 = (int)((int64_t)nv * (blockIdx.x + 1) / gridDim.x);
  unsigned long long best = 0ull;
  float floor_ = 0.f;                  // the best is at least this
  // (as bits: positive floats order as whole numbers)
  for (int v = v0; v < v1; v += U * kNT) {
    floor_ = fmaxf(floor_, __int_as_float(*(volatile int*)s_floor));
    float up[4 * U];
    float low = 0.f;
    // value j of vector i: 4 (v + i kNT + tid) - o + j, or without a common
    // phase 4 (v + i kNT) + j kNT + tid, in either case this thread's own
    float x[4 * U], y[4 * U], e[4 * U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int vi = v + i * kNT + tid, k = 4 * vi - o;
      if (VEC && vi < v1 && k >= 0 && k + 4 <= vocab) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(r.x + k));
        const float4 b = __ldcs(reinterpret_cast<const float4*>(r.e + k));
        x[4 * i] = a.x; x[4 * i + 1] = a.y; x[4 * i + 2] = a.z; x[4 * i + 3] = a.w;
        e[4 * i] = b.x; e[4 * i + 1] = b.y; e[4 * i + 2] = b.z; e[4 * i + 3] = b.w;
        if (Q) {
          const float4 q = __ldg(reinterpret_cast<const float4*>(r.y + k));
          y[4 * i] = q.x; y[4 * i + 1] = q.y; y[4 * i + 2] = q.z; y[4 * i + 3] = q.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int q = VEC ? k + j : 4 * (v + i * kNT) + j * kNT + tid;
          const bool in = VEC ? vi < v1 && q >= 0 && q < vocab
                              : q < min(4 * v1, vocab);
          x[4 * i + j] = in ? __ldg(r.x + q) : -INFINITY;
          e[4 * i + j] = in ? __ldcs(r.e + q) : 1.f;
          if (Q) y[4 * i + j] = in ? __ldg(r.y + q) : 0.f;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4 * U; ++i) {
      const float p = rough(clean(x[i]), r.m, r.ch) * r.iz;
      const float t = rcp(e[i]);
      float a = p * kUp, b = p * kDown;
      if (Q) {
        const float q = KIND == 1 ? y[i]
                                  : rough(clean(y[i]), r.mq, r.ch) * r.izq;
        a = fmaf(q, -kDown, a);
        b = fmaf(q, -kUp, b);
      }
      if (KIND == 3) {
        const int k = VEC ? 4 * (v + (i / 4) * kNT + tid) - o + i % 4
                          : 4 * (v + (i / 4) * kNT) + (i % 4) * kNT + tid;
        if (k == r.skip) a = b = 0.f;
      }
      // (a NaN compares false below and bounds nothing)
      up[i] = a * t * kUp;
      low = fmaxf(low, b * t * kDown);
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1)
      low = fmaxf(low, __shfl_xor_sync(0xffffffffu, low, s));
    // (an infinite one comes from noise below the smallest normal number,
    // which the fast reciprocal takes for 0: no bound)
    if (low > floor_ && low < INFINITY) {
      // the other warps have less to work out next turn
      floor_ = low;
      if ((tid & 31) == 0) atomicMax(s_floor, __float_as_int(low));
    }
    uint32_t mask = 0;
#pragma unroll
    for (int i = 0; i < 4 * U; ++i)
      if (up[i] > 0.f && up[i] >= floor_) mask |= 1u << i;
    while (mask) {
      const int i = __ffs(mask) - 1;
      mask &= mask - 1;
      const int k = VEC ? 4 * (v + (i / 4) * kNT + tid) - o + i % 4
                        : 4 * (v + (i / 4) * kNT) + (i % 4) * kNT + tid;
      best = max(best, race_exact(r, k, KIND != 0));
    }
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1)
    best = max(best, __shfl_xor_sync(0xffffffffu, best, s));
  return best;
}

__global__ void __launch_bounds__(kNT)
    verify_sample(const __grid_constant__ VerifyArgs a) {
  __shared__ VerifyRow s_row[2][kMaxOut];
  __shared__ int s_stop;       // first draft that is not accepted
  __shared__ int s_last;
  __shared__ int s_floor;      // a lower bound of the slice's best, as bits
  const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
  // (verify_stats has waited for what comes before it)
  RowInfo r = rows_of(a, b);
  const float T = temperature(a, b);
  if (r.n > a.max_out) {
    if (tid == 0) sv_latch(a.status, MPK_ERR_INVALID_ARG);
    r.n = a.max_out;
  }
  const bool greedy = !(T > 0.f);
  const float c = greedy ? 1.f : kLog2e / T;
  const bool dlog = a.draft && a.draft_is_logits;
  // log2(e) / T in two parts
  const float ch = greedy ? 1.f : kLog2e / T;
  const float cl = greedy ? 0.f : (fmaf(-ch, T, kLog2e) + kLog2eLow) / T;
  if (tid == 0) {
    s_stop = r.n - 1;
    s_floor = 0;
  }
  // The slice's noise does not depend on the verdicts: into the L2 while the
  // first pass drains.
  if (!greedy) {
    const float* e = a.noise + b * a.noise_stride;
    const int e0 = (int)((int64_t)a.vocab * blockIdx.x / gridDim.x);
    const int e1 = (int)((int64_t)a.vocab * (blockIdx.x + 1) / gridDim.x);
    for (int k = e0 + 32 * tid; k < e1; k += 32 * kNT)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(e + k));
  }
  // the rows' slices, a warp a row; lane 0 has what judges the draft ready
  bool waited = false;
  for (int i = tid >> 5; i < r.n; i += kNT / 32) {
    const int row = r.first + i;
    const int d = i < r.n - 1 ? a.tokens[row + 1] : -1;
    const bool have = d >= 0 && d < a.vocab;
    float xd = 0.f, yd = 1.f, u = 0.f;
    if (have && !greedy) {
      xd = clean(a.logits[row * a.logits_stride + d]);
      if (a.draft) yd = a.draft[row * a.draft_stride + d];
      u = a.uniform[row];
    }
    if (!waited) sv_grid_wait();
    waited = true;
    float pq[2] = {0.f, yd};             // of the drafted token
    int best = -1;
    for (int k = 0; k < (dlog && !greedy && i < r.n - 1 ? 2 : 1); ++k) {
      const float4* part =
          a.part + ((int64_t)k * a.n_tokens + row) * a.slices;
      float m = -INFINITY;
      int bi = 0x7fffffff;
      for (int s = lane; s < a.slices; s += 32) {
        const float4 v = part[s];
        if (v.x > m) bi = __float_as_int(v.z);
        m = fmaxf(m, v.x);
      }
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, s);
        const int b2 = __shfl_xor_sync(0xffffffffu, bi, s);
        if (m2 > m || (m2 == m && b2 < bi)) bi = b2;
        m = fmaxf(m, m2);
      }
      float z = 0.f;
      for (int s = lane; s < a.slices; s += 32) {
        const float4 v = part[s];
        z += v.y * (v.x == m ? 1.f : ex2a((v.x - m) * c));
      }
#pragma unroll
      for (int s = 16; s > 0; s >>= 1)
        z += __shfl_xor_sync(0xffffffffu, z, s);
      if (k == 0) best = m == -INFINITY ? -1 : bi;
      if (lane == 0) {
        s_row[k][i].z = z;
        s_row[k][i].m = m;
        s_row[k][i].best = best;
        if (have && !greedy)
          pq[k] = m == -INFINITY ? 0.f
                                 : weight(k ? clean(yd) : xd, m, ch, cl) / z;
      }
    }
    if (lane == 0 && i < r.n - 1) {
      const bool ok = have && (greedy ? best == d : u * pq[1] < pq[0]);
      if (!ok) atomicMin(&s_stop, i);
    }
  }
  if (!waited) sv_grid_wait();
  __syncthreads();
  const int n_acc = max(s_stop, 0);
  const int row = r.first + n_acc;
  const int refused = n_acc < r.n - 1 ? a.tokens[row + 1] : -1;
  const bool residual = refused >= 0 && refused < a.vocab;
  // ---- this slice of the race
  Race g;
  if (r.n > 0 && !greedy) {
    const VerifyRow w = s_row[0][n_acc];
    g.x = a.logits + row * a.logits_stride;
    g.e = a.noise + b * a.noise_stride;
    g.y = residual && a.draft ? a.draft + row * a.draft_stride : nullptr;
    g.m = w.m;
    g.iz = 1.f / w.z;
    g.ch = ch;
    g.cl = cl;
    g.skip = residual && !a.draft ? refused : -1;
    g.dlog = dlog;
    g.mq = g.izq = 0.f;
    if (g.y && dlog) {
      const VerifyRow y = s_row[1][n_acc];
      g.mq = y.m;
      g.izq = y.m == -INFINITY ? 0.f : 1.f / y.z;
    }
    unsigned long long best = 0ull;
    if (g.m > -INFINITY) {
      const unsigned o = ((uintptr_t)g.x >> 2) & 3;
      const bool same = (((uintptr_t)g.e >> 2) & 3) == o &&
                        (!g.y || (((uintptr_t)g.y >> 2) & 3) == o);
      if (g.y && dlog)
        best = same ? race_slice<2, true>(g, a.vocab, &s_floor)
                    : race_slice<2, false>(g, a.vocab, &s_floor);
      else if (g.y)
        best = same ? race_slice<1, true>(g, a.vocab, &s_floor)
                    : race_slice<1, false>(g, a.vocab, &s_floor);
      else
        best = same ? race_slice<3, true>(g, a.vocab, &s_floor)
                    : race_slice<3, false>(g, a.vocab, &s_floor);
    }
    if (lane == 0 && best) atomicMax(a.race + b, best);
  }
  // ---- the last slice to finish writes the answer
  __threadfence();
  __syncthreads();
  if (tid == 0) s_last = atomicAdd(a.arrived + b, 1u) == gridDim.x - 1;
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  int token = -1;
  if (r.n > 0) {
    if (greedy) {
      token = s_row[0][n_acc].best;
    } else {
      unsigned long long k = __ldcg(a.race + b);
      if (k == 0ull && residual && g.m > -INFINITY) k = race_plain(g, a.vocab);
      if (k) token = (int)(0xffffffffu - (uint32_t)k);
    }
  }
  for (int i = tid; i < a.max_out; i += kNT) {
    int t = -1;
    if (i < r.n) {
      if (i < n_acc) t = a.tokens[r.first + i + 1];
      else if (i == n_acc) t = token;
    }
    a.out_tokens[(int64_t)b * a.max_out + i] = t;
    if (a.logprobs) {
      float lp = 0.f;
      if (t >= 0 && !greedy) {
        const VerifyRow w = s_row[0][i];
        const float x =
            clean(a.logits[(r.first + i) * a.logits_stride + t]);
        lp = (x == w.m ? 0.f : (x - w.m) / T) - logf(w.z);
      }
      a.logprobs[(int64_t)b * a.max_out + i] = lp;
    }
  }
  if (tid == 0) {
    a.n_accepted[b] = n_acc;
    if (a.next_tokens) a.next_tokens[b] = token;
    if (a.seq_lens_out)
      a.seq_lens_out[b] = (a.seq_lens ? a.seq_lens[b] : 0) +
                          (r.n > 0 ? n_acc + 1 : 0);
  }
}

// Slices of a row in the first pass: those with the shortest time by waves of
// five CTAs an SM, each with 1.5 us to find out what its row is and its share
// of the 5.7 TB/s that such a wave reads (measured); 2048 values at least.
// (384 rows of 151936: 10 slices, 5.05 waves, took 49 us.)
int row_slices(const VerifyArgs& a, int64_t rows) {
  const double wave = 152 * 5, row_us = a.vocab * 4.0 * wave / 5.7e6;
  const int hi = (a.vocab + 2047) / 2048;
  int best = 1;
  double least = 1e30;
  for (int s = 1; s <= hi && s <= 128; ++s) {
    const double us = std::ceil(rows * s / wave) * (1.5 + row_us / s);
    if (us < least) {
      least = us;
      best = s;
    }
  }
  return best;
}

}  // namespace

size_t verify_workspace(VerifyArgs* a, char* base) {
  size_t off = 0;
  auto take = [&](size_t bytes) {
    char* p = base ? base + off : nullptr;
    off += (bytes + 255) / 256 * 256;
    return p;
  };
  const size_t rows = a->n_tokens > 0 ? a->n_tokens : 1;
  // (a call without drafts' logits has half the rows, and may have up to
  // twice the slices: room for either)
  const int one = row_slices(*a, rows), both = row_slices(*a, 2 * rows);
  a->slices = a->draft && a->draft_is_logits ? both : one;
  a->part = reinterpret_cast<float4*>(
      take(rows * (size_t)(one > 2 * both ? one : 2 * both) * 16));
  a->race = reinterpret_cast<unsigned long long*>(take((size_t)a->batch * 8));
  a->arrived = reinterpret_cast<uint32_t*>(take((size_t)a->batch * 4));
  return off;
}

cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t s) {
  const int rows = a.n_tokens > 0 ? a.n_tokens : 1;
  const bool dlog = a.draft && a.draft_is_logits;
  cudaError_t e = sv_launch(verify_stats, dim3(a.slices, rows, dlog ? 2 : 1),
                            kNT, 0, s, a);
  if (e != cudaSuccess) return e;
  // Slices of a race: whole turns of 4096 values a CTA, as few as keep the
  // grid within one wave of three CTAs an SM.
  const int64_t turns = ((int64_t)a.vocab + 4095) / 4096;
  const int64_t each = (turns * a.batch + 152 * 3 - 1) / (152 * 3);
  const int64_t n = (turns + each - 1) / each;
  return sv_launch(verify_sample, dim3((unsigned)n, a.batch), kNT, 0, s, a);
}

}  // namespace mpk
