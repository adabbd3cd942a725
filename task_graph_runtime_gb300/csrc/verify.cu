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
// verify_stats: (maximum, sum of exponentials) of every row, a row cut into
// slices so that few rows still fill the GPU; greedy rows (T <= 0) keep the
// index of the maximum instead.  verify_sample: every CTA of a sequence joins
// its rows' slices (in 64 bits), finds the first refused draft, and races its
// slice of that one row; slices meet in one 64-bit atomic maximum of (value,
// lowest index), whose result does not depend on their order.
// Bound by HBM: each row of logits leaves it once, the row that is sampled
// from once more with its draft and noise rows.
#include "serve_dev.cuh"

namespace mpk {
namespace {

constexpr int kNT = 256;
constexpr int kMaxOut = 128;     // rows of a sequence
constexpr float kLog2e = 1.4426950408889634f;

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

__global__ void __launch_bounds__(kNT)
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
      a.race[2 * b] = a.race[2 * b + 1] = 0ull;
      a.arrived[b] = 0u;
    }
  }
  const int row = blockIdx.y;
  if (row >= a.n_tokens) return;
  const int b = sv_seq_of(a.q_start, a.tokens_per_seq, a.batch, row);
  if (b < 0) return;
  const float T = a.temperature ? __ldg(a.temperature + b) : 1.f;
  const bool greedy = !(T > 0.f);
  if (blockIdx.z == 1) {
    // drafts' rows: the last row of a sequence has no draft after it, and a
    // greedy sequence does not ask for their distribution
    const RowInfo r = rows_of(a, b);
    if (row == r.first + r.n - 1 || greedy) return;
  }
  const float c = greedy ? 1.f : kLog2e / T;
  const float* x = blockIdx.z ? a.draft + row * a.draft_stride
                              : a.logits + row * a.logits_stride;
  // vectors of four on 16-byte boundaries: vector v holds values
  // [4 v - o, 4 v - o + 4)
  const int o = (int)(((uintptr_t)x >> 2) & 3);
  const int nv = (a.vocab + o + 3) / 4;
  const int v0 = (int)((int64_t)nv * blockIdx.x / gridDim.x);
  const int v1 = (int)((int64_t)nv * (blockIdx.x + 1) / gridDim.x);
  float m = -INFINITY, z = 0.f;
  int best = 0x7fffffff;
  constexpr int U = 4;
  for (int v = v0 + tid; v < v1; v += U * kNT) {
    float4 w[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int vi = v + i * kNT, k = 4 * vi - o;
      if (vi < v1 && k >= 0 && k + 4 <= a.vocab) {
        w[i] = __ldcs(reinterpret_cast<const float4*>(x + k));
      } else {
        float q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          q[j] = vi < v1 && k + j >= 0 && k + j < a.vocab ? x[k + j]
                                                          : -INFINITY;
        w[i] = make_float4(q[0], q[1], q[2], q[3]);
      }
      w[i].x = clean(w[i].x);
      w[i].y = clean(w[i].y);
      w[i].z = clean(w[i].z);
      w[i].w = clean(w[i].w);
    }
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < U; ++i)
      top = fmaxf(top, fmaxf(fmaxf(w[i].x, w[i].y), fmaxf(w[i].z, w[i].w)));
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
    a.stat[at] = make_float2(m, z);
    if (blockIdx.z == 0) a.amax[at] = best;
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

__global__ void __launch_bounds__(kNT)
    verify_sample(const __grid_constant__ VerifyArgs a) {
  __shared__ float s_m[2][kMaxOut];       // row maxima: target, draft
  __shared__ double s_z[2][kMaxOut];      // row sums
  __shared__ int s_best[kMaxOut];
  __shared__ int s_ok[kMaxOut];           // 1 accepted, 0 refused, 2 no draft
  __shared__ int s_last;
  const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31,
            warp = tid >> 5;
  sv_grid_wait();
  RowInfo r = rows_of(a, b);
  if (r.n > a.max_out) {
    if (tid == 0) sv_latch(a.status, MPK_ERR_INVALID_ARG);
    r.n = a.max_out;
  }
  const float T = a.temperature ? __ldg(a.temperature + b) : 1.f;
  const bool greedy = !(T > 0.f);
  const float c = greedy ? 1.f : kLog2e / T;
  const bool dlog = a.draft && a.draft_is_logits;
  // ---- the rows' statistics, and each draft's verdict
  for (int i = warp; i < r.n; i += kNT / 32) {
    for (int k = 0; k < (dlog && !greedy && i < r.n - 1 ? 2 : 1); ++k) {
      const int64_t at =
          ((int64_t)k * a.n_tokens + r.first + i) * a.splits;
      float m = -INFINITY;
      int best = 0x7fffffff;
      for (int s = lane; s < a.splits; s += 32) {
        const float v = a.stat[at + s].x;
        if (greedy && v > m) best = a.amax[at + s];
        m = fmaxf(m, v);
      }
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, s);
        const int b2 = __shfl_xor_sync(0xffffffffu, best, s);
        if (m2 > m || (m2 == m && b2 < best)) best = b2;
        m = fmaxf(m, m2);
      }
      double z = 0.0;
      for (int s = lane; s < a.splits; s += 32) {
        const float2 v = a.stat[at + s];
        z += (double)v.y * (v.x == m ? 1.0 : (double)ex2a((v.x - m) * c));
      }
#pragma unroll
      for (int s = 16; s > 0; s >>= 1)
        z += __shfl_xor_sync(0xffffffffu, z, s);
      if (lane == 0) {
        s_m[k][i] = m;
        s_z[k][i] = z;
        if (k == 0) s_best[i] = m == -INFINITY ? -1 : best;
      }
    }
    __syncwarp();
    if (lane == 0) {
      const int row = r.first + i;
      const int d = i < r.n - 1 ? a.tokens[row + 1] : -1;
      int ok = 2;
      if (d >= 0 && d < a.vocab) {
        if (greedy) {
          ok = d == s_best[i];
        } else {
          const float x = clean(a.logits[row * a.logits_stride + d]);
          const double p =
              s_m[0][i] == -INFINITY ? 0.0
              : x == s_m[0][i]       ? 1.0 / s_z[0][i]
                                     : exp(((double)x - s_m[0][i]) / T) /
                                     s_z[0][i];
          double q = 1.0;
          if (a.draft) {
            const float y = a.draft[row * a.draft_stride + d];
            if (!dlog) q = y;
            else if (s_m[1][i] == -INFINITY) q = 0.0;
            else if (clean(y) == s_m[1][i]) q = 1.0 / s_z[1][i];
            else q = exp(((double)clean(y) - s_m[1][i]) / T) / s_z[1][i];
          }
          ok = (double)a.uniform[row] * q < p ? 1 : 0;
        }
      }
      s_ok[i] = ok;
    }
  }
  __syncthreads();
  int n_acc = 0;
  while (n_acc < r.n - 1 && s_ok[n_acc] == 1) ++n_acc;
  const int row = r.first + n_acc;
  const bool residual = n_acc < r.n && s_ok[n_acc] == 0;
  // ---- this slice of the race
  if (r.n > 0 && !greedy) {
    const float m = s_m[0][n_acc];
    const float iz = (float)(1.0 / s_z[0][n_acc]);
    const double cd = 1.4426950408889634074 / (double)T;
    const float ch = (float)cd, cl = (float)(cd - (double)ch);
    const float* x = a.logits + row * a.logits_stride;
    const float* e = a.noise + b * a.noise_stride;
    const bool with_q = residual && a.draft;
    const float* y = with_q ? a.draft + row * a.draft_stride : x;
    const float mq = with_q && dlog ? s_m[1][n_acc] : 0.f;
    const float izq = with_q && dlog ? (float)(1.0 / s_z[1][n_acc]) : 0.f;
    const int skip = residual && !a.draft ? a.tokens[row + 1] : -1;
    unsigned long long best = 0ull, plain = 0ull;
    auto one = [&](int v, float xv, float yv, float ev) {
      if (m == -INFINITY) return;
      const float p = weight(clean(xv), m, ch, cl) * iz;
      float w = p;
      if (with_q) {
        const float q = !dlog ? yv
                        : mq == -INFINITY
                            ? 0.f
                            : weight(clean(yv), mq, ch, cl) * izq;
        w = p - q;
      } else if (v == skip) {
        w = 0.f;
      }
      if (w > 0.f) {
        const float s = w / ev;
        if (s >= 0.f) best = max(best, race_key(s, v));
      }
      if (residual && p > 0.f) {
        const float s = p / ev;
        if (s >= 0.f) plain = max(plain, race_key(s, v));
      }
    };
    const int o = (int)(((uintptr_t)x >> 2) & 3);
    const bool same = (((uintptr_t)e >> 2) & 3) == (unsigned)o &&
                      (((uintptr_t)y >> 2) & 3) == (unsigned)o;
    if (same) {
      const int nv = (a.vocab + o + 3) / 4;
      const int v0 = (int)((int64_t)nv * blockIdx.x / gridDim.x);
      const int v1 = (int)((int64_t)nv * (blockIdx.x + 1) / gridDim.x);
      for (int v = v0 + tid; v < v1; v += kNT) {
        const int k = 4 * v - o;
        if (k >= 0 && k + 4 <= a.vocab) {
          const float4 xv = __ldg(reinterpret_cast<const float4*>(x + k));
          const float4 ev = __ldcs(reinterpret_cast<const float4*>(e + k));
          const float4 yv =
              with_q ? __ldg(reinterpret_cast<const float4*>(y + k)) : xv;
          one(k, xv.x, yv.x, ev.x);
          one(k + 1, xv.y, yv.y, ev.y);
          one(k + 2, xv.z, yv.z, ev.z);
          one(k + 3, xv.w, yv.w, ev.w);
        } else {
          for (int j = 0; j < 4; ++j)
            if (k + j >= 0 && k + j < a.vocab)
              one(k + j, x[k + j], y[k + j], e[k + j]);
        }
      }
    } else {
      // rows on different 16-byte phases (an odd vocabulary)
      const int v0 = (int)((int64_t)a.vocab * blockIdx.x / gridDim.x);
      const int v1 = (int)((int64_t)a.vocab * (blockIdx.x + 1) / gridDim.x);
      constexpr int U = 4;
      for (int v = v0 + tid; v < v1; v += U * kNT) {
        float xv[U], yv[U], ev[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
          const int k = min(v + j * kNT, v1 - 1);
          xv[j] = __ldg(x + k);
          ev[j] = __ldcs(e + k);
          yv[j] = with_q ? __ldg(y + k) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < U; ++j)
          if (v + j * kNT < v1) one(v + j * kNT, xv[j], yv[j], ev[j]);
      }
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) {
      best = max(best, __shfl_xor_sync(0xffffffffu, best, s));
      plain = max(plain, __shfl_xor_sync(0xffffffffu, plain, s));
    }
    if (lane == 0) {
      if (best) atomicMax(a.race + 2 * b, best);
      if (plain) atomicMax(a.race + 2 * b + 1, plain);
    }
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
      token = s_best[n_acc];
    } else {
      unsigned long long k = __ldcg(a.race + 2 * b);
      // nothing of p lies above q (they agree to the last bit): sample p
      if (k == 0ull) k = __ldcg(a.race + 2 * b + 1);
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
        const float x =
            clean(a.logits[(r.first + i) * a.logits_stride + t]);
        const double d = x == s_m[0][i] ? 0.0 : (double)x - s_m[0][i];
        lp = (float)(d / T - log(s_z[0][i]));
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

}  // namespace

size_t verify_workspace(VerifyArgs* a, char* base) {
  size_t off = 0;
  auto take = [&](size_t bytes) {
    char* p = base ? base + off : nullptr;
    off += (bytes + 255) / 256 * 256;
    return p;
  };
  // Slices of at most 16384 values, fewer when there are few rows (about
  // four CTAs an SM), and no fewer than 2048.
  const int64_t rows = a->n_tokens > 0 ? a->n_tokens : 1;
  int64_t s = (152 * 4 + rows - 1) / rows;
  const int64_t lo = (a->vocab + 16383) / 16384, hi = (a->vocab + 2047) / 2048;
  s = s < lo ? lo : s > hi ? hi : s;
  a->splits = (int)s;
  a->stat = reinterpret_cast<float2*>(take((size_t)2 * rows * s * 8));
  a->amax = reinterpret_cast<int32_t*>(take((size_t)rows * s * 4));
  a->race = reinterpret_cast<unsigned long long*>(take((size_t)a->batch * 16));
  a->arrived = reinterpret_cast<uint32_t*>(take((size_t)a->batch * 4));
  return off;
}

cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t s) {
  const int rows = a.n_tokens > 0 ? a.n_tokens : 1;
  const bool dlog = a.draft && a.draft_is_logits;
  cudaError_t e = sv_launch(verify_stats, dim3(a.splits, rows, dlog ? 2 : 1),
                            kNT, 0, s, true, a);
  if (e != cudaSuccess) return e;
  int64_t n = (152 * 4 + a.batch - 1) / a.batch;
  const int64_t hi = (a.vocab + 2047) / 2048;
  n = n > hi ? hi : n;
  return sv_launch(verify_sample, dim3((unsigned)n, a.batch), kNT, 0, s, true,
                   a);
}

}  // namespace mpk
