// Appending new tokens to the paged KV cache (mpk_kv_append) and the
// rotation table it reads (mpk_rope_table).
//
// One thread takes 16 values of a head: two 16-byte chunks that hold both
// members of 8 rotation pairs (half layout: chunk i and the chunk rot/2 values
// later; interleaved: two neighbouring chunks), so that a rotation needs no
// exchange between threads.  A head's d/16 threads sit in one warp and sum its
// squares with log2(d/16) shuffles.  A thread stays with its token and its
// place in the head and goes over every HS-th head, so the cosines and sines
// (and what the token's position leads to) are found once, and the next two
// heads are on the way while two are worked on.  Arithmetic is on pairs of
// fp32 values (twice the rate), each operation rounded as by itself.
//
// Bound by HBM: every input and output byte moves once.  Measured (32 / 8
// heads of 128): 23 prompts of 1..4001 tokens, 921 MB, 158 us =
// 5.8 TB/s; 8192 tokens, 205 MB, 42 us; one token of 16 sequences 3.6 us.
#include "serve_dev.cuh"

namespace mpk {
namespace {

constexpr int kThreadsA = 256;

__device__ __forceinline__ float2 two(uint32_t w) {
  return make_float2(sv_lo(w), sv_hi(w));
}
// Products by pairs, sums one by one: with sums by pairs too, some of them
// come out fused with a product into one rounding (as instructions, as
// intrinsics, and as multiply-adds by 1), which is not what the decode step
// computes.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  return __fmul2_rn(a, b);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y));
}
__device__ __forceinline__ float2 sub2(float2 a, float2 b) {
  return make_float2(__fsub_rn(a.x, b.x), __fsub_rn(a.y, b.y));
}
__device__ __forceinline__ uint32_t pack2(float2 v) {
  return sv_pack(v.x, v.y);
}
__device__ __forceinline__ const uint32_t* words(const uint4& u) {
  return reinterpret_cast<const uint32_t*>(&u);
}

// LPH = d / 16 threads a head; HS threads share a token's heads at one place.
template <int LPH>
__global__ void __launch_bounds__(kThreadsA, 2)
    append_kernel(const __grid_constant__ AppendArgs a, int HS) {
  sv_grid_wait();
  const PagedArgs& p = a.p;
  constexpr int d = LPH * 16;
  const int c = threadIdx.x % LPH, hs = threadIdx.x / LPH % HS;
  const int n_tok = kThreadsA / (LPH * HS);
  const int t = blockIdx.x * n_tok + threadIdx.x / (LPH * HS);
  const bool row = t < p.n_tokens;
  const int h0 = (a.q_out ? 0 : p.Hq) + hs;   // no query output: keys on
  const int H = p.Hq + 2 * p.Hkv;
  // the two chunks of this thread, in values
  const bool turns = c < a.rot / 16;
  const int lo = !turns || a.interleaved ? 16 * c : 8 * c;
  const int hi = !turns || a.interleaved ? lo + 8 : lo + a.rot / 2;
  const uint16_t* rq = a.q + t * a.q_stride;
  const uint16_t* rk = a.k + t * a.k_stride - (int64_t)p.Hq * d;
  const uint16_t* rv = a.v + t * a.v_stride - (int64_t)(p.Hq + p.Hkv) * d;
  auto fetch = [&](int h, uint4& u, uint4& v) {
    if (!row || h >= H) return;
    const uint16_t* src =
        (h < p.Hq ? rq : h < p.Hq + p.Hkv ? rk : rv) + (int64_t)h * d;
    u = __ldcs(reinterpret_cast<const uint4*>(src + lo));
    v = __ldcs(reinterpret_cast<const uint4*>(src + hi));
  };
  uint4 u[2] = {}, v[2] = {};
  fetch(h0, u[0], v[0]);
  fetch(h0 + HS, u[1], v[1]);
  // where the token goes: the warp finds the sequence of its first token,
  // its others are a step or a few further
  const int tw = min(__shfl_sync(0xffffffffu, t, 0), p.n_tokens - 1);
  int b = sv_seq_of_warp(p.q_start, p.tokens_per_seq, p.batch, tw);
  if (t != tw && row) {
    if (p.q_start && b >= 0) {
      while (b < p.batch && __ldg(p.q_start + b + 1) <= t) ++b;
      if (b == p.batch) b = -1;
    } else {
      b = sv_seq_of(p.q_start, p.tokens_per_seq, p.batch, t);
    }
  }
  bool ok = row && b >= 0;
  int pos = 0;
  int64_t slot = 0;
  if (ok) {
    pos = __ldg(p.seq_lens + b) + t -
          sv_row(p.q_start, p.tokens_per_seq, p.n_tokens, b);
    const int pi = pos >= 0 ? (int)sv_div(pos, p.page_div) : p.max_pages;
    int page = -1;
    if (pi < p.max_pages)
      page = __ldg(p.page_table + (int64_t)b * p.max_pages + pi);
    if (page < 0 || page >= p.num_pages) {
      ok = false;
      sv_latch(p.status, MPK_ERR_KV_PAGE);
    } else if (a.rot > 0 && pos >= a.n_pos) {
      ok = false;
      sv_latch(p.status, MPK_ERR_INVALID_ARG);
    }
    slot = ((int64_t)page * p.Hkv * p.page_size + (pos - pi * p.page_size)) * d;
  }
  float2 cs[4], sn[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float4 f = make_float4(1.f, 0.f, 1.f, 0.f);
    if (turns && ok)
      f = __ldg(reinterpret_cast<const float4*>(
                    a.table + ((int64_t)pos * (a.rot / 2) + 8 * c) * 2) + i);
    cs[i] = make_float2(f.x, f.z);
    sn[i] = make_float2(f.y, f.w);
  }
  uint16_t* oq = a.q_out + t * a.q_out_stride;
  const int64_t head = (int64_t)p.page_size * d;
  const bool norms = a.q_norm || a.k_norm;
  // one head: chunks x and y of it to its place
  auto work = [&](int h, uint4 cu, uint4 cv) {
    const bool here = ok && h < H;
    const bool isq = h < p.Hq, isk = !isq && h < p.Hq + p.Hkv;
    const uint16_t* nw = isq ? a.q_norm : isk ? a.k_norm : nullptr;
    float2 x[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = two(words(cu)[i]);
      y[i] = two(words(cv)[i]);
    }
    float r = 0.f;
    if (norms) {
      // The sum of squares is fp32 over at most 128 values; threads without
      // a head of this turn join the shuffles.
      float2 ss = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        ss = __ffma2_rn(x[i], x[i], __ffma2_rn(y[i], y[i], ss));
      float sum = ss.x + ss.y;
#pragma unroll
      for (int o = LPH / 2; o > 0; o >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
      r = 1.0f / sqrtf(sum / (float)d + a.eps);
    }
    if (!here) return;
    if (nw) {
      // The norm's output is a bf16 tensor of the decode step, so it is
      // rounded here too: the cache holds what mpk_decode_step would write,
      // bit for bit.
      const uint4 wa = __ldg(reinterpret_cast<const uint4*>(nw + lo));
      const uint4 wb = __ldg(reinterpret_cast<const uint4*>(nw + hi));
      const float2 rr = make_float2(r, r);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = two(pack2(mul2(mul2(x[i], rr), two(words(wa)[i]))));
        y[i] = two(pack2(mul2(mul2(y[i], rr), two(words(wb)[i]))));
      }
    }
    const bool rot = turns && (isq || isk);
    if (rot) {
      if (a.interleaved) {
        // pairs lie side by side: (even, odd) of two values to (evens, odds)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float2* z = i < 2 ? x + 2 * i : y + 2 * (i - 2);
          const float2 e = make_float2(z[0].x, z[1].x);
          const float2 o = make_float2(z[0].y, z[1].y);
          const float2 q =
              sub2(mul2(e, cs[i]), mul2(o, sn[i]));
          const float2 w =
              add2(mul2(o, cs[i]), mul2(e, sn[i]));
          z[0] = make_float2(q.x, w.x);
          z[1] = make_float2(q.y, w.y);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 e = x[i], o = y[i];
          x[i] = sub2(mul2(e, cs[i]), mul2(o, sn[i]));
          y[i] = add2(mul2(o, cs[i]), mul2(e, sn[i]));
        }
      }
    }
    uint16_t* dst = isq   ? oq + (int64_t)h * d
                    : isk ? p.k + slot + (h - p.Hq) * head
                          : p.v + slot + (h - p.Hq - p.Hkv) * head;
    // untouched values keep their bits (NaN payloads among them)
    if (nw || rot) {
      cu = make_uint4(pack2(x[0]), pack2(x[1]), pack2(x[2]), pack2(x[3]));
      cv = make_uint4(pack2(y[0]), pack2(y[1]), pack2(y[2]), pack2(y[3]));
    }
    *reinterpret_cast<uint4*>(dst + lo) = cu;
    *reinterpret_cast<uint4*>(dst + hi) = cv;
  };
  // (the same number of turns for all threads of a warp)
  for (int h = h0; h - hs < H; h += 2 * HS) {
    uint4 nu[2] = {}, nv[2] = {};
    fetch(h + 2 * HS, nu[0], nv[0]);
    fetch(h + 3 * HS, nu[1], nv[1]);
    work(h, u[0], v[0]);
    work(h + HS, u[1], v[1]);
    u[0] = nu[0];
    u[1] = nu[1];
    v[0] = nv[0];
    v[1] = nv[1];
  }
}

// cos and sin of position * inverse frequency, times the attention factor.
// Angles, the scaled frequencies and the functions are in 64 bits: a
// position of 10^6 times a frequency near 1 leaves no bit of a fraction in
// 32.  Rounded once.
__global__ void rope_table_kernel(const __grid_constant__ RopeTableArgs a) {
  sv_grid_wait();
  const int half = a.rot / 2;
  const int64_t n = (int64_t)a.n_pos * half;
  const double kPi2 = 6.283185307179586476925286766559;
  for (int64_t k = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; k < n;
       k += (int64_t)gridDim.x * blockDim.x) {
    const int64_t row = k / half;
    const int i = (int)(k - row * half);
    double inv = pow(a.theta, -2.0 * i / a.rot);
    if (a.scaling == MPK_ROPE_LINEAR) {
      inv /= a.factor;
    } else if (a.scaling == MPK_ROPE_BANDS) {
      // wavelengths above old_ctx / low are stretched by the factor, those
      // below old_ctx / high stay, those between are mixed
      const double turns = a.old_ctx * inv / kPi2;
      const double m = fmin(fmax((turns - a.low) / (a.high - a.low), 0.0), 1.0);
      inv = (1.0 - m) * inv / a.factor + m * inv;
    } else if (a.scaling == MPK_ROPE_RAMP) {
      // the same mixture, linear in the pair's index between the indices
      // that make `high` and `low` turns over old_ctx positions
      const double den = 2.0 * log(a.theta);
      const double at_hi = a.rot * log(a.old_ctx / (a.high * kPi2)) / den;
      const double at_lo = a.rot * log(a.old_ctx / (a.low * kPi2)) / den;
      const double lo = fmax(floor(at_hi), 0.0);
      const double hi = fmin(ceil(at_lo), (double)a.rot - 1.0);
      const double m =
          fmin(fmax((i - lo) / (hi > lo ? hi - lo : 1e-3), 0.0), 1.0);
      inv = m * inv / a.factor + (1.0 - m) * inv;
    }
    double s, c;
    sincos((double)(a.first_pos + row) * inv, &s, &c);
    a.out[2 * k] = (float)(c * a.attn_factor);
    a.out[2 * k + 1] = (float)(s * a.attn_factor);
  }
}

template <int LPH>
cudaError_t append_d(const AppendArgs& a, cudaStream_t s) {
  const int H = (a.q_out ? a.p.Hq : 0) + 2 * a.p.Hkv;
  // Threads that share a token's heads: as many as there are heads while the
  // call fills the GPU at most once (its cost is the chain of loads), else
  // few, so that a thread's start serves many heads, but two waves of CTAs.
  const int64_t T = a.p.n_tokens;
  int HS = 1;
  while (HS < 32 && HS * LPH < kThreadsA && HS < H &&
         T * LPH * HS < (int64_t)152 * 512 * 2)
    HS *= 2;
  const int n_tok = kThreadsA / (LPH * HS);
  return sv_launch(append_kernel<LPH>,
                   dim3((unsigned)((T + n_tok - 1) / n_tok)), kThreadsA, 0, s,
                   a, HS);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, cudaStream_t s) {
  if (a.p.d == 128) return append_d<8>(a, s);
  if (a.p.d == 64) return append_d<4>(a, s);
  return append_d<2>(a, s);
}

cudaError_t launch_rope_table(const RopeTableArgs& a, cudaStream_t s) {
  const int64_t n = (int64_t)a.n_pos * (a.rot / 2);
  const int64_t blocks = (n + 127) / 128;
  return sv_launch(rope_table_kernel,
                   dim3((unsigned)(blocks < 4096 ? blocks : 4096)), 128, 0, s,
                   a);
}

}  // namespace mpk
