// Appending new tokens to the paged KV cache (mpk_kv_append) and the
// rotation table it reads (mpk_rope_table).
//
// One thread takes 16 values of one head of one token: two 16-byte chunks
// that hold both members of 8 rotation pairs (half layout: chunk i and the
// chunk rot/2 values later; interleaved: two neighbouring chunks), so that a
// rotation needs no exchange between threads.  A head's d/16 threads sit in
// one warp and sum its squares with log2(d/16) shuffles.  A thread repeats
// this for up to kHeads heads of its token with the same cosines and sines in
// registers: the table row is read once per kHeads heads.
//
// Bound by HBM: every input and output byte moves once.
#include "serve_dev.cuh"

namespace mpk {
namespace {

constexpr int kThreadsA = 128;

__device__ __forceinline__ void unpack8(uint4 u, float* x) {
  x[0] = sv_lo(u.x); x[1] = sv_hi(u.x);
  x[2] = sv_lo(u.y); x[3] = sv_hi(u.y);
  x[4] = sv_lo(u.z); x[5] = sv_hi(u.z);
  x[6] = sv_lo(u.w); x[7] = sv_hi(u.w);
}
__device__ __forceinline__ uint4 pack8f(const float* x) {
  return make_uint4(sv_pack(x[0], x[1]), sv_pack(x[2], x[3]),
                    sv_pack(x[4], x[5]), sv_pack(x[6], x[7]));
}
__device__ __forceinline__ float round_bf16(float x) {
  return sv_lo(sv_pack(x, 0.f));
}

// LPH = d / 16 threads a head; HPT heads a thread.
template <int LPH, int HPT>
__global__ void __launch_bounds__(kThreadsA)
    append_kernel(const __grid_constant__ AppendArgs a, int n_items, int HG) {
  sv_grid_wait();
  const PagedArgs& p = a.p;
  constexpr int d = LPH * 16;
  const int gt = blockIdx.x * kThreadsA + threadIdx.x;
  const bool live = gt < n_items * LPH;
  const int item = live ? gt / LPH : n_items - 1;
  const int c = gt % LPH;
  const int t = item / HG, hg = item - t * HG;
  const int H = p.Hq + 2 * p.Hkv;
  // the two chunks of this thread, in values
  int lo, hi;
  const bool turns = c < a.rot / 16;
  if (!turns || a.interleaved) {
    lo = 16 * c;
    hi = lo + 8;
  } else {
    lo = 8 * c;
    hi = lo + a.rot / 2;
  }
  uint4 u0[HPT], u1[HPT];
  const int h_first = a.q_out ? 0 : p.Hq;   // no query output: keys on
#pragma unroll
  for (int j = 0; j < HPT; ++j) {
    const int h = h_first + hg + j * HG;
    if (!live || h >= H) continue;
    const uint16_t* src =
        h < p.Hq ? a.q + t * a.q_stride + (int64_t)h * d
        : h < p.Hq + p.Hkv
            ? a.k + t * a.k_stride + (int64_t)(h - p.Hq) * d
            : a.v + t * a.v_stride + (int64_t)(h - p.Hq - p.Hkv) * d;
    u0[j] = __ldg(reinterpret_cast<const uint4*>(src + lo));
    u1[j] = __ldg(reinterpret_cast<const uint4*>(src + hi));
  }
  // where the token goes
  const int b = sv_seq_of(p.q_start, p.tokens_per_seq, p.batch, t);
  int pos = -1, page = -1;
  bool ok = live && b >= 0;
  if (ok) {
    pos = __ldg(p.seq_lens + b) + t -
          sv_row(p.q_start, p.tokens_per_seq, p.n_tokens, b);
    const int pi = pos >= 0 ? (int)sv_div(pos, p.page_div) : p.max_pages;
    if (pi < p.max_pages)
      page = __ldg(p.page_table + (int64_t)b * p.max_pages + pi);
    if (page < 0 || page >= p.num_pages) {
      ok = false;
      sv_latch(p.status, MPK_ERR_KV_PAGE);
    } else if (a.rot > 0 && pos >= a.n_pos) {
      ok = false;
      sv_latch(p.status, MPK_ERR_INVALID_ARG);
    }
  }
  float cs[8], sn[8];
  if (turns && ok) {
    const float4* tab = reinterpret_cast<const float4*>(
        a.table + ((int64_t)pos * (a.rot / 2) + 8 * c) * 2);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 w = __ldg(tab + i);
      cs[2 * i] = w.x;
      sn[2 * i] = w.y;
      cs[2 * i + 1] = w.z;
      sn[2 * i + 1] = w.w;
    }
  }
  const int64_t slot =
      ok ? ((int64_t)page * p.Hkv * p.page_size + (pos % p.page_size)) * d : 0;
#pragma unroll
  for (int j = 0; j < HPT; ++j) {
    const int h = h_first + hg + j * HG;
    const bool isq = h < p.Hq, isk = !isq && h < p.Hq + p.Hkv;
    const uint16_t* nw = isq ? a.q_norm : isk ? a.k_norm : nullptr;
    float x[8], y[8];
    if (live && h < H) {
      unpack8(u0[j], x);
      unpack8(u1[j], y);
    }
    // The norm's output is a bf16 tensor of the decode step, so it is
    // rounded here too: the cache holds what mpk_decode_step would write,
    // bit for bit.  The sum of squares is fp32 over at most 128 values.
    // Threads without a head of this pass join the shuffles.
    float ss = 0.f;
    if (a.q_norm || a.k_norm) {
      if (live && h < H)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], fmaf(y[i], y[i], ss));
#pragma unroll
      for (int o = LPH / 2; o > 0; o >>= 1)
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
    }
    if (!ok || h >= H) continue;
    if (nw) {
      const float r = 1.0f / sqrtf(ss / (float)d + a.eps);
      float wa[8], wb[8];
      unpack8(__ldg(reinterpret_cast<const uint4*>(nw + lo)), wa);
      unpack8(__ldg(reinterpret_cast<const uint4*>(nw + hi)), wb);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = round_bf16(__fmul_rn(__fmul_rn(x[i], r), wa[i]));
        y[i] = round_bf16(__fmul_rn(__fmul_rn(y[i], r), wb[i]));
      }
    }
    if (turns && (isq || isk)) {
      if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float* z = i < 4 ? x + 2 * i : y + 2 * (i - 4);
          const float e = z[0], o = z[1];
          z[0] = __fsub_rn(__fmul_rn(e, cs[i]), __fmul_rn(o, sn[i]));
          z[1] = __fadd_rn(__fmul_rn(o, cs[i]), __fmul_rn(e, sn[i]));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float e = x[i], o = y[i];
          x[i] = __fsub_rn(__fmul_rn(e, cs[i]), __fmul_rn(o, sn[i]));
          y[i] = __fadd_rn(__fmul_rn(o, cs[i]), __fmul_rn(e, sn[i]));
        }
      }
    }
    uint16_t* dst;
    if (isq)
      dst = a.q_out + t * a.q_out_stride + (int64_t)h * d;
    else if (isk)
      dst = p.k + slot + (int64_t)(h - p.Hq) * p.page_size * d;
    else
      dst = p.v + slot + (int64_t)(h - p.Hq - p.Hkv) * p.page_size * d;
    // untouched values keep their bits (NaN payloads among them)
    const bool same = !nw && !(turns && (isq || isk));
    *reinterpret_cast<uint4*>(dst + lo) = same ? u0[j] : pack8f(x);
    *reinterpret_cast<uint4*>(dst + hi) = same ? u1[j] : pack8f(y);
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
  // One head a thread while that fills the GPU at most once (the chain of
  // loads is what such a call costs), else three.
  const int64_t all = (int64_t)a.p.n_tokens * H * LPH;
  const bool few = all <= 152 * 2048;
  const int hpt = few ? 1 : 3;
  const int HG = (H + hpt - 1) / hpt;
  const int64_t items = (int64_t)a.p.n_tokens * HG;
  const int64_t threads = items * LPH;
  if (threads > 0x7fffffff) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)((threads + kThreadsA - 1) / kThreadsA));
  auto k = few ? append_kernel<LPH, 1> : append_kernel<LPH, 3>;
  return sv_launch(k, grid, kThreadsA, 0, s, true, a, (int)items, HG);
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
                   true, a);
}

}  // namespace mpk
