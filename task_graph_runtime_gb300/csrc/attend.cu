// Attention over the paged cache with shared prefixes (mpk_prefix_attention):
// the choice of launches and the merge of their results.  The kernels are in
// attend_kernel.cuh and attend_tc.cu.
#include "attend_plan.cuh"

namespace mpk {
namespace {

constexpr int kNT = 128;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The segments of a row's unit: the row in the first slot (an index into ml),
// and how many slots.
struct Found {
  int64_t at;
  int n;
};
__device__ __forceinline__ Found find(const AttendArgs& a, const AttnSet& s,
                                      int tok0, int e, int row, int h) {
  Found f{0, 0};
  if (row < 0) return f;
  const int tile = row >> s.shift;
  const int64_t at = meta_of(a.p, tok0, e, tile, s.shift, h);
  if (at >= s.units) return f;
  const int2 me = s.meta[at];
  // (only arrays that are not ascending leave anything else here)
  if (me.x < 0 || me.y < 0 || me.y > s.slots - me.x) return f;
  f.at = ((int64_t)me.x << s.shift) + (row & (s.M - 1));
  f.n = me.y;
  return f;
}

// One warp joins the segments of one (token, query head): the prefix's and
// the sequence's own.  Lane i fetches the maximum and sum of segment i, then
// the partial outputs are added with their final weights, four loads in
// flight.
// FEW: a grid of at most two CTAs an SM is all latency.  It goes through one
// turn of the same code on whatever the workspace holds while it waits for the
// kernels before it, so that the instructions and the pages' translations are
// at hand, and has the first four segments on their way before it knows their
// weights (16 sequences of 32 heads: the whole call 26.9 us, weights first
// 29.3).
// More CTAs hide each other's latency and need the registers: 64 sequences
// 49.7 us against 51.1.  (Eight or sixteen segments in flight: 0.4 and 1 us
// longer with 16 sequences; four heads a warp: 6 us longer.)
template <int D, bool FEW>
__global__ void __launch_bounds__(kNT)
    attend_merge(const __grid_constant__ AttendArgs a) {
  constexpr int V = D / 32, G = 4;
  const PagedArgs& p = a.p;
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * (kNT / 32) + (threadIdx.x >> 5);
  if (w >= (int64_t)p.n_tokens * p.Hq) return;
  const int t = (int)(w / p.Hq), hq = (int)(w - (int64_t)t * p.Hq);
  const int h = (int)sv_div(hq, p.grp_div), grp = p.Hq / p.Hkv;
  const int j = hq - h * grp;
  const int b = sv_seq_of_warp(p.q_start, p.tokens_per_seq, p.batch, t);
  if (b < 0) return;                     // behind the last sequence
  const Ent own = att_seq_ent(a, b);
  const int g = a.n_groups > 0 ? att_group(a, b) : 0;
  Ent pre{0, 0, 0, 0, 0};
  if (a.n_groups > 0) pre = att_group_ent(a, g);
  float m, l, acc[V];
  for (int pass = FEW ? 0 : 1; pass < 2; ++pass) {
    Found fp{0, 0}, fo{0, 1};            // (every set has a slot)
    if (pass == 1) {
      sv_grid_wait();
      fo.n = 0;
      if (pre.k1 > 0)
        fp = find(a, a.pre, pre.tok0, g, (t - pre.tok0) * grp + j, h);
      if (own.k1 > own.k0)
        fo = find(a, a.own, own.tok0, b, (t - own.tok0) * grp + j, h);
    }
    const int n = fp.n + fo.n;
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int i = i0 + lane;
      float2 ml = make_float2(-INFINITY, 0.f);
      const float* src = nullptr;
      if (i < n) {
        const bool q = i < fp.n;
        const int64_t at = q ? fp.at + ((int64_t)i << a.pre.shift)
                             : fo.at + ((int64_t)(i - fp.n) << a.own.shift);
        ml = q ? a.pre.ml[at] : a.own.ml[at];
        src = (q ? a.pre.part : a.own.part) + at * D;
      }
      const int k = min(32, n - i0);
      // segments q0 .. q0 + G - 1 on their way (a whole warp's row each)
      float v[G][V];
      auto row = [&](int q, float (&x)[V]) {
        const float* s = reinterpret_cast<const float*>(__shfl_sync(
            0xffffffffu, reinterpret_cast<unsigned long long>(src), q));
        if constexpr (V == 4) {
          const float4 u = *reinterpret_cast<const float4*>(s + lane * 4);
          x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
        } else if constexpr (V == 2) {
          const float2 u = *reinterpret_cast<const float2*>(s + lane * 2);
          x[0] = u.x; x[1] = u.y;
        } else {
          x[0] = s[lane];
        }
      };
      auto fetch = [&](int q0) {
#pragma unroll
        for (int j = 0; j < G; ++j) {
#pragma unroll
          for (int c = 0; c < V; ++c) v[j][c] = 0.f;
          if (q0 + j < k) row(q0 + j, v[j]);   // (the same for all lanes)
        }
      };
      if (FEW) fetch(0);
      float top = ml.x;
#pragma unroll
      for (int s = 16; s > 0; s >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
      const float mn = fmaxf(m, top);
      const float f = mn == -INFINITY ? 0.f : ex2(m - mn);
      const float wt = ml.x == -INFINITY ? 0.f : ex2(ml.x - mn);
      float sum = ml.x == -INFINITY ? 0.f : ml.y * wt;
#pragma unroll
      for (int s = 16; s > 0; s >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, s);
      m = mn;
      l = l * f + sum;
#pragma unroll
      for (int q = 0; q < V; ++q) acc[q] *= f;
      // (a segment in which the row saw nothing has weight 0 and zeros)
      auto add = [&](int q, const float (&x)[V]) {
        const float w = __shfl_sync(0xffffffffu, wt, q);
#pragma unroll
        for (int c = 0; c < V; ++c) acc[c] = fmaf(x[c], w, acc[c]);
      };
      if constexpr (FEW) {
        for (int q0 = 0;;) {
#pragma unroll
          for (int j = 0; j < G; ++j) add(q0 + j, v[j]);
          q0 += G;
          if (q0 >= k) break;
          fetch(q0);
        }
      } else {
#pragma unroll 4
        for (int q = 0; q < k; ++q) {
          float x[V];
          row(q, x);
          add(q, x);
        }
      }
    }
  }
  // no key seen: zeros, and -inf for the log sum
  const float inv = l > 0.f ? 1.0f / l : (l == 0.f ? 0.f : l);
  uint16_t* out = a.out + t * a.out_stride + (int64_t)hq * D + lane * V;
  if constexpr (V == 4) {
    *reinterpret_cast<uint2*>(out) =
        make_uint2(sv_pack(acc[0] * inv, acc[1] * inv),
                   sv_pack(acc[2] * inv, acc[3] * inv));
  } else if constexpr (V == 2) {
    *reinterpret_cast<uint32_t*>(out) = sv_pack(acc[0] * inv, acc[1] * inv);
  } else {
    *out = (uint16_t)sv_pack(acc[0] * inv, 0.f);
  }
  if (a.lse && lane == 0)
    a.lse[(int64_t)t * p.Hq + hq] =
        l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
}

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t,
                             void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*,
                             CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The layer's pool as rows of d values, in boxes of `box` rows x 128 bytes (the
// whole row of 64 for 32 values), swizzled as the kernels read them.
bool page_map(EncodeFn fn, const PagedArgs& p, const void* pool, int box,
              CUtensorMap* m) {
  const cuuint64_t dims[2] = {
      (cuuint64_t)p.d, (cuuint64_t)p.num_pages * p.Hkv * p.page_size};
  const cuuint64_t strides[1] = {(cuuint64_t)p.d * 2};
  const cuuint32_t boxes[2] = {p.d < 64 ? 32u : 64u, (cuuint32_t)box};
  const cuuint32_t steps[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(pool),
            dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
            p.d < 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool page_maps(AttendArgs* a) {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                         cudaEnableDefault, &r) !=
            cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn && page_map(fn, a->p, a->p.k, a->box, &a->map_k) &&
         page_map(fn, a->p, a->p.v, a->box, &a->map_v);
}

template <int D>
cudaError_t run_merge(const AttendArgs& a, cudaStream_t s) {
  const int64_t warps = (int64_t)a.p.n_tokens * a.p.Hq;
  const int64_t blocks = (warps + kNT / 32 - 1) / (kNT / 32);
  return sv_launch(blocks <= 152 * 2 ? attend_merge<D, true>
                                     : attend_merge<D, false>,
                   dim3((unsigned)blocks), kNT, 0, s, a);
}

}  // namespace

// at most: one CTA for each of four places on 152 SMs
int attend_ctas() { return 152 * 4; }

// Keys of a page that one TMA box takes: a power of two (so that a block of
// keys is whole boxes) that divides the page; 0, and no TMA, when that is
// below the 8 rows of a swizzle group or the pool's rows pass a coordinate.
int attend_box(const PagedArgs& p) {
  if ((int64_t)p.num_pages * p.Hkv * p.page_size > 0x7fffffff) return 0;
  const int box = p.page_size & -p.page_size;
  return box < 8 ? 0 : box > 64 ? 64 : box;
}

// Chooses the launches and places their results.
size_t attend_workspace(AttendArgs* a, char* base) {
  size_t off = 0;
  auto take = [&](size_t bytes) {
    char* p = base ? base + off : nullptr;
    off += (bytes + 255) / 256 * 256;
    return p;
  };
  // rows of one KV head, on average over the sequences and over the groups
  const int64_t rows = (int64_t)a->p.n_tokens * (a->p.Hq / a->p.Hkv);
  const int64_t per = (rows + a->p.batch - 1) / a->p.batch;
  const int64_t all = a->n_groups ? (rows + a->n_groups - 1) / a->n_groups : 0;
  // the smallest row tiles that hold them; few pairs are built
  a->wmo = per <= 8 ? 0 : per <= 16 ? 1 : per <= 32 ? 2 : 4;
  a->box = attend_box(a->p);
  // The tensor-memory kernel where it is the faster one for prefixes as long
  // as the page table allows.  Measured: it costs 8 us of its own (plan,
  // set-up, results; the sequences' kernel starts behind it) and 1.85 us a
  // tile of 256 rows x 128 keys on 152 SMs; the general kernel takes 2 us
  // (head_dim 128; 64: 1.2 us) a tile of 64 x 64 on 304 CTAs.
  if (a->n_groups && a->box && a->p.d >= 64 && a->scale_log2 > 0.f &&
      all > 64) {
    const double ctx = (double)a->p.page_size * a->p.max_pages;
    const double units = (double)a->n_groups * a->p.Hkv;
    const double gen = units * ((all + 63) / 64) * (ctx / 64) *
                       (a->p.d == 128 ? 2.0 : 1.2) / 304;
    const double tc =
        8 + units * ((all + 255) / 256) * (ctx / 128) * 1.85 / 152;
    a->tc = tc < gen;
  } else {
    a->tc = 0;
  }
  a->wmp = !a->n_groups || a->tc || all <= (a->wmo ? 16 * a->wmo : 8)
               ? a->wmo
               : 4;
  a->own.M = a->wmo ? 16 * a->wmo : 8;
  a->pre.M = a->tc ? attend_tc_rows() : a->wmp ? 16 * a->wmp : 8;
  // a set holds the results of n entities whose rows are disjoint
  auto place = [&](AttnSet* s, int64_t n, int ctas) {
    s->shift = 31 - __builtin_clz((unsigned)s->M);
    s->units = (rows / s->M + n) * a->p.Hkv;
    s->slots = s->units + ctas;
    s->meta = reinterpret_cast<int2*>(take(s->units * 8));
    s->ml = reinterpret_cast<float2*>(take(s->slots * s->M * 8));
    s->part = reinterpret_cast<float*>(
        take((size_t)s->slots * s->M * a->p.d * 4));
  };
  place(&a->own, a->p.batch, attend_ctas());
  if (a->n_groups)
    place(&a->pre, a->n_groups, a->tc ? attend_tc_ctas() : attend_ctas());
  return off;
}

cudaError_t launch_attend(AttendArgs& a, cudaStream_t s) {
  if (a.box && !page_maps(&a)) return cudaErrorNotSupported;
  cudaError_t e = cudaSuccess;
  if (a.tc) e = launch_attend_tc(a, s);
  if (e != cudaSuccess) return e;
  const int d = a.p.d;
  e = d == 128  ? launch_attend_128(a, s)
      : d == 64 ? launch_attend_64(a, s)
                : launch_attend_32(a, s);
  if (e != cudaSuccess) return e;
  return d == 128  ? run_merge<128>(a, s)
         : d == 64 ? run_merge<64>(a, s)
                   : run_merge<32>(a, s);
}

}  // namespace mpk
