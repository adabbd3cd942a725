// Attention of new tokens over the paged cache with shared prefixes
// (mpk_prefix_attention): the general kernel.  Included by one translation
// unit per head size.
//
// For a query row q of position t: o = sum_j p_j v_j, p_j = e^(s_j - M) / L,
// s_j = scale q.k_j over keys j <= t, with the running maximum M and sum L of
// a softmax in fp32.  The rows of a group (all tokens of its sequences, all
// query heads of a KV head) meet the prefix's keys together, so the prefix
// leaves HBM once; a sequence's own keys meet its own rows.  The two parts
// of a row, and the segments a long key axis is split into (attend_plan.cuh),
// are joined by their (M, L) in attend_merge (attend.cu).
//
// attend_kernel<D, WMP, WMO>: 4 warps; a group's row tile has 16 WMP rows, a
// sequence's 16 WMO.  A warp holds 16 rows and 64 / (4 / WM) keys of a block
// of 64; mma.sync m16n8k16, scores and weights stay in registers.  With few
// rows the warps split the keys, so that the tensor instructions per block
// stay few; the kernel is bound by the K/V bytes.  Blocks come through a ring
// of kStages shared-memory stages, 16-byte asynchronous copies, every token
// from its own page (any page size).  The copies run ahead over the whole
// stretch of the CTA, across the ends of segments, and the next segment's
// queries are fetched during the last block of the one before, so a stretch
// of many short sequences streams like one long one.
#pragma once

#include "attend_plan.cuh"

namespace mpk {
namespace {

constexpr int kNT = 128;
constexpr int kBN = 64;
constexpr int kStages = 3;

__device__ __forceinline__ uint32_t s_addr(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
// 16 bytes, or zeros when n == 0 (nothing is read then)
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
               "l"(src), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile(
      "ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile(
      "ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4],
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 2^x, exact 0 for -inf
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Byte offset of 16-byte chunk c of row r in a tile of D-value rows.  The
// chunk index is mixed with the row so that the 8 rows an ldmatrix reads lie
// in different banks.
template <int D>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  if (D == 32) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  return r * (D * 2) + ((c ^ (r & 7)) << 4);
}

template <int D>
struct Cfg {
  static constexpr int kTile = kBN * D * 2;            // bytes of K (or V)
  static constexpr int kStage = 2 * kTile;
  static constexpr int kSmem = kStages * kStage;
  static constexpr int CH = D / 8;                     // chunks a row
  static constexpr int kPitch = D + 4;                 // merge buffer, floats
  // rows that the merge of four key slices takes at a time (it lies over a
  // stage that has been consumed)
  static constexpr int kPass = 8;
  static_assert(4 * kPass * kPitch * 4 <= kStage, "merge buffer");
};

// A position on the CTA's stretch of the line.
struct Cursor {
  Ent E;
  int e, nb, units, u, blk, unit0;
  int64_t left;        // blocks of the stretch from here on
};

// What the blocks of a segment need to know.
struct Seg {
  int k1, key;         // end of the keys; first key of the next block
  int lim[2], lim_min; // keys this thread's two rows see
  bool prefix;
};

template <int D, int WMP, int WMO>
struct Attend {
  using C = Cfg<D>;
  static constexpr int CH = C::CH;
  static constexpr int RPT = kBN * CH / kNT;           // rows a thread loads
  static constexpr int RSTEP = kNT / CH;

  const AttendArgs& a;
  uint8_t* smem;
  float (*s_ml)[2];    // [4 * 16] of each warp's rows
  uint32_t* s_bad;     // [2] keys of a block whose V is not finite
  int G, n_ent;

  uint32_t qf[D / 16][4];
  float o[D / 8][4];
  float m[2], l[2];

  __device__ __forceinline__ Ent ent(int i) const {
    return i < G ? att_group_ent(a, i) : att_seq_ent(a, i - G);
  }
  __device__ __forceinline__ void enter(Cursor& c) const {
    const int M = c.e < G ? 16 * WMP : 16 * WMO;
    c.E = ent(c.e);
    c.nb = (c.E.k1 - c.E.k0 + kBN - 1) / kBN;
    c.units = c.nb > 0 ? ((c.E.rows + M - 1) / M) * a.p.Hkv : 0;
  }
  __device__ __forceinline__ void advance(Cursor& c) const {
    --c.left;
    if (++c.blk < c.nb) return;
    c.blk = 0;
    if (++c.u < c.units) return;
    if (c.left <= 0) return;
    do {
      c.unit0 = c.e + 1 == G ? 0 : c.unit0 + c.units;
      ++c.e;
      if (c.e >= n_ent) {
        c.left = 0;
        return;
      }
      enter(c);
    } while (c.units == 0);
    c.u = 0;
  }

  // K and V of the cursor's block into stage st
  __device__ __forceinline__ void load(const Cursor& cu, int st) {
    const PagedArgs& p = a.p;
    const uint32_t ks = s_addr(smem + st * C::kStage);
    const int c = threadIdx.x % CH, r0 = threadIdx.x / CH;
    const int h = cu.u % p.Hkv, key = cu.E.k0 + cu.blk * kBN;
    const int32_t* pt = p.page_table + (int64_t)cu.E.seq * p.max_pages;
    int pi[RPT], page[RPT];
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int t = key + r0 + i * RSTEP;
      pi[i] = (int)sv_div(t, p.page_div);
      page[i] = t < cu.E.k1 ? __ldg(pt + pi[i]) : -2;
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int r = r0 + i * RSTEP, t = key + r;
      const bool ok = page[i] >= 0 && page[i] < p.num_pages;
      if (!ok && page[i] != -2) sv_latch(p.status, MPK_ERR_KV_PAGE);
      const int64_t off =
          ok ? (((int64_t)page[i] * p.Hkv + h) * p.page_size +
                (t - pi[i] * p.page_size)) * D + c * 8
             : 0;
      const uint32_t dst = ks + swz<D>(r, c);
      cp16(dst, p.k + off, ok ? 16 : 0);
      cp16(dst + C::kTile, p.v + off, ok ? 16 : 0);
    }
  }

  // This thread's part of the queries of the cursor's unit, in the layout of
  // the product's first operand (rows past the entity's are zeros).
  template <int WM>
  __device__ __forceinline__ void queries(const Cursor& cu,
                                          uint32_t (&q)[D / 16][4]) {
    const PagedArgs& p = a.p;
    const int lane = threadIdx.x & 31, wm = (threadIdx.x >> 5) % WM;
    const int grp = p.Hq / p.Hkv, h = cu.u % p.Hkv, tile = cu.u / p.Hkv;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = tile * 16 * WM + wm * 16 + (lane >> 2) + 8 * r;
      const bool ok = row < cu.E.rows;
      const int tok = ok ? row / grp : 0;
      const uint16_t* src = a.q + (cu.E.tok0 + tok) * a.q_stride +
                            (int64_t)(h * grp + (ok ? row - tok * grp : 0)) * D +
                            2 * (lane & 3);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        q[k][r] = ok ? __ldg(reinterpret_cast<const uint32_t*>(src + 16 * k))
                     : 0u;
        q[k][2 + r] =
            ok ? __ldg(reinterpret_cast<const uint32_t*>(src + 16 * k + 8))
               : 0u;
      }
    }
  }

  template <int WM>
  __device__ __forceinline__ Seg begin(const Cursor& cu) {
    Seg s;
    s.k1 = cu.E.k1;
    s.key = cu.E.k0 + cu.blk * kBN;
    s.prefix = cu.e < G;
    if (s.prefix) {
      s.lim[0] = s.lim[1] = s.lim_min = s.k1;
    } else {
      // the last token's rows see all of k1; each token before one fewer
      const int grp = a.p.Hq / a.p.Hkv, n = cu.E.rows / grp;
      const int r0 = (cu.u / a.p.Hkv) * 16 * WM;
      const int lane = threadIdx.x & 31, wm = (threadIdx.x >> 5) % WM;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        s.lim[i] = s.k1 - (n - 1) +
                   min((r0 + wm * 16 + (lane >> 2) + 8 * i) / grp, n - 1);
      s.lim_min = s.k1 - (n - 1) + min(r0 / grp, n - 1);
    }
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
    return s;
  }

  template <int WM>
  __device__ __forceinline__ void block(const Seg& sg, int st) {
    constexpr int WN = 4 / WM, NK = kBN / WN;   // keys a warp and block
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int wn = warp / WM;
    uint8_t* kt = smem + st * C::kStage;
    uint8_t* vt = kt + C::kTile;
    const int kb = sg.key;
    // ---- scores
    float s[NK / 8][4];
#pragma unroll
    for (int i = 0; i < NK / 8; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
#pragma unroll
      for (int i = 0; i < NK / 16; ++i) {
        uint32_t b[4];
        ldm4(s_addr(kt) + swz<D>(wn * NK + i * 16 + (lane & 7) +
                                     ((lane >> 4) << 3),
                                 2 * k + ((lane >> 3) & 1)),
             b);
        mma16816(s[2 * i], qf[k], b[0], b[1]);
        mma16816(s[2 * i + 1], qf[k], b[2], b[3]);
      }
    }
    const bool masked = kb + kBN > sg.lim_min;
#pragma unroll
    for (int i = 0; i < NK / 8; ++i) {
#pragma unroll
      for (int q = 0; q < 4; ++q) s[i][q] *= a.scale_log2;
      if (masked) {
        const int key = kb + wn * NK + i * 8 + 2 * (lane & 3);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (key + (q & 1) >= sg.lim[q >> 1]) s[i][q] = -INFINITY;
      }
    }
    // ---- running maximum and sum
    float mn[2] = {m[0], m[1]};
#pragma unroll
    for (int i = 0; i < NK / 8; ++i) {
      mn[0] = fmaxf(mn[0], fmaxf(s[i][0], s[i][1]));
      mn[1] = fmaxf(mn[1], fmaxf(s[i][2], s[i][3]));
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      mn[r] = fmaxf(mn[r], __shfl_xor_sync(0xffffffffu, mn[r], 1));
      mn[r] = fmaxf(mn[r], __shfl_xor_sync(0xffffffffu, mn[r], 2));
    }
    float base[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      // nothing seen yet: any finite base keeps every weight 0
      base[r] = mn[r] == -INFINITY ? 0.f : mn[r];
      const float f = ex2(m[r] - base[r]);
      m[r] = mn[r];
      l[r] *= f;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        o[i][2 * r] *= f;
        o[i][2 * r + 1] *= f;
      }
    }
    // Weights go to the product as bf16 (the type of V); the sum takes
    // them unrounded.  Each weight is off by at most 2^-8 of itself, and
    // independently, so the output's error stays about its own rounding.
    uint32_t pf[NK / 16][4];
#pragma unroll
    for (int i = 0; i < NK / 8; ++i) {
      const float p0 = ex2(s[i][0] - base[0]), p1 = ex2(s[i][1] - base[0]);
      const float p2 = ex2(s[i][2] - base[1]), p3 = ex2(s[i][3] - base[1]);
      l[0] += p0 + p1;
      l[1] += p2 + p3;
      pf[i / 2][(i & 1) * 2] = sv_pack(p0, p1);
      pf[i / 2][(i & 1) * 2 + 1] = sv_pack(p2, p3);
    }
    // A weight of 0 times an infinite or NaN value of V would spoil a row
    // that does not see that key.  Keys past k1 are zeros; in a block that
    // some rows see only in part, values that are not finite are taken out
    // of the tile and added, key by key, to the rows that do see them.  (One
    // row per tile's limit: a block whose only limit is k1 has none.)
    if (masked && !sg.prefix && sg.lim_min < sg.k1)
      fix_values<NK>(vt, kb, wn, sg.lim, pf);
    // ---- weighted values
#pragma unroll
    for (int i = 0; i < NK / 16; ++i) {
#pragma unroll
      for (int n = 0; n < D / 16; ++n) {
        uint32_t b[4];
        ldm4t(s_addr(vt) + swz<D>(wn * NK + i * 16 + (lane & 15),
                                  2 * n + (lane >> 4)),
              b);
        mma16816(o[2 * n], pf[i], b[0], b[1]);
        mma16816(o[2 * n + 1], pf[i], b[2], b[3]);
      }
    }
  }

  // The segment's result: its first `valid` rows to slot `slot` of the set.
  // st: a stage that this block has consumed.
  template <int WM>
  __device__ __forceinline__ void finish(const AttnSet& set, int64_t slot,
                                         int valid, int st) {
    constexpr int WN = 4 / WM, M = 16 * WM;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int wm = warp % WM, wn = warp / WM;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    }
    float* part = set.part + slot * M * D;
    float2* ml = set.ml + slot * M;
    if constexpr (WN == 1) {
      // rows of a warp are complete
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = wm * 16 + (lane >> 2) + 8 * r;
        if (row >= valid) continue;
        if ((lane & 3) == 0) ml[row] = make_float2(m[r], l[r]);
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
          *reinterpret_cast<float2*>(part + row * D + i * 8 + 2 * (lane & 3)) =
              make_float2(o[i][2 * r], o[i][2 * r + 1]);
      }
    } else {
      // ---- join the WN warps that share these rows
      if ((lane & 3) == 0)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = wm * 16 + (lane >> 2) + 8 * r;
          s_ml[wn * M + row][0] = m[r];
          s_ml[wn * M + row][1] = l[r];
        }
      __syncthreads();
      float* buf = reinterpret_cast<float*>(smem + st * C::kStage);
      float f[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = wm * 16 + (lane >> 2) + 8 * r;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < WN; ++w) top = fmaxf(top, s_ml[w * M + row][0]);
        f[r] = m[r] == -INFINITY ? 0.f : ex2(m[r] - top);
      }
      if (tid < valid && tid < M) {
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < WN; ++w) top = fmaxf(top, s_ml[w * M + tid][0]);
#pragma unroll
        for (int w = 0; w < WN; ++w) {
          const float mw = s_ml[w * M + tid][0];
          sum += mw == -INFINITY ? 0.f : s_ml[w * M + tid][1] * ex2(mw - top);
        }
        ml[tid] = make_float2(top, sum);
      }
      // kPass rows at a time: warps write them, all threads add them up
#pragma unroll
      for (int r0 = 0; r0 < M; r0 += C::kPass) {
        if (r0 >= valid) break;
        if (r0 > 0) __syncthreads();
#pragma unroll
        for (int r = 0; r < 2; ++r)
          if (wm * 16 + 8 * r == r0) {
            const int row = lane >> 2;
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
              *reinterpret_cast<float2*>(buf +
                                         (wn * C::kPass + row) * C::kPitch +
                                         i * 8 + 2 * (lane & 3)) =
                  make_float2(o[i][2 * r] * f[r], o[i][2 * r + 1] * f[r]);
          }
        __syncthreads();
        const int n = min(valid - r0, C::kPass);
        for (int i = tid; i < n * (D / 4); i += kNT) {
          const int row = i / (D / 4), c = i % (D / 4);
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < WN; ++w) {
            const float4 u = *reinterpret_cast<const float4*>(
                buf + (w * C::kPass + row) * C::kPitch + c * 4);
            v.x += u.x;
            v.y += u.y;
            v.z += u.z;
            v.w += u.w;
          }
          *reinterpret_cast<float4*>(part + (r0 + row) * D + c * 4) = v;
        }
      }
    }
  }

  template <int NK>
  __device__ void fix_values(uint8_t* vt, int kb, int wn, const int (&lim)[2],
                             const uint32_t (&pf)[NK / 16][4]) {
    const int tid = threadIdx.x, lane = tid & 31;
    if (tid < 2) s_bad[tid] = 0;
    __syncthreads();
    bool any = false;
    for (int i = tid; i < kBN * CH; i += kNT) {
      const int r = i / CH;
      const uint4 u = *reinterpret_cast<const uint4*>(vt + swz<D>(r, i % CH));
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
      bool bad = false;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        bad |= (w[q] & 0x7f80u) == 0x7f80u ||
               (w[q] & 0x7f800000u) == 0x7f800000u;
      if (bad) atomicOr(&s_bad[r >> 5], 1u << (r & 31));
      any |= bad;
    }
    if (!__syncthreads_or(any)) return;
    for (int k = 0; k < NK; ++k) {
      const int r = wn * NK + k;
      if (!((s_bad[r >> 5] >> (r & 31)) & 1u)) continue;
      // the weights of key k: held by lane (k % 8) / 2 of each quad
      uint32_t w0 = 0, w1 = 0;
#pragma unroll
      for (int i = 0; i < NK / 8; ++i)
        if (i == k / 8) {
          w0 = pf[i / 2][(i & 1) * 2];
          w1 = pf[i / 2][(i & 1) * 2 + 1];
        }
      const int src = (lane & ~3) | ((k & 7) >> 1);
      w0 = __shfl_sync(0xffffffffu, w0, src);
      w1 = __shfl_sync(0xffffffffu, w1, src);
      const float p[2] = {(k & 1) ? sv_hi(w0) : sv_lo(w0),
                          (k & 1) ? sv_hi(w1) : sv_lo(w1)};
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const uint32_t u = *reinterpret_cast<const uint32_t*>(
            vt + swz<D>(r, i) + 4 * (lane & 3));
        const float v[2] = {sv_lo(u), sv_hi(u)};
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (!isfinite(v[q & 1]) && kb + r < lim[q >> 1])
            o[i][q] += p[q >> 1] * v[q & 1];
      }
    }
    __syncthreads();
    for (int i = tid; i < kBN * CH; i += kNT) {
      uint32_t* w = reinterpret_cast<uint32_t*>(vt + swz<D>(i / CH, i % CH));
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t u = w[q];
        if ((u & 0x7f80u) == 0x7f80u) u &= 0xffff0000u;
        if ((u & 0x7f800000u) == 0x7f800000u) u &= 0xffffu;
        w[q] = u;
      }
    }
    __syncthreads();
  }
};

template <int D, int WMP, int WMO>
__global__ void __launch_bounds__(kNT, 2)
    attend_kernel(const __grid_constant__ AttendArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_ml[64][2];
  __shared__ uint32_t s_bad[2];
  // Behind the tensor-memory kernel (which has waited for everything before
  // it) nothing here depends on its results: start at once, and wait for it
  // at the end so that the merge, which waits for this kernel, has both.
  if (!a.tc) sv_grid_wait();
  sv_grid_launch();
  using A = Attend<D, WMP, WMO>;
  A t{a, smem, s_ml, s_bad, a.tc ? 0 : a.n_groups, 0};
  t.n_ent = t.G + a.p.batch;
  const PlanStart ps = plan_start<kNT, 16 * WMP, 16 * WMO, kBN>(
      t.G, t.n_ent, a.p.Hkv, [&](int i) { return t.ent(i); }, blockIdx.x,
      gridDim.x);
  if (ps.x0 < ps.x1) {
    Cursor c;                    // the block being computed
    c.e = ps.e;
    c.unit0 = ps.unit0;
    c.left = ps.x1 - ps.x0;
    t.enter(c);
    c.u = (int)(ps.off / c.nb);
    c.blk = (int)(ps.off - (int64_t)c.u * c.nb);
    Cursor f = c;                // the block to be copied next
    for (int s = 0; s < kStages - 1; ++s) {
      if (f.left > 0) {
        t.load(f, s);
        t.advance(f);
      }
      cp_commit();
    }
    if (c.e < t.G) t.template queries<WMP>(c, t.qf);
    else t.template queries<WMO>(c, t.qf);
    int64_t x = ps.x0;
    int st = 0;
    bool fresh = true;
    Seg sg;
    while (c.left > 0) {
      cp_wait<kStages - 2>();
      __syncthreads();
      if (f.left > 0) {
        t.load(f, st == 0 ? kStages - 1 : st - 1);
        t.advance(f);
      }
      cp_commit();
      const bool prefix = c.e < t.G;
      if (fresh) {
        sg = prefix ? t.template begin<WMP>(c) : t.template begin<WMO>(c);
        const AttnSet& set = prefix ? a.pre : a.own;
        if (c.unit0 + c.u >= set.units) {
          // q_start or group_start not ascending
          sv_latch(a.p.status, MPK_ERR_INVALID_ARG);
          break;
        }
        if (c.blk == 0 && threadIdx.x == 0) {
          const int last = plan_owner(x + c.nb - 1, ps.total, ps.n);
          set.meta[c.unit0 + c.u] = make_int2(
              c.unit0 + c.u + (int)blockIdx.x, last - (int)blockIdx.x + 1);
          if (c.u == 0) set.ebase[prefix ? c.e : c.e - t.G] = c.unit0 / a.p.Hkv;
        }
      }
      const int64_t slot = (int64_t)c.unit0 + c.u + blockIdx.x;
      const int tile = c.u / a.p.Hkv, rows = c.E.rows;
      const bool last = c.blk + 1 == c.nb || c.left == 1;
      t.advance(c);
      uint32_t qn[D / 16][4];
      if (last && c.left > 0) {
        if (c.e < t.G) t.template queries<WMP>(c, qn);
        else t.template queries<WMO>(c, qn);
      }
      if (prefix) {
        t.template block<WMP>(sg, st);
        if (last)
          t.template finish<WMP>(a.pre, slot, rows - tile * 16 * WMP, st);
      } else {
        t.template block<WMO>(sg, st);
        if (last)
          t.template finish<WMO>(a.own, slot, rows - tile * 16 * WMO, st);
      }
      if (last) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) t.qf[k][i] = qn[k][i];
      }
      fresh = last;
      sg.key += kBN;
      ++x;
      st = st + 1 == kStages ? 0 : st + 1;
    }
    cp_wait<0>();
  }
  if (a.tc) sv_grid_wait();
}

template <int D, int WMP, int WMO>
cudaError_t run_tiles(const AttendArgs& a, cudaStream_t s) {
  auto k = attend_kernel<D, WMP, WMO>;
  cudaError_t e = cudaFuncSetAttribute(
      k, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem);
  if (e != cudaSuccess) return e;
  return sv_launch(k, dim3(attend_ctas()), kNT, Cfg<D>::kSmem, s, true, a);
}

template <int D>
cudaError_t run_attend(const AttendArgs& a, cudaStream_t s) {
  if (a.wmo == 4) return run_tiles<D, 4, 4>(a, s);
  if (a.wmo == 2) return run_tiles<D, 4, 2>(a, s);
  if (a.wmp == 4) return run_tiles<D, 4, 1>(a, s);
  return run_tiles<D, 1, 1>(a, s);
}

}  // namespace
}  // namespace mpk
