// Attention of new tokens over the paged cache with shared prefixes
// (mpk_prefix_attention): the general kernel and the merge.
//
// For a query row q of position t: o = sum_j p_j v_j, p_j = e^(s_j - M) / L,
// s_j = scale q.k_j over keys j <= t, with the running maximum M and sum L of
// a softmax in fp32.  The rows of a group (all tokens of its sequences, all
// query heads of a KV head) meet the prefix's keys together, so the prefix
// leaves HBM once; a sequence's own keys meet its own rows.  The two parts
// of a row, and the segments a long key axis is split into (attend_plan.cuh),
// are joined by their (M, L) in attend_merge.
//
// attend_kernel<D, WM>: 4 warps, row tile M = 16 WM, key blocks of 64 in a
// ring of kStages shared-memory stages filled with 16-byte asynchronous
// copies (any page size: every token finds its own page).  A warp holds 16
// rows and 64 / WN keys of a block, WN = 4 / WM; mma.sync m16n8k16, scores
// and weights stay in registers.  With few rows the warps split the keys, so
// the tensor instructions per key block stay few; the kernel is bound by the
// K/V bytes.
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

template <int D, int WM>
struct Cfg {
  static constexpr int WN = 4 / WM;
  static constexpr int M = 16 * WM;
  static constexpr int kTile = kBN * D * 2;            // bytes of K (or V)
  static constexpr int kQ = M * D * 2;
  static constexpr int kPitch = D + 4;                 // merge buffer, floats
  static constexpr int kMerge = WN > 1 ? WN * M * kPitch * 4 : 0;
  static constexpr int kRing = kStages * 2 * kTile;
  static constexpr int kSmem = kQ + (kRing > kMerge ? kRing : kMerge);
};

template <int D, int WM>
struct Body {
  using C = Cfg<D, WM>;
  static constexpr int WN = C::WN, M = C::M;
  static constexpr int CH = D / 8;                     // chunks a row
  static constexpr int NK = kBN / WN;                  // keys a warp and block
  static constexpr int RPT = kBN * CH / kNT;           // rows a thread loads
  static constexpr int RSTEP = kNT / CH;

  const AttendArgs& a;
  const AttnSet& set;
  uint8_t* smem;
  float (*s_ml)[2];   // [WN][M] of each warp
  uint32_t* s_bad;    // [2] keys of a block whose V is not finite

  // K and V of keys [key, key + 64) below k1 into stage st
  __device__ __forceinline__ void load(const Ent& e, int h, int key, int st) {
    const PagedArgs& p = a.p;
    const uint32_t ks = s_addr(smem + C::kQ + st * 2 * C::kTile);
    const int c = threadIdx.x % CH, r0 = threadIdx.x / CH;
    const int32_t* pt = p.page_table + (int64_t)e.seq * p.max_pages;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int r = r0 + i * RSTEP, t = key + r;
      bool ok = t < e.k1;
      int64_t off = 0;
      if (ok) {
        const int pi = (int)sv_div(t, p.page_div);
        const int page = __ldg(pt + pi);
        if (page < 0 || page >= p.num_pages) {
          sv_latch(p.status, MPK_ERR_KV_PAGE);
          ok = false;
        } else {
          off = (((int64_t)page * p.Hkv + h) * p.page_size +
                 (t - pi * p.page_size)) * D + c * 8;
        }
      }
      const uint32_t dst = ks + swz<D>(r, c);
      cp16(dst, p.k + off, ok ? 16 : 0);
      cp16(dst + C::kTile, p.v + off, ok ? 16 : 0);
    }
    cp_commit();
  }

  // One segment: blocks [blk, blk + nb) of unit (tile, h) of entity e.
  __device__ __forceinline__ void segment(const Ent& e, bool prefix, int tile,
                                          int h, int blk, int nb,
                                          int64_t slot) {
    const PagedArgs& p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int wm = warp % WM, wn = warp / WM;
    const int grp = p.Hq / p.Hkv;
    const int key0 = e.k0 + blk * kBN;
    // queries (rows past the entity's are zeros)
    for (int i = tid; i < M * CH; i += kNT) {
      const int r = i / CH, c = i % CH, row = tile * M + r;
      const bool ok = row < e.rows;
      const int tok = ok ? e.tok0 + row / grp : 0;
      const int hq = h * grp + (ok ? row % grp : 0);
      cp16(s_addr(smem) + swz<D>(r, c),
           a.q + tok * a.q_stride + (int64_t)hq * D + c * 8, ok ? 16 : 0);
    }
    cp_commit();
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) {
      if (s < nb) load(e, h, key0 + s * kBN, s);
      else cp_commit();
    }
    // keys each of this thread's two rows sees: [.., lim)
    int lim[2];
    int lim_min;
    if (prefix) {
      lim[0] = lim[1] = lim_min = e.k1;
    } else {
      // the last row sees all of k1; a row i tokens earlier i keys fewer
      const int n = e.rows / grp;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = tile * M + wm * 16 + (lane >> 2) + 8 * i;
        lim[i] = e.k1 - (n - 1) + min(row / grp, n - 1);
      }
      lim_min = e.k1 - (n - 1) + min(tile * M / grp, n - 1);
    }
    cp_wait<kStages - 1>();
    __syncthreads();
    uint32_t qf[D / 16][4];
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
      ldm4(s_addr(smem) + swz<D>(wm * 16 + (lane & 15), 2 * k + (lane >> 4)),
           qf[k]);
    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    for (int j = 0; j < nb; ++j) {
      cp_wait<kStages - 2>();
      __syncthreads();
      if (j + kStages - 1 < nb)
        load(e, h, key0 + (j + kStages - 1) * kBN, (j + kStages - 1) % kStages);
      else cp_commit();
      uint8_t* kt = smem + C::kQ + (j % kStages) * 2 * C::kTile;
      uint8_t* vt = kt + C::kTile;
      const int kb = key0 + j * kBN;
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
      const bool masked = kb + kBN > lim_min;
#pragma unroll
      for (int i = 0; i < NK / 8; ++i) {
#pragma unroll
        for (int q = 0; q < 4; ++q) s[i][q] *= a.scale_log2;
        if (masked) {
          const int key = kb + wn * NK + i * 8 + 2 * (lane & 3);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (key + (q & 1) >= lim[q >> 1]) s[i][q] = -INFINITY;
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
      // them unrounded.  Each weight is off by at most 2^-9 of itself, and
      // independently, so the output's error stays below its own rounding.
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
      // of the tile and added, key by key, to the rows that do see them.
      if (masked && !prefix) fix_values(vt, kb, wn, lim, pf, o);
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
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    }
    cp_wait<0>();
    __syncthreads();      // the ring is free
    float* part = set.part + slot * M * D;
    float2* ml = set.ml + slot * M;
    if (WN == 1) {
      // rows of a warp are complete
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = wm * 16 + (lane >> 2) + 8 * r;
        if ((lane & 3) == 0) ml[row] = make_float2(m[r], l[r]);
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
          *reinterpret_cast<float2*>(part + row * D + i * 8 + 2 * (lane & 3)) =
              make_float2(o[i][2 * r], o[i][2 * r + 1]);
      }
      return;
    }
    // ---- join the WN warps that share these rows
    if ((lane & 3) == 0)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = wm * 16 + (lane >> 2) + 8 * r;
        s_ml[wn * M + row][0] = m[r];
        s_ml[wn * M + row][1] = l[r];
      }
    __syncthreads();
    float* buf = reinterpret_cast<float*>(smem + C::kQ);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = wm * 16 + (lane >> 2) + 8 * r;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < WN; ++w) top = fmaxf(top, s_ml[w * M + row][0]);
      const float f = m[r] == -INFINITY ? 0.f : ex2(m[r] - top);
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        *reinterpret_cast<float2*>(buf + (wn * M + row) * C::kPitch + i * 8 +
                                   2 * (lane & 3)) =
            make_float2(o[i][2 * r] * f, o[i][2 * r + 1] * f);
    }
    __syncthreads();
    if (tid < M) {
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
    for (int i = tid; i < M * D / 4; i += kNT) {
      const int row = i / (D / 4), c = i % (D / 4);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < WN; ++w) {
        const float4 u = *reinterpret_cast<const float4*>(
            buf + (w * M + row) * C::kPitch + c * 4);
        v.x += u.x;
        v.y += u.y;
        v.z += u.z;
        v.w += u.w;
      }
      *reinterpret_cast<float4*>(part + row * D + c * 4) = v;
    }
    __syncthreads();      // buf before the next segment's copies
  }

  __device__ void fix_values(uint8_t* vt, int kb, int wn, const int (&lim)[2],
                             const uint32_t (&pf)[NK / 16][4],
                             float (&o)[D / 8][4]) {
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

// Entities of a launch: groups and sequences, or only one of the two.
enum { ENT_BOTH, ENT_GROUPS, ENT_SEQS };

template <int D, int WM>
__global__ void __launch_bounds__(kNT)
    attend_kernel(const __grid_constant__ AttendArgs a, int what) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int M = Cfg<D, WM>::M, WN = Cfg<D, WM>::WN;
  __shared__ float s_ml[WN * M][2];
  __shared__ uint32_t s_bad[2];
  // Behind a launch for the prefixes (which has waited for everything before
  // it) nothing here depends on its results: start at once, and wait for it
  // at the end so that the merge, which waits for this kernel, has both.
  if (what != ENT_SEQS || a.split == ATT_ONE) sv_grid_wait();
  sv_grid_launch();
  const int G = what == ENT_SEQS ? 0 : a.n_groups;
  const int n_ent = what == ENT_GROUPS ? G : G + a.p.batch;
  auto ent = [&](int i) {
    return i < G ? att_group_ent(a, i) : att_seq_ent(a, i - G);
  };
  const AttnSet& set = what == ENT_GROUPS ? a.pre : a.own;
  const int Hkv = a.p.Hkv;
  const PlanStart st =
      plan_start<kNT, M, kBN>(n_ent, Hkv, ent, blockIdx.x, gridDim.x);
  Body<D, WM> body{a, set, smem, s_ml, s_bad};
  int64_t x = st.x0, off = st.off, unit0 = st.unit0;
  int e = st.e;
  while (x < st.x1 && e < n_ent) {
    const Ent E = ent(e);
    const int nb = (E.k1 - E.k0 + kBN - 1) / kBN;
    const int64_t units = nb > 0 ? (int64_t)((E.rows + M - 1) / M) * Hkv : 0;
    while (x < st.x1 && off < units * nb) {
      const int u = (int)(off / nb), blk = (int)(off - (int64_t)u * nb);
      const int n = (int)min((int64_t)(nb - blk), st.x1 - x);
      const int64_t unit = unit0 + u;
      if (unit >= set.units) {   // q_start or group_start not ascending
        sv_latch(a.p.status, MPK_ERR_INVALID_ARG);
        off = units * nb;
        x = st.x1;
        break;
      }
      if (blk == 0 && threadIdx.x == 0) {
        const int last = plan_owner(x + nb - 1, st.total, st.n);
        set.meta[unit] =
            make_int2((int)(unit + blockIdx.x), last - (int)blockIdx.x + 1);
        if (u == 0) set.ebase[e] = (int)(unit0 / Hkv);
      }
      body.segment(E, e < G, u / Hkv, u % Hkv, blk, n, unit + blockIdx.x);
      x += n;
      off += n;
    }
    off = 0;
    unit0 += units;
    ++e;
  }
  if (what == ENT_SEQS && a.split != ATT_ONE) sv_grid_wait();
}

// One warp joins the segments of one (token, query head): the prefix's and
// the sequence's own.
template <int D>
__global__ void __launch_bounds__(kNT)
    attend_merge(const __grid_constant__ AttendArgs a) {
  constexpr int V = D / 32;
  const PagedArgs& p = a.p;
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * (kNT / 32) + (threadIdx.x >> 5);
  if (w >= (int64_t)p.n_tokens * p.Hq) return;
  const int t = (int)(w / p.Hq), hq = (int)(w - (int64_t)t * p.Hq);
  const int grp = p.Hq / p.Hkv, h = hq / grp, j = hq % grp;
  const int b = sv_seq_of(p.q_start, p.tokens_per_seq, p.batch, t);
  sv_grid_wait();
  if (b < 0) return;                     // behind the last sequence
  float m = -INFINITY, l = 0.f, acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
  auto take = [&](const AttnSet& s, int e, int tok0) {
    const int row = (t - tok0) * grp + j, r = row % s.M;
    const int64_t unit = ((int64_t)s.ebase[e] + row / s.M) * p.Hkv + h;
    if (row < 0 || unit < 0 || unit >= s.units) return;
    const int2 me = s.meta[unit];
    // (only arrays that are not ascending leave anything else here)
    if (me.x < 0 || me.y < 0 || me.y > s.slots - me.x) return;
    for (int i = 0; i < me.y; ++i) {
      const int64_t at = (int64_t)(me.x + i) * s.M + r;
      const float2 ml = s.ml[at];
      const float* src = s.part + at * D + lane * V;
      float v[V];
      if constexpr (V == 4) {
        const float4 u = *reinterpret_cast<const float4*>(src);
        v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
      } else if constexpr (V == 2) {
        const float2 u = *reinterpret_cast<const float2*>(src);
        v[0] = u.x; v[1] = u.y;
      } else {
        v[0] = *src;
      }
      if (ml.x == -INFINITY) continue;
      const float mn = fmaxf(m, ml.x);
      const float f = ex2(m - mn), g = ex2(ml.x - mn);
      m = mn;
      l = l * f + ml.y * g;
#pragma unroll
      for (int q = 0; q < V; ++q) acc[q] = acc[q] * f + v[q] * g;
    }
  };
  if (a.n_groups > 0) {
    const int g = att_group(a, b);
    const Ent e = att_group_ent(a, g);
    if (e.k1 > 0) take(a.pre, g, e.tok0);
  }
  const Ent e = att_seq_ent(a, b);
  if (e.k1 > e.k0)
    take(a.own, (a.split == ATT_ONE ? a.n_groups : 0) + b, e.tok0);
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
        l == 0.f ? -INFINITY
                 : (float)(((double)m + (double)log2f(l)) *
                           0.69314718055994530942);
}

int grid_ctas() { return 152 * 2; }

// Row tile for entities of `rows` rows: the smallest that holds them, at
// most 64.
int row_tile(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

template <int D, int WM>
cudaError_t run_m(const AttendArgs& a, int what, cudaStream_t s) {
  using C = Cfg<D, WM>;
  auto k = attend_kernel<D, WM>;
  cudaError_t e = cudaFuncSetAttribute(
      k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  return sv_launch(k, dim3(grid_ctas()), kNT, C::kSmem, s, true, a, what);
}
template <int D>
cudaError_t run(const AttendArgs& a, int M, int what, cudaStream_t s) {
  return M == 16   ? run_m<D, 1>(a, what, s)
         : M == 32 ? run_m<D, 2>(a, what, s)
                   : run_m<D, 4>(a, what, s);
}

template <int D>
cudaError_t attend_d(const AttendArgs& a, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (a.split == ATT_TC) e = launch_attend_tc(a, s);
  if (a.split == ATT_SPLIT) e = run<D>(a, a.pre.M, ENT_GROUPS, s);
  if (e != cudaSuccess) return e;
  e = run<D>(a, a.own.M, a.split == ATT_ONE ? ENT_BOTH : ENT_SEQS, s);
  if (e != cudaSuccess) return e;
  const int64_t warps = (int64_t)a.p.n_tokens * a.p.Hq;
  const int64_t blocks = (warps + kNT / 32 - 1) / (kNT / 32);
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  return sv_launch(attend_merge<D>, dim3((unsigned)blocks), kNT, 0, s, true,
                   a);
}

}  // namespace

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
  const int64_t all = a->n_groups ? rows / a->n_groups : 0;
  a->own.M = row_tile(per);
  a->split = ATT_ONE;
  if (a->n_groups && all > a->own.M) {
    a->split = ATT_SPLIT;
    a->pre.M = row_tile(all);
    if (attend_tc_box(a->p) && a->scale_log2 > 0.f) {
      a->split = ATT_TC;
      a->pre.M = attend_tc_rows();
    }
  }
  // a set holds the results of n entities whose rows are disjoint, `times`
  // over (each row is in one sequence's and at most one group's tiles)
  auto place = [&](AttnSet* s, int64_t n, int times, int ctas) {
    s->units = (times * (rows / s->M) + n) * a->p.Hkv;
    s->slots = s->units + ctas;
    s->ebase = reinterpret_cast<int32_t*>(take(n * 4));
    s->meta = reinterpret_cast<int2*>(take(s->units * 8));
    s->ml = reinterpret_cast<float2*>(take(s->slots * s->M * 8));
    s->part = reinterpret_cast<float*>(
        take((size_t)s->slots * s->M * a->p.d * 4));
  };
  if (a->split == ATT_ONE) {
    place(&a->own, a->p.batch + a->n_groups, a->n_groups ? 2 : 1, grid_ctas());
    a->pre = a->own;
  } else {
    place(&a->own, a->p.batch, 1, grid_ctas());
    place(&a->pre, a->n_groups, 1,
          a->split == ATT_TC ? attend_tc_ctas() : grid_ctas());
  }
  return off;
}

cudaError_t launch_attend(const AttendArgs& a, cudaStream_t s) {
  if (a.p.d == 128) return attend_d<128>(a, s);
  if (a.p.d == 64) return attend_d<64>(a, s);
  return attend_d<32>(a, s);
}

}  // namespace mpk
