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
// stay few; the kernel is bound by the K/V bytes.
// WM = 0 is a tile of 8 rows, one token's heads as a rule: the products are
// turned over (S^T = K Q^T, O^T = V^T P^T) so that the keys fill the 16 rows
// of the instruction and the queries its 8 columns.  That is half the tensor
// instructions, half the registers, and three or four CTAs an SM.
// A fifth warp walks the stretch ahead of them: it looks up the pages (one
// block early), copies K, V and the queries of a 16-row tile into a ring of
// kStages shared-memory stages, and leaves a description of the block there.
// Pages that are a multiple of 8 tokens come as TMA boxes (blocks begin at
// multiples of 64 keys, so that boxes do not cross pages), others key by key
// in 16-byte copies; the computing warps clear the values of keys outside the
// entity's.  These touch no list, table or length, and a stretch of many short
// sequences streams like one long one: the chain lengths -> pages -> keys that
// starts a sequence runs while earlier blocks are computed.
//
// Measured (head_dim 128, 32 / 8 heads): 256 sequences with 1..512 own keys,
// 269 MB, 53 us = 5.1 TB/s; 16 sequences of 1..2048 own keys behind a prefix
// of 2048, 79 MB, 22 us: there 5 us go into the plan and the first block's
// way, and 1100 to 1700 cycles a block are the chain of its instructions.
#pragma once

#include "attend_plan.cuh"

namespace mpk {
namespace {

constexpr int kNT = 160;       // four warps that compute, one that copies
constexpr int kComp = 128;
constexpr uint64_t kDrainNs = 200000000ull;   // for copies at the end
constexpr int kBN = 64;
constexpr float kSlack = 8.f;

// 16 bytes, or zeros when n == 0 (nothing is read then)
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
               "l"(src), "r"(n)
               : "memory");
}
// an arrival on `bar` once this thread's copies so far have landed
__device__ __forceinline__ void cp_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar)
               : "memory");
}
__device__ __forceinline__ void cp_wait_all() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}
__device__ __forceinline__ void sync_threads(int id, int n) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
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
// The 8 x 8 matrix of 16-bit values that the warp holds, turned over.
__device__ __forceinline__ uint32_t turn8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
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
// (rows of 128 values: two panels of 64).  These are the 64- and 128-byte
// swizzles of TMA.
template <int D, int ROWS>
__device__ __forceinline__ uint32_t swz(int r, int c) {
  if (D == 32) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  return (c >> 3) * (ROWS * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// What the copying warp says of the block in a stage.
struct Blk {
  int k0, k1;          // the unit's keys
  int key;             // first key of the block (a multiple of kBN)
  int tok0, rows;      // its entity's first token row and rows
  int tile, h;         // row tile, KV head
  int unit;
  int flags;           // BLK_*
};
enum {
  BLK_PREFIX = 1,
  BLK_FIRST = 2,       // of its segment
  BLK_LAST = 4,
  BLK_END = 8,         // last of the CTA's stretch
  BLK_STOP = 16        // bad arrays: no more blocks
};

__host__ __device__ constexpr int tile_rows(int wm) {
  return wm ? 16 * wm : 8;
}

// FEW: 8-row tiles alone.
template <int D, bool FEW = false>
struct Cfg {
  // CTAs an SM and stages a CTA: what the consumers' registers allow; the
  // stages fill the shared memory that they share.
  static constexpr int kCtas = FEW && D == 128 ? 3 : D == 128 ? 2 : 4;
  static constexpr int kStages = FEW && D == 128 ? 2 : D == 32 ? 4 : 3;
  static constexpr int kTile = kBN * D * 2;            // bytes of K (or V)
  static constexpr int kQ = 16 * D * 2;                // queries of 16 rows
  // (stages on 1024 bytes: the period of the swizzle)
  static constexpr int kStage = (2 * kTile + kQ + 1023) / 1024 * 1024;
  static constexpr int kSmem = kStages * kStage + 1024;
  static constexpr int CH = D / 8;                     // chunks a row
  static constexpr int kPitch = D + 4;                 // merge buffer, floats
  // rows that the merge of four key slices takes at a time (it lies over a
  // stage that has been consumed)
  static constexpr int kPass = 8;
  static_assert(4 * kPass * kPitch * 4 <= 2 * kTile, "merge buffer");
};

// A position on the CTA's stretch of the line.
struct Cursor {
  Ent E;
  int e, nb, units, u, blk, unit0;
  int64_t pos;         // its first place on the line
};

// Places of the line that a group's block takes: its time over that of a
// sequence's block (measured with a tile of 64 rows and one of 8 or 16:
// 3160 and 1100 cycles at head_dim 128, 2300 and 1200 at 64).
__host__ __device__ constexpr int block_places(int d, int wmp, int wmo) {
  return wmp == wmo ? 1 : wmo <= 1 && d == 128 ? 3 : 2;
}

// The copying warp.
template <int D, int WMP, int WMO>
struct Copier {
  using C = Cfg<D, WMP == 0>;
  static constexpr int CH = C::CH;
  const AttendArgs& a;
  uint8_t* smem;
  Blk* blk;
  uint32_t full, empty;
  volatile int* dead;
  int G, n_ent;
  static constexpr int W = block_places(D, WMP, WMO);

  __device__ __forceinline__ Ent ent(int i) const {
    return i < G ? att_group_ent(a, i) : att_seq_ent(a, i - G);
  }
  __device__ __forceinline__ void enter(Cursor& c) const {
    const int M = c.e < G ? tile_rows(WMP) : tile_rows(WMO);
    c.E = ent(c.e);
    c.nb = blocks_of<kBN>(c.E);
    c.units = c.nb > 0 ? ((c.E.rows + M - 1) / M) * a.p.Hkv : 0;
  }
  __device__ __forceinline__ void next_entity(Cursor& c) const {
    c.u = c.blk = 0;
    do {
      c.unit0 = c.e + 1 == G ? 0 : c.unit0 + c.units;
      if (++c.e >= n_ent) return;
      enter(c);
    } while (c.units == 0);
  }
  __device__ __forceinline__ void advance(Cursor& c, int64_t end) const {
    c.pos += c.e < G ? W : 1;
    if (++c.blk < c.nb) return;
    c.blk = 0;
    if (++c.u < c.units || c.pos >= end) return;
    next_entity(c);
  }
  __device__ __forceinline__ int first_key(const Cursor& c) const {
    return (c.E.k0 / kBN + c.blk) * kBN;
  }
  // Lane i looks up the pages of keys (boxes) i and i + 32 of the cursor's
  // block; -2 for those outside the entity's keys.
  __device__ __forceinline__ void pages(const Cursor& c, int (&pg)[2]) const {
    const int lane = threadIdx.x & 31;
    const int32_t* pt = a.p.page_table + (int64_t)c.E.seq * a.p.max_pages;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // with TMA, one lane a box
      const int t = first_key(c) + (lane + 32 * i) * (a.box ? a.box : 1);
      const int n = a.box ? a.box : 1;
      pg[i] = t + n > c.E.k0 && t < c.E.k1 && (lane + 32 * i) * n < kBN
                  ? __ldg(pt + sv_div(t, a.p.page_div))
                  : -2;
    }
  }

  __device__ __forceinline__ void run(const PlanStart& ps) {
    const PagedArgs& p = a.p;
    const int lane = threadIdx.x & 31;
    const int grp = p.Hq / p.Hkv;
    Cursor c;
    c.e = ps.e;
    c.unit0 = ps.unit0;
    enter(c);
    {
      // the first block that begins in the stretch
      const int w = c.e < G ? W : 1;
      const int64_t i = (ps.off + w - 1) / w;
      c.pos = ps.x0 - ps.off + i * w;
      c.u = (int)(i / c.nb);
      c.blk = (int)(i - (int64_t)c.u * c.nb);
      if (c.u >= c.units) next_entity(c);
    }
    int64_t sent = 0;
    const int64_t dv = reinterpret_cast<const char*>(p.v) -
                       reinterpret_cast<const char*>(p.k);
    const int ch = lane % CH, r0 = lane / CH;
    constexpr int RW = 32 / CH;                        // keys a step
    int pg[2];
    pages(c, pg);
    bool first = true;
    int st = 0;
    uint32_t ph = 1;
    for (bool end = false; !end; ++sent) {
      const bool prefix = c.e < G;
      const int wm = prefix ? WMP : WMO;
      Blk d;
      d.k0 = c.E.k0;
      d.k1 = c.E.k1;
      d.key = first_key(c);
      d.tok0 = c.E.tok0;
      d.rows = c.E.rows;
      d.tile = c.u / p.Hkv;
      d.h = c.u - d.tile * p.Hkv;
      d.unit = c.unit0 + c.u;
      const AttnSet& set = prefix ? a.pre : a.own;
      const bool stop = d.unit >= set.units;
      end = c.pos + (prefix ? W : 1) >= ps.x1;
      const bool last = c.blk + 1 == c.nb || end;
      d.flags = (end ? BLK_END : 0) | (prefix ? BLK_PREFIX : 0) |
                (first ? BLK_FIRST : 0) | (last ? BLK_LAST : 0) |
                (stop ? BLK_STOP : 0);
      // rows of the pool (32-bit numbers: 2^32 rows of 64 bytes are more
      // than the memory)
      uint32_t row[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = d.key + (lane + 32 * i) * (a.box ? a.box : 1);
        const bool ok = pg[i] >= 0 && pg[i] < p.num_pages;
        if (!ok && pg[i] != -2) sv_latch(p.status, MPK_ERR_KV_PAGE);
        row[i] = ok ? ((uint32_t)pg[i] * p.Hkv + d.h) * p.page_size +
                          (t - (int)sv_div(t, p.page_div) * p.page_size)
                    : 0xffffffffu;
      }
      // the next block's pages, on the way while this one waits for its stage
      const bool starts = c.blk == 0;
      const int ent_ = c.e, nb = c.nb;
      const int64_t pos = c.pos;
      if (!end) {
        advance(c, ps.x1);
        pages(c, pg);
      }
      if (!bar_wait(empty + 8 * st, ph, dead)) break;
      const uint32_t ks = t_addr(smem + st * C::kStage);
      if (a.box) {
        const bool ok = row[0] != 0xffffffffu;
        const uint32_t bytes =
            __popc(__ballot_sync(0xffffffffu, ok)) * a.box * D * 4;
        // (the bytes are announced first)
        if (lane == 0) {
          blk[st] = d;
          bar_expect(full + 8 * st, bytes);
        }
        __syncwarp();
        if (ok) {
          const uint32_t dst = ks + lane * a.box * (D < 64 ? 64 : 128);
#pragma unroll
          for (int q = 0; q < (D + 63) / 64; ++q) {
            tma_2d(dst + q * kBN * 128, &a.map_k, 64 * q, (int)row[0],
                   full + 8 * st);
            tma_2d(dst + C::kTile + q * kBN * 128, &a.map_v, 64 * q,
                   (int)row[0], full + 8 * st);
          }
        }
      } else {
        const char* kp = reinterpret_cast<const char*>(p.k) + ch * 16;
#pragma unroll 4
        for (int i = 0; i < kBN / RW; ++i) {
          const int r = r0 + i * RW;
          const uint32_t lo = __shfl_sync(0xffffffffu, row[0], r & 31);
          const uint32_t hi = __shfl_sync(0xffffffffu, row[1], r & 31);
          const uint32_t rr = r < 32 ? lo : hi;
          const bool ok = rr != 0xffffffffu;
          const char* src = kp + (uint64_t)(ok ? rr : 0u) * (D * 2);
          const uint32_t dst = ks + swz<D, kBN>(r, ch);
          cp16(dst, src, ok ? 16 : 0);
          cp16(dst + C::kTile, src + dv, ok ? 16 : 0);
        }
        if (lane == 0) {
          blk[st] = d;
          bar_arrive(full + 8 * st);
        }
      }
      if (first && wm <= 1 && !stop) {
#pragma unroll
        for (int i = 0; i < 16 / RW; ++i) {
          const int r = r0 + i * RW, rw = d.tile * tile_rows(wm) + r;
          if (wm == 0 && r >= 8) break;
          const bool ok = rw < d.rows;
          const int tok = ok ? (int)sv_div(rw, p.grp_div) : 0;
          cp16(ks + 2 * C::kTile + swz<D, 16>(r, ch),
               a.q + (d.tok0 + tok) * a.q_stride +
                   (int64_t)(d.h * grp + (ok ? rw - tok * grp : 0)) * D +
                   ch * 8,
               ok ? 16 : 0);
        }
      }
      cp_arrive(full + 8 * st);
      if (lane == 0 && starts && !stop) {
        const int to = plan_owner(pos + (int64_t)(nb - 1) * (prefix ? W : 1),
                                  ps.total, ps.n);
        const int64_t at = meta_of(p, d.tok0, prefix ? ent_ : ent_ - G, d.tile,
                                   set.shift, d.h);
        if (at < set.units)
          set.meta[at] =
              make_int2(d.unit + (int)blockIdx.x, to - (int)blockIdx.x + 1);
      }
      if (stop) {   // q_start or group_start not ascending
        sv_latch(p.status, MPK_ERR_INVALID_ARG);
        ++sent;
        break;
      }
      first = last;
      if (++st == C::kStages) {
        st = 0;
        ph ^= 1u;
      }
    }
    cp_wait_all();
    // no box may land after the CTA has left
    int late = 0;
    for (int64_t i = sent < C::kStages ? 0 : sent - C::kStages;
         a.box && i < sent; ++i)
      bar_wait(full + 8 * (int)(i % C::kStages),
               (uint32_t)(i / C::kStages) & 1u, &late, kDrainNs);
  }
};

// What the blocks of a segment need to know.
struct Seg {
  int k0, k1;          // the keys
  int lim[2], lim_min; // keys this thread's two rows see: [k0, lim)
  bool prefix;
};

// The warps that compute.
template <int D, bool FEW>
struct Attend {
  using C = Cfg<D, FEW>;
  static constexpr int CH = C::CH;

  const AttendArgs& a;
  uint8_t* smem;
  float (*s_ml)[2];    // [4 * 16] of each warp's rows

  // (a tile of 8 rows uses two words of each of qf and half of o, and its
  // thread's rows are 2 (lane % 4) and the next)
  uint32_t qf[D / 16][4];
  float o[D / 8][4];
  float m[2], l[2];

  // This thread's part of the queries of the block's unit, in the layout of
  // the product's first operand (rows past the entity's are zeros): from the
  // stage, or for a larger tile from memory.
  template <int WM>
  __device__ __forceinline__ void queries(const Blk& b, int st) {
    const int lane = threadIdx.x & 31;
    if constexpr (WM == 0) {
      const uint32_t q = t_addr(smem + st * C::kStage + 2 * C::kTile);
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        uint32_t b[4];
        ldm4(q + swz<D, 16>(lane & 7, 4 * k + (lane >> 3)), b);
        qf[2 * k][0] = b[0];
        qf[2 * k][1] = b[1];
        qf[2 * k + 1][0] = b[2];
        qf[2 * k + 1][1] = b[3];
      }
    } else if constexpr (WM == 1) {
      const uint32_t q = t_addr(smem + st * C::kStage + 2 * C::kTile);
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        ldm4(q + swz<D, 16>(lane & 15, 2 * k + (lane >> 4)), qf[k]);
    } else {
      const PagedArgs& p = a.p;
      const int wm = (threadIdx.x >> 5) % WM, grp = p.Hq / p.Hkv;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = b.tile * 16 * WM + wm * 16 + (lane >> 2) + 8 * r;
        const bool ok = row < b.rows;
        const int tok = ok ? (int)sv_div(row, p.grp_div) : 0;
        const int j = ok ? row - tok * grp : 0;
        const uint16_t* src = a.q + (b.tok0 + tok) * a.q_stride +
                              (int64_t)(b.h * grp + j) * D + 2 * (lane & 3);
        auto word = [&](int c) {
          return ok ? __ldg(reinterpret_cast<const uint32_t*>(src + c)) : 0u;
        };
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          qf[k][r] = word(16 * k);
          qf[k][2 + r] = word(16 * k + 8);
        }
      }
    }
  }

  template <int WM>
  __device__ __forceinline__ Seg begin(const Blk& b, int st) {
    queries<WM>(b, st);
    Seg s;
    s.k0 = b.k0;
    s.k1 = b.k1;
    s.prefix = b.flags & BLK_PREFIX;
    if (s.prefix) {
      s.lim[0] = s.lim[1] = s.lim_min = s.k1;
    } else {
      // the last token's rows see all of k1; each token before one fewer
      const int grp = a.p.Hq / a.p.Hkv, n = b.rows / grp;
      const int r0 = b.tile * tile_rows(WM);
      const int lane = threadIdx.x & 31;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = WM == 0 ? 2 * (lane & 3) + i
                              : (threadIdx.x >> 5) % (WM ? WM : 1) * 16 +
                                    (lane >> 2) + 8 * i;
        s.lim[i] = s.k1 - (n - 1) + min((r0 + r) / grp, n - 1);
      }
      s.lim_min = s.k1 - (n - 1) + min(r0 / grp, n - 1);
    }
#pragma unroll
    for (int i = 0; i < (WM == 0 ? D / 16 : D / 8); ++i)
      o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
    return s;
  }

  // The same for a tile of 8 rows; a warp has 16 keys.
  __device__ __forceinline__ void block8(const Seg& sg, int kb, int st) {
    const int lane = threadIdx.x & 31, wn = threadIdx.x >> 5;
    uint8_t* kt = smem + st * C::kStage;
    uint8_t* vt = kt + C::kTile;
    // ---- scores: s[2 i + r] is key lane / 4 + 8 i, row 2 (lane % 4) + r
    float s[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < D / 16; k += 2) {
      uint32_t b[4];
      ldm4(t_addr(kt) + swz<D, kBN>(wn * 16 + (lane & 15), 2 * k + (lane >> 4)),
           b);
      mma16816(s, b, qf[k][0], qf[k][1]);
      ldm4(t_addr(kt) +
               swz<D, kBN>(wn * 16 + (lane & 15), 2 * k + 2 + (lane >> 4)),
           b);
      mma16816(s2, b, qf[k + 1][0], qf[k + 1][1]);
    }
    const bool masked = kb + kBN > sg.lim_min || kb < sg.k0;
    const int key0 = kb + wn * 16 + (lane >> 2);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      s[q] = (s[q] + s2[q]) * a.scale_log2;
      const int key = key0 + 8 * (q >> 1);
      if (masked && (key >= sg.lim[q & 1] || key < sg.k0)) s[q] = -INFINITY;
    }
    // ---- running maximum and sum, as in block()
    float top[2] = {fmaxf(s[0], s[2]), fmaxf(s[1], s[3])};
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 4));
      top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 8));
      top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 16));
    }
    if (__any_sync(0xffffffffu,
                   top[0] > m[0] + kSlack || top[1] > m[1] + kSlack)) {
      float f[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float mn = fmaxf(m[r], top[r]);
        f[r] = mn == -INFINITY ? 1.f : ex2(m[r] - mn);
        m[r] = mn;
        l[r] *= f[r];
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) o[i][q] *= f[q & 1];
    }
    float w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      w[q] = ex2(s[q] - (m[q & 1] == -INFINITY ? 0.f : m[q & 1]));
    l[0] += w[0] + w[2];
    l[1] += w[1] + w[3];
    const uint32_t p0 = sv_pack(w[0], w[1]), p1 = sv_pack(w[2], w[3]);
    if (a.box && (kb < sg.k0 || kb + kBN > sg.k1))
      clear_values<0>(vt, sg.k0 - kb, sg.k1 - kb, wn);
    if (masked && !sg.prefix && sg.lim_min < sg.k1)
      fix_values8(vt, kb, wn, sg.lim, p0, p1);
    // ---- weighted values: rows and keys of the weights change places
    const uint32_t b0 = turn8(p0), b1 = turn8(p1);
#pragma unroll
    for (int n = 0; n < D / 16; ++n) {
      uint32_t b[4];
      ldm4t(t_addr(vt) + swz<D, kBN>(wn * 16 + (lane & 7) + ((lane >> 4) << 3),
                                     2 * n + ((lane >> 3) & 1)),
            b);
      mma16816(o[n], b, b0, b1);
    }
  }

  template <int WM>
  __device__ __forceinline__ void block(const Seg& sg, int kb, int st) {
    constexpr int WN = 4 / WM, NK = kBN / WN;   // keys a warp and block
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int wn = warp / WM;
    uint8_t* kt = smem + st * C::kStage;
    uint8_t* vt = kt + C::kTile;
    // ---- scores
    float s[NK / 8][4];
#pragma unroll
    for (int i = 0; i < NK / 8; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
#pragma unroll
      for (int i = 0; i < NK / 16; ++i) {
        uint32_t b[4];
        ldm4(t_addr(kt) + swz<D, kBN>(wn * NK + i * 16 + (lane & 7) +
                                     ((lane >> 4) << 3),
                                 2 * k + ((lane >> 3) & 1)),
             b);
        mma16816(s[2 * i], qf[k], b[0], b[1]);
        mma16816(s[2 * i + 1], qf[k], b[2], b[3]);
      }
    }
    const bool masked = kb + kBN > sg.lim_min || kb < sg.k0;
#pragma unroll
    for (int i = 0; i < NK / 8; ++i) {
#pragma unroll
      for (int q = 0; q < 4; ++q) s[i][q] *= a.scale_log2;
      if (masked) {
        const int key = kb + wn * NK + i * 8 + 2 * (lane & 3);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (key + (q & 1) >= sg.lim[q >> 1] || key + (q & 1) < sg.k0)
            s[i][q] = -INFINITY;
      }
    }
    // ---- running maximum and sum
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < NK / 8; ++i) {
      top[0] = fmaxf(top[0], fmaxf(s[i][0], s[i][1]));
      top[1] = fmaxf(top[1], fmaxf(s[i][2], s[i][3]));
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
      top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
    }
    // Weights are taken to a maximum that may lag behind by kSlack (their
    // ratio cancels in o / l, and 2^kSlack is far from any limit), so few
    // blocks rescale.
    if (__any_sync(0xffffffffu,
                   top[0] > m[0] + kSlack || top[1] > m[1] + kSlack)) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float mn = fmaxf(m[r], top[r]);
        const float f = mn == -INFINITY ? 1.f : ex2(m[r] - mn);
        m[r] = mn;
        l[r] *= f;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          o[i][2 * r] *= f;
          o[i][2 * r + 1] *= f;
        }
      }
    }
    // nothing seen yet: any finite base keeps every weight 0
    const float base[2] = {m[0] == -INFINITY ? 0.f : m[0],
                           m[1] == -INFINITY ? 0.f : m[1]};
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
    // that does not see that key.  Values of keys outside [k0, k1) become
    // zeros; in a block that some rows see only in part, values that are not
    // finite are taken out of the tile and added, key by key, to the rows
    // that do see them.
    if (a.box && (kb < sg.k0 || kb + kBN > sg.k1))
      clear_values<WM>(vt, sg.k0 - kb, sg.k1 - kb, wn);
    if (masked && !sg.prefix && sg.lim_min < sg.k1)
      fix_values<WM>(vt, kb, wn, sg.lim, pf);
    // ---- weighted values
#pragma unroll
    for (int i = 0; i < NK / 16; ++i) {
#pragma unroll
      for (int n = 0; n < D / 16; ++n) {
        uint32_t b[4];
        ldm4t(t_addr(vt) + swz<D, kBN>(wn * NK + i * 16 + (lane & 15),
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
    constexpr int WN = WM ? 4 / (WM ? WM : 1) : 4, M = tile_rows(WM);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int wm = WM ? warp % (WM ? WM : 1) : 0;
    const int wn = WM ? warp / (WM ? WM : 1) : warp;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (WM) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      } else {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 4);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 8);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 16);
      }
    }
    // row of value r of m, l and (by halves) o, and the lanes that speak for it
    auto row_of = [&](int r) {
      return WM ? wm * 16 + (lane >> 2) + 8 * r : 2 * (lane & 3) + r;
    };
    const bool speaks = WM ? (lane & 3) == 0 : lane < 4;
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
      if (speaks)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = row_of(r);
          s_ml[wn * M + row][0] = m[r];
          s_ml[wn * M + row][1] = l[r];
        }
      sync_threads(1, kComp);
      float* buf = reinterpret_cast<float*>(smem + st * C::kStage);
      float f[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = row_of(r);
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
        if (r0 > 0) sync_threads(1, kComp);
        if (WM == 0) {
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              buf[(wn * C::kPass + 2 * (lane & 3) + (q & 1)) * C::kPitch +
                  i * 16 + (lane >> 2) + 8 * (q >> 1)] = o[i][q] * f[q & 1];
        }
#pragma unroll
        for (int r = 0; r < 2; ++r)
          if (WM > 0 && wm * 16 + 8 * r == r0) {
            const int row = lane >> 2;
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
              *reinterpret_cast<float2*>(buf +
                                         (wn * C::kPass + row) * C::kPitch +
                                         i * 8 + 2 * (lane & 3)) =
                  make_float2(o[i][2 * r] * f[r], o[i][2 * r + 1] * f[r]);
          }
        sync_threads(1, kComp);
        const int n = min(valid - r0, C::kPass);
        for (int i = tid; i < n * (D / 4); i += kComp) {
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
      fence_async();   // the buffer, before a box lands on it
    }
  }

  // Zeros for the keys of this warp's slice outside [lo, hi).
  template <int WM>
  __device__ __forceinline__ void clear_values(uint8_t* vt, int lo, int hi,
                                               int wn) {
    constexpr int W = WM ? WM : 1, NK = 16 * W;
    const int lane = threadIdx.x & 31, wm = (threadIdx.x >> 5) % W;
    for (int i = wm * 32 + lane; i < NK * CH; i += 32 * W) {
      const int r = wn * NK + i / CH;
      if (r < lo || r >= hi)
        *reinterpret_cast<uint4*>(vt + swz<D, kBN>(r, i % CH)) =
            make_uint4(0, 0, 0, 0);
    }
    if (WM > 1) sync_threads(2 + wn, 32 * WM);
    else __syncwarp();
    fence_async();     // before a box lands here again
  }

  // The 4 / WM slices of keys are private to the WM warps of a slice, which
  // meet at a barrier of their own.
  template <int WM>
  __device__ __forceinline__ void fix_values(uint8_t* vt, int kb, int wn,
                                          const int (&lim)[2],
                                          const uint32_t (&pf)[4 * WM / 4][4]) {
    constexpr int NK = 16 * WM;
    const int lane = threadIdx.x & 31;
    uint32_t bad[2] = {0, 0};    // keys of the slice with such a value
    find_bad<NK>(vt, wn, bad);
    if (!(bad[0] | bad[1])) return;
    for (int k = 0; k < NK; ++k) {
      const int r = wn * NK + k;
      if (!((bad[k >> 5] >> (k & 31)) & 1u)) continue;
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
            vt + swz<D, kBN>(r, i) + 4 * (lane & 3));
        const float v[2] = {sv_lo(u), sv_hi(u)};
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (!isfinite(v[q & 1]) && kb + r < lim[q >> 1])
            o[i][q] += p[q >> 1] * v[q & 1];
      }
    }
    if (WM > 1) sync_threads(2 + wn, 32 * WM);
    else __syncwarp();
    drop_bad<NK>(vt, wn);
    if (WM > 1) sync_threads(2 + wn, 32 * WM);
    else __syncwarp();
    fence_async();
  }
  // Tile of 8 rows: p0, p1 hold the weights of keys lane / 4 and + 8.
  __device__ __forceinline__ void fix_values8(uint8_t* vt, int kb, int wn,
                                              const int (&lim)[2], uint32_t p0,
                                              uint32_t p1) {
    const int lane = threadIdx.x & 31;
    uint32_t bad[2] = {0, 0};
    find_bad<16>(vt, wn, bad);
    if (!bad[0]) return;
    for (int k = 0; k < 16; ++k) {
      const int r = wn * 16 + k;
      if (!((bad[0] >> k) & 1u)) continue;
      const uint32_t w = __shfl_sync(0xffffffffu, k < 8 ? p0 : p1,
                                     ((k & 7) << 2) | (lane & 3));
      const float p[2] = {sv_lo(w), sv_hi(w)};
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int c = i * 16 + (lane >> 2) + 8 * (q >> 1);
          const float v = sv_lo(*reinterpret_cast<const uint16_t*>(
              vt + swz<D, kBN>(r, c / 8) + 2 * (c % 8)));
          if (!isfinite(v) && kb + r < lim[q & 1]) o[i][q] += p[q & 1] * v;
        }
    }
    __syncwarp();
    drop_bad<16>(vt, wn);
    __syncwarp();
    fence_async();
  }
  // Keys of slice wn with a value that is not finite.
  template <int NK>
  __device__ __forceinline__ void find_bad(const uint8_t* vt, int wn,
                                           uint32_t (&bad)[2]) {
    for (int i = threadIdx.x & 31; i < NK * CH; i += 32) {
      const int k = i / CH;
      const uint4 u = *reinterpret_cast<const uint4*>(
          vt + swz<D, kBN>(wn * NK + k, i % CH));
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
      bool b = false;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        b |= (w[q] & 0x7f80u) == 0x7f80u ||
             (w[q] & 0x7f800000u) == 0x7f800000u;
      if (b) bad[k >> 5] |= 1u << (k & 31);
    }
    bad[0] = __reduce_or_sync(0xffffffffu, bad[0]);
    bad[1] = __reduce_or_sync(0xffffffffu, bad[1]);
  }
  // Zeros in their places.
  template <int NK>
  __device__ __forceinline__ void drop_bad(uint8_t* vt, int wn) {
    for (int i = threadIdx.x & 31; i < NK * CH; i += 32) {
      uint32_t* w = reinterpret_cast<uint32_t*>(
          vt + swz<D, kBN>(wn * NK + i / CH, i % CH));
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t u = w[q];
        if ((u & 0x7f80u) == 0x7f80u) u &= 0xffff0000u;
        if ((u & 0x7f800000u) == 0x7f800000u) u &= 0xffffu;
        w[q] = u;
      }
    }
  }

  template <int WM>
  __device__ __forceinline__ void step(Seg& sg, const Blk& b,
                                       const AttnSet& set, int64_t slot,
                                       int st) {
    if (b.flags & BLK_FIRST) sg = begin<WM>(b, st);
    if constexpr (WM == 0) block8(sg, b.key, st);
    else block<WM>(sg, b.key, st);
    if (b.flags & BLK_LAST)
      finish<WM>(set, slot, b.rows - b.tile * tile_rows(WM), st);
  }

  // The whole stretch of n blocks.
  template <int WMP, int WMO>
  __device__ __forceinline__ void run(const Blk* blk, uint32_t full,
                                      uint32_t empty, volatile int* dead,
                                      bool starts_prefix) {
    int st = 0;
    uint32_t ph = 0;
    Seg sg;
    // A turn without a block while the first one is on its way: it brings the
    // loop's code into the instruction caches (a first block took 5000
    // cycles, the next ones 1100).  It reads whatever the stage holds and
    // writes nothing; begin() sets the state anew.
    bool warm = true;
    sg.k0 = 0;
    sg.k1 = sg.lim[0] = sg.lim[1] = sg.lim_min = 0x7fffffff;
    sg.prefix = true;
    m[0] = m[1] = l[0] = l[1] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) qf[i][0] = qf[i][1] = qf[i][2] = qf[i][3] = 0u;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    while (true) {
      Blk b;
      if (warm) {
        b.key = b.unit = b.rows = b.tile = 0;
        b.flags = starts_prefix ? BLK_PREFIX : 0;
      } else {
        if (!bar_wait(full + 8 * st, ph, dead)) return;
        b = blk[st];
        if (b.flags & BLK_STOP) return;
      }
      const bool prefix = b.flags & BLK_PREFIX;
      const AttnSet& set = prefix ? a.pre : a.own;
      const int64_t slot = (int64_t)b.unit + blockIdx.x;
      if (WMP != WMO && prefix) {
        if constexpr (WMP != WMO) step<WMP>(sg, b, set, slot, st);
      } else {
        step<WMO>(sg, b, set, slot, st);
      }
      if (warm) {
        warm = false;
        continue;
      }
      __syncwarp();
      if ((threadIdx.x & 31) == 0) bar_arrive(empty + 8 * st);
      if (b.flags & BLK_END) return;
      if (++st == C::kStages) {
        st = 0;
        ph ^= 1u;
      }
    }
  }
};

template <int D, int WMP, int WMO>
__global__ void __launch_bounds__(kNT, WMP > 1 ? 2 : Cfg<D, WMP == 0>::kCtas)
    attend_kernel(const __grid_constant__ AttendArgs a) {
  extern __shared__ uint8_t raw[];
  uint8_t* const smem = raw + (1024 - (t_addr(raw) & 1023)) % 1024;
  constexpr int kStages = Cfg<D, WMP == 0>::kStages;
  __shared__ float s_ml[64][2];
  __shared__ Blk s_blk[kStages];
  __shared__ __align__(8) uint64_t bars[2 * kStages];
  __shared__ int s_dead;
  const uint32_t full = t_addr(bars), empty = full + 8 * kStages;
  if (threadIdx.x == kComp && a.box) {
    prefetch_map(&a.map_k);
    prefetch_map(&a.map_v);
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      bar_init(full + 8 * i, 33);      // the copying lanes and one of them
      bar_init(empty + 8 * i, 4);      // the computing warps
    }
    s_dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // Behind the tensor-memory kernel (which has waited for everything before
  // it) nothing here depends on its results: start at once, and wait for it
  // at the end so that the merge, which waits for this kernel, has both.
  if (!a.tc) sv_grid_wait();
  sv_grid_launch();
  Copier<D, WMP, WMO> cp{a,     smem,    s_blk, full,
                         empty, &s_dead, a.tc ? 0 : a.n_groups, 0};
  cp.n_ent = cp.G + a.p.batch;
  // (its barriers also publish the initialisation above)
  const PlanStart ps = plan_start<kNT, tile_rows(WMP), tile_rows(WMO), kBN,
                                  block_places(D, WMP, WMO)>(
      cp.G, cp.n_ent, a.p.Hkv, [&](int i) { return cp.ent(i); }, blockIdx.x,
      gridDim.x);
  if (ps.x0 < ps.x1) {
    if (threadIdx.x >= kComp) {
      cp.run(ps);
    } else {
      Attend<D, WMP == 0> t{a, smem, s_ml};
      t.template run<WMP, WMO>(s_blk, full, empty, &s_dead, ps.e < cp.G);
    }
    __syncthreads();
    if (threadIdx.x == 0 && s_dead) sv_latch(a.p.status, MPK_ERR_TIMEOUT);
  }
  if (a.tc) sv_grid_wait();
}

template <int D, int WMP, int WMO>
cudaError_t run_tiles(const AttendArgs& a, cudaStream_t s) {
  using C = Cfg<D, WMP == 0>;
  auto k = attend_kernel<D, WMP, WMO>;
  static SmemLimit limit;
  cudaError_t e = limit.set((const void*)k, C::kSmem);
  if (e != cudaSuccess) return e;
  const int ctas = WMP > 1 ? 2 : C::kCtas;
  return sv_launch(k, dim3(attend_ctas() / 4 * ctas), kNT, C::kSmem, s, a);
}

template <int D>
cudaError_t run_attend(const AttendArgs& a, cudaStream_t s) {
  if (a.wmo == 4) return run_tiles<D, 4, 4>(a, s);
  if (a.wmo == 2) return run_tiles<D, 4, 2>(a, s);
  if (a.wmo == 1 && a.wmp == 4) return run_tiles<D, 4, 1>(a, s);
  if (a.wmo == 1) return run_tiles<D, 1, 1>(a, s);
  if (a.wmp == 4) return run_tiles<D, 4, 0>(a, s);
  return run_tiles<D, 0, 0>(a, s);
}

}  // namespace
}  // namespace mpk
