// Attention over a shared prefix on the 5th-generation tensor cores.
//
// Many rows (all tokens of a group, all query heads of a KV head) meet the
// same keys, so a prefix is a dense product: S = Q K^T, P = e^(S - m),
// O += P V.  One persistent CTA an SM; a tile is two slots of 128 rows that
// share every K and V block of 128 keys.
//
//   warps 0-3, 4-7  slot 0, slot 1: a thread owns one row.  It loads its row
//                   of Q, reads its 128 scores from tensor memory, keeps the
//                   row's maximum and sum in registers, and writes the weights
//                   back to tensor memory as bf16 over the scores.
//   warp 8          page lookups and TMA loads of K and V (rings of 2).
//   warp 9          one thread issues tcgen05.mma: S_i = Q_i K^T (both from
//                   shared memory), O_i += P_i V (P from tensor memory).
//
// While one slot's softmax runs, the tensor core works for the other.  Tensor
// memory: S (and P) of the slots in columns 0 and 128, O in 256 and 384.
// O stays there over all key blocks.  It is rescaled only when a row's maximum
// has grown by more than 2^kSlack over the one its weights are taken to
// (their ratio cancels in O / l; 2^8 is far from any limit of fp32 or bf16), so
// nearly every block leaves it alone.
//
// Measured: 256 rows x 32 heads over a prefix of 16384 (8 KV heads of 128),
// 70 GFLOP, 68 us = 1.03 PFLOP/s.  A block of 256 x 128 takes 3520 cycles
// against 2050 of its products: softmax (1590), product and next scores of a
// slot follow one another, since weights and scores share their columns and
// the 512 are full.  (Blocks of 64 keys with two score buffers a slot: 93 us,
// the narrower products cost more than the wait.)
#include "attend_plan.cuh"

namespace mpk {
namespace {

constexpr int kThreadsT = 384;   // two softmax warpgroups, one for the rest
// Registers move from the third warpgroup to the softmax threads, which hold
// a row of 128 scores: 2 x 128 x 216 + 128 x 72 = 384 x 168, what the CTA is
// launched with.
constexpr int kSoftRegs = 216, kOtherRegs = 72;
constexpr int kRows = 256;        // rows of a tile
constexpr int kKeys = 128;        // keys of a block
constexpr float kSlack = 8.f;
constexpr uint64_t kDrainNs = 200000000ull;    // longest wait for copies at
                                               // the end

__device__ __forceinline__ void tc_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 "
      "[%0];" ::"r"(bar)
      : "memory");
}
// Shared-memory operands: 128-byte swizzled rows in 8-row groups 1024 bytes
// apart.  The upper word of the descriptor says that; the lower one has the
// address, and for an operand whose rows run along the product's inner
// dimension the distance of its 64-value column panels.
constexpr uint32_t kOperandHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t operand(uint32_t addr, uint32_t panel) {
  return ((addr & 0x3ffff) >> 4) | ((panel >> 4) << 16);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b,
                                       uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)acc), "r"(kOperandHi)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b,
                                       uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tmov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(
          d),
      "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)acc), "r"(kOperandHi)
      : "memory");
}
__device__ __forceinline__ void tm_ld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]),
        "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
        "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tm_ld16(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]),
        "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tm_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
      "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
      "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ void tm_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tm_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ float ex2t(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// bf16 x bf16 to fp32, M = 128
__device__ constexpr uint32_t product(int n, bool b_columns) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((b_columns ? 1u : 0u) << 16) |
         ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

template <int D>
struct TcSmem {
  static constexpr int kPanels = D / 64;
  static constexpr int kPanel = 128 * 128;             // 128 rows x 128 bytes
  static constexpr int kTile = kPanels * kPanel;
  static constexpr int kQ = 0;                         // [2] tiles
  static constexpr int kK = 2 * kTile;                 // [2]
  static constexpr int kV = 4 * kTile;                 // [2]
  // the output's staging area lies over Q: 8 warps x 32 rows x 36 floats
  static constexpr int kStage = 32 * 36 * 4;
  static constexpr int kOver = kTile >= 4 * kStage ? 0 : 1;
  static constexpr int kExtra = 6 * kTile;             // staging if Q is small
  static constexpr int kSmem =
      6 * kTile + (kOver ? 8 * kStage : 0) + 1024;     // + alignment
};

template <int D>
__global__ void __launch_bounds__(kThreadsT, 1)
    attend_tc(const __grid_constant__ AttendArgs a) {
  using L = TcSmem<D>;
  extern __shared__ uint8_t raw[];
  __shared__ __align__(8) uint64_t bars[20];
  __shared__ uint32_t s_tmem;
  __shared__ int s_dead;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = (t_addr(raw) + 1023u) & ~1023u;
  uint8_t* const smem = raw + (base - t_addr(raw));
  // full / empty of the K and V rings; per slot: Q loaded, scores ready,
  // weights ready, output complete; the copies of a prefix's last V block
  const uint32_t b0 = t_addr(bars);
  const uint32_t k_full = b0, k_empty = b0 + 16, v_full = b0 + 32,
                 v_empty = b0 + 48, q_full = b0 + 64, s_full = b0 + 80,
                 p_full = b0 + 96, o_full = b0 + 112, tail = b0 + 128;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      bar_init(k_full + 8 * i, 1);
      bar_init(k_empty + 8 * i, 1);
      bar_init(v_full + 8 * i, 1);
      bar_init(v_empty + 8 * i, 1);
      bar_init(s_full + 8 * i, 1);
      bar_init(p_full + 8 * i, 128);
      bar_init(o_full + 8 * i, 1);
      bar_init(q_full + 8 * i, 128);
    }
    bar_init(tail, 1);
    s_dead = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 8) {
    prefetch_map(&a.map_k);
    prefetch_map(&a.map_v);
    asm volatile(
        "tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::
            "r"(t_addr(&s_tmem))
        : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::
                     : "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tm = s_tmem;
  sv_grid_wait();
  // everything before this kernel is complete: the next one may start
  sv_grid_launch();
  const PagedArgs& p = a.p;
  const int box = a.box;
  const int Hkv = p.Hkv, grp = p.Hq / p.Hkv;
  const PlanStart st = plan_start<kThreadsT, kRows, kRows, kKeys, 1>(
      a.n_groups, a.n_groups, Hkv, [&](int g) { return att_group_ent(a, g); }, blockIdx.x,
      gridDim.x);
  volatile int* dead = &s_dead;

  // All roles walk the same segments.  f(E, tile, h, blk, n, slot, two):
  // `two`: the tile has rows in its second slot.  f returns false to stop.
  auto walk = [&](bool writes_meta, auto f) {
    int64_t left = st.x1 - st.x0;
    if (left <= 0) return;
    int e = st.e, unit0 = st.unit0;
    Ent E = att_group_ent(a, e);
    int nb = blocks_of<kKeys>(E);
    int u = (int)(st.off / nb), blk = (int)(st.off - (int64_t)u * nb);
    while (true) {
      const int unit = unit0 + u, tile = u / Hkv;
      const int n = (int)min((int64_t)(nb - blk), left);
      if (unit >= a.pre.units) {   // q_start or group_start not ascending
        sv_latch(p.status, MPK_ERR_INVALID_ARG);
        return;
      }
      if (writes_meta && blk == 0) {
        const int last = plan_owner(st.x1 - left + nb - 1, st.total, st.n);
        const int64_t at = meta_of(p, E.tok0, e, tile, a.pre.shift, u - tile * Hkv);
        if (at < a.pre.units)
          a.pre.meta[at] =
              make_int2(unit + (int)blockIdx.x, last - (int)blockIdx.x + 1);
      }
      if (!f(E, tile, u - tile * Hkv, blk, n, unit + (int)blockIdx.x,
             E.rows > tile * kRows + 128))
        return;
      left -= n;
      if (left <= 0) return;
      blk = 0;
      ++u;
      int units = (E.rows + kRows - 1) / kRows * Hkv;
      while (u >= units) {
        unit0 += units;
        if (++e >= a.n_groups) return;
        E = att_group_ent(a, e);
        nb = blocks_of<kKeys>(E);
        units = nb > 0 ? (E.rows + kRows - 1) / kRows * Hkv : 0;
        u = 0;
      }
    }
  };

  if (warp >= 8) {
    // (warps 10 and 11 fill up the warpgroup)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 8) {
    // ---------------------------------------------------------- loads
    int it = 0, sent[2] = {0, 0};
    uint32_t tail_ph = 0;
    walk(lane == 0, [&](const Ent& E, int, int h, int blk, int n, int,
                        bool) {
      const int32_t* pt = p.page_table + (int64_t)E.seq * p.max_pages;
      for (int j = 0; j < n; ++j, ++it) {
        const int st_ = it & 1;
        const uint32_t ph = (uint32_t)((it >> 1) & 1);
        const int key0 = (blk + j) * kKeys;
        // lane i finds the page of box i
        const int t = key0 + lane * box;
        int row = -1;
        if (lane < kKeys / box && t < E.k1) {
          const int pi = (int)sv_div(t, p.page_div);
          const int page = __ldg(pt + pi);
          if (page >= 0 && page < p.num_pages)
            row = (page * Hkv + h) * p.page_size + (t - pi * p.page_size);
          else
            sv_latch(p.status, MPK_ERR_KV_PAGE);
        }
        const int boxes = __popc(__ballot_sync(0xffffffffu, row >= 0));
        const uint32_t bytes = (uint32_t)boxes * box * D * 2;
        const bool last = key0 + kKeys > E.k1;
        for (int kv = 0; kv < 2; ++kv) {
          const uint32_t empty = (kv ? v_empty : k_empty) + 8 * st_;
          const uint32_t full = (kv ? v_full : k_full) + 8 * st_;
          const uint32_t dst =
              base + (kv ? L::kV : L::kK) + st_ * L::kTile;
          if (!bar_wait(empty, ph ^ 1u, dead)) return false;
          const bool fill = kv && last;
          const uint32_t bar = fill ? tail : full;
          if (lane == 0) bar_expect(bar, bytes);
          if (!fill) sent[kv] = it + 1;   // `full` will be reached
          __syncwarp();
          if (row >= 0)
#pragma unroll
            for (int q = 0; q < L::kPanels; ++q)
              tma_2d(dst + q * L::kPanel + lane * box * 128, kv ? &a.map_v : &a.map_k,
                     q * 64, row, bar);
          if (fill) {
            // values of keys past the end: zeros, because a weight of 0
            // times whatever the page holds there need not be 0
            if (!bar_wait(tail, tail_ph, dead)) return false;
            tail_ph ^= 1u;
            uint8_t* v = smem + L::kV + st_ * L::kTile;
            const int r0 = E.k1 - key0;
            for (int i = lane; i < (kKeys - r0) * 8; i += 32)
#pragma unroll
              for (int q = 0; q < L::kPanels; ++q)
                *reinterpret_cast<uint4*>(v + q * L::kPanel +
                                          (r0 + i / 8) * 128 + (i % 8) * 16) =
                    make_uint4(0, 0, 0, 0);
            fence_async();
            __syncwarp();
            if (lane == 0) bar_arrive(full);
            sent[kv] = it + 1;
          }
        }
      }
      return true;
    });
    // no copy may land after the CTA has left, nor the tensor core's arrivals
    // for the last two blocks
    int late = 0;
    for (int kv = 0; kv < 2; ++kv)
      for (int k = sent[kv] - 2; k < sent[kv]; ++k)
        if (k >= 0)
          bar_wait((kv ? v_full : k_full) + 8 * (k & 1), (k >> 1) & 1, &late,
                   kDrainNs);
    for (int k = it - 2; k < it; ++k)
      if (k >= 0 && !*dead) {
        bar_wait(k_empty + 8 * (k & 1), (k >> 1) & 1, dead);
        bar_wait(v_empty + 8 * (k & 1), (k >> 1) & 1, dead);
      }
    } else if (warp == 9) {
    // ------------------------------------------------------- products
    constexpr uint32_t iqk = product(kKeys, false), ipv = product(D, true);
    int it = 0;
    uint32_t pn[2] = {0, 0}, qn[2] = {0, 0};
    const uint32_t dq = operand(base + L::kQ, 16),
                   dk = operand(base + L::kK, 16),
                   dv = operand(base + L::kV, L::kPanel);
    constexpr uint32_t kTileD = L::kTile >> 4;
    auto qk = [&](int i, int stage) {
      if (lane == 0) {
        const uint32_t aq = dq + i * kTileD, ak = dk + stage * kTileD;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t o = ((k / 4) * L::kPanel + (k % 4) * 32) >> 4;
          mma_ss(tm + 128 * i, aq + o, ak + o, iqk, k > 0);
        }
        tc_commit(s_full + 8 * i);
      }
    };
    walk(false, [&](const Ent&, int, int, int, int n, int, bool two) {
      for (int i = 0; i < (two ? 2 : 1); ++i) {
        if (!bar_wait(q_full + 8 * i, qn[i] & 1, dead)) return false;
        ++qn[i];
      }
      if (!bar_wait(k_full + 8 * (it & 1), (it >> 1) & 1, dead)) return false;
      tc_after();
      qk(0, it & 1);
      if (two) qk(1, it & 1);
      if (lane == 0) tc_commit(k_empty + 8 * (it & 1));
      for (int j = 0; j < n; ++j, ++it) {
        const int sv = it & 1, sk = (it + 1) & 1;
        if (!bar_wait(v_full + 8 * sv, (it >> 1) & 1, dead)) return false;
        const bool more = j + 1 < n;
        if (more && !bar_wait(k_full + 8 * sk, ((it + 1) >> 1) & 1, dead))
          return false;
        for (int i = 0; i < (two ? 2 : 1); ++i) {
          if (!bar_wait(p_full + 8 * i, pn[i] & 1, dead)) return false;
          ++pn[i];
          tc_after();
          if (lane == 0) {
#pragma unroll
            for (int k = 0; k < kKeys / 16; ++k)
              mma_ts(tm + 256 + 128 * i, tm + 128 * i + 8 * k,
                     dv + sv * kTileD + (k * 2048 >> 4), ipv, j > 0 || k > 0);
            if (!more) tc_commit(o_full + 8 * i);
          }
          if (more) qk(i, sk);
        }
        if (lane == 0) {
          tc_commit(v_empty + 8 * sv);
          if (more) tc_commit(k_empty + 8 * sk);
        }
        __syncwarp();
      }
      return true;
    });
    }
  } else {
    // -------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    const int slot = warp >> 2, r = tid & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // 32 lanes a warp
    const uint32_t tS = tm + lanes + 128 * slot, tO = tS + 256;
    uint32_t sn = 0, on = 0;
    walk(false, [&](const Ent& E, int tile, int h, int blk, int n,
                    int part_slot, bool two) {
      if (slot == 1 && !two) return true;
      // the slot's rows of Q, swizzled as the tensor core expects: D / 8
      // neighbouring threads a row
      uint8_t* q = smem + L::kQ + slot * L::kTile;
#pragma unroll
      for (int k = 0; k < D / 8; ++k) {
        const int i = k * 128 + r, rr = i / (D / 8), c = i % (D / 8);
        const int row = tile * kRows + slot * 128 + rr;
        uint4 u = make_uint4(0, 0, 0, 0);
        if (row < E.rows) {
          const int tok = (int)sv_div(row, p.grp_div);
          u = __ldg(reinterpret_cast<const uint4*>(
              a.q + (E.tok0 + tok) * a.q_stride +
              (int64_t)(h * grp + row - tok * grp) * D + c * 8));
        }
        *reinterpret_cast<uint4*>(q + (c / 8) * L::kPanel + rr * 128 +
                                  (((c & 7) ^ (rr & 7)) << 4)) = u;
      }
      fence_async();
      bar_arrive(q_full + 8 * slot);
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j) {
        if (!bar_wait(s_full + 8 * slot, sn & 1, dead)) return false;
        ++sn;
        tc_after();
        // The row's 128 scores pass through 64 registers: the second half
        // first for its maximum, then the first half, whose weights are taken
        // while it is at hand, then the second half again.  (All 128 at once
        // spilled.)
        const int valid = E.k1 - (blk + j) * kKeys;
        uint32_t s0[32], s1[32];
        auto load = [&](int c) {
          tm_ld32(tS + 64 * c, s0);
          tm_ld32(tS + 64 * c + 32, s1);
        };
        auto mask = [&](uint32_t* s, int c) {
          if (valid < 32 * c + 32)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (32 * c + i >= valid) s[i] = 0xff800000u;
        };
        auto most = [&](const uint32_t* s, float t) {
#pragma unroll
          for (int i = 0; i < 32; i += 2)
            t = max3(t, __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
          return t;
        };
        load(1);
        tm_wait_ld();
        mask(s0, 2);
        mask(s1, 3);
        float t0 = most(s0, -INFINITY), t1 = most(s1, -INFINITY);
        load(0);
        tm_wait_ld();
        mask(s0, 0);
        mask(s1, 1);
        t0 = most(s0, t0);
        t1 = most(s1, t1);
        const float top = fmaxf(t0, t1) * a.scale_log2;
        const bool grow = top > m + kSlack || m == -INFINITY;
        if (__any_sync(0xffffffffu, grow)) {
          const float mn = grow ? fmaxf(m, top) : m;
          const float f = m == -INFINITY ? 0.f : ex2t(m - mn);
          l *= f;
          m = mn;
          if (j > 0) {
            // S of this block was committed behind the product before, so
            // O is at rest
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              uint32_t o[16];
              tm_ld16(tO + 16 * c, o);
              tm_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i)
                o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tm_st16(tO + 16 * c, o);
            }
          }
        }
        const float neg = m == -INFINITY ? 0.f : -m;
        const float2 neg2 = make_float2(neg, neg);
        const float2 sc2 = make_float2(a.scale_log2, a.scale_log2);
        float2 la = make_float2(0.f, 0.f), lb = la;
        auto weights = [&](const uint32_t* s, int c) {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            float2 x = __ffma2_rn(make_float2(__uint_as_float(s[2 * i]),
                                              __uint_as_float(s[2 * i + 1])),
                                  sc2, neg2);
            float2 y = __ffma2_rn(make_float2(__uint_as_float(s[2 * i + 2]),
                                              __uint_as_float(s[2 * i + 3])),
                                  sc2, neg2);
            x = make_float2(ex2t(x.x), ex2t(x.y));
            y = make_float2(ex2t(y.x), ex2t(y.y));
            la = __fadd2_rn(la, x);
            lb = __fadd2_rn(lb, y);
            // rounded to bf16 as in attend_kernel.cuh; the sum takes them
            // unrounded
            w[i] = sv_pack(x.x, x.y);
            w[i + 1] = sv_pack(y.x, y.y);
          }
          tm_st16(tS + 16 * c, w);
        };
        weights(s0, 0);
        weights(s1, 1);
        load(1);
        tm_wait_ld();
        mask(s0, 2);
        mask(s1, 3);
        weights(s0, 2);
        weights(s1, 3);
        l += (la.x + la.y) + (lb.x + lb.y);
        tm_wait_st();
        tc_before();
        bar_arrive(p_full + 8 * slot);
      }
      // ---- the segment's result
      if (!bar_wait(o_full + 8 * slot, on & 1, dead)) return false;
      ++on;
      tc_after();
      const int64_t at = (int64_t)part_slot * kRows + slot * 128;
      a.pre.ml[at + r] = make_float2(m, l);
      // through shared memory (over Q, which the products have finished
      // with), so that rows leave in whole lines
      float* out = a.pre.part + (at + (warp & 3) * 32) * D;
      float* stage = reinterpret_cast<float*>(
          smem + (L::kOver ? L::kExtra + warp * L::kStage
                           : L::kQ + slot * L::kTile + (warp & 3) * L::kStage));
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tm_ld32(tO + 32 * c, o);
        tm_wait_ld();
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<uint4*>(stage + lane * 36 + 4 * i) =
              make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int rr = i * 4 + (lane >> 3);
          *reinterpret_cast<float4*>(out + rr * D + 32 * c + 4 * (lane & 7)) =
              *reinterpret_cast<const float4*>(stage + rr * 36 +
                                               4 * (lane & 7));
        }
        __syncwarp();
      }
      tc_before();
      return true;
    });
  }
  __syncthreads();
  if (tid == 0 && s_dead) sv_latch(p.status, MPK_ERR_TIMEOUT);
  if (warp == 8) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(
        tm));
  }
}

template <int D>
cudaError_t tc_d(const AttendArgs& a, cudaStream_t s) {
  static SmemLimit limit;
  cudaError_t e = limit.set((const void*)attend_tc<D>, TcSmem<D>::kSmem);
  if (e != cudaSuccess) return e;
  return sv_launch(attend_tc<D>, dim3(attend_tc_ctas()), kThreadsT,
                   TcSmem<D>::kSmem, s, a);
}

}  // namespace

int attend_tc_ctas() { return 152; }
int attend_tc_rows() { return kRows; }

cudaError_t launch_attend_tc(const AttendArgs& a, cudaStream_t s) {
  return a.p.d == 128 ? tc_d<128>(a, s) : tc_d<64>(a, s);
}

}  // namespace mpk
