// How the attention kernels share out their work, worked out by every CTA
// from the device arrays (sequence lengths are not known to the host).
//
// Entities are the groups (a prefix and the rows of all its sequences) and
// then the sequences (own keys and own rows).  An entity's rows are cut into
// tiles of MP (groups) or MO (sequences), its keys into blocks of BN; a unit
// is one (row tile, KV head), numbered among the groups' or the sequences'.
// All blocks of all units form one line, of which every CTA takes an equal
// stretch: the load is even whatever the lengths are, and a long key axis is
// split when there are few rows.  A group's block takes W places of the line
// (what its larger row tile costs), and belongs to the CTA with its first.  A
// stretch of one unit's blocks is a segment; its partial result goes to slot
// (unit + CTA), which is unique because along the line either number grows
// from one segment to the next.  The unit's slots are consecutive, so the
// merge needs only the first and the count.  The plan takes 2 us of a call
// (one scan over the entities by all threads).
#pragma once

#include "serve_dev.cuh"

namespace mpk {

// ---- shared-memory barriers
__device__ __forceinline__ uint32_t t_addr(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}

// Longest wait of a role for another one of its CTA.
constexpr uint64_t kWaitNs = 2000000000ull;

__device__ __forceinline__ void bar_init(uint32_t b, uint32_t n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(b), "r"(n)
               : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(b) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(
                   b),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(b), "r"(parity)
      : "memory");
  return ok != 0;
}
// Waits for a phase, for two seconds at most; after that (or when another
// role has given up) false, and every role leaves its loop.
__device__ __forceinline__ bool bar_wait(uint32_t b, uint32_t parity,
                                         volatile int* dead,
                                         uint64_t limit = kWaitNs) {
  bool ok = bar_try(b, parity);
  if (!ok) {
    uint64_t t0, t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
    for (uint32_t i = 1; !ok; ++i) {
      ok = bar_try(b, parity);
      if (!ok && (i & 63u) == 0u) {
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
        if (*dead || t - t0 > limit) {
          *dead = 1;
          break;
        }
      }
    }
  }
  // a warp goes on, or leaves, as one
  return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map,
                                       int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ---- the plan
struct Ent {
  int tok0, rows;   // first token row, rows = tokens * query heads per KV head
  int k0, k1;       // keys
  int seq;          // whose page table row
};

__device__ __forceinline__ int att_ctx(const PagedArgs& p) {
  const int64_t c = (int64_t)p.max_pages * p.page_size;
  return c > 0x7fffffff ? 0x7fffffff : (int)c;
}
__device__ __forceinline__ int att_group(const AttendArgs& a, int b) {
  if (a.n_groups <= 1) return 0;
  int lo = 0, hi = a.n_groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(a.group_start + mid) <= b) lo = mid;
    else hi = mid;
  }
  return lo;
}
__device__ __forceinline__ int att_prefix(const AttendArgs& a, int g) {
  if (a.n_groups == 0) return 0;
  return min(max(__ldg(a.prefix_len + g), 0), att_ctx(a.p));
}
__device__ __forceinline__ Ent att_group_ent(const AttendArgs& a, int g) {
  const PagedArgs& p = a.p;
  Ent e;
  const int b0 = min(max(__ldg(a.group_start + g), 0), p.batch);
  const int b1 = min(max(__ldg(a.group_start + g + 1), b0), p.batch);
  e.tok0 = sv_row(p.q_start, p.tokens_per_seq, p.n_tokens, b0);
  const int t1 = sv_row(p.q_start, p.tokens_per_seq, p.n_tokens, b1);
  e.rows = max(t1 - e.tok0, 0) * (p.Hq / p.Hkv);
  e.k0 = 0;
  e.k1 = att_prefix(a, g);
  e.seq = min(b0, p.batch - 1);
  return e;
}
__device__ __forceinline__ Ent att_seq_ent(const AttendArgs& a, int b) {
  const PagedArgs& p = a.p;
  Ent e;
  e.tok0 = sv_row(p.q_start, p.tokens_per_seq, p.n_tokens, b);
  const int n =
      max(sv_row(p.q_start, p.tokens_per_seq, p.n_tokens, b + 1) - e.tok0, 0);
  e.rows = n * (p.Hq / p.Hkv);
  const int len = __ldg(p.seq_lens + b), g = att_group(a, b);
  e.k0 = att_prefix(a, g);
  if (a.n_groups > 0 && (__ldg(a.group_start + g) > b ||
                         __ldg(a.group_start + g + 1) <= b)) {
    // in no group: the groups do not go from 0 to the batch
    if (n > 0) sv_latch(p.status, MPK_ERR_INVALID_ARG);
    e.k0 = 0;
  }
  const int64_t end = (int64_t)len + n;
  const int ctx = att_ctx(p);
  e.k1 = end > ctx ? ctx : (int)end;
  e.seq = b;
  if (n > 0 && (end > ctx || len < 0)) sv_latch(p.status, MPK_ERR_KV_PAGE);
  // the prefix is read for every row of the group, so each sequence has to
  // hold all of it
  if (n > 0 && len < e.k0) {
    sv_latch(p.status, MPK_ERR_INVALID_ARG);
    e.k1 = e.k0;
  }
  if (e.k1 < e.k0) e.k1 = e.k0;
  return e;
}

// Blocks of an entity's keys; they begin at multiples of BN.
template <int BN>
__device__ __forceinline__ int blocks_of(const Ent& e) {
  return e.k1 > e.k0 ? (e.k1 + BN - 1) / BN - e.k0 / BN : 0;
}

// Where the segments of a unit are noted: a number that a row gives without
// looking anything up.  Tiles of entity e (of its kind) begin at row
// tok0 * heads of all rows; the entities' tiles do not meet because each
// entity adds one to the quotient.  Below rows / M + entities.
// (Rows of a KV head and entities times KV heads are below 2^30.)
__device__ __forceinline__ int64_t meta_of(const PagedArgs& p, int tok0, int e,
                                           int tile, int shift, int h) {
  return (int64_t)((tok0 * (p.Hq / p.Hkv) >> shift) + e + tile) * p.Hkv + h;
}

// Where a CTA starts on the line.
struct PlanStart {
  int64_t x0, x1;      // this CTA's stretch
  int64_t total;       // places of all units
  int64_t off;         // x0 within entity e, in places
  int unit0;           // units before entity e, of its kind
  int e;
  int n;               // CTAs that take part
};

// Finds the CTA's stretch with one scan over the entities (NT threads).
// Both passes of a batch of more than NT entities read the arrays again.
// `ent(e)` gives entity e; the first G are groups.
template <int NT, int MP, int MO, int BN, int W, typename F>
__device__ __forceinline__ PlanStart plan_start(int G, int n_ent, int Hkv,
                                                F ent, int cta, int n_cta) {
  __shared__ int64_t sh_cost[NT / 32], sh_unit[NT / 32];
  __shared__ int64_t sh_off, sh_base;
  __shared__ int sh_e;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto blocks = [&](int i, int64_t& cost, int64_t& unit) {
    cost = unit = 0;
    if (i < n_ent) {
      const Ent e = ent(i);
      const int64_t nb = blocks_of<BN>(e);
      const int64_t nt =
          i < G ? (e.rows + MP - 1) / MP : (e.rows + MO - 1) / MO;
      cost = nb * nt * Hkv * (i < G ? W : 1);
      // groups in the low half, sequences in the high half
      unit = nb > 0 ? nt * Hkv : 0;
      if (i >= G) unit <<= 32;
    }
  };
  // prefix sums over NT entities: this thread's (exclusive) and the sum
  auto scan = [&](int64_t& cost, int64_t& unit, int64_t& sum_c,
                  int64_t& sum_u) {
    int64_t ic = cost, iu = unit;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t vc = __shfl_up_sync(0xffffffffu, ic, o);
      const int64_t vu = __shfl_up_sync(0xffffffffu, iu, o);
      if (lane >= o) {
        ic += vc;
        iu += vu;
      }
    }
    if (lane == 31) {
      sh_cost[warp] = ic;
      sh_unit[warp] = iu;
    }
    __syncthreads();
    int64_t bc = 0, bu = 0;
    sum_c = sum_u = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
      const int64_t wc = sh_cost[w], wu = sh_unit[w];
      if (w < warp) {
        bc += wc;
        bu += wu;
      }
      sum_c += wc;
      sum_u += wu;
    }
    cost = bc + ic - cost;
    unit = bu + iu - unit;
  };
  if (tid == 0) sh_e = n_ent;
  int64_t cost, unit, bc, bu, total, units;
  blocks(tid, cost, unit);
  bc = cost;
  bu = unit;
  scan(bc, bu, total, units);
  int64_t more = 0;
  for (int i0 = NT; i0 < n_ent; i0 += NT) {
    int64_t c2, u2, s2, v2;
    blocks(i0 + tid, c2, u2);
    __syncthreads();
    scan(c2, u2, s2, v2);
    more += s2;
  }
  const int64_t first = total;   // of the first NT entities
  total += more;
  PlanStart st;
  st.total = total;
  // every CTA that takes part has a block, so a unit's segments belong to
  // consecutive CTAs
  st.n = total / W < n_cta ? max((int)(total / W), 1) : n_cta;
  if (total <= 0xffffffffll / (n_cta + 1)) {
    const uint32_t t = (uint32_t)total, n = (uint32_t)st.n;
    st.x0 = cta < st.n ? t * (uint32_t)cta / n : t;
    st.x1 = cta < st.n ? t * (uint32_t)(cta + 1) / n : t;
  } else {
    st.x0 = cta < st.n ? total * cta / st.n : total;
    st.x1 = cta < st.n ? total * (cta + 1) / st.n : total;
  }
  auto here = [&](int i, int64_t c, int64_t bc, int64_t bu) {
    if (c > 0 && st.x0 >= bc && st.x0 < bc + c) {
      sh_e = i;
      sh_off = st.x0 - bc;
      sh_base = bu;
    }
  };
  here(tid, cost, bc, bu);
  int64_t run_c = first, run_u = units;
  for (int i0 = NT; i0 < n_ent && run_c <= st.x0; i0 += NT) {
    int64_t c2, u2, s2, v2;
    blocks(i0 + tid, c2, u2);
    int64_t e2 = c2;
    __syncthreads();
    scan(e2, u2, s2, v2);
    here(i0 + tid, c2, run_c + e2, run_u + u2);
    run_c += s2;
    run_u += v2;
  }
  __syncthreads();
  st.e = sh_e;
  st.off = sh_off;
  st.unit0 = (int)(st.e < G ? sh_base : sh_base >> 32);
  return st;
}

// CTA that owns position x of the line.
__device__ __forceinline__ int plan_owner(int64_t x, int64_t total,
                                          int n_cta) {
  if (total <= 0xffffffffll / (n_cta + 1))
    return (int)(((uint32_t)(x + 1) * (uint32_t)n_cta - 1) / (uint32_t)total);
  return (int)(((x + 1) * n_cta - 1) / total);
}

}  // namespace mpk
