// Causal attention over packed sequences with grouped heads on tcgen05 tensor
// cores (sm_100a), head_dim 128, bf16 in / bf16 out, fp32 softmax.
//
// Sequence s has ql queries and kl keys; query i sees keys 0 .. kl - ql + i
// (keys before the first query are a cached prefix).  With
//   S = Q K^T scale,  m = max S,  P = 2^((S - m) log2 e),  O = P V / sum P
// over the visible keys, one pass over the keys keeps a running reference
// maximum and sum per row, rescaling O only when the maximum grows by more
// than 8 (base 2); the final division makes the result independent of it.
//
// Layout of the work.  The G = heads / kv_heads query heads that share a
// key/value head are packed into the rows of one 128-row tile: row r of a
// tile is head r mod G at query position p0 + r / G, so one load of K and V
// serves all of them and a short prompt still fills its tiles.  A tile
// holds P = 128 / G positions; rows past P G and past the sequence's last
// query are computed and dropped.  Two CTAs share an SM.
//
// Keys come in steps of 64.  S = Q K^T (both operands in shared memory), one
// thread per row takes the softmax, writes P as bf16 over S, and O += P V reads
// P from TMEM.  P is rounded to bf16 for the tensor core; the row sum adds the
// unrounded fp32 values.  A CTA's 256 TMEM columns are two slots for S and P
// and O, so S of the next step is there when a softmax ends, and the tensor
// core works through P V (i), S (i + 2) of one slot under the softmax of the
// other; K and V have two stages each, and S of the next query tile's first
// steps follows while this one's last softmax runs and O is divided and stored.
// (Steps of 128 keys leave room for one S, so that every softmax waits for P V
// and S, and compute more that the causal cut drops: 24 ragged prompts, 8500
// tokens, 59 us against 52.5; 32 prompts of 128 tokens 23 against 21.4; 4096
// tokens the same 135.)
//
// What bounds it: the base-2 exponentials (16 a clock per SM) and the tensor
// core are each busy half the time, between the dependent steps of four softmax
// warps per CTA.  16384 tokens take 1.98 ms, 1.11 PFLOP/s, at 1.8 GHz; over
// seconds the power limit holds the clock at 1.62 GHz (2.29 ms).
//
// The last step is cut to the keys that some row sees (in steps of 16 for the MMAs, 32 for the softmax).
//
// Rows that a sequence does not own: the last step may reach into the
// next sequence or into rows of a cache that were never written.  Their
// scores are masked, and their V rows, whose weight is 0 but whose values may
// be infinite or NaN, are kept out of the product: P V runs over the 16-key
// steps that hold a visible key, and the softmax warps clear the rows between
// the last visible key and the end of its step.
//
// Few rows (single tokens: ql G <= AT_MAX_ROWS) leave such a tile almost empty
// and are bound by reading the keys once; they run in a second kernel that
// feeds warp-level MMAs straight from memory (ap_token_kernel).
//
// Few rows and many keys: the key range of a tile is split over nsp CTAs,
// which write unnormalised O, maximum and sum to scratch; a third kernel
// joins them in a fixed order.
#include <string.h>

#include <algorithm>
#include <atomic>
#include <vector>

#include "qi_common.cuh"
#include "qi_internal.h"
#include "qi_tc.cuh"

namespace qi {

constexpr int AP_ROWS = 128;
constexpr int AP_THREADS = 192;   // 4 softmax warps, TMA, MMA
constexpr int AP_KEYS = 64;        // keys of a step
constexpr int AP_TILE = 128 * 128 * 2;
constexpr int AP_HALF = 128 * 128;          // bytes of 64 columns of the Q tile
constexpr int AP_STEP = AP_KEYS * 128 * 2;  // bytes of K or V of a step
constexpr int AP_STEP_HALF = AP_KEYS * 128;
constexpr int AP_OUT = 32 * 64;   // bytes of a softmax warp's staged output: 32 rows x 32 columns
constexpr int AP_SMEM = AP_TILE + 4 * AP_STEP + 8 * AP_OUT + 128 + 512;   // Q, two stages of K and V, two of O per warp
static_assert(2 * (AP_SMEM + 1024) <= 233472, "two CTAs per SM");

// A kernel's parameters carry the plan.  Most tables are short, and a launch with
// 12 KB of parameters takes 1 us longer, so the kernels exist for two sizes.
using ApFewPlan = PackedTable<16, 64>;

template <class Plan>
struct ApKernelParams {
  Plan plan;
  const uint16_t* q;   // for the token kernel (the tile kernel reads it through a tensor map)
  int ldq;
  uint16_t* o;
  int ldo, kv_heads;
  int tma_out;       // tile kernel: the output map's box holds 32 rows of a tile
  int row_blocks;    // token kernel: 16-row blocks per unit
  float sm_scale;
  float* part_o;     // [slots][slot_rows][128]
  float* part_ml;    // [slots][slot_rows][2]
  int* status;
};

// Unit -> (sequence, query tile, key/value head, key split).  Sequences are
// sorted by their number of units per head, E = query tiles x splits;
// level e takes unit e, counted from the sequence's end, of every sequence
// that has one, so long key ranges start first and the last CTAs are short.
struct ApUnit {
  int s, ct, h, j;
};
template <class Plan>
__host__ __device__ __forceinline__ int ap_tiles(const Plan& d, int s) {
  return (d.seq[s].ql + d.P - 1) / d.P;
}
template <class Plan>
__host__ __device__ __forceinline__ ApUnit ap_unit(const Plan& d, int kv_heads, int b) {
  if (d.n_order > 0) {
    const int i = b / kv_heads;
    ApUnit u;
    u.s = static_cast<int>(d.order[i] >> 24);
    u.ct = static_cast<int>(d.order[i] & 0xFFFFFFu);
    u.h = b - i * kv_heads;
    u.j = 0;
    return u;
  }
  // ustart falls with i: the levels shared by sequences 0..i begin at ustart[i]
  int lo = 0, hi = d.n_seqs - 1;
  while (lo < hi) {   // the first i whose levels begin at or before b
    const int mid = (lo + hi) >> 1;
    if (d.seq[mid].ustart <= b) hi = mid;
    else lo = mid + 1;
  }
  const int per_level = (lo + 1) * kv_heads;
  const int e0 = lo + 1 < d.n_seqs ? ap_tiles(d, lo + 1) * d.seq[lo + 1].nsp : 0;
  const int r = b - d.seq[lo].ustart;
  const int e = e0 + r / per_level, w = r % per_level;
  ApUnit u;
  u.s = w / kv_heads;
  u.h = w - u.s * kv_heads;
  const int nsp = d.seq[u.s].nsp;
  u.ct = ap_tiles(d, u.s) - 1 - e / nsp;
  u.j = e % nsp;
  return u;
}
template <class Plan>
__host__ __device__ __forceinline__ int ap_slot(const Plan& d, int kv_heads, int s, int ct, int h, int j) {
  return d.seq[s].sbase + (ct * d.seq[s].nsp + j) * kv_heads + h;
}

// Ask for a tile in L2.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y)
               : "memory");
}

// Unit number of a CTA's round: one of every gridDim.x, alternately from the
// front and the back of each round, so that longest-first order evens out.
__device__ __forceinline__ int ap_unit_of(int round) {
  const int n = static_cast<int>(gridDim.x), i = static_cast<int>(blockIdx.x);
  return round * n + ((round & 1) ? n - 1 - i : i);
}

// tmem_ld32 without the wait, and the wait that releases its registers: every
// use of the values comes after an asm statement that "changes" them, so none
// can be scheduled before the data has arrived.
__device__ __forceinline__ void tmem_ld32_start(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
               : "r"(taddr)
               : "memory");
}
template <bool WAIT>
__device__ __forceinline__ void tmem_ld32_ready(uint32_t (&r)[32]) {
  if (WAIT) asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]) :: "memory");
}

// 16 columns, loaded and waited for in one statement.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// Whether a phase is complete, without waiting.
__device__ __forceinline__ bool mbar_done(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// One arrival for the warp, after what all its lanes did before.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// A unit of the tile kernel: a query tile over steps [lo, lo + n) of the keys.
struct ApWork {
  ApUnit u;
  int lo, n;
  int tail;     // keys of the last of them that some row sees (AP_KEYS: all)
};
template <class Plan>
__device__ __forceinline__ ApWork ap_work(const Plan& d, int kv_heads, int b) {
  ApWork w;
  w.u = ap_unit(d, kv_heads, b);
  const PackedSeq& s = d.seq[w.u.s];
  const int end = max(0, s.kl - s.ql + min((w.u.ct + 1) * d.P, s.ql));   // keys that some row sees
  const int steps = (end + AP_KEYS - 1) / AP_KEYS;
  w.lo = 0;
  int hi = steps;
  if (s.nsp > 1) {
    w.lo = static_cast<int>(static_cast<long long>(steps) * w.u.j / s.nsp);
    hi = static_cast<int>(static_cast<long long>(steps) * (w.u.j + 1) / s.nsp);
  }
  w.n = hi - w.lo;
  w.tail = w.n > 0 && hi == steps ? end - (steps - 1) * AP_KEYS : AP_KEYS;
  if (w.n == 0) {   // no keys: one step that is masked throughout
    w.n = 1;
    w.tail = 0;
  }
  return w;
}

// The units of a CTA.  The grid has one CTA per unit, longest first; a running
// CTA takes the next one that has not started from the hardware (cluster launch
// control: it is cancelled and its number handed over), so that SMs which are
// done early go on.  The producer warp asks shortly before a unit's last loads
// (earlier, and long units would be handed to CTAs that still have long ones
// to finish), decodes the answer and puts it into a ring that every warp reads.  (A unit's reading warps are never
// further apart than the ring is long: a step's S, and so the loads behind it,
// waits for the P V two steps before.)
constexpr int AP_RING = 8;
constexpr int AP_AHEAD = 4;   // steps before the end of a unit's loads at which the next unit is asked for
struct ApRing {
  int4 unit[AP_RING];       // sequence | head << 8, query tile, steps (-1: behind the last), key split
  int2 range[AP_RING];      // first step, keys of the last
  uint4 answer;             // of the launch control
  uint64_t full[AP_RING], empty[AP_RING], asked;
};
static_assert(AP_MAX_SEQS <= 256, "sequence in 8 bits");
constexpr int AP_READERS = 5;   // the softmax warps and the MMA warp; the producer keeps its own order

__device__ __forceinline__ void ap_ask(ApRing* r) {
  mbar_expect_elect(&r->asked, 16);
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];\n\t}" ::"r"(
          smem_u32(&r->answer)),
      "r"(smem_u32(&r->asked))
      : "memory");
}
// The CTA that was handed over, or -1.
__device__ __forceinline__ int ap_answer(ApRing* r) {
  uint32_t got, x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 a;\n\t"
      "ld.shared.b128 a, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, a;\n\t}"
      : "=r"(got), "=r"(x)
      : "r"(smem_u32(&r->answer))
      : "memory");
  return got ? static_cast<int>(x) : -1;
}

// Unit k of the CTA into its place of the ring.
__device__ __forceinline__ void ap_publish(ApRing* r, int k, const ApWork& w, int lane) {
  if (lane == 0) {
    r->unit[k % AP_RING] = make_int4(w.u.s | (w.u.h << 8), w.u.ct, w.n, w.u.j);
    r->range[k % AP_RING] = make_int2(w.lo, w.tail);
  }
  warp_arrive(&r->full[k % AP_RING], lane);
}
// Unit k of the CTA, once it is in the ring (every lane gets it).
__device__ __forceinline__ bool ap_read(ApRing* r, int k, ApWork* w, int* status) {
  if (!mbar_wait_warp(&r->full[k % AP_RING], (k / AP_RING) & 1, status)) return false;
  const int4 u = r->unit[k % AP_RING];
  const int2 t = r->range[k % AP_RING];
  w->u.s = u.x & 255;
  w->u.h = u.x >> 8;
  w->u.ct = u.y;
  w->n = u.z;
  w->u.j = u.w;
  w->lo = t.x;
  w->tail = t.y;
  return true;
}

// A place in the sequence of steps that a CTA's units make up; w.n < 0 behind
// the last (and after a wait that ran out).
struct ApCursor {
  ApWork w;
  int k, j;    // unit of the CTA, step of the unit
  __device__ __forceinline__ bool live() const { return w.n >= 0; }
};

template <class Plan>
__global__ void __launch_bounds__(AP_THREADS, 2)
    ap_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
              const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
              const __grid_constant__ ApKernelParams<Plan> p) {
  const Plan& d = p.plan;
  int* status = p.status;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {   // (two CTAs leave no room to align it by hand)
    if (threadIdx.x == 0) set_error(status, QI_DEV_ERR_BOUNDS);
    return;
  }
  uint8_t* sQ = smem;
  uint8_t* sK = smem + AP_TILE;          // [2][AP_STEP]
  uint8_t* sV = sK + 2 * AP_STEP;        // [2][AP_STEP]
  uint8_t* sO = sV + 2 * AP_STEP;        // [4 warps][2][AP_OUT]
  // step i uses stage, slot and barriers i & 1, their phase is i >> 1
  uint64_t* q_full = reinterpret_cast<uint64_t*>(sO + 8 * AP_OUT);
  uint64_t* k_full = q_full + 1;   // [2]
  uint64_t* v_full = q_full + 3;   // [2]
  uint64_t* s_full = q_full + 5;   // [2] S complete
  uint64_t* p_full = q_full + 7;   // [2] P written
  uint64_t* pv_full = q_full + 9;  // [2] P V complete
  uint64_t* drain = q_full + 11;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(q_full + 12);
  ApRing* ring = reinterpret_cast<ApRing*>(q_full + 16);
  static_assert(sizeof(ApRing) <= 512, "shared memory");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&v_full[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_full[i], 1);
    }
    mbar_init(drain, 1);
    for (int i = 0; i < AP_RING; ++i) {
      mbar_init(&ring->full[i], 1);
      mbar_init(&ring->empty[i], AP_READERS);
    }
    mbar_init(&ring->asked, 1);
    fence_mbar_init();
  }
  if (warp == 4 && lane == 0) {
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
    prefetch_tmap(&tmO);
  }
  if (warp == 5) {
    tmem_alloc(tmem_slot, 256);
    tmem_relinquish();
  }
  const int G = d.G, P = d.P;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  if (warp == 4) {   // the first unit, from the launch's arguments alone
    ap_publish(ring, 0, ap_work(d, p.kv_heads, static_cast<int>(blockIdx.x)), lane);
  }
  pdl_wait();
  pdl_trigger();

  if (warp == 4) {
    // ------------------------------------------------------------ TMA producer (the whole warp, one lane issues)
    bool ok = true;
    int units = 0, nk = 0, nv = 0;   // loads of Q, K and V asked for
    int known = 1;                   // units in the ring
    int asked = 0, answered = 0;     // questions to the launch control
    auto take = [&] {   // the answer into the ring
      if (!mbar_wait_warp(&ring->asked, answered & 1, status)) { ok = false; return; }
      ++answered;
      const int b = ap_answer(ring);
      fence_proxy_async_smem();   // read before it is written again
      __syncwarp();
      if (known >= AP_RING &&
          !mbar_wait_warp(&ring->empty[known % AP_RING], (known / AP_RING - 1) & 1, status)) {
        ok = false;
        return;
      }
      ApWork w{};
      w.n = -1;
      if (b >= 0) w = ap_work(d, p.kv_heads, b);
      ap_publish(ring, known++, w, lane);
    };
    auto unit = [&](ApCursor& c) {   // unit c.k, step 0
      c.j = 0;
      if (ok && c.k == known) take();
      if (!ok || !ap_read(ring, c.k, &c.w, status)) {
        ok = false;
        c.w.n = -1;
      }
    };
    auto advance = [&](ApCursor& c) {
      if (++c.j < c.w.n) return;
      ++c.k;
      unit(c);
    };
    ApCursor at{{}, 0, 0};     // the step whose S is waited for; K and V cursors run ahead
    unit(at);
    ApCursor kc = at, vc = at;
    auto load_q = [&](const ApWork& x) {
      // a box holds P positions x G heads x 64 head columns: rows in tile order
      mbar_expect_elect(q_full, static_cast<uint32_t>(P * G) * 128 * 2);
      for (int half = 0; half < 2; ++half)
        tma_load_3d_elect(&tmQ, smem_u32(q_full), sQ + half * AP_HALF, 64 * half, x.u.h * G,
                          d.seq[x.u.s].q0 + x.u.ct * P);
      ++units;
    };
    auto load = [&](const CUtensorMap* map, uint64_t* full, uint8_t* dst, ApCursor& c, int& n) {
      if (!c.live()) return;
      if (map == &tmK && asked == answered && c.k + 1 == known && c.w.n - c.j <= AP_AHEAD) {
        ap_ask(ring);
        ++asked;
      }
      const int st = n++ & 1;
      mbar_expect_elect(&full[st], AP_STEP);
      for (int half = 0; half < 2; ++half)
        tma_load_2d_elect<false>(map, smem_u32(&full[st]), dst + st * AP_STEP + half * AP_STEP_HALF,
                                 c.w.u.h * 128 + 64 * half, d.seq[c.w.u.s].k0 + (c.w.lo + c.j) * AP_KEYS);
      advance(c);
    };
    if (at.live()) load_q(at.w);
    for (int i = 0; i < 2; ++i) {
      load(&tmK, k_full, sK, kc, nk);
      load(&tmV, v_full, sV, vc, nv);
    }
    for (int i = 0; ok && at.live(); ++i) {
      // S(i) complete: its K stage is free, and Q after a unit's last S
      if (!mbar_wait_warp(&s_full[i & 1], (i >> 1) & 1, status)) { ok = false; break; }
      const bool last = at.j + 1 == at.w.n;
      advance(at);
      if (last && at.live()) load_q(at.w);
      load(&tmK, k_full, sK, kc, nk);
      if (i > 0 && vc.live()) {   // P V(i - 1) complete: its V stage is free
        if (!mbar_wait_warp(&pv_full[(i - 1) & 1], ((i - 1) >> 1) & 1, status)) { ok = false; break; }
        load(&tmV, v_full, sV, vc, nv);
      }
    }
    if (!ok) {   // bounded drain of what is on its way: the answer, the loads already armed
      auto landed = [&](uint64_t* bar, int n) {   // n phases
        const uint64_t t0 = globaltimer_ns();
        while (n > 0 && !mbar_try_wait(bar, (n - 1) & 1) && globaltimer_ns() - t0 < QI_WAIT_NS) {
        }
      };
      landed(&ring->asked, asked);
      landed(q_full, units);
      for (int st = 0; st < 2; ++st) {
        landed(&k_full[st], (nk + 1 - st) / 2);
        landed(&v_full[st], (nv + 1 - st) / 2);
      }
    }
  } else if (warp == 5) {
    // ------------------------------------------------------------ MMA issuer (the whole warp, one lane issues)
    constexpr uint32_t idesc_m = umma_idesc(false, 128, 0);
    constexpr uint32_t idesc_pv = umma_idesc(false, 128, 128) | (1u << 16);   // B MN-major
    const uint64_t qd = umma_desc_kmajor_sw128(smem_u32(sQ)), kd = umma_desc_kmajor_sw128(smem_u32(sK));
    const uint64_t vd = umma_desc_mnmajor_sw128(smem_u32(sV), AP_STEP_HALF);
    bool ok = true;
    int x = 0, i = 0, units = 0;   // next S, next P V, units whose Q has been used
    auto unit = [&](ApCursor& c, bool release) {
      c.j = 0;
      if (!ap_read(ring, c.k, &c.w, status)) {
        ok = false;
        c.w.n = -1;
      } else if (release) {
        warp_arrive(&ring->empty[c.k % AP_RING], lane);
      }
    };
    ApCursor pc{{}, 0, 0}, sc{{}, 0, 0};
    unit(sc, false);
    unit(pc, true);
    while (ok && pc.live()) {
      // S(x) goes into the slot of P V(x - 2), issued before it: the tensor core takes them in
      // order.  A unit's first S waits for Q, and lets the P V before it pass.
      if (sc.live() && x <= i + 1 &&
          (sc.j > 0 || x == i || __all_sync(0xffffffffu, mbar_done(q_full, units & 1)))) {
        if ((sc.j == 0 && !mbar_wait_warp(q_full, units & 1, status)) ||
            !mbar_wait_warp(&k_full[x & 1], (x >> 1) & 1, status)) { ok = false; break; }
        if (sc.j == 0) ++units;
        tc_fence_after();
        const uint32_t cols = sc.j == sc.w.n - 1 ? static_cast<uint32_t>(max(sc.w.tail, 1) + 15) / 16 * 16 : AP_KEYS;
        const uint32_t idesc = idesc_m | ((cols >> 3) << 17);
        const uint64_t ks = kd + static_cast<uint64_t>((x & 1) * AP_STEP >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          umma_f16_elect<false>(tmem_base + 64 * (x & 1),
                                qd + (static_cast<uint64_t>((kk >> 2) * AP_HALF + (kk & 3) * 32) >> 4),
                                ks + (static_cast<uint64_t>((kk >> 2) * AP_STEP_HALF + (kk & 3) * 32) >> 4), idesc,
                                kk > 0);
        umma_commit_elect<false>(&s_full[x & 1]);
        if (++sc.j == sc.w.n) {
          ++sc.k;
          unit(sc, false);
        }
        ++x;
        continue;
      }
      if (!mbar_wait_warp(&v_full[i & 1], (i >> 1) & 1, status) ||
          !mbar_wait_warp(&p_full[i & 1], (i >> 1) & 1, status)) { ok = false; break; }
      tc_fence_after();
      const int steps = pc.j == pc.w.n - 1 ? (pc.w.tail + 15) / 16 : AP_KEYS / 16;
      const uint64_t vs = vd + static_cast<uint64_t>((i & 1) * AP_STEP >> 4);
#pragma unroll
      for (int kk = 0; kk < AP_KEYS / 16; ++kk)   // 16 keys per instruction
        if (kk < steps)
          umma_f16_ts_elect(tmem_base + 128, tmem_base + 64 * (i & 1) + kk * 8, vs + static_cast<uint64_t>(kk * 2048 >> 4),
                            idesc_pv, (pc.j > 0 || kk > 0) ? 1u : 0u);
      umma_commit_elect<false>(&pv_full[i & 1]);
      if (++pc.j == pc.w.n) {
        ++pc.k;
        unit(pc, true);
      }
      ++i;
    }
    if (!ok) {   // no MMA may still run when TMEM is released
      umma_commit_elect<false>(drain);
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(drain, 0) && globaltimer_ns() - t0 < QI_WAIT_NS) {
      }
    }
  } else {
    // ------------------------------------------------------------ softmax + epilogue
    const int row = warp * 32 + lane;
    const uint32_t lane_bits = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t tO = tmem_base + lane_bits + 128;
    const int row_pos = row / G, row_head = row - row_pos * G;
    const float sl2 = p.sm_scale * 1.4426950408889634f;
    bool ok = true;
    int t = 0;   // steps of the units before this one
    for (int k = 0; ok; ++k) {
      ApWork w;
      if (!ap_read(ring, k, &w, status)) break;
      warp_arrive(&ring->empty[k % AP_RING], lane);
      if (w.n < 0) break;
      const PackedSeq& sq = d.seq[w.u.s];
      const int pos = w.u.ct * P + row_pos;           // query position of this row
      const bool live = row < P * G && pos < sq.ql;
      const int lim = live ? max(0, sq.kl - sq.ql + 1 + pos) : 0;   // keys this row sees
      // keys that every live row of this warp sees: steps below need no mask
      const int lim_min = __reduce_min_sync(0xffffffffu, live ? lim : 0x7fffffff);
      const bool warp_live = __any_sync(0xffffffffu, live);
      float m_ref = -INFINITY;   // reference maximum, base-2 scaled; -inf: no score yet
      float l = 0.f;
      for (int j = 0; j < w.n; ++j) {
        const int g = t + j, slot = g & 1;
        if (!mbar_wait_warp(&s_full[slot], (g >> 1) & 1, status)) { ok = false; break; }
        tc_fence_after();
        const uint32_t tS = tmem_base + lane_bits + 64 * slot;
        const int k0 = (w.lo + j) * AP_KEYS;
        const int ncols = j == w.n - 1 ? w.tail : AP_KEYS;   // the same for every row
        if (warp_live) {   // (otherwise: no query in these 32 rows, and whatever O gets is dropped)
          // columns past the cut are masked
          uint32_t r[2][32];
          tmem_ld32_start(tS, r[0]);
          tmem_ld32_start(tS + 32, r[1]);
          tmem_ld32_ready<true>(r[0]);
          tmem_ld32_ready<false>(r[1]);
          if (k0 + AP_KEYS > lim_min) {
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (k0 + i >= lim) r[i >> 5][i & 31] = __float_as_uint(-INFINITY);
          }
          float m8[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) m8[k] = fmaxf(__uint_as_float(r[0][2 * k]), __uint_as_float(r[0][2 * k + 1]));
#pragma unroll
          for (int i = 16; i < 64; i += 16)
#pragma unroll
            for (int k = 0; k < 8; ++k)
              m8[k] = fmax3(m8[k], __uint_as_float(r[i >> 5][(i & 31) + 2 * k]),
                            __uint_as_float(r[i >> 5][(i & 31) + 2 * k + 1]));
          float mx2 = fmax3(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7]));
          mx2 *= sl2;
          // the reference moves only when the maximum exceeds it by more than 8 (P <= 256)
          const float old = m_ref;
          if (mx2 > old + 8.0f || old == -INFINITY) m_ref = mx2;
          const bool grow = m_ref != old && old != -INFINITY;
          if (__any_sync(0xffffffffu, grow)) {
            const float f = grow ? exp2f(old - m_ref) : 1.0f;
            l *= f;
            // (a row that has a score to rescale: a step of this unit came before)
            if (!mbar_wait_warp(&pv_full[(g - 1) & 1], ((g - 1) >> 1) & 1, status)) { ok = false; break; }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t o[16];
              tmem_ld16(tO + c * 16, o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tmem_st16(tO + c * 16, o);
            }
            tmem_st_wait();
          }
          const float neg = m_ref == -INFINITY ? 0.f : -m_ref;
          const uint64_t sl2x2 = f2_pack(sl2, sl2);
          const uint64_t negm2 = f2_pack(neg, neg);
          uint64_t acc2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (32 * c >= ncols) continue;   // P V does not read further
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              uint32_t pk[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float s0 = __uint_as_float(r[c][16 * q + 2 * i]), s1 = __uint_as_float(r[c][16 * q + 2 * i + 1]);
                const uint64_t x2 = f2_fma(f2_pack(s0, s1), sl2x2, negm2);
                float x0, x1;
                f2_unpack(x2, x0, x1);
                const float e0 = ex2_approx(x0);
                const float e1 = ex2_approx(x1);
                acc2[i & 3] = f2_add(acc2[i & 3], f2_pack(e0, e1));
                pk[i] = pack_bf16x2(e0, e1);
              }
              tmem_st8(tS + c * 16 + q * 8, pk);
            }
          }
          float a0, a1, b0, b1;
          f2_unpack(f2_add(acc2[0], acc2[1]), a0, a1);
          f2_unpack(f2_add(acc2[2], acc2[3]), b0, b1);
          l += (a0 + b0) + (a1 + b1);
          tmem_st_wait();
        }
        if (ncols & 15) {
          // clear V from the last visible key to the end of its 16-key step (the swizzle permutes
          // inside a 128-byte row)
          if (!mbar_wait_warp(&v_full[slot], (g >> 1) & 1, status)) { ok = false; break; }
          const int n_clear = ((ncols + 15) & ~15) - ncols;
          for (int i = row; i < n_clear * 16; i += 128)
            *reinterpret_cast<uint4*>(sV + slot * AP_STEP + ((i >> 3) & 1) * AP_STEP_HALF + (ncols + (i >> 4)) * 128 +
                                      (i & 7) * 16) =
                make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
        }
        tc_fence_before();
        warp_arrive(&p_full[slot], lane);
      }
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (!mbar_wait_warp(&pv_full[(t + w.n - 1) & 1], ((t + w.n - 1) >> 1) & 1, status)) { ok = false; break; }
      tc_fence_after();
      // where this row goes: fp32 partial of the key range, or the output.  32 whole rows leave
      // through TMA, 32 columns at a time (a warp's own stores, 32 rows of 16 bytes each, keep the
      // load/store unit busy for 2000 clocks per tile); a cut tile, or a G that does not divide 32,
      // is stored row by row.
      const bool split = sq.nsp > 1;
      const float inv = l > 0.f ? __fdividef(1.0f, l) : 0.f;
      const uint64_t inv2 = f2_pack(inv, inv);
      const size_t at = split ? static_cast<size_t>(ap_slot(d, p.kv_heads, w.u.s, w.u.ct, w.u.h, w.u.j)) *
                                        d.slot_rows + row
                              : static_cast<size_t>(sq.q0 + pos) * p.ldo + (w.u.h * G + row_head) * 128;
      if (split && live) *reinterpret_cast<float2*>(p.part_ml + 2 * at) = make_float2(m_ref, l);
      if (warp_live) {   // (a range without a key has weight 0, whatever its O)
        const bool whole = !split && p.tma_out && __all_sync(0xffffffffu, live);
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t r[32];
          tmem_ld32(tO + 32 * c, r);
          if (split) {
            if (!live) continue;
            float4* dst = reinterpret_cast<float4*>(p.part_o + at * 128 + c * 32);
#pragma unroll
            for (int v = 0; v < 8; ++v)
              dst[v] = make_float4(__uint_as_float(r[4 * v]), __uint_as_float(r[4 * v + 1]),
                                   __uint_as_float(r[4 * v + 2]), __uint_as_float(r[4 * v + 3]));
            continue;
          }
          uint8_t* mine = sO + (warp * 2 + (c & 1)) * AP_OUT;
          if (whole) {   // the stage's last store has read it
            if (lane == 0) bulk_wait_group_read<1>();
            __syncwarp();
          }
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            uint32_t y[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float a, b;
              f2_unpack(f2_mul(f2_pack(__uint_as_float(r[8 * v + 2 * e]), __uint_as_float(r[8 * v + 2 * e + 1])), inv2), a, b);
              y[e] = lim == 0 ? 0u : pack_bf16x2(a, b);   // a row that sees no key: 0
            }
            const uint4 x = make_uint4(y[0], y[1], y[2], y[3]);
            // (the 64-byte swizzle: chunk v of row i at chunk v ^ (i / 2 mod 4))
            if (whole) *reinterpret_cast<uint4*>(mine + lane * 64 + ((v ^ ((lane >> 1) & 3)) << 4)) = x;
            else if (live) *reinterpret_cast<uint4*>(p.o + at + c * 32 + v * 8) = x;
          }
          if (whole) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_3d(&tmO, mine, 32 * c, w.u.h * G + (warp * 32) % G, sq.q0 + w.u.ct * P + warp * 32 / G);
              bulk_commit_group();
            }
          }
        }
      }
      t += w.n;
      tc_fence_before();   // O has been read before the next unit's P lets P V write it
    }
  }

  if (warp < 4 && lane == 0) bulk_wait_group_read<0>();   // the staged rows are read before the CTA leaves
  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 256);
  }
}

// ---------------------------------------------------------------- few rows
//
// A unit of work is 16 rows (query heads of one key/value head, at one or more
// positions) over a range of keys.  A producer thread streams the keys with
// TMA, 64 at a time, through a ring of stages deep enough to keep the memory
// busy (two CTAs per SM hold 192 KB in flight) and runs ahead into the CTA's
// next units; each of four warps takes 16 keys of a stage with its own
// running maximum, sum and O (m16n8k16 MMAs, K and V fragments by ldmatrix
// from the swizzled tile), and the warps are joined at the unit's end in
// shared memory.  A 128-row tcgen05 tile would be almost empty here, and its
// fixed steps (TMEM, the S / P round trip) longer than the loads.  Before it
// waits for the previous kernel of the stream, a CTA asks for the keys of its
// first unit in L2 (no value is read then, so nothing stale is seen).
constexpr int AT_WARPS = 4;
constexpr int AT_THREADS = 32 * (AT_WARPS + 1);
constexpr int AT_MAX_ROWS = 32;
constexpr int AT_KEYS = 64;                        // keys of a stage
constexpr int AT_STAGES = 3;
constexpr int AT_HALF = AT_KEYS * 128;             // bytes of one 64-column half of K or V
constexpr int AT_STAGE = 4 * AT_HALF;              // K | V, two halves each
constexpr int AT_SMEM = 1024 + AT_STAGES * AT_STAGE + 128;
static_assert(AT_WARPS * 16 == AT_KEYS, "a warp takes 16 keys of a stage");

__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Named barrier over the compute warps: plain, and with an AND of a predicate.
__device__ __forceinline__ void at_bar() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool at_all(bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 1, 128, p;\n\t"
      "selp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(pred))
      : "memory");
  return r != 0;
}

template <class Plan>
__global__ void __launch_bounds__(AT_THREADS, 2)
    ap_token_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const __grid_constant__ ApKernelParams<Plan> p) {
  const Plan& d = p.plan;
  int* status = p.status;
  __shared__ float s_ml[AT_WARPS][16][2];
  __shared__ float s_o[AT_WARPS][4][128];
  extern __shared__ uint8_t at_smem_raw[];
  const uint32_t raw_addr = smem_u32(at_smem_raw);
  uint8_t* smem = at_smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + AT_STAGES * AT_STAGE);   // [AT_STAGES]
  uint64_t* empty = full + AT_STAGES;                                          // [AT_STAGES]
  const int G = d.G, total = d.units * p.row_blocks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  if (threadIdx.x == 0) {
    for (int i = 0; i < AT_STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], AT_WARPS);
    }
    fence_mbar_init();
  }
  __syncthreads();

  struct Work {
    ApUnit u;
    int r0, rows, lo, hi;   // first of 16 rows, rows of the unit, 64-key steps
  };
  auto work_of = [&](int w) {
    Work x;
    x.u = ap_unit(d, p.kv_heads, w / p.row_blocks);
    x.r0 = w % p.row_blocks * 16;
    x.rows = d.seq[x.u.s].ql * G;
    const int nsp = d.seq[x.u.s].nsp, steps = x.r0 < x.rows ? (d.seq[x.u.s].kl + AT_KEYS - 1) / AT_KEYS : 0;
    x.lo = static_cast<int>(static_cast<long long>(steps) * x.u.j / nsp);
    x.hi = static_cast<int>(static_cast<long long>(steps) * (x.u.j + 1) / nsp);
    return x;
  };

  if (warp == AT_WARPS) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      prefetch_tmap(&tmK);
      prefetch_tmap(&tmV);
      if (ap_unit_of(0) < total) {
        const Work w = work_of(ap_unit_of(0));
        for (int st = w.lo; st < w.hi; ++st)
          for (int half = 0; half < 2; ++half) {
            tma_prefetch_2d(&tmK, w.u.h * 128 + 64 * half, d.seq[w.u.s].k0 + st * AT_KEYS);
            tma_prefetch_2d(&tmV, w.u.h * 128 + 64 * half, d.seq[w.u.s].k0 + st * AT_KEYS);
          }
      }
    }
    pdl_wait();
    pdl_trigger();
    if (lane == 0) {
      bool ok = true;
      int i = 0;   // steps loaded, over all units
      for (int round = 0; ok && ap_unit_of(round) < total; ++round) {
        const Work w = work_of(ap_unit_of(round));
        for (int st = w.lo; st < w.hi; ++st, ++i) {
          const int sl = i % AT_STAGES;
          if (!mbar_wait(&empty[sl], ((i / AT_STAGES) & 1) ^ 1u, status)) { ok = false; break; }
          mbar_arrive_expect_tx(&full[sl], AT_STAGE);
          uint8_t* dst = smem + sl * AT_STAGE;
          const int row = d.seq[w.u.s].k0 + st * AT_KEYS;
          for (int half = 0; half < 2; ++half) {
            tma_load_2d(&tmK, &full[sl], dst + half * AT_HALF, w.u.h * 128 + 64 * half, row);
            tma_load_2d(&tmV, &full[sl], dst + (2 + half) * AT_HALF, w.u.h * 128 + 64 * half, row);
          }
        }
      }
      if (!ok) {   // bounded drain of the loads already armed
        for (int k = max(0, i - AT_STAGES); k < i; ++k) {
          const uint64_t t0 = globaltimer_ns();
          while (!mbar_try_wait(&full[k % AT_STAGES], (k / AT_STAGES) & 1) && globaltimer_ns() - t0 < QI_WAIT_NS) {
          }
        }
      }
    }
    return;
  }

  // -------------------------------------------------------------- compute warps
  Work w = work_of(min(ap_unit_of(0), total - 1));
  pdl_wait();
  pdl_trigger();
  const float sl2 = p.sm_scale * 1.4426950408889634f;
  // ldmatrix row addresses: lane gives row (lane & 7) of matrix lane >> 3.
  // K: matrices (keys 0-7, 8-15) x (columns 0-7, 8-15 of a 16-column step)
  // V: matrices (keys 0-7, 8-15) x (two 8-column groups)
  const int mrow = warp * 16 + (lane & 7) + ((lane >> 3) & 1) * 8, mcol = lane >> 4;
  int i = 0;   // steps taken, over all units
  for (int round = 0; ap_unit_of(round) < total; ++round) {
    if (round > 0) w = work_of(ap_unit_of(round));
    const PackedSeq& sq = d.seq[w.u.s];
    const int ql = sq.ql, kl = sq.kl, nsp = sq.nsp, r0 = w.r0, rows = w.rows;
    if (r0 >= rows) continue;
    uint32_t qa[8][4];   // A fragments of 16 head columns each
    int lim[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = r0 + g + 8 * e;
      const bool live = r < rows;
      lim[e] = live ? max(0, kl - ql + r / G + 1) : 0;   // keys the row sees
      const uint16_t* row = p.q + static_cast<size_t>(sq.q0 + (live ? r / G : 0)) * p.ldq +
                            (w.u.h * G + r % G) * 128 + 2 * t;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        qa[kk][e] = live ? *reinterpret_cast<const uint32_t*>(row + 16 * kk) : 0u;
        qa[kk][2 + e] = live ? *reinterpret_cast<const uint32_t*>(row + 16 * kk + 8) : 0u;
      }
    }
    const int lim_min = max(0, kl - ql + r0 / G + 1);   // keys that every row sees
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};   // rows g, g + 8; m: base-2 scaled reference
    float o[16][4];   // head columns 8 c + 2 t, + 1 of rows g and g + 8
#pragma unroll
    for (int c = 0; c < 16; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[c][e] = 0.f;
    bool ok = true;
#pragma unroll 1
    for (int st = w.lo; st < w.hi; ++st, ++i) {
      const int sl = i % AT_STAGES;
      if (!mbar_wait_warp(&full[sl], (i / AT_STAGES) & 1, status)) { ok = false; break; }
      uint8_t* stage = smem + sl * AT_STAGE;
      const int key0 = st * AT_KEYS + warp * 16;
      if (key0 < kl) {
        if (key0 + 16 > kl) {
          // rows behind the last key: weight 0, but whatever they hold must not be multiplied
          for (int x = lane; x < (key0 + 16 - kl) * 16; x += 32)
            *reinterpret_cast<uint4*>(stage + (2 + ((x >> 3) & 1)) * AT_HALF + (kl - st * AT_KEYS + (x >> 4)) * 128 +
                                      (x & 7) * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();   // before TMA writes the stage again
          __syncwarp();
        }
        const uint32_t kbase = smem_u32(stage) + mrow * 128, vbase = kbase + 2 * AT_HALF;
        float s[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const int chunk = (kk & 3) * 2 + mcol;   // 16-byte chunk of the 128-byte row, swizzled
          uint32_t b[4];                           // keys 0-7 | 8-15 at columns 0-7, then at 8-15
          ldsm_x4(b, kbase + (kk >> 2) * AT_HALF + ((chunk ^ (mrow & 7)) << 4));
          mma_16816(s[0], qa[kk][0], qa[kk][1], qa[kk][2], qa[kk][3], b[0], b[2]);
          mma_16816(s[1], qa[kk][0], qa[kk][1], qa[kk][2], qa[kk][3], b[1], b[3]);
        }
        if (key0 + 16 > lim_min) {
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (key0 + 8 * n + 2 * t + (e & 1) >= lim[e >> 1]) s[n][e] = -INFINITY;
        }
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = fmaxf(fmaxf(s[0][2 * e], s[0][2 * e + 1]), fmaxf(s[1][2 * e], s[1][2 * e + 1]));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2)) * sl2;
          // the reference moves only when the maximum exceeds it by more than 8 (P <= 256)
          f[e] = 1.f;
          if (x > m[e] + 8.f || m[e] == -INFINITY) {
            f[e] = m[e] == -INFINITY ? 1.f : exp2f(m[e] - x);   // no key seen yet: O and l are 0
            m[e] = x;
          }
        }
        if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
          for (int e = 0; e < 2; ++e) l[e] *= f[e];
#pragma unroll
          for (int c = 0; c < 16; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[c][e] *= f[e >> 1];
        }
        uint32_t pa[4];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float ref = m[e] == -INFINITY ? 0.f : m[e];
            const float x0 = ex2_approx(fmaf(s[n][2 * e], sl2, -ref)), x1 = ex2_approx(fmaf(s[n][2 * e + 1], sl2, -ref));
            l[e] += x0 + x1;
            pa[2 * n + e] = pack_bf16x2(x0, x1);
          }
#pragma unroll
        for (int c = 0; c < 8; ++c) {   // 16 head columns: two 8-column products
          const int chunk = (c & 3) * 2 + mcol;
          uint32_t b[4];
          ldsm_x4_trans(b, vbase + (c >> 2) * AT_HALF + ((chunk ^ (mrow & 7)) << 4));
          mma_16816(o[2 * c], pa[0], pa[1], pa[2], pa[3], b[0], b[1]);
          mma_16816(o[2 * c + 1], pa[0], pa[1], pa[2], pa[3], b[2], b[3]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[sl]);
    }
    // join the warps: m = max over those that saw a key
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
      if (t == 0) {
        s_ml[warp][g + 8 * e][0] = m[e];
        s_ml[warp][g + 8 * e][1] = l[e];
      }
    }
    if (!at_all(ok)) return;
    float f[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float mx = -INFINITY;
#pragma unroll
      for (int x = 0; x < AT_WARPS; ++x) mx = fmaxf(mx, s_ml[x][g + 8 * e][0]);
      f[e] = m[e] == -INFINITY ? 0.f : exp2f(m[e] - mx);
    }
    const int n_rows = min(16, rows - r0), col = threadIdx.x;
    const size_t slot = nsp > 1 ? static_cast<size_t>(ap_slot(d, p.kv_heads, w.u.s, 0, w.u.h, w.u.j)) * d.slot_rows + r0 : 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) {   // four rows at a time
      if (4 * b >= n_rows) break;
      if ((g >> 2) == (b & 1)) {
#pragma unroll
        for (int c = 0; c < 16; ++c)
          *reinterpret_cast<float2*>(&s_o[warp][g & 3][8 * c + 2 * t]) =
              make_float2(o[c][2 * (b >> 1)] * f[b >> 1], o[c][2 * (b >> 1) + 1] * f[b >> 1]);
      }
      at_bar();
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int r = 4 * b + x;
        if (r >= n_rows) break;
        float mx = -INFINITY, sum = 0.f, v = 0.f;
#pragma unroll
        for (int y = 0; y < AT_WARPS; ++y) mx = fmaxf(mx, s_ml[y][r][0]);
#pragma unroll
        for (int y = 0; y < AT_WARPS; ++y) {
          const float my = s_ml[y][r][0];
          if (my == -INFINITY && s_ml[y][r][1] == 0.f) continue;   // saw no key
          sum = fmaf(s_ml[y][r][1], exp2f(my - mx), sum);
          v += s_o[y][x][col];
        }
        if (nsp > 1) {
          p.part_o[(slot + r) * 128 + col] = v;
          if (col == 0) {
            p.part_ml[2 * (slot + r)] = mx;
            p.part_ml[2 * (slot + r) + 1] = sum;
          }
        } else {
          const int row = r0 + r;
          v = sum == 0.f ? 0.f : v / sum;
          p.o[static_cast<size_t>(sq.q0 + row / G) * p.ldo + (w.u.h * G + row % G) * 128 + col] =
              static_cast<uint16_t>(pack_bf16x2(v, 0.f));
        }
      }
      at_bar();   // s_o and, after the last rows, s_ml may be written again
    }
  }
}

// Join the key ranges of a split tile: with m = max m_j over the ranges that
// have weight, O = sum O_j 2^(m_j - m) / sum l_j 2^(m_j - m), always in the
// same order.  One CTA per row: warp w adds ranges w, w + 4, ..., 32 lanes
// cover the 128 columns, and the four sums are added in shared memory.
constexpr int AP_JOIN_WARPS = 4;
template <class Plan>
__global__ void __launch_bounds__(32 * AP_JOIN_WARPS) ap_join_kernel(const __grid_constant__ ApKernelParams<Plan> p) {
  const Plan& d = p.plan;
  __shared__ float4 s_o[AP_JOIN_WARPS][32];
  __shared__ float s_l[AP_JOIN_WARPS];
  const int b = static_cast<int>(blockIdx.x), r = static_cast<int>(blockIdx.y);
  // the last sequence whose groups begin at or before b (an unsplit one has none and begins
  // where the next split one does)
  int s = 0, s_hi = d.n_seqs - 1;
  while (s < s_hi) {
    const int mid = (s + s_hi + 1) >> 1;
    if (d.seq[mid].cbase <= b) s = mid;
    else s_hi = mid - 1;
  }
  const int ct = (b - d.seq[s].cbase) / p.kv_heads, h = (b - d.seq[s].cbase) % p.kv_heads;
  const int G = d.G, nsp = d.seq[s].nsp, p0 = ct * d.P;
  const int n_rows = min(d.P, d.seq[s].ql - p0) * G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const size_t step = static_cast<size_t>(p.kv_heads) * d.slot_rows;
  const size_t at = static_cast<size_t>(ap_slot(d, p.kv_heads, s, ct, h, 0)) * d.slot_rows + r;
  pdl_wait();   // (all of the above comes from the launch's own arguments)
  pdl_trigger();
  if (r >= n_rows) return;
  float m = -INFINITY;
  for (int j = lane; j < nsp; j += 32) {
    const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + 2 * (at + j * step));
    if (ml.y != 0.f) m = fmaxf(m, ml.x);   // NaN sums count too
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float lsum = 0.f;
#pragma unroll 4
  for (int j = warp; j < nsp; j += AP_JOIN_WARPS) {
    const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + 2 * (at + j * step));
    float4 o = *reinterpret_cast<const float4*>(p.part_o + (at + j * step) * 128 + lane * 4);
    const bool none = ml.y == 0.f;   // no key of this range is visible: O_j may be unwritten
    const float f = none ? 0.f : exp2f(ml.x - m);
    if (none) o = make_float4(0.f, 0.f, 0.f, 0.f);
    acc.x = fmaf(o.x, f, acc.x);
    acc.y = fmaf(o.y, f, acc.y);
    acc.z = fmaf(o.z, f, acc.z);
    acc.w = fmaf(o.w, f, acc.w);
    lsum = fmaf(ml.y, f, lsum);
  }
  s_o[warp][lane] = acc;
  if (lane == 0) s_l[warp] = lsum;
  __syncthreads();
  if (warp > 0) return;
#pragma unroll
  for (int w = 1; w < AP_JOIN_WARPS; ++w) {
    const float4 x = s_o[w][lane];
    acc = make_float4(acc.x + x.x, acc.y + x.y, acc.z + x.z, acc.w + x.w);
    lsum += s_l[w];
  }
  const float inv = lsum == 0.f ? 0.f : 1.0f / lsum;
  const uint2 w = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  *reinterpret_cast<uint2*>(p.o + static_cast<size_t>(d.seq[s].q0 + p0 + r / G) * p.ldo +
                            (h * G + r % G) * 128 + lane * 4) = w;
}

// ---------------------------------------------------------------- host side

// Launch plans of a table of sequences, one for the tile kernel and one for the
// token kernel: a pure function of the arguments.
//  * sequences of at most AT_MAX_ROWS rows go to the token kernel, except short
//    ones beside sequences that need the tile kernel anyway: a unit more there
//    costs less than a second kernel (about 12 us).
//  * tile kernel: key ranges are split when the longest unit would outlast the
//    average load of an SM, into ranges of about that average, at least
//    AP_MIN_RANGE steps of keys (a range costs a partial result and the joining
//    kernel).
//  * token kernel: two CTAs fit on an SM; ranges are as long as gives every
//    place one CTA, but between AT_MIN_KEYS (fewer keys do not pay for a
//    partial result) and AT_MAX_KEYS (shorter CTAs even out ragged lengths).
constexpr int AP_MIN_RANGE = 8;
constexpr int AT_MIN_KEYS = 256, AT_MAX_KEYS = 512, AT_JOIN_KEYS = 2048;

struct PlanSeq {
  int q0, ql, k0, kl, e, nsp;
};

// Launch order, partial results and CTA numbers of a plan whose splits are chosen.
static void plan_finish(std::vector<PlanSeq>& seq, int kv_heads, PackedPlan* d) {
  d->n_seqs = static_cast<int>(seq.size());
  auto tiles = [&](const PlanSeq& s) { return (s.ql + d->P - 1) / d->P; };
  for (PlanSeq& s : seq) s.e = tiles(s) * s.nsp;
  std::stable_sort(seq.begin(), seq.end(), [](const PlanSeq& a, const PlanSeq& b) {
    return a.e != b.e ? a.e > b.e : a.kl > b.kl;
  });
  for (int i = 0; i < d->n_seqs; ++i) {
    const PlanSeq& s = seq[i];
    d->seq[i] = {s.q0, s.ql, s.k0, s.kl, s.nsp, 0, d->slots, d->groups};
    if (s.nsp > 1) {
      d->slots += s.e * kv_heads;
      d->groups += tiles(s) * kv_heads;
      d->slot_rows = std::max(d->slot_rows, std::min(s.ql, d->P) * d->G);
    }
  }
  int at = 0;
  for (int i = d->n_seqs - 1; i >= 0; --i) {
    d->seq[i].ustart = at;
    const int below = i + 1 < d->n_seqs ? seq[i + 1].e : 0;
    at += (seq[i].e - below) * (i + 1) * kv_heads;
  }
  d->units = at;
}

void packed_plan(const int32_t* spans, int n, int heads, int kv_heads, int num_sms, PackedPlan* tile,
                 PackedPlan* token) {
  for (PackedPlan* d : {tile, token}) d->n_seqs = d->units = d->slots = d->slot_rows = d->groups = d->n_order = 0;
  tile->G = token->G = heads / kv_heads;
  tile->P = token->P = AP_ROWS / tile->G;
  std::vector<PlanSeq> big, few;
  long long few_keys = 0;
  bool any_big = false;
  for (int i = 0; i < n; ++i) any_big = any_big || static_cast<long long>(spans[4 * i + 1]) * tile->G > AT_MAX_ROWS;
  for (int i = 0; i < n; ++i) {
    const int32_t* t = spans + 4 * i;
    if (t[1] == 0) continue;
    const PlanSeq s{t[0], t[1], t[2], t[3], 0, 1};
    if (static_cast<long long>(s.ql) * tile->G <= AT_MAX_ROWS && !(any_big && s.kl <= AT_JOIN_KEYS)) {
      few.push_back(s);
      few_keys += static_cast<long long>(s.kl) * kv_heads;
    } else {
      big.push_back(s);
    }
  }
  if (!few.empty()) {
    const long long places = 2ll * num_sms;
    const long long range = std::min<long long>(
        AT_MAX_KEYS, std::max<long long>(AT_MIN_KEYS, (few_keys + places - 1) / places));
    for (PlanSeq& s : few) s.nsp = std::max(1, static_cast<int>((s.kl + range - 1) / range));
    plan_finish(few, kv_heads, token);
  }
  if (big.empty()) return;
  PackedPlan* d = tile;
  auto tiles = [&](const PlanSeq& s) { return (s.ql + d->P - 1) / d->P; };
  auto steps = [&](const PlanSeq& s, int ct) {   // of query tile ct over its keys
    const long long end = static_cast<long long>(s.kl) - s.ql + std::min((ct + 1) * d->P, s.ql);
    return end > 0 ? (end + AP_KEYS - 1) / AP_KEYS : 0ll;
  };
  long long total = 0, longest = 0;
  for (const PlanSeq& s : big) {
    const int t = tiles(s);
    for (int c = 0; c < t; ++c) total += steps(s, c) * kv_heads;
    longest = std::max(longest, steps(s, t - 1));
  }
  const long long share = (total + num_sms - 1) / num_sms;
  const long long range = std::max<long long>(AP_MIN_RANGE, share);
  if (longest >= 2 * range)
    for (PlanSeq& s : big) {
      const long long k = steps(s, tiles(s) - 1);
      if (k >= 2 * range) s.nsp = static_cast<int>((k + range - 1) / range);
    }
  plan_finish(big, kv_heads, d);
  // Exact order, longest unit first, where the table holds it and no unit is split (a counting
  // sort over the steps of a unit).
  if (d->slots > 0 || d->units > AP_MAX_ORDER * kv_heads || longest > AP_MAX_ORDER) return;
  std::vector<int> at(static_cast<size_t>(longest) + 2, 0);
  for (int pass = 0; pass < 2; ++pass) {
    for (int i = 0; i < d->n_seqs; ++i)
      for (int c = tiles(big[i]) - 1; c >= 0; --c) {
        const size_t cost = static_cast<size_t>(longest - steps(big[i], c));   // 0: the longest
        if (pass == 0) ++at[cost + 1];
        else d->order[at[cost]++] = static_cast<uint32_t>(i) << 24 | static_cast<uint32_t>(c);
      }
    if (pass == 0)
      for (size_t i = 1; i < at.size(); ++i) at[i] += at[i - 1];
  }
  d->n_order = d->units / kv_heads;
}

size_t packed_plan_bytes(const PackedPlan& d) {
  return (static_cast<size_t>(d.slots) * d.slot_rows * (128 + 2) * sizeof(float) + 15) & ~static_cast<size_t>(15);
}

// Largest dynamic shared memory of a kernel, set once per device.
template <class K>
static bool allow_smem(K kern, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return true;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  done.fetch_or(bit, std::memory_order_release);
  return true;
}

template <class Plan>
static int launch_join(const ApKernelParams<Plan>& p, cudaStream_t st) {
  if (p.plan.groups == 0) return 0;
  launch_pdl(ap_join_kernel<Plan>, dim3(p.plan.groups, p.plan.slot_rows), dim3(32 * AP_JOIN_WARPS), 0, st, 1, p);
  return launch_result();
}

// The parameters that both kernels take, with the plan's partial results from `scratch`.
template <class Plan>
static void ap_params(const PackedAttnParams& a, const PackedPlan& d, uint8_t* scratch, ApKernelParams<Plan>* p) {
  Plan& t = p->plan;
  t.n_seqs = d.n_seqs;
  t.G = d.G;
  t.P = d.P;
  t.units = d.units;
  t.slots = d.slots;
  t.slot_rows = d.slot_rows;
  t.groups = d.groups;
  t.n_order = d.n_order;
  memcpy(t.seq, d.seq, sizeof(PackedSeq) * static_cast<size_t>(d.n_seqs));
  memcpy(t.order, d.order, sizeof(uint32_t) * static_cast<size_t>(d.n_order));
  p->q = a.q;
  p->ldq = a.ldq;
  p->o = a.o;
  p->ldo = a.ldo;
  p->kv_heads = a.kv_heads;
  p->tma_out = 0;
  p->row_blocks = 0;
  p->sm_scale = a.sm_scale;
  p->status = a.status;
  p->part_o = reinterpret_cast<float*>(scratch);
  p->part_ml = p->part_o + static_cast<size_t>(d.slots) * d.slot_rows * 128;
}

// K and V maps; without any key row nothing is loaded and they lie over q.
static bool ap_kv_maps(const PackedAttnParams& a, CUtensorMap* tk, CUtensorMap* tv, uint32_t keys) {
  const bool none = a.k_rows == 0;
  const uint64_t width = static_cast<uint64_t>(a.kv_heads) * 128, n = none ? a.q_rows : a.k_rows;
  return make_tmap_2d(tk, none ? a.q : a.k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, width, n,
                      static_cast<uint64_t>(none ? a.ldq : a.ldk) * 2, 64, keys) &&
         make_tmap_2d(tv, none ? a.q : a.v, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, width, n,
                      static_cast<uint64_t>(none ? a.ldq : a.ldv) * 2, 64, keys);
}

template <class Plan>
static int launch_tile(const PackedAttnParams& a, const PackedPlan& d, uint8_t* scratch, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  if (!allow_smem(ap_kernel<Plan>, AP_SMEM, done)) {
    launch_result();
    return -1;
  }
  ApKernelParams<Plan> p;
  ap_params(a, d, scratch, &p);
  CUtensorMap tq, tk, tv, to;
  if (!make_tmap_rows3(&tq, a.q, 128, a.heads, a.q_rows, static_cast<uint64_t>(a.ldq) * 2, 64, d.G, d.P) ||
      !ap_kv_maps(a, &tk, &tv, AP_KEYS))
    return -2;
  // output boxes: the 32 rows of a softmax warp, min(G, 32) heads x 32 / G positions
  p.tma_out = 32 % d.G == 0 || d.G % 32 == 0;
  const uint32_t box_heads = d.G < 32 ? d.G : 32;
  if (!p.tma_out) to = tq;
  else if (!make_tmap_rows3(&to, a.o, 128, a.heads, a.q_rows, static_cast<uint64_t>(a.ldo) * 2, 32, box_heads,
                            32 / box_heads))
    return -2;
  launch_pdl(ap_kernel<Plan>, dim3(d.units), dim3(AP_THREADS), AP_SMEM, st, 1, tq, tk, tv, to,
             p);
  return launch_result() || launch_join(p, st) ? -1 : 0;
}

template <class Plan>
static int launch_token(const PackedAttnParams& a, const PackedPlan& d, uint8_t* scratch, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  if (!allow_smem(ap_token_kernel<Plan>, AT_SMEM, done)) {
    launch_result();
    return -1;
  }
  ApKernelParams<Plan> p;
  ap_params(a, d, scratch, &p);
  int rows = 0;
  for (int i = 0; i < d.n_seqs; ++i) rows = std::max(rows, d.seq[i].ql * d.G);
  p.row_blocks = (rows + 15) / 16;
  CUtensorMap tk, tv;
  if (!ap_kv_maps(a, &tk, &tv, AT_KEYS)) return -2;
  const long long total = static_cast<long long>(d.units) * p.row_blocks;
  const int grid = static_cast<int>(std::min<long long>(total, 2ll * a.num_sms));
  launch_pdl(ap_token_kernel<Plan>, dim3(grid), dim3(AT_THREADS), AT_SMEM, st, 1, tk, tv, p);
  return launch_result() || launch_join(p, st) ? -1 : 0;
}

template <class Plan>
static bool ap_holds(const PackedPlan& d) {
  return d.n_seqs <= static_cast<int>(sizeof(Plan::seq) / sizeof(PackedSeq)) &&
         d.n_order <= static_cast<int>(sizeof(Plan::order) / sizeof(uint32_t));
}

int launch_attention_packed(const PackedAttnParams& a, const PackedPlan& tile, const PackedPlan& token,
                            cudaStream_t st) {
  uint8_t* scratch = static_cast<uint8_t*>(a.scratch);
  int r = 0;
  if (tile.units > 0)
    r = ap_holds<ApFewPlan>(tile) ? launch_tile<ApFewPlan>(a, tile, scratch, st)
                                  : launch_tile<PackedPlan>(a, tile, scratch, st);
  if (r == 0 && token.units > 0) {
    scratch += packed_plan_bytes(tile);
    r = ap_holds<ApFewPlan>(token) ? launch_token<ApFewPlan>(a, token, scratch, st)
                                   : launch_token<PackedPlan>(a, token, scratch, st);
  }
  return r;
}

}  // namespace qi
