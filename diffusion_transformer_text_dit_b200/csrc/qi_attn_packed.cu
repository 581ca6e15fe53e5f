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
// tile is head r mod G at query position p0 + r / G, so one 128-key tile of K
// and V serves all of them and a short prompt or a single token (G rows)
// still reads each key once.  A tile holds P = 128 / G positions; rows past
// P G and past the sequence's last query are computed and dropped.  A CTA
// takes nq = 2 neighbouring tiles A and B of a sequence, whose MMAs and
// softmax alternate, or nq = 1 when there are too few tiles to fill the GPU.
//
// TMEM (512 columns): S_A | S_B | O_A | O_B.  Per key tile: S = Q K^T (both
// operands in shared memory), one thread per row takes the softmax, writes P
// as bf16 over S, and O += P V reads P from TMEM.  P is rounded to bf16 for
// the tensor core; the row sum adds the unrounded fp32 values.
//
// Rows that a sequence does not own: the last key tile may reach into the
// next sequence or into rows of a cache that were never written.  Their
// scores are masked, and their V rows, whose weight is 0 but whose values may
// be infinite or NaN, are kept out of the product: P V runs over the 16-key
// steps that hold a visible key, and the producer warp clears the rows between
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
constexpr int AP_THREADS = 320;   // 8 softmax warps, TMA (and the V tail), MMA
constexpr int AP_KST = 3;
constexpr int AP_VST = 2;
constexpr int AP_TILE = 128 * 128 * 2;
constexpr int AP_HALF = 128 * 128;
constexpr int AP_SMEM = 1024 + (2 + AP_KST + AP_VST) * AP_TILE + 256;

struct ApKernelParams {
  PackedPlan plan;
  const uint16_t* q;   // for the token kernel (the tile kernel reads it through a tensor map)
  int ldq;
  uint16_t* o;
  int ldo, kv_heads;
  int row_blocks;    // token kernel: 16-row blocks per unit
  float sm_scale;
  float* part_o;     // [slots][slot_rows][128]
  float* part_ml;    // [slots][slot_rows][2]
  int* status;
};

// CTA -> (sequence, query tile group, key/value head, key split).  Sequences
// are sorted by their number of units per head, E = tile groups x splits;
// level e takes unit e, counted from the sequence's end, of every sequence
// that has one, so long key ranges start first and the last CTAs are short.
struct ApUnit {
  int s, ct, h, j;
};
__host__ __device__ __forceinline__ int ap_tiles(const PackedPlan& d, int s) {
  const int per = d.P * d.nq;
  return (d.seq[s].ql + per - 1) / per;
}
__host__ __device__ __forceinline__ ApUnit ap_unit(const PackedPlan& d, int kv_heads, int b) {
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
__host__ __device__ __forceinline__ int ap_slot(const PackedPlan& d, int kv_heads, int s, int ct, int h, int j) {
  return d.seq[s].sbase + (ct * d.seq[s].nsp + j) * kv_heads + h;
}

__device__ __forceinline__ void ap_softmax_bar() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

__device__ __forceinline__ void tma_load_3d(const CUtensorMap* map, uint64_t* bar, void* smem, int x,
                                            int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(smem)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Ask for a tile in L2.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y)
               : "memory");
}

__global__ void __launch_bounds__(AP_THREADS, 1)
    ap_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
              const __grid_constant__ CUtensorMap tmV, const __grid_constant__ ApKernelParams p) {
  const PackedPlan& d = p.plan;
  int* status = p.status;
  extern __shared__ uint8_t ap_smem_raw[];
  const uint32_t raw_addr = smem_u32(ap_smem_raw);
  uint8_t* smem = ap_smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  uint8_t* sQ = smem;                              // [2][AP_TILE]
  uint8_t* sK = smem + 2 * AP_TILE;                // [AP_KST][AP_TILE]
  uint8_t* sV = smem + (2 + AP_KST) * AP_TILE;     // [AP_VST][AP_TILE]
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + (2 + AP_KST + AP_VST) * AP_TILE);
  uint64_t* q_full = bars + 0;
  uint64_t* k_full = bars + 1;                     // [AP_KST]
  uint64_t* k_empty = k_full + AP_KST;             // [AP_KST]
  uint64_t* v_full = k_empty + AP_KST;             // [AP_VST]
  uint64_t* v_empty = v_full + AP_VST;             // [AP_VST]
  uint64_t* s_full = v_empty + AP_VST;             // [2] per query tile
  uint64_t* p_full = s_full + 2;                   // [2]
  uint64_t* o_full = p_full + 2;
  uint64_t* drain = o_full + 1;
  uint64_t* v_landed = drain + 1;                  // the last V tile is in shared memory ...
  uint64_t* v_tail = v_landed + 1;                 // ... and its rows past the keys are cleared
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(v_tail + 1);
  uint8_t* stage = smem;   // output rows, over Q (free once every MMA has completed)

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const ApUnit u = ap_unit(d, p.kv_heads, static_cast<int>(blockIdx.x));
  const int G = d.G, P = d.P, nq = d.nq;
  const int ql = d.seq[u.s].ql, kl = d.seq[u.s].kl, k0s = d.seq[u.s].k0, nsp = d.seq[u.s].nsp;
  const int p0 = u.ct * P * nq;                    // first query position of this CTA
  const int first = kl - ql + 1;                   // keys that query position 0 sees (may be negative)
  // keys that the last position of tile X sees, and its key tiles
  int n_all[2];
#pragma unroll
  for (int X = 0; X < 2; ++X) {
    const int last = min(p0 + (X + 1) * P, ql) - 1;   // < p0 + X P: the tile has no query
    const int end = X < nq && last >= p0 + X * P ? max(0, first + last) : 0;
    n_all[X] = (end + AP_ROWS - 1) / AP_ROWS;
  }
  const int kv_end = max(0, first + min(p0 + nq * P, ql) - 1);   // keys that some row of this CTA sees
  const int n_tot = max(n_all[0], n_all[1]);
  const int lo = static_cast<int>(static_cast<long long>(n_tot) * u.j / nsp);
  const int hi = static_cast<int>(static_cast<long long>(n_tot) * (u.j + 1) / nsp);
  // this CTA's key tiles are [lo, hi); local tile i drives the rings and phases
  const int n_x0 = max(0, min(n_all[0], hi) - lo), n_x1 = max(0, min(n_all[1], hi) - lo);
  const int n_kv = hi - lo;
  // keys of the last tile some row sees; < 128: rows behind them must not reach P V
  const int tail = hi == n_tot && n_kv > 0 ? kv_end - (n_tot - 1) * AP_ROWS : AP_ROWS;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int s = 0; s < AP_KST; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
    }
    for (int s = 0; s < AP_VST; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], 128);
    }
    mbar_init(o_full, 1);
    mbar_init(drain, 1);
    mbar_init(v_landed, 1);
    mbar_init(v_tail, 1);
    fence_mbar_init();
  }
  if (warp == 8 && lane == 0) {
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();
  pdl_trigger();

  if (warp == 8) {
    // ------------------------------------------------------------ TMA producer
    bool ok = true;
    if (lane == 0 && n_kv > 0) {
      // a box holds P positions x G heads x 64 head columns: rows in tile order
      const uint32_t q_bytes = static_cast<uint32_t>(P * G) * 128 * 2;
      mbar_arrive_expect_tx(q_full, nq * q_bytes);
      for (int t = 0; t < nq; ++t)
        for (int half = 0; half < 2; ++half)
          tma_load_3d(&tmQ, q_full, sQ + t * AP_TILE + half * AP_HALF, 64 * half, u.h * G,
                      d.seq[u.s].q0 + p0 + t * P);
      int jk = 0, jv = 0;   // tiles whose loads were issued
      for (int j = 0; j < n_kv; ++j) {
        const int row = k0s + (lo + j) * AP_ROWS;
        const int ks = j % AP_KST, kr = j / AP_KST;
        if (!mbar_wait(&k_empty[ks], (kr & 1) ^ 1u, status)) { ok = false; break; }
        mbar_arrive_expect_tx(&k_full[ks], AP_TILE);
        for (int half = 0; half < 2; ++half)
          tma_load_2d(&tmK, &k_full[ks], sK + ks * AP_TILE + half * AP_HALF, u.h * 128 + 64 * half, row);
        jk = j + 1;
        const int vs = j % AP_VST, vr = j / AP_VST;
        if (!mbar_wait(&v_empty[vs], (vr & 1) ^ 1u, status)) { ok = false; break; }
        mbar_arrive_expect_tx(&v_full[vs], AP_TILE);
        for (int half = 0; half < 2; ++half)
          tma_load_2d(&tmV, &v_full[vs], sV + vs * AP_TILE + half * AP_HALF, u.h * 128 + 64 * half, row);
        jv = j + 1;
      }
      if (!ok) {
        // bounded drain of the loads already armed (Q, the last K and V tiles)
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(q_full, 0) && globaltimer_ns() - t0 < QI_WAIT_NS) {
        }
        for (int jj = (jk > AP_KST ? jk - AP_KST : 0); jj < jk; ++jj) {
          const uint64_t t1 = globaltimer_ns();
          while (!mbar_try_wait(&k_full[jj % AP_KST], (jj / AP_KST) & 1) &&
                 globaltimer_ns() - t1 < QI_WAIT_NS) {
          }
        }
        for (int jj = (jv > AP_VST ? jv - AP_VST : 0); jj < jv; ++jj) {
          const uint64_t t1 = globaltimer_ns();
          while (!mbar_try_wait(&v_full[jj % AP_VST], (jj / AP_VST) & 1) &&
                 globaltimer_ns() - t1 < QI_WAIT_NS) {
          }
        }
      }
    }
    // V tail: clear the last tile's rows from the last visible key to the end
    // of its 16-key step (the swizzle permutes inside a 128-byte row)
    if (__all_sync(0xffffffffu, ok) && tail < AP_ROWS && n_kv > 0) {
      const int st = (n_kv - 1) % AP_VST;
      if (mbar_wait_warp(v_landed, 0, status) &&
          mbar_wait_warp(&v_full[st], ((n_kv - 1) / AP_VST) & 1, status)) {
        const int rows = ((tail + 15) & ~15) - tail;
        for (int i = lane; i < rows * 16; i += 32)
          *reinterpret_cast<uint4*>(sV + st * AP_TILE + ((i >> 3) & 1) * AP_HALF + (tail + (i >> 4)) * 128 +
                                    (i & 7) * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(v_tail);
      }
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0 && n_kv > 0) {
      constexpr uint32_t idesc_s = umma_idesc(false, 128, 128);
      constexpr uint32_t idesc_pv = umma_idesc(false, 128, 128) | (1u << 16);   // B MN-major
      bool ok = mbar_wait(q_full, 0, status);
      bool landed = false;
      auto issue_s = [&](int X, int jj) -> bool {
        const int st = jj % AP_KST;
        if (!mbar_wait(&k_full[st], (jj / AP_KST) & 1, status)) return false;
        tc_fence_after();
        const uint32_t qa = smem_u32(sQ + X * AP_TILE), kb = smem_u32(sK + st * AP_TILE);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t off = (kk >> 2) * AP_HALF + (kk & 3) * 32;
          umma_f16(tmem_base + X * 128, umma_desc_kmajor_sw128(qa + off),
                   umma_desc_kmajor_sw128(kb + off), idesc_s, kk > 0);
        }
        umma_commit(&s_full[X]);
        return true;
      };
      auto issue_pv = [&](int X, int jj) -> bool {
        const int st = jj % AP_VST;
        const bool cut = jj == n_kv - 1 && tail < AP_ROWS;
        if (!mbar_wait(&v_full[st], (jj / AP_VST) & 1, status)) return false;
        if (cut && !landed) {   // cleared while the softmax runs
          mbar_arrive(v_landed);
          landed = true;
        }
        if (!mbar_wait(&p_full[X], jj & 1, status)) return false;
        if (cut && !mbar_wait(v_tail, 0, status)) return false;
        tc_fence_after();
        const uint32_t vb = smem_u32(sV + st * AP_TILE);
        const int steps = cut ? (tail + 15) / 16 : 8;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)   // 16 keys per instruction
          if (kk < steps)
            umma_f16_ts(tmem_base + 256 + X * 128, tmem_base + X * 128 + kk * 8,
                        umma_desc_mnmajor_sw128(vb + kk * 2048, AP_HALF), idesc_pv,
                        (jj > 0 || kk > 0) ? 1u : 0u);
        return true;
      };
      if (ok) {
        if (n_x0 > 0) ok = issue_s(0, 0);
        if (ok && n_x1 > 0) ok = issue_s(1, 0);
        if (ok) umma_commit(&k_empty[0]);
      }
      for (int j = 0; ok && j < n_kv; ++j) {
        if (j < n_x0) ok = issue_pv(0, j);
        if (ok && j + 1 < n_x0) ok = issue_s(0, j + 1);
        if (ok && j < n_x1) ok = issue_pv(1, j);
        if (ok) umma_commit(&v_empty[j % AP_VST]);
        if (ok && j + 1 < n_kv) {
          if (j + 1 < n_x1) ok = issue_s(1, j + 1);
          if (ok) umma_commit(&k_empty[(j + 1) % AP_KST]);
        }
      }
      if (ok) {
        umma_commit(o_full);
      } else {
        umma_commit(drain);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(drain, 0) && globaltimer_ns() - t0 < QI_WAIT_NS) {
        }
      }
    }
  } else {
    // ------------------------------------------------------------ softmax + epilogue
    const int X = warp >> 2;
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lane_bits = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem_base + lane_bits + X * 128;
    const uint32_t tO = tmem_base + lane_bits + 256 + X * 128;
    const int n_mine = X == 0 ? n_x0 : n_x1;
    const int pos = p0 + X * P + row / G;           // query position of this row
    const bool live = X < nq && row < P * G && pos < ql;
    const int lim = live ? max(0, first + pos) : 0;   // keys this row sees
    // keys that every live row of this warp sees: tiles below need no mask
    const int lim_min = __reduce_min_sync(0xffffffffu, live ? lim : 0x7fffffff);
    const float sl2 = p.sm_scale * 1.4426950408889634f;
    float m_ref = 0.f;   // reference maximum, base-2 scaled
    float l = 0.f;
    bool seen = false;   // m_ref holds a score
    const bool warp_live = __any_sync(0xffffffffu, live);
    bool ok = true;
    for (int j = 0; j < n_mine; ++j) {
      if (!mbar_wait_warp(&s_full[X], j & 1, status)) { ok = false; break; }
      tc_fence_after();
      if (!warp_live) {   // no query in these 32 rows: whatever O gets is dropped
        mbar_arrive(&p_full[X]);
        continue;
      }
      const int k0 = (lo + j) * AP_ROWS;
      uint32_t r[128];
      tmem_ld128(tS, r);
      if (k0 + AP_ROWS > lim_min) {
#pragma unroll
        for (int i = 0; i < 128; ++i)
          if (k0 + i >= lim) r[i] = __float_as_uint(-INFINITY);
      }
      float m8[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) m8[k] = fmaxf(__uint_as_float(r[2 * k]), __uint_as_float(r[2 * k + 1]));
#pragma unroll
      for (int i = 16; i < 128; i += 16)
#pragma unroll
        for (int k = 0; k < 8; ++k)
          m8[k] = fmax3(m8[k], __uint_as_float(r[i + 2 * k]), __uint_as_float(r[i + 2 * k + 1]));
      const float mx2 = fmax3(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7])) * sl2;
      if (!seen && mx2 > -INFINITY) {   // the row's first score: P was 0 until now
        seen = true;
        m_ref = mx2;
      }
      const bool grow = mx2 > m_ref + 8.0f;
      if (__any_sync(0xffffffffu, grow)) {
        float f = 1.0f;
        if (grow) {
          f = exp2f(m_ref - mx2);
          l *= f;
          m_ref = mx2;
        }
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32];
          tmem_ld32(tO + c * 32, o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
          tmem_st32(tO + c * 32, o);
        }
        tmem_st_wait();
      }
      const uint64_t sl2x2 = f2_pack(sl2, sl2);
      const uint64_t negm2 = f2_pack(-m_ref, -m_ref);
      uint64_t acc2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float s0 = __uint_as_float(r[32 * c + 2 * i]), s1 = __uint_as_float(r[32 * c + 2 * i + 1]);
          const uint64_t x2 = f2_fma(f2_pack(s0, s1), sl2x2, negm2);
          float x0, x1;
          f2_unpack(x2, x0, x1);
          const float e0 = ex2_approx(x0);
          const float e1 = ex2_approx(x1);
          acc2[i & 3] = f2_add(acc2[i & 3], f2_pack(e0, e1));
          pk[i] = pack_bf16x2(e0, e1);
        }
        tmem_st16(tS + c * 16, pk);
      }
      float a0, a1, b0, b1;
      f2_unpack(f2_add(acc2[0], acc2[1]), a0, a1);
      f2_unpack(f2_add(acc2[2], acc2[3]), b0, b1);
      l += (a0 + b0) + (a1 + b1);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&p_full[X]);
    }
    ok = __all_sync(0xffffffffu, ok);
    if (ok && n_kv > 0) ok = mbar_wait_warp(o_full, 0, status);
    tc_fence_after();
    const bool have = n_mine > 0;   // O of this tile was written
    if (X < nq && ok && nsp > 1) {
      // partial result of this key range (rows packed from the CTA's first)
      const int prow = X * P * G + row;
      const size_t at = static_cast<size_t>(ap_slot(d, p.kv_heads, u.s, u.ct, u.h, u.j)) * d.slot_rows + prow;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t r[32];
        if (have) tmem_ld32(tO + c * 32, r);
        if (live && have) {
          float4* dst = reinterpret_cast<float4*>(p.part_o + at * 128 + c * 32);
#pragma unroll
          for (int v = 0; v < 8; ++v)
            dst[v] = make_float4(__uint_as_float(r[4 * v]), __uint_as_float(r[4 * v + 1]),
                                 __uint_as_float(r[4 * v + 2]), __uint_as_float(r[4 * v + 3]));
        }
      }
      if (live) {
        p.part_ml[2 * at] = m_ref;
        p.part_ml[2 * at + 1] = have ? l : 0.f;   // 0: this range has no weight
      }
    } else if (X < nq && ok) {
      const float inv = l > 0.f ? 1.0f / l : 0.f;
      const uint64_t inv2 = f2_pack(inv, inv);
      uint8_t* rows = stage + X * AP_TILE + quarter * 32 * 256;   // this warp's 32 rows of 256 bytes
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t r[32];
        if (have) {
          tmem_ld32(tO + c * 32, r);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) r[i] = 0u;
        }
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float a, b;
            f2_unpack(f2_mul(f2_pack(__uint_as_float(r[8 * v + 2 * e]), __uint_as_float(r[8 * v + 2 * e + 1])), inv2), a, b);
            w[e] = lim == 0 ? 0u : pack_bf16x2(a, b);   // a row that sees no key: 0
          }
          // 16-byte chunk x of row i at chunk x ^ (i mod 16): no bank conflicts either way
          *reinterpret_cast<uint4*>(rows + lane * 256 + (((c * 4 + v) ^ (lane & 15)) << 4)) =
              make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      __syncwarp();
      // each half warp copies one row: 256 contiguous bytes of the output
#pragma unroll 4
      for (int i = 0; i < 16; ++i) {
        const int rr = 2 * i + (lane >> 4), x = lane & 15;
        const int tr = quarter * 32 + rr, ps = p0 + X * P + tr / G;
        if (tr < P * G && ps < ql) {
          const uint4 w = *reinterpret_cast<const uint4*>(rows + rr * 256 + ((x ^ (rr & 15)) << 4));
          *reinterpret_cast<uint4*>(p.o + static_cast<size_t>(d.seq[u.s].q0 + ps) * p.ldo +
                                    (u.h * G + tr % G) * 128 + x * 8) = w;
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
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

__global__ void __launch_bounds__(AT_THREADS, 2)
    ap_token_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                    const __grid_constant__ ApKernelParams p) {
  const PackedPlan& d = p.plan;
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

  // The units of this CTA: one of every gridDim.x, alternately from the front
  // and the back of each round, so that longest-first order evens out.
  auto unit_of = [&](int round) {
    const int n = static_cast<int>(gridDim.x), i = static_cast<int>(blockIdx.x);
    return round * n + ((round & 1) ? n - 1 - i : i);
  };
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
      if (unit_of(0) < total) {
        const Work w = work_of(unit_of(0));
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
      for (int round = 0; ok && unit_of(round) < total; ++round) {
        const Work w = work_of(unit_of(round));
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
  Work w = work_of(min(unit_of(0), total - 1));
  pdl_wait();
  pdl_trigger();
  const float sl2 = p.sm_scale * 1.4426950408889634f;
  // ldmatrix row addresses: lane gives row (lane & 7) of matrix lane >> 3.
  // K: matrices (keys 0-7, 8-15) x (columns 0-7, 8-15 of a 16-column step)
  // V: matrices (keys 0-7, 8-15) x (two 8-column groups)
  const int mrow = warp * 16 + (lane & 7) + ((lane >> 3) & 1) * 8, mcol = lane >> 4;
  int i = 0;   // steps taken, over all units
  for (int round = 0; unit_of(round) < total; ++round) {
    if (round > 0) w = work_of(unit_of(round));
    const PackedPlan::Seq& sq = d.seq[w.u.s];
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
__global__ void __launch_bounds__(32 * AP_JOIN_WARPS) ap_join_kernel(const __grid_constant__ ApKernelParams p) {
  const PackedPlan& d = p.plan;
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
  const int G = d.G, nsp = d.seq[s].nsp, p0 = ct * d.P * d.nq;
  const int n_rows = min(d.P * d.nq, d.seq[s].ql - p0) * G;
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
//  * sequences of at most AT_MAX_ROWS rows go to the token kernel.
//  * tile kernel: nq = 2 (two query tiles share a CTA's key stream and hide each
//    other's softmax) unless that leaves SMs without a CTA or every sequence
//    has no more positions than one tile holds; key ranges are split when the
//    longest CTA would outlast the average load of an SM, into ranges of about
//    that average, at least AP_MIN_RANGE key tiles (a range costs a partial
//    result and the joining kernel).
//  * token kernel: two CTAs fit on an SM; ranges are as long as gives every
//    place one CTA, but between AT_MIN_KEYS (fewer keys do not pay for a
//    partial result) and AT_MAX_KEYS (shorter CTAs even out ragged lengths).
constexpr int AP_MIN_RANGE = 4;
constexpr int AT_MIN_KEYS = 256, AT_MAX_KEYS = 512;

struct PlanSeq {
  int q0, ql, k0, kl, e, nsp;
};

// Launch order, partial results and CTA numbers of a plan whose nq and splits are chosen.
static void plan_finish(std::vector<PlanSeq>& seq, int kv_heads, PackedPlan* d) {
  d->n_seqs = static_cast<int>(seq.size());
  auto tiles = [&](const PlanSeq& s) { return (s.ql + d->P * d->nq - 1) / (d->P * d->nq); };
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
      d->slot_rows = std::max(d->slot_rows, std::min(s.ql, d->P * d->nq) * d->G);
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
  memset(tile, 0, sizeof(*tile));
  memset(token, 0, sizeof(*token));
  tile->G = token->G = heads / kv_heads;
  tile->P = token->P = AP_ROWS / tile->G;
  std::vector<PlanSeq> big, few;
  int max_ql = 0;
  long long few_keys = 0;
  for (int i = 0; i < n; ++i) {
    const int32_t* t = spans + 4 * i;
    if (t[1] == 0) continue;
    const PlanSeq s{t[0], t[1], t[2], t[3], 0, 1};
    if (static_cast<long long>(s.ql) * tile->G <= AT_MAX_ROWS) {
      few.push_back(s);
      few_keys += static_cast<long long>(s.kl) * kv_heads;
    } else {
      big.push_back(s);
      max_ql = std::max(max_ql, s.ql);
    }
  }
  if (!few.empty()) {
    const long long places = 2ll * num_sms;
    const long long range = std::min<long long>(
        AT_MAX_KEYS, std::max<long long>(AT_MIN_KEYS, (few_keys + places - 1) / places));
    for (PlanSeq& s : few) s.nsp = std::max(1, static_cast<int>((s.kl + range - 1) / range));
    token->nq = 1;
    plan_finish(few, kv_heads, token);
  }
  if (big.empty()) return;
  PackedPlan* d = tile;
  auto tiles = [&](const PlanSeq& s, int nq) { return (s.ql + d->P * nq - 1) / (d->P * nq); };
  auto key_tiles = [&](const PlanSeq& s, int nq, int ct) {   // of query tile group ct
    const long long end = static_cast<long long>(s.kl) - s.ql + std::min((ct + 1) * d->P * nq, s.ql);
    return end > 0 ? (end + AP_ROWS - 1) / AP_ROWS : 0ll;
  };
  long long units2 = 0;
  for (const PlanSeq& s : big) units2 += static_cast<long long>(tiles(s, 2)) * kv_heads;
  d->nq = max_ql > d->P && units2 >= num_sms ? 2 : 1;
  long long total = 0, longest = 0;
  for (const PlanSeq& s : big) {
    const int t = tiles(s, d->nq);
    for (int c = 0; c < t; ++c) total += key_tiles(s, d->nq, c) * kv_heads;
    longest = std::max(longest, key_tiles(s, d->nq, t - 1));
  }
  const long long share = (total + num_sms - 1) / num_sms;
  const long long range = std::max<long long>(AP_MIN_RANGE, share);
  if (longest >= 2 * range)
    for (PlanSeq& s : big) {
      const long long k = key_tiles(s, d->nq, tiles(s, d->nq) - 1);
      if (k >= 2 * range) s.nsp = static_cast<int>((k + range - 1) / range);
    }
  plan_finish(big, kv_heads, d);
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

static int launch_join(const ApKernelParams& p, cudaStream_t st) {
  if (p.plan.groups == 0) return 0;
  launch_pdl(ap_join_kernel, dim3(p.plan.groups, p.plan.slot_rows), dim3(32 * AP_JOIN_WARPS), 0, st, 1, p);
  return launch_result();
}

int launch_attention_packed(const PackedAttnParams& a, const PackedPlan& tile, const PackedPlan& token,
                            cudaStream_t st) {
  ApKernelParams p;
  p.q = a.q;
  p.ldq = a.ldq;
  p.o = a.o;
  p.ldo = a.ldo;
  p.kv_heads = a.kv_heads;
  p.sm_scale = a.sm_scale;
  p.status = a.status;
  uint8_t* scratch = static_cast<uint8_t*>(a.scratch);
  auto partials = [&](const PackedPlan& d, size_t at) {
    p.plan = d;
    p.part_o = reinterpret_cast<float*>(scratch + at);
    p.part_ml = p.part_o + static_cast<size_t>(d.slots) * d.slot_rows * 128;
  };
  // K and V maps; without any key row nothing is loaded and they lie over q
  auto kv_maps = [&](CUtensorMap* tk, CUtensorMap* tv, uint32_t keys) {
    const bool none = a.k_rows == 0;
    const uint64_t width = static_cast<uint64_t>(a.kv_heads) * 128, n = none ? a.q_rows : a.k_rows;
    return make_tmap_2d(tk, none ? a.q : a.k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, width, n,
                        static_cast<uint64_t>(none ? a.ldq : a.ldk) * 2, 64, keys) &&
           make_tmap_2d(tv, none ? a.q : a.v, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, width, n,
                        static_cast<uint64_t>(none ? a.ldq : a.ldv) * 2, 64, keys);
  };
  if (tile.units > 0) {
    static std::atomic<uint64_t> done{0};
    if (!allow_smem(ap_kernel, AP_SMEM, done)) {
      launch_result();
      return -1;
    }
    CUtensorMap tq, tk, tv;
    if (!make_tmap_rows3(&tq, a.q, 128, a.heads, a.q_rows, static_cast<uint64_t>(a.ldq) * 2, 64, tile.G, tile.P) ||
        !kv_maps(&tk, &tv, AP_ROWS))
      return -2;
    partials(tile, 0);
    launch_pdl(ap_kernel, dim3(tile.units), dim3(AP_THREADS), AP_SMEM, st, 1, tq, tk, tv, p);
    if (launch_result() || launch_join(p, st)) return -1;
  }
  if (token.units > 0) {
    int rows = 0;
    for (int i = 0; i < token.n_seqs; ++i) rows = std::max(rows, token.seq[i].ql * token.G);
    static std::atomic<uint64_t> done{0};
    if (!allow_smem(ap_token_kernel, AT_SMEM, done)) {
      launch_result();
      return -1;
    }
    CUtensorMap tk, tv;
    if (!kv_maps(&tk, &tv, AT_KEYS)) return -2;
    partials(token, packed_plan_bytes(tile));
    p.row_blocks = (rows + 15) / 16;
    const long long total = static_cast<long long>(token.units) * p.row_blocks;
    const int grid = static_cast<int>(std::min<long long>(total, 2ll * a.num_sms));
    launch_pdl(ap_token_kernel, dim3(grid), dim3(AT_THREADS), AT_SMEM, st, 1, tk, tv, p);
    if (launch_result() || launch_join(p, st)) return -1;
  }
  return 0;
}

}  // namespace qi
