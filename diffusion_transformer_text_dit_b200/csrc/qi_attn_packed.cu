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
// Few rows and many keys (single tokens): the key range of a tile is split
// over nsp CTAs, which write unnormalised O, maximum and sum to scratch; a
// second kernel joins them in a fixed order.
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
  uint16_t* o;
  int ldo, heads, kv_heads;
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
  return (d.ql[s] + per - 1) / per;
}
__host__ __device__ __forceinline__ ApUnit ap_unit(const PackedPlan& d, int kv_heads, int b) {
  // ustart falls with i: the levels shared by sequences 0..i begin at ustart[i]
  int lo = 0, hi = d.n_seqs - 1;
  while (lo < hi) {   // the first i whose levels begin at or before b
    const int mid = (lo + hi) >> 1;
    if (d.ustart[mid] <= b) hi = mid;
    else lo = mid + 1;
  }
  const int per_level = (lo + 1) * kv_heads;
  const int e0 = lo + 1 < d.n_seqs ? ap_tiles(d, lo + 1) * d.nsp[lo + 1] : 0;
  const int r = b - d.ustart[lo];
  const int e = e0 + r / per_level, w = r % per_level;
  ApUnit u;
  u.s = w / kv_heads;
  u.h = w - u.s * kv_heads;
  const int nsp = d.nsp[u.s];
  u.ct = ap_tiles(d, u.s) - 1 - e / nsp;
  u.j = e % nsp;
  return u;
}
__host__ __device__ __forceinline__ int ap_slot(const PackedPlan& d, int kv_heads, int s, int ct, int h, int j) {
  return d.sbase[s] + (ct * d.nsp[s] + j) * kv_heads + h;
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
  const int ql = d.ql[u.s], kl = d.kl[u.s], k0s = d.k0[u.s], nsp = d.nsp[u.s];
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
                      d.q0[u.s] + p0 + t * P);
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
          *reinterpret_cast<uint4*>(p.o + static_cast<size_t>(d.q0[u.s] + ps) * p.ldo +
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

// Join the key ranges of a split tile: with m = max m_j over the ranges that
// have weight, O = sum O_j 2^(m_j - m) / sum l_j 2^(m_j - m), j ascending.
// One CTA per (sequence, query tile group, key/value head); 32 lanes cover a
// row's 128 columns.
constexpr int AP_JOIN_THREADS = 256;
__global__ void __launch_bounds__(AP_JOIN_THREADS) ap_join_kernel(const __grid_constant__ ApKernelParams p) {
  const PackedPlan& d = p.plan;
  const int b = static_cast<int>(blockIdx.x);
  int s = 0;
  while (!(d.nsp[s] > 1 && b >= d.cbase[s] && b < d.cbase[s] + ap_tiles(d, s) * p.kv_heads)) {
    if (s == d.n_seqs - 1) return;
    ++s;
  }
  const int ct = (b - d.cbase[s]) / p.kv_heads, h = (b - d.cbase[s]) % p.kv_heads;
  const int G = d.G, nsp = d.nsp[s], p0 = ct * d.P * d.nq;
  const int rows = min(d.P * d.nq, d.ql[s] - p0) * G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  for (int r = warp; r < rows; r += AP_JOIN_THREADS / 32) {
    const size_t step = static_cast<size_t>(p.kv_heads) * d.slot_rows;
    const size_t at = static_cast<size_t>(ap_slot(d, p.kv_heads, s, ct, h, 0)) * d.slot_rows + r;
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
    for (int j = 0; j < nsp; ++j) {
      const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + 2 * (at + j * step));
      if (ml.y == 0.f) continue;   // no key of this range is visible: O_j may be unwritten
      const float f = exp2f(ml.x - m);
      const float4 o = *reinterpret_cast<const float4*>(p.part_o + (at + j * step) * 128 + lane * 4);
      acc.x = fmaf(o.x, f, acc.x);
      acc.y = fmaf(o.y, f, acc.y);
      acc.z = fmaf(o.z, f, acc.z);
      acc.w = fmaf(o.w, f, acc.w);
      lsum = fmaf(ml.y, f, lsum);
    }
    const float inv = lsum == 0.f ? 0.f : 1.0f / lsum;
    const uint2 w = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    *reinterpret_cast<uint2*>(p.o + static_cast<size_t>(d.q0[s] + p0 + r / G) * p.ldo +
                              (h * G + r % G) * 128 + lane * 4) = w;
  }
}

// ---------------------------------------------------------------- host side

// Launch plan of a table of sequences: a pure function of its arguments.
//  * nq = 2 (two query tiles share a CTA's key stream and hide each other's
//    softmax) unless that leaves SMs without a CTA or every sequence has no
//    more positions than one tile holds.
//  * key ranges are split when the longest CTA would outlast the average load
//    of an SM: ranges of about that average, at least AP_MIN_RANGE key tiles
//    (a range costs a partial result and the joining kernel).
constexpr int AP_MIN_RANGE = 4;

void packed_plan(const int32_t* spans, int n, int heads, int kv_heads, int num_sms, PackedPlan* d) {
  memset(d, 0, sizeof(*d));
  d->G = heads / kv_heads;
  d->P = AP_ROWS / d->G;
  struct Seq {
    int q0, ql, k0, kl, e, nsp;
  };
  std::vector<Seq> seq;
  int max_ql = 0;
  for (int i = 0; i < n; ++i) {
    const int32_t* t = spans + 4 * i;
    if (t[1] == 0) continue;
    seq.push_back({t[0], t[1], t[2], t[3], 0, 1});
    max_ql = std::max(max_ql, t[1]);
  }
  d->n_seqs = static_cast<int>(seq.size());
  if (seq.empty()) return;
  auto tiles = [&](const Seq& s, int nq) { return (s.ql + d->P * nq - 1) / (d->P * nq); };
  auto key_tiles = [&](const Seq& s, int nq, int ct) {   // of query tile group ct
    const long long end = static_cast<long long>(s.kl) - s.ql + std::min((ct + 1) * d->P * nq, s.ql);
    return end > 0 ? (end + AP_ROWS - 1) / AP_ROWS : 0ll;
  };
  long long units2 = 0;
  for (const Seq& s : seq) units2 += static_cast<long long>(tiles(s, 2)) * kv_heads;
  d->nq = max_ql > d->P && units2 >= num_sms ? 2 : 1;
  long long total = 0, longest = 0, units = 0;
  for (const Seq& s : seq) {
    const int t = tiles(s, d->nq);
    units += static_cast<long long>(t) * kv_heads;
    for (int c = 0; c < t; ++c) total += key_tiles(s, d->nq, c) * kv_heads;
    longest = std::max(longest, key_tiles(s, d->nq, t - 1));
  }
  const long long share = (total + num_sms - 1) / num_sms;
  const long long range = std::max<long long>(AP_MIN_RANGE, share);
  if (longest >= 2 * range)
    for (Seq& s : seq) {
      const long long k = key_tiles(s, d->nq, tiles(s, d->nq) - 1);
      if (k >= 2 * range) s.nsp = static_cast<int>((k + range - 1) / range);
    }
  for (Seq& s : seq) s.e = tiles(s, d->nq) * s.nsp;
  std::stable_sort(seq.begin(), seq.end(), [](const Seq& a, const Seq& b) {
    return a.e != b.e ? a.e > b.e : a.kl > b.kl;
  });
  int rows = 0;
  for (int i = 0; i < d->n_seqs; ++i) {
    const Seq& s = seq[i];
    d->q0[i] = s.q0;
    d->ql[i] = s.ql;
    d->k0[i] = s.k0;
    d->kl[i] = s.kl;
    d->nsp[i] = s.nsp;
    d->sbase[i] = d->slots;
    d->cbase[i] = d->groups;
    if (s.nsp > 1) {
      d->slots += s.e * kv_heads;
      d->groups += tiles(s, d->nq) * kv_heads;
      rows = std::max(rows, std::min(s.ql, d->P * d->nq) * d->G);
    }
  }
  d->slot_rows = rows;
  int at = 0;
  for (int i = d->n_seqs - 1; i >= 0; --i) {
    d->ustart[i] = at;
    const int below = i + 1 < d->n_seqs ? seq[i + 1].e : 0;
    at += (seq[i].e - below) * (i + 1) * kv_heads;
  }
  d->units = at;
}

size_t packed_plan_bytes(const PackedPlan& d) {
  return static_cast<size_t>(d.slots) * d.slot_rows * (128 + 2) * sizeof(float);
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

int launch_attention_packed(const PackedAttnParams& a, const PackedPlan& plan, cudaStream_t st) {
  if (plan.units == 0) return 0;
  static std::atomic<uint64_t> done{0};
  if (!allow_smem(ap_kernel, AP_SMEM, done)) {
    launch_result();
    return -1;
  }
  CUtensorMap tq, tk, tv;
  if (!make_tmap_rows3(&tq, a.q, 128, a.heads, a.q_rows, static_cast<uint64_t>(a.ldq) * 2, 64, plan.G, plan.P))
    return -2;
  if (a.k_rows == 0) {   // no keys at all: every row is 0 and nothing is loaded
    tk = tq;
    tv = tq;
  } else if (!make_tmap_2d(&tk, a.k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<uint64_t>(a.kv_heads) * 128,
                    a.k_rows, static_cast<uint64_t>(a.ldk) * 2, 64, AP_ROWS) ||
      !make_tmap_2d(&tv, a.v, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<uint64_t>(a.kv_heads) * 128,
                    a.k_rows, static_cast<uint64_t>(a.ldv) * 2, 64, AP_ROWS))
    return -2;
  ApKernelParams p;
  p.plan = plan;
  p.o = a.o;
  p.ldo = a.ldo;
  p.heads = a.heads;
  p.kv_heads = a.kv_heads;
  p.sm_scale = a.sm_scale;
  p.part_o = static_cast<float*>(a.scratch);
  p.part_ml = a.scratch ? p.part_o + static_cast<size_t>(plan.slots) * plan.slot_rows * 128 : nullptr;
  p.status = a.status;
  launch_pdl(ap_kernel, dim3(plan.units), dim3(AP_THREADS), AP_SMEM, st, 1, tq, tk, tv, p);
  if (launch_result()) return -1;
  if (plan.groups > 0) {
    launch_pdl(ap_join_kernel, dim3(plan.groups), dim3(AP_JOIN_THREADS), 0, st, 1, p);
    return launch_result();
  }
  return 0;
}

}  // namespace qi
