// Step 2-3 of a ForwardPass over a cache of 8-bit codes (Pie "The forward
// pass", State geometry: kv_len; Attention masks): split-KV grouped-query
// attention over paged e4m3 codes with one power-of-two scale per (page, kv
// head).
//
// Mathematics, for query vector q, slot s in a page with scales 2^ek, 2^ev and
// codes ck, cv:
//   x_s = log2(e) sm_scale 2^ek <q, ck> + ev,     p_s = 2^(x_s - M),
//   o = sum_s p_s cv_s / sum_s p_s 2^-ev,         lse = ln 2 (M + log2 sum_s p_s 2^-ev).
// K's scale multiplies a score.  V's scale is added to the exponent, so that
// the weights p_s, already scaled, multiply the bare codes and pages of
// unequal scales share one fp32 accumulator; the softmax sum takes it back
// out, exactly.  M is a whole number (the running maximum, rounded up): the
// constant ev - M is then exact and x_s - M is rounded once, near zero where
// the weight is large.
//
// Operands are fp16: a code is exact in it (one conversion instruction per two
// codes, where bf16 would take three), a query vector is brought to its range by a
// power of two of its own (which leaves bf16's 8 bits exact), and the weights
// keep 11 bits.  An fp32 pass splits query vectors and weights into two fp16
// halves (22 bits) and issues every product twice.
//
// Both products are transposed, S^T = K Q^T and O^T += V^T P^T, so that query
// vectors are the 8 columns of a 16 x 8 x 16 MMA and no row is padding for a
// decode row.  The codes are fetched with ldmatrix, which moves pairs of bytes:
//   * a K fragment holds codes 4t .. 4t + 3 of a slot where the MMA wants
//     elements 2t, 2t + 1, 2t + 8, 2t + 9: a permutation of d, applied to the
//     query vectors as well, which the dot product does not see;
//   * a transposed V fragment holds two neighbouring elements of d for two
//     slots; one byte permutation makes them two pairs of slots, and the rows of
//     O^T come out in the order 0, 2, .. 14, 1, 3, .. 15 of each 16.
// One CTA (4 compute warps and a producer warp) streams an item's chunk through a
// ring of 64-slot stages, filled by tensor copies with a swizzle that keeps
// ldmatrix free of bank conflicts.  Two warps share a stage, 32 slots each, and
// the pairs take turns: at 2 d bytes per slot it is the issue slots that run
// short, and two 16-slot units side by side share one softmax step's shuffles and
// tests.  Units that every query vector sees in full skip the tests.  A persistent
// grid takes items from a counter.  Items hold up to 8 query vectors (NT = 1: decode rows, bound by
// HBM: a slot and kv head costs 2 d bytes) or 32 (NT = 4: drafts and prompts
// that attend_kv8_tc.cu does not take, every code converted once for all of them).
// Masked passes skip stages that no row of the item sees.  Every wait is
// bounded in time.

#include <cfloat>
#include <climits>

#include <algorithm>

#include "fp8.cuh"
#include "tc_util.cuh"

namespace pie {

namespace a8 {

constexpr int WARPS = 4;
constexpr int THREADS = (WARPS + 1) * 32;
constexpr int MAX_PAGES = kStageSlots / 8;  // pages per stage at most
constexpr float kLog2e = 1.4426950408889634f;

template <int D, int NT, bool SPLIT>
struct Cfg {
  static constexpr int KS = D / 16;                      // 16-wide steps of d
  static constexpr int HALF = kStageSlots * D;           // K (or V) codes of a stage
  static constexpr int STAGE = 2 * HALF;
  // 48 KB of ring per CTA at d 128: three CTAs per SM keep 144 KB in flight
  static constexpr int STAGES = D == 128 ? 3 : 6;
  // barriers of the stages: an even number, at least the ring's, so that each
  // belongs to one pair of warps, which then sees every phase of it
  static constexpr int BARS = (STAGES + 1) / 2 * 2;
  static constexpr int QROW = D * 2 + 32;                // fp16 query vector, padded by 32 bytes:
                                                         // 8 rows' 8-byte reads cover all banks
  static constexpr int Q = 8 * NT * QROW * (SPLIT ? 2 : 1);
  static constexpr int OROW = D + 4;                     // (float2 stores of 4 rows on distinct banks)
  static constexpr int MERGE = WARPS * 8 * (OROW + 2) * 4;  // the warps' states of one query tile
  static constexpr int SCALES = STAGES * 2 * MAX_PAGES * 4;
  static constexpr int SMEM = STAGES * STAGE + Q + MERGE + SCALES + 8 * NT * 4 +
                              (2 * BARS + 4) * 8 + 32 + 1024;
  static constexpr int MIN_CTAS = NT == 1 ? 3 : 1;
};

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
// D (16 x 8, fp32) += A (16 x 16, fp16) B (16 x 8, fp16)
__device__ __forceinline__ void mma(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// what packing left out, itself packed
__device__ __forceinline__ uint32_t pack_rest(float lo, float hi, uint32_t packed) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&packed));
  return pack_half(lo - f.x, hi - f.y);
}

// byte offset of 16-byte chunk c of slot row r in a K or V block (128-byte
// swizzle for d 128, 64-byte for d 64)
template <int D>
__device__ __forceinline__ uint32_t chunk(int r, int c) {
  if constexpr (D == 128) return uint32_t(r * 128 + ((c ^ (r & 7)) << 4));
  else return uint32_t(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

__device__ __forceinline__ void tma_3d(void* dst, const CUtensorMap* map, int z, uint64_t* bar,
                                       uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
      "l"(map), "r"(0), "r"(0), "r"(z), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// The stages of an item that some row of it sees, in order: all of them
// without a mask; with one, 32 stages' words are looked through at a time,
// a lane each.  Every warp of the CTA walks the same ones.
struct Stages {
  const uint32_t* words;
  const int64_t* wind;
  int row0, nrows, kb, ke, n, base;
  uint32_t bits;
  __device__ __forceinline__ Stages(const DevMeta& m, const uint32_t* mask_words, const DecItem& it)
      : words(mask_words), wind(m.mask_word_indptr), row0(it.row0), nrows(it.nrows),
        kb(it.kv_begin), ke(it.kv_end), base(-1), bits(~0u) {
    n = ke > kb ? (ke - kb + kStageSlots - 1) / kStageSlots : 0;
  }
  // the first stage from s on that is seen, or n
  __device__ __forceinline__ int from(int s) {
    if (!words) return s;
    while (s < n) {
      if (base < 0 || s >= base + 32) {
        base = s;
        const int sb = kb + (s + int(threadIdx.x & 31)) * kStageSlots;
        bool seen = false;
        if (sb < ke)
          for (int r = 0; r < nrows && !seen; ++r) {
            const uint32_t* w = words + wind[row0 + r] + (sb >> 5);
#pragma unroll
            for (int i = 0; i < kStageSlots / 32; ++i) {
              const int left = ke - sb - 32 * i;
              if (left > 0) seen = seen || (w[i] & (left < 32 ? (1u << left) - 1u : ~0u)) != 0;
            }
          }
        bits = __ballot_sync(0xffffffffu, seen);
      }
      const uint32_t rest = bits >> (s - base);
      if (rest) return s + __ffs(rest) - 1;
      s = base + 32;
    }
    return n;
  }
};

}  // namespace a8

template <typename T, int D, int NT>
__global__ void __launch_bounds__(a8::THREADS, a8::Cfg<D, NT, sizeof(T) == 4>::MIN_CTAS)
    attend_kv8_kernel(DevMeta m, int Hq, int Hkv, int G, int P, float scale_log2, const T* q_rot,
                      const uint8_t* k_scale, const uint8_t* v_scale, const uint32_t* mask_words,
                      const DecItem* items, int num_items, int* work, uint32_t* status,
                      const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap) {
  using namespace a8;
  constexpr bool SPLIT = sizeof(T) == 4;
  using C = Cfg<D, NT, SPLIT>;
  constexpr int STAGES = C::STAGES, BARS = C::BARS, KS = C::KS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* qs = ring + STAGES * C::STAGE;                        // fp16 query vectors (then rests)
  float* merge = reinterpret_cast<float*>(qs + C::Q);            // [WARPS][8] m, l, then o
  int* exps = reinterpret_cast<int*>(merge + C::MERGE / 4);      // [STAGES][K, V][pages] exponents
  float* zq = reinterpret_cast<float*>(exps + C::SCALES / 4);    // [8 NT] score factors
  uint64_t* full = reinterpret_cast<uint64_t*>(zq + 8 * NT);
  uint64_t* empty = full + BARS;
  uint64_t* item_full = empty + BARS;
  uint64_t* item_empty = item_full + 2;
  int* qidx = reinterpret_cast<int*>(item_empty + 2);
  int* decision = qidx + 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < BARS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], WARPS / 2);  // the pair of warps that reads it
    }
    for (int q = 0; q < 2; ++q) {
      mbar_init(&item_full[q], 1);
      mbar_init(&item_empty[q], 1);
    }
    fence_barrier_init();
  }
  __syncthreads();
  grid_dep_wait();
  grid_dep_launch();
  const uint64_t wait_ns = m.test_wait_us ? uint64_t(m.test_wait_us) * 1000ull : kWaitLimitNs;

  if (warp == WARPS) {
    // ---------------- producer warp -----------------------------------------
    // Lane 2i + c copies the K (c = 0) or V (1) block of the stage's page i and,
    // while they are on their way, leaves its scale's exponent beside the stage.
    const uint64_t pol = policy_evict_first();
    const int c = lane & 1, pi = lane >> 1, lp = fp8::log2i(P), ppt = kStageSlots >> lp;
    int gs = 0;  // stages issued by this CTA so far
    // every way out counts the CTA done; the last one sets the counter back
    auto finish = [&]() {
      if (lane == 0) {
        __threadfence();
        if (atomicAdd(work + 1, 1) == int(gridDim.x) - 1) {
          atomicExch(work, 0);
          atomicExch(work + 1, 0);
        }
      }
    };
    int ticket = 0;  // lane 0: the next item, asked for while the last one streams
    if (lane == 0) ticket = atomicAdd(work, 1);
    for (int k = 0;; ++k) {
      int idx = __shfl_sync(0xffffffffu, ticket, 0);
      if (idx >= num_items) idx = -1;
      const int q = k & 1;
      if (k >= 2 && !mbar_wait_ns(&item_empty[q], ((k >> 1) - 1) & 1, wait_ns)) {
        if (lane == 0) set_status(status, PIE_STATUS_TIMEOUT);
        finish();
        return;
      }
      if (lane == 0) {
        qidx[q] = idx;
        mbar_arrive(&item_full[q]);
      }
      if (idx < 0) break;
      if (lane == 0) ticket = atomicAdd(work, 1);
      const DecItem it = items[idx];
      Stages seen(m, mask_words, it);
      auto issue_stage = [&](int ord, int s, int pid, int ek, int ev) -> bool {
        if (ord == m.test_stall - 1) return false;  // test hook: nothing from here on
        // the stage that held this one's place in the ring has been read
        const int st = gs % STAGES, before = gs - STAGES;
        uint64_t* bar = &full[gs % BARS];
        if (before >= 0 && !mbar_wait_ns(&empty[before % BARS], (before / BARS) & 1, wait_ns)) {
          if (lane == 0) set_status(status, PIE_STATUS_TIMEOUT);
          return false;
        }
        const bool issue = pi < ppt && pid >= 0;
        const uint32_t copies = __popc(__ballot_sync(0xffffffffu, issue));
        if (lane == 0) {
          const int sb = it.kv_begin + s * kStageSlots;
          if (copies != 2u * uint32_t(((min(sb + kStageSlots, it.kv_end) - 1) >> lp) - (sb >> lp) + 1))
            set_status(status, PIE_STATUS_BOUNDS);
          mbar_expect_tx(bar, copies * uint32_t(P) * D);
        }
        __syncwarp();
        if (issue)
          tma_3d(ring + st * C::STAGE + c * C::HALF + pi * P * D, c ? &vmap : &kmap,
                 int(int64_t(pid) * Hkv + it.kv_head), bar, pol);
        if (pi < MAX_PAGES) exps[(st * 2 + c) * MAX_PAGES + pi] = (c ? ev : ek) - fp8::kBias;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
        ++gs;
        return true;
      };
      const int i = pi < ppt ? pi : 0;
      auto stage_at = [&](int j) { return it.kv_begin + j * kStageSlots; };
      fp8::PageBatches pb(m, it.lane, window_pages(it.block), it.kv_head, it.kv_end, seen.n, Hkv, P,
                          k_scale, v_scale, stage_at);
      int next = seen.from(0);
      for (int s = 0, ord = 0; s < seen.n; ++s) {
        pb.at(s);
        if (s != next) continue;
        const int pid = pb.page(s, i), ek = pb.k_exp(s, i), ev = pb.v_exp(s, i);
        if (!issue_stage(ord, s, pid, ek, ev)) {
          finish();
          return;
        }
        ++ord;
        next = seen.from(s + 1);
      }
    }
    finish();
    return;
  }

  // ---------------- compute warps ---------------------------------------------
  // Fragments (g = lane / 4, t = lane % 4): scores S^T[slot g, g + 8][query 2t,
  // 2t + 1]; outputs O^T[d 16n + 2g, 16n + 2g + 1][query 2t, 2t + 1].
  const int g = lane >> 2, t = lane & 3;
  const int mi = lane >> 3, mr = lane & 7;  // ldmatrix: lane i serves row i & 7 of matrix i >> 3
  const uint32_t ring_s = smem_u32(ring);
  const int half = (warp & 1) * 32, pair = warp >> 1, lp = fp8::log2i(P);
  int gs = 0;
  bool dead = false;  // a wait ran out: no more work, but every barrier is still taken
  for (int k = 0;; ++k) {
    if (warp == 0) {
      const int q = k & 1;
      const bool ok = mbar_wait_ns(&item_full[q], (k >> 1) & 1, wait_ns);
      int v = ok ? qidx[q] : -2;
      v = __shfl_sync(0xffffffffu, v, 0);
      if (lane == 0) {
        decision[k & 1] = v;
        if (v != -2) mbar_arrive(&item_empty[q]);
        if (v == -2) set_status(status, PIE_STATUS_TIMEOUT);
      }
    }
    asm volatile("bar.sync 1, %0;" ::"n"(WARPS * 32) : "memory");
    const int idx = decision[k & 1];
    if (idx < 0) break;
    const DecItem it = items[idx];
    const int nqv = it.nrows * G;
    const WindowView view(m, P, window_pages(it.block));
    Stages st_it(m, mask_words, it);

    // the query vectors, scaled into fp16's range by a power of two each (the
    // largest magnitude to [2^13, 2^14)); 16 threads per vector
    {
      constexpr int EPT = D / 16;
      const int ch = threadIdx.x & 15;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int qv = nt * 8 + (threadIdx.x >> 4);
        float x[EPT];
#pragma unroll
        for (int e = 0; e < EPT; ++e) x[e] = 0.f;
        if (qv < nqv) {
          const int row = it.row0 + qv / G, head = it.kv_head * G + qv % G;
          const T* src = q_rot + (int64_t(row) * Hq + head) * D + ch * EPT;
          if constexpr (sizeof(T) * EPT == 8) {
            unpack8<T>(*reinterpret_cast<const uint2*>(src), x);
          } else {
#pragma unroll
            for (int e = 0; e < EPT; e += 16 / int(sizeof(T)))
              unpack16<T>(*reinterpret_cast<const uint4*>(src + e), x + e);
          }
        }
        float big = 0.f;
#pragma unroll
        for (int e = 0; e < EPT; ++e) big = fmaxf(big, fabsf(x[e]));
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, off));
        const int up = fp8::query_exp(big);
#pragma unroll
        for (int e = 0; e < EPT; ++e) x[e] = fp8::scale2(x[e], up);
        uint32_t* dst = reinterpret_cast<uint32_t*>(qs + qv * C::QROW + ch * EPT * 2);
#pragma unroll
        for (int e = 0; e < EPT; e += 2) {
          const uint32_t h = pack_half(x[e], x[e + 1]);
          dst[e / 2] = h;
          if constexpr (SPLIT) dst[8 * NT * C::QROW / 4 + e / 2] = pack_rest(x[e], x[e + 1], h);
        }
        if (ch == 0) zq[qv] = fp8::scale2(scale_log2, -up);
      }
    }
    asm volatile("bar.sync 1, %0;" ::"n"(WARPS * 32) : "memory");
    // this lane's query vectors 8 nt + 2t + i; the slots that every one sees
    bool valid_q[NT][2];
    int slot_lim[NT][2];
    float zf[NT][2];
    const uint32_t* mrow[NT][2];
    int lim_min = INT_MAX, lim_max = -1;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int qv = nt * 8 + 2 * t + i;
        valid_q[nt][i] = qv < nqv;
        const int row = it.row0 + (valid_q[nt][i] ? qv : 0) / G;
        slot_lim[nt][i] = valid_q[nt][i] ? m.slots[row] : -1;
        if (valid_q[nt][i]) {
          lim_min = min(lim_min, slot_lim[nt][i]);
          lim_max = max(lim_max, slot_lim[nt][i]);
        }
        zf[nt][i] = zq[qv];
        mrow[nt][i] = valid_q[nt][i] && mask_words ? mask_words + m.mask_word_indptr[row] : nullptr;
      }
    lim_min = __reduce_min_sync(0xffffffffu, lim_min);
    lim_max = __reduce_max_sync(0xffffffffu, lim_max);
    // Q^T fragments: d elements 16k + 4t .. 4t + 3 of query g (one bf16 query
    // tile keeps them in registers)
    constexpr bool QREG = NT == 1 && !SPLIT;
    uint32_t qb[QREG ? KS : 1][2];
    auto load_q = [&](int nt, int kk, uint32_t* b) {
      const uint8_t* src = qs + (nt * 8 + g) * C::QROW + kk * 32 + t * 8;
      const uint2 u = *reinterpret_cast<const uint2*>(src);
      b[0] = u.x;
      b[1] = u.y;
      if constexpr (SPLIT) {
        const uint2 w = *reinterpret_cast<const uint2*>(src + 8 * NT * C::QROW);
        b[2] = w.x;
        b[3] = w.y;
      }
    };
    if constexpr (QREG) {
#pragma unroll
      for (int kk = 0; kk < KS; ++kk) load_q(0, kk, qb[kk]);
    }
    float o[NT][KS][4];
    float m_used[NT][2], l_part[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int n = 0; n < KS; ++n) o[nt][n][0] = o[nt][n][1] = o[nt][n][2] = o[nt][n][3] = 0.f;
      m_used[nt][0] = m_used[nt][1] = -INFINITY;
      l_part[nt][0] = l_part[nt][1] = 0.f;
    }

    for (int s = st_it.from(0); s < st_it.n; s = st_it.from(s + 1), ++gs) {
      if ((gs & 1) != pair || dead) continue;  // the other pair's stage
      const int st = gs % STAGES;
      const int base = it.kv_begin + s * kStageSlots + half;  // this warp's first position
      const int left = it.kv_end - base;
      // the rows' mask words of these positions, on their way while the stage lands
      uint32_t word[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) word[nt][i] = mrow[nt][i] && left > 0 ? mrow[nt][i][base >> 5] : ~0u;
      if (!mbar_wait_ns(&full[gs % BARS], (gs / BARS) & 1, wait_ns)) {
        dead = true;
        if (lane == 0) set_status(status, PIE_STATUS_TIMEOUT);
        continue;
      }
      // U units of 16 slots side by side: two, or one after the other where the
      // query tiles take the registers
      constexpr int U = NT == 1 ? 2 : 1;
#pragma unroll 1
      for (int u0 = 0; u0 < 2 && left > 16 * u0; u0 += U) {
        const int unit = half + 16 * u0;  // first row within the stage
        const int ub = base + 16 * u0;
        const int nvalid = min(16 * U, left - 16 * u0);
        const uint32_t kbase = ring_s + st * C::STAGE, vbase = kbase + C::HALF;
        if (nvalid < 16 * U) {
          // V rows past the end: zero codes, so that their zero weights give zero
          for (int i = lane; i < (16 * U - nvalid) * (D / 16); i += 32)
            *reinterpret_cast<uint4*>(ring + st * C::STAGE + C::HALF +
                                      (unit + nvalid + i / (D / 16)) * D + i % (D / 16) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();  // the stage is later rewritten by the copy engine
          __syncwarp();
        }
        // ---- S^T = K Q^T: matrices (slots 0-7, chunk 2kk), (8-15, 2kk),
        // (0-7, 2kk + 1), (8-15, 2kk + 1)
        float cc[U][NT][4];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            cc[u][nt][0] = cc[u][nt][1] = cc[u][nt][2] = cc[u][nt][3] = 0.f;
#pragma unroll
        for (int kk = 0; kk < KS; kk += 2) {
          uint32_t w[U][4];
#pragma unroll
          for (int u = 0; u < U; ++u)
            ldsm_x4(kbase + chunk<D>(unit + 16 * u + (mi & 1) * 8 + mr, kk + (mi >> 1)), w[u]);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t a[U][4];
#pragma unroll
            for (int u = 0; u < U; ++u) {
              fp8::to_half2x2(w[u][2 * h], a[u][0], a[u][2]);
              fp8::to_half2x2(w[u][2 * h + 1], a[u][1], a[u][3]);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              uint32_t b[SPLIT ? 4 : 2];
              if constexpr (QREG) {
                b[0] = qb[kk + h][0];
                b[1] = qb[kk + h][1];
              } else {
                load_q(nt, kk + h, b);
              }
#pragma unroll
              for (int u = 0; u < U; ++u) {
                mma(cc[u][nt], a[u], b[0], b[1]);
                if constexpr (SPLIT) mma(cc[u][nt], a[u], b[2], b[3]);
              }
            }
          }
        }
        // this lane's slots g and g + 8 of each unit: their pages' scales
        float sk[U][2], unsv[U][2], lv[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int pg = (unit + 16 * u + g + 8 * j) >> lp;
            const int ek = exps[st * 2 * MAX_PAGES + pg], ev = exps[(st * 2 + 1) * MAX_PAGES + pg];
            sk[u][j] = fp8::pow2i(ek);
            unsv[u][j] = fp8::pow2i(-ev);
            lv[u][j] = float(ev);
          }
        // positions that every query vector sees (slots rise with them)
        const int s0 = view.slot(ub), s1 = view.slot(ub + 16 * U - 1);
        const bool all = !mask_words && nvalid == 16 * U && s1 <= lim_min &&
                         (view.window == 0 || s0 > lim_max - view.window || s1 < view.sinks);
        if (!all) {
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int i = e & 1, cs = 16 * u + g + 8 * (e >> 1);
                const bool vis = valid_q[nt][i] && cs < nvalid &&
                                 (mrow[nt][i] ? ((word[nt][i] >> (16 * u0 + cs)) & 1u) != 0
                                              : view.sees(slot_lim[nt][i], view.slot(ub + cs)));
                if (!vis) cc[u][nt][e] = -INFINITY;
              }
        }
        uint32_t pb[U][NT][SPLIT ? 4 : 2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          // cc[u][nt][e]: slot 16u + g + 8 (e >> 1), query 2t + (e & 1); the
          // factors stay above zero, so that -inf stays -inf
          float zs[U][4], mt[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              zs[u][e] = fmaxf(zf[nt][e & 1] * sk[u][e >> 1], FLT_MIN);
              mt[e & 1] = fmaxf(mt[e & 1], fmaf(cc[u][nt][e], zs[u][e], lv[u][e >> 1]));
            }
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) {
            mt[0] = fmaxf(mt[0], __shfl_xor_sync(0xffffffffu, mt[0], off));
            mt[1] = fmaxf(mt[1], __shfl_xor_sync(0xffffffffu, mt[1], off));
          }
          // (m_used + 8 is -inf at first: any visible score moves it)
          if (__any_sync(0xffffffffu, mt[0] > m_used[nt][0] + 8.f || mt[1] > m_used[nt][1] + 8.f)) {
            float alpha[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float m_new = mt[i] > m_used[nt][i] + 8.f ? ceilf(mt[i]) : m_used[nt][i];
              alpha[i] = m_new == m_used[nt][i] ? 1.f : ex2(m_used[nt][i] - m_new);
              l_part[nt][i] *= alpha[i];
              m_used[nt][i] = m_new;
            }
#pragma unroll
            for (int n = 0; n < KS; ++n) {
              o[nt][n][0] *= alpha[0];
              o[nt][n][1] *= alpha[1];
              o[nt][n][2] *= alpha[0];
              o[nt][n][3] *= alpha[1];
            }
          }
          // (no visible slot yet: every score is -inf, and so is every exponent)
          const float neg_m[2] = {m_used[nt][0] == -INFINITY ? 0.f : -m_used[nt][0],
                                  m_used[nt][1] == -INFINITY ? 0.f : -m_used[nt][1]};
#pragma unroll
          for (int u = 0; u < U; ++u) {
            float p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              p[e] = ex2(fmaf(cc[u][nt][e], zs[u][e], lv[u][e >> 1] + neg_m[e & 1]));
            l_part[nt][0] = fmaf(p[0], unsv[u][0], fmaf(p[2], unsv[u][1], l_part[nt][0]));
            l_part[nt][1] = fmaf(p[1], unsv[u][0], fmaf(p[3], unsv[u][1], l_part[nt][1]));
            const uint32_t h0 = pack_half(p[0], p[1]), h1 = pack_half(p[2], p[3]);
            pb[u][nt][0] = movmatrix_t(h0);
            pb[u][nt][1] = movmatrix_t(h1);
            if constexpr (SPLIT) {
              pb[u][nt][2] = movmatrix_t(pack_rest(p[0], p[1], h0));
              pb[u][nt][3] = movmatrix_t(pack_rest(p[2], p[3], h1));
            }
          }
        }
        // ---- O^T += V^T P^T: matrices (slots 0-7, chunk n), (8-15, n), (0-7,
        // n + 1), (8-15, n + 1), transposed
#pragma unroll
        for (int n = 0; n < KS; n += 2) {
          uint32_t w[U][4];
#pragma unroll
          for (int u = 0; u < U; ++u)
            ldsm_x4_t(vbase + chunk<D>(unit + 16 * u + (mi & 1) * 8 + mr, n + (mi >> 1)), w[u]);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int u = 0; u < U; ++u) {
              uint32_t a[4];
              fp8::to_half2x2(__byte_perm(w[u][2 * h], 0, 0x3120), a[0], a[1]);
              fp8::to_half2x2(__byte_perm(w[u][2 * h + 1], 0, 0x3120), a[2], a[3]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma(o[nt][n + h], a, pb[u][nt][0], pb[u][nt][1]);
                if constexpr (SPLIT) mma(o[nt][n + h], a, pb[u][nt][2], pb[u][nt][3]);
              }
            }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[gs % BARS]);
    }

    // ---- merge the warps' states into the item's partials, a query tile at a
    // time (the buffer's last readers have passed the barriers since)
    float* mw = merge;            // [WARPS][8]
    float* lw = mw + WARPS * 8;   // [WARPS][8]
    float* ow = lw + WARPS * 8;   // [WARPS][8][OROW]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (nt * 8 >= nqv) break;
      if (nt > 0) asm volatile("bar.sync 1, %0;" ::"n"(WARPS * 32) : "memory");
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float l = l_part[nt][i];
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
        const int q = 2 * t + i;
        if (g == 0) {
          mw[warp * 8 + q] = m_used[nt][i];
          lw[warp * 8 + q] = l;
        }
        float* orow = ow + (warp * 8 + q) * C::OROW;
#pragma unroll
        for (int n = 0; n < KS; ++n)
          *reinterpret_cast<float2*>(orow + 16 * n + 2 * g) = make_float2(o[nt][n][i], o[nt][n][2 + i]);
      }
      asm volatile("bar.sync 1, %0;" ::"n"(WARPS * 32) : "memory");
      for (int i = threadIdx.x; i < min(8, nqv - nt * 8) * D; i += WARPS * 32) {
        const int qq = i / D, cd = i % D;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) M = fmaxf(M, mw[w * 8 + qq]);
        float O = 0.f, L = 0.f;
        if (M != -INFINITY) {
#pragma unroll
          for (int w = 0; w < WARPS; ++w) {
            const float mv = mw[w * 8 + qq];
            const float f = mv == -INFINITY ? 0.f : ex2(mv - M);
            O = fmaf(f, ow[(w * 8 + qq) * C::OROW + cd], O);
            L = fmaf(f, lw[w * 8 + qq], L);
          }
        }
        const int64_t at = int64_t(it.part_base) + nt * 8 + qq;
        m.part_o[at * D + cd] = O;
        if (cd == 0) m.part_ml[at] = make_float2(M, L);
      }
    }
  }
}

template <typename T, int D, int NT>
static cudaError_t launch_a8(const pie_fwd_plan_t& p, const void* q_rot, const uint8_t* k_scale,
                             const uint8_t* v_scale, const uint32_t* mask_words, uint32_t* status,
                             const CUtensorMap& km, const CUtensorMap& vm, cudaStream_t s) {
  using C = a8::Cfg<D, NT, sizeof(T) == 4>;
  const int n = NT == 1 ? p.num_dec_items : p.num_wide_items;
  if (n == 0) return cudaSuccess;
  static std::atomic<uint64_t> configured{0};  // per instantiation and device
  cudaError_t e = set_smem_limit(attend_kv8_kernel<T, D, NT>, C::SMEM, configured);
  if (e != cudaSuccess) return e;
  DevMeta m = p.dev;
  test_wait_hook(&m.test_stall, &m.test_wait_us);
  const int per_sm = std::max(1, std::min(C::MIN_CTAS, 227 * 1024 / (C::SMEM + 1024)));
  const int grid = std::min(n, per_sm * std::max(1, p.dev.num_sms));
  return launch_dependent(attend_kv8_kernel<T, D, NT>, dim3(grid), dim3(a8::THREADS), C::SMEM, s,
                          true, m, p.desc.num_q_heads, p.desc.num_kv_heads, p.G, p.desc.page_size,
                          p.desc.sm_scale * a8::kLog2e, static_cast<const T*>(q_rot), k_scale,
                          v_scale, mask_words, NT == 1 ? m.dec_items : m.wide_items, n,
                          m.dec_work + (NT == 1 ? 0 : 2), status, km, vm);
}

template <typename T, int D>
static cudaError_t launch_a8_all(const pie_fwd_plan_t& p, const void* q_rot, const uint8_t* k_scale,
                                 const uint8_t* v_scale, const uint32_t* mask_words,
                                 uint32_t* status, const CUtensorMap& km, const CUtensorMap& vm,
                                 cudaStream_t s) {
  cudaError_t e = launch_a8<T, D, 1>(p, q_rot, k_scale, v_scale, mask_words, status, km, vm, s);
  if (e == cudaSuccess)
    e = launch_a8<T, D, 4>(p, q_rot, k_scale, v_scale, mask_words, status, km, vm, s);
  return e;
}

cudaError_t launch_attend_kv8(const pie_fwd_plan_t& p, const void* q_rot, const uint8_t* k_pool,
                              const uint8_t* v_pool, const uint8_t* k_scale,
                              const uint8_t* v_scale, const uint32_t* mask_words,
                              uint32_t* status, cudaStream_t s) {
  const int D = p.desc.head_dim, P = p.desc.page_size;
  CUtensorMap km, vm;
  const cuuint64_t dims[3] = {cuuint64_t(D), cuuint64_t(P),
                              cuuint64_t(p.dev.num_pool_pages) * p.desc.num_kv_heads};
  const cuuint64_t str[2] = {cuuint64_t(D), cuuint64_t(D) * P};
  const cuuint32_t box[3] = {cuuint32_t(D), cuuint32_t(P), 1};
  const CUtensorMapSwizzle sw = D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  if (!tc::make_map(&km, k_pool, 3, dims, str, box, sw, CU_TENSOR_MAP_DATA_TYPE_UINT8) ||
      !tc::make_map(&vm, v_pool, 3, dims, str, box, sw, CU_TENSOR_MAP_DATA_TYPE_UINT8))
    return cudaErrorInvalidValue;
  const bool bf = p.desc.dtype == PIE_BF16;
  auto f = D == 128 ? (bf ? launch_a8_all<__nv_bfloat16, 128> : launch_a8_all<float, 128>)
                    : (bf ? launch_a8_all<__nv_bfloat16, 64> : launch_a8_all<float, 64>);
  return f(p, q_rot, k_scale, v_scale, mask_words, status, km, vm, s);
}

}  // namespace pie
