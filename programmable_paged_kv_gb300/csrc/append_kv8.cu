// Step 1 of a ForwardPass into a cache of 8-bit codes (Pie "The forward pass",
// State geometry: positions, slots): RoPE of the rows, and the write of their
// K and V as e4m3 codes with one power-of-two scale per (page, kv head).
//
// One page is one unit: its slots share their scales, so the rows of the pass
// that write it (the plan's WriteBlock) are quantised together with the page's
// live codes.  One warp takes one kv head of one page, K and V, and the query
// heads of its group for the same rows; the warps of a CTA share the rows'
// rotation angles.  The scale is a power of two: e4m3 is a floating format, so
// a finer scale would buy no precision, products with it are exact, and a page
// whose scale grows shifts its codes' exponents (only values that fall under
// e4m3's smallest normal lose bits).  A page's codes are read only then.
//
// A code is the nearest to the exactly rotated value, so it does not depend on
// how the rotation was evaluated:
//   * the angle is positions[r] * base^(-2i/d) / (2 pi) turns in 0.64 fixed
//     point: the 64-bit product wraps, which is the reduction modulo a turn,
//     without error;
//   * sine and cosine of the remaining eighth of a turn are their power series
//     in 64-bit fixed point (error below 2^-40), kept as two floats each;
//   * x cos - y sin is a sum of exact products (FMA residuals), rounded to odd
//     in fp32, so that the rounding to e4m3 that follows is the only one.
// Queries need no more than fp32 and take the leading floats alone.
//
// Bound: HBM for prompts (q, k, v in, q_rot and codes out), latency for a
// decode step.

#include "fp8.cuh"

namespace pie {

namespace ak {

constexpr int WARPS = 4;

// cos and sin of 2 pi t / 2^64, each as a sum of two floats
struct Angle {
  float ch, cl, sh, sl;
};

// v / 2^63 as two floats (v <= 2^63)
__device__ __forceinline__ void split63(uint64_t v, float& hi, float& lo) {
  const float h = __ull2float_rz(v);
  lo = __ull2float_rn(v - static_cast<uint64_t>(h)) * 0x1p-63f;
  hi = h * 0x1p-63f;
}

__device__ __forceinline__ Angle angle(uint64_t turns) {
  // the nearest quarter turn, and what is left of it: |r| <= 2^61
  const uint32_t quarter = static_cast<uint32_t>((turns + (uint64_t(1) << 61)) >> 62);
  const int64_t r = static_cast<int64_t>(turns - (uint64_t(quarter) << 62));
  const uint64_t a = static_cast<uint64_t>(r < 0 ? -r : r);
  // theta = 2 pi a / 2^64 <= pi/4, times 2^63 (pi in 2.62 fixed point)
  const uint64_t theta = __umul64hi(a << 2, 0xC90FDAA22168C235ull);
  const uint64_t x = __umul64hi(theta << 1, theta << 1);  // theta^2, 0.64
  // 1 - cos = x (1/2! - x (1/4! - ...)), theta - sin = theta x (1/3! - ...):
  // Horner in 0.64 fixed point, 1/k! times 2^64
  constexpr double one = 18446744073709551616.0;
  constexpr uint64_t i2 = uint64_t(one / 2), i4 = uint64_t(one / 24), i6 = uint64_t(one / 720),
                     i8 = uint64_t(one / 40320), i10 = uint64_t(one / 3628800),
                     i12 = uint64_t(one / 479001600), i3 = uint64_t(one / 6),
                     i5 = uint64_t(one / 120), i7 = uint64_t(one / 5040),
                     i9 = uint64_t(one / 362880), i11 = uint64_t(one / 39916800),
                     i13 = uint64_t(one / 6227020800.0);
  uint64_t c = i10 - __umul64hi(x, i12);
  c = i8 - __umul64hi(x, c);
  c = i6 - __umul64hi(x, c);
  c = i4 - __umul64hi(x, c);
  c = i2 - __umul64hi(x, c);
  const uint64_t cosv = (uint64_t(1) << 63) - (__umul64hi(x, c) >> 1);
  uint64_t s = i11 - __umul64hi(x, i13);
  s = i9 - __umul64hi(x, s);
  s = i7 - __umul64hi(x, s);
  s = i5 - __umul64hi(x, s);
  s = i3 - __umul64hi(x, s);
  const uint64_t sinv = theta - __umul64hi(theta, __umul64hi(x, s));
  float ch, cl, sh, sl;
  split63(cosv, ch, cl);
  split63(sinv, sh, sl);
  if (r < 0) sh = -sh, sl = -sl;
  // turn by the quarters
  Angle o;
  const bool swap = quarter & 1;
  o.ch = swap ? sh : ch;
  o.cl = swap ? sl : cl;
  o.sh = swap ? ch : sh;
  o.sl = swap ? cl : sl;
  const uint32_t qd = quarter & 3;
  if (qd == 1 || qd == 2) o.ch = -o.ch, o.cl = -o.cl;
  if (qd >= 2) o.sh = -o.sh, o.sl = -o.sl;
  return o;
}

// x c - y s for c = ch + cl, s = sh + sl, rounded to odd in fp32: the nearest
// float, moved to its odd neighbour towards the exact value when the float is
// even and inexact (a later rounding to fewer bits then sees on which side of
// its ties the value lies)
__device__ __forceinline__ float rot_odd(float x, float ch, float cl, float y, float sh, float sl) {
  // (the intrinsics keep the compiler from contracting into other FMAs)
  const float p = __fmul_rn(x, ch), pe = fmaf(x, ch, -p);
  const float q = __fmul_rn(y, sh), qe = fmaf(y, sh, -q);
  const float t = __fsub_rn(p, q);  // t + te = p - q exactly (Knuth's two-sum)
  if (!(fabsf(t) < INFINITY)) return t;
  const float b = __fsub_rn(t, p);
  const float te = __fsub_rn(__fsub_rn(p, __fsub_rn(t, b)), __fadd_rn(q, b));
  const float lo = __fadd_rn(te, __fadd_rn(__fsub_rn(pe, qe), fmaf(x, cl, -__fmul_rn(y, sl))));
  const float h = __fadd_rn(t, lo);
  const float rest = __fsub_rn(lo, __fsub_rn(h, t));
  uint32_t u = __float_as_uint(h);
  if (rest != 0.f && !(u & 1u) && (u & 0x7FFFFFFFu) != 0u) u += ((rest > 0.f) == (h > 0.f)) ? 1u : -1u;
  return __uint_as_float(u);
}

// the smallest e in [kMinExp, kMaxExp] with amax <= 448 * 2^e
__device__ __forceinline__ int needed_exp(float amax) {
  const uint32_t u = __float_as_uint(amax);
  // 448 = 1.75 * 2^8
  const int e = int(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return max(fp8::kMinExp, min(fp8::kMaxExp, e));
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
  return x;
}

template <typename T, int N>
__device__ __forceinline__ void load_n(const T* p, float* f) {
  if constexpr (sizeof(T) * N == 16) {
    unpack16<T>(*reinterpret_cast<const uint4*>(p), f);
  } else if constexpr (sizeof(T) * N == 8) {
    unpack8<T>(*reinterpret_cast<const uint2*>(p), f);
  } else if constexpr (sizeof(T) * N == 4 && N == 2) {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
    f[0] = __uint_as_float(u << 16);
    f[1] = __uint_as_float(u & 0xFFFF0000u);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = Elem<T>::to_f(p[i]);
  }
}
template <typename T, int N>
__device__ __forceinline__ void store_n(T* p, const float* f) {
  if constexpr (sizeof(T) == 2 && N == 2) {
    __nv_bfloat162 h = __floats2bfloat162_rn(f[0], f[1]);
    *reinterpret_cast<__nv_bfloat162*>(p) = h;
  } else if constexpr (sizeof(T) == 4 && N == 2) {
    *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = Elem<T>::from_f(f[i]);
  }
}
template <int N>
__device__ __forceinline__ void store_codes(uint8_t* p, const float* f) {
  if constexpr (N == 4)
    *reinterpret_cast<uint32_t*>(p) =
        fp8::from_float2(f[0], f[1]) | (fp8::from_float2(f[2], f[3]) << 16);
  else if constexpr (N == 2)
    *reinterpret_cast<uint16_t*>(p) = uint16_t(fp8::from_float2(f[0], f[1]));
  else
    *p = uint8_t(fp8::from_float2(f[0], 0.f));
}

// The page's live codes of one kv head (rows of D bytes, offsets `keep`) from
// scale 2^old to 2^e.
template <int D>
__device__ __forceinline__ void regrow(uint8_t* rows, uint32_t keep, int old, int e, int lane) {
  constexpr int N = D / 32;  // codes per lane
  const int diff = old - e;  // < 0
  while (keep) {
    const int o = __ffs(keep) - 1;
    keep &= keep - 1;
    uint8_t* p = rows + o * D + lane * N;
    const uint32_t c = N == 4 ? *reinterpret_cast<const uint32_t*>(p)
                              : uint32_t(*reinterpret_cast<const uint16_t*>(p));
    uint32_t h[2];
    fp8::to_half2x2(c, h[0], h[1]);
    float f[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
      f[2 * i] = fp8::scale2(v.x, diff);
      f[2 * i + 1] = fp8::scale2(v.y, diff);
    }
    store_codes<N>(p, f);
  }
}

}  // namespace ak

template <typename T, int D>
__global__ void __launch_bounds__(ak::WARPS * 32) append_kv8_kernel(
    DevMeta m, int Hq, int Hkv, int P, const T* q, const T* k, const T* v, T* q_rot,
    uint8_t* k_pool, uint8_t* v_pool, uint8_t* k_scale, uint8_t* v_scale,
    const int32_t* frozen_len, uint32_t* status) {
  using namespace ak;
  constexpr int H = D / 2;
  constexpr int PL = H / 32;  // rotation pairs per lane: elements i0 .. and H + i0 ..
  constexpr int VL = D / 32;  // V elements per lane
  extern __shared__ Angle ang[];  // [rows of the page][H]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the plan's own data (uploaded before any kernel of the pass) and the
  // angles, while the kernel before this one may still run
  const WriteBlock wb = m.wblocks[blockIdx.x];
  const int32_t* rows = m.wrow + wb.row0;
  for (int i = threadIdx.x; i < wb.nrows * H; i += WARPS * 32)
    ang[i] = angle(uint64_t(uint32_t(m.positions[rows[i / H]])) * m.rope_turn[i % H]);
  const int slot0 = wb.lpage * P;
  const int kv_len = m.kv_len[wb.lane];
  grid_dep_wait();
  grid_dep_launch();
  __syncthreads();
  const int frozen = frozen_len[wb.lane];
  if (blockIdx.y == 0 && threadIdx.x < wb.nrows) {
    const int r = rows[threadIdx.x], slot = m.slots[r];
    if (slot < frozen) set_status(status, PIE_STATUS_FROZEN_WRITE);
    if (r == m.row_indptr[wb.lane] && m.fold_mode[wb.lane] != PIE_FOLD_NONE && slot != frozen)
      set_status(status, PIE_STATUS_FOLD_GAP);
  }
  const int g = blockIdx.y * WARPS + warp;
  if (g >= Hkv) return;
  const int G = Hq / Hkv;
  const int i0 = lane * PL;

  // ---- K and V: the slots written now, the live ones that stay
  const bool wr = lane < P && ((wb.written >> lane) & 1u) && slot0 + lane >= frozen;
  const bool live = lane < P && slot0 + lane < max(kv_len, frozen);
  const uint32_t writes = __ballot_sync(0xffffffffu, wr);
  const uint32_t keep = __ballot_sync(0xffffffffu, live && !wr);
  if (writes) {
    const int64_t cell = int64_t(wb.page) * Hkv + g;
    auto rotated = [&](int i, float* lo, float* hi) {  // row i of the page, this lane's pairs
      const T* src = k + (int64_t(rows[i]) * Hkv + g) * D;
      float x[PL], y[PL];
      load_n<T, PL>(src + i0, x);
      load_n<T, PL>(src + H + i0, y);
#pragma unroll
      for (int e = 0; e < PL; ++e) {
        const Angle a = ang[i * H + i0 + e];
        lo[e] = rot_odd(x[e], a.ch, a.cl, y[e], a.sh, a.sl);
        hi[e] = rot_odd(y[e], a.ch, a.cl, -x[e], a.sh, a.sl);
      }
    };
    float ka = 0.f, va = 0.f;
    for (int i = 0; i < wb.nrows; ++i) {
      const int r = rows[i];
      if (m.slots[r] < frozen) continue;
      float lo[PL], hi[PL], f[VL];
      rotated(i, lo, hi);
      load_n<T, VL>(v + (int64_t(r) * Hkv + g) * D + lane * VL, f);
#pragma unroll
      for (int e = 0; e < PL; ++e) ka = fmaxf(ka, fmaxf(fabsf(lo[e]), fabsf(hi[e])));
#pragma unroll
      for (int e = 0; e < VL; ++e) va = fmaxf(va, fabsf(f[e]));
    }
    const int k_old = int(k_scale[cell]) - fp8::kBias, v_old = int(v_scale[cell]) - fp8::kBias;
    int ke = needed_exp(warp_max(ka)), ve = needed_exp(warp_max(va));
    uint8_t* kc = k_pool + cell * P * D;
    uint8_t* vc = v_pool + cell * P * D;
    if (keep) {
      ke = max(ke, k_old);
      ve = max(ve, v_old);
      if (ke > k_old) regrow<D>(kc, keep, k_old, ke, lane);
      if (ve > v_old) regrow<D>(vc, keep, v_old, ve, lane);
    }
    __syncwarp();  // every lane has read the old scales
    if (lane == 0) {
      k_scale[cell] = uint8_t(ke + fp8::kBias);
      v_scale[cell] = uint8_t(ve + fp8::kBias);
    }
    for (int i = 0; i < wb.nrows; ++i) {
      const int r = rows[i], slot = m.slots[r];
      if (slot < frozen) continue;
      const int o = (slot - slot0) * D;
      float lo[PL], hi[PL], f[VL];
      rotated(i, lo, hi);
#pragma unroll
      for (int e = 0; e < PL; ++e) {
        lo[e] = fp8::scale2(lo[e], -ke);
        hi[e] = fp8::scale2(hi[e], -ke);
      }
      store_codes<PL>(kc + o + i0, lo);
      store_codes<PL>(kc + o + H + i0, hi);
      load_n<T, VL>(v + (int64_t(r) * Hkv + g) * D + lane * VL, f);
#pragma unroll
      for (int e = 0; e < VL; ++e) f[e] = fp8::scale2(f[e], -ve);
      store_codes<VL>(vc + o + lane * VL, f);
    }
  }

  // ---- the group's query heads, frozen rows included
  for (int u = 0; u < wb.nrows * G; ++u) {
    const int i = u / G;
    const int64_t at = (int64_t(rows[i]) * Hq + g * G + u % G) * D;
    float x[PL], y[PL], lo[PL], hi[PL];
    load_n<T, PL>(q + at + i0, x);
    load_n<T, PL>(q + at + H + i0, y);
#pragma unroll
    for (int e = 0; e < PL; ++e) {
      const Angle a = ang[i * H + i0 + e];
      lo[e] = fmaf(x[e], a.ch, -(y[e] * a.sh));
      hi[e] = fmaf(y[e], a.ch, x[e] * a.sh);
    }
    store_n<T, PL>(q_rot + at + i0, lo);
    store_n<T, PL>(q_rot + at + H + i0, hi);
  }
}

template <typename T, int D>
static cudaError_t launch_ak(const pie_fwd_plan_t& p, const void* q, const void* k, const void* v,
                             void* q_rot, uint8_t* k_pool, uint8_t* v_pool, uint8_t* k_scale,
                             uint8_t* v_scale, const int32_t* frozen, uint32_t* status,
                             cudaStream_t s) {
  const int Hkv = p.desc.num_kv_heads;
  const dim3 grid(p.num_wblocks, (Hkv + ak::WARPS - 1) / ak::WARPS);
  const size_t smem = size_t(p.desc.page_size) * (D / 2) * sizeof(ak::Angle);  // at most 32 KB
  return launch_dependent(append_kv8_kernel<T, D>, grid, dim3(ak::WARPS * 32), smem, s, true, p.dev,
                          p.desc.num_q_heads, Hkv, p.desc.page_size, static_cast<const T*>(q),
                          static_cast<const T*>(k), static_cast<const T*>(v),
                          static_cast<T*>(q_rot), k_pool, v_pool, k_scale, v_scale, frozen, status);
}

cudaError_t launch_append_kv8(const pie_fwd_plan_t& p, const void* q, const void* k, const void* v,
                              void* q_rot, uint8_t* k_pool, uint8_t* v_pool, uint8_t* k_scale,
                              uint8_t* v_scale, const int32_t* frozen, uint32_t* status,
                              cudaStream_t s) {
  const bool bf = p.desc.dtype == PIE_BF16;
  auto f = p.desc.head_dim == 128 ? (bf ? launch_ak<__nv_bfloat16, 128> : launch_ak<float, 128>)
                                  : (bf ? launch_ak<__nv_bfloat16, 64> : launch_ak<float, 64>);
  return f(p, q, k, v, q_rot, k_pool, v_pool, k_scale, v_scale, frozen, status, s);
}

}  // namespace pie
