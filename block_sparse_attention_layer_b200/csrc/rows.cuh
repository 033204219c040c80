// Rows of one head in registers, shared by the kernels around the attention
// (norm + rotation forward and backward, 8-bit checkpoints).
//
// A row of D elements (64 or 128) lies over G = D / 8 neighbouring lanes,
// eight elements a lane, so a warp holds R = 32 / G rows.  bf16: elements
// 8 l .. 8 l + 7 (one 16-byte access).  fp32: 4 l .. 4 l + 3 and the same in
// the row's second half (two 16-byte accesses, each contiguous over the
// lanes).  Adjacent elements (2p, 2p + 1) always share a lane.
//
// 8-bit checkpoints: a group of values with a = max |x| is stored as codes
// round-half-even(127 x / a) of the exact quotient and the fp32 scale a / 127;
// it reads back as code * scale, off by at most a / 254 (+ the rounding of
// the scale).  A group with an infinity or NaN gets a NaN scale and reads back
// as NaN throughout; one with a < 2^-119 (whose scale would be subnormal) is
// stored as zeros.
#pragma once

#include <atomic>

#include "common.cuh"

namespace vmoba {
namespace rows {

constexpr unsigned kAll = 0xFFFFFFFFu;

// n / d for 0 <= n < 2^31 by a multiplication (round-up reciprocal in 33 bits).
struct FastDiv {
  uint32_t mul, shift;
  FastDiv() = default;
  explicit FastDiv(uint32_t d) {
    shift = 0;
    while ((1u << shift) < d) ++shift;
    mul = (uint32_t)((((1ull << shift) - d) << 32) / d + 1);
  }
  __host__ __device__ __forceinline__ int div(int n) const {
#ifdef __CUDA_ARCH__
    return (int)((__umulhi(mul, (uint32_t)n) + (uint32_t)n) >> shift);
#else
    return (int)(((uint32_t)(((uint64_t)mul * (uint32_t)n) >> 32) + (uint32_t)n) >> shift);
#endif
  }
};

template <typename E>
struct Raw;  // a lane's eight elements as loaded
template <>
struct Raw<__nv_bfloat16> { uint4 u; };
template <>
struct Raw<float> { float4 a, b; };

// Element i (0..7) of lane l within the row.
template <typename E, int D>
__device__ __forceinline__ int elem_at(int l, int i) {
  if (sizeof(E) == 2) return l * 8 + i;
  return i < 4 ? l * 4 + i : D / 2 + l * 4 + i - 4;
}

// Values pass once: no place in L1.
__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ float4 as_float4(const uint4& v) {
  return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z),
                     __uint_as_float(v.w));
}

// Asynchronous copies of a lane's own values into its own place in shared
// memory: only the lane that asked for them reads them, so its own wait is the
// only one needed, and loads stay in flight without holding registers.
template <int Bytes>
__device__ __forceinline__ void fetch(void* to, const void* from) {
  const uint32_t dst = (uint32_t)__cvta_generic_to_shared(to);
  if constexpr (Bytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(from) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" :: "r"(dst), "l"(from), "n"(Bytes)
                 : "memory");
}
__device__ __forceinline__ void fetch_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>  // at most the N newest groups still in flight
__device__ __forceinline__ void fetch_wait() {
  asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory");
}

// A lane's pointer into one tensor, held in registers through a loop (the
// compiler otherwise forms it anew at every use), and `n` strides from it.
template <typename T>
__device__ __forceinline__ T* pinned(T* p) {
  asm volatile("" : "+l"(p));
  return p;
}
template <typename T>
__device__ __forceinline__ T* at_bytes(T* p, int n, uint32_t stride) {
  return reinterpret_cast<T*>(
      reinterpret_cast<uintptr_t>(p) + (unsigned long long)(uint32_t)n * stride);
}

// A warp's place for one access of its R rows, in the order of the lanes;
// `from` is where the lane's first 16 bytes lie.
template <typename E, int D>
struct Slot {
  static constexpr int kBytes = 32 * sizeof(Raw<E>);
  __device__ __forceinline__ static void ask(char* s, const char* from, int lane) {
    fetch<16>(s + lane * 16, from);
    if constexpr (sizeof(E) == 4) fetch<16>(s + 512 + lane * 16, from + D * 2);
  }
  __device__ __forceinline__ static Raw<E> get(const char* s, int lane) {
    Raw<E> r;
    if constexpr (sizeof(E) == 2) {
      r.u = *reinterpret_cast<const uint4*>(s + lane * 16);
    } else {
      r.a = *reinterpret_cast<const float4*>(s + lane * 16);
      r.b = *reinterpret_cast<const float4*>(s + 512 + lane * 16);
    }
    return r;
  }
  // `to` is where the lane's first 16 bytes go
  __device__ __forceinline__ static void put(char* to, const Raw<E>& r) {
    if constexpr (sizeof(E) == 2) {
      __stcg(reinterpret_cast<uint4*>(to), r.u);
    } else {
      __stcg(reinterpret_cast<float4*>(to), r.a);
      __stcg(reinterpret_cast<float4*>(to + D * 2), r.b);
    }
  }
};

// T rows of codes (raw q, k and, if T = 3, v of a token and head) and their
// scales, of two neighbouring heads of R tokens or of one head of two times R.
// Two heads' codes of a token are neighbours, so sixteen of them are one copy
// and a lane reads what others asked for: a __syncwarp stands between its
// wait and its reads, and between those and the next copies.
template <typename E, int D, int T, bool TwoHeads>
struct CodeRows {
  static constexpr int G = D / 8, R = 32 / G, kVec = TwoHeads ? 16 : 8;
  static constexpr int kScales = T * 512, kBytes = kScales + 2 * R * T * 4;
  // the lane's pointers for head h: codes of kind i, and the scale of kind l
  __device__ __forceinline__ static const char* codes_at(const int8_t* codes, int i, int h,
                                                         int n_h, int l) {
    return reinterpret_cast<const char*>(codes) + ((long long)i * n_h + h) * D + l * kVec;
  }
  __device__ __forceinline__ static const float* scale_at(const float* scales, int h, int n_h,
                                                          int l) {
    return scales + min(l, T - 1) * n_h + h;
  }
  __device__ __forceinline__ static void ask(char* s, const char* const (&codes)[T],
                                             const float* scale, int n, int n_h, int u, int sub,
                                             int l) {
    if (TwoHeads && u == 1) return;
    const uint32_t stride = 3 * n_h;
#pragma unroll
    for (int i = 0; i < T; ++i)
      fetch<kVec>(s + i * 512 + (TwoHeads ? 0 : u * 256) + (sub * G + l) * kVec,
                  at_bytes(codes[i], n, stride * D));
    if (l < T) {
      const float* from = at_bytes(scale, n, stride * 4);
      float* to = reinterpret_cast<float*>(s + kScales);
      if constexpr (TwoHeads)
        fetch<8>(to + (sub * T + l) * 2, from);
      else
        fetch<4>(to + (u * R + sub) * T + l, from);
    }
  }
  __device__ __forceinline__ static uint2 codes(const char* s, int i, int u, int sub, int l) {
    s += i * 512 + (TwoHeads ? (sub * 2 + u) * D : u * 256 + sub * D);
    if constexpr (sizeof(E) == 2) return reinterpret_cast<const uint2*>(s)[l];
    const uint32_t* p = reinterpret_cast<const uint32_t*>(s);
    return make_uint2(p[l], p[D / 8 + l]);
  }
  __device__ __forceinline__ static float scale(const char* s, int i, int u, int sub) {
    const float* p = reinterpret_cast<const float*>(s + kScales);
    return TwoHeads ? p[(sub * T + i) * 2 + u] : p[(u * R + sub) * T + i];
  }
};

// A lane's eight values as four adjacent pairs: fp32 arithmetic runs on pairs
// (two lanes of one instruction each), and a rotation turns one.
struct Vals {
  float2 p[4];
  __device__ __forceinline__ float& at(int i) { return i & 1 ? p[i >> 1].y : p[i >> 1].x; }
  __device__ __forceinline__ float at(int i) const { return i & 1 ? p[i >> 1].y : p[i >> 1].x; }
};

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

__device__ __forceinline__ Vals unpack(const Raw<__nv_bfloat16>& r) {
  const uint32_t w[4] = {r.u.x, r.u.y, r.u.z, r.u.w};
  Vals v;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v.p[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  return v;
}
__device__ __forceinline__ Vals unpack(const Raw<float>& r) {
  return {make_float2(r.a.x, r.a.y), make_float2(r.a.z, r.a.w), make_float2(r.b.x, r.b.y),
          make_float2(r.b.z, r.b.w)};
}

// The one rounding of a result: to the storage type, nearest even.
__device__ __forceinline__ uint32_t bf16x2(float2 v) {
  const __nv_bfloat162 w = __float22bfloat162_rn(v);
  return *reinterpret_cast<const uint32_t*>(&w);
}
__device__ __forceinline__ void pack(const Vals& v, Raw<__nv_bfloat16>& r) {
  r.u = make_uint4(bf16x2(v.p[0]), bf16x2(v.p[1]), bf16x2(v.p[2]), bf16x2(v.p[3]));
}
__device__ __forceinline__ void pack(const Vals& v, Raw<float>& r) {
  r.a = make_float4(v.p[0].x, v.p[0].y, v.p[1].x, v.p[1].y);
  r.b = make_float4(v.p[2].x, v.p[2].y, v.p[3].x, v.p[3].y);
}

// Four rows' sums over their G lanes at once (every lane of the warp takes
// part).  Two exchange steps leave each lane with a quarter of one sum, the
// rest of the tree adds those; nine shuffles instead of 4 log2 G.  The lane
// that holds sum k is k * G / 4 of the group.
template <int G>
__device__ __forceinline__ float quarter_sums(const float (&v)[4], int l) {
  const bool hi = l & (G / 2), hi2 = l & (G / 4);
  float s0 = hi ? v[2] : v[0], s1 = hi ? v[3] : v[1];
  s0 += __shfl_xor_sync(kAll, hi ? v[0] : v[2], G / 2);
  s1 += __shfl_xor_sync(kAll, hi ? v[1] : v[3], G / 2);
  float s = (hi2 ? s1 : s0) + __shfl_xor_sync(kAll, hi2 ? s0 : s1, G / 4);
#pragma unroll
  for (int o = G / 8; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
  return s;
}
template <int G>
__device__ __forceinline__ void spread(float s, float (&v)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = __shfl_sync(kAll, s, k * (G / 4), G);
}

// Sum over the G lanes of a row.
template <int G>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
template <int G>
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

__device__ __forceinline__ float lane_dot(const Vals& a, const Vals& b) {
  float2 s = __fmul2_rn(a.p[0], b.p[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) s = __ffma2_rn(a.p[i], b.p[i], s);
  return s.x + s.y;
}

// Waits until the stream's previous kernel has finished and its writes are
// visible (every access to global memory comes after this), and lets the next
// one be set up once all of this grid's CTAs run.  Global memory is read by
// plain loads only: a read-only one (__ldg, or through a const __restrict__
// parameter) holds its data to be constant for as long as the kernel lives,
// which begins before this, and may be moved up across it.
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ---- 8-bit groups ----

// Group maxima of |x| as bits: an infinity or NaN sorts above every finite
// value.  bf16 works on the stored 16 bits, two values an instruction, and
// two groups share the words of one shuffle tree.
__device__ __forceinline__ uint32_t max16x2(uint32_t a, uint32_t b) {
  uint32_t m;
  asm("max.u16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
  return m;
}
__device__ __forceinline__ uint32_t lane_max(const Raw<__nv_bfloat16>& r) {
  constexpr uint32_t kAbs = 0x7FFF7FFFu;
  return max16x2(max16x2(r.u.x & kAbs, r.u.y & kAbs), max16x2(r.u.z & kAbs, r.u.w & kAbs));
}
template <int G>
__device__ __forceinline__ void group_max(const Raw<__nv_bfloat16>& a,
                                          const Raw<__nv_bfloat16>& b, uint32_t& ma,
                                          uint32_t& mb) {
  const uint32_t wa = lane_max(a), wb = lane_max(b);
  uint32_t m = max16x2(__byte_perm(wa, wb, 0x5410), __byte_perm(wa, wb, 0x7632));
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) m = max16x2(m, __shfl_xor_sync(kAll, m, o));
  ma = m << 16;
  mb = m & 0xFFFF0000u;
}
__device__ __forceinline__ uint32_t lane_max(const Raw<float>& r) {
  const Vals v = unpack(r);
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v.at(i)) & 0x7FFFFFFFu);
  return m;
}
template <int G>
__device__ __forceinline__ void group_max(const Raw<float>& a, const Raw<float>& b, uint32_t& ma,
                                          uint32_t& mb) {
  ma = row_max<G>(lane_max(a));
  mb = row_max<G>(lane_max(b));
}

// The code of one value for which the fp32 quotient cannot decide: rounds by
// the sign of 127 x - T a, T the half integer next to c.  Both products are
// taken with their rounding errors (an fma gives each exactly) and subtracted
// leading parts first, so the sign is the exact one; zero is a tie, which
// goes to the even code.
__device__ __forceinline__ float settle(float x, float a, float c, float d) {
  const float T = c + copysignf(0.5f, d);
  const float q = 127.0f * x, p = T * a;
  const float s = (q - p) + (fmaf(127.0f, x, -q) - fmaf(T, a, -p));
  return s > 0.f ? T + 0.5f : (s < 0.f ? T - 0.5f : 2.0f * rintf(0.5f * T));
}

__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float m;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(fabsf(b)), "f"(fabsf(c)));
  return m;
}

// Codes of a lane's eight values, byte i = element i, for a group whose
// max |x| has the bits `m`; scale gets the group's.  The quotient is x *
// (127 / a) with the factor in fp32 (reciprocal, product: off by less than
// 2^-22 of it), rounded to an integer by the fma that adds 1.5 * 2^23.
//
// bf16: x and a have eight bits each, so a quotient that is no tie is at least
// 2^-16 of itself away from one, and unless a's significand is 254 / 128 the
// only tie is 63.5 (x = a / 2), which goes up to 64.  A factor 2^-19 larger
// than 127 / a therefore rounds every quotient as asked (for every pair of
// significands: test_every_pair_of_bf16_significands); with 254 / 128 each
// value is settled exactly.  That is one fma a value; testing every quotient's distance from a border
// instead, as fp32 does, sent half of the groups the settling way (an element
// is a / 2 in that many) and took 71 us against 55 for 55296 x 1536.
// fp32: where a quotient's distance from its integer is so close to a half
// that the factor's error could decide, the lane settles its eight.
// A group with a outside [2^-119, 2^100] (nothing to scale, not finite, or
// with a subnormal reciprocal) goes the settling way too.
template <typename E>
__device__ __forceinline__ uint2 encode8(const Vals& v, uint32_t m, float& scale) {
  const float a = __uint_as_float(m);
  // a / 127 correctly rounded: a first quotient and one step with its exact
  // remainder (Markstein's division; test_every_fp32_scale has every significand)
  constexpr float kInv = 1.0f / 127.0f;
  const float q = a * kInv;
  scale = fmaf(fmaf(-127.0f, q, a), kInv, q);
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(a));
  inv *= sizeof(E) == 2 ? 127.0f * (1.0f + 0x1p-19f) : 127.0f;
  constexpr float kMagic = 12582912.0f;
  Vals z;
#pragma unroll
  for (int i = 0; i < 4; ++i) z.p[i] = __ffma2_rn(v.p[i], both(inv), both(kMagic));
  constexpr uint32_t kLow = 0x04000000u, kHigh = 0x71800000u;      // 2^-119, 2^100
  bool rare = m - kLow > kHigh - kLow;
  if constexpr (sizeof(E) == 2) {
    rare = rare || (m & 0x007F0000u) == 0x007E0000u;
  } else {
    float border = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 d =
          __ffma2_rn(v.p[i], both(inv), __ffma2_rn(z.p[i], both(-1.f), both(kMagic)));
      border = max_abs3(border, d.x, d.y);
    }
    rare = rare || border > 0.5f - 0x1p-14f;
  }
  if (rare) {
    const bool bad = m >= 0x7F800000u, none = m < kLow;
    if (bad) scale = __uint_as_float(0x7FC00000u);
    if (none) scale = 0.f;
    // the largest fp32 number: 127 a / 127 must not read back as infinite
    if (!bad && scale * 127.0f > 0x1.fffffep127f)
      scale = __uint_as_float(__float_as_uint(scale) - 1u);
    const float down = m > kHigh ? 0x1p-8f : 1.0f;
    const float by = __fdividef(127.0f, a * down) * down;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float c = rintf(v.at(i) * by);
      const float code = settle(v.at(i) * down, a * down, c, fmaf(v.at(i), by, -c));
      z.at(i) = bad || none ? kMagic : code + kMagic;
    }
  }
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(z.at(i));
  const uint32_t lo = __byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040),
                                  0x5410);
  const uint32_t hi = __byte_perm(__byte_perm(w[4], w[5], 0x0040), __byte_perm(w[6], w[7], 0x0040),
                                  0x5410);
  return make_uint2(lo, hi);
}

// Eight codes as fp32.  A byte c + 128 in the mantissa of 2^23 is 2^23 + 128 + c.
__device__ __forceinline__ Vals code_values(uint2 c) {
  const uint32_t w[2] = {c.x ^ 0x80808080u, c.y ^ 0x80808080u};
  Vals v;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v.at(i) = __uint_as_float(__byte_perm(w[i >> 2], 0x4B000000u, 0x7440 + (i & 3)));
#pragma unroll
  for (int i = 0; i < 4; ++i) v.p[i] = __fadd2_rn(v.p[i], both(-8388736.0f));
  return v;
}

__device__ __forceinline__ Vals scaled(Vals v, float by) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v.p[i] = __fmul2_rn(v.p[i], both(by));
  return v;
}

// code * scale, one rounding.
__device__ __forceinline__ Vals decode8(uint2 c, float scale) {
  return scaled(code_values(c), scale);
}

// A lane's eight codes into a row of D codes, from the element order of E;
// `to` is where its first go.
template <typename E, int D>
__device__ __forceinline__ void store_codes(char* to, uint2 c) {
  if (sizeof(E) == 2) {
    __stcg(reinterpret_cast<uint2*>(to), c);
  } else {
    __stcg(reinterpret_cast<uint32_t*>(to), c.x);
    __stcg(reinterpret_cast<uint32_t*>(to + D / 2), c.y);
  }
}

// ---- norm ----

// 1 / sqrt(v) within 2 ulp; v is never subnormal here (eps >= 1e-30).
__device__ __forceinline__ float rsqrt_normal(float v) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// r[k] = 1 / sqrt(mean x^2 + eps) of four rows.  Where a row's squares leave
// fp32's range it is first scaled by pre[k] = 2^-80 (x changes, and eps is
// taken times its square); else pre[k] = 1.
template <int D>
__device__ __forceinline__ void inv_rms(Vals (&x)[4], float eps, int l, float (&r)[4],
                                        float (&pre)[4]) {
  constexpr int G = D / 8;
  float ss[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    ss[k] = lane_dot(x[k], x[k]);
    pre[k] = 1.f;
  }
  const float s = quarter_sums<G>(ss, l);
  spread<G>(rsqrt_normal(fmaf(s, 1.0f / D, eps)), r);
  if (__any_sync(kAll, !(s < 0x1p100f))) {
    float sum[4];
    spread<G>(s, sum);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const bool big = !(sum[k] < 0x1p100f);
      if (big) {
        pre[k] = 0x1p-80f;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[k].at(i) *= 0x1p-80f;
      }
      const float again = row_sum<G>(lane_dot(x[k], x[k]));
      if (big) r[k] = rsqrt_normal(fmaf(again, 1.0f / D, eps * 0x1p-80f * 0x1p-80f));
    }
  }
}

// x r of four rows (and r) from raw values: x becomes x r.
template <int D>
__device__ __forceinline__ void normalise(Vals (&x)[4], float eps, int l, float (&r)[4]) {
  float pre[4];
  inv_rms<D>(x, eps, l, r, pre);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    x[k] = scaled(x[k], r[k]);
    r[k] *= pre[k];
  }
}

// The same from codes, without their scales s where these are ordinary:
// x r = c / sqrt(mean c^2 + eps / s^2), the sum of squared codes an exact
// integer.  Where eps / s^2 is huge (or s is zero or NaN) the values are formed.
template <int D>
__device__ __forceinline__ void normalise(const uint2 (&c)[4], const float (&s)[4], float eps,
                                          int l, Vals (&x)[4], float (&r)[4]) {
  constexpr int G = D / 8;
  float ss[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    ss[k] = (float)__dp4a((int)c[k].x, (int)c[k].x, __dp4a((int)c[k].y, (int)c[k].y, 0));
  const bool hi = l & (G / 2), hi2 = l & (G / 4);
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;"
      : "=f"(inv) : "f"(hi ? (hi2 ? s[3] : s[2]) : (hi2 ? s[1] : s[0])));
  const float e = eps * inv * inv;
  const float sum = quarter_sums<G>(ss, l);
  if (!__any_sync(kAll, !(e < 0x1p100f))) {
    const float rc = rsqrt_normal(fmaf(sum, 1.0f / D, e));
    float rx[4];
    spread<G>(rc, rx);
    spread<G>(rc * inv, r);
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = scaled(code_values(c[k]), rx[k]);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = decode8(c[k], s[k]);
    normalise<D>(x, eps, l, r);
  }
}

// ---- rotation ----

// A token's place as the lanes of its row share it, in shared memory: the
// table rows of its t, y and x and its index.
struct __align__(16) Spot {
  int row[3];
  int n;
};

// Where a lane's four pairs find their table entry: the axis whose table row
// counts (0, 1, 2 = t, y, x) and the pair's place in that row; `still` has a
// bit for each pair that does not turn.
struct PairRefs {
  int place[4], axis[4];
  uint32_t still;
};

template <typename E, int D>
__device__ __forceinline__ PairRefs pair_refs(int l, int ht, int hh, int hw) {
  PairRefs r;
  r.still = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    int p = elem_at<E, D>(l, 2 * i) / 2;
    int axis = 0;
    if (p >= ht) { p -= ht; axis = 1; }
    if (axis == 1 && p >= hh) { p -= hh; axis = 2; }
    if (axis == 2 && p >= hw) { p = 0; r.still |= 1u << i; }
    r.place[i] = p;
    r.axis[i] = axis;
  }
  return r;
}

// some_still: whether any pair of a head stays (then the entry read for it,
// if the table has one at all, is replaced by no turn).
__device__ __forceinline__ void load_turns(const PairRefs& r, const float2* table, bool some_still,
                                           const Spot* spot, float2 (&cs)[4]) {
  if (some_still) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      cs[i] = r.still >> i & 1u ? make_float2(1.f, 0.f)
                                : table[spot->row[r.axis[i]] + r.place[i]];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) cs[i] = table[spot->row[r.axis[i]] + r.place[i]];
  }
}

// (y0, y1) -> (y0 c - y1 s, y0 s + y1 c)
__device__ __forceinline__ void turn(Vals& x, const float2 (&cs)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = x.p[i], c = cs[i];
    x.p[i] = make_float2(fmaf(y.x, c.x, -(y.y * c.y)), fmaf(y.x, c.y, y.y * c.x));
  }
}
// the transpose (= the inverse)
__device__ __forceinline__ void turn_back(Vals& x, const float2 (&cs)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = x.p[i], c = cs[i];
    x.p[i] = make_float2(fmaf(y.x, c.x, y.y * c.y), fmaf(y.y, c.x, -(y.x * c.y)));
  }
}

// A lane's eight weights of a row (ones where there are none).
template <typename E, int D>
__device__ __forceinline__ Vals load_weights(const float* g, int l) {
  Vals w;
#pragma unroll
  for (int i = 0; i < 8; ++i) w.at(i) = g ? g[elem_at<E, D>(l, i)] : 1.f;
  return w;
}

}  // namespace rows

// Launches a kernel that begins with after_previous(): it may be set up while
// the stream's previous kernel still runs its last CTAs.
template <typename K, typename... A>
cudaError_t launch(K kernel, dim3 grid, int block, int smem, int cluster, cudaStream_t st,
                   const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// A kernel's opt-in to more than 48 KB of shared memory, once per device.
class SmemOptIn {
 public:
  template <typename K>
  cudaError_t set(K kernel, int bytes, int dev) {
    if (dev < 64 && (done_.load(std::memory_order_relaxed) >> dev & 1)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) done_.fetch_or(1ull << dev);
    return e;
  }
 private:
  std::atomic<unsigned long long> done_{0};
};

// What the norm + rotation kernels are given, besides the layer's geometry.
struct NormRopeArgs {
  const void* in[3];          // raw q, k, v: [s] rows of n_h * d, `ld` elements apart
  long long ld;
  const int8_t* codes;        // or their 8-bit checkpoint [s][3][n_h][d] ...
  const float* scales;        // ... with a scale for each row of d: [s][3][n_h]
  const float *gq, *gk;       // norm weights [d], or null
  float eps;
  const float2* table;        // (cos, sin): T * ht, then H * hh, then W * hw entries
  int ht, hh, hw;             // pairs that turn with t, y, x
  bool still;                 // whether some pairs do not turn (the table has nothing for them)
};

struct NormRopeOut {
  void *q, *k, *v;
  float* blocks;              // block means of k ([n_h][N_b][d]), or null: k, v in token order
  int8_t* codes;              // checkpoint to write, or null
  float* scales;
};

cudaError_t launch_norm_rope(const Prob& P, const NormRopeArgs& a, const NormRopeOut& o,
                             int num_sms, cudaStream_t st);
size_t norm_rope_bwd_ws_bytes(const Prob& P);
cudaError_t launch_norm_rope_bwd(const Prob& P, const NormRopeArgs& a, const void* dq,
                                 const void* dk, const void* dv, void* const (&out)[3],
                                 long long ld_out, float* dweight, void* ws, int num_sms,
                                 cudaStream_t st);
cudaError_t launch_rope_table(int T, int H, int W, int ht, int hh, int hw, double base,
                              const long long (&origin)[3], float2* table, cudaStream_t st);
cudaError_t launch_act8_pack(int dtype, const void* x, long long n_rows, int cols, long long ld,
                             int group, int8_t* codes, float* scales, int num_sms,
                             cudaStream_t st);
cudaError_t launch_act8_unpack(int dtype, const int8_t* codes, const float* scales,
                               long long n_rows, int cols, int group, void* out, long long ld,
                               int num_sms, cudaStream_t st);

}  // namespace vmoba
