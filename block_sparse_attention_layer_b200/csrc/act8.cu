// Activation checkpoints in 8 bits: [rows][cols] values as int8 codes and one
// fp32 scale for each group of `group` neighbouring columns (the last group of
// a row may be short), and back.  Arithmetic of a group: rows.cuh.  Both passes
// are HBM bound: one read of the values, one write of 1 + 4 / group bytes for
// each, or the reverse.
//
// A group lies over group / 8 lanes, eight values a lane: neighbouring columns
// in 16-byte accesses where every row starts on a 16-byte boundary and its
// codes on an 8-byte one, else columns group / 8 apart, one by one.
#include "rows.cuh"

namespace vmoba {
namespace {

using namespace rows;

constexpr int kThreads = 256;

__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }

// Eight neighbouring values.
__device__ __forceinline__ Vals load8(const __nv_bfloat16* p) {
  return unpack(Raw<__nv_bfloat16>{load16(p)});
}
__device__ __forceinline__ Vals load8(const float* p) {
  return unpack(Raw<float>{as_float4(load16(p)), as_float4(load16(p + 4))});
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const Vals& v) {
  Raw<__nv_bfloat16> r;
  pack(v, r);
  *reinterpret_cast<uint4*>(p) = r.u;
}
__device__ __forceinline__ void store8(float* p, const Vals& v) {
  Raw<float> r;
  pack(v, r);
  reinterpret_cast<float4*>(p)[0] = r.a;
  reinterpret_cast<float4*>(p)[1] = r.b;
}

template <typename E, int Group, bool Vec>
__global__ void __launch_bounds__(kThreads)
k_act8_pack(const E* __restrict__ x, long long n_groups, int per_row, int cols, long long ld,
            int8_t* __restrict__ codes, float* __restrict__ scales) {
  constexpr int G = Group / 8;
  const int l = threadIdx.x % G;
  const long long g0 = ((long long)blockIdx.x * kThreads + threadIdx.x) / G;
  const bool mine = g0 < n_groups;
  const long long g = mine ? g0 : n_groups - 1;
  const long long row = g / per_row;
  const int c0 = (int)(g - row * per_row) * Group;
  const E* src = x + row * ld;
  int8_t* dst = codes + row * cols;
  Vals v;
  const int at = c0 + l * 8;
  if constexpr (Vec) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v.p[i] = both(0.f);
    if (at < cols) v = load8(src + at);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = c0 + l + i * G;
      v.at(i) = c < cols ? load1(src + c) : 0.f;
    }
  }
  float scale;
  const uint2 w = encode8(v, row_max<G>(abs_max_bits(v)), scale);
  if (!mine) return;
  if (l == 0) scales[g] = scale;
  if constexpr (Vec) {
    if (at < cols) *reinterpret_cast<uint2*>(dst + at) = w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = c0 + l + i * G;
      if (c < cols) dst[c] = (int8_t)((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
    }
  }
}

template <typename E, int Group, bool Vec>
__global__ void __launch_bounds__(kThreads)
k_act8_unpack(const int8_t* __restrict__ codes, const float* __restrict__ scales,
              long long n_groups, int per_row, int cols, E* __restrict__ out, long long ld) {
  constexpr int G = Group / 8;
  const int l = threadIdx.x % G;
  const long long g = ((long long)blockIdx.x * kThreads + threadIdx.x) / G;
  if (g >= n_groups) return;
  const long long row = g / per_row;
  const int c0 = (int)(g - row * per_row) * Group;
  const int8_t* src = codes + row * cols;
  E* dst = out + row * ld;
  const float scale = __ldg(scales + g);
  if constexpr (Vec) {
    const int at = c0 + l * 8;
    if (at < cols)
      store8(dst + at, decode8(__ldg(reinterpret_cast<const uint2*>(src + at)), scale));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = c0 + l + i * G;
      if (c < cols) store1(dst + c, (float)src[c] * scale);
    }
  }
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

template <typename E, int Group>
cudaError_t pack_t(const void* x, long long n_rows, int cols, long long ld, int8_t* codes,
                   float* scales, cudaStream_t st) {
  const int per_row = (cols + Group - 1) / Group;
  const long long n = n_rows * per_row;
  const long long ctas = (n * (Group / 8) + kThreads - 1) / kThreads;
  const bool vec = aligned(x, 16) && (ld * sizeof(E)) % 16 == 0 && cols % 8 == 0 &&
                   aligned(codes, 8);
  {
    VMOBA_TRACE("k_act8_pack", st);
    if (vec)
      k_act8_pack<E, Group, true><<<(unsigned)ctas, kThreads, 0, st>>>(
          static_cast<const E*>(x), n, per_row, cols, ld, codes, scales);
    else
      k_act8_pack<E, Group, false><<<(unsigned)ctas, kThreads, 0, st>>>(
          static_cast<const E*>(x), n, per_row, cols, ld, codes, scales);
  }
  count_launches(1);
  return cudaGetLastError();
}

template <typename E, int Group>
cudaError_t unpack_t(const int8_t* codes, const float* scales, long long n_rows, int cols,
                     void* out, long long ld, cudaStream_t st) {
  const int per_row = (cols + Group - 1) / Group;
  const long long n = n_rows * per_row;
  const long long ctas = (n * (Group / 8) + kThreads - 1) / kThreads;
  const bool vec = aligned(out, 16) && (ld * sizeof(E)) % 16 == 0 && cols % 8 == 0 &&
                   aligned(codes, 8);
  {
    VMOBA_TRACE("k_act8_unpack", st);
    if (vec)
      k_act8_unpack<E, Group, true><<<(unsigned)ctas, kThreads, 0, st>>>(
          codes, scales, n, per_row, cols, static_cast<E*>(out), ld);
    else
      k_act8_unpack<E, Group, false><<<(unsigned)ctas, kThreads, 0, st>>>(
          codes, scales, n, per_row, cols, static_cast<E*>(out), ld);
  }
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_act8_pack(int dtype, const void* x, long long n_rows, int cols, long long ld,
                             int group, int8_t* codes, float* scales, cudaStream_t st) {
  if (dtype == VMOBA_BF16)
    return group == 64
               ? pack_t<__nv_bfloat16, 64>(x, n_rows, cols, ld, codes, scales, st)
               : pack_t<__nv_bfloat16, 128>(x, n_rows, cols, ld, codes, scales, st);
  return group == 64 ? pack_t<float, 64>(x, n_rows, cols, ld, codes, scales, st)
                     : pack_t<float, 128>(x, n_rows, cols, ld, codes, scales, st);
}

cudaError_t launch_act8_unpack(int dtype, const int8_t* codes, const float* scales,
                               long long n_rows, int cols, int group, void* out, long long ld,
                               cudaStream_t st) {
  if (dtype == VMOBA_BF16)
    return group == 64
               ? unpack_t<__nv_bfloat16, 64>(codes, scales, n_rows, cols, out, ld, st)
               : unpack_t<__nv_bfloat16, 128>(codes, scales, n_rows, cols, out, ld, st);
  return group == 64 ? unpack_t<float, 64>(codes, scales, n_rows, cols, out, ld, st)
                     : unpack_t<float, 128>(codes, scales, n_rows, cols, out, ld, st);
}

}  // namespace vmoba
