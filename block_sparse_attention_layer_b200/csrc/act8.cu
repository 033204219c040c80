// Activation checkpoints in 8 bits: [rows][cols] values as int8 codes and one
// fp32 scale for each group of `group` neighbouring columns (the last group of
// a row may be short), and back.  Arithmetic of a group: rows.cuh.  Bound: HBM,
// one read of the values and one write of 1 + 4 / group bytes for each, or the
// reverse.  55296 x 1536 bf16 in groups of 128: 49 us to store (5.2 TB/s, 0.81
// of a plain copy's rate; half of its instructions are integer ones, for the
// codes), 40 us to read back (0.99).
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
__device__ __forceinline__ Raw<__nv_bfloat16> load8(const __nv_bfloat16* p) { return {load16(p)}; }
__device__ __forceinline__ Raw<float> load8(const float* p) {
  return {as_float4(load16(p)), as_float4(load16(p + 4))};
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

// Groups in order of rows.  A CTA takes kUnroll * kThreads / G of them in a
// row, a lane kUnroll with all their loads in flight (store and read back with
// two: 97 us, four: 94, eight: 104); the 64-bit division that finds the first one's row is the CTA's, a
// lane finds its own from there by a 32-bit multiplication.
constexpr int kUnroll = 4;

struct Shape {
  long long n_groups, ld;
  int per_row, cols;
  FastDiv div;                     // per_row
};

struct Place {
  long long row;
  int c0;                          // first column
};
__device__ __forceinline__ Place place(const Shape& s, long long row0, int g0, int offset) {
  const int g = g0 + offset, down = s.div.div(g);
  return {row0 + down, g - down * s.per_row};
}

template <typename E, int Group, bool Vec>
__global__ void __launch_bounds__(kThreads)
k_act8_pack(const E* __restrict__ x, const __grid_constant__ Shape s, int8_t* __restrict__ codes,
            float* __restrict__ scales) {
  constexpr int G = Group / 8, kPer = kThreads / G;
  const int l = threadIdx.x % G;
  const long long base = (long long)blockIdx.x * (kUnroll * kPer);
  const long long row0 = base / s.per_row;
  const int g0 = (int)(base - row0 * s.per_row);
  const int most = (int)min(s.n_groups - base, (long long)(kUnroll * kPer));
  Raw<E> r[kUnroll];
  Place at[kUnroll];
  after_previous();
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int k = u * kPer + threadIdx.x / G;
    at[u] = place(s, row0, g0, min(k, most - 1));
    at[u].c0 *= Group;
    const E* src = x + at[u].row * s.ld;
    if constexpr (Vec) {
      const int c = at[u].c0 + l * 8;
      Vals zero{};
      pack(zero, r[u]);
      if (c < s.cols) r[u] = load8(src + c);
    } else {
      Vals v;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = at[u].c0 + l + i * G;
        v.at(i) = c < s.cols ? load1(src + c) : 0.f;
      }
      pack(v, r[u]);               // exact: the values are the type's
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; u += 2) {
    uint32_t m[2];
    group_max<G>(r[u], r[u + 1], m[0], m[1]);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int k = (u + b) * kPer + threadIdx.x / G;
      if (k >= most) continue;
      float scale;
      const uint2 w = encode8<E>(unpack(r[u + b]), m[b], scale);
      if (l == 0) scales[base + k] = scale;
      int8_t* dst = codes + at[u + b].row * s.cols;
      if constexpr (Vec) {
        const int c = at[u + b].c0 + l * 8;
        if (c < s.cols) *reinterpret_cast<uint2*>(dst + c) = w;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = at[u + b].c0 + l + i * G;
          if (c < s.cols) dst[c] = (int8_t)((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
        }
      }
    }
  }
}

template <typename E, int Group, bool Vec>
__global__ void __launch_bounds__(kThreads)
k_act8_unpack(const int8_t* __restrict__ codes, const float* __restrict__ scales,
              const __grid_constant__ Shape s, E* __restrict__ out) {
  constexpr int G = Group / 8, kPer = kThreads / G;
  const int l = threadIdx.x % G;
  const long long base = (long long)blockIdx.x * (kUnroll * kPer);
  const long long row0 = base / s.per_row;
  const int g0 = (int)(base - row0 * s.per_row);
  const int most = (int)min(s.n_groups - base, (long long)(kUnroll * kPer));
  uint2 w[kUnroll];
  float scale[kUnroll];
  Place at[kUnroll];
  after_previous();
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int k = min(u * kPer + (int)threadIdx.x / G, most - 1);
    at[u] = place(s, row0, g0, k);
    at[u].c0 *= Group;
    scale[u] = __ldg(scales + base + k);
    const int8_t* src = codes + at[u].row * s.cols;
    if constexpr (Vec) {
      const int c = at[u].c0 + l * 8;
      w[u] = make_uint2(0u, 0u);
      if (c < s.cols) w[u] = __ldg(reinterpret_cast<const uint2*>(src + c));
    } else {
      uint32_t b[2] = {0u, 0u};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = at[u].c0 + l + i * G;
        if (c < s.cols) b[i >> 2] |= (uint32_t)(uint8_t)src[c] << (8 * (i & 3));
      }
      w[u] = make_uint2(b[0], b[1]);
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    if (u * kPer + (int)threadIdx.x / G >= most) break;
    const Vals v = decode8(w[u], scale[u]);
    E* dst = out + at[u].row * s.ld;
    if constexpr (Vec) {
      const int c = at[u].c0 + l * 8;
      if (c < s.cols) store8(dst + c, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = at[u].c0 + l + i * G;
        if (c < s.cols) store1(dst + c, v.at(i));
      }
    }
  }
}

template <int Group>
Shape shape_of(long long n_rows, int cols, long long ld, unsigned* ctas) {
  Shape s{};
  s.per_row = (cols + Group - 1) / Group;
  s.cols = cols;
  s.ld = ld;
  s.n_groups = n_rows * s.per_row;
  s.div = FastDiv(s.per_row);
  constexpr int per_cta = kUnroll * kThreads / (Group / 8);
  *ctas = (unsigned)((s.n_groups + per_cta - 1) / per_cta);
  return s;
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

template <typename E>
bool vectors(const void* x, long long ld, int cols, const int8_t* codes) {
  return aligned(x, 16) && (ld * sizeof(E)) % 16 == 0 && cols % 8 == 0 && aligned(codes, 8);
}

template <typename E, int Group>
cudaError_t pack_t(const void* x, long long n_rows, int cols, long long ld, int8_t* codes,
                   float* scales, cudaStream_t st) {
  unsigned ctas;
  const Shape s = shape_of<Group>(n_rows, cols, ld, &ctas);
  const auto kernel = vectors<E>(x, ld, cols, codes) ? k_act8_pack<E, Group, true>
                                                     : k_act8_pack<E, Group, false>;
  VMOBA_TRACE("k_act8_pack", st);
  return launch(kernel, dim3(ctas), kThreads, 0, 1, st, static_cast<const E*>(x), s, codes, scales);
}

template <typename E, int Group>
cudaError_t unpack_t(const int8_t* codes, const float* scales, long long n_rows, int cols,
                     void* out, long long ld, cudaStream_t st) {
  unsigned ctas;
  const Shape s = shape_of<Group>(n_rows, cols, ld, &ctas);
  const auto kernel = vectors<E>(out, ld, cols, codes) ? k_act8_unpack<E, Group, true>
                                                       : k_act8_unpack<E, Group, false>;
  VMOBA_TRACE("k_act8_unpack", st);
  return launch(kernel, dim3(ctas), kThreads, 0, 1, st, codes, scales, s, static_cast<E*>(out));
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
