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

// Groups in order of rows.  A CTA takes U * kThreads / G of them in a row, a
// lane U with all their loads in flight.  U is kUnroll with vectors (store and
// read back 55296 x 1536 with two: 97 us, four: 94, eight: 104), but one where
// that makes no more than kFewCtas CTAs an SM (16 x 1536: 2.5 us against 3.1;
// 1200 x 1536: 4.4 against 4.5; 3000 x 1536: 7.4 against 6.9), and one for
// single values, eight loads each (40000 x 1003 fp32: 83 us against 115).  The
// 64-bit division that finds a CTA's first row is done once for it, a lane
// finds its own from there by a 32-bit multiplication.
constexpr int kUnroll = 4;
constexpr int kFewCtas = 6;

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

template <typename E, int Group, bool Vec, int U>
__global__ void __launch_bounds__(kThreads)
k_act8_pack(const E* x, const __grid_constant__ Shape s, int8_t* codes, float* scales) {
  constexpr int G = Group / 8, kPer = kThreads / G;
  const int l = threadIdx.x % G;
  const long long base = (long long)blockIdx.x * (U * kPer);
  const long long row0 = base / s.per_row;
  const int g0 = (int)(base - row0 * s.per_row);
  const int most = (int)min(s.n_groups - base, (long long)(U * kPer));
  Raw<E> r[U];
  Place at[U];
  after_previous();
#pragma unroll
  for (int u = 0; u < U; ++u) {
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
  for (int u = 0; u < U; u += 2) {
    uint32_t m[2];
    group_max<G>(r[u], r[min(u + 1, U - 1)], m[0], m[1]);
#pragma unroll
    for (int b = 0; b < min(2, U); ++b) {
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

template <typename E, int Group, bool Vec, int U>
__global__ void __launch_bounds__(kThreads)
k_act8_unpack(const int8_t* codes, const float* scales,
              const __grid_constant__ Shape s, E* out) {
  constexpr int G = Group / 8, kPer = kThreads / G;
  const int l = threadIdx.x % G;
  const long long base = (long long)blockIdx.x * (U * kPer);
  const long long row0 = base / s.per_row;
  const int g0 = (int)(base - row0 * s.per_row);
  const int most = (int)min(s.n_groups - base, (long long)(U * kPer));
  uint2 w[U];
  float scale[U];
  Place at[U];
  after_previous();
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int k = min(u * kPer + (int)threadIdx.x / G, most - 1);
    at[u] = place(s, row0, g0, k);
    at[u].c0 *= Group;
    scale[u] = scales[base + k];
    const int8_t* src = codes + at[u].row * s.cols;
    if constexpr (Vec) {
      const int c = at[u].c0 + l * 8;
      w[u] = make_uint2(0u, 0u);
      if (c < s.cols) w[u] = *reinterpret_cast<const uint2*>(src + c);
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
  for (int u = 0; u < U; ++u) {
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

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Calls f(shape, CTAs, vectors?, groups a lane) with compile-time flags.
template <typename E, int Group, typename F>
cudaError_t with_shape(const void* x, long long n_rows, int cols, long long ld,
                       const int8_t* codes, int num_sms, F f) {
  Shape s{};
  s.per_row = (int)(((long long)cols + Group - 1) / Group);    // cols may be the largest int
  s.cols = cols;
  s.ld = ld;
  s.n_groups = n_rows * s.per_row;
  s.div = FastDiv(s.per_row);
  constexpr int per = kThreads / (Group / 8);          // groups of a CTA, one a lane
  const bool vec = aligned(x, 16) && (ld * sizeof(E)) % 16 == 0 && cols % 8 == 0 &&
                   aligned(codes, 8);
  const bool few = s.n_groups <= (long long)per * kFewCtas * num_sms;
  const auto go = [&](auto v, auto u) {
    constexpr int U = decltype(u)::value;
    return f(s, dim3((unsigned)((s.n_groups + U * per - 1) / (U * per))), v, u);
  };
  using Yes = std::true_type;
  using No = std::false_type;
  using One = std::integral_constant<int, 1>;
  using Many = std::integral_constant<int, kUnroll>;
  if (!vec) return go(No{}, One{});
  return few ? go(Yes{}, One{}) : go(Yes{}, Many{});
}

template <typename E, int Group>
cudaError_t pack_t(const void* x, long long n_rows, int cols, long long ld, int8_t* codes,
                   float* scales, int num_sms, cudaStream_t st) {
  VMOBA_TRACE("k_act8_pack", st);
  return with_shape<E, Group>(x, n_rows, cols, ld, codes, num_sms,
                              [&](const Shape& s, dim3 ctas, auto v, auto u) {
    return launch(k_act8_pack<E, Group, decltype(v)::value, decltype(u)::value>, ctas, kThreads, 0,
                  1, st, static_cast<const E*>(x), s, codes, scales);
  });
}

template <typename E, int Group>
cudaError_t unpack_t(const int8_t* codes, const float* scales, long long n_rows, int cols,
                     void* out, long long ld, int num_sms, cudaStream_t st) {
  VMOBA_TRACE("k_act8_unpack", st);
  return with_shape<E, Group>(out, n_rows, cols, ld, codes, num_sms,
                              [&](const Shape& s, dim3 ctas, auto v, auto u) {
    return launch(k_act8_unpack<E, Group, decltype(v)::value, decltype(u)::value>, ctas, kThreads,
                  0, 1, st, codes, scales, s, static_cast<E*>(out));
  });
}

}  // namespace

cudaError_t launch_act8_pack(int dtype, const void* x, long long n_rows, int cols, long long ld,
                             int group, int8_t* codes, float* scales, int num_sms,
                             cudaStream_t st) {
  if (dtype == VMOBA_BF16)
    return group == 64
               ? pack_t<__nv_bfloat16, 64>(x, n_rows, cols, ld, codes, scales, num_sms, st)
               : pack_t<__nv_bfloat16, 128>(x, n_rows, cols, ld, codes, scales, num_sms, st);
  return group == 64 ? pack_t<float, 64>(x, n_rows, cols, ld, codes, scales, num_sms, st)
                     : pack_t<float, 128>(x, n_rows, cols, ld, codes, scales, num_sms, st);
}

cudaError_t launch_act8_unpack(int dtype, const int8_t* codes, const float* scales,
                               long long n_rows, int cols, int group, void* out, long long ld,
                               int num_sms, cudaStream_t st) {
  if (dtype == VMOBA_BF16)
    return group == 64
               ? unpack_t<__nv_bfloat16, 64>(codes, scales, n_rows, cols, out, ld, num_sms, st)
               : unpack_t<__nv_bfloat16, 128>(codes, scales, n_rows, cols, out, ld, num_sms, st);
  return group == 64 ? unpack_t<float, 64>(codes, scales, n_rows, cols, out, ld, num_sms, st)
                     : unpack_t<float, 128>(codes, scales, n_rows, cols, out, ld, num_sms, st);
}

}  // namespace vmoba
