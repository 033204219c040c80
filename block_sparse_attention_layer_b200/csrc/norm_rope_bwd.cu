// Backward of the norm + rotation: from the gradients of the rotated q and k
// (token order) to those of the raw rows and of the norm weights.  With u the
// gradient rotated back, r = 1 / sqrt(mean(x^2) + eps), xh = x r, w = u g:
//   dx = r (w - xh mean(w xh)),   dg = sum over tokens and heads of u xh;
// dv is moved into its place in the projection's gradient.  x comes from the
// projection's output or from its 8-bit checkpoint.  HBM bound: 8 s n_h d
// elements (two of them bytes when x is a checkpoint).
//
// A CTA walks chunks of tokens of one head; each lane keeps fp32 sums of its
// weight gradients over a chunk (at most kChunk / 16 rows) and adds them to
// fp64 sums in shared memory, the CTA's total goes to the workspace, and a
// second kernel adds the totals in a fixed order, so results do not depend on
// scheduling.
#include "rows.cuh"

namespace vmoba {
namespace {

using namespace rows;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kChunk = 256;         // tokens of one work item
constexpr int kMaxCtas = 1024;      // partial weight gradients in the workspace

template <typename E, int D, bool From8>
__global__ void __launch_bounds__(kThreads)
k_norm_rope_bwd(Prob P, NormRopeArgs a, const E* __restrict__ dq, const E* __restrict__ dk,
                const E* __restrict__ dv, E* oq, E* ok, E* ov, long long ld_out, float* part,
                int n_items, int n_chunks) {
  constexpr int G = D / 8, R = 32 / G;
  __shared__ double sums[16][kThreads];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / G, l = lane % G;
  float gq[8], gk[8];
  load_weights<E, D>(a.gq, l, gq);
  load_weights<E, D>(a.gk, l, gk);
  const PairRefs refs = pair_refs<E, D>(l, a.ht, a.hh, a.hw);
  const long long row3 = (long long)P.n_h * D;
#pragma unroll
  for (int i = 0; i < 16; ++i) sums[i][threadIdx.x] = 0.0;

  for (int item = blockIdx.x; item < n_items; item += gridDim.x) {
    const int h = item / n_chunks, c0 = (item - h * n_chunks) * kChunk;
    const int last = min(c0 + kChunk, P.s);
    float wq[8], wk[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) wq[i] = wk[i] = 0.f;
    for (int n0 = c0 + warp * R; n0 < last; n0 += kWarps * R) {
      const bool mine = n0 + sub < last;
      const int n = mine ? n0 + sub : last - 1;
      const int t = n / (P.H * P.W), yx = n - t * (P.H * P.W), y = yx / P.W, x = yx - y * P.W;
      const long long at = n * row3 + (long long)h * D;
      const Raw<E> uq = load_row<D>(dq + at, l), uk = load_row<D>(dk + at, l),
                   uv = load_row<D>(dv + at, l);
      float xq[8], xk[8];
      if constexpr (From8) {
        const long long ckpt = ((long long)n * 3 * P.n_h + h) * D;
        const float* sc = a.scales + (long long)n * 3 * P.n_h + h;
        decode8(load_codes<E, D>(a.codes + ckpt, l), __ldg(sc), xq);
        decode8(load_codes<E, D>(a.codes + ckpt + row3, l), __ldg(sc + P.n_h), xk);
      } else {
        const long long raw = n * a.ld + (long long)h * D;
        unpack(load_row<D>(static_cast<const E*>(a.in[0]) + raw, l), xq);
        unpack(load_row<D>(static_cast<const E*>(a.in[1]) + raw, l), xk);
      }
      float2 cs[4];
      load_turns(refs, a.table, t * a.ht, P.T * a.ht + y * a.hh,
                 P.T * a.ht + P.H * a.hh + x * a.hw, cs);
      const long long out = n * ld_out + (long long)h * D;
      if (mine) store_raw<D>(ov + out, l, uv);
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        float(&xx)[8] = which ? xk : xq;
        const float(&g)[8] = which ? gk : gq;
        float(&wsum)[8] = which ? wk : wq;
        float u[8];
        unpack(which ? uk : uq, u);
        turn_back(u, cs);
        float pre;
        const float r = inv_rms<D>(xx, a.eps, pre);
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          xx[i] *= r;                                // xh
          if (mine) wsum[i] = fmaf(u[i], xx[i], wsum[i]);
          u[i] *= g[i];
          dot = fmaf(u[i], xx[i], dot);
        }
        dot = row_sum<G>(dot) * (1.0f / D);
        const float rr = r * pre;
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = rr * fmaf(-xx[i], dot, u[i]);
        if (mine) {
          Raw<E> w;
          pack(u, w);
          store_raw<D>((which ? ok : oq) + out, l, w);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      sums[i][threadIdx.x] += (double)wq[i];
      sums[8 + i][threadIdx.x] += (double)wk[i];
    }
  }
  if (part == nullptr) return;
  __syncthreads();
  // column c of the 2 D gradients: element i of lane l in every warp and row
  for (int c = threadIdx.x; c < 2 * D; c += kThreads) {
    const int e = c % D;
    int ll, i;
    if (sizeof(E) == 2) {
      ll = e / 8; i = e % 8;
    } else {
      const int f = e % (D / 2);
      ll = f / 4; i = f % 4 + (e >= D / 2 ? 4 : 0);
    }
    double sum = 0.0;
    for (int w = 0; w < kWarps; ++w)
      for (int b = 0; b < R; ++b) sum += sums[i + (c >= D ? 8 : 0)][w * 32 + b * G + ll];
    part[(size_t)blockIdx.x * 2 * D + c] = (float)sum;
  }
}

__global__ void k_norm_dweight(const float* __restrict__ part, int n, int cols,
                               float* __restrict__ out) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= cols) return;
  double sum = 0.0;
  for (int i = 0; i < n; ++i) sum += (double)part[(size_t)i * cols + c];
  out[c] = (float)sum;
}

template <typename E, int D, bool From8>
cudaError_t launch_t(const Prob& P, const NormRopeArgs& a, const void* dq, const void* dk,
                     const void* dv, void* const (&out)[3], long long ld_out, float* dweight,
                     void* ws, int num_sms, cudaStream_t st) {
  const int n_chunks = (P.s + kChunk - 1) / kChunk, n_items = n_chunks * P.n_h;
  const int ctas = min(min(n_items, num_sms * 4), kMaxCtas);
  float* part = dweight ? static_cast<float*>(ws) : nullptr;
  {
    VMOBA_TRACE("k_norm_rope_bwd", st);
    k_norm_rope_bwd<E, D, From8><<<ctas, kThreads, 0, st>>>(
        P, a, static_cast<const E*>(dq), static_cast<const E*>(dk), static_cast<const E*>(dv),
        static_cast<E*>(out[0]), static_cast<E*>(out[1]), static_cast<E*>(out[2]), ld_out, part,
        n_items, n_chunks);
  }
  count_launches(1);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !dweight) return e;
  {
    VMOBA_TRACE("k_norm_dweight", st);
    k_norm_dweight<<<(2 * D + 31) / 32, 32, 0, st>>>(part, ctas, 2 * D, dweight);
  }
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace

size_t norm_rope_bwd_ws_bytes(const Prob& P) {
  return align_up((size_t)kMaxCtas * 2 * P.d * sizeof(float), 256);
}

cudaError_t launch_norm_rope_bwd(const Prob& P, const NormRopeArgs& a, const void* dq,
                                 const void* dk, const void* dv, void* const (&out)[3],
                                 long long ld_out, float* dweight, void* ws, int num_sms,
                                 cudaStream_t st) {
  auto go = [&](auto e, auto d) {
    using E = decltype(e);
    constexpr int D = decltype(d)::value;
    return a.codes ? launch_t<E, D, true>(P, a, dq, dk, dv, out, ld_out, dweight, ws, num_sms, st)
                   : launch_t<E, D, false>(P, a, dq, dk, dv, out, ld_out, dweight, ws, num_sms,
                                           st);
  };
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  if (P.dtype == VMOBA_BF16)
    return P.d == 128 ? go(__nv_bfloat16{}, D128{}) : go(__nv_bfloat16{}, D64{});
  return P.d == 128 ? go(float{}, D128{}) : go(float{}, D64{});
}

}  // namespace vmoba
