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

struct Walk {
  int T, H, W, s, n_h;
  FastDiv hw, w;                   // H * W, W
  uint32_t ld, ld_out;             // bytes between tokens
  int n_items, n_chunks;
};

template <typename E, int D, bool From8, bool TwoHeads>
__global__ void __launch_bounds__(kThreads, 2)
k_norm_rope_bwd(const __grid_constant__ Walk w, const __grid_constant__ NormRopeArgs a,
                const E* __restrict__ dq, const E* __restrict__ dk, const E* __restrict__ dv,
                E* __restrict__ oq, E* __restrict__ ok, E* __restrict__ ov, float* part) {
  constexpr int G = D / 8, R = 32 / G;
  __shared__ double sums[16][kThreads];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / G, l = lane % G;
  const Vals gq = load_weights<E, D>(a.gq, l), gk = load_weights<E, D>(a.gk, l);
  const PairRefs refs = pair_refs<E, D>(l, a.ht, a.hh, a.hw);
  const int y_rows = w.T * a.ht, x_rows = y_rows + w.H * a.hh;
  const uint32_t row3 = w.n_h * D * sizeof(E);
#pragma unroll
  for (int i = 0; i < 16; ++i) sums[i][threadIdx.x] = 0.0;

  for (int item = blockIdx.x; item < w.n_items; item += gridDim.x) {
    const int unit = item / w.n_chunks, c0 = (item - unit * w.n_chunks) * kChunk;
    const int h0 = unit * (TwoHeads ? 2 : 1);
    const int last = min(c0 + kChunk, w.s);
    Vals wq, wk;
#pragma unroll
    for (int i = 0; i < 4; ++i) wq.p[i] = wk.p[i] = both(0.f);
    constexpr int kStep = kWarps * R;
    for (int n0 = c0 + warp * R; n0 < last; n0 += kStep * (TwoHeads ? 1 : 2)) {
      int n[2];
      bool mine[2];
      float2 cs[TwoHeads ? 1 : 2][4];
      Raw<E> uq[2], uk[2], uv[2];
      Vals x[4];
      [[maybe_unused]] Raw<E> xq[2], xk[2];
      [[maybe_unused]] uint2 cq[2], ck[2];
      [[maybe_unused]] float sq[2], sk[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (TwoHeads && u == 1) {
          n[1] = n[0]; mine[1] = mine[0];
        } else {
          mine[u] = n0 + u * kStep + sub < last;
          n[u] = min(n0 + u * kStep + sub, last - 1);
          const int t = w.hw.div(n[u]), yx = n[u] - t * (w.H * w.W), y = w.w.div(yx);
          load_turns(refs, a.table, t * a.ht, y_rows + y * a.hh, x_rows + (yx - y * w.W) * a.hw,
                     cs[u]);
        }
        const int h = h0 + (TwoHeads ? u : 0);
        uq[u] = load_row<D>(at_bytes(dq + h * D, n[u], row3), l);
        uk[u] = load_row<D>(at_bytes(dk + h * D, n[u], row3), l);
        uv[u] = load_row<D>(at_bytes(dv + h * D, n[u], row3), l);
        if constexpr (From8) {
          const uint32_t row = (uint32_t)(n[u] * 3 * w.n_h + h);
          cq[u] = load_codes<E, D>(at_bytes(a.codes, row, D), l);
          ck[u] = load_codes<E, D>(at_bytes(a.codes, row + w.n_h, D), l);
          sq[u] = __ldg(a.scales + row);
          sk[u] = __ldg(a.scales + row + w.n_h);
        } else {
          xq[u] = load_row<D>(at_bytes(static_cast<const E*>(a.in[0]) + h * D, n[u], w.ld), l);
          xk[u] = load_row<D>(at_bytes(static_cast<const E*>(a.in[1]) + h * D, n[u], w.ld), l);
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if constexpr (From8) {
          x[2 * u] = decode8(cq[u], sq[u]);
          x[2 * u + 1] = decode8(ck[u], sk[u]);
        } else {
          x[2 * u] = unpack(xq[u]);
          x[2 * u + 1] = unpack(xk[u]);
        }
        if (mine[u])
          store_raw<D>(at_bytes(ov + (h0 + (TwoHeads ? u : 0)) * D, n[u], w.ld_out), l, uv[u]);
      }
      float r[4], pre[4], dot[4];
      inv_rms<D>(x, a.eps, l, r, pre);
      Vals g[4];                                // the gradients, then w = u g
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        g[k] = unpack(k & 1 ? uk[k / 2] : uq[k / 2]);
        turn_back(g[k], cs[TwoHeads ? 0 : k / 2]);
        Vals& sum = k & 1 ? wk : wq;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[k].p[i] = __fmul2_rn(x[k].p[i], both(r[k]));                // xh
          if (mine[k / 2]) sum.p[i] = __ffma2_rn(g[k].p[i], x[k].p[i], sum.p[i]);
          g[k].p[i] = __fmul2_rn(g[k].p[i], k & 1 ? gk.p[i] : gq.p[i]);
        }
        dot[k] = lane_dot(g[k], x[k]);
      }
      spread<G>(quarter_sums<G>(dot, l) * (-1.0f / D), dot);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float rr = r[k] * pre[k];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          g[k].p[i] = __fmul2_rn(__ffma2_rn(x[k].p[i], both(dot[k]), g[k].p[i]), both(rr));
        if (mine[k / 2]) {
          Raw<E> s;
          pack(g[k], s);
          const int h = h0 + (TwoHeads ? k / 2 : 0);
          store_raw<D>(at_bytes((k & 1 ? ok : oq) + h * D, n[k / 2], w.ld_out), l, s);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      sums[i][threadIdx.x] += (double)wq.at(i);
      sums[8 + i][threadIdx.x] += (double)wk.at(i);
    }
  }
  if (part == nullptr) return;
  __syncthreads();
  // column e of the q and k gradients: element i of lane ll, over warps and rows
  for (int c = threadIdx.x; c < 2 * D; c += kThreads) {
    const int which = c / D, i = c % D / G, ll = c % G;
    double sum = 0.0;
    for (int v = 0; v < kWarps; ++v)
#pragma unroll
      for (int b = 0; b < R; ++b) sum += sums[8 * which + i][v * 32 + b * G + ll];
    part[(size_t)blockIdx.x * 2 * D + which * D + elem_at<E, D>(ll, i)] = (float)sum;
  }
}

// The CTAs' totals added up: 32 columns a block, 32 threads a column, each
// over every 32nd CTA, and their sums in order.
__global__ void __launch_bounds__(1024)
k_norm_dweight(const float* __restrict__ part, int n, int cols, float* __restrict__ out) {
  __shared__ double sums[32][33];
  const int c = threadIdx.x & 31, k = threadIdx.x >> 5;
  const float* p = part + blockIdx.x * 32 + c;
  double sum = 0.0;
#pragma unroll 8
  for (int i = k; i < n; i += 32) sum += (double)__ldg(p + (size_t)i * cols);
  sums[k][c] = sum;
  __syncthreads();
  if (k == 0) {
    for (int i = 1; i < 32; ++i) sum += sums[i][c];
    out[blockIdx.x * 32 + c] = (float)sum;
  }
}

template <typename E, int D, bool From8, bool TwoHeads>
cudaError_t launch_t(const Prob& P, const NormRopeArgs& a, const void* dq, const void* dk,
                     const void* dv, void* const (&out)[3], long long ld_out, float* dweight,
                     void* ws, int num_sms, cudaStream_t st) {
  Walk w{};
  w.T = P.T; w.H = P.H; w.W = P.W; w.s = P.s; w.n_h = P.n_h;
  w.hw = FastDiv(P.H * P.W);
  w.w = FastDiv(P.W);
  w.ld = (uint32_t)(a.ld * sizeof(E));
  w.ld_out = (uint32_t)(ld_out * sizeof(E));
  w.n_chunks = (P.s + kChunk - 1) / kChunk;
  w.n_items = w.n_chunks * (TwoHeads ? P.n_h / 2 : P.n_h);
  const int ctas = min(min(w.n_items, num_sms * 2), kMaxCtas);
  float* part = dweight ? static_cast<float*>(ws) : nullptr;
  {
    VMOBA_TRACE("k_norm_rope_bwd", st);
    k_norm_rope_bwd<E, D, From8, TwoHeads><<<ctas, kThreads, 0, st>>>(
        w, a, static_cast<const E*>(dq), static_cast<const E*>(dk), static_cast<const E*>(dv),
        static_cast<E*>(out[0]), static_cast<E*>(out[1]), static_cast<E*>(out[2]), part);
  }
  count_launches(1);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !dweight) return e;
  {
    VMOBA_TRACE("k_norm_dweight", st);
    k_norm_dweight<<<2 * D / 32, 1024, 0, st>>>(part, ctas, 2 * D, dweight);
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
    auto call = [&](auto fn) {
      return fn(P, a, dq, dk, dv, out, ld_out, dweight, ws, num_sms, st);
    };
    if (P.n_h % 2 == 0)
      return a.codes ? call(launch_t<E, D, true, true>) : call(launch_t<E, D, false, true>);
    return a.codes ? call(launch_t<E, D, true, false>) : call(launch_t<E, D, false, false>);
  };
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  if (P.dtype == VMOBA_BF16)
    return P.d == 128 ? go(__nv_bfloat16{}, D128{}) : go(__nv_bfloat16{}, D64{});
  return P.d == 128 ? go(float{}, D128{}) : go(float{}, D64{});
}

}  // namespace vmoba
