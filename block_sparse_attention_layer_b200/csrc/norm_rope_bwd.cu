// Backward of the norm + rotation: from the gradients of the rotated q and k
// (token order) to those of the raw rows and of the norm weights.  With u the
// gradient rotated back, r = 1 / sqrt(mean(x^2) + eps), xh = x r, w = u g:
//   dx = r (w - xh mean(w xh)),   dg = sum over tokens and heads of u xh;
// dv is moved into its place in the projection's gradient.  x comes from the
// projection's output or from its 8-bit checkpoint (x r is then formed from
// the codes, whose squares sum to an exact integer, without their scales).
//
// Bound: HBM, 8 s n_h d elements (two of them 1.03 bytes when x is a
// checkpoint).  12 heads of 128, bf16: 75600 tokens 286 to 302 us by card (0.95 to
// 1.00 of a plain copy's 6.46 TB/s), 55296 tokens 211 us, or from a checkpoint 194 to
// 205 us (0.91 to 0.95; 2.4 instructions a cycle and SM).
//
// As in the forward, a lane works on two rows of q, k (and v) at a time, two
// neighbouring heads of a token where the head count is even, fed through
// shared memory by asynchronous copies one step ahead.  CTAs stay resident and
// walk items of neighbouring tokens of one unit of heads; neighbouring items
// are the units of the same tokens, so that whole rows pass at one time.  Each
// lane keeps fp32 sums of its weight gradients over at most kFlush rows and
// adds them to fp64 sums in shared memory, the CTA's total goes to the
// workspace, and a second kernel adds the totals in a fixed order, so results
// do not depend on scheduling.
#include "rows.cuh"

namespace vmoba {
namespace {

using namespace rows;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kFlush = 64;          // rows a lane adds in fp32 before they go to its fp64 sums
constexpr int kMaxCtas = 1024;      // partial weight gradients in the workspace

struct Walk {
  int T, H, W, s, n_h;
  int chunk;                       // tokens of a work item
  FastDiv hw, w;                   // H * W, W
  uint32_t ld, ld_out;             // bytes between tokens
  int n_items, units;              // units of heads
};

// The gradients and the raw q and k of two rows on their way through shared
// memory.
template <typename E, int D, bool From8, bool TwoHeads>
struct Feed {
  using C = CodeRows<E, D, 2, TwoHeads>;
  static constexpr int kSlot = Slot<E, D>::kBytes, kRaw = 6 * kSlot;
  static constexpr int kBytes = kRaw + (From8 ? C::kBytes : 4 * kSlot);
  __device__ __forceinline__ static Raw<E> grad(const char* s, int i, int u, int lane) {
    return Slot<E, D>::get(s + (3 * u + i) * kSlot, lane);
  }
  // x r of q and k of both rows, and r
  __device__ __forceinline__ static void load(const char* s, float eps, int sub, int l,
                                              Vals (&x)[4], float (&r)[4]) {
    s += kRaw;
    if constexpr (From8) {
      uint2 c[4];
      float sc[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        c[k] = C::codes(s, k & 1, k / 2, sub, l);
        sc[k] = C::scale(s, k & 1, k / 2, sub);
      }
      normalise<D>(c, sc, eps, l, x, r);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        x[k] = unpack(Slot<E, D>::get(s + k * kSlot, sub * (D / 8) + l));
      normalise<D>(x, eps, l, r);
    }
  }
};

// Iterations a warp's loads run ahead.
constexpr int kStages = 2;

template <typename E, int D, bool From8, bool TwoHeads>
struct Smem {
  static constexpr int kRing = kStages * kWarps * Feed<E, D, From8, TwoHeads>::kBytes;
  static constexpr int kSpots = kStages * kWarps * 8 * (int)sizeof(Spot);
  static constexpr int kLanes = kWarps * (D / 8);      // lanes of one row in every warp
  static constexpr int kBytes =
      kRing + kSpots + 16 * kLanes * (int)sizeof(double) + 2 * D * (int)sizeof(float);
};

// The weights of q and k (2 D) in shared memory, 16 registers a lane fewer: a
// lane's first four and last four elements lie in separate halves, for 16-byte
// reads without bank conflicts.
template <typename E, int D>
__device__ __forceinline__ void place_weight(const NormRopeArgs& a, int c, float* to) {
  const float* g = c < D ? a.gq : a.gk;
  const int half = c % D / (D / 2), l = c % (D / 2) / 4;
  to[c] = g ? g[elem_at<E, D>(l, half * 4 + c % 4)] : 1.f;
}
template <int D>
__device__ __forceinline__ Vals weights(const float* g, int l) {
  const float4 a = reinterpret_cast<const float4*>(g)[l];
  const float4 b = reinterpret_cast<const float4*>(g + D / 2)[l];
  return {make_float2(a.x, a.y), make_float2(a.z, a.w), make_float2(b.x, b.y),
          make_float2(b.z, b.w)};
}

// n strides and so many bytes more.
__device__ __forceinline__ unsigned long long offset(int n, uint32_t stride, uint32_t more) {
  return (unsigned long long)(uint32_t)n * stride + more;
}

template <typename E, int D, bool From8, bool TwoHeads>
__global__ void __launch_bounds__(kThreads, 2)
k_norm_rope_bwd(const __grid_constant__ Walk w, const __grid_constant__ NormRopeArgs a,
                const E* dq, const E* dk, const E* dv, E* oq, E* ok, E* ov, float* part) {
  constexpr int G = D / 8, R = 32 / G, S = kStages;
  constexpr int kStep = kWarps * R, kStride = kStep * (TwoHeads ? 1 : 2);
  using F = Feed<E, D, From8, TwoHeads>;
  using M = Smem<E, D, From8, TwoHeads>;
  extern __shared__ __align__(16) char smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / G, l = lane % G;
  char* ring = smem + warp * (S * F::kBytes);
  Spot* spots = reinterpret_cast<Spot*>(smem + M::kRing) + warp * (S * 8);
  double(&sums)[16][M::kLanes] =
      *reinterpret_cast<double(*)[16][M::kLanes]>(smem + M::kRing + M::kSpots);
  float* g_smem = reinterpret_cast<float*>(&sums[16][0]);
  after_previous();
  for (int c = threadIdx.x; c < 2 * D; c += kThreads) place_weight<E, D>(a, c, g_smem);
  __syncthreads();
  const PairRefs refs = pair_refs<E, D>(l, a.ht, a.hh, a.hw);
  const int y_rows = w.T * a.ht, x_rows = y_rows + w.H * a.hh;
  const uint32_t row3 = w.n_h * D * sizeof(E);
  if (sub == 0) {
#pragma unroll
    for (int i = 0; i < 16; ++i) sums[i][warp * G + l] = 0.0;
  }

  // A warp walks the tokens of its CTA's items as one sequence, so that its
  // loads run ahead over the end of an item too.
  struct At {
    int item, n0, last, h0;
  };
  auto enter = [&](At& p) {          // the warp's first token of the item
    if (p.item >= w.n_items) return;
    const int c = p.item / w.units, unit = p.item - c * w.units, c0 = c * w.chunk;
    p.h0 = unit * (TwoHeads ? 2 : 1);
    p.n0 = c0 + warp * R;
    p.last = min(c0 + w.chunk, w.s);
  };
  auto skip_empty = [&](At& p) {     // an item may have no token for this warp
    while (p.item < w.n_items && p.n0 >= p.last) {
      p.item += gridDim.x;
      enter(p);
    }
  };
  At cur{(int)blockIdx.x, 0, 0, 0};
  enter(cur);
  skip_empty(cur);
  At ahead = cur;
  // the lane's first bytes of head 0, token 0
  const char* in_dq = reinterpret_cast<const char*>(dq) + l * 16;
  const char* in_dk = reinterpret_cast<const char*>(dk) + l * 16;
  const char* in_dv = reinterpret_cast<const char*>(dv) + l * 16;
  const char* in_raw[2];
  [[maybe_unused]] const float* in_scale = nullptr;
  if constexpr (From8) {
    for (int i = 0; i < 2; ++i) in_raw[i] = F::C::codes_at(a.codes, i, 0, w.n_h, l);
    in_scale = F::C::scale_at(a.scales, 0, w.n_h, l);
  } else {
    for (int i = 0; i < 2; ++i) in_raw[i] = static_cast<const char*>(a.in[i]) + l * 16;
  }
  char* const to_q = reinterpret_cast<char*>(oq) + l * 16;
  char* const to_k = reinterpret_cast<char*>(ok) + l * 16;
  char* const to_v = reinterpret_cast<char*>(ov) + l * 16;
  auto ask = [&](int stage) {
    if (ahead.item < w.n_items) {
      int n = 0;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (!TwoHeads || u == 0) {
          n = min(ahead.n0 + u * kStep + sub, ahead.last - 1);
          if (l == 0) {
            const int t = w.hw.div(n), yx = n - t * (w.H * w.W), y = w.w.div(yx);
            spots[stage * 8 + u * 4 + sub] =
                Spot{{t * a.ht, y_rows + y * a.hh, x_rows + (yx - y * w.W) * a.hw}, n};
          }
        }
        char* to = ring + stage * F::kBytes;
        constexpr int kHead = D * sizeof(E);
        const uint32_t first = ahead.h0 * kHead, more = TwoHeads ? u * kHead : 0;
        const unsigned long long at = offset(n, row3, first);
        Slot<E, D>::ask(to + 3 * u * F::kSlot, in_dq + at + more, lane);
        Slot<E, D>::ask(to + (3 * u + 1) * F::kSlot, in_dk + at + more, lane);
        Slot<E, D>::ask(to + (3 * u + 2) * F::kSlot, in_dv + at + more, lane);
        to += F::kRaw;
        if constexpr (From8) {
          const char* const codes[2] = {in_raw[0] + ahead.h0 * D, in_raw[1] + ahead.h0 * D};
          F::C::ask(to, codes, in_scale + ahead.h0, n, w.n_h, u, sub, l);
        } else {
          const unsigned long long raw = offset(n, w.ld, first);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            Slot<E, D>::ask(to + (2 * u + i) * F::kSlot, in_raw[i] + raw + more, lane);
        }
      }
      ahead.n0 += kStride;
      skip_empty(ahead);
    }
    fetch_commit();
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) ask(i);
  int stage = 0;
  Vals wq, wk;
#pragma unroll
  for (int i = 0; i < 4; ++i) wq.p[i] = wk.p[i] = both(0.f);
  int rows = 0;
  while (cur.item < w.n_items) {
    {
      __syncwarp();                  // the spots of the stage that is refilled have been read
      ask(stage == 0 ? S - 1 : stage - 1);
      __syncwarp();                  // and this stage's are visible
      int n[2];
      bool mine[2];
      float2 cs[TwoHeads ? 1 : 2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (TwoHeads && u == 1) {
          n[1] = n[0]; mine[1] = mine[0];
        } else {
          mine[u] = cur.n0 + u * kStep + sub < cur.last;
          const Spot* spot = spots + stage * 8 + u * 4 + sub;
          n[u] = spot->n;
          load_turns(refs, a.table, a.still, spot, cs[u]);
        }
      }
      unsigned long long out[2];
#pragma unroll
      for (int u = 0; u < 2; ++u)
        out[u] = TwoHeads && u ? out[0] + D * sizeof(E)
                               : offset(n[u], w.ld_out, cur.h0 * (int)(D * sizeof(E)));
      fetch_wait<S - 1>();
      if constexpr (From8) __syncwarp();
      const char* in = ring + stage * F::kBytes;
      stage = stage == S - 1 ? 0 : stage + 1;
#pragma unroll
      for (int u = 0; u < 2; ++u)
        if (mine[u])
          Slot<E, D>::put(to_v + out[u], F::grad(in, 2, u, lane));
      Vals x[4];
      float r[4], dot[4];
      F::load(in, a.eps, sub, l, x, r);          // xh = x r
      Vals g[4];                                // the gradients, then w = u g
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        g[k] = unpack(F::grad(in, k & 1, k / 2, lane));
        turn_back(g[k], cs[TwoHeads ? 0 : k / 2]);
        Vals& sum = k & 1 ? wk : wq;
        const Vals weight = weights<D>(g_smem + (k & 1) * D, l);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (mine[k / 2]) sum.p[i] = __ffma2_rn(g[k].p[i], x[k].p[i], sum.p[i]);
          g[k].p[i] = __fmul2_rn(g[k].p[i], weight.p[i]);
        }
        dot[k] = lane_dot(g[k], x[k]);
      }
      spread<G>(quarter_sums<G>(dot, l) * (-1.0f / D), dot);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          g[k].p[i] = __fmul2_rn(__ffma2_rn(x[k].p[i], both(dot[k]), g[k].p[i]), both(r[k]));
        if (mine[k / 2]) {
          Raw<E> s;
          pack(g[k], s);
          Slot<E, D>::put((k & 1 ? to_k : to_q) + out[k / 2], s);
        }
      }
    }
    cur.n0 += kStride;
    skip_empty(cur);
    if ((rows += 2) < kFlush && cur.item < w.n_items) continue;
    rows = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float v = i < 8 ? wq.at(i) : wk.at(i - 8);
#pragma unroll
      for (int o = G; o < 32; o <<= 1) v += __shfl_xor_sync(kAll, v, o);
      if (sub == 0) sums[i][warp * G + l] += (double)v;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) wq.p[i] = wk.p[i] = both(0.f);
  }
  if (part == nullptr) return;
  __syncthreads();
  // column e of the q and k gradients: element i of lane ll, over the warps
  for (int c = threadIdx.x; c < 2 * D; c += kThreads) {
    const int which = c / D, i = c % D / G, ll = c % G;
    double sum = 0.0;
#pragma unroll
    for (int v = 0; v < kWarps; ++v) sum += sums[8 * which + i][v * G + ll];
    part[(size_t)blockIdx.x * 2 * D + which * D + elem_at<E, D>(ll, i)] = (float)sum;
  }
}

// The CTAs' totals added up: 32 columns a block, 32 threads a column, each
// over every 32nd CTA, and their sums in order.
__global__ void __launch_bounds__(1024)
k_norm_dweight(const float* part, int n, int cols, float* out) {
  __shared__ double sums[32][33];
  const int c = threadIdx.x & 31, k = threadIdx.x >> 5;
  after_previous();
  const float* p = part + blockIdx.x * 32 + c;
  double sum = 0.0;
#pragma unroll 8
  for (int i = k; i < n; i += 32) sum += (double)p[(size_t)i * cols];
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
  // Items are strides of the CTA's warps.  From raw rows one each: the CTAs then
  // walk one window of neighbouring rows together, where longer items keep each
  // CTA on a distance of its own from the next, which DRAM takes badly (75600
  // tokens: 290 us with one, 306 with two, 318 with eight, 327 with 32).  From
  // codes up to 32, of the length for which the CTA with the most items has the
  // fewest strides (267 us; 279 with one).
  constexpr int stride = kWarps * (256 / D) * (TwoHeads ? 1 : 2);
  const int units = TwoHeads ? P.n_h / 2 : P.n_h, slots = min(2 * num_sms, kMaxCtas);
  const long long strides = (P.s + stride - 1) / stride;
  long long best = -1;
  for (int k = From8 ? 32 : 1; k >= 1; --k) {
    const long long items = (strides + k - 1) / k * units, most = (items + slots - 1) / slots * k;
    if (best < 0 || most < best) {
      best = most;
      w.chunk = k * stride;
    }
  }
  w.units = units;
  w.n_items = (P.s + w.chunk - 1) / w.chunk * units;
  const int ctas = min(w.n_items, slots);
  float* part = dweight ? static_cast<float*>(ws) : nullptr;
  const auto kernel = k_norm_rope_bwd<E, D, From8, TwoHeads>;
  constexpr int smem = Smem<E, D, From8, TwoHeads>::kBytes;
  static SmemOptIn opt_in;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = opt_in.set(kernel, smem, dev);
  if (e != cudaSuccess) return e;
  {
    VMOBA_TRACE("k_norm_rope_bwd", st);
    e = launch(kernel, dim3(ctas), kThreads, smem, 1, st, w, a, static_cast<const E*>(dq),
               static_cast<const E*>(dk), static_cast<const E*>(dv), static_cast<E*>(out[0]),
               static_cast<E*>(out[1]), static_cast<E*>(out[2]), part);
  }
  if (e != cudaSuccess || !dweight) return e;
  VMOBA_TRACE("k_norm_dweight", st);
  return launch(k_norm_dweight, dim3(2 * D / 32), 1024, 0, 1, st, static_cast<const float*>(part),
                ctas, 2 * D, dweight);
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
