// Between the projection and the attention: the RMS norm of each head's query
// and key row, y = x g / sqrt(mean(x^2) + eps), and its rotation by the
// token's (t, y, x) position, in one pass that also moves v.  q leaves in
// token order; k and v leave in token order (dense attention) or in the
// layer's partition order together with the fp32 block means of k, so that
// the sparse layer needs no partition pass over them.  The raw rows come from
// the projection or from an 8-bit checkpoint, and the pass can write that
// checkpoint.  A row's raw value is read once and its result written once:
// HBM bound, 6 s n_h d elements.
//
// A lane works on two rows of q, k and v at a time, two neighbouring heads of
// one token where the head count is even (they share the position and its
// table entries), else one head of two tokens: six loads in flight before the
// first is used, and the four sums of squares go through one shuffle tree.  A
// CTA's eight warps take `up` neighbouring units of heads, the rest of the
// warps further tokens.  A block of keys is cut into chunks, one CTA each;
// the CTAs of a block are a cluster, whose members add their column sums over
// distributed shared memory in a fixed order.  Token order is the case of a
// single block that is the whole latent, without clusters.
#include <cooperative_groups.h>

#include "rows.cuh"

namespace vmoba {
namespace {

using namespace rows;
namespace cg = cooperative_groups;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxUp = 2;          // units of a CTA
constexpr int kFlush = 64;         // rows a lane adds in fp32 before they go to its fp64 sums

// Where the rows of one launch lie.
struct Walk {
  int T, H, W, n_h;
  int bt, bh, bw;                  // box of a block
  int nbh, nbw, Nb, L;
  FastDiv hw, w;                   // bh * bw, bw
  int chunk, chunks;               // rows of a chunk, chunks of a block
  int up;                          // units of heads of a CTA
  uint32_t ld, kv_tok;             // bytes between tokens of the raw rows; positions of k and v
  long long kv_head;               // elements between heads of k and v
};

// One row of q, k and v on its way through shared memory.
template <typename E, int D, bool From8>
struct Feed {
  static constexpr int kSlot = Slot<E, D>::kBytes, kBytes = 3 * kSlot;
  __device__ __forceinline__ static void ask(char* s, const Walk& w, const NormRopeArgs& a, int n,
                                             int h, int lane, int l) {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      Slot<E, D>::ask(s + i * kSlot, at_bytes(static_cast<const E*>(a.in[i]) + h * D, n, w.ld),
                      lane, l);
  }
  __device__ __forceinline__ static Raw<E> raw(const char* s, int i, int lane) {
    return Slot<E, D>::get(s + i * kSlot, lane);
  }
  __device__ __forceinline__ static Vals get(const char* s, int i, int lane) {
    return unpack(raw(s, i, lane));
  }
  __device__ __forceinline__ static Raw<E> value(const char* s, int lane) {
    return raw(s, 2, lane);
  }
};
template <typename E, int D>
struct Feed<E, D, true> {
  static constexpr int kSlot = Slot8<E, D>::kBytes, kBytes = 3 * kSlot;
  __device__ __forceinline__ static void ask(char* s, const Walk& w, const NormRopeArgs& a, int n,
                                             int h, int lane, int l) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const uint32_t row = (uint32_t)((n * 3 + i) * w.n_h + h);
      Slot8<E, D>::ask(s + i * kSlot, at_bytes(a.codes, row, D), a.scales + row, lane, l);
    }
  }
  __device__ __forceinline__ static Vals get(const char* s, int i, int lane) {
    return decode8(Slot8<E, D>::codes(s + i * kSlot, lane), Slot8<E, D>::scale(s + i * kSlot, lane));
  }
  __device__ __forceinline__ static Raw<E> value(const char* s, int lane) {
    Raw<E> r;
    pack(get(s, 2, lane), r);
    return r;
  }
};

// Iterations a warp's loads run ahead, and the CTAs of an SM that this leaves
// shared memory for.
template <typename E, bool From8>
constexpr int stages() { return From8 || sizeof(E) == 2 ? 3 : 2; }

template <typename E, int D, bool From8, bool TwoHeads>
constexpr int smem_bytes() {
  return stages<E, From8>() * kWarps * 2 * Feed<E, D, From8>::kBytes +
         (TwoHeads ? 2 : 1) * (8 * kThreads + kMaxUp * D) * (int)sizeof(double);
}

template <typename E, int D, bool From8, bool To8, bool TwoHeads>
__global__ void __launch_bounds__(kThreads, 2)
k_norm_rope(const __grid_constant__ Walk w, const __grid_constant__ NormRopeArgs a,
            const __grid_constant__ NormRopeOut o) {
  constexpr int G = D / 8, R = 32 / G, NA = TwoHeads ? 2 : 1;
  using F = Feed<E, D, From8>;
  constexpr int S = stages<E, From8>();
  extern __shared__ __align__(16) char smem[];
  double(&sums)[NA][8][kThreads] =               // a thread's fp64 column sums
      *reinterpret_cast<double(*)[NA][8][kThreads]>(smem);
  double* total = &sums[0][0][0] + NA * 8 * kThreads;    // the CTA's, read by its cluster
  char* ring = reinterpret_cast<char*>(total + kMaxUp * NA * D) +
               (threadIdx.x >> 5) * (S * 2 * F::kBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / G, l = lane % G;
  const int h0 = (blockIdx.y * w.up + warp % w.up) * NA;
  const int j = blockIdx.x / w.chunks;
  const int first = (blockIdx.x - j * w.chunks) * w.chunk, last = min(first + w.chunk, w.L);
  const int step = kWarps / w.up * R;

  const Vals gq = load_weights<E, D>(a.gq, l), gk = load_weights<E, D>(a.gk, l);
  const PairRefs refs = pair_refs<E, D>(l, a.ht, a.hh, a.hw);
  const int y_rows = w.T * a.ht, x_rows = y_rows + w.H * a.hh;
  const int pw = j % w.nbw, jj = j / w.nbw, ph = jj % w.nbh, pt = jj / w.nbh;
  const int t0 = pt * w.bt, y0 = ph * w.bh, x0 = pw * w.bw;
  Vals acc[NA];
#pragma unroll
  for (int u = 0; u < NA; ++u)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      acc[u].at(i) = 0.f;
      sums[u][i][threadIdx.x] = 0.0;
    }

  const int stride = step * (TwoHeads ? 1 : 2);
  const int r_begin = first + warp / w.up * R;
  // row r of the block is token n = (t, y, x)
  auto locate = [&](int r, int& t, int& y, int& x) {
    const int bt = w.hw.div(r), rest = r - bt * (w.bh * w.bw), by = w.w.div(rest);
    t = t0 + bt;
    y = y0 + by;
    x = x0 + rest - by * w.bw;
    return (t * w.H + y) * w.W + x;
  };
  auto ask = [&](int r0, int stage) {
    if (r0 < last) {
      int n = 0, t, y, x;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (!TwoHeads || u == 0) n = locate(min(r0 + u * step + sub, last - 1), t, y, x);
        F::ask(ring + (stage * 2 + u) * F::kBytes, w, a, n, h0 + (TwoHeads ? u : 0), lane, l);
      }
    }
    fetch_commit();
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) ask(r_begin + i * stride, i);
  int rows = 0, stage = 0;
  for (int r0 = r_begin; r0 < last; r0 += stride) {
    ask(r0 + (S - 1) * stride, stage == 0 ? S - 1 : stage - 1);
    int r[2], n[2];
    bool mine[2];
    float2 cs[TwoHeads ? 1 : 2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (TwoHeads && u == 1) {
        r[1] = r[0]; n[1] = n[0]; mine[1] = mine[0];
      } else {
        r[u] = r0 + u * step + sub;
        mine[u] = r[u] < last;
        int t, y, x;
        n[u] = locate(min(r[u], last - 1), t, y, x);
        load_turns(refs, a.table, t * a.ht, y_rows + y * a.hh, x_rows + x * a.hw, cs[u]);
      }
    }
    fetch_wait<S - 1>();
    const char* in[2] = {ring + stage * 2 * F::kBytes, ring + (stage * 2 + 1) * F::kBytes};
    stage = stage == S - 1 ? 0 : stage + 1;
    Vals x[4] = {F::get(in[0], 0, lane), F::get(in[0], 1, lane), F::get(in[1], 0, lane),
                 F::get(in[1], 1, lane)};
    if constexpr (To8) {
      const Raw<E> raw[6] = {F::raw(in[0], 0, lane), F::raw(in[0], 1, lane),
                             F::raw(in[0], 2, lane), F::raw(in[1], 0, lane),
                             F::raw(in[1], 1, lane), F::raw(in[1], 2, lane)};
      uint32_t m[6];
#pragma unroll
      for (int i = 0; i < 3; ++i) group_max<G>(raw[i], raw[i + 3], m[i], m[i + 3]);
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        float sc[2];
        uint2 c[2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
          c[u] = encode8(i < 2 ? x[2 * u + i] : unpack(raw[2 + 3 * u]), m[i + 3 * u], sc[u]);
        const uint32_t row[2] = {(uint32_t)((n[0] * 3 + i) * w.n_h + h0),
                                 (uint32_t)((n[1] * 3 + i) * w.n_h + h0 + (TwoHeads ? 1 : 0))};
#pragma unroll
        for (int u = 0; u < 2; ++u)
          if (mine[u]) store_codes<E, D>(at_bytes(o.codes, row[u], D), l, c[u]);
        if (l == 0) {
          if constexpr (TwoHeads) {      // an even row: two scales in one access
            if (mine[0])
              *reinterpret_cast<float2*>(o.scales + row[0]) = make_float2(sc[0], sc[1]);
          } else {
            if (mine[0]) o.scales[row[0]] = sc[0];
            if (mine[1]) o.scales[row[1]] = sc[1];
          }
        }
      }
    }
    float rms[4], pre[4];
    inv_rms<D>(x, a.eps, l, rms, pre);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      Vals &q = x[2 * u], &k = x[2 * u + 1];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        q.p[i] = __fmul2_rn(__fmul2_rn(q.p[i], both(rms[2 * u])), gq.p[i]);
        k.p[i] = __fmul2_rn(__fmul2_rn(k.p[i], both(rms[2 * u + 1])), gk.p[i]);
      }
      turn(q, cs[TwoHeads ? 0 : u]);
      turn(k, cs[TwoHeads ? 0 : u]);
      if (mine[u]) {
        const int h = h0 + (TwoHeads ? u : 0);
        Raw<E> s;
        pack(q, s);
        store_raw<D>(at_bytes(static_cast<E*>(o.q) + h * D, n[u], w.n_h * D * sizeof(E)), l, s);
        pack(k, s);
        const int p = j * w.L + r[u];
        store_raw<D>(at_bytes(static_cast<E*>(o.k) + h * w.kv_head, p, w.kv_tok), l, s);
        store_raw<D>(at_bytes(static_cast<E*>(o.v) + h * w.kv_head, p, w.kv_tok), l,
                     F::value(in[u], lane));
        Vals& to = acc[TwoHeads ? u : 0];
#pragma unroll
        for (int i = 0; i < 4; ++i) to.p[i] = __fadd2_rn(to.p[i], k.p[i]);
      }
    }
    rows += TwoHeads ? 1 : 2;
    if (rows >= kFlush) {
      rows = 0;
#pragma unroll
      for (int u = 0; u < NA; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          sums[u][i][threadIdx.x] += (double)acc[u].at(i);
          acc[u].at(i) = 0.f;
        }
    }
  }
  if (o.blocks == nullptr) return;
#pragma unroll
  for (int u = 0; u < NA; ++u)
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[u][i][threadIdx.x] += (double)acc[u].at(i);
  __syncthreads();
  const int cols = w.up * NA * D;
  for (int c = threadIdx.x; c < cols; c += kThreads) {
    const int hh = c / D, i = c % D / G, ll = c % G;      // lanes apart: no bank conflicts
    double sum = 0.0;
    for (int v = hh / NA; v < kWarps; v += w.up)
#pragma unroll
      for (int b = 0; b < R; ++b) sum += sums[hh % NA][i][v * 32 + b * G + ll];
    total[hh * D + elem_at<E, D>(ll, i)] = sum;
  }
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  const int rank = cluster.block_rank(), size = cluster.num_blocks();
  for (int c = rank * kThreads + threadIdx.x; c < cols; c += size * kThreads) {
    double sum = 0.0;
    for (int m = 0; m < size; ++m) sum += cluster.map_shared_rank(total, m)[c];
    o.blocks[((size_t)(blockIdx.y * w.up * NA + c / D) * w.Nb + j) * D + c % D] =
        (float)(sum / (double)w.L);
  }
  cluster.sync();                    // a member's sums are read until here
}

template <typename E, int D, bool From8, bool To8, bool TwoHeads>
cudaError_t launch_t(const Prob& P, const NormRopeArgs& a, const NormRopeOut& o, int num_sms,
                     cudaStream_t st) {
  constexpr int R = 256 / D;
  const int units = TwoHeads ? P.n_h / 2 : P.n_h;
  Walk w{};
  w.T = P.T; w.H = P.H; w.W = P.W; w.n_h = P.n_h;
  w.bt = P.bt; w.bh = P.bh; w.bw = P.bw;
  w.nbh = P.nbh; w.nbw = P.nbw; w.Nb = P.Nb; w.L = P.L;
  w.ld = (uint32_t)(a.ld * sizeof(E));
  w.up = units % 2 == 0 ? 2 : 1;
  const int step = kWarps / w.up * R, groups = units / w.up;
  if (o.blocks) {
    w.kv_tok = D * sizeof(E);
    w.kv_head = (long long)P.s * D;
    // the chunk count whose CTAs, two on an SM at a time, get through the
    // steps of the slowest slot first; each further CTA of a slot costs about
    // two steps of filling and reducing
    const int slots = 2 * num_sms;
    long long best = -1;
    for (int c = 1; c <= 8; ++c) {
      const long long waves = ((long long)P.Nb * c * groups + slots - 1) / slots;
      const long long cost = waves * (((P.L + c - 1) / c + step - 1) / step + 2);
      if (best < 0 || cost < best) {
        best = cost;
        w.chunks = c;
      }
    }
    w.chunk = (P.L + w.chunks - 1) / w.chunks;
  } else {                             // token order: one block that is the whole latent
    w.bt = P.T; w.bh = P.H; w.bw = P.W;
    w.nbh = w.nbw = w.Nb = 1;
    w.L = P.s;
    w.kv_tok = P.n_h * D * sizeof(E);
    w.kv_head = D;
    const long long want = 8LL * num_sms / groups + 1;
    w.chunk = (int)((P.s + want - 1) / want);
    w.chunk = (w.chunk + step - 1) / step * step;
    w.chunks = (P.s + w.chunk - 1) / w.chunk;
  }
  w.hw = FastDiv(w.bh * w.bw);
  w.w = FastDiv(w.bw);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(w.Nb * w.chunks, groups);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes<E, D, From8, TwoHeads>();
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = o.blocks ? w.chunks : 1;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const auto kernel = k_norm_rope<E, D, From8, To8, TwoHeads>;
  static SmemOptIn opt_in;
  cudaError_t e = opt_in.set(kernel, (int)cfg.dynamicSmemBytes);
  if (e != cudaSuccess) return e;
  {
    VMOBA_TRACE("k_norm_rope", st);
    e = cudaLaunchKernelEx(&cfg, kernel, w, a, o);
  }
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename E, int D, bool TwoHeads>
cudaError_t launch_h(const Prob& P, const NormRopeArgs& a, const NormRopeOut& o, int num_sms,
                     cudaStream_t st) {
  if (a.codes) return launch_t<E, D, true, false, TwoHeads>(P, a, o, num_sms, st);
  if (o.codes) return launch_t<E, D, false, true, TwoHeads>(P, a, o, num_sms, st);
  return launch_t<E, D, false, false, TwoHeads>(P, a, o, num_sms, st);
}

template <typename E, int D>
cudaError_t launch_d(const Prob& P, const NormRopeArgs& a, const NormRopeOut& o, int num_sms,
                     cudaStream_t st) {
  return P.n_h % 2 == 0 ? launch_h<E, D, true>(P, a, o, num_sms, st)
                        : launch_h<E, D, false>(P, a, o, num_sms, st);
}

// (cos, sin) of every axis position and pair: the angle (origin + position) *
// base^(-2 i / dim) in fp64, since a far position times a frequency near one
// has no correct fp32 fraction, each result rounded once.
__global__ void k_rope_table(int T, int H, int W, int ht, int hh, int hw, double base,
                             long long ot, long long oy, long long ox, float2* table) {
  const int nt = T * ht, ny = H * hh, nx = W * hw;
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= nt + ny + nx) return;
  const int k = i < nt ? i : (i < nt + ny ? i - nt : i - nt - ny);
  const int half = i < nt ? ht : (i < nt + ny ? hh : hw);
  const long long origin = i < nt ? ot : (i < nt + ny ? oy : ox);
  const int pos = k / half, pair = k - pos * half;
  double s, c;
  sincos((double)(origin + pos) * pow(base, -(double)pair / (double)half), &s, &c);
  table[i] = make_float2((float)c, (float)s);
}

}  // namespace

cudaError_t launch_norm_rope(const Prob& P, const NormRopeArgs& a, const NormRopeOut& o,
                             int num_sms, cudaStream_t st) {
  if (P.dtype == VMOBA_BF16)
    return P.d == 128 ? launch_d<__nv_bfloat16, 128>(P, a, o, num_sms, st)
                      : launch_d<__nv_bfloat16, 64>(P, a, o, num_sms, st);
  return P.d == 128 ? launch_d<float, 128>(P, a, o, num_sms, st)
                    : launch_d<float, 64>(P, a, o, num_sms, st);
}

cudaError_t launch_rope_table(int T, int H, int W, int ht, int hh, int hw, double base,
                              const long long (&origin)[3], float2* table, cudaStream_t st) {
  const int n = T * ht + H * hh + W * hw;
  if (n == 0) return cudaSuccess;
  {
    VMOBA_TRACE("k_rope_table", st);
    k_rope_table<<<(n + 127) / 128, 128, 0, st>>>(T, H, W, ht, hh, hw, base, origin[0], origin[1],
                                                  origin[2], table);
  }
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace vmoba
