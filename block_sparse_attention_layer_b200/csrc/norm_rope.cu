// Between the projection and the attention: the RMS norm of each head's query
// and key row, y = x g / sqrt(mean(x^2) + eps), and its rotation by the
// token's (t, y, x) position, in one pass that also moves v.  q leaves in
// token order; k and v leave in token order (dense attention) or in the
// layer's partition order together with the fp32 block means of k, so that
// the sparse layer needs no partition pass over them.  The raw rows come from
// the projection or from an 8-bit checkpoint, and the pass can write that
// checkpoint.
//
// Bound: HBM.  Each raw value is read once, each result written once: 6 s n_h d
// elements (3 of them 1.03 bytes when they come from codes, 3.1 s n_h d bytes
// more when a checkpoint is written).  55296 tokens, 12 heads of 128, bf16:
// 161 us in token order or into 288 blocks (6.3 TB/s, 0.98 of a plain copy's
// 6.46), 175 us into eight blocks, 214 us with the checkpoint written (0.93),
// 137 us from it (0.88).
//
// A lane works on two rows of q, k and v at a time, two neighbouring heads of
// one token where the head count is even (they share the position and its
// table entries), else one head of two tokens; the four sums of squares go
// through one shuffle tree.  Rows reach a lane through its own place in shared
// memory by asynchronous copies, two steps ahead: loads in registers at two
// CTAs an SM left 55296 tokens at 244 us where these took 202.  A CTA's eight
// warps take `up` neighbouring units of heads, the rest of the warps further
// tokens.  A block of keys may be cut into chunks, one CTA each; the CTAs of a
// block are then a cluster, whose members add their column sums over
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
  int chunks;                      // CTAs that share a block's rows
  int up;                          // units of heads of a CTA
  uint32_t ld, q_tok, kv_tok;      // bytes between tokens of the raw rows and q; positions of k, v
  long long kv_head;               // elements between heads of k and v
};

// Two rows of q, k and v on their way through shared memory.
template <typename E, int D, bool From8, bool TwoHeads>
struct Feed {
  static constexpr int kSlot = Slot<E, D>::kBytes, kBytes = 6 * kSlot;
  const char* in[3];                 // the lane's first 16 bytes of head h0, token 0
  __device__ __forceinline__ Feed(const Walk& w, const NormRopeArgs& a, int h0, int l) {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      in[i] = pinned(static_cast<const char*>(a.in[i]) + h0 * D * (int)sizeof(E) + l * 16);
  }
  __device__ __forceinline__ void ask(char* s, const Walk& w, int n, int u, int sub,
                                      int l) const {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      Slot<E, D>::ask(s + (3 * u + i) * kSlot,
                      at_bytes(in[i], n, w.ld) + (TwoHeads ? u * D * (int)sizeof(E) : 0),
                      sub * (D / 8) + l);
  }
  __device__ __forceinline__ static Raw<E> raw(const char* s, int i, int u, int sub, int l) {
    return Slot<E, D>::get(s + (3 * u + i) * kSlot, sub * (D / 8) + l);
  }
  // x r of q and k of both rows
  __device__ __forceinline__ static void load(const char* s, float eps, int sub, int l,
                                              Vals (&x)[4]) {
    float r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = unpack(raw(s, k & 1, k / 2, sub, l));
    normalise<D>(x, eps, l, r);
  }
  __device__ __forceinline__ static Raw<E> value(const char* s, int u, int sub, int l) {
    return raw(s, 2, u, sub, l);
  }
};
template <typename E, int D, bool TwoHeads>
struct Feed<E, D, true, TwoHeads> {
  using C = CodeRows<E, D, 3, TwoHeads>;
  static constexpr int kBytes = C::kBytes;
  const char* codes[3];
  const float* scale;
  __device__ __forceinline__ Feed(const Walk& w, const NormRopeArgs& a, int h0, int l) {
#pragma unroll
    for (int i = 0; i < 3; ++i) codes[i] = pinned(C::codes_at(a.codes, i, h0, w.n_h, l));
    scale = pinned(C::scale_at(a.scales, h0, w.n_h, l));
  }
  __device__ __forceinline__ void ask(char* s, const Walk& w, int n, int u, int sub,
                                      int l) const {
    C::ask(s, codes, scale, n, w.n_h, u, sub, l);
  }
  __device__ __forceinline__ static void load(const char* s, float eps, int sub, int l,
                                              Vals (&x)[4]) {
    uint2 c[4];
    float sc[4], r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      c[k] = C::codes(s, k & 1, k / 2, sub, l);
      sc[k] = C::scale(s, k & 1, k / 2, sub);
    }
    normalise<D>(c, sc, eps, l, x, r);
  }
  __device__ __forceinline__ static Raw<E> value(const char* s, int u, int sub, int l) {
    Raw<E> r;
    pack(decode8(C::codes(s, 2, u, sub, l), C::scale(s, 2, u, sub)), r);
    return r;
  }
};

// Steps of a warp in shared memory: the one at work and those being loaded
// (as many as leave room for two CTAs an SM, or for fp32 rows one).
template <typename E, bool From8>
constexpr int stages() { return From8 || sizeof(E) == 2 ? 3 : 2; }

// Shared memory: the loads under way and their tokens, the column sums of the
// CTA and those of its warps' lanes (one for each part of a row).
template <typename E, int D, bool From8, bool TwoHeads>
struct Smem {
  static constexpr int kNA = TwoHeads ? 2 : 1;
  static constexpr int kLanes = kWarps * (D / 8);
  static constexpr int kRing = stages<E, From8>() * kWarps * Feed<E, D, From8, TwoHeads>::kBytes;
  static constexpr int kSpots = stages<E, From8>() * kWarps * 8 * (int)sizeof(Spot);
  static constexpr int kTotal = kMaxUp * kNA * D * (int)sizeof(double);
  static constexpr int kBytes = kRing + kSpots + kTotal + kNA * 8 * kLanes * (int)sizeof(double);
};

template <typename E, int D, bool From8, bool To8, bool TwoHeads>
__global__ void __launch_bounds__(kThreads, 2)
k_norm_rope(const __grid_constant__ Walk w, const __grid_constant__ NormRopeArgs a,
            const __grid_constant__ NormRopeOut o) {
  constexpr int G = D / 8, R = 32 / G, NA = TwoHeads ? 2 : 1;
  using F = Feed<E, D, From8, TwoHeads>;
  using M = Smem<E, D, From8, TwoHeads>;
  constexpr int S = stages<E, From8>();
  extern __shared__ __align__(16) char smem[];
  char* ring = smem + (threadIdx.x >> 5) * (S * F::kBytes);
  Spot* spots = reinterpret_cast<Spot*>(smem + M::kRing) + (threadIdx.x >> 5) * (S * 8);
  double* total = reinterpret_cast<double*>(smem + M::kRing + M::kSpots);
  double(&sums)[NA][8][M::kLanes] =
      *reinterpret_cast<double(*)[NA][8][M::kLanes]>(total + kMaxUp * NA * D);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / G, l = lane % G;
  const int h0 = (blockIdx.y * w.up + warp % w.up) * NA;
  // partition order: chunk x of block z; token order: chunk z.  The chunks of a
  // block are interleaved strides of its rows, so that their CTAs walk one
  // window of it together (1 to 3 % faster than stretches of their own).
  const int j = o.blocks ? blockIdx.z : 0;
  const int step = kWarps / w.up * R, own = step * (TwoHeads ? 1 : 2);
  const int first = (o.blocks ? blockIdx.x : blockIdx.z) * own, last = w.L;
  after_previous();
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
      if (sub == 0) sums[u][i][warp * G + l] = 0.0;
    }
  // adds the lanes' fp32 sums of a row part to its fp64 sums
  auto flush = [&] {
#pragma unroll
    for (int u = 0; u < NA; ++u)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float v = acc[u].at(i);
#pragma unroll
        for (int m = G; m < 32; m <<= 1) v += __shfl_xor_sync(kAll, v, m);
        if (sub == 0) sums[u][i][warp * G + l] += (double)v;
        acc[u].at(i) = 0.f;
      }
  };

  const int stride = own * w.chunks;
  const int r_begin = first + warp / w.up * R;
  // row r of the block is token n = (t, y, x)
  auto locate = [&](int r) {
    const int bt = w.hw.div(r), rest = r - bt * (w.bh * w.bw), by = w.w.div(rest);
    const int t = t0 + bt, y = y0 + by, x = x0 + rest - by * w.bw;
    return Spot{{t * a.ht, y_rows + y * a.hh, x_rows + x * a.hw}, (t * w.H + y) * w.W + x};
  };
  const F feed(w, a, h0, l);
  auto ask = [&](int r0, int stage) {
    if (r0 < last) {
      int n = 0;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (!TwoHeads || u == 0) {
          const Spot spot = locate(min(r0 + u * step + sub, last - 1));
          n = spot.n;
          if (l == 0) spots[stage * 8 + u * 4 + sub] = spot;
        }
        feed.ask(ring + stage * F::kBytes, w, n, u, sub, l);
      }
    }
    fetch_commit();
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) ask(r_begin + i * stride, i);
  // the lane's first bytes of head h0, token or position 0
  char* const to_q = pinned(static_cast<char*>(o.q) + h0 * D * (int)sizeof(E) + l * 16);
  char* const to_k =
      pinned(static_cast<char*>(o.k) + h0 * w.kv_head * (int)sizeof(E) + l * 16);
  char* const to_v =
      pinned(static_cast<char*>(o.v) + h0 * w.kv_head * (int)sizeof(E) + l * 16);
  [[maybe_unused]] char* to_codes = nullptr;
  [[maybe_unused]] float* to_scales = nullptr;
  if constexpr (To8) {
    to_codes = pinned(reinterpret_cast<char*>(o.codes) + h0 * D + l * (sizeof(E) == 2 ? 8 : 4));
    to_scales = pinned(o.scales + h0);
  }
  int rows = 0, stage = 0;
  for (int r0 = r_begin; r0 < last; r0 += stride) {
    __syncwarp();                    // the spots of the stage that is refilled have been read
    ask(r0 + (S - 1) * stride, stage == 0 ? S - 1 : stage - 1);
    __syncwarp();                    // and this stage's, written S - 1 steps ago, are visible
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
        const Spot* spot = spots + stage * 8 + u * 4 + sub;
        n[u] = spot->n;
        load_turns(refs, a.table, a.still, spot, cs[u]);
      }
    }
    fetch_wait<S - 1>();
    if constexpr (From8) __syncwarp();
    const char* in = ring + stage * F::kBytes;
    stage = stage == S - 1 ? 0 : stage + 1;
    if constexpr (To8) {
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const Raw<E> raw[2] = {F::raw(in, i, 0, sub, l), F::raw(in, i, 1, sub, l)};
        uint32_t m[2];
        float sc[2];
        uint2 c[2];
        group_max<G>(raw[0], raw[1], m[0], m[1]);
#pragma unroll
        for (int u = 0; u < 2; ++u) c[u] = encode8<E>(unpack(raw[u]), m[u], sc[u]);
        // row (n, i) of the checkpoint: n_h heads of D codes
        const int row[2] = {(n[0] * 3 + i) * w.n_h, (n[1] * 3 + i) * w.n_h};
#pragma unroll
        for (int u = 0; u < 2; ++u)
          if (mine[u])
            store_codes<E, D>(at_bytes(to_codes, row[u], D) + (TwoHeads ? u * D : 0), c[u]);
        if (l == 0) {
          if constexpr (TwoHeads) {      // an even row: two scales in one access
            if (mine[0])
              *reinterpret_cast<float2*>(to_scales + row[0]) = make_float2(sc[0], sc[1]);
          } else {
            if (mine[0]) to_scales[row[0]] = sc[0];
            if (mine[1]) to_scales[row[1]] = sc[1];
          }
        }
      }
    }
    Vals x[4];
    F::load(in, a.eps, sub, l, x);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      Vals &q = x[2 * u], &k = x[2 * u + 1];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        q.p[i] = __fmul2_rn(q.p[i], gq.p[i]);
        k.p[i] = __fmul2_rn(k.p[i], gk.p[i]);
      }
      turn(q, cs[TwoHeads ? 0 : u]);
      turn(k, cs[TwoHeads ? 0 : u]);
      if (mine[u]) {
        Raw<E> s;
        pack(q, s);
        Slot<E, D>::put(at_bytes(to_q, n[u], w.q_tok) + (TwoHeads ? u * D * (int)sizeof(E) : 0),
                        s);
        pack(k, s);
        const int p = j * w.L + r[u];
        const long long head = TwoHeads && u ? w.kv_head * (int)sizeof(E) : 0;
        Slot<E, D>::put(at_bytes(to_k, p, w.kv_tok) + head, s);
        Slot<E, D>::put(at_bytes(to_v, p, w.kv_tok) + head, F::value(in, u, sub, l));
        Vals& to = acc[TwoHeads ? u : 0];
#pragma unroll
        for (int i = 0; i < 4; ++i) to.p[i] = __fadd2_rn(to.p[i], k.p[i]);
      }
    }
    rows += TwoHeads ? 1 : 2;
    if (rows >= kFlush) {
      rows = 0;
      flush();
    }
  }
  if (o.blocks == nullptr) return;
  flush();
  __syncthreads();
  const int cols = w.up * NA * D;
  auto write = [&](int c, double sum) {
    o.blocks[((size_t)(blockIdx.y * w.up * NA + c / D) * w.Nb + j) * D + c % D] =
        (float)(sum / (double)w.L);
  };
  for (int c = threadIdx.x; c < cols; c += kThreads) {
    const int hh = c / D, i = c % D / G, ll = c % G;      // lanes apart: no bank conflicts
    double sum = 0.0;
    for (int v = hh / NA; v < kWarps; v += w.up)
      sum += sums[hh % NA][i][v * G + ll];
    const int col = hh * D + elem_at<E, D>(ll, i);
    if (w.chunks == 1)
      write(col, sum);
    else
      total[col] = sum;
  }
  if (w.chunks == 1) return;
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  const int rank = cluster.block_rank();
  for (int c = rank * kThreads + threadIdx.x; c < cols; c += w.chunks * kThreads) {
    double sum = 0.0;
    for (int m = 0; m < w.chunks; ++m) sum += cluster.map_shared_rank(total, m)[c];
    write(c, sum);
  }
  cluster.sync();                    // a member's sums are read until here
}

// CTAs of a kernel that the device runs at once in clusters of each size
// (clusters do not cross GPCs, whose sizes differ), asked once per device.
class Capacity {
 public:
  template <typename K>
  int ctas(K kernel, int dev, int cluster, int smem, int num_sms) {
    if (dev < 0 || dev >= kDevices) return num_sms;
    std::atomic<int>& known = known_[dev][cluster];
    int n = known.load(std::memory_order_relaxed);
    if (n) return n;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(cluster);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
      (void)cudaGetLastError();
      return num_sms;
    }
    known.store(n * cluster, std::memory_order_relaxed);
    return n * cluster;
  }

 private:
  static constexpr int kDevices = 16;
  std::atomic<int> known_[kDevices][9] = {};
};

template <typename E, int D, bool From8, bool To8, bool TwoHeads>
cudaError_t launch_t(const Prob& P, const NormRopeArgs& a, const NormRopeOut& o, int num_sms,
                     cudaStream_t st) {
  constexpr int R = 256 / D;
  using M = Smem<E, D, From8, TwoHeads>;
  const auto kernel = k_norm_rope<E, D, From8, To8, TwoHeads>;
  static SmemOptIn opt_in;
  static Capacity capacity;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = opt_in.set(kernel, M::kBytes, dev);
  if (e != cudaSuccess) return e;
  const int units = TwoHeads ? P.n_h / 2 : P.n_h;
  Walk w{};
  w.T = P.T; w.H = P.H; w.W = P.W; w.n_h = P.n_h;
  w.bt = P.bt; w.bh = P.bh; w.bw = P.bw;
  w.nbh = P.nbh; w.nbw = P.nbw; w.Nb = P.Nb; w.L = P.L;
  w.ld = (uint32_t)(a.ld * sizeof(E));
  w.q_tok = P.n_h * D * sizeof(E);
  if (o.blocks) {
    w.kv_tok = D * sizeof(E);
    w.kv_head = (long long)P.s * D;
    // One CTA for each block and unit of heads where these are at least one and
    // a half rounds of CTAs (1.6 rounds: 108 us against 113 of the search
    // below on 32760 tokens in 78 blocks; 5.8 rounds: 162 against 165 on 55296
    // tokens in 288 blocks; but from codes 141 against 137).  Else the units
    // and chunks of a CTA for which the slowest of the places that CTAs run in
    // has the fewest strides; a CTA's filling and reducing costs about two, a
    // cluster's two more (55296 tokens in 8 blocks: 174 us against 189 with
    // eight chunks of two units, 433 with one CTA a block; 2048 tokens of 4
    // heads in 64 blocks: 3.2 us against 4.2 with clusters of two).
    w.up = w.chunks = 1;
    long long best = -1;
    const bool many = !From8 && 2LL * P.Nb * units >=
                                    3LL * capacity.ctas(kernel, dev, 1, M::kBytes, num_sms);
    for (int up = 1; up <= (units % 2 ? 1 : 2) && !many; ++up) {
      const int own = kWarps / up * R * (TwoHeads ? 1 : 2), strides = (P.L + own - 1) / own;
      for (int c = 1; c <= 8 && c <= strides; ++c) {
        const long long ctas = (long long)P.Nb * c * (units / up);
        const int slots = capacity.ctas(kernel, dev, c, M::kBytes, num_sms);
        const long long cost =
            ((ctas + slots - 1) / slots) * ((strides + c - 1) / c + (c > 1 ? 4 : 2));
        if (best < 0 || cost < best) {
          best = cost;
          w.up = up;
          w.chunks = c;
        }
      }
    }
  } else {                             // token order: one block that is the whole latent
    w.bt = P.T; w.bh = P.H; w.bw = P.W;
    w.nbh = w.nbw = w.Nb = 1;
    w.L = P.s;
    w.kv_tok = P.n_h * D * sizeof(E);
    w.kv_head = D;
    // eight CTAs an SM (11520 tokens: 36.5 us; two 40.9, sixteen 36.6, 32 43.8)
    w.up = units % 2 == 0 ? 2 : 1;
    const int own = kWarps / w.up * R * (TwoHeads ? 1 : 2);
    const long long strides = (P.s + own - 1) / own, want = 8LL * num_sms * w.up / units + 1;
    w.chunks = (int)(strides < want ? strides : want);
  }
  w.hw = FastDiv(w.bh * w.bw);
  w.w = FastDiv(w.bw);
  VMOBA_TRACE("k_norm_rope", st);
  // all heads of neighbouring tokens run at one time: whole rows of DRAM pages
  const int groups = units / w.up;
  return o.blocks ? launch(kernel, dim3(w.chunks, groups, w.Nb), kThreads, M::kBytes, w.chunks,
                           st, w, a, o)
                  : launch(kernel, dim3(1, groups, w.chunks), kThreads, M::kBytes, 1, st, w, a, o);
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
  after_previous();
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
  VMOBA_TRACE("k_rope_table", st);
  return launch(k_rope_table, dim3((n + 127) / 128), 128, 0, 1, st, T, H, W, ht, hh, hw, base,
                origin[0], origin[1], origin[2], table);
}

}  // namespace vmoba
