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
// A CTA's eight warps take `hp` neighbouring heads; a warp holds R = 256 / d
// rows of its head at a time and asks for the next ones before it works on
// these.  A block of keys is cut into C chunks, one CTA each; the C CTAs are a
// cluster, whose members add their column sums over distributed shared memory
// in a fixed order.  Token order is the case of a single block that is the
// whole latent, without clusters.
#include <cooperative_groups.h>

#include "rows.cuh"

namespace vmoba {
namespace {

using namespace rows;
namespace cg = cooperative_groups;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxHp = 4;
constexpr int kFlush = 64;         // rows a lane adds in fp32 before they go to its fp64 sums

// Where the rows of one launch lie.
struct Walk {
  int T, H, W, s, n_h;
  int bt, bh, bw;                  // box of a block
  int nbh, nbw, Nb, L;
  FastDiv hw, w;                   // bh * bw, bw
  int chunk, chunks;               // rows of a chunk, chunks of a block
  int hp;                          // heads of a CTA
  long long kv_tok, kv_head;       // strides of k and v by position and head
};

// One row of q, k and v as loaded.
template <typename E, int D, bool From8>
struct Rows {
  Raw<E> q, k, v;
  __device__ __forceinline__ void load(const NormRopeArgs& a, int n, int h, int n_h, int l) {
    const long long at = n * a.ld + (long long)h * D;
    q = load_row<D>(static_cast<const E*>(a.in[0]) + at, l);
    k = load_row<D>(static_cast<const E*>(a.in[1]) + at, l);
    v = load_row<D>(static_cast<const E*>(a.in[2]) + at, l);
  }
  __device__ __forceinline__ void values(float (&xq)[8], float (&xk)[8]) const {
    unpack(q, xq);
    unpack(k, xk);
  }
  __device__ __forceinline__ Raw<E> value() const { return v; }
};
template <typename E, int D>
struct Rows<E, D, true> {
  uint2 c[3];
  float sc[3];
  __device__ __forceinline__ void load(const NormRopeArgs& a, int n, int h, int n_h, int l) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const long long row = ((long long)n * 3 + i) * n_h + h;
      c[i] = load_codes<E, D>(a.codes + row * D, l);
      sc[i] = __ldg(a.scales + row);
    }
  }
  __device__ __forceinline__ void values(float (&xq)[8], float (&xk)[8]) const {
    decode8(c[0], sc[0], xq);
    decode8(c[1], sc[1], xk);
  }
  __device__ __forceinline__ Raw<E> value() const {
    float x[8];
    decode8(c[2], sc[2], x);
    Raw<E> r;
    pack(x, r);
    return r;
  }
};

template <typename E, int D, bool From8, bool To8>
__global__ void __launch_bounds__(kThreads, 2)
k_norm_rope(Walk w, NormRopeArgs a, NormRopeOut o) {
  constexpr int G = D / 8, R = 32 / G;
  __shared__ double sums[8][kThreads];       // a thread's fp64 column sums
  __shared__ double total[kMaxHp * D];       // the CTA's, summed over the cluster at the end
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / G, l = lane % G;
  const int h = blockIdx.y * w.hp + warp % w.hp;
  const int j = blockIdx.x / w.chunks;
  const int first = (blockIdx.x - j * w.chunks) * w.chunk, last = min(first + w.chunk, w.L);
  const int step = kWarps / w.hp * R;

  float gq[8], gk[8];
  load_weights<E, D>(a.gq, l, gq);
  load_weights<E, D>(a.gk, l, gk);
  const PairRefs refs = pair_refs<E, D>(l, a.ht, a.hh, a.hw);
  const int y_rows = w.T * a.ht, x_rows = y_rows + w.H * a.hh;
  const long long row3 = (long long)w.n_h * D;
  const int pw = j % w.nbw, jj = j / w.nbw, ph = jj % w.nbh, pt = jj / w.nbh;
  const int t0 = pt * w.bt, y0 = ph * w.bh, x0 = pw * w.bw;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    acc[i] = 0.f;
    sums[i][threadIdx.x] = 0.0;
  }

  // row r of the block is token n = (t, y, x)
  int t, y, x, n;
  auto locate = [&](int r) {
    t = w.hw.div(r);
    const int rest = r - t * (w.bh * w.bw);
    y = w.w.div(rest);
    x = x0 + rest - y * w.bw;
    t += t0;
    y += y0;
    n = (t * w.H + y) * w.W + x;
  };
  Rows<E, D, From8> cur, next;
  int r = first + warp / w.hp * R + sub;
  if (r - sub < last) {
    locate(min(r, last - 1));
    cur.load(a, n, h, w.n_h, l);
  }
  int rows = 0;
  for (; r - sub < last; r += step) {
    const bool mine = r < last;
    const int nn = n, rt = t * a.ht, ry = y_rows + y * a.hh, rx = x_rows + x * a.hw;
    float2 cs[4];
    load_turns(refs, a.table, rt, ry, rx, cs);
    if (r - sub + step < last) {
      locate(min(r + step, last - 1));
      next.load(a, n, h, w.n_h, l);
    }
    float xq[8], xk[8];
    cur.values(xq, xk);
    const Raw<E> rv = cur.value();
    if constexpr (To8) {
      float sc[3], xv[8];
      uint2 c[3];
      unpack(rv, xv);
      c[0] = encode8(xq, row_max<G>(abs_max_bits(xq)), sc[0]);
      c[1] = encode8(xk, row_max<G>(abs_max_bits(xk)), sc[1]);
      c[2] = encode8(xv, row_max<G>(abs_max_bits(xv)), sc[2]);
      if (mine) {
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          const long long row = ((long long)nn * 3 + i) * w.n_h + h;
          store_codes<E, D>(o.codes + row * D, l, c[i]);
          if (l == 0) o.scales[row] = sc[i];
        }
      }
    }
    float pre;
    const float rq = inv_rms<D>(xq, a.eps, pre), rk = inv_rms<D>(xk, a.eps, pre);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      xq[i] = xq[i] * rq * gq[i];
      xk[i] = xk[i] * rk * gk[i];
    }
    turn(xq, cs);
    turn(xk, cs);
    if (mine) {
      Raw<E> u;
      pack(xq, u);
      store_raw<D>(static_cast<E*>(o.q) + nn * row3 + (long long)h * D, l, u);
      pack(xk, u);
      const long long at = ((long long)j * w.L + r) * w.kv_tok + h * w.kv_head;
      store_raw<D>(static_cast<E*>(o.k) + at, l, u);
      store_raw<D>(static_cast<E*>(o.v) + at, l, rv);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += xk[i];
    }
    if (++rows == kFlush) {
      rows = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sums[i][threadIdx.x] += (double)acc[i];
        acc[i] = 0.f;
      }
    }
    cur = next;
  }
  if (o.blocks == nullptr) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) sums[i][threadIdx.x] += (double)acc[i];
  __syncthreads();
  const int cols = w.hp * D;
  for (int c = threadIdx.x; c < cols; c += kThreads) {
    const int hh = c / D, i = c % D / G, ll = c % G;      // lanes apart: no bank conflicts
    double sum = 0.0;
    for (int v = hh; v < kWarps; v += w.hp)
#pragma unroll
      for (int b = 0; b < R; ++b) sum += sums[i][v * 32 + b * G + ll];
    total[hh * D + elem_at<E, D>(ll, i)] = sum;
  }
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  const int rank = cluster.block_rank(), size = cluster.num_blocks();
  for (int c = rank * kThreads + threadIdx.x; c < cols; c += size * kThreads) {
    double sum = 0.0;
    for (int m = 0; m < size; ++m) sum += cluster.map_shared_rank(total, m)[c];
    o.blocks[((size_t)(blockIdx.y * w.hp + c / D) * w.Nb + j) * D + c % D] =
        (float)(sum / (double)w.L);
  }
  cluster.sync();                    // a member's sums are read until here
}

template <typename E, int D, bool From8, bool To8>
cudaError_t launch_t(const Prob& P, const NormRopeArgs& a, const NormRopeOut& o, int num_sms,
                     cudaStream_t st) {
  constexpr int R = 256 / D;
  Walk w{};
  w.T = P.T; w.H = P.H; w.W = P.W; w.s = P.s; w.n_h = P.n_h;
  w.bt = P.bt; w.bh = P.bh; w.bw = P.bw;
  w.nbh = P.nbh; w.nbw = P.nbw; w.Nb = P.Nb; w.L = P.L;
  w.hp = P.n_h % 4 == 0 ? 4 : (P.n_h % 2 == 0 ? 2 : 1);
  const int step = kWarps / w.hp * R, groups = P.n_h / w.hp;
  if (o.blocks) {
    w.kv_tok = D;
    w.kv_head = (long long)P.s * D;
    w.chunks = 1;
    while (w.chunks < 8 && (long long)P.Nb * w.chunks * groups < 4 * num_sms &&
           P.L > w.chunks * step * 2)
      w.chunks *= 2;
    w.chunk = (P.L + w.chunks - 1) / w.chunks;
  } else {                             // token order: one block that is the whole latent
    w.bt = P.T; w.bh = P.H; w.bw = P.W;
    w.nbh = w.nbw = w.Nb = 1;
    w.L = P.s;
    w.kv_tok = (long long)P.n_h * D;
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
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = o.blocks ? w.chunks : 1;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cudaError_t e;
  {
    VMOBA_TRACE("k_norm_rope", st);
    e = cudaLaunchKernelEx(&cfg, k_norm_rope<E, D, From8, To8>, w, a, o);
  }
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename E, int D>
cudaError_t launch_d(const Prob& P, const NormRopeArgs& a, const NormRopeOut& o, int num_sms,
                     cudaStream_t st) {
  if (a.codes) return launch_t<E, D, true, false>(P, a, o, num_sms, st);
  if (o.codes) return launch_t<E, D, false, true>(P, a, o, num_sms, st);
  return launch_t<E, D, false, false>(P, a, o, num_sms, st);
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
