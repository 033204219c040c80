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
// One CTA per (block, head); a warp holds R = 256 / d rows of that head, and
// consecutive groups of R tokens go round the warps.  Token order is the case
// of a single block that is the whole latent.
#include "rows.cuh"

namespace vmoba {
namespace {

using namespace rows;

constexpr int kWarps = 8;

template <typename E, int D, bool From8, bool To8>
__global__ void __launch_bounds__(kWarps * 32)
k_norm_rope(Prob P, NormRopeArgs a, NormRopeOut o, int chunk, long long kv_tok,
            long long kv_head) {
  constexpr int G = D / 8, R = 32 / G;
  __shared__ double red[kWarps * R][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / G, l = lane % G;
  const int h = blockIdx.y;
  // rows [first, last) of the partition order; a chunk never leaves its block
  const int first = blockIdx.x * chunk, last = min(first + chunk, P.s);

  float gq[8], gk[8];
  load_weights<E, D>(a.gq, l, gq);
  load_weights<E, D>(a.gk, l, gk);
  const PairRefs refs = pair_refs<E, D>(l, P.T, P.H, a.ht, a.hh, a.hw);
  const long long row3 = (long long)P.n_h * D;
  double acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0;

  for (int p0 = first + warp * R; p0 < last; p0 += kWarps * R) {
    const bool mine = p0 + sub < last;
    const int p = mine ? p0 + sub : last - 1;
    const int n = perm_token(P, p);
    const int t = n / (P.H * P.W), yx = n - t * (P.H * P.W), y = yx / P.W, x = yx - y * P.W;
    float xq[8], xk[8], xv[8];
    Raw<E> rv;
    const long long ckpt = ((long long)n * 3 * P.n_h + h) * D;   // its q row; k, v: + row3, 2 row3
    if constexpr (From8) {
      float sc[3];
      uint2 c[3];
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        c[i] = load_codes<E, D>(a.codes + ckpt + i * row3, l);
        sc[i] = __ldg(a.scales + ((long long)n * 3 + i) * P.n_h + h);
      }
      decode8(c[0], sc[0], xq);
      decode8(c[1], sc[1], xk);
      decode8(c[2], sc[2], xv);
      pack(xv, rv);
    } else {
      const long long at = n * a.ld + (long long)h * D;
      const Raw<E> rq = load_row<D>(static_cast<const E*>(a.in[0]) + at, l);
      const Raw<E> rk = load_row<D>(static_cast<const E*>(a.in[1]) + at, l);
      rv = load_row<D>(static_cast<const E*>(a.in[2]) + at, l);
      unpack(rq, xq);
      unpack(rk, xk);
    }
    if constexpr (To8) {
      unpack(rv, xv);
      float sc[3];
      uint2 c[3];
      c[0] = encode8(xq, row_max<G>(abs_max_bits(xq)), sc[0]);
      c[1] = encode8(xk, row_max<G>(abs_max_bits(xk)), sc[1]);
      c[2] = encode8(xv, row_max<G>(abs_max_bits(xv)), sc[2]);
      if (mine) {
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          store_codes<E, D>(o.codes + ckpt + i * row3, l, c[i]);
          if (l == 0) o.scales[((long long)n * 3 + i) * P.n_h + h] = sc[i];
        }
      }
    }
    float2 cs[4];
    load_turns(refs, a.table, t, y, x, cs);
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
      Raw<E> w;
      pack(xq, w);
      store_raw<D>(static_cast<E*>(o.q) + n * row3 + (long long)h * D, l, w);
      pack(xk, w);
      const long long at = p * kv_tok + h * kv_head;
      store_raw<D>(static_cast<E*>(o.k) + at, l, w);
      store_raw<D>(static_cast<E*>(o.v) + at, l, rv);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += (double)xk[i];
    }
  }
  if (o.blocks == nullptr) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) red[warp * R + sub][elem_at<E, D>(l, i)] = acc[i];
  __syncthreads();
  for (int c = threadIdx.x; c < D; c += blockDim.x) {
    double sum = 0.0;
    for (int w = 0; w < kWarps * R; ++w) sum += red[w][c];
    o.blocks[((size_t)h * P.Nb + blockIdx.x) * D + c] = (float)(sum / (double)P.L);
  }
}

template <typename E, int D, bool From8, bool To8>
cudaError_t launch_t(Prob P, const NormRopeArgs& a, const NormRopeOut& o, cudaStream_t st) {
  int chunk = P.L;
  long long kv_tok = D, kv_head = (long long)P.s * D;
  if (o.blocks == nullptr) {            // token order: one block that is the whole latent
    P.bt = P.T; P.bh = P.H; P.bw = P.W;
    P.nbt = P.nbh = P.nbw = P.Nb = 1;
    P.L = P.s;
    kv_tok = (long long)P.n_h * D;
    kv_head = D;
    chunk = 64;
  }
  const dim3 grid((P.s + chunk - 1) / chunk, P.n_h);
  {
    VMOBA_TRACE("k_norm_rope", st);
    k_norm_rope<E, D, From8, To8><<<grid, kWarps * 32, 0, st>>>(P, a, o, chunk, kv_tok, kv_head);
  }
  count_launches(1);
  return cudaGetLastError();
}

template <typename E, int D>
cudaError_t launch_d(const Prob& P, const NormRopeArgs& a, const NormRopeOut& o, cudaStream_t st) {
  if (a.codes) return launch_t<E, D, true, false>(P, a, o, st);
  if (o.codes) return launch_t<E, D, false, true>(P, a, o, st);
  return launch_t<E, D, false, false>(P, a, o, st);
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
                             cudaStream_t st) {
  if (P.dtype == VMOBA_BF16)
    return P.d == 128 ? launch_d<__nv_bfloat16, 128>(P, a, o, st)
                      : launch_d<__nv_bfloat16, 64>(P, a, o, st);
  return P.d == 128 ? launch_d<float, 128>(P, a, o, st) : launch_d<float, 64>(P, a, o, st);
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
