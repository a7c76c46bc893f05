// Eviction from the block-scaled 8-bit KV cache (format: cache8.cuh) by accumulated attention
// weight: which tokens stay, and their move to another cache.
#include "cache8.cuh"

namespace sgqa {
namespace {

constexpr int kSelThr = 1024;

// Order-preserving key of a weight; NaN ranks as -infinity.
__device__ __forceinline__ uint32_t weight_key(float w) { return score_key(w != w ? -INFINITY : w); }

// One CTA per (sequence, group). Of more than `keep` tokens the `recent` last stay, and of the N
// before them the c = keep - recent heaviest: an exact radix select (8 bits a pass) finds the key of
// the c-th heaviest and how many of its equals stay, the lowest positions first; an ordered pass
// writes the positions.
__global__ void __launch_bounds__(kSelThr) cache8_keep_kernel(C8EvictArgs a) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t s_prefix, s_need, s_base[2];
  __shared__ uint32_t wsum[2][32];
  const int unit = blockIdx.x, b = unit / a.G, g = unit % a.G;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int L = c8_len(a.lens, b, a.T, a.status);
  const int m = min(L, a.keep);
  int32_t* kept = a.kept + (long)unit * a.keep;
  if (g == 0 && tid == 0) a.lens_out[b] = m;
  for (int i = m + tid; i < a.keep; i += kSelThr) kept[i] = -1;
  if (L <= a.keep) {
    for (int i = tid; i < L; i += kSelThr) kept[i] = i;
    return;
  }
  const int N = L - a.recent, c = a.keep - a.recent;
  for (int i = tid; i < a.recent; i += kSelThr) kept[c + i] = N + i;
  if (c == 0) return;
  const float* w = a.weight + (long)unit * a.T;
  if (tid == 0) {
    s_prefix = 0u;
    s_need = (uint32_t)c;
  }
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0u;
    __syncthreads();
    const uint32_t prefix = s_prefix, mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
    for (int i = tid; i < N; i += kSelThr) {
      const uint32_t k = weight_key(w[i]);
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (tid == 0) {
      uint32_t need = s_need;
      int x = 255;
      while (x > 0 && hist[x] < need) need -= hist[x--];
      s_need = need;
      s_prefix = prefix | ((uint32_t)x << shift);
    }
    __syncthreads();
  }
  const uint32_t thr = s_prefix, ties = s_need;
  if (tid < 2) s_base[tid] = 0u;
  __syncthreads();
  for (int i0 = 0; i0 < N; i0 += kSelThr) {
    const int i = i0 + tid;
    const uint32_t k = i < N ? weight_key(w[i]) : 0u;
    const bool gt = i < N && k > thr, eq = i < N && k == thr;
    const uint32_t bg = __ballot_sync(0xFFFFFFFFu, gt), be = __ballot_sync(0xFFFFFFFFu, eq);
    if (lane == 0) {
      wsum[0][warp] = __popc(bg);
      wsum[1][warp] = __popc(be);
    }
    __syncthreads();
    uint32_t ng = s_base[0], ne = s_base[1];
    for (int x = 0; x < warp; ++x) {
      ng += wsum[0][x];
      ne += wsum[1][x];
    }
    const uint32_t below = (1u << lane) - 1u;
    ng += __popc(bg & below);
    ne += __popc(be & below);
    if (gt || (eq && ne < ties)) kept[ng + min(ne, ties)] = i;
    __syncthreads();
    if (tid == kSelThr - 1) {
      s_base[0] = ng + (gt ? 1 : 0);
      s_base[1] = ne + (eq ? 1 : 0);
    }
    __syncthreads();
  }
}

constexpr int kThr = 256;

// Largest |code * scale| of 16 codes but for NaN, as fp32 bits.
__device__ __forceinline__ uint32_t amax16(const uint4& x, float scale) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t m = 0;  // the largest magnitude code that is no NaN
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t c = (w[i] >> (8 * j)) & 0x7Fu;
      if (c != 0x7Fu) m = max(m, c);
    }
  }
  return __float_as_uint(c8_decode2(m).x * scale);
}
__device__ __forceinline__ uint4 rescale16(const uint4& x, int k) {
  if (k == 0) return x;
  const float f = c8_shift(k);
  return make_uint4(c8_rescale4(x.x, f), c8_rescale4(x.y, f), c8_rescale4(x.z, f), c8_rescale4(x.w, f));
}

// One item per block of the new cache and group, rows as in the append kernel.
template <int D, int BLK>
__global__ void __launch_bounds__(kThr) cache8_move_kernel(C8EvictArgs a, int blocks_per_seq) {
  constexpr int kTpr = D / 16, kRows = kThr / kTpr;
  constexpr int kItems = kRows > BLK ? kRows / BLK : 1;
  constexpr int kPass = BLK > kRows ? BLK / kRows : 1;
  __shared__ uint32_t amax[kItems][2];
  const int tid = threadIdx.x;
  if (tid < kItems * 2) amax[tid / 2][tid & 1] = 0u;
  __syncthreads();
  const int sub = kItems > 1 ? (tid / kTpr) / BLK : 0;
  const int row0 = kItems > 1 ? (tid / kTpr) % BLK : tid / kTpr;
  const int col = (tid % kTpr) * 16;
  const long item = (long)blockIdx.x * kItems + sub;
  const long per_seq = (long)blocks_per_seq * a.G;
  const int b = (int)(item / per_seq), g = (int)(item % a.G), j = (int)((item % per_seq) / a.G);
  int m = 0;
  if (b < a.batch) m = min(c8_len(a.lens, b, a.T, a.status), a.keep);
  const long nblk = (a.T + BLK - 1) / BLK, nblk_out = (a.T_out + BLK - 1) / BLK;
  uint4 xk[kPass], xv[kPass];
  int ek[kPass], ev[kPass];
  uint32_t mk = 0, mv = 0;
#pragma unroll
  for (int p = 0; p < kPass; ++p) {
    const int i = j * BLK + row0 + p * kRows;
    xk[p] = xv[p] = make_uint4(0, 0, 0, 0);
    ek[p] = ev[p] = -126;
    if (i < m) {
      const int u = __ldg(a.kept + ((long)b * a.G + g) * a.keep + i);
      const long src = (((long)b * a.T + u) * a.G + g) * D + col;
      const long si = ((long)b * nblk + u / BLK) * a.G + g;
      xk[p] = __ldg(reinterpret_cast<const uint4*>(a.src.k8 + src));
      xv[p] = __ldg(reinterpret_cast<const uint4*>(a.src.v8 + src));
      ek[p] = c8_scale_exponent(__ldg(a.src.ks + si));
      ev[p] = c8_scale_exponent(__ldg(a.src.vs + si));
      if (col == 0) a.w_out[((long)b * a.G + g) * a.T_out + i] = __ldg(a.weight + ((long)b * a.G + g) * a.T + u);
    }
  }
#pragma unroll
  for (int p = 0; p < kPass; ++p) {
    mk = max(mk, amax16(xk[p], c8_pow2(ek[p])));
    mv = max(mv, amax16(xv[p], c8_pow2(ev[p])));
  }
  mk = __reduce_max_sync(0xFFFFFFFFu, mk);
  mv = __reduce_max_sync(0xFFFFFFFFu, mv);
  if ((tid & 31) == 0) {
    atomicMax(&amax[sub][0], mk);
    atomicMax(&amax[sub][1], mv);
  }
  __syncthreads();
  const int nk = c8_exponent(amax[sub][0]), nv = c8_exponent(amax[sub][1]);
#pragma unroll
  for (int p = 0; p < kPass; ++p) {
    const int i = j * BLK + row0 + p * kRows;
    if (i >= m) break;
    const long dst = (((long)b * a.T_out + i) * a.G + g) * D + col;
    *reinterpret_cast<uint4*>(a.dst.k8 + dst) = rescale16(xk[p], ek[p] - nk);
    *reinterpret_cast<uint4*>(a.dst.v8 + dst) = rescale16(xv[p], ev[p] - nv);
  }
  if (row0 == 0 && col == 0 && j * BLK < m) {
    const long so = ((long)b * nblk_out + j) * a.G + g;
    a.dst.ks[so] = c8_pow2(nk);
    a.dst.vs[so] = c8_pow2(nv);
  }
}

template <int D, int BLK>
cudaError_t launch_move(const C8EvictArgs& a, cudaStream_t s) {
  constexpr int kRows = kThr / (D / 16);
  constexpr int kItems = kRows > BLK ? kRows / BLK : 1;
  const int most = a.keep < a.T ? a.keep : a.T;  // tokens a sequence can keep
  const int per_seq = (most + BLK - 1) / BLK;
  const long ctas = ((long)a.batch * per_seq * a.G + kItems - 1) / kItems;
  if (ctas > 0x7FFFFFFFL) return cudaErrorInvalidConfiguration;
  cache8_move_kernel<D, BLK><<<(unsigned)ctas, kThr, 0, s>>>(a, per_seq);
  return cudaGetLastError();
}
template <int D>
cudaError_t launch_d(const C8EvictArgs& a, cudaStream_t s) {
  switch (a.block) {
    case 8: return launch_move<D, 8>(a, s);
    case 16: return launch_move<D, 16>(a, s);
    case 32: return launch_move<D, 32>(a, s);
    case 64: return launch_move<D, 64>(a, s);
    default: return launch_move<D, 128>(a, s);
  }
}

}  // namespace

cudaError_t launch_cache8_evict(const C8EvictArgs& a, cudaStream_t s) {
  cache8_keep_kernel<<<(unsigned)(a.batch * a.G), kSelThr, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return a.d == 64 ? launch_d<64>(a, s) : launch_d<128>(a, s);
}

}  // namespace sgqa
