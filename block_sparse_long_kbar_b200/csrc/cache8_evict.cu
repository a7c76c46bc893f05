// Eviction from the block-scaled 8-bit KV cache (format: cache8.cuh) by accumulated attention
// weight: which tokens stay, and their move to another cache.
#include <cooperative_groups.h>

#include "cache8.cuh"

namespace cg = cooperative_groups;

namespace sgqa {
namespace {

constexpr int kSelThr = 1024;
constexpr int kSelVec = 4;                       // 16-byte loads a lane keeps in flight (or in registers)
constexpr int kSelWarp = kSelVec * 32;           // and a warp: 512 weights
constexpr int kSelCta = kSelWarp * 4 * 32;       // weights a CTA can hold in registers: 16384

// Order-preserving key of a weight; NaN ranks as -infinity. No weight's key is 0.
__device__ __forceinline__ uint32_t weight_key(float w) { return score_key(w != w ? -INFINITY : w); }

// Sum of x over the block's threads before this one; *all: over all.
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* buf, uint32_t* all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t y = x;
#pragma unroll
  for (int h = 1; h < 32; h <<= 1) {
    const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, y, h);
    if (lane >= h) y += v;
  }
  if (lane == 31) buf[warp] = y;
  __syncthreads();
  uint32_t v = buf[lane], z = v;
#pragma unroll
  for (int h = 1; h < 32; h <<= 1) {
    const uint32_t q = __shfl_up_sync(0xFFFFFFFFu, z, h);
    if (lane >= h) z += q;
  }
  *all = __shfl_sync(0xFFFFFFFFu, z, 31);
  const uint32_t before = __shfl_sync(0xFFFFFFFFu, z - v, warp);
  __syncthreads();
  return before + y - x;
}

// Of more than `keep` tokens the `recent` last stay, and of the N before them the c = keep - recent
// heaviest: a radix select (11, 11 and 10 bits) finds the key of the c-th heaviest and how many of its
// equals stay, the lowest positions first; an ordered pass writes the positions. A cluster of CTAs
// serves one (sequence, group): each histograms its part of the weights (a contiguous range, split
// into one per warp) in its own shared memory and adds up the others' over distributed shared memory.
// REG: a part fits the CTA's registers and is read once; else it is read in every pass (from L2).
template <bool REG>
__global__ void __launch_bounds__(kSelThr) cache8_keep_kernel(C8EvictArgs a) {
  __shared__ alignas(16) uint32_t hist[3][2048];
  __shared__ uint32_t buf[32], s_bin, s_need, s_count[2];
  const cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
  const int unit = blockIdx.x / ctas, b = unit / a.G, g = unit % a.G;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int L = c8_len(a.lens, b, a.T, a.status);
  const int m = min(L, a.keep);
  int32_t* kept = a.kept + (long)unit * a.keep;
  const int t = rank * kSelThr + tid, step = ctas * kSelThr;
  if (g == 0 && t == 0) a.lens_out[b] = m;
  for (int i = m + t; i < a.keep; i += step) kept[i] = -1;
  if (L <= a.keep) {
    for (int i = t; i < L; i += step) kept[i] = i;
    return;
  }
  const int N = L - a.recent, c = a.keep - a.recent;
  for (int i = t; i < a.recent; i += step) kept[c + i] = N + i;
  if (c == 0) return;
  // 16-byte aligned vectors: vector v holds weights 4 v - off ..
  const long w0 = (long)unit * a.T;
  const int off = (int)(w0 & 3);
  const float* w = a.weight + (w0 - off);
  const int nv = (N + off + 3) / 4, per_cta = (nv + ctas - 1) / ctas, per_warp = (per_cta + 31) / 32;
  const int end_cta = min(nv, (rank + 1) * per_cta), v0 = rank * per_cta + warp * per_warp;
  const int v1 = min(end_cta, v0 + per_warp);
  uint32_t key[kSelVec][4];
  auto load = [&](int base) {  // keys of this lane's vectors; 0 where there is no weight
#pragma unroll
    for (int s = 0; s < kSelVec; ++s) {
      const int v = base + s * 32 + lane, e = 4 * v - off;
      if (v < v1 && e >= 0 && e + 3 < N) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(w) + v);
        key[s][0] = weight_key(x.x);
        key[s][1] = weight_key(x.y);
        key[s][2] = weight_key(x.z);
        key[s][3] = weight_key(x.w);
      } else {
#pragma unroll
        for (int x = 0; x < 4; ++x)
          key[s][x] = v < v1 && e + x >= 0 && e + x < N ? weight_key(__ldg(w + 4L * v + x)) : 0u;
      }
    }
  };
  if (REG) load(v0);
  for (int i = tid; i < 3 * 2048; i += kSelThr) hist[0][i] = 0u;
  __syncthreads();
  uint32_t prefix = 0u, need = (uint32_t)c;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t mask = pass == 0 ? 0u : pass == 1 ? 0xFFE00000u : 0xFFFFFC00u, digit = pass == 2 ? 1023u : 2047u;
    for (int base = v0; base < v1; base += kSelWarp) {
      if (!REG) load(base);
#pragma unroll
      for (int s = 0; s < kSelVec; ++s)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (key[s][x] && (key[s][x] & mask) == prefix) atomicAdd(&hist[pass][(key[s][x] >> shift) & digit], 1u);
      if (REG) break;
    }
    cluster.sync();
    // bins from the top: the one that holds the need-th
    uint32_t n0 = 0u, n1 = 0u;
    for (int r = 0; r < ctas; ++r) {
      const uint2 h = *cluster.map_shared_rank(reinterpret_cast<uint2*>(&hist[pass][2046 - 2 * tid]), r);
      n0 += h.y;
      n1 += h.x;
    }
    uint32_t all;
    const uint32_t before = block_scan(n0 + n1, buf, &all);
    if (before < need && need <= before + n0 + n1) {
      const bool second = need > before + n0;
      s_bin = 2047u - 2u * tid - (second ? 1u : 0u);
      s_need = need - before - (second ? n0 : 0u);
    }
    __syncthreads();
    prefix |= s_bin << shift;
    need = s_need;
  }
  const uint32_t thr = prefix, ties = need;
  // heavier ones and equals in this warp, this CTA's warps before it, the CTAs before this one
  uint32_t gt = 0u, eq = 0u;
  for (int base = v0; base < v1; base += kSelWarp) {
    if (!REG) load(base);
#pragma unroll
    for (int s = 0; s < kSelVec; ++s)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        gt += key[s][x] > thr ? 1u : 0u;
        eq += key[s][x] == thr ? 1u : 0u;
      }
    if (REG) break;
  }
  gt = __reduce_add_sync(0xFFFFFFFFu, gt);
  eq = __reduce_add_sync(0xFFFFFFFFu, eq);
  uint32_t all_gt, all_eq;
  uint32_t ng = block_scan(lane == 0 ? gt : 0u, buf, &all_gt), ne = block_scan(lane == 0 ? eq : 0u, buf, &all_eq);
  ng = __shfl_sync(0xFFFFFFFFu, ng, 0);
  ne = __shfl_sync(0xFFFFFFFFu, ne, 0);
  if (tid == 0) {
    s_count[0] = all_gt;
    s_count[1] = all_eq;
  }
  cluster.sync();
  for (int r = 0; r < rank; ++r) {
    const uint32_t* x = cluster.map_shared_rank(&s_count[0], r);
    ng += x[0];
    ne += x[1];
  }
  const uint32_t below = (1u << lane) - 1u;
  for (int base = v0; base < v1; base += kSelWarp) {
    if (!REG) load(base);
#pragma unroll
    for (int s = 0; s < kSelVec; ++s) {
      uint32_t lg = 0u, le = 0u, ag = 0u, ae = 0u;  // in the lanes below, in all lanes
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const uint32_t bg = __ballot_sync(0xFFFFFFFFu, key[s][x] > thr);
        const uint32_t be = __ballot_sync(0xFFFFFFFFu, key[s][x] == thr);
        lg += __popc(bg & below);
        le += __popc(be & below);
        ag += __popc(bg);
        ae += __popc(be);
      }
      uint32_t pg = ng + lg, pe = ne + le;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const bool is_gt = key[s][x] > thr, is_eq = key[s][x] == thr;
        if (is_gt || (is_eq && pe < ties)) kept[pg + min(pe, ties)] = 4 * (base + s * 32 + lane) - off + x;
        pg += is_gt ? 1u : 0u;
        pe += is_eq ? 1u : 0u;
      }
      ng += ag;
      ne += ae;
    }
    if (REG) break;
  }
  cluster.sync();  // no CTA leaves while another reads its shared memory
}

constexpr int kThr = 256;

// Largest |code * scale| of 16 codes but for NaN, as fp32 bits.
__device__ __forceinline__ uint32_t amax16(const uint4& x, float scale) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t m = 0;  // the largest magnitude code that is no NaN
#pragma unroll
  for (int i = 0; i < 4; ++i) m = c8_max_u16x2(m, c8_max_u16x2(w[i] & 0x007F007Fu, (w[i] >> 8) & 0x007F007Fu));
  m = max(m & 0xFFFFu, m >> 16);
  if (m == 0x7Fu) {
    m = 0;
    for (int i = 0; i < 16; ++i) {
      const uint32_t c = (w[i >> 2] >> (8 * (i & 3))) & 0x7Fu;
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

// One item per block of the new cache and group, rows and items as in the append kernel. HBM bound: a
// kept row is read and written once.
constexpr int kLoop = 8;
template <int D, int BLK>
__global__ void __launch_bounds__(kThr) cache8_move_kernel(C8EvictArgs a, int loop) {
  constexpr int kTpr = D / 16, kRows = kThr / kTpr;
  constexpr int kItems = kRows > BLK ? kRows / BLK : 1;
  constexpr int kPass = BLK > kRows ? BLK / kRows : 1;
  __shared__ uint32_t amax[kLoop][kItems][2];
  const int tid = threadIdx.x, b = blockIdx.y;
  const int m = min(c8_len(a.lens, b, a.T, a.status), a.keep);
  const int first = (int)blockIdx.x * loop * kItems;
  if (first / a.G * BLK >= m) return;
  for (int i = tid; i < kLoop * kItems * 2; i += kThr) (&amax[0][0][0])[i] = 0u;
  __syncthreads();
  const int sub = kItems > 1 ? (tid / kTpr) / BLK : 0;
  const int row0 = kItems > 1 ? (tid / kTpr) % BLK : tid / kTpr;
  const int col = (tid % kTpr) * 16;
  const int nblk = (a.T + BLK - 1) / BLK, nblk_out = (a.T_out + BLK - 1) / BLK;
  int j = (first + sub) / a.G, g = (first + sub) % a.G;
  for (int it = 0; it < loop; ++it) {
    uint4 xk[kPass], xv[kPass];
    int ek[kPass], ev[kPass], u[kPass];
    uint32_t mk = 0, mv = 0;
    const int i0 = j * BLK + row0;
#pragma unroll
    for (int p = 0; p < kPass; ++p)
      u[p] = i0 + p * kRows < m ? __ldg(a.kept + (long)(b * a.G + g) * a.keep + i0 + p * kRows) : -1;
#pragma unroll
    for (int p = 0; p < kPass; ++p) {
      xk[p] = xv[p] = make_uint4(0, 0, 0, 0);
      ek[p] = ev[p] = -126;
      if (u[p] >= 0) {
        const long src = (long)((b * a.T + u[p]) * a.G + g) * D + col;
        const long si = (long)(b * nblk + u[p] / BLK) * a.G + g;
        xk[p] = __ldg(reinterpret_cast<const uint4*>(a.src.k8 + src));
        xv[p] = __ldg(reinterpret_cast<const uint4*>(a.src.v8 + src));
        ek[p] = c8_scale_exponent(__ldg(a.src.ks + si));
        ev[p] = c8_scale_exponent(__ldg(a.src.vs + si));
      }
    }
    if (col == 0) {
#pragma unroll
      for (int p = 0; p < kPass; ++p)
        if (u[p] >= 0)
          a.w_out[(long)(b * a.G + g) * a.T_out + i0 + p * kRows] = __ldg(a.weight + (long)(b * a.G + g) * a.T + u[p]);
    }
#pragma unroll
    for (int p = 0; p < kPass; ++p) {
      mk = max(mk, amax16(xk[p], c8_pow2(ek[p])));
      mv = max(mv, amax16(xv[p], c8_pow2(ev[p])));
    }
    mk = __reduce_max_sync(0xFFFFFFFFu, mk);
    mv = __reduce_max_sync(0xFFFFFFFFu, mv);
    if ((tid & 31) == 0) {
      atomicMax(&amax[it][sub][0], mk);
      atomicMax(&amax[it][sub][1], mv);
    }
    __syncthreads();
    const int nk = c8_exponent(amax[it][sub][0]), nv = c8_exponent(amax[it][sub][1]);
#pragma unroll
    for (int p = 0; p < kPass; ++p) {
      if (u[p] < 0) break;
      const long dst = (long)((b * a.T_out + i0 + p * kRows) * a.G + g) * D + col;
      *reinterpret_cast<uint4*>(a.dst.k8 + dst) = rescale16(xk[p], ek[p] - nk);
      *reinterpret_cast<uint4*>(a.dst.v8 + dst) = rescale16(xv[p], ev[p] - nv);
    }
    if (row0 == 0 && col == 0 && u[0] >= 0) {
      const long so = (long)(b * nblk_out + j) * a.G + g;
      a.dst.ks[so] = c8_pow2(nk);
      a.dst.vs[so] = c8_pow2(nv);
    }
    for (g += kItems; g >= a.G; g -= a.G) ++j;
  }
}

template <int D, int BLK>
cudaError_t launch_move(const C8EvictArgs& a, cudaStream_t s) {
  constexpr int kRows = kThr / (D / 16);
  constexpr int kItems = kRows > BLK ? kRows / BLK : 1;
  const int most = a.keep < a.T ? a.keep : a.T;  // tokens a sequence can keep
  const long items = (long)((most + BLK - 1) / BLK) * a.G;  // of a sequence; T * G is below 2^31
  const long groups = (items + kItems - 1) / kItems, full = groups * a.batch / (148 * 6 * 4);
  const int loop = (int)(full < 1 ? 1 : full > kLoop ? kLoop : full);
  cache8_move_kernel<D, BLK><<<dim3((unsigned)((groups + loop - 1) / loop), (unsigned)a.batch), kThr, 0, s>>>(
      a, loop);
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

// A part that starts and ends inside a vector still fits the registers of ctas CTAs.
bool keep_fits(int T, int ctas) { return (long)T + 6 <= (long)kSelCta * ctas; }
// CTAs per (sequence, group): as few as hold its weights in registers, up to a cluster's 8, and more
// while that leaves SMs without a CTA and a part 2048 weights or more.
int keep_ctas(long units, int T) {
  int c = 1;
  while (c < 8 && (!keep_fits(T, c) || (units * c * 2 <= 148 && T >= c * 2 * 2048))) c *= 2;
  return c;
}
template <bool REG>
cudaError_t launch_keep(const C8EvictArgs& a, int ctas, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)ctas;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)(a.batch * a.G * ctas));
  cfg.blockDim = dim3(kSelThr);
  cfg.stream = s;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache8_keep_kernel<REG>, a);
}

}  // namespace

cudaError_t launch_cache8_evict(const C8EvictArgs& a, cudaStream_t s) {
  const int ctas = keep_ctas((long)a.batch * a.G, a.T);
  const cudaError_t e = keep_fits(a.T, ctas) ? launch_keep<true>(a, ctas, s) : launch_keep<false>(a, ctas, s);
  if (e != cudaSuccess) return e;
  return a.d == 64 ? launch_d<64>(a, s) : launch_d<128>(a, s);
}

}  // namespace sgqa
