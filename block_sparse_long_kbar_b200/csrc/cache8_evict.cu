// Eviction from the block-scaled 8-bit KV cache (format: cache8.cuh) by accumulated attention
// weight: which tokens stay, and their move to another cache.
// Bytes: a weight per token and group once, a kept row of K and of V read and written once. Measured: 32
// sequences of 8K tokens to 4K (277 MB) 59 us on the device, of which the selection 13 us and the move 47
// us = 5.8 TB/s (rows of 128 bytes, a random half of them); 1M tokens to 131072 (289 MB) 85 us, of which
// the selection 38 us (five launches over 16 MB of weights, each a chain of load, scan and count) and
// the move 48 us.
#include <cooperative_groups.h>

#include "cache8.cuh"
#include "clusters.h"

namespace cg = cooperative_groups;

namespace sgqa {
namespace {

constexpr int kSelThr = 512;           // (1024: 11.1 instead of 9.7 us for 3 sequences of 777, no less for 8K)
constexpr int kSelPart = 4 * kSelThr;  // weights of a CTA per 16-byte load of its threads

// Words of global memory that the selection over the whole GPU has per unit.
__device__ __host__ constexpr long keep_grid_words(int ctas) { return 3 * 2048 + 8 + 2L * ((ctas + 1) & ~1); }

// Order-preserving key of a weight: -0 as +0, NaN as -infinity. No weight's key is 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  const float x = w + 0.f;
  const int u = __float_as_int(x);
  const uint32_t k = (uint32_t)(u ^ ((u >> 31) | (int)0x80000000));
  return x == x ? k : 0x007FFFFFu;
}

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
  const uint32_t v = lane < (int)(blockDim.x >> 5) ? buf[lane] : 0u;
  uint32_t z = v;
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

// The weights of one (sequence, group) that compete, and the part of them that one warp takes: 16-byte
// aligned vectors v0 .. v1 - 1, vector v holding weights 4 v - off ..; VEC vectors of a lane at a time.
template <int VEC>
struct Part {
  const float* w;
  int off, N, v0, v1;
  int w0, w1;  // vectors all of whose weights compete: [w0, w1)
  uint32_t key[VEC][4];
  float4 ahead[VEC];
  __device__ __forceinline__ void set(const C8EvictArgs& a, int unit, int n, int ctas, int rank, int warps) {
    const long at = (long)unit * a.T;
    off = (int)(at & 3);
    w = a.weight + (at - off);
    N = n;
    const int nv = (N + off + 3) / 4, per_cta = (nv + ctas - 1) / ctas, per_warp = (per_cta + warps - 1) / warps;
    v0 = rank * per_cta + (int)(threadIdx.x >> 5) * per_warp;
    v1 = min(min(nv, (rank + 1) * per_cta), v0 + per_warp);
    w0 = off ? 1 : 0;
    w1 = min(v1, (N + off) >> 2);
  }
  __device__ __forceinline__ void fetch(int base) {
    const int v = base + (int)(threadIdx.x & 31);
    const float4* p = reinterpret_cast<const float4*>(w) + v;
#pragma unroll
    for (int s = 0; s < VEC; ++s)
      if (v + s * 32 >= w0 && v + s * 32 < w1) ahead[s] = __ldg(p + s * 32);
  }
  __device__ __forceinline__ void keys(int base) {  // 0 where there is no weight
    const int v = base + (int)(threadIdx.x & 31);
#pragma unroll
    for (int s = 0; s < VEC; ++s) {
      const bool whole = v + s * 32 >= w0 && v + s * 32 < w1;
      key[s][0] = whole ? weight_key(ahead[s].x) : 0u;
      key[s][1] = whole ? weight_key(ahead[s].y) : 0u;
      key[s][2] = whole ? weight_key(ahead[s].z) : 0u;
      key[s][3] = whole ? weight_key(ahead[s].w) : 0u;
    }
    if (base < w0 || w1 < min(v1, base + VEC * 32)) {  // the unit's first or last vector, in part
#pragma unroll
      for (int s = 0; s < VEC; ++s) {
        const int y = v + s * 32;
        if (y < v1 && (y < w0 || y >= w1))
          for (int x = 0; x < 4; ++x) {
            const int e = 4 * y - off + x;
            const uint32_t k = e >= 0 && e < N ? weight_key(__ldg(w + 4L * y + x)) : 0u;
            if (x == 0) key[s][0] = k;
            else if (x == 1) key[s][1] = k;
            else if (x == 2) key[s][2] = k;
            else key[s][3] = k;
          }
      }
    }
  }
  __device__ __forceinline__ void count(uint32_t* hist, int pass, uint32_t prefix) const {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t mask = pass == 0 ? 0u : pass == 1 ? 0xFFE00000u : 0xFFFFFC00u, digit = pass == 2 ? 1023u : 2047u;
#pragma unroll
    for (int s = 0; s < VEC; ++s)
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (key[s][x] && (key[s][x] & mask) == prefix) atomicAdd(&hist[(key[s][x] >> shift) & digit], 1u);
  }
  __device__ __forceinline__ void above(uint32_t thr, uint32_t& gt, uint32_t& eq) const {
#pragma unroll
    for (int s = 0; s < VEC; ++s)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        gt += key[s][x] > thr ? 1u : 0u;
        eq += key[s][x] == thr ? 1u : 0u;
      }
  }
  // ng0 heavier ones and ne0 equals precede these vectors. A lane's counts in two vectors, heavier and
  // equal, are four bytes of a word (a warp has at most 128 of each), so that one scan over the lanes
  // serves both.
  __device__ __forceinline__ void emit(const C8EvictArgs& a, int base, uint32_t thr, uint32_t ties, uint32_t ng0,
                                       uint32_t ne0, int32_t* kept, uint32_t* ng_out = nullptr, uint32_t* ne_out = nullptr) const {
    const int lane = threadIdx.x & 31;
    uint32_t ng = ng0, ne = ne0;
#pragma unroll
    for (int s0 = 0; s0 < VEC; s0 += 2) {
      uint32_t own = 0u;
#pragma unroll
      for (int s = s0; s < min(VEC, s0 + 2); ++s)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t one = 1u << (16 * (s - s0));
          own += key[s][x] > thr ? one : 0u;
          own += key[s][x] == thr ? one << 8 : 0u;
        }
      uint32_t upto = own;
#pragma unroll
      for (int h = 1; h < 32; h <<= 1) {
        const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, upto, h);
        if (lane >= h) upto += y;
      }
      const uint32_t all = __shfl_sync(0xFFFFFFFFu, upto, 31), before = upto - own;
#pragma unroll
      for (int s = s0; s < min(VEC, s0 + 2); ++s) {
        const int sh = 16 * (s - s0);
        uint32_t pg = ng + (before >> sh & 255u), pe = ne + (before >> (sh + 8) & 255u);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const bool is_gt = key[s][x] > thr, is_eq = key[s][x] == thr;
          if ((is_gt || (is_eq && pe < ties)) &&
              SGQA_CHECK(pg + min(pe, ties) < (uint32_t)(a.keep - a.recent), a.status))
            kept[pg + min(pe, ties)] = 4 * (base + s * 32 + lane) - off + x;
          pg += is_gt ? 1u : 0u;
          pe += is_eq ? 1u : 0u;
        }
        ng += all >> sh & 255u;
        ne += all >> (sh + 8) & 255u;
      }
    }
    if (ng_out) {
      *ng_out = ng;
      *ne_out = ne;
    }
  }
};

// Thread t of 2048 / BINS holds the counts n[] of bins 2047 - BINS t and below: extends the prefix by
// the bin of the need-th heaviest, and counts need from the top of that bin.
template <int BINS>
__device__ __forceinline__ void find_bin(const uint32_t (&n)[BINS], int pass, uint32_t& prefix, uint32_t& need,
                                         uint32_t* buf, uint32_t* found) {
  uint32_t sum = 0u, all;
#pragma unroll
  for (int i = 0; i < BINS; ++i) sum += n[i];
  uint32_t before = block_scan(sum, buf, &all);
  if (before < need && need <= before + sum) {
#pragma unroll
    for (int i = 0; i < BINS; ++i) {
      if (before < need && need <= before + n[i]) {
        found[0] = 2047u - BINS * threadIdx.x - i;
        found[1] = need - before;
      }
      before += n[i];
    }
  }
  __syncthreads();
  prefix |= found[0] << (pass == 0 ? 21 : pass == 1 ? 10 : 0);
  need = found[1];
}

// What needs no selection: thread t of n writes its share. True if there is nothing more to do.
__device__ __forceinline__ bool keep_simple(const C8EvictArgs& a, int unit, int L, int t, int n) {
  const int m = min(L, a.keep), c = a.keep - a.recent;
  int32_t* kept = a.kept + (long)unit * a.keep;
  if (unit % a.G == 0 && t == 0) a.lens_out[unit / a.G] = m;
  for (int i = m + t; i < a.keep; i += n) kept[i] = -1;
  if (L <= a.keep) {
    for (int i = t; i < L; i += n) kept[i] = i;
    return true;
  }
  for (int i = t; i < a.recent; i += n) kept[c + i] = L - a.recent + i;
  return c == 0;
}

// Of more than `keep` tokens the `recent` last stay, and of the N before them the c = keep - recent
// heaviest: a radix select (11, 11 and 10 bits) finds the key of the c-th heaviest and how many of its
// equals stay, the lowest positions first; an ordered pass writes the positions. A cluster of CTAs
// serves one (sequence, group): each histograms its part of the weights (a contiguous range, split
// into one per warp) in its own shared memory and adds up the others' over distributed shared memory.
// REG: a part fits the CTA's registers, VEC 16-byte loads a lane, and is read once; else it is read in
// every pass (from L2), the next loads under way while the present ones are counted.
template <int VEC, bool REG>
__global__ void __launch_bounds__(kSelThr) cache8_keep_kernel(C8EvictArgs a) {
  __shared__ alignas(16) uint32_t hist[3][2048];
  __shared__ uint32_t buf[32], found[2], s_count[2];
  const cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
  const int unit = blockIdx.x / ctas, tid = threadIdx.x, lane = tid & 31;
  grid_dependents();
  const int L = c8_len(a.lens, unit / a.G, a.T, a.status);
  if (keep_simple(a, unit, L, rank * kSelThr + tid, ctas * kSelThr)) return;
  Part<VEC> part;
  part.set(a, unit, L - a.recent, ctas, rank, kSelThr / 32);
  // a pass over the part: take(base) with the keys of vectors base ..
  auto pass_over = [&](auto&& take) {
    if (REG) {
      take(part.v0);
    } else {
      part.fetch(part.v0);
      for (int base = part.v0; base < part.v1; base += VEC * 32) {
        part.keys(base);
        if (base + VEC * 32 < part.v1) part.fetch(base + VEC * 32);
        take(base);
      }
    }
  };
  if (REG) part.fetch(part.v0);
  for (int i = tid; i < 3 * 2048; i += kSelThr) hist[0][i] = 0u;
  if (REG) part.keys(part.v0);
  __syncthreads();
  uint32_t prefix = 0u, need = (uint32_t)(a.keep - a.recent);
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    pass_over([&](int) { part.count(hist[pass], pass, prefix); });
    cluster.sync();
    uint32_t bins[4] = {0u, 0u, 0u, 0u};
    for (int r = 0; r < ctas; ++r) {
      const uint4 h = *cluster.map_shared_rank(reinterpret_cast<uint4*>(&hist[pass][2044 - 4 * tid]), r);
      bins[0] += h.w;
      bins[1] += h.z;
      bins[2] += h.y;
      bins[3] += h.x;
    }
    find_bin(bins, pass, prefix, need, buf, found);
  }
  // heavier ones and equals in this warp, this CTA's warps before it, the CTAs before this one
  uint32_t gt = 0u, eq = 0u;
  pass_over([&](int) { part.above(prefix, gt, eq); });
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
  int32_t* kept = a.kept + (long)unit * a.keep;
  pass_over([&](int base) { part.emit(a, base, prefix, need, ng, ne, kept, &ng, &ne); });
  cluster.sync();  // no CTA leaves while another reads its shared memory
}

// The same selection for few (sequence, group)s of very many weights, which need the whole GPU: a part
// of 16384 weights per CTA, and a launch per pass (STEP 0 to 2: histograms, added up in global memory;
// 3: counts of every part; 4: positions). The weights come from L2 after the first pass, and are read
// while the launch before ends.
// Global memory, per unit: 3 histograms, (prefix, need) after each, (heavier, equal) of every part.
constexpr int kGridThr = 512, kGridVec = 8;
template <int STEP>
__global__ void __launch_bounds__(kGridThr, 2) cache8_keep_grid_kernel(C8EvictArgs a) {
  __shared__ alignas(16) uint32_t hist[STEP < 3 ? 2048 : 2];
  __shared__ uint32_t buf[32], found[2];
  const int unit = blockIdx.y, rank = blockIdx.x, ctas = gridDim.x, tid = threadIdx.x, lane = tid & 31;
  grid_dependents();
  const int L = c8_len(a.lens, unit / a.G, a.T, a.status);
  if (STEP == 0) {
    grid_wait();
    if (keep_simple(a, unit, L, rank * kGridThr + tid, ctas * kGridThr)) return;
  } else if (L <= a.keep || a.keep == a.recent) {
    grid_wait();  // (no kernel ends before the one it was started behind)
    return;
  }
  uint32_t* g = a.grid_ws + (long)unit * keep_grid_words(ctas);
  uint32_t* state = g + 3 * 2048;  // [3][2]
  uint2* counts = reinterpret_cast<uint2*>(state + 8);
  Part<kGridVec> part;
  part.set(a, unit, L - a.recent, ctas, rank, kGridThr / 32);
  part.fetch(part.v0);
  uint32_t prefix = 0u, need = (uint32_t)(a.keep - a.recent);
  if (STEP < 3)
    for (int i = tid; i < 2048; i += kGridThr) hist[i] = 0u;
  part.keys(part.v0);
  if (STEP > 0) grid_wait();
  if (STEP > 1) {
    prefix = state[2 * (min(STEP, 4) - 2)];
    need = state[2 * (min(STEP, 4) - 2) + 1];
  }
  if (STEP > 0 && STEP < 4) {
    const uint4 h = *reinterpret_cast<const uint4*>(g + (STEP - 1) * 2048 + 2044 - 4 * tid);
    const uint32_t bins[4] = {h.w, h.z, h.y, h.x};
    find_bin(bins, STEP - 1, prefix, need, buf, found);
    if (rank == 0 && tid == 0) {
      state[2 * (STEP - 1)] = prefix;
      state[2 * (STEP - 1) + 1] = need;
    }
  } else {
    __syncthreads();
  }
  if constexpr (STEP < 3) {
    part.count(hist, STEP, prefix);
    __syncthreads();
    for (int i = tid; i < 2048; i += kGridThr)
      if (hist[i]) atomicAdd(g + STEP * 2048 + i, hist[i]);
  } else {
    uint32_t gt = 0u, eq = 0u, all_gt, all_eq;
    part.above(prefix, gt, eq);
    gt = __reduce_add_sync(0xFFFFFFFFu, gt);
    eq = __reduce_add_sync(0xFFFFFFFFu, eq);
    uint32_t ng = block_scan(lane == 0 ? gt : 0u, buf, &all_gt), ne = block_scan(lane == 0 ? eq : 0u, buf, &all_eq);
    if constexpr (STEP == 3) {
      if (tid == 0) counts[rank] = make_uint2(all_gt, all_eq);
    } else {
      ng = __shfl_sync(0xFFFFFFFFu, ng, 0);
      ne = __shfl_sync(0xFFFFFFFFu, ne, 0);
      uint32_t bg = 0u, be = 0u, before_g, before_e;
      for (int r = tid; r < rank; r += kGridThr) {
        const uint2 x = counts[r];
        bg += x.x;
        be += x.y;
      }
      block_scan(bg, buf, &before_g);
      block_scan(be, buf, &before_e);
      part.emit(a, part.v0, prefix, need, ng + before_g, ne + before_e, a.kept + (long)unit * a.keep);
    }
  }
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
// One item per block of the new cache and group, rows and items as in the append kernel. HBM bound: a
// kept row is read and written once (with streaming stores 32 sequences of 8K take 59 us on the device instead of
// 63, of which the write-back of ordinary ones took the difference).
constexpr int kLoop = 8;
template <int D, int BLK>
__global__ void __launch_bounds__(kThr, BLK * D == 128 * 128 ? 4 : 0) cache8_move_kernel(C8EvictArgs a, int loop) {
  constexpr int kTpr = D / 16, kRows = kThr / kTpr;
  constexpr int kItems = kRows > BLK ? kRows / BLK : 1;
  constexpr int kPass = BLK > kRows ? BLK / kRows : 1;
  constexpr int kSide = kPass == 1 ? 2 : 1;
  __shared__ uint32_t amax[kLoop + 1][kItems][2];
  const int tid = threadIdx.x, b = blockIdx.y;
  grid_dependents();
  const int m = min(c8_len(a.lens, b, a.T, a.status), a.keep);
  const int first = (int)blockIdx.x * loop * kItems;
  for (int i = tid; i < (kLoop + 1) * kItems * 2; i += kThr) (&amax[0][0][0])[i] = 0u;
  grid_wait();
  if (first / a.G * BLK >= m) return;
  __syncthreads();
  const int sub = kItems > 1 ? (tid / kTpr) / BLK : 0;
  const int row0 = kItems > 1 ? (tid / kTpr) % BLK : tid / kTpr;
  const int col = (tid % kTpr) * 16;
  const int nblk = (a.T + BLK - 1) / BLK, nblk_out = (a.T_out + BLK - 1) / BLK;
  // kSide items side by side, so that every thread has several rows under way, and their positions one
  // step ahead
  struct Item {
    int j, g, u[kPass];
    uint4 xk[kPass], xv[kPass];
    int ek[kPass], ev[kPass];
  };
  auto positions = [&](Item& x, bool there) {
#pragma unroll
    for (int p = 0; p < kPass; ++p) {
      const int i = x.j * BLK + row0 + p * kRows;
      // (a plain load: written by the kernel before, whose end is waited for in this one)
      x.u[p] = there && i < m ? a.kept[(long)(b * a.G + x.g) * a.keep + i] : -1;
      if (!SGQA_CHECK(!(there && i < m) || (x.u[p] >= 0 && x.u[p] < a.T && i < a.T_out && x.j < nblk_out), a.status))
        x.u[p] = -1;
    }
  };
  auto step = [&](Item& x) {
    for (x.g += kItems * kSide; x.g >= a.G; x.g -= a.G) ++x.j;
  };
  Item x[kSide], y[kSide];
#pragma unroll
  for (int q = 0; q < kSide; ++q) {
    x[q].j = (first + sub + q * kItems) / a.G;
    x[q].g = (first + sub + q * kItems) % a.G;
    positions(x[q], q < loop);
  }
  for (int it = 0; it < loop; it += kSide) {
#pragma unroll
    for (int q = 0; q < kSide; ++q) {
      Item& z = x[q];
#pragma unroll
      for (int p = 0; p < kPass; ++p) {
        z.xk[p] = z.xv[p] = make_uint4(0, 0, 0, 0);
        z.ek[p] = z.ev[p] = -126;
        if (z.u[p] >= 0) {
          const long src = (long)((b * a.T + z.u[p]) * a.G + z.g) * D + col;
          const long si = (long)(b * nblk + z.u[p] / BLK) * a.G + z.g;
          z.xk[p] = __ldcs(reinterpret_cast<const uint4*>(a.src.k8 + src));
          z.xv[p] = __ldcs(reinterpret_cast<const uint4*>(a.src.v8 + src));
          z.ek[p] = c8_scale_exponent(__ldg(a.src.ks + si));
          z.ev[p] = c8_scale_exponent(__ldg(a.src.vs + si));
        }
      }
      y[q].j = z.j;
      y[q].g = z.g;
      step(y[q]);
      positions(y[q], it + kSide + q < loop);
    }
    if (col == 0) {
#pragma unroll
      for (int q = 0; q < kSide; ++q)
#pragma unroll
        for (int p = 0; p < kPass; ++p)
          if (x[q].u[p] >= 0)
            a.w_out[(long)(b * a.G + x[q].g) * a.T_out + x[q].j * BLK + row0 + p * kRows] =
                __ldg(a.weight + (long)(b * a.G + x[q].g) * a.T + x[q].u[p]);
    }
#pragma unroll
    for (int q = 0; q < kSide; ++q) {
      uint32_t mk = 0, mv = 0;
#pragma unroll
      for (int p = 0; p < kPass; ++p) {
        mk = max(mk, amax16(x[q].xk[p], c8_pow2(x[q].ek[p])));
        mv = max(mv, amax16(x[q].xv[p], c8_pow2(x[q].ev[p])));
      }
      mk = __reduce_max_sync(0xFFFFFFFFu, mk);
      mv = __reduce_max_sync(0xFFFFFFFFu, mv);
      if ((tid & 31) == 0) {
        atomicMax(&amax[it + q][sub][0], mk);
        atomicMax(&amax[it + q][sub][1], mv);
      }
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kSide; ++q) {
      const Item& z = x[q];
      const int nk = c8_exponent(amax[it + q][sub][0]), nv = c8_exponent(amax[it + q][sub][1]);
#pragma unroll
      for (int p = 0; p < kPass; ++p) {
        if (z.u[p] < 0) break;
        const long dst = (long)((b * a.T_out + z.j * BLK + row0 + p * kRows) * a.G + z.g) * D + col;
        __stcs(reinterpret_cast<uint4*>(a.dst.k8 + dst), c8_rescale16(z.xk[p], z.ek[p] - nk));
        __stcs(reinterpret_cast<uint4*>(a.dst.v8 + dst), c8_rescale16(z.xv[p], z.ev[p] - nv));
      }
      if (row0 == 0 && col == 0 && z.u[0] >= 0) {
        const long so = (long)(b * nblk_out + z.j) * a.G + z.g;
        a.dst.ks[so] = c8_pow2(nk);
        a.dst.vs[so] = c8_pow2(nv);
      }
      x[q].j = y[q].j;
      x[q].g = y[q].g;
#pragma unroll
      for (int p = 0; p < kPass; ++p) x[q].u[p] = y[q].u[p];
    }
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
  return launch_behind(cache8_move_kernel<D, BLK>, dim3((unsigned)((groups + loop - 1) / loop), (unsigned)a.batch), kThr,
                       0, s, true, a, loop);
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
bool keep_fits(int T, int vec, int ctas) { return (long)T + (T % 4 ? 6 : 0) <= (long)kSelPart * vec * ctas; }

// Clusters of 16 where the device can hold one (8 are always possible).
template <int VEC, bool REG>
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
  const auto kernel = cache8_keep_kernel<VEC, REG>;
  int most = 0;
  const int n = cluster_ctas(
      ctas,
      [&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess; },
      [&] { return cudaOccupancyMaxActiveClusters(&most, kernel, &cfg) == cudaSuccess ? most : 0; });
  if (n != ctas) {
    (void)cudaGetLastError();
    at.val.clusterDim.x = (unsigned)n;
    cfg.gridDim = dim3((unsigned)(a.batch * a.G * n));
  }
  return cudaLaunchKernelEx(&cfg, kernel, a);
}
// Which selection: clusters of as few CTAs as hold a (sequence, group)'s weights in registers with eight
// loads a lane, up to 8; of more while that leaves SMs without a CTA and a part 2048 weights or more.
// Where 8 do not hold them: launches over the whole GPU if clusters of 16 would leave SMs without a CTA
// (1M weights, 4 groups: 38 us, against 76 us with 4 clusters of 16), else those.
bool keep_on_grid(long units, int T) { return !keep_fits(T, 8, 8) && units * 16 <= 148; }
int keep_grid_ctas(int T) { return (int)(((long)T + 6 + 4 * kGridVec * kGridThr - 1) / (4 * kGridVec * kGridThr)); }
cudaError_t launch_keep_any(const C8EvictArgs& a, cudaStream_t s) {
  const long units = (long)a.batch * a.G;
  if (keep_on_grid(units, a.T)) {
    const int ctas = keep_grid_ctas(a.T);
    cudaError_t e = cudaMemsetAsync(a.grid_ws, 0, (size_t)units * keep_grid_words(ctas) * 4, s);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)ctas, (unsigned)units);
    cache8_keep_grid_kernel<0><<<grid, kGridThr, 0, s>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if ((e = launch_behind(cache8_keep_grid_kernel<1>, grid, kGridThr, 0, s, true, a)) != cudaSuccess) return e;
    if ((e = launch_behind(cache8_keep_grid_kernel<2>, grid, kGridThr, 0, s, true, a)) != cudaSuccess) return e;
    if ((e = launch_behind(cache8_keep_grid_kernel<3>, grid, kGridThr, 0, s, true, a)) != cudaSuccess) return e;
    return launch_behind(cache8_keep_grid_kernel<4>, grid, kGridThr, 0, s, true, a);
  }
  int c = 1;
  while (c < 8 && (!keep_fits(a.T, 8, c) || (units * c * 2 <= 148 && a.T >= c * 2 * 2048))) c *= 2;
  if (keep_fits(a.T, 1, c)) return launch_keep<1, true>(a, c, s);
  if (keep_fits(a.T, 2, c)) return launch_keep<2, true>(a, c, s);
  if (keep_fits(a.T, 4, c)) return launch_keep<4, true>(a, c, s);
  if (keep_fits(a.T, 8, c)) return launch_keep<8, true>(a, c, s);
  return launch_keep<4, false>(a, 16, s);
}

}  // namespace

size_t cache8_keep_bytes(int batch, int G, int T) {
  const long units = (long)batch * G;
  return keep_on_grid(units, T) ? (size_t)units * keep_grid_words(keep_grid_ctas(T)) * 4 : 0;
}

cudaError_t launch_cache8_evict(const C8EvictArgs& a, cudaStream_t s) {
  const cudaError_t e = launch_keep_any(a, s);
  if (e != cudaSuccess) return e;
  return a.d == 64 ? launch_d<64>(a, s) : launch_d<128>(a, s);
}

}  // namespace sgqa
