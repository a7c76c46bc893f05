// Appending tokens to the block-scaled 8-bit KV cache (format: cache8.cuh).
//
// A work item is one touched block of one (sequence, group), K and V together: every thread loads
// 16 dims of a row (32 bytes of bf16 for K, 32 for V), the item's largest finite magnitudes meet in
// shared memory, and the codes go out as one 16-byte store per row piece: each new element is read
// once and written once, no second pass. A block that held tokens before keeps its scale unless a new
// token needs a larger one; only then are its codes read, rounded again and rewritten. HBM bound: 2
// bytes read and 1 written per element. Item indices are 32-bit, the sequence is a grid dimension and a
// CTA goes through several items: with 64-bit divisions for every item the kernel was bound by them.
// Measured: 8 prompts of up to 24K tokens (258 MB) 47 us a call, the kernel 39 us = 6.6 TB/s (105 us
// before); four tokens of 32 sequences 2.9 us on the device.
#include "cache8.cuh"

namespace sgqa {
namespace {

constexpr int kThr = 256;

// Largest finite magnitude (bf16 bits) of 16 bf16 values.
__device__ __forceinline__ uint32_t amax16(const uint4 (&x)[2]) {
  const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = c8_max_u16x2(m, w[i] & 0x7FFF7FFFu);
  m = max(m & 0xFFFFu, m >> 16);
  if (m < 0x7F80u) return m;
  m = 0;  // an infinity or NaN among them
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;
    m = max(m, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
  }
  return m;
}
__device__ __forceinline__ uint2 encode8(const uint4& x, float inv) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = c8_encode2(bf16_lo(w[i]) * inv, bf16_hi(w[i]) * inv);
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// D: head dim; BLK: tokens per block. Rows of a block are spread over the threads, D / 16 to a row;
// small blocks share a CTA (a warp always serves one item), large ones take several passes. A CTA goes
// through `loop` groups of items, so that what every thread works out once is shared by all of them.
constexpr int kLoop = 8;
template <int D, int BLK>
__global__ void __launch_bounds__(kThr) cache8_append_kernel(C8AppendArgs a, int items, int loop) {
  constexpr int kTpr = D / 16, kRows = kThr / kTpr;
  constexpr int kItems = kRows > BLK ? kRows / BLK : 1;
  constexpr int kPass = BLK > kRows ? BLK / kRows : 1;
  __shared__ uint32_t amax[kLoop][kItems][2];
  const int tid = threadIdx.x, b = blockIdx.y;
  const int cnt = a.counts ? __ldg(a.counts + b) : a.n_t, L = __ldg(a.lens + b);
  if (L < 0 || cnt < 0 || cnt > a.n_t || (long)L + cnt > a.T) {
    if (tid == 0) report(a.status, SGQA_ERR_DEVICE_CHECK);
    return;
  }
  const int end = L + cnt, j0 = L / BLK;
  const int first = (int)blockIdx.x * loop * kItems;  // item: (touched block, g), g fastest
  if (cnt == 0 || (j0 + first / a.G) * BLK >= end) return;
  for (int i = tid; i < kLoop * kItems * 2; i += kThr) (&amax[0][0][0])[i] = 0u;
  __syncthreads();
  const int sub = kItems > 1 ? (tid / kTpr) / BLK : 0;
  const int row0 = kItems > 1 ? (tid / kTpr) % BLK : tid / kTpr;
  const int col = (tid % kTpr) * 16;
  const int nblk = (a.T + BLK - 1) / BLK;
  int item = first + sub, j = j0 + item / a.G, g = item % a.G;
  for (int it = 0; it < loop; ++it) {
    const int u0 = j * BLK;
    const bool live = item < items && u0 < end && SGQA_CHECK(j < nblk && g < a.G, a.status);
    uint4 xk[kPass][2], xv[kPass][2];
    uint32_t mk = 0, mv = 0;
#pragma unroll
    for (int p = 0; p < kPass; ++p) {
      const int u = u0 + row0 + p * kRows;
      xk[p][0] = xk[p][1] = xv[p][0] = xv[p][1] = make_uint4(0, 0, 0, 0);
      if (live && u >= L && u < end) {
        const long src = (long)((b * a.n_t + (u - L)) * a.G + g) * D + col;
        const uint4* pk = reinterpret_cast<const uint4*>(a.k + src);
        const uint4* pv = reinterpret_cast<const uint4*>(a.v + src);
        xk[p][0] = __ldg(pk);
        xk[p][1] = __ldg(pk + 1);
        xv[p][0] = __ldg(pv);
        xv[p][1] = __ldg(pv + 1);
      }
    }
    // the scales of a block that holds tokens already (read by all before one thread writes them)
    const long si = (long)(b * nblk + j) * a.G + g;
    const bool held = live && u0 < L;
    const int ek_old = held ? c8_scale_exponent(a.c.ks[si]) : -126;
    const int ev_old = held ? c8_scale_exponent(a.c.vs[si]) : -126;
#pragma unroll
    for (int p = 0; p < kPass; ++p) {
      mk = max(mk, amax16(xk[p]));
      mv = max(mv, amax16(xv[p]));
    }
    mk = __reduce_max_sync(0xFFFFFFFFu, mk);
    mv = __reduce_max_sync(0xFFFFFFFFu, mv);
    if ((tid & 31) == 0) {
      atomicMax(&amax[it][sub][0], mk);
      atomicMax(&amax[it][sub][1], mv);
    }
    __syncthreads();
    if (live) {
      const int ek = max(ek_old, c8_exponent(amax[it][sub][0] << 16)), ev = max(ev_old, c8_exponent(amax[it][sub][1] << 16));
      const float ik = c8_pow2(-ek), iv = c8_pow2(-ev);
#pragma unroll
      for (int p = 0; p < kPass; ++p) {
        const int u = u0 + row0 + p * kRows;
        if (u >= end || !SGQA_CHECK(u < a.T, a.status)) break;
        const long dst = (long)((b * a.T + u) * a.G + g) * D + col;
        uint4* ok = reinterpret_cast<uint4*>(a.c.k8 + dst);
        uint4* ov = reinterpret_cast<uint4*>(a.c.v8 + dst);
        if (u >= L) {
          const uint2 k0 = encode8(xk[p][0], ik), k1 = encode8(xk[p][1], ik);
          const uint2 v0 = encode8(xv[p][0], iv), v1 = encode8(xv[p][1], iv);
          *ok = make_uint4(k0.x, k0.y, k1.x, k1.y);
          *ov = make_uint4(v0.x, v0.y, v1.x, v1.y);
        } else {
          if (ek > ek_old) *ok = c8_rescale16(*ok, ek_old - ek);
          if (ev > ev_old) *ov = c8_rescale16(*ov, ev_old - ev);
        }
      }
      if (row0 == 0 && col == 0) {
        a.c.ks[si] = c8_pow2(ek);
        a.c.vs[si] = c8_pow2(ev);
      }
    }
    item += kItems;
    for (g += kItems; g >= a.G; g -= a.G) ++j;
  }
}

template <int D, int BLK>
cudaError_t launch(const C8AppendArgs& a, cudaStream_t s) {
  constexpr int kRows = kThr / (D / 16);
  constexpr int kItems = kRows > BLK ? kRows / BLK : 1;
  // n_t tokens can touch one block more than they fill, but never more than there are
  const long nblk = ((long)a.T + BLK - 1) / BLK;
  const long touched = ((long)a.n_t + BLK - 1) / BLK + 1;
  const long items = (touched < nblk ? touched : nblk) * a.G;  // of a sequence; T * G is below 2^31
  const long groups = (items + kItems - 1) / kItems;
  // groups of items per CTA: several once the GPU is full several times over without
  const long full = groups * a.batch / (148 * 6 * 4);
  const int loop = (int)(full < 1 ? 1 : full > kLoop ? kLoop : full);
  cache8_append_kernel<D, BLK><<<dim3((unsigned)((groups + loop - 1) / loop), (unsigned)a.batch), kThr, 0, s>>>(
      a, (int)items, loop);
  return cudaGetLastError();
}
template <int D>
cudaError_t launch_d(const C8AppendArgs& a, cudaStream_t s) {
  switch (a.block) {
    case 8: return launch<D, 8>(a, s);
    case 16: return launch<D, 16>(a, s);
    case 32: return launch<D, 32>(a, s);
    case 64: return launch<D, 64>(a, s);
    default: return launch<D, 128>(a, s);
  }
}

}  // namespace

cudaError_t launch_cache8_append(const C8AppendArgs& a, cudaStream_t s) {
  return a.d == 64 ? launch_d<64>(a, s) : launch_d<128>(a, s);
}

}  // namespace sgqa
