// Dense gated attention of a step's tokens over the block-scaled 8-bit KV cache (format:
// cache8.cuh), and the attention weight every token received.
#include "cache8.cuh"

namespace sgqa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kWarps = 8;

// One CTA per query row (sequence, new token, head); warps take tokens in turn, each with a running
// maximum and sum.
template <int D>
__global__ void __launch_bounds__(kWarps * 32) cache8_attend_row_kernel(C8AttendArgs a) {
  constexpr int kE = D / 32;
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][D];
  const int h = blockIdx.x % a.Hq, i = (blockIdx.x / a.Hq) % a.n_new, b = blockIdx.x / (a.Hq * a.n_new);
  const int R = a.Hq / a.G, g = h / R;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int L = c8_len(a.lens, b, a.T, a.status);
  const int end = L - a.n_new + i + 1;
  const long nblk = (a.T + a.block - 1) / a.block;
  const long row = (((long)b * a.n_new + i) * a.Hq + h) * D;
  const float sc = kLog2e / sqrtf((float)D);
  float q[kE], o[kE];
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    q[e] = bf16_to_f32(a.q[row + lane * kE + e]);
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int u = warp; u < end; u += kWarps) {
    const long at = (((long)b * a.T + u) * a.G + g) * D + lane * kE;
    const long si = ((long)b * nblk + u / a.block) * a.G + g;
    float z = 0.f, v[kE];
#pragma unroll
    for (int e = 0; e < kE; e += 2) {
      const float2 k2 = c8_decode2(*reinterpret_cast<const uint16_t*>(a.c.k8 + at + e));
      const float2 v2 = c8_decode2(*reinterpret_cast<const uint16_t*>(a.c.v8 + at + e));
      z = fmaf(q[e], k2.x, fmaf(q[e + 1], k2.y, z));
      v[e] = v2.x;
      v[e + 1] = v2.y;
    }
#pragma unroll
    for (int x = 16; x; x >>= 1) z += __shfl_xor_sync(0xFFFFFFFFu, z, x);
    z *= sc * a.c.ks[si];
    const float mn = fmaxf(m, z), f = exp2f(m - mn), p = exp2f(z - mn), pv = p * a.c.vs[si];
    l = l * f + p;
#pragma unroll
    for (int e = 0; e < kE; ++e) o[e] = fmaf(pv, v[e], o[e] * f);
    m = mn;
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < kE; ++e) so[warp][lane * kE + e] = o[e];
  __syncthreads();
  float ms = -INFINITY;
  for (int w = 0; w < kWarps; ++w) ms = fmaxf(ms, sm[w]);
  float den = 0.f;
  for (int w = 0; w < kWarps; ++w) den += sm[w] == -INFINITY ? 0.f : sl[w] * exp2f(sm[w] - ms);
  if (tid < D) {
    float y = 0.f;
    for (int w = 0; w < kWarps; ++w) y += sm[w] == -INFINITY ? 0.f : so[w][tid] * exp2f(sm[w] - ms);
    y = end > 0 ? y / den : 0.f;
    a.out[row + tid] = f32_to_bf16_rne(y * sigmoid_fast(bf16_to_f32(a.gate[row + tid])));
  }
  if (tid == 0) a.lse[((long)b * a.G + g) * a.n_new * R + i * R + h % R] = ms + log2f(den);
}

// One thread per token: its probabilities under all rows of its group.
template <int D>
__global__ void __launch_bounds__(128) cache8_weight_kernel(C8AttendArgs a) {
  const int R = a.Hq / a.G, g = blockIdx.y, b = blockIdx.z;
  const int u = blockIdx.x * blockDim.x + threadIdx.x;
  const int L = c8_len(a.lens, b, a.T, a.status);
  if (u >= L) return;
  const long nblk = (a.T + a.block - 1) / a.block;
  const float sc = kLog2e / sqrtf((float)D) * a.c.ks[((long)b * nblk + u / a.block) * a.G + g];
  const uint8_t* k = a.c.k8 + (((long)b * a.T + u) * a.G + g) * D;
  float sum = 0.f;
  for (int i = 0; i < a.n_new; ++i) {
    if (u > L - a.n_new + i) continue;
    for (int r = 0; r < R; ++r) {
      const uint16_t* q = a.q + (((long)b * a.n_new + i) * a.Hq + g * R + r) * D;
      float z = 0.f;
      for (int e = 0; e < D; e += 2) {
        const float2 k2 = c8_decode2(*reinterpret_cast<const uint16_t*>(k + e));
        z = fmaf(bf16_to_f32(q[e]), k2.x, fmaf(bf16_to_f32(q[e + 1]), k2.y, z));
      }
      sum += exp2f(z * sc - a.lse[((long)b * a.G + g) * a.n_new * R + i * R + r]);
    }
  }
  const long wi = ((long)b * a.G + g) * a.T + u;
  a.w_out[wi] = (a.w_in && u < L - a.n_new ? a.w_in[wi] : 0.f) + sum;
}

template <int D>
cudaError_t launch(const C8AttendArgs& a, cudaStream_t s) {
  cache8_attend_row_kernel<D><<<(unsigned)(a.batch * a.n_new * a.Hq), kWarps * 32, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !a.w_out) return e;
  cache8_weight_kernel<D><<<dim3((unsigned)((a.T + 127) / 128), (unsigned)a.G, (unsigned)a.batch), 128, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t cache8_part_bytes(int, int, int, int) { return 0; }

cudaError_t launch_cache8_attend(const C8AttendArgs& a, cudaStream_t s) {
  return a.d == 64 ? launch<64>(a, s) : launch<128>(a, s);
}

}  // namespace sgqa
