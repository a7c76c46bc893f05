// The block-scaled 8-bit KV cache: its format, the arguments of its kernels, and the device helpers
// they share.
//
// Format. K and V rows are E4M3 codes [batch, T, G, d] with one scale per block of `block` tokens
// and KV group, [batch, ceil(T / block), G] fp32: s = 2^e with e the smallest integer of [-126, 119]
// such that max |x| <= 448 s over the block's finite values (448: E4M3's largest value; at 119 code
// times scale stays finite); a code is x / s rounded to nearest even, saturating; NaN stays NaN and
// counts for no scale. A power of two makes the value code * s exact in bf16 and fp32, and moving a row to
// a block of another scale loses nothing but what falls below that block's subnormal step.
#pragma once
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace sgqa {

constexpr int kC8MaxRows = 64;  // query rows (n_new * Hq / G) of a sequence and group in one step

struct Cache8 {
  uint8_t* k8;
  float* ks;
  uint8_t* v8;
  float* vs;
};

struct C8AppendArgs {
  const int32_t* lens;
  const int32_t* counts;  // may be null: n_t tokens each
  const uint16_t* k;      // [batch, n_t, G, d] bf16
  const uint16_t* v;
  Cache8 c;
  int batch, T, G, d, block, n_t;
  int* status;
};
cudaError_t launch_cache8_append(const C8AppendArgs& a, cudaStream_t s);

struct C8AttendArgs {
  const int32_t* lens;
  const uint16_t* q;  // [batch, n_new, Hq, d] bf16
  const uint16_t* gate;
  Cache8 c;
  uint16_t* out;
  const float* w_in;  // [batch, G, T], may be null
  float* w_out;       // [batch, G, T], null: no weights
  float* lse;         // [batch, G, n_new * R]: log2 of each row's softmax sum
  float* part;
  int batch, T, Hq, G, d, block, n_new;
  int stall_cta;  // failure-detection test hook: this CTA issues no loads (-1: none)
  // set by the launch: chunks of rows per (sequence, group), rows of each, log2 of block
  int nch, chunk_rows, block_log2;
  int main_ctas;  // and, for the join, the CTAs of the launch before
  int* status;
};
size_t cache8_part_bytes(int batch, int G, int rows, int d);
cudaError_t launch_cache8_attend(const C8AttendArgs& a, cudaStream_t s);

struct C8EvictArgs {
  const int32_t* lens;
  const float* weight;  // [batch, G, T]
  Cache8 src, dst;
  float* w_out;         // [batch, G, T_out]
  int32_t* kept;        // [batch, G, keep]
  int32_t* lens_out;
  uint32_t* grid_ws;  // cache8_keep_bytes
  int batch, T, T_out, G, d, block, keep, recent;
  int* status;
};
size_t cache8_keep_bytes(int batch, int G, int T);
cudaError_t launch_cache8_evict(const C8EvictArgs& a, cudaStream_t s);

// Launch whose start overlaps the end of the kernel before it on the stream (after which it waits
// where it needs that kernel's results) or, with ahead false, an ordinary one.
template <class... P, class... A>
inline cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t s, bool ahead,
                          A... args) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &at;
  cfg.numAttrs = ahead ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ---- device helpers ----------------------------------------------------------------------------
// Exponent of the scale from the bits of the largest finite |x| (an fp32): amax = m 2^E with m in
// [1, 2) and 448 = 1.75 2^8, so e = E - 8, plus one when m > 1.75, within [-126, 119]. Zeros and fp32
// subnormals have an exponent field that reads E = -127 and get -126 as they should.
__device__ __forceinline__ int c8_exponent(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23) - 127 - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return max(-126, min(119, e));
}
// 2^e for the exponents a scale and its inverse can have
__device__ __forceinline__ float c8_pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// exponent of a scale as the format has them (anything else is read as the nearest that it has)
__device__ __forceinline__ int c8_scale_exponent(float s) {
  return max(-126, min(119, (int)((__float_as_uint(s) >> 23) & 255u) - 127));
}

// two fp32 values as two E4M3 codes (nearest even, saturating; the first in the low byte)
__device__ __forceinline__ uint32_t c8_encode2(float x0, float x1) {
  return __nv_cvt_float2_to_fp8x2(make_float2(x0, x1), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 c8_decode2(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xFFFFu), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// four codes times f, rounded to E4M3 again (one rounding: the products are exact in fp32)
__device__ __forceinline__ uint32_t c8_rescale4(uint32_t w, float f) {
  const float2 a = c8_decode2(w), b = c8_decode2(w >> 16);
  return c8_encode2(a.x * f, a.y * f) | (c8_encode2(b.x * f, b.y * f) << 16);
}
// two codes times 2^k, rounded to E4M3 again, for k of [-24, 15] in fp16: a product of 2^-11 or more is exact there,
// one below becomes 0 as it should.
__device__ __forceinline__ uint32_t c8_rescale2_half(uint32_t two, __half2 f) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(two & 0xFFFFu), __NV_E4M3);
  const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&h), f);
  return __nv_cvt_halfraw2_to_fp8x2(*reinterpret_cast<const __half2_raw*>(&y), __NV_SATFINITE, __NV_E4M3);
}
// 2^k for rescaling codes; beyond +-40 every code but 0 saturates or vanishes anyway
__device__ __forceinline__ float c8_shift(int k) { return c8_pow2(max(-40, min(40, k))); }

// 16 codes times 2^k, rounded to E4M3 again
__device__ __forceinline__ uint4 c8_rescale16(const uint4& x, int k) {
  if (k == 0) return x;
  if (k > 15) {
    const float f = c8_shift(k);
    return make_uint4(c8_rescale4(x.x, f), c8_rescale4(x.y, f), c8_rescale4(x.z, f), c8_rescale4(x.w, f));
  }
  const __half2 f = __float2half2_rn(c8_pow2(max(-24, k)));
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = c8_rescale2_half(w[i], f) | (c8_rescale2_half(w[i] >> 16, f) << 16);
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// the larger of each 16-bit half
__device__ __forceinline__ uint32_t c8_max_u16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}

// A kernel launched with programmatic serialization starts when every CTA of the one before it has
// called grid_dependents() or ended; grid_wait() returns when that kernel has ended and its writes are seen.
__device__ __forceinline__ void grid_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// lens[b] if it is a length this cache can have, else 0 and a device check
__device__ __forceinline__ int c8_len(const int32_t* lens, int b, int T, int* status) {
  const int n = __ldg(lens + b);
  if (n >= 0 && n <= T) return n;
  report(status, SGQA_ERR_DEVICE_CHECK);
  return 0;
}

}  // namespace sgqa
