// C ABI of the block-scaled 8-bit KV cache (include/sgqa.h): argument checks, workspace layout and
// the kernels of each call. No allocation, no host synchronisation, no global state.
#include "api_common.h"
#include "cache8.cuh"

using namespace sgqa;

namespace {

int check_cache8(const sgqa_dims* d, int block) {
  const int rc = check_dims(d);
  if (rc) return rc;
  if (block != 8 && block != 16 && block != 32 && block != 64 && block != 128) return SGQA_ERR_UNSUPPORTED;
  return SGQA_OK;
}

struct Cache8Ws {
  int* status;
  float* lse;
  float* part;
  size_t bytes;
};

Cache8Ws cache8_layout(const sgqa_dims* d, int n_new, void* ws) {
  Cache8Ws w{};
  uint8_t* base = static_cast<uint8_t*>(ws);
  size_t off = kStatusBytes;
  w.status = reinterpret_cast<int*>(base);
  w.lse = reinterpret_cast<float*>(base + off);
  off += align256((size_t)d->batch * n_new * d->Hq * 4);
  w.part = reinterpret_cast<float*>(base + off);
  off += align256(cache8_part_bytes(d->batch, d->G, n_new * (d->Hq / d->G), d->d));
  w.bytes = off;
  return w;
}

// attention's and eviction's workspaces lie at the same place: no call keeps anything there
size_t evict_bytes(const sgqa_dims* d) { return kStatusBytes + align256(cache8_keep_bytes(d->batch, d->G, d->T)); }

bool ws_ok(const void* ws, size_t have, size_t need) {
  return ws && (reinterpret_cast<uintptr_t>(ws) & 255u) == 0 && have >= need;
}

bool cache_ok(const uint8_t* k8, const float* ks, const uint8_t* v8, const float* vs) {
  return aligned16(k8) && aligned16(ks) && aligned16(v8) && aligned16(vs);
}

// Memory of a call's tensors: whether an output shares some with an input or another output.
struct Span {
  const void* p;
  long bytes;
};
bool meet(const Span& x, const Span& y) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
  return x.p && y.p && a < b + (uintptr_t)y.bytes && b < a + (uintptr_t)x.bytes;
}
template <int IN, int OUT>
bool overlap(const Span (&in)[IN], const Span (&out)[OUT]) {
  for (int i = 0; i < OUT; ++i) {
    for (const Span& x : in)
      if (meet(x, out[i])) return true;
    for (int j = 0; j < i; ++j)
      if (meet(out[j], out[i])) return true;
  }
  return false;
}
// bytes of a cache's codes (K or V) and of their scales
long code_bytes(const sgqa_dims* d, int T) { return (long)d->batch * T * d->G * d->d; }
long scale_bytes(const sgqa_dims* d, int T, int block) { return (long)d->batch * (((long)T + block - 1) / block) * d->G * 4; }

Cache8 cache_of(const uint8_t* k8, const float* ks, const uint8_t* v8, const float* vs) {
  return {const_cast<uint8_t*>(k8), const_cast<float*>(ks), const_cast<uint8_t*>(v8), const_cast<float*>(vs)};
}

}  // namespace

extern "C" {

size_t sgqa_cache8_workspace_size(const sgqa_dims* dims, int block, int n_new) {
  if (check_cache8(dims, block) != SGQA_OK || n_new <= 0 || (long)n_new * (dims->Hq / dims->G) > kC8MaxRows) return 0;
  const size_t at = cache8_layout(dims, n_new, nullptr).bytes, ev = evict_bytes(dims);
  return at > ev ? at : ev;
}

int sgqa_cache8_append(const sgqa_dims* dims, int block, const int32_t* lens, const int32_t* counts, int n_t,
                       const uint16_t* k_new, const uint16_t* v_new, uint8_t* k8, float* k_scale, uint8_t* v8,
                       float* v_scale, void* ws, size_t ws_bytes, void* stream) {
  const int rc = check_cache8(dims, block);
  if (rc) return rc;
  if (n_t < 0 || n_t > dims->T) return SGQA_ERR_INVALID_ARG;
  if (!aligned16(lens) || (counts && !aligned16(counts)) || !cache_ok(k8, k_scale, v8, v_scale))
    return SGQA_ERR_INVALID_ARG;
  if (n_t > 0 && (!aligned16(k_new) || !aligned16(v_new))) return SGQA_ERR_INVALID_ARG;
  if (!ws_ok(ws, ws_bytes, kStatusBytes)) return SGQA_ERR_WORKSPACE;
  if (n_t == 0) return SGQA_OK;
  const long c = code_bytes(dims, dims->T), s = scale_bytes(dims, dims->T, block), x = code_bytes(dims, n_t) * 2;
  if (overlap<4, 5>({{lens, dims->batch * 4L}, {counts, dims->batch * 4L}, {k_new, x}, {v_new, x}},
                    {{k8, c}, {v8, c}, {k_scale, s}, {v_scale, s}, {ws, kStatusBytes}}))
    return SGQA_ERR_INVALID_ARG;
  C8AppendArgs a{};
  a.lens = lens; a.counts = counts; a.k = k_new; a.v = v_new; a.c = cache_of(k8, k_scale, v8, v_scale);
  a.batch = dims->batch; a.T = dims->T; a.G = dims->G; a.d = dims->d; a.block = block; a.n_t = n_t;
  a.status = static_cast<int*>(ws);
  return cuda_status(launch_cache8_append(a, static_cast<cudaStream_t>(stream)));
}

int sgqa_cache8_attend(const sgqa_dims* dims, int block, const int32_t* lens, int n_new, const uint16_t* q,
                       const uint16_t* gate, const uint8_t* k8, const float* k_scale, const uint8_t* v8,
                       const float* v_scale, uint16_t* out, const float* weight_in, float* weight_out, void* ws,
                       size_t ws_bytes, void* stream) {
  const int rc = check_cache8(dims, block);
  if (rc) return rc;
  if (n_new <= 0 || (weight_in && !weight_out)) return SGQA_ERR_INVALID_ARG;
  if ((long)n_new * (dims->Hq / dims->G) > kC8MaxRows) return SGQA_ERR_UNSUPPORTED;
  if (!aligned16(lens) || !aligned16(q) || !aligned16(gate) || !aligned16(out) ||
      !cache_ok(k8, k_scale, v8, v_scale) || (weight_in && !aligned16(weight_in)) ||
      (weight_out && !aligned16(weight_out)))
    return SGQA_ERR_INVALID_ARG;
  const Cache8Ws w = cache8_layout(dims, n_new, ws);
  if (!ws_ok(ws, ws_bytes, w.bytes)) return SGQA_ERR_WORKSPACE;
  const long c = code_bytes(dims, dims->T), s = scale_bytes(dims, dims->T, block), x = (long)dims->batch * n_new * dims->Hq * dims->d * 2;
  const long wt = (long)dims->batch * dims->G * dims->T * 4;
  // (the gate of an element is read by the thread that writes it, and so is a weight's past: out may be gate,
  // weight_out may be weight_in, whole)
  if (overlap<8, 3>({{lens, dims->batch * 4L}, {q, x}, {k8, c}, {v8, c}, {k_scale, s}, {v_scale, s},
                     {gate == out ? nullptr : gate, x}, {weight_in == weight_out ? nullptr : weight_in, wt}},
                    {{out, x}, {weight_out, wt}, {ws, (long)w.bytes}}))
    return SGQA_ERR_INVALID_ARG;
  C8AttendArgs a{};
  a.lens = lens; a.q = q; a.gate = gate; a.c = cache_of(k8, k_scale, v8, v_scale); a.out = out;
  a.w_in = weight_in; a.w_out = weight_out; a.lse = w.lse; a.part = w.part;
  a.batch = dims->batch; a.T = dims->T; a.Hq = dims->Hq; a.G = dims->G; a.d = dims->d; a.block = block;
  a.n_new = n_new; a.status = w.status; a.stall_cta = g_test_stall_cta;
  return cuda_status(launch_cache8_attend(a, static_cast<cudaStream_t>(stream)));
}

int sgqa_cache8_evict(const sgqa_dims* dims, int block, const int32_t* lens, int keep, int recent, int T_out,
                      const float* weight, const uint8_t* k8, const float* k_scale, const uint8_t* v8,
                      const float* v_scale, uint8_t* k8_out, float* k_scale_out, uint8_t* v8_out,
                      float* v_scale_out, float* weight_out, int32_t* kept, int32_t* lens_out, void* ws,
                      size_t ws_bytes, void* stream) {
  const int rc = check_cache8(dims, block);
  if (rc) return rc;
  if (keep <= 0 || recent < 0 || recent > keep || T_out < keep || T_out >= (1 << 28)) return SGQA_ERR_INVALID_ARG;
  if ((long)dims->batch * T_out * dims->G >= (1L << 31)) return SGQA_ERR_UNSUPPORTED;  // row indices are 32-bit
  if (!aligned16(lens) || !aligned16(weight) || !cache_ok(k8, k_scale, v8, v_scale) ||
      !cache_ok(k8_out, k_scale_out, v8_out, v_scale_out) || !aligned16(weight_out) || !aligned16(kept) ||
      !aligned16(lens_out))
    return SGQA_ERR_INVALID_ARG;
  if (!ws_ok(ws, ws_bytes, evict_bytes(dims))) return SGQA_ERR_WORKSPACE;
  const long c = code_bytes(dims, dims->T), s = scale_bytes(dims, dims->T, block), w = (long)dims->batch * dims->G * dims->T * 4;
  const long co = code_bytes(dims, T_out), so = scale_bytes(dims, T_out, block), n = (long)dims->batch * dims->G * 4;
  if (overlap<6, 8>({{lens, dims->batch * 4L}, {weight, w}, {k8, c}, {v8, c}, {k_scale, s}, {v_scale, s}},
                    {{k8_out, co}, {v8_out, co}, {k_scale_out, so}, {v_scale_out, so}, {weight_out, n * T_out},
                     {kept, n * keep}, {lens_out, dims->batch * 4L}, {ws, (long)evict_bytes(dims)}}))
    return SGQA_ERR_INVALID_ARG;
  C8EvictArgs a{};
  a.grid_ws = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(ws) + kStatusBytes);
  a.lens = lens; a.weight = weight; a.src = cache_of(k8, k_scale, v8, v_scale);
  a.dst = cache_of(k8_out, k_scale_out, v8_out, v_scale_out); a.w_out = weight_out; a.kept = kept;
  a.lens_out = lens_out; a.batch = dims->batch; a.T = dims->T; a.T_out = T_out; a.G = dims->G; a.d = dims->d;
  a.block = block; a.keep = keep; a.recent = recent; a.status = static_cast<int*>(ws);
  return cuda_status(launch_cache8_evict(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
