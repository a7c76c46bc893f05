// Dense gated attention of a step's tokens over the block-scaled 8-bit KV cache (format:
// cache8.cuh), and the attention weight every token received.
//
// With z_u = s_u q . k_u / sqrt(d) (k_u the codes, s_u their block's scale) a row's output is
// sum_u 2^(z_u - m) t_u v_u / sum_u 2^(z_u - m) (t_u the V scale, z in units of log2 e). The cache is
// read once, 2 d bytes per token and group against at most 8 d * 32 operations: HBM bound. So the
// codes go to the tensor cores as they are, without a conversion, as the wide operand (M = 128 tokens
// or head dims), and the few query rows of a (sequence, group) are the narrow one:
//   S^T[128 tokens x 2 NR] = K_tile . [q1; q2]^T       q = (q1 + q2 / 16) 2^e, both E4M3
//   O^T[d x 2 NR]          = V_tile^T . [P1 | P2]      p t = (P1 + P2 / 28) 2^E / 448, both E4M3
// Two E4M3 terms hold q exactly down to 2^-22 of its row's largest element and p t to 2^-8 of itself
// or 2^-23 of the tile's largest. P is relative to its own tile's maxima (of z per row, of t over the
// tile), so O^T starts anew in every tile and is added up in registers in fp32: a token that takes
// nearly all attention costs the far ones none of their digits. The denominator and the maxima are
// taken from fp32 scores.
//
// Work: the tiles of 128 tokens of all (sequence, group) units, in that order, cut into one equal
// contiguous piece per CTA (one CTA per SM), so that ragged lengths, one long sequence and many
// short ones all balance; the lengths are read on the device. A unit's pieces leave partial sums,
// which a second kernel joins in the order of the tiles.
// Roles: warp 0 issues TMA loads, warp 1 the MMAs, warps 2-3 split the rows of q, warps 4-7 and
// 8-11 take tiles in turn (a thread per token) from S^T to P, warps 12-15 (a thread per head dim)
// add O^T up. Waits are bounded as everywhere (tc_common.cuh).
// The received weights need each row's final sum: a further pass over K recomputes the scores.
#include <cuda.h>

#include "cache8.cuh"
#include "tc_common.cuh"

namespace sgqa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegMax = -3.4028234663852886e38f;  // maximum of a row that no token has reached
constexpr int kTok = 128;                           // tokens per tile
constexpr int kGridMax = 148;                       // one CTA per SM
constexpr int kThreads = 512;
constexpr int kMaxNR = 32;                          // rows per unit; more make several units
constexpr int kNever = 0x7FFFFFFF;

template <int D, int NR, bool W>
struct Cfg {
  static constexpr int N = 2 * NR;                       // MMA columns: both terms of every row
  static constexpr int kTile = kTok * D;
  static constexpr int kStage = W ? kTile : 2 * kTile;   // K, then V
  static constexpr int kStages = D == 128 ? (W ? 8 : 5) : (W ? 8 : 8);
  static constexpr int kQ = N * D;
  static constexpr int kP = W ? 0 : kTok * N;
  static constexpr int kTmem = (W ? 2 : 4) * N < 32 ? 32 : (W ? 2 : 4) * N;
  static constexpr int kRowsT = D == 128 ? NR : NR / 2;  // rows per accumulating thread
};

template <int NR>
struct Shared {
  uint64_t full[8], empty[8];
  uint64_t s_full[2], s_empty[2], p_full[2], o_full[2], o_empty[2], q_full[2], q_empty[2];
  uint32_t tmem;
  volatile int abort_flag;
  int start_b, start_off, total;
  int wsum[16];
  int nan_any[2];
  int nan_at[2][128];       // per head dim: first token not visible to all rows whose V is NaN there
  int wev[2][4];
  int e_tile[2];
  float fac[2][NR];         // per unit parity: 2^e log2 e / sqrt(d) of a row
  float lse[2][NR];
  int lim[2][NR];           // a row's own position; -1: no row
  float wmax[2][4][NR];
  float mt[2][NR];          // per softmax group: a row's maximum over the tile
  float2 ab[2][NR];         // factors of the sums so far and of this tile
  float2 acc_ab[2][NR];
};

// The tiles of one CTA in order. unit = ((sequence, group), chunk of rows).
struct Walk {
  int b, gu, tile, ntiles, L, left, piece;
  bool first;  // the first tile of this CTA's piece of the unit
};
__device__ __forceinline__ int tiles_of(int L) { return (L + kTok - 1) / kTok; }
__device__ __forceinline__ int len_of(const C8AttendArgs& a, int b) {
  const int n = __ldg(a.lens + b);
  return n >= 0 && n <= a.T ? n : 0;
}
__device__ __forceinline__ void walk_begin(Walk& w, const C8AttendArgs& a, int b, int off, int left) {
  w.b = b;
  w.L = len_of(a, b);
  w.ntiles = tiles_of(w.L);
  w.gu = off / w.ntiles;
  w.tile = off % w.ntiles;
  w.left = left;
  w.piece = 0;
  w.first = true;
}
__device__ __forceinline__ bool walk_last(const Walk& w) { return w.left == 1 || w.tile + 1 == w.ntiles; }
__device__ __forceinline__ void walk_next(Walk& w, const C8AttendArgs& a) {
  w.first = false;
  if (--w.left == 0) return;
  if (++w.tile < w.ntiles) return;
  w.tile = 0;
  w.first = true;
  ++w.piece;
  if (++w.gu < a.G * a.nch) return;
  w.gu = 0;
  do {
    ++w.b;
    w.L = len_of(a, w.b);
  } while (w.L == 0);
  w.ntiles = tiles_of(w.L);
}

// Per launch: partial sums of every piece, and the CTAs that hold a unit's first and last tile.
template <int D, int NR>
struct Part {
  static constexpr long kRec = (long)NR * D + NR * 11 + 4;  // O, M, l of eight warps, m of two groups; E
  float* base;
  int* first;
  int* last;
  __device__ __host__ Part(float* p, long units) {
    first = reinterpret_cast<int*>(p);
    last = first + ((units + 3) & ~3L);
    base = p + 2 * ((units + 3) & ~3L);
  }
  __device__ float* o(long slot) const { return base + slot * kRec; }
  __device__ float* m(long slot) const { return base + slot * kRec + NR * D; }
  __device__ float* l(long slot) const { return base + slot * kRec + NR * D + NR; }       // [8][NR]
  __device__ float* lm(long slot) const { return base + slot * kRec + NR * D + 9 * NR; }  // [2][NR]
  __device__ int* e(long slot) const { return reinterpret_cast<int*>(base + slot * kRec + NR * D + 11 * NR); }
};

// ---- PTX ---------------------------------------------------------------------------------------
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p; }" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(acc)
      : "memory");
}
// kind::f8f6f4, E4M3 x E4M3 -> F32, M = 128; MN-major operands where set
__host__ __device__ constexpr uint32_t idesc_f8(int N, bool a_mn, bool b_mn) {
  return (1u << 4) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
}
// MN-major operand whose rows along K are 64 bytes (64B swizzle), 8-row groups 512 bytes apart; the
// second 64 elements along MN lie where the first do (stride 0), so M = 128 holds every dim twice.
__device__ __forceinline__ uint64_t smem_desc_mnmajor_sw64_twice(const void* tile) {
  return (uint64_t)((smem_u32(tile) & 0x3FFFFu) >> 4) | ((uint64_t)(512 >> 4) << 32) | (1ull << 46) | (4ull << 61);
}
__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void group_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }

// A warp's wait. After a wait has run out none waits any longer, but the roles go on through their
// tiles (with whatever is in the buffers), so that no group's barrier is left short of a warp.
__device__ __forceinline__ void warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int* status) {
  if ((threadIdx.x & 31) == 0 && !*abort && !tc::mbar_wait(bar, parity, abort, status)) {
    if (!*abort) report(status, SGQA_ERR_TIMEOUT);
    *abort = 1;
  }
  __syncwarp();
}

// Sums of x[r] over the warp's lanes, in a fixed order; lane r (mod NR) gets row r's.
template <int NR>
__device__ __forceinline__ float warp_sums(float (&x)[NR], int lane) {
#pragma unroll
  for (int h = NR / 2; h >= 1; h >>= 1) {
    const bool up = lane & h;
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const float give = up ? x[i] : x[i + h], have = up ? x[i + h] : x[i];
      x[i] = have + __shfl_xor_sync(0xFFFFFFFFu, give, h);
    }
  }
  float y = x[0];
#pragma unroll
  for (int h = NR; h < 32; h <<= 1) y += __shfl_xor_sync(0xFFFFFFFFu, y, h);
  return y;
}

// A token's V codes of a tile, as TMA's swizzle has laid them out.
template <int D>
__device__ __forceinline__ int v_chunk(int row, int c) {
  return D == 128 ? c ^ (row & 7) : c ^ ((row >> 1) & 3);
}

template <int D, int NR, bool W>
__global__ void __launch_bounds__(kThreads, 1)
    cache8_attend_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                         const C8AttendArgs a) {
  using C = Cfg<D, NR, W>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared<NR> sh;
  uint8_t* sKV = smem_align<1024>(smem_raw);
  uint8_t* sQ = sKV + C::kStages * C::kStage;
  uint8_t* sP = sQ + 2 * C::kQ;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int units_b = a.G * a.nch;

  // ---- this CTA's piece of the tiles ----
  int sum = 0;
  for (int b = tid; b < a.batch; b += kThreads) sum += tiles_of(c8_len(a.lens, b, a.T, a.status)) * units_b;
  sum = __reduce_add_sync(0xFFFFFFFFu, sum);
  if (lane == 0) sh.wsum[warp] = sum;
  if (tid == 0) {
    for (int i = 0; i < 8; ++i) {
      tc::mbar_init(&sh.full[i], 1);
      tc::mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sh.s_full[i], 1);
      tc::mbar_init(&sh.s_empty[i], 4);
      tc::mbar_init(&sh.p_full[i], 128);
      tc::mbar_init(&sh.o_full[i], 1);
      tc::mbar_init(&sh.o_empty[i], 4);
      tc::mbar_init(&sh.q_full[i], 64);
      tc::mbar_init(&sh.q_empty[i], 1 + 8);
      sh.nan_any[i] = 0;
    }
    sh.abort_flag = 0;
    tc::fence_mbar_init();
    tc::prefetch_tensormap(&map_k);
    if (!W) tc::prefetch_tensormap(&map_v);
  }
  if (tid < 256) sh.nan_at[tid >> 7][tid & 127] = kNever;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) total += sh.wsum[i];
  // (every CTA below n has a tile: the CTAs between a unit's first and last have all written)
  const int n = min((int)gridDim.x, total), cta = (int)blockIdx.x;
  if (cta >= n) return;
  const int t0 = (int)((long)total * cta / n), t1 = (int)((long)total * (cta + 1) / n);
  __syncthreads();
  for (int b0 = 0, run = 0; b0 < a.batch; b0 += kThreads) {
    const int b = b0 + tid;
    const int nb = b < a.batch ? tiles_of(len_of(a, b)) * units_b : 0;
    int x = nb;
#pragma unroll
    for (int h = 1; h < 32; h <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, x, h);
      if (lane >= h) x += y;
    }
    if (lane == 31) sh.wsum[warp] = x;
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (i < warp) x += sh.wsum[i];
      all += sh.wsum[i];
    }
    if (run + x > t0 && run + x - nb <= t0) {
      sh.start_b = b;
      sh.start_off = t0 - (run + x - nb);
    }
    run += all;
    __syncthreads();
    if (run > t0) break;
  }
  if (warp == 1) tc::tmem_alloc(&sh.tmem, C::kTmem);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sh.tmem;
  const uint32_t tmem_o = tmem + 2 * C::N;
  volatile int* abort = &sh.abort_flag;
  Walk w;
  walk_begin(w, a, sh.start_b, sh.start_off, t1 - t0);
  const int R = a.Hq / a.G, rows = a.n_new * R;
  const long units = (long)a.batch * units_b;
  const Part<D, NR> part(a.part, units);

  if (warp == 0) {
    // ---- TMA: K and V tiles ----
    if (lane == 0) {
      int k = 0;
      for (; w.left > 0; walk_next(w, a), ++k) {
        const int st = k % C::kStages;
        if (k >= C::kStages && !tc::mbar_wait(&sh.empty[st], (uint32_t)((k / C::kStages - 1) & 1), abort, a.status)) {
          if (!*abort) report(a.status, SGQA_ERR_TIMEOUT);
          *abort = 1;
          break;
        }
        uint8_t* dst = sKV + st * C::kStage;
        const int g = w.gu / a.nch, z = w.b * a.T + w.tile * kTok;
        tc::mbar_arrive_expect_tx(&sh.full[st], C::kStage);
        tc::tma_load_3d(dst, &map_k, &sh.full[st], 0, g, z);
        if (!W) tc::tma_load_3d(dst + C::kTile, &map_v, &sh.full[st], 0, g, z);
      }
      // copies in flight land before the CTA leaves (all have, unless a wait ran out)
      for (int j = max(0, k - C::kStages); j < k; ++j) {
        volatile int none = 0;
        tc::mbar_wait(&sh.full[j % C::kStages], (uint32_t)((j / C::kStages) & 1), &none);
      }
    }
  } else if (warp == 1) {
    // ---- MMA ----
    if (lane == 0) {
      constexpr uint32_t id_s = idesc_f8(C::N, false, false), id_o = idesc_f8(C::N, true, true);
      int k = 0, pv = 0, pieces = 0;
      bool ok = true;
      auto issue_pv = [&]() -> bool {
        const int pb = pv & 1, st = pv % C::kStages;
        if (!tc::mbar_wait(&sh.p_full[pb], (uint32_t)((pv >> 1) & 1), abort, a.status)) return false;
        if (pv >= 2 && !tc::mbar_wait(&sh.o_empty[pb], (uint32_t)(((pv >> 1) - 1) & 1), abort, a.status)) return false;
        tc::fence_after_sync();
        const uint8_t* v = sKV + st * C::kStage + C::kTile;
        const uint8_t* p = sP + pb * C::kP;
#pragma unroll
        for (int kk = 0; kk < kTok / 32; ++kk) {
          const uint64_t da = D == 128 ? tc::smem_desc_mnmajor_sw128(v + kk * 32 * D, 1024, 1024)
                                       : smem_desc_mnmajor_sw64_twice(v + kk * 32 * D);
          // P: [16 columns][128 tokens][16 bytes]: 8 tokens are 128 bytes, 16 columns 2048
          mma_f8(tmem_o + (uint32_t)(pb * C::N), da, tc::smem_desc_kmajor_noswz(p + kk * 512, 128, 2048), id_o, kk > 0);
        }
        tc::mma_commit(&sh.empty[st]);
        tc::mma_commit(&sh.o_full[pb]);
        ++pv;
        return true;
      };
      for (; w.left > 0; walk_next(w, a), ++k) {
        const int st = k % C::kStages, sb = k & 1;
        if ((w.first && !tc::mbar_wait(&sh.q_full[w.piece & 1], (uint32_t)((w.piece >> 1) & 1), abort, a.status)) ||
            !tc::mbar_wait(&sh.full[st], (uint32_t)((k / C::kStages) & 1), abort, a.status) ||
            (k >= 2 && !tc::mbar_wait(&sh.s_empty[sb], (uint32_t)(((k >> 1) - 1) & 1), abort, a.status))) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        const uint8_t* kt = sKV + st * C::kStage;
        const uint8_t* q = sQ + (w.piece & 1) * C::kQ;
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk)
          mma_f8(tmem + (uint32_t)(sb * C::N), tc::smem_desc_kmajor(kt + kk * 32, D),
                 tc::smem_desc_kmajor_noswz(q + kk * 256, 128, D * 8), id_s, kk > 0);
        tc::mma_commit(&sh.s_full[sb]);
        if (W) tc::mma_commit(&sh.empty[st]);
        if (walk_last(w)) {
          tc::mma_commit(&sh.q_empty[w.piece & 1]);
          pieces = w.piece + 1;
        }
        if (!W && k > 0 && !(ok = issue_pv())) {
          ++k;
          break;
        }
      }
      if (!W && ok) ok = issue_pv();
      if (!ok) {
        if (!*abort) report(a.status, SGQA_ERR_TIMEOUT);
        *abort = 1;
      }
      // the MMAs in flight end before the CTA leaves
      volatile int none = 0;
      if (k > 0) tc::mbar_wait(&sh.s_full[(k - 1) & 1], (uint32_t)(((k - 1) >> 1) & 1), &none);
      const int freed = W ? k : pv;
      for (int j = max(0, freed - C::kStages); j < freed; ++j)
        tc::mbar_wait(&sh.empty[j % C::kStages], (uint32_t)((j / C::kStages) & 1), &none);
      if (!W && pv > 0) tc::mbar_wait(&sh.o_full[(pv - 1) & 1], (uint32_t)(((pv - 1) >> 1) & 1), &none);
      if (ok && pieces > 0) tc::mbar_wait(&sh.q_empty[(pieces - 1) & 1], (uint32_t)(((pieces - 1) >> 1) & 1), abort);
    }
  } else if (warp < 4) {
    // ---- a unit's rows of q as two E4M3 terms; a warp per row ----
    constexpr int kE = D / 32;
    for (; w.left > 0; walk_next(w, a)) {
      if (!w.first) continue;
      const int pb = w.piece & 1, g = w.gu / a.nch, r0 = (w.gu % a.nch) * a.chunk_rows;
      if (w.piece >= 2) warp_wait(&sh.q_empty[pb], (uint32_t)(((w.piece >> 1) - 1) & 1), abort, a.status);
      uint8_t* dst = sQ + pb * C::kQ;
#pragma unroll 4
      for (int r = warp - 2; r < NR; r += 2) {
        const int gr = r0 + r;
        const bool real = r < a.chunk_rows && gr < rows;
        uint32_t x[kE / 2];
#pragma unroll
        for (int e = 0; e < kE / 2; ++e) x[e] = 0u;
        if (real) {
          const long src = (((long)w.b * a.n_new + gr / R) * a.Hq + (long)g * R + gr % R) * D + lane * kE;
          if constexpr (kE == 4) {
            const uint2 y = __ldg(reinterpret_cast<const uint2*>(a.q + src));
            x[0] = y.x;
            x[1] = y.y;
          } else {
            x[0] = __ldg(reinterpret_cast<const uint32_t*>(a.q + src));
          }
        }
        uint32_t amax = 0u;
#pragma unroll
        for (int e = 0; e < kE / 2; ++e) {
          const uint32_t lo = x[e] & 0x7FFFu, hi = (x[e] >> 16) & 0x7FFFu;
          amax = max(amax, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
        }
        amax = __reduce_max_sync(0xFFFFFFFFu, amax);
        const int ex = c8_exponent(amax << 16);
        const float inv = c8_pow2(-ex);
        uint32_t c1 = 0u, c2 = 0u;
#pragma unroll
        for (int e = 0; e < kE / 2; ++e) {
          const float y0 = bf16_lo(x[e]) * inv, y1 = bf16_hi(x[e]) * inv;
          // an infinity becomes NaN, as which it would end in the scores
          uint32_t t1 = c8_encode2(y0, y1);
          const float2 f = c8_decode2(t1);
          uint32_t t2 = c8_encode2((y0 - f.x) * 16.f, (y1 - f.y) * 16.f);
          if ((x[e] & 0x7F80u) == 0x7F80u) t1 |= 0x7Fu;
          if ((x[e] & 0x7F800000u) == 0x7F800000u) t1 |= 0x7F00u;
          c1 |= t1 << (16 * e);
          c2 |= t2 << (16 * e);
        }
        const int at = (lane * kE / 16) * 128 + lane * kE % 16;
        uint8_t* p1 = dst + (r >> 3) * (D * 8) + (r & 7) * 16 + at;
        uint8_t* p2 = dst + ((NR + r) >> 3) * (D * 8) + (r & 7) * 16 + at;
        if constexpr (kE == 4) {
          *reinterpret_cast<uint32_t*>(p1) = c1;
          *reinterpret_cast<uint32_t*>(p2) = c2;
        } else {
          *reinterpret_cast<uint16_t*>(p1) = (uint16_t)c1;
          *reinterpret_cast<uint16_t*>(p2) = (uint16_t)c2;
        }
        if (lane == 0) {
          sh.fac[pb][r] = c8_pow2(ex) * (kLog2e / sqrtf((float)D));
          sh.lim[pb][r] = real ? w.L - a.n_new + gr / R : -1;
          if (W) sh.lse[pb][r] = real ? a.lse[((long)w.b * a.G + g) * rows + gr] : 0.f;
        }
      }
      tc::fence_proxy_async();
      tc::mbar_arrive(&sh.q_full[pb]);
    }
  } else if (warp < 12) {
    // ---- a thread per token: scores, probabilities ----
    const int wg = (warp >> 2) - 1, q4 = warp & 3, row = q4 * 32 + lane, t = tid & 127;
    const uint32_t lane_base = (uint32_t)(q4 * 32) << 16;
    const uint32_t ts = tmem + lane_base + (uint32_t)(wg * C::N);
    const long nblk = (a.T + a.block - 1) / a.block;
    float l[W ? 1 : NR];
#pragma unroll
    for (int r = 0; r < (W ? 1 : NR); ++r) l[r] = 0.f;
    float m_run = kNegMax;  // row t's, in the group's first threads
    int k = 0;
    for (; w.left > 0; walk_next(w, a), ++k) {
      const int pb = w.piece & 1;
      if (w.first) warp_wait(&sh.q_full[pb], (uint32_t)((w.piece >> 1) & 1), abort, a.status);
      if ((k & 1) == wg) {
        const int u = w.tile * kTok + row, g = w.gu / a.nch;
        const bool live = u < w.L;
        const int vis = w.L - a.n_new;               // tokens up to here are visible to every row
        const bool edge = (w.tile + 1) * kTok - 1 > vis;
        float sk = 0.f;
        int ev = -126;
        if (live) {
          const long si = ((long)w.b * nblk + u / a.block) * a.G + g;
          sk = c8_pow2(c8_scale_exponent(__ldg(a.c.ks + si)));
          if (!W) ev = c8_scale_exponent(__ldg(a.c.vs + si));
        }
        if constexpr (W) {
          const long wi = ((long)w.b * a.G + g) * a.T + u;
          float sum = a.w_in && u < vis ? a.w_in[wi] : 0.f;
          warp_wait(&sh.s_full[wg], (uint32_t)((k >> 1) & 1), abort, a.status);
          tc::fence_after_sync();
          float add = 0.f;
#pragma unroll
          for (int r0 = 0; r0 < NR; r0 += 16) {
            constexpr int kH = NR < 16 ? NR : 16;
            uint32_t c1[16], c2[16];
            tc::tmem_ld16_nowait(ts + r0, c1);
            if constexpr (NR >= 16) tc::tmem_ld16_nowait(ts + NR + r0, c2);
            tc::tmem_wait_ld2(c1, c2);
            if constexpr (NR < 16) {
#pragma unroll
              for (int r = 0; r < kH; ++r) c2[r] = c1[NR + r];
            }
#pragma unroll
            for (int r = 0; r < kH; ++r) {
              const float z = fmaf(__uint_as_float(c2[r]), 0.0625f, __uint_as_float(c1[r])) * sh.fac[pb][r0 + r] * sk;
              const float p = ex2_approx(z - sh.lse[pb][r0 + r]);
              const int lim = sh.lim[pb][r0 + r];
              add += lim >= u ? p : 0.f;
            }
          }
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&sh.s_empty[wg]);
          if (live) a.w_out[wi] = sum + add;
        } else {
          warp_wait(&sh.s_full[wg], (uint32_t)((k >> 1) & 1), abort, a.status);
          tc::fence_after_sync();
          float z[NR];
#pragma unroll
          for (int r0 = 0; r0 < NR; r0 += 16) {
            constexpr int kH = NR < 16 ? NR : 16;
            uint32_t c1[16], c2[16];
            tc::tmem_ld16_nowait(ts + r0, c1);
            if constexpr (NR >= 16) tc::tmem_ld16_nowait(ts + NR + r0, c2);
            tc::tmem_wait_ld2(c1, c2);
            if constexpr (NR < 16) {
#pragma unroll
              for (int r = 0; r < kH; ++r) c2[r] = c1[NR + r];
            }
#pragma unroll
            for (int r = 0; r < kH; ++r)
              z[r0 + r] = fmaf(__uint_as_float(c2[r]), 0.0625f, __uint_as_float(c1[r])) * sh.fac[pb][r0 + r] * sk;
          }
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&sh.s_empty[wg]);
          if (edge) {
#pragma unroll
            for (int r = 0; r < NR; ++r)
              if (u > sh.lim[pb][r]) z[r] = -INFINITY;
          }
          // maxima of the tile; NaN counts for none (it reaches the sums by itself)
          float mine = kNegMax;
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            const float x = warp_max(fmaxf(z[r], kNegMax));
            if (lane == r) mine = x;
          }
          const int we = __reduce_max_sync(0xFFFFFFFFu, ev);
          if (lane < NR) sh.wmax[wg][q4][lane] = mine;
          if (lane == 0) sh.wev[wg][q4] = we;
          group_sync(1 + wg);
          // the P buffer and the tile's numbers two tiles back have been read
          if (k >= 2) warp_wait(&sh.o_empty[wg], (uint32_t)(((k >> 1) - 1) & 1), abort, a.status);
          if (t < NR) {
            const float mt = fmaxf(fmaxf(sh.wmax[wg][0][t], sh.wmax[wg][1][t]), fmaxf(sh.wmax[wg][2][t], sh.wmax[wg][3][t]));
            const float mn = fmaxf(m_run, mt);
            sh.mt[wg][t] = mt;
            sh.ab[wg][t] = make_float2(ex2_approx(m_run - mn), ex2_approx(mt - mn));
            m_run = mn;
          }
          const int et = max(max(sh.wev[wg][0], sh.wev[wg][1]), max(sh.wev[wg][2], sh.wev[wg][3]));
          if (t == 0) sh.e_tile[wg] = et;
          group_sync(1 + wg);
          const float cv = 448.f * c8_pow2(max(-126, ev - et));
          uint8_t* pd = sP + wg * C::kP + row * 16;
#pragma unroll
          for (int r0 = 0; r0 < NR; r0 += 16) {
            constexpr int kH = NR < 16 ? NR : 16;
            uint32_t p1[kH / 4], p2[kH / 4];
#pragma unroll
            for (int r = 0; r < kH; r += 2) {
              float y[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float p = ex2_approx(z[r0 + r + e] - sh.mt[wg][r0 + r + e]);
                const float2 ab = sh.ab[wg][r0 + r + e];
                l[r0 + r + e] = fmaf(l[r0 + r + e], ab.x, p * ab.y);
                y[e] = p * cv;
              }
              const uint32_t t1 = c8_encode2(y[0], y[1]);
              const float2 f = c8_decode2(t1);
              const uint32_t t2 = c8_encode2((y[0] - f.x) * 28.f, (y[1] - f.y) * 28.f);
              if (r & 2) {
                p1[r / 4] |= t1 << 16;
                p2[r / 4] |= t2 << 16;
              } else {
                p1[r / 4] = t1;
                p2[r / 4] = t2;
              }
            }
            if constexpr (NR < 16) {
              *reinterpret_cast<uint4*>(pd) = make_uint4(p1[0], p1[1], p2[0], p2[1]);
            } else {
              *reinterpret_cast<uint4*>(pd + (r0 / 16) * 2048) = make_uint4(p1[0], p1[1], p1[2], p1[3]);
              *reinterpret_cast<uint4*>(pd + ((NR + r0) / 16) * 2048) = make_uint4(p2[0], p2[1], p2[2], p2[3]);
            }
          }
          if (edge) {
            // A zero probability must not meet a NaN code: rows behind the last token become zeros,
            // and a NaN of a token that some row does not see is noted and taken out; the rows that
            // see it get it back at the end.
            warp_wait(&sh.full[k % C::kStages], (uint32_t)((k / C::kStages) & 1), abort, a.status);
            uint8_t* v = sKV + (k % C::kStages) * C::kStage + C::kTile + row * D;
            if (!live) {
#pragma unroll
              for (int c = 0; c < D / 16; ++c) *reinterpret_cast<uint4*>(v + c * 16) = make_uint4(0u, 0u, 0u, 0u);
            } else if (u > vis) {
              for (int c = 0; c < D / 16; ++c) {
                for (int x = 0; x < 16; ++x) {
                  uint8_t* code = v + v_chunk<D>(row, c) * 16 + x;
                  if ((*code & 0x7F) == 0x7F) {
                    *code = 0;
                    atomicMin(&sh.nan_at[pb][c * 16 + x], u);
                    sh.nan_any[pb] = 1;
                  }
                }
              }
            }
          }
          tc::fence_proxy_async();
          tc::mbar_arrive(&sh.p_full[wg]);
        }
      }
      if (walk_last(w)) {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sh.q_empty[pb]);
        if constexpr (!W) {
          // this piece's sums
          const long slot = (long)w.b * units_b + w.gu + blockIdx.x;
          const float s = warp_sums<NR>(l, lane);
          if (lane < NR) part.l(slot)[(wg * 4 + q4) * NR + lane] = s;
          if (t < NR) part.lm(slot)[wg * NR + t] = m_run;
          m_run = kNegMax;
#pragma unroll
          for (int r = 0; r < NR; ++r) l[r] = 0.f;
        }
      }
    }
  } else if (!W) {
    // ---- a thread per head dim: outputs ----
    const int q4 = warp & 3, t = tid & 127;
    const int dim = D == 128 ? t : t & 63, rb = D == 128 ? 0 : (t >> 6) * C::kRowsT;
    const uint32_t to = tmem_o + ((uint32_t)(q4 * 32) << 16) + (uint32_t)rb;
    float o[C::kRowsT];
#pragma unroll
    for (int r = 0; r < C::kRowsT; ++r) o[r] = 0.f;
    float m_run = kNegMax;
    int e_run = -126;
    int first_tile = 0;
    int k = 0;
    for (; w.left > 0; walk_next(w, a), ++k) {
      const int pb = w.piece & 1, sb = k & 1;
      if (w.first) first_tile = w.tile;
      warp_wait(&sh.p_full[sb], (uint32_t)((k >> 1) & 1), abort, a.status);
      const int et = sh.e_tile[sb], en = max(e_run, et);
      if (t < NR) {
        const float mt = sh.mt[sb][t], mn = fmaxf(m_run, mt);
        sh.acc_ab[sb][t] = make_float2(ex2_approx(m_run - mn) * c8_pow2(max(-126, e_run - en)),
                                       ex2_approx(mt - mn) * c8_pow2(max(-126, et - en)) * (1.f / 448.f));
        m_run = mn;
      }
      e_run = en;
      group_sync(3);
      warp_wait(&sh.o_full[sb], (uint32_t)((k >> 1) & 1), abort, a.status);
      tc::fence_after_sync();
#pragma unroll
      for (int r0 = 0; r0 < C::kRowsT; r0 += 16) {
        constexpr int kH = C::kRowsT < 16 ? C::kRowsT : 16;
        uint32_t c1[16], c2[16];
        if constexpr (NR >= 16) {
          // 16 columns of each term (with 8 rows a thread the upper half is not used)
          tc::tmem_ld16_nowait(to + (uint32_t)(sb * C::N + r0), c1);
          tc::tmem_ld16_nowait(to + (uint32_t)(sb * C::N + NR + r0) - (kH < 16 && D == 64 ? (uint32_t)rb : 0u), c2);
        } else {
          tc::tmem_ld16_nowait(to - (uint32_t)rb + (uint32_t)(sb * C::N), c1);
        }
        tc::tmem_wait_ld2(c1, c2);
#pragma unroll
        for (int r = 0; r < kH; ++r) {
          float x1, x2;
          if constexpr (NR >= 16) {
            x1 = __uint_as_float(c1[r]);
            if constexpr (kH < 16) x2 = __uint_as_float(rb ? c2[kH + r] : c2[r]);
            else x2 = __uint_as_float(c2[r]);
          } else if constexpr (D == 128) {
            x1 = __uint_as_float(c1[r]);
            x2 = __uint_as_float(c1[NR + r]);
          } else {
            x1 = __uint_as_float(rb ? c1[C::kRowsT + r] : c1[r]);
            x2 = __uint_as_float(rb ? c1[NR + C::kRowsT + r] : c1[NR + r]);
          }
          const float2 ab = sh.acc_ab[sb][rb + r0 + r];
          o[r0 + r] = fmaf(o[r0 + r], ab.x, fmaf(x2, 1.f / 28.f, x1) * ab.y);
        }
      }
      tc::fence_before_sync();
      const bool last = walk_last(w);
      const long unit = (long)w.b * units_b + w.gu, slot = unit + blockIdx.x;
      if (last) {
        if (sh.nan_any[pb]) {
          const int np = sh.nan_at[pb][dim], r0 = (w.gu % a.nch) * a.chunk_rows + rb;
#pragma unroll
          for (int r = 0; r < C::kRowsT; ++r)
            if (np <= w.L - a.n_new + (r0 + r) / R) o[r] = __int_as_float(0x7FC00000);
        }
        group_sync(3);
        sh.nan_at[pb][t] = kNever;
        if (t == 0) sh.nan_any[pb] = 0;
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sh.o_empty[sb]);
      if (last) {
        float* po = part.o(slot) + rb * D + dim;
#pragma unroll
        for (int r = 0; r < C::kRowsT; ++r) {
          po[r * D] = o[r];
          o[r] = 0.f;
        }
        if (t < NR) part.m(slot)[t] = m_run;
        if (t == 0) {
          *part.e(slot) = e_run;
          if (first_tile == 0) part.first[unit] = (int)blockIdx.x;
          if (w.tile + 1 == w.ntiles) part.last[unit] = (int)blockIdx.x;
        }
        m_run = kNegMax;
        e_run = -126;
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, C::kTmem);
  }
}

// Joins the pieces of a unit in the order of their tiles: a CTA per (sequence, group, row), a thread
// per head dim.
template <int D, int NR>
__global__ void __launch_bounds__(D) cache8_join_kernel(C8AttendArgs a) {
  if (tc::grid_timed_out(a.status)) return;
  const int R = a.Hq / a.G, rows = a.n_new * R;
  const int gr = blockIdx.x % rows, bg = blockIdx.x / rows, b = bg / a.G, g = bg % a.G;
  const int r = gr % a.chunk_rows, t = threadIdx.x;
  const long unit = (long)bg * a.nch + gr / a.chunk_rows;
  const int L = len_of(a, b);
  const Part<D, NR> part(a.part, (long)a.batch * a.G * a.nch);
  float den = 0.f, num = 0.f, m = kNegMax;
  int e = -126;
  if (L > a.n_new - 1 - gr / R) {
    const int c0 = part.first[unit], c1 = part.last[unit];
    for (int c = c0; c <= c1; ++c) {
      m = fmaxf(m, part.m(unit + c)[r]);
      e = max(e, *part.e(unit + c));
    }
    for (int c = c0; c <= c1; ++c) {
      const long slot = unit + c;
      const float f = ex2_approx(part.m(slot)[r] - m) * c8_pow2(max(-126, *part.e(slot) - e));
      num = fmaf(part.o(slot)[r * D + t], f, num);
#pragma unroll
      for (int wg = 0; wg < 2; ++wg) {
        const float* l = part.l(slot) + wg * 4 * NR + r;
        den = fmaf((l[0] + l[NR]) + (l[2 * NR] + l[3 * NR]), ex2_approx(part.lm(slot)[wg * NR + r] - m), den);
      }
    }
  }
  const long at = (((long)b * a.n_new + gr / R) * a.Hq + (long)g * R + gr % R) * D + t;
  const float y = den == 0.f ? 0.f : num / den * c8_pow2(e);
  a.out[at] = f32_to_bf16_rne(y * sigmoid_fast(bf16_to_f32(__ldg(a.gate + at))));
  if (t == 0 && a.w_out) a.lse[(long)bg * rows + gr] = den == 0.f ? 0.f : m + log2f(den);
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled get_encode() {
  static EncodeTiled fn = nullptr;
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiled>(p);
  }
  return fn;
}
// [batch * T tokens][G][d] codes, box = one group's codes of 128 tokens; zeros behind the last token
bool make_map(CUtensorMap* map, const void* base, long tokens, int G, int d) {
  EncodeTiled enc = get_encode();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)G, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)d, (cuuint64_t)G * d};
  const cuuint32_t box[3] = {(cuuint32_t)d, 1, kTok};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int NR, bool W>
cudaError_t launch_main(const CUtensorMap& mk, const CUtensorMap& mv, C8AttendArgs a, int nch, int chunk_rows,
                        cudaStream_t s) {
  using C = Cfg<D, NR, W>;
  constexpr int kSmem = C::kStages * C::kStage + 2 * C::kQ + 2 * C::kP + 1024;
  cudaError_t e = cudaFuncSetAttribute(cache8_attend_kernel<D, NR, W>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  a.nch = nch;
  a.chunk_rows = chunk_rows;
  const long tiles = (long)a.batch * a.G * nch * ((a.T + kTok - 1) / kTok);
  const unsigned grid = (unsigned)(tiles < kGridMax ? tiles : kGridMax);
  cache8_attend_kernel<D, NR, W><<<grid, kThreads, kSmem, s>>>(mk, mv, a);
  return cudaGetLastError();
}

// rows of a unit: all of a (sequence, group), or halves of them
struct Rows {
  int nch, chunk_rows, nr;
};
Rows rows_of(int rows) {
  const int nch = (rows + kMaxNR - 1) / kMaxNR, c = (rows + nch - 1) / nch;
  return {nch, c, c <= 8 ? 8 : c <= 16 ? 16 : 32};
}

template <int D, int NR>
cudaError_t launch_rows(const CUtensorMap& mk, const CUtensorMap& mv, C8AttendArgs a, const Rows& rw, cudaStream_t s) {
  cudaError_t e = launch_main<D, NR, false>(mk, mv, a, rw.nch, rw.chunk_rows, s);
  if (e != cudaSuccess) return e;
  a.nch = rw.nch;
  a.chunk_rows = rw.chunk_rows;
  const int rows = a.n_new * (a.Hq / a.G);
  const long ctas = (long)a.batch * a.G * rows;
  if (ctas > 0x7FFFFFFFL) return cudaErrorInvalidConfiguration;
  cache8_join_kernel<D, NR><<<(unsigned)ctas, D, 0, s>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess || !a.w_out) return e;
  return rw.nch == 1 ? launch_main<D, NR, true>(mk, mv, a, 1, rows, s) : launch_main<D, 64, true>(mk, mv, a, 1, rows, s);
}
template <int D>
cudaError_t launch_d(const C8AttendArgs& a, cudaStream_t s) {
  CUtensorMap mk, mv;
  const long tokens = (long)a.batch * a.T;
  if (!make_map(&mk, a.c.k8, tokens, a.G, D) || !make_map(&mv, a.c.v8, tokens, a.G, D)) return cudaErrorInvalidValue;
  const Rows rw = rows_of(a.n_new * (a.Hq / a.G));
  switch (rw.nr) {
    case 8: return launch_rows<D, 8>(mk, mv, a, rw, s);
    case 16: return launch_rows<D, 16>(mk, mv, a, rw, s);
    default: return launch_rows<D, 32>(mk, mv, a, rw, s);
  }
}

}  // namespace

size_t cache8_part_bytes(int batch, int G, int rows, int d) {
  const Rows rw = rows_of(rows);
  const long units = (long)batch * G * rw.nch;
  const long rec = (long)rw.nr * d + rw.nr * 11 + 4;
  return (size_t)(2 * ((units + 3) & ~3L) + (units + kGridMax) * rec) * 4;
}

cudaError_t launch_cache8_attend(const C8AttendArgs& a, cudaStream_t s) {
  return a.d == 64 ? launch_d<64>(a, s) : launch_d<128>(a, s);
}

}  // namespace sgqa
