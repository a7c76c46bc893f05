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
// Two E4M3 terms hold q exactly down to 2^-14 of its row's largest element and p t to 1/289 of itself
// or, where they are subnormal, 2^-23 of 2^E. 2^E is at most 16 times the row's own largest p t of the
// tile: where the V scales of a tile's blocks are within 2^kSpread of one another it is the tile's largest,
// against the row's largest p; else a further pass over the scores finds every row's own, since a block of
// a far larger scale that the row does not see, or hardly, would take the digits of the others. P and E
// belong to one tile, so O^T starts anew in every tile and is added up in registers in fp32: a token that
// takes nearly all attention costs the far ones none of their digits. The denominator and the maxima are
// taken from fp32 scores.
//
// Work: the tiles of 128 tokens of all (sequence, group) units, in that order, cut into one equal
// contiguous piece per CTA (one CTA per SM), so that ragged lengths, one long sequence and many
// short ones all balance; the lengths are read on the device. A unit's pieces leave partial sums,
// which a second kernel joins in the order of the tiles.
// Roles: warp 0 issues TMA loads, warp 1 the MMAs of S^T, warp 2 those of O^T, warp 3 keeps the rows'
// running maxima and sums, then come two or three groups of four warps that take tiles in turn from
// S^T to P, and four warps (a thread per head dim) that add O^T up and split the next unit's rows of
// q. Waits are bounded as everywhere (tc_common.cuh): after one has run out nobody waits any more, and
// the roles run through their tiles to the end.
// S^T is read in the 16x256b shape: a lane holds NR / 4 rows of 4 tokens (q's rows are placed so that
// both terms of a row and pairs of rows land in one lane), so that row factors take NR / 4 registers,
// maxima and sums over tokens start inside the thread, and products run on packed pairs.
// The received weights need each row's final sum: a further pass over K recomputes the scores, from
// the last tile to the first, so that it finds in L2 what the first pass has read last.
//
// Measured (B200, inputs changing from pass to pass): 32 sequences of up to 32K tokens, 8 rows a group
// (762 MB): 128 us a call, 121 on the device, at 97% of a copy's rate. 1M tokens, 4 groups of 32 rows
// (1.07 GB): 194 us on the device on a cool GPU, 240 us a call in a long run, where the SM clock falls to
// 1.67 GHz under the power cap (4.5 TB/s): the 32 rows take 1100 to 1250 cycles a tile, the accumulating
// warps first (96 registers for every role, with 92 bytes spilled at d 128). With weights, 8 sequences of
// 64K (454 MB and K again): 118 us, of which 70 the first kernel and 32 the pass over K, a third of it from
// L2. Small calls are launches, one chain of cold loads and instruction fetch: 8 us on the device for 1900
// tokens. More than 32 rows make two units, which read K and V once each.
// Not taken: two terms added up in one column of S^T or O^T (the second would need its scale inside the
// MMA), a maximum carried over from earlier tiles (loses the digits above), converting to fp16 (0.4
// us of a tile's 0.75 for the conversions alone, and twice the shared memory).
#include <cuda.h>

#include "cache8.cuh"
#include "tc_common.cuh"

namespace sgqa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegMax = -3.4028234663852886e38f;  // maximum of a row that no token has reached
constexpr int kTok = 128;                           // tokens per tile
constexpr int kGridMax = 148;                       // one CTA per SM
constexpr int kMaxNR = 32;                          // rows per unit; more make several units
constexpr int kNever = 0x7FFFFFFF;
constexpr int kSpread = 4;  // of a tile's V exponents, up to which its rows share a reference

template <int D, int NR, bool W>
struct Cfg {
  static constexpr int N = 2 * NR;                       // MMA columns: both terms of every row
  static constexpr int kTile = kTok * D;
  static constexpr int kStage = W ? kTile : 2 * kTile;   // K, then V
  static constexpr int kStages = D == 64 || W ? 8 : 5;
  static constexpr int kQ = N * D;
  static constexpr int kP = W ? 0 : kTok * N;
  // Softmax groups of four warps, each with a buffer of S^T, P and O^T of its own. Two keep up with
  // HBM where a tile is 32 KB and has up to 16 rows; 32 rows took 1350 cycles a tile with two, and
  // tiles of 16 KB (5000 tokens, 15 rows) 22 us a call instead of 18.
  static constexpr int kGroups = W || D == 64 || NR == 32 ? 3 : 2;
  static constexpr int kThreads = 128 + 128 * kGroups + (W ? 0 : 128);
  static constexpr int kTmemUsed = (W ? 1 : 2) * kGroups * N;
  static constexpr int kTmem = kTmemUsed <= 64 ? 64 : kTmemUsed <= 128 ? 128 : kTmemUsed <= 256 ? 256 : 512;
  // Warps that split q, and that fetch tiles: the weights' pass reads half as much a tile, and one warp
  // needed 0.35 us for each.
  static constexpr int kQWarps = W ? 4 * kGroups : 4, kFetch = W ? 2 : 1;
  static constexpr int kRowsT = D == 128 ? NR : NR / 2;  // rows per accumulating thread
  static constexpr int q = NR / 4;                       // rows per lane of the softmax warps
};

constexpr int kMaxGroups = 3;
// Where a CTA's tiles begin (the weights' pass: end): unit and tile, and how many there are (0: none).
struct Start {
  int b, g, ch, L, ntiles, tile, left;
};
template <int NR>
struct Shared {
  uint64_t full[8], empty[8];
  uint64_t s_full[kMaxGroups], s_empty[kMaxGroups], p_full[kMaxGroups], o_full[kMaxGroups], o_empty[kMaxGroups];
  uint64_t f_full[kMaxGroups], q_full[2], q_empty[2];
  float scale[8][32];                      // per stage: K scales of the tile's blocks, then V scales
  uint32_t tmem;
  volatile int abort_flag;
  Start start;
  int wsum[32], wmore[32];
  // per unit modulo the groups (the softmax warps can be that many units ahead of the accumulating ones):
  int nan_any[kMaxGroups];
  int nan_at[kMaxGroups][128];             // per head dim: first token not visible to all rows whose V is NaN there
  int2 wev[kMaxGroups][4];  // per softmax group and warp: largest and smallest V exponent of its tokens
  alignas(16) float fac[2][NR];            // per unit parity: 2^e log2 e / sqrt(d) of a row
  float lse[2][NR];
  int lim[2][NR];                          // a row's own position; -1: no row
  alignas(16) float wmax[kMaxGroups][4][NR];    // per softmax group and warp: a row's maximum over the tile
  alignas(16) float wsum_p[kMaxGroups][4][NR];  // and the sum of its probabilities
  // where V's exponents differ: a row's largest score (less the row's maximum) plus V exponent, and over the group
  alignas(16) float wref[kMaxGroups][4][NR];
  int ref[kMaxGroups][NR];
  // per softmax group, for the accumulating warps: factors of the sums so far, and whether any is not 1;
  // of this tile's first (x, y) and second (z, w) terms for pairs of rows
  alignas(16) float fa[kMaxGroups][NR];
  int any_fa[kMaxGroups];
  float4 fb[kMaxGroups][NR / 2];
};

__device__ __forceinline__ int warp_scan(int x, int lane) {
#pragma unroll
  for (int h = 1; h < 32; h <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, x, h);
    if (lane >= h) x += y;
  }
  return x;
}

// The tiles of one CTA in order, a piece of a unit at a time: tiles [t0, t1) of unit ((sequence b,
// group g), chunk ch of its rows). A loop over a piece's tiles has nothing else to keep track of: with
// four roles on every scheduler, instruction fetch is what short loops are for. The weights' pass goes
// from the last tile to the first, for K tiles that the first pass has left in L2.
struct Walk {
  int b, g, ch, L, ntiles, t0, t1, left;  // left: tiles of this and later pieces
  int piece, k;                           // pieces and tiles of this CTA before
};
__device__ __forceinline__ int tiles_of(int L) { return (L + kTok - 1) / kTok; }
__device__ __forceinline__ int len_of(const C8AttendArgs& a, int b) {
  const int n = __ldg(a.lens + b);
  return n >= 0 && n <= a.T ? n : 0;
}
template <bool BACK>
__device__ __forceinline__ void walk_begin(Walk& w, const Start& s) {
  w.b = s.b;
  w.g = s.g;
  w.ch = s.ch;
  w.L = s.L;
  w.ntiles = s.ntiles;
  w.left = s.left;
  w.t0 = BACK ? max(0, s.tile + 1 - s.left) : s.tile;
  w.t1 = BACK ? s.tile + 1 : min(s.ntiles, s.tile + s.left);
  w.piece = w.k = 0;
}
// This CTA's share of `total` tiles: [t0, t0 + left). Every CTA below min(CTAs, tiles) has one: the CTAs
// between a unit's first and last have all written.
__device__ __forceinline__ int share_of(int total, int& t0) {
  const int n = min((int)gridDim.x, total), cta = (int)blockIdx.x;
  if (cta >= n) return 0;
  const int each = total / n, odd = total - each * n;
  t0 = each * cta + min(cta, odd);
  return each + (cta < odd ? 1 : 0);
}
// off: the tile's place among those of sequence b
__device__ __forceinline__ void set_start(Start& s, const C8AttendArgs& a, int b, int L, int off, int left) {
  s.b = b;
  s.L = L;
  s.ntiles = tiles_of(L);
  const int gu = off / s.ntiles;
  s.tile = off - gu * s.ntiles;
  s.g = a.nch == 1 ? gu : gu / a.nch;
  s.ch = gu - s.g * a.nch;
  s.left = left;
}
// The start, found by one warp from up to 256 lengths. (Short loops: this runs once, from a cold
// instruction cache, and everything waits for it.)
constexpr int kWarpLens = 256;
template <bool BACK>
__device__ __forceinline__ void warp_start(Start& s, const C8AttendArgs& a, int lane) {
  const int units_b = a.G * a.nch;
  int total = 0;
  const bool stopped = tc::grid_timed_out(a.status);
#pragma unroll 1
  for (int b = lane; b < a.batch; b += 32) total += tiles_of(c8_len(a.lens, b, a.T, a.status));
  total = __reduce_add_sync(0xFFFFFFFFu, total) * units_b;
  int t0 = 0;
  const int left = __any_sync(0xFFFFFFFFu, stopped) ? 0 : share_of(total, t0);
  if (left == 0) {
    if (lane == 0) s.left = 0;
    return;
  }
  const int from = BACK ? t0 + left - 1 : t0;
#pragma unroll 1
  for (int b = lane, seen = 0;; b += 32) {
    const int L = b < a.batch ? len_of(a, b) : 0, n = tiles_of(L) * units_b;
    int x = n;
#pragma unroll 1
    for (int h = 1; h < 32; h <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, x, h);
      if (lane >= h) x += y;
    }
    x += seen;
    if (x > from && x - n <= from) set_start(s, a, b, L, from - (x - n), left);
    seen = __shfl_sync(0xFFFFFFFFu, x, 31);
    if (seen > from) break;
  }
}
// The start from any number of lengths: all threads of the CTA.
template <int THREADS, bool BACK, class SH>
__device__ __forceinline__ void block_start(SH& sh, const C8AttendArgs& a, int tid) {
  const int warp = tid >> 5, lane = tid & 31;
  if (tid == 0) sh.wmore[31] = tc::grid_timed_out(a.status);
  int mine = 0;
  for (int b = tid; b < a.batch; b += THREADS) mine += tiles_of(c8_len(a.lens, b, a.T, a.status)) * a.G * a.nch;
  mine = __reduce_add_sync(0xFFFFFFFFu, mine);
  if (lane == 0) sh.wmore[warp] = mine;
  __syncthreads();
  int total = 0, t0 = 0;
  for (int i = 0; i < THREADS / 32; ++i) total += sh.wmore[i];
  const int left = sh.wmore[31] ? 0 : share_of(total, t0), from = BACK ? t0 + left - 1 : t0;
  if (left == 0) {
    if (tid == 0) sh.start.left = 0;
    return;
  }
  for (int b0 = 0, seen = 0; seen <= from; b0 += THREADS) {
    const int b = b0 + tid, L = b < a.batch ? len_of(a, b) : 0, n = tiles_of(L) * a.G * a.nch;
    int x = warp_scan(n, lane);
    __syncthreads();
    if (lane == 31) sh.wsum[warp] = x;
    __syncthreads();
    x += seen;
    for (int i = 0; i < THREADS / 32; ++i) {
      if (i < warp) x += sh.wsum[i];
      seen += sh.wsum[i];
    }
    if (x > from && x - n <= from) set_start(sh.start, a, b, L, from - (x - n), left);
  }
}
template <bool BACK>
__device__ __forceinline__ void walk_next(Walk& w, const C8AttendArgs& a) {
  w.left -= w.t1 - w.t0;
  w.k += w.t1 - w.t0;
  ++w.piece;
  if (w.left == 0) return;
  w.ch += BACK ? -1 : 1;
  if (w.ch < 0 || w.ch == a.nch) {
    w.ch = BACK ? a.nch - 1 : 0;
    w.g += BACK ? -1 : 1;
    if (w.g < 0 || w.g == a.G) {
      w.g = BACK ? a.G - 1 : 0;
      do {
        w.b += BACK ? -1 : 1;
        w.L = len_of(a, w.b);
      } while (w.L == 0);
      w.ntiles = tiles_of(w.L);
    }
  }
  w.t0 = BACK ? max(0, w.ntiles - w.left) : 0;
  w.t1 = BACK ? w.ntiles : min(w.ntiles, w.left);
}
template <bool BACK>
__device__ __forceinline__ int walk_tile(const Walk& w, int x) { return BACK ? w.t1 - 1 - x : w.t0 + x; }

// Per launch: partial sums of every piece, and the CTAs that hold a unit's first and last tile.
template <int D, int NR>
struct Part {
  static constexpr long kRec = (long)NR * D + NR * 3;  // O; M, l, E
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
  __device__ float* l(long slot) const { return base + slot * kRec + NR * D + NR; }
  __device__ int* e(long slot) const { return reinterpret_cast<int*>(base + slot * kRec + NR * D + 2 * NR); }
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
// 8 q columns of the warp's 32 TMEM lanes, as matrix fragments: c[16 h + ...]: lane / 4 + 8 e + 16 h is
// the token, 8 j + 2 (lane % 4) + x the column of c[4 q h + 4 j + 2 e + x].
template <int Q>
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&c)[8 * Q]);
template <>
__device__ __forceinline__ void tmem_ld_frag<2>(uint32_t taddr, uint32_t (&c)[16]) {
  asm volatile(
      "{ .reg .b32 t; add.u32 t, %16, 0x100000;\n"
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%16];\n"
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%8,%9,%10,%11,%12,%13,%14,%15}, [t];\n"
      "tcgen05.wait::ld.sync.aligned; }"
      : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3]), "=r"(c[4]), "=r"(c[5]), "=r"(c[6]), "=r"(c[7]), "=r"(c[8]), "=r"(c[9]), "=r"(c[10]), "=r"(c[11]), "=r"(c[12]), "=r"(c[13]), "=r"(c[14]), "=r"(c[15])
      : "r"(taddr)
      : "memory");
}
template <>
__device__ __forceinline__ void tmem_ld_frag<4>(uint32_t taddr, uint32_t (&c)[32]) {
  asm volatile(
      "{ .reg .b32 t; add.u32 t, %32, 0x100000;\n"
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n"
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [t];\n"
      "tcgen05.wait::ld.sync.aligned; }"
      : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3]), "=r"(c[4]), "=r"(c[5]), "=r"(c[6]), "=r"(c[7]), "=r"(c[8]), "=r"(c[9]), "=r"(c[10]), "=r"(c[11]), "=r"(c[12]), "=r"(c[13]), "=r"(c[14]), "=r"(c[15]), "=r"(c[16]), "=r"(c[17]), "=r"(c[18]), "=r"(c[19]), "=r"(c[20]), "=r"(c[21]), "=r"(c[22]), "=r"(c[23]), "=r"(c[24]), "=r"(c[25]), "=r"(c[26]), "=r"(c[27]), "=r"(c[28]), "=r"(c[29]), "=r"(c[30]), "=r"(c[31])
      : "r"(taddr)
      : "memory");
}
template <>
__device__ __forceinline__ void tmem_ld_frag<8>(uint32_t taddr, uint32_t (&c)[64]) {
  asm volatile(
      "{ .reg .b32 t; add.u32 t, %64, 0x100000;\n"
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%64];\n"
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [t];\n"
      "tcgen05.wait::ld.sync.aligned; }"
      : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3]), "=r"(c[4]), "=r"(c[5]), "=r"(c[6]), "=r"(c[7]), "=r"(c[8]), "=r"(c[9]), "=r"(c[10]), "=r"(c[11]), "=r"(c[12]), "=r"(c[13]), "=r"(c[14]), "=r"(c[15]), "=r"(c[16]), "=r"(c[17]), "=r"(c[18]), "=r"(c[19]), "=r"(c[20]), "=r"(c[21]), "=r"(c[22]), "=r"(c[23]), "=r"(c[24]), "=r"(c[25]), "=r"(c[26]), "=r"(c[27]), "=r"(c[28]), "=r"(c[29]), "=r"(c[30]), "=r"(c[31]), "=r"(c[32]), "=r"(c[33]), "=r"(c[34]), "=r"(c[35]), "=r"(c[36]), "=r"(c[37]), "=r"(c[38]), "=r"(c[39]), "=r"(c[40]), "=r"(c[41]), "=r"(c[42]), "=r"(c[43]), "=r"(c[44]), "=r"(c[45]), "=r"(c[46]), "=r"(c[47]), "=r"(c[48]), "=r"(c[49]), "=r"(c[50]), "=r"(c[51]), "=r"(c[52]), "=r"(c[53]), "=r"(c[54]), "=r"(c[55]), "=r"(c[56]), "=r"(c[57]), "=r"(c[58]), "=r"(c[59]), "=r"(c[60]), "=r"(c[61]), "=r"(c[62]), "=r"(c[63])
      : "r"(taddr)
      : "memory");
}

// the largest; NaN only if all are
__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}
__device__ __forceinline__ uint64_t evict_first_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void tma_load_3d_once(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z,
                                                 uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%3, %4, "
      "%5}], [%2], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "l"(policy)
      : "memory");
}
// True in one lane of the warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.b32 %0, 1, 0, p; }" : "=r"(p));
  return p != 0;
}
// pairs of fp32
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// A 4-byte copy to shared memory, and an arrival once this thread's copies so far have landed.
__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ void group_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }

// A warp's wait. After a wait has run out none waits any longer, but the roles go on through their
// tiles (with whatever is in the buffers), so that no group's barrier is left short of a warp.
__device__ __noinline__ void slow_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int* status) {
  if (*abort || tc::mbar_wait(bar, parity, abort, status)) return;
  if (!*abort) report(status, SGQA_ERR_TIMEOUT);
  *abort = 1;
}
__device__ __forceinline__ void warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int* status) {
  if (!tc::mbar_try_wait(bar, parity)) slow_wait(bar, parity, abort, status);
  __syncwarp();
}

// Exponents (largest, smallest) of V over a tile, from those of a group's warps.
__device__ __forceinline__ int2 spread_of(const int2 (&w)[4]) {
  return make_int2(max(max(w[0].x, w[1].x), max(w[2].x, w[3].x)), min(min(w[0].y, w[1].y), min(w[2].y, w[3].y)));
}
// A row's sums are held in units of 2^(m + e): m its largest score so far, e an integer with 2^(m + e) at least
// the references of what it holds. x: such a sum of m and e, less the new m.
__device__ __forceinline__ int ref_of(float x) { return max(-126, __float2int_ru(x)); }

// x[j] over the eight lanes that share rows (lane / 4), joined by op in a fixed order; the lane gets
// row (lane / 4) mod Q.
template <int Q, class Op>
__device__ __forceinline__ float across_tokens(float (&x)[Q], int lane, Op op) {
#pragma unroll
  for (int h = Q / 2; h >= 1; h >>= 1) {
    const bool up = lane & (4 * h);
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const float give = up ? x[i] : x[i + h], have = up ? x[i + h] : x[i];
      x[i] = op(have, __shfl_xor_sync(0xFFFFFFFFu, give, 4 * h));
    }
  }
  float y = x[0];
#pragma unroll
  for (int h = Q; h < 8; h <<= 1) y = op(y, __shfl_xor_sync(0xFFFFFFFFu, y, 4 * h));
  return y;
}

// A token's V codes of a tile, as TMA's swizzle has laid them out.
template <int D>
__device__ __forceinline__ int v_chunk(int row, int c) {
  return D == 128 ? c ^ (row & 7) : c ^ ((row >> 1) & 3);
}

// A unit's rows of q as two E4M3 terms, and what else a row needs: warp `first` of `warps`, D / 16 lanes
// to a row, 16 dims a lane. (A loop of little code: it runs once per unit, mostly from a cold
// instruction cache; with eight rows unrolled it took 9 us.)
template <int D, int NR, bool W>
__device__ __forceinline__ void split_q(const C8AttendArgs& a, const Walk& w, Shared<NR>& sh, uint8_t* sQ, int first,
                                        int warps, int lane) {
  using C = Cfg<D, NR, W>;
  constexpr int kLanes = D / 16, kRows = 32 / kLanes;
  const int R = a.Hq / a.G, rows = a.n_new * R;
  const int pb = w.piece & 1, r0 = w.ch * a.chunk_rows, real = min(a.chunk_rows, rows - r0);
  const int chunk = lane % kLanes;
  uint8_t* dst = sQ + pb * C::kQ + chunk * 128;
#pragma unroll 1
  for (int r = first * kRows + lane / kLanes; r < NR; r += warps * kRows) {
    const int gr = r0 + r, i = gr / R;
    uint4 x[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
    float lse = INFINITY;  // no row: 2^-inf
    if (r < real && SGQA_CHECK(w.b < a.batch && w.g < a.G && gr < rows, a.status)) {
      const uint4* src = reinterpret_cast<const uint4*>(
          a.q + (((long)w.b * a.n_new + i) * a.Hq + (long)w.g * R + gr - i * R) * D + chunk * 16);
      x[0] = __ldg(src);
      x[1] = __ldg(src + 1);
      if (W) lse = a.lse[((long)w.b * a.G + w.g) * rows + gr];
    }
    const uint32_t y[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
    uint32_t amax = 0u;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t lo = y[e] & 0x7FFFu, hi = (y[e] >> 16) & 0x7FFFu;
      amax = max(amax, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
    }
#pragma unroll
    for (int h = 1; h < kLanes; h <<= 1) amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, h));
    const int ex = c8_exponent(amax << 16);
    const float inv = c8_pow2(-ex);
    uint32_t c1[4], c2[4];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float y0 = bf16_lo(y[e]) * inv, y1 = bf16_hi(y[e]) * inv;
      uint32_t t1 = c8_encode2(y0, y1);
      const float2 f = c8_decode2(t1);
      const uint32_t t2 = c8_encode2((y0 - f.x) * 16.f, (y1 - f.y) * 16.f);
      // an infinity becomes NaN, as which it would end in the scores
      if ((y[e] & 0x7F80u) == 0x7F80u) t1 |= 0x7Fu;
      if ((y[e] & 0x7F800000u) == 0x7F800000u) t1 |= 0x7F00u;
      c1[e / 2] = e & 1 ? c1[e / 2] | (t1 << 16) : t1;
      c2[e / 2] = e & 1 ? c2[e / 2] | (t2 << 16) : t2;
    }
    // columns 8 j + 2 i + x of S^T: row i q + (j / 2) 2 + x, term j % 2
    const int jj = r % C::q, n1 = 16 * (jj >> 1) + 2 * (r / C::q) + (jj & 1), n2 = n1 + 8;
    *reinterpret_cast<uint4*>(dst + (n1 >> 3) * (D * 8) + (n1 & 7) * 16) = make_uint4(c1[0], c1[1], c1[2], c1[3]);
    *reinterpret_cast<uint4*>(dst + (n2 >> 3) * (D * 8) + (n2 & 7) * 16) = make_uint4(c2[0], c2[1], c2[2], c2[3]);
    if (chunk == 0) {
      sh.fac[pb][r] = c8_pow2(ex) * (kLog2e / sqrtf((float)D));
      sh.lim[pb][r] = r < real ? w.L - a.n_new + i : -1;
      if (W) sh.lse[pb][r] = lse;
    }
  }
  __syncwarp();
  tc::fence_proxy_async();
}

// One of the kQWarps warps that split q: its rows of the piece w.
template <int D, int NR, bool W>
__device__ __forceinline__ void split_piece(const C8AttendArgs& a, const Walk& w, Shared<NR>& sh, uint8_t* sQ, int first,
                                            volatile int* abort, int lane) {
  const int pb = w.piece & 1;
  if (w.piece >= 2) warp_wait(&sh.q_empty[pb], (uint32_t)(((w.piece >> 1) - 1) & 1), abort, a.status);
  split_q<D, NR, W>(a, w, sh, sQ, first, Cfg<D, NR, W>::kQWarps, lane);
  tc::mbar_arrive(&sh.q_full[pb]);
}
template <int D, int NR, bool W>
__global__ void __launch_bounds__(Cfg<D, NR, W>::kThreads, 1)
    cache8_attend_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                         const C8AttendArgs a) {
  using C = Cfg<D, NR, W>;
  constexpr int kThreads = C::kThreads, kGroups = C::kGroups;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared<NR> sh;
  uint8_t* sKV = smem_align<1024>(smem_raw);
  uint8_t* sQ = sKV + C::kStages * C::kStage;
  uint8_t* sP = sQ + 2 * C::kQ;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int units_b = a.G * a.nch;

  grid_dependents();  // (the kernels behind wait for this one's end where they need it)
  // ---- barriers; this CTA's piece of the tiles ----
  // The first warp makes what it needs by itself and goes on to fetch the first tiles, while the others
  // wait for what it leaves behind. (Lengths of more sequences than a warp reads: all together.)
  if (a.batch > kWarpLens) {
    block_start<kThreads, W>(sh, a, tid);
    __syncthreads();
  }
  if (warp == 0) {
    if (lane < 8) {
      tc::mbar_init(&sh.full[lane], 1 + 32);
      tc::mbar_init(&sh.empty[lane], W ? 1 + 4 : 1);  // the weights' pass reads scales after the MMA
    } else if (lane < 8 + kGroups) {
      const int i = lane - 8;
      tc::mbar_init(&sh.s_full[i], 1);
      tc::mbar_init(&sh.s_empty[i], 4);
      tc::mbar_init(&sh.p_full[i], 128);
      tc::mbar_init(&sh.f_full[i], 32);
      tc::mbar_init(&sh.o_full[i], 1);
      tc::mbar_init(&sh.o_empty[i], 4);
    } else if (lane >= 16 && lane < 18) {
      tc::mbar_init(&sh.q_full[lane - 16], 32 * C::kQWarps);
      tc::mbar_init(&sh.q_empty[lane - 16], 1 + 4 * kGroups);
    } else if (lane == 18) {
      sh.abort_flag = 0;
    }
    tc::fence_mbar_init();
    if (a.batch <= kWarpLens) warp_start<W>(sh.start, a, lane);
    __syncwarp();
    asm volatile("bar.arrive 9, %0;" ::"n"(kThreads) : "memory");
  } else {
    if (warp == 1) tc::tmem_alloc(&sh.tmem, C::kTmem);
    if (tid == 64) {
      tc::prefetch_tensormap(&map_k);
      if (!W) tc::prefetch_tensormap(&map_v);
    }
    if (tid >= 128 && tid < 128 + 128 * kMaxGroups) (&sh.nan_at[0][0])[tid - 128] = kNever;
    if (tid >= 96 && tid < 96 + kMaxGroups) sh.nan_any[tid - 96] = 0;
    tc::fence_before_sync();
    asm volatile("bar.sync 9, %0;" ::"n"(kThreads) : "memory");
    tc::fence_after_sync();
  }
  if (sh.start.left == 0) {
    if (W) grid_wait();  // (no kernel ends before the one it was started behind)
    if (warp == 1) tc::tmem_dealloc(sh.tmem, C::kTmem);
    return;
  }
  const uint32_t tmem = warp == 0 ? 0u : sh.tmem;  // (the first warp may be ahead of its allocation)
  const uint32_t tmem_o = tmem + kGroups * C::N;
  volatile int* abort = &sh.abort_flag;
  Walk w;
  walk_begin<W>(w, sh.start);
  const Part<D, NR> part(a.part, (long)a.batch * units_b);

  // the first piece's rows of q: all warps but those that have tiles to fetch and to multiply
  constexpr int kQFirst = W ? 4 : 4 + 4 * kGroups;  // the warps that split the later pieces' rows
  constexpr int kNoQ = 1 + C::kFetch;
  if (warp >= kNoQ) {
    if (W) grid_wait();  // the rows' sums, and what the weights so far were written by
    split_q<D, NR, W>(a, w, sh, sQ, warp - kNoQ, kThreads / 32 - kNoQ, lane);
    if (warp >= kQFirst && warp < kQFirst + C::kQWarps) {
      asm volatile("bar.sync 8, %0;" ::"n"(kThreads - 32 * kNoQ) : "memory");
      tc::mbar_arrive(&sh.q_full[0]);
    } else {
      asm volatile("bar.arrive 8, %0;" ::"n"(kThreads - 32 * kNoQ) : "memory");
    }
  }
  if (warp == 0 || (C::kFetch == 2 && warp == 2)) {
    // ---- TMA: K and V tiles; a lane per block: their scales ----
    const int me = warp >> 1;
    const int nblk = (a.T + a.block - 1) >> a.block_log2, per = kTok >> a.block_log2;  // (batch * T * G is below 2^31)
    const int part_v = lane >> 4, j = lane & 15;
    const float* scales = part_v ? a.c.vs : a.c.ks;
    const bool mine = j < per && !(W && part_v);
    int issued = 0, st = me;
    uint32_t ph = 1;
    bool stop = (int)blockIdx.x == a.stall_cta - (W ? SGQA_TEST_STALL_WEIGHTS : 0);
    const uint64_t once = evict_first_policy();  // V where K is read again for the weights
    for (; w.left > 0 && !stop; walk_next<W>(w, a)) {
      const int src = (w.b * nblk + j) * a.G + w.g, z = w.b * a.T;
      for (int x = (me + C::kFetch - w.k % C::kFetch) % C::kFetch; x < w.t1 - w.t0; x += C::kFetch) {
        const int tile = walk_tile<W>(w, x);
        // (a tile that is none reads zeros or another's rows)
        const bool in = SGQA_CHECK(w.b < a.batch && w.g < a.G && tile >= 0 && tile * kTok < w.L, a.status);
        if (w.k + x >= C::kStages) {
          warp_wait(&sh.empty[st], ph, abort, a.status);
          if ((stop = __any_sync(0xFFFFFFFFu, *abort))) break;
        }
        if (lane == 0) {
          uint8_t* dst = sKV + st * C::kStage;
          tc::mbar_arrive_expect_tx(&sh.full[st], C::kStage);
          tc::tma_load_3d(dst, &map_k, &sh.full[st], 0, w.g, z + tile * kTok);
          if (W) {
          } else if (a.w_out) {
            tma_load_3d_once(dst + C::kTile, &map_v, &sh.full[st], 0, w.g, z + tile * kTok, once);
          } else {
            tc::tma_load_3d(dst + C::kTile, &map_v, &sh.full[st], 0, w.g, z + tile * kTok);
          }
        }
        const int blk = tile * per;
        if (mine && in && blk + j < nblk) cp_async4(&sh.scale[st][lane], scales + (src + blk * a.G));
        cp_async_arrive(&sh.full[st]);
        issued = w.k + x + 1;
        st += C::kFetch;
        if (st >= C::kStages) {
          st -= C::kStages;
          ph ^= 1;
        }
      }
    }
    // copies in flight land before the CTA leaves (all have, unless a wait ran out)
    cp_async_wait_all();
    if (lane == 0) {
      volatile int none = 0;
      for (int i = max(0, issued - C::kStages); i < issued; ++i)
        if (i % C::kFetch == me) tc::mbar_wait(&sh.full[i % C::kStages], (uint32_t)((i / C::kStages) & 1), &none);
    }
  } else if (warp == 1) {
    // ---- MMAs of S^T: the warp waits, one lane issues ----
    constexpr uint32_t id_s = idesc_f8(C::N, false, false);
    const uint64_t dk = tc::smem_desc_kmajor(sKV, D), dq = tc::smem_desc_kmajor_noswz(sQ, 128, D * 8);
    int k = 0, st = 0, sb = 0;
    uint32_t ph = 0, sph = 1;  // phases of the stages and of S^T's buffers
    for (; w.left > 0; walk_next<W>(w, a)) {
      const int pb = w.piece & 1;
      const uint64_t db = dq + (uint32_t)(pb * (C::kQ >> 4));
      warp_wait(&sh.q_full[pb], (uint32_t)((w.piece >> 1) & 1), abort, a.status);
      for (int n = __shfl_sync(0xFFFFFFFFu, w.t1 - w.t0, 0); n > 0; --n, ++k) {
        warp_wait(&sh.full[st], ph, abort, a.status);
        if (k >= kGroups) warp_wait(&sh.s_empty[sb], sph, abort, a.status);
        tc::fence_after_sync();
        if (elect_one()) {
          const uint64_t da = dk + (uint32_t)(st * (C::kStage >> 4));
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk)
            mma_f8(tmem + (uint32_t)(sb * C::N), da + kk * 2, db + kk * 16, id_s, kk > 0);
          tc::mma_commit(&sh.s_full[sb]);
          if (W) tc::mma_commit(&sh.empty[st]);
          if (n == 1) tc::mma_commit(&sh.q_empty[pb]);
        }
        __syncwarp();
        if (++sb == kGroups) {
          sb = 0;
          sph ^= 1u;
        }
        if (++st == C::kStages) {
          st = 0;
          ph ^= 1;
        }
      }
    }
    // the MMAs in flight end before the CTA leaves
    if (lane == 0) {
      volatile int none = 0;
      tc::mbar_wait(&sh.s_full[(k - 1) % kGroups], (uint32_t)(((k - 1) / kGroups) & 1), &none);
      if (W)
        for (int j = max(0, k - C::kStages); j < k; ++j)
          tc::mbar_wait(&sh.empty[j % C::kStages], (uint32_t)((j / C::kStages) & 1), abort);
      tc::mbar_wait(&sh.q_empty[(w.piece - 1) & 1], (uint32_t)(((w.piece - 1) >> 1) & 1), abort);
    }
  } else if (W && warp < 4) {
    // (no O^T in the weights' pass)
  } else if (warp == 2) {
    // ---- MMAs of O^T ----
    {
      constexpr uint32_t id_o = idesc_f8(C::N, true, true);
      const uint64_t dv = D == 128 ? tc::smem_desc_mnmajor_sw128(sKV + C::kTile, 1024, 1024)
                                   : smem_desc_mnmajor_sw64_twice(sKV + C::kTile);
      // P: [16 columns][128 tokens][16 bytes]: 8 tokens are 128 bytes, 16 columns 2048
      const uint64_t dp = tc::smem_desc_kmajor_noswz(sP, 128, 2048);
      const int count = __shfl_sync(0xFFFFFFFFu, w.left, 0);
      int st = 0, pb = 0;
      uint32_t ph = 0;
      for (int k = 0; k < count; ++k) {
        warp_wait(&sh.p_full[pb], ph, abort, a.status);
        if (k >= kGroups) warp_wait(&sh.o_empty[pb], ph ^ 1u, abort, a.status);
        tc::fence_after_sync();
        if (elect_one()) {
          const uint64_t da = dv + (uint32_t)(st * (C::kStage >> 4)), db = dp + (uint32_t)(pb * (C::kP >> 4));
#pragma unroll
          for (int kk = 0; kk < kTok / 32; ++kk)
            mma_f8(tmem_o + (uint32_t)(pb * C::N), da + kk * (32 * D >> 4), db + kk * 32, id_o, kk > 0);
          tc::mma_commit(&sh.empty[st]);
          tc::mma_commit(&sh.o_full[pb]);
        }
        __syncwarp();
        if (++st == C::kStages) st = 0;
        if (++pb == kGroups) {
          pb = 0;
          ph ^= 1u;
        }
      }
      if (lane == 0) {
        volatile int none = 0;
        tc::mbar_wait(&sh.o_full[(count - 1) % kGroups], (uint32_t)(((count - 1) / kGroups) & 1), &none);
        for (int j = max(0, count - C::kStages); j < count; ++j)
          tc::mbar_wait(&sh.empty[j % C::kStages], (uint32_t)((j / C::kStages) & 1), &none);
      }
    }
  } else if (warp == 3) {
    {
      // ---- a lane per row: running maxima, denominators, factors for the accumulating warps ----
      float m_run = kNegMax, l = 0.f;
      int e_run = -126, sb = 0;  // (the row's)
      uint32_t ph = 0;
      for (; w.left > 0; walk_next<W>(w, a)) {
        for (int n = w.t1 - w.t0; n > 0; --n) {
          warp_wait(&sh.p_full[sb], ph, abort, a.status);
          float now = 1.f;
          const int2 ev = spread_of(sh.wev[sb]);
          if (lane < NR) {
            const float(&wm)[4][NR] = sh.wmax[sb];
            const float(&ws)[4][NR] = sh.wsum_p[sb];
            const float mt = fmaxf(fmaxf(wm[0][lane], wm[1][lane]), fmaxf(wm[2][lane], wm[3][lane]));
            const float mn = fmaxf(m_run, mt), da = m_run - mn, db = mt - mn;
            const int et = ev.x - ev.y > kSpread ? sh.ref[sb][lane] : ev.x;
            const int en = max(ref_of(da + (float)e_run), ref_of(db + (float)et));
            const float b = ex2_approx(db + (float)(et - en)) * (1.f / 448.f);
            float* f = reinterpret_cast<float*>(&sh.fb[sb][lane >> 1]) + (lane & 1);
            f[0] = b;
            f[2] = b * (1.f / 28.f);
            now = ex2_approx(da + (float)(e_run - en));
            sh.fa[sb][lane] = now;
            l = fmaf(l, ex2_approx(da), ((ws[0][lane] + ws[1][lane]) + (ws[2][lane] + ws[3][lane])) * ex2_approx(db));
            m_run = mn;
            e_run = en;
          }
          const bool any = __any_sync(0xFFFFFFFFu, now != 1.f);
          if (lane == 0) sh.any_fa[sb] = any;
          tc::mbar_arrive(&sh.f_full[sb]);
          if (++sb == kGroups) {
            sb = 0;
            ph ^= 1u;
          }
        }
        const long slot = (long)w.b * units_b + w.g * a.nch + w.ch + blockIdx.x;
        if (lane < NR && SGQA_CHECK(slot < (long)a.batch * units_b + kGridMax, a.status)) {
          part.m(slot)[lane] = m_run;
          part.l(slot)[lane] = l;
          part.e(slot)[lane] = e_run;
        }
        m_run = kNegMax;
        l = 0.f;
        e_run = -126;
      }
    }
  } else if (warp < 4 + 4 * kGroups) {
    // ---- scores, probabilities: lane = rows (lane % 4) q .. + q - 1 of tokens lane / 4 + 8 e ----
    constexpr int q = C::q;
    const int wg = (warp >> 2) - 1, q4 = warp & 3, t = tid & 127;
    const int i = lane & 3, tok = q4 * 32 + (lane >> 2), row0 = i * q;
    const uint32_t ts = tmem + ((uint32_t)(q4 * 32) << 16) + (uint32_t)(wg * C::N);
    uint64_t fac[q / 2];
#pragma unroll
    for (int j = 0; j < q / 2; ++j) fac[j] = 0ull;
    const bool stopped = W && tc::grid_timed_out(a.status);  // the rows' sums were not written
    // tiles k = wg, wg + groups, ..: stage k mod the stages, phase of the buffers kp = k / groups
    int st = wg;
    uint32_t ph = 0, kp = 0;
    for (Walk ahead = w; w.left > 0; w = ahead) {
      walk_next<W>(ahead, a);
      if (W && ahead.left > 0) split_piece<D, NR, W>(a, ahead, sh, sQ, warp - 4, abort, lane);
      const int pb = w.piece & 1;
      warp_wait(&sh.q_full[pb], (uint32_t)((w.piece >> 1) & 1), abort, a.status);
#pragma unroll
      for (int j = 0; j < q / 2; ++j) fac[j] = pack2(sh.fac[pb][row0 + 2 * j], sh.fac[pb][row0 + 2 * j + 1]);
      const int vis = w.L - a.n_new;  // tokens up to here are visible to every row
      const long wi0 = ((long)w.b * a.G + w.g) * a.T;
      for (int x = (wg + kGroups - w.k % kGroups) % kGroups; x < w.t1 - w.t0; x += kGroups, ++kp) {
        const int tile = walk_tile<W>(w, x);
        const int u0 = tile * kTok + tok;
        const bool edge = (tile + 1) * kTok - 1 > vis;
        const int uw = tile * kTok + q4 * 32 + (lane >> 2) + 8 * i;  // the token whose weight this lane writes
        const long wi = wi0 + uw;
        float sum = 0.f;
        if constexpr (W) {
          if (a.w_in && uw < vis && SGQA_CHECK(w.b < a.batch && uw >= 0 && uw < a.T, a.status)) sum = a.w_in[wi];
        }
        warp_wait(&sh.s_full[wg], kp & 1u, abort, a.status);
        warp_wait(&sh.full[st], ph, abort, a.status);
        tc::fence_after_sync();
        float sk[4];
        int ev[4], we = -127, wl = 127;
        const int sb = tok >> a.block_log2;
        sk[0] = sh.scale[st][sb];
        ev[0] = W ? 0 : (int)(__float_as_uint(sh.scale[st][16 + sb]) >> 23 & 255u) - 127;
#pragma unroll
        for (int e = 1; e < 4; ++e) {
          sk[e] = sk[0];
          ev[e] = ev[0];
        }
        if (a.block_log2 < 5) {  // else a lane's four tokens, all within 32, are in one block
#pragma unroll
          for (int e = 1; e < 4; ++e) {
            const int sb = (tok + 8 * e) >> a.block_log2;
            sk[e] = sh.scale[st][sb];
            ev[e] = W ? 0 : (int)(__float_as_uint(sh.scale[st][16 + sb]) >> 23 & 255u) - 127;
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (edge && u0 + 8 * e >= w.L) {  // whatever lies behind the last token
            sk[e] = 0.f;
            ev[e] = -127;
          } else {
            wl = min(wl, ev[e]);
          }
          we = max(we, ev[e]);
        }
        if constexpr (W) {
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&sh.empty[st]);
        }
        constexpr int qh = q < 8 ? q : 8;  // rows of one pass over S^T
        uint64_t z[4][qh / 2];             // [token][pair of rows]
        float add[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int h = 0; h < q / qh; ++h) {
          uint32_t c[8 * qh];
          tmem_ld_frag<qh>(ts + (uint32_t)(8 * qh * h), c);
          if (h == q / qh - 1) {
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&sh.s_empty[wg]);
          }
          const uint64_t sixteenth = pack2(0.0625f, 0.0625f);
          const int rh = row0 + qh * h;
#pragma unroll
          for (int j = 0; j < qh / 2; ++j) {
            // (the weights' pass takes the factors from shared memory: it may have several passes)
            const uint64_t f = W ? pack2(sh.fac[pb][rh + 2 * j], sh.fac[pb][rh + 2 * j + 1]) : fac[j];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t* x = c + 4 * qh * (e >> 1) + 8 * j + 2 * (e & 1);
              const uint64_t q1 = pack2(__uint_as_float(x[0]), __uint_as_float(x[1]));
              const uint64_t q2 = pack2(__uint_as_float(x[4]), __uint_as_float(x[5]));
              z[e][j] = mul2(mul2(fma2(q2, sixteenth, q1), f), pack2(sk[e], sk[e]));
            }
          }
          if (edge) {
#pragma unroll
            for (int j = 0; j < qh / 2; ++j) {
              const int lim0 = sh.lim[pb][rh + 2 * j], lim1 = sh.lim[pb][rh + 2 * j + 1];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 x = unpack2(z[e][j]);
                z[e][j] = pack2(u0 + 8 * e > lim0 ? -INFINITY : x.x, u0 + 8 * e > lim1 ? -INFINITY : x.y);
              }
            }
          }
          if constexpr (W) {
#pragma unroll
            for (int j = 0; j < qh / 2; ++j) {
              const uint64_t lse = pack2(-sh.lse[pb][rh + 2 * j], -sh.lse[pb][rh + 2 * j + 1]);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float2 x = unpack2(add2(z[e][j], lse)), y = unpack2(z[e][j]);
                // (a masked token gets nothing from a row of NaN either)
                add[e] += y.x == -INFINITY ? 0.f : ex2_approx(x.x);
                add[e] += y.y == -INFINITY ? 0.f : ex2_approx(x.y);
              }
            }
          }
        }
        if constexpr (W) {
          // over the four lanes of a token; lane i gets token i
          const bool up2 = i & 2, up1 = i & 1;
          const float g0 = up2 ? add[0] : add[2], g1 = up2 ? add[1] : add[3];
          const float h0 = (up2 ? add[2] : add[0]) + __shfl_xor_sync(0xFFFFFFFFu, g0, 2);
          const float h1 = (up2 ? add[3] : add[1]) + __shfl_xor_sync(0xFFFFFFFFu, g1, 2);
          const float tot = (up1 ? h1 : h0) + __shfl_xor_sync(0xFFFFFFFFu, up1 ? h0 : h1, 1);
          // (after a wait of this CTA has run out the scores may be anything: the weight, which may be summed up
          // in place, stays as it is)
          if (uw < w.L && !stopped && !*abort && SGQA_CHECK(w.b < a.batch && uw >= 0 && uw < a.T, a.status))
            a.w_out[wi] = sum + tot;
        } else {
          // maxima of the tile; NaN counts for none (it reaches the sums by itself)
          float mx[q];
#pragma unroll
          for (int j = 0; j < q / 2; ++j) {
            const float2 z0 = unpack2(z[0][j]), z1 = unpack2(z[1][j]), z2 = unpack2(z[2][j]), z3 = unpack2(z[3][j]);
            mx[2 * j] = max3(max3(z0.x, z1.x, z2.x), z3.x, kNegMax);
            mx[2 * j + 1] = max3(max3(z0.y, z1.y, z2.y), z3.y, kNegMax);
          }
          const float mine = across_tokens<q>(mx, lane, [](float x, float y) { return fmaxf(x, y); });
          we = __reduce_max_sync(0xFFFFFFFFu, we);
          wl = __reduce_min_sync(0xFFFFFFFFu, wl);
          // the P buffer and the numbers of the group's tile before have been read
          if (kp > 0) warp_wait(&sh.o_empty[wg], (kp & 1u) ^ 1u, abort, a.status);
          if ((lane >> 2) < q) sh.wmax[wg][q4][row0 + (lane >> 2)] = mine;
          if (lane == 0) sh.wev[wg][q4] = make_int2(we, wl);
          if (edge) {
            // A zero probability must not meet a NaN code: rows behind the last token become zeros,
            // and a NaN of a token that some row does not see is noted and taken out; the rows that
            // see it get it back at the end.
            uint8_t* v = sKV + st * C::kStage + C::kTile;
            const int after = w.L - tile * kTok;  // the tile's first row behind the last token
            if (t >= after) {
#pragma unroll
              for (int c = 0; c < D / 16; ++c) *reinterpret_cast<uint4*>(v + t * D + c * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            // 16 codes a thread of the rows vis + 1 .. L - 1 of this tile
            for (int x = max(0, vis + 1 - tile * kTok) * (D / 16) + t; x < min(kTok, after) * (D / 16); x += 128) {
              const int r = x / (D / 16), c = x % (D / 16);
              uint4* p = reinterpret_cast<uint4*>(v + r * D + v_chunk<D>(r, c) * 16);
              uint32_t y[4] = {p->x, p->y, p->z, p->w}, any = 0u;
#pragma unroll
              for (int e = 0; e < 4; ++e) any |= __vcmpeq4(y[e] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
              if (any) {
                for (int e = 0; e < 16; ++e) {
                  const uint32_t code = 0x7Fu << (8 * (e & 3));
                  if ((y[e >> 2] & code) != code) continue;
                  y[e >> 2] &= ~(0xFFu << (8 * (e & 3)));
                  atomicMin(&sh.nan_at[w.piece % kGroups][c * 16 + e], tile * kTok + r);
                }
                sh.nan_any[w.piece % kGroups] = 1;
                *p = make_uint4(y[0], y[1], y[2], y[3]);
              }
            }
          }
          group_sync(1 + wg);
          uint64_t mt[q / 2], ps[q / 2];
#pragma unroll
          for (int j = 0; j < q / 2; ++j) {
            float2 x = *reinterpret_cast<const float2*>(&sh.wmax[wg][0][row0 + 2 * j]);
#pragma unroll
            for (int y = 1; y < 4; ++y) {
              const float2 v = *reinterpret_cast<const float2*>(&sh.wmax[wg][y][row0 + 2 * j]);
              x.x = fmaxf(x.x, v.x);
              x.y = fmaxf(x.y, v.y);
            }
            mt[j] = pack2(-x.x, -x.y);
            ps[j] = 0ull;
          }
          const int2 es = spread_of(sh.wev[wg]);
          uint8_t* pd = sP + wg * C::kP + (i * 2 * q / 16) * 2048 + (i * 2 * q % 16) + tok * 16;
          const __half2 c28 = __floats2half2_rn(28.f, 28.f);
          // y (448 p t over the reference) of a token's rows as two terms. Both from y rounded to fp16 (2^-11
          // of itself): the first's rest is exact there (a multiple of y's last bit, at most 2^-4 of it), and
          // so is its 28-fold.
          auto terms = [&](int j, uint64_t y2, uint32_t(&p1)[q / 2], uint32_t(&p2)[q / 2]) {
            const float2 y = unpack2(y2);
            const __half2 h = __floats2half2_rn(y.x, y.y);
            p1[j] = __nv_cvt_halfraw2_to_fp8x2(h, __NV_SATFINITE, __NV_E4M3);
            const __half2_raw f = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)p1[j], __NV_E4M3);
            p2[j] = __nv_cvt_halfraw2_to_fp8x2(__hmul2(__hsub2(h, __half2(f)), c28), __NV_SATFINITE, __NV_E4M3);
          };
          auto store = [&](uint8_t* d, const uint32_t(&p1)[q / 2], const uint32_t(&p2)[q / 2]) {
            if constexpr (q == 8) {
              *reinterpret_cast<uint4*>(d) = make_uint4(p1[0] | p1[1] << 16, p1[2] | p1[3] << 16, p2[0] | p2[1] << 16,
                                                        p2[2] | p2[3] << 16);
            } else if constexpr (q == 4) {
              *reinterpret_cast<uint2*>(d) = make_uint2(p1[0] | p1[1] << 16, p2[0] | p2[1] << 16);
            } else {
              *reinterpret_cast<uint32_t*>(d) = p1[0] | p2[0] << 16;
            }
          };
          if (es.x - es.y <= kSpread) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float cs = 448.f * c8_pow2(max(-126, ev[e] - es.x));
              const uint64_t c2 = pack2(cs, cs);
              uint32_t p1[q / 2], p2[q / 2];  // two codes each
#pragma unroll
              for (int j = 0; j < q / 2; ++j) {
                const float2 x = unpack2(add2(z[e][j], mt[j]));
                const uint64_t p = pack2(ex2_approx(x.x), ex2_approx(x.y));
                ps[j] = add2(ps[j], p);
                terms(j, mul2(p, c2), p1, p2);
              }
              store(pd + e * 128, p1, p2);
            }
          } else {
            // The rows' own references: the largest score plus V exponent, rounded up. (A tile that comes here
            // takes up to 25% longer with 32 rows, 1% with 8, where HBM binds; so it is not the only way.)
            float mr[q];
#pragma unroll
            for (int j = 0; j < q; ++j) mr[j] = kNegMax;
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
              for (int j = 0; j < q / 2; ++j) {
                const float2 x = unpack2(add2(z[e][j], mt[j]));
                mr[2 * j] = fmaxf(mr[2 * j], x.x + (float)ev[e]);
                mr[2 * j + 1] = fmaxf(mr[2 * j + 1], x.y + (float)ev[e]);
              }
            const float own = across_tokens<q>(mr, lane, [](float x, float y) { return fmaxf(x, y); });
            if ((lane >> 2) < q) sh.wref[wg][q4][row0 + (lane >> 2)] = own;
            group_sync(1 + wg);
            // (row t; the softmax warps' and the maxima's both read it behind another barrier)
            if (t < NR)
              sh.ref[wg][t] = ref_of(fmaxf(fmaxf(sh.wref[wg][0][t], sh.wref[wg][1][t]), fmaxf(sh.wref[wg][2][t], sh.wref[wg][3][t])));
            group_sync(1 + wg);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t p1[q / 2], p2[q / 2];
#pragma unroll
              for (int j = 0; j < q / 2; ++j) {
                const float2 x = unpack2(add2(z[e][j], mt[j]));
                ps[j] = add2(ps[j], pack2(ex2_approx(x.x), ex2_approx(x.y)));
                const float y0 = ex2_approx(x.x + (float)(ev[e] - sh.ref[wg][row0 + 2 * j]));
                const float y1 = ex2_approx(x.y + (float)(ev[e] - sh.ref[wg][row0 + 2 * j + 1]));
                terms(j, pack2(448.f * y0, 448.f * y1), p1, p2);
              }
              store(pd + e * 128, p1, p2);
            }
          }
          tc::fence_proxy_async();
          float x[q];
#pragma unroll
          for (int j = 0; j < q / 2; ++j) {
            const float2 y = unpack2(ps[j]);
            x[2 * j] = y.x;
            x[2 * j + 1] = y.y;
          }
          const float s = across_tokens<q>(x, lane, [](float x, float y) { return x + y; });
          if ((lane >> 2) < q) sh.wsum_p[wg][q4][row0 + (lane >> 2)] = s;
          tc::mbar_arrive(&sh.p_full[wg]);
        }
        st += kGroups;
        if (st >= C::kStages) {
          st -= C::kStages;
          ph ^= 1;
        }
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sh.q_empty[pb]);
    }
  } else {
    const int q_first = warp - 4 - 4 * kGroups;
    if constexpr (!W) {
      // ---- a thread per head dim: outputs ----
      const int q4 = warp & 3, t = tid & 127;
      const int dim = D == 128 ? t : t & 63, rb = D == 128 ? 0 : (t >> 6) * C::kRowsT;
      // columns of O^T: rows i q .. of the first terms, then of the second, for i = 0 .. 3
      const uint32_t to = tmem_o + ((uint32_t)(q4 * 32) << 16) + (uint32_t)(C::kRowsT < 8 ? 0 : 2 * rb);
      uint64_t o[C::kRowsT / 2];
#pragma unroll
      for (int r = 0; r < C::kRowsT / 2; ++r) o[r] = 0ull;
      int sb = 0;
      uint32_t ph = 0;
      for (Walk ahead = w; w.left > 0; w = ahead) {
        walk_next<W>(ahead, a);
        if (ahead.left > 0) split_piece<D, NR, W>(a, ahead, sh, sQ, q_first, abort, lane);
        const int nb = w.piece % kGroups;
        const long unit = (long)w.b * units_b + w.g * a.nch + w.ch, slot = unit + blockIdx.x;
        for (int n = w.t1 - w.t0; n > 0; --n) {
          warp_wait(&sh.f_full[sb], ph, abort, a.status);
          if (sh.any_fa[sb]) {
#pragma unroll
            for (int r = 0; r < C::kRowsT; r += 2)
              o[r / 2] = mul2(o[r / 2], *reinterpret_cast<const uint64_t*>(&sh.fa[sb][rb + r]));
          }
          warp_wait(&sh.o_full[sb], ph, abort, a.status);
          tc::fence_after_sync();
#pragma unroll
          for (int r0 = 0; r0 < C::kRowsT; r0 += 16) {
            constexpr int kH = C::kRowsT < 16 ? C::kRowsT : 16, q = C::q;
            uint32_t c[2][16];
            tc::tmem_ld16_nowait(to + (uint32_t)(sb * C::N + 2 * r0), c[0]);
            if constexpr (kH == 16) tc::tmem_ld16_nowait(to + (uint32_t)(sb * C::N + 2 * r0 + 16), c[1]);
            tc::tmem_wait_ld2(c[0], c[1]);
#pragma unroll
            for (int r = 0; r < kH; r += 2) {
              const int h = r >> 3, x = (r & 7) / q * 2 * q + (r & 7) % q;
              float x1 = __uint_as_float(c[h][x]), y1 = __uint_as_float(c[h][x + 1]);
              float x2 = __uint_as_float(c[h][x + q]), y2 = __uint_as_float(c[h][x + q + 1]);
              if constexpr (C::kRowsT < 8) {  // the upper rows' threads: 8 columns on
                if (rb) {
                  x1 = __uint_as_float(c[0][x + 8]), y1 = __uint_as_float(c[0][x + 9]);
                  x2 = __uint_as_float(c[0][x + q + 8]), y2 = __uint_as_float(c[0][x + q + 9]);
                }
              }
              const float4 f = sh.fb[sb][(rb + r0 + r) / 2];
              uint64_t& y = o[(r0 + r) / 2];
              y = fma2(pack2(x2, y2), pack2(f.z, f.w), fma2(pack2(x1, y1), pack2(f.x, f.y), y));
            }
          }
          tc::fence_before_sync();
          if (n == 1) {
            if (sh.nan_any[nb]) {
              const int np = sh.nan_at[nb][dim], r0 = w.ch * a.chunk_rows + rb, R = a.Hq / a.G;
#pragma unroll
              for (int r = 0; r < C::kRowsT; r += 2) {
                const float nan = __int_as_float(0x7FC00000);
                const float2 y = unpack2(o[r / 2]);
                o[r / 2] = pack2(np <= w.L - a.n_new + (r0 + r) / R ? nan : y.x,
                                 np <= w.L - a.n_new + (r0 + r + 1) / R ? nan : y.y);
              }
            }
            group_sync(7);
            sh.nan_at[nb][t] = kNever;
            if (t == 0) sh.nan_any[nb] = 0;
          }
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&sh.o_empty[sb]);
          if (++sb == kGroups) {
            sb = 0;
            ph ^= 1u;
          }
        }
        float* po = part.o(slot) + rb * D + dim;
        const bool in = SGQA_CHECK(unit < (long)a.batch * units_b && slot < (long)a.batch * units_b + kGridMax, a.status);
#pragma unroll
        for (int r = 0; r < C::kRowsT; r += 2) {
          if (!in) break;
          const float2 y = unpack2(o[r / 2]);
          po[r * D] = y.x;
          po[(r + 1) * D] = y.y;
          o[r / 2] = 0ull;
        }
        if (t == 0 && in) {
          if (w.t0 == 0) part.first[unit] = (int)blockIdx.x;
          if (w.t1 == w.ntiles) part.last[unit] = (int)blockIdx.x;
        }
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

// Joins the pieces of a unit: PER warps per (sequence, group, row), which take its pieces in turn; a
// lane per piece for the factors, per D / 32 head dims for the sums. The order is fixed.
constexpr int kJoinWarps = 8, kJoinLens = 256;  // (with more sequences the first kernel's notes are read)
template <int D, int NR, int PER>
__global__ void __launch_bounds__(kJoinWarps * 32) cache8_join_kernel(C8AttendArgs a) {
  constexpr int kV = D / 32;
  __shared__ float s_m[kJoinWarps], s_l[kJoinWarps], s_o[PER > 1 ? kJoinWarps : 1][D];
  __shared__ int s_e[kJoinWarps];
  grid_dependents();
  const int R = a.Hq / a.G, rows = a.n_new * R, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int item = min((int)((blockIdx.x * kJoinWarps + warp) / PER), a.batch * a.G * rows - 1), part_of = warp % PER;
  const int gr = item % rows, bg = item / rows, b = bg / a.G, g = bg % a.G;
  const int r = gr % a.chunk_rows, ch = gr / a.chunk_rows;
  const long unit = (long)bg * a.nch + ch;
  const Part<D, NR> part(a.part, (long)a.batch * a.G * a.nch);
  const long at = (((long)b * a.n_new + gr / R) * a.Hq + (long)g * R + gr % R) * D + lane * kV;
  // what the call's inputs say, while the kernel before still runs
  uint32_t gate[kV / 2];
#pragma unroll
  for (int v = 0; v < kV / 2; ++v) gate[v] = __ldg(reinterpret_cast<const uint32_t*>(a.gate + at) + v);
  const int L = len_of(a, b);
  const bool some = L > a.n_new - 1 - gr / R;
  int c0 = 0, c1 = -1;  // the CTAs whose pieces this unit has
  if (a.batch <= kJoinLens) {
    int before = 0, total = 0;
    for (int x = lane; x < a.batch; x += 32) {
      const int n = tiles_of(len_of(a, x)) * a.G * a.nch;
      total += n;
      if (x < b) before += n;
    }
    total = __reduce_add_sync(0xFFFFFFFFu, total);
    before = __reduce_add_sync(0xFFFFFFFFu, before) + (g * a.nch + ch) * tiles_of(L);
    const int n = max(1, min(a.main_ctas, total)), each = total / n, odd = total - each * n;
    auto cta_of = [&](int t) { return t < odd * (each + 1) ? t / (each + 1) : odd + (t - odd * (each + 1)) / max(1, each); };
    if (some) {
      c0 = cta_of(before);
      c1 = cta_of(before + tiles_of(L) - 1);
    }
  }
  grid_wait();
  if (tc::grid_timed_out(a.status) || (blockIdx.x * kJoinWarps + warp) / PER > item) return;
  if (some && a.batch > kJoinLens) {
    c0 = part.first[unit];
    c1 = part.last[unit];
  }
  if (!SGQA_CHECK(!some || (c0 >= 0 && c0 <= c1 && c1 < a.main_ctas), a.status)) c0 = 0, c1 = -1;
  const int n = c1 - c0 + 1;  // pieces; this warp's are part_of, part_of + PER, ..
  float m = kNegMax, den = 0.f, o[kV];
  int e = -126;
#pragma unroll
  for (int v = 0; v < kV; ++v) o[v] = 0.f;
  for (int p0 = part_of; p0 < n; p0 += 32 * PER) {
    const long slot = unit + c0 + p0 + lane * PER;
    const bool has = p0 + lane * PER < n;
    const float pm = has ? part.m(slot)[r] : kNegMax, pl = has ? part.l(slot)[r] : 0.f;
    const int pe = has ? part.e(slot)[r] : -126;
    // the sums so far and these pieces' on common references
    float mn = fmaxf(m, pm);
#pragma unroll
    for (int h = 16; h; h >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xFFFFFFFFu, mn, h));
    const int en = max(ref_of(m - mn + (float)e), __reduce_max_sync(0xFFFFFFFFu, ref_of(pm - mn + (float)pe)));
    const float old = ex2_approx(m - mn), f = ex2_approx(pm - mn);
    float l = pl * f;
#pragma unroll
    for (int h = 16; h; h >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, h);
    den = fmaf(den, old, l);
    const float fe = ex2_approx(pm - mn + (float)(pe - en)), olde = ex2_approx(m - mn + (float)(e - en));
#pragma unroll
    for (int v = 0; v < kV; ++v) o[v] *= olde;
    m = mn;
    e = en;
    const float* src = part.o(unit + c0 + p0) + r * D + lane * kV;
    const int last = min(32, (n - p0 + PER - 1) / PER);
#pragma unroll 8
    for (int x = 0; x < last; ++x) {
      const float fx = __shfl_sync(0xFFFFFFFFu, fe, x);
      const float* y = src + (long)x * PER * Part<D, NR>::kRec;
#pragma unroll
      for (int v = 0; v < kV; v += 2) {
        const float2 y2 = *reinterpret_cast<const float2*>(y + v);
        o[v] = fmaf(y2.x, fx, o[v]);
        o[v + 1] = fmaf(y2.y, fx, o[v + 1]);
      }
    }
  }
  if constexpr (PER > 1) {
    if (lane == 0) {
      s_m[warp] = m;
      s_e[warp] = e;
      s_l[warp] = den;
    }
#pragma unroll
    for (int v = 0; v < kV; ++v) s_o[warp][lane * kV + v] = o[v];
    __syncthreads();  // (all warps of the CTA have the same item)
    if (warp > 0) return;
    for (int x = 1; x < PER; ++x) m = fmaxf(m, s_m[x]);
    e = -126;
    for (int x = 0; x < PER; ++x) e = max(e, ref_of(s_m[x] - m + (float)s_e[x]));
    den = 0.f;
#pragma unroll
    for (int v = 0; v < kV; ++v) o[v] = 0.f;
#pragma unroll
    for (int x = 0; x < PER; ++x) {
      const float f = ex2_approx(s_m[x] - m), fe = ex2_approx(s_m[x] - m + (float)(s_e[x] - e));
      den = fmaf(s_l[x], f, den);
#pragma unroll
      for (int v = 0; v < kV; ++v) o[v] = fmaf(s_o[x][lane * kV + v], fe, o[v]);
    }
  }
  const float scale = c8_pow2(e);
#pragma unroll
  for (int v = 0; v < kV; v += 2) {
    const float y0 = den == 0.f ? 0.f : o[v] / den * scale, y1 = den == 0.f ? 0.f : o[v + 1] / den * scale;
    const uint32_t gt = gate[v / 2];
    reinterpret_cast<uint32_t*>(a.out + at)[v / 2] =
        f32_to_bf16_rne(y0 * sigmoid_fast(bf16_lo(gt))) | ((uint32_t)f32_to_bf16_rne(y1 * sigmoid_fast(bf16_hi(gt))) << 16);
  }
  if (lane == 0 && a.w_out) a.lse[item] = den == 0.f ? 0.f : m + log2f(den);
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
// [batch * T tokens][G][d] codes, box = one group's codes of 128 tokens; zeros behind the last token.
// (With promotion to 256 bytes L2 fetches the neighbouring group along: 32 x 32K 164 us on the device instead of 121.)
bool make_map(CUtensorMap* map, const void* base, long tokens, int G, int d) {
  EncodeTiled enc = get_encode();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)G, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)d, (cuuint64_t)G * d};
  const cuuint32_t box[3] = {(cuuint32_t)d, 1, kTok};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

unsigned main_grid(const C8AttendArgs& a) {
  const long tiles = (long)a.batch * a.G * a.nch * ((a.T + kTok - 1) / kTok);
  return (unsigned)(tiles < kGridMax ? tiles : kGridMax);
}

template <int D, int NR, bool W>
cudaError_t launch_main(const CUtensorMap& mk, const CUtensorMap& mv, C8AttendArgs a, int nch, int chunk_rows,
                        cudaStream_t s) {
  using C = Cfg<D, NR, W>;
  constexpr int kSmem = C::kStages * C::kStage + 2 * C::kQ + C::kGroups * C::kP + 1024;
  cudaError_t e = cudaFuncSetAttribute(cache8_attend_kernel<D, NR, W>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  a.nch = nch;
  a.chunk_rows = chunk_rows;
  a.block_log2 = a.block == 8 ? 3 : a.block == 16 ? 4 : a.block == 32 ? 5 : a.block == 64 ? 6 : 7;
  const unsigned grid = main_grid(a);
  return launch_behind(cache8_attend_kernel<D, NR, W>, grid, C::kThreads, kSmem, s, W, mk, mv, a);
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
  a.main_ctas = (int)main_grid(a);
  const int rows = a.n_new * (a.Hq / a.G);
  const long items = (long)a.batch * a.G * rows;
  if (items > 0x7FFFFFF0L) return cudaErrorInvalidConfiguration;
  // eight warps a row where a unit has four pieces or more (1M tokens, 4 groups: 8 us instead of 15), else
  // one (128 units of 2 pieces: 6 us instead of 9)
  if ((long)a.batch * a.G * rw.nch * 4 <= kGridMax)
    e = launch_behind(cache8_join_kernel<D, NR, kJoinWarps>, (unsigned)items, kJoinWarps * 32, 0, s, true, a);
  else
    e = launch_behind(cache8_join_kernel<D, NR, 1>, (unsigned)((items + kJoinWarps - 1) / kJoinWarps), kJoinWarps * 32, 0,
                      s, true, a);
  if (e != cudaSuccess || !a.w_out) return e;
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
  const long rec = (long)rw.nr * d + rw.nr * 3;
  return (size_t)(2 * ((units + 3) & ~3L) + (units + kGridMax) * rec) * 4;
}

cudaError_t launch_cache8_attend(const C8AttendArgs& a, cudaStream_t s) {
  return a.d == 64 ? launch_d<64>(a, s) : launch_d<128>(a, s);
}

}  // namespace sgqa
