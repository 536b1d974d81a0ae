// Attention over the block-scaled 8-bit cache (mkv_blk8_attention), head_dim D, on tcgen05.
//
// Mathematics.  For query row r of a kv head (rows: nq query tokens x G heads), token t of a page with scales
// sk, sv and codes K_t, V_t (e4m3):
//   s_rt = c sk (q_r . K_t),  c = softmax scale * log2(e);   out_r = sum_t 2^(s_rt - m_r) sv V_t / sum_t 2^(s_rt - m_r)
// in one pass with running references (m for the sum, M for the weights 2^(s + log2 sv - M) of the codes; M is kept as
// M - m, and s - m is a difference of rounded scores, so that neither loses the page's scale nor the slack to the size
// of the scores: ones of 1e30 still give their largest token's V).
//
// The codes are read as the first to leave L2, so that they do not push out what every CTA wants (the kernel's own
// code, page ids, scales, the pieces for the join): 68.7 -> 65.2 us for 8 requests of 8K .. 32K tokens; with several
// row tiles, which read them again, 265 -> 263 us (4 x 16K, 64 query tokens).
//
// The codes go into the tensor cores as they lie in memory: S = K q^T with the 128 tokens of a tile as the M
// rows (A, K-major) and the query rows as N columns, O^T += V^T P with head dims as M (A = V, MN-major) and the
// weights as N.  tcgen05.mma kind::f8f6f4 wants 8-bit operands on both sides, so q and the weights are split
// into e4m3 parts that share N: a row q scaled by a power of two is q = q1 + q2 / 16 (+ q3 / 256), each part the
// rounded remainder of the one before.  Four significant bits a part: two parts hold a bf16 q exactly and three an
// fp16 one (up to its smallest elements: below 2^-17 of the row's largest a part is subnormal).
// The weights (times 2^6, of their fp16 rounding) take four parts, of steps 1, 2^-4, 2^-11 and 2^-15.  What matters is
// not how many bits a weight has but what all of them miss together: a long context behind one dominant token is
// a hundred thousand weights of 2^-17, whose sum counts as much as that token, and parts of steps 1 and 2^-4 alone
// round every one of them to the same wrong value (65,536 tokens 11 nats below the first: outputs 23 to 56 % off).  The
// first two parts hold the 8 leading bits of weights above 2^-10 of the reference and the last two, 2^7 further down,
// their remainder (11 bits in all) and the leading bits of the weights below: 2^-8 or better down to 2^-22 of the
// reference, and an error of 2^-31 of it for what is smaller still, against a largest weight of 2^-2 or more: a million
// tokens lose 2^-9 together.  The row sums use the unrounded fp32 weights.
// P is the B operand with N contiguous (16-byte groups of one token), so that a thread stores its token's weights in
// two 16-byte words.
// An N of 32 costs the tensor pipe what N = 8 does (reading A bounds it), and no code is ever converted, so the ALUs see
// only the scores: nothing in the kernel scales with head_dim but the copies and the MMAs.
//
// Bound: memory, 2 D bytes a token and kv head.  Work is cut into tiles of 128 tokens of one (sequence, kv head,
// row tile); every CTA takes the same number of tiles, one after another, whatever sequences they belong to (the
// lengths live on the device; the CTAs sum the tile counts themselves).  A CTA that holds all tiles of a unit
// writes its rows, the others leave (m, l, o) in the workspace for the join kernel.
//
// A CTA: one warp copies pages by TMA (boxes of one page, swizzled) into a ring of slots, K and V tiles in turn;
// another issues the MMAs; a warpgroup for every eight rows of the row tile runs their softmax, thread t on token t
// (TMEM lane t).  (Two warpgroups for row tiles of 24 and 32, 12 or 16 rows a thread: 69.1 us against 66.6 for
// 8 x 8K .. 32K tokens with 24 rows, head_dim 256, fp16; 42 against 37 for 6 x 4K .. 18K with 30 rows, head_dim 64:
// a tile's softmax is a chain of short dependent steps, and more warps hide them.)  S is double-buffered: the next
// tile's QK runs while this tile's softmax does.  The maximum is looked at by one vote a tile (does any
// score exceed its reference by 2^2?) and reduced only then, to a reference 2^2 above it, which is rare after the
// first tile of a piece; weights therefore lie in [0, 4] and their first parts, scaled by 2^6, in e4m3's range.
// What is not done every tile (the references, a piece's end, the producer's start) is written as rolled loops over rows
// kept in shared memory: a launch meets its instructions cold, about 80 cycles per 128 bytes of code, and unrolled those
// paths cost 7,000 cycles the first time against a tile's 2,600.  For the same reason nothing is divided where a product
// does (all divisions by the call's counts, and the join's loads without branches: one request of 4,096 13.0 -> 12.3 us,
// of 14,584 with heads of 128 16.9 -> 15.2, the ragged batch 305 -> 297 .. 300).  The next piece's query rows are split
// behind this piece's first tile, not before it, where they delayed every CTA's first softmax by 5,000 cycles.
//
// Measured (HBM copy rate 6,695 GB/s): 64 requests of 1,024 .. 65,536 tokens, 32 / 8 heads of 128, bf16: 305 .. 308 us
// for 2.02 GB, 98 % (297 with two parts a weight).  8 requests of 8K .. 32K, four query tokens, 24 / 4 heads of 256,
// fp16: 65.5 us for 314 MB (72 %; 63 with three parts); of 64K and 128K each: 168 and 323 us (95 and 99 %), so long
// calls are bound by memory and some 20 us are the start (cold code, the first codes), the pieces' ends and the join; 12 us
// for one query token.  One request of 4,096: 12.5 us, that latency alone.
// Tried and not kept: tiles drawn from a counter in chunks (the ragged batch 316 us, the 8 requests 108: every change
// of piece costs about four tiles); QK and PV issued by two warps (the ragged batch 327 us); whole runs of page ids
// fetched ahead (330: a faster mean, a slower last CTA).
// Every wait is bounded; one that runs out sets the error word and the CTA leaves after its copies have landed.
#pragma once

#include "mkv_blk8.cuh"
#include "mkv_internal.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <climits>

namespace mkv {
namespace b8 {

constexpr unsigned kFull = 0xffffffffu;
constexpr long long kWaitCycles = 4000000000LL;   // ~2 s: bound on any wait
constexpr float kRise = 2.0f;                      // log2 units a score may exceed its reference by
constexpr float kRoom = 2.0f;                      // and that a raised reference lies above the largest score
constexpr float kNone = -1e30f;                    // reference before any visible token
constexpr float kUp = 6.0f;                        // log2 of the factor that weights carry into their parts
constexpr int kWP = 4;                             // parts of a weight
constexpr __host__ __device__ float part_step(int k) { return k == 2 ? 128.f : 16.f; }   // step of part k - 1 over part k's
constexpr int kScaleRing = 8;                      // tiles whose page scales are kept

// ------------------------------------------------------------------ PTX
__device__ __forceinline__ uint32_t sptr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void bar_init(uint64_t* b, uint32_t n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(sptr(b)), "r"(n) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(sptr(b)) : "memory");
}
__device__ __forceinline__ void bar_expect(uint64_t* b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(sptr(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(sptr(b)), "r"(parity) : "memory");
  return ok != 0;
}
__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t* b) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(sptr(b)) : "memory");
}
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tma_page(void* dst, const CUtensorMap* map, int x, int z, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(sptr(dst)),
      "l"(map), "r"(x), "r"(0), "r"(z), "r"(sptr(bar)), "l"(policy)
      : "memory");
}
// consecutive columns of this warp's TMEM lanes (the caller waits)
__device__ __forceinline__ void tm_ld4(uint32_t at, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void tm_st4(uint32_t at, const float* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3])
               : "memory");
}
__device__ __forceinline__ void tm_ld8(uint32_t at, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(at) : "memory");
}
__device__ __forceinline__ void tm_st8(uint32_t at, const float* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at), "f"(v[0]), "f"(v[1]),
               "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}
// N (a multiple of 4) columns
template <int N>
__device__ __forceinline__ void tm_ld(uint32_t at, float* v) {
#pragma unroll
  for (int i = 0; i + 8 <= N; i += 8) tm_ld8(at + i, v + i);
  if constexpr (N % 8) tm_ld4(at + N / 8 * 8, v + N / 8 * 8);
}
template <int N>
__device__ __forceinline__ void tm_st(uint32_t at, const float* v) {
#pragma unroll
  for (int i = 0; i + 8 <= N; i += 8) tm_st8(at + i, v + i);
  if constexpr (N % 8) tm_st4(at + N / 8 * 8, v + N / 8 * 8);
}
// the loaded registers are tied to the wait, so that no use of them moves above it
template <int N>
__device__ __forceinline__ void tm_wait_ld(float (&v)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2(__half2 x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t*>(&x)));
  return r;
}
__device__ __forceinline__ __half2 half2_of(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return *reinterpret_cast<const __half2*>(&r);
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return __half22float2(*reinterpret_cast<const __half2*>(&r));
}
// a maximum over the warp, on integers of the same order
__device__ __forceinline__ float warp_max(float x) {
  const int b = __float_as_int(x);
  const int m = __reduce_max_sync(kFull, b ^ ((b >> 31) & 0x7fffffff));
  return __int_as_float(m ^ ((m >> 31) & 0x7fffffff));
}

// ------------------------------------------------------------------ layout
constexpr int round16(int x) { return (x + 15) & ~15; }
constexpr int pow2_cols(int x) { return x <= 32 ? 32 : x <= 64 ? 64 : x <= 128 ? 128 : x <= 256 ? 256 : 512; }

template <int D, int RT, int QP>
struct Cfg {
  static constexpr int kW = D < 128 ? D : 128;            // bytes of a row in a sub-tile: the swizzle's width
  static constexpr int kSub = D / kW;
  static constexpr int kSubBytes = kB8Tile * kW;
  static constexpr int kTileBytes = kB8Tile * D;
  static constexpr int kNS = round16(QP * RT);            // columns of S
  static constexpr int kWG = RT / 8;            // softmax warpgroups
  static constexpr int kRows = RT / kWG;                  // rows of one
  static constexpr int kPG = kWP * kRows / 16;            // 16-byte groups of a warpgroup's weights
  static constexpr int kNP = 16 * kPG * kWG;              // columns of O
  static constexpr int kSoft = 128 * kWG, kThreads = kSoft + 64;
  static_assert(kRows % 4 == 0, "rows of a warpgroup");
  static constexpr int kQBytes = kNS * D, kPBytes = kNP * kB8Tile;
  static constexpr int kQSub = kNS * kW;
  static constexpr int kCols = pow2_cols(2 * kNS + kSub * kNP);
  static constexpr int kTO = 2 * kNS;                     // first column of O
  static constexpr int kCtas = b8_ctas_per_sm(D, RT);
  static_assert(2 * kNS + kSub * kNP <= 512 && kCols * kCtas <= 512, "tensor memory");
  // fixed part of shared memory behind the slots
  static constexpr int kQ = 0, kP = kQ + 2 * kQBytes, kX = kP + 2 * kPBytes;         // x: [RT][128] floats
  static constexpr int kRefs = kX + RT * 128 * 4;         // [2 pieces][WG][4][rows]: m, M - m, factors of l and O
  static constexpr int kFac = kRefs + 2 * 4 * RT * 4;     // [2][RT] q factors, then [2][RT] visible limits
  static constexpr int kScale = kFac + 4 * RT * 4;        // [ring][8] k scale, [ring][8] log2 v scale
  static constexpr int kBars = kScale + kScaleRing * 16 * 4;
  static constexpr int kNBars = 2 * 8 + 4 * 2 + 2 * 4 + 2;   // full, empty [8]; s, p, pv, q [2]; vote, red [WG]; drain; one to spare
  static constexpr int kMisc = kBars + kNBars * 8;        // tmem base, abort, issued, -, flags[WG][2][4]
  static constexpr int kNan = kMisc + 16 + kWG * 32;      // [1 or 2 pieces][D]: first token of the piece with a NaN there
  static constexpr int kPre = kNan + (kWG > 1 ? 2 : 1) * D * 4;
  static constexpr int kFixed = kPre;                     // then pre [n + 1], lens [n]: sized by the call
  // the ring leaves room for the largest batch, or, where CTAs share an SM, for 256 sequences (more cost residency)
  static constexpr int kRoomFor = kB8MaxBatch < 256 || kCtas == 1 ? kB8MaxBatch : 256;
  static constexpr int kLimit = (kCtas == 1 ? 232448 : 233472 / kCtas - 1024) - 1024;   // less the alignment
  static constexpr int kFit = (kLimit - kFixed - (2 * kRoomFor + 1) * 4) / kTileBytes;
  static constexpr int kSlots = kFit > 8 ? 8 : kFit;
  static_assert(kSlots >= 4, "ring");
  static_assert(kBars % 8 == 0 && kMisc % 16 == 0 && kP % 1024 == 0 && kX % 1024 == 0 && kScale % 16 == 0, "alignment");
  static constexpr int kSmem = kSlots * kTileBytes + kFixed + 1024;
  // tcgen05 instruction descriptors: D fp32, A and B e4m3, M = 128
  static constexpr uint32_t kIdesc = (1u << 4) | (8u << 24);
  static constexpr uint32_t kIdescS = kIdesc | (uint32_t(kNS / 8) << 17);
  static constexpr uint32_t kIdescO = kIdesc | (3u << 15) | (uint32_t(kNP / 8) << 17);   // A and B are MN-major
  static constexpr uint64_t kSw = kW == 128 ? 2 : 4;      // descriptor's swizzle code: 128 or 64 bytes
};
// shared-memory operand descriptor; sbo: bytes between groups of 8 rows (K-major) or of 8 K-rows (MN-major,
// swizzled; without swizzle that is lbo, and sbo is the bytes between 16-byte groups of N)
__device__ __forceinline__ uint64_t sdesc(uint32_t addr, uint32_t lbo, uint32_t sbo, uint64_t swizzle) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFF) | (static_cast<uint64_t>(lbo >> 4) << 16) |
         (static_cast<uint64_t>(sbo >> 4) << 32) | (1ull << 46) | (swizzle << 61);
}

// ------------------------------------------------------------------ work
// kv tokens that the rows of row tile rt see, 0 .. len
__device__ __forceinline__ int kv_end(const B8AttnParams& p, int len, int rt, int RT) {
  const int last = p.by_G(min(p.rows, (rt + 1) * RT) - 1);
  return max(0, min(len, len - p.nq + last + 1));
}
__device__ __forceinline__ int clamp_len(const B8AttnParams& p, int len) { return min(max(len, 0), p.width * p.P); }
__device__ __forceinline__ int seq_len(const B8AttnParams& p, int b) { return clamp_len(p, p.lens[b]); }
__device__ __forceinline__ int tiles_of(const B8AttnParams& p, int len, int rt, int RT) {
  return (kv_end(p, len, rt, RT) + kB8Tile - 1) / kB8Tile;
}
struct Unit {
  int b, kvh, rt, len, tile0, tiles;
};
// the unit and the tile within it of global tile g; pre[b]: tiles of sequences before b (and lens behind it, in
// shared memory)
template <int RT>
__device__ __forceinline__ Unit unit_at(const B8AttnParams& p, const int* pre, int g) {
  const int* lens = pre + p.n + 1;
  int lo = 0, hi = p.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= g) lo = mid; else hi = mid - 1;
  }
  Unit u;
  u.b = lo;
  u.len = lens[lo];
  const int per = p.by_Hkv(pre[lo + 1] - pre[lo]);
  int rest = g - pre[lo];
  u.kvh = static_cast<int>(__fdividef(static_cast<float>(rest), static_cast<float>(per)));   // at most one off: below 4,096
  rest -= u.kvh * per;
  if (rest < 0) {
    --u.kvh;
    rest += per;
  } else if (rest >= per) {
    ++u.kvh;
    rest -= per;
  }
  u.rt = 0;
  u.tiles = tiles_of(p, u.len, 0, RT);
  while (rest >= u.tiles) {
    rest -= u.tiles;
    u.tiles = tiles_of(p, u.len, ++u.rt, RT);
  }
  u.tile0 = rest;
  return u;
}
// first tile, total c / ctas, of CTA c of min(p.ctas, total) (each has one tile at least: the join reads a piece of every
// CTA of a unit)
__device__ __forceinline__ int cta_first(const B8AttnParams& p, int total, int c) {
  if (total <= p.ctas) return c;
  const int each = p.by_ctas(total);                      // (total = each ctas + rest, and rest c fits 32 bits)
  return each * c + static_cast<int>(p.by_ctas((total - each * p.ctas) * c));
}
// the last CTA c with cta_first(c) <= g
__device__ __forceinline__ int cta_of(const B8AttnParams& p, int total, int g) {
  if (total <= p.ctas) return g;
  int c = static_cast<int>(__fdividef(static_cast<float>(g) * static_cast<float>(p.ctas), static_cast<float>(total)));
  while (cta_first(p, total, c) > g) --c;                 // (at most one off)
  while (c + 1 < p.ctas && cta_first(p, total, c + 1) <= g) ++c;
  return c;
}

// E consecutive elements (aligned to their own size) as floats
template <int E>
__device__ __forceinline__ void load_q(const void* q, bool f16, int64_t i, float (&x)[E]) {
  uint32_t w[E / 2];
  const uint16_t* at = static_cast<const uint16_t*>(q) + i;
  if constexpr (E == 8) *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(at);
  else if constexpr (E == 4) *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(at);
  else w[0] = *reinterpret_cast<const uint32_t*>(at);
#pragma unroll
  for (int k = 0; k < E / 2; ++k) {
    const float2 f = f16 ? __half22float2(*reinterpret_cast<const __half2*>(w + k))
                         : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(w + k));
    x[2 * k] = f.x;
    x[2 * k + 1] = f.y;
  }
}
__device__ __forceinline__ void store_out(void* out, bool f16, int64_t i, float v) {
  if (f16) static_cast<__half*>(out)[i] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
}

// Clears tokens `to` .. 127 of a V tile, and the NaNs of tokens `from` .. `to` - 1, whose places go to nan_from (thread t
// of 128; a call, so that its registers are not the softmax's).
template <int D>
__device__ __noinline__ void hide(uint8_t* tile, int t, int from, int to, int token0, int* nan_from) {
  constexpr int W = D < 128 ? D : 128;
  if (t >= to) {
#pragma unroll
    for (int d = 0; d < D / W; ++d) {
      uint4* row = reinterpret_cast<uint4*>(tile + d * kB8Tile * W + t * W);
#pragma unroll
      for (int i = 0; i < W / 16; ++i) row[i] = make_uint4(0, 0, 0, 0);
    }
  }
#pragma unroll 1
  for (int x = max(from, 0) * (D / 4) + t; x < min(to, kB8Tile) * (D / 4); x += 128) {   // four dims d0 .. of token k
    const int k = x / (D / 4), d0 = x % (D / 4) * 4;
    const int sw = W == 128 ? (k & 7) : ((k >> 1) & 3);
    uint32_t* at = reinterpret_cast<uint32_t*>(tile + d0 / W * kB8Tile * W + k * W + ((d0 % W) ^ (sw << 4)));
    uint32_t nan = __vcmpeq4(*at & 0x7f7f7f7fu, 0x7f7f7f7fu);
    if (!nan) continue;
    *at &= ~nan;
#pragma unroll 1
    for (int d = d0; nan; nan >>= 8, ++d)
      if (nan & 1) atomicMin(nan_from + d, token0 + k);
  }
}

// ------------------------------------------------------------------ kernel
template <int D, int RT, int QP>
__global__ void __launch_bounds__(Cfg<D, RT, QP>::kThreads, Cfg<D, RT, QP>::kCtas)
mkv_blk8_attn_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                     const __grid_constant__ B8AttnParams p) {
  using C = Cfg<D, RT, QP>;
  constexpr int kThreads = C::kThreads, kCopyWarp = C::kWG * 4, kMmaWarp = kCopyWarp + 1;
  extern __shared__ uint8_t raw[];
  uint8_t* const slots = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const fix = slots + C::kSlots * C::kTileBytes;
  uint8_t* const qbuf = fix + C::kQ;
  uint8_t* const pbuf = fix + C::kP;
  float* const xbuf = reinterpret_cast<float*>(fix + C::kX);
  float* const refs = reinterpret_cast<float*>(fix + C::kRefs);
  float* const qfac = reinterpret_cast<float*>(fix + C::kFac);
  int* const qlim = reinterpret_cast<int*>(qfac + 2 * RT);
  float* const kscale = reinterpret_cast<float*>(fix + C::kScale);
  float* const vscale = kscale + kScaleRing * 8;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(fix + C::kBars);
  uint64_t *const b_full = bars, *const b_empty = bars + 8, *const b_s = bars + 16, *const b_p = bars + 18,
           *const b_pv = bars + 20, *const b_q = bars + 22, *const b_votes = bars + 24, *const b_reds = bars + 28,
           *const b_drain = bars + 32;
  uint32_t* const misc = reinterpret_cast<uint32_t*>(fix + C::kMisc);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  int* const issued = reinterpret_cast<int*>(misc + 2);
  int* const flags = reinterpret_cast<int*>(misc + 4);    // [WG][2][4]
  int* const nan_from = reinterpret_cast<int*>(fix + C::kNan);
  int* const pre = reinterpret_cast<int*>(fix + C::kPre);
  int* const lens = pre + p.n + 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 32) {
    for (int i = 0; i < 8; ++i) {
      bar_init(b_full + i, 2);       // the copies' bytes, and the page scales beside a K tile
      bar_init(b_empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(b_s + i, 2);          // the MMAs' commit, and the issuing thread (it has seen the page scales)
      bar_init(b_p + i, C::kSoft);
      bar_init(b_pv + i, 1);
      bar_init(b_q + i, C::kSoft);
    }
    for (int i = 0; i < C::kWG; ++i) {
      bar_init(b_votes + i, 4);
      bar_init(b_reds + i, 4);
    }
    bar_init(b_drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    pre[0] = 0;
    *abort_flag = 0;
    *issued = 0;
  }
  if (warp == kCopyWarp && lane < 2)
    asm volatile("prefetch.tensormap [%0];" ::"l"(lane ? &vmap : &kmap) : "memory");
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sptr(misc)), "r"(C::kCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == 0) {
    // tile counts of the sequences, summed: 128 lengths at a time are on their way together
    int carry = 0;
    for (int b0 = 0; b0 < p.n; b0 += 128) {
      int len[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int b = b0 + 32 * i + lane;
        len[i] = b < p.n ? p.lens[b] : 0;
      }
#pragma unroll 1
      for (int i = 0; i < 4 && b0 + 32 * i < p.n; ++i) {
        const int b = b0 + 32 * i + lane;
        const int want = i == 0 ? len[0] : i == 1 ? len[1] : i == 2 ? len[2] : len[3], got = clamp_len(p, want);
        if (want > got && blockIdx.x == 0) atomicOr(p.err, kErrBadPage);
        int v = 0;
        for (int rt = 0; rt < p.row_tiles; ++rt) v += tiles_of(p, got, rt, RT);
        v = b < p.n ? v * p.Hkv : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int up = __shfl_up_sync(kFull, v, o);
          if (lane >= o) v += up;
        }
        v += carry;
        if (b < p.n) {
          pre[b + 1] = v;
          lens[b] = got;
        }
        carry = __shfl_sync(kFull, v, 31);
      }
    }
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = misc[0];
  const int total = pre[p.n];
  if (blockIdx.x == 0)
    for (int b = tid; b <= p.n; b += kThreads) p.plan[b] = pre[b];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int ctas = min(p.ctas, total), cta = min(static_cast<int>(blockIdx.x), ctas);   // (CTAs past the tiles: none)
  const int g0 = cta_first(p, total, cta), g1 = cta < ctas ? cta_first(p, total, cta + 1) : g0;

  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (bar_try(bar, parity)) return true;
    const long long t0 = clock64();
    for (;;) {
      if (*abort_flag) return false;
      if (bar_try(bar, parity)) return true;
      if (clock64() - t0 > kWaitCycles) {
        atomicOr(p.err, kErrWaitTimeout);
        *abort_flag = 1;
        return false;
      }
    }
  };

  const int T = g1 - g0;                                  // tiles of this CTA
  const int pshift = 31 - __clz(p.P);                     // tokens of a page: a power of two
  if (warp == kCopyWarp) {
    // ============================================================ copies
    const int ppt = kB8Tile >> pshift;                    // pages of a tile, one a lane
    uint64_t policy;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    struct At {
      int g, left, b, kvh, tile, end;
    };
    auto enter = [&](At& a) {
      const Unit u = unit_at<RT>(p, pre, a.g);
      a.left = u.tiles - u.tile0;
      a.b = u.b;
      a.kvh = u.kvh;
      a.tile = u.tile0;
      a.end = kv_end(p, u.len, u.rt, RT);
    };
    auto step = [&](At& a) {
      ++a.g;
      ++a.tile;
      if (--a.left == 0 && a.g < g1) enter(a);
    };
    // the page of this lane in the tile: -1 where the lane has none
    auto page_of = [&](const At& a) -> int {
      const int pg = a.tile * ppt + lane;
      if (a.g >= g1 || lane >= ppt || pg * p.P >= a.end) return -1;
      const int id = p.table[static_cast<int64_t>(a.b) * p.width + pg];
      return id < 0 || id >= p.pages ? -2 : id;
    };
    if (T > 0) {
      At a{g0, 0, 0, 0, 0, 0};
      enter(a);
      At ahead = a;
      int id = page_of(a), id1, id2, was = -1, was_z = 0;
      step(ahead);
      id1 = page_of(ahead);
      auto scale = [&](const float* s, int page, int kvh) { return page >= 0 ? s[static_cast<int64_t>(page) * p.Hkv + kvh] : 0.f; };
      float ks = scale(p.k_scale, id, a.kvh), vs = scale(p.v_scale, id, a.kvh);
      At next = ahead;                                    // tile j + 1; `ahead` runs to tile j + 2
      int used = 0;
      auto issue = [&](const CUtensorMap* map, int page, int z) -> bool {
        const int slot = used % C::kSlots, round = used / C::kSlots;
        if (!__all_sync(kFull, round == 0 || wait(b_empty + slot, (round - 1) & 1))) return false;
        const uint32_t have = __ballot_sync(kFull, page >= 0);
        if (lane == 0) {
          bar_expect(b_full + slot, __popc(have) * p.P * D);
          *issued = used + 1;
        }
        __syncwarp();
        if (page >= 0) {
#pragma unroll
          for (int s = 0; s < C::kSub; ++s)
            tma_page(slots + slot * C::kTileBytes + s * C::kSubBytes + lane * p.P * C::kW, map, s * 128, z, b_full + slot, policy);
        }
        ++used;
        return true;
      };
      // the second arrival of the tile just issued: this warp's stores so far are seen by who waits for it
      auto release = [&]() {
        __syncwarp();
        if (lane == 0) bar_arrive(b_full + (used - 1) % C::kSlots);
      };
      for (int j = 0; j <= T; ++j) {
        if (j < T) {
          if (__any_sync(kFull, id == -2)) {              // a page outside the cache: nothing of the tile is read
            if (lane == 0) {
              atomicOr(p.err, kErrBadPage);
              *abort_flag = 1;
            }
            break;
          }
          const float nk = scale(p.k_scale, id1, next.kvh), nv = scale(p.v_scale, id1, next.kvh);
          step(ahead);
          id2 = page_of(ahead);
          const int z = (p.page0 + id) * p.Hkv + a.kvh;
          if (!issue(&kmap, id, z)) break;
          if (lane < ppt) {
            kscale[(j & (kScaleRing - 1)) * 8 + lane] = ks;
            vscale[(j & (kScaleRing - 1)) * 8 + lane] = __log2f(vs) + kUp;
          }
          release();
          if (j > 0) {
            if (!issue(&vmap, was, was_z)) break;
            release();
          }
          was = id;
          was_z = z;
          id = id1;
          id1 = id2;
          ks = nk;
          vs = nv;
          a = next;
          next = ahead;
        } else {
          if (!issue(&vmap, was, was_z)) break;
          release();
        }
      }
      // the MMAs' last arrivals land before the CTA's shared memory goes
      for (int k = max(0, used - C::kSlots); k < used && !*abort_flag; ++k) wait(b_empty + k % C::kSlots, (k / C::kSlots) & 1);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ============================================================ MMAs
    if (lane == 0 && T > 0) {
      const uint64_t dk = sdesc(sptr(slots), 16, 8 * C::kW, C::kSw), dv = sdesc(sptr(slots), 8 * C::kW, 8 * C::kW, C::kSw),
                     dq = sdesc(sptr(qbuf), 16, 8 * C::kW, C::kSw), dp = sdesc(sptr(pbuf), 128, 2048, 0);
      int used = 0, piece = -1, left = 0, g = g0;
      bool o_new = true, pv_new = true;
      auto full = [&]() { return wait(b_full + used % C::kSlots, (used / C::kSlots) & 1); };
      for (int j = 0; j <= T; ++j) {
        if (j < T) {
          const bool first = left == 0;
          if (first) {                                    // a new piece: its query rows
            const Unit u = unit_at<RT>(p, pre, g);
            left = min(u.tiles - u.tile0, g1 - g);
            g += left;
            ++piece;
            if (!wait(b_q + (piece & 1), (piece >> 1) & 1)) break;
          }
          --left;
          if (!full()) break;
          tc_after();
          // (an address field counts 16 bytes and has no carry out: shared memory ends below 2^18)
          const uint64_t ka = dk + (used % C::kSlots) * (C::kTileBytes / 16), qq = dq + (piece & 1) * (C::kQBytes / 16);
#pragma unroll
          for (int s = 0; s < C::kSub; ++s)
#pragma unroll
            for (int k = 0; k < C::kW / 32; ++k)
              tc_mma(tmem + (j & 1) * C::kNS, ka + (s * C::kSubBytes + k * 32) / 16, qq + (s * C::kQSub + k * 32) / 16,
                     C::kIdescS, s | k);
          tc_commit(b_s + (j & 1));
          bar_arrive(b_s + (j & 1));
          tc_commit(b_empty + used % C::kSlots);
          ++used;
          o_new = first;
        }
        if (j > 0) {                                      // the weights of tile j - 1
          const int i = j - 1;
          if (!wait(b_p + (i & 1), (i >> 1) & 1)) break;
          if (!full()) break;
          tc_after();
          const uint64_t va = dv + (used % C::kSlots) * (C::kTileBytes / 16), pp = dp + (i & 1) * (C::kPBytes / 16);
#pragma unroll
          for (int s = 0; s < C::kSub; ++s)
#pragma unroll
            for (int k = 0; k < kB8Tile / 32; ++k)
              tc_mma(tmem + C::kTO + s * C::kNP, va + (s * C::kSubBytes + k * 32 * C::kW) / 16, pp + k * 512 / 16, C::kIdescO,
                     (pv_new && k == 0) ? 0u : 1u);
          tc_commit(b_empty + used % C::kSlots);
          tc_commit(b_pv + (i & 1));
          ++used;
        }
        pv_new = o_new;                                   // PV lags QK by one tile
      }
    }
    __syncwarp();
  } else {
    // ============================================================ softmax: thread t is token t of the tile
    constexpr int R = C::kRows;
    const int wg = C::kWG > 1 ? warp >> 2 : 0, w4 = warp & 3, t = tid & 127, row0 = wg * R;   // this warpgroup's rows
    const uint32_t lanes = static_cast<uint32_t>(w4 * 32) << 16;
    uint64_t *const b_vote = b_votes + wg, *const b_red = b_reds + wg;
    float* const my_x = xbuf + wg * R * 128;
    int* const my_flags = flags + wg * 8;
    bool ok = true;
    // query rows of a unit -> parts in qbuf[i & 1], factors and limits
    auto prepare = [&](int i, const Unit& u) {
      uint8_t* dst = qbuf + (i & 1) * C::kQBytes;
      constexpr int E = D / 32;                           // elements of a lane
      float next[E];                                      // the next row's elements, on their way
      int qi = 0, next_qi = 0;
      auto fetch = [&](int r) {
        const int row = u.rt * RT + r;
#pragma unroll
        for (int e = 0; e < E; ++e) next[e] = 0.f;
        if (r >= row0 + R || row >= p.rows) return;
        next_qi = p.by_G(row);
        load_q<E>(p.q, p.q_f16,
                  ((static_cast<int64_t>(u.b) * p.nq + next_qi) * p.Hq + u.kvh * p.G + (row - next_qi * p.G)) * D + lane * E, next);
      };
      fetch(row0 + w4);
#pragma unroll 1
      for (int r = row0 + w4; r < row0 + R; r += 4) {     // its own rows: the other warpgroup may be a piece behind
        const bool have = u.rt * RT + r < p.rows;
        float x[E];
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = next[e];
        qi = next_qi;
        fetch(r + 4);
        float amax = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) amax = fmaxf(amax, fabsf(x[e]));
        amax = warp_max(amax);
        // amax 2^ex in [128, 256); a subnormal amax is brought up by 2^126
        const int ex = min(134 - static_cast<int>(__float_as_uint(amax) >> 23), 126);
        const float up = __uint_as_float(static_cast<uint32_t>(ex + 127) << 23);
        const float down = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
        uint32_t part[QP][(E + 3) / 4];
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] *= up;
#pragma unroll
        for (int k = 0; k < QP; ++k) {
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            const uint32_t two = e4m3x2(x[e], x[e + 1]);
            const float2 f = from_e4m3x2(two);
            x[e] = (x[e] - f.x) * 16.f;
            x[e + 1] = (x[e + 1] - f.y) * 16.f;
            part[k][e / 4] = (e & 2) ? part[k][e / 4] | (two << 16) : two;
          }
          const int n = QP * r + k, col = (lane * E) % C::kW;
          const int sw = C::kW == 128 ? (n & 7) : ((n >> 1) & 3);
          uint8_t* to = dst + (lane * E) / C::kW * C::kQSub + n * C::kW + (((col >> 4) ^ sw) << 4) + (col & 15);
          if constexpr (E == 8) *reinterpret_cast<uint2*>(to) = make_uint2(part[k][0], part[k][1]);
          else if constexpr (E == 4) *reinterpret_cast<uint32_t*>(to) = part[k][0];
          else *reinterpret_cast<uint16_t*>(to) = static_cast<uint16_t>(part[k][0]);
        }
        if (lane == 0) {
          qfac[(i & 1) * RT + r] = amax < INFINITY ? down * p.scale_log2 : NAN;   // (e4m3 has no infinity: its row is NaN)
          qlim[(i & 1) * RT + r] = have ? min(u.len, u.len - p.nq + qi + 1) : kv_end(p, u.len, u.rt, RT);
        }
      }
      proxy_fence();
      bar_arrive(b_q + (i & 1));
    };
    int votes = 0, reds = 0;                              // uses of the exchange barriers
    auto meet = [&](uint64_t* bar, int& uses) {           // a warpgroup's warps (their stores before it are seen after)
      __syncwarp();
      if (lane == 0) bar_arrive(bar);
      ok = __all_sync(kFull, wait(bar, uses & 1));
      ++uses;
      return ok;
    };
    int gnext = g0, j = 0, cnt = 0;
    Unit u{};
    for (int piece = -1; T > 0 && ok; ++piece) {          // (piece -1 has no tiles: it prepares the first)
      Unit nu{};
      int ncnt = 0;                                       // the next piece's tiles; 0 behind the last
      float m[R], md[R], l[R];                            // m, M - m, the sum
#pragma unroll
      for (int r = 0; r < R; ++r) {
        m[r] = kNone;
        md[r] = l[r] = 0.f;
      }
      // the references again, for the rolled loops (another buffer than the last piece's, which may still be read)
      float* const my_refs = refs + ((piece & 1) * C::kWG + wg) * 4 * R;
      if (t < 2 * R) my_refs[t] = t < R ? kNone : 0.f;
      int* const my_nan = nan_from + (C::kWG > 1 ? (piece & 1) * D : 0);    // (one warpgroup: a thread resets what it read)
      if (wg == 0)
        for (int d = t; d < D; d += 128) my_nan[d] = INT_MAX;
      const float* fac = qfac + (piece & 1) * RT + row0;
      const int* lim = qlim + (piece & 1) * RT + row0;
      const int end = kv_end(p, u.len, u.rt, RT);
      const int first_lim = u.len - p.nq + static_cast<int>(p.by_G(u.rt * RT)) + 1;   // the least limit of the tile's rows
#pragma unroll 1
      for (int c = 0;; ++c, ++j) {
        if (c == min(cnt, 1) && gnext < g1) {             // the next piece's query rows, behind this one's first tile
          nu = unit_at<RT>(p, pre, gnext);
          ncnt = min(nu.tiles - nu.tile0, g1 - gnext);
          gnext += ncnt;
          prepare(piece + 1, nu);
        }
        if (c >= cnt) break;
        const int buf = j & 1;
        if (!(ok = __all_sync(kFull, wait(b_s + buf, (j >> 1) & 1)))) break;
        if (j >= 2 && !(ok = __all_sync(kFull, wait(b_pv + buf, ((j >> 1) - 1) & 1)))) break;
        tc_after();
        const int tile = u.tile0 + c, tok = tile * kB8Tile + t;
        const int ring = (j & (kScaleRing - 1)) * 8 + (t >> pshift);
        const float ks = kscale[ring], lv = vscale[ring];
        float a[R], d1[R], d2[R];                         // q . K; exponents of the weight for the sum and for the codes
        {
          float v[QP * R];
          tm_ld<QP * R>(tmem + lanes + buf * C::kNS + QP * row0, v);
          tm_wait_ld(v);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            a[r] = v[QP * r + QP - 1];
#pragma unroll
            for (int k = QP - 2; k >= 0; --k) a[r] = fmaf(a[r], 0.0625f, v[QP * r + k]);
          }
        }
        uint32_t hidden = 0;                              // rows that do not see this token
        if (tile * kB8Tile + kB8Tile > first_lim) {
#pragma unroll
          for (int r = 0; r < R; ++r) hidden |= static_cast<uint32_t>(tok >= lim[r]) << r;
        }
        for (bool raised = false;; raised = true) {       // twice when the references rise
          float most1 = -INFINITY, most2 = -INFINITY;
#pragma unroll
          for (int r = 0; r < R; ++r) {
            d1[r] = __fmul_rn(a[r], fac[r] * ks) - m[r];  // (the score that m was taken from, not a more exact one)
            d2[r] = d1[r] + (lv - md[r]);
          }
          if (hidden) {
#pragma unroll
            for (int r = 0; r < R; ++r)
              if (hidden >> r & 1) d1[r] = d2[r] = -INFINITY;
          }
#pragma unroll
          for (int r = 0; r < R; ++r) {
            most1 = fmaxf(most1, d1[r]);
            most2 = fmaxf(most2, d2[r]);
          }
          if (raised) break;
          const bool any = __any_sync(kFull, most1 > kRise || most2 > kRise + kUp);
          int* const flag = my_flags + (votes & 1) * 4;
          if (lane == 0) flag[w4] = any;
          if (!meet(b_vote, votes)) break;
          const int4 f4 = *reinterpret_cast<const int4*>(flag);
          if (!(f4.x | f4.y | f4.z | f4.w)) break;
          // raise the references: the scores to shared memory, a warp a row
#pragma unroll
          for (int r = 0; r < R; ++r) my_x[r * 128 + t] = hidden >> r & 1 ? -INFINITY : __fmul_rn(a[r], fac[r] * ks);
          if (!meet(b_red, reds)) break;
          const float lv4 = vscale[(j & (kScaleRing - 1)) * 8 + (4 * lane >> pshift)] - kUp;    // of the page of tokens 4 lane ..
#pragma unroll 1
          for (int r = w4; r < R; r += 4) {
            const float4 x = *reinterpret_cast<const float4*>(my_x + r * 128 + 4 * lane);
            const float top = fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w));
            const float om = my_refs[r], od = my_refs[R + r];
            float nm = fmaxf(om, warp_max(top) + kRoom);
            if (nm == INFINITY) nm = NAN;                 // a score that overflowed: its row is NaN from here on
            const float nd = fmaxf(od + (om - nm), warp_max((top - nm) + lv4) + kRoom);
            if (lane == 0) {
              my_refs[r] = nm;
              my_refs[R + r] = nd;
              my_refs[2 * R + r] = ex2(om - nm);
              my_refs[3 * R + r] = ex2((om - nm) + (od - nd));
            }
          }
          if (!meet(b_red, reds)) break;
#pragma unroll
          for (int r = 0; r < R; ++r) {
            m[r] = my_refs[r];
            md[r] = my_refs[R + r];
            l[r] *= my_refs[2 * R + r];
          }
          if (c > 0) {
            if (!(ok = __all_sync(kFull, wait(b_pv + (buf ^ 1), ((j - 1) >> 1) & 1)))) break;
            tc_after();
#pragma unroll 1
            for (int i = 0; i < R / 4 * C::kSub; ++i) {   // four rows of O, 128 dims
              const int r0 = i / C::kSub * 4, d = i % C::kSub;
              const uint32_t at = tmem + lanes + C::kTO + d * C::kNP + wg * C::kPG * 16 + kWP * r0;
              const float4 fo = *reinterpret_cast<const float4*>(my_refs + 3 * R + r0);
              float o[4 * kWP];
              tm_ld<4 * kWP>(at, o);
              tm_wait_ld(o);
#pragma unroll
              for (int k = 0; k < 4 * kWP; ++k)
                o[k] *= k / (2 * kWP) ? (k % 2 ? fo.w : fo.z) : (k % 2 ? fo.y : fo.x);
              tm_st<4 * kWP>(at, o);
            }
            tm_wait_st();
          }
        }
        if (!ok) break;
        // weights: byte n = kWP (r - r % 2) + 2 part + r % 2 of this token's row, 16 bytes a group
        uint32_t words[4 * C::kPG];
#pragma unroll
        for (int i = 0; i < 4 * C::kPG; ++i) words[i] = 0;
#pragma unroll
        for (int r = 0; r < R; r += 2) {
          l[r] += ex2(d1[r]);
          l[r + 1] += ex2(d1[r + 1]);
          __half2 w = __floats2half2_rn(ex2(d2[r]), ex2(d2[r + 1]));
#pragma unroll
          for (int k = 0; k < kWP; ++k) {                 // (a remainder past e4m3's range is cut to it: it only errs less)
            const int hw = kWP * r / 2 + k;
            const uint32_t two = e4m3x2(w);
            words[hw / 2] |= two << (16 * (hw % 2));
            if (k + 1 < kWP) w = __hmul2(__hsub2(w, half2_of(two)), __float2half2_rn(part_step(k + 1)));
          }
        }
#pragma unroll
        for (int i = 0; i < C::kPG; ++i)
          *reinterpret_cast<uint4*>(pbuf + buf * C::kPBytes + (wg * C::kPG + i) * 2048 + t * 16) =
              make_uint4(words[4 * i], words[4 * i + 1], words[4 * i + 2], words[4 * i + 3]);
        if (wg == 0 && tile * kB8Tile + kB8Tile > first_lim) {
          // What a row does not see may be any code, and weight 0 does not silence a NaN, so this changes V in shared
          // memory (the slot is this tile's until its PV is done): tokens past the last one are cleared, and so are
          // the NaNs of tokens that some rows of the tile see; those rows get them back at the piece's end.
          const int vn = j < T - 1 ? 2 * j + 2 : 2 * j + 1;
          if (!(ok = __all_sync(kFull, wait(b_full + vn % C::kSlots, (vn / C::kSlots) & 1)))) break;
          hide<D>(slots + (vn % C::kSlots) * C::kTileBytes, t, first_lim - tile * kB8Tile, end - tile * kB8Tile, tile * kB8Tile,
                  my_nan);
        }
        proxy_fence();
        tc_before();
        bar_arrive(b_p + buf);
      }
      if (!ok) break;
      if (piece >= 0) {
        // ---------------------------------------------------------- the piece's rows
#pragma unroll
        for (int r = 0; r < R; ++r) my_x[r * 128 + t] = l[r];
        if (!meet(b_red, reds)) break;
#pragma unroll 1
        for (int r = w4; r < R; r += 4) {
          const float4 x = *reinterpret_cast<const float4*>(my_x + r * 128 + 4 * lane);
          float sum = (x.x + x.y) + (x.z + x.w);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
          if (lane == 0) my_refs[2 * R + r] = sum;
        }
        if (!meet(b_red, reds)) break;
        if (!(ok = __all_sync(kFull, wait(b_pv + ((j - 1) & 1), ((j - 1) >> 1) & 1)))) break;
        tc_after();
        const bool whole = cnt == u.tiles;
        const int slot = 2 * blockIdx.x + (piece ? 1 : 0);
        int nan_at[C::kSub];
#pragma unroll
        for (int d = 0; d < C::kSub; ++d) nan_at[d] = my_nan[d * 128 + min(t, C::kW - 1)];
#pragma unroll 1
        for (int r0 = 0; r0 < R && u.rt * RT + row0 + r0 < p.rows; r0 += 4) {
          float o[C::kSub][4 * kWP];
#pragma unroll
          for (int d = 0; d < C::kSub; ++d) tm_ld<4 * kWP>(tmem + lanes + C::kTO + d * C::kNP + wg * C::kPG * 16 + kWP * r0, o[d]);
#pragma unroll
          for (int d = 0; d < C::kSub; ++d) tm_wait_ld(o[d]);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int rr = r0 + r, row = u.rt * RT + row0 + rr;
            if (row >= p.rows) break;
            const float mr = my_refs[rr], L = my_refs[2 * R + rr];
            const bool empty = L == 0.f;                    // no token that counts; of a whole unit:
            const bool lost = whole && empty && lim[rr] > 0;        // tokens, but all their scores fell below kNone
            // O holds 2^kUp times the weights, relative to M
            float f = ex2(my_refs[R + rr] - kUp);
            if (whole) f = f / L;
            float out[C::kSub];
#pragma unroll
            for (int d = 0; d < C::kSub; ++d) {
              const float* c4 = o[d] + r / 2 * 2 * kWP + r % 2;     // the row's parts lie two columns apart
              out[d] = c4[2 * (kWP - 1)];
#pragma unroll
              for (int k = kWP - 2; k >= 0; --k) out[d] = fmaf(out[d], 1.f / part_step(k + 1), c4[2 * k]);
              out[d] = empty ? 0.f : out[d] * f;
              if (lim[rr] > nan_at[d] || lost) out[d] = NAN;
            }
            if (whole) {
              const int qi = p.by_G(row);
              const int64_t hrow = (static_cast<int64_t>(u.b) * p.nq + qi) * p.Hq + u.kvh * p.G + (row - qi * p.G);
#pragma unroll
              for (int d = 0; d < C::kSub; ++d)
                if (t < C::kW) store_out(p.out, p.q_f16, hrow * D + d * 128 + t, out[d]);
              if (t == 0) p.lse[hrow] = lost ? NAN : empty ? -INFINITY : (mr + log2f(L)) * 0.69314718055994530942f;
            } else {
              float* to = p.part + (static_cast<int64_t>(slot) * RT + row0 + rr) * (D + 4);
#pragma unroll
              for (int d = 0; d < C::kSub; ++d)
                if (t < C::kW) to[d * 128 + t] = out[d];
              if (t == 0) *reinterpret_cast<float2*>(to + D) = make_float2(mr, L);
            }
          }
        }
        tc_before();                                        // (the next piece's first weights order its PV behind this)
        __syncwarp();
      }
      if (ncnt == 0) break;
      u = nu;
      cnt = ncnt;
    }
  }
  __syncthreads();
  if (*abort_flag) {                                      // leave nothing in flight: the copies, then the MMAs
    if (tid == 0) {
      const int n = *issued;
      for (int k = max(0, n - C::kSlots); k < n; ++k) {
        const long long t0 = clock64();
        while (!bar_try(b_full + k % C::kSlots, (k / C::kSlots) & 1) && clock64() - t0 < kWaitCycles) {}
      }
    }
    if (tid == kMmaWarp * 32) {
      tc_commit(b_drain);
      const long long t0 = clock64();
      while (!bar_try(b_drain, 0) && clock64() - t0 < kWaitCycles) {}
    }
    __syncthreads();
  }
  tc_before();
  __syncthreads();
  tc_after();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kCols) : "memory");
}

// ------------------------------------------------------------------ join
// One block per (sequence, query token, query head): the rows of units that several CTAs share, and the rows of units
// without a tile (nothing is visible: out 0, lse -inf).  Bound: latency, a chain of three loads (the tile counts, the
// pieces' m and l, their rows); the four warps take the pieces in turn, eight rows in flight each, a lane four dims of
// every 128, and add up in shared memory.
constexpr int kJoinWarps = 4;
template <int D, int RT>
__global__ void __launch_bounds__(32 * kJoinWarps) mkv_blk8_join_kernel(const __grid_constant__ B8AttnParams p) {
  constexpr int kV = (D + 127) / 128;                     // float4 of a lane
  __shared__ __align__(16) float sums[kJoinWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t hrow = blockIdx.x;
  const uint32_t bq = p.by_Hq(hrow), hq = hrow - bq * p.Hq, b = p.by_nq(bq), qi = bq - b * p.nq;
  const int kvh = p.by_G(hq), row = qi * p.G + hq - kvh * p.G, rt = row / RT;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int total = p.plan[p.n], base = p.plan[b], per = p.by_Hkv(p.plan[b + 1] - base);
  const int len = seq_len(p, b);
  const int tiles = tiles_of(p, len, rt, RT);
  int c0 = 0, pieces = 0, ga = base + kvh * per;
  if (tiles > 0) {
    for (int i = 0; i < rt; ++i) ga += tiles_of(p, len, i, RT);
    c0 = cta_of(p, total, ga);
    pieces = cta_of(p, total, ga + tiles - 1) - c0 + 1;
    if (pieces == 1) return;                              // written by its CTA
  }
  const int64_t stride = static_cast<int64_t>(2) * RT * (D + 4);       // of a CTA's two pieces
  // the first CTA's piece is its second one unless the unit starts its range; the others' is their first
  const float* part = p.part + c0 * stride + static_cast<int64_t>(row - rt * RT) * (D + 4);
  const int64_t first = cta_first(p, total, c0) == ga ? 0 : stride / 2;
  const bool mine = D >= 128 || lane < D / 4;
  // lane i weighs piece i of 32
  float M = kNone, L = 0.f, o[4 * kV];
#pragma unroll
  for (int x = 0; x < 4 * kV; ++x) o[x] = 0.f;
  for (int i0 = 0; i0 < pieces; i0 += 32) {
    const int i = i0 + lane, cnt = min(32, pieces - i0);
    float4 v[8][kV];
#pragma unroll
    for (int k = 0; k < 8; ++k) {                         // (past the last piece that one again, with weight 0: no branch)
      const int n = min(i0 + kJoinWarps * k + warp, pieces - 1);
      const float* q = part + (n ? n * stride : first) + (mine ? 4 * lane : 0);
#pragma unroll
      for (int x = 0; x < kV; ++x) v[k][x] = *reinterpret_cast<const float4*>(q + 128 * x);
    }
    const float2 ml = i < pieces ? *reinterpret_cast<const float2*>(part + (i ? i * stride : first) + D) : make_float2(kNone, 0.f);
    const float top = fmaxf(M, warp_max(ml.x));
    const float w = i < pieces ? ex2(ml.x - top) : 0.f, keep = ex2(M - top);
    float sum = w * ml.y;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(kFull, sum, x);
    L = fmaf(L, keep, sum);
    M = top;
#pragma unroll
    for (int x = 0; x < 4 * kV; ++x) o[x] *= keep;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float wk = __shfl_sync(kFull, w, kJoinWarps * k + warp);
      if (kJoinWarps * k + warp < cnt) {
#pragma unroll
        for (int x = 0; x < kV; ++x) {
          o[4 * x] = fmaf(v[k][x].x, wk, o[4 * x]);
          o[4 * x + 1] = fmaf(v[k][x].y, wk, o[4 * x + 1]);
          o[4 * x + 2] = fmaf(v[k][x].z, wk, o[4 * x + 2]);
          o[4 * x + 3] = fmaf(v[k][x].w, wk, o[4 * x + 3]);
        }
      }
    }
  }
  if (mine) {
#pragma unroll
    for (int x = 0; x < kV; ++x)
      *reinterpret_cast<float4*>(&sums[warp][128 * x + 4 * lane]) = make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
  }
  __syncthreads();
  const bool empty = L == 0.f;
  const float none = len - p.nq + static_cast<int>(qi) + 1 > 0 ? NAN : 0.f;      // (tokens, but no score above kNone; or no token)
#pragma unroll
  for (int d = threadIdx.x; d < D; d += 32 * kJoinWarps)
    store_out(p.out, p.q_f16, static_cast<int64_t>(hrow) * D + d,
              empty ? none : ((sums[0][d] + sums[1][d]) + (sums[2][d] + sums[3][d])) / L);
  if (threadIdx.x == 0) p.lse[hrow] = empty ? (none == 0.f ? -INFINITY : none) : (M + log2f(L)) * 0.69314718055994530942f;
}

template <int D, int RT, int QP>
cudaError_t go(const CUtensorMap& k, const CUtensorMap& v, const B8AttnParams& p, cudaStream_t s) {
  using C = Cfg<D, RT, QP>;
  // the shared-memory limit is a per-device attribute: set once per device (twice from racing threads is harmless)
  static std::atomic<uint64_t> set{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!bit || !(set.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(mkv_blk8_attn_kernel<D, RT, QP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::kSmem + (2 * kB8MaxBatch + 1) * 4);
    if (e != cudaSuccess) return e;
    set.fetch_or(bit, std::memory_order_acq_rel);
  }
  mkv_blk8_attn_kernel<D, RT, QP><<<p.ctas, C::kThreads, C::kSmem + (2 * p.n + 1) * 4, s>>>(k, v, p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(p.n) * unsigned(p.nq) * unsigned(p.Hq));
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, mkv_blk8_join_kernel<D, RT>, p);
}

template <int D>
cudaError_t pick(const CUtensorMap& k, const CUtensorMap& v, const B8AttnParams& p, cudaStream_t s) {
  switch (b8_row_tile(p.rows, D, p.q_f16)) {
    case 8: return p.q_f16 ? go<D, 8, 3>(k, v, p, s) : go<D, 8, 2>(k, v, p, s);
    case 16: return p.q_f16 ? go<D, 16, 3>(k, v, p, s) : go<D, 16, 2>(k, v, p, s);
    case 24: return p.q_f16 ? go<D, 24, 3>(k, v, p, s) : go<D, 24, 2>(k, v, p, s);
    default:
      if constexpr (D < 256) {
        if (p.q_f16) return go<D, 32, 3>(k, v, p, s);
      }
      return go<D, 32, 2>(k, v, p, s);
  }
}

}  // namespace b8
}  // namespace mkv
