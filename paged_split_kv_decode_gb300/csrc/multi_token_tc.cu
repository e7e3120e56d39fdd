// Attention of several new tokens a request on the 5th-generation tensor cores
// (tcgen05.mma kind::f16: bf16 operands, f16 with fp8 pools; f32 accumulators in TMEM).
//
// Rows.  The G query heads of one KV head and the request's new tokens are stacked
// token-major into row tiles of TH = floor(128 / G) tokens (TH * G <= 128 TMEM lanes), so
// every K/V element crosses into shared memory once for up to 256 rows.  A unit is one
// (request, KV head, one or two row tiles); its work is its key tiles of NK tokens.
//
// Split.  The key tiles of all units lie on one line, request by request and KV head by KV
// head, and each CTA takes a stretch of it that costs the same (a unit costs some tiles beside
// its own: Lay): every SM gets its share whatever the lengths, with one CTA per SM and no
// second wave.  The host finds where the stretches begin.  A stretch that
// holds a whole unit writes its output; a piece of a unit writes a normalised partial
// and its LSE to the workspace (at most two pieces a CTA, so the workspace does not
// grow with the batch), and a second kernel joins the pieces of each split unit in key
// order.  Nothing is added atomically: results repeat bit for bit.
//
// Pipeline.  Two softmax slots alternate on the tensor cores: op t is S = Q K^T and, after
// the slot's warpgroup has turned S into P, O += P V; while one slot's rows take their
// softmax the other slot's MMAs run.  A unit of two row tiles gives each slot one of them
// (op 2j and 2j + 1 share key tile j); a unit of one row tile gives the slots its even and
// odd key tiles, with an O, maximum and sum each, joined when the unit ends.  Each slot has an
// MMA thread, which issues S(t + 2) right after P V(t): they use the same TMEM columns (P lies
// over S), and a thread's MMAs execute in issue order.
// A tile's P goes in parts of 64 keys, so that PV of the first runs while the second is made.
//   TMEM (512 columns): per slot S [128 x NK] f32 with P over it, and O [128 x D] f32.
//   Shared memory: two row tiles of Q (fp8 pools: none), a ring of K and V half-tiles (K, V, ...).
//   Warps: 0-3 softmax of slot 0, 4-7 of slot 1 (thread = row = TMEM lane), 8 and 11 (one
//   thread each) the MMAs of the slots, 9 loads Q and K, 10 loads V.
//
// Tiles are read by TMA through a 5-D view of the pool, [groups of 8 token slots][KV head]
// [64-column halves][8 slots][64 columns], whose box of a page's part lands as complete
// 128-byte-swizzle atoms: one copy carries a whole head row (both halves at D = 128) of up
// to 128 slots of a page.  Page positions past the request's pages load as zeros.
//
// fp8 pools: the copies bring codes (swizzled rows of a head) into a ring of their own, and eight more
// warps (12-19) turn them into f16 tiles of 64 keys in the layout above, half-tile by half-tile: one
// conversion for two codes, where bf16 takes four.  Q lies in TMEM, D / 2 columns a slot, written by
// the softmax warps as f16 scaled row by row: S of 64 keys reads K alone from shared memory, which
// copies, conversion and MMAs otherwise fill.  With bf16 operands and Q in shared memory 16 requests'
// trees of 9 to 24 tokens over 512 to 8192 keys took 61 us against 54.  (K's codes taken as they are by
// kind::f8f6f4, against Q in two e4m3 terms, were no faster.)
//
// Precision.  S and O are f32.  P meets V as TERMS bf16 terms: one for bf16 outputs (P off
// by at most 2^-8 of itself, as the output is), three for f32 outputs (24 bits).  Three
// terms of NK keys need 3 NK / 2 columns, which is why f32 outputs take tiles of 64 keys.
// With fp8 pools the terms are f16: one (2^-11) or two (2^-22; with O, S and Q there is no room
// for a third), and P's scale is 2^7 higher, so that what f16 loses at its low end is 2^-32 of
// the row's largest P.
// The tensor cores' f32 accumulation cuts low bits at every step of 16 keys and term, always
// towards zero: over 8000 keys it cost 1.3e-5 of the result's norm.  bf16 outputs do not
// see that; for f32 outputs O starts anew every kFlush ops of a slot (36 steps), and the rows add
// what they read out to a sum in the workspace, rounded to nearest.  3 single tokens over 20000 to
// 65536 keys: 8e-7 of the norm and 127 us, against 3.5e-6 and 113 us with 16 ops and 5e-7 and
// some 180 us with one.
// The row maximum follows lazily: O and l are rescaled only when it grows by more than
// 2^8, so P <= 2^8 (2^15 as f16).
//
// Measured, 32 query and 8 KV heads of 128, cold caches, the join beside it: 32 requests of 5 tokens
// over 512 to 4096 keys 55 + 5 us (286 MB, 0.77 of a plain copy's rate: copies bound it); with f32
// outputs 85 + 6 us (322 MB); 3 single tokens over 20000 to 65536 keys, f32 outputs, 126 + 8 us (0.75); a
// 4096-token chunk over 4096 283 + 12 us (1460 TFLOP/s: tensor cores 64 % active, the rest is what one
// slot's chain of S, softmax and P V leaves uncovered by the other's); fp8 trees as above, bound by that
// chain over tiles of 64 keys and by the conversion.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cstring>

#include "device.cuh"
#include "multi_token.h"

namespace psd {

namespace {

constexpr int kRows = 128;       // TMEM lanes of a row tile
constexpr float kLazy = 8.f;     // log2 units
constexpr int kMmaWarp = 8, kKWarp = 9, kVWarp = 10, kMmaWarp1 = 11;
constexpr int kConvertWarp = 12, kConvertWarps = 4;  // fp8 pools only: 4 warps for K, then 4 for V
constexpr uint32_t kRingBytes = 128 * 1024;
constexpr int kMaxStages = 16;

template <int D, int TERMS, bool FP8>
struct Lay {
  static constexpr int NK = TERMS == 1 && !FP8 ? 128 : 64;     // keys per tile
  static constexpr int kFlush = 9 / TERMS;                     // f32 outputs: ops of a slot that O holds at most
  static constexpr int kParts = NK / 64;                       // parts of a tile whose P go separately
  static constexpr int kHalves = D / 64;                       // 64-column halves of a row
  static constexpr uint32_t kGroupBytes = kHalves * 1024;      // 8 slots of one head
  static constexpr uint32_t kTileBytes = NK / 8 * kGroupBytes; // K or V of a tile
  static constexpr uint32_t kRawBytes = NK * D;                // its fp8 codes
  // half-tiles in the ring; fp8 pools have a ring of codes beside it
  static constexpr int kStages = FP8 ? 8 : int(kRingBytes / kTileBytes);
  static constexpr int kRaw = FP8 ? (D == 64 ? 16 : 8) : 0;
  static constexpr uint32_t kOffRaw = kStages * kTileBytes;
  static constexpr uint32_t kQHalfBytes = kRows * 128;
  static constexpr uint32_t kQBytes = kHalves * kQHalfBytes;   // one row tile
  static constexpr uint32_t kOffQ = kOffRaw + kRaw * kRawBytes;
  static constexpr uint32_t kOffOut = kOffQ + (FP8 ? 0 : 2 * kQBytes);  // 32 rows of 128 bytes for each softmax warp
  static constexpr uint32_t kOffBar = kOffOut + 8 * 32 * 128;
  static constexpr uint32_t kSmem = kOffBar + 1024 + 1024;     // barriers, alignment slack
  static constexpr uint32_t kPCols = NK / 2;                   // 32-bit columns of one P term
  static constexpr uint32_t kSCols = TERMS == 3 ? 96 : NK;     // a slot's S, or its P terms if they are wider
  static constexpr uint32_t kColS = 2 * D;                     // after the two O
  static constexpr uint32_t kColQ = kColS + 2 * kSCols;        // fp8 pools: a slot's Q, D / 2 columns
  // P = 2^(s - m) with the row's top at 2^kBias: f16 holds P down to 2^-31 of it.
  static constexpr float kBias = FP8 ? 7.f : 0.f;
  static constexpr int kThreads = FP8 ? 20 * 32 : 12 * 32;
  // What a CTA's time is made of, in halves of a key tile of one row tile: such a tile, a tile of
  // two row tiles, and what a unit costs beside its tiles (three tiles of 128 keys, five of 64, and
  // fourteen where Q comes through registers).  Stretches equal in tiles alone left the CTAs with
  // most units 15 % behind the mean.  Tiles of two row tiles counted as one: 34 us for 24 requests of
  // 1 to 4 tokens and one of 200 over 100 to 3000 keys against 27 (f32 outputs: 36 against 25); fp8
  // units counted as four tiles: 65 us for 16 requests' trees against 54.
  static constexpr int kOneCost = 2, kTwoCost = 4, kUnitCost = NK == 128 ? 6 : FP8 ? 28 : 10;
  // Registers a thread: 168 at launch of 384 threads, 96 of 640; the softmax warps hold a
  // part's scores and weights and take what the others do without.
  static constexpr int kLaunchRegs = FP8 ? 96 : 168;
  static constexpr int kSoftmaxRegs = FP8 ? 144 : 208, kOtherRegs = FP8 ? 64 : 88;
  static_assert(256 * kSoftmaxRegs + (kThreads - 256) * kOtherRegs <= kThreads * kLaunchRegs, "registers of the launch");
  static_assert(TERMS * kPCols <= kSCols && NK <= int(kSCols), "S region");
  static_assert(kColQ + (FP8 ? D : 0) <= 512, "TMEM columns");
  static_assert(kStages >= 4 && kStages <= kMaxStages && kRaw <= kMaxStages, "S runs two tiles ahead of PV");
  static_assert(kSmem <= 227u * 1024u, "shared memory");
  static_assert(kTileBytes % 1024 == 0, "128-byte-swizzle atoms");
};

enum {
  T_FULL = 0, T_EMPTY = kMaxStages,  // per half-tile: landed (or converted) / its MMAs have read it
  T_RFULL = 2 * kMaxStages, T_REMPTY = 3 * kMaxStages,  // per half-tile of codes: landed / converted
  T_QFULL = 4 * kMaxStages,          // [2] the row tile of Q landed; fp8 pools: the slot's is written (4 warps)
  T_QFREE = T_QFULL + 2,             // [2] every S that reads it is done
  T_SFULL = T_QFREE + 2,             // [2] S of the slot's next op is complete
  T_PFULL = T_SFULL + 2,             // [part][2] the part's P is written (4 warps)
  T_HALF = T_PFULL + 4,              // [2] the first part's PV of the slot's op is complete
  T_TURN = T_HALF + 2,               // [2] the MMAs of the other slot's op before are issued
  T_OFULL = T_TURN + 2,              // every PV of the unit is complete
  T_OFREE,                           // the unit's O are read out (8 warps)
  T_XREADY,                          // [2] the other slot's (m, l) of the rows are there (4 warps)
  T_DRAIN = T_XREADY + 2, T_SLOT, T_TAIL
};
static_assert(T_TAIL * 8 + 16 <= 1024, "barrier area");

struct TCParams {
  const int32_t *page_indices;
  const uint64_t *tree;
  const __nv_bfloat16 *q;
  int64_t q_stride;  // elements between tokens
  void *o;
  float *lse;
  float *part_o;    // [CTAs][2][2 * 128 rows][D]
  float *part_lse;  // [CTAs][2][2 * 128 rows]
  float *sum_o;     // [CTAs][2 slots][128 rows][D], f32 outputs only
  FaultRef fault;
  int64_t num_pages;
  int Hq, Hkv, G, TH, page_size, sub, out_f32;
  float q_scale, v_scale;
  uint32_t wait_limit;
  int withhold_from;  // testing aid: no loads for a unit's key tiles from this index on
};
// Requests with new tokens, and where each CTA's stretch of the line of key tiles begins.
constexpr int kMaxCtas = 192;
struct Start {
  uint16_t b, kv;  // request, KV head
  int32_t tok0, j; // first token and key tile of the unit
  int32_t tiles;   // key tiles of the stretch
};
struct TCRequests {
  psd_token_request r[kStepRequests];
  Start start[kMaxCtas];
};

// ------------------------------------------------------------------ walking the units
struct Unit {
  psd_token_request r;
  int kv, tok0;      // KV head, first new token of the unit
  int two;           // 1: two row tiles
  int j0, j1, n;     // this CTA's key tiles of the unit's n
  bool first;        // the CTA's first unit
};

// Key tiles of the unit whose first token is tok0.
__host__ __device__ __forceinline__ int unit_tiles(const psd_token_request &r, int tok0, int TH, int NK, bool tree) {
  const int start = r.kv_len - r.num_new;
  const int end = tok0 + 2 * TH < r.num_new ? tok0 + 2 * TH : r.num_new;  // tokens up to here
  const int keys = tree ? r.kv_len : start + end;
  return (keys + NK - 1) / NK;
}

// Walks the units of this CTA's stretch.
template <int NK>
struct Walk {
  const TCParams &p;
  const TCRequests &req;
  int left, b, kv, tok0, j;  // key tiles left; the next unit and tile
  bool first = true;
  __device__ Walk(const TCParams &p_, const TCRequests &req_) : p(p_), req(req_) {
    const int c = blockIdx.x;
    left = req.start[c].tiles;
    b = req.start[c].b;
    kv = req.start[c].kv;
    tok0 = req.start[c].tok0;
    j = req.start[c].j;
  }
  __device__ bool next(Unit &u) {
    if (left == 0) return false;
    u.r = req.r[b];
    u.kv = kv;
    u.tok0 = tok0;
    u.two = u.r.num_new - tok0 > p.TH ? 1 : 0;
    u.n = unit_tiles(u.r, tok0, p.TH, NK, p.tree != nullptr);
    u.j0 = j;
    u.j1 = min(u.n, j + left);
    u.first = first;
    left -= u.j1 - u.j0;
    first = false;
    j = 0;
    tok0 += 2 * p.TH;
    if (tok0 >= u.r.num_new) {
      tok0 = 0;
      if (++kv == p.Hkv) kv = 0, ++b;
    }
    return true;
  }
};

// ------------------------------------------------------------------------ PTX wrappers
// Shared-memory matrix descriptor, 128-byte swizzle (layout code 2), version 1.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return uint64_t((saddr & 0x3FFFFu) >> 4) | (uint64_t((lbo >> 4) & 0x3FFFu) << 16) |
         (uint64_t((sbo >> 4) & 0x3FFFu) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
}
// kind::f16: f32 accumulate, A and B both bf16 or both f16, A K-major, B K-major or (b_mn) MN-major.
__host__ __device__ constexpr uint32_t idesc_16bit(bool bf16, int M, int N, bool b_mn) {
  return (1u << 4) | (uint32_t(bf16) << 7) | (uint32_t(bf16) << 10) | (uint32_t(b_mn) << 16) | (uint32_t(N >> 3) << 17) |
         (uint32_t(M >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool elect() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
        "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
        "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
      "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
      "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&v);
}
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, int c3, int c4,
                                            uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, uint32_t bar,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void *at) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(at) : "memory");
}
__device__ __forceinline__ uint64_t l2_normal_policy() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

__device__ __forceinline__ float max3(float a, float b, float c) {  // NaN operands lose, as in fmaxf
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// 16 e4m3 codes to f16, exactly.
__device__ __forceinline__ void codes_to_f16(const uint4 &codes, uint32_t (&out)[8]) {
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
        : "=r"(out[2 * i]), "=r"(out[2 * i + 1])
        : "r"(w[i]));
}
__device__ __forceinline__ uint32_t f16x2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}
// Two values of P as the MMAs take them, and back.
template <bool F16>
__device__ __forceinline__ uint32_t p_bits(float lo, float hi) {
  return F16 ? f16x2_bits(lo, hi) : bf16x2_bits(lo, hi);
}
template <bool F16>
__device__ __forceinline__ float2 p_values(uint32_t w) {
  if constexpr (F16) return __half22float2(*reinterpret_cast<const __half2 *>(&w));
  else return make_float2(bf16_lo(w), bf16_hi(w));
}

// Waits for phase `parity` of the barrier, at most `limit` cycles.  The kernel's waits are many
// and inlined, so that they leave the fault word to the end of their role.
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, uint32_t limit) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint32_t t0 = uint32_t(clock());
  while (!mbar_try_wait(bar, parity))
    if (uint32_t(clock()) - t0 > limit) return false;
  return true;
}

// The visible keys of one row among the 32 from `base` on, one bit each.
__device__ __forceinline__ uint32_t visible(int base, int seen, int start, uint64_t tree, bool has_tree) {
  const int n = (has_tree ? start : seen) - base;  // keys before this one are visible
  uint32_t bits = n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
  if (has_tree) {
    const int sh = start - base;                   // the tree's bit 0 is key `start`
    if (sh >= 0 && sh < 32) bits |= uint32_t(tree << sh);
    else if (sh < 0 && sh > -64) bits |= uint32_t(tree >> -sh);
  }
  return bits;
}

template <int D, int TERMS, bool FP8>
__global__ void __launch_bounds__(Lay<D, TERMS, FP8>::kThreads, 1)
    step_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const TCParams p, const __grid_constant__ TCRequests req) {
  using L = Lay<D, TERMS, FP8>;
  constexpr int NK = L::NK, NS = L::kStages;
  // the ring that the copies fill
  constexpr int NC = FP8 ? L::kRaw : NS, kLanded = FP8 ? T_RFULL : T_FULL, kFreed = FP8 ? T_REMPTY : T_EMPTY;
  constexpr uint32_t kCopied = FP8 ? L::kRawBytes : L::kTileBytes;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  dependents_may_launch();  // the joining kernel waits for this grid on its own
  uint8_t *sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::kOffBar);
  uint32_t *tslot = reinterpret_cast<uint32_t *>(bars + T_SLOT);
  int *tail = reinterpret_cast<int *>(bars + T_TAIL);  // what the load warps issued
  auto bar = [&](int i) { return smem_u32(bars + i); };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool has_tree = p.tree != nullptr;

  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(bar(T_FULL + i), FP8 ? kConvertWarps : 1);
      mbar_init(bar(T_EMPTY + i), 2);
    }
    for (int i = 0; i < L::kRaw; ++i) {
      mbar_init(bar(T_RFULL + i), 1);
      mbar_init(bar(T_REMPTY + i), kConvertWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(T_SFULL + i), 1);
      mbar_init(bar(T_PFULL + i), 4);
      mbar_init(bar(T_PFULL + 2 + i), 4);
      mbar_init(bar(T_HALF + i), 1);
      mbar_init(bar(T_TURN + i), 1);
      mbar_init(bar(T_QFULL + i), FP8 ? 4 : 1);
      mbar_init(bar(T_QFREE + i), 2);
      mbar_init(bar(T_XREADY + i), 4);
    }
    mbar_init(bar(T_OFULL), 2);
    mbar_init(bar(T_OFREE), 8);
    mbar_init(bar(T_DRAIN), 2);
    fence_mbar_init();
  }
  if (warp == kKWarp || warp == kVWarp) {
    // what the first copies need, on its way while the CTA sets up: the tensor maps and page ids
    const Start &a = req.start[blockIdx.x];
    const psd_token_request &r = req.r[a.b];
    const int pos = (a.j * NK + lane * p.sub) / p.page_size;
    if (lane * p.sub < NK && int64_t(pos) * p.page_size < r.kv_len) prefetch_l2(p.page_indices + r.page_off + pos);
    if (lane == 0) {
      prefetch_map(warp == kKWarp ? &tmK : &tmV);
      if (!FP8 && warp == kKWarp) prefetch_map(&tmQ);
    }
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)), "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tslot;
  uint32_t bad = 0;  // what this thread has to report when its role ends
  auto wait_all = [&](int b, uint32_t parity) {  // a warp's bounded wait
    return __all_sync(0xffffffffu, wait_bounded(bar(b), parity & 1u, p.wait_limit)) != 0;
  };
  // (Each role sets its register share inside its own branch: where the branches met again
  // the compiler would hold every role to the smallest.)
  if (warp >= kMmaWarp) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::kOtherRegs));
  Walk<NK> walk(p, req);
  Unit u;
  if (warp == kKWarp || warp == kVWarp) {
    // ----------------------------------------------------------------- loads
    // Half-tile i of the ring: K of key tile i / 2 (even) or V of it (odd).
    const bool is_v = warp == kVWarp;
    const CUtensorMap *map = is_v ? &tmV : &tmK;
    const uint64_t pol = l2_normal_policy();
    const int n_copies = NK / p.sub;          // a lane each; p.sub tokens of one page
    const uint32_t copy_bytes = FP8 ? uint32_t(p.sub * D) : uint32_t(p.sub / 8) * L::kGroupBytes;
    const int P = p.page_size, pages_a_tile = NK / P, rest_a_tile = NK % P;
    int g = 0, q_next = 0, q_uses0 = 0, q_uses1 = 0;  // key tiles so far; the Q buffers' uses
    bool ok = true, withheld = false;
    while (ok && !withheld && walk.next(u)) {
      if (!FP8 && !is_v) {
        // A unit of one row tile uses the Q buffers in turn, so that its Q comes while the unit
        // before is worked on; a unit of two uses both.
        const int h0 = u.two ? 0 : q_next;
        for (int h = h0; h <= h0 + u.two && ok; ++h) {
          const int uses = h ? q_uses1 : q_uses0;
          if (uses > 0) ok = wait_all(T_QFREE + h, uint32_t(uses - 1));
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(bar(T_QFULL + h), uint32_t(L::kHalves * p.TH * p.G) * 128u);
          __syncwarp();
          if (lane < L::kHalves)
            tma_load_4d(smem_u32(sm + L::kOffQ + h * L::kQBytes + lane * L::kQHalfBytes), &tmQ, 0, u.kv * p.G,
                        u.r.token0 + u.tok0 + (u.two ? h * p.TH : 0), lane, bar(T_QFULL + h), pol);
          __syncwarp();
          if (h) ++q_uses1;
          else ++q_uses0;
        }
        if (!ok) break;
        if (!u.two) q_next ^= 1;
      }
      const int n_pages = (u.r.kv_len + P - 1) / P;
      // This lane's copy: its page of the tile and the token in it, a tile at a time without a division,
      // and page ids fetched two tiles ahead.
      int pos = (u.j0 * NK + lane * p.sub) / P, off = u.j0 * NK + lane * p.sub - pos * P;
      int ahead = pos, ahead_off = off;
      auto step = [&](int &page, int &at) {
        page += pages_a_tile;
        at += rest_a_tile;
        if (at >= P) at -= P, ++page;
      };
      auto next_id = [&]() {
        const int id = lane < n_copies && ahead < n_pages ? __ldg(p.page_indices + u.r.page_off + ahead) : -1;
        step(ahead, ahead_off);
        return id;
      };
      int id = next_id(), id_next = next_id();
      for (int j = u.j0; j < u.j1; ++j, ++g) {
        if (j >= p.withhold_from) {
          withheld = true;
          break;
        }
        const int id_after = next_id();
        const int i = 2 * g + (is_v ? 1 : 0), st = i % NC;
        if (i >= NC && !wait_all(kFreed + st, uint32_t(i / NC - 1))) {
          ok = false;
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(bar(kLanded + st), kCopied);
        __syncwarp();
        if (lane < n_copies) {
          const bool there = pos < n_pages && id >= 0 && int64_t(id) < p.num_pages;
          if (pos < n_pages && !there) bad |= PSD_FAULT_PAGE_ID;
          // the first token slot; not there: wholly outside the view, which reads as zeros
          const int64_t first = there ? int64_t(id) * P + off : -1024;
          if constexpr (FP8)
            tma_load_3d(smem_u32(sm + L::kOffRaw + st * kCopied + lane * copy_bytes), map, 0, u.kv, int(first),
                        bar(kLanded + st), pol);
          else
            tma_load_5d(smem_u32(sm + st * kCopied + lane * copy_bytes), map, 0, 0, 0, u.kv, int(first / 8),
                        bar(kLanded + st), pol);
        }
        __syncwarp();
        step(pos, off);
        id = id_next;
        id_next = id_after;
      }
    }
    if (!ok) bad |= PSD_FAULT_WAIT_TIMEOUT;
    if (lane == 0) {
      tail[is_v] = g;
      if (!is_v) tail[2] = q_uses0, tail[3] = q_uses1;
    }
  } else if (FP8 && warp >= kConvertWarp) {
    // ------------------------------------------------------- fp8 codes to f16
    // Four warps take the K half-tiles and four the V, in the order of the ring: 16 codes a thread
    // and step, exact (the scales are in the scores' and the output's factors), into the
    // swizzled layout the MMAs read.  V rows past the request's last token become zeros.
    const int th = (tid - 32 * kConvertWarp) & 127, v = warp >= kConvertWarp + kConvertWarps ? 1 : 0;
    int g = 0;
    bool ok = true;
    while (ok && walk.next(u)) {
      for (int j = u.j0; j < u.j1; ++j, ++g) {
        const int i = 2 * g + v, st = i % NS, rs = i % NC;
        {  // the codes have landed (lane 0 asks) and the stage is free (lane 1)
          const int b = lane == 0 ? T_RFULL + rs : lane == 1 && i >= NS ? T_EMPTY + st : -1;
          ok = b < 0 || wait_bounded(bar(b), uint32_t(lane == 0 ? i / NC : i / NS - 1) & 1u, p.wait_limit);
          ok = __all_sync(0xffffffffu, ok) != 0;
          if (!ok) break;
          __syncwarp();  // (a vote orders no memory: what two lanes have seen holds for all from here on)
        }
        const uint8_t *src = sm + L::kOffRaw + rs * L::kRawBytes;
        uint8_t *dst = sm + st * L::kTileBytes;
        const int left = v ? u.r.kv_len - j * NK : NK;
        // A warp's step: 8 tokens, 4 chunks of 16 codes each; 8 lanes that move together have the 8
        // tokens of a swizzle atom, codes and f16, and so 8 different banks.
        constexpr int kSteps = NK * D / 16 / 128;
        const int step0 = (th >> 5) * kSteps;
        auto place = [&](int c, int &tk, int &chunk) {
          const int s = step0 + c;
          tk = (D == 128 ? s >> 1 : s) * 8 + (lane & 7);
          chunk = (D == 128 ? (s & 1) * 4 : 0) + (lane >> 3);
        };
        uint4 w[kSteps];
#pragma unroll
        for (int c = 0; c < kSteps; ++c) {
          int tk, chunk;
          place(c, tk, chunk);
          w[c] = *reinterpret_cast<const uint4 *>(src + tk * D + ((chunk ^ (D == 128 ? tk & 7 : (tk >> 1) & 3)) << 4));
        }
#pragma unroll
        for (int c = 0; c < kSteps; ++c) {
          int tk, chunk;
          place(c, tk, chunk);
          uint32_t out[8];
          codes_to_f16(w[c], out);
          if (tk >= left) {
#pragma unroll
            for (int y = 0; y < 8; ++y) out[y] = 0u;
          }
          const int k = (2 * chunk) & 7;
          uint8_t *row = dst + (tk >> 3) * L::kGroupBytes + (chunk >> 2) * 1024 + (tk & 7) * 128;
          *reinterpret_cast<uint4 *>(row + ((k ^ (tk & 7)) << 4)) = make_uint4(out[0], out[1], out[2], out[3]);
          *reinterpret_cast<uint4 *>(row + (((k + 1) ^ (tk & 7)) << 4)) = make_uint4(out[4], out[5], out[6], out[7]);
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(T_FULL + st));
          mbar_arrive(bar(T_REMPTY + rs));
        }
      }
    }
    if (!ok) bad |= PSD_FAULT_WAIT_TIMEOUT;
  } else if (elect()) {
    // ------------------------------------------------------- the MMAs of a slot
    // One thread a slot: an op costs its thread about 1300 cycles (16 issues, six waits of over
    // 100 cycles on barriers that are ready), more than the 1024 its MMAs take.  The ops go in
    // turn, so that the slots stay half a period apart: left alone they fall into step, and the
    // tensor cores idle while both take their softmax (the 4096-token prompt took 6 % longer).
    // The tiles of an op are waited for before its P, and S(t + 2) follows P V(t) without a wait.
    // A half-tile is released by two commits: one from each slot where both read it, two
    // from the slot that has it alone.
    // A wait tells a phase of its barrier from the one before, not from the one before that.  So a
    // thread may wait for a half-tile only when the stage's last half-tile has landed for certain,
    // also where that was the other slot's: within a unit a stage keeps its slot (or both see
    // every tile), and between units a thread waits first until every S of the unit before is
    // done (its K landed), and before its first P V until that unit is read out (its V landed).
    const int slot = warp == kMmaWarp1 ? 1 : 0;
    const uint32_t id_s = idesc_16bit(!FP8, kRows, NK, false);
    const uint32_t id_pv = idesc_16bit(!FP8, kRows, D, true);
    // Q: 8-row groups 1024 B apart.  K (K-major): 8-token groups kGroupBytes apart, a half 1024 B
    // further.  V (MN-major): 64-column atoms 1024 B apart, 8-token groups kGroupBytes apart.
    const uint64_t qd = desc_sw128(smem_u32(sm + L::kOffQ), 16, 1024);
    const uint64_t kd = desc_sw128(smem_u32(sm), 16, L::kGroupBytes);
    const uint64_t vd = desc_sw128(smem_u32(sm), 1024, L::kGroupBytes);
    const uint32_t d = tmem + D * slot, sp = tmem + L::kColS + slot * L::kSCols;  // O; S and P
    const uint32_t qt = tmem + L::kColQ + slot * (D / 2);  // fp8 pools: Q
    auto wait = [&](int b, uint32_t parity) { return wait_bounded(bar(b), parity & 1u, p.wait_limit); };
    int g = 0, units = 0;
    uint32_t ops = 0, turns = 0;  // this slot's ops, and turns waited for
    int q_next = 0;
    uint32_t q_parity = 0;        // bit h: parity of Q buffer h's uses
    int h_before = 0;             // a Q buffer of the unit before
    bool ok = true;
    while (ok && walk.next(u)) {
      const int nt = u.j1 - u.j0, T = u.two ? 2 * nt : nt;
      auto half_tile = [&](int t) { return 2 * (g + (u.two ? t >> 1 : t)); };  // K of op t; V is the next
      auto k_ready = [&](int t) {
        const int i = half_tile(t);
        return wait(T_FULL + i % NS, uint32_t(i / NS));
      };
      const int h = u.two ? slot : q_next;  // the Q buffer
      const uint64_t q = qd + ((h ? L::kQBytes : 0u) >> 4);
      // Each slot's commit, to every buffer of the unit: a buffer's phase then needs both slots, and
      // neither can run two phases ahead of the other's wait below.
      auto q_free = [&]() {
        commit(bar(T_QFREE + h));
        if (u.two) commit(bar(T_QFREE + (h ^ 1)));
      };
      auto issue_s = [&](int t) {
        const int st = half_tile(t) % NS;
        const uint64_t b = kd + ((st * L::kTileBytes) >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t bk = b + (((k >> 2) * 1024 + (k & 3) * 32) >> 4);
          if constexpr (FP8) mma_ts(sp, qt + 8 * k, bk, id_s, k > 0);
          else mma_ss(sp, q + (((k >> 2) * L::kQHalfBytes + (k & 3) * 32) >> 4), bk, id_s, k > 0);
        }
        commit(bar(T_SFULL + slot));
        commit(bar(T_EMPTY + st));
        if (!u.two) commit(bar(T_EMPTY + st));
        if (t + 2 >= T) q_free();
      };
      ok = (units == 0 || wait(T_QFREE + h_before, (q_parity >> h_before) ^ 1u)) && 
           (FP8 ? wait(T_QFULL + slot, uint32_t(units)) : wait(T_QFULL + h, q_parity >> h)) &&
           (slot >= T || k_ready(slot));
      h_before = h;
      if (!ok) break;
      fence_after();
      if (slot < T) {
        issue_s(slot);
      } else {
        // One key tile, slot 0's.  The unit before is read out first: its phase of T_OFULL must
        // not take this slot's arrival for slot 0's.
        if (units > 0 && !(ok = wait(T_OFREE, uint32_t(units - 1)))) break;
        q_free();
        commit(bar(T_OFULL));
      }
      q_parity ^= u.two ? 3u : 1u << q_next;
      if (!u.two) q_next ^= 1;
      for (int t = slot; t < T; t += 2) {
        const int i = half_tile(t) + 1, st = i % NS;
        // K of op t + 2 has a stage that op t or an earlier one freed: no P stands before it
        ok = (t > 1 || units == 0 || wait(T_OFREE, uint32_t(units - 1))) && wait(T_FULL + st, uint32_t(i / NS)) &&
             (t + 2 >= T || k_ready(t + 2)) && (t == 0 || wait(T_TURN + slot, turns));
        if (!ok) break;
        if (t > 0) ++turns;
        const uint64_t b = vd + ((st * L::kTileBytes) >> 4);
        const bool fresh = TERMS > 1 ? (t >> 1) % L::kFlush == 0 : t < 2;  // O starts at zero
#pragma unroll
        for (int part = 0; part < L::kParts; ++part) {
          ok = wait(T_PFULL + 2 * part + slot, ops);
          if (!ok) break;
          fence_after();
#pragma unroll
          for (int k = 4 * part; k < 4 * part + 4; ++k)
#pragma unroll
            for (int x = 0; x < TERMS; ++x)
              mma_ts(d, sp + x * L::kPCols + 8 * k, b + ((k * 2 * L::kGroupBytes) >> 4), id_pv, !fresh || k > 0 || x > 0);
          if (part == 0 && L::kParts > 1) commit(bar(T_HALF + slot));
        }
        if (!ok) break;
        ++ops;
        if (t + 2 < T) issue_s(t + 2);  // before the commits below: a softmax waits for it
        commit(bar(T_EMPTY + st));
        if (!u.two) commit(bar(T_EMPTY + st));
        if (t + 2 >= T) commit(bar(T_OFULL));
        if (t + 1 < T) mbar_arrive(bar(T_TURN + (slot ^ 1)));
      }
      g += nt;
      ++units;
    }
    // every MMA issued has completed before TMEM is released
    commit(bar(T_DRAIN));
    if (!wait(T_DRAIN, 0u) || !ok) bad |= PSD_FAULT_WAIT_TIMEOUT;
  }
  } else {
    // ---------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(L::kSoftmaxRegs));
    Walk<NK> walk(p, req);
    Unit u;
    const int slot = warp >> 2, r = tid & 127;       // row of the tile = TMEM lane
    const uint32_t lane_base = tmem + (uint32_t(32 * (warp & 3)) << 16);
    const uint32_t s_col = lane_base + L::kColS + slot * L::kSCols;
    [[maybe_unused]] float qs = p.q_scale;
    const int rt = r / p.G, rg = r - rt * p.G;        // token of the tile, head of the group
    // fp8 pools: the row's Q of a unit as f16, times the power of two that puts its top in [2^14, 2^15):
    // exact but for elements 2^-31 below the top.  Returns the row's score factor.
    auto q_row = [&](const Unit &v, bool &there) {
      const int t = v.tok0 + (v.two && slot ? p.TH : 0) + rt;
      there = rt < p.TH && t < v.r.num_new;
      return reinterpret_cast<const uint4 *>(p.q + (int64_t(v.r.token0) + t) * p.q_stride + (int64_t(v.kv) * p.G + rg) * D);
    };
    auto give_q = [&](const Unit &v) {
      bool there;
      const uint4 *src = q_row(v, there);
      float f_inv = 1.f;
      if (__any_sync(0xffffffffu, there)) {
        const uint4 none = make_uint4(0u, 0u, 0u, 0u);
        float top = 0.f;
        {
          uint4 w[D / 8];
#pragma unroll
          for (int c = 0; c < D / 8; ++c) w[c] = there ? __ldg(src + c) : none;
#pragma unroll
          for (int c = 0; c < D / 8; ++c) {
            const uint32_t y[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) top = max3(top, fabsf(bf16_lo(y[k])), fabsf(bf16_hi(y[k])));
          }
        }
        // the factor stays a normal number: times a score of -inf, 0 would be NaN (a row so small beside
        // the scale scores 0 anyway)
        const int most = min(100, int(__float_as_uint(p.q_scale) >> 23) - 1);
        const int e = min(most, max(-114, 14 - (int(__float_as_uint(top) >> 23) - 127)));
        const float f = __uint_as_float(uint32_t(127 + e) << 23);
        f_inv = __uint_as_float(uint32_t(127 - e) << 23);
        const uint32_t q_col = lane_base + L::kColQ + slot * (D / 2);
        // 64 elements at a time, from the first-level cache (held since the pass above they would spill)
#pragma unroll 1
        for (int c0 = 0; c0 < D / 8; c0 += 8) {
          uint32_t x[32];
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const uint4 w = there ? __ldg(src + c0 + c) : none;
            const uint32_t y[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) x[4 * c + k] = f16x2_bits(bf16_lo(y[k]) * f, bf16_hi(y[k]) * f);
          }
          tmem_st32(q_col + 4 * c0, x);
        }
      }
      st_wait();
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(T_QFULL + slot));
      return p.q_scale * f_inv;
    };
    [[maybe_unused]] float qs_next = p.q_scale;
    if constexpr (FP8) {
      Walk<NK> ahead = walk;
      if (ahead.next(u)) qs_next = give_q(u);
    }
    int g = 0, units = 0, singles = 0;                // key tiles, units, units of one row tile so far
    uint32_t ops = 0;
    bool ok = true;
    while (ok && walk.next(u)) {
      const int nt = u.j1 - u.j0, T = u.two ? 2 * nt : nt;
      const int tile_tok = u.tok0 + (u.two && slot ? p.TH : 0);
      const int tok = tile_tok + rt;                  // new token of the request
      const bool live = rt < p.TH && tok < u.r.num_new;
      const bool warp_live = __any_sync(0xffffffffu, live);
      const int start = u.r.kv_len - u.r.num_new;
      uint64_t tree = 0;
      if (has_tree && live) {
        tree = __ldg(reinterpret_cast<const unsigned long long *>(p.tree) + u.r.token0 + tok);
        if (u.r.num_new < 64) tree &= (uint64_t(1) << u.r.num_new) - 1;
      }
      if constexpr (FP8) {
        qs = qs_next;
        Walk<NK> ahead = walk;
        Unit v;
        bool there;
        if (ahead.next(v)) {  // its Q on the way to the second-level cache
          const uint4 *src = q_row(v, there);
          if (there) {
            prefetch_l2(src);
            if constexpr (D == 128) prefetch_l2(src + 8);
          }
        }
      }
      const int seen = start + tok + 1;               // causal: keys before this one
      const int clear = has_tree ? start : seen;      // every key before this one is visible
      float m = neg_inf(), l = 0.f;
      // f32 outputs: the row's O of the ops before the last flush, relative to 2^m_sum; columns
      // c .. c + 3 at sum_row + c kRows, so that a warp's rows lie side by side
      float *sum_row = p.sum_o + (int64_t(blockIdx.x) * 2 + slot) * kRows * D + 4 * r;
      float m_sum = neg_inf();
      bool flushed = false;
      for (int t = slot; t < T; t += 2, ++ops) {
        const int j = u.j0 + (u.two ? t >> 1 : t), base = j * NK;
        ok = wait_all(T_SFULL + slot, ops);
        if (!ok) break;
        fence_after();
        bool empty = t < 2;                             // O holds nothing
        if (warp_live) {
          if constexpr (TERMS > 1) {
            if (t >= 2 && (t >> 1) % L::kFlush == 0) {
              // S(t) is complete, so PV(t - 2), issued before it, is too
              const float keep = m_sum == neg_inf() ? 0.f : ex2(m_sum - m);
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tmem_ld32(lane_base + D * slot + c, o);
                ld_wait();
                if (live) {
#pragma unroll
                  for (int k = 0; k < 32; k += 4) {
                    float4 *at = reinterpret_cast<float4 *>(sum_row + (c + k) * kRows);
                    float4 x = flushed ? *at : make_float4(0.f, 0.f, 0.f, 0.f);
                    x.x = fmaf(x.x, keep, __uint_as_float(o[k]));
                    x.y = fmaf(x.y, keep, __uint_as_float(o[k + 1]));
                    x.z = fmaf(x.z, keep, __uint_as_float(o[k + 2]));
                    x.w = fmaf(x.w, keep, __uint_as_float(o[k + 3]));
                    *at = x;
                  }
                }
              }
              m_sum = m;
              flushed = empty = true;
            }
          }
        }
        // V rows past the request's last token may hold anything, NaN included: the slot whose PV
        // comes first zeroes them before it gives its P, so that P = 0 never meets a NaN.
        const int left = u.r.kv_len - base;
        if (!FP8 && left < NK && !(u.two && slot)) {
          const int i = 2 * (g + (u.two ? t >> 1 : t)) + 1, st = i % NS;
          ok = wait_all(T_FULL + st, uint32_t(i / NS));
          if (!ok) break;
          uint8_t *vt = sm + st * L::kTileBytes;
          // 16-byte chunks of the tokens [left, NK): token tk's row of half h
          for (int c = r; c < (NK - left) * L::kHalves * 8; c += 128) {
            const int tk = left + c / (L::kHalves * 8), h = (c >> 3) % L::kHalves;
            *reinterpret_cast<uint4 *>(vt + (tk >> 3) * L::kGroupBytes + h * 1024 + (tk & 7) * 128 + (c & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async();
        }
        const bool masked = __any_sync(0xffffffffu, live && clear < base + NK);
        auto give_part = [&](auto which) -> bool {
          constexpr int part = decltype(which)::value;
          if (warp_live) {
            // P with the row's running maximum as it stands, and the part's own maximum beside it: on
            // most tiles no row grows by more than 2^8 and the maximum is off the critical path.
            // Otherwise (a unit's first tile among them) O and l are rescaled and P is taken again.
            uint32_t pk[32];                            // two bf16 each
            [[maybe_unused]] float pf[TERMS > 1 ? 64 : 1];
            float2 sum[2];
            for (;;) {
              const float nm = m == neg_inf() ? 0.f : -m;
              const float2 qs2 = make_float2(qs, qs), nm2 = make_float2(nm, nm);
              float t4[4] = {neg_inf(), neg_inf(), neg_inf(), neg_inf()};
              sum[0] = sum[1] = make_float2(0.f, 0.f);
#pragma unroll
              for (int c0 = 0; c0 < 64; c0 += 32) {
                uint32_t x[32];
                tmem_ld32(s_col + 64 * part + c0, x);
                ld_wait();
                if (masked) {
                  const uint32_t bits = visible(base + 64 * part + c0, seen, start, tree, has_tree);
#pragma unroll
                  for (int c = 0; c < 32; ++c) x[c] = (bits >> c) & 1u ? x[c] : 0xff800000u;
                }
#pragma unroll
                for (int c = 0; c < 32; c += 8)
#pragma unroll
                  for (int y = 0; y < 4; ++y)
                    t4[y] = max3(t4[y], __uint_as_float(x[c + 2 * y]), __uint_as_float(x[c + 2 * y + 1]));
#pragma unroll
                for (int c = 0; c < 32; c += 2) {
                  const float2 z =
                      __ffma2_rn(make_float2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), qs2, nm2);
                  const float a = ex2(z.x), b = ex2(z.y);
                  sum[(c >> 1) & 1] = __fadd2_rn(sum[(c >> 1) & 1], make_float2(a, b));
                  if constexpr (TERMS == 1) {
                    pk[(c0 + c) / 2] = p_bits<FP8>(a, b);
                  } else {
                    pf[c0 + c] = a;
                    pf[c0 + c + 1] = b;
                  }
                }
              }
              float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
              top = live ? top * qs : neg_inf();        // qs > 0; (a dead row's scores are whatever Q held)
              const bool grow = top > m + (L::kBias + kLazy);
              if (!__any_sync(0xffffffffu, grow)) break;
              // O may be changed: S(t) is complete, so PV(t - 2), issued before it, is too; the first
              // part's PV of this op is waited for
              if (part > 0) {
                if (!wait_all(T_HALF + slot, ops)) return false;
                fence_after();
              }
              const float m_new = grow ? top - L::kBias : m;
              const float alpha = grow ? ex2(m - m_new) : 1.f;
              l *= alpha;
              if (part > 0 || !empty) {
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                  uint32_t o[32];
                  tmem_ld32(lane_base + D * slot + c, o);
                  ld_wait();
#pragma unroll
                  for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * alpha);
                  tmem_st32(lane_base + D * slot + c, o);
                }
              }
              m = m_new;
            }
            if constexpr (TERMS == 1) {
              tmem_st32(s_col + 32 * part, pk);
            } else {
#pragma unroll
              for (int y = 0; y < TERMS; ++y) {         // each term takes what the ones before left
#pragma unroll
                for (int c = 0; c < 64; c += 2) {
                  pk[c / 2] = p_bits<FP8>(pf[c], pf[c + 1]);
                  const float2 got = p_values<FP8>(pk[c / 2]);
                  pf[c] -= got.x;
                  pf[c + 1] -= got.y;
                }
                tmem_st32(s_col + y * L::kPCols, pk);
              }
            }
            sum[0] = __fadd2_rn(sum[0], sum[1]);
            l += sum[0].x + sum[0].y;
          }
          st_wait();
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(T_PFULL + 2 * part + slot));
          return true;
        };
        ok = give_part(std::integral_constant<int, 0>{});
        if constexpr (L::kParts > 1) ok = ok && give_part(std::integral_constant<int, 1>{});
        if (!ok) break;
      }
      if (!ok) break;

      // ------------------------------------------------------------- epilogue
      ok = wait_all(T_OFULL, uint32_t(units));
      if (!ok) break;
      fence_after();
      if constexpr (FP8) {
        // Q of the next unit, so that its S need not wait for what follows.  (Not before the wait: both
        // MMA threads must have seen this unit's Q.)
        Walk<NK> ahead = walk;
        Unit v;
        if (ahead.next(v)) qs_next = give_q(v);
      }
      const bool whole = u.j0 == 0 && u.j1 == u.n;
      const int row = tile_tok * p.G + r - u.tok0 * p.G;   // row of the unit (p.TH * p.G a tile)
      const int piece = 2 * blockIdx.x + (u.first ? 0 : 1);  // the CTA's first piece, or its last
      const int64_t out = (int64_t(u.r.token0) + tok) * p.Hq + u.kv * p.G + rg;
      // Where this row goes, in elements: the output, or a piece's rows in the workspace.
      const int64_t dst = live ? (whole ? out : int64_t(piece) * 2 * kRows + row) * D : -1;
      // 32 columns of the warp's rows, as f32, from the rows' lanes to coalesced stores through
      // shared memory: chunk k of row `lane` lies at k ^ lane % 8; then 4 lanes a row, 8 columns each,
      // 8 rows a step.  (Lanes that store their own rows touch 32 lines at once: 10000 cycles a unit
      // of 256 rows.  One rolled copy of the code: it runs once or a few times a CTA, and what it
      // costs then is fetching it.)
      uint8_t *stage = sm + L::kOffOut + warp * (32 * 128);
      auto put32 = [&](const float (&x)[32], int c) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          *reinterpret_cast<float4 *>(stage + lane * 128 + ((k ^ (lane & 7)) << 4)) =
              make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
        __syncwarp();
        const int k = 2 * (lane & 3), at = c + 4 * k;
#pragma unroll 1
        for (int rr = lane >> 2; rr < 32; rr += 8) {
          const int64_t to = __shfl_sync(0xffffffffu, dst, rr);
          const float4 y = *reinterpret_cast<const float4 *>(stage + rr * 128 + ((k ^ (rr & 7)) << 4));
          const float4 z = *reinterpret_cast<const float4 *>(stage + rr * 128 + (((k + 1) ^ (rr & 7)) << 4));
          if (to < 0) continue;
          if (whole && TERMS == 1) {
            *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.o) + to + at) =
                make_uint4(bf16x2_bits(y.x, y.y), bf16x2_bits(y.z, y.w), bf16x2_bits(z.x, z.y), bf16x2_bits(z.z, z.w));
          } else {
            float4 *out4 = reinterpret_cast<float4 *>((whole ? static_cast<float *>(p.o) : p.part_o) + to + at);
            out4[0] = y;
            out4[1] = z;
          }
        }
        __syncwarp();
      };
      const float keep = m_sum == neg_inf() ? 0.f : ex2(m_sum - m);  // flushed sums to 2^m
      auto add_flushed = [&](float (&x)[32], const float *from, float scale) {
#pragma unroll
        for (int k = 0; k < 32; k += 4) {
          const float4 y = *reinterpret_cast<const float4 *>(from + k * kRows);
          x[k] = fmaf(y.x, scale, x[k]);
          x[k + 1] = fmaf(y.y, scale, x[k + 1]);
          x[k + 2] = fmaf(y.z, scale, x[k + 2]);
          x[k + 3] = fmaf(y.w, scale, x[k + 3]);
        }
      };
      // The slots have the even and odd tiles of a unit of one row tile: they tell each other m and
      // l (and the factor of their flushed sums) through the other's staging rows, and join the two O
      // of half the columns each.  (Those rows are free: their warp is past its last unit's stores,
      // which this unit's O waited for, and waits here before its next.)
      const bool joint = !u.two && T > 1;
      float m1 = neg_inf(), l1 = 0.f, keep1 = 0.f;
      if (joint) {
        if constexpr (TERMS > 1) __threadfence_block();  // sum_row is read by the other slot
        reinterpret_cast<float4 *>(sm + L::kOffOut + (warp ^ 4) * (32 * 128))[lane] =
            make_float4(m, l, flushed ? keep : 0.f, 0.f);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(T_XREADY + (slot ^ 1)));
        if (!(ok = wait_all(T_XREADY + slot, uint32_t(singles)))) break;
        const float4 other = reinterpret_cast<const float4 *>(stage)[lane];
        m1 = other.x, l1 = other.y, keep1 = other.z;
        __syncwarp();
        ++singles;
      }
      if (warp_live && (u.two || joint || slot == 0)) {
        const float top = fmaxf(m, m1), from = top == neg_inf() ? 0.f : top;
        const float w0 = ex2(m - from), w1 = ex2(m1 - from);  // 0 where a slot saw no key
        const float all = l * w0 + l1 * w1, inv = all == 0.f ? 0.f : p.v_scale / all;
        const float f0 = l == 0.f ? 0.f : w0 * inv, f1 = l1 == 0.f ? 0.f : w1 * inv;
        const int c_end = joint ? D / 2 * (slot + 1) : D;
#pragma unroll 1
        for (int c = joint ? D / 2 * slot : 0; c < c_end; c += 32) {
          float x[32];
          tmem_ld32(lane_base + D * slot + c, reinterpret_cast<uint32_t *>(x));
          ld_wait();
#pragma unroll
          for (int k = 0; k < 32; ++k) x[k] = l == 0.f ? 0.f : x[k] * f0;
          if (joint) {
            uint32_t y[32];
            tmem_ld32(lane_base + D * (slot ^ 1) + c, y);
            ld_wait();
#pragma unroll
            for (int k = 0; k < 32; ++k) x[k] = l1 == 0.f ? x[k] : fmaf(__uint_as_float(y[k]), f1, x[k]);
          }
          if constexpr (TERMS > 1) {
            if (live && flushed && l != 0.f) add_flushed(x, sum_row + c * kRows, keep * f0);
            if (live && keep1 != 0.f && l1 != 0.f)
              add_flushed(x, sum_row + (slot ? -kRows * D : kRows * D) + c * kRows, keep1 * f1);
          }
          put32(x, c);
        }
        if (live && (u.two || slot == 0)) {
          const float v = all == 0.f ? neg_inf() : top + log2f(all);
          if (!whole) p.part_lse[int64_t(piece) * 2 * kRows + row] = v;
          else if (p.lse) p.lse[out] = v;
        }
      }
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(T_OFREE));
      g += nt;
      ++units;
    }
    if (!ok) bad |= PSD_FAULT_WAIT_TIMEOUT;
  }
  __syncwarp();
  st_wait();
  fence_before();
  __syncthreads();
  if (warp == kKWarp) {
    // No copy may be in flight when the CTA exits, after a wait that ran out either: the last
    // half-tile issued into each stage, by either load warp, and the last Q.
    if (lane < NC) {
      int last = -1;
      for (int v = 0; v < 2; ++v) {
        const int top = 2 * (tail[v] - 1) + v;
        for (int i = top; i > last && i > top - 2 * NC; i -= 2)
          if (i % NC == lane) last = i;
      }
      if (last >= 0 && !wait_bounded(bar(kLanded + lane), uint32_t(last / NC) & 1u, p.wait_limit))
        bad |= PSD_FAULT_WAIT_TIMEOUT;
    }
    if (!FP8 && lane < 2 && tail[2 + lane] > 0 &&
        !wait_bounded(bar(T_QFULL + lane), uint32_t(tail[2 + lane] - 1) & 1u, p.wait_limit))
      bad |= PSD_FAULT_WAIT_TIMEOUT;
  }
  if (bad) raise_fault(p.fault, bad);
  if (warp == kMmaWarp) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
  }
}

// A unit that the CTAs' bounds cut.
struct Cut {
  int64_t out;   // output row of the unit's first token and head
  int16_t rows;  // live rows
  int16_t n;     // its pieces, one a CTA
  int16_t first; // the CTA of the first
  int16_t late;  // the first piece is the second of its CTA
};
struct Cuts {
  Cut c[kMaxCtas - 1];
};

// Joins the pieces of the cut units (blockIdx.x), in key order: LANES lanes a row.  The host
// names them: found by a walk on the device, as the main kernel's stretches are, they cost
// 30 us more behind a 4096-token prompt.
template <int D, int LANES>
__global__ void __launch_bounds__(256) step_join_kernel(const TCParams p, const __grid_constant__ Cuts cuts) {
  constexpr int kCols = D / LANES;  // of a row, a lane: chunks of 4, LANES chunks apart
  const Cut &u = cuts.c[blockIdx.x];
  const int lane = threadIdx.x % LANES, row = blockIdx.y * (256 / LANES) + threadIdx.x / LANES;
  wait_for_prior_grid();
  const bool live = row < u.rows;
  auto at = [&](int i) {
    return int64_t(2 * (u.first + i) + (i == 0 ? u.late : 0)) * 2 * kRows + (live ? row : 0);
  };
  // The first two pieces (there are two at least) are on their way beside the LSEs.
  float y[2][kCols];
  auto fetch = [&](int i, float (&to)[kCols]) {
    const float *src = p.part_o + at(i) * D + 4 * lane;
#pragma unroll
    for (int k = 0; k < kCols; k += 4)
      *reinterpret_cast<float4 *>(to + k) = *reinterpret_cast<const float4 *>(src + LANES * k);
  };
  fetch(0, y[0]);
  fetch(1, y[1]);
  float m = neg_inf();
  for (int i = lane; i < u.n; i += LANES) m = fmaxf(m, p.part_lse[at(i)]);
#pragma unroll
  for (int x = LANES / 2; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  const float from = m == neg_inf() ? 0.f : m;
  float x[kCols] = {}, sum = 0.f;
  for (int i = 0; i < u.n; i += 2) {
    if (i > 0) {
      fetch(i, y[0]);
      if (i + 1 < u.n) fetch(i + 1, y[1]);
    }
#pragma unroll
    for (int k2 = 0; k2 < 2; ++k2) {
      if (i + k2 >= u.n) break;
      const float s = p.part_lse[at(i + k2)], w = ex2(s - from);
      sum += w;
#pragma unroll
      for (int k = 0; k < kCols; ++k) x[k] = s == neg_inf() ? x[k] : fmaf(w, y[k2][k], x[k]);
    }
  }
  if (!live) return;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int64_t out = u.out + int64_t(row / p.G) * p.Hq + row % p.G;
#pragma unroll
  for (int k = 0; k < kCols; k += 4) {
    const int64_t o = out * D + 4 * lane + LANES * k;
    const float4 y = make_float4(x[k] * inv, x[k + 1] * inv, x[k + 2] * inv, x[k + 3] * inv);
    if (p.out_f32)
      *reinterpret_cast<float4 *>(static_cast<float *>(p.o) + o) = y;
    else
      *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.o) + o) = make_uint2(bf16x2_bits(y.x, y.y), bf16x2_bits(y.z, y.w));
  }
  if (lane == 0 && p.lse) p.lse[out] = sum == 0.f ? neg_inf() : m + log2f(sum);
}

// ------------------------------------------------------------------------- launch
bool encode(CUtensorMap *map, const DeviceInfo &dev, int rank, const void *base, const cuuint64_t *dims,
            const cuuint64_t *strides, const cuuint32_t *box, int codes = 0) {  // bytes of a row of codes
  auto fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(dev.encode_tiled);
  const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
  return fn && fn(map, codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, cuuint32_t(rank),
                  const_cast<void *>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  codes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int TERMS, bool FP8>
psd_status run(const StepParams &S, const StepRequests &sreq, const StepPlace &place, const DeviceInfo &dev,
               cudaStream_t s) {
  using L = Lay<D, TERMS, FP8>;
  TCParams p;
  p.page_indices = S.page_indices;
  p.tree = S.tree;
  p.q = static_cast<const __nv_bfloat16 *>(S.q);
  p.q_stride = S.q_stride;
  p.o = S.o;
  p.lse = S.lse;
  p.fault = S.fault;
  p.num_pages = S.num_pages;
  p.Hq = S.Hq;
  p.Hkv = S.Hkv;
  p.G = S.G;
  p.TH = kRows / S.G;
  p.page_size = S.page_size;
  p.sub = 8;
  while (p.sub < L::NK && S.page_size % (2 * p.sub) == 0) p.sub *= 2;
  p.out_f32 = S.out_f32;
  p.q_scale = S.q_scale;
  p.v_scale = S.v_scale;
  p.wait_limit = uint32_t(dev.test_wait_limit > 0 ? dev.test_wait_limit : kWaitLimitCycles);
  p.withhold_from = dev.test_withhold_from >= 0 ? dev.test_withhold_from : 0x7fffffff;
  TCRequests req;
  std::memcpy(req.r, sreq.r, sizeof(psd_token_request) * size_t(S.B));
  const bool tree = S.tree != nullptr;
  // The units on their line, each with its tiles and its cost.
  auto unit_cost = [&](const psd_token_request &r, int tok0, int n) {
    return L::kUnitCost + n * (r.num_new - tok0 > p.TH ? L::kTwoCost : L::kOneCost);
  };
  int64_t tiles = 0, cost = 0;
  struct {
    int64_t tiles, cost;
  } head[kStepRequests];  // of one KV head of a request
  for (int b = 0; b < S.B; ++b) {
    const psd_token_request &r = req.r[b];
    head[b] = {0, 0};
    for (int t = 0; t < r.num_new; t += 2 * p.TH) {
      const int n = unit_tiles(r, t, p.TH, L::NK, tree);
      head[b].tiles += n;
      head[b].cost += unit_cost(r, t, n);
    }
    tiles += head[b].tiles * S.Hkv;
    cost += head[b].cost * S.Hkv;
  }
  if (tiles > 0x7fffffffLL) return fail(PSD_ERR_UNSUPPORTED, "multi_token_decode: more than 2^31 key tiles in one launch");
  // One CTA per SM; a stretch costs at least a tile, so that two bounds inside a unit differ.
  constexpr int kTile = L::kOneCost > L::kTwoCost ? L::kOneCost : L::kTwoCost;
  const int ctas = int(std::min<int64_t>({tiles, cost / kTile, place.ctas, kMaxCtas}));
  // Where the CTAs' stretches begin, and the units that a bound cuts.
  Cuts cuts;
  int n_cuts = 0, most = 0;
  {
    int b = 0, kv = 0, tok0 = 0, n = 0;          // the unit
    int64_t at_tile = 0, at_cost = 0;            // tiles and cost before it
    int64_t req_tile = 0, req_cost = 0;          // before its request
    int64_t before = 0;                          // the tile at which the CTA before begins
    bool cut = false;                            // the unit is in `cuts` already
    auto enter = [&](int kv_, int tok0_) {
      kv = kv_, tok0 = tok0_, n = unit_tiles(req.r[b], tok0, p.TH, L::NK, tree);
      cut = false;
    };
    enter(0, 0);
    for (int c = 0; c <= ctas; ++c) {
      const int64_t at = c * cost / ctas;
      int64_t tile = tiles;
      if (c < ctas) {
        bool moved = false;
        while (at >= req_cost + head[b].cost * S.Hkv) {
          req_tile += head[b].tiles * S.Hkv;
          req_cost += head[b].cost * S.Hkv;
          ++b, moved = true;
        }
        const int h = int((at - req_cost) / head[b].cost);
        if (moved || h != kv) {
          at_tile = req_tile + h * head[b].tiles;
          at_cost = req_cost + h * head[b].cost;
          enter(h, 0);
        }
        while (at >= at_cost + unit_cost(req.r[b], tok0, n)) {
          at_tile += n;
          at_cost += unit_cost(req.r[b], tok0, n);
          enter(kv, tok0 + 2 * p.TH);
        }
        const psd_token_request &r = req.r[b];
        const int per = r.num_new - tok0 > p.TH ? L::kTwoCost : L::kOneCost;
        const int j = int(std::max<int64_t>(0, (at - at_cost - L::kUnitCost) / per));
        tile = at_tile + j;
        req.start[c] = Start{uint16_t(b), uint16_t(kv), tok0, j, 0};
        if (j > 0 && !cut) {  // CTA c - 1 has the first piece
          cut = true;
          Cut &u = cuts.c[n_cuts++];
          u.out = (int64_t(r.token0) + tok0) * S.Hq + int64_t(kv) * S.G;
          u.rows = int16_t(std::min(r.num_new - tok0, 2 * p.TH) * S.G);
          u.first = int16_t(c - 1);
          u.late = before < at_tile;
          u.n = 1;
          most = std::max(most, int(u.rows));
        }
        if (j > 0) ++cuts.c[n_cuts - 1].n;
      }
      if (c > 0) req.start[c - 1].tiles = int32_t(tile - before);
      before = tile;
    }
  }
  p.part_o = place.part_o;
  p.part_lse = place.part_lse;
  p.sum_o = place.sum_o;

  CUtensorMap tmQ = {}, tmK, tmV;
  if (!FP8) {
    const cuuint64_t dims[4] = {64, cuuint64_t(S.Hq), cuuint64_t(S.num_tokens), cuuint64_t(L::kHalves)};
    const cuuint64_t strides[3] = {cuuint64_t(D) * 2, cuuint64_t(S.q_stride) * 2, 128};
    const cuuint32_t box[4] = {64, cuuint32_t(S.G), cuuint32_t(p.TH), 1};
    if (!encode(&tmQ, dev, 4, S.q, dims, strides, box))
      return fail(PSD_ERR_CUDA, "cuTensorMapEncodeTiled failed for the queries");
  }
  const cuuint64_t slots = cuuint64_t(S.num_pages) * cuuint64_t(S.page_size);
  bool mapped;
  if constexpr (FP8) {  // token slots of D codes a head, as they lie
    const cuuint64_t dims[3] = {cuuint64_t(D), cuuint64_t(S.Hkv), slots};
    const cuuint64_t strides[2] = {cuuint64_t(D), cuuint64_t(S.Hkv) * D};
    const cuuint32_t box[3] = {cuuint32_t(D), 1, cuuint32_t(p.sub)};
    mapped = encode(&tmK, dev, 3, S.k_pool, dims, strides, box, D) && encode(&tmV, dev, 3, S.v_pool, dims, strides, box, D);
  } else {
    const cuuint64_t row = cuuint64_t(S.Hkv) * D * 2;  // bytes of a token slot
    const cuuint64_t dims[5] = {64, 8, cuuint64_t(L::kHalves), cuuint64_t(S.Hkv), slots / 8};
    const cuuint64_t strides[4] = {row, 128, cuuint64_t(D) * 2, 8 * row};
    const cuuint32_t box[5] = {64, 8, cuuint32_t(L::kHalves), 1, cuuint32_t(p.sub / 8)};
    mapped = encode(&tmK, dev, 5, S.k_pool, dims, strides, box) && encode(&tmV, dev, 5, S.v_pool, dims, strides, box);
  }
  if (!mapped) return fail(PSD_ERR_CUDA, "cuTensorMapEncodeTiled failed for the KV pool");

  auto kern = step_tc_kernel<D, TERMS, FP8>;
  // once a device: the attribute stays, and setting it is a microsecond of every call
  static std::atomic<uint64_t> ready{0};
  const uint64_t bit = dev.device < 64 ? uint64_t(1) << dev.device : 0;
  cudaError_t e = cudaSuccess;
  if (!(ready.load(std::memory_order_acquire) & bit)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(L::kSmem));
    if (e != cudaSuccess) return fail(PSD_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    ready.fetch_or(bit, std::memory_order_release);
  }
  kern<<<ctas, L::kThreads, L::kSmem, s>>>(tmQ, tmK, tmV, p, req);
  e = cudaGetLastError();
  if (e != cudaSuccess) return fail(PSD_ERR_CUDA, "multi_token_decode launch: %s", cudaGetErrorString(e));
  if (n_cuts == 0) return PSD_OK;
  cudaLaunchConfig_t cfg = {};
  // Few rows have many pieces and want lanes, many rows have two and want loads in flight: 32 lanes a
  // row against 8 took 6.3 us against 8.6 for 4 rows of 24 units in six pieces each, 4.4 against 4.9
  // for 20 rows of 132 units, the same for 96 of 103, and 12.5 against 10 for 256 of 128.
  const bool few = most <= 32;
  constexpr int kWide = D / 4, kNarrow = 8;  // lanes a row
  const int rows = 256 / (few ? kWide : kNarrow);
  cfg.gridDim = dim3(unsigned(n_cuts), unsigned((most + rows - 1) / rows));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = few ? cudaLaunchKernelEx(&cfg, step_join_kernel<D, kWide>, p, cuts)
          : cudaLaunchKernelEx(&cfg, step_join_kernel<D, kNarrow>, p, cuts);
  if (e != cudaSuccess) return fail(PSD_ERR_CUDA, "multi_token_decode join launch: %s", cudaGetErrorString(e));
  return PSD_OK;
}

}  // namespace

bool step_tc_supports(const StepParams &p) {
  // q_scale > 0: the kernel takes the row maximum of the raw scores before scaling
  return (p.D == 64 || p.D == 128) && p.page_size % 8 == 0 && p.G <= kRows && p.q_scale > 0.f &&
         p.num_pages * p.page_size <= 0x7fffffffLL;
}

StepPlace step_tc_place(int ctas, int D, float *base) {
  StepPlace x;
  x.ctas = ctas;
  x.part_o = base;
  x.sum_o = x.part_o + size_t(ctas) * 4 * kRows * size_t(D);
  x.part_lse = x.sum_o + size_t(ctas) * 2 * kRows * size_t(D);
  x.floats = size_t(ctas) * kRows * (6 * size_t(D) + 4);
  return x;
}

psd_status launch_step_tc(const StepParams &p, const StepRequests &req, const StepPlace &place, const DeviceInfo &dev,
                          cudaStream_t s) {
  auto go = [&](auto d) {
    constexpr int D = decltype(d)::value;
    if (p.fp8) return p.out_f32 ? run<D, 2, true>(p, req, place, dev, s) : run<D, 1, true>(p, req, place, dev, s);
    return p.out_f32 ? run<D, 3, false>(p, req, place, dev, s) : run<D, 1, false>(p, req, place, dev, s);
  };
  return p.D == 64 ? go(std::integral_constant<int, 64>{}) : go(std::integral_constant<int, 128>{});
}

}  // namespace psd
