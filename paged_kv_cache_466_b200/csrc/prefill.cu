// Attention of many query tokens per sequence over the paged cache
// (pa_prefill): prompts, chunks of prompts, draft tokens, on the
// fifth-generation tensor cores (tcgen05, accumulators in tensor memory).
//
// Eq. 1 of "KV-Cache Optimization Techniques", section "PagedAttention
// (vLLM)", for every query token of a ragged batch, with an online softmax:
// per KV head, the (token, query head) rows of a sequence that read that head
// are packed (row r is token r / G, head r % G), so the K and V tiles are read
// once for the whole group. A CTA takes 256 rows as two tiles of 128 and walks
// the 128-key tiles between the first and the last key any of its rows sees,
// from the last to the first.
//
//   warps 0-3, 4-7   softmax of row tile 0, 1: thread = row = TMEM lane
//   warp 8           issues the MMAs
//   warps 9-         bring K and V tiles into shared memory: bf16 pools by TMA
//                    (one box per page and 64 columns; warp 9 K, warp 10 V),
//                    quantised pools by copies and exact conversion of the
//                    codes to bf16
//
//   S[128 x 128] = Q K^T  : Q and K K-major, 128-byte-swizzled in shared memory
//   O[128 x D]  += P V    : P from tensor memory (bf16, over the scores' own
//                           columns), V as the page rows lie (MN-major)
//
// PV of tile k and S of tile k + 1 of one row tile are issued together, while
// the other row tile is in its softmax, and one commit covers both: a thread
// that has seen it may read the new scores and may rescale O.
//
// Quantised pools (x = s c + z per row): codes reach the MMA exactly (INT8 as
// c - 128, INT4 as c - 8, E4M3 as it is); q.x = s (q.c) + z sum(q) and
// sum p x = sum (p s) c + sum p z are applied once per score.
//
// P is rounded to bf16, by at most 2^-8 of a weight, as the output is (quantised
// pools: the weight times its row's V scale); the denominator and all statistics
// stay fp32. The weights' roundings are independent and weigh as much as the
// output's one: 1.95e-3 to 2.5e-3 off in the 2-norm against 1.65e-3 for an fp32
// product rounded once. Carrying the rest of P in a second operand ends that
// (1.65e-3), but costs 512 more clocks of MMAs per row tile and key tile in
// series with the rest: capped prompt of 8192 tokens 615 -> 828 us, INT8 draft
// rows 98.9 -> 128 us, FP8 chunk 1409 -> 1836 us. Not taken for a bf16 output.
//
// What bounds it: the chain of one row tile. A tile of 256 rows and 128 keys
// takes 3180 clocks: softmax 1720 (128 exponentials a thread are 1024 clocks of
// the special-function unit), hand-over 140, PV and S 1024, their completion
// 290; the MMAs of both row tiles fill 2048 of them. Around the tiles a CTA
// spends about 10,000 clocks (finding its rows, first loads, output).
// Measured on B200, 32/8 heads of 128, one prompt of 8192 bf16 tokens, causal:
// 450 us, 1220 TFLOP/s (75 % of the measured library rate), capped 560 us.
// Tried and slower: two threads per row (535 against 494 us then), 64-key tiles
// with the next scores computed early (765; an N of 64 reads A from shared
// memory twice as often), P handed over in halves (471 against 452), a quarter
// of the exponentials on the FMA pipe (492 against 474).
#include <atomic>
#include <cmath>
#include <cstddef>
#include <type_traits>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_tcgen05.cuh"

namespace pa {
namespace {

constexpr float kLn2 = 0.693147180559945309f;
constexpr float kRescaleLog2 = 8.0f;   // raise the running max only past this
constexpr float kQuickMost = 1048576.f;  // largest weight sum of a tile done without a maximum pass
constexpr int kTile = 128;            // query rows of a tile (the MMA's M)
constexpr int kKeys = 128;            // keys of a tile
constexpr int kCtaRows = 2 * kTile;
constexpr int kSoftmaxThreads = 256;
constexpr int kMmaWarp = 8;
constexpr int kLoadWarp0 = 9;
constexpr int kTmemCols = 512;        // scores (P over them) of two row tiles, two outputs
// Threads, and registers per thread at launch and after the launch's are split
// anew: a softmax thread holds the 128 scores of its row.
template <int KVT>
constexpr int kThreads = KVT == PA_KV_BF16 ? 384 : 512;
template <int KVT>
constexpr int kLoaders = kThreads<KVT> / 32 - kLoadWarp0;  // warps (bf16 pools use two)
template <int KVT>
constexpr int kLaunchRegs = KVT == PA_KV_BF16 ? 168 : 128;
template <int KVT>
constexpr int kSoftmaxRegs = KVT == PA_KV_BF16 ? 224 : 200;
template <int KVT>
constexpr int kOtherRegs = 56;
template <int KVT>
constexpr int kSplitRegs = kSoftmaxRegs<KVT> * kSoftmaxThreads +
                           kOtherRegs<KVT> * (kThreads<KVT> - kSoftmaxThreads);
static_assert(kSplitRegs<PA_KV_BF16> <= kLaunchRegs<PA_KV_BF16> * kThreads<PA_KV_BF16> &&
                  kSplitRegs<PA_KV_U8_PER_TOKEN> <=
                      kLaunchRegs<PA_KV_U8_PER_TOKEN> * kThreads<PA_KV_U8_PER_TOKEN>,
              "register split");
constexpr uint64_t kWaitLimitNs = 1000000000ull;  // 1 s (a tile takes microseconds)

template <int D, int KVT>
struct Layout {
  static constexpr int kQBytes = kTile * D * 2;      // one row tile's queries
  static constexpr int kSlotBytes = kKeys * D * 2;   // one K or V tile, bf16
  static constexpr int kSlots = (KVT == PA_KV_BF16 ? 5 : 4) * (D == 64 ? 2 : 1);
  // Tiles whose page and scale records are kept. A loader that writes those of
  // tile k has seen the slot of K tile k - kSlots / 2 (or, bf16, of the tile
  // before that one) freed, so the softmax has left the tile before it.
  static constexpr int kRing = D == 64 ? 8 : 4;
  static_assert(kRing > kSlots / 2 + 1 || (KVT != PA_KV_BF16 && kRing > kSlots / 2), "records");
  static constexpr int kQOff = 0;
  static constexpr int kSlotOff = 2 * kQBytes;
  // of the last tiles: K scale, K zero, V scale, V zero of every key
  static constexpr int kSzOff = kSlotOff + kSlots * kSlotBytes;
  static constexpr int kSzTile = 4 * kKeys * 4;
  static constexpr int kSzBytes = KVT == PA_KV_BF16 ? 0 : kRing * kSzTile;
  // quantised pools: per loader warp a 16-key block of codes (and the scales
  // and zeros of its keys) as it comes from the pool. (A fourth slot instead
  // of deeper staging: 8192 FP8 tokens 880 us with three slots and three
  // stages, 699 us with four slots and one.)
  static constexpr int kRawOff = kSzOff + kSzBytes;
  static constexpr int kRawBlock = 16 * (KVT == PA_KV_U4_PER_TOKEN ? D / 2 : D);
  static constexpr int kRawBytes =
      KVT == PA_KV_BF16 ? 0 : kLoaders<KVT> * (kRawBlock + 256);
  static constexpr int kBarOff = kRawOff + kRawBytes;
  static constexpr int kBytes = kBarOff + 512;
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

// Shared control block behind the tiles.
struct Control {
  uint64_t full[10], empty[10];  // K / V slots
  uint64_t q_full;               // queries in shared memory
  uint64_t s_full[2];            // scores of a row tile (and the PV before them) done
  uint64_t p_full[2];            // P of a row tile stored, O rescaled
  uint64_t stopped;              // MMAs in flight when the block gives up are done
  uint32_t tmem;
  int32_t dead;                  // a bounded wait ran out: everybody stops
  int32_t seq, blk, q0, qlen, ctx;
  int32_t lo, hi;                // first / past-the-last key of any row
  alignas(8) uint8_t valid[8][8];      // per tile: 16-key blocks in valid pages
};
static_assert(offsetof(Control, valid) % 8 == 0 && sizeof(Control) <= 512, "control block");

__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}

// Waits for a phase; gives up after kWaitLimitNs, or at once when another
// warp has given up.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int32_t *dead) {
  if (try_wait(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  for (int i = 0; i < (1 << 26); ++i) {
    if (try_wait(bar, parity)) return true;
    if ((i & 15) == 15 && (*dead || global_ns() - t0 > kWaitLimitNs)) break;
  }
  *dead = 1;
  return false;
}

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count));
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_arrive_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
// One lane of a converged warp, the same every time. The MMA and copy loops run
// warp-uniformly and only the issue itself is elected: their operands then
// stay in uniform registers (in a branch of one lane every operand of every
// MMA is moved there again, 97 clocks an MMA instead of 64).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void proxy_fence() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// One page's block of one KV head, 64 columns: [64][P][1][1] of the pool seen
// as [D][P][Hkv][num_pages]. A page id past the pool reads zeros.
__device__ __forceinline__ void tma_page(const CUtensorMap *map, uint32_t dst, uint32_t bar, int x,
                                         int h, int page) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, "
      "{%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(x), "r"(0), "r"(h), "r"(page)
      : "memory");
}

__device__ __forceinline__ void sts_u4(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

// ---- exact conversions of codes to bf16 pairs ---------------------------------------

__device__ __forceinline__ uint32_t bf16x2_sub(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Two codes in bits 0..7 and 16..23 of w (the other bits anything). INT8: 0x4300
// | (c & 127) is 128 + (c & 127); subtracting 128 where bit 7 is set and 256
// where it is not leaves c - 128.
__device__ __forceinline__ uint32_t u8x2_to_bf16(uint32_t w) {
  return bf16x2_sub((w & 0x007F007Fu) | 0x43004300u, (w & 0x00800080u) ^ 0x43804380u);
}
// Two nibbles in bits 0..3 and 16..19 -> c - 8.
__device__ __forceinline__ uint32_t u4x2_to_bf16(uint32_t w) {
  return bf16x2_sub((w & 0x000F000Fu) | 0x43004300u, 0x43084308u);
}
// Two E4M3 codes whose signs lie in bits 15 and 31 of `sign` and whose other
// bits in 4..10 and 20..26 of `mag`: read as bf16 they are the value times
// 2^-120 (subnormals included).
__device__ __forceinline__ uint32_t e4m3x2_to_bf16(uint32_t sign, uint32_t mag) {
  return bf16x2_mul((sign & 0x80008000u) | (mag & 0x07F007F0u), 0x7B807B80u);
}

// A 16-key block of codes as a warp holds it, 16 bytes per lane and piece, and
// its conversion into a K-major tile. Codes are taken in the order in which
// they pair up without byte shuffles: element e of every 8 lands in
// place place_of(e). The queries are put in the same order, and the columns of O are
// taken back out of it. Zero bytes of keys that do not exist become the code
// shift, whose scale and zero are 0 and whose V weight is 0.
template <int D, int KVT>
struct Rows {
  static constexpr int kRowBytes = KVT == PA_KV_U4_PER_TOKEN ? D / 2 : D;
  static constexpr int kPieces = 16 * kRowBytes / 512;  // per lane
  static __device__ __forceinline__ uint4 convert8(uint32_t w0, uint32_t w1) {  // 8 codes
    if constexpr (KVT == PA_KV_FP8_PER_TOKEN)
      return make_uint4(e4m3x2_to_bf16(w0 << 8, w0 << 4), e4m3x2_to_bf16(w0, w0 >> 4),
                        e4m3x2_to_bf16(w1 << 8, w1 << 4), e4m3x2_to_bf16(w1, w1 >> 4));
    else
      return make_uint4(u8x2_to_bf16(w0), u8x2_to_bf16(w0 >> 8), u8x2_to_bf16(w1),
                        u8x2_to_bf16(w1 >> 8));
  }
  static __device__ __forceinline__ uint4 convert8(uint32_t w) {  // 8 INT4 codes
    return make_uint4(u4x2_to_bf16(w), u4x2_to_bf16(w >> 4), u4x2_to_bf16(w >> 8),
                      u4x2_to_bf16(w >> 12));
  }
  static __device__ __forceinline__ void store(uint32_t tile, int blk, int lane, uint32_t raw) {
    uint4 v[kPieces];
#pragma unroll
    for (int k = 0; k < kPieces; ++k) v[k] = lds128(raw + (lane + 32 * k) * 16);
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      const int at = (lane + 32 * k) * 16;
      const int r = blk * 16 + at / kRowBytes;
      if constexpr (KVT == PA_KV_U4_PER_TOKEN) {
        const int c0 = at % kRowBytes / 4;  // four 16-byte chunks of bf16
        const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) sts_u4(tile + sw128(r, c0 + j, kKeys), convert8(w[j]));
      } else {
        // lanes of the second 64 columns write their chunks in the other order:
        // both halves' chunks would share banks
        const int pc = at % kRowBytes / 16, o = (pc >> 2) & 1;
        const uint4 a = convert8(v[k].x, v[k].y), b = convert8(v[k].z, v[k].w);
        sts_u4(tile + sw128(r, 2 * pc + o, kKeys), o ? b : a);
        sts_u4(tile + sw128(r, 2 * pc + 1 - o, kKeys), o ? a : b);
      }
    }
  }
};
// Place of element e (0..7) among eight converted codes.
template <int KVT>
__host__ __device__ constexpr int place_of(int e) {
  if (KVT == PA_KV_BF16) return e;
  if (KVT == PA_KV_U4_PER_TOKEN) return e < 4 ? 2 * e : 2 * e - 7;  // 0 4 1 5 2 6 3 7
  return (e & 4) | ((e & 1) << 1) | ((e & 2) >> 1);                 // 0 2 1 3 of every four
}
// Eight bf16 queries in that order.
template <int KVT>
__device__ __forceinline__ uint4 place8(uint4 v) {
  if constexpr (KVT == PA_KV_U4_PER_TOKEN)
    return make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632),
                      __byte_perm(v.y, v.w, 0x5410), __byte_perm(v.y, v.w, 0x7632));
  else
    return make_uint4(__byte_perm(v.x, v.y, 0x5410), __byte_perm(v.x, v.y, 0x7632),
                      __byte_perm(v.z, v.w, 0x5410), __byte_perm(v.z, v.w, 0x7632));
}
template <int KVT>
constexpr float kCodeShift = KVT == PA_KV_U8_PER_TOKEN ? 128.f : KVT == PA_KV_U4_PER_TOKEN ? 8.f : 0.f;

// ---- two fp32 values per instruction ---------------------------------------------------

using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pack2(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

// How the scores are changed.
enum { kCapped = 1, kBiased = 2 };

// ---- the kernel ----------------------------------------------------------------------

template <int D, int KVT, int MODE>  // MODE: kCapped | kBiased
__global__ void __launch_bounds__(kThreads<KVT>, 1)
    prefill_kernel(const __grid_constant__ PrefillArgs a) {
  using L = Layout<D, KVT>;
  constexpr bool kQuant = KVT != PA_KV_BF16;
  constexpr bool kCap = (MODE & kCapped) != 0, kBias = (MODE & kBiased) != 0;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char *smem = smem_raw;  // the swizzled tiles need the 1024-byte alignment
  Control &c = *reinterpret_cast<Control *>(smem + L::kBarOff);
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait_primary();

  const int h = blockIdx.x % a.hkv;
  const int split = blockIdx.x / a.hkv % a.S;
  const int flat = blockIdx.x / a.hkv / a.S;
  const int G = a.hq / a.hkv;

  // ---- which sequence and rows: warp 0 adds up the sequences' blocks, 32
  // sequences at a time (their lengths stay in registers when that is all).
  // Blocks are taken from the last to the first, so that with causal masks the
  // ones with most keys start first.
  if (warp == 0) {
    int s = 0, len = 0, ctx = 0, nb = 0;
    auto load = [&](int b) {
      s = len = ctx = nb = 0;
      if (b >= a.B) return;
      const int q0 = __ldg(a.q_begin + b), q1 = __ldg(a.q_begin + b + 1);
      ctx = __ldg(a.ctx + b);
      s = max(q0, 0);
      len = max(min(q1, a.n), s) - s;  // (no entry makes the difference wrap)
      if (blockIdx.x == 0 && (q0 < 0 || q1 > a.n || q1 < q0)) flag_error(a.d_err, PA_DERR_BAD_SEQ);
      nb = (int)(((long long)len * G + kCtaRows - 1) / kCtaRows);
    };
    if (lane == 0) c.seq = -1;
    int total = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      load(b0 + lane);
      total += __reduce_add_sync(0xffffffffu, nb);
    }
    const int want = total - 1 - flat;
    int before = 0;
    for (int b0 = 0; b0 < a.B && want >= before; b0 += 32) {  // (want < 0: past the last block)
      if (a.B > 32) load(b0 + lane);
      int incl = nb;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (want >= before + incl - nb && want < before + incl) {
        c.seq = b0 + lane;
        c.blk = want - (before + incl - nb);
        c.q0 = s;
        c.qlen = len;
        if (ctx < len || ctx > a.max_pages * a.P) {  // no such context: sees nothing
          flag_error(a.d_err, PA_DERR_BAD_CTX);
          ctx = 0;
        }
        c.ctx = ctx;
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
  } else if (tid == 32) {
    c.lo = 0x7fffffff;
    c.hi = 0;
    c.dead = 0;
    for (int i = 0; i < L::kSlots; ++i) {
      bar_init(smem_u32(&c.full[i]), kQuant ? kKeys / 16 : 1);
      bar_init(smem_u32(&c.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(smem_u32(&c.s_full[i]), 1);
      bar_init(smem_u32(&c.p_full[i]), kTile);
    }
    bar_init(smem_u32(&c.q_full), kSoftmaxThreads);
    bar_init(smem_u32(&c.stopped), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  if (c.seq < 0) return;  // CTA-uniform: past the last block
  const int b = c.seq, qlen = c.qlen, ctx = c.ctx;
  const int rows = qlen * G - c.blk * kCtaRows;  // of this CTA; may pass 256

  // ---- this thread's row: what it sees
  int lo = 0, hi = 0x7fffffff;  // an unused row masks nothing
  int pos = 0;
  bool row_ok = false;
  size_t orow = 0;
  const int sub = warp >> 2, rl = tid & 127;  // row tile and row of a softmax thread
  if (tid < kSoftmaxThreads) {
    row_ok = tid < rows;
    if (row_ok) {
      const int r = c.blk * kCtaRows + tid;
      const int tok = r / G, head = h * G + r % G;
      orow = (size_t)(c.q0 + tok) * a.hq + head;
      pos = ctx - qlen + tok;
      hi = pos + 1;
      if (a.prefix_end != nullptr) hi = max(hi, __ldg(a.prefix_end + c.q0 + tok));
      hi = min(hi, ctx);
      if (a.doc_begin != nullptr) lo = max(__ldg(a.doc_begin + c.q0 + tok), 0);
      if (hi <= lo) lo = hi = 0;
    }
    const bool sees = row_ok && hi > lo;
    const int wlo = __reduce_min_sync(0xffffffffu, sees ? lo : 0x7fffffff);
    const int whi = __reduce_max_sync(0xffffffffu, sees ? hi : 0);
    if (lane == 0 && whi > 0) {
      atomicMin(&c.lo, wlo);
      atomicMax(&c.hi, whi);
    }
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&c.tmem)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();  // the key range and the TMEM address: the loads may begin
  tc_fence_after();

  // ---- this split's key tiles [t0, t1), walked from t1 - 1 down
  int t0 = 0, t1 = 0;
  if (c.hi > 0) {
    const int f = c.lo / kKeys, e = (c.hi + kKeys - 1) / kKeys;
    const int per = (e - f + a.S - 1) / a.S;
    t0 = f + split * per;
    t1 = min(t0 + per, e);
    if (t1 < t0) t1 = t0;
  }
  const int n = t1 - t0;
  // Of the first tile, blocks (bf16 pools: pages) that end at or before this key
  // are not read and their table entries not looked at: the cache may have
  // dropped the pages before the first document.
  const int first = c.lo;
  const int subs = rows > kTile ? 2 : 1;  // row tiles in use
  const uint32_t tmem = c.tmem;
  volatile int32_t *dead = &c.dead;

  // With one row tile the other tile's softmax warps help with the codes.
  const int NW = kLoaders<KVT> + (subs == 1 ? 4 : 0);
  auto load_codes = [&](int w, uint32_t raw) {
    // ---- quantised pools: the loader warps (w of NW) take the tiles' 16-key
    // blocks in turn: a block's codes, and the scales and zeros of its keys, are copied
    // to shared memory while its slot is waited for, and a lane converts what
    // it copied itself.
    using R = Rows<D, KVT>;
    const int p_log2 = a.P == 32 ? 5 : 4;
    const int total = n * 2 * (kKeys / 16);
    const int32_t *table = a.block_tables + (size_t)b * a.max_pages;
    auto token_of = [&](int m) { return (t1 - 1 - (m >> 4)) * kKeys + (m & 7) * 16; };
    auto there = [&](int m) {
      return m < total && token_of(m) < ctx && token_of(m) + 16 > first;
    };
    // the table's entry for block m, not looked at yet (the load is waited
    // for where it is used, a block later)
    auto entry_of = [&](int m) { return there(m) ? __ldg(table + (token_of(m) >> p_log2)) : 0; };
    auto fetch = [&](int m, int page) {
      if (m < total) {
        const int tok = token_of(m);
        const bool good = there(m) && page >= 0 && page < a.num_pages;
        const int live = good ? min(ctx - tok, 16) : 0;
        const bool is_v = (m >> 3) & 1;
        const size_t row0 = (((size_t)(good ? page : 0) * a.hkv + h) << p_log2) + (tok & (a.P - 1));
        const unsigned char *src =
            static_cast<const unsigned char *>(is_v ? a.v_pool : a.k_pool) + row0 * R::kRowBytes;
#pragma unroll
        for (int k = 0; k < R::kPieces; ++k) {
          const int at = (lane + 32 * k) * 16;
          cp_async16(raw + at, src + at, at / R::kRowBytes < live ? 16u : 0u);
        }
        if (!is_v)
          cp_async8(raw + L::kRawBlock + lane * 8,
                    reinterpret_cast<const float2 *>(lane < 16 ? a.k_sz : a.v_sz) + row0 + (lane & 15),
                    (lane & 15) < live ? 8u : 0u);
      }
      cp_async_commit();
    };
    int page = entry_of(w), next = entry_of(w + NW);
    fetch(w, page);
    for (int m = w; m < total; m += NW) {
      const int i = m >> 3, blk = m & 7, slot = i % L::kSlots;
      const bool is_v = i & 1;
      const bool bad = there(m) && (page < 0 || page >= a.num_pages);
      bool ok = true;
      if (i >= L::kSlots) ok = wait_bar(smem_u32(&c.empty[slot]), (i / L::kSlots - 1) & 1, dead);
      if (!__all_sync(0xffffffffu, ok)) break;
      cp_async_wait<0>();
      if (!is_v) {
        const int ring = (i >> 1) % L::kRing;
        float *sz = reinterpret_cast<float *>(smem + L::kSzOff + ring * L::kSzTile) +
                    (lane < 16 ? 0 : 2 * kKeys) + blk * 16 + (lane & 15);
        const uint2 v = lds64(raw + L::kRawBlock + lane * 8);
        const float x = __uint_as_float(v.x), z = __uint_as_float(v.y);
        const float f = lane < 16 ? a.scale_log2 : 1.f;  // K rows carry the score scale
        sz[0] = x * f;
        sz[kKeys] = fmaf(x, kCodeShift<KVT>, z) * f;
        if (lane == 0) {
          c.valid[ring][blk] = !bad;
          if (bad) flag_error(a.d_err, PA_DERR_BAD_PAGE);
        }
      }
      R::store(sbase + L::kSlotOff + slot * L::kSlotBytes, blk, lane, raw);
      proxy_fence();
      __syncwarp();
      if (lane == 0) bar_arrive(smem_u32(&c.full[slot]));
      page = next;
      fetch(m + NW, page);
      next = entry_of(m + 2 * NW);
    }
    cp_async_wait<0>();
  };

  if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs<KVT>));
    if (warp == kMmaWarp) {
      if (n > 0) {
        // ---- MMA issue
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        auto wait_slot = [&](int i) {
          const bool done =
              wait_bar(smem_u32(&c.full[i % L::kSlots]), (i / L::kSlots) & 1, dead);
          return (bool)__all_sync(0xffffffffu, done);
        };
        // operands advance by constants inside a tile: one addition per MMA
        const uint64_t q_desc = smem_desc(sbase + L::kQOff, 16, 1024);
        const uint64_t k_desc = smem_desc(sbase + L::kSlotOff, 16, 1024);
        const uint64_t v_desc = smem_desc(sbase + L::kSlotOff, kKeys * 128, 1024);
        auto issue_s = [&](int sb, int k) {
          const uint64_t q0 = q_desc + sb * (L::kQBytes >> 4);
          const uint64_t k0 = k_desc + (2 * k) % L::kSlots * (L::kSlotBytes >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            umma_bf16(tm + sb * kKeys, q0 + (((kk >> 2) * (kTile * 128) + (kk & 3) * 32) >> 4),
                      k0 + (((kk >> 2) * (kKeys * 128) + (kk & 3) * 32) >> 4),
                      instr_desc(kKeys, false), kk > 0);
        };
        auto issue_pv = [&](int sb, int k) {
          const uint64_t v0 = v_desc + (2 * k + 1) % L::kSlots * (L::kSlotBytes >> 4);
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)
            umma_bf16_ts(tm + 2 * kKeys + sb * D, tm + sb * kKeys + kk * 8, v0 + ((kk * 2048) >> 4),
                         instr_desc(D, true), k > 0 || kk > 0);
        };
        bool ok = __all_sync(0xffffffffu, wait_bar(smem_u32(&c.q_full), 0, dead));
        ok = ok && wait_slot(0);
        tc_fence_after();
        if (ok && elect_one()) {
          for (int sb = 0; sb < subs; ++sb) {
            issue_s(sb, 0);
            umma_commit(smem_u32(&c.s_full[sb]));
          }
          umma_commit(smem_u32(&c.empty[0]));
        }
        __syncwarp();
        for (int k = 0; ok && k < n; ++k) {
          ok = wait_slot(2 * k + 1);
          if (ok && k + 1 < n) ok = wait_slot(2 * k + 2);
          for (int sb = 0; ok && sb < subs; ++sb) {
            ok = __all_sync(0xffffffffu, wait_bar(smem_u32(&c.p_full[sb]), k & 1, dead));
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
              issue_pv(sb, k);
              if (k + 1 < n) issue_s(sb, k + 1);
              umma_commit(smem_u32(&c.s_full[sb]));
            }
            __syncwarp();
          }
          if (ok && elect_one()) {
            umma_commit(smem_u32(&c.empty[(2 * k + 1) % L::kSlots]));
            if (k + 1 < n) umma_commit(smem_u32(&c.empty[(2 * k + 2) % L::kSlots]));
          }
          __syncwarp();
        }
        if (!ok) {
          // stopped early: the MMAs in flight must end before their tensor memory is freed
          if (elect_one()) umma_commit(smem_u32(&c.stopped));
          __syncwarp();
          mbar_wait_bounded(smem_u32(&c.stopped), 0, kWaitLimitNs);
        }
      }
    } else if constexpr (!kQuant) {
      // ---- K tiles (warp 9) and V tiles (warp 10) by TMA, page by page
      if (warp < kLoadWarp0 + 2 && n > 0) {
        const bool is_v = warp != kLoadWarp0;
        const CUtensorMap *map = is_v ? &a.tmv : &a.tmk;
        const int per_tile = kKeys / a.P;
        const uint32_t box = (uint32_t)a.P * 128;
        const int32_t *table = a.block_tables + (size_t)b * a.max_pages;
        // lane x: the id of page x of tile k; past the context or before the
        // first key -1
        auto outside = [&](int tok) { return tok >= ctx || tok + a.P <= first; };
        auto page_of = [&](int k) {
          const int tok = (t1 - 1 - k) * kKeys + lane * a.P;
          return k < n && lane < per_tile && !outside(tok) ? __ldg(table + tok / a.P) : -1;
        };
        int id = page_of(0);
        bool ok = true;
        for (int k = 0; k < n; ++k) {
          const int tile = t1 - 1 - k;
          const int next = page_of(k + 1);
          const bool none = outside(tile * kKeys + lane * a.P);
          const bool bad = lane < per_tile && !none && (id < 0 || id >= a.num_pages);
          const int page = none || bad ? a.num_pages : id;  // past the pool: zeros
          if (!is_v && lane < per_tile) {
            if (bad) flag_error(a.d_err, PA_DERR_BAD_PAGE);
            for (int x = 0; x < a.P / 16; ++x) c.valid[k % L::kRing][lane * (a.P / 16) + x] = !bad;
          }
          const int i = 2 * k + is_v, slot = i % L::kSlots;
          if (i >= L::kSlots)
            ok = wait_bar(smem_u32(&c.empty[slot]), (i / L::kSlots - 1) & 1, dead);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const uint32_t dst = sbase + L::kSlotOff + slot * L::kSlotBytes;
          const uint32_t bar = smem_u32(&c.full[slot]);
          // the page the context ends in: its rows past the end hold anything
          // (NaN too), so that block is copied by hand and filled with zeros
          const int end = ctx - tile * kKeys;
          const int cut = end < kKeys && end % a.P != 0 ? end / a.P : -1;  // warp-uniform
          if (cut >= 0) {
            const int pg = __shfl_sync(0xffffffffu, page, cut);
            const unsigned char *src =
                static_cast<const unsigned char *>(is_v ? a.v_pool : a.k_pool) +
                ((size_t)(pg < a.num_pages ? pg : 0) * a.hkv + h) * a.P * D * 2;
            const int live = pg < a.num_pages ? end % a.P : 0;
            for (int x = lane; x < a.P * (D / 8); x += 32) {
              const int r = x / (D / 8), j = x % (D / 8);
              const uint4 v = r < live ? ldg_nc128(src + ((size_t)r * D + j * 8) * 2)
                                       : make_uint4(0, 0, 0, 0);
              sts_u4(dst + sw128(cut * a.P + r, j, kKeys), v);
            }
            proxy_fence();
          }
          __syncwarp();
          if (elect_one()) bar_arrive_tx(bar, box * (per_tile - (cut >= 0 ? 1 : 0)) * (D / 64));
          for (int x = 0; x < per_tile; ++x) {
            const int pg = __shfl_sync(0xffffffffu, page, x);
            if (x != cut && elect_one()) {
#pragma unroll
              for (int half = 0; half < D / 64; ++half)
                tma_page(map, dst + half * (kKeys * 128) + x * box, bar, half * 64, h, pg);
            }
            __syncwarp();
          }
          id = next;
        }
        if (!ok) {
          // stopped early: the copies in flight must land before the CTA ends
          for (int s = 0; s < L::kSlots; ++s)
            for (int par = 0; par < 2; ++par) mbar_wait_bounded(smem_u32(&c.full[s]), par, 1000000ull);
        }
      }
    } else if (n > 0) {
      load_codes(warp - kLoadWarp0, sbase + L::kRawOff + (warp - kLoadWarp0) * (L::kRawBlock + 256));
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs<KVT>));
    // the warp's 32 query rows, D / 8 lanes a row (rows past the last: zeros)
    const uint32_t dst = sbase + L::kQOff + sub * L::kQBytes;
    constexpr int kRowLanes = D / 8;
    // (a second row tile that is not used leaves its place to the loaders;
    // without a key tile nothing waits for the queries of the other warps, which
    // the rows staged below would meet in shared memory)
    if (sub < subs && n > 0) {
#pragma unroll
      for (int i = 0; i < kRowLanes; ++i) {
        const int r = i * (32 / kRowLanes) + lane / kRowLanes, k = lane % kRowLanes;
        const size_t from = __shfl_sync(0xffffffffu, (unsigned long long)orow, r);
        const bool live = __shfl_sync(0xffffffffu, (int)row_ok, r) != 0;
        const unsigned char *src = static_cast<const unsigned char *>(a.q) + from * D * 2 + k * 16;
        const uint32_t to = dst + sw128((warp & 3) * 32 + r, k, kTile);
        if constexpr (kQuant)
          sts_u4(to, place8<KVT>(live ? ldg_nc128(src) : make_uint4(0, 0, 0, 0)));
        else
          cp_async16(to, src, live ? 16u : 0u);
      }
    }
    cp_async_commit();
    cp_async_wait<0>();
    proxy_fence();
    bar_arrive(smem_u32(&c.q_full));
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + sub * kKeys + lane_off;
    const uint32_t t_o = tmem + 2 * kKeys + sub * D + lane_off;
    float m_run = -INFINITY, l_run = 0.f, z_run = 0.f;
    bool ok = true;
    if constexpr (kQuant) {
      if (sub >= subs && n > 0)  // (in the place of the other row tile's queries)
        load_codes(kLoaders<KVT> + warp - 4,
                   sbase + L::kQOff + L::kQBytes + (warp - 4) * (L::kRawBlock + 256));
    }
    if (sub < subs && n > 0) {
      constexpr bool kZero = kQuant && KVT != PA_KV_FP8_PER_TOKEN;  // rows have a zero point
      float qsum = 0.f;
      if constexpr (kZero) {
        __syncwarp();  // a warp's rows are loaded by the warp
        const uint32_t qs = sbase + L::kQOff + sub * L::kQBytes;
        for (int k = 0; k < D / 8; ++k) {
          const uint4 v = lds128(qs + sw128(rl, k, kTile));
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int x = 0; x < 4; ++x) qsum += bf16_lo(w[x]) + bf16_hi(w[x]);
        }
      }
      float slope = 0.f;
      if constexpr (kBias)
        if (row_ok)
          slope = __ldg(a.slopes + orow % a.hq) * 1.4426950408889634f;
      for (int k = 0; k < n; ++k) {
        // (a wait that runs out makes all later ones end at once)
        ok = ok && wait_bar(smem_u32(&c.s_full[sub]), k & 1, dead);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const int k0 = (t1 - 1 - k) * kKeys;
        float s[kKeys];
#pragma unroll
        for (int c0 = 0; c0 < kKeys; c0 += 32)
          tmem_ld32(t_s + c0, reinterpret_cast<uint32_t(&)[32]>(s[c0]));
        tmem_wait_ld();
        const uint32_t sz = sbase + L::kSzOff + k % L::kRing * L::kSzTile;
        const uint2 valid = lds64(smem_u32(c.valid[k % L::kRing]));
        const bool all_valid = valid.x == 0x01010101u && valid.y == 0x01010101u;
        // warp-uniform: every row of the warp sees every key of the tile
        const bool full = __all_sync(0xffffffffu, lo <= k0 && hi >= k0 + kKeys) && all_valid;

        // Weights p = 2^(x - m) of all keys of the tile, x = mul s (or the
        // polynomial of the cap), into P over the scores' columns, two keys
        // per column. Adds them to lt and, for pools with zeros, p z to zt;
        // returns the largest s^2 with kPoly (else 0).
        float lt, zt;
        // bias_0, the bias of the tile's first key, and sl, the bias' step from
        // key to key, are added to x (a quick way of a biased kernel).
        auto weights = [&](auto poly_c, auto bias_c, float mul, float m, float bias_0, float sl) {
          constexpr bool kPoly = decltype(poly_c)::value, kAdd = decltype(bias_c)::value;
          const f32x2 mul_2 = pack2(mul, mul), neg_2 = pack2(bias_0 - m, bias_0 - m);
          const f32x2 sl_2 = pack2(sl, sl);
          f32x2 l2[2] = {0, 0}, z2 = 0;
          float y4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c0 = 0; c0 < kKeys; c0 += 32) {
            uint32_t w[16];
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              f32x2 p[2];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int e = c0 + 2 * (j + i);
                const f32x2 u = pack2(s[e], s[e + 1]);
                f32x2 x = neg_2;
                if constexpr (kAdd) x = fma2(sl_2, pack2((float)e, (float)(e + 1)), neg_2);
                if constexpr (kPoly) {
                  const f32x2 y = mul2(u, u);
                  float y0, y1;
                  unpack2(y, y0, y1);
                  y4[(j + i) & 3] = max3(y4[(j + i) & 3], y0, y1);
                  f32x2 r = pack2(a.cap_r[3], a.cap_r[3]);
#pragma unroll
                  for (int q = 2; q >= 0; --q) r = fma2(r, y, pack2(a.cap_r[q], a.cap_r[q]));
                  x = fma2(u, r, x);
                } else {
                  x = fma2(u, mul_2, x);
                }
                float x0, x1;
                unpack2(x, x0, x1);
                p[i] = pack2(fast_exp2(x0), fast_exp2(x1));
                l2[i] = add2(l2[i], p[i]);
              }
              if constexpr (kQuant) {
                const uint4 vs = lds128(sz + 2 * kKeys * 4 + (c0 + 2 * j) * 4);
                if constexpr (kZero) {
                  const uint4 vz = lds128(sz + 3 * kKeys * 4 + (c0 + 2 * j) * 4);
                  z2 = fma2(p[0], pack2(__uint_as_float(vz.x), __uint_as_float(vz.y)), z2);
                  z2 = fma2(p[1], pack2(__uint_as_float(vz.z), __uint_as_float(vz.w)), z2);
                }
                p[0] = mul2(p[0], pack2(__uint_as_float(vs.x), __uint_as_float(vs.y)));
                p[1] = mul2(p[1], pack2(__uint_as_float(vs.z), __uint_as_float(vs.w)));
              }
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                float p0, p1;
                unpack2(p[i], p0, p1);
                w[j + i] = pack_bf16(p0, p1);
              }
            }
            tmem_st16(t_s + c0 / 2, w);
          }
          float x0, x1;
          unpack2(add2(l2[0], l2[1]), x0, x1);
          lt = x0 + x1;
          unpack2(z2, x0, x1);
          zt = x0 + x1;
          return fmaxf(fmaxf(y4[0], y4[1]), fmaxf(y4[2], y4[3]));
        };

        float mul = a.scale_log2;  // brings s to log2 units
        if constexpr (kQuant) {    // codes to scores in log2 units
          mul = 1.f;
          const f32x2 qq = pack2(qsum, qsum);
#pragma unroll
          for (int j = 0; j < kKeys; j += 4) {
            const uint4 ks = lds128(sz + j * 4);
            f32x2 u0 = pack2(s[j], s[j + 1]), u1 = pack2(s[j + 2], s[j + 3]);
            const f32x2 f0 = pack2(__uint_as_float(ks.x), __uint_as_float(ks.y)),
                        f1 = pack2(__uint_as_float(ks.z), __uint_as_float(ks.w));
            if constexpr (kZero) {
              const uint4 kz = lds128(sz + kKeys * 4 + j * 4);
              u0 = fma2(u0, f0, mul2(pack2(__uint_as_float(kz.x), __uint_as_float(kz.y)), qq));
              u1 = fma2(u1, f1, mul2(pack2(__uint_as_float(kz.z), __uint_as_float(kz.w)), qq));
            } else {
              u0 = mul2(u0, f0);
              u1 = mul2(u1, f1);
            }
            unpack2(u0, s[j], s[j + 1]);
            unpack2(u1, s[j + 2], s[j + 3]);
          }
        }
        // The quick way: weights against the running reference as it stands,
        // without a look at the tile's maximum first. It holds when every row
        // has a reference, no key is masked, no weight sum has outgrown
        // kQuickMost (weights above 1 are carried as exactly as those below) and, capped, all
        // scores lie where the polynomial is good. Else the tile is done
        // again, below, from the scores still in registers.
        // (a biased tile also needs all its keys before the query: the bias is
        // then linear in the key)
        bool quick = full && mul > 0.f && __all_sync(0xffffffffu, m_run > -INFINITY);
        if constexpr (kBias)
          quick = quick && (a.prefix_end == nullptr ||
                            __all_sync(0xffffffffu, !row_ok || pos >= k0 + kKeys - 1));
        if (quick) {
          bool good = true;
          const std::integral_constant<bool, kBias> bias_c{};
          const float bias_0 = kBias ? slope * (float)(k0 - pos) : 0.f;
          if constexpr (kCap)
            good = weights(std::true_type{}, bias_c, mul, m_run, bias_0, slope) <= a.cap_u * a.cap_u;
          else
            weights(std::false_type{}, bias_c, mul, m_run, bias_0, slope);
          quick = __all_sync(0xffffffffu, good && lt < kQuickMost);
          if (!quick) tmem_wait_st();  // this P is written over
        }
        if (!quick) {
          if constexpr (MODE == 0) {
            const f32x2 mul_2 = pack2(mul, mul);
#pragma unroll
            for (int j = 0; j < kKeys; j += 2) unpack2(mul2(pack2(s[j], s[j + 1]), mul_2), s[j], s[j + 1]);
          } else {
#pragma unroll
            for (int j = 0; j < kKeys; ++j) {
              s[j] *= mul;
              if constexpr (kCap) s[j] = a.cap_l2 * tanh_f32(s[j] * a.inv_cap);
              if constexpr (kBias) s[j] -= slope * fabsf((float)(pos - k0 - j));
            }
          }
          if (!full) {
            // 32 keys at a time: most such blocks are seen by all the warp's rows
            // (packed documents 242 -> 239 us; the capped kernel, whose registers
            // it costs, 562 -> 606 us, does without)
            const int begin = lo - k0, end = hi - k0;
#pragma unroll
            for (int c0 = 0; c0 < kKeys; c0 += 32) {
              if (MODE == kCapped || !__all_sync(0xffffffffu, begin <= c0 && end >= c0 + 32)) {
#pragma unroll
                for (int j = c0; j < c0 + 32; ++j)
                  if ((unsigned)(j - begin) >= (unsigned)(end - begin)) s[j] = -INFINITY;
              }
            }
            if (!all_valid) {
#pragma unroll
              for (int j = 0; j < kKeys; ++j)
                if (((j < 64 ? valid.x : valid.y) >> (j / 16 % 4 * 8) & 1u) == 0) s[j] = -INFINITY;
            }
          }
          float m4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int j = 0; j < kKeys; j += 8)
#pragma unroll
            for (int i = 0; i < 4; ++i) m4[i] = max3(m4[i], s[j + 2 * i], s[j + 2 * i + 1]);
          const float mx = max3(fmaxf(m4[0], m4[1]), m4[2], m4[3]);
          const bool need = mx > m_run + kRescaleLog2 || (m_run == -INFINITY && mx > -INFINITY);
          if (__any_sync(0xffffffffu, need)) {  // tcgen05.ld / st are warp-wide
            const float m_new = need ? fmaxf(m_run, mx) : m_run;
            const float alpha = need && m_run != -INFINITY ? fast_exp2(m_run - m_new) : 1.f;
            m_run = m_new;
            l_run *= alpha;
            z_run *= alpha;
            if (k > 0) {
#pragma unroll 1
              for (int c0 = 0; c0 < D; c0 += 16) {
                uint32_t u[16];
                tmem_ld16(t_o + c0, u);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) u[j] = __float_as_uint(__uint_as_float(u[j]) * alpha);
                tmem_st16(t_o + c0, u);
              }
            }
          }
          weights(std::false_type{}, std::false_type{}, 1.f, m_run == -INFINITY ? 0.f : m_run, 0.f, 0.f);
        }
        l_run += lt;
        z_run += zt;
        tmem_wait_st();
        tc_fence_before();
        bar_arrive(smem_u32(&c.p_full[sub]));
      }
      if (ok) ok = wait_bar(smem_u32(&c.s_full[sub]), n & 1, dead);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
    }
    // ---- the row's result
    if (sub < subs) {
      const bool none = l_run == 0.f || !ok;  // no key seen (a NaN goes through)
      const float inv = none ? 0.f : 1.f / l_run;
      const float zero = z_run * inv;
      const float lse = none ? -INFINITY : (m_run + log2f(l_run)) * kLn2;
      // The row tile's queries are not needed any more: the warp's rows go
      // through their place in shared memory, 256 bytes (16 pieces, swizzled by
      // row) a row and turn, and out in whole lines.
      const uint32_t stage = sbase + L::kQOff + sub * L::kQBytes + (warp & 3) * (L::kQBytes / 4);
      constexpr int kRowPieces = D / 8;  // of bf16; a turn of fp32 partials holds D / 2 columns
      auto out_rows = [&](auto part_c, int c0) {
        constexpr bool kPart = decltype(part_c)::value;
        constexpr int kCols = kPart ? D / 2 : D;
#pragma unroll
        for (int x = 0; x < kCols; x += 32) {
          uint32_t u[32];
          if (n > 0) {  // CTA-uniform
            tmem_ld32(t_o + c0 + x, u);
            tmem_wait_ld();
          }
          float o[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const float v = __uint_as_float(u[(j & ~7) + place_of<KVT>(j & 7)]);
            o[j] = none ? 0.f : fmaf(v, inv, zero);
          }
          constexpr int kEach = kPart ? 4 : 8;  // columns per piece
#pragma unroll
          for (int j = 0; j < 32 / kEach; ++j) {
            const int pc = x / kEach + j;
            const uint32_t to = stage + lane * kRowPieces * 16 + ((pc ^ (lane & (kRowPieces - 1))) << 4);
            if constexpr (kPart)
              sts_u4(to, make_uint4(__float_as_uint(o[4 * j]), __float_as_uint(o[4 * j + 1]),
                                    __float_as_uint(o[4 * j + 2]), __float_as_uint(o[4 * j + 3])));
            else
              sts_u4(to, make_uint4(pack_bf16(o[8 * j], o[8 * j + 1]), pack_bf16(o[8 * j + 2], o[8 * j + 3]),
                                    pack_bf16(o[8 * j + 4], o[8 * j + 5]),
                                    pack_bf16(o[8 * j + 6], o[8 * j + 7])));
          }
        }
        __syncwarp();
#pragma unroll 4
        for (int i = 0; i < kRowPieces; ++i) {
          const int r = i * (32 / kRowPieces) + lane / kRowPieces, pc = lane % kRowPieces;
          const uint4 v = lds128(stage + r * kRowPieces * 16 + ((pc ^ (r & (kRowPieces - 1))) << 4));
          const size_t to = __shfl_sync(0xffffffffu, (unsigned long long)orow, r);
          const bool live = __shfl_sync(0xffffffffu, (int)(row_ok && !(kPart && none)), r) != 0;
          if (live) {
            if constexpr (kPart)
              reinterpret_cast<uint4 *>(a.o_part + (to * a.S + split) * D + c0)[pc] = v;
            else
              reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + to * D)[pc] = v;
          }
        }
        __syncwarp();
      };
      if (a.S > 1) {
        out_rows(std::true_type{}, 0);
        out_rows(std::true_type{}, D / 2);
      } else {
        out_rows(std::false_type{}, 0);
      }
      if (row_ok) {
        if (a.S > 1) a.lse_part[orow * a.S + split] = lse;
        else if (a.lse_out != nullptr) a.lse_out[orow] = lse;
      }
    }
    if (!ok) flag_error(a.d_err, PA_DERR_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    if (*dead && lane == 0) flag_error(a.d_err, PA_DERR_TIMEOUT);
    __syncwarp();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols));
  }
}

// Merge of S partials per (token, query head) row: one warp per row, weights
// exp(lse_s - max); a partial without weight is not read.
template <int D>
__global__ void __launch_bounds__(128) prefill_merge_kernel(const PrefillArgs a) {
  pdl_wait_primary();
  const int lane = threadIdx.x & 31;
  const size_t row = (size_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= (size_t)a.n * a.hq) return;  // (the grid is rounded up to whole CTAs)
  // Rows outside the sequences, clamped as prefill_kernel clamps them, have no
  // partials and are left as they were.
  const float *lse = a.lse_part + row * a.S;
  float M = lane < a.S ? __ldcg(lse + lane) : -INFINITY;  // on its way meanwhile
  const int tok = (int)((uint32_t)row / (uint32_t)a.hq);  // (at most 2^31 rows)
  bool mine = false;
#pragma unroll 1
  for (int b0 = 0; b0 < a.B && !mine; b0 += 32) {
    const int b = min(b0 + lane, a.B - 1);
    const int q0 = __ldg(a.q_begin + b), q1 = __ldg(a.q_begin + b + 1);
    mine = __any_sync(0xffffffffu, tok >= max(q0, 0) && tok < min(q1, a.n));
  }
  if (!mine) return;
  for (int s = lane + 32; s < a.S; s += 32) M = fmaxf(M, __ldcg(lse + s));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  constexpr int E = D / 32;
  float acc[E] = {};
  float den = 0.f;
  for (int s = 0; s < a.S; ++s) {
    // (the maximum drops NaN; a partial that is NaN keeps a NaN weight, so the
    // row is NaN however its keys are split)
    const float l = __ldcg(lse + s);
    const float w = l == -INFINITY ? 0.f : expf(l - M);
    if (w == 0.f) continue;
    den += w;
    const float *o = a.o_part + (row * a.S + s) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(w, __ldcg(o + e), acc[e]);
  }
  const float inv = den == 0.f ? 0.f : 1.f / den;
  uint32_t *out = reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(a.out) + row * D + lane * E);
#pragma unroll
  for (int e = 0; e < E; e += 2) out[e / 2] = pack_bf16(acc[e] * inv, acc[e + 1] * inv);
  if (a.lse_out != nullptr && lane == 0) a.lse_out[row] = den == 0.f ? -INFINITY : M + logf(den);
}

bool encode_pool(CUtensorMap *map, const void *pool, int D, int P, int hkv, int num_pages) {
  const TmapEncodeFn f = tmap_encoder();
  if (f == nullptr) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)P, (cuuint64_t)hkv, (cuuint64_t)num_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)P * D * 2, (cuuint64_t)hkv * P * D * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)P, 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return f(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(pool), dims, strides, box, estr,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Once per device and kernel: shared memory opt-in, and a check that the
// launch brings the registers that the kernel's register split hands out.
template <int D, int KVT, int MODE>
cudaError_t ensure_attr() {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
  if (bit && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  cudaFuncAttributes fa;
  e = cudaFuncGetAttributes(&fa, prefill_kernel<D, KVT, MODE>);
  if (e != cudaSuccess) return e;
  if (fa.numRegs * kThreads<KVT> < kSplitRegs<KVT>) return cudaErrorInvalidConfiguration;
  e = cudaFuncSetAttribute(prefill_kernel<D, KVT, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           Layout<D, KVT>::kBytes);
  if (e == cudaSuccess && bit) done.fetch_or(bit, std::memory_order_acq_rel);
  return e;
}

template <int D, int KVT, int MODE>
cudaError_t launch_mode(const PrefillArgs &a_in, cudaStream_t stream) {
  PrefillArgs a = a_in;
  cudaError_t e = ensure_attr<D, KVT, MODE>();
  if (e != cudaSuccess) return e;
  if (KVT == PA_KV_BF16 && (!encode_pool(&a.tmk, a.k_pool, D, a.P, a.hkv, a.num_pages) ||
                            !encode_pool(&a.tmv, a.v_pool, D, a.P, a.hkv, a.num_pages)))
    return cudaErrorNotSupported;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)prefill_blocks(a.n, a.B, a.hq / a.hkv) * a.hkv * a.S));
  cfg.blockDim = dim3(kThreads<KVT>);
  cfg.dynamicSmemBytes = Layout<D, KVT>::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, prefill_kernel<D, KVT, MODE>, a);
  if (e != cudaSuccess || a.S == 1) return e;
  cfg.gridDim = dim3((unsigned)(((long long)a.n * a.hq + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, prefill_merge_kernel<D>, a);
}

template <int D, int KVT>
cudaError_t launch_t(const PrefillArgs &a_in, cudaStream_t stream) {
  PrefillArgs a = a_in;
  // cap tanh(z), z = cap_z u, as u R(u^2), fitted for the least absolute error
  // of tanh, 1.9e-7, on |z| <= 1/2; u is q.k (bf16 pools) or the score in log2
  // units. Coefficients that fp32 cannot hold, or not to its full precision (a
  // tiny cap or scale, a huge cap), leave the bound at 0: such scores take the
  // other way.
  const double z = KVT == PA_KV_BF16 ? (double)a.scale_log2 * a.inv_cap : (double)a.inv_cap;
  const double c[4] = {1.0, -0.333264608, 0.131858621, -0.044229293};
  double zz = z;
  bool fits = a.cap_l2 > 0.f && z > 0.0 && 0.5 / z < 1e18;  // (the bound is used squared)
  for (int i = 0; i < 4; ++i, zz *= z * z) {
    a.cap_r[i] = (float)(a.cap_l2 * c[i] * zz);
    fits = fits && std::isnormal(a.cap_r[i]);
  }
  a.cap_u = fits ? (float)(0.5 / z) : 0.f;
  if (a.slopes != nullptr)
    return a.cap_l2 > 0.f ? launch_mode<D, KVT, kCapped | kBiased>(a, stream)
                          : launch_mode<D, KVT, kBiased>(a, stream);
  return a.cap_l2 > 0.f ? launch_mode<D, KVT, kCapped>(a, stream)
                        : launch_mode<D, KVT, 0>(a, stream);
}

}  // namespace

// Blocks of 256 rows over all sequences: no more than this, whatever the lengths.
long long prefill_blocks(int n, int B, int G) { return ((long long)n * G) / kCtaRows + B; }

cudaError_t launch_prefill(int D, int kv_dtype, const PrefillArgs &a, cudaStream_t stream) {
#define PA_PF(D_, K_) if (D == D_ && kv_dtype == K_) return launch_t<D_, K_>(a, stream)
  PA_PF(128, PA_KV_BF16); PA_PF(128, PA_KV_U8_PER_TOKEN);
  PA_PF(128, PA_KV_FP8_PER_TOKEN); PA_PF(128, PA_KV_U4_PER_TOKEN);
  PA_PF(64, PA_KV_BF16); PA_PF(64, PA_KV_U8_PER_TOKEN);
  PA_PF(64, PA_KV_FP8_PER_TOKEN); PA_PF(64, PA_KV_U4_PER_TOKEN);
#undef PA_PF
  return cudaErrorInvalidValue;
}

}  // namespace pa
