// Cache write with the rotary position embedding applied on the way.
//
// A pair (a, b) of a head's elements is turned by the angle of its token's
// position: a' = a c - b s, b' = b c + a s, with c and s read from the
// caller's table (row p: the cosines, then the sines, of position p). Each
// product and each sum is one IEEE fp32 rounding (no contraction) and the
// result is rounded to bf16 once, so that the stored bits are those of
// rotating the rows first and calling pa_kv_append on them; quantised pools
// then quantise the bf16 row by the formulas of pa_quant.cuh.
//
// Bound by bytes: every q, k and v row is read and written once. A thread
// holds 16 elements of a row: eight pairs, two 16-byte chunks; with the pairs
// half a row apart these are chunks u and u + r / 16, so no element leaves
// its thread. D / 16 lanes make a row and a warp takes kRows rows per lane
// group, all loads issued before the first use. Queries, keys and values of a
// token are one list of rows, cut into items of one warp: the cosines, sines
// and the page slot are looked up once per item.
#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_quant.cuh"

namespace pa {
namespace {

constexpr int kWarps = 4;       // items per CTA at a time
constexpr int kMaxAxes = 4;

__device__ __forceinline__ uint4 ldg128(const void *p) {
  // not the read-only path: q may be rotated in place
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

__device__ __forceinline__ void unpack(const uint4 &v, float *x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(w[i]);
    x[2 * i + 1] = bf16_hi(w[i]);
  }
}

__device__ __forceinline__ uint4 pack8(const float *x) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                    pack_bf16(x[6], x[7]));
}

// (Quantised pools: six CTAs per SM, 80 registers, 70.6 -> 67.7 us for 8,000
// image tokens of 64/8 heads into an FP8 cache; bf16 pools lose by it.)
template <int D, int KVT, bool IL, int kRows>  // kRows: rows per lane group and item
__global__ void __launch_bounds__(kWarps * 32, KVT == PA_KV_BF16 ? 0 : 6) append_rope_kernel(const AppendRopeArgs a) {
  pdl_launch_dependents();
  pdl_wait_primary();
  constexpr int kLanes = D / 16;         // lanes of one row
  constexpr int kGroups = 32 / kLanes;   // rows a warp holds at a time
  constexpr int kItemRows = kGroups * kRows;
  const int lane = threadIdx.x & 31;
  const int u = lane % kLanes;
  const int grp = lane / kLanes;
  const int half = a.rot / 2;
  // this thread's pairs 8u .. 8u + 7 and the chunks that hold them
  const bool turn = 16 * u < a.rot;
  const int c0 = IL ? 2 * u : (turn ? u : 2 * u);
  const int c1 = IL ? 2 * u + 1 : (turn ? u + a.rot / 16 : 2 * u + 1);
  const int rows = a.hq + 2 * a.hkv;
  const int per_token = (rows + kItemRows - 1) / kItemRows;
  const long long items = (long long)a.n * per_token;
  for (long long it = blockIdx.x * (long long)kWarps + (threadIdx.x >> 5); it < items;
       it += (long long)gridDim.x * kWarps) {
    const int i = (int)(it / per_token);
    const int r0 = (int)(it % per_token) * kItemRows + grp;
    // ---- all row loads first
    uint4 v[kRows][2];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int r = r0 + k * kGroups;
      if (r < rows) {
        const unsigned char *src =
            r < a.hq ? a.q + ((size_t)i * a.q_stride + (size_t)r * D) * 2
            : r < a.hq + a.hkv
                ? a.k_new + ((size_t)i * a.k_stride + (size_t)(r - a.hq) * D) * 2
                : a.v_new + ((size_t)i * a.v_stride + (size_t)(r - a.hq - a.hkv) * D) * 2;
        v[k][0] = ldg128(src + c0 * 16);
        v[k][1] = ldg128(src + c1 * 16);
      } else {
        v[k][0] = v[k][1] = make_uint4(0, 0, 0, 0);
      }
    }
    // ---- the token's angles
    int p[kMaxAxes];
    bool pos_ok = true;
#pragma unroll
    for (int x = 0; x < kMaxAxes; ++x) {
      p[x] = 0;
      if (x < a.num_axes) {
        p[x] = __ldg(a.rope_pos + (size_t)(a.rope_pos_axes > 1 ? x : 0) * a.n + i);
        if (p[x] < 0 || p[x] >= a.table_len) {
          pos_ok = false;
          p[x] = 0;
        }
      }
    }
    float c[8], s[8];
    if (turn) {
      bool same = true;  // the thread's eight pairs follow one axis
#pragma unroll
      for (int e = 1; e < 8; ++e) same &= a.axis_of_pair[8 * u + e] == a.axis_of_pair[8 * u];
      auto row = [&](int e) {
        const int x = a.axis_of_pair[8 * u + e];
        const int px = x == 0 ? p[0] : x == 1 ? p[1] : x == 2 ? p[2] : p[3];
        return a.table + (size_t)px * a.rot + 8 * u;
      };
      if (same) {
        const float *t = row(0);
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          const float4 cv = __ldg(reinterpret_cast<const float4 *>(t + e));
          const float4 sv = __ldg(reinterpret_cast<const float4 *>(t + half + e));
          c[e] = cv.x; c[e + 1] = cv.y; c[e + 2] = cv.z; c[e + 3] = cv.w;
          s[e] = sv.x; s[e + 1] = sv.y; s[e + 2] = sv.z; s[e + 3] = sv.w;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float *t = row(e);
          c[e] = __ldg(t + e);
          s[e] = __ldg(t + half + e);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        c[e] = 1.f;
        s[e] = 0.f;
      }
    }
    // ---- the token's page slot: row (page * Hkv + h) * P + slot of the pool
    long long slot0 = -1;  // the row of KV head 0
    int bits = pos_ok ? 0 : PA_DERR_BAD_POS;
    if (r0 - grp + kItemRows > a.hq) {  // warp-uniform: the item holds key or value rows
      const int seq = __ldg(a.seq_idx + i);
      const int ps = __ldg(a.pos + i);
      if (seq < 0 || seq >= a.num_seqs) {
        bits |= PA_DERR_BAD_SEQ;
      } else if (ps < 0 || ps / a.P >= a.max_pages) {
        bits |= PA_DERR_BAD_POS;
      } else {
        const int page = __ldg(a.block_tables + (size_t)seq * a.max_pages + ps / a.P);
        if (page < 0 || page >= a.num_pages)
          bits |= PA_DERR_BAD_PAGE;
        else
          slot0 = (long long)page * a.hkv * a.P + ps % a.P;
      }
    }
    if (bits != 0 && lane == 0) flag_error(a.d_err, bits);
    if (!pos_ok) continue;  // warp-uniform: nothing of this token is written

#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int r = r0 + k * kGroups;
      const bool rotates = r < a.hq + a.hkv;
      if (rotates && turn) {
        float x[16];
        unpack(v[k][0], x);
        unpack(v[k][1], x + 8);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int ia = IL ? 2 * e : e, ib = IL ? 2 * e + 1 : e + 8;
          const float xa = x[ia], xb = x[ib];
          x[ia] = __fsub_rn(__fmul_rn(xa, c[e]), __fmul_rn(xb, s[e]));
          x[ib] = __fadd_rn(__fmul_rn(xb, c[e]), __fmul_rn(xa, s[e]));
        }
        v[k][0] = pack8(x);
        v[k][1] = pack8(x + 8);
      }
      if (r < a.hq) {
        unsigned char *dst = a.q_out + ((size_t)i * a.hq + r) * D * 2;
        *reinterpret_cast<uint4 *>(dst + c0 * 16) = v[k][0];
        *reinterpret_cast<uint4 *>(dst + c1 * 16) = v[k][1];
      }
      if constexpr (KVT == PA_KV_BF16) {
        if (r >= a.hq && r < rows && slot0 >= 0) {
          const int h = rotates ? r - a.hq : r - a.hq - a.hkv;
          unsigned char *dst = (rotates ? a.k_pool : a.v_pool) + (size_t)(slot0 + (long long)h * a.P) * D * 2;
          *reinterpret_cast<uint4 *>(dst + c0 * 16) = v[k][0];
          *reinterpret_cast<uint4 *>(dst + c1 * 16) = v[k][1];
        }
      } else {
        // warp-uniform: some row of this step goes to the cache
        if (r - grp + kGroups > a.hq && r - grp < rows) {
          const bool live = r >= a.hq && r < rows && slot0 >= 0;
          const int h = rotates ? r - a.hq : r - a.hq - a.hkv;
          const size_t row = live ? (size_t)(slot0 + (long long)h * a.P) : 0;
          float x[16];
          unpack(v[k][0], x);
          unpack(v[k][1], x + 8);
          uint32_t codes[2][2];
          const float2 sz = quantise_lanes<KVT, kLanes>(x, codes);
          if (live) {
            unsigned char *dst = rotates ? a.k_pool : a.v_pool;
            if constexpr (KVT == PA_KV_U4_PER_TOKEN) {
              dst += row * (D / 2);
              *reinterpret_cast<uint32_t *>(dst + c0 * 4) = codes[0][0];
              *reinterpret_cast<uint32_t *>(dst + c1 * 4) = codes[1][0];
            } else {
              dst += row * D;
              *reinterpret_cast<uint2 *>(dst + c0 * 8) = make_uint2(codes[0][0], codes[0][1]);
              *reinterpret_cast<uint2 *>(dst + c1 * 8) = make_uint2(codes[1][0], codes[1][1]);
            }
            if (u == 0)
              *reinterpret_cast<float2 *>((rotates ? a.k_sz : a.v_sz) + row * 2) = sz;
          }
        }
      }
    }
  }
}

template <int D, int KVT, int kRows>
cudaError_t launch_rows(const AppendRopeArgs &a, bool interleaved, cudaStream_t stream) {
  const int item_rows = 32 / (D / 16) * kRows;
  const long long items =
      (long long)a.n * ((a.hq + 2 * a.hkv + item_rows - 1) / item_rows);
  const long long want = (items + kWarps - 1) / kWarps;
  // a few items per warp even out the costly key and value rows (8,000 tokens,
  // FP8: 16 CTAs per SM 69.0 us, 32 70.6, one item per warp 75.6; at 5 per SM
  // the same warps get those rows every time, 96.8)
  const long long most = 16LL * device_sm_count();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(want < most ? want : most));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return interleaved ? cudaLaunchKernelEx(&cfg, append_rope_kernel<D, KVT, true, kRows>, a)
                     : cudaLaunchKernelEx(&cfg, append_rope_kernel<D, KVT, false, kRows>, a);
}

// Items of two rows per lane group where four would leave lanes without a row
// (16 rows of 64 elements a token: 14.1 -> 12.2 us for 10,982 tokens) or
// warps without an item (a step of eight tokens: 2.96 -> 2.57 us); else four,
// which look the angles and slots up half as often (8192 tokens of 48 rows of
// 128: 34.1 us, with two 38).
template <int D, int KVT>
cudaError_t launch_t(const AppendRopeArgs &a, bool interleaved, cudaStream_t stream) {
  const int rows = a.hq + 2 * a.hkv, two = 32 / (D / 16) * 2;
  const int items2 = (rows + two - 1) / two, items4 = (rows + 2 * two - 1) / (2 * two);
  const bool few = (long long)a.n * items4 < 4LL * device_sm_count();
  return items2 < 2 * items4 || few ? launch_rows<D, KVT, 2>(a, interleaved, stream)
                                    : launch_rows<D, KVT, 4>(a, interleaved, stream);
}

}  // namespace

cudaError_t launch_append_rope(int D, int kv_dtype, const AppendRopeArgs &a, bool interleaved,
                               cudaStream_t stream) {
#define PA_AR(D_, K_) \
  if (D == D_ && kv_dtype == K_) return launch_t<D_, K_>(a, interleaved, stream)
  PA_AR(128, PA_KV_BF16); PA_AR(128, PA_KV_U8_PER_TOKEN);
  PA_AR(128, PA_KV_FP8_PER_TOKEN); PA_AR(128, PA_KV_U4_PER_TOKEN);
  PA_AR(64, PA_KV_BF16); PA_AR(64, PA_KV_U8_PER_TOKEN);
  PA_AR(64, PA_KV_FP8_PER_TOKEN); PA_AR(64, PA_KV_U4_PER_TOKEN);
#undef PA_AR
  return cudaErrorInvalidValue;
}

}  // namespace pa
