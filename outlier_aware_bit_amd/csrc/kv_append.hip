// Appending rows to the paged key/value cache (qlin_kv_append).
//
// Per row and kv head: K after the Hadamard (t = (k d) H, a butterfly in
// registers, 8 values a lane and four exchanges between 16 lanes), then for K
// and V the row's minimum and maximum, its (step, lo) and codes, all in
// registers; a row is read once and written once.
//
// One token per sequence is a launch: 2.6 us for one, 3.4 for 48 sequences.  For
// prompts vector instructions are what is short: 18,381 tokens of 8 heads of 128
// channels, int4 with the Hadamard, 97 MB, 24.4 us (4.0 TB/s; vector
// instructions 66 % of the time, 165 of them per eight values); 18,786 of 4 heads
// of 256 channels, int8, 116 MB, 23.1 us (5.0 TB/s, where a copy reaches 5.2).
#include <type_traits>

#include "kv.hpp"

namespace qlin {
namespace {

struct AppendArgs {
  KvPool c;
  const uint16_t* k;
  const uint16_t* v;
  int64_t ld_k, ld_v;  // elements between two tokens
  int64_t T;
  const int32_t* row;  // null: token t belongs to row t
  const int32_t* slot;
  const int32_t* table;
  int64_t B, max_pages;
  const int32_t* position;  // with mass and pos, or all null
  float* mass;
  int32_t* pos;
  int64_t ld;
};

constexpr int kAppendThreads = 256;

// 1 / s of a positive fp16 value, correctly rounded: one Newton step on the
// approximate reciprocal gives the quotient for each of them (all 31743 were
// compared).  An infinite s gives a NaN where 1 / s is 0: codes of such a row
// stand for nothing.
__device__ __forceinline__ float inverse(float s) {
  const float r = __builtin_amdgcn_rcpf(s);
  return __builtin_fmaf(__builtin_fmaf(-s, r, 1.0f), r, r);
}

// One row as stored: fp16 as it is; else, in fp32 with one rounding per
// operation, lo = fp16(min t), step = fp16((max t - lo) * (1 / qmax)),
// code = clamp(rint((t - lo) * (1 / step)), 0, qmax).  LANES neighbouring lanes
// hold the row, 8 values each.  A NaN makes lo a NaN, an infinity makes step or
// lo one, so a row that was not finite does not read back as if it were.
template <int BITS, int LANES, bool ROT>
__device__ __forceinline__ void store_row(const v4i raw, int c, uint8_t* dst, uint32_t* meta, const int8_t* signs) {
  if constexpr (BITS == 16) {
    reinterpret_cast<v4i*>(dst)[c] = raw;
  } else {
    float t[8];
    if constexpr (ROT) {
      signed8(raw, *reinterpret_cast<const uint2*>(signs + 8 * c), t);
      hadamard128(t, c);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        t[i] = h2f(static_cast<uint16_t>(static_cast<uint32_t>(raw[i >> 1]) >> (16 * (i & 1))));
    }
    float mn = t[0], mx = t[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      mn = min_nan(mn, t[i]);
      mx = max_nan(mx, t[i]);
    }
    mn = min_nan(mn, lane_xor<1>(mn));
    mx = max_nan(mx, lane_xor<1>(mx));
    mn = min_nan(mn, lane_xor<2>(mn));
    mx = max_nan(mx, lane_xor<2>(mx));
    mn = min_nan(mn, dpp_f32<0x141>(mn));  // eight lanes reversed: the quads are uniform
    mx = max_nan(mx, dpp_f32<0x141>(mx));
    if constexpr (LANES >= 16) {
      mn = min_nan(mn, lane_xor<8>(mn));
      mx = max_nan(mx, lane_xor<8>(mx));
    }
    if constexpr (LANES == 32) {
      mn = min_nan(mn, __shfl_xor(mn, 16, 64));
      mx = max_nan(mx, __shfl_xor(mx, 16, 64));
    }
    constexpr float qmax = (BITS == 4) ? 15.0f : 255.0f;
    const uint16_t lo16 = f2h(mn);
    const float lo = h2f(lo16);
    const uint16_t step16 = f2h_mul(sub_rn(mx, lo), 1.0f / qmax);
    const float step = h2f(step16);
    const float inv = (step == 0.0f) ? 0.0f : inverse(step);
    // A code per byte.  The conversion to a byte rounds to the nearest integer,
    // ties to even, and saturates (all 2^32 arguments were compared with rint
    // and a clamp to [0, 255]).
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float code = mul_rn(sub_rn(t[i], lo), inv);
      if constexpr (BITS == 4) code = __builtin_amdgcn_fmed3f(code, 0.0f, qmax);
      w[i >> 2] = __builtin_amdgcn_cvt_pk_u8_f32(code, i & 3, w[i >> 2]);
    }
    if constexpr (BITS == 8) {
      reinterpret_cast<uint2*>(dst)[c] = make_uint2(w[0], w[1]);
    } else {
      // Bytes 0 and 2 of w | w >> 4 hold two codes each.
      w[0] |= w[0] >> 4;
      w[1] |= w[1] >> 4;
      reinterpret_cast<uint32_t*>(dst)[c] = __builtin_amdgcn_perm(w[1], w[0], 0x06040200u);
    }
    if (c == 0) *meta = static_cast<uint32_t>(step16) | static_cast<uint32_t>(lo16) << 16;
  }
}

// A workgroup takes 2048 / D consecutive tokens of one kv head, D / 8 lanes per
// row, and stores each token's K and V row: the rows, their (step, lo)
// pairs and the mass / pos entries of neighbouring tokens of a prompt lie side
// by side in a page, so a workgroup's stores fill whole lines.
template <int BITS, int D, bool ROT>
__global__ __launch_bounds__(kAppendThreads) void kv_append_kernel(AppendArgs a) {
  constexpr int LANES = D / 8;
  constexpr int RB = D * BITS / 8;  // bytes of a stored row
  const int c = threadIdx.x % LANES;
  constexpr int TOKENS = kAppendThreads / LANES;
  const uint32_t h = blockIdx.x, heads = a.c.heads;
  const int ps = a.c.page_shift;
  const int64_t step = static_cast<int64_t>(gridDim.y) * TOKENS;
  int64_t t = static_cast<int64_t>(blockIdx.y) * TOKENS + threadIdx.x / LANES;
  for (int64_t lot = static_cast<int64_t>(blockIdx.y) * TOKENS; lot < a.T; lot += step, t += step) {  // uniform
    const int64_t tt = t < a.T ? t : a.T - 1;  // every lane takes part in the exchanges
    const v4i k = *reinterpret_cast<const v4i*>(a.k + tt * a.ld_k + h * D + 8 * c);
    const v4i v = *reinterpret_cast<const v4i*>(a.v + tt * a.ld_v + h * D + 8 * c);
    const int32_t slot = a.slot[tt];
    const int64_t b = a.row != nullptr ? a.row[tt] : tt;
    bool ok = t < a.T && b >= 0 && b < a.B && slot >= 0 && (slot >> ps) < a.max_pages;
    const uint32_t entry = ok ? slot >> ps : 0;
    const uint32_t id = a.table[static_cast<uint64_t>(static_cast<uint32_t>(ok ? b : 0)) *
                                static_cast<uint32_t>(a.max_pages) + entry];
    ok = ok && id < static_cast<uint32_t>(a.c.pages);
    if (!ok) continue;  // uniform over a row's lanes
    const uint64_t at = ((static_cast<uint64_t>(id) * heads + h) << ps) + (slot & ((1 << ps) - 1));
    store_row<BITS, LANES, ROT>(k, c, a.c.k + at * RB, a.c.kmeta + at, a.c.signs);
    store_row<BITS, LANES, false>(v, c, a.c.v + at * RB, a.c.vmeta + at, nullptr);
    if (a.mass != nullptr && c == 0 && slot < a.ld) {
      const uint64_t i = static_cast<uint64_t>(static_cast<uint32_t>(b) * heads + h) * static_cast<uint32_t>(a.ld) + slot;
      a.mass[i] = 0.0f;
      a.pos[i] = a.position[tt];
    }
  }
}

template <int BITS, int D, bool ROT>
void launch(const AppendArgs& a, hipStream_t st) {
  constexpr int tokens = kAppendThreads / (D / 8);
  const int64_t lots = (a.T + tokens - 1) / tokens;
  // Neighbouring workgroups take the heads of the same tokens, which lie side by
  // side.  One lot each: 2,048 workgroups that go over the lots, the next one's
  // rows loaded ahead, took 28 - 30 us where this takes 25.
  const dim3 grid(static_cast<unsigned>(a.c.heads), static_cast<unsigned>(lots < 65535 ? lots : 65535));
  kv_append_kernel<BITS, D, ROT><<<grid, kAppendThreads, 0, st>>>(a);
}

template <int BITS>
void launch_d(const AppendArgs& a, int D, hipStream_t st) {
  if (D == 64) {
    launch<BITS, 64, false>(a, st);
  } else if (D == 256) {
    launch<BITS, 256, false>(a, st);
  } else {
    if constexpr (BITS < 16) {
      if (a.c.signs != nullptr) return launch<BITS, 128, true>(a, st);
    }
    launch<BITS, 128, false>(a, st);
  }
}

}  // namespace
}  // namespace qlin

using namespace qlin;

extern "C" qlin_status qlin_kv_append(const qlin_kv_cache* cache, const uint16_t* k, int64_t ld_k, const uint16_t* v,
                                      int64_t ld_v, int64_t T, const int32_t* row, const int32_t* slot,
                                      const int32_t* table, int64_t B, int64_t max_pages, const int32_t* position,
                                      float* mass, int32_t* pos, int64_t ld, void* stream) {
  QLIN_KV_CACHE(cache);
  QLIN_KV_TABLE(cache, B, max_pages);
  QLIN_REQUIRE(T >= 0, QLIN_ERR_INVALID_ARG, "T=%lld is negative", (long long)T);
  const int64_t width = static_cast<int64_t>(cache->kv_heads) * cache->head_dim;
  QLIN_REQUIRE(ld_k >= width && ld_k % 8 == 0, QLIN_ERR_SHAPE,
               "ld_k=%lld must be a multiple of 8, at least kv_heads * head_dim", (long long)ld_k);
  QLIN_REQUIRE(ld_v >= width && ld_v % 8 == 0, QLIN_ERR_SHAPE,
               "ld_v=%lld must be a multiple of 8, at least kv_heads * head_dim", (long long)ld_v);
  QLIN_DIMS(T, ld_k);
  QLIN_DIMS(T, ld_v);
  QLIN_REQUIRE(row != nullptr || T <= B, QLIN_ERR_SHAPE, "T=%lld tokens without rows: at most B=%lld", (long long)T,
               (long long)B);
  const bool track = mass != nullptr;
  QLIN_REQUIRE((pos != nullptr) == track && (position != nullptr) == track, QLIN_ERR_INVALID_ARG,
               "mass, pos and position come together or not at all");
  if (track) {
    QLIN_KV_TRACK(cache, B, ld);
    QLIN_REQUIRE(B < kMaxDim / cache->kv_heads, QLIN_ERR_SHAPE, "B * kv_heads: fewer than 2^31");
  }
  if (T == 0 || B == 0) return QLIN_OK;
  QLIN_PTR(k);
  QLIN_PTR(v);
  QLIN_OPT_PTR(row);
  QLIN_PTR(slot);
  QLIN_PTR(table);
  if (track) {
    QLIN_PTR(position);
    QLIN_PTR(mass);
    QLIN_PTR(pos);
  }
  const AppendArgs a{kv_pool(*cache), k, v, ld_k, ld_v, T, row, slot, table, B, max_pages, position, mass, pos, ld};
  hipStream_t st = as_stream(stream);
  if (cache->bits == 16)
    launch_d<16>(a, cache->head_dim, st);
  else if (cache->bits == 8)
    launch_d<8>(a, cache->head_dim, st);
  else
    launch_d<4>(a, cache->head_dim, st);
  QLIN_LAUNCH_CHECK("kv_append_kernel");
  return QLIN_OK;
}
