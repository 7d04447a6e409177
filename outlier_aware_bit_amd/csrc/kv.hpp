// The paged key/value cache shared by qlin_kv_append, qlin_attn_decode and
// qlin_kv_evict: host-side checks and the device helpers more than one of them
// uses.
#pragma once

#include "common.hpp"

namespace qlin {

// A slot's rows of one kv head lie at row index (page id * kv_heads + head) *
// page + line in every array of the pool (k, v, kmeta, vmeta), so one index
// serves all four.
struct KvPool {
  uint8_t* k;
  uint8_t* v;
  uint32_t* kmeta;  // (step, lo) fp16 pairs; null for fp16 rows
  uint32_t* vmeta;
  const int8_t* signs;
  int64_t pages;
  int32_t heads;
  int32_t page_shift;
};

inline int kv_page_shift(int32_t page) {
  int s = 0;
  while ((1 << s) < page) ++s;
  return s;
}

inline KvPool kv_pool(const qlin_kv_cache& c) {
  return KvPool{static_cast<uint8_t*>(c.k), static_cast<uint8_t*>(c.v), reinterpret_cast<uint32_t*>(c.kmeta),
                reinterpret_cast<uint32_t*>(c.vmeta), c.signs, c.pages, c.kv_heads, kv_page_shift(c.page)};
}

// The parts of a cache's description that need no pointers (enough for the
// workspace sizes), then the whole of it with the block table's size.
inline bool kv_shape_ok(const qlin_kv_cache* c) {
  return c != nullptr && (c->bits == 4 || c->bits == 8 || c->bits == 16) &&
         (c->head_dim == 64 || c->head_dim == 128 || c->head_dim == 256) && c->page >= 16 && c->page <= 1024 &&
         (c->page & (c->page - 1)) == 0 && c->kv_heads >= 1 && c->kv_heads <= 65535;
}

#define QLIN_KV_CACHE(c)                                                                                     \
  do {                                                                                                       \
    QLIN_REQUIRE((c) != nullptr, QLIN_ERR_INVALID_ARG, "cache: null pointer");                               \
    QLIN_REQUIRE((c)->bits == 4 || (c)->bits == 8 || (c)->bits == 16, QLIN_ERR_UNSUPPORTED,                  \
                 "bits=%d: 4, 8 and 16 are provided", (c)->bits);                                            \
    QLIN_REQUIRE((c)->head_dim == 64 || (c)->head_dim == 128 || (c)->head_dim == 256, QLIN_ERR_UNSUPPORTED,  \
                 "head_dim=%d: 64, 128 and 256 are provided", (c)->head_dim);                                \
    QLIN_REQUIRE((c)->page >= 16 && (c)->page <= 1024 && ((c)->page & ((c)->page - 1)) == 0,                 \
                 QLIN_ERR_UNSUPPORTED, "page=%d: a power of two from 16 to 1024", (c)->page);                \
    QLIN_REQUIRE((c)->kv_heads >= 1 && (c)->kv_heads <= 65535, QLIN_ERR_SHAPE,                               \
                 "kv_heads=%d must be in [1, 65535]", (c)->kv_heads);                                        \
    QLIN_REQUIRE((c)->pages >= 1 && (c)->pages < ::qlin::kMaxDim &&                                          \
                     (c)->pages * (c)->page <= ::qlin::kMaxElems / (c)->head_dim / (c)->kv_heads,            \
                 QLIN_ERR_SHAPE, "pages=%lld: at least 1, the pool at most 2^40 elements",                   \
                 (long long)(c)->pages);                                                                     \
    QLIN_PTR((c)->k);                                                                                        \
    QLIN_PTR((c)->v);                                                                                        \
    if ((c)->bits == 16) {                                                                                   \
      QLIN_REQUIRE((c)->kmeta == nullptr && (c)->vmeta == nullptr && (c)->signs == nullptr,                  \
                   QLIN_ERR_INVALID_ARG, "kmeta, vmeta and signs must be NULL when bits == 16");             \
    } else {                                                                                                 \
      QLIN_PTR((c)->kmeta);                                                                                  \
      QLIN_PTR((c)->vmeta);                                                                                  \
      QLIN_OPT_PTR((c)->signs);                                                                              \
      QLIN_REQUIRE((c)->signs == nullptr || (c)->head_dim == 128, QLIN_ERR_UNSUPPORTED,                      \
                   "signs: only head_dim 128 has the block-128 Hadamard");                                   \
    }                                                                                                        \
  } while (0)

// B rows of max_pages page ids; the slots of a row stay below 2^31.
#define QLIN_KV_TABLE(c, B, max_pages)                                                                        \
  do {                                                                                                        \
    QLIN_REQUIRE((B) >= 0, QLIN_ERR_INVALID_ARG, "B=%lld is negative", (long long)(B));                       \
    QLIN_REQUIRE((max_pages) >= 1 && (max_pages) <= (::qlin::kMaxDim - 1) / (c)->page, QLIN_ERR_SHAPE,        \
                 "max_pages=%lld: at least 1, and fewer than 2^31 slots", (long long)(max_pages));            \
    QLIN_DIMS(B, max_pages);                                                                                  \
  } while (0)

// mass / pos [B x kv_heads x ld]
#define QLIN_KV_TRACK(c, B, ld)                                                                                \
  QLIN_REQUIRE((ld) >= 1 && (ld) < ::qlin::kMaxDim && (B) < ::qlin::kMaxDim &&                                 \
                   (B) * (ld) <= ::qlin::kMaxElems / (c)->kv_heads,                                            \
               QLIN_ERR_SHAPE, "ld=%lld: at least 1, B * kv_heads * ld at most 2^40", (long long)(ld))

// ---------------------------------------------------------------- device side
// Minimum and maximum that pass a NaN on (fminf and fmaxf drop it).
__device__ __forceinline__ float min_nan(float a, float b) { return __builtin_elementwise_minimum(a, b); }
__device__ __forceinline__ float max_nan(float a, float b) { return __builtin_elementwise_maximum(a, b); }

template <int CTRL>
__device__ __forceinline__ float dpp_f32(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
// The value of the lane whose number differs in bit MASK (1, 2, 4 or 8: within
// a row of 16 lanes).  quad_perm swaps bits 0 and 1; a reversal of each 8 lanes
// (xor 7) after a reversal of each quad (xor 3) is xor 4; a rotation by 8 in a
// row of 16 is xor 8.
template <int MASK>
__device__ __forceinline__ float lane_xor(float v) {
  static_assert(MASK == 1 || MASK == 2 || MASK == 4 || MASK == 8, "");
  if constexpr (MASK == 1) return dpp_f32<0xB1>(v);
  if constexpr (MASK == 2) return dpp_f32<0x4E>(v);
  if constexpr (MASK == 4) return dpp_f32<0x141>(dpp_f32<0x1B>(v));
  return dpp_f32<0x128>(v);
}

// Inclusive sum over the lanes of a wave.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // one lane up, in rows of 16
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // lane 15 to rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // lane 31 to rows 2 and 3
  return v;
}

// u += s * (u, or v, of the lane that CTRL names) for eight values: s is +-1, so
// the product is exact and the sum rounded once.  (A DPP operand may be read
// two wait states after it was written.)
#define QLIN_FMAC_DPP8(u, s, CTRL)                                                                  \
  asm("s_nop 1\n\t"                                                                                 \
      "v_fmac_f32_dpp %0, %0, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                           \
      "v_fmac_f32_dpp %1, %1, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                           \
      "v_fmac_f32_dpp %2, %2, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                           \
      "v_fmac_f32_dpp %3, %3, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                           \
      "v_fmac_f32_dpp %4, %4, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                           \
      "v_fmac_f32_dpp %5, %5, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                           \
      "v_fmac_f32_dpp %6, %6, %8 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                           \
      "v_fmac_f32_dpp %7, %7, %8 " CTRL " row_mask:0xf bank_mask:0xf"                               \
      : "+v"(u[0]), "+v"(u[1]), "+v"(u[2]), "+v"(u[3]), "+v"(u[4]), "+v"(u[5]), "+v"(u[6]), "+v"(u[7])\
      : "v"(s))
#define QLIN_FMAC_DPP8_OF(u, v, s, CTRL)                                                            \
  asm("s_nop 1\n\t"                                                                                 \
      "v_fmac_f32_dpp %0, %8, %16 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                          \
      "v_fmac_f32_dpp %1, %9, %16 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                          \
      "v_fmac_f32_dpp %2, %10, %16 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                         \
      "v_fmac_f32_dpp %3, %11, %16 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                         \
      "v_fmac_f32_dpp %4, %12, %16 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                         \
      "v_fmac_f32_dpp %5, %13, %16 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                         \
      "v_fmac_f32_dpp %6, %14, %16 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                         \
      "v_fmac_f32_dpp %7, %15, %16 " CTRL " row_mask:0xf bank_mask:0xf"                             \
      : "+&v"(u[0]), "+&v"(u[1]), "+&v"(u[2]), "+&v"(u[3]), "+&v"(u[4]), "+&v"(u[5]), "+&v"(u[6]),  \
        "+&v"(u[7])                                                                                 \
      : "v"(v[0]), "v"(v[1]), "v"(v[2]), "v"(v[3]), "v"(v[4]), "v"(v[5]), "v"(v[6]), "v"(v[7]), "v"(s))

// t = (x * d) H_128 for 128 values held by 16 neighbouring lanes, 8 each
// (lane c of the 16 holds 8c .. 8c + 7): a butterfly of spans 1, 2, .., 64 in
// fp32, every sum and difference rounded once.  Across lanes the lower one of a
// pair takes u + other and the upper one u - other, the negative of what is
// due, which goes on through the later spans and is put right at the end.
__device__ __forceinline__ void hadamard128(float (&u)[8], int c) {
#pragma unroll
  for (int h = 1; h < 8; h <<= 1) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if ((e & h) == 0) {
        const float a = u[e], b = u[e + h];
        u[e] = add_rn(a, b);
        u[e + h] = sub_rn(a, b);
      }
    }
  }
  const float s1 = (c & 1) ? -1.0f : 1.0f, s2 = (c & 2) ? -1.0f : 1.0f;
  const float s4 = (c & 4) ? -1.0f : 1.0f, s8 = (c & 8) ? -1.0f : 1.0f;
  QLIN_FMAC_DPP8(u, s1, "quad_perm:[1,0,3,2]");
  QLIN_FMAC_DPP8(u, s2, "quad_perm:[2,3,0,1]");
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = dpp_f32<0x1B>(u[e]);  // each quad reversed, then each eight lanes
  QLIN_FMAC_DPP8_OF(u, v, s4, "row_half_mirror");
  QLIN_FMAC_DPP8(u, s8, "row_ror:8");
  const float sign = (s1 * s2) * (s4 * s8);
#pragma unroll
  for (int e = 0; e < 8; ++e) u[e] = __builtin_fmaf(u[e], sign, 0.0f);
}

// Eight fp16 values times the signs (a negative entry: -1), as fp32: the sign
// bits (bit 7 of each byte) are moved to the fp16 pairs and flipped in.
__device__ __forceinline__ void signed8(const v4i raw, const uint2 s, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t mask = __builtin_amdgcn_perm(0u, i < 2 ? s.x : s.y, (i & 1) ? 0x030c020cu : 0x010c000cu) & 0x80008000u;
    const uint32_t w = static_cast<uint32_t>(raw[i]) ^ mask;
    f[2 * i] = h2f(static_cast<uint16_t>(w));
    f[2 * i + 1] = h2f(static_cast<uint16_t>(w >> 16));
  }
}

}  // namespace qlin
