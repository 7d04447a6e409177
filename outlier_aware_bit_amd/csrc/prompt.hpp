// Attention over whole prompts, shared by qlin_attn_prompt and its backward pass:
// the packed sequences' borders, tiles of rows in LDS, host-side checks.
#pragma once

#include "common.hpp"

namespace qlin {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

struct Borders {
  const int32_t* cu_q;
  const int32_t* cu_k;
  int64_t B;
  int32_t Tq, Tk;
};

// Queries [q0, q1) and keys [k0, k1) of a sequence; a border outside the arrays
// is taken to their ends.
struct Seq {
  int32_t q0, q1, k0, k1;
};

__device__ __forceinline__ int32_t clamp_i32(int32_t v, int32_t lo, int32_t hi) {
  return v < lo ? lo : v > hi ? hi : v;
}

// The sequence of the slot-th tile of ROWS rows, and which of its tiles that is.
// Sequence b's tiles have the slots from cu[b] / ROWS + b on, which leaves room
// for each (and a few slots without a tile): ceil(n / ROWS) <=
// floor((cu + n) / ROWS) - floor(cu / ROWS) + 1.  A search with 64 probes at a
// time, the same in every wave.
template <int ROWS>
__device__ __forceinline__ int64_t find_tile(const int32_t* cu, int64_t B, int64_t slot, int64_t& tile) {
  int64_t lo = 0, n = B;  // the last b in [lo, lo + n) whose slots begin at or before `slot`
  const int lane = threadIdx.x & 63;
  while (true) {
    const int64_t step = (n + 63) / 64;
    const int64_t b = lo + lane * step;
    const bool at = b < lo + n && cu[b] / ROWS + b <= slot;
    const int hits = __builtin_popcountll(__ballot(at));
    const int64_t from = lo + (hits > 0 ? hits - 1 : 0) * step;
    n = lo + n - from < step ? lo + n - from : step;
    lo = from;
    if (step == 1) break;
  }
  const int32_t b = __builtin_amdgcn_readfirstlane(static_cast<int32_t>(lo));  // B < 2^31
  tile = slot - (cu[b] / ROWS + b);
  return b;
}

__device__ __forceinline__ Seq sequence(const Borders& s, int64_t b) {
  Seq r;
  r.q0 = clamp_i32(s.cu_q[b], 0, s.Tq);
  r.q1 = clamp_i32(s.cu_q[b + 1], r.q0, s.Tq);
  r.k0 = clamp_i32(s.cu_k[b], 0, s.Tk);
  r.k1 = clamp_i32(s.cu_k[b + 1], r.k0, s.Tk);
  return r;
}

// Workgroups are handed to the 8 XCDs in turn.  Heads that are a multiple of 8
// are dealt out so that an XCD works on neighbouring ones, which share kv heads
// and so its L2's lines.
__device__ __forceinline__ void head_and_slot(uint32_t id, uint32_t heads, uint32_t& head, uint32_t& slot) {
  slot = id / heads;
  const uint32_t h = id - slot * heads;
  head = (heads & 7) == 0 ? (h & 7) * (heads >> 3) + (h >> 3) : h;
}

// Rows of D fp16 values lie in LDS as 16-byte chunks, chunk c of a row at c ^
// swizzle(row): 16 neighbouring rows then have their chunk c in 16 different
// places of the 256 bytes that the banks span, and so do four neighbouring
// rows' runs of four chunks.
template <int D>
__device__ __forceinline__ int swizzle(int row) {
  if constexpr (D == 64) {
    const int r = row >> 1;
    return ((r & 1) << 2) | ((r >> 1) & 3);
  } else {
    return ((row & 3) << 2) | ((row >> 2) & 3);
  }
}
template <int D>
__device__ __forceinline__ int lds_at(int row, int chunk) {  // in bytes
  return row * (2 * D) + ((chunk ^ swizzle<D>(row)) << 4);
}

typedef __attribute__((address_space(3))) void* lds_ptr;
typedef _Float16 v4h __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef float v2f __attribute__((ext_vector_type(2)));

// BYTES per lane from `base` + off, lane after lane into LDS from `lds` on, without
// registers in between; what lies past `bytes` arrives as zeros.  (The buffer's
// type is one that only the device's compiler knows.)
template <int BYTES>
__device__ __forceinline__ void load_to_lds(const void* base, int32_t bytes, uint32_t off, void* lds) {
#ifdef __HIP_DEVICE_COMPILE__
  const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, bytes, 0x00027000);
  static_assert(BYTES == 4 || BYTES == 16, "");
  if constexpr (BYTES == 16)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)lds, 16, off, 0, 0, 0);
  else
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)lds, 4, off, 0, 0, 0);
#endif
}

// Loads ROWS rows of D values, `ld` elements apart, into LDS; rows from `rows` on become zeros.  The lanes' source offsets do not
// depend on the tile.  WAVES waves share the rows.
template <int D, int ROWS, int WAVES>
struct TileLoad {
  static constexpr int kEach = ROWS * D * 2 / 1024 / WAVES;  // instructions of a wave, 1024 bytes each
  static_assert(kEach * WAVES * 1024 == ROWS * D * 2, "");
  uint32_t off[kEach];

  __device__ __forceinline__ void init(int64_t ld, int wave, int lane) {
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int at = (wave * kEach + i) * 64 + lane;  // chunk in LDS
      const int row = at / (D / 8), pos = at % (D / 8);
      off[i] = static_cast<uint32_t>(row) * static_cast<uint32_t>(2 * ld) + ((pos ^ swizzle<D>(row)) << 4);
    }
  }
  __device__ __forceinline__ void load(const uint16_t* base, int64_t ld, int rows, uint8_t* lds, int wave) const {
    const int32_t n = rows <= 0 ? 0 : static_cast<int32_t>((rows < ROWS ? rows - 1 : ROWS - 1) * (2 * ld) + 2 * D);
#pragma unroll
    for (int i = 0; i < kEach; ++i) load_to_lds<16>(base, n, off[i], lds + (wave * kEach + i) * 1024);
  }
};
// 64 fp32 values, those from `n` on as zeros.
__device__ __forceinline__ void load64(const float* src, int n, float* lds, int lane) {
  load_to_lds<4>(src, 4 * (n < 64 ? n : 64), 4 * lane, lds);
}
// Tokens at most this many elements apart: a tile's offsets stay in 31 bits.
constexpr int64_t kMaxPromptLd = int64_t(1) << 22;

// Waits for this wave's loads into LDS and its reads of it, then for every wave.
__device__ __forceinline__ void tile_barrier() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Four rows by 16 columns of LDS, transposed: each 16 lanes read the rows' four
// runs of four, and lane i of them gets column i of the four rows.
__device__ __forceinline__ v4h lds_transposed(const uint8_t* p) {
  return __builtin_bit_cast(v4h, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)p));
}
__device__ __forceinline__ v8h join_halves(v4h a, v4h b) {
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}
// Two fp32 to fp16, to the nearest even.
__device__ __forceinline__ uint32_t pack_half(float a, float b) {
  const v2f f = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, v2h));
}
__device__ __forceinline__ v8h pack8(float a, float b, float c, float d, float e, float f, float g, float h) {
  const v4i w = {static_cast<int>(pack_half(a, b)), static_cast<int>(pack_half(c, d)),
                 static_cast<int>(pack_half(e, f)), static_cast<int>(pack_half(g, h))};
  return __builtin_bit_cast(v8h, w);
}

#define QLIN_PROMPT_ROWS(name, T, ld, n, head_dim)                                                          \
  do {                                                                                                      \
    QLIN_REQUIRE((ld) >= static_cast<int64_t>(n) * (head_dim) && (ld) % 8 == 0, QLIN_ERR_SHAPE,             \
                 "%s=%lld must be a multiple of 8, at least a token's row", name, (long long)(ld));         \
    QLIN_REQUIRE((ld) <= ::qlin::kMaxPromptLd, QLIN_ERR_SHAPE, "%s=%lld: at most 2^22", name, (long long)(ld)); \
    QLIN_DIMS(T, ld);                                                                                       \
  } while (0)

// At most 2^30 tokens, so that positions, tiles and windows add up within 32 bits;
// a window of that many is every key.
constexpr int64_t kMaxTokens = int64_t(1) << 30;
inline int32_t prompt_window(int32_t window) { return window < kMaxTokens ? window : static_cast<int32_t>(kMaxTokens); }

// What both passes require of their sizes (a grid's workgroups stay below 2^31).
inline bool prompt_heads_ok(int32_t heads, int32_t kv_heads) {
  return kv_heads >= 1 && heads >= 1 && heads <= 65535 && heads % kv_heads == 0;
}
inline bool prompt_sizes_ok(int32_t heads, int64_t B, int64_t Tq, int64_t Tk) {
  return B <= 65535 && Tq <= kMaxTokens && Tk <= kMaxTokens && (Tq / 32 + B) * heads < kMaxDim &&
         (Tk / 32 + B) * heads < kMaxDim;
}
inline bool prompt_shape_ok(int32_t heads, int32_t kv_heads, int32_t head_dim, int64_t B, int64_t Tq, int64_t Tk,
                            int32_t causal, int32_t window) {
  return (head_dim == 64 || head_dim == 128 || head_dim == 256) && prompt_heads_ok(heads, kv_heads) && B >= 0 &&
         Tq >= 0 && Tk >= 0 && prompt_sizes_ok(heads, B, Tq, Tk) && window >= 0 && (window == 0 || causal != 0) &&
         dims_ok(Tq, static_cast<int64_t>(heads) * head_dim) && dims_ok(Tk, static_cast<int64_t>(kv_heads) * head_dim);
}
#define QLIN_PROMPT_SHAPE(heads, kv_heads, head_dim, B, Tq, Tk, scale, causal, window)                         \
  do {                                                                                                         \
    QLIN_REQUIRE((head_dim) == 64 || (head_dim) == 128 || (head_dim) == 256, QLIN_ERR_UNSUPPORTED,             \
                 "head_dim=%d: 64, 128 and 256 are provided", (head_dim));                                     \
    QLIN_REQUIRE(::qlin::prompt_heads_ok((heads), (kv_heads)), QLIN_ERR_SHAPE,                                 \
                 "heads=%d must be in [1, 65535] and a multiple of kv_heads=%d", (heads), (kv_heads));         \
    QLIN_REQUIRE((B) >= 0 && (Tq) >= 0 && (Tk) >= 0, QLIN_ERR_INVALID_ARG, "B=%lld, Tq=%lld, Tk=%lld: negative", \
                 (long long)(B), (long long)(Tq), (long long)(Tk));                                            \
    QLIN_REQUIRE(::qlin::prompt_sizes_ok((heads), (B), (Tq), (Tk)), QLIN_ERR_SHAPE,                            \
                 "B=%lld, Tq=%lld, Tk=%lld: at most 65535 sequences and 2^30 tokens, fewer than 2^31 tiles",        \
                 (long long)(B), (long long)(Tq), (long long)(Tk));                                            \
    QLIN_REQUIRE((scale) - (scale) == 0.0f, QLIN_ERR_INVALID_ARG, "scale is not finite");                      \
    QLIN_REQUIRE((window) >= 0 && ((window) == 0 || (causal)), QLIN_ERR_INVALID_ARG,                           \
                 "window=%d: not negative, and for causal attention only", (window));                          \
    QLIN_DIMS(Tq, static_cast<int64_t>(heads) * (head_dim));                                                   \
    QLIN_DIMS(Tk, static_cast<int64_t>(kv_heads) * (head_dim));                                                \
  } while (0)

// |scale| log2(e); never 0, so that a hidden key's -inf stays what it is (logits
// are below 2^41: this makes them nothing).
inline float prompt_scale(float scale) {
  const float c = (scale < 0.0f ? -scale : scale) * kLog2e;
  return c > 1.0e-30f ? c : 1.0e-30f;
}

}  // namespace qlin
