// Attention of one new token over the paged key/value cache (qlin_attn_decode).
//
// Per sequence and kv head, with up to eight of the group's query heads:
//   S = K q^T   (slots x heads),   P = exp2(S - m),   O^T = V^T P^T  (D x heads)
// on 16x16x32 fp16 matrix instructions, whose 16 columns hold every head twice:
// columns 8 .. 15 carry what rounding P (and a rotated q) to fp16 left over, so
// that a weight or a channel of q is good to 2^-22 of itself, the smallest to
// 2^-27 of the row's largest weight or 2^-35 of the head's largest channel, for no
// further matrix instruction.  Both results hold a head in lane & 7, so the
// softmax state and the rescaling of O never leave the lane, and P comes out of
// the first product in the registers where the second one takes it: the
// eight slots 8g .. 8g + 7 of lane group g = lane >> 4 are one k-group of the
// second product.  K rows are read as its A operand directly; V rows are read
// eight slots by D / 16 channels per lane and transposed in registers by byte
// permutes.  Nothing of K, V, S or P goes through LDS.
//
// Rows of codes stand for lo + step * code, and are never expanded to that: with
// w_i = p_i step_i,  s_i = step_i (q . code_i) + lo_i sum(q)  and
// o = sum_i w_i code_i + sum_i p_i lo_i,  so the codes enter the products as
// small integers and each row costs two multiplications more.  K after the
// Hadamard is met by q after the Hadamard: (k d H)(q d H) = 128 k q.
//
// The work is a sequence of tiles of 32 slots, row after row (a row: a sequence,
// a kv head, and up to 32 of its query heads).  As many workgroups as the GPU
// holds at a time take equal runs of it, wherever rows begin and end, so ragged
// batches and single long rows fill it alike; a row that lies in several
// workgroups leaves a maximum, a sum and a vector in each, which a second launch
// joins.  Rows that are one short run each need no second launch.
//
// Bound by the bytes of K and V, read once (each eight query heads of a larger
// group read them again, from cache where it holds them): 32 sequences of 500 - 4,000 slots,
// 32 kv heads of 128 channels, fp16, 1,180 MB, 209 us or 5.6 TB/s (a plain read
// of that size reaches 6.4); 64 of 1,500 - 12,000, 8 kv heads, int4, 471 MB and
// 55 MB of logits, 118 us or 4.5 TB/s (a copy reaches 5.2), vector instructions
// 40 % and matrix instructions 9 % of the time.  Small calls are bound by their
// chain of waits: launch, lens, page ids, q and the first tile, the join of the
// waves: 7 us for 100 slots; 65,537 slots of 8 kv heads int4, 71 MB, 21 us and 4
// for the second launch, of which reading is 10.
#include <type_traits>

#include "kv.hpp"

namespace qlin {
namespace {

struct AttnArgs {
  KvPool c;
  const uint16_t* q;
  int64_t ld_q;
  int32_t heads;  // query heads
  int32_t group;  // query heads per kv head
  int32_t parts;  // rows per kv head: its query heads, 32 at a time
  const int32_t* table;
  const int32_t* lens;
  int64_t B, max_pages;
  int32_t max_len;
  int32_t window;  // 0: the whole length
  float scale_log2;  // scale * log2(e)
  uint16_t* out;
  const float* mass_in;
  float* mass_out;
  int64_t ld_mass;
  int32_t groups;   // workgroups that share the tiles; 0: one row each, whole
  int2* runs;       // [rows]: slot of a row's first part, and its last workgroup
  float* part_o;    // [2 * groups x row_heads x D]: a workgroup's first and last row, if cut
  float2* part_ml;  // [2 * groups x row_heads]: reference exponent and sum
  int32_t row_heads;
  float2* head_ml;  // [B * heads] of rows that are not cut (with mass)
  float* logits;    // [B * heads x ld_logits], log2 domain (with mass)
  int64_t ld_logits;
};

constexpr int kAttnWaves = 4;
constexpr int kAttnThreads = 64 * kAttnWaves;
constexpr int kCus = 256;
constexpr int kTile = 32;       // slots
constexpr int kTileHeads = 8;   // query heads of a wave
constexpr int kRowHeads = kTileHeads * kAttnWaves;

// A head's weights are exp2(s - m), for codes times the row's step, with m such
// that the largest is 2^kTop when m is set; m moves when one would pass kCeil, so
// fp16 holds them (below 2^16).  m begins as a guess, for logits near zero and V
// near one, and is set if a lane's first weights lie below kFloor: the largest
// is then never smaller, and slots down to 2^-26 of it still count.  (Set by the
// first tile of every row, without a guess: 65,537 slots 24.2 us against 23.1.)
// The sum's own terms may grow to 2^kSumTop where steps are small (or zero: those
// weights are all 0).
constexpr float kTop = 7.0f, kCeil = 0x1p15f, kFloor = 0x1p2f, kSumTop = 30.0f, kSumCeil = 0x1p40f;
template <int BITS>
constexpr float kFirstRef = BITS == 16 ? -8.0f : BITS == 8 ? -13.0f : -9.0f;
// The reference of nothing: below any finite logit.
constexpr float kNoRef = -3.0e38f;

__device__ __forceinline__ v8h as_v8h(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const v4i w = {static_cast<int>(a), static_cast<int>(b), static_cast<int>(c), static_cast<int>(d)};
  return __builtin_bit_cast(v8h, w);
}

__device__ __forceinline__ float lo_half(uint32_t w) { return h2f(static_cast<uint16_t>(w)); }
__device__ __forceinline__ float hi_half(uint32_t w) { return h2f(static_cast<uint16_t>(w >> 16)); }

// Four channels of the output, fp16; zero where nothing has weight.
__device__ __forceinline__ uint2 out4(float4 acc, float sum) {
  const bool none = sum == 0.0f;
  const uint32_t x = f2h(none ? 0.0f : div_rn(acc.x, sum)), y = f2h(none ? 0.0f : div_rn(acc.y, sum));
  const uint32_t z = f2h(none ? 0.0f : div_rn(acc.z, sum)), w = f2h(none ? 0.0f : div_rn(acc.w, sum));
  return make_uint2(x | y << 16, z | w << 16);
}

__device__ __forceinline__ float max_groups(float v) {  // over the four lane groups of a head
  v = fmaxf(v, __shfl_xor(v, 16, 64));
  return fmaxf(v, __shfl_xor(v, 32, 64));
}
__device__ __forceinline__ float sum_groups(float v) {
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

// A value that no kernel here writes, at an address that is the same for the
// whole wave: a scalar load, apart from the vector loads' counter.
__device__ __forceinline__ int32_t scalar_i32(const int32_t* p) {
  return *(const __attribute__((address_space(4))) int32_t*)(p);
}
// Some values are the same in every lane without the compiler seeing it (a
// division's result, a sum after a branch of one lane); it would keep them, and
// all that follows from them, in vector registers.
__device__ __forceinline__ int uniform_i32(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform_i64(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(static_cast<uint64_t>(v) >> 32));
  return static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo);
}

// Powers of two (f, 1 / f) that bring a head's largest |q| to 2^14 .. 2^15, so
// that rounding to fp16 goes by its own size: what the smallest channels lose is
// 2^-39 of the largest, 2^-35 where int4 divides by 16.  (1, 1) for no size.
__device__ __forceinline__ float2 q_power(float top) {
  const uint32_t e = __builtin_bit_cast(uint32_t, top) >> 23;
  if (top == 0.0f || !(top < INFINITY)) return make_float2(1.0f, 1.0f);
  return make_float2(__builtin_bit_cast(float, (268u - e) << 23), __builtin_bit_cast(float, (e - 14u) << 23));
}

// First slot that a sequence of `len` attends to, and one past the last.
__device__ __forceinline__ void attn_range(const AttnArgs& a, int len, int& low, int& n) {
  n = len < 0 ? 0 : len;
  n = n > a.max_len ? a.max_len : n;  // at most the table's slots
  low = (a.window > 0 && n > a.window) ? n - a.window : 0;
}
// A row's tiles: those of its sequence that hold a slot in the range.
__device__ __forceinline__ void attn_tiles(int low, int n, int& t0, int& t1) {
  t0 = low / kTile;
  t1 = (n + kTile - 1) / kTile;
}
// x / y of numbers that are the same in every lane, y > 0: 32 bits where they do.
__device__ __forceinline__ int64_t attn_div(int64_t x, int64_t y) {
  if (x <= 0x7fffffff && y <= 0x7fffffff) return uniform_i32(static_cast<uint32_t>(x) / static_cast<uint32_t>(y));
  return uniform_i64(x / y);
}
// A workgroup's share of `total` tiles.
__device__ __forceinline__ int64_t attn_share(const AttnArgs& a, int64_t total) {
  const int64_t share = attn_div(total + a.groups - 1, a.groups);
  return share < kAttnWaves ? kAttnWaves : share;
}
// Where a workgroup leaves its part of a row: apart if it is a row that begins
// inside the workgroup's run (its last), not at its start or before.
__device__ __forceinline__ int64_t part_slot(int64_t group, int64_t row_begin, int64_t share) {
  return 2 * group + (row_begin > group * share ? 1 : 0);
}

// Codes enter the matrix products as the low 11 bits of an fp16, which are
// linear (denormals, then the first binade): bits * 2^-24.  An AND or a byte
// permute then makes an operand, and the power of two goes into the row's step.
// Of the four nibbles of a 16-bit half, two sit four bits higher, 16 times
// larger; the first product divides q by 16 there, the second one its result.
// The matrix instructions align such operands as if they were normal numbers
// and drop what falls off the end, always downwards: measured, -1.4e-7 of the
// sum for nibbles in bits 0 .. 3, which shows where V's codes cancel against
// the rows' lo over a long cache.  V's nibbles go to bits 3 .. 6 and 7 .. 10
// instead, one shift more (2^-3 of that, and nothing).
template <int BITS>
struct Codes {
  static constexpr float k_unit = 16777216.0f;                              // 2^24
  static constexpr float v_unit = (BITS == 4) ? 2097152.0f : 16777216.0f;  // 2^21
};

// What a workgroup does once per row (q, the join of the waves, the output)
// takes about as long as reading this many bytes, and counts as so many tiles
// before the row's own when the work is divided.  65,537 slots of 8 heads, int4:
// 23.5 us with 0, 22.5 with half of it, 20.2, 19.6 with twice; 64 sequences of
// 1,500 - 12,000 slots: 122, 119, 116 and 120 us.
constexpr int kRowBytes = 65536;

template <int BITS, int D>
struct Attn {
  static constexpr int RB = D * BITS / 8;                  // bytes of a stored row
  static constexpr int KS = D / 32;                        // k steps of the first product
  static constexpr int NT = D / 16;                        // channel tiles of the second
  static constexpr int KW = RB / 16;                       // dwords of K of a lane and row
  static constexpr int DPL = D / 16;                       // channels of V of a lane and row
  static constexpr int VW = (DPL * BITS + 31) / 32;        // dwords of them
  static constexpr int VC = VW > 4 ? 2 : 1;                // 16-byte pieces of them, D / VC channels apart
  static constexpr int DPC = DPL / VC;
  static constexpr bool QUANT = BITS < 16;
  static constexpr int PAD = kRowBytes / (kTile * (2 * RB + (QUANT ? 8 : 0)));  // tiles

  // K: the bytes of lane group g in a row are 16-byte pieces j at 64 j + 16 g
  // (8 bytes at 8 g for 32-byte rows).  Channel of element e of piece j:
  static constexpr int EPP = (RB == 32) ? 16 : 128 / BITS;  // elements of a piece
  static __device__ __forceinline__ int k_channel(int j, int g) { return j * 4 * EPP + g * EPP; }

  // The order of a lane's eight elements in a k step of the first product.
  static __device__ __forceinline__ int k_order(int i) {
    if constexpr (BITS == 4) {
      constexpr int o[8] = {0, 4, 1, 5, 2, 6, 3, 7};
      return o[i];
    }
    return i;
  }

  // Operand of k step s from the row's dwords.
  static __device__ __forceinline__ v8h k_operand(const uint32_t (&w)[KW], int s) {
    if constexpr (BITS == 16) {
      return as_v8h(w[4 * s], w[4 * s + 1], w[4 * s + 2], w[4 * s + 3]);
    } else if constexpr (BITS == 8) {
      const uint32_t a = w[2 * s], b = w[2 * s + 1];
      return as_v8h(__builtin_amdgcn_perm(0u, a, 0x0c010c00u), __builtin_amdgcn_perm(0u, a, 0x0c030c02u),
                    __builtin_amdgcn_perm(0u, b, 0x0c010c00u), __builtin_amdgcn_perm(0u, b, 0x0c030c02u));
    } else {
      const uint32_t x = w[s], y = x >> 8;
      return as_v8h(x & 0x000f000fu, x & 0x00f000f0u, y & 0x000f000fu, y & 0x00f000f0u);
    }
  }

  // Channel of row m of tile t of the second product.
  static __device__ __forceinline__ int v_channel(int t, int m) { return (t / DPC) * 16 * DPC + m * DPC + t % DPC; }

  // Dword of tile t's operand that holds slots a and b (lower, upper half).
  static __device__ __forceinline__ uint32_t v_pair(const uint32_t (&wa)[VW], const uint32_t (&wb)[VW], int t) {
    if constexpr (BITS == 16) {
      return __builtin_amdgcn_perm(wb[t >> 1], wa[t >> 1], (t & 1) ? 0x07060302u : 0x05040100u);
    } else if constexpr (BITS == 8) {
      const uint32_t d = t & 3;
      return __builtin_amdgcn_perm(wb[t >> 2], wa[t >> 2], 0x0c000c00u | ((4 + d) << 16) | d);
    } else {
      const uint32_t w = __builtin_amdgcn_perm(wb[t >> 3], wa[t >> 3], (t & 4) ? 0x07060302u : 0x05040100u);
      const uint32_t y = (t & 2) ? w >> 5 : w << 3;
      return y & ((t & 1) ? 0x07800780u : 0x00780078u);
    }
  }

  static __device__ __forceinline__ void load_k(const uint8_t* p, uint32_t (&w)[KW]) {
    if constexpr (KW == 2) {
      const uint2 x = *reinterpret_cast<const uint2*>(p);
      w[0] = x.x;
      w[1] = x.y;
    } else {
#pragma unroll
      for (int j = 0; j < KW / 4; ++j) {
        const uint4 x = *reinterpret_cast<const uint4*>(p + 64 * j);
        w[4 * j] = x.x;
        w[4 * j + 1] = x.y;
        w[4 * j + 2] = x.z;
        w[4 * j + 3] = x.w;
      }
    }
  }
  static __device__ __forceinline__ void load_v(const uint8_t* p, uint32_t (&w)[VW]) {
    if constexpr (DPL * BITS == 16) {
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    } else if constexpr (VW == 1) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (VW == 2) {
      const uint2 x = *reinterpret_cast<const uint2*>(p);
      w[0] = x.x;
      w[1] = x.y;
    } else {
#pragma unroll
      for (int j = 0; j < VC; ++j) {
        const uint4 x = *reinterpret_cast<const uint4*>(p + 256 * j);
        w[4 * j] = x.x;
        w[4 * j + 1] = x.y;
        w[4 * j + 2] = x.z;
        w[4 * j + 3] = x.w;
      }
    }
  }
};

// Bytes of the kernel's dynamic LDS: the waves' sums, then their vectors or the
// rotated q, whichever is larger.
constexpr int kRotLd = 132;  // of a rotated q: eight heads in different banks
constexpr int kMlBytes = kAttnWaves * kTileHeads * 8;
inline size_t attn_lds(int D, int row_heads, bool rot) {
  const int tiles = (row_heads + kTileHeads - 1) / kTileHeads;
  const int hs = row_heads < kTileHeads ? row_heads : kTileHeads;
  const size_t o = static_cast<size_t>(kAttnWaves) * hs * (D + 4) * sizeof(float);
  const size_t q = rot ? static_cast<size_t>(tiles) * kTileHeads * kRotLd * sizeof(float) : 0;
  return kMlBytes + (o > q ? o : q);
}

// Workgroups that a CU holds: as many as fit with two tiles in registers, so
// that the next one is on its way while one is computed on.  One more spills
// (D = 256, int4, 64 sequences: 282 us against 192).  fp16 rows of D = 256 do not
// quite fit even so: 5 registers a lane go to scratch, 12 with logits (16 sequences
// of 2,000 - 8,000 slots, 4 kv heads, 72 us, 4.5 TB/s).  The launch has as many as
// the GPU holds at a time; twice or three times as many, each with half or a
// third of the work, took 38 and 47 us where one does 65,537 slots in 29.
constexpr int attn_resident(int D) { return D == 64 ? 3 : D == 128 ? 2 : 1; }

template <int BITS, int D, bool ROT, bool LOGITS>
__global__ __launch_bounds__(kAttnThreads, attn_resident(D)) void attn_kernel(AttnArgs a) {
  using A = Attn<BITS, D>;
  constexpr int RB = A::RB, KS = A::KS, NT = A::NT, KW = A::KW, VW = A::VW;
  constexpr bool QUANT = A::QUANT;
  extern __shared__ uint8_t lds[];
  float2* lds_ml = reinterpret_cast<float2*>(lds);         // [wave][kTileHeads]
  float* lds_o = reinterpret_cast<float*>(lds + kMlBytes);  // [wave][head][D + 4]

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ps = a.c.page_shift, line_mask = (1 << ps) - 1;
  const int rows_b = a.c.heads * a.parts;  // rows of a sequence

  // The run of this workgroup: rows (b, r) from place `at` of the flat sequence
  // of places up to `stop`; a row takes PAD places and one for each of its tiles,
  // from row_at on.  len: the sequence's length.
  int64_t at = 0, stop = 0, row_at = 0, share = 0;
  int b, r, len;
  if (a.groups == 0) {
    b = uniform_i32(static_cast<int>(blockIdx.x) / rows_b);
    len = scalar_i32(a.lens + b);
    r = static_cast<int>(blockIdx.x) - b * rows_b;
  } else {
    // Every wave for itself: the tiles of all sequences, then the one where the
    // run begins.
    auto len_of = [&](int i) { return i < a.B ? a.lens[i] : 0; };
    auto tiles_of = [&](int len) {
      int low, n, t0, t1;
      attn_range(a, len, low, n);
      attn_tiles(low, n, t0, t1);
      return t1 == t0 ? 0 : t1 - t0 + A::PAD;
    };
    const int len0 = len_of(lane), tiles0 = tiles_of(len0);
    const uint32_t sum0 = wave_scan(tiles0);  // 64 times 2^25 at most
    int64_t total = static_cast<uint32_t>(__builtin_amdgcn_readlane(sum0, 63));
    for (int b0 = 64; b0 < a.B; b0 += 64)
      total += static_cast<uint32_t>(__builtin_amdgcn_readlane(wave_scan(tiles_of(len_of(b0 + lane))), 63));
    total *= rows_b;
    share = attn_share(a, total);
    at = blockIdx.x * share;
    stop = min(at + share, total);
    if (at >= stop) return;
    int64_t before = 0;  // tiles of the sequences before b0
    for (int b0 = 0;; b0 += 64) {
      const int row_len = b0 == 0 ? len0 : len_of(b0 + lane), tiles = b0 == 0 ? tiles0 : tiles_of(row_len);
      const uint32_t sum = b0 == 0 ? sum0 : wave_scan(tiles);
      const uint64_t past = __ballot((before + sum) * rows_b > at);
      if (past != 0) {
        const int i = __builtin_ctzll(past);
        const int own = __builtin_amdgcn_readlane(tiles, i);
        b = b0 + i;
        len = __builtin_amdgcn_readlane(row_len, i);
        row_at = (before + static_cast<uint32_t>(__builtin_amdgcn_readlane(sum, i)) - own) * rows_b;
        r = static_cast<int>(attn_div(at - row_at, own));
        row_at += static_cast<int64_t>(r) * own;
        break;
      }
      before += static_cast<uint32_t>(__builtin_amdgcn_readlane(sum, 63));
    }
  }

  // A row, or the part of it in this run: tiles [t0, t1) of sequence b.
  struct Row {
    int low, n, t0, t1, tiles;  // slots attended to, tiles here and in all
    int h, hrow, hq0;           // kv head; query heads, and the first of them
    int per, ht, hs, end;       // waves of a head tile; this wave's head tile, its heads (none: it idles)
    const int32_t* table;
    int last_page;
  };
  auto row_of = [&]() {
    Row w;
    attn_range(a, len, w.low, w.n);
    attn_tiles(w.low, w.n, w.t0, w.t1);
    w.tiles = w.t1 - w.t0;
    if (a.groups != 0) {
      const int64_t first = at > row_at + A::PAD ? at - row_at - A::PAD : 0;
      const int64_t last = stop - row_at - A::PAD < w.tiles ? stop - row_at - A::PAD : w.tiles;
      w.t1 = w.t0 + static_cast<int>(last);
      w.t0 += static_cast<int>(first);
    }
    w.h = a.parts == 1 ? r : uniform_i32(r / a.parts);
    const int part = r - w.h * a.parts;
    w.hrow = min(kRowHeads, a.group - part * kRowHeads);
    w.hq0 = w.h * a.group + part * kRowHeads;
    // The waves share out the head tiles, then the slots.
    const int head_tiles = (w.hrow + kTileHeads - 1) / kTileHeads;
    const int shift = head_tiles == 1 ? 2 : head_tiles == 2 ? 1 : 0;
    w.per = 1 << shift;
    w.ht = wave >> shift;
    w.hs = min(kTileHeads, w.hrow - w.ht * kTileHeads);
    w.end = min(w.n, w.t1 * kTile);
    w.table = a.table + static_cast<int64_t>(b) * a.max_pages;
    w.last_page = max(w.n - 1, 0) >> ps;
    return w;
  };
  struct Tile {
    uint32_t k[2][KW], v[8][VW], km[8], vm[8];
    bool ok0, ok1;  // its halves are on pages of the pool
  };
  auto load = [&](Tile& x, const Row& w, int tile, int g, int col) {
    // The rows where the halves of the tile begin: pages hold 16 slots or
    // more.  A half beyond the last page, or on a page outside the pool,
    // reads another row instead, and its values are dropped below.
    const int slot = tile * kTile;
    const int32_t id0 = scalar_i32(w.table + (slot >> ps));
    const int32_t id1 = scalar_i32(w.table + min((slot + 16) >> ps, w.last_page));
    const uint32_t pages = static_cast<uint32_t>(a.c.pages), heads = static_cast<uint32_t>(a.c.heads);
    x.ok0 = static_cast<uint32_t>(id0) < pages;
    x.ok1 = static_cast<uint32_t>(id1) < pages;
    const uint32_t p0 = x.ok0 ? id0 : 0, p1 = x.ok1 ? id1 : 0;
    const int64_t row0 = ((static_cast<uint64_t>(p0) * heads + w.h) << ps) + (slot & line_mask);
    const int64_t row1 = ((static_cast<uint64_t>(p1) * heads + w.h) << ps) + ((slot + 16) & line_mask);
    // Row 8 * (run & 1) + line of the lane's run of eight slots, from the row
    // where its half of the tile begins.
    const int krun = col >> 2;
    const int64_t krow = krun < 2 ? row0 : row1, vrow = g < 2 ? row0 : row1;
    const int v_row = 8 * (g & 1);
    const uint8_t* kp = a.c.k + krow * RB + (8 * (krun & 1) + (col & 3)) * RB + (RB == 32 ? 8 : 16) * g;
    const uint8_t* vp = a.c.v + vrow * RB + v_row * RB + col * (RB / 16 / A::VC);
    A::load_k(kp, x.k[0]);
    A::load_k(kp + 4 * RB, x.k[1]);
    if constexpr (QUANT) {
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        const uint4 m = *reinterpret_cast<const uint4*>(a.c.kmeta + vrow + v_row + i);
        x.km[i] = m.x, x.km[i + 1] = m.y, x.km[i + 2] = m.z, x.km[i + 3] = m.w;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) A::load_v(vp + i * RB, x.v[i]);
    if constexpr (QUANT) {
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        const uint4 m = *reinterpret_cast<const uint4*>(a.c.vmeta + vrow + v_row + i);
        x.vm[i] = m.x, x.vm[i + 1] = m.y, x.vm[i + 2] = m.z, x.vm[i + 3] = m.w;
      }
    }
  };
  if (a.groups != 0 && row_at + A::PAD >= stop) return;  // the run ends before the row's first tile
  while (true) {
    const Row w = row_of();
    const int low = w.low, end = w.end, hrow = w.hrow, hs = w.hs, ht = w.ht, per = w.per;
    const int64_t head0 = static_cast<int64_t>(b) * a.heads + w.hq0;
    // What depends on the lane alone is worked out anew for each row: kept
    // across rows, it would take the registers of a tile.
    int lane_again = lane;
    asm volatile("" : "+v"(lane_again));
    const int g = lane_again >> 4, col = lane_again & 15;

    // Two tiles, in turn: one is loaded while the other is computed on; the
    // first is on its way while q is prepared.  (A wave without a tile loads one
    // as well: of the row, or of page 0 for a row without slots.)
    // q's loads go out before the tile's: loads are waited for in order.
    constexpr int SPP = A::EPP / 8;  // k steps of a piece
    const int hcol = col & 7, rem = col >> 3;
    const bool here = hcol < hs;
    const int c = tid & 15;  // of a rotated q: 16 lanes a head, heads tid >> 4 and on
    const uint16_t* q_row0 = a.q + b * a.ld_q + static_cast<int64_t>(w.hq0) * D;
    v4i qr;
    uint2 qsigns;
    v8h qf[KS];
    if constexpr (ROT) {
      qr = *reinterpret_cast<const v4i*>(q_row0 + min(tid >> 4, hrow - 1) * D + 8 * c);
      qsigns = *reinterpret_cast<const uint2*>(a.c.signs + 8 * c);
    } else {
      const uint16_t* qp = q_row0 + (here ? ht * kTileHeads + hcol : 0) * D;
#pragma unroll
      for (int s = 0; s < KS; ++s)
        qf[s] = *reinterpret_cast<const v8h*>(qp + A::k_channel(s / SPP, g) + 8 * (s % SPP));
    }
    __builtin_amdgcn_sched_barrier(0);
    Tile x, y;
    int tile = w.t0 + (wave & (per - 1));  // uniform per wave
    load(x, w, max(min(tile, w.t1 - 1), 0), g, col);

    // q in the operand order of the first product, and sum_d q_d for the rows'
    // lo.  Columns 8 .. 15: the same q, or what fp16 leaves of a rotated one.
    const float frem = static_cast<float>(rem);
    float qsum = 0.0f, unit = 1.0f;  // q is the operand times unit
    if constexpr (ROT) {
      float* q_lds = lds_o;  // [head][kRotLd]
      for (int hd = tid >> 4; hd < (hrow + kTileHeads - 1) / kTileHeads * kTileHeads; hd += kAttnThreads / 16) {
        float u[8];  // uniform per wave: 16 lanes a head
        if (hd >= kAttnThreads / 16) qr = *reinterpret_cast<const v4i*>(q_row0 + min(hd, hrow - 1) * D + 8 * c);
        signed8(qr, qsigns, u);
        hadamard128(u, c);
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(u[i]));
        top = fmaxf(top, lane_xor<1>(top));
        top = fmaxf(top, lane_xor<2>(top));
        top = fmaxf(top, lane_xor<4>(top));
        top = fmaxf(top, lane_xor<8>(top));
        const float2 power = q_power(top);
        const float f = hd < hrow ? power.x : 0.0f;
        if (c == 0) q_lds[hd * kRotLd + 128] = power.y * 0.0078125f;
        float4* dst = reinterpret_cast<float4*>(q_lds + hd * kRotLd + 8 * c);
        dst[0] = make_float4(u[0] * f, u[1] * f, u[2] * f, u[3] * f);
        dst[1] = make_float4(u[4] * f, u[5] * f, u[6] * f, u[7] * f);
      }
      lds_barrier();
      const float* q_row = q_lds + ((hs > 0 ? ht : 0) * kTileHeads + hcol) * kRotLd;
      unit = q_row[128];
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const float4* src = reinterpret_cast<const float4*>(q_row + A::k_channel(s / SPP, g) + 8 * (s % SPP));
        const float4 lo4 = src[0], hi4 = src[1];
        const float u[8] = {lo4.x, lo4.y, lo4.z, lo4.w, hi4.x, hi4.y, hi4.z, hi4.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float v = u[A::k_order(i)];
          qsum += v;
          if (BITS == 4 && (i & 2)) v *= 0.0625f;
          const _Float16 hi = static_cast<_Float16>(v);
          qf[s][i] = rem ? static_cast<_Float16>(v - static_cast<float>(hi)) : hi;
        }
      }
      lds_barrier();  // lds_o takes the vectors next
    } else {
      float f = 1.0f;
      if constexpr (BITS == 4) {
        float top = 0.0f;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
#pragma unroll
          for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(static_cast<float>(qf[s][i])));
        }
        const float2 power = q_power(max_groups(top));
        f = power.x;
        unit = power.y;
      }
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const v8h raw = qf[s];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const _Float16 v = here ? raw[A::k_order(i)] : static_cast<_Float16>(0.0f);
          if constexpr (QUANT) qsum += static_cast<float>(v);
          if constexpr (BITS == 4)
            qf[s][i] = static_cast<_Float16>(static_cast<float>(v) * ((i & 2) ? f * 0.0625f : f));
          else
            qf[s][i] = v;
        }
      }
    }
    if constexpr (QUANT) qsum = sum_groups(qsum) * (ROT ? a.scale_log2 * unit : a.scale_log2);
    const float qscale = QUANT ? a.scale_log2 * Codes<BITS>::k_unit * unit : a.scale_log2;

    v4f o[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) o[t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    float m = kFirstRef<BITS>, l = 0.0f, olo = 0.0f;  // olo: the weights times the rows' lo

    auto compute = [&](Tile& x, int tile) {
      const int base = tile * kTile;
      float s[8];  // logits less m
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < KS; ++k)
          acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(A::k_operand(x.k[t], k), qf[k], acc, 0, 0, 0);
#pragma unroll
        for (int i = 4 * t; i < 4 * t + 4; ++i) {
          if constexpr (ROT) acc[i & 3] += lane_xor<8>(acc[i & 3]);
          if constexpr (QUANT)
            s[i] = __builtin_fmaf(acc[i & 3] * qscale, lo_half(x.km[i]), __builtin_fmaf(hi_half(x.km[i]), qsum, -m));
          else
            s[i] = __builtin_fmaf(acc[i & 3], qscale, -m);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      if (!(x.ok0 && x.ok1 && base >= low && base + kTile <= end)) {  // uniform
        const bool on_page = g < 2 ? x.ok0 : x.ok1;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int slot = base + 8 * g + i;
          const bool ok = on_page && slot >= low && slot < end;
          s[i] = ok ? s[i] : -INFINITY;
#pragma unroll
          for (int w = 0; w < VW; ++w) x.v[i][w] = ok ? x.v[i][w] : 0u;
          if constexpr (QUANT) x.vm[i] = ok ? x.vm[i] : 0u;
        }
      }
      if constexpr (LOGITS) {
        if (col < hs) {
          float* lp = a.logits + (head0 + ht * kTileHeads + col) * a.ld_logits + base + 8 * g;
          *reinterpret_cast<float4*>(lp) = make_float4(s[0] + m, s[1] + m, s[2] + m, s[3] + m);
          *reinterpret_cast<float4*>(lp + 4) = make_float4(s[4] + m, s[5] + m, s[6] + m, s[7] + m);
        }
      }
      float e[8], w[8], sum, wmax;
      auto weights = [&]() {
        sum = 0.0f;
        wmax = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          e[i] = __builtin_amdgcn_exp2f(s[i]);
          sum += e[i];
          w[i] = QUANT ? __builtin_fmaf(e[i], lo_half(x.vm[i]), 0.0f) : e[i];
          wmax = fmaxf(wmax, w[i]);
        }
      };
      weights();
      // Out of range, or the lane's first weights and too small: against an m far
      // above their logits fp16 keeps little of them, or nothing.
      if (__any(wmax > kCeil || sum > kSumCeil || !(l > 0.0f || wmax >= kFloor))) {
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          top = fmaxf(top, s[i] - kSumTop);
          // A step that is not finite makes its own weight so, whatever m is.
          const float step = QUANT ? lo_half(x.vm[i]) : 1.0f;
          if (step > 0.0f && step < INFINITY) top = fmaxf(top, s[i] + __builtin_amdgcn_logf(step) - kTop);
        }
        top = max_groups(top);
        const bool none = sum_groups(l) == 0.0f;
        const float up = top == -INFINITY ? 0.0f : (none ? top : fmaxf(top, 0.0f));
        const float alpha = none ? 1.0f : __builtin_amdgcn_exp2f(-up);
        m += up;
        l *= alpha;
        olo *= alpha;
#pragma unroll
        for (int t = 0; t < NT; ++t) o[t] *= alpha;
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] -= up;
        weights();
      }
      l += sum;
      v8h p;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (QUANT) olo = __builtin_fmaf(e[i], hi_half(x.vm[i]), olo);
        p[i] = static_cast<_Float16>(w[i]);
      }
      // Columns 8 .. 15 take the remainders.
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = static_cast<_Float16>(__builtin_fmaf(-frem, static_cast<float>(p[i]), w[i]));
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (t % 4 == 0) __builtin_amdgcn_sched_barrier(0);
        const v8h vf = as_v8h(A::v_pair(x.v[0], x.v[1], t), A::v_pair(x.v[2], x.v[3], t),
                              A::v_pair(x.v[4], x.v[5], t), A::v_pair(x.v[6], x.v[7], t));
        o[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, p, o[t], 0, 0, 0);
      }
    };
    if (hs > 0 && tile < w.t1) {
      // The last load of a row reads its last tile again: without a branch
      // around it, what is in flight is known, and only what is used is waited
      // for.
      while (true) {
        load(y, w, min(tile + per, w.t1 - 1), g, col);
        __builtin_amdgcn_sched_barrier(0);
        compute(x, tile);
        tile += per;
        if (tile >= w.t1) break;
        load(x, w, min(tile + per, w.t1 - 1), g, col);
        __builtin_amdgcn_sched_barrier(0);
        compute(y, tile);
        tile += per;
        if (tile >= w.t1) break;
      }
    }
    // The wave's sums in the values' own units, then the waves of each head tile.
    l = sum_groups(l);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // An infinite value of V times a remainder of 0 is a NaN that is not the sum's.
        const float both = o[t][i] + lane_xor<8>(o[t][i]);
        o[t][i] = both == both ? both : o[t][i];
      }
    }
    if constexpr (QUANT) {
      olo = sum_groups(olo);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        constexpr float unit = Codes<BITS>::v_unit;
        const float f = (BITS == 4 && (t & 1)) ? unit / 16.0f : unit;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[t][i] = __builtin_fmaf(o[t][i], f, olo);
      }
    }
    const int lds_heads = min(hrow, kTileHeads);
    if (lane < kTileHeads) lds_ml[wave * kTileHeads + lane] = make_float2(l == 0.0f ? kNoRef : m, l);
    if (col < hs) {
      float* dst = lds_o + (wave * lds_heads + col) * (D + 4);
#pragma unroll
      for (int t = 0; t < NT; t += 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<float4*>(dst + A::v_channel(t, 4 * g + i)) =
              make_float4(o[t][i], o[t + 1][i], o[t + 2][i], o[t + 3][i]);
      }
    }
    const bool whole = w.t1 - w.t0 == w.tiles;
    lds_barrier();
    const int64_t slot = whole ? 0 : part_slot(blockIdx.x, row_at + A::PAD, share) * a.row_heads;
    for (int i = tid; i < hrow * (D / 4); i += kAttnThreads) {
      const int hd = i / (D / 4), d = i % (D / 4) * 4, w0 = hd / kTileHeads * per, hl = hd % kTileHeads;
      float mx = kNoRef;
      for (int v = w0; v < w0 + per; ++v) mx = fmaxf(mx, lds_ml[v * kTileHeads + hl].x);
      float sum = 0.0f;
      float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int v = w0; v < w0 + per; ++v) {
        const float2 ml = lds_ml[v * kTileHeads + hl];
        const float4 u = *reinterpret_cast<const float4*>(lds_o + (v * lds_heads + hl) * (D + 4) + d);
        const float f = __builtin_amdgcn_exp2f(ml.x - mx);
        sum = __builtin_fmaf(ml.y, f, sum);
        acc.x = __builtin_fmaf(u.x, f, acc.x);
        acc.y = __builtin_fmaf(u.y, f, acc.y);
        acc.z = __builtin_fmaf(u.z, f, acc.z);
        acc.w = __builtin_fmaf(u.w, f, acc.w);
      }
      if (whole) {
        *reinterpret_cast<uint2*>(a.out + (head0 + hd) * D + d) = out4(acc, sum);
        if (LOGITS && d == 0) a.head_ml[head0 + hd] = make_float2(mx, sum);
      } else {
        *reinterpret_cast<float4*>(a.part_o + (slot + hd) * D + d) = acc;
        if (d == 0) a.part_ml[slot + hd] = make_float2(mx, sum);
      }
    }
    if (a.groups == 0) return;
    // A row that begins here says where its first part is, and its last workgroup.
    row_at += A::PAD;
    const int last_group = whole ? blockIdx.x : static_cast<int>(attn_div(row_at + w.tiles - 1, share));
    if (tid == 0 && at <= row_at)
      a.runs[static_cast<int64_t>(b) * rows_b + r] =
          make_int2(static_cast<int>(part_slot(blockIdx.x, row_at, share)), last_group);
    row_at = uniform_i64(row_at + w.tiles);
    if (row_at + A::PAD >= stop) return;
    at = row_at;
    if (++r == rows_b) {
      r = 0;
      int next_low, next_n;
      do {  // the next sequence with a tile; there is one, as row_at < stop
        ++b;
        len = scalar_i32(a.lens + b);
        attn_range(a, len, next_low, next_n);
      } while (next_n == 0);
    }
    lds_barrier();  // lds_o and lds_ml are read
  }
}

// The weights of every slot need the sums over all of them, and the logits are
// 4 bytes per query head where K is D / 2 and more per kv head, so the first
// kernel leaves its logits in memory and this one takes the exponential again:
// 55 MB of logits and 28 MB of mass in 20 us (64 sequences as above); 4 us where
// there is only the join, three dependent reads.
//
// Per (row, kv head): the first join_blocks workgroups (one for each query head
// of the group, or none) join the parts of a row that several workgroups took;
// each of the others adds the group's weights of kMassSlots slots to mass.
constexpr int kJoinThreads = 256;
// Sets of 1,024 slots, and heads whose logits are loaded together: 64 sequences
// as above, groups of 4 and 8 heads, 19.7 and 31 us; 26 and 29.5 with one set, 22
// and 36 with four, 24 and 38 with eight heads.
constexpr int kMassSets = 2, kMassHeads = 4;
constexpr int kMassSlots = kMassSets * 4 * kJoinThreads;

// The parts of one query head of a row: index of part i in part_ml.
struct Parts {
  int64_t first, rest;
  int count, step;
  __device__ __forceinline__ int64_t at(int i) const { return i == 0 ? first : rest + static_cast<int64_t>(i) * step; }
};
__device__ __forceinline__ int2 attn_run(const AttnArgs& a, int64_t row) {
  const int32_t* p = reinterpret_cast<const int32_t*>(a.runs + row);
  return a.groups == 0 ? make_int2(0, 0) : make_int2(scalar_i32(p), scalar_i32(p + 1));
}
__device__ __forceinline__ Parts attn_parts(const AttnArgs& a, const int2 run, int hd) {
  if (a.groups == 0) return Parts{0, 0, 1, 0};
  const int w0 = run.x >> 1;
  return Parts{static_cast<int64_t>(run.x) * a.row_heads + hd, static_cast<int64_t>(2 * w0) * a.row_heads + hd,
               run.y - w0 + 1, 2 * a.row_heads};
}

template <int D>
__global__ __launch_bounds__(kJoinThreads) void attn_join_kernel(AttnArgs a, int join_blocks) {
  constexpr int LANES = D / 4, ROWS = kJoinThreads / LANES;
  __shared__ float4 acc_lds[kJoinThreads];
  __shared__ float2 row_ml[ROWS];
  __shared__ float2 head_ml[kRowHeads];
  const int tid = threadIdx.x;
  const int h = blockIdx.y;
  const int64_t b = blockIdx.z;
  const int len = scalar_i32(a.lens + b);
  int low, n;
  if (static_cast<int>(blockIdx.x) < join_blocks) {
    const int hd = blockIdx.x;
    // (Of a row without slots, which left no run, nothing is done with it.)
    const Parts p = attn_parts(a, attn_run(a, (b * a.c.heads + h) * a.parts + hd / kRowHeads), hd % kRowHeads);
    attn_range(a, len, low, n);
    uint2* out = reinterpret_cast<uint2*>(a.out + (b * a.heads + h * a.group + hd) * D);
    if (n == 0) {
      if (tid < LANES) out[tid] = make_uint2(0, 0);
      return;
    }
    if (p.count == 1) return;
    // Thread r0 * LANES + d4 takes parts r0, r0 + ROWS, .. with a reference of
    // its own, so no pass over the maxima comes first.
    const int d4 = tid % LANES, r0 = tid / LANES;
    float mx = kNoRef, sum = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int i = r0; i < p.count; i += ROWS) {
      const int64_t at = p.at(i);
      const float2 x = a.part_ml[at];
      const float4 v = reinterpret_cast<const float4*>(a.part_o + at * D)[d4];
      const float to = fmaxf(mx, x.x), f0 = __builtin_amdgcn_exp2f(mx - to), f = __builtin_amdgcn_exp2f(x.x - to);
      mx = to;
      sum = __builtin_fmaf(x.y, f, sum * f0);
      acc.x = __builtin_fmaf(v.x, f, acc.x * f0);
      acc.y = __builtin_fmaf(v.y, f, acc.y * f0);
      acc.z = __builtin_fmaf(v.z, f, acc.z * f0);
      acc.w = __builtin_fmaf(v.w, f, acc.w * f0);
    }
    acc_lds[tid] = acc;
    if (d4 == 0) row_ml[r0] = make_float2(mx, sum);
    __syncthreads();
    if (tid < LANES) {
      float top = kNoRef, total = 0.0f;
#pragma unroll
      for (int i = 0; i < ROWS; ++i) top = fmaxf(top, row_ml[i].x);
      float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        const float4 v = acc_lds[i * LANES + tid];
        const float f = __builtin_amdgcn_exp2f(row_ml[i].x - top);
        total = __builtin_fmaf(row_ml[i].y, f, total);
        t.x = __builtin_fmaf(v.x, f, t.x);
        t.y = __builtin_fmaf(v.y, f, t.y);
        t.z = __builtin_fmaf(v.z, f, t.z);
        t.w = __builtin_fmaf(v.w, f, t.w);
      }
      out[tid] = out4(t, total);
    }
    return;
  }
  // mass of slots [s0, s0 + kMassSlots) of one (row, kv head)
  const int64_t bh = b * a.c.heads + h;
  int2 run = attn_run(a, bh * a.parts);
  attn_range(a, len, low, n);
  const int s0 = (static_cast<int>(blockIdx.x) - join_blocks) * kMassSlots;
  if (s0 >= n) return;  // uniform
  const int64_t head0 = b * a.heads + h * a.group;
  // What needs no statistics is loaded before they are known: mass, and the
  // logits of the first heads.  Below the window there are none.
  const bool any = s0 + kMassSlots > low;
  const uintptr_t ends = reinterpret_cast<uintptr_t>(a.mass_out) | reinterpret_cast<uintptr_t>(a.mass_in);
  const bool wide = ((a.ld_mass & 3) | (ends & 15)) == 0;  // four slots at once
  float w[kMassSets][4], base[kMassSets][4];
  float4 s[kMassSets][kMassHeads];
  auto first = [&](int j) { return s0 + j * 4 * kJoinThreads + 4 * tid; };  // four slots each
  auto load = [&](int h0, int hd, int hs) {
    const float* lp = a.logits + (head0 + h0 + hd) * a.ld_logits;
#pragma unroll
    for (int j = 0; j < kMassSets; ++j) {
      const bool seen = first(j) + 3 >= low && first(j) < n;
#pragma unroll
      for (int i = 0; i < kMassHeads; ++i) {
        s[j][i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (hd + i < hs && seen) s[j][i] = *reinterpret_cast<const float4*>(lp + i * a.ld_logits + first(j));
      }
    }
  };
  load(0, 0, min(kRowHeads, a.group));
#pragma unroll
  for (int j = 0; j < kMassSets; ++j) {
    const int slot0 = first(j);
    const int64_t mass_at = bh * a.ld_mass + slot0;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[j][i] = base[j][i] = 0.0f;
    if (a.mass_in != nullptr) {
      if (wide) {
        if (slot0 < n) {
          const float4 v = *reinterpret_cast<const float4*>(a.mass_in + mass_at);
          base[j][0] = v.x, base[j][1] = v.y, base[j][2] = v.z, base[j][3] = v.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (slot0 + i < n) base[j][i] = a.mass_in[mass_at + i];
      }
    }
  }
  for (int h0 = 0; any && h0 < a.group; h0 += kRowHeads) {  // uniform
    const int hs = min(kRowHeads, a.group - h0);
    if (h0 > 0) run = attn_run(a, bh * a.parts + h0 / kRowHeads);
    __syncthreads();
    // Each wave takes heads in turn: maximum, then sum, over the parts.
    for (int hd = tid >> 6; hd < hs; hd += kJoinThreads / 64) {
      const Parts p = attn_parts(a, run, hd);
      float mx, sum;
      if (p.count == 1) {
        const float2 ml = a.head_ml[head0 + h0 + hd];
        mx = ml.x;
        sum = ml.y;
      } else {
        float own = kNoRef;
        sum = 0.0f;
        for (int i = tid & 63; i < p.count; i += 64) {
          const float2 ml = a.part_ml[p.at(i)];
          const float to = fmaxf(own, ml.x);
          sum = __builtin_fmaf(ml.y, __builtin_amdgcn_exp2f(ml.x - to), sum * __builtin_amdgcn_exp2f(own - to));
          own = to;
        }
        mx = wave_max(own);
        sum *= __builtin_amdgcn_exp2f(own - mx);
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
      }
      if ((tid & 63) == 0) head_ml[hd] = make_float2(mx, sum == 0.0f ? 0.0f : div_rn(1.0f, sum));
    }
    __syncthreads();
    for (int hd = 0; hd < hs; hd += kMassHeads) {
      if (h0 + hd > 0) load(h0, hd, hs);
#pragma unroll
      for (int i = 0; i < kMassHeads; ++i) {
        if (hd + i < hs) {
          const float2 ml = head_ml[hd + i];
#pragma unroll
          for (int j = 0; j < kMassSets; ++j) {
            w[j][0] = __builtin_fmaf(__builtin_amdgcn_exp2f(s[j][i].x - ml.x), ml.y, w[j][0]);
            w[j][1] = __builtin_fmaf(__builtin_amdgcn_exp2f(s[j][i].y - ml.x), ml.y, w[j][1]);
            w[j][2] = __builtin_fmaf(__builtin_amdgcn_exp2f(s[j][i].z - ml.x), ml.y, w[j][2]);
            w[j][3] = __builtin_fmaf(__builtin_amdgcn_exp2f(s[j][i].w - ml.x), ml.y, w[j][3]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < kMassSets; ++j) {
    const int slot0 = first(j);
    const int64_t mass_at = bh * a.ld_mass + slot0;
    // (Logits outside the range were never written.)
#pragma unroll
    for (int i = 0; i < 4; ++i) base[j][i] += slot0 + i >= low ? w[j][i] : 0.0f;
    if (wide && slot0 + 3 < n) {
      *reinterpret_cast<float4*>(a.mass_out + mass_at) = make_float4(base[j][0], base[j][1], base[j][2], base[j][3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (slot0 + i < n) a.mass_out[mass_at + i] = base[j][i];
    }
  }
}

struct AttnPlan {
  int parts, row_heads, groups;
  int64_t ld_logits;
  size_t run_bytes, ml_bytes, head_bytes, o_bytes, logit_bytes;
  size_t total() const { return run_bytes + ml_bytes + head_bytes + o_bytes + logit_bytes; }
};

inline size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Rows of at most this many tiles are one workgroup each: no second launch.
// Both launches, replayed from a graph, 128 channels, 4 query heads a kv head, as
// one workgroup each against divided and joined: one row of 512 slots 8.9 against
// 9.1 us (fp16), 7.7 against 9.4 (int8), 8.1 against 10.0 (int4), of 1,024 13.1
// against 9.4, 10.6 against 9.2, 10.8 against 10.0; 32 rows of 512 9.2 against 10.4,
// 8.0 against 10.0, 8.5 against 10.5, of 1,024 14.6 against 11.6, 11.3 against 10.4,
// 11.5 against 10.8.  (128 rows of 1,024 would be faster whole: 15.4 against 18.7,
// 12.2 against 17.6, 12.3 against 14.8.)
constexpr int64_t kWholeTiles = 16;

AttnPlan attn_plan(const qlin_kv_cache& c, int32_t heads, int64_t B, int64_t max_len, int32_t window, bool mass) {
  AttnPlan p;
  const int group = heads / c.kv_heads;
  p.parts = (group + kRowHeads - 1) / kRowHeads;
  p.row_heads = group < kRowHeads ? group : kRowHeads;
  int64_t tiles = (max_len + kTile - 1) / kTile;
  if (window > 0) {  // a window may begin inside a tile
    const int64_t w = (static_cast<int64_t>(window) + kTile - 2) / kTile + 1;
    tiles = w < tiles ? w : tiles;
  }
  const int64_t rows = B * c.kv_heads * p.parts;
  const int64_t most = int64_t(kCus) * attn_resident(c.head_dim);
  const int64_t runs = (rows * tiles + kAttnWaves - 1) / kAttnWaves;
  p.groups = tiles <= kWholeTiles ? 0 : static_cast<int>(runs < most ? runs : most);
  const size_t parts = static_cast<size_t>(2) * p.groups * p.row_heads;
  const size_t n = static_cast<size_t>(B) * heads;
  p.run_bytes = p.groups ? up256(static_cast<size_t>(rows) * sizeof(int2)) : 0;
  p.ml_bytes = up256(parts * sizeof(float2));
  p.o_bytes = up256(parts * c.head_dim * sizeof(float));
  p.head_bytes = mass ? up256(n * sizeof(float2)) : 0;
  p.ld_logits = (max_len + kTile - 1) / kTile * kTile;
  p.logit_bytes = mass ? n * static_cast<size_t>(p.ld_logits) * sizeof(float) : 0;
  return p;
}

template <int BITS, int D, bool ROT>
void launch_attn(const AttnArgs& a, const dim3 grid, hipStream_t st) {
  const size_t lds = attn_lds(D, a.row_heads, ROT);
  if (a.logits != nullptr)
    attn_kernel<BITS, D, ROT, true><<<grid, kAttnThreads, lds, st>>>(a);
  else
    attn_kernel<BITS, D, ROT, false><<<grid, kAttnThreads, lds, st>>>(a);
}

template <int BITS>
void launch_bits(const AttnArgs& a, int D, const dim3 grid, hipStream_t st) {
  if (D == 64) return launch_attn<BITS, 64, false>(a, grid, st);
  if (D == 256) return launch_attn<BITS, 256, false>(a, grid, st);
  if constexpr (BITS < 16) {
    if (a.c.signs != nullptr) return launch_attn<BITS, 128, true>(a, grid, st);
  }
  launch_attn<BITS, 128, false>(a, grid, st);
}

}  // namespace
}  // namespace qlin

using namespace qlin;

extern "C" size_t qlin_attn_decode_work_bytes(const qlin_kv_cache* cache, int32_t heads, int64_t B, int64_t max_len,
                                              int32_t window, int32_t mass) {
  if (!kv_shape_ok(cache) || heads < 1 || heads % cache->kv_heads != 0 || B < 1 || max_len < 0 ||
      max_len > kMaxDim / 2 || window < 0 || !dims_ok(B, max_len) || !dims_ok(B * heads, max_len + 1) ||
      !dims_ok(B * heads, cache->head_dim))
    return 0;
  const AttnPlan p = attn_plan(*cache, heads, B, max_len, window, mass != 0);
  return p.total();
}

extern "C" qlin_status qlin_attn_decode(const qlin_kv_cache* cache, const uint16_t* q, int64_t ld_q, int32_t heads,
                                        const int32_t* table, const int32_t* lens, int64_t B, int64_t max_pages,
                                        int64_t max_len, float scale, int32_t window, uint16_t* out,
                                        const float* mass_in, float* mass_out, int64_t ld, void* work, void* stream) {
  QLIN_KV_CACHE(cache);
  QLIN_KV_TABLE(cache, B, max_pages);
  QLIN_REQUIRE(heads >= 1 && heads % cache->kv_heads == 0, QLIN_ERR_SHAPE,
               "heads=%d must be a positive multiple of kv_heads=%d", heads, cache->kv_heads);
  const int64_t width = static_cast<int64_t>(heads) * cache->head_dim;
  QLIN_REQUIRE(ld_q >= width && ld_q % 8 == 0, QLIN_ERR_SHAPE,
               "ld_q=%lld must be a multiple of 8, at least heads * head_dim", (long long)ld_q);
  QLIN_DIMS(B, ld_q);
  QLIN_REQUIRE(max_len >= 0, QLIN_ERR_INVALID_ARG, "max_len=%lld is negative", (long long)max_len);
  QLIN_REQUIRE(max_len <= max_pages * cache->page, QLIN_ERR_SHAPE, "max_len=%lld: the table holds %lld slots",
               (long long)max_len, (long long)(max_pages * cache->page));
  QLIN_REQUIRE(max_len <= kMaxDim / 2, QLIN_ERR_SHAPE, "max_len=%lld: at most 2^30", (long long)max_len);
  QLIN_REQUIRE(window >= 0, QLIN_ERR_INVALID_ARG, "window=%d is negative", window);
  QLIN_REQUIRE(scale == scale, QLIN_ERR_INVALID_ARG, "scale is NaN");
  QLIN_REQUIRE(B <= 65535, QLIN_ERR_SHAPE, "B=%lld: at most 65535", (long long)B);
  QLIN_REQUIRE(B * heads < kMaxDim, QLIN_ERR_SHAPE, "B * heads: at most 2^31 - 1");
  QLIN_DIMS(B * heads, max_len + 1);
  const bool mass = mass_out != nullptr;
  QLIN_REQUIRE(mass || mass_in == nullptr, QLIN_ERR_INVALID_ARG, "mass_in needs mass_out");
  if (mass) {
    QLIN_KV_TRACK(cache, B, ld);
    QLIN_REQUIRE(max_len <= ld, QLIN_ERR_SHAPE, "ld=%lld: at least max_len=%lld", (long long)ld, (long long)max_len);
  }
  if (B == 0) return QLIN_OK;
  QLIN_PTR(q);
  QLIN_PTR(table);
  QLIN_PTR(lens);
  QLIN_PTR(out);
  QLIN_OPT_PTR(mass_in);
  QLIN_OPT_PTR(mass_out);
  const AttnPlan p = attn_plan(*cache, heads, B, max_len, window, mass);
  const int64_t rows = B * cache->kv_heads * p.parts;
  QLIN_REQUIRE(rows < kMaxDim, QLIN_ERR_SHAPE, "B * kv_heads: fewer than 2^31");
  const dim3 grid(static_cast<unsigned>(p.groups ? p.groups : rows));
  const int join_blocks = p.groups ? heads / cache->kv_heads : 0;
  const int mass_blocks = mass ? static_cast<int>((max_len + kMassSlots - 1) / kMassSlots) : 0;
  if (p.total() > 0) QLIN_PTR(work);

  uint8_t* w = static_cast<uint8_t*>(work);
  AttnArgs a{};
  a.c = kv_pool(*cache);
  a.q = q;
  a.ld_q = ld_q;
  a.heads = heads;
  a.group = heads / cache->kv_heads;
  a.table = table;
  a.lens = lens;
  a.B = B;
  a.max_pages = max_pages;
  a.max_len = static_cast<int32_t>(max_len);
  a.window = window;
  a.scale_log2 = scale * 1.44269504088896340736f;
  a.out = out;
  a.mass_in = mass_in;
  a.mass_out = mass_out;
  a.ld_mass = ld;
  a.parts = p.parts;
  a.groups = p.groups;
  a.row_heads = p.row_heads;
  a.ld_logits = p.ld_logits;
  auto take = [&](size_t bytes) {
    uint8_t* at = bytes ? w : nullptr;
    w += bytes;
    return at;
  };
  a.runs = reinterpret_cast<int2*>(take(p.run_bytes));
  a.part_ml = reinterpret_cast<float2*>(take(p.ml_bytes));
  a.part_o = reinterpret_cast<float*>(take(p.o_bytes));
  a.head_ml = reinterpret_cast<float2*>(take(p.head_bytes));
  a.logits = reinterpret_cast<float*>(take(p.logit_bytes));
  hipStream_t st = as_stream(stream);
  if (cache->bits == 16)
    launch_bits<16>(a, cache->head_dim, grid, st);
  else if (cache->bits == 8)
    launch_bits<8>(a, cache->head_dim, grid, st);
  else
    launch_bits<4>(a, cache->head_dim, grid, st);
  QLIN_LAUNCH_CHECK("attn_kernel");
  if (join_blocks + mass_blocks > 0) {
    const dim3 jgrid(static_cast<unsigned>(join_blocks + mass_blocks), static_cast<unsigned>(cache->kv_heads),
                     static_cast<unsigned>(B));
    if (cache->head_dim == 64)
      attn_join_kernel<64><<<jgrid, kJoinThreads, 0, st>>>(a, join_blocks);
    else if (cache->head_dim == 128)
      attn_join_kernel<128><<<jgrid, kJoinThreads, 0, st>>>(a, join_blocks);
    else
      attn_join_kernel<256><<<jgrid, kJoinThreads, 0, st>>>(a, join_blocks);
    QLIN_LAUNCH_CHECK("attn_join_kernel");
  }
  return QLIN_OK;
}
