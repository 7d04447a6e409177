// Attention of one new token over the paged key/value cache (qlin_attn_decode).
//
// Per sequence and kv head, with up to eight of the group's query heads:
//   S = K q^T   (slots x heads),   P = exp2(S - m),   O^T = V^T P^T  (D x heads)
// on 16x16x32 fp16 matrix instructions, whose 16 columns hold every head twice:
// columns 8 .. 15 carry what rounding P (and a rotated q) to fp16 left over, so
// that both products are good to 2^-21 for no further matrix instruction.
// Both results hold a head in lane & 7, so the softmax state and the rescaling
// of O never leave the lane, and P comes
// out of the first product in the registers where the second one takes it: the
// eight slots 8g .. 8g + 7 of lane group g = lane >> 4 are one k-group of the
// second product.  K rows are read as its A operand directly; V rows are read
// eight slots by D / 16 channels per lane and transposed in registers by byte
// permutes.  Nothing of K, V, S or P goes through LDS.
//
// The cache is split over its length: a workgroup takes `chunk` slots of one
// kv head, its four waves 32 * U slots at a time; a second launch joins the
// chunks of a head by their maxima and sums (none when one chunk is enough).
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
  int32_t chunk, splits, head_tiles;
  float* part_o;    // [B * heads x splits x D] (splits > 1)
  float2* part_ml;  // [B * heads x splits]: reference exponent and sum
  float* logits;    // [B * heads x ld_logits], log2 domain (with mass)
  int64_t ld_logits;
};

constexpr int kAttnWaves = 4;
constexpr int kAttnThreads = 64 * kAttnWaves;
constexpr int kMaxChunk = 2048;
constexpr int kTileHeads = 8;  // query heads of a workgroup

// A wave's exponent reference m starts below any finite logit.
constexpr float kNoRef = -3.0e38f;
// exp2(s - m) reaches 2^kTop at the maximum that m was set from and may grow to
// 2^kCeil before m is moved, so fp16 holds it (below 2^16) and slots down to
// 2^-(24 + kTop) of that maximum still count.
constexpr float kTop = 7.0f, kCeil = 15.0f;

__device__ __forceinline__ v8h as_v8h(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const v4i w = {static_cast<int>(a), static_cast<int>(b), static_cast<int>(c), static_cast<int>(d)};
  return __builtin_bit_cast(v8h, w);
}

__device__ __forceinline__ float lo_half(uint32_t w) { return h2f(static_cast<uint16_t>(w)); }
__device__ __forceinline__ float hi_half(uint32_t w) { return h2f(static_cast<uint16_t>(w >> 16)); }

__device__ __forceinline__ float max_groups(float v) {  // over the four lane groups of a head
  v = fmaxf(v, __shfl_xor(v, 16, 64));
  return fmaxf(v, __shfl_xor(v, 32, 64));
}
__device__ __forceinline__ float sum_groups(float v) {
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

// First slot that row b attends to, and one past the last.
__device__ __forceinline__ void attn_range(const AttnArgs& a, int64_t b, int& low, int& n) {
  const int64_t cap = a.max_pages << a.c.page_shift;
  n = a.lens[b];
  n = n < 0 ? 0 : n;
  n = n > a.max_len ? a.max_len : n;
  n = n > cap ? static_cast<int>(cap) : n;
  low = (a.window > 0 && n > a.window) ? n - a.window : 0;
}
// The chunks of a row start at the 32-slot block of its first slot.
__device__ __forceinline__ int attn_base(int low) { return low & ~31; }

// Codes enter the matrix products as fp16 denormals, code * 2^-24, which the
// matrix instructions keep exactly: an AND or a byte permute then makes an
// operand, and 2^24 goes into the row's step.  The second and fourth nibble of
// a 16-bit half stay where they are, 16 times larger; the first product
// divides q by 16 there, the second one its result.
template <int BITS>
struct Codes {
  static constexpr float unit = 16777216.0f;  // 2^24
  static constexpr float mid = (BITS == 4) ? 7.5f : 127.5f;
};

template <int BITS, int D, bool ROT, bool LOGITS>
struct Attn {
  static constexpr int RB = D * BITS / 8;                  // bytes of a stored row
  static constexpr int U = (BITS == 4 && D <= 128) ? 2 : 1;  // 32-slot blocks of a wave at a time
  static constexpr int KS = D / 32;                        // k steps of the first product
  static constexpr int NT = D / 16;                        // channel tiles of the second
  static constexpr int KW = RB / 16;                       // dwords of K of a lane and row
  static constexpr int DPL = D / 16;                       // channels of V of a lane and row
  static constexpr int VW = (DPL * BITS + 31) / 32;        // dwords of them
  static constexpr int VC = VW > 4 ? 2 : 1;                // 16-byte pieces of them, D / VC channels apart
  static constexpr int DPC = DPL / VC;
  static constexpr bool QUANT = BITS < 16;

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
      const uint32_t y = (t & 2) ? w >> 8 : w;
      return y & ((t & 1) ? 0x00f000f0u : 0x000f000fu);
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

// Bytes of the split kernel's dynamic LDS: the row indices of the chunk's
// pages, and either the rotated q or the waves' results, whichever is larger.
constexpr int kIdBytes = (kMaxChunk / 16 + 1) * 8 + 8;
constexpr int kMlBytes = kAttnWaves * kTileHeads * 8;
inline size_t attn_lds(int D, int group, bool rot) {
  const int hs = group < kTileHeads ? group : kTileHeads;
  const size_t o = static_cast<size_t>(kAttnWaves) * hs * (D + 4) * sizeof(float);
  const size_t qr = rot ? kTileHeads * 128 * sizeof(float) : 0;
  return kIdBytes + kMlBytes + (o > qr ? o : qr);
}

template <int BITS, int D, bool ROT, bool LOGITS>
__global__ __launch_bounds__(kAttnThreads) void attn_split_kernel(AttnArgs a) {
  using A = Attn<BITS, D, ROT, LOGITS>;
  constexpr int RB = A::RB, U = A::U, KS = A::KS, NT = A::NT, KW = A::KW, VW = A::VW;
  constexpr bool QUANT = A::QUANT;
  extern __shared__ uint8_t lds[];
  int64_t* ids = reinterpret_cast<int64_t*>(lds);                      // row index of each page, or -1
  float2* lds_ml = reinterpret_cast<float2*>(lds + kIdBytes);          // [wave][kTileHeads]
  float* lds_o = reinterpret_cast<float*>(lds + kIdBytes + kMlBytes);  // [wave][head][D + 4]

  // Head tiles of one chunk are eight workgroups apart: the same XCD's cache.
  const int64_t idx = blockIdx.x;
  const int64_t rest = idx / (8 * a.head_tiles) * 8 + (idx & 7);
  const int ht = static_cast<int>((idx >> 3) % a.head_tiles);
  if (rest >= a.B * a.c.heads * a.splits) return;
  const int split = static_cast<int>(rest % a.splits);
  const int64_t bh = rest / a.splits;
  const int h = static_cast<int>(bh % a.c.heads);
  const int64_t b = bh / a.c.heads;
  int low, n;
  attn_range(a, b, low, n);
  const int c0 = attn_base(low) + split * a.chunk;
  const int hs = min(kTileHeads, a.group - kTileHeads * ht);  // query heads here
  const int hfirst = h * a.group + kTileHeads * ht;           // the first of them
  const int64_t head0 = b * a.heads + hfirst;
  if (c0 >= n) {  // uniform
    if (a.splits == 1)
      for (int i = threadIdx.x; i < hs * D; i += kAttnThreads) a.out[head0 * D + i] = 0;
    return;
  }
  const int end = min(n, c0 + a.chunk);

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane >> 4, col = lane & 15;
  const int ps = a.c.page_shift, line_mask = (1 << ps) - 1;
  const int page0 = c0 >> ps, page_count = ((end - 1) >> ps) - page0 + 1;
  for (int i = threadIdx.x; i < page_count; i += kAttnThreads) {
    const int32_t id = a.table[b * a.max_pages + page0 + i];
    ids[i] = (id >= 0 && id < a.c.pages) ? (static_cast<int64_t>(id) * a.c.heads + h) << ps : -1;
  }

  // q in the operand order of the first product, and sum_d q_d for the rows'
  // lo.  Columns 8 .. 15: the same q, or what fp16 leaves of a rotated one.
  const int hcol = col & 7, rem = col >> 3;
  const float frem = static_cast<float>(rem);
  v8h qf[KS];
  float qsum = 0.0f;
  constexpr int SPP = A::EPP / 8;  // k steps of a piece
  if constexpr (ROT) {
    float* q_lds = lds_o;  // [head][128]
    const int hd = threadIdx.x >> 4, c = threadIdx.x & 15;
    if (hd < kTileHeads) {  // uniform per wave
      float u[8];
      const int hq = hd < hs ? hd : 0;
      const v4i raw = *reinterpret_cast<const v4i*>(a.q + b * a.ld_q + (hfirst + hq) * D + 8 * c);
      signed8(raw, a.c.signs + 8 * c, u);
      hadamard128(u, c);
#pragma unroll
      for (int i = 0; i < 8; ++i) q_lds[hd * 128 + 8 * c + i] = hd < hs ? u[i] * 0.0078125f : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int d0 = A::k_channel(s / SPP, g) + 8 * (s % SPP);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float x = q_lds[hcol * 128 + d0 + A::k_order(i)];
        qsum += x;
        if (BITS == 4 && (i & 2)) x *= 0.0625f;
        const _Float16 hi = static_cast<_Float16>(x);
        qf[s][i] = rem ? static_cast<_Float16>(x - static_cast<float>(hi)) : hi;
      }
    }
  } else {
    const bool here = hcol < hs;
    const uint16_t* qp = a.q + b * a.ld_q + (hfirst + (here ? hcol : 0)) * D;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const v8h raw = *reinterpret_cast<const v8h*>(qp + A::k_channel(s / SPP, g) + 8 * (s % SPP));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const _Float16 x = here ? raw[A::k_order(i)] : static_cast<_Float16>(0.0f);
        if constexpr (QUANT) qsum += static_cast<float>(x);
        qf[s][i] = (BITS == 4 && (i & 2)) ? x * static_cast<_Float16>(0.0625f) : x;
      }
    }
  }
  if constexpr (QUANT) qsum = sum_groups(qsum) * a.scale_log2;
  const float qscale = QUANT ? a.scale_log2 * Codes<BITS>::unit : a.scale_log2;
  __syncthreads();  // ids

  v4f o[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) o[t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  v4f psum = {0.0f, 0.0f, 0.0f, 0.0f};  // sum of the rounded P, for the codes' midpoint
  float m = kNoRef, l = 0.0f, omid = 0.0f, inv_ref = 0.0f, ref = 0.0f;

  const int krun = col >> 2, kline = col & 3;
  for (int base = c0 + wave * 32 * U; base < end; base += kAttnWaves * 32 * U) {  // uniform per wave
    // Slots beyond the last page read another row of the same page, whose
    // values are dropped below.
    uint32_t kw[U][2][KW], vw[U][8][VW], km[QUANT ? U : 1][8], vm[QUANT ? U : 1][8];
    bool run_ok[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int ks = base + 32 * u + 8 * krun, vs = base + 32 * u + 8 * g;
      const int64_t ki = ids[min((ks >> ps) - page0, page_count - 1)];
      const int64_t vi = ids[min((vs >> ps) - page0, page_count - 1)];
      run_ok[u] = vi >= 0;
      const int64_t krow = (ki < 0 ? 0 : ki) + (ks & line_mask) + kline;
      const int64_t vrow = (vi < 0 ? 0 : vi) + (vs & line_mask);
      const uint8_t* kp = a.c.k + krow * RB + (RB == 32 ? 8 : 16) * g;
      const uint8_t* vp = a.c.v + vrow * RB + col * (RB / 16 / A::VC);
      A::load_k(kp, kw[u][0]);
      A::load_k(kp + 4 * RB, kw[u][1]);
      if constexpr (QUANT) {
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          const uint4 x = *reinterpret_cast<const uint4*>(a.c.kmeta + vrow + i);
          km[u][i] = x.x, km[u][i + 1] = x.y, km[u][i + 2] = x.z, km[u][i + 3] = x.w;
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) A::load_v(vp + i * RB, vw[u][i]);
      if constexpr (QUANT) {
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          const uint4 x = *reinterpret_cast<const uint4*>(a.c.vmeta + vrow + i);
          vm[u][i] = x.x, vm[u][i + 1] = x.y, vm[u][i + 2] = x.z, vm[u][i + 3] = x.w;
        }
      }
    }

    float s[U][8];
    float smax = -INFINITY;
    bool whole = base >= low && base + 32 * U <= end;
#pragma unroll
    for (int u = 0; u < U; ++u) whole = whole && run_ok[u];
    const bool all_whole = __all(whole);
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const v8h kf = A::k_operand(kw[u][t], k);
          acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[k], acc, 0, 0, 0);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if constexpr (ROT) acc[r] += lane_xor<8>(acc[r]);
          const int i = 4 * t + r;
          if constexpr (QUANT)
            s[u][i] = __builtin_fmaf(acc[r], lo_half(km[u][i]) * qscale, hi_half(km[u][i]) * qsum);
          else
            s[u][i] = acc[r] * qscale;
        }
      }
    }
    if (!all_whole) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int slot = base + 32 * u + 8 * g + i;
          const bool ok = run_ok[u] && slot >= low && slot < end;
          s[u][i] = ok ? s[u][i] : -INFINITY;
#pragma unroll
          for (int w = 0; w < VW; ++w) vw[u][i][w] = ok ? vw[u][i][w] : 0u;
          if constexpr (QUANT) vm[u][i] = ok ? vm[u][i] : 0u;
        }
      }
    }
    if constexpr (LOGITS) {
      if (col < hs) {
        float* lp = a.logits + (head0 + col) * a.ld_logits + base + 8 * g;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (base + 32 * u + 8 * g < a.ld_logits) {
            *reinterpret_cast<float4*>(lp + 32 * u) = make_float4(s[u][0], s[u][1], s[u][2], s[u][3]);
            *reinterpret_cast<float4*>(lp + 32 * u + 4) = make_float4(s[u][4], s[u][5], s[u][6], s[u][7]);
          }
        }
      }
    }
    float vmax = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        smax = fmaxf(smax, s[u][i]);
        if constexpr (QUANT) vmax = fmaxf(vmax, lo_half(vm[u][i]));
      }
    }
    // The references move only when a weight would leave fp16's range.
    bool move = smax > m + kCeil;
    if constexpr (QUANT) move = move || vmax * inv_ref > 1.0f || ref == 0.0f;
    if (__any(move)) {
      const float top = max_groups(smax);
      const float mn = top > m + kCeil ? top - kTop : m;
      float alpha = __builtin_amdgcn_exp2f(m - mn), beta = alpha;
      if constexpr (QUANT) {
        // A power of two at least four times the largest step so far.
        float big = max_groups(vmax);
        big = __shfl(big, 0, 64);
        if (!(big * inv_ref <= 1.0f) || ref == 0.0f) {
          const int e = big > 0.0f ? static_cast<int>((__builtin_bit_cast(uint32_t, big) >> 23) & 255u) - 127 + 3 : -24;
          const float nr = __builtin_bit_cast(float, static_cast<uint32_t>(e + 127) << 23);
          const float ni = __builtin_bit_cast(float, static_cast<uint32_t>(127 - e) << 23);
          beta *= ref * ni;
          ref = nr;
          inv_ref = ni;
        }
      }
      l *= alpha;
      omid *= alpha;
      m = mn;
#pragma unroll
      for (int t = 0; t < NT; ++t) o[t] *= beta;
      psum *= beta;
    }

#pragma unroll
    for (int u = 0; u < U; ++u) {
      float w[8];
      v8h p;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float e = __builtin_amdgcn_exp2f(s[u][i] - m);
        l += e;
        if constexpr (QUANT) {
          // The step goes into the weight, the codes' midpoint apart.
          const float step = lo_half(vm[u][i]);
          omid = __builtin_fmaf(e, __builtin_fmaf(step, Codes<BITS>::mid, hi_half(vm[u][i])), omid);
          w[i] = e * (step * inv_ref);
        } else {
          w[i] = e;
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = static_cast<_Float16>(w[i]);
      // Columns 8 .. 15 take the remainders.
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = static_cast<_Float16>(__builtin_fmaf(-frem, static_cast<float>(p[i]), w[i]));
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const v8h vf = as_v8h(A::v_pair(vw[u][0], vw[u][1], t), A::v_pair(vw[u][2], vw[u][3], t),
                              A::v_pair(vw[u][4], vw[u][5], t), A::v_pair(vw[u][6], vw[u][7], t));
        o[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, p, o[t], 0, 0, 0);
      }
      if constexpr (QUANT) {
        const v8h ones = as_v8h(0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u);
        psum = __builtin_amdgcn_mfma_f32_16x16x32_f16(ones, p, psum, 0, 0, 0);
      }
    }
  }

  // The wave's sums in the values' own units.
  l = sum_groups(l);
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int r = 0; r < 4; ++r) o[t][r] += lane_xor<8>(o[t][r]);
  }
  if constexpr (QUANT) {
    omid = sum_groups(omid) - (psum[0] + lane_xor<8>(psum[0])) * (ref * Codes<BITS>::mid);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float unit = ref * ((BITS == 4 && (t & 1)) ? Codes<BITS>::unit / 16.0f : Codes<BITS>::unit);
#pragma unroll
      for (int r = 0; r < 4; ++r) o[t][r] = __builtin_fmaf(o[t][r], unit, omid);
    }
  }
  if (lane < kTileHeads) lds_ml[wave * kTileHeads + lane] = make_float2(m, l);
  if (col < hs) {
    float* dst = lds_o + (wave * hs + col) * (D + 4);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int r = 0; r < 4; ++r) dst[A::v_channel(t, 4 * g + r)] = o[t][r];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < hs * D; i += kAttnThreads) {
    const int hd = i / D, d = i % D;
    float mx = kNoRef;
#pragma unroll
    for (int w = 0; w < kAttnWaves; ++w) mx = fmaxf(mx, lds_ml[w * kTileHeads + hd].x);
    float sum = 0.0f, acc = 0.0f;
#pragma unroll
    for (int w = 0; w < kAttnWaves; ++w) {
      const float2 ml = lds_ml[w * kTileHeads + hd];
      const float f = __builtin_amdgcn_exp2f(ml.x - mx);
      sum = __builtin_fmaf(ml.y, f, sum);
      acc = __builtin_fmaf(lds_o[(w * hs + hd) * (D + 4) + d], f, acc);
    }
    if (a.splits == 1) a.out[(head0 + hd) * D + d] = f2h(sum == 0.0f ? 0.0f : div_rn(acc, sum));
    if (a.splits > 1) a.part_o[((head0 + hd) * a.splits + split) * D + d] = acc;
    if (d == 0 && a.part_ml != nullptr) a.part_ml[(head0 + hd) * a.splits + split] = make_float2(mx, sum);
  }
}

// Joins the chunks of a head (blocks below B * heads, when there are several),
// then adds the heads' weights of each slot to mass (the other blocks).
constexpr int kJoinThreads = 256;
constexpr int kMassSlots = 1024;

template <int D>
__global__ __launch_bounds__(kJoinThreads) void attn_join_kernel(AttnArgs a, int64_t join_blocks, int mass_blocks) {
  __shared__ float4 acc_lds[kJoinThreads];
  __shared__ float red[kJoinThreads / 64];
  __shared__ float sums[16];  // ROWS of them: 16, 8 or 4
  __shared__ float2 head_ml[16];
  const int tid = threadIdx.x;
  if (blockIdx.x < join_blocks) {
    const int64_t head = blockIdx.x;  // b * heads + query head
    int low, n;
    attn_range(a, head / a.heads, low, n);
    const int used = n <= 0 ? 0 : (n - attn_base(low) + a.chunk - 1) / a.chunk;
    const float2* ml = a.part_ml + head * a.splits;
    float mx = kNoRef;
    for (int i = tid; i < used; i += kJoinThreads) mx = fmaxf(mx, ml[i].x);
    mx = wave_max(mx);
    if ((tid & 63) == 0) red[tid >> 6] = mx;
    __syncthreads();
    mx = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    constexpr int LANES = D / 4, ROWS = kJoinThreads / LANES;
    const int d4 = tid % LANES, r0 = tid / LANES;
    const float4* po = reinterpret_cast<const float4*>(a.part_o + head * a.splits * D) + d4;
    float sum = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i = r0; i < used; i += ROWS) {
      const float2 x = ml[i];
      const float f = __builtin_amdgcn_exp2f(x.x - mx);
      const float4 v = po[static_cast<int64_t>(i) * LANES];
      sum = __builtin_fmaf(x.y, f, sum);
      acc.x = __builtin_fmaf(v.x, f, acc.x);
      acc.y = __builtin_fmaf(v.y, f, acc.y);
      acc.z = __builtin_fmaf(v.z, f, acc.z);
      acc.w = __builtin_fmaf(v.w, f, acc.w);
    }
    acc_lds[tid] = acc;
    if (d4 == 0) sums[r0] = sum;
    __syncthreads();
    if (tid < LANES) {
      float total = 0.0f;
      float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        const float4 v = acc_lds[i * LANES + tid];
        total += sums[i];
        t.x += v.x, t.y += v.y, t.z += v.z, t.w += v.w;
      }
      const bool none = total == 0.0f;
      uint2 w;
      w.x = f2h(none ? 0.0f : div_rn(t.x, total)) | static_cast<uint32_t>(f2h(none ? 0.0f : div_rn(t.y, total))) << 16;
      w.y = f2h(none ? 0.0f : div_rn(t.z, total)) | static_cast<uint32_t>(f2h(none ? 0.0f : div_rn(t.w, total))) << 16;
      reinterpret_cast<uint2*>(a.out + head * D)[tid] = w;
    }
    return;
  }
  // mass of slots [s0, s0 + kMassSlots) of one (row, kv head)
  const int64_t idx = blockIdx.x - join_blocks;
  const int64_t bh = idx / mass_blocks;
  const int s0 = static_cast<int>(idx % mass_blocks) * kMassSlots;
  const int64_t b = bh / a.c.heads;
  const int h = static_cast<int>(bh % a.c.heads);
  int low, n;
  attn_range(a, b, low, n);
  if (s0 >= n) return;  // uniform
  const int base = attn_base(low);
  const int used = (n - base + a.chunk - 1) / a.chunk;
  const int64_t head0 = b * a.heads + h * a.group;
  float w[kMassSlots / kJoinThreads];
#pragma unroll
  for (int i = 0; i < kMassSlots / kJoinThreads; ++i) w[i] = 0.0f;
  for (int h0 = 0; h0 < a.group; h0 += 16) {
    const int hs = min(16, a.group - h0);
    __syncthreads();
    // Each wave takes heads in turn: maximum, then sum, over the chunks.
    for (int hd = tid >> 6; hd < hs; hd += kJoinThreads / 64) {
      const float2* ml = a.part_ml + (head0 + h0 + hd) * a.splits;
      float mx = kNoRef;
      for (int i = tid & 63; i < used; i += 64) mx = fmaxf(mx, ml[i].x);
      mx = wave_max(mx);
      float sum = 0.0f;
      for (int i = tid & 63; i < used; i += 64) sum = __builtin_fmaf(ml[i].y, __builtin_amdgcn_exp2f(ml[i].x - mx), sum);
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o, 64);
      if ((tid & 63) == 0) head_ml[hd] = make_float2(mx, sum == 0.0f ? 0.0f : div_rn(1.0f, sum));
    }
    __syncthreads();
    for (int hd = 0; hd < hs; ++hd) {
      const float2 ml = head_ml[hd];
      const float* lp = a.logits + (head0 + h0 + hd) * a.ld_logits;
#pragma unroll
      for (int i = 0; i < kMassSlots / kJoinThreads; ++i) {
        const int slot = s0 + i * kJoinThreads + tid;
        if (slot >= low && slot < n) w[i] = __builtin_fmaf(__builtin_amdgcn_exp2f(lp[slot] - ml.x), ml.y, w[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kMassSlots / kJoinThreads; ++i) {
    const int slot = s0 + i * kJoinThreads + tid;
    if (slot < n && slot < a.ld_mass) {
      const int64_t at = bh * a.ld_mass + slot;
      a.mass_out[at] = (a.mass_in != nullptr ? a.mass_in[at] : 0.0f) + w[i];
    }
  }
}

struct AttnPlan {
  int chunk, splits, head_tiles;
  int64_t ld_logits;
  size_t o_bytes, ml_bytes, logit_bytes;
};

// Slots a wave takes at a time, times the waves: the unit of a chunk.
inline int attn_unit(const qlin_kv_cache& c) { return kAttnWaves * 32 * ((c.bits == 4 && c.head_dim <= 128) ? 2 : 1); }

AttnPlan attn_plan(const qlin_kv_cache& c, int32_t heads, int64_t B, int64_t max_len, int32_t window, bool mass) {
  AttnPlan p;
  const int group = heads / c.kv_heads;
  p.head_tiles = (group + kTileHeads - 1) / kTileHeads;
  // A window may begin 31 slots into its first 32-slot block.
  int64_t span = max_len;
  if (window > 0 && window + 31 < span) span = window + 31;
  if (span < 1) span = 1;
  const int unit = attn_unit(c);
  // Workgroups for every CU several times over, so that ragged rows even out;
  // but no chunk below two units, where the fixed work would show, and none
  // above kMaxChunk.
  const int64_t rows = B * c.kv_heads * p.head_tiles;
  int64_t chunk = (span * rows + 2047) / 2048;
  chunk = (chunk + unit - 1) / unit * unit;
  if (chunk < 2 * unit) chunk = 2 * unit;
  if (chunk > kMaxChunk) chunk = kMaxChunk;
  p.chunk = static_cast<int>(chunk);
  p.splits = static_cast<int>((span + chunk - 1) / chunk);
  const size_t n = static_cast<size_t>(B) * heads;
  p.o_bytes = p.splits > 1 ? n * p.splits * c.head_dim * sizeof(float) : 0;
  p.ml_bytes = (p.splits > 1 || mass) ? (n * p.splits * sizeof(float2) + 255) / 256 * 256 : 0;
  p.ld_logits = (max_len + 31) / 32 * 32;
  p.logit_bytes = mass ? n * static_cast<size_t>(p.ld_logits) * sizeof(float) : 0;
  return p;
}

template <int BITS, int D, bool ROT>
void launch_split(const AttnArgs& a, int64_t blocks, hipStream_t st) {
  const size_t lds = attn_lds(D, a.group, ROT);
  const dim3 grid(static_cast<unsigned>(blocks));
  if (a.logits != nullptr)
    attn_split_kernel<BITS, D, ROT, true><<<grid, kAttnThreads, lds, st>>>(a);
  else
    attn_split_kernel<BITS, D, ROT, false><<<grid, kAttnThreads, lds, st>>>(a);
}

template <int BITS>
void launch_bits(const AttnArgs& a, int D, int64_t blocks, hipStream_t st) {
  if (D == 64) return launch_split<BITS, 64, false>(a, blocks, st);
  if (D == 256) return launch_split<BITS, 256, false>(a, blocks, st);
  if constexpr (BITS < 16) {
    if (a.c.signs != nullptr) return launch_split<BITS, 128, true>(a, blocks, st);
  }
  launch_split<BITS, 128, false>(a, blocks, st);
}

}  // namespace
}  // namespace qlin

using namespace qlin;

extern "C" size_t qlin_attn_decode_work_bytes(const qlin_kv_cache* cache, int32_t heads, int64_t B, int64_t max_len,
                                              int32_t window, int32_t mass) {
  if (!kv_shape_ok(cache) || heads < 1 || heads % cache->kv_heads != 0 || B < 1 || max_len < 0 || window < 0 ||
      !dims_ok(B, max_len) || !dims_ok(B * heads, max_len + 1) || !dims_ok(B * heads, cache->head_dim))
    return 0;
  const AttnPlan p = attn_plan(*cache, heads, B, max_len, window, mass != 0);
  return p.o_bytes + p.ml_bytes + p.logit_bytes;
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
  QLIN_REQUIRE(window >= 0, QLIN_ERR_INVALID_ARG, "window=%d is negative", window);
  QLIN_REQUIRE(scale == scale, QLIN_ERR_INVALID_ARG, "scale is NaN");
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
  const int64_t rest = B * cache->kv_heads * p.splits;
  const int64_t blocks = p.head_tiles == 1 ? rest : (rest + 7) / 8 * 8 * p.head_tiles;
  const int mass_blocks = static_cast<int>((max_len + kMassSlots - 1) / kMassSlots);
  const int64_t join = p.splits > 1 ? B * heads : 0;
  const int64_t join_blocks = join + (mass ? B * cache->kv_heads * mass_blocks : 0);
  QLIN_REQUIRE(blocks < kMaxDim && join_blocks < kMaxDim, QLIN_ERR_SHAPE, "B * heads * max_len too large");
  if (p.o_bytes + p.ml_bytes + p.logit_bytes > 0) QLIN_PTR(work);

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
  a.chunk = p.chunk;
  a.splits = p.splits;
  a.head_tiles = p.head_tiles;
  a.part_o = p.o_bytes ? reinterpret_cast<float*>(w) : nullptr;
  a.part_ml = p.ml_bytes ? reinterpret_cast<float2*>(w + p.o_bytes) : nullptr;
  a.logits = p.logit_bytes ? reinterpret_cast<float*>(w + p.o_bytes + p.ml_bytes) : nullptr;
  a.ld_logits = p.ld_logits;
  hipStream_t st = as_stream(stream);
  if (cache->bits == 16)
    launch_bits<16>(a, cache->head_dim, blocks, st);
  else if (cache->bits == 8)
    launch_bits<8>(a, cache->head_dim, blocks, st);
  else
    launch_bits<4>(a, cache->head_dim, blocks, st);
  QLIN_LAUNCH_CHECK("attn_split_kernel");
  if (join_blocks > 0) {
    const dim3 grid(static_cast<unsigned>(join_blocks));
    if (cache->head_dim == 64)
      attn_join_kernel<64><<<grid, kJoinThreads, 0, st>>>(a, join, mass_blocks);
    else if (cache->head_dim == 128)
      attn_join_kernel<128><<<grid, kJoinThreads, 0, st>>>(a, join, mass_blocks);
    else
      attn_join_kernel<256><<<grid, kJoinThreads, 0, st>>>(a, join, mass_blocks);
    QLIN_LAUNCH_CHECK("attn_join_kernel");
  }
  return QLIN_OK;
}
