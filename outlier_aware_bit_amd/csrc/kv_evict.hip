// Eviction from the paged key/value cache by accumulated attention weight
// (qlin_kv_evict).
//
// Which slots stay is a selection of the `left` largest 32-bit keys of a row
// (sequence, kv head): one workgroup per row counts 8-bit digits from the top
// (four passes at most), then numbers the slots that leave the front and those
// that move into them.  A second launch copies the moved rows.  Attention does
// not depend on the order of slots, so only slots that stay past the new
// length move, never the whole cache: a step that evicts one slot of each head
// copies at most one row of each.
#include "kv.hpp"

namespace qlin {
namespace {

struct EvictArgs {
  KvPool c;
  const int32_t* table;
  const int32_t* lens;
  int64_t B, max_pages;
  int32_t max_len, budget, recent;
  const float* mass;
  const int32_t* pos;
  int64_t ld;
  float* mass_out;
  int32_t* pos_out;
  int32_t* lens_out;
  int32_t* kept;   // [B * heads x budget]
  int32_t* count;  // [B * heads]: moves of each row
  int32_t* from;   // [B * heads x move_cap]
  int32_t* to;
  int32_t move_cap;
};

constexpr int kSelThreads = 1024, kSelWaves = kSelThreads / 64;
constexpr int kCopies = 32;                 // of the digit counts, one per lane pair
constexpr int kKeysMax = 24576;             // keys held in LDS (96 KiB)

__device__ __forceinline__ int evict_len(const EvictArgs& a, int64_t b) {
  const int64_t cap = a.max_pages << a.c.page_shift;
  int n = a.lens[b];
  n = n < 0 ? 0 : n;
  n = n > a.max_len ? a.max_len : n;
  return n > cap ? static_cast<int>(cap) : n;
}

// Larger keys stay: the newest tokens above everything, then by mass as an
// ordered integer (-0 as +0; a NaN below everything).
__device__ __forceinline__ uint32_t evict_key(float mass, int32_t pos, int64_t newest_gone) {
  if (pos > newest_gone) return 0xffffffffu;
  if (mass != mass) return 0u;
  const uint32_t u = __builtin_bit_cast(uint32_t, add_rn(mass, 0.0f));
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// Exclusive sums over the waves of per-wave counts; every thread gets its
// wave's.  lds holds kSelWaves words; total is the whole sum.
__device__ __forceinline__ int wave_base(int count, int* lds, int& total) {
  const int w = threadIdx.x >> 6;
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[w] = count;
  __syncthreads();
  int base = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < kSelWaves; ++i) {
    const int x = lds[i];
    base += i < w ? x : 0;
    total += x;
  }
  return base;
}

template <bool KEYS_IN_LDS>
__global__ __launch_bounds__(kSelThreads) void kv_select_kernel(EvictArgs a) {
  extern __shared__ uint32_t keys[];
  __shared__ uint32_t hist[256 * kCopies];
  __shared__ uint32_t bins[256];
  __shared__ int small[kSelWaves];
  __shared__ uint32_t found[2];
  __shared__ int newest_lds[kSelWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t row = blockIdx.x;
  const int64_t b = row / a.c.heads;
  const int n = evict_len(a, b);
  const int left = min(n, a.budget);
  const float* mass = a.mass + row * a.ld;
  const int32_t* pos = a.pos + row * a.ld;
  float* mass_out = a.mass_out + row * a.ld;
  int32_t* pos_out = a.pos_out + row * a.ld;
  int32_t* kept = a.kept + row * a.budget;
  if (tid == 0 && row % a.c.heads == 0) a.lens_out[b] = left;
  for (int i = left + tid; i < a.budget; i += kSelThreads) kept[i] = -1;
  if (n <= left) {  // uniform: nothing goes
    for (int i = tid; i < n; i += kSelThreads) {
      kept[i] = i;
      mass_out[i] = mass[i];
      pos_out[i] = pos[i];
    }
    if (tid == 0) a.count[row] = 0;
    return;
  }

  int newest = INT32_MIN;
  for (int i = tid; i < n; i += kSelThreads) newest = max(newest, pos[i]);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) newest = max(newest, __shfl_xor(newest, o, 64));
  if (lane == 0) newest_lds[wave] = newest;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSelWaves; ++i) newest = max(newest, newest_lds[i]);
  const int64_t gone = static_cast<int64_t>(newest) - a.recent;  // positions up to here are not protected

  if constexpr (KEYS_IN_LDS) {
    for (int i = tid; i < n; i += kSelThreads) keys[i] = evict_key(mass[i], pos[i], gone);
  }
  auto key_of = [&](int i) { return KEYS_IN_LDS ? keys[i] : evict_key(mass[i], pos[i], gone); };

  // The left-th largest key, digit by digit: `prefix` holds the digits found,
  // `need` how many slots with that prefix stay.
  uint32_t prefix = 0;
  int need = left;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256 * kCopies; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    const uint32_t mask = shift == 24 ? 0u : ~0u << (shift + 8);
    for (int i = tid; i < n; i += kSelThreads) {
      const uint32_t k = key_of(i);
      if ((k & mask) == prefix) atomicAdd(&hist[((k >> shift) & 255u) * kCopies + (lane & (kCopies - 1))], 1u);
    }
    __syncthreads();
    {  // four threads sum a digit's copies, from different banks
      const int digit = tid >> 2, part = tid & 3;
      uint32_t s = 0;
#pragma unroll
      for (int i = 0; i < kCopies / 4; ++i) s += hist[digit * kCopies + ((part * (kCopies / 4) + i + digit) & (kCopies - 1))];
      s += __shfl_xor(s, 1, 64);
      s += __shfl_xor(s, 2, 64);
      if (part == 0) bins[digit] = s;
    }
    __syncthreads();
    if (wave == 0) {  // lane l: digits 255 - 4l .. 252 - 4l, from the top
      uint32_t c[4], sum = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[i] = bins[255 - 4 * lane - i];
        sum += c[i];
      }
      uint32_t above = sum;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const uint32_t x = __shfl_up(above, o, 64);
        above += lane >= o ? x : 0;
      }
      above -= sum;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t want = static_cast<uint32_t>(need);
        if (above < want && above + c[i] >= want) {
          found[0] = static_cast<uint32_t>(255 - 4 * lane - i);
          found[1] = want - above;
        }
        above += c[i];
      }
    }
    __syncthreads();
    prefix |= found[0] << shift;
    need = static_cast<int>(found[1]);
    // All slots with this prefix stay: the prefix, as the least key that has
    // it, already separates the rest.
    if (bins[found[0]] == found[1]) break;  // uniform
  }

  // Wave w numbers the slots of one contiguous part of the row: ties at the
  // threshold first (the lowest slots stay), then the freed front slots and the
  // slots that move.
  const int part = (n + kSelThreads - 1) / kSelThreads * 64;
  const int i0 = min(n, wave * part), i1 = min(n, i0 + part);
  int ties = 0;
  for (int i = i0 + lane; i - lane < i1; i += 64) ties += __popcll(__ballot(i < i1 && key_of(i) == prefix));
  int total;
  const uint64_t below = (uint64_t(1) << lane) - 1;
  const int tie0 = wave_base(ties, small, total);
  auto walk = [&](auto&& emit) {
    int tie = tie0;
    for (int base = i0; base < i1; base += 64) {
      const int i = base + lane;
      const uint32_t k = i < i1 ? key_of(i) : 0u;
      const bool eq = i < i1 && k == prefix;
      const uint64_t eqs = __ballot(eq);
      const bool keep = i < i1 && (k > prefix || (eq && tie + __popcll(eqs & below) < need));
      tie += __popcll(eqs);
      emit(i, keep, i < i1 && !keep && i < left, keep && i >= left);
    }
  };
  int frees = 0, moves = 0;
  walk([&](int, bool, bool free_slot, bool move) {
    frees += __popcll(__ballot(free_slot));
    moves += __popcll(__ballot(move));
  });
  int free_at = wave_base(frees, small, total);
  int move_at = wave_base(moves, small, total);
  int32_t* from = a.from + row * a.move_cap;
  int32_t* to = a.to + row * a.move_cap;
  if (tid == 0) a.count[row] = total;
  {
    int at = move_at;
    walk([&](int i, bool, bool, bool move) {
      const uint64_t ms = __ballot(move);
      if (move) from[at + __popcll(ms & below)] = i;
      at += __popcll(ms);
    });
  }
  __syncthreads();  // the row's list of moving slots is read below
  walk([&](int i, bool keep, bool free_slot, bool) {
    const uint64_t fs = __ballot(free_slot);
    int src = i;
    if (free_slot) {
      const int k = free_at + __popcll(fs & below);
      src = from[k];
      to[k] = i;
    }
    free_at += __popcll(fs);
    if (free_slot || (keep && i < left)) {
      kept[i] = src;
      mass_out[i] = mass[src];
      pos_out[i] = pos[src];
    }
  });
}

constexpr int kMoveThreads = 256;

// LANES lanes copy a moved slot: the K row's 16-byte pieces, then the V row's.
template <int RB>
__global__ __launch_bounds__(kMoveThreads) void kv_move_kernel(EvictArgs a) {
  constexpr int HALF = RB / 16, LANES = 2 * HALF;
  const int64_t row = blockIdx.x;
  const int64_t b = row / a.c.heads;
  const int h = static_cast<int>(row % a.c.heads);
  const int count = a.count[row];
  const int ps = a.c.page_shift, mask = (1 << ps) - 1;
  const int l = threadIdx.x % LANES;
  const int32_t* table = a.table + b * a.max_pages;
  const int step = static_cast<int>(gridDim.y) * (kMoveThreads / LANES);
  for (int i = blockIdx.y * (kMoveThreads / LANES) + threadIdx.x / LANES; i < count; i += step) {
    const int src = a.from[row * a.move_cap + i], dst = a.to[row * a.move_cap + i];
    const int64_t sp = table[src >> ps], dp = table[dst >> ps];
    if (sp < 0 || sp >= a.c.pages || dp < 0 || dp >= a.c.pages) continue;
    const int64_t s = ((sp * a.c.heads + h) << ps) + (src & mask), d = ((dp * a.c.heads + h) << ps) + (dst & mask);
    uint8_t* p = l < HALF ? a.c.k : a.c.v;
    const int piece = l < HALF ? l : l - HALF;
    reinterpret_cast<uint4*>(p + d * RB)[piece] = reinterpret_cast<const uint4*>(p + s * RB)[piece];
    if (a.c.kmeta != nullptr && piece == 0) {
      uint32_t* meta = l < HALF ? a.c.kmeta : a.c.vmeta;
      meta[d] = meta[s];
    }
  }
}

template <int RB>
void launch_move(const EvictArgs& a, int64_t rows, hipStream_t st) {
  const int per = kMoveThreads / (RB / 8);
  // A workgroup goes over several moves of its row when there are many.
  const int64_t most = (a.move_cap + per - 1) / per;
  const int64_t want = (4096 + rows - 1) / rows;
  const dim3 grid(static_cast<unsigned>(rows), static_cast<unsigned>(most < want ? most : want));
  kv_move_kernel<RB><<<grid, kMoveThreads, 0, st>>>(a);
}

// At most this many slots of a row move: each fills a slot below the budget
// and comes from one past it.
inline int64_t evict_move_cap(int64_t max_len, int64_t budget) {
  const int64_t over = max_len > budget ? max_len - budget : 0;
  return over < budget ? over : budget;
}

inline size_t evict_count_bytes(int64_t rows) { return (static_cast<size_t>(rows) * 4 + 255) / 256 * 256; }

}  // namespace
}  // namespace qlin

using namespace qlin;

extern "C" size_t qlin_kv_evict_work_bytes(const qlin_kv_cache* cache, int64_t B, int64_t max_len, int32_t budget) {
  if (!kv_shape_ok(cache) || B < 1 || B >= kMaxDim / cache->kv_heads || max_len < 0 || max_len >= kMaxDim - 1 ||
      budget < 0 || !dims_ok(B * cache->kv_heads, max_len + 1))
    return 0;
  const int64_t rows = B * cache->kv_heads;
  return evict_count_bytes(rows) + static_cast<size_t>(rows) * evict_move_cap(max_len, budget) * 8;
}

extern "C" qlin_status qlin_kv_evict(const qlin_kv_cache* cache, const int32_t* table, const int32_t* lens, int64_t B,
                                     int64_t max_pages, int64_t max_len, int32_t budget, int32_t recent,
                                     const float* mass, const int32_t* pos, int64_t ld, float* mass_out,
                                     int32_t* pos_out, int32_t* lens_out, int32_t* kept, void* work, void* stream) {
  QLIN_KV_CACHE(cache);
  QLIN_KV_TABLE(cache, B, max_pages);
  QLIN_REQUIRE(max_len >= 0, QLIN_ERR_INVALID_ARG, "max_len=%lld is negative", (long long)max_len);
  QLIN_REQUIRE(max_len <= max_pages * cache->page, QLIN_ERR_SHAPE, "max_len=%lld: the table holds %lld slots",
               (long long)max_len, (long long)(max_pages * cache->page));
  QLIN_REQUIRE(budget >= 1, QLIN_ERR_INVALID_ARG, "budget=%d must be at least 1", budget);
  QLIN_REQUIRE(recent >= 0 && recent <= budget, QLIN_ERR_INVALID_ARG, "recent=%d must be in [0, budget]", recent);
  QLIN_KV_TRACK(cache, B, ld);
  QLIN_REQUIRE(max_len <= ld, QLIN_ERR_SHAPE, "ld=%lld: at least max_len=%lld", (long long)ld, (long long)max_len);
  QLIN_REQUIRE(B < kMaxDim / cache->kv_heads, QLIN_ERR_SHAPE, "B * kv_heads: fewer than 2^31");
  QLIN_DIMS(B * cache->kv_heads, budget);
  if (B == 0) return QLIN_OK;
  QLIN_PTR(table);
  QLIN_PTR(lens);
  QLIN_PTR(mass);
  QLIN_PTR(pos);
  QLIN_PTR(mass_out);
  QLIN_PTR(pos_out);
  QLIN_PTR(lens_out);
  QLIN_PTR(kept);
  QLIN_PTR(work);
  const int64_t rows = B * cache->kv_heads;
  EvictArgs a{};
  a.c = kv_pool(*cache);
  a.table = table;
  a.lens = lens;
  a.B = B;
  a.max_pages = max_pages;
  a.max_len = static_cast<int32_t>(max_len);
  a.budget = budget;
  a.recent = recent;
  a.mass = mass;
  a.pos = pos;
  a.ld = ld;
  a.mass_out = mass_out;
  a.pos_out = pos_out;
  a.lens_out = lens_out;
  a.kept = kept;
  a.move_cap = static_cast<int32_t>(evict_move_cap(max_len, budget));
  uint8_t* w = static_cast<uint8_t*>(work);
  a.count = reinterpret_cast<int32_t*>(w);
  a.from = reinterpret_cast<int32_t*>(w + evict_count_bytes(rows));
  a.to = a.from + rows * a.move_cap;
  hipStream_t st = as_stream(stream);
  if (max_len <= kKeysMax)
    kv_select_kernel<true><<<dim3(static_cast<unsigned>(rows)), kSelThreads, static_cast<size_t>(max_len) * 4, st>>>(a);
  else
    kv_select_kernel<false><<<dim3(static_cast<unsigned>(rows)), kSelThreads, 0, st>>>(a);
  QLIN_LAUNCH_CHECK("kv_select_kernel");
  if (a.move_cap > 0) {
    switch (cache->head_dim * cache->bits / 8) {
      case 32: launch_move<32>(a, rows, st); break;
      case 64: launch_move<64>(a, rows, st); break;
      case 128: launch_move<128>(a, rows, st); break;
      case 256: launch_move<256>(a, rows, st); break;
      default: launch_move<512>(a, rows, st); break;
    }
    QLIN_LAUNCH_CHECK("kv_move_kernel");
  }
  return QLIN_OK;
}
