// Eviction from the paged key/value cache by accumulated attention weight
// (qlin_kv_evict).
//
// Which slots stay is a selection of the `left` largest 32-bit keys of a row
// (sequence, kv head): one workgroup per row counts 8-bit digits from the top
// (four passes at most), then numbers the slots that leave the front and those
// that move into them.  A second launch copies the moved rows.  Attention does
// not depend on the order of slots, so only slots that stay past the new
// length move, never the whole cache: a step that evicts one slot of each head
// copies at most one row of each.  A row with slots that do not exist, or with
// more of the newest tokens than can stay, looks every slot up in memory for each
// digit: 128 rows of 1,025 slots 21 us in all against 12, 256 rows of 3,000 - 9,000
// 90 against 71.
//
// The selection waits and counts rather than reads: 256 rows of 3,000 - 9,000
// slots 18 us, of which about 5 are the first loads, 1.3 each digit and 3 the
// lists; 128 rows of 1,025 slots with the move 9.6 us.  The copies are bound by
// memory: rows of 128 and 256 bytes at scattered places, 197 MB (int8) in 50 us,
// 3.9 TB/s, where a copy of neighbouring rows reaches 5.2; 62 MB (fp16) in 14 us.
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

// Digit counts are kept in copies, one for every fourth lane: the masses of a
// row share their leading digits, and lanes that count into one word wait for
// each other.  A copy holds the counts from digit 255 down; copies begin eight
// banks apart.  Selection of 256 rows of 3,000 - 9,000 slots: 21.4 us with one
// copy, 17.8 with 4 and with 8, 18.0 with 16.
constexpr int kCopies = 4, kCopyLd = 264;

__device__ __forceinline__ int evict_len(const EvictArgs& a, int64_t b) {
  const int64_t cap = a.max_pages << a.c.page_shift;
  int n = a.lens[b];
  n = n < 0 ? 0 : n;
  n = n > a.max_len ? a.max_len : n;
  return n > cap ? static_cast<int>(cap) : n;
}

// Larger keys stay: the newest tokens, then by mass as an ordered integer (-0 as
// +0; a NaN last).  Above and below them all are slots that do not exist: one
// before `left` keeps its place, one past it goes.
constexpr uint32_t kKeyHeld = 0xffffffffu, kKeyNewest = 0xfffffffeu, kKeyNan = 1u, kKeyGone = 0u;
__device__ __forceinline__ uint32_t mass_key(float mass) {
  if (mass != mass) return kKeyNan;
  const uint32_t u = __builtin_bit_cast(uint32_t, add_rn(mass, 0.0f));
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int lanes_below(uint64_t mask) {  // set bits below the lane's
  return __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(mask >> 32),
                                   __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(mask), 0));
}
// Maximum over the lanes, in every lane.
__device__ __forceinline__ int max_wave(int v) {
  v = max(v, __builtin_amdgcn_update_dpp(v, v, 0x111, 0xF, 0xF, false));  // one lane up, in rows of 16
  v = max(v, __builtin_amdgcn_update_dpp(v, v, 0x112, 0xF, 0xF, false));
  v = max(v, __builtin_amdgcn_update_dpp(v, v, 0x114, 0xF, 0xF, false));
  v = max(v, __builtin_amdgcn_update_dpp(v, v, 0x118, 0xF, 0xF, false));
  v = max(v, __builtin_amdgcn_update_dpp(v, v, 0x142, 0xA, 0xF, false));  // lane 15 to rows 1 and 3
  v = max(v, __builtin_amdgcn_update_dpp(v, v, 0x143, 0xC, 0xF, false));  // lane 31 to rows 2 and 3
  return __builtin_amdgcn_readlane(v, 63);
}

// Rows of which no more bytes than this can move are moved by the workgroup
// that selected them: 128 rows, 1 and 128 slots of 128 bytes over, 9.9 and 11.0
// us against 9.2 and 3.8, 9.4 and 4.5 with a second launch; 512 slots over, 16.6
// against 8.8 and 6.7.
constexpr int64_t kOwnMoveBytes = 16384;
// Slots that a thread moves at a time (1, 2, 4, 8: 53, 52.5, 51 and 54 us for
// the 197 MB above), and workgroups over all rows (2,048, 16,384, 65,536: 67, 51
// and 50 us).
constexpr int kMoveThreads = 256;
constexpr int kMovesAtOnce = 4;
constexpr int64_t kMoveGroups = 16384;

// A row's moves, by `groups` workgroups of THREADS of which this is number
// `group`: each takes neighbouring moves, whose slots lie close together.  LANES
// lanes copy a slot's K and V rows, 16 bytes each, several slots at a time so
// that their loads wait together; two lanes take its mass and position as well.
template <int RB, int THREADS>
__device__ __forceinline__ void move_slots(const EvictArgs& a, int64_t row, const int32_t* from, const int32_t* to,
                                           int count, int group, int groups) {
  constexpr int HALF = RB / 16, LANES = 2 * HALF, step = THREADS / LANES;
  const int first = group * kMovesAtOnce * step + threadIdx.x / LANES;
  const int64_t b = row / a.c.heads;
  const int h = static_cast<int>(row - b * a.c.heads);
  const int ps = a.c.page_shift, mask = (1 << ps) - 1;
  const int l = threadIdx.x % LANES, piece = l < HALF ? l : l - HALF;
  const int32_t* table = a.table + b * a.max_pages;
  uint8_t* pool = l < HALF ? a.c.k : a.c.v;
  uint32_t* metas = l < HALF ? a.c.kmeta : a.c.vmeta;
  const int64_t track = row * a.ld;
  const uint32_t* tracked = reinterpret_cast<const uint32_t*>(l == 0 ? static_cast<const void*>(a.mass) : a.pos) + track;
  uint32_t* tracked_out = reinterpret_cast<uint32_t*>(l == 0 ? static_cast<void*>(a.mass_out) : a.pos_out) + track;
  for (int i0 = first; i0 < count; i0 += groups * kMovesAtOnce * step) {
    int src[kMovesAtOnce], dst[kMovesAtOnce];
    int64_t s[kMovesAtOnce], d[kMovesAtOnce];
    bool ok[kMovesAtOnce];
    v4i w[kMovesAtOnce];
    uint32_t m[kMovesAtOnce], t[kMovesAtOnce];
#pragma unroll
    for (int u = 0; u < kMovesAtOnce; ++u) {
      const int i = min(i0 + u * step, count - 1);
      src[u] = from[i];
      dst[u] = to[i];
    }
#pragma unroll
    for (int u = 0; u < kMovesAtOnce; ++u) {
      const int64_t sp = table[src[u] >> ps], dp = table[dst[u] >> ps];  // in the pool, as when selected
      ok[u] = i0 + u * step < count && sp >= 0 && sp < a.c.pages && dp >= 0 && dp < a.c.pages;
      s[u] = (((ok[u] ? sp : 0) * a.c.heads + h) << ps) + (src[u] & mask);
      d[u] = (((ok[u] ? dp : 0) * a.c.heads + h) << ps) + (dst[u] & mask);
    }
#pragma unroll
    for (int u = 0; u < kMovesAtOnce; ++u) {
      w[u] = reinterpret_cast<const v4i*>(pool + s[u] * RB)[piece];
      m[u] = (metas != nullptr && piece == 0) ? metas[s[u]] : 0;
      t[u] = l < 2 ? tracked[src[u]] : 0;
    }
#pragma unroll
    for (int u = 0; u < kMovesAtOnce; ++u) {
      if (ok[u]) {
        reinterpret_cast<v4i*>(pool + d[u] * RB)[piece] = w[u];
        if (metas != nullptr && piece == 0) metas[d[u]] = m[u];
      }
      if (i0 + u * step < count) {
        if (l < 2) tracked_out[dst[u]] = t[u];
        if (l == 2) a.kept[row * a.budget + dst[u]] = src[u];
      }
    }
  }
}

// Workgroups of 256 threads take rows up to this many times their size, and of
// 1,024 longer ones: 128 rows of 1,025 slots 10.0 us against 10.5, of 2,000 slots
// 10.4 against 8.1.  Rows of up to 8 and 20 slots a thread are held in registers
// (20, with keys, masses and positions, take 93 of the 128 that a lane has):
// 32 rows of 9,001 - 16,384 slots 18.6 us, read from memory for every digit 51.
constexpr int kSmallSteps = 6;

// Selects the slots of one row.  Each wave holds a contiguous part of it, up to
// STEPS times 64 slots in registers (STEPS == 0: any number, read from memory
// each time).  RB > 0: the workgroup moves the rows as well.
template <int THREADS, int STEPS, int RB>
__global__ __launch_bounds__(THREADS) void kv_select_kernel(EvictArgs a) {
  constexpr int WAVES = THREADS / 64;
  __shared__ uint4 hist4[2][kCopyLd * kCopies / 4];
  __shared__ uint4 digits4[64];
  __shared__ int newest_lds[WAVES], holes_lds[WAVES], ties_lds[WAVES];
  __shared__ int2 counts_lds[WAVES];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t row = blockIdx.x;
  const int64_t b = blockIdx.x / static_cast<uint32_t>(a.c.heads);
  const int n = evict_len(a, b);
  const int left = min(n, a.budget);
  const float* mass = a.mass + row * a.ld;
  const int32_t* pos = a.pos + row * a.ld;
  float* mass_out = a.mass_out + row * a.ld;
  int32_t* pos_out = a.pos_out + row * a.ld;
  int32_t* kept = a.kept + row * a.budget;
  if (tid == 0 && row == b * a.c.heads) a.lens_out[b] = left;
  for (int i = left + tid; i < a.budget; i += THREADS) kept[i] = -1;

  const int steps = (n + THREADS - 1) / THREADS;  // STEPS at most where that is not 0
  const int i0 = wave * steps * 64 + lane;
  float mv[STEPS > 0 ? STEPS : 1];
  int32_t pv[STEPS > 0 ? STEPS : 1];
  auto slot = [&](int s) { return i0 + 64 * s; };
  // each(f): f(step, slot, whether it is in the row) over the lane's slots.
  auto each = [&](auto&& f) {
    if constexpr (STEPS > 0) {
#pragma unroll
      for (int s = 0; s < STEPS; ++s)
        if (s < steps) f(s, slot(s), slot(s) < n);  // uniform
    } else {
      for (int s = 0; s < steps; ++s) f(s, slot(s), slot(s) < n);
    }
  };
  if constexpr (STEPS > 0) {
    each([&](int s, int i, bool in) {
      mv[s] = in ? mass[i] : 0.0f;
      pv[s] = in ? pos[i] : INT32_MIN;
    });
  }
  // Slots that do not exist lie on pages outside the pool.  The row's page ids:
  // two a thread are enough for rows in registers, as pages hold 16 slots or more.
  const int32_t* table = a.table + b * a.max_pages;
  const int ps = a.c.page_shift;
  auto outside = [&](int32_t id) { return static_cast<uint32_t>(id) >= static_cast<uint32_t>(a.c.pages); };
  auto absent = [&](int i) { return outside(table[i >> ps]); };
  const int32_t id0 = table[tid << ps < n ? tid : 0];
  const int32_t id1 = STEPS > 8 ? table[(tid + THREADS) << ps < n ? tid + THREADS : 0] : id0;
  auto mass_at = [&](int s, int i) { return STEPS > 0 ? mv[s] : mass[i]; };
  auto pos_at = [&](int s, int i) { return STEPS > 0 ? pv[s] : pos[i]; };
  // Slots below `left` as if all of them stayed; the moves overwrite those that
  // do not (and read only slots from `left` on).
  const bool copy_mass = mass_out != mass, copy_pos = pos_out != pos;
  each([&](int s, int i, bool) {
    if (i >= left) return;
    kept[i] = i;
    if (copy_mass) mass_out[i] = mass_at(s, i);
    if (copy_pos) pos_out[i] = pos_at(s, i);
  });
  if (n <= left) {  // uniform: nothing goes
    if (RB == 0 && tid == 0) a.count[row] = 0;
    return;
  }

  uint32_t* hist0 = reinterpret_cast<uint32_t*>(hist4[0]);
  uint32_t* hist1 = reinterpret_cast<uint32_t*>(hist4[1]);
  for (int i = tid; i < kCopyLd * kCopies / 4; i += THREADS) hist4[0][i] = make_uint4(0, 0, 0, 0);
  int newest = INT32_MIN;
  each([&](int s, int i, bool in) {
    if (in) newest = max(newest, pos_at(s, i));
  });
  newest = max_wave(newest);
  bool holes = outside(id0) || outside(id1);
  if constexpr (STEPS == 0) {
    for (int i = (THREADS + tid) << ps; i < n; i += THREADS << ps) holes = holes || absent(i);
  }
  holes = __any(holes);
  if (lane == 0) {
    newest_lds[wave] = newest;
    holes_lds[wave] = holes;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < WAVES; ++i) {
    newest = max(newest, newest_lds[i]);
    holes = holes || holes_lds[i] != 0;
  }
  if (holes) {  // uniform, and rare: only then are slots looked up
    newest = INT32_MIN;
#pragma unroll 1
    for (int s = 0; s < steps; ++s) {
      if (slot(s) < n && !absent(slot(s))) newest = max(newest, pos[slot(s)]);
    }
    newest = max_wave(newest);
    __syncthreads();
    if (lane == 0) newest_lds[wave] = newest;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < WAVES; ++i) newest = max(newest, newest_lds[i]);
  }
  const int64_t gone = static_cast<int64_t>(newest) - a.recent;  // positions up to here are not protected
  // Past the row keys are those of slots that go: as many slots as stay have
  // larger ones.
  auto key_of = [&](bool in, float m, int32_t p) {
    return !in ? kKeyGone : p > gone ? kKeyNewest : mass_key(m);
  };
  // The same from memory and slot by slot, for rows with holes, and where there are
  // more of the newest than can stay (positions that repeat): those by mass, and
  // no others.
  bool crowded = false;
  auto each_slot = [&](auto&& f) {
#pragma unroll 1
    for (int s = 0; s < steps; ++s) f(s, slot(s), slot(s) < n);
  };
  auto careful_key = [&](int, int i, bool in) {
    if (!in) return kKeyGone;
    if (holes && absent(i)) return i < left ? kKeyHeld : kKeyGone;
    return crowded ? (pos[i] > gone ? mass_key(mass[i]) : kKeyGone) : key_of(true, mass[i], pos[i]);
  };

  // The left-th largest key, digit by digit: `prefix` holds the digits found,
  // `need` how many slots with that prefix stay.  Every wave sums the copies
  // and finds the digit for itself; the next digit's counts are cleared
  // meanwhile.
  uint32_t prefix, need;
  bool all_stay;
  auto find = [&](auto&& each, auto&& key_at) {
    prefix = 0;
    need = static_cast<uint32_t>(left);
    all_stay = false;
#pragma unroll 1
    for (int shift = 24; shift >= 0; shift -= 8) {
      uint32_t* hist = (shift & 8) ? hist0 : hist1;
      uint32_t* next = (shift & 8) ? hist1 : hist0;
      // With the prefix (zero below it) taken off, what is left is below 2^(shift + 8).
      const uint32_t bound = shift == 24 ? 0xffffffffu : (256u << shift) - 1u;
      uint32_t* copy = hist + (lane & (kCopies - 1)) * kCopyLd + 255;
      each([&](int s, int i, bool in) {
        const uint32_t k = key_at(s, i, in) ^ prefix;
        if (k <= bound) atomicAdd(copy - (k >> shift), 1u);
      });
      __syncthreads();
      for (int i = tid; i < kCopyLd * kCopies / 4; i += THREADS) reinterpret_cast<uint4*>(next)[i] = make_uint4(0, 0, 0, 0);
      // A thread per digit sums the copies, then lane l of every wave takes digits
      // 255 - 4l .. 252 - 4l, from the top.
      if (tid < 256) {
        uint32_t of_digit = 0;
#pragma unroll
        for (int i = 0; i < kCopies; ++i) of_digit += hist[i * kCopyLd + tid];
        reinterpret_cast<uint32_t*>(digits4)[tid] = of_digit;
      }
      __syncthreads();
      const uint4 digits = digits4[lane];
      const uint32_t c[4] = {digits.x, digits.y, digits.z, digits.w};
      const uint32_t sum = c[0] + c[1] + c[2] + c[3];
      uint32_t above = wave_scan(sum) - sum;
      uint32_t digit = 0, rest = 0, whole = 0, here = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (above < need && above + c[i] >= need) {
          digit = static_cast<uint32_t>(255 - 4 * lane - i);
          rest = need - above;
          whole = c[i];
          here = 1;
        }
        above += c[i];
      }
      const int at = __builtin_ctzll(__ballot(here != 0));
      prefix |= static_cast<uint32_t>(__builtin_amdgcn_readlane(digit, at)) << shift;
      need = static_cast<uint32_t>(__builtin_amdgcn_readlane(rest, at));
      // All slots with this prefix stay: the prefix, as the least key that has
      // it, already separates the rest.
      all_stay = static_cast<uint32_t>(__builtin_amdgcn_readlane(whole, at)) == need;
      if (all_stay) break;  // uniform
    }
  };

  // Ties at the threshold in slot order (the lowest stay), then the freed front
  // slots and the slots that move, numbered over the row.
  // The lists of the moves: for the second launch, or in LDS.
  __shared__ int32_t own_lists[RB > 0 ? 2 * kOwnMoveBytes / (2 * RB) : 1];
  int32_t* from = RB > 0 ? own_lists : a.from + row * a.move_cap;
  int32_t* to = RB > 0 ? own_lists + a.move_cap : a.to + row * a.move_cap;
  int total = 0;
  auto list = [&](auto&& each, auto&& key_at) {
    int tie0 = 0;
    if (!all_stay) {
      int ties = 0;
      each([&](int s, int i, bool in) { ties += __popcll(__ballot(key_at(s, i, in) == prefix)); });
      if (lane == 0) ties_lds[wave] = ties;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < WAVES; ++i) tie0 += i < wave ? ties_lds[i] : 0;
    }
    auto walk = [&](auto&& f) {
      int tie = tie0;
      each([&](int s, int i, bool in) {
        const uint32_t k = key_at(s, i, in);
        bool keep = k >= prefix;
        if (!all_stay) {
          const uint64_t eqs = __ballot(k == prefix);
          keep = keep && (k > prefix || tie + lanes_below(eqs) < static_cast<int>(need));
          tie += __popcll(eqs);
        }
        f(!keep && i < left, keep && i >= left, i);
      });
    };
    int2 counts = make_int2(0, 0);
    walk([&](bool free_slot, bool move, int) {
      counts.x += __popcll(__ballot(free_slot));
      counts.y += __popcll(__ballot(move));
    });
    if (lane == 0) counts_lds[wave] = counts;
    __syncthreads();
    int free_at = 0, move_at = 0;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) {
      const int2 x = counts_lds[i];
      free_at += i < wave ? x.x : 0;
      move_at += i < wave ? x.y : 0;
      total += x.y;
    }
    walk([&](bool free_slot, bool move, int i) {
      const uint64_t fs = __ballot(free_slot), ms = __ballot(move);
      if (free_slot) to[free_at + lanes_below(fs)] = i;
      if (move) from[move_at + lanes_below(ms)] = i;
      free_at += __popcll(fs);
      move_at += __popcll(ms);
    });
  };

  if (!holes) {
    uint32_t kv[STEPS > 0 ? STEPS : 1];
    if constexpr (STEPS > 0) each([&](int s, int, bool in) { kv[s] = key_of(in, mv[s], pv[s]); });
    auto key_at = [&](int s, int i, bool in) {
      if constexpr (STEPS > 0) return kv[s];
      return in ? key_of(true, mass[i], pos[i]) : kKeyGone;
    };
    find(each, key_at);
    crowded = !all_stay && prefix == kKeyNewest;
    if (!crowded) list(each, key_at);
  }
  if (holes || crowded) {
    find(each_slot, careful_key);
    if (!crowded && !all_stay && prefix == kKeyNewest) {
      crowded = true;
      find(each_slot, careful_key);
    }
    list(each_slot, careful_key);
  }
  if constexpr (RB > 0) {
    __syncthreads();  // the lists
    move_slots<RB, THREADS>(a, row, from, to, total, 0, 1);
  } else {
    if (tid == 0) a.count[row] = total;
  }
}

template <int RB>
__global__ __launch_bounds__(kMoveThreads) void kv_move_kernel(EvictArgs a) {
  const int64_t row = blockIdx.x;
  move_slots<RB, kMoveThreads>(a, row, a.from + row * a.move_cap, a.to + row * a.move_cap, a.count[row], blockIdx.y,
                               static_cast<int>(gridDim.y));
}

template <int RB>
void launch_evict(const EvictArgs& a, int64_t rows, hipStream_t st) {
  const dim3 grid(static_cast<unsigned>(rows));
  const bool own = static_cast<int64_t>(a.move_cap) * 2 * RB <= kOwnMoveBytes;
  if (a.max_len <= 256 * kSmallSteps) {
    if (own)
      kv_select_kernel<256, kSmallSteps, RB><<<grid, 256, 0, st>>>(a);
    else
      kv_select_kernel<256, kSmallSteps, 0><<<grid, 256, 0, st>>>(a);
  } else if (a.max_len <= 1024 * 8) {
    if (own)
      kv_select_kernel<1024, 8, RB><<<grid, 1024, 0, st>>>(a);
    else
      kv_select_kernel<1024, 8, 0><<<grid, 1024, 0, st>>>(a);
  } else if (a.max_len <= 1024 * 20) {
    kv_select_kernel<1024, 20, 0><<<grid, 1024, 0, st>>>(a);
  } else {
    kv_select_kernel<1024, 0, 0><<<grid, 1024, 0, st>>>(a);
  }
  if (a.move_cap == 0 || (own && a.max_len <= 1024 * 8)) return;
  constexpr int per = kMoveThreads / (RB / 8) * kMovesAtOnce;
  // A workgroup goes over several lots of its row's moves when there are many.
  const int64_t most = (a.move_cap + per - 1) / per;
  const int64_t want = (kMoveGroups + rows - 1) / rows;
  kv_move_kernel<RB><<<dim3(static_cast<unsigned>(rows), static_cast<unsigned>(most < want ? most : want)), kMoveThreads,
                       0, st>>>(a);
}

// At most this many slots of a row move: each fills a slot below the budget
// and comes from one past it.
inline int64_t evict_move_cap(int64_t max_len, int64_t budget) {
  const int64_t over = max_len > budget ? max_len - budget : 0;
  return over < budget ? over : budget;
}

// Slots and budgets at most: the kernels step past them by up to a workgroup's
// reach (2^21 slots) in 32 bits.
constexpr int64_t kMaxSlots = kMaxDim / 2;

inline size_t evict_count_bytes(int64_t rows) { return (static_cast<size_t>(rows) * 4 + 255) / 256 * 256; }

}  // namespace
}  // namespace qlin

using namespace qlin;

extern "C" size_t qlin_kv_evict_work_bytes(const qlin_kv_cache* cache, int64_t B, int64_t max_len, int32_t budget) {
  if (!kv_shape_ok(cache) || B < 1 || B >= kMaxDim / cache->kv_heads || max_len < 0 || max_len > kMaxSlots ||
      budget < 0 || budget > kMaxSlots || !dims_ok(B * cache->kv_heads, max_len + 1))
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
  QLIN_REQUIRE(max_len <= kMaxSlots, QLIN_ERR_SHAPE, "max_len=%lld: at most 2^30", (long long)max_len);
  QLIN_REQUIRE(budget <= kMaxSlots, QLIN_ERR_SHAPE, "budget=%d: at most 2^30", budget);
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
  QLIN_REQUIRE(lens_out != lens, QLIN_ERR_INVALID_ARG, "lens_out: must not be the array lens");
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
  switch (cache->head_dim * cache->bits / 8) {
    case 32: launch_evict<32>(a, rows, st); break;
    case 64: launch_evict<64>(a, rows, st); break;
    case 128: launch_evict<128>(a, rows, st); break;
    case 256: launch_evict<256>(a, rows, st); break;
    default: launch_evict<512>(a, rows, st); break;
  }
  QLIN_LAUNCH_CHECK("kv_select_kernel, kv_move_kernel");
  return QLIN_OK;
}
