// Backward of the event rows x_i = item_table[id_i] + action_table[a_i]
// (events.cu): the tables' gradients,
//   d_item[v] = sum over {i : id_i = v} of dX_i,   d_action[a] likewise,
// dense, fp32, without floating-point atomics: the same inputs give the same
// bits.  A row whose id or action is outside its table was zero in the forward,
// so it counts for neither table (and sets the device error word).
//
// The rows are ordered by item id with a stable radix sort of (id, event) pairs (an
// LSD pass per kMaxBits bits of the vocabulary's size: two for a million items), so
// every table row's gradient is the sum of a contiguous run of the list, in the order
// of the events.  The list is cut into equal windows, one per half-warp: runs inside a
// window are written at once, the sums of the runs that cross its ends are kept, and a
// second kernel adds those.  So every row of dX is read once and every half-warp has
// the same work however popular an item is (under Zipf(1.1) ids over a million items
// one item has 1 event in 8).  The same pass adds each row to its action's sum, in a
// table per warp in shared memory.
//
// Bound by memory: dX read once, the item gradient written once.  The sort is one
// cooperative launch (its CTAs exchange digit counts through memory between the passes'
// steps): half of each CTA's warps sort, which waits on latency and leaves the memory
// idle, and the other half zero the whole item gradient meanwhile (most of it stays
// zero: a million items, 680K events); the rows with events are written over that.
#include <algorithm>
#include <mutex>

#include "sa_internal.cuh"
#include "tma_map.cuh"

namespace sa {

namespace {
constexpr int kMaxBits = 10;                 // of the id per pass: 1024 bins
constexpr int kSortThreads = 512, kSortWarps = kSortThreads / 32;   // of a CTA; as many again write zeros
constexpr int kSortPer = 1024;               // events per sorting CTA, at least
constexpr int kMinWin = 32;                  // list positions per window, at least
constexpr int kSumThreads = 256, kSumWarps = kSumThreads / 32, kHalves = 2 * kSumWarps;
constexpr int kCols = 8;                     // columns per lane: a half-warp covers 128
constexpr int kBatch = 8;                    // rows in flight per half-warp
constexpr int kLong = 32;                    // windows of a run that one half-warp adds; longer: the whole CTA
constexpr int kFusedActions = 16;            // action tables that the window kernel keeps in shared memory

// the key of an event: its item id, or `vocab` (behind every item) when the event's id or
// action is outside its table
__device__ __forceinline__ uint32_t event_key(const int32_t* ids, const uint8_t* acts, int64_t i, int64_t vocab,
                                              int n_actions) {
  const int64_t id = ids[i];
  return id >= 0 && id < vocab && acts[i] < n_actions ? (uint32_t)id : (uint32_t)vocab;
}

// where a pass reads its keys: the events themselves (the first), or the last pass's list
struct FromEvents {
  const int32_t* ids;
  const uint8_t* acts;
  int64_t vocab;
  int n_actions;
  __device__ uint32_t key(int64_t i) const { return event_key(ids, acts, i, vocab, n_actions); }
  __device__ uint32_t event(int64_t i) const { return (uint32_t)i; }
  __device__ bool outside(uint32_t key) const { return key == (uint32_t)vocab; }
};
struct FromList {
  const uint32_t* keys;
  const uint32_t* events;
  // written by other CTAs of this launch: not through L1
  __device__ uint32_t key(int64_t i) const { return __ldcg(keys + i); }
  __device__ uint32_t event(int64_t i) const { return __ldcg(events + i); }
  __device__ bool outside(uint32_t) const { return false; }
};

// barrier of a CTA's sorting warps
__device__ __forceinline__ void sort_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kSortThreads) : "memory"); }

// Barrier number `round` (from 1) of the sorting CTAs over a counter that starts at zero.  All of
// them are resident (cooperative launch); the wait is bounded all the same: past the limit it sets
// the device error word, and the sort goes on over incomplete counts, every index of which is
// checked before it is used.
__device__ __forceinline__ void grid_sync(unsigned* counter, unsigned ctas, unsigned round, int* err) {
  __threadfence();
  sort_sync();
  if (threadIdx.x == 0) {
    atomicAdd(counter, 1u);
    const long long t0 = clock64();
    while (*(volatile unsigned*)counter < ctas * round)
      if (clock64() - t0 > 4000000000LL) {
        atomicOr(err, DEV_ERR_TIMEOUT);
        break;
      }
    __threadfence();
  }
  sort_sync();
}

struct SortArgs {
  FromEvents in;
  int64_t n, per;            // events, and events per sorting CTA
  int bits, passes, ctas;    // of the keys; sorting CTAs
  uint32_t *keys[2], *events[2];   // the list after pass q is in buffer q & 1
  int* hist;                 // [ctas][bins] digit counts of a pass, one array per pass parity
  unsigned* counter;
  float4* zero;              // the item gradient, and its 16-byte pieces
  int64_t zeros;
  int* err;
};
constexpr int sort_smem(int bits) { return (kSortWarps + 3) * (1 << bits) * 4; }

// One pass over the digit at `shift`: moves the CTA's events behind those with smaller digits, and
// those with the same digit in earlier CTAs.  Each warp owns a contiguous part, counts its digits,
// and places its events in order, so equal digits keep their order.
template <class In>
__device__ void sort_pass(const In& in, const SortArgs& s, int q, int shift, int bits, int* smem, unsigned& round) {
  __shared__ int warp_sum[kSortWarps];
  const int bins = 1 << bits, cta = blockIdx.x;
  int *wcnt = smem, *base = smem + kSortWarps * bins, *half = base + bins;   // [warps][bins], [bins], [2][bins]
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  for (int b = threadIdx.x; b < kSortWarps * bins; b += kSortThreads) wcnt[b] = 0;
  sort_sync();
  const int64_t begin = min((int64_t)cta * s.per, s.n), end = min(begin + s.per, s.n);
  const int64_t size = ((end - begin + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
  const int64_t wb = min(begin + warp * size, end), we = min(wb + size, end);
  int* mine = wcnt + warp * bins;
  bool bad = false;
  for (int64_t i0 = wb + lane; i0 < we; i0 += 128) {
    uint32_t key[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) key[x] = i0 + 32 * x < we ? in.key(i0 + 32 * x) : 0u;
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (i0 + 32 * x < we) {
        bad |= in.outside(key[x]);
        atomicAdd(&mine[(key[x] >> shift) & (bins - 1)], 1);
      }
  }
  if (bad) atomicOr(s.err, DEV_ERR_INDEX);
  sort_sync();
  // half[h][b]: events with digit b of the CTAs g = h mod 2; base[b]: of the earlier CTAs
  int* hist = s.hist + (int64_t)(q & 1) * s.ctas * (1 << kMaxBits);
  for (int b = threadIdx.x; b < bins; b += kSortThreads) {
    int total = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) total += wcnt[w * bins + b];
    if (s.ctas > 1) {
      hist[(int64_t)cta * bins + b] = total;
    } else {
      base[b] = 0;
      half[b] = total;
      half[bins + b] = 0;
    }
  }
  if (s.ctas > 1) {
    grid_sync(s.counter, s.ctas, ++round, s.err);
    // two halves of the CTAs, four bins per thread (bins >= 4)
    const int quads = bins / 4, x = threadIdx.x % quads, h = threadIdx.x / quads;
    int4 total = make_int4(0, 0, 0, 0), before = make_int4(0, 0, 0, 0);
    if (h < 2) {
#pragma unroll 16
      for (int g = h; g < s.ctas; g += 2) {
        const int4 c = __ldcg((const int4*)(hist + (int64_t)g * bins + 4 * x));
        total.x += c.x; total.y += c.y; total.z += c.z; total.w += c.w;
        if (g < cta) { before.x += c.x; before.y += c.y; before.z += c.z; before.w += c.w; }
      }
      *(int4*)(half + h * bins + 4 * x) = total;
      if (h == 0) *(int4*)(base + 4 * x) = before;
    }
    sort_sync();
    if (h == 1) {
      int4 o = *(int4*)(base + 4 * x);
      o.x += before.x; o.y += before.y; o.z += before.z; o.w += before.w;
      *(int4*)(base + 4 * x) = o;
    }
  }
  sort_sync();
  // each warp's first place for each digit
  int carry = 0;
  for (int b0 = 0; b0 < bins; b0 += kSortThreads) {
    const int b = b0 + threadIdx.x;
    const int total = b < bins ? half[b] + half[bins + b] : 0;
    int incl = total;
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) warp_sum[warp] = incl;
    sort_sync();
    int off = carry, all = carry;
    for (int w = 0; w < kSortWarps; ++w) {
      if (w < warp) off += warp_sum[w];
      all += warp_sum[w];
    }
    carry = all;
    if (b < bins) {
      int run = off + incl - total + base[b];
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) {
        const int c = wcnt[w * bins + b];
        wcnt[w * bins + b] = run;
        run += c;
      }
    }
    sort_sync();
  }
  uint32_t *keys = s.keys[q & 1], *events = s.events[q & 1];
  for (int64_t i0 = wb; i0 < we; i0 += 32) {
    const int64_t i = i0 + lane;
    const bool there = i < we;
    const uint32_t key = there ? in.key(i) : 0u;
    const int digit = there ? (int)((key >> shift) & (bins - 1)) : -1;
    const unsigned same = __match_any_sync(0xffffffffu, digit);
    const int rank = __popc(same & ((1u << lane) - 1));
    const int at = there ? mine[digit] : 0;
    __syncwarp();
    if (there) {
      if (rank == 0) mine[digit] = at + __popc(same);
      if ((unsigned)(at + rank) < (uint64_t)s.n) {
        keys[at + rank] = key;
        events[at + rank] = in.event(i);
      }
    }
    __syncwarp();
  }
  if (s.ctas > 1 && q + 1 < s.passes) grid_sync(s.counter, s.ctas, ++round, s.err);
  else sort_sync();
}

__global__ void __launch_bounds__(2 * kSortThreads, 1) sort_events_kernel(SortArgs s) {
  extern __shared__ __align__(16) int smem[];
  if (threadIdx.x >= kSortThreads) {
    const int64_t stride = (int64_t)gridDim.x * kSortThreads;
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int64_t i = (int64_t)blockIdx.x * kSortThreads + threadIdx.x - kSortThreads; i < s.zeros; i += stride)
      __stcs(s.zero + i, zero);
    return;
  }
  if ((int)blockIdx.x >= s.ctas) return;
  unsigned round = 0;
  for (int q = 0; q < s.passes; ++q) {
    const int shift = s.bits * q / s.passes, bits = s.bits * (q + 1) / s.passes - shift;
    if (q == 0) sort_pass(s.in, s, q, shift, bits, smem, round);
    else sort_pass(FromList{s.keys[(q - 1) & 1], s.events[(q - 1) & 1]}, s, q, shift, bits, smem, round);
  }
}

// 8 columns of a row, as they lie in memory
struct RawB {
  uint4 w;
};
struct RawF {
  float4 a, b;
};
__device__ __forceinline__ RawB load_raw(const __nv_bfloat16* p) { return {__ldcs((const uint4*)p)}; }
__device__ __forceinline__ RawF load_raw(const float* p) {
  return {__ldcs((const float4*)p), __ldcs((const float4*)p + 1)};
}
struct Cols {                                // 8 fp32 columns, added in pairs
  float2 x[4];
};
__device__ __forceinline__ Cols widen(const RawB& r) {
  const uint32_t w[4] = {r.w.x, r.w.y, r.w.z, r.w.w};
  Cols c;
#pragma unroll
  for (int i = 0; i < 4; ++i) c.x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  return c;
}
__device__ __forceinline__ Cols widen(const RawF& r) {
  return {{make_float2(r.a.x, r.a.y), make_float2(r.a.z, r.a.w), make_float2(r.b.x, r.b.y), make_float2(r.b.z, r.b.w)}};
}
__device__ __forceinline__ Cols zero_cols() {
  const float2 z = make_float2(0.f, 0.f);
  return {{z, z, z, z}};
}
__device__ __forceinline__ void add_cols(Cols& a, const Cols& b) {
#pragma unroll
  for (int i = 0; i < 4; ++i) a.x[i] = __fadd2_rn(a.x[i], b.x[i]);
}
__device__ __forceinline__ Cols load_cols(const float* p) {
  const float4 a = *(const float4*)p, b = *((const float4*)p + 1);
  return {{make_float2(a.x, a.y), make_float2(a.z, a.w), make_float2(b.x, b.y), make_float2(b.z, b.w)}};
}
__device__ __forceinline__ void store_cols(float* p, const Cols& c) {
  *(float4*)p = make_float4(c.x[0].x, c.x[0].y, c.x[1].x, c.x[1].y);
  *((float4*)p + 1) = make_float4(c.x[2].x, c.x[2].y, c.x[3].x, c.x[3].y);
}

// A warp's table of action sums in shared memory: [n_actions][2][16 lanes] float4, so that the
// lanes' 16-byte accesses are consecutive
struct Table {
  float4* base;
  __device__ void clear(int n_actions) const {
    for (int a = 0; a < n_actions; ++a) base[a * 32 + threadIdx.x % 32] = make_float4(0.f, 0.f, 0.f, 0.f);
    __syncwarp();
  }
  __device__ void add(int a, int l, const Cols& c) const {
    float4* p = base + a * 32 + l;
    float4 u = p[0], v = p[16];
    u.x += c.x[0].x; u.y += c.x[0].y; u.z += c.x[1].x; u.w += c.x[1].y;
    v.x += c.x[2].x; v.y += c.x[2].y; v.z += c.x[3].x; v.w += c.x[3].y;
    p[0] = u;
    p[16] = v;
  }
};
// the CTA's tables, added in order, to out[n_actions][d] (columns c0 .. c0 + 127 of it)
__device__ __forceinline__ void store_tables(const float4* tables, int count, int n_actions, int c0, int d, float* out) {
  for (int e = threadIdx.x; e < n_actions * 32; e += blockDim.x) {
    const int col = c0 + (e % 16) * kCols + (e / 16) % 2 * 4;
    float4 acc = tables[e];
    for (int h = 1; h < count; ++h) {
      const float4 x = tables[h * n_actions * 32 + e];
      acc.x += x.x; acc.y += x.y; acc.z += x.z; acc.w += x.w;
    }
    if (col < d) *(float4*)(out + (int64_t)(e / 32) * d + col) = acc;
  }
}

// What a window leaves for the second kernel: its first key, and the key of its last run if that
// starts in it and goes on behind it (else kNone).
constexpr uint32_t kNone = 0xFFFFFFFFu;

// Window w is list positions [win w, win (w + 1)), a half-warp's.  It walks them row by row: a run
// that lies inside is written to its table row; the sum before the window's first run head goes to
// first[w], that of a run which goes on behind the window to last[w].  With kActions every row is
// also added to the warp's table of action sums, one half-warp after the other (a table per
// half-warp would halve the CTAs per SM); the CTA's tables go to action_part[CTA][n_actions][d].
template <class T, bool kActions>
__global__ void __launch_bounds__(kSumThreads, 3) window_rows_kernel(const T* __restrict__ dX,
                                                                     const uint32_t* __restrict__ keys,
                                                                     const uint32_t* __restrict__ events,
                                                                     const uint8_t* __restrict__ acts, int64_t n,
                                                                     int64_t win, int64_t vocab, int n_actions, int d,
                                                                     float* __restrict__ first, float* __restrict__ last,
                                                                     uint32_t* __restrict__ first_key,
                                                                     uint32_t* __restrict__ open_key,
                                                                     float* __restrict__ d_item,
                                                                     float* __restrict__ action_part) {
  extern __shared__ float4 tables[];                 // [kSumWarps][n_actions][32]
  const int half = threadIdx.x / 16, l = threadIdx.x % 16;
  const Table table{tables + threadIdx.x / 32 * n_actions * 32};
  const int64_t w = (int64_t)blockIdx.x * kHalves + half, p0 = min(w * win, n), p1 = min(p0 + win, n);
  for (int c0 = 0; c0 < d; c0 += 16 * kCols) {
    const int c = c0 + l * kCols;
    const bool in = c < d;
    if (kActions) table.clear(n_actions);
    Cols acc = zero_cols();
    uint32_t run = p0 > 0 ? keys[p0 - 1] : kNone;    // key of the run that acc belongs to
    const uint32_t behind = p1 < n ? keys[p1] : kNone;
    bool inside = false;                             // a head was seen: acc starts at it
    // (an event number is below n, unless the sort gave up at a barrier)
    auto event_at = [&](int64_t i) { const uint32_t e = events[i]; return e < (uint64_t)n ? e : 0u; };
    uint32_t key_n = p0 + l < p1 ? keys[p0 + l] : kNone, ev_n = p0 + l < p1 ? event_at(p0 + l) : 0u;
    if (l == 0 && c0 == 0 && p0 < p1) first_key[w] = key_n;
    // both half-warps take the same steps (win is theirs in common); cnt <= 0: behind the window
    for (int64_t b = p0; b < p0 + win; b += 16) {
      const int cnt = (int)min((int64_t)16, p1 - b);
      const uint32_t key = key_n, ev = ev_n;
      if (b + 16 + l < p1) {                         // the next 16 positions, a step ahead
        key_n = keys[b + 16 + l];
        ev_n = event_at(b + 16 + l);
      }
      int act = -1;
      if (kActions && l < cnt && key < (uint32_t)vocab) act = acts[ev];
#pragma unroll
      for (int j = 0; j < 16; j += kBatch) {
        decltype(load_raw(dX)) x[kBatch];
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
          const uint32_t e = __shfl_sync(0xffffffffu, ev, j + q, 16);
          if (j + q < cnt && in) x[q] = load_raw(dX + (int64_t)e * d + c);
        }
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
          const uint32_t kq = __shfl_sync(0xffffffffu, key, j + q, 16);
          const int aq = kActions ? __shfl_sync(0xffffffffu, act, j + q, 16) : -1;
          if (j + q < cnt && in) {                   // the same for the whole half-warp, but for idle lanes
            if (kq != run) {
              if (!inside) store_cols(first + w * d + c, acc);
              else if (run < (uint32_t)vocab) store_cols(d_item + (int64_t)run * d + c, acc);
              acc = zero_cols();
            }
            add_cols(acc, widen(x[q]));
          }
          if (j + q < cnt && kq != run) {
            inside = true;
            run = kq;
          }
          if (kActions) {
            const bool add = aq >= 0 && j + q < cnt && in;
            if (add && half % 2 == 0) table.add(aq, l, widen(x[q]));
            __syncwarp();
            if (add && half % 2 == 1) table.add(aq, l, widen(x[q]));
            __syncwarp();
          }
        }
      }
    }
    const bool on = behind == run;                   // the run goes on in the next window
    if (in && p0 < p1) {
      if (!inside) store_cols(first + w * d + c, acc);
      else if (on) store_cols(last + w * d + c, acc);
      else if (run < (uint32_t)vocab) store_cols(d_item + (int64_t)run * d + c, acc);
    }
    if (l == 0 && c0 == 0 && p0 < p1) open_key[w] = inside && on && run < (uint32_t)vocab ? run : kNone;
    if (kActions) {
      __syncthreads();
      store_tables(tables, kSumWarps, n_actions, c0, d, action_part + (int64_t)blockIdx.x * n_actions * d);
      __syncthreads();
    }
  }
}

// sum of rows [b, e) of a [., pitch] array at 8 columns, in order
__device__ __forceinline__ Cols sum_range(const float* __restrict__ part, int64_t b, int64_t e, int64_t pitch, bool in) {
  Cols acc = zero_cols();
  if (!in) return acc;
  int64_t v = b;
  for (; v + kBatch <= e; v += kBatch) {
    Cols x[kBatch];
#pragma unroll
    for (int q = 0; q < kBatch; ++q) x[q] = load_cols(part + (v + q) * pitch);
#pragma unroll
    for (int q = 0; q < kBatch; ++q) add_cols(acc, x[q]);
  }
  for (; v < e; ++v) add_cols(acc, load_cols(part + v * pitch));
  return acc;
}

// the half-warps' sums added in order; the result is in half-warp 0
__device__ __forceinline__ Cols sum_halves(const Cols& mine, Cols (*part)[16]) {
  const int half = threadIdx.x / 16, l = threadIdx.x % 16;
  __syncthreads();
  part[half][l] = mine;
  __syncthreads();
  Cols acc = part[0][l];
  for (int h = 1; h < kHalves; ++h) add_cols(acc, part[h][l]);
  return acc;
}

// CTAs [0, action_ctas): the action sums, one action each, from `parts` CTAs' tables.  The others: a
// half-warp per window whose last run goes on: the run's sum is last[w] + first[w + 1] + ... up to
// the window where it ends.  Runs over more than kLong windows are added by the whole CTA.
__global__ void __launch_bounds__(kSumThreads) crossing_rows_kernel(const uint32_t* __restrict__ first_key,
                                                                    const uint32_t* __restrict__ open_key,
                                                                    int64_t windows, int d,
                                                                    const float* __restrict__ first,
                                                                    const float* __restrict__ last,
                                                                    float* __restrict__ d_item, int action_ctas,
                                                                    const float* __restrict__ action_part, int parts,
                                                                    float* __restrict__ d_action) {
  __shared__ Cols part[kHalves][16];
  __shared__ int64_t long_end[kHalves];
  const int half = threadIdx.x / 16, l = threadIdx.x % 16;
  if ((int)blockIdx.x < action_ctas) {
    const int a = (int)blockIdx.x;
    for (int c0 = 0; c0 < d; c0 += 16 * kCols) {
      const int c = c0 + l * kCols;
      const Cols acc = sum_halves(sum_range(action_part + (int64_t)a * d + c, (int64_t)parts * half / kHalves,
                                            (int64_t)parts * (half + 1) / kHalves, (int64_t)action_ctas * d, c < d), part);
      if (half == 0 && c < d) store_cols(d_action + (int64_t)a * d + c, acc);
    }
    return;
  }
  const unsigned mask = 0xFFFFu << (threadIdx.x & 16);
  const int64_t w0 = (int64_t)(blockIdx.x - action_ctas) * kHalves, w = w0 + half;
  const uint32_t run = w + 1 < windows ? open_key[w] : kNone;
  int64_t end = 0;                                   // one behind the last window of the run (0: none to add)
  if (run != kNone) {
    // window v > w holds a part of the run iff its first key is the run's
    end = w + 1;
    for (int i = 0; i < kLong; i += 16) {
      const int64_t v = end + l;
      const int more = __popc(__ballot_sync(mask, v < windows && first_key[v] == run) & mask);
      end += more;
      if (more < 16) break;
    }
    if (end == w + 1 + kLong) {                      // find the end, 16 probes at a time
      int64_t lo = end, hi = windows;                // all windows before lo start with the run, hi does not
      while (lo < hi) {
        const int64_t step = (hi - lo + 15) / 16, v = lo + l * step;
        const int more = __popc(__ballot_sync(mask, v < hi && first_key[v] == run) & mask);
        if (more == 0) break;
        hi = min(hi, lo + more * step);
        lo = lo + (more - 1) * step + 1;
      }
      end = lo;
    }
  }
  const bool is_long = end - w - 1 >= kLong;
  if (l == 0) long_end[half] = is_long ? end : 0;
  if (end > 0 && !is_long)
    for (int c = l * kCols; c < d; c += 16 * kCols) {
      Cols acc = load_cols(last + w * d + c);
      add_cols(acc, sum_range(first + c, w + 1, end, d, true));
      store_cols(d_item + (int64_t)run * d + c, acc);
    }
  __syncthreads();
  for (int i = 0; i < kHalves; ++i) {
    const int64_t e = long_end[i], b = w0 + i;
    if (e == 0) continue;
    const int64_t cnt = e - b - 1;
    const uint32_t key = open_key[b];
    for (int c0 = 0; c0 < d; c0 += 16 * kCols) {
      const int c = c0 + l * kCols;
      Cols acc = sum_range(first + c, b + 1 + cnt * half / kHalves, b + 1 + cnt * (half + 1) / kHalves, d, c < d);
      if (half == 0 && c < d) add_cols(acc, load_cols(last + b * d + c));
      acc = sum_halves(acc, part);
      if (half == 0 && c < d) store_cols(d_item + (int64_t)key * d + c, acc);
    }
  }
}

// part[CTA][action][d]: the sums of the CTA's contiguous events by action (more actions than the
// window kernel's tables, or the action gradient alone).  Each warp adds its own contiguous part
// into its own table in shared memory, two rows at a time, one after the other; the tables are added
// in order.
template <class T>
__global__ void action_rows_kernel(const T* __restrict__ dX, const int32_t* __restrict__ ids,
                                   const uint8_t* __restrict__ acts, int64_t n, int64_t per, int64_t vocab,
                                   int n_actions, int d, float* __restrict__ part, int* err) {
  extern __shared__ float4 tables[];                 // [warps][n_actions][32]
  const int warp = threadIdx.x / 32, warps = blockDim.x / 32, lane = threadIdx.x % 32, l = lane % 16, h = lane / 16;
  const int c = blockIdx.y * 16 * kCols + l * kCols;
  const bool in = c < d;
  const Table table{tables + warp * n_actions * 32};
  table.clear(n_actions);
  const int64_t begin = min((int64_t)blockIdx.x * per, n), end = min(begin + per, n);
  const int64_t size = (end - begin + warps - 1) / warps;
  const int64_t wb = min(begin + warp * size, end), we = min(wb + size, end);
  bool bad = false;
  for (int64_t i0 = wb; i0 < we; i0 += 32) {
    const int cnt = (int)min((int64_t)32, we - i0);
    int a = -1;
    if (lane < cnt) {
      const bool ok = event_key(ids, acts, i0 + lane, vocab, n_actions) < (uint64_t)vocab;
      a = ok ? (int)acts[i0 + lane] : -1;
      bad |= !ok;
    }
    for (int j = 0; j < cnt; j += 2 * kBatch) {      // rows j + 2 q + h
      decltype(load_raw(dX)) x[kBatch];
#pragma unroll
      for (int q = 0; q < kBatch; ++q)
        if (j + 2 * q + h < cnt && in) x[q] = load_raw(dX + (i0 + j + 2 * q + h) * d + c);
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        const int aq = __shfl_sync(0xffffffffu, a, j + 2 * q + h);
        const bool add = j + 2 * q + h < cnt && aq >= 0 && in;
        if (add && h == 0) table.add(aq, l, widen(x[q]));
        __syncwarp();
        if (add && h == 1) table.add(aq, l, widen(x[q]));
        __syncwarp();
      }
    }
  }
  if (bad && blockIdx.y == 0) atomicOr(err, DEV_ERR_INDEX);
  __syncthreads();
  store_tables(tables, warps, n_actions, blockIdx.y * 16 * kCols, d, part + (int64_t)blockIdx.x * n_actions * d);
}

int key_bits(int64_t vocab) {
  int b = 2;                                          // a digit of at least 4 bins
  while (((int64_t)1 << b) <= vocab) ++b;             // keys 0 .. vocab
  return b;
}
int sort_ctas(int64_t n) {
  return (int)std::max<int64_t>(1, std::min<int64_t>(device_info().sm_count, (n + kSortPer - 1) / kSortPer));
}
// warps of an action CTA: their tables (512 bytes per action) fit in 128 KB of shared memory
int action_warps(int n_actions) { return std::max(1, std::min(kSumWarps, 256 / n_actions)); }
int action_ctas(int64_t n) {
  return (int)std::max<int64_t>(1, std::min<int64_t>(4 * device_info().sm_count, (n + 255) / 256));
}
// Windows: one per half-warp of the CTAs that are resident at once (three per SM, their registers'
// limit: 16 tables take 64 KB of a CTA's shared memory), so that all have the same work.
int64_t window_size(int64_t n) {
  const int64_t halves = (int64_t)3 * device_info().sm_count * kHalves;
  return std::max<int64_t>(kMinWin, (n + halves - 1) / halves);
}

template <class T>
sa_status run(const T* dX, const int32_t* ids, const uint8_t* acts, int64_t n, int64_t vocab, int n_actions, int d,
              float* d_item, float* d_action, const EventsBwdWork& w, cudaStream_t st) {
  static unsigned long long done[3] = {};          // one per kernel
  static std::mutex mu;
  int* err = device_status_word();
  const bool fused = d_item && d_action && n_actions <= kFusedActions;
  const int64_t win = window_size(n), windows = (n + win - 1) / win;
  const int window_ctas = (int)((windows + kHalves - 1) / kHalves);
  const int parts = fused ? window_ctas : action_ctas(n);
  if (d_action && !fused) {
    const int warps = action_warps(n_actions);
    const int smem = warps * n_actions * 512;
    set_smem_limit_once((const void*)action_rows_kernel<T>, 256 * 512, &done[0], mu);
    SA_TIMED("action_rows_kernel", st,
             (action_rows_kernel<T><<<dim3(parts, (d + 127) / 128), warps * 32, smem, st>>>(
                 dX, ids, acts, n, (n + parts - 1) / parts, vocab, n_actions, d, w.action_part, err)));
  }
  if (d_item) {
    const int bits = key_bits(vocab), passes = (bits + kMaxBits - 1) / kMaxBits;
    SortArgs s{{ids, acts, vocab, n_actions}, n, 0, bits, passes, sort_ctas(n), {w.keys[0], w.keys[1]},
               {w.events[0], w.events[1]}, w.hist, w.counter, (float4*)d_item, vocab * d / 4, err};
    s.per = (n + s.ctas - 1) / s.ctas;
    set_smem_limit_once((const void*)sort_events_kernel, sort_smem(kMaxBits), &done[1], mu);
    const int smem = sort_smem((bits + passes - 1) / passes);
    if (s.ctas == 1) {
      SA_TIMED("sort_events_kernel", st,
               (sort_events_kernel<<<device_info().sm_count, 2 * kSortThreads, smem, st>>>(s)));
    } else {
      SA_CUDA(cudaMemsetAsync(w.counter, 0, sizeof(unsigned), st));
      void* args[] = {&s};
      SA_TIMED("sort_events_kernel", st,
               cudaLaunchCooperativeKernel((const void*)sort_events_kernel, dim3(device_info().sm_count),
                                           dim3(2 * kSortThreads), args, (size_t)smem, st));
    }
    const uint32_t *keys = w.keys[(passes - 1) & 1], *events = w.events[(passes - 1) & 1];
    if (fused) {
      const int smem = kSumWarps * n_actions * 512;
      set_smem_limit_once((const void*)window_rows_kernel<T, true>, kSumWarps * kFusedActions * 512, &done[2], mu);
      SA_TIMED("window_rows_kernel", st,
               (window_rows_kernel<T, true><<<window_ctas, kSumThreads, smem, st>>>(
                   dX, keys, events, acts, n, win, vocab, n_actions, d, w.first, w.last, w.first_key, w.open_key, d_item,
                   w.action_part)));
    } else {
      SA_TIMED("window_rows_kernel", st,
               (window_rows_kernel<T, false><<<window_ctas, kSumThreads, 0, st>>>(
                   dX, keys, events, acts, n, win, vocab, 0, d, w.first, w.last, w.first_key, w.open_key, d_item, nullptr)));
    }
  }
  const int ac = d_action ? n_actions : 0;
  SA_TIMED("crossing_rows_kernel", st,
           (crossing_rows_kernel<<<ac + (d_item ? window_ctas : 0), kSumThreads, 0, st>>>(
               w.first_key, w.open_key, windows, d, w.first, w.last, d_item, ac, w.action_part, parts, d_action)));
  return SA_OK;
}
}  // namespace

size_t events_bwd_layout(void* base, int64_t n, int64_t vocab, int n_actions, int d, EventsBwdWork* w) {
  Carve c(base);
  EventsBwdWork v;
  (void)vocab;
  const size_t rows = (size_t)std::max<int64_t>(n, 1);
  const int64_t win = window_size(n);
  const size_t windows = (size_t)std::max<int64_t>((n + win - 1) / win, 1);
  for (int i = 0; i < 2; ++i) {
    v.keys[i] = c.take<uint32_t>(rows);
    v.events[i] = c.take<uint32_t>(rows);
  }
  v.hist = c.take<int>((size_t)2 * sort_ctas(n) << kMaxBits);
  v.counter = c.take<unsigned>(1);
  v.first = c.take<float>(windows * d);
  v.last = c.take<float>(windows * d);
  v.first_key = c.take<uint32_t>(windows);
  v.open_key = c.take<uint32_t>(windows);
  v.action_part = c.take<float>(std::max((size_t)action_ctas(n), (windows + kHalves - 1) / kHalves) * n_actions * d);
  if (w) *w = v;
  return c.bytes();
}

sa_status events_bwd_run(const void* dX, sa_dtype dtype, const int32_t* ids, const uint8_t* acts, int64_t n,
                         int64_t vocab, int n_actions, int d, float* d_item, float* d_action, const EventsBwdWork& w,
                         cudaStream_t st) {
  if (!d_item && !d_action) return SA_OK;
  if (n == 0) {
    if (d_item) SA_CUDA(cudaMemsetAsync(d_item, 0, sizeof(float) * vocab * d, st));
    if (d_action) SA_CUDA(cudaMemsetAsync(d_action, 0, sizeof(float) * n_actions * d, st));
    return SA_OK;
  }
  if (dtype == SA_BF16)
    return run((const __nv_bfloat16*)dX, ids, acts, n, vocab, n_actions, d, d_item, d_action, w, st);
  return run((const float*)dX, ids, acts, n, vocab, n_actions, d, d_item, d_action, w, st);
}

}  // namespace sa
