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
// of the events.  The list is cut into equal windows, one per warp: runs inside a
// window are written at once, the sums of the runs that cross its ends are kept, and a
// second kernel adds those.  So every row of dX is read once and every warp has
// the same work however popular an item is (under Zipf(1.1) ids over a million items
// one item has 1 event in 8).  The same pass adds each row to its action's sum, in a
// table per warp in shared memory.
//
// Bound by memory: dX read once, the item gradient written once.  The sort is one
// cooperative launch (its CTAs exchange digit counts through memory between the passes'
// steps) that waits on latency and leaves the memory idle, so a thread of each CTA zeroes
// the whole item gradient meanwhile (most of it stays zero: a million items, 680K events)
// with bulk stores out of shared memory, a bounded number in flight: written by ordinary
// stores of half the warps, the zeros held up the sort's loads until they were all out
// (40 us for a load, 124 us for both; bulk stores of 16 KB 114, of 2 KB, a few at once, 103;
// zeros alone 82, sort alone 38).  The rows with events are written over that.  680K events
// of a million items (bf16 dX, d = 128), us: sort and zeros 103, windows 53, crossing runs 9: the
// call 174, 690 MB at 4.0 TB/s.
#include <algorithm>
#include <mutex>

#include "sa_internal.cuh"
#include "tc_ptx.cuh"
#include "tma_map.cuh"

namespace sa {

namespace {
constexpr int kMaxBits = 10;                 // of the id per pass: 1024 bins
constexpr int kSortThreads = 512, kSortWarps = kSortThreads / 32;   // sorting; one more warp zeroes
constexpr int kZeroBytes = 2048;             // a bulk store of zeros
// Bytes of zeros from which two stores are in flight, not one: faster alone, more in the way of the sort.  A
// replayed call's us, one and two (bf16 rows, cold L2):
//   table, GB          0.20       0.27       0.36       0.51       1.0
//   20,000 events    66,  68    80,  74    98,  84   127, 107   227, 188
//   200,000          82,  88    94,  97   113, 107   143, 127   244, 207
//   680,000         133, 141   139, 151   152, 164   184, 178   285, 261
//   2,000,000       278, 283   285, 295   301, 305   324, 324   413, 418
// (the border lies higher the more events there are to sort, which the rule does not follow)
constexpr int64_t kManyZeros = 256 << 20;
constexpr int kSortPer = 1024;               // events per sorting CTA, at least
constexpr int kAlone = 4096;                 // events that one CTA sorts alone (3000: 27 us a call, 40 with three CTAs)
// CTAs that add up each other's counts, a barrier less a pass, where more have them scanned by a warp per digit.  A
// replayed call's us, added and scanned: 6 to 12 CTAs 45, 49; 20 47, 51; 38 49, 51; 49 to 69 the same; 76 55,
// 53-55; 98 57, 55; 118 61, 57; 148 66, 61
constexpr int kFewCtas = 64;
constexpr int kHeld = 12;                    // keys (and events) that a sorting lane holds in registers
constexpr int kMinWin = 32;                  // list positions per window, at least
constexpr int kSumThreads = 256, kSumWarps = kSumThreads / 32;
constexpr int kCrossThreads = 512, kCrossWarps = kCrossThreads / 32;
constexpr int kWindowCtas = 3;               // window CTAs per SM: 16 tables take 64 KB of shared memory each
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
  __device__ uint2 at(int64_t i) const { return make_uint2(event_key(ids, acts, i, vocab, n_actions), (uint32_t)i); }
  __device__ bool outside(uint32_t key) const { return key == (uint32_t)vocab; }
};
struct FromList {
  const uint2* list;
  // written by other CTAs of this launch: not through L1
  __device__ uint2 at(int64_t i) const { return __ldcg(list + i); }
  __device__ bool outside(uint32_t) const { return false; }
};

// barrier of a CTA's sorting warps
__device__ __forceinline__ void sort_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kSortThreads) : "memory"); }

// Barrier number `round` (from 1) of the sorting CTAs over a counter that starts at zero.  All of
// them are resident (cooperative launch); the wait is bounded all the same: past the limit it sets
// the device error word, and the sort goes on over incomplete counts.  The list may then hold any
// words, so every kernel checks an index that comes from it before it is used.
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
  uint2* list[2];            // (key, event) after pass q in list[q & 1]: one scattered store per event
  int* hist;                 // [ctas][bins] digit counts of a pass
  int* before;               // [bins][ctas] the same of the earlier CTAs, and [bins] the digits' totals
  unsigned* counter;
  char* zero;                // the item gradient, and its bytes
  int64_t zeros;
  int* err;
};
// zeros, then counts [warps][bins], digit totals [bins], and the earlier CTAs' counts [bins]
constexpr int sort_smem(int bits) { return kZeroBytes + (kSortWarps + 2) * (1 << bits) * 4; }

// One pass over the digit at `shift`: moves the CTA's events behind those with smaller digits, and
// those with the same digit in earlier CTAs.  Each warp owns a contiguous part, counts its digits,
// and places its events in order, so equal digits keep their order.
template <class In>
__device__ void sort_pass(const In& in, const SortArgs& s, int q, int shift, int bits, int* smem, unsigned& round) {
  __shared__ int warp_sum[kSortWarps];
  const int bins = 1 << bits, cta = blockIdx.x;
  int *wcnt = smem, *totals = smem + kSortWarps * bins, *base = totals + bins;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  for (int b = threadIdx.x; b < kSortWarps * bins; b += kSortThreads) wcnt[b] = 0;
  sort_sync();
  const int64_t begin = min((int64_t)cta * s.per, s.n), end = min(begin + s.per, s.n);
  const int64_t size = ((end - begin + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
  const int64_t wb = min(begin + warp * size, end), we = min(wb + size, end);
  int* mine = wcnt + warp * bins;
  bool bad = false;
  // the first kHeld keys of each lane stay in registers until they are placed (under the writes of
  // the zeros a load takes microseconds); longer parts are read again, kHeld at a time
  uint2 held[kHeld];
  auto load = [&](int64_t i0) {
#pragma unroll
    for (int x = 0; x < kHeld; ++x) {
      const int64_t i = i0 + 32 * x + lane;
      held[x] = i < we ? in.at(i) : make_uint2(0u, 0u);
    }
  };
  for (int64_t i0 = wb + 32 * kHeld; i0 < we; i0 += 32 * kHeld) {
    load(i0);
#pragma unroll
    for (int x = 0; x < kHeld; ++x)
      if (i0 + 32 * x + lane < we) {
        bad |= in.outside(held[x].x);
        atomicAdd(&mine[(held[x].x >> shift) & (bins - 1)], 1);
      }
  }
  load(wb);
#pragma unroll
  for (int x = 0; x < kHeld; ++x)
    if (wb + 32 * x + lane < we) {
      bad |= in.outside(held[x].x);
      atomicAdd(&mine[(held[x].x >> shift) & (bins - 1)], 1);
    }
  if (bad) atomicOr(s.err, DEV_ERR_INDEX);
  sort_sync();
  // the CTA's counts; then totals[b]: all events with digit b, base[b]: those of earlier CTAs
  for (int b = threadIdx.x; b < bins; b += kSortThreads) {
    int total = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) total += wcnt[w * bins + b];
    if (s.ctas > 1) {
      s.hist[(int64_t)cta * bins + b] = total;
    } else {
      totals[b] = total;
      base[b] = 0;
    }
  }
  if (s.ctas > 1 && s.ctas <= kFewCtas) {
    // few CTAs: each adds up the others' counts itself, which saves a barrier
    grid_sync(s.counter, s.ctas, ++round, s.err);
    for (int b = threadIdx.x; b < bins; b += kSortThreads) {
      int total = 0, earlier = 0;
      for (int g0 = 0; g0 < s.ctas; g0 += 16) {
        int c[16];
#pragma unroll
        for (int x = 0; x < 16; ++x) c[x] = g0 + x < s.ctas ? __ldcg(s.hist + (int64_t)(g0 + x) * bins + b) : 0;
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          total += c[x];
          if (g0 + x < cta) earlier += c[x];
        }
      }
      base[b] = earlier;
      totals[b] = total;
    }
  } else if (s.ctas > 1) {
    grid_sync(s.counter, s.ctas, ++round, s.err);
    // a warp per digit scans it over the CTAs (every CTA reading all counts takes twice as long)
    for (int b = cta + s.ctas * warp; b < bins; b += s.ctas * kSortWarps) {
      int carry = 0;
      for (int g0 = 0; g0 < s.ctas; g0 += 128) {
        int c[4], incl[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int g = g0 + 32 * x + lane;
          c[x] = g < s.ctas ? __ldcg(s.hist + (int64_t)g * bins + b) : 0;
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          incl[x] = c[x];
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl[x], o);
            if (lane >= o) incl[x] += y;
          }
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int g = g0 + 32 * x + lane;
          if (g < s.ctas) s.before[(int64_t)b * s.ctas + g] = carry + incl[x] - c[x];
          carry += __shfl_sync(0xffffffffu, incl[x], 31);
        }
      }
      if (lane == 0) s.before[(int64_t)bins * s.ctas + b] = carry;
    }
    grid_sync(s.counter, s.ctas, ++round, s.err);
    for (int b = threadIdx.x; b < bins; b += kSortThreads) {
      base[b] = __ldcg(s.before + (int64_t)b * s.ctas + cta);
      totals[b] = __ldcg(s.before + (int64_t)bins * s.ctas + b);
    }
  }
  sort_sync();
  // each warp's first place for each digit
  int carry = 0;
  for (int b0 = 0; b0 < bins; b0 += kSortThreads) {
    const int b = b0 + threadIdx.x;
    const int total = b < bins ? totals[b] : 0;
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
  uint2* list = s.list[q & 1];
  for (int64_t i0 = wb; i0 < we; i0 += 32 * kHeld) {
    if (i0 > wb) load(i0);
#pragma unroll
    for (int x = 0; x < kHeld; ++x) {
      if (i0 + 32 * x >= we) break;
      const bool there = i0 + 32 * x + lane < we;
      const int digit = (int)((held[x].x >> shift) & (bins - 1));
      unsigned same = __ballot_sync(0xffffffffu, there);          // the lanes with this digit
      for (int i = 0; i < bits; ++i) {
        const unsigned set = __ballot_sync(0xffffffffu, (digit >> i) & 1);
        same &= (digit >> i) & 1 ? set : ~set;
      }
      const int rank = __popc(same & ((1u << lane) - 1));
      const int at = there ? mine[digit] : 0;
      __syncwarp();
      if (there) {
        if (rank == 0) mine[digit] = at + __popc(same);
        if ((unsigned)(at + rank) < (uint64_t)s.n) list[at + rank] = held[x];
      }
      __syncwarp();
    }
  }
  if (s.ctas > 1 && q + 1 < s.passes) grid_sync(s.counter, s.ctas, ++round, s.err);
  else sort_sync();
}

__global__ void __launch_bounds__(kSortThreads + 32, 1) sort_events_kernel(SortArgs s) {
  extern __shared__ __align__(128) char smem_raw[];
  let_next_start();
  if (threadIdx.x >= kSortThreads) {
    const int lane = threadIdx.x % 32;
    for (int i = lane; i < kZeroBytes / 16; i += 32) ((float4*)smem_raw)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    tc::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      const int64_t step = (int64_t)gridDim.x * kZeroBytes, first = (int64_t)blockIdx.x * kZeroBytes;
      if (s.zeros >= kManyZeros) {
        for (int64_t at = first; at < s.zeros; at += step)
          tc::bulk_store_limited<2>(s.zero + at, smem_raw, (uint32_t)min((int64_t)kZeroBytes, s.zeros - at));
      } else {
        for (int64_t at = first; at < s.zeros; at += step)
          tc::bulk_store_limited<1>(s.zero + at, smem_raw, (uint32_t)min((int64_t)kZeroBytes, s.zeros - at));
      }
      tc::bulk_store_wait();
    }
    return;
  }
  if ((int)blockIdx.x >= s.ctas) return;
  int* smem = (int*)(smem_raw + kZeroBytes);
  unsigned round = 0;
  for (int q = 0; q < s.passes; ++q) {
    const int shift = s.bits * q / s.passes, bits = s.bits * (q + 1) / s.passes - shift;
    if (q == 0) sort_pass(s.in, s, q, shift, bits, smem, round);
    else sort_pass(FromList{s.list[(q - 1) & 1]}, s, q, shift, bits, smem, round);
  }
}

// 4 columns of a row, as they lie in memory
__device__ __forceinline__ uint2 load_raw(const __nv_bfloat16* p) { return __ldcs((const uint2*)p); }
__device__ __forceinline__ float4 load_raw(const float* p) { return __ldcs((const float4*)p); }
struct Cols {                                // 4 fp32 columns, added in pairs
  float2 a, b;
};
__device__ __forceinline__ Cols widen(const uint2& w) {
  return {make_float2(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u)),
          make_float2(__uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u))};
}
__device__ __forceinline__ Cols widen(const float4& r) { return {make_float2(r.x, r.y), make_float2(r.z, r.w)}; }
__device__ __forceinline__ Cols zero_cols() { return {make_float2(0.f, 0.f), make_float2(0.f, 0.f)}; }
__device__ __forceinline__ void add_cols(Cols& x, const Cols& y) {
  x.a = __fadd2_rn(x.a, y.a);
  x.b = __fadd2_rn(x.b, y.b);
}
__device__ __forceinline__ Cols load_cols(const float* p) { return widen(*(const float4*)p); }
__device__ __forceinline__ void store_cols(float* p, const Cols& c) {
  *(float4*)p = make_float4(c.a.x, c.a.y, c.b.x, c.b.y);
}
template <class T>
constexpr int batch_rows() { return sizeof(T) == 2 ? 16 : 8; }   // rows in flight per warp: 32 registers

// the CTA's tables of action sums (per warp [n_actions][32 lanes] float4), added in order, to
// out[n_actions][d] (columns c0 .. c0 + 127 of it)
__device__ __forceinline__ void store_tables(const float4* tables, int count, int n_actions, int c0, int d, float* out) {
  for (int e = threadIdx.x; e < n_actions * 32; e += blockDim.x) {
    const int col = c0 + e % 32 * 4;
    Cols acc = widen(tables[e]);
    for (int h = 1; h < count; ++h) add_cols(acc, widen(tables[h * n_actions * 32 + e]));
    if (col < d) store_cols(out + (int64_t)(e / 32) * d + col, acc);
  }
}
__device__ __forceinline__ void add_to_table(float4* row, const Cols& v) {
  Cols s = widen(*row);
  add_cols(s, v);
  *row = make_float4(s.a.x, s.a.y, s.b.x, s.b.y);
}

constexpr uint32_t kNone = 0xFFFFFFFFu;      // no item

// Window w is list positions [win w, win (w + 1)), a warp's.  It walks them row by row: a run that
// lies inside is written to its table row; the sum before the window's first run head goes to
// first[w], that of a run which starts in it and goes on behind it to last[w]; first_key[w] and
// open_key[w] (kNone: no run goes on) tell the second kernel which.  With kActions every row is also
// added to the warp's table of action sums; the CTA's tables go to action_part[CTA][n_actions][d].
template <class T, bool kActions>
__global__ void __launch_bounds__(kSumThreads, kWindowCtas) window_rows_kernel(
    const T* __restrict__ dX, const uint2* list, const uint8_t* __restrict__ acts, int64_t n, int64_t win, int64_t vocab,
    int n_actions, int d, float* first, float* last, uint32_t* first_key, uint32_t* open_key, float* d_item,
    float* action_part) {
  extern __shared__ float4 tables[];                 // [kSumWarps][n_actions][32]
  let_next_start();
  wait_for_previous();
  constexpr int kBatch = batch_rows<T>();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  float4* mine = tables + warp * n_actions * 32 + lane;
  const int64_t w = (int64_t)blockIdx.x * kSumWarps + warp, p0 = min(w * win, n), p1 = min(p0 + win, n);
  for (int c0 = 0; c0 < d; c0 += 128) {
    const int c = c0 + lane * 4;
    const bool in = c < d;
    if (kActions)
      for (int a = 0; a < n_actions; ++a) mine[a * 32] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p0 < p1) {
      const T* col = dX + (in ? c : 0);              // idle lanes read (and drop) the first columns
      Cols acc = zero_cols();
      uint32_t run = p0 > 0 ? list[p0 - 1].x : kNone;  // key of the run that acc belongs to
      const uint32_t behind = p1 < n ? list[p1].x : kNone;
      bool inside = false;                           // a head was seen: acc starts at it
      // (an event number is below n, unless the sort gave up at a barrier)
      auto list_at = [&](int64_t i) {
        const uint2 x = list[i];
        return make_uint2(x.x, x.y < (uint64_t)n ? x.y : 0u);
      };
      uint2 next = p0 + lane < p1 ? list_at(p0 + lane) : make_uint2(kNone, 0u);
      if (lane == 0 && c0 == 0) first_key[w] = next.x;
      for (int64_t b = p0; b < p1; b += 32) {
        const int cnt = (int)min((int64_t)32, p1 - b);
        const uint32_t key = next.x, ev = next.y;
        if (b + 32 + lane < p1) next = list_at(b + 32 + lane);   // the next 32 positions, a step ahead
        int act = -1;
        if (kActions && lane < cnt && key < (uint32_t)vocab) {
          const int a = acts[ev];                    // below n_actions, unless the key is not this event's
          act = a < n_actions ? a : -1;
        }
        uint32_t prev = __shfl_up_sync(0xffffffffu, key, 1);
        if (lane == 0) prev = run;
        const unsigned heads = __ballot_sync(0xffffffffu, lane < cnt && key != prev);
#pragma unroll
        for (int j = 0; j < 32; j += kBatch) {
          if (j >= cnt) break;
          decltype(load_raw(dX)) x[kBatch];
#pragma unroll
          for (int q = 0; q < kBatch; ++q)           // behind the window's end: event 0, dropped
            x[q] = load_raw(col + (int64_t)__shfl_sync(0xffffffffu, ev, j + q) * d);
#pragma unroll
          for (int q = 0; q < kBatch; ++q) {
            if (j + q >= cnt) break;
            if ((heads >> (j + q)) & 1) {            // the same for the whole warp
              if (in) {
                if (!inside) store_cols(first + w * d + c, acc);
                else if (run < (uint32_t)vocab) store_cols(d_item + (int64_t)run * d + c, acc);
              }
              inside = true;
              run = __shfl_sync(0xffffffffu, key, j + q);
              acc = zero_cols();
            }
            const Cols v = widen(x[q]);
            add_cols(acc, v);
            if (kActions) {
              const int a = __shfl_sync(0xffffffffu, act, j + q);
              if (a >= 0) add_to_table(mine + a * 32, v);
            }
          }
        }
      }
      const bool on = behind == run;                 // the run goes on in the next window
      if (in) {
        if (!inside) store_cols(first + w * d + c, acc);
        else if (on) store_cols(last + w * d + c, acc);
        else if (run < (uint32_t)vocab) store_cols(d_item + (int64_t)run * d + c, acc);
      }
      if (lane == 0 && c0 == 0) open_key[w] = inside && on && run < (uint32_t)vocab ? run : kNone;
    }
    if (kActions) {
      __syncthreads();
      store_tables(tables, kSumWarps, n_actions, c0, d, action_part + (int64_t)blockIdx.x * n_actions * d);
      __syncthreads();
    }
  }
}

// sum of rows [b, e) of a [., pitch] array at 4 columns, in order
__device__ __forceinline__ Cols sum_range(const float* part, int64_t b, int64_t e, int64_t pitch, bool in) {
  Cols acc = zero_cols();
  if (!in) return acc;
  int64_t v = b;
  for (; v + 16 <= e; v += 16) {
    Cols x[16];
#pragma unroll
    for (int q = 0; q < 16; ++q) x[q] = load_cols(part + (v + q) * pitch);
#pragma unroll
    for (int q = 0; q < 16; ++q) add_cols(acc, x[q]);
  }
  if (v < e) {                               // the rest, in one batch too
    Cols x[15];
#pragma unroll
    for (int q = 0; q < 15; ++q) x[q] = v + q < e ? load_cols(part + (v + q) * pitch) : zero_cols();
#pragma unroll
    for (int q = 0; q < 15; ++q) add_cols(acc, x[q]);
  }
  return acc;
}

// the warps' sums added in order; the result is in warp 0
__device__ __forceinline__ Cols sum_warps(const Cols& mine, Cols (*part)[32]) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  __syncthreads();
  part[warp][lane] = mine;
  __syncthreads();
  Cols acc = part[0][lane];
  for (int w = 1; w < kCrossWarps; ++w) add_cols(acc, part[w][lane]);
  return acc;
}

// CTAs [0, action_ctas): the action sums, one action each, from `parts` CTAs' tables.  The others: a
// warp per window whose last run goes on: the run's sum is last[w] + first[w + 1] + ... up to the
// window where it ends.  Runs over 32 windows or more are added by the whole CTA.
__global__ void __launch_bounds__(kCrossThreads) crossing_rows_kernel(
    const uint32_t* first_key, const uint32_t* open_key, int64_t windows, int d, const float* first, const float* last,
    float* d_item, int action_ctas, const float* action_part, int parts, float* d_action) {
  __shared__ Cols part[kCrossWarps][32];
  __shared__ int64_t long_end[kCrossWarps];
  wait_for_previous();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if ((int)blockIdx.x < action_ctas) {
    const int a = (int)blockIdx.x;
    for (int c0 = 0; c0 < d; c0 += 128) {
      const int c = c0 + lane * 4;
      const Cols acc = sum_warps(sum_range(action_part + (int64_t)a * d + c, (int64_t)parts * warp / kCrossWarps,
                                           (int64_t)parts * (warp + 1) / kCrossWarps, (int64_t)action_ctas * d, c < d), part);
      if (warp == 0 && c < d) store_cols(d_action + (int64_t)a * d + c, acc);
    }
    return;
  }
  const int64_t w0 = (int64_t)(blockIdx.x - action_ctas) * kCrossWarps, w = w0 + warp;
  const uint32_t run = w + 1 < windows ? open_key[w] : kNone;
  int64_t end = 0;                                   // one behind the last window of the run (0: none to add)
  bool is_long = false;
  if (run != kNone) {
    // window v > w holds a part of the run iff its first key is the run's
    const int64_t v = w + 1 + lane;
    const int more = __popc(__ballot_sync(0xffffffffu, v < windows && first_key[v] == run));
    end = w + 1 + more;
    is_long = more == 32;
    if (is_long) {                                   // find the end, 32 probes at a time
      int64_t lo = end, hi = windows;                // the windows before lo start with the run, hi does not
      while (lo < hi) {
        const int64_t step = (hi - lo + 31) / 32, at = lo + lane * step;
        const int yes = __popc(__ballot_sync(0xffffffffu, at < hi && first_key[at] == run));
        if (yes == 0) break;
        hi = min(hi, lo + yes * step);
        lo = lo + (yes - 1) * step + 1;
      }
      end = lo;
    }
  }
  if (lane == 0) long_end[warp] = is_long ? end : 0;
  if (end > 0 && !is_long)
    for (int c = lane * 4; c < d; c += 128) {
      Cols acc = load_cols(last + w * d + c);
      add_cols(acc, sum_range(first + c, w + 1, end, d, true));
      store_cols(d_item + (int64_t)run * d + c, acc);
    }
  __syncthreads();
  for (int i = 0; i < kCrossWarps; ++i) {
    const int64_t e = long_end[i], b = w0 + i;
    if (e == 0) continue;
    const int64_t cnt = e - b - 1;
    const uint32_t key = open_key[b];
    for (int c0 = 0; c0 < d; c0 += 128) {
      const int c = c0 + lane * 4;
      Cols acc = sum_range(first + c, b + 1 + cnt * warp / kCrossWarps, b + 1 + cnt * (warp + 1) / kCrossWarps, d, c < d);
      if (warp == 0 && c < d) add_cols(acc, load_cols(last + b * d + c));
      acc = sum_warps(acc, part);
      if (warp == 0 && c < d) store_cols(d_item + (int64_t)key * d + c, acc);
    }
  }
}

// part[CTA][action][d]: the sums of the CTA's contiguous events by action (more actions than the
// window kernel's tables, or the action gradient alone).  Each warp adds its own contiguous part
// into its own table in shared memory; the tables are added in order.
template <class T>
__global__ void action_rows_kernel(const T* __restrict__ dX, const int32_t* __restrict__ ids,
                                   const uint8_t* __restrict__ acts, int64_t n, int64_t per, int64_t vocab,
                                   int n_actions, int d, float* __restrict__ part, int* err) {
  extern __shared__ float4 tables[];                 // [warps][n_actions][32]
  let_next_start();
  constexpr int kBatch = batch_rows<T>();
  const int warp = threadIdx.x / 32, warps = blockDim.x / 32, lane = threadIdx.x % 32;
  const int c = blockIdx.y * 128 + lane * 4;
  const bool in = c < d;
  float4* mine = tables + warp * n_actions * 32 + lane;
  for (int a = 0; a < n_actions; ++a) mine[a * 32] = make_float4(0.f, 0.f, 0.f, 0.f);
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
#pragma unroll
    for (int j = 0; j < 32; j += kBatch) {
      if (j >= cnt) break;
      decltype(load_raw(dX)) x[kBatch];
#pragma unroll
      for (int q = 0; q < kBatch; ++q)
        if (j + q < cnt && in) x[q] = load_raw(dX + (i0 + j + q) * d + c);
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        const int aq = __shfl_sync(0xffffffffu, a, j + q);
        if (j + q < cnt && aq >= 0 && in) add_to_table(mine + aq * 32, widen(x[q]));
      }
    }
  }
  if (bad && blockIdx.y == 0) atomicOr(err, DEV_ERR_INDEX);
  __syncthreads();
  store_tables(tables, warps, n_actions, blockIdx.y * 128, d, part + (int64_t)blockIdx.x * n_actions * d);
}

int key_bits(int64_t vocab) {
  int b = 2;                                          // a digit of at least 4 bins
  while (((int64_t)1 << b) <= vocab) ++b;             // keys 0 .. vocab
  return b;
}
int sort_ctas(int64_t n) {
  if (n <= kAlone) return 1;
  return (int)std::max<int64_t>(1, std::min<int64_t>(device_info().sm_count, (n + kSortPer - 1) / kSortPer));
}
// warps of an action CTA: their tables (512 bytes per action) fit in 128 KB of shared memory
int action_warps(int n_actions) { return std::max(1, std::min(kSumWarps, 256 / n_actions)); }
int action_ctas(int64_t n) {
  return (int)std::max<int64_t>(1, std::min<int64_t>(4 * device_info().sm_count, (n + 255) / 256));
}
// Windows: one per warp of the CTAs that are resident at once, so that all have the same work.
int64_t window_size(int64_t n) {
  const int64_t warps = (int64_t)kWindowCtas * device_info().sm_count * kSumWarps;
  return std::max<int64_t>(kMinWin, (n + warps - 1) / warps);
}

// whether the window kernel adds up the actions too
bool fused_actions(const float* d_item, const float* d_action, int n_actions) {
  return d_item && d_action && n_actions <= kFusedActions;
}

// The windows' sums of the list's rows into d_item, and the action sums with them if fused_actions.
template <class T>
sa_status sum_windows(const T* dX, const uint2* list, const uint8_t* acts, int64_t n, int64_t vocab, int n_actions, int d,
                      float* d_item, float* d_action, const EventsBwdWork& w, cudaStream_t st) {
  static unsigned long long done = 0;
  static std::mutex mu;
  const int64_t win = window_size(n), windows = (n + win - 1) / win;
  const int ctas = (int)((windows + kSumWarps - 1) / kSumWarps);
  if (fused_actions(d_item, d_action, n_actions)) {
    const int smem = kSumWarps * n_actions * 512;
    set_smem_limit_once((const void*)window_rows_kernel<T, true>, kSumWarps * kFusedActions * 512, &done, mu);
    SA_TIMED("window_rows_kernel", st,
             launch_after(window_rows_kernel<T, true>, ctas, kSumThreads, smem, st, dX, list, acts, n, win, vocab, n_actions,
                          d, w.first, w.last, w.first_key, w.open_key, d_item, w.action_part));
  } else {
    SA_TIMED("window_rows_kernel", st,
             launch_after(window_rows_kernel<T, false>, ctas, kSumThreads, 0, st, dX, list, acts, n, win, vocab, 0, d,
                          w.first, w.last, w.first_key, w.open_key, d_item, nullptr));
  }
  return SA_OK;
}

// The runs that cross windows into d_item, and the action sums from their parts.
sa_status sum_crossing(int64_t n, int n_actions, int d, float* d_item, float* d_action, const EventsBwdWork& w,
                       cudaStream_t st) {
  const int64_t win = window_size(n), windows = (n + win - 1) / win;
  const int parts = fused_actions(d_item, d_action, n_actions) ? (int)((windows + kSumWarps - 1) / kSumWarps) : action_ctas(n);
  const int ac = d_action ? n_actions : 0;
  SA_TIMED("crossing_rows_kernel", st,
           launch_after(crossing_rows_kernel, ac + (d_item ? (int)((windows + kCrossWarps - 1) / kCrossWarps) : 0),
                        kCrossThreads, 0, st, w.first_key, w.open_key,
                        windows, d, w.first, w.last, d_item, ac, w.action_part, parts, d_action));
  return SA_OK;
}

template <class T>
sa_status run(const T* dX, const int32_t* ids, const uint8_t* acts, int64_t n, int64_t vocab, int n_actions, int d,
              float* d_item, float* d_action, const EventsBwdWork& w, cudaStream_t st) {
  static unsigned long long done[2] = {};          // one per kernel
  static std::mutex mu;
  int* err = device_status_word();
  if (d_action && !fused_actions(d_item, d_action, n_actions)) {
    const int warps = action_warps(n_actions), parts = action_ctas(n);
    const int smem = warps * n_actions * 512;
    set_smem_limit_once((const void*)action_rows_kernel<T>, 256 * 512, &done[0], mu);
    SA_TIMED("action_rows_kernel", st,
             (action_rows_kernel<T><<<dim3(parts, (d + 127) / 128), warps * 32, smem, st>>>(
                 dX, ids, acts, n, (n + parts - 1) / parts, vocab, n_actions, d, w.action_part, err)));
  }
  if (d_item) {
    const int bits = key_bits(vocab), passes = (bits + kMaxBits - 1) / kMaxBits;
    SortArgs s{{ids, acts, vocab, n_actions}, n, 0, bits, passes, sort_ctas(n), {w.list[0], w.list[1]},
               w.hist, w.before, w.counter, (char*)d_item, vocab * d * 4, err};
    s.per = (n + s.ctas - 1) / s.ctas;
    set_smem_limit_once((const void*)sort_events_kernel, sort_smem(kMaxBits), &done[1], mu);
    const int smem = sort_smem((bits + passes - 1) / passes);
    if (s.ctas == 1) {
      SA_TIMED("sort_events_kernel", st,
               (sort_events_kernel<<<device_info().sm_count, kSortThreads + 32, smem, st>>>(s)));
    } else {
      SA_CUDA(cudaMemsetAsync(w.counter, 0, sizeof(unsigned), st));
      void* args[] = {&s};
      SA_TIMED("sort_events_kernel", st,
               cudaLaunchCooperativeKernel((const void*)sort_events_kernel, dim3(device_info().sm_count),
                                           dim3(kSortThreads + 32), args, (size_t)smem, st));
    }
    const uint2* list = w.list[(passes - 1) & 1];
    const sa_status done_windows = sum_windows(dX, list, acts, n, vocab, n_actions, d, d_item, d_action, w, st);
    if (done_windows != SA_OK) return done_windows;
  }
  return sum_crossing(n, n_actions, d, d_item, d_action, w, st);
}
}  // namespace

size_t events_bwd_layout(void* base, int64_t n, int64_t vocab, int n_actions, int d, EventsBwdWork* w) {
  Carve c(base);
  EventsBwdWork v;
  (void)vocab;
  const size_t rows = (size_t)std::max<int64_t>(n, 1);
  const int64_t win = window_size(n);
  const size_t windows = (size_t)std::max<int64_t>((n + win - 1) / win, 1);
  for (int i = 0; i < 2; ++i) v.list[i] = c.take<uint2>(rows);
  v.hist = c.take<int>((size_t)sort_ctas(n) << kMaxBits);
  v.before = c.take<int>((size_t)(sort_ctas(n) + 1) << kMaxBits);
  v.counter = c.take<unsigned>(1);
  v.first = c.take<float>(windows * d);
  v.last = c.take<float>(windows * d);
  v.first_key = c.take<uint32_t>(windows);
  v.open_key = c.take<uint32_t>(windows);
  v.action_part = c.take<float>(std::max((size_t)action_ctas(n), (windows + kSumWarps - 1) / kSumWarps) * n_actions * d);
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

sa_status selftest_unsorted_events(const void* list, const float* dX, const uint8_t* acts, int64_t n, int64_t vocab,
                                   int n_actions, int d, float* d_item, float* d_action, const EventsBwdWork& w,
                                   cudaStream_t st) {
  SA_CUDA(cudaMemsetAsync(d_item, 0, sizeof(float) * vocab * d, st));
  const sa_status s = sum_windows(dX, (const uint2*)list, acts, n, vocab, n_actions, d, d_item, d_action, w, st);
  return s != SA_OK ? s : sum_crossing(n, n_actions, d, d_item, d_action, w, st);
}

}  // namespace sa
