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
// of the events.  The list is cut into windows of 64 positions, one per warp: runs
// inside a window are written at once, the sums of the runs that cross its ends are
// kept, and a second kernel adds those.  So every row of dX is read once and every
// warp has the same work however popular an item is (under Zipf(1.1) ids over a
// million items one item has 1 event in 8).  The same pass adds each row to its
// action's sum, in a table per warp in shared memory.
//
// Bound by memory: dX read once, the item gradient written once.  Most of it is zero
// rows (a million items, 680K events); they are written by extra CTAs of the sort's
// kernels, which by themselves wait on latency and leave the memory idle.
#include <algorithm>
#include <mutex>

#include "sa_internal.cuh"
#include "tma_map.cuh"

namespace sa {

namespace {
constexpr int kMaxBits = 10;                 // of the id per pass: 1024 bins
constexpr int kSortThreads = 512, kSortWarps = kSortThreads / 32;
constexpr int kSmallN = 4096;                // events that one CTA sorts in one launch
constexpr int kWin = 64;                     // list positions per window
constexpr int kSumThreads = 256, kSumWarps = kSumThreads / 32;
constexpr int kLong = 32;                    // windows of a run that one warp adds; longer: the whole CTA
constexpr int kFusedActions = 16;            // action tables that the window kernel keeps in shared memory

struct Pass {
  int shift, bits;
  int64_t n, per;          // events, and events per CTA
};

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
  __device__ uint32_t key(int64_t i) const { return keys[i]; }
  __device__ uint32_t event(int64_t i) const { return events[i]; }
  __device__ bool outside(uint32_t) const { return false; }
};

// hist[CTA][bin]: the CTA's events with each digit.  The first pass also marks the items that
// have events in `seen` (a bit per item).
template <class In>
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(In in, Pass ps, int* __restrict__ hist,
                                                                  unsigned* __restrict__ seen, int* err) {
  __shared__ int cnt[1 << kMaxBits];
  const int bins = 1 << ps.bits;
  for (int b = threadIdx.x; b < bins; b += kSortThreads) cnt[b] = 0;
  __syncthreads();
  const int64_t begin = (int64_t)blockIdx.x * ps.per, end = min(begin + ps.per, ps.n);
  for (int64_t i = begin + threadIdx.x; i < end; i += kSortThreads) {
    const uint32_t key = in.key(i);
    atomicAdd(&cnt[(key >> ps.shift) & (bins - 1)], 1);
    if (in.outside(key)) {
      atomicOr(err, DEV_ERR_INDEX);
    } else if (seen) {
      const unsigned bit = 1u << (key & 31);
      if (!(__ldcg(seen + (key >> 5)) & bit)) atomicOr(seen + (key >> 5), bit);
    }
  }
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += kSortThreads) hist[(int64_t)blockIdx.x * bins + b] = cnt[b];
}

// Zero rows of the item gradient that no event names: table rows [begin, end), `d` floats each,
// spread over the CTA's and its peers' warps; with seen = NULL all of them.
struct ZeroRows {
  float* out;
  const unsigned* seen;
  int64_t begin, end;
  int d;
};
__device__ __forceinline__ void zero_rows(const ZeroRows& z, int cta, int ctas) {
  const int lane = threadIdx.x % 32;
  const int64_t warp = (int64_t)cta * (blockDim.x / 32) + threadIdx.x / 32, warps = (int64_t)ctas * (blockDim.x / 32);
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  // 32 rows (one word of `seen`) at a time
  for (int64_t w = z.begin / 32 + warp; w * 32 < z.end; w += warps) {
    const unsigned have = z.seen ? z.seen[w] : 0u;
    const int64_t r0 = w * 32, r1 = min(r0 + 32, z.end);
    for (int64_t r = max(r0, z.begin); r < r1; ++r) {
      if ((have >> (r - r0)) & 1) continue;
      for (int c = lane * 4; c < z.d; c += 128) *(float4*)(z.out + r * z.d + c) = zero;
    }
  }
}

// Shared memory of a sorting CTA: wcnt [kSortWarps][bins], base [bins], half [2][bins]
struct SortSmem {
  int *wcnt, *base, *half;
  __device__ SortSmem(int* smem, int bins) : wcnt(smem), base(smem + kSortWarps * bins), half(base + bins) {}
};
constexpr int sort_smem(int bits) { return (kSortWarps + 3) * (1 << bits) * 4; }

// Moves the CTA's events [begin, end) to their places in (keys, events): behind those with smaller
// digits, and those with the same digit in earlier CTAs (hist, `ctas` of them; NULL: there is one
// CTA).  Each warp owns a contiguous part, counts its digits, and places its events in order, so
// equal digits keep their order.
template <class In>
__device__ void place(const In& in, const Pass& ps, int cta, int ctas, const int* __restrict__ hist, int* smem,
                      uint32_t* __restrict__ keys, uint32_t* __restrict__ events) {
  __shared__ int warp_sum[kSortWarps];
  const int bins = 1 << ps.bits;
  const SortSmem sm(smem, bins);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  for (int b = threadIdx.x; b < kSortWarps * bins; b += kSortThreads) sm.wcnt[b] = 0;
  __syncthreads();
  const int64_t begin = (int64_t)cta * ps.per, end = min(begin + ps.per, ps.n);
  const int64_t size = ((end - begin + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
  const int64_t wb = min(begin + warp * size, end), we = min(wb + size, end);
  int* mine = sm.wcnt + warp * bins;
  for (int64_t i = wb + lane; i < we; i += 32) atomicAdd(&mine[(in.key(i) >> ps.shift) & (bins - 1)], 1);
  // half[h][b]: events with digit b of the CTAs g = h mod 2; base[b]: of the earlier CTAs
  if (hist) {
    // two halves of the CTAs, four bins per thread (bins >= 4)
    const int quads = bins / 4, q = threadIdx.x % quads, h = threadIdx.x / quads;
    int4 total = make_int4(0, 0, 0, 0), before = make_int4(0, 0, 0, 0);
    if (h < 2) {
#pragma unroll 16
      for (int g = h; g < ctas; g += 2) {
        const int4 c = *(const int4*)(hist + (int64_t)g * bins + 4 * q);
        total.x += c.x; total.y += c.y; total.z += c.z; total.w += c.w;
        if (g < cta) { before.x += c.x; before.y += c.y; before.z += c.z; before.w += c.w; }
      }
      *(int4*)(sm.half + h * bins + 4 * q) = total;
      if (h == 0) *(int4*)(sm.base + 4 * q) = before;
    }
    __syncthreads();
    if (h == 1) {
      int4 o = *(int4*)(sm.base + 4 * q);
      o.x += before.x; o.y += before.y; o.z += before.z; o.w += before.w;
      *(int4*)(sm.base + 4 * q) = o;
    }
  } else {
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += kSortThreads) {
      int total = 0;
      for (int w = 0; w < kSortWarps; ++w) total += sm.wcnt[w * bins + b];
      sm.base[b] = 0;
      sm.half[b] = total;
      sm.half[bins + b] = 0;
    }
  }
  __syncthreads();
  // each warp's first place for each digit
  int carry = 0;
  for (int b0 = 0; b0 < bins; b0 += kSortThreads) {
    const int b = b0 + threadIdx.x;
    const int total = b < bins ? sm.half[b] + sm.half[bins + b] : 0;
    int incl = total;
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int off = carry, all = carry;
    for (int w = 0; w < kSortWarps; ++w) {
      if (w < warp) off += warp_sum[w];
      all += warp_sum[w];
    }
    carry = all;
    if (b < bins) {
      int run = off + incl - total + sm.base[b];
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) {
        const int c = sm.wcnt[w * bins + b];
        sm.wcnt[w * bins + b] = run;
        run += c;
      }
    }
    __syncthreads();
  }
  for (int64_t i0 = wb; i0 < we; i0 += 32) {
    const int64_t i = i0 + lane;
    const bool there = i < we;
    const uint32_t key = there ? in.key(i) : 0u;
    const int digit = there ? (int)((key >> ps.shift) & (bins - 1)) : -1;
    const unsigned same = __match_any_sync(0xffffffffu, digit);
    const int rank = __popc(same & ((1u << lane) - 1));
    const int at = there ? mine[digit] : 0;
    __syncwarp();
    if (there) {
      if (rank == 0) mine[digit] = at + __popc(same);
      keys[at + rank] = key;
      events[at + rank] = in.event(i);
    }
    __syncwarp();
  }
}

// CTAs [0, ctas) sort, the others write zero rows
template <class In>
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(In in, Pass ps, int ctas, const int* __restrict__ hist,
                                                                  uint32_t* __restrict__ keys,
                                                                  uint32_t* __restrict__ events, ZeroRows z) {
  extern __shared__ __align__(16) int smem[];
  if ((int)blockIdx.x >= ctas) {
    zero_rows(z, (int)blockIdx.x - ctas, (int)gridDim.x - ctas);
    return;
  }
  place(in, ps, (int)blockIdx.x, ctas, hist, smem, keys, events);
}

// All passes of a short list in CTA 0 (into buffer (passes - 1) & 1); the others write zero rows
struct Buffers {
  uint32_t *keys[2], *events[2];
};
__global__ void __launch_bounds__(kSortThreads) sort_small_kernel(FromEvents in, int64_t n, int bits, int passes,
                                                                  Buffers buf, ZeroRows z, int* err) {
  extern __shared__ __align__(16) int smem[];
  if (blockIdx.x > 0) {
    zero_rows(z, (int)blockIdx.x - 1, (int)gridDim.x - 1);
    return;
  }
  for (int64_t i = threadIdx.x; i < n; i += kSortThreads)
    if (in.outside(in.key(i))) atomicOr(err, DEV_ERR_INDEX);
  for (int q = 0; q < passes; ++q) {
    const int shift = bits * q / passes;
    const Pass ps{shift, bits * (q + 1) / passes - shift, n, n};
    if (q == 0) {
      place(in, ps, 0, 1, nullptr, smem, buf.keys[0], buf.events[0]);
    } else {
      const FromList from{buf.keys[(q - 1) & 1], buf.events[(q - 1) & 1]};
      place(from, ps, 0, 1, nullptr, smem, buf.keys[q & 1], buf.events[q & 1]);
    }
    __syncthreads();                                 // the next pass reads what every warp wrote
  }
}

__device__ __forceinline__ float4 row4(const __nv_bfloat16* p) {
  const uint2 w = *(const uint2*)p;
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xFFFF0000u));
}
__device__ __forceinline__ float4 row4(const float* p) { return *(const float4*)p; }
__device__ __forceinline__ void add4(float4& a, const float4& b) {
  a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
}

// Window w is list positions [kWin w, kWin (w + 1)).  A warp walks its windows row by row: a run
// that lies inside is written to its table row; the sum before the window's first run head goes to
// first[w], that of a run which goes on behind the window to last[w].  With kActions every row is
// also added to the warp's table of action sums; the CTA's tables are added in order at the end,
// into action_part[CTA][n_actions][d].
template <class T, bool kActions>
__global__ void __launch_bounds__(kSumThreads) window_rows_kernel(const T* __restrict__ dX,
                                                                  const uint32_t* __restrict__ keys,
                                                                  const uint32_t* __restrict__ events,
                                                                  const uint8_t* __restrict__ acts, int64_t n,
                                                                  int64_t vocab, int n_actions, int d,
                                                                  float* __restrict__ first, float* __restrict__ last,
                                                                  float* __restrict__ d_item,
                                                                  float* __restrict__ action_part) {
  extern __shared__ float4 table[];                  // [kSumWarps][n_actions][32]
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  float4* mine = table + warp * n_actions * 32;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  const int64_t windows = (n + kWin - 1) / kWin, stride = (int64_t)gridDim.x * kSumWarps;
  for (int c0 = 0; c0 < d; c0 += 128) {
    const int c = c0 + lane * 4;
    const bool in = c < d;
    if (kActions)
      for (int a = 0; a < n_actions; ++a) mine[a * 32 + lane] = zero;
    for (int64_t w = (int64_t)blockIdx.x * kSumWarps + warp; w < windows; w += stride) {
      const int64_t p0 = w * kWin;
      float4 acc = zero;
      uint32_t run = p0 > 0 ? keys[p0 - 1] : 0xFFFFFFFFu;      // key of the run that acc belongs to
      bool inside = false;                                      // a head was seen: acc starts at it
      for (int b = 0; b < kWin && p0 + b < n; b += 32) {
        const int cnt = (int)min((int64_t)32, n - p0 - b);
        const uint32_t key = lane < cnt ? keys[p0 + b + lane] : 0xFFFFFFFFu;
        const uint32_t ev = lane < cnt ? events[p0 + b + lane] : 0u;
        int act = 0;
        if (kActions && lane < cnt && key < (uint32_t)vocab) act = acts[ev];
        for (int j = 0; j < cnt; j += 8) {
          float4 x[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const uint32_t e = __shfl_sync(0xffffffffu, ev, j + q);
            x[q] = j + q < cnt && in ? row4(dX + (int64_t)e * d + c) : zero;
          }
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            if (j + q >= cnt) break;
            const uint32_t kq = __shfl_sync(0xffffffffu, key, j + q);
            if (kq != run) {                                    // the same for the whole warp
              if (in) {
                if (!inside) *(float4*)(first + w * d + c) = acc;
                else if (run < (uint32_t)vocab) *(float4*)(d_item + (int64_t)run * d + c) = acc;
              }
              inside = true;
              run = kq;
              acc = zero;
            }
            add4(acc, x[q]);
            if (kActions) {
              const int aq = __shfl_sync(0xffffffffu, act, j + q);
              if (kq < (uint32_t)vocab) add4(mine[aq * 32 + lane], x[q]);
            }
          }
        }
      }
      const bool on = p0 + kWin < n && keys[p0 + kWin] == run;  // the run goes on in the next window
      if (in) {
        if (!inside) *(float4*)(first + w * d + c) = acc;
        else if (on) *(float4*)(last + w * d + c) = acc;
        else if (run < (uint32_t)vocab) *(float4*)(d_item + (int64_t)run * d + c) = acc;
      }
    }
    if (kActions) {
      __syncthreads();
      for (int e = threadIdx.x; e < n_actions * 32; e += kSumThreads) {
        const int col = c0 + (e % 32) * 4;
        float4 acc = table[e];
        for (int w = 1; w < kSumWarps; ++w) add4(acc, table[w * n_actions * 32 + e]);
        if (col < d) *(float4*)(action_part + ((int64_t)blockIdx.x * n_actions + e / 32) * d + col) = acc;
      }
      __syncthreads();
    }
  }
}

// sum of rows [b, e) of part [., d] at columns c..c+3, in order
__device__ __forceinline__ float4 sum_range(const float* __restrict__ part, int64_t b, int64_t e, int64_t pitch, bool in) {
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int64_t v = b; v < e; ++v)
    if (in) add4(acc, *(const float4*)(part + v * pitch));
  return acc;
}

// the warps' sums added in warp order; the result is in warp 0
__device__ __forceinline__ float4 sum_warps(float4 mine, float4 (*part)[32]) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  __syncthreads();
  part[warp][lane] = mine;
  __syncthreads();
  float4 acc = part[0][lane];
  for (int w = 1; w < kSumWarps; ++w) add4(acc, part[w][lane]);
  return acc;
}

// CTAs [0, window_ctas): a warp per window whose last run started in it and goes on: the run's sum
// is last[w] + first[w + 1] + ... up to the window where it ends.  Runs over more than kLong
// windows are added by the whole CTA.  The other CTAs: the action sums, one action each.
__global__ void __launch_bounds__(kSumThreads) crossing_rows_kernel(const uint32_t* __restrict__ keys, int64_t n,
                                                                    int64_t vocab, int d,
                                                                    const float* __restrict__ first,
                                                                    const float* __restrict__ last,
                                                                    float* __restrict__ d_item, int window_ctas,
                                                                    const float* __restrict__ action_part, int parts,
                                                                    int n_actions, float* __restrict__ d_action) {
  __shared__ float4 part[kSumWarps][32];
  __shared__ int64_t long_end[kSumWarps];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if ((int)blockIdx.x >= window_ctas) {
    const int a = (int)blockIdx.x - window_ctas;
    for (int c0 = 0; c0 < d; c0 += 128) {
      const int c = c0 + lane * 4;
      const float* p = action_part + (int64_t)a * d + c;
      const float4 acc = sum_warps(sum_range(p, (int64_t)parts * warp / kSumWarps, (int64_t)parts * (warp + 1) / kSumWarps,
                                             (int64_t)n_actions * d, c < d), part);
      if (warp == 0 && c < d) *(float4*)(d_action + (int64_t)a * d + c) = acc;
    }
    return;
  }
  const int64_t w = (int64_t)blockIdx.x * kSumWarps + warp, windows = (n + kWin - 1) / kWin;
  int64_t end = 0;                                   // one behind the last window of the run (0: none to add)
  uint32_t run = 0xFFFFFFFFu;
  if (w + 1 < windows) {
    run = keys[w * kWin + kWin - 1];
    if (run < (uint32_t)vocab && keys[(w + 1) * kWin] == run && (w == 0 || keys[w * kWin - 1] != run)) {
      // window v > w holds a part of the run iff its first key is the run's
      const int64_t v = w + 1 + lane;
      const unsigned more = __ballot_sync(0xffffffffu, v < windows && keys[v * kWin] == run);
      end = w + 1 + __popc(more);
      if (more == 0xffffffffu) {                     // kLong = 32 windows or more: find the end
        int64_t lo = w + 33, hi = windows;           // the first window at or behind lo that does not start with it
        while (lo < hi) {
          const int64_t mid = (lo + hi) >> 1;
          if (keys[mid * kWin] == run) lo = mid + 1; else hi = mid;
        }
        end = lo;
      }
    }
  }
  const bool is_long = end - w - 1 >= kLong;
  if (lane == 0) long_end[warp] = is_long ? end : 0;
  if (end > 0 && !is_long)
    for (int c = lane * 4; c < d; c += 128) {
      float4 acc = *(const float4*)(last + w * d + c);
      add4(acc, sum_range(first + c, w + 1, end, d, true));
      *(float4*)(d_item + (int64_t)run * d + c) = acc;
    }
  __syncthreads();
  for (int i = 0; i < kSumWarps; ++i) {
    const int64_t e = long_end[i], b = (int64_t)blockIdx.x * kSumWarps + i;
    if (e == 0) continue;
    const int64_t cnt = e - b - 1;
    const uint32_t key = keys[b * kWin + kWin - 1];
    for (int c0 = 0; c0 < d; c0 += 128) {
      const int c = c0 + lane * 4;
      float4 acc = sum_range(first + c, b + 1 + cnt * warp / kSumWarps, b + 1 + cnt * (warp + 1) / kSumWarps, d, c < d);
      if (warp == 0 && c < d) add4(acc, *(const float4*)(last + b * d + c));
      acc = sum_warps(acc, part);
      if (warp == 0 && c < d) *(float4*)(d_item + (int64_t)key * d + c) = acc;
    }
  }
}

// part[CTA][action][d]: the sums of the CTA's contiguous events by action.  Each warp adds its
// own contiguous part into its own table in shared memory; the warps' tables are added in order.
template <class T>
__global__ void action_rows_kernel(const T* __restrict__ dX, const int32_t* __restrict__ ids,
                                   const uint8_t* __restrict__ acts, int64_t n, int64_t per, int64_t vocab,
                                   int n_actions, int d, float* __restrict__ part, int* err) {
  extern __shared__ float4 table[];                  // [warps][n_actions][32]
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, warps = blockDim.x / 32;
  const int c = blockIdx.y * 128 + lane * 4;
  float4* mine = table + warp * n_actions * 32;
  for (int a = 0; a < n_actions; ++a) mine[a * 32 + lane] = make_float4(0.f, 0.f, 0.f, 0.f);
  __syncwarp();
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
    for (int j = 0; j < cnt; j += 8) {
      float4 x[8];
#pragma unroll
      for (int q = 0; q < 8; ++q)
        x[q] = j + q < cnt && c < d ? row4(dX + (i0 + j + q) * d + c) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int aq = __shfl_sync(0xffffffffu, a, (j + q) & 31);
        if (j + q < cnt && aq >= 0) add4(mine[aq * 32 + lane], x[q]);
      }
    }
  }
  if (bad && blockIdx.y == 0) atomicOr(err, DEV_ERR_INDEX);
  __syncthreads();
  for (int e = threadIdx.x; e < n_actions * 32; e += blockDim.x) {
    const int col = blockIdx.y * 128 + (e % 32) * 4;
    float4 acc = table[e];
    for (int w = 1; w < warps; ++w) add4(acc, table[w * n_actions * 32 + e]);
    if (col < d) *(float4*)(part + ((int64_t)blockIdx.x * n_actions + e / 32) * d + col) = acc;
  }
}

int key_bits(int64_t vocab) {
  int b = 2;                                          // a digit of at least 4 bins
  while (((int64_t)1 << b) <= vocab) ++b;             // keys 0 .. vocab
  return b;
}
int sort_ctas(int64_t n) {
  return (int)std::max<int64_t>(1, std::min<int64_t>(device_info().sm_count, (n + 1023) / 1024));
}
// warps of an action CTA: their tables (512 bytes per action) fit in 128 KB of shared memory
int action_warps(int n_actions) { return std::max(1, std::min(8, 256 / n_actions)); }
int action_ctas(int64_t n) { return (int)std::max<int64_t>(1, std::min<int64_t>(4 * device_info().sm_count, (n + 255) / 256)); }
// CTAs of the window kernel: as many as are resident with their action tables (n_actions 4 KB each)
int window_ctas(int64_t n, int n_actions) {
  const int64_t ctas = ((n + kWin - 1) / kWin + kSumWarps - 1) / kSumWarps;
  const int per_sm = n_actions <= 8 ? 6 : 3;
  return (int)std::max<int64_t>(1, std::min<int64_t>(ctas, (int64_t)per_sm * device_info().sm_count));
}

template <class T>
sa_status run(const T* dX, const int32_t* ids, const uint8_t* acts, int64_t n, int64_t vocab, int n_actions, int d,
              float* d_item, float* d_action, const EventsBwdWork& w, cudaStream_t st) {
  static unsigned long long done[5] = {};          // one per kernel
  static std::mutex mu;
  int* err = device_status_word();
  const bool fused = d_item && d_action && n_actions <= kFusedActions;
  int parts = fused ? window_ctas(n, n_actions) : action_ctas(n);
  if (d_action && !fused) {
    const int warps = action_warps(n_actions);
    const int smem = warps * n_actions * 512;
    set_smem_limit_once((const void*)action_rows_kernel<T>, 131072, &done[0], mu);
    SA_TIMED("action_rows_kernel", st,
             (action_rows_kernel<T><<<dim3(parts, (d + 127) / 128), warps * 32, smem, st>>>(
                 dX, ids, acts, n, (n + parts - 1) / parts, vocab, n_actions, d, w.action_part, err)));
  }
  const uint32_t* keys = nullptr;
  if (d_item) {
    const int bits = key_bits(vocab), passes = (bits + kMaxBits - 1) / kMaxBits, G = sort_ctas(n);
    const int zero_ctas = 2 * device_info().sm_count;
    const FromEvents from{ids, acts, vocab, n_actions};
    if (n <= kSmallN) {
      const int smem = sort_smem((bits + passes - 1) / passes);
      set_smem_limit_once((const void*)sort_small_kernel, sort_smem(kMaxBits), &done[3], mu);
      const ZeroRows z{d_item, nullptr, 0, vocab, d};
      const unsigned grid = 1 + (unsigned)std::min<int64_t>(zero_ctas, (vocab + 511) / 512);
      const Buffers buf{{w.keys[0], w.keys[1]}, {w.events[0], w.events[1]}};
      SA_TIMED("sort_small_kernel", st,
               (sort_small_kernel<<<grid, kSortThreads, smem, st>>>(from, n, bits, passes, buf, z, err)));
    } else {
      SA_CUDA(cudaMemsetAsync(w.seen, 0, (size_t)(vocab + 31) / 32 * 4, st));
      set_smem_limit_once((const void*)sort_place_kernel<FromEvents>, sort_smem(kMaxBits), &done[1], mu);
      set_smem_limit_once((const void*)sort_place_kernel<FromList>, sort_smem(kMaxBits), &done[2], mu);
      for (int q = 0; q < passes; ++q) {
        Pass ps;
        ps.shift = bits * q / passes;
        ps.bits = bits * (q + 1) / passes - ps.shift;
        ps.n = n;
        ps.per = (n + G - 1) / G;
        const int smem = sort_smem(ps.bits);
        uint32_t *ko = w.keys[q & 1], *eo = w.events[q & 1];
        // every pass writes its share of the zero rows
        const ZeroRows z{d_item, w.seen, vocab * q / passes, vocab * (q + 1) / passes, d};
        if (q == 0) {
          SA_TIMED("sort_count_kernel", st, (sort_count_kernel<<<G, kSortThreads, 0, st>>>(from, ps, w.hist, w.seen, err)));
          SA_TIMED("sort_place_kernel", st,
                   (sort_place_kernel<<<G + zero_ctas, kSortThreads, smem, st>>>(from, ps, G, w.hist, ko, eo, z)));
        } else {
          const FromList in{w.keys[(q - 1) & 1], w.events[(q - 1) & 1]};
          SA_TIMED("sort_count_kernel", st, (sort_count_kernel<<<G, kSortThreads, 0, st>>>(in, ps, w.hist, nullptr, err)));
          SA_TIMED("sort_place_kernel", st,
                   (sort_place_kernel<<<G + zero_ctas, kSortThreads, smem, st>>>(in, ps, G, w.hist, ko, eo, z)));
        }
      }
    }
    keys = w.keys[(passes - 1) & 1];
    const uint32_t* events = w.events[(passes - 1) & 1];
    const int ctas = window_ctas(n, fused ? n_actions : 0);
    if (fused) {
      const int smem = kSumWarps * n_actions * 512;
      set_smem_limit_once((const void*)window_rows_kernel<T, true>, kSumWarps * kFusedActions * 512, &done[4], mu);
      SA_TIMED("window_rows_kernel", st,
               (window_rows_kernel<T, true><<<ctas, kSumThreads, smem, st>>>(
                   dX, keys, events, acts, n, vocab, n_actions, d, w.first, w.last, d_item, w.action_part)));
    } else {
      SA_TIMED("window_rows_kernel", st,
               (window_rows_kernel<T, false><<<ctas, kSumThreads, 0, st>>>(dX, keys, events, acts, n, vocab, 0, d, w.first,
                                                                            w.last, d_item, nullptr)));
    }
  }
  const int64_t windows = d_item ? (n + kWin - 1) / kWin : 0;
  const int wc = (int)((windows + kSumWarps - 1) / kSumWarps);
  SA_TIMED("crossing_rows_kernel", st,
           (crossing_rows_kernel<<<wc + (d_action ? n_actions : 0), kSumThreads, 0, st>>>(
               keys, n, vocab, d, w.first, w.last, d_item, wc, w.action_part, parts, n_actions, d_action)));
  return SA_OK;
}
}  // namespace

size_t events_bwd_layout(void* base, int64_t n, int64_t vocab, int n_actions, int d, EventsBwdWork* w) {
  Carve c(base);
  EventsBwdWork v;
  const size_t rows = (size_t)std::max<int64_t>(n, 1), windows = (rows + kWin - 1) / kWin;
  for (int i = 0; i < 2; ++i) {
    v.keys[i] = c.take<uint32_t>(rows);
    v.events[i] = c.take<uint32_t>(rows);
  }
  v.hist = c.take<int>((size_t)sort_ctas(n) << kMaxBits);
  v.seen = c.take<unsigned>((size_t)(vocab + 31) / 32);
  v.first = c.take<float>(windows * d);
  v.last = c.take<float>(windows * d);
  v.action_part = c.take<float>((size_t)std::max(action_ctas(n), window_ctas(n, n_actions)) * n_actions * d);
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
