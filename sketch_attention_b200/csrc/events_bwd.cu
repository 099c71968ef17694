// Backward of the event rows x_i = item_table[id_i] + action_table[a_i]
// (events.cu): the tables' gradients,
//   d_item[v] = sum over {i : id_i = v} of dX_i,   d_action[a] likewise,
// dense, fp32, without floating-point atomics: the same inputs give the same
// bits.  A row whose id or action is outside its table was zero in the forward,
// so it counts for neither table (and sets the device error word).
//
// The rows are ordered by item id with a stable radix sort of (id, i) pairs (an
// LSD pass per kMaxBits bits of the vocabulary's size: two for a million items),
// so every table row's gradient is the sum of a contiguous run of the list, in
// the order of the events.  Bound by memory: dX is read once for the items and
// the table gradient is written once, zeros included; the sort moves 8 bytes per
// event and pass.  A popular item's run is long (under Zipf(1.1) ids over a
// million items one item has 1 event in 8): runs are cut at multiples of kRun
// list positions, pieces that one item fills are summed first, by a CTA each,
// and the item's row then adds the pieces, so no row is one warp's serial work.
#include <algorithm>
#include <mutex>

#include "sa_internal.cuh"
#include "tma_map.cuh"

namespace sa {

namespace {
constexpr int kMaxBits = 10;                 // of the id per pass: 1024 bins
constexpr int kSortThreads = 512, kSortWarps = kSortThreads / 32;
constexpr int kRun = 256;                    // list positions per piece of a long run
constexpr int kSumThreads = 256, kSumWarps = kSumThreads / 32;
constexpr int kShort = 32;                   // runs up to this length are one warp's work
constexpr int kMaxRows = 64;                 // table rows per CTA of the row kernel

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

// hist[CTA][bin]: the CTA's events with each digit
template <class In>
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(In in, Pass ps, int* __restrict__ hist, int* err) {
  __shared__ int cnt[1 << kMaxBits];
  const int bins = 1 << ps.bits;
  for (int b = threadIdx.x; b < bins; b += kSortThreads) cnt[b] = 0;
  __syncthreads();
  const int64_t begin = (int64_t)blockIdx.x * ps.per, end = min(begin + ps.per, ps.n);
  for (int64_t i = begin + threadIdx.x; i < end; i += kSortThreads) {
    const uint32_t key = in.key(i);
    if (in.outside(key)) atomicOr(err, DEV_ERR_INDEX);
    atomicAdd(&cnt[(key >> ps.shift) & (bins - 1)], 1);
  }
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += kSortThreads) hist[(int64_t)blockIdx.x * bins + b] = cnt[b];
}

// Moves the CTA's events behind those with smaller digits, and those with the same digit in
// earlier CTAs.  Each warp owns a contiguous part, counts its digits, and places its events
// in order, so equal digits keep their order.
template <class In>
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(In in, Pass ps, const int* __restrict__ hist,
                                                                  uint32_t* __restrict__ keys,
                                                                  uint32_t* __restrict__ events) {
  extern __shared__ int smem[];
  int* wcnt = smem;                                  // [kSortWarps][bins]
  const int bins = 1 << ps.bits;
  int* base = smem + kSortWarps * bins;              // [bins]
  __shared__ int warp_sum[kSortWarps];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  for (int b = threadIdx.x; b < kSortWarps * bins; b += kSortThreads) wcnt[b] = 0;
  // base[b] = events with a smaller digit + events of earlier CTAs with digit b
  int carry = 0;
  for (int b0 = 0; b0 < bins; b0 += kSortThreads) {
    const int b = b0 + threadIdx.x;
    int total = 0, before = 0;
    if (b < bins) {
#pragma unroll 8
      for (int g = 0; g < (int)gridDim.x; ++g) {
        const int c = hist[(int64_t)g * bins + b];
        if (g < (int)blockIdx.x) before += c;
        total += c;
      }
    }
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
    if (b < bins) base[b] = off + incl - total + before;
    carry = all;
    __syncthreads();
  }
  const int64_t begin = (int64_t)blockIdx.x * ps.per, end = min(begin + ps.per, ps.n);
  const int64_t part = ((end - begin + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
  const int64_t wb = min(begin + warp * part, end), we = min(wb + part, end);
  int* mine = wcnt + warp * bins;
  for (int64_t i = wb + lane; i < we; i += 32) atomicAdd(&mine[(in.key(i) >> ps.shift) & (bins - 1)], 1);
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += kSortThreads) {
    int run = base[b];
    for (int w = 0; w < kSortWarps; ++w) {
      const int c = wcnt[w * bins + b];
      wcnt[w * bins + b] = run;
      run += c;
    }
  }
  __syncthreads();
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

__device__ __forceinline__ float4 row4(const __nv_bfloat16* p) {
  const uint2 w = *(const uint2*)p;
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xFFFF0000u));
}
__device__ __forceinline__ float4 row4(const float* p) { return *(const float4*)p; }
__device__ __forceinline__ void add4(float4& a, const float4& b) {
  a.x += b.x; a.y += b.y; a.z += b.z; a.w += b.w;
}

// a warp's sum, in order, of the rows events[s..e) at columns c..c+3 (c < d, else zero)
template <class T>
__device__ __forceinline__ float4 sum_rows(const T* __restrict__ dX, const uint32_t* __restrict__ events, int64_t s,
                                           int64_t e, int d, int c) {
  const int lane = threadIdx.x % 32;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int64_t i0 = s; i0 < e; i0 += 32) {
    const int cnt = (int)min((int64_t)32, e - i0);
    const uint32_t ev = lane < cnt ? events[i0 + lane] : 0u;
    for (int j = 0; j < cnt; j += 8) {
      float4 x[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const uint32_t r = __shfl_sync(0xffffffffu, ev, (j + q) & 31);
        x[q] = j + q < cnt && c < d ? row4(dX + (int64_t)r * d + c) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) add4(acc, x[q]);
    }
  }
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

// pieces[c] = sum of the rows of list positions [kRun c, kRun (c + 1)), where one item fills them
template <class T>
__global__ void __launch_bounds__(kSumThreads) piece_kernel(const T* __restrict__ dX, const uint32_t* __restrict__ keys,
                                                            const uint32_t* __restrict__ events, int64_t vocab, int d,
                                                            float* __restrict__ pieces) {
  __shared__ float4 part[kSumWarps][32];
  const int64_t s = (int64_t)blockIdx.x * kRun;
  const uint32_t key = keys[s];
  if (key != keys[s + kRun - 1] || key >= (uint64_t)vocab) return;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  for (int c0 = 0; c0 < d; c0 += 128) {
    const int c = c0 + lane * 4;
    const int64_t b = s + warp * (kRun / kSumWarps);
    const float4 acc = sum_warps(sum_rows(dX, events, b, b + kRun / kSumWarps, d, c), part);
    if (warp == 0 && c < d) *(float4*)(pieces + (int64_t)blockIdx.x * d + c) = acc;
  }
}

// first position of keys[lo..hi) that is not below `key`
__device__ __forceinline__ int64_t lower_bound(const uint32_t* __restrict__ keys, int64_t lo, int64_t hi, uint64_t key) {
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (keys[mid] < key) lo = mid + 1; else hi = mid;
  }
  return lo;
}

// the CTA's `rows` table rows: each is the sum of its run of the list (zero without one)
template <class T>
__global__ void __launch_bounds__(kSumThreads) item_rows_kernel(const T* __restrict__ dX,
                                                                const uint32_t* __restrict__ keys,
                                                                const uint32_t* __restrict__ events, int64_t n,
                                                                int64_t vocab, int rows, int d,
                                                                const float* __restrict__ pieces,
                                                                float* __restrict__ d_item) {
  __shared__ int64_t start[kMaxRows + 1];
  __shared__ float4 part[kSumWarps][32];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t v0 = (int64_t)blockIdx.x * rows;
  const int here = (int)min((int64_t)rows, vocab - v0);
  if (threadIdx.x <= here) start[threadIdx.x] = lower_bound(keys, 0, n, (uint64_t)(v0 + threadIdx.x));
  __syncthreads();
  for (int c0 = 0; c0 < d; c0 += 128) {
    const int c = c0 + lane * 4;
    for (int r = warp; r < here; r += kSumWarps) {
      const int64_t s = start[r], e = start[r + 1];
      if (e - s > kShort) continue;
      const float4 acc = sum_rows(dX, events, s, e, d, c);
      if (c < d) *(float4*)(d_item + (v0 + r) * d + c) = acc;
    }
    for (int r = 0; r < here; ++r) {
      const int64_t s = start[r], e = start[r + 1];
      if (e - s <= kShort) continue;
      // whole pieces [p0, p1), and the rows before and behind them, spread over the warps
      const int64_t p0 = (s + kRun - 1) / kRun, p1 = e / kRun;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      if (p0 < p1) {
        const int64_t head = p0 * kRun - s, tail = e - p1 * kRun;
        acc = sum_rows(dX, events, s + head * warp / kSumWarps, s + head * (warp + 1) / kSumWarps, d, c);
        const int64_t q0 = p0 + (p1 - p0) * warp / kSumWarps, q1 = p0 + (p1 - p0) * (warp + 1) / kSumWarps;
#pragma unroll 8
        for (int64_t q = q0; q < q1; ++q)
          if (c < d) add4(acc, *(const float4*)(pieces + q * d + c));
        const int64_t tb = p1 * kRun;
        add4(acc, sum_rows(dX, events, tb + tail * warp / kSumWarps, tb + tail * (warp + 1) / kSumWarps, d, c));
      } else {
        acc = sum_rows(dX, events, s + (e - s) * warp / kSumWarps, s + (e - s) * (warp + 1) / kSumWarps, d, c);
      }
      acc = sum_warps(acc, part);
      if (warp == 0 && c < d) *(float4*)(d_item + (v0 + r) * d + c) = acc;
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
  int b = 1;
  while (((int64_t)1 << b) <= vocab) ++b;             // keys 0 .. vocab
  return b;
}
int sort_ctas(int64_t n) {
  return (int)std::max<int64_t>(1, std::min<int64_t>(device_info().sm_count, (n + 1023) / 1024));
}
// warps of an action CTA: their tables (512 bytes per action) fit in 128 KB of shared memory
int action_warps(int n_actions) { return std::max(1, std::min(8, 256 / n_actions)); }
int action_ctas(int64_t n) { return (int)std::max<int64_t>(1, std::min<int64_t>(device_info().sm_count, (n + 255) / 256)); }

template <class T>
sa_status run(const T* dX, const int32_t* ids, const uint8_t* acts, int64_t n, int64_t vocab, int n_actions, int d,
              float* d_item, float* d_action, const EventsBwdWork& w, cudaStream_t st) {
  if (d_action) {
    const int warps = action_warps(n_actions), ctas = action_ctas(n);
    const int smem = warps * n_actions * 512;
    static unsigned long long done = 0;
    static std::mutex mu;
    set_smem_limit_once((const void*)action_rows_kernel<T>, 131072, &done, mu);
    SA_TIMED("action_rows_kernel", st,
             (action_rows_kernel<T><<<dim3(ctas, (d + 127) / 128), warps * 32, smem, st>>>(
                 dX, ids, acts, n, (n + ctas - 1) / ctas, vocab, n_actions, d, w.action_part, device_status_word())));
    sa_status s = sa_sum_slices(w.action_part, ctas, (int64_t)n_actions * d, d_action, st);
    if (s != SA_OK) return s;
  }
  if (!d_item) return SA_OK;
  const int bits = key_bits(vocab), passes = (bits + kMaxBits - 1) / kMaxBits, G = sort_ctas(n);
  static unsigned long long done_e = 0, done_l = 0;
  static std::mutex mu;
  int* err = device_status_word();
  const int limit = (kSortWarps + 1) * (1 << kMaxBits) * 4;
  set_smem_limit_once((const void*)sort_place_kernel<FromEvents>, limit, &done_e, mu);
  set_smem_limit_once((const void*)sort_place_kernel<FromList>, limit, &done_l, mu);
  const uint32_t *keys = nullptr, *events = nullptr;
  for (int q = 0; q < passes; ++q) {
    Pass ps;
    ps.shift = bits * q / passes;
    ps.bits = bits * (q + 1) / passes - ps.shift;
    ps.n = n;
    ps.per = (n + G - 1) / G;
    const int smem = (kSortWarps + 1) * (1 << ps.bits) * 4;
    uint32_t *ko = w.keys[q & 1], *eo = w.events[q & 1];
    if (q == 0) {
      FromEvents in{ids, acts, vocab, n_actions};
      SA_TIMED("sort_count_kernel", st, (sort_count_kernel<<<G, kSortThreads, 0, st>>>(in, ps, w.hist, err)));
      SA_TIMED("sort_place_kernel", st, (sort_place_kernel<<<G, kSortThreads, smem, st>>>(in, ps, w.hist, ko, eo)));
    } else {
      FromList in{keys, events};
      SA_TIMED("sort_count_kernel", st, (sort_count_kernel<<<G, kSortThreads, 0, st>>>(in, ps, w.hist, err)));
      SA_TIMED("sort_place_kernel", st, (sort_place_kernel<<<G, kSortThreads, smem, st>>>(in, ps, w.hist, ko, eo)));
    }
    keys = ko;
    events = eo;
  }
  if (n >= kRun)
    SA_TIMED("piece_kernel", st,
             (piece_kernel<T><<<(unsigned)(n / kRun), kSumThreads, 0, st>>>(dX, keys, events, vocab, d, w.pieces)));
  // enough CTAs for every SM with a small vocabulary, 64 rows each with a large one
  const int rows = (int)std::max<int64_t>(1, std::min<int64_t>(kMaxRows, vocab / (8 * device_info().sm_count)));
  SA_TIMED("item_rows_kernel", st,
           (item_rows_kernel<T><<<(unsigned)((vocab + rows - 1) / rows), kSumThreads, 0, st>>>(
               dX, keys, events, n, vocab, rows, d, w.pieces, d_item)));
  return SA_OK;
}
}  // namespace

size_t events_bwd_layout(void* base, int64_t n, int64_t vocab, int n_actions, int d, EventsBwdWork* w) {
  Carve c(base);
  EventsBwdWork v;
  const size_t rows = (size_t)std::max<int64_t>(n, 1);
  for (int i = 0; i < 2; ++i) {
    v.keys[i] = c.take<uint32_t>(rows);
    v.events[i] = c.take<uint32_t>(rows);
  }
  v.hist = c.take<int>((size_t)sort_ctas(n) << kMaxBits);
  v.pieces = c.take<float>((size_t)(n / kRun) * d);
  v.action_part = c.take<float>((size_t)action_ctas(n) * n_actions * d);
  if (w) *w = v;
  return c.bytes();
}

sa_status events_bwd_run(const void* dX, sa_dtype dtype, const int32_t* ids, const uint8_t* acts, int64_t n,
                         int64_t vocab, int n_actions, int d, float* d_item, float* d_action, const EventsBwdWork& w,
                         cudaStream_t st) {
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
