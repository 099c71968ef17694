// Backward of the token-wise normalisation variant (sa_tokenwise.cu): k folded
// prototypes attend over each user's events, keys = values = X, and the
// probabilities are recomputed from X.  With U = P W_Q W_K^T / sqrt(d),
// A = softmax over the user's events of U X^T, H = A X, i = 1/(m + eps):
//   dW_V = sum_u (i H)^T dS,  dH = i dS W_V^T,  c_j = dH_j . H_j
//   dZ = A o (dH X^T - c)     (per prototype: both the normaliser and c are row constants)
//   dX = A^T dH + dZ^T U,  E = sum_u dZ X   (dP, dW_Q, dW_K follow from E by small GEMMs)
//
// Accuracy.  dX is bf16; the weight gradients are fp32 and hold fp32-grade
// accuracy: X is exact in bf16, so the products that feed E take only their
// other operand (U, dH, dZ) as a bf16 pair hi + lo (16 bits, 2^-17 relative),
// two tensor-core products each.  The tensor core's fp32 accumulation truncates:
// a K = 8192 product reads 9e-6 off and drifts with K (85000: 1.6e-5 with signs
// mixed, 6.6e-5 without), K = 1024 1e-6; so E leaves TMEM every kDrain token
// tiles (1024 events) and is summed in registers, rounded to nearest.  For dX,
// Z takes U hi + lo (an error of Z is a relative error of A), the rest (dH in G and in
// A^T dH, U in dZ^T U, A, dZ) is bf16, since dX itself is: 2.7e-3 to 3.4e-3 of its norm off
// where its own rounding is 1.7e-3.  All that for the H that is given: c comes from it, and an
// H that is off by e adds -(dH . e) A X to E (the forward's H, 1e-3 to 5e-3 off, makes 4e-4 of
// dP at logits of a standard deviation of 1 and 1e-2 at 8).  c from the recomputed A and G
// would need G in the statistics' pass, a third product there, and another meaning of H.
//
// Three tensor-core passes over the events, each bounded by its products
// (per 128 events x 128 prototypes, 512 clocks per product at the bf16 rate):
//   tw_lse_kernel  row maximum and sum: 2 products; one CTA per (128-prototype
//     slice, token chunk), lane = prototype, so a row's statistics stay in a thread.
//   e_cta          6 products, same split.  [Z; G] = [U; dH] X^T with lane =
//     prototype; dZ goes back to TMEM as the A operand of E += dZ X, so nothing
//     but operands crosses shared memory.
//   dx_cta         5 products; one CTA per token chunk, 256 events (two tiles) per
//     pass over the prototypes (halves the prototype traffic out of L2), lane =
//     token.  The tiles alternate: while one tile's A and dZ are computed the
//     tensor core works on the other's.  A and dZ overwrite the logits in TMEM.
// 340,000 events x 1024 prototypes (4 users), us: statistics 113 (1.58 PFLOP/s of its 2 products), dX 357
// and E 394 alone (1.25 and 1.36 PFLOP/s of their 5 and 6), 727 in one launch; rows, weights and sums 50; a
// call 1.01 ms (0.88-0.93 in a loop over the same buffers).  The clock is at 1.56-1.7 GHz there (power cap).
// E's operands come through shared memory at 128 bytes a clock, 2750 clocks a tile beside the 6 x 512 of its
// products.  Short calls are bound by the chain of six kernels and by the host (one user of 300 events: 37 us,
// 31 replayed from a graph).
#include <algorithm>
#include <mutex>

#include "sa_internal.cuh"
#include "tc_ptx.cuh"
#include "tma_map.cuh"

namespace sa {

namespace {
using namespace tc;

constexpr int TILE = 128, DD = 128;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr uint32_t XT_BYTES = 32768;         // [128 rows x 128] bf16: 2 SW128 halves of 16 KB

// f(t, piece, u, first event, end of the piece, first, last) for every 128-event tile of
// chunk g, user by user (a piece: the chunk's events of one user)
template <class F>
__device__ __forceinline__ void for_each_tile(const int64_t* off, int B, const Chunking& ch, int g, F&& f) {
  const int64_t cb = (int64_t)g * ch.T, ce = min(cb + ch.T, ch.n_total);
  int t = 0, piece = 0;
  for (int u = user_of_token(off, B, cb); u < B && off[u] < ce; ++u) {
    const int64_t pb = max(off[u], cb), pe = min(off[u + 1], ce);
    if (pb >= pe) continue;
    for (int64_t tb = pb; tb < pe; tb += TILE, ++t)
      if (!f(t, piece, u, tb, pe, tb == pb, tb + TILE >= pe)) return;
    ++piece;
  }
}

// Descriptors of an operand's 16-deep K steps: a base, computed once per stage, plus a constant
// (added to the address field, which does not overflow).
//
// Every kernel has two threads that issue MMAs.  The tensor core takes a 128 x 128 x 16 product every
// 64 clocks and queues only a few, so a thread that issues a stage's products, waits for the next
// stage's barriers and loops (500 clocks even when all are ready) leaves it idle meanwhile: one
// thread for 16 products a tile measured 1665 clocks instead of 1024.  The two take turns, a stage
// each, waiting for their own barriers during the other's turn.  Without turns they issue at the same
// time and then wait at the same time: both stages finish late, and the tensor core idles while the
// warps work on both (dX: 4130 clocks per two stages of 1408).
constexpr uint32_t kHi = desc_hi(1024, SWZ_128B);
__device__ __forceinline__ uint32_t kmajor(uint32_t addr) { return desc_lo(addr, 16); }
__device__ constexpr uint32_t kstep(int ks) { return ((ks >> 2) * 16384 + (ks & 3) * 32) >> 4; }
__device__ __forceinline__ uint32_t mnmajor(uint32_t addr) { return desc_lo(addr, 16384); }
__device__ constexpr uint32_t mnstep(int ks) { return ks * 2048 >> 4; }

__device__ __forceinline__ float round_bf16(float x) { return __bfloat162float(__float2bfloat16_rn(x)); }
// x = hi + lo as bf16 pairs
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(a, b);
  lo = pack_bf16x2(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xFFFF0000u));
}

// waits for this thread's TMEM loads; names their registers, so no use moves above the wait
template <int N>
__device__ __forceinline__ void wait_ld(float* v) {
#pragma unroll
  for (int i = 0; i < N; i += 16) tmem_wait_ld16(v + i);
}

// mbar_wait of a whole warp, with one answer: the lanes leave together when the kernel gives up, so
// that no warp-wide instruction (tcgen05.ld) waits for lanes that have left.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int* err) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, err));
}

// The turns of the two issuing threads: thread 0 goes first, then they alternate (n: turns taken so
// far).  A turn is passed on kEarly products before its last is issued: the other thread's wake-up takes
// about as long as those run.
constexpr int kEarly = 4;
struct Turns {
  uint64_t bar[2];
};
__device__ __forceinline__ bool turn_wait(Turns* t, int i, int n, volatile int* abort, int* err) {
  return mbar_wait(&t->bar[i], i == 0 ? (n & 1) ^ 1 : n & 1, abort, err);
}
__device__ __forceinline__ void turn_pass(Turns* t, int i) { mbar_arrive(&t->bar[1 - i]); }

__device__ __forceinline__ void load_rows(uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int row) {
  tma_load_2d(dst, map, bar, 0, row);
  tma_load_2d(dst + XT_BYTES / 2, map, bar, 64, row);
}
// the same through a map of 64-row boxes (U and dH: the dX kernel takes 64 at a time)
__device__ __forceinline__ void load_rows64(uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int row) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    tma_load_2d(dst + i * (XT_BYTES / 4), map, bar, 64 * (i / 2), row + 64 * (i % 2));
}

// ============================================================== row statistics
constexpr int S_NXS = 4;
constexpr uint32_t S_OFF_U = 0;                                  // U hi, U lo
constexpr uint32_t S_OFF_X = 2 * XT_BYTES;
constexpr uint32_t S_OFF_BAR = S_OFF_X + S_NXS * XT_BYTES;
constexpr uint32_t S_SMEM = S_OFF_BAR + 256 + 1024;
// warp 0 TMA, 1 and 18 the MMAs of the even and the odd tiles, 2-9 the even tiles' statistics and
// 10-17 the odd ones', two threads per prototype: the teams are in different phases, so that the
// exponentials of one (1024 clocks a tile) fill the other's waits
constexpr int S_THREADS = 608, S_PARTS = 4;  // (max, sum) pairs per prototype: team, column half

struct SBars {
  uint64_t u_full, x_full[S_NXS], x_empty[S_NXS], z_full[2], z_empty[2], mma_done[2];
  Turns turns;
  uint32_t tmem_base;
  int abort;
};

struct SParams {
  const int64_t* off;
  int B;
  Chunking ch;
  int slices, kp;
  float2* user;          // [B, S_PARTS, kp] (max, sum) of users inside one chunk
  float2* slot;          // [G, 2, S_PARTS, kp] of the pieces of users that span chunks
  int* err;
};

__global__ void __launch_bounds__(S_THREADS, 1)
    tw_lse_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmR, SParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  SBars* bars = (SBars*)(smem + S_OFF_BAR);
  volatile int* abort = &bars->abort;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int sl = blockIdx.x % p.slices, g = blockIdx.x / p.slices;

  if (threadIdx.x == 0) {
    mbar_init(&bars->u_full, 1);
    for (int s = 0; s < S_NXS; ++s) { mbar_init(&bars->x_full[s], 1); mbar_init(&bars->x_empty[s], 1); }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars->z_full[b], 1);
      mbar_init(&bars->z_empty[b], 256);
      mbar_init(&bars->mma_done[b], 1);
      mbar_init(&bars->turns.bar[b], 1);
    }
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&bars->tmem_base, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  let_next_start();
  wait_for_previous();

  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&tmX);
    mbar_arrive_expect_tx(&bars->u_full, 2 * XT_BYTES);
    load_rows64(smem + S_OFF_U, &tmR, &bars->u_full, sl * TILE);
    load_rows64(smem + S_OFF_U + XT_BYTES, &tmR, &bars->u_full, p.kp + sl * TILE);
    int issued = 0;
    for_each_tile(p.off, p.B, p.ch, g, [&](int t, int, int, int64_t tb, int64_t, bool, bool) {
      const int s = t % S_NXS;
      if (t >= S_NXS && !mbar_wait(&bars->x_empty[s], ((t / S_NXS) - 1) & 1, abort, p.err)) return false;
      mbar_arrive_expect_tx(&bars->x_full[s], XT_BYTES);
      load_rows(smem + S_OFF_X + s * XT_BYTES, &tmX, &bars->x_full[s], (int)tb);
      issued = t + 1;
      return true;
    });
    if (*abort) {                            // no copy may be in flight when the CTA ends
      mbar_wait_bounded(&bars->u_full, 0);
      for (int t = std::max(0, issued - S_NXS); t < issued; ++t)
        mbar_wait_bounded(&bars->x_full[t % S_NXS], (t / S_NXS) & 1);
    }
  } else if (warp == 1 || warp == 18) {
    const int b = warp == 18;                // the parity of this thread's tiles
    const uint32_t id = idesc_bf16(128, 128, false, false), z = tmem + 128 * b;
    const uint32_t du = kmajor(smem_u32(smem + S_OFF_U)), dulo = kmajor(smem_u32(smem + S_OFF_U + XT_BYTES));
    if (lane == 0) {
      if (mbar_wait(&bars->u_full, 0, abort, p.err))
        for_each_tile(p.off, p.B, p.ch, g, [&](int t, int, int, int64_t, int64_t, bool, bool) {
          if ((t & 1) != b) return true;
          const int s = t % S_NXS;
          if (!mbar_wait(&bars->x_full[s], (t / S_NXS) & 1, abort, p.err)) return false;
          if (t >= 2 && !mbar_wait(&bars->z_empty[b], ((t >> 1) - 1) & 1, abort, p.err)) return false;
          if (!turn_wait(&bars->turns, b, t >> 1, abort, p.err)) return false;
          tc_fence_after();
          const uint32_t dx = kmajor(smem_u32(smem + S_OFF_X + s * XT_BYTES));
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) mma_ss_lo(z, du + kstep(ks), dx + kstep(ks), kHi, id, ks > 0);
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            if (ks == 8 - kEarly) turn_pass(&bars->turns, b);
            mma_ss_lo(z, dulo + kstep(ks), dx + kstep(ks), kHi, id, 1u);
          }
          mma_commit(&bars->z_full[b]);
          mma_commit(&bars->x_empty[s]);
          return true;
        });
      mma_commit(&bars->mma_done[b]);
      mbar_wait_bounded(&bars->mma_done[b], 0);
    }
  } else if (warp >= 2 && warp < 18) {
    // column half h: events 64 h .. 64 h + 63 of a tile
    const int q = warp % 4, team = (warp - 2) / 8, h = (warp - 2) / 4 % 2;
    const uint32_t at = tmem + ((uint32_t)(q * 32) << 16) + 128 * team + 64 * h;
    const int j = sl * TILE + q * 32 + lane;
    const int64_t cb = (int64_t)g * p.ch.T, ce = min(cb + p.ch.T, p.ch.n_total);
    float m = -INFINITY, sum = 0.f;
    for_each_tile(p.off, p.B, p.ch, g, [&](int t, int, int u, int64_t tb, int64_t pe, bool first, bool last) {
      if (first) { m = -INFINITY; sum = 0.f; }
      const int nv = (int)min(pe - tb - 64 * h, (int64_t)64);   // events of this half that are the user's
      if ((t & 1) == team) {
        if (!warp_wait(&bars->z_full[team], (t >> 1) & 1, abort, p.err)) return false;
        tc_fence_after();
        float z[64];
        tmem_ld32(at, z);
        tmem_ld32(at + 32, z + 32);
        wait_ld<64>(z);
        tc_fence_before();
        mbar_arrive(&bars->z_empty[team]);
        if (nv > 0) {
          if (nv < 64) {
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (i >= nv) z[i] = -INFINITY;
          }
          float mx[4] = {z[0], z[1], z[2], z[3]};
#pragma unroll
          for (int i = 4; i < 64; ++i) mx[i & 3] = fmaxf(mx[i & 3], z[i]);
          const float mn = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
          const float2 nm = make_float2(-mn, -mn);
          float2 s2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int i = 0; i < 64; i += 2) {
            const float2 e = __fadd2_rn(make_float2(z[i], z[i + 1]), nm);
            s2[(i >> 1) & 1] = __fadd2_rn(s2[(i >> 1) & 1], make_float2(ex2(e.x), ex2(e.y)));
          }
          sum = fmaf(sum, ex2(m - mn), (s2[0].x + s2[0].y) + (s2[1].x + s2[1].y));
          m = mn;
        }
      }
      if (last) {
        const int dest = piece_dest(p.off[u], p.off[u + 1], cb, ce);
        float2* out = dest == DEST_USER ? p.user + (int64_t)u * S_PARTS * p.kp
                                        : p.slot + ((int64_t)g * 2 + dest) * S_PARTS * p.kp;
        out[(int64_t)(2 * team + h) * p.kp + j] = make_float2(m, sum);
      }
      return true;
    });
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// lse2[u, j] = log2 of the row's sum of 2^z over the user's events, from its pieces' parts; +inf for
// a padding prototype (its A = 2^(z - inf) = 0) and for a user without events.  A CTA takes 32
// prototypes of a user; its 8 warps take the pieces in turn, and their results are added in order.
__global__ void __launch_bounds__(256) tw_lse_combine_kernel(const int64_t* __restrict__ off, Chunking ch, int k, int kp,
                                                             const float2* user, const float2* slot, float* lse2) {
  __shared__ float2 part[8][32];
  let_next_start();
  wait_for_previous();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int u = blockIdx.x / (kp / 32), j = blockIdx.x % (kp / 32) * 32 + lane;
  const int64_t ub = off[u], ue = off[u + 1];
  float m = -INFINITY, s = 0.f;
  auto add = [&](const float2& v) {
    if (v.x == -INFINITY && v.y == 0.f) return;          // a part without events
    const float mn = fmaxf(m, v.x);
    s = s * exp2f(m - mn) + v.y * exp2f(v.x - mn);
    m = mn;
  };
  if (ue > ub) {
    const int64_t gf = ub / ch.T, gl = (ue - 1) / ch.T;
    for (int64_t g = gf + warp; g <= gl; g += 8) {
      const float2* p = gf == gl ? user + (int64_t)u * S_PARTS * kp : slot + (g * 2 + (g == gf ? 1 : 0)) * S_PARTS * kp;
      float2 v[S_PARTS];
#pragma unroll
      for (int h = 0; h < S_PARTS; ++h) v[h] = p[(int64_t)h * kp + j];
#pragma unroll
      for (int h = 0; h < S_PARTS; ++h) add(v[h]);
    }
  }
  part[warp][lane] = make_float2(m, s);
  __syncthreads();
  if (warp > 0) return;
  for (int w = 1; w < 8; ++w) add(part[w][lane]);
  lse2[(int64_t)u * kp + j] = j < k && ue > ub ? m + log2f(s) : INFINITY;
}

// ============================================================== E kernel
constexpr int E_NXS = 3, kDrain = 8;         // token tiles per stay of E in TMEM
constexpr uint32_t E_OFF_U = 0;                                  // U hi, U lo, dH hi, dH lo
constexpr uint32_t E_OFF_X = 4 * XT_BYTES;
constexpr uint32_t E_OFF_BAR = E_OFF_X + E_NXS * XT_BYTES;
constexpr uint32_t E_SMEM = E_OFF_BAR + 256 + 1024;
constexpr int E_THREADS = 608;               // warp 0 TMA, 1 the MMAs of Z and G, 18 of E, 2-17 four threads per prototype
constexpr uint32_t E_TM_Z = 0, E_TM_G = 128, E_TM_E = 256, E_TM_DZ = 384;   // dZ: hi 64 columns, lo 64

struct EBars {
  uint64_t u_full, h_full, h_empty, x_full[E_NXS], x_empty[E_NXS], zg_full, zg_empty, dz_full, e_done, mma_done[2], zg_turn, e_turn;
  uint32_t tmem_base;
  int abort;
};

struct EParams {
  const int64_t* off;
  int B;
  Chunking ch;
  int slices, k, kp;
  const float* lse2;     // [B, kp]
  const float* c;        // [B, kp]
  float* Epart;          // [G, k, d]
  int* err;
};

__device__ __forceinline__ void e_cta(const CUtensorMap& tmX, const CUtensorMap& tmR, const EParams& p, int cta) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  EBars* bars = (EBars*)(smem + E_OFF_BAR);
  volatile int* abort = &bars->abort;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int sl = cta % p.slices, g = cta / p.slices;

  if (threadIdx.x == 0) {
    mbar_init(&bars->u_full, 1);
    mbar_init(&bars->h_full, 1);
    mbar_init(&bars->h_empty, 1);
    // X is read by the MMAs of both threads
    for (int s = 0; s < E_NXS; ++s) { mbar_init(&bars->x_full[s], 1); mbar_init(&bars->x_empty[s], 2); }
    mbar_init(&bars->zg_full, 1);
    mbar_init(&bars->zg_empty, 512);
    mbar_init(&bars->dz_full, 512);
    mbar_init(&bars->e_done, 1);
    mbar_init(&bars->zg_turn, 1);
    mbar_init(&bars->e_turn, 1);
    mbar_init(&bars->mma_done[0], 1);
    mbar_init(&bars->mma_done[1], 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  let_next_start();
  wait_for_previous();

  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&tmX);
    mbar_arrive_expect_tx(&bars->u_full, 2 * XT_BYTES);
    load_rows64(smem + E_OFF_U, &tmR, &bars->u_full, sl * TILE);
    load_rows64(smem + E_OFF_U + XT_BYTES, &tmR, &bars->u_full, p.kp + sl * TILE);
    int issued_x = 0, issued_h = 0;
    for_each_tile(p.off, p.B, p.ch, g, [&](int t, int piece, int u, int64_t tb, int64_t, bool first, bool) {
      if (first) {
        if (piece > 0 && !mbar_wait(&bars->h_empty, (piece - 1) & 1, abort, p.err)) return false;
        mbar_arrive_expect_tx(&bars->h_full, 2 * XT_BYTES);
        const int row = (2 + u) * p.kp + sl * TILE;
        load_rows64(smem + E_OFF_U + 2 * XT_BYTES, &tmR, &bars->h_full, row);
        load_rows64(smem + E_OFF_U + 3 * XT_BYTES, &tmR, &bars->h_full, row + p.B * p.kp);
        issued_h = piece + 1;
      }
      const int s = t % E_NXS;
      if (t >= E_NXS && !mbar_wait(&bars->x_empty[s], ((t / E_NXS) - 1) & 1, abort, p.err)) return false;
      mbar_arrive_expect_tx(&bars->x_full[s], XT_BYTES);
      load_rows(smem + E_OFF_X + s * XT_BYTES, &tmX, &bars->x_full[s], (int)tb);
      issued_x = t + 1;
      return true;
    });
    if (*abort) {
      mbar_wait_bounded(&bars->u_full, 0);
      if (issued_h > 0) mbar_wait_bounded(&bars->h_full, (issued_h - 1) & 1);
      for (int t = std::max(0, issued_x - E_NXS); t < issued_x; ++t)
        mbar_wait_bounded(&bars->x_full[t % E_NXS], (t / E_NXS) & 1);
    }
  } else if (warp == 1 && lane == 0) {
    // Z = (U hi + U lo) X^T, G = (dH hi + dH lo) X^T.  The turns are Z G (t + 1), then E (t): E's
    // products run while the warps read this tile's Z and G.
    const uint32_t id_zg = idesc_bf16(128, 128, false, false);
    const uint32_t du = kmajor(smem_u32(smem + E_OFF_U));
    int tiles = 0;
    if (mbar_wait(&bars->u_full, 0, abort, p.err))
      for_each_tile(p.off, p.B, p.ch, g, [&](int t, int piece, int, int64_t, int64_t, bool first, bool last) {
        if (first && !mbar_wait(&bars->h_full, piece & 1, abort, p.err)) return false;
        if (!mbar_wait(&bars->x_full[t % E_NXS], (t / E_NXS) & 1, abort, p.err)) return false;
        if (t > 0 && !mbar_wait(&bars->zg_empty, (t - 1) & 1, abort, p.err)) return false;
        if (t > 1 && !mbar_wait(&bars->zg_turn, t & 1, abort, p.err)) return false;
        tc_fence_after();
        const uint32_t dx = kmajor(smem_u32(smem + E_OFF_X + t % E_NXS * XT_BYTES));
#pragma unroll
        for (int o = 0; o < 4; ++o)
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            if (o == 3 && ks == 8 - kEarly && t > 0) mbar_arrive(&bars->e_turn);
            mma_ss_lo(tmem + (o < 2 ? E_TM_Z : E_TM_G), du + (o * XT_BYTES >> 4) + kstep(ks), dx + kstep(ks), kHi,
                      id_zg, (o & 1) || ks > 0);
          }
        mma_commit(&bars->zg_full);
        mma_commit(&bars->x_empty[t % E_NXS]);
        if (last) mma_commit(&bars->h_empty);
        tiles = t + 1;
        return true;
      });
    // the last tile's E, once the turn before it was taken (a barrier two phases on looks unfinished)
    if (tiles < 2 || mbar_wait(&bars->zg_turn, tiles & 1, abort, p.err)) mbar_arrive(&bars->e_turn);
    mma_commit(&bars->mma_done[0]);
    mbar_wait_bounded(&bars->mma_done[0], 0);
  } else if (warp == 18 && lane == 0) {
    // E += dZ X, afresh after every drain
    const uint32_t id_e = idesc_bf16(128, 128, false, true);     // A from TMEM, B MN-major
    for_each_tile(p.off, p.B, p.ch, g, [&](int t, int, int, int64_t, int64_t, bool, bool) {
      // dZ was computed from Z and G of this tile, so its X is there
      if (!mbar_wait(&bars->x_full[t % E_NXS], (t / E_NXS) & 1, abort, p.err)) return false;
      if (!mbar_wait(&bars->dz_full, t & 1, abort, p.err)) return false;
      if (!mbar_wait(&bars->e_turn, t & 1, abort, p.err)) return false;
      tc_fence_after();
      const uint32_t dx = mnmajor(smem_u32(smem + E_OFF_X + t % E_NXS * XT_BYTES));
      const uint32_t kept = t % kDrain != 0 ? 1u : 0u;
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        if (ks == 8 - kEarly / 2) mbar_arrive(&bars->zg_turn);
        mma_ts_lo(tmem + E_TM_E, tmem + E_TM_DZ + ks * 8, dx + mnstep(ks), kHi, id_e, ks > 0 ? 1u : kept);
        mma_ts_lo(tmem + E_TM_E, tmem + E_TM_DZ + 64 + ks * 8, dx + mnstep(ks), kHi, id_e, 1u);
      }
      mma_commit(&bars->e_done);
      mma_commit(&bars->x_empty[t % E_NXS]);
      return true;
    });
    mma_commit(&bars->mma_done[1]);
    mbar_wait_bounded(&bars->mma_done[1], 0);
  } else if (warp >= 2 && warp < 18) {
    const int q = warp % 4, w = (warp - 2) / 4;          // events 32 w .. 32 w + 31 of a tile, columns 32 w .. of E
    const uint32_t own = tmem + ((uint32_t)(q * 32) << 16) + 32 * w;
    const uint32_t dz_at = tmem + ((uint32_t)(q * 32) << 16) + E_TM_DZ + 16 * w;
    const int j = sl * TILE + q * 32 + lane;
    float acc[32];                                       // this thread's quarter row of E
#pragma unroll
    for (int i = 0; i < 32; ++i) acc[i] = 0.f;
    auto drain = [&]() {
#pragma unroll
      for (int i = 0; i < 32; i += 16) {
        float v[16];
        tmem_ld16(own + E_TM_E + i, v);
        wait_ld<16>(v);
#pragma unroll
        for (int x = 0; x < 16; ++x) acc[i + x] += v[x];
      }
    };
    float2 nl2 = make_float2(0.f, 0.f), nc = make_float2(0.f, 0.f);
    int tiles = 0;
    bool ok = true;
    for_each_tile(p.off, p.B, p.ch, g, [&](int t, int, int u, int64_t tb, int64_t pe, bool first, bool) {
      if (first) {
        // one event: its probability is 1 whatever Z, so dZ is zero exactly (dA - c would leave
        // the rounding of two equal numbers)
        const float l2 = p.off[u + 1] - p.off[u] == 1 ? INFINITY : p.lse2[(int64_t)u * p.kp + j];
        const float c = p.c[(int64_t)u * p.kp + j];
        nl2 = make_float2(-l2, -l2);
        nc = make_float2(-c, -c);
      }
      const int nv = (int)min(pe - tb - 32 * w, (int64_t)32);   // events of this quarter that are the user's
      if (!warp_wait(&bars->zg_full, t & 1, abort, p.err)) return ok = false;
      tc_fence_after();
      float z[32], gv[32];
      tmem_ld32(own + E_TM_Z, z);
      tmem_ld32(own + E_TM_G, gv);
      wait_ld<32>(z);
      wait_ld<32>(gv);
      tc_fence_before();
      mbar_arrive(&bars->zg_empty);
      uint32_t hi[16], lo[16];
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const float2 e = __fadd2_rn(make_float2(z[i], z[i + 1]), nl2);
        const float2 d = __fadd2_rn(make_float2(gv[i], gv[i + 1]), nc);
        float2 dz = __fmul2_rn(make_float2(ex2(e.x), ex2(e.y)), d);
        if (nv < 32) {
          if (i >= nv) dz.x = 0.f;
          if (i + 1 >= nv) dz.y = 0.f;
        }
        split2(dz.x, dz.y, hi[i / 2], lo[i / 2]);
      }
      // the last tile's E MMA has read dZ, and E is complete up to that tile
      if (t > 0 && !warp_wait(&bars->e_done, (t - 1) & 1, abort, p.err)) return ok = false;
      tc_fence_after();
      if (t > 0 && t % kDrain == 0) drain();
      tmem_st16(dz_at, hi);
      tmem_st16(dz_at + 64, lo);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&bars->dz_full);
      tiles = t + 1;
      return true;
    });
    if (ok && tiles > 0 && warp_wait(&bars->e_done, (tiles - 1) & 1, abort, p.err)) {
      tc_fence_after();
      drain();
      if (j < p.k) {
        float* dst = p.Epart + ((int64_t)g * p.k + j) * DD + 32 * w;
#pragma unroll
        for (int i = 0; i < 32; i += 4) *(float4*)(dst + i) = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ============================================================== dX kernel
constexpr int KC = 64, X_NCS = 3;            // prototypes per stage, stages
constexpr uint32_t CH_BYTES = 49152;         // [U h0 | dH h0 | U h1 | dH h1 | Ulo h0 | Ulo h1], 8 KB each
constexpr uint32_t X_OFF_X = 0;                                  // two token tiles
constexpr uint32_t X_OFF_CH = 2 * XT_BYTES;
constexpr uint32_t X_OFF_ROW = X_OFF_CH + X_NCS * CH_BYTES;      // [X_NCS][lse2 64 | ln2 c 64]
constexpr uint32_t X_OFF_BAR = X_OFF_ROW + X_NCS * 2 * KC * 4;
constexpr uint32_t X_SMEM = X_OFF_BAR + 256 + 1024;
// warp 0 TMA, 1 and 18 the MMAs of tile 0 and tile 1, 2-17 four threads per token, both tiles in turn
constexpr int X_THREADS = 608;
// TMEM columns of tile i: [Z|G] at 128 i, later A and ln2 dZ as bf16 pairs in the columns of Z;
// dX at 256 + 128 i
constexpr uint32_t X_TM_ZG = 0, X_TM_Q = 256;

struct XBars {
  uint64_t x_full[2], x_empty[2], c_full[X_NCS], c_empty[X_NCS], zg_full[2], aa_full[2], q_full[2], mma_done[2];
  Turns turns;
  uint32_t tmem_base;
  int abort;
};

struct XParams {
  const int64_t* off;
  int B;
  Chunking ch;
  int kp;
  const float* lse2;     // [B, kp]
  const float* c2;       // [B, kp] ln2 c
  __nv_bfloat16* dX;     // [n, d]
  int* err;
};

// The units of a chunk in order: up to 256 events of one user.
struct Units {
  const int64_t* off;
  int B, u;
  int64_t ce, tb, pe;                        // the current unit starts at tb, its piece ends at pe
  __device__ Units(const XParams& p, int g) : off(p.off), B(p.B) {
    const int64_t cb = (int64_t)g * p.ch.T;
    ce = min(cb + p.ch.T, p.ch.n_total);
    u = user_of_token(off, B, cb);
    tb = cb;
    pe = min(off[u + 1], ce);
  }
  __device__ bool done() const { return tb >= ce; }
  __device__ bool two() const { return pe - tb > TILE; }
  __device__ void next() {
    tb += 2 * TILE;
    if (tb < pe) return;
    tb = pe;
    if (tb >= ce) return;
    do ++u; while (off[u + 1] <= tb);        // tb < ce <= n: a user with events follows
    pe = min(off[u + 1], ce);
  }
};

__device__ __forceinline__ void dx_cta(const CUtensorMap& tmX, const CUtensorMap& tmR, const XParams& p, int cta) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  XBars* bars = (XBars*)(smem + X_OFF_BAR);
  volatile int* abort = &bars->abort;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = cta, nch = p.kp / KC;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->x_full[i], 1);
      mbar_init(&bars->x_empty[i], 1);
      mbar_init(&bars->zg_full[i], 1);
      mbar_init(&bars->aa_full[i], 512);
      mbar_init(&bars->q_full[i], 1);
      mbar_init(&bars->mma_done[i], 1);
      mbar_init(&bars->turns.bar[i], 1);
    }
    for (int s = 0; s < X_NCS; ++s) { mbar_init(&bars->c_full[s], 1); mbar_init(&bars->c_empty[s], 2); }
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  let_next_start();
  wait_for_previous();

  if (warp == 0 && lane == 0) {
    // ------------------------------------------------------------ TMA producer
    prefetch_tensormap(&tmX);
    int cc = 0, tiles[2] = {0, 0};           // stages and tiles issued so far
    bool ok = true;
    for (Units un(p, g); ok && !un.done(); un.next()) {
      const int n_tiles = un.two() ? 2 : 1;
      for (int i = 0; ok && i < n_tiles; ++i) {
        if (tiles[i] > 0 && !mbar_wait(&bars->x_empty[i], (tiles[i] - 1) & 1, abort, p.err)) { ok = false; break; }
        mbar_arrive_expect_tx(&bars->x_full[i], XT_BYTES);
        load_rows(smem + X_OFF_X + i * XT_BYTES, &tmX, &bars->x_full[i], (int)(un.tb + i * TILE));
        ++tiles[i];
      }
      for (int c = 0; ok && c < nch; ++c, ++cc) {
        const int s = cc % X_NCS;
        if (cc >= X_NCS && !mbar_wait(&bars->c_empty[s], ((cc / X_NCS) - 1) & 1, abort, p.err)) { ok = false; break; }
        mbar_arrive_expect_tx(&bars->c_full[s], CH_BYTES + 2 * KC * 4);
        uint8_t* cd = smem + X_OFF_CH + s * CH_BYTES;
        const int64_t row = (int64_t)un.u * p.kp + c * KC;
        const int h_row = 2 * p.kp + (int)row;
        tma_load_2d(cd, &tmR, &bars->c_full[s], 0, c * KC);
        tma_load_2d(cd + 8192, &tmR, &bars->c_full[s], 0, h_row);
        tma_load_2d(cd + 16384, &tmR, &bars->c_full[s], 64, c * KC);
        tma_load_2d(cd + 24576, &tmR, &bars->c_full[s], 64, h_row);
        tma_load_2d(cd + 32768, &tmR, &bars->c_full[s], 0, p.kp + c * KC);
        tma_load_2d(cd + 40960, &tmR, &bars->c_full[s], 64, p.kp + c * KC);
        uint8_t* rd = smem + X_OFF_ROW + s * 2 * KC * 4;
        bulk_load(rd, p.lse2 + row, KC * 4, &bars->c_full[s]);
        bulk_load(rd + KC * 4, p.c2 + row, KC * 4, &bars->c_full[s]);
      }
    }
    if (*abort) {
      for (int i = 0; i < 2; ++i)
        if (tiles[i] > 0) mbar_wait_bounded(&bars->x_full[i], (tiles[i] - 1) & 1);
      for (int c = std::max(0, cc - X_NCS); c < cc; ++c)
        mbar_wait_bounded(&bars->c_full[c % X_NCS], (c / X_NCS) & 1);
    }
  } else if (warp == 1 || warp == 18) {
    // ------------------------------------------------------------ MMA issuers: tile i of every unit
    const int i = warp == 18;
    const uint32_t id_zg = idesc_bf16(128, 128, false, false), id_lo = idesc_bf16(128, 64, false, false);
    const uint32_t id_q = idesc_bf16(128, 128, false, true);     // A from TMEM, B MN-major
    const uint32_t zg = tmem + X_TM_ZG + 128 * i, q = tmem + X_TM_Q + 128 * i;
    const uint32_t dx = kmajor(smem_u32(smem + X_OFF_X + i * XT_BYTES));
    if (lane == 0) {
      int cc = 0, x = 0, a = 0, n = 0;       // stages, tiles, aggregated stages and turns so far
      // A turn is the aggregation of a stage and the next stage's logits.
      // Logits for stage counter cc: Z = X (U hi + U lo)^T, G = X dH^T
      auto logits_ready = [&](int cc, bool first) -> bool {
        return (!first || mbar_wait(&bars->x_full[i], x++ & 1, abort, p.err)) &&
               mbar_wait(&bars->c_full[cc % X_NCS], (cc / X_NCS) & 1, abort, p.err);
      };
      auto logits = [&](int cc, bool two) {
        const uint32_t dc = kmajor(smem_u32(smem + X_OFF_CH + cc % X_NCS * CH_BYTES));
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) mma_ss_lo(zg, dx + kstep(ks), dc + kstep(ks), kHi, id_zg, ks > 0);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          if (ks == 8 - kEarly && two) turn_pass(&bars->turns, i);
          mma_ss_lo(zg, dx + kstep(ks), dc + ((32768 + (ks >> 2) * 8192 + (ks & 3) * 32) >> 4), kHi, id_lo, 1u);
        }
      };
      bool ok = true;
      for (Units un(p, g); ok && !un.done(); un.next()) {
        const bool two = un.two();
        if (i == 1 && !two) {
          // no tile of this thread's: its share of freeing the unit's stages (once they were full, so
          // that no arrival counts for an earlier use of the stage)
          for (int c = 0; ok && c < nch; ++c, ++cc) {
            ok = mbar_wait(&bars->c_full[cc % X_NCS], (cc / X_NCS) & 1, abort, p.err);
            if (ok) mbar_arrive(&bars->c_empty[cc % X_NCS]);
          }
          continue;
        }
        // the first logits, then turns of aggregation and logits, then the last aggregation
        for (int c = -1; c < nch; ++c) {
          if (c >= 0 && !mbar_wait(&bars->aa_full[i], a++ & 1, abort, p.err)) { ok = false; break; }
          if (c + 1 < nch && !logits_ready(cc + c + 1, c < 0)) { ok = false; break; }
          if (two && !turn_wait(&bars->turns, i, n++, abort, p.err)) { ok = false; break; }
          tc_fence_after();
          if (c >= 0) {
            // dX += A dH + (ln2 dZ) U (U in base-2 units) over the stage's 64 prototypes
            const uint32_t dc = mnmajor(smem_u32(smem + X_OFF_CH + (cc + c) % X_NCS * CH_BYTES));
            const uint32_t kept = c > 0 ? 1u : 0u;
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
              // prototypes 16 ks ..: written by the threads of quarter ks, A then dZ, 8 columns each
              mma_ts_lo(q, zg + 16 * ks, dc + (8192 >> 4) + mnstep(ks), kHi, id_q, ks > 0 ? 1u : kept);
              mma_ts_lo(q, zg + 16 * ks + 8, dc + mnstep(ks), kHi, id_q, 1u);
            }
            mma_commit(&bars->c_empty[(cc + c) % X_NCS]);
            if (c == nch - 1) mma_commit(&bars->q_full[i]);
          }
          if (c + 1 < nch) logits(cc + c + 1, two);
          else if (two) turn_pass(&bars->turns, i);
          if (c + 1 < nch) mma_commit(&bars->zg_full[i]);
          if (c + 1 == nch - 1) mma_commit(&bars->x_empty[i]);
        }
        cc += nch;
      }
      mma_commit(&bars->mma_done[i]);
      mbar_wait_bounded(&bars->mma_done[i], 0);
    }
  } else if (warp >= 2) {
    // ------------------------------------------------------------ four threads per token
    const int q = warp % 4, w = (warp - 2) / 4;          // prototypes 16 w .. 16 w + 15 of a stage
    const int row = q * 32 + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)(q * 32) << 16);
    const float2 ln2v = make_float2(kLn2, kLn2);
    int cc = 0, a[2] = {0, 0}, t[2] = {0, 0};            // stage counter; stages and units per tile
    bool ok = true;
    for (Units un(p, g); ok && !un.done(); un.next()) {
      const int n_tiles = un.two() ? 2 : 1;
      for (int c = 0; ok && c < nch; ++c, ++cc) {
        const int s = cc % X_NCS;
        const float4* l4 = (const float4*)(smem + X_OFF_ROW + s * 2 * KC * 4) + 4 * w;
        const float4* c4 = l4 + KC / 4;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (i >= n_tiles) break;
          const uint32_t own = lane_addr + X_TM_ZG + 128 * i + 16 * w;
          if (!warp_wait(&bars->zg_full[i], a[i] & 1, abort, p.err) ||
              !warp_wait(&bars->c_full[s], (cc / X_NCS) & 1, abort, p.err)) { ok = false; break; }
          ++a[i];
          tc_fence_after();
          float z[16], gv[16];
          tmem_ld16(own, z);
          tmem_ld16(own + 64, gv);
          wait_ld<16>(z);
          wait_ld<16>(gv);
          uint32_t pk[16];                   // A in 0..7, ln2 dZ in 8..15 (even prototype low)
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const float4 l = l4[b], cv = c4[b];
            const float2 lp[2] = {make_float2(-l.x, -l.y), make_float2(-l.z, -l.w)};
            const float2 cp[2] = {make_float2(-cv.x, -cv.y), make_float2(-cv.z, -cv.w)};
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int j = 4 * b + 2 * x;
              const float2 e = __fadd2_rn(make_float2(z[j], z[j + 1]), lp[x]);
              const float2 A = make_float2(ex2(e.x), ex2(e.y));
              const float2 dz = __fmul2_rn(A, __ffma2_rn(make_float2(gv[j], gv[j + 1]), ln2v, cp[x]));
              pk[j / 2] = pack_bf16x2(A.x, A.y);
              pk[8 + j / 2] = pack_bf16x2(dz.x, dz.y);
            }
          }
          tmem_st16(own, pk);
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(&bars->aa_full[i]);
        }
      }
      // this thread's 32 columns of its token's dX, in both tiles
      for (int i = 0; ok && i < n_tiles; ++i) {
        if (!warp_wait(&bars->q_full[i], t[i] & 1, abort, p.err)) { ok = false; break; }
        ++t[i];
        tc_fence_after();
        const int64_t r = un.tb + i * TILE + row;
        float v[32];
        tmem_ld32(lane_addr + X_TM_Q + 128 * i + 32 * w, v);
        wait_ld<32>(v);
        tc_fence_before();                   // read before this thread's next arrival at aa_full
        if (r < un.pe) {
          uint4* dst = (uint4*)(p.dX + r * DD + 32 * w);
#pragma unroll
          for (int x = 0; x < 4; ++x)
            dst[x] = make_uint4(pack_bf16x2(v[8 * x], v[8 * x + 1]), pack_bf16x2(v[8 * x + 2], v[8 * x + 3]),
                                pack_bf16x2(v[8 * x + 4], v[8 * x + 5]), pack_bf16x2(v[8 * x + 6], v[8 * x + 7]));
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Both in one launch: CTAs [0, x_ctas) compute dX, the others E.  Neither needs the other; a small
// call's run side by side, and a large one's E starts on the SMs that finish their dX first.
static_assert(E_THREADS == X_THREADS, "one launch for both");
constexpr uint32_t GRADS_SMEM = E_SMEM > X_SMEM ? E_SMEM : X_SMEM;

__global__ void __launch_bounds__(X_THREADS, 1)
    tw_grads_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmR,
                    const __grid_constant__ XParams xp, const __grid_constant__ EParams ep, int x_ctas) {
  if ((int)blockIdx.x < x_ctas) dx_cta(tmX, tmR, xp, (int)blockIdx.x);
  else e_cta(tmX, tmR, ep, (int)blockIdx.x - x_ctas);
}

// ============================================================== rows of 128 columns
// The products with the d x d weights, in fp32 FMA, 16 or 8 rows per CTA step (the framework's tiled fp32
// GEMM takes 12 us for such a product at any k up to 1024; the eleven that fold the prototypes and
// carry E back to the weights took two thirds of a small call; the four stages of them here take about
// 6 us each).  A weight matrix lies in shared memory as it is in memory, with a pitch of 132 floats: rows and columns of it are then both read
// without bank conflicts, so it serves W and W^T.
constexpr int R_THREADS = 256, W_PITCH = DD + 4;
constexpr int RB = 16, RW = 8;                // rows per step of the prepare and the weights kernel
constexpr uint32_t W_BYTES = DD * W_PITCH * 4, ROW_BYTES = DD * 4;
constexpr uint32_t PREP_SMEM = W_BYTES + 3 * RB * ROW_BYTES, WEIGHTS_SMEM = 2 * W_BYTES + 4 * RW * ROW_BYTES;

__device__ __forceinline__ void copy16(float* dst, const float* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// the copies of a weight matrix, and of `have` rows (the others zeros); copies_done, then a barrier
__device__ __forceinline__ void load_weight(float* w, const float* W) {
#pragma unroll
  for (int x = 0; x < DD * DD / 4 / R_THREADS; ++x) {
    const int i = x * R_THREADS + threadIdx.x;
    copy16(w + i / 32 * W_PITCH + i % 32 * 4, W + i * 4);
  }
}
template <int R>
__device__ __forceinline__ void load_block(float (*rows)[DD], const float* src, int have) {
#pragma unroll
  for (int x = 0; x < R * DD / 4 / R_THREADS; ++x) {
    const int i = x * R_THREADS + threadIdx.x;
    if (i / 32 < have) copy16(&rows[0][0] + i * 4, src + i * 4);
    else ((float4*)rows)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
}

// dst[r][c] = f sum_e rows[r][e] W[e][c], or (kT) f sum_e rows[r][e] W[c][e].  A thread has a 4 x 4 tile and
// every KS-th four of the 128 terms (8 shared loads of 16 bytes for 64 FMA); its neighbours in the warp
// have the others, and each of them stores a part of the tile.
template <int R, bool kT>
__device__ __forceinline__ void rows_product(const float (*rows)[DD], const float* w, float (*dst)[DD], float f) {
  constexpr int KS = 32 / R, T = R;             // lanes that share a tile, tiles side by side in a warp
  static_assert(R == 8 || R == 16, "a warp has 16 or 8 tiles");
  const int warp = threadIdx.x / 32, h = threadIdx.x % 32 / T, t = threadIdx.x % T;
  const int r0 = warp / (DD / (4 * T)) * 4, c0 = warp % (DD / (4 * T)) * 4 * T;
  float v[4][4] = {};
#pragma unroll 2
  for (int e = 4 * h; e < DD; e += 4 * KS) {
    float4 x[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) x[r] = *(const float4*)&rows[r0 + r][e];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (kT) {                                 // column c0 + t + T j
        const float4 y = *(const float4*)(w + (c0 + t + T * j) * W_PITCH + e);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          v[r][j] = fmaf(x[r].x, y.x, fmaf(x[r].y, y.y, fmaf(x[r].z, y.z, fmaf(x[r].w, y.w, v[r][j]))));
      } else {                                  // term e + j of columns c0 + 4 t ..
        const float4 y = *(const float4*)(w + (e + j) * W_PITCH + c0 + 4 * t);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float xe = j == 0 ? x[r].x : j == 1 ? x[r].y : j == 2 ? x[r].z : x[r].w;
          v[r][0] = fmaf(xe, y.x, v[r][0]);
          v[r][1] = fmaf(xe, y.y, v[r][1]);
          v[r][2] = fmaf(xe, y.z, v[r][2]);
          v[r][3] = fmaf(xe, y.w, v[r][3]);
        }
      }
    }
  }
  // rows 2 h', 2 h' + 1 of the tile to the lanes with bit 16 of h', and (KS = 4) one row each
  float u[2][4], s[4];
  const bool up = threadIdx.x & 16;
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      u[r][j] = (up ? v[2 + r][j] : v[r][j]) + __shfl_xor_sync(0xffffffffu, up ? v[r][j] : v[2 + r][j], 16);
  const int row = r0 + (up ? 2 : 0);
  if (KS == 4) {
    const bool up8 = threadIdx.x & 8;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      s[j] = (up8 ? u[1][j] : u[0][j]) + __shfl_xor_sync(0xffffffffu, up8 ? u[0][j] : u[1][j], 8);
#pragma unroll
    for (int j = 0; j < 4; ++j) dst[row + (up8 ? 1 : 0)][kT ? c0 + t + T * j : c0 + 4 * t + j] = f * s[j];
  } else {
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int j = 0; j < 4; ++j) dst[row + r][kT ? c0 + t + T * j : c0 + 4 * t + j] = f * u[r][j];
  }
}

// acc[8][8] += sum_r a[r][8 ty ..] b[r][4 tx .. and 64 + 4 tx ..]: a thread's tile of a^T b
template <int R>
__device__ __forceinline__ void add_outer(const float (*a)[DD], const float (*b)[DD], float (*acc)[8]) {
  const int ty = threadIdx.x / 16 % 16, tx = threadIdx.x % 16;
#pragma unroll 2
  for (int r = 0; r < R; ++r) {
    const float4 a0 = *(const float4*)&a[r][8 * ty], a1 = *(const float4*)&a[r][8 * ty + 4];
    const float4 b0 = *(const float4*)&b[r][4 * tx], b1 = *(const float4*)&b[r][64 + 4 * tx];
    const float av[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
    const float bv[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int x = 0; x < 8; ++x) acc[i][x] = fmaf(av[i], bv[x], acc[i][x]);
  }
}
__device__ __forceinline__ void store_outer(float* part, const float (*acc)[8], float f) {
  const int ty = threadIdx.x / 16 % 16, tx = threadIdx.x % 16;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float* dst = part + (8 * ty + i) * DD + 4 * tx;
    *(float4*)dst = make_float4(f * acc[i][0], f * acc[i][1], f * acc[i][2], f * acc[i][3]);
    *(float4*)(dst + 64) = make_float4(f * acc[i][4], f * acc[i][5], f * acc[i][6], f * acc[i][7]);
  }
}
// four columns of a row as hi + lo bf16
__device__ __forceinline__ void store_split(__nv_bfloat16* hi, __nv_bfloat16* lo, int64_t at, const float4& x) {
  uint2 h, l;
  split2(x.x, x.y, h.x, l.x);
  split2(x.z, x.w, h.y, l.y);
  *(uint2*)(hi + at) = h;
  *(uint2*)(lo + at) = l;
}

// CTAs [0, kp / 16): Q = P W_Q and U = Q W_K^T log2(e) / sqrt(d) as hi + lo (zero rows behind k).
// The others (where the rows are few), 16 prototypes of a user each: dH = i dS W_V^T as hi + lo, c = (hi + lo) . H
// and c2 = ln2 hi . H (zeros for a user without events and behind k), and the CTA's part of sum H^T dS.
// G - c is small beside G where a softmax has one large weight (x is near H there), so each c is that of
// the dH which its kernel's G has, hi + lo in E and hi in dX: the rest then costs rest (x - H), not rest x.
__global__ void __launch_bounds__(R_THREADS, 2) tw_prepare_kernel(
    const int64_t* __restrict__ off, int B, int k, int kp, float inv, float u_scale, const float* __restrict__ P,
    const float* __restrict__ W_Q, const float* __restrict__ W_K, const float* __restrict__ W_V,
    const float* __restrict__ dS, const float* __restrict__ H, float* __restrict__ Q, __nv_bfloat16* __restrict__ Uhi,
    __nv_bfloat16* __restrict__ Ulo, __nv_bfloat16* __restrict__ Hhi, __nv_bfloat16* __restrict__ Hlo,
    float* __restrict__ cj, float* __restrict__ c2, float* __restrict__ part_v) {
  extern __shared__ __align__(16) float sm[];
  float (*a)[DD] = (float (*)[DD])(sm + DD * W_PITCH), (*b)[DD] = a + RB, (*o)[DD] = b + RB;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, groups = kp / RB;
  let_next_start();
  if ((int)blockIdx.x < groups) {
    const int j0 = blockIdx.x * RB;
    load_block<RB>(a, P + (int64_t)j0 * DD, k - j0);
    load_weight(sm, W_Q);
    copies_done();
    __syncthreads();
    rows_product<RB, false>(a, sm, b, 1.f);
    __syncthreads();
    load_weight(sm, W_K);
    for (int r = warp; r < RB; r += R_THREADS / 32)
      if (j0 + r < k) *(float4*)(Q + (int64_t)(j0 + r) * DD + lane * 4) = *(const float4*)&b[r][lane * 4];
    copies_done();
    __syncthreads();
    rows_product<RB, true>(b, sm, o, u_scale);
    __syncthreads();
    for (int r = warp; r < RB; r += R_THREADS / 32)
      store_split(Uhi, Ulo, (int64_t)(j0 + r) * DD + lane * 4, *(const float4*)&o[r][lane * 4]);
    return;
  }
  const int g = blockIdx.x - groups, u = g / groups, j0 = g % groups * RB;
  const int have = off[u + 1] > off[u] ? k - j0 : 0;
  const int64_t in = ((int64_t)u * k + j0) * DD, row0 = (int64_t)u * kp + j0;
  load_weight(sm, W_V);
  load_block<RB>(a, dS + in, have);
  load_block<RB>(b, H + in, have);
  copies_done();
  __syncthreads();
  rows_product<RB, true>(a, sm, o, inv);
  float dwv[8][8] = {};
  add_outer<RB>(b, a, dwv);
  __syncthreads();
  for (int r = warp; r < RB; r += R_THREADS / 32) {
    const float4 x = *(const float4*)&o[r][lane * 4], hv = *(const float4*)&b[r][lane * 4];
    const float4 hi = make_float4(round_bf16(x.x), round_bf16(x.y), round_bf16(x.z), round_bf16(x.w));
    float dot_hi = fmaf(hi.x, hv.x, fmaf(hi.y, hv.y, fmaf(hi.z, hv.z, hi.w * hv.w)));
    float dot = fmaf(round_bf16(x.x - hi.x), hv.x, fmaf(round_bf16(x.y - hi.y), hv.y,
                fmaf(round_bf16(x.z - hi.z), hv.z, fmaf(round_bf16(x.w - hi.w), hv.w, dot_hi))));
    for (int s = 16; s > 0; s >>= 1) {
      dot += __shfl_xor_sync(0xffffffffu, dot, s);
      dot_hi += __shfl_xor_sync(0xffffffffu, dot_hi, s);
    }
    if (lane == 0) {
      cj[row0 + r] = dot;
      c2[row0 + r] = kLn2 * dot_hi;
    }
    store_split(Hhi, Hlo, (row0 + r) * DD + lane * 4, x);
  }
  store_outer(part_v + (int64_t)g * DD * DD, dwv, 1.f);
}

// The same dH, c, c2 and parts of sum H^T dS where there are many rows (many users), on the tensor
// cores in fp32 grade: dS, H and W_V as three bf16 parts each (24 bits), six products of the parts, the
// small ones first (the accumulation truncates at the size of the sum).  64 rows a step:
//   dH^T = W_V dS^T (lane = column of dH, 64 TMEM columns, two buffers),
//   dW_V += H^T dS  (K = the rows; the large product and the small ones in accumulators of their own,
//   which leave TMEM every kVDrain steps and are summed in fp32, rounded to nearest).
// 16 warps split a step's rows into shared memory, then write the step before while the tensor core
// works (4400 clocks) and the next rows are on their way: 11,000 clocks a step, 0.34 ms for 524,288 rows
// (2.4 TB/s; the L1 and shared-memory array serves the loads and the MMAs' operands).  Every CTA has a
// first step: the grid is no larger than the number of steps.
constexpr int V_ROWS = 64, V_THREADS = 544, kVDrain = 8;
constexpr uint32_t VS_BYTES = V_ROWS * DD * 2;                   // a part of a step's dS or H
constexpr uint32_t V_OFF_S = 3 * XT_BYTES, V_OFF_H = V_OFF_S + 3 * VS_BYTES, V_OFF_RED = V_OFF_H + 3 * VS_BYTES;
constexpr uint32_t V_OFF_BAR = V_OFF_RED + 2 * 2 * 4 * V_ROWS * 4;
constexpr uint32_t VALUES_SMEM = V_OFF_BAR + 64 + 1024;
constexpr uint32_t V_TM_DW = 128, V_TM_DW_LOW = 256;             // dH: columns 0-63 and 64-127

struct VBars {
  uint64_t full, done, mma_done;
  uint32_t tmem_base;
  int abort;
};

// four columns of a row (c4: which four) as three bf16 parts, into swizzled tiles of 64-column halves
__device__ __forceinline__ void store_parts(uint32_t base, uint32_t part_bytes, int row, int c4, float4 x) {
  const uint32_t at = base + (c4 >> 4) * (part_bytes / 2) + row * 128 + ((((c4 & 15) >> 1) ^ (row & 7)) << 4) + (c4 & 1) * 8;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const uint32_t a = pack_bf16x2(x.x, x.y), b = pack_bf16x2(x.z, x.w);
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at + i * part_bytes), "r"(a), "r"(b) : "memory");
    x.x -= __uint_as_float(a << 16); x.y -= __uint_as_float(a & 0xFFFF0000u);
    x.z -= __uint_as_float(b << 16); x.w -= __uint_as_float(b & 0xFFFF0000u);
  }
}

__global__ void __launch_bounds__(V_THREADS, 1) tw_values_kernel(
    const int64_t* __restrict__ off, int B, int k, int kp, float inv, const float* __restrict__ W_V,
    const float* __restrict__ dS, const float* __restrict__ H, __nv_bfloat16* Hhi, __nv_bfloat16* Hlo, float* cj, float* c2,
    float* part_v, int* err) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  VBars* bars = (VBars*)(smem + V_OFF_BAR);
  float* red = (float*)(smem + V_OFF_RED);                       // [buffer][c2, c][quarter of the columns][row]
  volatile int* abort = &bars->abort;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, groups = kp / V_ROWS;
  const int steps = B * groups;                                  // B kp < 2^31
  const uint32_t at_w = smem_u32(smem), at_s = at_w + V_OFF_S, at_h = at_w + V_OFF_H;

  if (threadIdx.x == 0) {
    mbar_init(&bars->full, 512);
    mbar_init(&bars->done, 1);
    mbar_init(&bars->mma_done, 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == 16) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  let_next_start();

  if (warp == 16) {
    if (lane == 0) {
      const uint32_t id_h = idesc_bf16(128, V_ROWS, false, false), id_w = idesc_bf16(128, 128, true, true);
      const uint32_t dw = kmajor(at_w), ds = kmajor(at_s);
      const uint32_t ms = desc_lo(at_s, VS_BYTES / 2), mh = desc_lo(at_h, VS_BYTES / 2);
      constexpr int pi[6] = {0, 1, 2, 0, 1, 0}, pj[6] = {2, 1, 0, 1, 0, 0};      // parts of the products
      int n = 0;
      for (int g = blockIdx.x; g < steps; g += gridDim.x, ++n) {
        mbar_wait(&bars->full, n & 1, abort, err);
        tc_fence_after();
        const uint32_t d = tmem + (n & 1) * V_ROWS, kept = n % kVDrain != 0 ? 1u : 0u;
#pragma unroll
        for (int o = 0; o < 6; ++o)
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            mma_ss_lo(d, dw + (pi[o] * XT_BYTES >> 4) + kstep(ks),
                      ds + ((pj[o] * VS_BYTES + (ks >> 2) * (VS_BYTES / 2) + (ks & 3) * 32) >> 4), kHi, id_h, o > 0 || ks > 0);
#pragma unroll
        for (int o = 0; o < 6; ++o)
#pragma unroll
          for (int ks = 0; ks < V_ROWS / 16; ++ks)
            mma_ss_lo(tmem + (o < 5 ? V_TM_DW_LOW : V_TM_DW), mh + (pi[o] * VS_BYTES >> 4) + mnstep(ks),
                      ms + (pj[o] * VS_BYTES >> 4) + mnstep(ks), kHi, id_w, ks > 0 || (o > 0 && o < 5) ? 1u : kept);
        mma_commit(&bars->done);
      }
      mma_commit(&bars->mma_done);               // nothing in flight when the CTA ends, whatever gave up
      mbar_wait_bounded(&bars->mma_done, 0);
    }
  } else {
    const int q = warp % 4, p = warp / 4, c = 32 * q + lane;     // dH's column; rows 16 p .. of a step, 32 p .. of dW_V
    const uint32_t own = tmem + ((uint32_t)(q * 32) << 16);
    struct Step {
      int u, j0, have;                                           // user, first row, rows of H that count
    };
    float4 sv[4], hv[4];
    auto load = [&](int g) {
      Step s{g / groups, g % groups * V_ROWS, 0};
      if (off[s.u + 1] > off[s.u]) s.have = k - s.j0;
      const int64_t in = ((int64_t)s.u * k + s.j0) * DD;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int i = x * 512 + threadIdx.x;
        sv[x] = hv[x] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i / 32 < s.have) {
          sv[x] = *(const float4*)(dS + in + i * 4);
          hv[x] = *(const float4*)(H + in + i * 4);
        }
      }
      return s;
    };
    // the CTA's part of sum H^T dS lies in memory (L2): a thread's 32 values of it
    float* part = part_v + (int64_t)blockIdx.x * DD * DD + c * DD + 32 * p;
    auto drain = [&](bool first) {
#pragma unroll
      for (int i = 0; i < 32; i += 16) {
        float lo[16], v[16];
        tmem_ld16(own + V_TM_DW_LOW + 32 * p + i, lo);
        tmem_ld16(own + V_TM_DW + 32 * p + i, v);
        wait_ld<16>(lo);
        wait_ld<16>(v);
#pragma unroll
        for (int x = 0; x < 16; x += 4) {
          float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
          if (!first) s = *(const float4*)(part + i + x);
          *(float4*)(part + i + x) = make_float4(s.x + (lo[x] + v[x]), s.y + (lo[x + 1] + v[x + 1]),
                                                 s.z + (lo[x + 2] + v[x + 2]), s.w + (lo[x + 3] + v[x + 3]));
        }
      }
    };
    // dH of a step, in TMEM buffer b: hi and lo, c and c2
    auto write = [&](const Step& at_step, int b) {
      const int u = at_step.u, j0 = at_step.j0 + 16 * p, have = at_step.have - 16 * p;
      const float* h_at = H + ((int64_t)u * k + j0) * DD + c;
      const int64_t row0 = (int64_t)u * kp + j0;
      float v[16], sum[32];
      tmem_ld16(own + b * V_ROWS + 16 * p, v);
#pragma unroll
      for (int r = 0; r < 16; ++r) sum[r] = r < have ? h_at[r * DD] : 0.f;
      wait_ld<16>(v);
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        v[r] *= inv;
        const float hi = round_bf16(v[r]), lo = round_bf16(v[r] - hi);
        sum[16 + r] = fmaf(hi, sum[r], lo * sum[r]);
        sum[r] *= hi;
      }
      // the 32 sums over the warp's columns, one to a lane
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < o; ++i) {
          const bool up = lane & o;
          const float send = up ? sum[i] : sum[i + o], keep = up ? sum[i + o] : sum[i];
          sum[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
      red[((b * 2 + lane / 16) * 4 + q) * V_ROWS + 16 * p + lane % 16] = sum[0];
      // neighbours exchange columns: an even lane stores rows 0, 2, .., an odd one 1, 3, ..
      const bool odd = lane & 1;
#pragma unroll
      for (int r = 0; r < 16; r += 2) {
        const float got = __shfl_xor_sync(0xffffffffu, odd ? v[r] : v[r + 1], 1);
        uint32_t hi, lo;
        split2(odd ? got : v[r], odd ? v[r + 1] : got, hi, lo);
        const int64_t at = (row0 + r + odd) * DD + (c & ~1);
        *(uint32_t*)(Hhi + at) = hi;
        *(uint32_t*)(Hlo + at) = lo;
      }
      asm volatile("bar.sync 1, 512;" ::: "memory");
      if (threadIdx.x < 2 * V_ROWS) {
        const int which = threadIdx.x / V_ROWS, r = threadIdx.x % V_ROWS;
        const float* s = red + (b * 2 + which) * 4 * V_ROWS + r;
        const float x = (s[0] + s[V_ROWS]) + (s[2 * V_ROWS] + s[3 * V_ROWS]);
        const int64_t at = (int64_t)u * kp + at_step.j0 + r;
        if (which == 0) c2[at] = kLn2 * x;
        else cj[at] = x;
      }
    };
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const int i = x * 512 + threadIdx.x;
      store_parts(at_w, XT_BYTES, i / 32, i % 32, *(const float4*)(W_V + i * 4));
    }
    Step next = load(blockIdx.x), last{};
    int n = 0;
    for (int g = blockIdx.x; g < steps; g += gridDim.x, ++n) {
      if (n > 0) {                                         // a wait that gave up leaves numbers that mean nothing
        warp_wait(&bars->done, (n - 1) & 1, abort, err);
        tc_fence_after();
        if (n % kVDrain == 0) drain(n == kVDrain);
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int i = x * 512 + threadIdx.x;
        store_parts(at_s, VS_BYTES, i / 32, i % 32, sv[x]);
        store_parts(at_h, VS_BYTES, i / 32, i % 32, hv[x]);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(&bars->full);
      const Step now = next;
      if (g + (int)gridDim.x < steps) next = load(g + gridDim.x);
      if (n > 0) write(last, (n - 1) & 1);
      last = now;
    }
    warp_wait(&bars->done, (n - 1) & 1, abort, err);
    tc_fence_after();
    drain(n <= kVDrain);
    write(last, (n - 1) & 1);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 16) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  wait_for_previous();                       // so that what follows this kernel follows U's too
}

// the sum of four columns of n parts, in order, 16 loads at a time (the last few too: one by one they
// cost a trip to L2 each)
__device__ __forceinline__ float4 sum_parts(const float* src, int64_t pitch, int n) {
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < n; i0 += 16) {
    float4 x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i)
      x[i] = i0 + i < n ? *(const float4*)(src + (i0 + i) * pitch) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 16; ++i) { s.x += x[i].x; s.y += x[i].y; s.z += x[i].z; s.w += x[i].w; }
  }
  return s;
}

// 8 prototypes at a time: E = the chunks' parts in order, dQ = E W_K / sqrt(d), dP = dQ W_Q^T, and
// the CTA's parts of dW_Q = P^T dQ and dW_K = E^T Q / sqrt(d)
__global__ void __launch_bounds__(R_THREADS, 1) tw_weights_kernel(int k, int G, float rs, const float* Epart,
                                                                  const float* __restrict__ P, const float* Q,
                                                                  const float* __restrict__ W_Q,
                                                                  const float* __restrict__ W_K, float* dP,
                                                                  float* part_qk) {
  extern __shared__ __align__(16) float sm[];
  float *w0 = sm, *w1 = sm + DD * W_PITCH;
  float (*e)[DD] = (float (*)[DD])(w1 + DD * W_PITCH), (*q)[DD] = e + RW, (*dq)[DD] = q + RW, (*pr)[DD] = dq + RW;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  float dwq[8][8] = {}, dwk[8][8] = {};
  let_next_start();
  load_weight(w0, W_K);
  load_weight(w1, W_Q);
  wait_for_previous();
  for (int j0 = blockIdx.x * RW; j0 < k; j0 += gridDim.x * RW) {
    __syncthreads();
    load_block<RW>(q, Q + (int64_t)j0 * DD, k - j0);
    load_block<RW>(pr, P + (int64_t)j0 * DD, k - j0);
    for (int r = warp; r < RW; r += R_THREADS / 32) {
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
      if (j0 + r < k) s = sum_parts(Epart + (int64_t)(j0 + r) * DD + lane * 4, (int64_t)k * DD, G);
      *(float4*)&e[r][lane * 4] = s;
    }
    copies_done();
    __syncthreads();
    rows_product<RW, false>(e, w0, dq, rs);
    add_outer<RW>(e, q, dwk);
    __syncthreads();                         // e is no longer read: dP replaces it
    rows_product<RW, true>(dq, w1, e, 1.f);
    add_outer<RW>(pr, dq, dwq);
    __syncthreads();
    for (int r = warp; r < RW; r += R_THREADS / 32)
      if (j0 + r < k) *(float4*)(dP + (int64_t)(j0 + r) * DD + lane * 4) = *(const float4*)&e[r][lane * 4];
  }
  store_outer(part_qk + (int64_t)blockIdx.x * 2 * DD * DD, dwq, 1.f);
  store_outer(part_qk + ((int64_t)blockIdx.x * 2 + 1) * DD * DD, dwk, rs);
}

// dW_V = i times the sum of its parts, dW_Q and dW_K the sums of theirs: a CTA per 128 values, its
// 8 warps over the parts, added in order
__global__ void __launch_bounds__(R_THREADS) tw_sum_kernel(const float* part_v, int n_v, float inv, const float* part_qk,
                                                           int n_qk, float* dW_V, float* dW_Q, float* dW_K) {
  __shared__ float4 sums[R_THREADS / 32][32];
  wait_for_previous();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int which = blockIdx.x / DD, at = blockIdx.x % DD * DD + lane * 4;
  const float* src = (which == 0 ? part_v : part_qk + (which - 1) * DD * DD) + at;
  const int n = which == 0 ? n_v : n_qk;
  const int64_t pitch = which == 0 ? DD * DD : 2 * DD * DD;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int i = n * warp / 8; i < n * (warp + 1) / 8; ++i) {
    const float4 x = *(const float4*)(src + i * pitch);
    s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp > 0) return;
  for (int w = 1; w < R_THREADS / 32; ++w) {
    const float4 x = sums[w][lane];
    s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
  }
  const float f = which == 0 ? inv : 1.f;
  float* dst = which == 0 ? dW_V : which == 1 ? dW_Q : dW_K;
  *(float4*)(dst + at) = make_float4(f * s.x, f * s.y, f * s.z, f * s.w);
}

int padded_k(int k) { return (k + TILE - 1) / TILE * TILE; }

// token chunks of the per-slice kernels: one CTA per (slice, chunk), one wave
Chunking slice_chunks(int64_t n, int k) {
  return make_chunking(n, std::max(1, device_info().sm_count / (padded_k(k) / TILE)), TILE);
}
// whether the rows of dS are many enough for tw_values_kernel: more blocks of rows, U's among them, than
// SMs.  A call's time with tw_prepare_kernel alone and with it (us): 1 user x 1024 prototypes 80.0, 83.5;
// 16 x 128 49.3, 53.4; 4 x 512 100.4, 96.1; 4 x 1024 130.6, 118.4; 8 x 512 88.2, 74.5; 64 x 1024 510, 240
bool many_rows(int B, int k) { return (B + 1LL) * (padded_k(k) / RB) > device_info().sm_count; }
// CTAs that keep a part of the d x d gradient of W_V each (64 KB written and read again)
int value_parts(int B, int k) {
  const int64_t rows = (int64_t)B * padded_k(k);
  return (int)(many_rows(B, k) ? std::min<int64_t>(rows / V_ROWS, device_info().sm_count) : rows / RB);
}
int weight_parts(int k) { return std::min((k + RW - 1) / RW, 64); }
Chunking token_chunks(int64_t n) { return make_chunking(n, device_info().sm_count, TILE); }

sa_status map_rows(CUtensorMap* map, const void* base, int64_t rows, uint32_t box_rows) {
  return tma_map_bf16(map, base, DD, (uint64_t)rows, 64, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}
}  // namespace

size_t tokenwise_bwd_layout(void* base, int B, int64_t n, int k, int d, TokenwiseBwdWork* w) {
  Carve c(base);
  TokenwiseBwdWork v;
  const size_t kp = padded_k(k), kd = (size_t)k * d, dd = (size_t)d * d;
  v.chE = slice_chunks(n, k);
  v.chX = token_chunks(n);
  const size_t G = (size_t)std::max(v.chE.G, 1);
  v.Q = c.take<float>(kd);
  v.Uhi = c.take<__nv_bfloat16>(2 * (1 + (size_t)B) * kp * d);   // one array, one tensor map
  v.Ulo = v.Uhi + kp * d;
  v.Hhi = v.Ulo + kp * d;
  v.Hlo = v.Hhi + (size_t)B * kp * d;
  for (float** p : {&v.c, &v.c2, &v.lse2}) *p = c.take<float>((size_t)B * kp);
  v.stat_user = c.take<float2>((size_t)B * S_PARTS * kp);
  v.stat_slot = c.take<float2>(G * 2 * S_PARTS * kp);
  v.Epart = c.take<float>(G * kd);
  v.part_v = c.take<float>(value_parts(B, k) * dd);
  v.part_qk = c.take<float>(weight_parts(k) * 2 * dd);
  if (w) *w = v;
  return c.bytes();
}

sa_status sa_tokenwise_backward_run(const SaBwdArgs& a, const TokenwiseBwdWork& w, cudaStream_t st) {
  static unsigned long long done_s = 0, done_g = 0, done_p = 0, done_w = 0, done_v = 0;
  static std::mutex mu;
  set_smem_limit_once((const void*)tw_lse_kernel, S_SMEM, &done_s, mu);
  set_smem_limit_once((const void*)tw_grads_kernel, GRADS_SMEM, &done_g, mu);
  set_smem_limit_once((const void*)tw_prepare_kernel, PREP_SMEM, &done_p, mu);
  set_smem_limit_once((const void*)tw_values_kernel, VALUES_SMEM, &done_v, mu);
  set_smem_limit_once((const void*)tw_weights_kernel, WEIGHTS_SMEM, &done_w, mu);
  const int kp = padded_k(a.k), slices = kp / TILE, n_v = value_parts(a.B, a.k), n_qk = weight_parts(a.k);
  const bool many = many_rows(a.B, a.k);
  const float inv = 1.f / (1.f + a.eps);                // m = 1 for a user with events
  const float rs = 1.f / sqrtf((float)a.d);
  sa_status s;
  SA_TIMED("tw_prepare_kernel", st,
           (tw_prepare_kernel<<<kp / RB + (many ? 0 : n_v), R_THREADS, PREP_SMEM, st>>>(
               a.off_dev, a.B, a.k, kp, inv, 1.4426950408889634f * rs, a.P, a.W_Q, a.W_K, a.W_V, a.dS, a.H, w.Q, w.Uhi,
               w.Ulo, w.Hhi, w.Hlo, w.c, w.c2, w.part_v)));
  if (many)
    SA_TIMED("tw_values_kernel", st,
             launch_after(tw_values_kernel, n_v, V_THREADS, VALUES_SMEM, st, a.off_dev, a.B, a.k, kp, inv, a.W_V, a.dS, a.H,
                          w.Hhi, w.Hlo, w.c, w.c2, w.part_v, device_status_word()));
  if (a.n_total > 0) {
    CUtensorMap tmX, tmR;                               // the events; U and dH, hi and lo
    const int64_t hrows = (int64_t)a.B * kp;
    if ((s = map_rows(&tmX, a.X, a.n_total, 128)) != SA_OK) return s;
    if ((s = map_rows(&tmR, w.Uhi, 2 * (kp + hrows), 64)) != SA_OK) return s;
    SParams sp{a.off_dev, a.B, w.chE, slices, kp, w.stat_user, w.stat_slot, device_status_word()};
    SA_TIMED("tw_lse_kernel", st,
             launch_after(tw_lse_kernel, w.chE.G * slices, S_THREADS, S_SMEM, st, tmX, tmR, sp));
    SA_TIMED("tw_lse_combine_kernel", st,
             launch_after(tw_lse_combine_kernel, (unsigned)(hrows / 32), 256, 0, st, a.off_dev, w.chE, a.k, kp, w.stat_user,
                          w.stat_slot, w.lse2));
    XParams xp{a.off_dev, a.B, w.chX, kp, w.lse2, w.c2, (__nv_bfloat16*)a.dX, device_status_word()};
    EParams ep{a.off_dev, a.B, w.chE, slices, a.k, kp, w.lse2, w.c, w.Epart, device_status_word()};
    SA_TIMED("tw_grads_kernel", st,
             launch_after(tw_grads_kernel, w.chX.G + w.chE.G * slices, X_THREADS, GRADS_SMEM, st, tmX, tmR, xp, ep,
                          w.chX.G));
  }
  SA_TIMED("tw_weights_kernel", st,
           launch_after(tw_weights_kernel, n_qk, R_THREADS, WEIGHTS_SMEM, st, a.k, w.chE.G, rs, w.Epart, a.P, w.Q, a.W_Q,
                        a.W_K, a.dP, w.part_qk));
  SA_TIMED("tw_sum_kernel", st,
           launch_after(tw_sum_kernel, 3 * DD, R_THREADS, 0, st, w.part_v, n_v, inv, w.part_qk, n_qk, a.dW_V, a.dW_Q, a.dW_K));
  return SA_OK;
}

}  // namespace sa
