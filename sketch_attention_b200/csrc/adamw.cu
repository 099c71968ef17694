// AdamW over many tensors in one launch (decoupled weight decay, bias-corrected
// moments), the moments held in fp32 or in 8 bits.  Per value, in fp32:
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2        (g = gradient * grad_scale)
//   p = p (1 - lr w) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// 8-bit states: m and sqrt(v) in e4m3, one fp32 scale (largest magnitude / 448)
// per 128 consecutive values -- a row of a 128-wide table.  The square root
// halves v's range in octaves, so e4m3's 2^-9 .. 448 covers a ratio of 5e10 in
// v inside one block; a positive sqrt(v) below that range is held as the
// smallest code, not as zero, so a value whose second moment is tiny is never
// divided by eps alone (its step gets smaller instead).  The update itself uses
// the fp32 moments of this step, before they are rounded.
//
// Bound by memory: every value is read and written once (28 bytes in 32 bits, 16
// in 8, + 2 for the bf16 copy).  A thread owns 8 consecutive values (16-byte
// accesses; a block of 128 is half a warp, so its maximum is four shuffles), a
// CTA one chunk of 2048 values; the tensor of a chunk is found by a binary search
// over the list, which travels as the kernel's parameter: nothing is copied to the
// device beforehand, and a captured launch keeps its own list.  128 M values with
// the bf16 copy: 32 bits 0.557 ms (6.9 TB/s), 8 bits 0.385 ms (6.0 TB/s).  With
// resident CTAs that walk the chunks instead, 4 or 8 per SM, 0.65-0.68 and 0.41-0.43
// ms: the CTAs drift apart and touch more DRAM pages at once.  Streaming hints on
// the accesses cost 3-5%.
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>

#include "sa_internal.cuh"

namespace sa {

namespace {
constexpr int kBlock = 128;            // values per scale of an 8-bit state
constexpr int kPer = 8;                // values per thread
constexpr int kThreads = 256;
constexpr int kChunk = kThreads * kPer;
constexpr float kE4m3Max = 448.f, kE4m3Tiny = 0.001953125f;
// a block whose largest magnitude is below this has scale 0 and zeros: its scale would be denormal soon
constexpr float kScaleMin = 7.88860905e-31f;   // 2^-100

enum : int { GRAD_BF16 = 1, STATE_8 = 2 };

struct Item {
  float* param;
  const void* grad;
  void *m, *v;
  float *m_scale, *v_scale;
  __nv_bfloat16* copy;
  int64_t n;
  int64_t first;        // chunks of the tensors before this one
  float decay;
  int flags;
};
// lists up to kFew fit in 4 KB of parameters
constexpr int kFew = 48, kMany = 192;

// N tensors of 80 bytes each (the parameter space takes 32764 bytes)
template <int N>
struct List {
  Item item[N];
  int64_t chunks;
  int count;
  float b1, b1c, b2, b2c, eps;          // b1c = 1 - b1, b2c = 1 - b2, from double
  float lr, rbc1, rbc2;                 // 1 / (1 - b1^t), 1 / sqrt(1 - b2^t) of the host's step
  double log_b1, log_b2;
  const int64_t* step;
  const float* lr_dev;
  const float* grad_scale;
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// largest of 16 lanes' values (both halves of the warp at once); NaN if any is NaN
__device__ __forceinline__ float max16(float x) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) x = max_nan(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

__device__ __forceinline__ void from_e4m3(uint2 q, float* x) {
  const uint32_t w[2] = {q.x, q.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i / 2] >> (16 * (i % 2))), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ uint2 to_e4m3(const float* x) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(x[4 * i], x[4 * i + 1]), __NV_SATFINITE, __NV_E4M3) |
           (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2], x[4 * i + 3]), __NV_SATFINITE, __NV_E4M3) << 16;
  return make_uint2(w[0], w[1]);
}

// `left` of a thread's 8 values are there (left >= 8: all, by 16-byte accesses)
__device__ __forceinline__ void load8(const float* p, int64_t left, float* x) {
  if (left >= kPer) {
    const float4 a = *(const float4*)p, b = *(const float4*)(p + 4);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[i] = i < left ? p[i] : 0.f;
  }
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, int64_t left, float* x) {
  if (left >= kPer) {
    const uint4 a = *(const uint4*)p;
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[i] = i < left ? __bfloat162float(p[i]) : 0.f;
  }
}
__device__ __forceinline__ uint2 load_codes(const uint8_t* p, int64_t left) {
  if (left >= kPer) return *(const uint2*)p;
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (i < left) w[i / 4] |= (uint32_t)p[i] << (8 * (i % 4));
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store8(float* p, int64_t left, const float* x) {
  if (left >= kPer) {
    *(float4*)p = make_float4(x[0], x[1], x[2], x[3]);
    *(float4*)(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i < left) p[i] = x[i];
  }
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, int64_t left, const float* x) {
  if (left >= kPer) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *(const uint32_t*)&h;
    }
    *(uint4*)p = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i < left) p[i] = __float2bfloat16_rn(x[i]);
  }
}
__device__ __forceinline__ void store_codes(uint8_t* p, int64_t left, uint2 q) {
  if (left >= kPer) {
    *(uint2*)p = q;
  } else {
    const uint32_t w[2] = {q.x, q.y};
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i < left) p[i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
  }
}

// rounds 8 values of a block of 128 to e4m3 under the block's scale (`top`: the block's
// largest magnitude); `floor`: x >= 0 and no positive value becomes zero
template <bool kFloor>
__device__ __forceinline__ uint2 quantise(const float* x, float top, float* scale) {
  const bool some = !(top < kScaleMin);          // a NaN counts: it spreads over its block
  *scale = some ? top * (1.f / kE4m3Max) : 0.f;
  // x / scale, rounded to nearest: the reciprocal's product and one step on its residual (Markstein,
  // IBM Journal of Research and Development 34, 1990: exact where the reciprocal is rounded to nearest
  // and the residual does not underflow; it does for quotients below 2^-16 only, whose code is zero)
  const float inv = some ? __frcp_rn(*scale) : 0.f;
  float y[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const float q = x[i] * inv;
    y[i] = __fmaf_rn(__fmaf_rn(-q, *scale, x[i]), inv, q);
    if (kFloor && y[i] > 0.f) y[i] = fmaxf(y[i], kE4m3Tiny);
  }
  return to_e4m3(y);
}

template <int N>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ List<N> L) {
  // the step's scalars: the host's, or those in device memory when the kernel runs
  __shared__ float s_bc[2];
  const float gs = L.grad_scale ? *L.grad_scale : 1.f;
  if (L.grad_scale && !isfinite(gs)) return;     // an overflowed gradient: the step is left out
  float rbc1 = L.rbc1, rbc2 = L.rbc2;
  if (L.step) {
    if (threadIdx.x < 2) {
      const double t = (double)*L.step;
      s_bc[threadIdx.x] = threadIdx.x == 0 ? (float)(-1.0 / expm1(t * L.log_b1))
                                           : (float)(1.0 / sqrt(-expm1(t * L.log_b2)));
    }
    __syncthreads();
    rbc1 = s_bc[0];
    rbc2 = s_bc[1];
  }
  const float lr = L.lr_dev ? *L.lr_dev : L.lr;
  const float step_size = lr * rbc1;

  for (int64_t c = blockIdx.x; c < L.chunks; c += gridDim.x) {
    int lo = 0, hi = L.count - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (L.item[mid].first <= c) lo = mid; else hi = mid - 1;
    }
    const Item& t = L.item[lo];
    const int64_t at = (c - t.first) * kChunk + threadIdx.x * kPer;
    const int64_t left = t.n - at;               // <= 0: no value of this thread is there
    const bool is8 = t.flags & STATE_8;
    float p[kPer] = {}, g[kPer] = {}, m[kPer] = {}, v[kPer] = {};
    if (left > 0) {
      load8(t.param + at, left, p);
      if (t.flags & GRAD_BF16) load8((const __nv_bfloat16*)t.grad + at, left, g);
      else load8((const float*)t.grad + at, left, g);
      if (is8) {
        const float ms = t.m_scale[at / kBlock], vs = t.v_scale[at / kBlock];
        from_e4m3(load_codes((const uint8_t*)t.m + at, left), m);
        from_e4m3(load_codes((const uint8_t*)t.v + at, left), v);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          m[i] *= ms;
          v[i] *= vs;
          v[i] *= v[i];
        }
      } else {
        load8((const float*)t.m + at, left, m);
        load8((const float*)t.v + at, left, v);
      }
    }
    const float keep = 1.f - lr * t.decay;
    float r[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      // each rounding is spelled out, so that an 8-bit code does not depend on how the compiler
      // contracts: m = fl(b1c g + fl(b1 m)), v = fl(b2c fl(g g) + fl(b2 v))
      const float gi = g[i] * gs;
      m[i] = __fmaf_rn(L.b1c, gi, __fmul_rn(L.b1, m[i]));
      v[i] = __fmaf_rn(L.b2c, __fmul_rn(gi, gi), __fmul_rn(L.b2, v[i]));
      r[i] = sqrtf(v[i]);
      p[i] = p[i] * keep - step_size * __fdividef(m[i], fmaf(r[i], rbc2, L.eps));   // 2 ulp of the step
    }
    if (is8) {
      // all lanes take part in the block's maximum; the values past the end are zero
      float tm = fabsf(m[0]), tv = r[0];
#pragma unroll
      for (int i = 1; i < kPer; ++i) {
        tm = max_nan(tm, fabsf(m[i]));
        tv = max_nan(tv, r[i]);
      }
      tm = max16(tm);
      tv = max16(tv);
      float ms, vs;
      const uint2 qm = quantise<false>(m, tm, &ms), qv = quantise<true>(r, tv, &vs);
      if (left > 0) {
        store_codes((uint8_t*)t.m + at, left, qm);
        store_codes((uint8_t*)t.v + at, left, qv);
        if (at % kBlock == 0) {
          t.m_scale[at / kBlock] = ms;
          t.v_scale[at / kBlock] = vs;
        }
      }
    } else if (left > 0) {
      store8((float*)t.m + at, left, m);
      store8((float*)t.v + at, left, v);
    }
    if (left > 0) {
      store8(t.param + at, left, p);
      if (t.copy) store8(t.copy + at, left, p);
    }
  }
}
template <int N>
sa_status launch(const sa_adamw_tensor* tensors, int n_tensors, const sa_adamw_config& c, cudaStream_t st) {
  List<N> L;
  L.b1 = (float)c.beta1; L.b1c = (float)(1.0 - c.beta1);
  L.b2 = (float)c.beta2; L.b2c = (float)(1.0 - c.beta2);
  L.eps = (float)c.eps;
  L.lr = (float)c.lr;
  L.log_b1 = std::log(c.beta1);                  // log(0) = -inf: 1 - 0^t = 1 on both sides
  L.log_b2 = std::log(c.beta2);
  L.rbc1 = L.rbc2 = 1.f;
  if (!c.step_dev) {
    L.rbc1 = (float)(-1.0 / std::expm1((double)c.step * L.log_b1));
    L.rbc2 = (float)(1.0 / std::sqrt(-std::expm1((double)c.step * L.log_b2)));
  }
  L.step = c.step_dev;
  L.lr_dev = c.lr_dev;
  L.grad_scale = c.grad_scale_dev;
  for (int i = 0; i < n_tensors;) {
    L.count = 0;
    L.chunks = 0;
    for (; i < n_tensors && L.count < N; ++i) {
      const sa_adamw_tensor& t = tensors[i];
      if (t.n == 0) continue;
      L.item[L.count++] = {t.param, t.grad, t.m, t.v, t.m_scale, t.v_scale, (__nv_bfloat16*)t.param_bf16, t.n,
                           L.chunks, t.weight_decay,
                           (t.grad_dtype == SA_BF16 ? GRAD_BF16 : 0) | (t.state == SA_STATE_8BIT ? STATE_8 : 0)};
      L.chunks += (t.n + kChunk - 1) / kChunk;
    }
    if (L.count == 0) break;
    const unsigned grid = (unsigned)std::min<int64_t>(L.chunks, (int64_t)1 << 30);   // a CTA per chunk
    SA_TIMED("adamw_kernel", st, (adamw_kernel<N><<<grid, kThreads, 0, st>>>(L)));
  }
  return SA_OK;
}
}  // namespace

sa_status adamw_run(const sa_adamw_tensor* tensors, int n_tensors, const sa_adamw_config& c, cudaStream_t st) {
  return n_tensors <= kFew ? launch<kFew>(tensors, n_tensors, c, st) : launch<kMany>(tensors, n_tensors, c, st);
}

}  // namespace sa
