// gdn_step_internal.h — structures shared by the kernels around the recurrent layers (short
// convolution, selective scan, norm, sampling) and their C entry points.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/gdn.h"

namespace gdn {

constexpr int kMaxRequests = 4096;  // of one packed call
// Its rows: the kernels step past a request's last row by a block of 512 at most.
constexpr int32_t kMaxRows = INT32_MAX - 4096;

struct ConvArgs {
  gdn_conv_config cfg;
  gdn_requests req;
  const void* x;
  void* y;
  int64_t x_stride, y_stride;
  void* pool;
  void* ckpt;
  int32_t* status;
};
int launch_conv_packed(const ConvArgs& a, void* stream);
// batch = req.num_tokens, slots from req.slot_idx
int launch_conv_step(const ConvArgs& a, void* stream);

struct SsmArgs {
  gdn_ssm_config cfg;
  gdn_requests req;
  gdn_ssm_rows rows;
  float* pool;
  float* ckpt;
  float* ends;    // [units][C][N] end states of the segments of cut requests (workspace)
  float* steps;   // [units][C] their sums of dt
  int32_t segment;  // tokens of a segment; 0: requests run whole
  int32_t units;    // end states that the workspace holds
  int32_t* status;
};
// Tokens of a segment for calls of this shape, or 0 when requests run whole.
int32_t ssm_segment(const gdn_ssm_config& cfg, const gdn_requests& req);
// Segments behind their requests' first that the workspace has room for: those of disjoint requests.
int64_t ssm_units(const gdn_requests& req, int32_t segment);
// The most units of any call with at most as many requests and tokens, no longer ones.
int64_t ssm_most_units(const gdn_ssm_config& cfg, const gdn_requests& req);
int launch_ssm_packed(const SsmArgs& a, void* stream);
int launch_ssm_step(const SsmArgs& a, void* stream);

struct NormArgs {
  gdn_norm_config cfg;
  int32_t num_tokens;
  const void *x, *residual, *gate;
  void *sum, *y, *codes;
  int64_t x_stride, residual_stride, gate_stride, sum_stride, y_stride, codes_stride;
  float* scales;
};
constexpr int kMaxNormRow = 32768;
int launch_rms_norm(const NormArgs& a, void* stream);

struct SampleArgs {
  int32_t io_dtype, num_rows, vocab;
  const void* logits;
  int64_t stride;
  const float* temperature;
  const int32_t* top_k;
  const float *top_p, *min_p, *u;
  int32_t* token;
  float* logprob;
  int32_t* status;
};
constexpr int kMaxVocab = 1 << 18;
int launch_sample(const SampleArgs& a, void* stream);

#ifdef __CUDACC__

__device__ __forceinline__ void raise_status(int32_t* status, int32_t code) {
  if (status) atomicMax(status, code);
}

// A request as the device finds it: rows [lo, lo + len) and the state's slot; len < 0: not served.
struct Request {
  int32_t lo, len, slot;
  bool zero;
};
__device__ __forceinline__ Request load_request(const gdn_requests& r, int32_t n, int32_t* status) {
  const int32_t lo = r.cu[n], hi = r.cu[n + 1];
  const int32_t slot = r.slot_idx ? r.slot_idx[n] : n;
  Request q = {lo, hi - lo, slot, r.start_zero && r.start_zero[n] != 0};
  if (lo < 0 || hi < lo || hi > r.num_tokens || hi - lo > r.max_len || slot >= r.num_slots) {
    raise_status(status, GDN_ERR_INVALID_ARGUMENT);
    q.len = -1;
  } else if (slot < 0) {
    q.len = -1;
  }
  return q;
}

// The checkpoints of request n: [begin, end) of the CSR, held to what the arrays have.
__device__ __forceinline__ int2 load_checkpoints(const gdn_requests& r, int32_t n,
                                                 int32_t* status) {
  if (!r.ckpt_cu) return make_int2(0, 0);
  const int32_t lo = r.ckpt_cu[n], hi = r.ckpt_cu[n + 1];
  if (lo < 0 || hi < lo || hi > r.num_ckpt) {
    raise_status(status, GDN_ERR_INVALID_ARGUMENT);
    return make_int2(0, 0);
  }
  return make_int2(lo, hi);
}

// Work units of the requests in order, request n having units(n): the request that unit `u`
// belongs to, the unit's place in it, and the sum of extra(n) over the requests in front of it.
// Every thread of a block of THREADS calls it; seq < 0 when there is no unit u. Sums are held at
// 2^31 - 1 (requests that overlap may ask for any number of units).
struct Unit {
  int32_t seq, place, extra;
};
template <int THREADS, class Units, class Extra>
__device__ Unit find_unit(int32_t num_seqs, int32_t u, Units units, Extra extra) {
  __shared__ uint32_t warp_units[THREADS / 32], warp_extra[THREADS / 32];
  __shared__ Unit found;
  constexpr uint32_t kTop = 0x7fffffffu;
  const int per = (num_seqs + THREADS - 1) / THREADS;
  const int first = threadIdx.x * per, last = min(num_seqs, first + per);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t mine = 0, more = 0;
  for (int n = first; n < last; ++n) {
    mine = min(kTop, mine + (uint32_t)units(n));
    more = min(kTop, more + (uint32_t)extra(n));
  }
  uint32_t upto = mine, upto_more = more;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t a = __shfl_up_sync(0xffffffffu, upto, off);
    const uint32_t b = __shfl_up_sync(0xffffffffu, upto_more, off);
    if (lane >= off) {
      upto = min(kTop, upto + a);
      upto_more = min(kTop, upto_more + b);
    }
  }
  if (threadIdx.x == 0) found = {-1, 0, 0};
  if (lane == 31) {
    warp_units[warp] = upto;
    warp_extra[warp] = upto_more;
  }
  __syncthreads();
  uint32_t at = __shfl_up_sync(0xffffffffu, upto, 1);  // sums in front of this thread's requests
  uint32_t at_more = __shfl_up_sync(0xffffffffu, upto_more, 1);
  if (lane == 0) at = at_more = 0;
  uint32_t base = 0, base_more = 0;
  for (int w = 0; w < warp; ++w) {
    base = min(kTop, base + warp_units[w]);
    base_more = min(kTop, base_more + warp_extra[w]);
  }
  at = min(kTop, base + at);
  at_more = min(kTop, base_more + at_more);
  if (at <= (uint32_t)u && (uint32_t)u < min(kTop, base + upto)) {
    for (int n = first; n < last; ++n) {
      const uint32_t k = (uint32_t)units(n);
      if ((uint32_t)u - at < k) {
        found = {n, (int32_t)((uint32_t)u - at), (int32_t)at_more};
        break;
      }
      at += k;
      at_more = min(kTop, at_more + (uint32_t)extra(n));
    }
  }
  __syncthreads();
  return found;
}

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Two fp32 numbers in a register pair, worked on together. A pair takes an fma pipe as long as its
// two numbers would one by one, but leaves issue slots and does not hold up the special functions:
// 64 fma beside 16 ex2 take 106 clocks a warp, 32 pairs 69.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pair(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ f32x2 both(float v) { return pair(v, v); }
__device__ __forceinline__ void unpair(f32x2 p, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ f32x2 ex2(f32x2 x) {
  float lo, hi;
  unpair(x, lo, hi);
  return pair(ex2(lo), ex2(hi));
}
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
constexpr float kLog2e = 1.4426950408889634f;
// v / (1 + exp(-v)); past 2^126 the reciprocal is 0, and so is the result to 1e-36; -inf gives NaN, as
// the formula does
__device__ __forceinline__ float silu(float v) { return v * rcp(1.f + ex2(-kLog2e * v)); }
__device__ __forceinline__ f32x2 silu(f32x2 v) {
  float a, b;
  unpair(add2(ex2(mul2(v, both(-kLog2e))), both(1.f)), a, b);
  return mul2(v, pair(rcp(a), rcp(b)));
}

// 16 bytes of T, and their values
template <typename T>
struct Vec {
  static constexpr int N = 16 / sizeof(T);
  uint4 raw;
};
template <typename T>
__device__ __forceinline__ void unpack(const Vec<T>& v, float* f);
template <>
__device__ __forceinline__ void unpack<float>(const Vec<float>& v, float* f) {
  f[0] = __uint_as_float(v.raw.x);
  f[1] = __uint_as_float(v.raw.y);
  f[2] = __uint_as_float(v.raw.z);
  f[3] = __uint_as_float(v.raw.w);
}
template <>
__device__ __forceinline__ void unpack<__nv_bfloat16>(const Vec<__nv_bfloat16>& v, float* f) {
  const uint32_t w[4] = {v.raw.x, v.raw.y, v.raw.z, v.raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <typename T>
__device__ __forceinline__ Vec<T> pack(const float* f);
template <>
__device__ __forceinline__ Vec<float> pack<float>(const float* f) {
  return {make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                     __float_as_uint(f[3]))};
}
template <>
__device__ __forceinline__ Vec<__nv_bfloat16> pack<__nv_bfloat16>(const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = reinterpret_cast<const uint32_t&>(h);
  }
  return {make_uint4(w[0], w[1], w[2], w[3])};
}

// `count` elements at p (N of them: one 16-byte access where `whole`; the rest read as 0)
template <typename T>
__device__ __forceinline__ Vec<T> load_vec(const T* p, int count, bool whole) {
  Vec<T> v;
  v.raw = make_uint4(0, 0, 0, 0);
  if (whole) {
    v.raw = *reinterpret_cast<const uint4*>(p);
  } else {
    T* e = reinterpret_cast<T*>(&v.raw);
#pragma unroll
    for (int i = 0; i < Vec<T>::N; ++i)
      if (i < count) e[i] = p[i];
  }
  return v;
}
template <typename T>
__device__ __forceinline__ void store_vec(T* p, const Vec<T>& v, int count, bool whole) {
  if (whole) {
    *reinterpret_cast<uint4*>(p) = v.raw;
  } else {
    const T* e = reinterpret_cast<const T*>(&v.raw);
#pragma unroll
    for (int i = 0; i < Vec<T>::N; ++i)
      if (i < count) p[i] = e[i];
  }
}

#endif  // __CUDACC__

}  // namespace gdn
