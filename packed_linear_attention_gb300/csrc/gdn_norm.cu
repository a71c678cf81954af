// gdn_norm.cu — root-mean-square norm with the residual's addition in front, a gate and an 8-bit
// output behind.
//
//     s = x + residual;  v = s / sqrt(mean(s^2) + eps) * (w + offset) * silu(gate)
//     y = v,  codes = e4m3(v / scale)
//
// Two passes over a row that stays in registers: each input is read once and each output written
// once, 16 or 32 bytes a thread (8 elements). A row belongs to `team` threads with VPT vectors of
// 8 elements each; a head of 64, 128 or 256 elements is 8, 16 or 32 neighbouring lanes of one
// vector, and so is a group of columns with one scale, so only whole rows need shared memory.
// Bound by HBM; a few rows alone by the launch and one chain of loads and sums.
#include <algorithm>

#include "gdn_step_internal.h"

namespace gdn {
namespace {

#ifndef NV
#define NV 2
#endif
constexpr float kMinScale = 0x1p-100f, kTop = 448.f;

// 8 elements: 16 bytes of bf16, 32 of fp32
template <typename T>
struct Eight {
  Vec<T> v[8 / Vec<T>::N];
  __device__ __forceinline__ Eight(const T* p, int count) {
#pragma unroll
    for (int i = 0; i < 8 / Vec<T>::N; ++i)
      v[i] = load_vec(p + i * Vec<T>::N, count - i * Vec<T>::N, count >= 8);
  }
  __device__ __forceinline__ Eight() {}
  __device__ __forceinline__ void values(float* f) const {
#pragma unroll
    for (int i = 0; i < 8 / Vec<T>::N; ++i) unpack(v[i], f + i * Vec<T>::N);
  }
};
template <typename T>
__device__ __forceinline__ void store8(T* p, int count, const float* f) {
  constexpr int N = Vec<T>::N;
#pragma unroll
  for (int i = 0; i < 8; i += N) store_vec(p + i, pack<T>(f + i), count - i, count >= 8);
}

// Sum (or maximum) over `width` neighbouring lanes.
template <bool MAX>
__device__ __forceinline__ float lanes(float v, int width) {
  for (int off = width >> 1; off > 0; off >>= 1) {
    const float o = __shfl_xor_sync(0xffffffffu, v, off);
    v = MAX ? fmaxf(v, o) : v + o;
  }
  return v;
}
// Over the `team` threads of a row (a power of two); every thread of the block calls it.
template <bool MAX>
__device__ __forceinline__ float team_reduce(float v, int team, float* shared) {
  v = lanes<MAX>(v, min(team, 32));
  if (team <= 32) return v;
  const int warps = team / 32, warp = threadIdx.x / 32, first = warp / warps * warps;
  if (threadIdx.x % 32 == 0) shared[warp] = v;
  __syncthreads();
  float r = shared[first];
  for (int i = 1; i < warps; ++i) r = MAX ? fmaxf(r, shared[first + i]) : r + shared[first + i];
  return r;
}

// The scale of values up to `top`: top / 448, or the least power of two at least that.
__device__ __forceinline__ float scale_of(float top, bool pow2) {
  if (pow2) {
    // top = m 2^e, m in [1, 2): 448 is 1.75 2^8
    const uint32_t bits = __float_as_uint(top);
    const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u);
    return e <= -100 ? kMinScale : __uint_as_float((uint32_t)(e + 127) << 23);
  }
  return fmaxf(__fdiv_rn(top, kTop), kMinScale);
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return lo | (uint32_t)hi << 16;
}

// HEADS: heads of `dim` elements, each by itself; else the row is one.
template <typename T, int VPT, bool HEADS, int THREADS>
__global__ void __launch_bounds__(THREADS) norm_kernel(NormArgs p, int team) {
  __shared__ float sums[32], tops[32];
  const int rows = blockDim.x / team;
  const int64_t row = (int64_t)blockIdx.x * rows + threadIdx.x / team;
  const int me = threadIdx.x % team;
  const int width = p.cfg.num_heads * p.cfg.dim;
  const bool live = row < p.num_tokens;
  const int64_t r = live ? row : p.num_tokens - 1;
  float s[VPT][8], sum[VPT];
  int count[VPT];
  Eight<T> gate[VPT];
  {
    Eight<T> x[VPT], residual[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * team + me) * 8;
      count[i] = max(0, min(8, width - c));
      x[i] = Eight<T>(static_cast<const T*>(p.x) + r * p.x_stride + c, count[i]);
      if (p.residual)
        residual[i] = Eight<T>(static_cast<const T*>(p.residual) + r * p.residual_stride + c, count[i]);
      if (p.gate)
        gate[i] = Eight<T>(static_cast<const T*>(p.gate) + r * p.gate_stride + c, count[i]);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      x[i].values(s[i]);
      if (p.residual) {
        float f[8];
        residual[i].values(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[i][e] += f[e];
      }
    }
  }
  float all = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    sum[i] = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[i] = fmaf(s[i][e], s[i][e], sum[i]);
    if (HEADS) sum[i] = lanes<false>(sum[i], p.cfg.dim / 8);
    all += sum[i];
  }
  if (!HEADS) all = team_reduce<false>(all, team, sums);
  const float inv_dim = 1.f / (float)p.cfg.dim;
  if (p.sum && live) {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      store8(static_cast<T*>(p.sum) + r * p.sum_stride + (i * team + me) * 8, count[i], s[i]);
  }
  float top[VPT], row_top = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * team + me) * 8;
    const float inv = rsqrtf(fmaf(HEADS ? sum[i] : all, inv_dim, p.cfg.eps));
    float w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = 1.f;
    if (p.cfg.weight && count[i] > 0) {
      Eight<float>(p.cfg.weight + (HEADS ? c % p.cfg.dim : c), count[i]).values(w);
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] += p.cfg.weight_offset;
    }
    float g[8];
    if (p.gate) {
      gate[i].values(g);
#pragma unroll
      for (int e = 0; e < 8; e += 2) unpair(silu(pair(g[e], g[e + 1])), g[e], g[e + 1]);
    }
    top[i] = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float v = s[i][e] * inv * w[e];
      if (p.gate) v *= g[e];
      s[i][e] = v;
      const float m = fabsf(v);
      if (e < count[i] && m <= 3.4028234e38f) top[i] = fmaxf(top[i], m);
    }
    row_top = fmaxf(row_top, top[i]);
    if (p.y && live) store8(static_cast<T*>(p.y) + r * p.y_stride + c, count[i], s[i]);
  }
  if (!p.codes) return;
  const int group = p.cfg.scale_group;
  if (group == 0) row_top = team_reduce<true>(row_top, team, tops);
  uint8_t* codes = static_cast<uint8_t*>(p.codes) + r * p.codes_stride;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * team + me) * 8;
    const float t = group == 0 ? row_top : lanes<true>(top[i], group / 8);
    const float scale = scale_of(t, p.cfg.scale_pow2 != 0);
    const float inv = __fdiv_rn(1.f, scale);
    if (!live || count[i] == 0) continue;
    if (group == 0) {
      if (c == 0) p.scales[r] = scale;
    } else if (c % group == 0) {
      p.scales[r * (width / group) + c / group] = scale;
    }
    uint2 q;
    q.x = e4m3x4(s[i][0] * inv, s[i][1] * inv, s[i][2] * inv, s[i][3] * inv);
    q.y = e4m3x4(s[i][4] * inv, s[i][5] * inv, s[i][6] * inv, s[i][7] * inv);
    if (count[i] == 8) {
      *reinterpret_cast<uint2*>(codes + c) = q;
    } else {
      for (int e = 0; e < count[i]; ++e) codes[c + e] = (uint8_t)((e < 4 ? q.x : q.y) >> (8 * (e & 3)));
    }
  }
}

template <typename T, int VPT, bool HEADS>
int launch_rows(const NormArgs& a, int team, cudaStream_t s) {
  const int threads = std::max(team, 128), rows = threads / team;
  const unsigned grid = (unsigned)((a.num_tokens + (int64_t)rows - 1) / rows);
  if (threads <= 256) norm_kernel<T, VPT, HEADS, 256><<<grid, threads, 0, s>>>(a, team);
  else norm_kernel<T, VPT, HEADS, 1024><<<grid, threads, 0, s>>>(a, team);
  return (int)cudaGetLastError();
}

template <typename T, bool HEADS>
int launch(const NormArgs& a, cudaStream_t s) {
  const int vecs = (a.cfg.num_heads * a.cfg.dim + 7) / 8;
  int vpt = a.num_tokens > 1024 ? NV : 1;  // 64 bytes of a thread's row
  while (vecs > 1024 * vpt) vpt *= 2;
  int team = 32;
  while (team * vpt < vecs) team *= 2;
  switch (vpt) {
    case 1: return launch_rows<T, 1, HEADS>(a, team, s);
    case 2: return launch_rows<T, 2, HEADS>(a, team, s);
    case 4: return launch_rows<T, 4, HEADS>(a, team, s);
  }
  return (int)cudaErrorInvalidValue;
}

}  // namespace

int launch_rms_norm(const NormArgs& a, void* stream) {
  if (a.num_tokens == 0) return 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a.cfg.io_dtype == GDN_BF16)
    return a.cfg.num_heads > 1 ? launch<__nv_bfloat16, true>(a, s) : launch<__nv_bfloat16, false>(a, s);
  return a.cfg.num_heads > 1 ? launch<float, true>(a, s) : launch<float, false>(a, s);
}

}  // namespace gdn
