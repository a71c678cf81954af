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

constexpr float kMinScale = 0x1p-100f, kTop = 448.f;

// 8 elements as they lie in memory: 16 bytes of bf16, 32 of fp32. `count` of them are the row's; WHOLE:
// all 8 or none.
template <typename T>
struct Eight {
  static constexpr int kVecs = 8 / Vec<T>::N;
  Vec<T> v[kVecs];
  template <bool WHOLE>
  __device__ __forceinline__ void load(const T* p, int count) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      if constexpr (WHOLE) {
        v[i].raw = make_uint4(0, 0, 0, 0);
        if (count > 0) v[i].raw = reinterpret_cast<const uint4*>(p)[i];
      } else {
        v[i] = load_vec(p + i * Vec<T>::N, count - i * Vec<T>::N, count >= 8);
      }
    }
  }
  __device__ __forceinline__ void values(f32x2* f) const {
    float x[8];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) unpack(v[i], x + i * Vec<T>::N);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = pair(x[2 * i], x[2 * i + 1]);
  }
  template <bool WHOLE>
  __device__ __forceinline__ static void store(T* p, int count, const f32x2* f) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) unpair(f[i], x[2 * i], x[2 * i + 1]);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      if constexpr (WHOLE) {
        if (count > 0) reinterpret_cast<uint4*>(p)[i] = pack<T>(x + i * Vec<T>::N).raw;
      } else {
        store_vec(p + i * Vec<T>::N, pack<T>(x + i * Vec<T>::N), count - i * Vec<T>::N, count >= 8);
      }
    }
  }
};

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

// The scale of values up to `top` and its reciprocal: top / 448, or the least power of two at least
// that.
__device__ __forceinline__ void scale_of(float top, bool pow2, float& scale, float& inv) {
  if (pow2) {
    // top = m 2^e, m in [1, 2): 448 is 1.75 2^8
    const uint32_t bits = __float_as_uint(top);
    const int e = max(-100, (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u));
    scale = __uint_as_float((uint32_t)(127 + e) << 23);
    inv = __uint_as_float((uint32_t)(127 - e) << 23);
  } else {
    scale = fmaxf(top * (1.f / kTop), kMinScale);
    inv = rcp(scale);
  }
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return lo | (uint32_t)hi << 16;
}

// Blocks of 256 threads on an SM; 0: as many as the registers give. 32 gated heads of 128, 32,768 rows, four
// vectors a thread: 139 us at 64 registers (76 bytes a thread spill), 147 at the 78 that it would take.
template <typename T, int VPT, bool HEADS, int THREADS>
constexpr int kResident = sizeof(T) == 2 && VPT == 4 && HEADS && THREADS == 256 ? 4 : 0;

// HEADS: heads of `dim` elements, each by itself; else the row is one. WHOLE: rows of a multiple of 8.
template <typename T, int VPT, bool HEADS, bool WHOLE, int THREADS>
__global__ void __launch_bounds__(THREADS, kResident<T, VPT, HEADS, THREADS>) norm_kernel(NormArgs p, int team) {
  __shared__ float sums[32], tops[32];
  const int rows = blockDim.x / team;
  const int64_t row = (int64_t)blockIdx.x * rows + threadIdx.x / team;
  const int me = threadIdx.x % team;
  const int width = p.cfg.num_heads * p.cfg.dim;
  const bool live = row < p.num_tokens;
  const int64_t r = live ? row : p.num_tokens - 1;
  f32x2 s[VPT][4];
  float sum[VPT];
  int count[VPT];
  Eight<T> gate[VPT];
  {
    Eight<T> x[VPT], residual[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * team + me) * 8;
      count[i] = max(0, min(8, width - c));
      x[i].template load<WHOLE>(static_cast<const T*>(p.x) + r * p.x_stride + c, count[i]);
      if (p.residual)
        residual[i].template load<WHOLE>(static_cast<const T*>(p.residual) + r * p.residual_stride + c, count[i]);
      if (p.gate)
        gate[i].template load<WHOLE>(static_cast<const T*>(p.gate) + r * p.gate_stride + c, count[i]);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      x[i].values(s[i]);
      if (p.residual) {
        f32x2 f[4];
        residual[i].values(f);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[i][e] = add2(s[i][e], f[e]);
      }
    }
  }
  float all = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    f32x2 q = mul2(s[i][0], s[i][0]);
#pragma unroll
    for (int e = 1; e < 4; ++e) q = fma2(s[i][e], s[i][e], q);
    float lo, hi;
    unpair(q, lo, hi);
    sum[i] = lo + hi;
    if (HEADS) sum[i] = lanes<false>(sum[i], p.cfg.dim / 8);
    all += sum[i];
    if (p.sum && live)
      Eight<T>::template store<WHOLE>(static_cast<T*>(p.sum) + r * p.sum_stride + (i * team + me) * 8, count[i], s[i]);
  }
  if (!HEADS) all = team_reduce<false>(all, team, sums);
  const float inv_dim = 1.f / (float)p.cfg.dim;
  float top[VPT], row_top = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * team + me) * 8;
    const f32x2 inv = both(rsqrtf(fmaf(HEADS ? sum[i] : all, inv_dim, p.cfg.eps)));
#pragma unroll
    for (int e = 0; e < 4; ++e) s[i][e] = mul2(s[i][e], inv);
    if (p.cfg.weight) {
      Eight<float> raw;
      f32x2 w[4];
      raw.load<WHOLE>(p.cfg.weight + (HEADS ? c % p.cfg.dim : c), count[i]);
      raw.values(w);
#pragma unroll
      for (int e = 0; e < 4; ++e) s[i][e] = mul2(s[i][e], add2(w[e], both(p.cfg.weight_offset)));
    }
    if (p.gate) {
      f32x2 g[4];
      gate[i].values(g);
#pragma unroll
      for (int e = 0; e < 4; ++e) s[i][e] = mul2(s[i][e], silu(g[e]));
    }
    if (p.y && live)
      Eight<T>::template store<WHOLE>(static_cast<T*>(p.y) + r * p.y_stride + c, count[i], s[i]);
    if (!p.codes) continue;
    // the largest finite value (what lies past the row is 0, or the weights' NaN times it)
    float v[8];
    top[i] = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      unpair(s[i][e], v[2 * e], v[2 * e + 1]);
      top[i] = fmaxf(top[i], fmaxf(fabsf(v[2 * e]), fabsf(v[2 * e + 1])));
    }
    if (top[i] == INFINITY) {
      top[i] = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (fabsf(v[e]) < INFINITY) top[i] = fmaxf(top[i], fabsf(v[e]));
    }
    row_top = fmaxf(row_top, top[i]);
  }
  if (!p.codes) return;
  const int group = p.cfg.scale_group;
  if (group == 0) row_top = team_reduce<true>(row_top, team, tops);
  uint8_t* codes = static_cast<uint8_t*>(p.codes) + r * p.codes_stride;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * team + me) * 8;
    const float t = group == 0 ? row_top : lanes<true>(top[i], group / 8);
    float scale, inv;
    scale_of(t, p.cfg.scale_pow2 != 0, scale, inv);
    if (!live || count[i] == 0) continue;
    if (group == 0) {
      if (c == 0) p.scales[r] = scale;
    } else if ((c & (group - 1)) == 0) {
      p.scales[r * (width / group) + c / group] = scale;
    }
    float v[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) unpair(mul2(s[i][e], both(inv)), v[2 * e], v[2 * e + 1]);
    uint2 q;
    q.x = e4m3x4(v[0], v[1], v[2], v[3]);
    q.y = e4m3x4(v[4], v[5], v[6], v[7]);
    if (WHOLE || count[i] == 8) {
      *reinterpret_cast<uint2*>(codes + c) = q;
    } else {
      for (int e = 0; e < count[i]; ++e) codes[c + e] = (uint8_t)((e < 4 ? q.x : q.y) >> (8 * (e & 3)));
    }
  }
}

template <typename T, int VPT, bool HEADS, bool WHOLE>
int launch_rows(const NormArgs& a, int team, cudaStream_t s) {
  const int threads = std::max(team, 128), rows = threads / team;
  const unsigned grid = (unsigned)((a.num_tokens + (int64_t)rows - 1) / rows);
  if (threads <= 256) norm_kernel<T, VPT, HEADS, WHOLE, 256><<<grid, threads, 0, s>>>(a, team);
  else norm_kernel<T, VPT, HEADS, WHOLE, 1024><<<grid, threads, 0, s>>>(a, team);
  return (int)cudaGetLastError();
}

template <typename T, bool HEADS, bool WHOLE>
int launch(const NormArgs& a, cudaStream_t s) {
  const int vecs = (a.cfg.num_heads * a.cfg.dim + 7) / 8;
  // Few rows: as many threads a row as there are vectors. Many: two or four vectors a thread (32,768
  // rows of 2,048 with residual and codes: 121 us with one, 92 with two, 98 with four; 32 gated heads
  // of 128: 171, 152 and 139). Measured at these widths: rows of fewer vectors than a warp's leave some
  // empty (4 gated heads of 64: 33 us, 7.4 of them bytes).
  int vpt = a.num_tokens <= 1024 ? 1 : HEADS && sizeof(T) == 2 ? 4 : 2;
  while (vecs > 1024 * vpt) vpt *= 2;
  int team = 32;
  while (team * vpt < vecs) team *= 2;
  switch (vpt) {
    case 1: return launch_rows<T, 1, HEADS, WHOLE>(a, team, s);
    case 2: return launch_rows<T, 2, HEADS, WHOLE>(a, team, s);
    case 4: return launch_rows<T, 4, HEADS, WHOLE>(a, team, s);
  }
  return (int)cudaErrorInvalidValue;
}
template <typename T>
int launch(const NormArgs& a, cudaStream_t s) {
  if (a.cfg.num_heads > 1) return launch<T, true, true>(a, s);  // heads are multiples of 8
  return a.cfg.dim % 8 == 0 ? launch<T, false, true>(a, s) : launch<T, false, false>(a, s);
}

}  // namespace

int launch_rms_norm(const NormArgs& a, void* stream) {
  if (a.num_tokens == 0) return 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return a.cfg.io_dtype == GDN_BF16 ? launch<__nv_bfloat16>(a, s) : launch<float>(a, s);
}

}  // namespace gdn
