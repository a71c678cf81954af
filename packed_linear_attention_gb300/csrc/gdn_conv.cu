// gdn_conv.cu — the short causal convolution in front of a recurrent layer, for packs of
// requests and for single tokens.
//
//     y[t][c] = act(bias[c] + sum_j w[c][j] x[t - W + 1 + j][c])
//
// Every output needs W inputs of its own channel and nothing else, so a thread takes 16 bytes of
// channels, keeps the last W - 1 rows in registers and walks down its rows: x is read once (and
// W - 1 rows more for every kTile rows), y written once, both 16 bytes a thread. Bound by HBM.
//
// A block takes kTile rows of one request and 128 threads' channels. The block of a request's
// first rows is the only one that touches its state: it reads the rows in front from the slot,
// then writes the slot and the request's checkpoints, copies of rows of x (or of the old state
// where the request is shorter than W - 1).
#include "gdn_step_internal.h"

namespace gdn {
namespace {

constexpr int kThreads = 128;
constexpr int kTile = 32;  // rows of a block
constexpr int kAhead = 8;  // rows loaded at once

template <typename T>
struct Channels {
  int c0, count;
  bool whole;         // 16 bytes of x and y
  bool whole_state;   // and of the state, whose rows are C elements apart
};
template <typename T>
__device__ __forceinline__ Channels<T> my_channels(int block, int channels) {
  Channels<T> k;
  k.c0 = (block * kThreads + (int)threadIdx.x) * Vec<T>::N;
  k.count = min(Vec<T>::N, channels - k.c0);
  k.whole = k.count == Vec<T>::N;
  k.whole_state = k.whole && channels % Vec<T>::N == 0;
  return k;
}

template <typename T, int W>
struct Taps {
  float w[Vec<T>::N][W], bias[Vec<T>::N];
  __device__ __forceinline__ Taps(const gdn_conv_config& cfg, int c0, int count) {
#pragma unroll
    for (int i = 0; i < Vec<T>::N; ++i) {
#pragma unroll
      for (int j = 0; j < W; ++j)
        w[i][j] = i < count ? __ldg(cfg.weight + (size_t)(c0 + i) * W + j) : 0.f;
      bias[i] = cfg.bias && i < count ? __ldg(cfg.bias + c0 + i) : 0.f;
    }
  }
  // rows: the W - 1 rows in front, oldest first
  __device__ __forceinline__ void apply(const float (*rows)[Vec<T>::N], const float* x, bool act,
                                        float* y) const {
#pragma unroll
    for (int i = 0; i < Vec<T>::N; ++i) {
      float s = fmaf(w[i][W - 1], x[i], bias[i]);
#pragma unroll
      for (int j = 0; j < W - 1; ++j) s = fmaf(w[i][j], rows[j][i], s);
      y[i] = act ? silu(s) : s;
    }
  }
};

template <typename T, int W>
__global__ void __launch_bounds__(kThreads) conv_kernel(ConvArgs p, int channel_blocks) {
  const int unit = blockIdx.x / channel_blocks, block = blockIdx.x % channel_blocks;
  int32_t* status = blockIdx.x == 0 ? p.status : nullptr;
  const gdn_requests& req = p.req;
  // a request has a unit for every kTile rows, one at least: that of its state
  const Unit u = find_unit<kThreads>(
      req.num_seqs, unit,
      [&](int n) {
        const Request q = load_request(req, n, status);
        return q.len < 0 ? 0 : max(1, (q.len + kTile - 1) / kTile);
      },
      [](int) { return 0; });
  if (u.seq < 0) return;
  const Request q = load_request(req, u.seq, nullptr);
  const int channels = p.cfg.channels;
  const Channels<T> k = my_channels<T>(block, channels);
  if (k.count <= 0) return;
  constexpr int N = Vec<T>::N;
  const T* x = static_cast<const T*>(p.x) + (size_t)q.lo * p.x_stride + k.c0;
  T* y = static_cast<T*>(p.y) + (size_t)q.lo * p.y_stride + k.c0;
  T* state = static_cast<T*>(p.pool) + (size_t)q.slot * (W - 1) * channels + k.c0;
  const int t0 = u.place * kTile, t1 = min(q.len, t0 + kTile);

  float rows[W - 1][N];
  if (t0 == 0) {
    Vec<T> old[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      old[j].raw = make_uint4(0, 0, 0, 0);
      if (!q.zero) old[j] = load_vec(state + (size_t)j * channels, k.count, k.whole_state);
      unpack(old[j], rows[j]);
    }
    // the last W - 1 inputs of the first `len` ones: rows of x, or of the old state
    auto save = [&](T* to, int len) {
#pragma unroll
      for (int j = 0; j < W - 1; ++j) {
        Vec<T> v = old[W - 2];
        const int at = len - (W - 1) + j;
        if (at >= 0) {
          v = load_vec(x + (size_t)at * p.x_stride, k.count, k.whole);
        } else {
#pragma unroll
          for (int i = 0; i < W - 1; ++i)
            if (W - 1 + at == i) v = old[i];
        }
        store_vec(to + (size_t)j * channels, v, k.count, k.whole_state);
      }
    };
    const int2 ck = load_checkpoints(req, u.seq, block == 0 && threadIdx.x == 0 ? p.status : nullptr);
    int before = 0;
    for (int i = ck.x; i < ck.y; ++i) {
      const int pos = req.ckpt_pos[i];
      if (pos <= before || pos > q.len) {
        if (block == 0 && threadIdx.x == 0) raise_status(p.status, GDN_ERR_INVALID_ARGUMENT);
        continue;
      }
      save(static_cast<T*>(p.ckpt) + (size_t)i * (W - 1) * channels + k.c0, pos);
      before = pos;
    }
    save(state, q.len);
  } else {
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      unpack(load_vec(x + (size_t)(t0 - (W - 1) + j) * p.x_stride, k.count, k.whole), rows[j]);
  }

  const Taps<T, W> taps(p.cfg, k.c0, k.count);
  const bool act = p.cfg.activation == GDN_ACT_SILU;
  for (int t = t0; t < t1; t += kAhead) {
    Vec<T> in[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (t + i < t1) in[i] = load_vec(x + (size_t)(t + i) * p.x_stride, k.count, k.whole);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (t + i >= t1) break;
      float v[N], out[N];
      unpack(in[i], v);
      taps.apply(rows, v, act, out);
#pragma unroll
      for (int j = 0; j + 1 < W - 1; ++j)
#pragma unroll
        for (int e = 0; e < N; ++e) rows[j][e] = rows[j + 1][e];
#pragma unroll
      for (int e = 0; e < N; ++e) rows[W - 2][e] = v[e];
      store_vec(y + (size_t)(t + i) * p.y_stride, pack<T>(out), k.count, k.whole);
    }
  }
}

// One token of a request: the state's rows move up by one.
template <typename T, int W>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(ConvArgs p, int channel_blocks) {
  const int b = blockIdx.x / channel_blocks;
  const int channels = p.cfg.channels;
  const Channels<T> k = my_channels<T>(blockIdx.x % channel_blocks, channels);
  if (k.count <= 0) return;
  const int slot = p.req.slot_idx[b];
  if (slot < 0 || slot >= p.req.num_slots) {
    if (slot >= 0) raise_status(p.status, GDN_ERR_INVALID_ARGUMENT);
    return;
  }
  constexpr int N = Vec<T>::N;
  T* state = static_cast<T*>(p.pool) + (size_t)slot * (W - 1) * channels + k.c0;
  Vec<T> old[W];
#pragma unroll
  for (int j = 0; j < W - 1; ++j)
    old[j] = load_vec(state + (size_t)j * channels, k.count, k.whole_state);
  old[W - 1] = load_vec(static_cast<const T*>(p.x) + (size_t)b * p.x_stride + k.c0, k.count, k.whole);
  const Taps<T, W> taps(p.cfg, k.c0, k.count);
  float rows[W - 1][N], v[N], out[N];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) unpack(old[j], rows[j]);
  unpack(old[W - 1], v);
  taps.apply(rows, v, p.cfg.activation == GDN_ACT_SILU, out);
#pragma unroll
  for (int j = 0; j < W - 1; ++j)
    store_vec(state + (size_t)j * channels, old[j + 1], k.count, k.whole_state);
  store_vec(static_cast<T*>(p.y) + (size_t)b * p.y_stride + k.c0, pack<T>(out), k.count, k.whole);
}

template <typename T>
int channel_blocks(int channels) {
  return (channels + kThreads * Vec<T>::N - 1) / (kThreads * Vec<T>::N);
}

template <typename T, int W>
int launch_packed(const ConvArgs& a, cudaStream_t s) {
  const int cb = channel_blocks<T>(a.cfg.channels);
  const int64_t units = (int64_t)a.req.num_tokens / kTile + a.req.num_seqs;
  conv_kernel<T, W><<<(unsigned)(units * cb), kThreads, 0, s>>>(a, cb);
  return (int)cudaGetLastError();
}
template <typename T, int W>
int launch_single(const ConvArgs& a, cudaStream_t s) {
  const int cb = channel_blocks<T>(a.cfg.channels);
  conv_step_kernel<T, W><<<(unsigned)((int64_t)a.req.num_tokens * cb), kThreads, 0, s>>>(a, cb);
  return (int)cudaGetLastError();
}
template <typename T>
int by_width(const ConvArgs& a, bool single, cudaStream_t s) {
  switch (a.cfg.width) {
    case 2: return single ? launch_single<T, 2>(a, s) : launch_packed<T, 2>(a, s);
    case 3: return single ? launch_single<T, 3>(a, s) : launch_packed<T, 3>(a, s);
    case 4: return single ? launch_single<T, 4>(a, s) : launch_packed<T, 4>(a, s);
  }
  return (int)cudaErrorInvalidValue;
}

int launch(const ConvArgs& a, bool single, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return a.cfg.io_dtype == GDN_BF16 ? by_width<__nv_bfloat16>(a, single, s)
                                    : by_width<float>(a, single, s);
}

}  // namespace

int launch_conv_packed(const ConvArgs& a, void* stream) { return launch(a, false, stream); }
int launch_conv_step(const ConvArgs& a, void* stream) {
  return a.req.num_tokens == 0 ? 0 : launch(a, true, stream);
}

}  // namespace gdn
