// gdn_conv.cu — the short causal convolution in front of a recurrent layer, for packs of
// requests and for single tokens.
//
//     y[t][c] = act(bias[c] + sum_j w[c][j] x[t - W + 1 + j][c])
//
// Every output needs W inputs of its own channel and nothing else, so a thread takes four channels,
// keeps their last W - 1 rows in registers and walks down its rows: x is read once (and W - 1 rows
// more for every block's rows), y written once, 8 or 16 bytes a thread. Bound by HBM: four channels
// are few enough registers for the loads in flight that it takes.
//
// A block takes `tile` rows of one request and 128 threads' channels. The block of a request's
// first rows is the only one that touches its state: it reads the rows in front from the slot,
// then writes the slot and the request's checkpoints, copies of rows of x (or of the old state
// where the request is shorter than W - 1).
#include "gdn_step_internal.h"

namespace gdn {
namespace {

constexpr int kThreads = 128;
// Rows loaded at once and blocks of an SM: loads on their way are what the wave waits for. bf16, 32 x
// 1,024 rows of 8,192 channels, blocks of 128 rows: four rows and as many blocks as fit (six) 210 us, six
// and seven 181 (124 bytes of a thread's registers spill), six and six 189, seven and seven 194 (472
// bytes), four and eight 196, eight and five 195. fp32: four and five 328, three and six 333.
template <typename T>
constexpr int kAhead = sizeof(T) == 2 ? 6 : 4;
template <typename T>
constexpr int kResident = sizeof(T) == 2 ? 7 : 5;

// Four channels of a row as they lie in memory.
template <typename T>
struct Four {
  uint32_t w[sizeof(T)];

  __device__ __forceinline__ void load(const T* p, int count, bool whole) {
    if (whole) {
      if constexpr (sizeof(T) == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x, w[1] = v.y;
      }
    } else {
      clear();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i >= count) continue;
        if constexpr (sizeof(T) == 4) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
        else w[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i % 2));
      }
    }
  }
  __device__ __forceinline__ void store(T* p, int count, bool whole) const {
    if (whole) {
      if constexpr (sizeof(T) == 4) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
      else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i >= count) continue;
        if constexpr (sizeof(T) == 4) reinterpret_cast<uint32_t*>(p)[i] = w[i];
        else reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(w[i / 2] >> (16 * (i % 2)));
      }
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) w[i] = 0;
  }
  __device__ __forceinline__ void values(f32x2* f) const {
    if constexpr (sizeof(T) == 4) {
      f[0] = pair(__uint_as_float(w[0]), __uint_as_float(w[1]));
      f[1] = pair(__uint_as_float(w[2]), __uint_as_float(w[3]));
    } else {
      f[0] = pair(__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xffff0000u));
      f[1] = pair(__uint_as_float(w[1] << 16), __uint_as_float(w[1] & 0xffff0000u));
    }
  }
  __device__ __forceinline__ explicit Four(const f32x2* f) {
    float v[4];
    unpair(f[0], v[0], v[1]);
    unpair(f[1], v[2], v[3]);
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(v[i]);
    } else {
      const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
      w[0] = reinterpret_cast<const uint32_t&>(a);
      w[1] = reinterpret_cast<const uint32_t&>(b);
    }
  }
  __device__ __forceinline__ Four() {}
};

struct Channels {
  int c0, count;
  bool whole;         // x and y in one access
  bool whole_state;   // and the state, whose rows are C elements apart
};
__device__ __forceinline__ Channels my_channels(int block, int channels) {
  Channels k;
  k.c0 = (block * kThreads + (int)threadIdx.x) * 4;
  k.count = min(4, channels - k.c0);
  k.whole = k.count == 4;
  k.whole_state = k.whole && channels % 4 == 0;
  return k;
}

template <int W>
struct Taps {
  f32x2 w[2][W], bias[2];
  __device__ __forceinline__ Taps(const gdn_conv_config& cfg, int c0, int count) {
    float f[4][W], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int j = 0; j < W; ++j)
        f[i][j] = i < count ? __ldg(cfg.weight + (size_t)(c0 + i) * W + j) : 0.f;
      b[i] = cfg.bias && i < count ? __ldg(cfg.bias + c0 + i) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int j = 0; j < W; ++j) w[i][j] = pair(f[2 * i][j], f[2 * i + 1][j]);
      bias[i] = pair(b[2 * i], b[2 * i + 1]);
    }
  }
  // rows: the W - 1 rows in front, oldest first
  __device__ __forceinline__ void apply(const f32x2 (*rows)[2], const f32x2* x, bool act,
                                        f32x2 (&y)[2]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f32x2 s = fma2(w[i][W - 1], x[i], bias[i]);
#pragma unroll
      for (int j = 0; j < W - 1; ++j) s = fma2(w[i][j], rows[j][i], s);
      y[i] = act ? silu(s) : s;
    }
  }
};

// Down `left` rows from x to y, `rows` being those in front.
template <typename T, int W, bool WHOLE>
__device__ __forceinline__ void walk(const Taps<W>& taps, f32x2 (&rows)[W - 1][2], const T* x, T* y,
                                     const ConvArgs& p, int left, int count, bool act) {
  constexpr int N = kAhead<T>;
  Four<T> next[N];  // on their way while the rows in front of them are worked on
  const auto fetch = [&](int n) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i < n) next[i].load(x, count, WHOLE);
      x += p.x_stride;
    }
  };
  const auto one = [&](const Four<T>& in) {
    f32x2 v[2], out[2];
    in.values(v);
    taps.apply(rows, v, act, out);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int j = 0; j + 1 < W - 1; ++j) rows[j][e] = rows[j + 1][e];
      rows[W - 2][e] = v[e];
    }
    Four<T>(out).store(y, count, WHOLE);
    y += p.y_stride;
  };
  fetch(left);
  for (; left >= 2 * N; left -= N) {
    Four<T> in[N];
#pragma unroll
    for (int i = 0; i < N; ++i) in[i] = next[i];
    fetch(N);
#pragma unroll
    for (int i = 0; i < N; ++i) one(in[i]);
  }
  while (left > 0) {  // the last rows, fewer than two groups
    Four<T> in[N];
#pragma unroll
    for (int i = 0; i < N; ++i) in[i] = next[i];
    fetch(left - N);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < left) one(in[i]);
    left -= N;
  }
}

template <typename T, int W>
__global__ void __launch_bounds__(kThreads, kResident<T>) conv_kernel(ConvArgs p, int channel_blocks, int tile) {
  const int unit = blockIdx.x / channel_blocks, block = blockIdx.x % channel_blocks;
  int32_t* status = blockIdx.x == 0 ? p.status : nullptr;
  const gdn_requests& req = p.req;
  // a request has a unit for every `tile` rows, one at least: that of its state
  const Unit u = find_unit<kThreads>(
      req.num_seqs, unit,
      [&](int n) {
        const Request q = load_request(req, n, status);
        return q.len < 0 ? 0 : max(1, (q.len + tile - 1) / tile);
      },
      [](int) { return 0; });
  if (u.seq < 0) return;
  const Request q = load_request(req, u.seq, nullptr);
  const int channels = p.cfg.channels;
  const Channels k = my_channels(block, channels);
  if (k.count <= 0) return;
  const T* x = static_cast<const T*>(p.x) + (size_t)q.lo * p.x_stride + k.c0;
  T* y = static_cast<T*>(p.y) + (size_t)q.lo * p.y_stride + k.c0;
  T* state = static_cast<T*>(p.pool) + (size_t)q.slot * (W - 1) * channels + k.c0;
  const int t0 = u.place * tile, t1 = min(q.len, t0 + tile);

  f32x2 rows[W - 1][2];
  if (t0 == 0) {
    Four<T> old[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      old[j].clear();
      if (!q.zero) old[j].load(state + (size_t)j * channels, k.count, k.whole_state);
      old[j].values(rows[j]);
    }
    // the last W - 1 inputs of the first `len` ones: rows of x, or of the old state
    auto save = [&](T* to, int len) {
#pragma unroll
      for (int j = 0; j < W - 1; ++j) {
        Four<T> v = old[W - 2];
        const int at = len - (W - 1) + j;
        if (at >= 0) {
          v.load(x + (size_t)at * p.x_stride, k.count, k.whole);
        } else {
#pragma unroll
          for (int i = 0; i < W - 1; ++i)
            if (W - 1 + at == i) v = old[i];
        }
        v.store(to + (size_t)j * channels, k.count, k.whole_state);
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
    for (int j = 0; j < W - 1; ++j) {
      Four<T> v;
      v.load(x + (size_t)(t0 - (W - 1) + j) * p.x_stride, k.count, k.whole);
      v.values(rows[j]);
    }
  }

  const Taps<W> taps(p.cfg, k.c0, k.count);
  x += (size_t)t0 * p.x_stride;
  y += (size_t)t0 * p.y_stride;
  const int left = t1 - t0;
  if (!k.whole) walk<T, W, false>(taps, rows, x, y, p, left, k.count, p.cfg.activation == GDN_ACT_SILU);
  else if (p.cfg.activation == GDN_ACT_SILU) walk<T, W, true>(taps, rows, x, y, p, left, 4, true);
  else walk<T, W, true>(taps, rows, x, y, p, left, 4, false);
}

// One token of a request: the state's rows move up by one.
template <typename T, int W>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(ConvArgs p, int channel_blocks) {
  const int b = blockIdx.x / channel_blocks;
  const int channels = p.cfg.channels;
  const Channels k = my_channels(blockIdx.x % channel_blocks, channels);
  if (k.count <= 0) return;
  const int slot = p.req.slot_idx[b];
  if (slot < 0 || slot >= p.req.num_slots) {
    if (slot >= 0) raise_status(p.status, GDN_ERR_INVALID_ARGUMENT);
    return;
  }
  T* state = static_cast<T*>(p.pool) + (size_t)slot * (W - 1) * channels + k.c0;
  Four<T> old[W];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) old[j].load(state + (size_t)j * channels, k.count, k.whole_state);
  old[W - 1].load(static_cast<const T*>(p.x) + (size_t)b * p.x_stride + k.c0, k.count, k.whole);
  const Taps<W> taps(p.cfg, k.c0, k.count);
  f32x2 rows[W][2], out[2];
#pragma unroll
  for (int j = 0; j < W; ++j) old[j].values(rows[j]);
  taps.apply(rows, rows[W - 1], p.cfg.activation == GDN_ACT_SILU, out);
#pragma unroll
  for (int j = 0; j < W - 1; ++j)
    old[j + 1].store(state + (size_t)j * channels, k.count, k.whole_state);
  Four<T>(out).store(static_cast<T*>(p.y) + (size_t)b * p.y_stride + k.c0, k.count, k.whole);
}

int channel_blocks(int channels) { return (channels + kThreads * 4 - 1) / (kThreads * 4); }

// Rows of a block: a start costs about as much as eight rows, and the last blocks run as long as all
// others. 32 x 1,024 rows of 8,192 channels, bf16: 212 us with blocks of 32 rows, 177 with 512 (all
// run at once); 4 x 1,024 rows of 2,048: 19 and 72.
template <typename T>
int tile_of(int64_t tokens, int cb) {
  constexpr int64_t kPlaces = 152 * kResident<T>;
  int best = 0;
  int64_t least = 0;
  for (int tile = 32; tile <= 512; tile *= 2) {
    const int64_t blocks = (tokens + tile - 1) / tile * cb;
    const int64_t cost = (blocks + kPlaces - 1) / kPlaces * (tile + 8);
    if (best == 0 || cost <= least) {
      best = tile;
      least = cost;
    }
  }
  return best;
}

template <typename T, int W>
int launch_packed(const ConvArgs& a, cudaStream_t s) {
  const int cb = channel_blocks(a.cfg.channels);
  const int tile = tile_of<T>(a.req.num_tokens, cb);
  const int64_t units = (int64_t)a.req.num_tokens / tile + a.req.num_seqs;
  conv_kernel<T, W><<<(unsigned)(units * cb), kThreads, 0, s>>>(a, cb, tile);
  return (int)cudaGetLastError();
}
template <typename T, int W>
int launch_single(const ConvArgs& a, cudaStream_t s) {
  const int cb = channel_blocks(a.cfg.channels);
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
