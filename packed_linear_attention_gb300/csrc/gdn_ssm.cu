// gdn_ssm.cu — the selective scan, for packs of requests and for single tokens.
//
//     dt = softplus(delta + bias)
//     h[n] = exp(dt a[n]) h[n] + dt x b[n]          (fp32, N states a channel)
//     y = (sum_n c[n] h[n] + d x) silu(z)
//
// Channels are independent and their states short, so a thread owns a channel (or SPLIT lanes
// share one, NS states each), keeps its states and decay rates in registers and walks down the
// rows. exp is one multiplication (the rates are held times log2 e) and one ex2; the rest are fused
// multiply-adds on pairs of states (f32x2).
//
// A block takes kCh channels of one request, kTile rows at a time, in two turns. In the first its
// threads share out the tile 8 elements each, 16-byte accesses side by side: dt and dt x go to shared
// memory, and what the last tile's scan left there is gated and stored; b and c, the same for all
// channels of a group, are widened to fp32. In the second every thread scans its channel from shared
// memory, at offsets known when compiled: what it costs is its 16 states, not their addresses.
#include <algorithm>
#include <climits>

#include "gdn_step_internal.h"

namespace gdn {
namespace {

constexpr int kThreads = 128;

// exp of dt times a rate (held times log2 e). Just below 0 the ex2 instruction errs low by 2e-8 on
// average, which slow decays would sum up; 3e-8 in its argument leaves 5e-9 (and 2^0 at 1).
constexpr float kNudge = 3e-8f;
__device__ __forceinline__ f32x2 decay(f32x2 dt, f32x2 a) {
  return ex2(fma2(dt, a, pair(kNudge, kNudge)));
}
// log(1 + exp(x)) = max(x, 0) + log1p(e), e = exp(-|x|) in (0, 1]. log1p(e) is e times a polynomial
// fitted to log1p(e) / e (least squares, reweighted towards an even relative error, 3e-8).
__device__ constexpr float kLog1p[9] = {0.99999994f,  -0.49999493f, 0.33319095f,   -0.24842976f, 0.1910598f,
                             -0.13663195f, 0.07822535f,  -0.029504869f, 0.0052326024f};
// exp(-|x|) = 2^y exp(r): y = -|x| log2 e as rounded (at |x| = 30 that is off by 2^-19, and so would be
// the result) and r = -|x| - y ln 2, what the rounding left, where exp(r) is 1 + r. So small results keep
// their relative precision, 2^-20, down to 2^-126. |x| is held at 127, past which 2^y is 0 anyway, for
// infinities to leave no NaN; a NaN stays.
constexpr float kLn2 = 0.6931471805599453f;
// -|x|, held at -127
__device__ __forceinline__ float minus_abs(float x) {
  float a;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(a) : "f"(fabsf(x)), "f"(127.f));
  return -a;
}
__device__ __forceinline__ f32x2 softplus(f32x2 x) {
  float x0, x1;
  unpair(x, x0, x1);
  const f32x2 a = pair(minus_abs(x0), minus_abs(x1)), y = mul2(a, both(kLog2e));
  f32x2 e = ex2(y);
  e = fma2(e, fma2(y, both(-kLn2), a), e);
  f32x2 p = both(kLog1p[8]);
#pragma unroll
  for (int i = 7; i >= 0; --i) p = fma2(e, p, both(kLog1p[i]));
  return fma2(e, p, pair(fmaxf(x0, 0.f), fmaxf(x1, 0.f)));
}
__device__ __forceinline__ float softplus(float x) {
  const float a = minus_abs(x), y = a * kLog2e;
  float e = ex2(y);
  e = fmaf(e, fmaf(y, -kLn2, a), e);
  float p = kLog1p[8];
#pragma unroll
  for (int i = 7; i >= 0; --i) p = fmaf(e, p, kLog1p[i]);
  return fmaf(e, p, fmaxf(x, 0.f));
}

// The states of one thread: NS of channel c, chunks of four that the SPLIT lanes take in turn
// (so that the lanes' reads of b and c in shared memory lie side by side).
template <int NS, int SPLIT>
struct States {
  f32x2 h[NS / 2], a[NS / 2];

  __device__ __forceinline__ static int chunk(int i, int part) { return 4 * (i * SPLIT + part); }

  __device__ __forceinline__ void rates(const float* a_row, int part, int n) {
#pragma unroll
    for (int i = 0; i < NS / 4; ++i) {
      float f[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int at = chunk(i, part) + e;
        f[e] = at < n ? kLog2e * __ldg(a_row + at) : 0.f;
      }
      a[2 * i] = pair(f[0], f[1]);
      a[2 * i + 1] = pair(f[2], f[3]);
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < NS / 2; ++i) h[i] = 0;
  }
  // row: N floats; 16-byte accesses where N is a multiple of 4
  __device__ __forceinline__ void load(const float* row, int part, int n) {
#pragma unroll
    for (int i = 0; i < NS / 4; ++i) {
      const int at = chunk(i, part);
      float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
      if (n % 4 == 0) {
        if (at < n) f = *reinterpret_cast<const float4*>(row + at);
      } else {
        if (at < n) f.x = row[at];
        if (at + 1 < n) f.y = row[at + 1];
        if (at + 2 < n) f.z = row[at + 2];
        if (at + 3 < n) f.w = row[at + 3];
      }
      h[2 * i] = pair(f.x, f.y);
      h[2 * i + 1] = pair(f.z, f.w);
    }
  }
  __device__ __forceinline__ void store(float* row, int part, int n) const {
#pragma unroll
    for (int i = 0; i < NS / 4; ++i) {
      const int at = chunk(i, part);
      float4 f;
      unpair(h[2 * i], f.x, f.y);
      unpair(h[2 * i + 1], f.z, f.w);
      if (n % 4 == 0) {
        if (at < n) *reinterpret_cast<float4*>(row + at) = f;
      } else {
        if (at < n) row[at] = f.x;
        if (at + 1 < n) row[at + 1] = f.y;
        if (at + 2 < n) row[at + 2] = f.z;
        if (at + 3 < n) row[at + 3] = f.w;
      }
    }
  }
  // one row; b and c: the padded row in shared memory. Returns this thread's part of c . h. Even and odd
  // chunks are added up apart: a thread with 16 states has two sums that are those of two lanes with 8
  // each. Which of the two shapes a call takes goes by the requests around a request, whose bits shall not.
  template <bool OUT>
  __device__ __forceinline__ float step(float dt, float dtx, const float* b, const float* c,
                                        int part) {
    constexpr int kSums = NS == 4 || (NS == 8 && SPLIT == 2) ? 1 : 2;
    const f32x2 t = pair(dt, dt), u = pair(dtx, dtx);
    f32x2 acc[kSums] = {};
#pragma unroll
    for (int i = 0; i < NS / 4; ++i) {
      const ulonglong2 bv = *reinterpret_cast<const ulonglong2*>(b + chunk(i, part));
      h[2 * i] = fma2(decay(t, a[2 * i]), h[2 * i], mul2(u, bv.x));
      h[2 * i + 1] = fma2(decay(t, a[2 * i + 1]), h[2 * i + 1], mul2(u, bv.y));
      if (OUT) {
        const ulonglong2 cv = *reinterpret_cast<const ulonglong2*>(c + chunk(i, part));
        f32x2& s = acc[i % kSums];
        s = i < kSums ? mul2(cv.x, h[2 * i]) : fma2(cv.x, h[2 * i], s);
        s = fma2(cv.y, h[2 * i + 1], s);
      }
    }
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < kSums; ++k) {
      float lo, hi;
      unpair(acc[k], lo, hi);
      sum = k == 0 ? lo + hi : sum + (lo + hi);
    }
    return sum;
  }
};

// What a block scans: rows [lo, lo + len) of request `seq` from `state`.
struct Span {
  int32_t seq, lo, len, first;  // first: rows of the request in front of them
};

template <typename T, int NS, int SPLIT>
struct Scan {
  static constexpr int kPadded = NS * SPLIT;
  static constexpr int kCh = kThreads / SPLIT;
  static constexpr int kTile = 16;
  static constexpr int kAcross = kCh / 8, kStep = kThreads / kAcross;  // shares of a row; rows between a thread's
  static constexpr int kShares = (kTile + kStep - 1) / kStep;          // of a thread
  static constexpr int kVecs = 8 / Vec<T>::N;
  static constexpr int kShare = (kTile * kPadded + kThreads - 1) / kThreads;  // of b and of c
  struct Shared {
    float4 f[kTile][kCh / 2];  // dt and dt x of two channels, at pair_at
    float4 y[kTile][kCh / 4];  // at quad_at
    float b[kTile][kPadded], c[kTile][kPadded];
    float4 bias[kCh / 4], skip[kCh / 4];  // at quad_at
    uint4 x[kShares][kVecs][kThreads], z[kShares][kVecs][kThreads];  // of the rows being scanned
  };
  // Where 16 bytes of a row lie, so that neither the 8 channels of a thread's share nor the channels
  // of a warp's lanes meet in a bank: chunk q of pairs, chunk q of fours.
  __device__ __forceinline__ static int pair_at(int q) { return q ^ ((q >> 3) & 3); }
  __device__ __forceinline__ static int quad_at(int q) { return q ^ ((q >> 3) & 1); }

  struct Eight {
    Vec<T> v[kVecs];
    __device__ __forceinline__ void load(const T* p, int count, bool whole) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
        v[i] = load_vec(p + i * Vec<T>::N, count - i * Vec<T>::N, whole);
    }
    __device__ __forceinline__ void values(float* f) const {
#pragma unroll
      for (int i = 0; i < kVecs; ++i) unpack(v[i], f + i * Vec<T>::N);
    }
  };

  const SsmArgs& p;
  Shared& sm;
  int group, channel, part, local;
  int my_f, my_y;  // this thread's channel in a row of f and of y
  bool live;
  // this thread's share of a tile: 8 channels of a row
  int task_row, task_col, task_channel, count;
  bool whole;
  States<NS, SPLIT> s;
  float total = 0.f;

  __device__ __forceinline__ Scan(const SsmArgs& args, Shared& shared, int block)
      : p(args), sm(shared) {
    const int per = p.cfg.channels / p.cfg.num_groups;
    const int tiles = (per + kCh - 1) / kCh;
    group = block / tiles;
    const int first = block % tiles * kCh;  // of the group
    local = threadIdx.x / SPLIT;
    part = threadIdx.x % SPLIT;
    live = first + local < per;
    channel = group * per + min(first + local, per - 1);
    task_row = threadIdx.x / kAcross;
    task_col = threadIdx.x % kAcross * 8;
    task_channel = group * per + first + task_col;
    count = max(0, min(8, per - first - task_col));
    whole = count == 8 && (p.cfg.num_groups == 1 || per % Vec<T>::N == 0);
    s.rates(p.cfg.a + (size_t)channel * p.cfg.state_dim, part, p.cfg.state_dim);
    my_f = 2 * pair_at(local / 2) + local % 2;
    my_y = 4 * quad_at(local / 4) + local % 4;
    if (part == 0) {
      reinterpret_cast<float*>(sm.bias)[my_y] = p.cfg.delta_bias ? __ldg(p.cfg.delta_bias + channel) : 0.f;
      reinterpret_cast<float*>(sm.skip)[my_y] = p.cfg.d ? __ldg(p.cfg.d + channel) : 0.f;
    }
  }

  __device__ __forceinline__ size_t state_row(int64_t slot) const {
    return ((size_t)slot * p.cfg.channels + channel) * p.cfg.state_dim;
  }

  // b and c of rows [row, row + kTile) on their way to a buffer; zeros past the states and the rows
  struct Shares {
    T b[kShare], c[kShare];
  };
  __device__ __forceinline__ void load_bc(Shares& w, int64_t row, int rows) {
    const int n = p.cfg.state_dim;
    const T* b = static_cast<const T*>(p.rows.b) + row * p.rows.b_stride + (size_t)group * n;
    const T* c = static_cast<const T*>(p.rows.c) + row * p.rows.c_stride + (size_t)group * n;
#pragma unroll
    for (int i = 0; i < kShare; ++i) {
      const int at = i * kThreads + threadIdx.x, t = at / kPadded, k = at % kPadded;
      const bool in = t < rows && k < n;
      w.b[i] = in ? b[(size_t)t * p.rows.b_stride + k] : from_f32<T>(0.f);
      w.c[i] = in ? c[(size_t)t * p.rows.c_stride + k] : from_f32<T>(0.f);
    }
  }
  __device__ __forceinline__ void store_bc(const Shares& w) {
#pragma unroll
    for (int i = 0; i < kShare; ++i) {
      const int at = i * kThreads + threadIdx.x;
      if (kTile * kPadded % kThreads == 0 || at < kTile * kPadded) {
        (&sm.b[0][0])[at] = to_f32(w.b[i]);
        (&sm.c[0][0])[at] = to_f32(w.c[i]);
      }
    }
  }

  // The rows of `span`, from the states in s. OUT: y and the checkpoints; else the sum of dt.
  template <bool OUT>
  __device__ __forceinline__ void run(const Span& span, bool report) {
    const int len = span.len;
    const bool gated = OUT && p.rows.z;
    // the first checkpoint past the rows in front (rows counted from span.lo from here on)
    int2 ck = make_int2(0, 0);
    int mark = INT_MAX, before = 0;
    auto next_mark = [&] {
      mark = INT_MAX;
      for (; ck.x < ck.y; ++ck.x) {
        const int pos = p.req.ckpt_pos[ck.x];
        if (pos <= before || pos > p.req.cu[span.seq + 1] - p.req.cu[span.seq]) {
          if (report) raise_status(p.status, GDN_ERR_INVALID_ARGUMENT);
          continue;
        }
        before = pos;
        if (pos > span.first) {
          mark = pos - span.first;
          return;
        }
      }
    };
    if (OUT) {
      ck = load_checkpoints(p.req, span.seq, report ? p.status : nullptr);
      next_mark();
    }

    // Addresses are worked out anew for each tile: registers are what is short while it is scanned.
    auto row_of = [&](const void* base, int64_t stride, int t) {
      int row = task_row;
      asm volatile("" : "+r"(row));
      return static_cast<const T*>(base) + (int64_t)(span.lo + t + row) * stride + task_channel;
    };
    // whether this thread has share i of the tile at t0
    auto mine = [&](int i, int t0) {
      return count > 0 && task_row + i * kStep < kTile && t0 + task_row + i * kStep < len;
    };
    Eight xn[kShares], dn[kShares], zn[kShares];  // the next tile's rows
    auto fetch = [&](int t0) {
#pragma unroll
      for (int i = 0; i < kShares; ++i) {
        if (mine(i, t0)) {
          xn[i].load(row_of(p.rows.x, p.rows.x_stride, t0 + i * kStep), count, whole);
          dn[i].load(row_of(p.rows.delta, p.rows.delta_stride, t0 + i * kStep), count, whole);
          if (gated) zn[i].load(row_of(p.rows.z, p.rows.z_stride, t0 + i * kStep), count, whole);
        }
      }
    };
    // this thread's 8 channels in a row of fours, as pairs
    auto quads = [&](const float4* row, f32x2* f) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(&row[quad_at(task_col / 4 + i)]);
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
      }
    };
    // dt and dt x of this thread's share
    auto prepare = [&](int s) {
      float xf[8], df[8];
      f32x2 bias[4];
      xn[s].values(xf);
      dn[s].values(df);
      quads(sm.bias, bias);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f32x2 dt = add2(pair(df[2 * i], df[2 * i + 1]), bias[i]);
        if (p.cfg.delta_softplus) dt = softplus(dt);
        float4 f;
        unpair(dt, f.x, f.z);
        unpair(mul2(dt, pair(xf[2 * i], xf[2 * i + 1])), f.y, f.w);
        sm.f[task_row + s * kStep][pair_at(task_col / 2 + i)] = f;
      }
      if (OUT) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
          sm.x[s][i][threadIdx.x] = xn[s].v[i].raw;
          if (gated) sm.z[s][i][threadIdx.x] = zn[s].v[i].raw;
        }
      }
    };
    auto finish = [&](int t0, int s) {
      if (!mine(s, t0)) return;
      float f[8], out[8];
      f32x2 skip[4], sum[4];
      Eight h;
#pragma unroll
      for (int i = 0; i < kVecs; ++i) h.v[i].raw = sm.x[s][i][threadIdx.x];
      h.values(f);
      quads(sm.skip, skip);
      quads(sm.y[task_row + s * kStep], sum);
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[i] = fma2(skip[i], pair(f[2 * i], f[2 * i + 1]), sum[i]);
      if (gated) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) h.v[i].raw = sm.z[s][i][threadIdx.x];
        h.values(f);
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] = mul2(sum[i], silu(pair(f[2 * i], f[2 * i + 1])));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) unpair(sum[i], out[2 * i], out[2 * i + 1]);
      T* y = const_cast<T*>(row_of(p.rows.y, p.rows.y_stride, t0 + s * kStep));
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
        store_vec(y + i * Vec<T>::N, pack<T>(out + i * Vec<T>::N), count - i * Vec<T>::N, whole);
    };
    auto one = [&](int r) {
      const float2 f = reinterpret_cast<const float2*>(sm.f[r])[my_f];
      if (!OUT) total += f.x;
      float sum = s.template step<OUT>(f.x, f.y, sm.b[r], sm.c[r], part);
      if (OUT) {
#pragma unroll
        for (int off = SPLIT / 2; off > 0; off >>= 1)
          sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (part == 0) reinterpret_cast<float*>(sm.y[r])[my_y] = sum;
      }
    };

    Shares w;  // the next tile's b and c
    load_bc(w, span.lo, min(len, kTile));
    fetch(0);
    __syncthreads();  // bias and skip
    for (int t0 = 0; t0 < len; t0 += kTile) {
      const bool more = t0 + kTile < len;
#pragma unroll
      for (int i = 0; i < kShares; ++i) {
        if (OUT && t0 > 0) finish(t0 - kTile, i);
        if (mine(i, t0)) prepare(i);
      }
      store_bc(w);
      if (more) {
        fetch(t0 + kTile);
        load_bc(w, span.lo + t0 + kTile, min(len - t0 - kTile, kTile));
      }
      __syncthreads();
      const int rows = min(len - t0, kTile);
      if (rows == kTile && (!OUT || mark > t0 + kTile)) {
#pragma unroll 8
        for (int r = 0; r < kTile; ++r) one(r);
      } else {
        for (int r = 0; r < rows; ++r) {
          one(r);
          if (OUT && mark == t0 + r + 1) {
            if (live) s.store(p.ckpt + state_row(ck.x), part, p.cfg.state_dim);
            ++ck.x;
            next_mark();
          }
        }
      }
      __syncthreads();
    }
    if (OUT && len > 0) {
#pragma unroll
      for (int i = 0; i < kShares; ++i) finish((len - 1) / kTile * kTile, i);
    }
  }
};

// Blocks of an SM: 128 registers a thread hold 16 states, their rates and the next rows without
// spilling. At 96 (five blocks) a wave of 32 x 1,024 x 4,096 channels takes 648 us against 620; fp32
// rows and wide shares of b and c want more.
template <typename T, int SPLIT>
constexpr int kResident = sizeof(T) == 2 && SPLIT < 4 ? 4 : 3;

// pass 0: whole requests, a unit each. With requests cut into segments, pass 1 runs every
// request's first segment and finds the end states of its middle ones from zeros; pass 2 joins
// them and runs the segments behind the first. exp(a dt_1) ... exp(a dt_k) is exp(a sum dt), so a
// segment's decay needs only its sum of dt.
template <typename T, int NS, int SPLIT>
__global__ void __launch_bounds__(kThreads, kResident<T, SPLIT>) ssm_kernel(SsmArgs p, int channel_blocks, int pass) {
  using S = Scan<T, NS, SPLIT>;
  __shared__ __align__(16) typename S::Shared sm;
  const int unit = blockIdx.x / channel_blocks;
  int32_t* status = blockIdx.x == 0 && pass < 2 ? p.status : nullptr;
  const int seg = p.segment;
  Unit u = {unit, 0, 0};
  if (pass > 0) {
    const auto behind = [&](int n) {  // segments behind the first
      const Request q = load_request(p.req, n, nullptr);
      return q.len <= 0 ? 0 : (q.len - 1) / seg;
    };
    u = find_unit<kThreads>(
        p.req.num_seqs, unit,
        [&](int n) {
          const Request q = load_request(p.req, n, status);
          if (q.len < 0) return 0;
          const int k = q.len == 0 ? 0 : (q.len - 1) / seg;
          return pass == 1 ? max(1, k) : k;
        },
        behind);
    if (u.seq < 0) return;
  } else {
    status = blockIdx.x % channel_blocks == 0 && threadIdx.x == 0 ? p.status : nullptr;
  }
  const Request q = load_request(p.req, u.seq, pass == 0 ? status : nullptr);
  if (q.len < 0) return;
  const int later = seg && q.len > 0 ? (q.len - 1) / seg : 0;
  const int k = pass == 2 ? u.place + 1 : u.place;  // this block's segment
  if (later > 0 && u.extra + later > p.units) {  // only where requests overlap
    if (threadIdx.x == 0) raise_status(p.status, GDN_ERR_INVALID_ARGUMENT);
    return;
  }
  S scan(p, sm, blockIdx.x % channel_blocks);
  const int n = p.cfg.state_dim;
  const Span span = {u.seq, q.lo + k * seg, seg ? min(q.len - k * seg, seg) : q.len, k * seg};
  const size_t ends = (size_t)u.extra;  // the request's first end state
  scan.s.clear();
  if (k == 0) {
    if (!q.zero) scan.s.load(p.pool + scan.state_row(q.slot), scan.part, n);
  } else if (pass == 2) {
    scan.s.load(p.ends + scan.state_row(ends), scan.part, n);
    for (int j = 1; j < k; ++j) {
      States<NS, SPLIT> end;
      end.load(p.ends + scan.state_row(ends + j), scan.part, n);
      const float dt = p.steps[(ends + j) * p.cfg.channels + scan.channel];
#pragma unroll
      for (int i = 0; i < NS / 2; ++i)
        scan.s.h[i] = fma2(decay(pair(dt, dt), scan.s.a[i]), scan.s.h[i], end.h[i]);
    }
  }
  const bool report = blockIdx.x % channel_blocks == 0 && threadIdx.x == 0;
  if (pass == 1 && k > 0) {
    scan.template run<false>(span, false);
    if (scan.live && scan.part == 0)
      p.steps[(ends + k) * p.cfg.channels + scan.channel] = scan.total;
  } else {
    scan.template run<true>(span, report);
  }
  if (!scan.live) return;
  if (k == later) scan.s.store(p.pool + scan.state_row(q.slot), scan.part, n);
  else if (pass == 1) scan.s.store(p.ends + scan.state_row(ends + k), scan.part, n);
}

// One token: LANES lanes a channel, eight states each (32 bytes, a sector of memory), so that a state
// goes through as accesses side by side while a channel's own work (softplus, gate, addresses) is
// repeated by as few lanes as that allows. Bound by HBM (the states, in and out).
template <typename T>
__device__ __forceinline__ void load_eight(const T* p, int count, bool aligned, f32x2* f) {
  float x[8];
  if (aligned && count >= 8) {
#pragma unroll
    for (int i = 0; i < 8 / Vec<T>::N; ++i)
      unpack(Vec<T>{reinterpret_cast<const uint4*>(p)[i]}, x + i * Vec<T>::N);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = i < count ? to_f32(p[i]) : 0.f;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = pair(x[2 * i], x[2 * i + 1]);
}

// Everything but the state is read before the slot is looked at. (Two rows a thread, their loads on the
// way together: 20.5 us for 128 rows of 4,096 channels and 16 states against 18.4; nine blocks an SM,
// at the 54 registers that it would take: 19.9.)
template <typename T, int LANES>
__global__ void __launch_bounds__(kThreads, 10) ssm_step_kernel(SsmArgs p, bool aligned) {
  const int64_t row = blockIdx.x;
  const int c = blockIdx.y * (kThreads / LANES) + (int)threadIdx.x / LANES;
  const int n0 = threadIdx.x % LANES * 8, n = p.cfg.state_dim;
  const bool live = c < p.cfg.channels;
  const int ch = min(c, p.cfg.channels - 1), count = n - n0;
  const int group = p.cfg.num_groups == 1 ? 0 : ch / (p.cfg.channels / p.cfg.num_groups);
  const bool whole = n % 8 == 0;
  const int slot = p.req.slot_idx[row];
  f32x2 a[4], b[4], cc[4], h[4];
  const float x = to_f32(static_cast<const T*>(p.rows.x)[row * p.rows.x_stride + ch]);
  float dt = to_f32(static_cast<const T*>(p.rows.delta)[row * p.rows.delta_stride + ch]);
  const float z = p.rows.z ? to_f32(static_cast<const T*>(p.rows.z)[row * p.rows.z_stride + ch]) : 0.f;
  load_eight(static_cast<const T*>(p.rows.b) + row * p.rows.b_stride + group * n + n0, count, aligned, b);
  load_eight(static_cast<const T*>(p.rows.c) + row * p.rows.c_stride + group * n + n0, count, aligned, cc);
  load_eight(p.cfg.a + (size_t)ch * n + n0, count, whole, a);
  const float bias = p.cfg.delta_bias ? __ldg(p.cfg.delta_bias + ch) : 0.f;
  const float skip = p.cfg.d ? __ldg(p.cfg.d + ch) : 0.f;
  if (slot < 0 || slot >= p.req.num_slots) {
    if (slot >= 0 && blockIdx.y == 0 && threadIdx.x == 0) raise_status(p.status, GDN_ERR_INVALID_ARGUMENT);
    return;
  }
  float* state = p.pool + ((size_t)slot * p.cfg.channels + ch) * n + n0;
  load_eight(state, count, whole, h);
  dt += bias;
  if (p.cfg.delta_softplus) dt = softplus(dt);
  const f32x2 t = both(kLog2e * dt), u = both(dt * x);
  f32x2 acc = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = fma2(decay(t, a[i]), h[i], mul2(u, b[i]));
    acc = i == 0 ? mul2(cc[i], h[i]) : fma2(cc[i], h[i], acc);
  }
  float sum, hi;
  unpair(acc, sum, hi);
  sum += hi;
#pragma unroll
  for (int off = LANES / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if (!live) return;
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) unpair(h[i], f[2 * i], f[2 * i + 1]);
  if (whole) {
    if (count >= 8) {
      reinterpret_cast<float4*>(state)[0] = make_float4(f[0], f[1], f[2], f[3]);
      reinterpret_cast<float4*>(state)[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < count) state[i] = f[i];
  }
  if (n0 == 0) {
    if (p.cfg.d) sum = fmaf(skip, x, sum);
    if (p.rows.z) sum *= silu(z);
    static_cast<T*>(p.rows.y)[row * p.rows.y_stride + ch] = from_f32<T>(sum);
  }
}

// States of a thread and lanes of a channel. 16 states a thread cost the least in all; 8 are done
// sooner where the GPU's 608 schedulers have less than four warps each (a prompt of 4,096 rows and
// 4,096 channels: 542 against 704 us; a wave, which has seven: 710 against 620).
struct Shape {
  int ns, split;
};
constexpr int64_t kSchedulers = 608;
Shape shape_of(int n) {
  if (n <= 4) return {4, 1};
  if (n <= 8) return {8, 1};
  int split = 1;
  while (16 * split < n) split *= 2;
  return {16, split};
}
// Warps of a request's channels.
int64_t channel_warps(const gdn_ssm_config& cfg) {
  return ((int64_t)cfg.channels * shape_of(cfg.state_dim).split + 31) / 32;
}
// Rows that the requests may have in all.
int64_t rows_of(const gdn_requests& req) {
  return std::min<int64_t>(req.num_tokens, (int64_t)req.num_seqs * req.max_len);
}
// Warps that run side by side: those of a request's channels, times the requests that the rows
// make up at their longest.
int64_t warps_of(const gdn_ssm_config& cfg, const gdn_requests& req) {
  return channel_warps(cfg) * std::max<int64_t>(1, rows_of(req) / std::max(1, req.max_len));
}

template <typename T, int NS, int SPLIT>
int launch_scan(const SsmArgs& a, cudaStream_t s) {
  const int per = a.cfg.channels / a.cfg.num_groups, ch = kThreads / SPLIT;
  const int cb = a.cfg.num_groups * ((per + ch - 1) / ch);
  if (a.segment == 0) {
    ssm_kernel<T, NS, SPLIT><<<(unsigned)((int64_t)a.req.num_seqs * cb), kThreads, 0, s>>>(a, cb, 0);
    return (int)cudaGetLastError();
  }
  // disjoint requests: at most a segment more than their whole ones each
  ssm_kernel<T, NS, SPLIT>
      <<<(unsigned)(((int64_t)a.units + a.req.num_seqs) * cb), kThreads, 0, s>>>(a, cb, 1);
  if (a.units > 0)
    ssm_kernel<T, NS, SPLIT><<<(unsigned)((int64_t)a.units * cb), kThreads, 0, s>>>(a, cb, 2);
  return (int)cudaGetLastError();
}

template <typename T>
int scan_by_shape(const SsmArgs& a, cudaStream_t s) {
  const Shape k = shape_of(a.cfg.state_dim);
  if (k.ns == 4) return launch_scan<T, 4, 1>(a, s);
  if (k.ns == 8) return launch_scan<T, 8, 1>(a, s);
  const int64_t pieces = a.segment ? ((int64_t)a.req.max_len + a.segment - 1) / a.segment : 1;
  if (k.split == 1 && warps_of(a.cfg, a.req) * pieces < 4 * kSchedulers)
    return launch_scan<T, 8, 2>(a, s);
  switch (k.split) {
    case 1: return launch_scan<T, 16, 1>(a, s);
    case 2: return launch_scan<T, 16, 2>(a, s);
    case 4: return launch_scan<T, 16, 4>(a, s);
    case 8: return launch_scan<T, 16, 8>(a, s);
  }
  return (int)cudaErrorInvalidValue;
}

template <typename T, int LANES>
int launch_one(const SsmArgs& a, cudaStream_t s) {
  constexpr int ch = kThreads / LANES;
  const auto at = [](const void* p, int64_t stride) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % (int64_t)(16 / sizeof(T)) == 0;
  };
  const bool aligned = at(a.rows.b, a.rows.b_stride) && at(a.rows.c, a.rows.c_stride) &&
                       a.cfg.state_dim % 8 == 0;
  const dim3 grid((unsigned)a.req.num_tokens, (unsigned)((a.cfg.channels + ch - 1) / ch));
  ssm_step_kernel<T, LANES><<<grid, kThreads, 0, s>>>(a, aligned);
  return (int)cudaGetLastError();
}
template <typename T>
int step_by_lanes(const SsmArgs& a, cudaStream_t s) {
  const int n = a.cfg.state_dim;
  if (n <= 8) return launch_one<T, 1>(a, s);
  if (n <= 16) return launch_one<T, 2>(a, s);
  if (n <= 32) return launch_one<T, 4>(a, s);
  if (n <= 64) return launch_one<T, 8>(a, s);
  return launch_one<T, 16>(a, s);
}

}  // namespace

// Cutting does the exponentials of most rows twice, so it pays where the schedulers have less than
// three quarters of a warp each: 32,768 rows of 2,048 channels take 3,620 us whole and 540 in 57
// pieces, four requests of 4,096 rows and 4,096 channels 542 and 550. Shorter pieces than 64 rows
// spend more on their starts than they win (a prompt of 100 rows: 17 us whole, 21 in four).
constexpr int64_t kFew = kSchedulers * 3 / 4, kWanted = 6 * kSchedulers, kLeast = 64, kMost = 64;
int32_t ssm_segment(const gdn_ssm_config& cfg, const gdn_requests& req) {
  const int64_t warps = warps_of(cfg, req);
  if (req.max_len < 1 || warps > kFew) return 0;
  const int64_t pieces = std::min<int64_t>(kMost, kWanted / warps);
  const int64_t seg = std::max<int64_t>(kLeast, ((int64_t)req.max_len + pieces - 1) / pieces + 31) / 32 * 32;
  return req.max_len >= 2 * seg ? (int32_t)seg : 0;
}

int64_t ssm_units(const gdn_requests& req, int32_t segment) { return segment ? rows_of(req) / segment : 0; }

// Fewer requests or shorter ones may be cut where the largest call is not. A segment has kLeast rows at
// least, and max_len / pieces. With R = rows / max_len requests side by side pieces are kWanted /
// (channel warps * R rounded down, 1 at least), so that rows / segment is below twice kWanted over the
// channel warps.
int64_t ssm_most_units(const gdn_ssm_config& cfg, const gdn_requests& req) {
  const int64_t warps = channel_warps(cfg);
  if (warps > kFew || req.max_len < 2 * kLeast) return 0;
  return std::min<int64_t>(rows_of(req) / kLeast, 2 * kWanted / warps);
}

int launch_ssm_packed(const SsmArgs& a, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return a.cfg.io_dtype == GDN_BF16 ? scan_by_shape<__nv_bfloat16>(a, s) : scan_by_shape<float>(a, s);
}

int launch_ssm_step(const SsmArgs& a, void* stream) {
  if (a.req.num_tokens == 0) return 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return a.cfg.io_dtype == GDN_BF16 ? step_by_lanes<__nv_bfloat16>(a, s) : step_by_lanes<float>(a, s);
}

}  // namespace gdn
