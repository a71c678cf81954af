// gdn_kv_plan.cu — the step plan of the paged cache: pages, slots and positions of a step's
// tokens from the requests' lengths, and the return of ended requests' pages.
//
// A request with c cached and n new tokens owns ceil(c / P) pages of P tokens and needs
// ceil((c + n) / P) - ceil(c / P) more. With the exclusive sums of the needs, page number k
// handed out in the step is the free stack's entry count - 1 - k, so every table entry and
// every slot is an independent lookup after two prefix sums over the requests, and the result
// does not depend on the order in which threads run. Pages are looked at before anything is
// decided: a request whose half-filled page is out of range asks for none, and the stack counts
// as ending in front of its first entry out of range. (The loads fall into the prefix sums.)
//
// One launch of one thread-block cluster (1 to 8 blocks of 1,024 threads): every block forms
// the prefix sums itself (at most 4,096 requests, four per thread), then the blocks share the
// rows. The free count may be updated in place, so block 0 writes it only after the cluster
// has met, when every block has read it. A decode step's plan is bound by the launch and a
// chain of dependent loads: 8.2 us for 256 requests of one token, 12.6 for 512 that bring 33,000
// tokens.
#include <cuda_runtime.h>

#include <atomic>

#include "gdn_attn_internal.h"
#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr int kThreads = 1024;
constexpr int kPerThread = kMaxSeqs / kThreads;

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// Exclusive sum over the block (64-bit: lengths are the caller's and may be any int32), the whole
// sum in warp_sums[32].
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();  // warp_sums of an earlier scan has been read
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    int64_t s = warp_sums[lane], t = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, t, o);
      if (lane >= o) t += y;
    }
    warp_sums[lane] = t - s;
    if (lane == 31) warp_sums[32] = t;
  }
  __syncthreads();
  return warp_sums[warp] + inc - x;
}

__device__ __forceinline__ int32_t ceil_div(int32_t a, int32_t b) {
  return (int32_t)(((int64_t)a + b - 1) / b);
}

// The last i in [0, n) with start[i] <= x (start non-decreasing, start[0] <= x).
__device__ __forceinline__ int32_t owner(const int32_t* start, int32_t n, int32_t x) {
  int32_t lo = 0, hi = n - 1;
  while (lo < hi) {
    const int32_t mid = (lo + hi + 1) >> 1;
    if (start[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) plan_kernel(PlanArgs p) {
  extern __shared__ int32_t sh[];
  __shared__ int64_t warp_sums[33];
  __shared__ int32_t taken, usable;  // pages handed out; pages in front of the first bad one
  const int n = p.num_seqs, tid = threadIdx.x, P = p.page_size;
  int32_t* cu = sh;               // [n + 1] first rows
  int32_t* page0 = cu + n + 1;    // [n + 1] first page handed out
  int32_t* ctx = page0 + n + 1;   // [n] cached tokens, -1: the request is not served
  const bool writer = cluster_rank() == 0;
  int32_t free_count = *p.free_count;
  int32_t raise = 0;
  if (free_count < 0 || free_count > p.num_pages) {
    raise = GDN_ERR_INVALID_ARGUMENT;
    free_count = free_count < 0 ? 0 : p.num_pages;
  }
  if (tid == 0) {
    taken = 0;
    usable = INT32_MAX;
  }
  auto bad_page = [&](int32_t k) {  // the k-th page from the top
    const int32_t id = p.free_pages[free_count - 1 - k];
    return id < 0 || id >= p.num_pages;
  };
  int32_t bad_at = INT32_MAX;  // this thread's first, of the 4,096 that most steps do with
#pragma unroll
  for (int i = kPerThread - 1; i >= 0; --i) {
    const int32_t k = tid + i * kThreads;
    if (k < free_count && bad_page(k)) bad_at = k;
  }

  // rows: exclusive sums of the new lengths
  const int per = (n + kThreads - 1) / kThreads, b0 = tid * per;
  int32_t c[kPerThread], m[kPerThread];
  bool ok[kPerThread];
  int64_t sum = 0;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int b = b0 + i;
    const bool in = i < per && b < n;
    c[i] = in ? p.ctx_len[b] : 0;
    m[i] = in ? p.new_len[b] : 0;
    sum += max(m[i], 0);
    ok[i] = in;
    if (m[i] > 0 && c[i] > 0 && (c[i] & (P - 1)) != 0 && c[i] / P < p.max_blocks) {
      const int32_t id = p.block_table[(size_t)b * p.max_blocks + c[i] / P];
      ok[i] = id >= 0 && id < p.num_pages;
    }
  }
  int64_t row = block_scan(sum, warp_sums);
  if (bad_at < INT32_MAX) atomicMin(&usable, bad_at);  // read behind the next sum's barriers
  int64_t need = 0;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int b = b0 + i;
    if (i < per && b < n) {
      const int64_t end = row + max(m[i], 0), len = (int64_t)c[i] + m[i];
      cu[b] = (int32_t)min(row, (int64_t)p.num_tokens);
      if (b == n - 1) cu[n] = (int32_t)min(end, (int64_t)p.num_tokens);
      ok[i] = ok[i] && c[i] >= 0 && m[i] >= 0 && end <= p.num_tokens &&
              len <= (int64_t)p.max_blocks * P && len <= INT32_MAX;
      if (!ok[i]) raise = GDN_ERR_INVALID_ARGUMENT;
      else need += ceil_div(c[i] + m[i], P) - ceil_div(c[i], P);
      row = end;
    }
  }
  // pages: exclusive sums of the needs; a request is served while the stack covers its sum
  int64_t page = block_scan(need, warp_sums);
  const int64_t asked = warp_sums[32];
  if (asked > kMaxSeqs) {  // the rest of the pages that may be handed out
    for (int32_t k = kMaxSeqs + tid; k < min(asked, (int64_t)free_count); k += kThreads)
      if (bad_page(k)) atomicMin(&usable, k);
    __syncthreads();
  }
  const int32_t have = min(usable, free_count);
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int b = b0 + i;
    if (i < per && b < n) {
      const int32_t want = ok[i] ? ceil_div(c[i] + m[i], P) - ceil_div(c[i], P) : 0;
      page0[b] = (int32_t)min(page, (int64_t)INT32_MAX);
      page += want;
      if (b == n - 1) page0[n] = (int32_t)min(page, (int64_t)INT32_MAX);
      if (want > 0) {
        if (page > have) {
          ok[i] = false;
          raise = max(raise, page > free_count ? (int32_t)GDN_ERR_POOL_EXHAUSTED
                                               : (int32_t)GDN_ERR_INVALID_ARGUMENT);
        } else {
          atomicMax(&taken, (int32_t)page);
        }
      }
      ctx[b] = ok[i] ? c[i] : -1;
      if (writer) p.kv_len[b] = ok[i] ? c[i] + m[i] : 0;
    }
  }
  __syncthreads();
  if (writer) {
    for (int b = tid; b <= n; b += kThreads) p.cu_new[b] = cu[b];
    if (raise) raise_status(p.status, raise);
  }

  const int gtid = (int)(blockIdx.x * kThreads) + tid, all = (int)(gridDim.x * kThreads);
  // new table entries
  const int32_t out = min(page0[n], have);
  for (int32_t k = gtid; k < out; k += all) {
    const int b = owner(page0, n, k);
    if (ctx[b] >= 0)
      p.block_table[(size_t)b * p.max_blocks + ceil_div(ctx[b], P) + k - page0[b]] =
          p.free_pages[free_count - 1 - k];
  }
  // slots and positions
  const int32_t rows = cu[n];
  for (int32_t r = gtid; r < p.num_tokens; r += all) {
    int32_t pos = 0;
    int64_t slot = -1;
    if (r < rows) {
      const int b = owner(cu, n, r);
      if (ctx[b] >= 0) {
        pos = ctx[b] + r - cu[b];
        const int32_t blk = pos / P, old = ceil_div(ctx[b], P);
        const int32_t id = blk < old
                               ? p.block_table[(size_t)b * p.max_blocks + blk]
                               : p.free_pages[free_count - 1 - (page0[b] + blk - old)];
        slot = (int64_t)id * P + (pos - blk * P);
      }
    }
    p.slots[r] = slot;
    if (p.positions) p.positions[r] = pos;
  }
  cluster_sync();  // every block has read *free_count
  if (writer && tid == 0) *p.free_count_out = free_count - taken;
}

__global__ void __launch_bounds__(kThreads) release_kernel(ReleaseArgs p) {
  extern __shared__ int32_t sh[];
  __shared__ int64_t warp_sums[33];
  __shared__ int32_t pushed;
  const int n = p.num_seqs, tid = threadIdx.x, lane = tid & 31;
  int32_t* cnt = sh;        // [n] pages of a row that is given back
  int32_t* at = sh + n;     // [n] their place on the stack
  int32_t count = *p.free_count, raise = 0;
  if (count < 0 || count > p.num_pages) {
    raise = GDN_ERR_INVALID_ARGUMENT;
    count = count < 0 ? 0 : p.num_pages;
  }
  if (tid == 0) pushed = 0;
  // a row is given back whole or not at all: look at its pages first (a warp per row)
  for (int b = tid >> 5; b < n; b += kThreads / 32) {
    int32_t k = 0;
    if (p.release[b] != 0) {
      const int32_t len = p.kv_len[b];
      k = len > 0 ? ceil_div(len, p.page_size) : 0;
      bool good = len >= 0 && k <= p.max_blocks;
      if (good)
        for (int j = lane; j < k; j += 32) {
          const int32_t id = p.block_table[(size_t)b * p.max_blocks + j];
          good = good && id >= 0 && id < p.num_pages;
        }
      if (!__all_sync(0xffffffffu, good)) {
        k = 0;
        raise = GDN_ERR_INVALID_ARGUMENT;
      }
    }
    if (lane == 0) cnt[b] = k;
  }
  __syncthreads();
  const int per = (n + kThreads - 1) / kThreads, b0 = tid * per;
  int64_t sum = 0;
  for (int b = b0; b < min(n, b0 + per); ++b) sum += cnt[b];
  int64_t place = count + block_scan(sum, warp_sums);
  for (int b = b0; b < min(n, b0 + per); ++b) {
    const int32_t k = cnt[b];
    if (place + k > p.num_pages) {  // more pages than there are: this row and the later stay
      raise = GDN_ERR_INVALID_ARGUMENT;
      cnt[b] = 0;
    } else if (k > 0) {
      atomicMax(&pushed, (int32_t)(place + k - count));
    }
    at[b] = (int32_t)min(place, (int64_t)p.num_pages);
    place += k;
  }
  __syncthreads();
  for (int b = tid >> 5; b < n; b += kThreads / 32)
    for (int j = lane; j < cnt[b]; j += 32) {
      int32_t* e = p.block_table + (size_t)b * p.max_blocks + j;
      p.free_pages[at[b] + j] = *e;
      *e = -1;
    }
  if (raise) raise_status(p.status, raise);
  if (tid == 0) *p.free_count = count + pushed;
}

std::atomic<int> g_plan_ready[kMaxDevices];

}  // namespace

int launch_kv_plan(const PlanArgs& a, void* stream) {
  const size_t smem = sizeof(int32_t) * (3 * (size_t)a.num_seqs + 2);
  int e = configure_once(g_plan_ready, [] {
    return (int)cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)(sizeof(int32_t) * (3 * kMaxSeqs + 2)));
  });
  if (e != 0) return e;
  // a block per 2,048 rows, up to the portable cluster size
  unsigned blocks = 1;
  while (blocks < 8 && (int64_t)blocks * 2048 < a.num_tokens) blocks *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = blocks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return (int)cudaLaunchKernelEx(&cfg, plan_kernel, a);
}

int launch_kv_release(const ReleaseArgs& a, void* stream) {
  const size_t smem = sizeof(int32_t) * 2 * (size_t)a.num_seqs;
  release_kernel<<<1, kThreads, smem, static_cast<cudaStream_t>(stream)>>>(a);
  return (int)cudaGetLastError();
}

}  // namespace gdn
