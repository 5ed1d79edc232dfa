// vkv_page_select: the pages one query per row attends to (Sparse Forcing summary,
// section 2 components 2 and 3, one query at a time): coarse scores of the pages' key
// means, then an exact top-k.
//
// The ranking decides which pages are read, so scores are accumulated in fp64: 16-bit
// queries times fp32 means leave no rounding that could swap two pages whose scores
// differ in fp32's last bits, whatever the order of the sum.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cstring>

#include "vkv_page.cuh"

namespace vkv {
namespace {

struct SelParams {
  FastDiv by_page;
  int score_steps, head_groups;
  int R, H, Hkv, G, page, n_pages, W, topk, first, last;
  const void* q;
  long long q_sb, q_sh;
  const float* kbar;
  const int* table;
  long long table_stride;
  const int* kv_len;
  int* sel;
  unsigned long long* keys;  // [R * Hkv][W]
  int* err;
};

// A score's order-preserving image: larger score, larger key; NaN lowest, -0 as +0.
// Real scores map below ~0, which marks the pages that are always kept.
__device__ __forceinline__ unsigned long long page_key(double v) {
  if (v != v) return 0ull;
  if (v == 0.0) v = 0.0;
  const unsigned long long u = (unsigned long long)__double_as_longlong(v);
  return u ^ ((u >> 63) ? ~0ull : 0x8000000000000000ull);
}

__device__ __forceinline__ double key_value(unsigned long long k) {  // the score of a real key
  return __longlong_as_double((long long)(k ^ ((k >> 63) ? 0x8000000000000000ull : ~0ull)));
}

constexpr int kScoreWarps = 8;
constexpr int kScoreStages = 3;
constexpr int kScoreStage = 4096;  // bytes of means that a warp fetches at a time

// One warp per key head (a block's warps take up to 8 neighbouring heads, whose means lie side
// by side), 8 lanes per page.  grid: x = row and head group, y = chunks of the table's width
// (p.score_steps steps of a warp).  HBM-bound (4 d bytes per page and key head): each lane
// streams the pieces of the means that it will use itself through a private cp.async ring, so
// that 128 KB per SM are in flight with no registers held and no barriers.  Length and table are
// asked for together, the queries while the first means are on their way.  The fp64 products
// hide behind the loads.
template <int D, typename T>
__global__ void __launch_bounds__(kScoreWarps * 32, 2) page_score_kernel(const SelParams p) {
  constexpr int PC = D / 32;                         // 16-byte pieces of a lane per page: 4 channels of each 32
  constexpr int PASSES = kScoreStage / (4 * 4 * D);  // pages of a lane group per stage
  constexpr int STEP = 4 * PASSES;                   // pages per step
  extern __shared__ __align__(16) char ring[];
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane & 7;
  const int r = blockIdx.x / p.head_groups, g = (blockIdx.x - r * p.head_groups) * kScoreWarps + warp;
  if (g >= p.Hkv) return;
  const int j0 = blockIdx.y * p.score_steps * STEP;
  const int raw = p.kv_len[r];
  const int* tab = p.table + r * p.table_stride;
  const int jl = j0 + (lane >> 3);  // the lane's first page
  int ahead[PASSES];                // table entries of the next step to fetch
#pragma unroll
  for (int e = 0; e < PASSES; ++e) ahead[e] = jl + e * 4 < p.W ? tab[jl + e * 4] : -1;
  const int len = page_row_len(raw, p.W, p.page, p.err);
  const int n = len <= 0 ? 0 : p.by_page(len) + (p.by_page(len) * p.page < len ? 1 : 0);
  if (j0 >= n || n <= p.topk) return;  // all of a short row's pages are kept: no ranking
  const int steps = min(p.score_steps, (n - j0 + STEP - 1) / STEP);
  const uint32_t mine = smem_u32(ring) + (uint32_t)(warp * kScoreStages * kScoreStage + lane * 16);
  int pg[kScoreStages][PASSES];  // pages of the steps in flight, the oldest first; -1: none
  auto fetch = [&](int step, int stage, int* got) {
#pragma unroll
    for (int e = 0; e < PASSES; ++e) {
      const int j = jl + step * STEP + e * 4, at = ahead[e];
      const bool in = step < steps && j < n, ok = in && at >= 0 && at < p.n_pages;
      if (in && !ok && sub == 0 && p.err) atomicCAS(p.err, 0, VKV_DEVERR_BAD_INDEX);
      got[e] = ok ? at : -1;
      if (ok) {
        const float* src = p.kbar + ((long long)at * p.Hkv + g) * D + sub * 4;
#pragma unroll
        for (int i = 0; i < PC; ++i)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(mine + stage * kScoreStage + (e * PC + i) * 512),
                       "l"(src + i * 32)
                       : "memory");
      }
      const int next = j + STEP;
      ahead[e] = next < n ? tab[next] : -1;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int s = 0; s < kScoreStages - 1; ++s) fetch(s, s, pg[s]);
  const T* q = reinterpret_cast<const T*>(p.q) + r * p.q_sb + (long long)g * p.G * p.q_sh + sub * 4;
  double qr[4 * PC];  // the group's summed queries, at the lane's channels
#pragma unroll
  for (int i = 0; i < 4 * PC; ++i) qr[i] = 0.0;
#pragma unroll 4
  for (int i = 0; i < p.G; ++i) {
    uint2 x[PC];
#pragma unroll
    for (int c = 0; c < PC; ++c) x[c] = *reinterpret_cast<const uint2*>(q + i * p.q_sh + c * 32);
#pragma unroll
    for (int c = 0; c < PC; ++c) {
      const T* e = reinterpret_cast<const T*>(&x[c]);
#pragma unroll
      for (int k = 0; k < 4; ++k) qr[4 * c + k] += (double)(float)e[k];
    }
  }
  unsigned long long* out = p.keys + ((size_t)r * p.Hkv + g) * p.W;
  int stage = 0;
#pragma unroll 1
  for (int step = 0; step < steps; ++step) {
    const int put = stage == 0 ? kScoreStages - 1 : stage - 1;
    fetch(step + kScoreStages - 1, put, pg[kScoreStages - 1]);
    asm volatile("cp.async.wait_group %0;" ::"n"(kScoreStages - 1) : "memory");
    double a[PASSES];
#pragma unroll
    for (int e = 0; e < PASSES; ++e) a[e] = 0.0;
#pragma unroll
    for (int i = 0; i < PC; ++i) {
#pragma unroll
      for (int e = 0; e < PASSES; ++e) {
        const float4 v = *reinterpret_cast<const float4*>(ring + (warp * kScoreStages + stage) * kScoreStage +
                                                          (e * PC + i) * 512 + lane * 16);
        a[e] = fma((double)v.x, qr[4 * i], a[e]);
        a[e] = fma((double)v.y, qr[4 * i + 1], a[e]);
        a[e] = fma((double)v.z, qr[4 * i + 2], a[e]);
        a[e] = fma((double)v.w, qr[4 * i + 3], a[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < PASSES; ++e) {
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) a[e] += __shfl_xor_sync(0xFFFFFFFFu, a[e], o);
      const int j = jl + step * STEP + e * 4;
      if (j < n && sub == 0) {
        const bool forced = j < p.first || j >= n - p.last;
        out[j] = forced ? ~0ull : pg[0][e] >= 0 ? page_key(a[e]) : 0ull;
      }
    }
#pragma unroll
    for (int s = 0; s + 1 < kScoreStages; ++s)
#pragma unroll
      for (int e = 0; e < PASSES; ++e) pg[s][e] = pg[s + 1][e];
    stage = stage + 1 == kScoreStages ? 0 : stage + 1;
  }
  griddep_launch_dependents();
}

constexpr int kPickThreads = 1024;
constexpr int kPickWarps = kPickThreads / 32;
constexpr int kBins = 2048;
constexpr int kCand = 512;  // keys of one bin that are ranked by comparing each with each
static_assert(kPickWarps == 32 && kBins == 2 * kPickThreads, "a lane per warp; two bins per thread");

// Inclusive sum over the block, in thread order; `total` is the block's sum.
__device__ __forceinline__ int warp_incl(int x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}
__device__ __forceinline__ int block_scan(int x, int* warp_sum, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  x = warp_incl(x, lane);
  __syncthreads();  // the last call's sums have been read
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  const int w = warp_incl(warp_sum[lane], lane);
  total = __shfl_sync(0xFFFFFFFFu, w, 31);
  const int before = __shfl_sync(0xFFFFFFFFu, w, (warp + 31) & 31);
  return warp ? x + before : x;
}

// A float's order-preserving image and back.
__device__ __forceinline__ uint32_t order_of(float f) {
  const uint32_t u = __float_as_uint(f);
  return u ^ (u >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t u) { return __uint_as_float(u ^ (u >> 31 ? 0x80000000u : 0xFFFFFFFFu)); }

// One block per (row, key head): the topk largest keys, of equal ones the lowest pages.
// The scores are dealt to bins of equal width between the least and the largest (a page's
// bin never decreases with its key, whatever the rounding); the bin that holds the topk-th
// key has few keys as a rule, and these are ranked one against the other.  Should it hold
// many (equal scores, outliers), a radix selection, 8 bits a pass, finds the key instead.
//
// Bound: latency, of the code's own fetch too (it runs once).  So many threads have few pages
// each: HELD (of up to 1024 HELD table columns) are kept in registers with their bins, 0 reads
// the keys again in every step.  2000 pages: 7.8 us with 256 threads of 8 pages.
template <int HELD>
__global__ void __launch_bounds__(kPickThreads) page_pick_kernel(const SelParams p) {
  __shared__ int hist[kBins];
  __shared__ int warp_sum[kPickWarps];
  __shared__ uint32_t warp_lo[kPickWarps], warp_hi[kPickWarps];
  __shared__ unsigned long long cand_key[kCand];
  __shared__ int cand_page[kCand];
  __shared__ int s_bin, s_above, s_in, s_n, s_page;
  __shared__ unsigned long long s_key;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  reinterpret_cast<int2*>(hist)[tid] = make_int2(0, 0);
  if (tid == 0) s_n = 0;
  griddep_wait();  // the scores
  const int r = blockIdx.x / p.Hkv;
  const int raw = p.kv_len[r];
  const int len = (raw >= -1 && (long long)raw <= (long long)p.W * p.page) ? raw : 0;
  const int n = len <= 0 ? 0 : p.by_page(len) + (p.by_page(len) * p.page < len ? 1 : 0);
  int* out = p.sel + (size_t)blockIdx.x * p.topk;
  const int kept = min(n, p.topk);
  for (int i = kept + tid; i < p.topk; i += kPickThreads) out[i] = -1;
  if (n <= p.topk) {
    if (p.W <= p.topk && tid == 0) page_row_len(raw, p.W, p.page, p.err);  // no score kernel has run
    // the row's pages are all kept and no score was taken: its first key head looks at their numbers
    const int* tab = p.table + r * p.table_stride;
    const bool look = p.err && blockIdx.x == r * p.Hkv;
    for (int i = tid; i < n; i += kPickThreads) {
      out[i] = i;
      if (look && (tab[i] < 0 || tab[i] >= p.n_pages)) atomicCAS(p.err, 0, VKV_DEVERR_BAD_INDEX);
    }
    return;
  }
  const unsigned long long* keys = p.keys + (size_t)blockIdx.x * p.W;
  // thread t has the t-th run of pages
  const int per = HELD ? HELD : (n - 1) / kPickThreads + 1;
  const int a = (int)min((long long)n, (long long)tid * per), b = min(n - a, per) + a;
  constexpr int N = HELD ? HELD : 1;
  unsigned long long own[N];
  float value[N];  // then the bin
  int own_bin[N];
  if (HELD) {
#pragma unroll
    for (int e = 0; e < N; ++e) own[e] = a + e < b ? keys[a + e] : 0ull;
#pragma unroll
    for (int e = 0; e < N; ++e) value[e] = (float)key_value(own[e]);
  }
  // the finite scores' range
  uint32_t lo_u = 0xFFFFFFFFu, hi_u = 0u;
  auto widen = [&](unsigned long long k, float f) {
    if (k != 0ull && k != ~0ull && fabsf(f) < INFINITY) {
      lo_u = min(lo_u, order_of(f));
      hi_u = max(hi_u, order_of(f));
    }
  };
  if (HELD) {
#pragma unroll
    for (int e = 0; e < N; ++e) widen(own[e], value[e]);
  } else {
    for (int j = a; j < b; ++j) widen(keys[j], (float)key_value(keys[j]));
  }
  lo_u = __reduce_min_sync(0xFFFFFFFFu, lo_u);
  hi_u = __reduce_max_sync(0xFFFFFFFFu, hi_u);
  if (lane == 0) {
    warp_lo[warp] = lo_u;
    warp_hi[warp] = hi_u;
  }
  __syncthreads();
  griddep_launch_dependents();
  lo_u = __reduce_min_sync(0xFFFFFFFFu, warp_lo[lane]);
  hi_u = __reduce_max_sync(0xFFFFFFFFu, warp_hi[lane]);
  const float lo = order_value(lo_u), scale = hi_u > lo_u ? (float)(kBins - 3) / (order_value(hi_u) - lo) : 0.f;
  auto bin_at = [&](unsigned long long k, float f) {
    if (k == 0ull) return 0;
    if (k == ~0ull) return kBins - 1;
    return 1 + max(0, min(kBins - 3, __float2int_rd((f - lo) * scale)));
  };
  if (HELD) {
#pragma unroll
    for (int e = 0; e < N; ++e) own_bin[e] = a + e < b ? bin_at(own[e], value[e]) : -1;
  }
  auto each = [&](auto&& f) {  // f(page, key, bin) for the thread's pages
    if (HELD) {
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (a + e < b) f(a + e, own[e], own_bin[e]);
    } else {
#pragma unroll 1
      for (int j = a; j < b; ++j) {
        const unsigned long long k = keys[j];
        f(j, k, bin_at(k, (float)key_value(k)));
      }
    }
  };
  each([&](int, unsigned long long, int at) { atomicAdd(&hist[at], 1); });
  __syncthreads();
  {  // the bin of the topk-th key: thread t has bins 2 t and 2 t + 1 from the top
    int total;
    const int2 c = reinterpret_cast<const int2*>(hist)[kPickThreads - 1 - tid];
    const int above = block_scan(c.x + c.y, warp_sum, total) - (c.x + c.y);
    const bool up = p.topk <= above + c.y;
    if (above < p.topk && p.topk <= above + c.x + c.y) {
      s_bin = kBins - 1 - 2 * tid - (up ? 0 : 1);
      s_above = above + (up ? 0 : c.y);
      s_in = up ? c.y : c.x;
    }
  }
  __syncthreads();
  const int bin = s_bin, n_in = s_in;
  int need = p.topk - s_above;  // keys of the bin to take: at least one, at most n_in
  if (n_in <= kCand) {
    each([&](int j, unsigned long long k, int at) {
      if (at == bin) {
        const int i = atomicAdd(&s_n, 1);
        cand_key[i] = k;
        cand_page[i] = j;
      }
    });
    __syncthreads();
    for (int i = tid; i < n_in; i += kPickThreads) {
      const unsigned long long k = cand_key[i];
      const int j = cand_page[i];
      int rank = 0;
      for (int x = 0; x < n_in; ++x) rank += cand_key[x] > k || (cand_key[x] == k && cand_page[x] < j);
      if (rank == need - 1) {
        s_key = k;
        s_page = j;
      }
    }
  } else {
    unsigned long long thr = 0ull, mask = 0ull;  // digits of the wanted key found so far
#pragma unroll 1
    for (int shift = 56; shift >= 0; shift -= 8) {
      __syncthreads();
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      each([&](int, unsigned long long k, int at) {
        if ((k & mask) == thr && at == bin) atomicAdd(&hist[(int)(k >> shift) & 255], 1);
      });
      __syncthreads();
      int total;
      const int cnt = tid < 256 ? hist[255 - tid] : 0, inc = block_scan(cnt, warp_sum, total);
      if (inc - cnt < need && need <= inc) {
        s_bin = 255 - tid;
        s_above = inc - cnt;
      }
      __syncthreads();
      thr |= (unsigned long long)s_bin << shift;
      mask |= 255ull << shift;
      need -= s_above;
    }
    // the page of the need-th of the keys equal to it
    int eq = 0, total;
    each([&](int, unsigned long long k, int) { eq += k == thr; });
    int before = block_scan(eq, warp_sum, total) - eq;
    if (before < need && need <= before + eq) {
      each([&](int j, unsigned long long k, int) {
        if (k == thr && ++before == need) s_page = j;
      });
      s_key = thr;
    }
  }
  __syncthreads();
  // ascending output
  const unsigned long long key = s_key;
  const int last = s_page;
  int mine = 0, total;
  each([&](int j, unsigned long long k, int) { mine += k > key || (k == key && j <= last); });
  int at = block_scan(mine, warp_sum, total) - mine;
  each([&](int j, unsigned long long k, int) {
    if (k > key || (k == key && j <= last)) out[at++] = j;
  });
}

}  // namespace
}  // namespace vkv

using namespace vkv;

extern "C" size_t vkv_page_select_workspace_size(int32_t R, int32_t Hkv, int32_t W) {
  if (R < 1 || Hkv < 1 || W < 1) return 0;
  return ((size_t)R * Hkv * W * sizeof(unsigned long long) + 255) & ~(size_t)255;
}

extern "C" vkv_status vkv_page_select(const vkv_page_select_args* a, vkv_stream_t stream) {
  if (!a) return VKV_ERR_NULL;
  if (a->d != 64 && a->d != 128) return VKV_ERR_UNSUPPORTED;
  if (a->q_dtype != VKV_BF16 && a->q_dtype != VKV_FP16) return VKV_ERR_UNSUPPORTED;
  if (a->R < 1 || a->R > VKV_PAGE_MAX_ROWS || a->H < 1 || a->Hkv < 1 || a->H % a->Hkv || a->page < 1 ||
      a->n_pages < 1 || a->W < 1 || a->topk < 1 || a->topk > 4096 || a->sink_pages < 0 || a->local_pages < 0 ||
      (long long)a->sink_pages + a->local_pages > a->topk || a->table_stride < a->W)
    return VKV_ERR_SHAPE;
  // a warp of the score kernel counts columns up to 4 steps of at most 16 past the row's last
  if ((long long)a->R * a->W > INT_MAX || (long long)a->W * a->page > INT_MAX || (long long)a->R * a->Hkv > INT_MAX ||
      a->W > INT_MAX - 256)
    return VKV_ERR_UNSUPPORTED;
  if (!a->q.ptr || !a->kbar || !a->table || !a->kv_len || !a->sel) return VKV_ERR_NULL;
  vkv_tensor q = a->q;
  q.st = 0;
  if (!page_tensor_aligned(q, a->q_dtype) || (reinterpret_cast<uintptr_t>(a->kbar) & 15u)) return VKV_ERR_ALIGN;
  if (!a->workspace || a->workspace_bytes < vkv_page_select_workspace_size(a->R, a->Hkv, a->W))
    return VKV_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(a->workspace) & 255u) return VKV_ERR_ALIGN;
  int dev = 0;
  const int n_sm = device_sm_count(&dev);
  if (n_sm <= 0) return VKV_ERR_CUDA;
  SelParams p;
  std::memset(&p, 0, sizeof(p));
  p.R = a->R; p.H = a->H; p.Hkv = a->Hkv; p.G = a->H / a->Hkv;
  p.page = a->page; p.n_pages = a->n_pages; p.W = a->W; p.topk = a->topk;
  p.by_page = fast_div(a->page);
  p.first = a->sink_pages; p.last = a->local_pages;
  p.q = a->q.ptr; p.q_sb = a->q.sb; p.q_sh = a->q.sh;
  p.kbar = a->kbar;
  p.table = a->table; p.table_stride = a->table_stride;
  p.kv_len = a->kv_len;
  p.sel = a->sel;
  p.keys = reinterpret_cast<unsigned long long*>(a->workspace);
  p.err = a->err_word;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int seqs = a->R * a->Hkv;
  if (a->W > a->topk) {
    // steps per warp: one round of the GPU's warps, or rounds of 16 steps (rows end at different
    // places; 32 rows of 16001 to 48000 tokens: 41.5 us with 4, 37.5 with 8, 35.2 with 16)
    const int step = kScoreStage / (4 * a->d);
    const long long row_steps = ((long long)a->W + step - 1) / step;
    const int warps = std::min(kScoreWarps, a->Hkv);
    p.head_groups = (a->Hkv + kScoreWarps - 1) / kScoreWarps;
    const long long round = 2ll * kScoreWarps * n_sm;
    p.score_steps = (int)std::min<long long>(16, (seqs * row_steps + round - 1) / round);
    p.score_steps = (int)std::max<long long>(p.score_steps, (row_steps + 65534) / 65535);
    const dim3 grid((unsigned)(a->R * p.head_groups), (unsigned)((row_steps + p.score_steps - 1) / p.score_steps));
    const size_t smem = (size_t)warps * kScoreStages * kScoreStage;
    const bool bf = a->q_dtype == VKV_BF16;
    auto score = a->d == 128 ? (bf ? page_score_kernel<128, __nv_bfloat16> : page_score_kernel<128, __half>)
                             : (bf ? page_score_kernel<64, __nv_bfloat16> : page_score_kernel<64, __half>);
    static std::atomic<uint64_t> ready[4];  // by kernel: devices (by bit) on which the shared memory limit is raised
    std::atomic<uint64_t>& rd = ready[(a->d == 128 ? 2 : 0) + (bf ? 1 : 0)];
    if (!(rd.load(std::memory_order_acquire) >> dev & 1u)) {
      if (cudaFuncSetAttribute(score, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kScoreWarps * kScoreStages * kScoreStage) != cudaSuccess) {
        cudaGetLastError();
        return VKV_ERR_CUDA;
      }
      rd.fetch_or(1ull << dev, std::memory_order_release);
    }
    if (launch_ahead(score, grid, dim3((unsigned)warps * 32), smem, st, p) != cudaSuccess) return VKV_ERR_CUDA;
  }
  auto pick = a->W <= 2 * kPickThreads ? page_pick_kernel<2> : a->W <= 8 * kPickThreads ? page_pick_kernel<8> : page_pick_kernel<0>;
  return launch_ahead(pick, dim3((unsigned)seqs), dim3(kPickThreads), 0, st, p) == cudaSuccess ? VKV_OK : VKV_ERR_CUDA;
}
