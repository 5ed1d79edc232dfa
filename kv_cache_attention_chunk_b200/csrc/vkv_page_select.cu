// vkv_page_select: the pages one query per row attends to (Sparse Forcing summary,
// section 2 components 2 and 3, one query at a time): coarse scores of the pages' key
// means, then an exact top-k.
//
// The ranking decides which pages are read, so scores are accumulated in fp64: 16-bit
// queries times fp32 means leave no rounding that could swap two pages whose scores
// differ in fp32's last bits, whatever the order of the sum.
#include <algorithm>
#include <climits>
#include <cstring>

#include "vkv_page.cuh"

namespace vkv {
namespace {

struct SelParams {
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

constexpr int kScoreThreads = 256;
constexpr int kScorePer = 2;                                // pages per 8 lanes, loads in flight together
constexpr int kScorePages = kScorePer * kScoreThreads / 8;  // pages per block

// grid: x = r * Hkv + g, y = page chunks of the table's width.  8 lanes per page; every
// load of a block (its means, 512 bytes a page at d = 128) is in flight while the queries
// are added up.
template <int D, typename T>
__global__ void __launch_bounds__(kScoreThreads) page_score_kernel(const SelParams p) {
  constexpr int PER = D / 8;  // channels per lane: 4 consecutive of each 32
  __shared__ double qs[D];
  griddep_launch_dependents();
  const int r = blockIdx.x / p.Hkv, g = blockIdx.x - r * p.Hkv;
  const int len = page_row_len(p.kv_len[r], p.W, p.page, p.err);
  const int n = len <= 0 ? 0 : (int)(((long long)len + p.page - 1) / p.page);
  const int j0 = blockIdx.y * kScorePages;
  if (j0 >= n || n <= p.topk) return;  // all of a short row's pages are kept: no ranking
  const int sub = threadIdx.x & 7, grp = threadIdx.x >> 3;
  const int* tab = p.table + r * p.table_stride;
  int pg[kScorePer];
  float4 v[kScorePer][PER / 4];
#pragma unroll
  for (int e = 0; e < kScorePer; ++e) {
    const int j = j0 + e * (kScoreThreads / 8) + grp;
    pg[e] = j < n ? tab[j] : -1;
    if (j < n && (pg[e] < 0 || pg[e] >= p.n_pages)) {
      if (p.err && sub == 0) atomicCAS(p.err, 0, VKV_DEVERR_BAD_INDEX);
      pg[e] = -1;
    }
  }
  const T* q = reinterpret_cast<const T*>(p.q) + r * p.q_sb + (long long)g * p.G * p.q_sh;
  if (threadIdx.x < D) {
    double s = 0.0;
    for (int i = 0; i < p.G; i += 4) {
      T x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = q[min(i + e, p.G - 1) * p.q_sh + threadIdx.x];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i + e < p.G) s += (double)(float)x[e];
    }
    qs[threadIdx.x] = s;
  }
#pragma unroll
  for (int e = 0; e < kScorePer; ++e) {
    const float4* kb = reinterpret_cast<const float4*>(p.kbar + ((long long)max(pg[e], 0) * p.Hkv + g) * D) + sub;
#pragma unroll
    for (int i = 0; i < PER / 4; ++i) v[e][i] = pg[e] >= 0 ? __ldg(kb + i * 8) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __syncthreads();
  unsigned long long* out = p.keys + (size_t)blockIdx.x * p.W;
#pragma unroll
  for (int e = 0; e < kScorePer; ++e) {
    double a = 0.0;
#pragma unroll
    for (int i = 0; i < PER / 4; ++i) {
      const double* qr = qs + i * 32 + sub * 4;
      a = fma((double)v[e][i].x, qr[0], a);
      a = fma((double)v[e][i].y, qr[1], a);
      a = fma((double)v[e][i].z, qr[2], a);
      a = fma((double)v[e][i].w, qr[3], a);
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
    const int j = j0 + e * (kScoreThreads / 8) + grp;
    if (j < n && sub == 0) {
      const bool forced = j < p.first || j >= n - p.last;
      out[j] = forced ? ~0ull : pg[e] >= 0 ? page_key(a) : 0ull;
    }
  }
}

constexpr int kPickThreads = 256;
constexpr int kPickWarps = kPickThreads / 32;
constexpr int kBins = 2048;
constexpr int kCand = 512;  // keys of one bin that are ranked by comparing each with each

// Inclusive sum over the block, in thread order; `total` is the block's sum.
__device__ __forceinline__ int block_scan(int x, int* warp_sum, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // the last call's sums have been read
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int w = 0; w < kPickWarps; ++w) {
    if (w < warp) x += warp_sum[w];
    total += warp_sum[w];
  }
  return x;
}

// One block per (row, key head): the topk largest keys, of equal ones the lowest pages.
// The scores are dealt to bins of equal width between the least and the largest (a page's
// bin never decreases with its key, whatever the rounding); the bin that holds the topk-th
// key has few keys as a rule, and these are ranked one against the other.  Should it hold
// many (equal scores, outliers), a radix selection, 8 bits a pass, finds the key instead.
__global__ void __launch_bounds__(kPickThreads) page_pick_kernel(const SelParams p) {
  __shared__ int hist[kBins];
  __shared__ int warp_sum[kPickWarps];
  __shared__ float warp_lo[kPickWarps], warp_hi[kPickWarps];
  __shared__ unsigned long long cand_key[kCand];
  __shared__ int cand_page[kCand];
  __shared__ int s_bin, s_above, s_in, s_n, s_page;
  __shared__ unsigned long long s_key;
  griddep_wait();  // the scores
  const int r = blockIdx.x / p.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int raw = p.kv_len[r];
  const int len = (raw >= -1 && (long long)raw <= (long long)p.W * p.page) ? raw : 0;
  const int n = len <= 0 ? 0 : (int)(((long long)len + p.page - 1) / p.page);
  int* out = p.sel + (size_t)blockIdx.x * p.topk;
  const int kept = min(n, p.topk);
  for (int i = kept + tid; i < p.topk; i += kPickThreads) out[i] = -1;
  if (n <= p.topk) {
    if (p.W <= p.topk && tid == 0) page_row_len(raw, p.W, p.page, p.err);  // no score kernel has run
    for (int i = tid; i < n; i += kPickThreads) out[i] = i;
    return;
  }
  const unsigned long long* keys = p.keys + (size_t)blockIdx.x * p.W;
  for (int i = tid; i < kBins; i += kPickThreads) hist[i] = 0;
  if (tid == 0) s_n = 0;
  // the finite scores' range
  float lo = INFINITY, hi = -INFINITY;
  for (int j = tid; j < n; j += kPickThreads) {
    const unsigned long long k = keys[j];
    const float f = (float)key_value(k);
    if (k != 0ull && k != ~0ull && fabsf(f) < INFINITY) {
      lo = fminf(lo, f);
      hi = fmaxf(hi, f);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
  }
  if (lane == 0) {
    warp_lo[warp] = lo;
    warp_hi[warp] = hi;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kPickWarps; ++w) {
    lo = fminf(lo, warp_lo[w]);
    hi = fmaxf(hi, warp_hi[w]);
  }
  const float scale = hi > lo ? (float)(kBins - 3) / (hi - lo) : 0.f;
  auto bin_of = [&](unsigned long long k) {
    if (k == 0ull) return 0;
    if (k == ~0ull) return kBins - 1;
    return 1 + max(0, min(kBins - 3, __float2int_rd(((float)key_value(k) - lo) * scale)));
  };
  for (int j = tid; j < n; j += kPickThreads) atomicAdd(&hist[bin_of(keys[j])], 1);
  __syncthreads();
  {  // the bin of the topk-th key: thread t scans bins from the top
    constexpr int B = kBins / kPickThreads;
    int c[B], sum = 0, total;
#pragma unroll
    for (int e = 0; e < B; ++e) sum += c[e] = hist[kBins - 1 - (tid * B + e)];
    int above = block_scan(sum, warp_sum, total) - sum;
#pragma unroll
    for (int e = 0; e < B; ++e) {
      if (above < p.topk && p.topk <= above + c[e]) {
        s_bin = kBins - 1 - (tid * B + e);
        s_above = above;
        s_in = c[e];
      }
      above += c[e];
    }
  }
  __syncthreads();
  const int bin = s_bin, n_in = s_in;
  int need = p.topk - s_above;  // keys of the bin to take: at least one, at most n_in
  if (n_in <= kCand) {
    for (int j = tid; j < n; j += kPickThreads) {
      const unsigned long long k = keys[j];
      if (bin_of(k) == bin) {
        const int at = atomicAdd(&s_n, 1);
        cand_key[at] = k;
        cand_page[at] = j;
      }
    }
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
      hist[tid] = 0;
      __syncthreads();
      for (int j = tid; j < n; j += kPickThreads) {
        const unsigned long long k = keys[j];
        if ((k & mask) == thr && bin_of(k) == bin) atomicAdd(&hist[(int)(k >> shift) & 255], 1);
      }
      __syncthreads();
      int total;
      const int cnt = hist[255 - tid], inc = block_scan(cnt, warp_sum, total);
      if (inc - cnt < need && need <= inc) {
        s_bin = 255 - tid;
        s_above = inc - cnt;
      }
      __syncthreads();
      thr |= (unsigned long long)s_bin << shift;
      mask |= 255ull << shift;
      need -= s_above;
    }
    // the page of the need-th of the keys equal to it; thread t has the t-th run of pages
    const int per = (n + kPickThreads - 1) / kPickThreads, a = min(n, tid * per), b = min(n, a + per);
    int eq = 0, total;
    for (int j = a; j < b; ++j) eq += keys[j] == thr;
    int before = block_scan(eq, warp_sum, total) - eq;
    if (before < need && need <= before + eq) {
      for (int j = a; j < b; ++j)
        if (keys[j] == thr && ++before == need) s_page = j;
      s_key = thr;
    }
  }
  __syncthreads();
  // ascending output; thread t has the t-th run of pages
  const unsigned long long key = s_key;
  const int last = s_page;
  const int per = (n + kPickThreads - 1) / kPickThreads, a = min(n, tid * per), b = min(n, a + per);
  int mine = 0, total;
  for (int j = a; j < b; ++j) {
    const unsigned long long k = keys[j];
    mine += k > key || (k == key && j <= last);
  }
  int at = block_scan(mine, warp_sum, total) - mine;
  for (int j = a; j < b; ++j) {
    const unsigned long long k = keys[j];
    if (k > key || (k == key && j <= last)) out[at++] = j;
  }
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
  if ((long long)a->R * a->W > INT_MAX || (long long)a->W * a->page > INT_MAX || (long long)a->R * a->Hkv > INT_MAX || a->W > 65535 * kScorePages)
    return VKV_ERR_UNSUPPORTED;
  if (!a->q.ptr || !a->kbar || !a->table || !a->kv_len || !a->sel) return VKV_ERR_NULL;
  vkv_tensor q = a->q;
  q.st = 0;
  if (!page_tensor_aligned(q, a->q_dtype) || (reinterpret_cast<uintptr_t>(a->kbar) & 15u)) return VKV_ERR_ALIGN;
  if (!a->workspace || a->workspace_bytes < vkv_page_select_workspace_size(a->R, a->Hkv, a->W))
    return VKV_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(a->workspace) & 255u) return VKV_ERR_ALIGN;
  int dev = 0;
  if (device_sm_count(&dev) <= 0) return VKV_ERR_CUDA;
  SelParams p;
  std::memset(&p, 0, sizeof(p));
  p.R = a->R; p.H = a->H; p.Hkv = a->Hkv; p.G = a->H / a->Hkv;
  p.page = a->page; p.n_pages = a->n_pages; p.W = a->W; p.topk = a->topk;
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
    const dim3 grid((unsigned)seqs, (unsigned)((a->W + kScorePages - 1) / kScorePages));
    const bool bf = a->q_dtype == VKV_BF16;
    if (a->d == 128) {
      if (bf) page_score_kernel<128, __nv_bfloat16><<<grid, kScoreThreads, 0, st>>>(p);
      else page_score_kernel<128, __half><<<grid, kScoreThreads, 0, st>>>(p);
    } else {
      if (bf) page_score_kernel<64, __nv_bfloat16><<<grid, kScoreThreads, 0, st>>>(p);
      else page_score_kernel<64, __half><<<grid, kScoreThreads, 0, st>>>(p);
    }
    if (cudaGetLastError() != cudaSuccess) return VKV_ERR_CUDA;
  }
  // the second kernel's blocks take their places while the first one ends
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)seqs);
  cfg.blockDim = dim3(kPickThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = a->W > a->topk ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, page_pick_kernel, p) != cudaSuccess) {
    cudaGetLastError();
    return VKV_ERR_CUDA;
  }
  return VKV_OK;
}
