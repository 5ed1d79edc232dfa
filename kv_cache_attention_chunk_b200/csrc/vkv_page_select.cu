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

constexpr int kScoreThreads = 256;
constexpr int kScorePages = 256;  // pages per CTA

// grid: x = page chunks of the table's width, y = r * Hkv + g.  8 lanes per page.
template <int D, typename T>
__global__ void __launch_bounds__(kScoreThreads) page_score_kernel(const SelParams p) {
  constexpr int PER = D / 8;  // channels per lane: 4 consecutive of each 32
  __shared__ double qs[D];
  const int r = blockIdx.y / p.Hkv, g = blockIdx.y - r * p.Hkv;
  const int len = page_row_len(p.kv_len[r], p.W, p.page, p.err);
  const int n = len <= 0 ? 0 : (int)(((long long)len + p.page - 1) / p.page);
  const int j0 = blockIdx.x * kScorePages;
  if (j0 >= n || n <= p.topk) return;  // all of a short row's pages are kept: no ranking
  const T* q = reinterpret_cast<const T*>(p.q) + r * p.q_sb + (long long)g * p.G * p.q_sh;
  for (int x = threadIdx.x; x < D; x += kScoreThreads) {
    double s = 0.0;
    for (int i = 0; i < p.G; ++i) s += (double)(float)q[i * p.q_sh + x];
    qs[x] = s;
  }
  __syncthreads();
  const int sub = threadIdx.x & 7, grp = threadIdx.x >> 3;
  double qr[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) qr[i] = qs[(i / 4) * 32 + sub * 4 + (i & 3)];
  unsigned long long* out = p.keys + (size_t)blockIdx.y * p.W;
  const int* tab = p.table + r * p.table_stride;
  const int j1 = min(n, j0 + kScorePages);
  for (int jb = j0; jb < j1; jb += kScoreThreads / 8) {
    const int j = jb + grp;
    const bool in = j < j1;
    const int pg = in ? tab[j] : -1;
    const bool ok = pg >= 0 && pg < p.n_pages;
    double a = 0.0;
    if (ok) {
      const float4* kb = reinterpret_cast<const float4*>(p.kbar + ((long long)pg * p.Hkv + g) * D) + sub;
      float4 v[PER / 4];
#pragma unroll
      for (int i = 0; i < PER / 4; ++i) v[i] = __ldg(kb + i * 8);
#pragma unroll
      for (int i = 0; i < PER / 4; ++i) {
        a = fma((double)v[i].x, qr[4 * i], a);
        a = fma((double)v[i].y, qr[4 * i + 1], a);
        a = fma((double)v[i].z, qr[4 * i + 2], a);
        a = fma((double)v[i].w, qr[4 * i + 3], a);
      }
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
    if (in && sub == 0) {
      if (!ok && p.err) atomicCAS(p.err, 0, VKV_DEVERR_BAD_INDEX);
      const bool forced = j < p.first || j >= n - p.last;
      out[j] = forced ? ~0ull : ok ? page_key(a) : 0ull;
    }
  }
}

constexpr int kPickThreads = 256;

// One CTA per (row, key head): radix selection of the topk-th largest key, 8 bits a pass
// from the top, until the keys that share the digits found so far are all to be taken;
// then the kept pages in ascending order, of the keys equal to the threshold the lowest.
__global__ void __launch_bounds__(kPickThreads) page_pick_kernel(const SelParams p) {
  __shared__ int hist[256];
  __shared__ int warp_sum[kPickThreads / 32];
  __shared__ int s_digit, s_above, s_in;
  const int r = blockIdx.x / p.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int raw = p.kv_len[r];
  const int len = (raw >= -1 && (long long)raw <= (long long)p.W * p.page) ? raw : 0;
  const int n = len <= 0 ? 0 : (int)(((long long)len + p.page - 1) / p.page);
  int* out = p.sel + (size_t)blockIdx.x * p.topk;
  const int kept = min(n, p.topk);
  for (int i = kept + tid; i < p.topk; i += kPickThreads) out[i] = -1;
  if (n <= p.topk) {
    for (int i = tid; i < n; i += kPickThreads) out[i] = i;
    return;
  }
  const unsigned long long* keys = p.keys + (size_t)blockIdx.x * p.W;
  unsigned long long thr = 0ull, mask = 0ull;  // digits of the threshold found so far
  int need = p.topk;                           // keys still to take among those in play
  bool all = false;                            // every key in play is taken
#pragma unroll 1
  for (int shift = 56; shift >= 0 && !all; shift -= 8) {
    hist[tid] = 0;
    __syncthreads();
    for (int j = tid; j < n; j += kPickThreads) {
      const unsigned long long k = keys[j];
      if ((k & mask) == thr) atomicAdd(&hist[(int)(k >> shift) & 255], 1);
    }
    __syncthreads();
    // thread t: digit 255 - t; keys in play with a digit above it
    const int cnt = hist[255 - tid];
    int inc = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += t;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    for (int w = 0; w < warp; ++w) inc += warp_sum[w];
    if (inc - cnt < need && need <= inc) {
      s_digit = 255 - tid;
      s_above = inc - cnt;
      s_in = cnt;
    }
    __syncthreads();
    thr |= (unsigned long long)s_digit << shift;
    mask |= 255ull << shift;
    need -= s_above;
    all = need == s_in;
    __syncthreads();
  }
  // ascending output; `need` of the keys equal to the threshold (on the digits found) are taken
  int written = 0, eq_seen = 0;
  for (int j0 = 0; j0 < n; j0 += kPickThreads) {
    const int j = j0 + tid;
    const unsigned long long k = j < n ? keys[j] : 0ull;
    const bool eq = j < n && (k & mask) == thr;
    const bool above = j < n && (k & mask) > thr;
    // equal keys before this one, then kept ones before it
    unsigned b = __ballot_sync(0xFFFFFFFFu, eq);
    if (lane == 0) warp_sum[warp] = __popc(b);
    __syncthreads();
    int before = eq_seen, tot = 0;
    for (int w = 0; w < kPickThreads / 32; ++w) {
      if (w < warp) before += warp_sum[w];
      tot += warp_sum[w];
    }
    eq_seen += tot;
    const bool keep = above || (eq && before + __popc(b & ((1u << lane) - 1u)) < need);
    __syncthreads();
    b = __ballot_sync(0xFFFFFFFFu, keep);
    if (lane == 0) warp_sum[warp] = __popc(b);
    __syncthreads();
    int at = written;
    tot = 0;
    for (int w = 0; w < kPickThreads / 32; ++w) {
      if (w < warp) at += warp_sum[w];
      tot += warp_sum[w];
    }
    written += tot;
    if (keep) out[at + __popc(b & ((1u << lane) - 1u))] = j;
    __syncthreads();
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
  if ((long long)a->R * a->W > INT_MAX || (long long)a->W * a->page > INT_MAX || (long long)a->R * a->Hkv > 65535 * 16)
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
    const dim3 grid((unsigned)((a->W + kScorePages - 1) / kScorePages), (unsigned)seqs);
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
  page_pick_kernel<<<(unsigned)seqs, kPickThreads, 0, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? VKV_OK : VKV_ERR_CUDA;
}
