// vkv_page_map: pages and slots of one step's new tokens, from the rows' lengths.
//
// Every block reads all rows (a few KB, from L2 after the first) and scans them for itself:
// tokens, pages taken and pages returned before each row.  So no block waits for another's
// result, and the tokens, the new table entries and the returned pages can be spread over
// the grid's threads, each of which finds its row by bisection of the scan in shared memory.
// Where lengths or ring positions are updated in place, they may be written only after every
// block has read them: those steps run as one cluster of up to 8 blocks, with a cluster barrier in
// between (256 rows that decode 5.9 us, apart 5.5; 48 rows' prompts of up to 4680 tokens 18, apart 4.3).
//
// Bound: latency.  A decoding step moves some tens of KB; its time is the launch, two
// dependent reads (lengths, then ring or table) and the stores.  A thread takes kTok tokens
// at a time, so that their bisections and look-ups overlap.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cstring>

#include "vkv_page.cuh"

namespace vkv {
namespace {

constexpr int kMapThreads = 512;
constexpr int kMapMaxCluster = 8;
constexpr int kTok = 4;

struct MapParams {
  int R, W, page, n_ring, max_tokens;
  FastDiv by_page;
  const int* kv_len;
  const int* new_len;
  int* table;
  long long table_stride;
  int* ring;
  const long long* ring_pos;
  int* kv_len_out;
  long long* ring_pos_out;
  long long* slot;
  int* row;
  int* pos;
  int* cu;
  int* err;
};

// All threads of the cluster; memory operations before it are visible after it.
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Entry `i` (< n) behind position `first` (< n) of a ring of n < 2^31 entries.
__device__ __forceinline__ unsigned ring_at(int first, int i, int n) {
  const unsigned x = (unsigned)first + (unsigned)i;
  return x >= (unsigned)n ? x - (unsigned)n : x;
}

// Where position t of a ring of n lies; a 64-bit remainder only once t has passed 2^32.
__device__ __forceinline__ int ring_start(long long t, int n) {
  return (unsigned long long)t >> 32 ? (int)(t % n) : (int)((unsigned)t % (unsigned)n);
}

template <bool IN_PLACE>
__global__ void __launch_bounds__(kMapThreads) page_map_kernel(const MapParams p) {
  griddep_wait();
  extern __shared__ int sm[];
  int* tok = sm;               // [R + 1] new tokens before row r
  int* need = tok + p.R + 1;   // [R + 1] pages taken before row r
  int* back = need + p.R + 1;  // [R + 1] pages returned before row r
  int* held = back + p.R + 1;  // [R] tokens held (0 for a free row)
  __shared__ long long warp_tok[kMapThreads / 32];
  __shared__ unsigned long long warp_pg[kMapThreads / 32];
  __shared__ int fault;  // bit 0: a length out of range, bit 1: a row that does not fit its table row
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int R = p.R, page = p.page;
  if (tid == 0) fault = 0;
  const long long taken = p.ring_pos[0], returned = p.ring_pos[1];
  const long long row_cap = (long long)p.W * page;
  auto pages_of = [&](int n) { return p.by_page(n) + (p.by_page(n) * page < n ? 1 : 0); };
  const int ring_t = ring_start(taken, p.n_ring), ring_b = ring_start(returned, p.n_ring);
  __syncthreads();
  // each thread: `per` consecutive rows; 64-bit token sum, pages as need | back << 32
  const int per = (R + kMapThreads - 1) / kMapThreads;
  const int r0 = min(R, tid * per), r1 = min(R, r0 + per);
  long long my_tok = 0;
  unsigned long long my_pg = 0;
  for (int r = r0; r < r1; ++r) {
    int len = p.kv_len[r], add = p.new_len[r], bad = 0;
    if (len < -1 || len > row_cap || add < -1) {
      bad = 1;
      len = add = 0;
    } else if ((long long)max(len, 0) + max(add, 0) > row_cap) {
      bad = 2;
      add = 0;
    }
    if (bad) atomicOr(&fault, bad);
    const int h = max(len, 0);
    const unsigned had = (unsigned)pages_of(h);
    unsigned nd = 0, bk = 0;
    if (add < 0) bk = had;
    else nd = (unsigned)pages_of(h + add) - had;  // h + add <= W * page
    held[r] = h;
    tok[r] = max(add, 0);
    need[r] = (int)nd;
    back[r] = (int)bk;
    my_tok += max(add, 0);
    my_pg += nd | ((unsigned long long)bk << 32);
  }
  long long it = my_tok;
  unsigned long long ip = my_pg;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xFFFFFFFFu, it, o);
    const unsigned long long b = __shfl_up_sync(0xFFFFFFFFu, ip, o);
    if (lane >= o) {
      it += a;
      ip += b;
    }
  }
  if (lane == 31) {
    warp_tok[warp] = it;
    warp_pg[warp] = ip;
  }
  __syncthreads();
  long long base_t = it - my_tok, all_t = 0;
  unsigned long long base_p = ip - my_pg, all_p = 0;
#pragma unroll
  for (int w = 0; w < kMapThreads / 32; ++w) {
    if (w < warp) {
      base_t += warp_tok[w];
      base_p += warp_pg[w];
    }
    all_t += warp_tok[w];
    all_p += warp_pg[w];
  }
  const unsigned n_need = (unsigned)all_p, n_back = (unsigned)(all_p >> 32);
  // the step as a whole (the same decision in every thread of every CTA)
  int bad = (fault & 1) ? VKV_DEVERR_BAD_OFFSETS : fault ? VKV_DEVERR_NO_SPACE : 0;
  if (taken < 0 || returned < taken || returned - taken > p.n_ring ||
      (long long)n_back > p.n_ring - (returned - taken))
    bad = VKV_DEVERR_BAD_OFFSETS;
  else if (!bad && (all_t > p.max_tokens || (long long)n_need > returned - taken))
    bad = VKV_DEVERR_NO_SPACE;
  if (!bad) {  // counts to offsets; sums fit (all_t <= max_tokens, pages <= n_ring)
    int t = (int)base_t, a = (int)(unsigned)base_p, b = (int)(unsigned)(base_p >> 32);
    for (int r = r0; r < r1; ++r) {
      const int ct = tok[r], ca = need[r], cb = back[r];
      tok[r] = t;
      need[r] = a;
      back[r] = b;
      t += ct;
      a += ca;
      b += cb;
    }
    if (tid == 0) {
      tok[R] = (int)all_t;
      need[R] = (int)n_need;
      back[R] = (int)n_back;
    }
  }
  if constexpr (IN_PLACE) cluster_barrier();  // the grid is one cluster: every block has read what is updated
  else __syncthreads();
  const int n_thr = (int)gridDim.x * kMapThreads, me = (int)blockIdx.x * kMapThreads + tid;
  const int total = bad ? 0 : (int)all_t;
  if (me == 0) {
    if (bad && p.err) atomicCAS(p.err, 0, bad);
    p.ring_pos_out[0] = bad ? taken : taken + n_need;
    p.ring_pos_out[1] = bad ? returned : returned + n_back;
  }
  // a refused step's kv_len_out = kv_len: the lengths were not kept, and where the two are
  // one array there is nothing to do
  if (bad) {
    if (p.kv_len_out != p.kv_len)
      for (int r = me; r < R; r += n_thr) p.kv_len_out[r] = p.kv_len[r];
  } else {
    for (int r = me; r < R; r += n_thr) {
      const int add = tok[r + 1] - tok[r];
      // a row ends with new_len = -1; a free row that receives nothing stays free
      const bool gone = p.new_len[r] < 0 || (add == 0 && p.kv_len[r] < 0);
      p.kv_len_out[r] = gone ? -1 : held[r] + add;
    }
  }
  if (p.cu)
    for (int r = me; r <= R; r += n_thr) p.cu[r] = bad ? 0 : tok[r];
  // per step of a thread: one new table entry, one returned page and kTok tokens, whose
  // bisections and look-ups are all under way before the first result is needed
  const int taken_n = bad ? 0 : (int)n_need, back_n = bad ? 0 : (int)n_back;
  const int pages_n = max(taken_n, back_n);
  long long i0 = me;  // tokens i0, i0 + n_thr, ..
  for (long long at = me; at < pages_n || i0 < p.max_tokens; at += n_thr, i0 += (long long)kTok * n_thr) {
    int row[kTok], t[kTok], pg[kTok], rn = 0, rb = 0;
#pragma unroll
    for (int e = 0; e < kTok; ++e) row[e] = 0;
    for (int n = R; n > 1;) {  // the largest row with offset <= item
      const int half = n >> 1;
#pragma unroll
      for (int e = 0; e < kTok; ++e)
        if (tok[row[e] + half] <= i0 + (long long)e * n_thr) row[e] += half;
      if (need[rn + half] <= at) rn += half;
      if (back[rb + half] <= at) rb += half;
      n -= half;
    }
    int fresh = 0, gone = 0;
    if (at < taken_n) fresh = p.ring[ring_at(ring_t, (int)at, p.n_ring)];
    if (at < back_n) gone = p.table[rb * p.table_stride + ((int)at - back[rb])];
#pragma unroll
    for (int e = 0; e < kTok; ++e) {
      const long long i = i0 + (long long)e * n_thr;
      pg[e] = -1;
      if (i >= total) continue;
      const int r = row[e], h = held[r];
      t[e] = h + (int)(i - tok[r]);
      const int j = p.by_page(t[e]), had = pages_of(h);
      pg[e] = j < had ? p.table[r * p.table_stride + j]
                      : p.ring[ring_at(ring_t, need[r] + (j - had), p.n_ring)];
    }
    if (at < taken_n) p.table[rn * p.table_stride + pages_of(held[rn]) + ((int)at - need[rn])] = fresh;
    if (at < back_n) p.ring[ring_at(ring_b, (int)at, p.n_ring)] = gone;
#pragma unroll
    for (int e = 0; e < kTok; ++e) {
      const long long i = i0 + (long long)e * n_thr;
      if (i >= p.max_tokens) break;
      const bool in = i < total;
      p.slot[i] = in && pg[e] >= 0 ? (long long)pg[e] * page + (t[e] - p.by_page(t[e]) * page) : -1;
      if (p.row) p.row[i] = in ? row[e] : -1;
      if (p.pos) p.pos[i] = in ? t[e] : -1;
    }
  }
  griddep_launch_dependents();
}

}  // namespace
}  // namespace vkv

using namespace vkv;

extern "C" vkv_status vkv_page_map(const vkv_page_map_args* a, vkv_stream_t stream) {
  if (!a) return VKV_ERR_NULL;
  if (a->R < 1 || a->R > VKV_PAGE_MAX_ROWS || a->W < 1 || a->page < 1 || a->n_ring < 1 || a->max_tokens < 1)
    return VKV_ERR_SHAPE;
  if ((long long)a->R * a->W > INT_MAX || (long long)a->W * a->page > INT_MAX) return VKV_ERR_UNSUPPORTED;
  if (a->table_stride < a->W) return VKV_ERR_SHAPE;
  if (!a->kv_len || !a->new_len || !a->table || !a->ring || !a->ring_pos || !a->kv_len_out || !a->ring_pos_out ||
      !a->slot)
    return VKV_ERR_NULL;
  int dev = 0;
  const int n_sm = device_sm_count(&dev);
  if (n_sm <= 0) return VKV_ERR_CUDA;
  MapParams p;
  std::memset(&p, 0, sizeof(p));
  p.R = a->R;
  p.W = a->W;
  p.page = a->page;
  p.n_ring = a->n_ring;
  p.max_tokens = a->max_tokens;
  p.kv_len = a->kv_len;
  p.new_len = a->new_len;
  p.table = a->table;
  p.table_stride = a->table_stride;
  p.ring = a->ring;
  p.ring_pos = reinterpret_cast<const long long*>(a->ring_pos);
  p.kv_len_out = a->kv_len_out;
  p.ring_pos_out = reinterpret_cast<long long*>(a->ring_pos_out);
  p.slot = reinterpret_cast<long long*>(a->slot);
  p.row = a->row;
  p.pos = a->pos;
  p.cu = a->cu;
  p.err = a->err_word;
  p.by_page = fast_div(a->page);
  const bool in_place = a->kv_len == a->kv_len_out || a->ring_pos == a->ring_pos_out;
  const int most = in_place ? kMapMaxCluster : n_sm;
  // a thread per token, or per four pages that a step could move: their number is known on the
  // device alone, and a block too many costs less than a second look-up after the first (256 rows
  // of which 16 end, with 1000 pages in all: 7.1 us in one block, 4.9 in many)
  const long long pages = std::min<long long>((long long)a->R * a->W, a->n_ring);
  const long long items = std::max<long long>(std::max(a->max_tokens, a->R), pages / 4);
  const int ctas = (int)std::min<long long>(most, (items + kMapThreads - 1) / kMapThreads);
  const size_t smem = (size_t)(4 * a->R + 3) * sizeof(int);
  auto fn = in_place ? page_map_kernel<true> : page_map_kernel<false>;
  // the limit is the kernel's, whoever calls it: raised once per device, to the most any call takes (set to
  // each call's own need, it could fall below a larger call's on another thread, before that one's launch)
  static std::atomic<uint64_t> ready[2];  // by kernel: devices (by bit) on which it is raised
  std::atomic<uint64_t>& rd = ready[in_place ? 1 : 0];
  if (smem > 48 * 1024 && !(rd.load(std::memory_order_acquire) >> dev & 1u)) {
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (4 * VKV_PAGE_MAX_ROWS + 3) * (int)sizeof(int)) != cudaSuccess) {
      cudaGetLastError();
      return VKV_ERR_CUDA;
    }
    rd.fetch_or(1ull << dev, std::memory_order_release);
  }
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (!in_place || ctas == 1)  // one block needs no cluster (a cluster launch takes a microsecond more)
    return launch_ahead(fn, dim3((unsigned)ctas), dim3(kMapThreads), smem, st,
                        p) == cudaSuccess ? VKV_OK : VKV_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kMapThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)ctas;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, fn, p) != cudaSuccess) {
    cudaGetLastError();
    return VKV_ERR_CUDA;
  }
  return VKV_OK;
}
