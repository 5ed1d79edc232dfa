// vkv_page_append: keys and values of a step's tokens into the pages of the cache, in
// the cache's element type, and the key means of the pages written to (the pages'
// representatives, Sparse Forcing summary section 2 component 2, kept as tokens arrive).
//
// Bandwidth-bound: each row is read once and written once.  16-byte chunks (8 values)
// per thread, all of a thread's loads issued before its first store.
#include <algorithm>
#include <cstring>

#include "vkv_page.cuh"

namespace vkv {
namespace {

struct AppendParams {
  int T, Hkv, page;
  long long n_slots;
  const uint4* kn;
  const uint4* vn;
  long long kn_st, kn_sh, vn_st, vn_sh;  // in 16-byte chunks of the input
  char* k;
  char* v;
  long long k_sb, k_st, k_sh, v_sb, v_st, v_sh;  // in bytes
  const long long* slot;
  const float* ks;
  const float* vs;
  float* kbar;
  int* err;
};

// One stored chunk: the bytes that go to the cache, and (for the mean) their values.
template <typename IN, bool E4M3>
__device__ __forceinline__ void store_chunk(char* dst, const uint4 x, float scale, float* val) {
  if constexpr (E4M3) {
    float f[8];
    unpack8<IN>(x, f);
    uint32_t w[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t lo = f32x2_to_e4m3x2(__fdiv_rn(f[4 * e], scale), __fdiv_rn(f[4 * e + 1], scale));
      const uint32_t hi = f32x2_to_e4m3x2(__fdiv_rn(f[4 * e + 2], scale), __fdiv_rn(f[4 * e + 3], scale));
      w[e] = lo | (hi << 16);
    }
    *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    if (val) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t h2 = e4m3x2_to_f16x2(w[e >> 1] >> (16 * (e & 1)));
        const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&h2));
        val[2 * e] = p.x;
        val[2 * e + 1] = p.y;
      }
    }
  } else {
    *reinterpret_cast<uint4*>(dst) = x;
    if (val) unpack8<IN>(x, val);
  }
}

// Eight stored values of a cache row.
template <typename IN, bool E4M3>
__device__ __forceinline__ void load_chunk(const char* src, float* val) {
  if constexpr (E4M3) {
    const uint2 u = *reinterpret_cast<const uint2*>(src);
    const uint32_t w[2] = {u.x, u.y};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t h2 = e4m3x2_to_f16x2(w[e >> 1] >> (16 * (e & 1)));
      const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&h2));
      val[2 * e] = p.x;
      val[2 * e + 1] = p.y;
    }
  } else {
    unpack8<IN>(*reinterpret_cast<const uint4*>(src), val);
  }
}

// Without means: thread = one chunk column (head, chunk) of kRows consecutive tokens.
// grid: x = token groups, y = column blocks of up to 256 threads.
constexpr int kAppendRows = 4;

template <int D, typename IN, bool E4M3>
__global__ void __launch_bounds__(256) append_kernel(const AppendParams p) {
  constexpr int CPR = D / 8;
  constexpr int OB = E4M3 ? 8 : 16;  // bytes of a stored chunk
  const int col = blockIdx.y * blockDim.x + threadIdx.x;
  if (col >= p.Hkv * CPR) return;
  const int h = col / CPR, c = col % CPR;
  const int i0 = blockIdx.x * kAppendRows;
  const float ks = E4M3 && p.ks ? p.ks[h] : 1.f, vs = E4M3 && p.vs ? p.vs[h] : 1.f;
  long long s[kAppendRows];
  uint4 kx[kAppendRows], vx[kAppendRows];
#pragma unroll
  for (int e = 0; e < kAppendRows; ++e) {
    const int i = i0 + e;
    s[e] = i < p.T ? p.slot[i] : -1;
    if (i < p.T) {
      kx[e] = __ldcs(p.kn + i * p.kn_st + h * p.kn_sh + c);
      vx[e] = __ldcs(p.vn + i * p.vn_st + h * p.vn_sh + c);
    }
  }
#pragma unroll
  for (int e = 0; e < kAppendRows; ++e) {
    if (s[e] < 0) continue;
    if (s[e] >= p.n_slots) {
      if (p.err) atomicCAS(p.err, 0, VKV_DEVERR_BAD_INDEX);
      continue;
    }
    const long long pg = s[e] / p.page, off = s[e] - pg * p.page;
    store_chunk<IN, E4M3>(p.k + pg * p.k_sb + off * p.k_st + h * p.k_sh + c * OB, kx[e], ks, nullptr);
    store_chunk<IN, E4M3>(p.v + pg * p.v_sb + off * p.v_st + h * p.v_sh + c * OB, vx[e], vs, nullptr);
  }
}

// With means: a CTA (128 threads) takes the runs that start among `slab` consecutive
// tokens, for one head.  A run is a page's tokens of this call (consecutive slots of one
// page).  The CTA's row groups (D/8 lanes each, one row per group and pass) first add the
// page's earlier rows, read from the cache, then copy the run's rows and add what they
// store; the groups' sums meet in shared memory, in a fixed order.
constexpr int kMeanThreads = 128;

template <int D, typename IN, bool E4M3>
__global__ void __launch_bounds__(kMeanThreads) append_mean_kernel(const AppendParams p, int slab) {
  constexpr int CPR = D / 8;
  constexpr int GROUPS = kMeanThreads / CPR;
  constexpr int OB = E4M3 ? 8 : 16;
  constexpr int U = 4;  // rows of a thread in flight
  __shared__ float part[GROUPS][D];
  const int h = blockIdx.y;
  const int c = threadIdx.x % CPR, g = threadIdx.x / CPR;
  const float ks = E4M3 && p.ks ? p.ks[h] : 1.f, vs = E4M3 && p.vs ? p.vs[h] : 1.f;
  const long long i_end = min((long long)p.T, ((long long)blockIdx.x + 1) * slab);
  for (long long i = (long long)blockIdx.x * slab; i < i_end; ++i) {
    const long long s0 = p.slot[i];
    if (s0 < 0) continue;
    if (s0 >= p.n_slots) {
      if (p.err) atomicCAS(p.err, 0, VKV_DEVERR_BAD_INDEX);
      continue;
    }
    const long long pg = s0 / p.page;
    const int off = (int)(s0 - pg * p.page);
    if (i > 0 && off > 0 && p.slot[i - 1] == s0 - 1) continue;  // inside a run that started before
    // the run's length: consecutive slots up to the page's end
    const int most = (int)min((long long)(p.page - off), (long long)p.T - i);
    int n = 1;
    for (int t0 = 1; t0 < most; t0 += 32) {
      const int t = t0 + (threadIdx.x & 31);
      const bool in = t < most && p.slot[i + t] == s0 + t;
      const unsigned b = __ballot_sync(0xFFFFFFFFu, in);
      const int run = __ffs(~b) == 0 ? 32 : __ffs(~b) - 1;
      n += run;
      if (run < 32) break;
    }
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
    const char* kp = p.k + pg * p.k_sb + h * p.k_sh + c * OB;
    for (int r0 = g; r0 < off; r0 += GROUPS * U) {  // the page's earlier rows
      float f[U][8];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 + u * GROUPS;
        if (r < off) {
          load_chunk<IN, E4M3>(kp + r * p.k_st, f[u]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) f[u][e] = 0.f;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += f[u][e];
    }
    char* kd = p.k + pg * p.k_sb + off * p.k_st + h * p.k_sh + c * OB;
    char* vd = p.v + pg * p.v_sb + off * p.v_st + h * p.v_sh + c * OB;
    for (int r0 = g; r0 < n; r0 += GROUPS * U) {
      uint4 kx[U], vx[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 + u * GROUPS;
        if (r < n) {
          kx[u] = __ldcs(p.kn + (i + r) * p.kn_st + h * p.kn_sh + c);
          vx[u] = __ldcs(p.vn + (i + r) * p.vn_st + h * p.vn_sh + c);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = r0 + u * GROUPS;
        if (r < n) {
          float f[8];
          store_chunk<IN, E4M3>(kd + r * p.k_st, kx[u], ks, f);
          store_chunk<IN, E4M3>(vd + r * p.v_st, vx[u], vs, nullptr);
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] += f[e];
        }
      }
    }
    __syncthreads();  // the previous run's sums have been read
#pragma unroll
    for (int e = 0; e < 8; ++e) part[g][c * 8 + e] = acc[e];
    __syncthreads();
    const float rows = (float)(off + n);
    for (int x = threadIdx.x; x < D; x += kMeanThreads) {
      float t = 0.f;
#pragma unroll
      for (int gg = 0; gg < GROUPS; ++gg) t += part[gg][x];
      p.kbar[(pg * p.Hkv + h) * D + x] = __fdiv_rn(t, rows) * ks;
    }
  }
}

template <int D, typename IN, bool E4M3>
cudaError_t launch(const AppendParams& p, int n_sm, cudaStream_t st) {
  if (p.kbar) {
    // few tokens: one run start per CTA; many: as many as leave about 16 CTAs per SM
    const long long want = 16ll * n_sm;
    const int slab = (int)std::min<long long>(32, std::max<long long>(1, (long long)p.T * p.Hkv / want));
    const dim3 grid((unsigned)((p.T + slab - 1) / slab), (unsigned)p.Hkv);
    append_mean_kernel<D, IN, E4M3><<<grid, kMeanThreads, 0, st>>>(p, slab);
  } else {
    const int cols = p.Hkv * (D / 8), n_cb = (cols + 255) / 256;
    const int width = (((cols + n_cb - 1) / n_cb) + 31) / 32 * 32;
    const dim3 grid((unsigned)((p.T + kAppendRows - 1) / kAppendRows), (unsigned)n_cb);
    append_kernel<D, IN, E4M3><<<grid, width, 0, st>>>(p);
  }
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const AppendParams& p, int x_dtype, int kv_dtype, int n_sm, cudaStream_t st) {
  if (kv_dtype == VKV_E4M3)
    return x_dtype == VKV_BF16 ? launch<D, __nv_bfloat16, true>(p, n_sm, st) : launch<D, __half, true>(p, n_sm, st);
  return x_dtype == VKV_BF16 ? launch<D, __nv_bfloat16, false>(p, n_sm, st) : launch<D, __half, false>(p, n_sm, st);
}

}  // namespace
}  // namespace vkv

using namespace vkv;

extern "C" vkv_status vkv_page_append(const vkv_page_append_args* a, vkv_stream_t stream) {
  if (!a) return VKV_ERR_NULL;
  if (a->d != 64 && a->d != 128) return VKV_ERR_UNSUPPORTED;
  if (a->x_dtype != VKV_BF16 && a->x_dtype != VKV_FP16) return VKV_ERR_UNSUPPORTED;
  if (a->kv_dtype != a->x_dtype && a->kv_dtype != VKV_E4M3) return VKV_ERR_UNSUPPORTED;
  if (a->T < 0 || a->T > (1 << 30) || a->Hkv < 1 || a->page < 1 || a->n_pages < 1) return VKV_ERR_SHAPE;
  if (a->Hkv > 4096) return VKV_ERR_UNSUPPORTED;
  if (a->kv_dtype != VKV_E4M3 && (a->k_scale || a->v_scale)) return VKV_ERR_UNSUPPORTED;
  if (!a->k.ptr || !a->v.ptr || (a->T > 0 && (!a->k_new.ptr || !a->v_new.ptr || !a->slot))) return VKV_ERR_NULL;
  if (!page_tensor_aligned(a->k, a->kv_dtype) || !page_tensor_aligned(a->v, a->kv_dtype)) return VKV_ERR_ALIGN;
  if (a->T > 0) {
    vkv_tensor kn = a->k_new, vn = a->v_new;
    kn.sb = vn.sb = 0;
    if (!page_tensor_aligned(kn, a->x_dtype) || !page_tensor_aligned(vn, a->x_dtype)) return VKV_ERR_ALIGN;
  }
  if (reinterpret_cast<uintptr_t>(a->kbar) & 15u) return VKV_ERR_ALIGN;
  int dev = 0;
  const int n_sm = device_sm_count(&dev);
  if (n_sm <= 0) return VKV_ERR_CUDA;
  if (a->T == 0) return VKV_OK;
  AppendParams p;
  std::memset(&p, 0, sizeof(p));
  p.T = a->T;
  p.Hkv = a->Hkv;
  p.page = a->page;
  p.n_slots = (long long)a->n_pages * a->page;
  p.kn = reinterpret_cast<const uint4*>(a->k_new.ptr);
  p.vn = reinterpret_cast<const uint4*>(a->v_new.ptr);
  p.kn_st = a->k_new.st / 8; p.kn_sh = a->k_new.sh / 8;
  p.vn_st = a->v_new.st / 8; p.vn_sh = a->v_new.sh / 8;
  const int e = dtype_bytes(a->kv_dtype);
  p.k = reinterpret_cast<char*>(a->k.ptr);
  p.v = reinterpret_cast<char*>(a->v.ptr);
  p.k_sb = a->k.sb * e; p.k_st = a->k.st * e; p.k_sh = a->k.sh * e;
  p.v_sb = a->v.sb * e; p.v_st = a->v.st * e; p.v_sh = a->v.sh * e;
  p.slot = reinterpret_cast<const long long*>(a->slot);
  p.ks = a->k_scale;
  p.vs = a->v_scale;
  p.kbar = a->kbar;
  p.err = a->err_word;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t rc = a->d == 128 ? launch_d<128>(p, a->x_dtype, a->kv_dtype, n_sm, st)
                                     : launch_d<64>(p, a->x_dtype, a->kv_dtype, n_sm, st);
  return rc == cudaSuccess ? VKV_OK : VKV_ERR_CUDA;
}
