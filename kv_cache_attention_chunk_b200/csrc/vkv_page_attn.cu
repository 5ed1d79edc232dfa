// vkv_page_attn: attention of one query per row over the row's paged cache.
//
// First form: one CTA per (row, query head).  Each of its warps takes every fourth
// visible token, the lanes share the head dimension, and each warp keeps a running
// maximum, sum and output; the warps' parts meet in shared memory.
#include <algorithm>
#include <climits>
#include <cstring>

#include "vkv_page.cuh"

namespace vkv {
namespace {

struct PageAttnParams {
  int R, H, Hkv, G, page, n_pages, W, sink, window, topk;
  float scale_log2;
  const void* q;
  long long q_sb, q_sh;
  void* o;
  long long o_sb, o_sh;
  const char* k;
  const char* v;
  long long k_sb, k_st, k_sh, v_sb, v_st, v_sh;  // bytes
  const int* table;
  long long table_stride;
  const int* kv_len;
  const int* sel;
  const float* ks;
  const float* vs;
  float* lse;
  int* err;
};

template <typename T>
__device__ __forceinline__ T from_float(float f);
template <>
__device__ __forceinline__ __nv_bfloat16 from_float(float f) { return __float2bfloat16_rn(f); }
template <>
__device__ __forceinline__ __half from_float(float f) { return __float2half_rn(f); }

template <typename T, bool E4M3>
__device__ __forceinline__ float elem(const char* row, int c) {
  if constexpr (E4M3) {
    const uint32_t h2 = e4m3x2_to_f16x2(reinterpret_cast<const uint8_t*>(row)[c]);
    return __low2float(*reinterpret_cast<const __half2*>(&h2));
  } else {
    return (float)reinterpret_cast<const T*>(row)[c];
  }
}

constexpr int kSimpleWarps = 4;

template <int D, typename T, bool E4M3>
__global__ void __launch_bounds__(kSimpleWarps * 32) page_attn_kernel(const PageAttnParams p) {
  constexpr int PL = D / 32;
  __shared__ float sm_m[kSimpleWarps], sm_l[kSimpleWarps], sm_o[kSimpleWarps][D];
  const int r = blockIdx.x / p.H, h = blockIdx.x - r * p.H, g = h / p.G;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int len = page_row_len(p.kv_len[r], p.W, p.page, p.err);
  if (len < 0) return;
  const T* q = reinterpret_cast<const T*>(p.q) + r * p.q_sb + h * p.q_sh;
  const float ks = (E4M3 && p.ks ? p.ks[g] : 1.f) * p.scale_log2, vs = E4M3 && p.vs ? p.vs[g] : 1.f;
  float qr[PL], acc[PL], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < PL; ++i) {
    qr[i] = (float)q[lane + 32 * i];
    acc[i] = 0.f;
  }
  const int* sel = p.sel ? p.sel + ((long long)r * p.Hkv + g) * p.topk : nullptr;
  const int lo = p.window > 0 ? min(p.sink, len) : len;
  const int gap = p.window > 0 ? max(0, len - p.window - lo) : 0;
  const long long count = p.sel ? (long long)p.topk * p.page : (long long)len - gap;
  for (long long x = warp; x < count; x += kSimpleWarps) {
    long long tok;
    if (sel) {
      const int j = sel[x / p.page];
      if (j < 0 || j >= p.W) {
        if (j != -1 && p.err && lane == 0) atomicCAS(p.err, 0, VKV_DEVERR_BAD_INDEX);
        continue;
      }
      tok = (long long)j * p.page + x % p.page;
      if (tok >= len) continue;
    } else {
      tok = x < lo ? x : x + gap;
    }
    const int pg = p.table[r * p.table_stride + tok / p.page];
    if (pg < 0 || pg >= p.n_pages) {
      if (p.err && lane == 0) atomicCAS(p.err, 0, VKV_DEVERR_BAD_INDEX);
      continue;
    }
    const char* kr = p.k + pg * p.k_sb + (tok % p.page) * p.k_st + g * p.k_sh;
    const char* vr = p.v + pg * p.v_sb + (tok % p.page) * p.v_st + g * p.v_sh;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < PL; ++i) s += qr[i] * elem<T, E4M3>(kr, lane + 32 * i);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    s *= ks;
    const float mn = fmaxf(m, s), ms = mn == -INFINITY ? 0.f : mn;
    const float a = exp2f(m - ms), w = exp2f(s - ms);
    m = mn;
    l = l * a + w;
#pragma unroll
    for (int i = 0; i < PL; ++i) acc[i] = acc[i] * a + w * elem<T, E4M3>(vr, lane + 32 * i);
  }
  if (lane == 0) {
    sm_m[warp] = m;
    sm_l[warp] = l;
  }
#pragma unroll
  for (int i = 0; i < PL; ++i) sm_o[warp][lane + 32 * i] = acc[i];
  __syncthreads();
  float M = -INFINITY, L = 0.f;
#pragma unroll
  for (int w = 0; w < kSimpleWarps; ++w) M = fmaxf(M, sm_m[w]);
  const float Ms = M == -INFINITY ? 0.f : M;
#pragma unroll
  for (int w = 0; w < kSimpleWarps; ++w) L += sm_l[w] * exp2f(sm_m[w] - Ms);
  T* o = reinterpret_cast<T*>(p.o) + r * p.o_sb + h * p.o_sh;
  for (int c = threadIdx.x; c < D; c += kSimpleWarps * 32) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < kSimpleWarps; ++w) t += sm_o[w][c] * exp2f(sm_m[w] - Ms);
    o[c] = from_float<T>(L == 0.f ? 0.f : t / L * vs);
  }
  if (threadIdx.x == 0) p.lse[(size_t)r * p.H + h] = L == 0.f ? -INFINITY : (Ms + log2f(L)) * 0.69314718055994531f;
}

template <int D, typename T, bool E4M3>
cudaError_t launch(const PageAttnParams& p, cudaStream_t st) {
  page_attn_kernel<D, T, E4M3><<<(unsigned)(p.R * p.H), kSimpleWarps * 32, 0, st>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const PageAttnParams& p, int q_dtype, int kv_dtype, cudaStream_t st) {
  if (kv_dtype == VKV_E4M3)
    return q_dtype == VKV_BF16 ? launch<D, __nv_bfloat16, true>(p, st) : launch<D, __half, true>(p, st);
  return q_dtype == VKV_BF16 ? launch<D, __nv_bfloat16, false>(p, st) : launch<D, __half, false>(p, st);
}

}  // namespace
}  // namespace vkv

using namespace vkv;

extern "C" size_t vkv_page_attn_workspace_size(int32_t H, int32_t Hkv, int32_t d) {
  if (H < 1 || Hkv < 1 || H % Hkv || (d != 64 && d != 128)) return 0;
  return 256;
}

extern "C" vkv_status vkv_page_attn(const vkv_page_attn_args* a, vkv_stream_t stream) {
  if (!a) return VKV_ERR_NULL;
  if (a->d != 64 && a->d != 128) return VKV_ERR_UNSUPPORTED;
  if (a->q_dtype != VKV_BF16 && a->q_dtype != VKV_FP16) return VKV_ERR_UNSUPPORTED;
  if (a->kv_dtype != a->q_dtype && a->kv_dtype != VKV_E4M3) return VKV_ERR_UNSUPPORTED;
  if (a->R < 1 || a->R > VKV_PAGE_MAX_ROWS || a->H < 1 || a->Hkv < 1 || a->H % a->Hkv || a->page < 1 ||
      a->n_pages < 1 || a->W < 1 || a->sink < 0 || a->window < 0 || a->table_stride < a->W)
    return VKV_ERR_SHAPE;
  if (!(a->scale > 0.f) || a->scale > 3.0e38f) return VKV_ERR_SHAPE;
  if (a->sel ? (a->topk < 1 || a->window != 0) : a->topk != 0) return VKV_ERR_SHAPE;
  if ((long long)a->R * a->W > INT_MAX || (long long)a->W * a->page > INT_MAX || a->H > 4096 ||
      (long long)a->topk * a->page > INT_MAX)
    return VKV_ERR_UNSUPPORTED;
  if (a->kv_dtype != VKV_E4M3 && (a->k_scale || a->v_scale)) return VKV_ERR_UNSUPPORTED;
  if (!a->q.ptr || !a->o.ptr || !a->k.ptr || !a->v.ptr || !a->table || !a->kv_len || !a->lse) return VKV_ERR_NULL;
  vkv_tensor q = a->q, o = a->o;
  q.st = o.st = 0;
  if (!page_tensor_aligned(q, a->q_dtype) || !page_tensor_aligned(o, a->q_dtype) ||
      !page_tensor_aligned(a->k, a->kv_dtype) || !page_tensor_aligned(a->v, a->kv_dtype))
    return VKV_ERR_ALIGN;
  int dev = 0;
  if (device_sm_count(&dev) <= 0) return VKV_ERR_CUDA;
  const size_t need = vkv_page_attn_workspace_size(a->H, a->Hkv, a->d);
  if (!a->workspace || a->workspace_bytes < need) return VKV_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(a->workspace) & 255u) return VKV_ERR_ALIGN;
  PageAttnParams p;
  std::memset(&p, 0, sizeof(p));
  p.R = a->R; p.H = a->H; p.Hkv = a->Hkv; p.G = a->H / a->Hkv;
  p.page = a->page; p.n_pages = a->n_pages; p.W = a->W; p.sink = a->sink; p.window = a->window; p.topk = a->topk;
  p.scale_log2 = a->scale * 1.4426950408889634f;
  p.q = a->q.ptr; p.q_sb = a->q.sb; p.q_sh = a->q.sh;
  p.o = a->o.ptr; p.o_sb = a->o.sb; p.o_sh = a->o.sh;
  const int e = dtype_bytes(a->kv_dtype);
  p.k = reinterpret_cast<const char*>(a->k.ptr);
  p.v = reinterpret_cast<const char*>(a->v.ptr);
  p.k_sb = a->k.sb * e; p.k_st = a->k.st * e; p.k_sh = a->k.sh * e;
  p.v_sb = a->v.sb * e; p.v_st = a->v.st * e; p.v_sh = a->v.sh * e;
  p.table = a->table; p.table_stride = a->table_stride;
  p.kv_len = a->kv_len;
  p.sel = a->sel;
  p.ks = a->k_scale; p.vs = a->v_scale;
  p.lse = a->lse;
  p.err = a->err_word;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t rc = a->d == 128 ? launch_d<128>(p, a->q_dtype, a->kv_dtype, st)
                                     : launch_d<64>(p, a->q_dtype, a->kv_dtype, st);
  return rc == cudaSuccess ? VKV_OK : VKV_ERR_CUDA;
}
