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
  int T, Hkv, page, slab;
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

// x / s, correctly rounded: the product with r = 1/s (rounded once) corrected by its exact
// remainder (Markstein, Computation of elementary functions on the IBM RISC System/6000
// processor, 1990), two values an instruction, where a division takes about ten.  Chunks with
// infinities or quotients that could pass 1e30, and s outside [2^-60, 2^60], where remainders
// could underflow, are divided.
// Both work on -x and give (-x) (-r) corrected by (q s - x) (-r): an exact remainder is +0
// whatever the signs of its terms, and with these the quotient -0 of x = -0 stays -0 where x r
// corrected by (x - q s) r would become +0 (s > 0; a scale below zero is divided by as well).
struct Divisor {
  float s, r;       // the scale, -1 / scale
  uint64_t s2, r2;  // the same, twice each
  bool plain;
  __device__ __forceinline__ explicit Divisor(float scale) {
    s = scale;
    r = __fdiv_rn(-1.f, scale);
    s2 = pack2f(s, s);
    r2 = pack2f(r, r);
    plain = !(scale >= 0x1p-60f && scale <= 0x1p60f);
  }
  template <typename IN>
  __device__ __forceinline__ void operator()(const uint4 x, float* f) const {
    constexpr uint32_t kSigns = 0x80008000u;
    unpack8<IN>(make_uint4(x.x ^ kSigns, x.y ^ kSigns, x.z ^ kSigns, x.w ^ kSigns), f);
    // the largest magnitude (NaN aside): the sign-free patterns are ordered like the values
    const uint32_t m01 = __vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu), m23 = __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu);
    const uint32_t m = __vmaxu2(m01, m23);
    float top;
    {
      const uint32_t h = max(m >> 16, m & 0xFFFFu);
      float t[8];
      unpack8<IN>(make_uint4(h, 0u, 0u, 0u), t);
      top = t[0];
    }
    if (plain || !(top * fabsf(r) < 1e30f)) {
#pragma unroll 1
      for (int e = 0; e < 8; ++e) {  // rotates, so that no register is indexed
        const float t = __fdiv_rn(f[0], -s);
#pragma unroll
        for (int k = 0; k < 7; ++k) f[k] = f[k + 1];
        f[7] = t;
      }
      return;
    }
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const uint64_t v = pack2f(f[e], f[e + 1]), q = mul2f(v, r2);
      unpack2f(fma2f(fma2f(q, s2, v), r2, q), f[e], f[e + 1]);
    }
  }
};

// One stored chunk: the bytes that go to the cache, and (for the mean) their values.
template <typename IN, bool E4M3>
__device__ __forceinline__ void store_chunk(char* dst, const uint4 x, const Divisor& by, float* val) {
  if constexpr (E4M3) {
    float f[8];
    by.template operator()<IN>(x, f);
    uint32_t w[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t lo = f32x2_to_e4m3x2(f[4 * e], f[4 * e + 1]);
      const uint32_t hi = f32x2_to_e4m3x2(f[4 * e + 2], f[4 * e + 3]);
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

// Eight stored values of a cache row: as they lie there, and as fp32.
template <bool E4M3>
struct Raw { using type = uint4; };
template <>
struct Raw<true> { using type = uint2; };
template <typename IN>
__device__ __forceinline__ void add_raw(const uint4 x, float* acc) {
  float f[8];
  unpack8<IN>(x, f);
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] += f[e];
}
template <typename IN>
__device__ __forceinline__ void add_raw(const uint2 x, float* acc) {
  const uint32_t w[2] = {x.x, x.y};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t h2 = e4m3x2_to_f16x2(w[e >> 1] >> (16 * (e & 1)));
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h2));
    acc[2 * e] += v.x;
    acc[2 * e + 1] += v.y;
  }
}

// Without means: thread = one chunk column (head, chunk) of kRows consecutive tokens.
// grid: x = token groups, y = column blocks of up to 256 threads.
constexpr int kAppendRows = 4;

template <int D, typename IN, bool E4M3>
__global__ void __launch_bounds__(256) append_kernel(const AppendParams p) {
  griddep_wait();
  constexpr int CPR = D / 8;
  constexpr int OB = E4M3 ? 8 : 16;  // bytes of a stored chunk
  const int col = blockIdx.y * blockDim.x + threadIdx.x;
  if (col >= p.Hkv * CPR) return;
  const int h = col / CPR, c = col % CPR;
  const int i0 = blockIdx.x * kAppendRows;
  const float ks = E4M3 && p.ks ? p.ks[h] : 1.f, vs = E4M3 && p.vs ? p.vs[h] : 1.f;
  const Divisor by_k(ks), by_v(vs);
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
    store_chunk<IN, E4M3>(p.k + pg * p.k_sb + off * p.k_st + h * p.k_sh + c * OB, kx[e], by_k, nullptr);
    store_chunk<IN, E4M3>(p.v + pg * p.v_sb + off * p.v_st + h * p.v_sh + c * OB, vx[e], by_v, nullptr);
  }
  griddep_launch_dependents();
}

// With means: a warp takes the runs that start among `slab` (<= 32) consecutive tokens, for
// one head; the block's warps take neighbouring heads, whose rows lie side by side.  A run is
// a page's tokens of this call (consecutive slots of one page).  The warp's lane groups (D/8
// lanes each, one row per group and load, kRun loads in flight) first add the page's earlier
// rows, read from the cache, then copy the run's rows and add what they store; the groups'
// sums meet by shuffles, in a fixed order.  SPLIT: the block's four warps share each run of one
// head instead, and meet in shared memory: for calls of few runs (64 rows' next tokens: 4.1
// us against 5.5 us) and pages of many tokens.
constexpr int kMeanWarps = 4;
constexpr int kRun = 4;

template <int D, typename IN, bool E4M3, bool SPLIT>
__global__ void __launch_bounds__(kMeanWarps * 32, 5) append_mean_kernel(const AppendParams p) {
  constexpr int CPR = D / 8;
  constexpr int GROUPS = 32 / CPR * (SPLIT ? kMeanWarps : 1);  // rows at a time
  constexpr int OB = E4M3 ? 8 : 16;
  __shared__ float part[SPLIT ? kMeanWarps : 1][D];
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = SPLIT ? blockIdx.y : blockIdx.y * kMeanWarps + warp;
  if (h >= p.Hkv) return;
  const int c = lane % CPR, g = (SPLIT ? threadIdx.x : lane) / CPR;
  const float ks = E4M3 && p.ks ? p.ks[h] : 1.f, vs = E4M3 && p.vs ? p.vs[h] : 1.f;
  const Divisor by_k(ks), by_v(vs);
  const long long i0 = (long long)blockIdx.x * p.slab;
  const int n_tok = (int)min((long long)p.slab, p.T - i0);
  const long long s = lane < n_tok ? p.slot[i0 + lane] : -1;
  const long long prev = lane < n_tok && i0 + lane > 0 ? p.slot[i0 + lane - 1] : -2;
  const bool bad = s >= p.n_slots;
  if (bad && h == 0 && p.err) atomicCAS(p.err, 0, VKV_DEVERR_BAD_INDEX);
  const bool ok = s >= 0 && !bad;
  const long long page_l = ok ? (s >> 32 ? s / p.page : (long long)((uint32_t)s / (uint32_t)p.page)) : 0;
  const int off_l = ok ? (int)(s - page_l * p.page) : 0;
  unsigned starts = __ballot_sync(0xFFFFFFFFu, ok && !(off_l > 0 && prev == s - 1));
#pragma unroll 1
  for (; starts; starts &= starts - 1) {
    const int b = __ffs(starts) - 1;
    const long long i = i0 + b, s0 = __shfl_sync(0xFFFFFFFFu, s, b), pg = __shfl_sync(0xFFFFFFFFu, page_l, b);
    const int off = __shfl_sync(0xFFFFFFFFu, off_l, b);
    // the run's length: consecutive slots up to the page's end, in the slab and behind it
    const int most = (int)min((long long)(p.page - off), (long long)p.T - i);
    const unsigned in = __ballot_sync(0xFFFFFFFFu, lane >= b && lane - b < most && s == s0 + (lane - b)) >> b;
    int n = in == 0xFFFFFFFFu ? 32 : __ffs(~in) - 1;
    if (b + n == n_tok) {
      while (n < most) {
        const unsigned more = __ballot_sync(0xFFFFFFFFu, n + lane < most && p.slot[i + n + lane] == s0 + n + lane);
        const int run = more == 0xFFFFFFFFu ? 32 : __ffs(~more) - 1;
        n += run;
        if (run < 32) break;
      }
    }
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
    // row pointers advance by additions: products for every row in flight would fill the registers
    const char* kp = p.k + pg * p.k_sb + g * p.k_st + h * p.k_sh + c * OB;
    const long long k_step = GROUPS * p.k_st, v_step = GROUPS * p.v_st;
    for (int r0 = g; r0 < off; r0 += GROUPS * kRun) {  // the page's earlier rows
      typename Raw<E4M3>::type x[kRun];
#pragma unroll
      for (int u = 0; u < kRun; ++u) {
        if (r0 + u * GROUPS < off) x[u] = *reinterpret_cast<const typename Raw<E4M3>::type*>(kp);
        kp += k_step;
      }
#pragma unroll
      for (int u = 0; u < kRun; ++u)
        if (r0 + u * GROUPS < off) add_raw<IN>(x[u], acc);
    }
    char* kd = p.k + pg * p.k_sb + (off + g) * p.k_st + h * p.k_sh + c * OB;
    char* vd = p.v + pg * p.v_sb + (off + g) * p.v_st + h * p.v_sh + c * OB;
    const uint4* kn = p.kn + (i + g) * p.kn_st + h * p.kn_sh + c;
    const uint4* vn = p.vn + (i + g) * p.vn_st + h * p.vn_sh + c;
    const long long kn_step = GROUPS * p.kn_st, vn_step = GROUPS * p.vn_st;
    for (int r0 = g; r0 < n; r0 += GROUPS * kRun) {
      uint4 kx[kRun], vx[kRun];
#pragma unroll
      for (int u = 0; u < kRun; ++u) {
        if (r0 + u * GROUPS < n) {
          kx[u] = __ldcs(kn);
          vx[u] = __ldcs(vn);
        }
        kn += kn_step;
        vn += vn_step;
      }
#pragma unroll
      for (int u = 0; u < kRun; ++u) {
        if (r0 + u * GROUPS < n) {
          float f[8];
          store_chunk<IN, E4M3>(kd, kx[u], by_k, f);
          store_chunk<IN, E4M3>(vd, vx[u], by_v, nullptr);
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] += f[e];
        }
        kd += k_step;
        vd += v_step;
      }
    }
#pragma unroll
    for (int o = CPR; o < 32; o <<= 1)
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += __shfl_xor_sync(0xFFFFFFFFu, acc[e], o);
    if constexpr (SPLIT) {  // the warps' sums, in their order
      __syncthreads();  // the last run's have been read
      if (lane < CPR) {
#pragma unroll
        for (int e = 0; e < 8; ++e) part[warp][c * 8 + e] = acc[e];
      }
      __syncthreads();
      if (g == 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          acc[e] = part[0][c * 8 + e];
#pragma unroll
          for (int w = 1; w < kMeanWarps; ++w) acc[e] += part[w][c * 8 + e];
        }
      }
    }
    if (g == 0) {
      const float rows = (float)(off + n);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = __fdiv_rn(acc[e], rows) * ks;
      float4* dst = reinterpret_cast<float4*>(p.kbar + (pg * p.Hkv + h) * D + c * 8);
      dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
    }
  }
  griddep_launch_dependents();
}

template <int D, typename IN, bool E4M3>
cudaError_t launch(AppendParams& p, int n_sm, cudaStream_t st) {
  if (p.kbar) {
    // four warps per run where runs are few or long (pages of 64 tokens: 29.2 against 31.0 us for
    // 17000 tokens; of 16 tokens, e4m3, 27.9 against 19.2 us, for half of the lanes have no row); tokens per
    // block so that about `warps` warps per SM have one
    const bool split = (long long)p.T * p.Hkv <= 8ll * n_sm || p.page >= 64;
    const long long warps = split ? 16 : 64;
    p.slab = (int)std::min<long long>(32, std::max<long long>(1, (long long)p.T * p.Hkv / (warps * n_sm)));
    const dim3 grid((unsigned)((p.T + p.slab - 1) / p.slab), (unsigned)(split ? p.Hkv : (p.Hkv + kMeanWarps - 1) / kMeanWarps));
    return launch_ahead(split ? append_mean_kernel<D, IN, E4M3, true> : append_mean_kernel<D, IN, E4M3, false>, grid,
                        dim3(kMeanWarps * 32), 0, st, p);
  } else {
    const int cols = p.Hkv * (D / 8), n_cb = (cols + 255) / 256;
    const int width = (((cols + n_cb - 1) / n_cb) + 31) / 32 * 32;
    const dim3 grid((unsigned)((p.T + kAppendRows - 1) / kAppendRows), (unsigned)n_cb);
    return launch_ahead(append_kernel<D, IN, E4M3>, grid, dim3((unsigned)width), 0, st, p);
  }
}

template <int D>
cudaError_t launch_d(AppendParams& p, int x_dtype, int kv_dtype, int n_sm, cudaStream_t st) {
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
  // the loops over a page's rows step up to 64 past the last
  if (a->Hkv > 4096 || a->page > (1 << 30)) return VKV_ERR_UNSUPPORTED;
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
