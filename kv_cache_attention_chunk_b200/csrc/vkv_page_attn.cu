// vkv_page_attn: attention of one query per row over the row's paged cache.
//
//   s_t = scale <q_h, k_t>,  o = sum_t 2^(c s_t - m) v_t / sum_t 2^(c s_t - m),  c = scale log2 e
//
// Every cached byte is used by the G = H / Hkv queries that share its head and by nothing
// else: 4 G flops per 16-bit key-value pair of numbers, far below what the tensor cores
// could do meanwhile, so HBM bounds the call and the kernel is built as a stream.
//
// Work: the visible tokens of a (row, key head, chunk of up to 16 query heads) are a unit,
// cut into tiles of TT tokens; all units' tiles form one line, which is dealt out to the
// warps of a grid of two or three blocks per SM in equal contiguous shares.  So rows of any
// length mix, one long row fills the GPU, and no host code needs the lengths.  Short calls are
// latencies, and joins are the longest of them: there the line is made of blocks, whole ones
// for each unit, so that no block has parts of two units to join one after the other.  Each warp streams
// its own share through a private ring of cp.async stages (K and V of a tile, addresses from
// the block table, masked tokens zero-filled); warps never wait for one another until the
// end.  A unit within one warp's share is finished there.  A unit cut by shares leaves its
// parts (m, l, O) in shared memory, one block joins its own, and parts of a unit that spans
// blocks go to the workspace, where the block that arrives last joins them, in block order:
// no atomics on data, equal inputs give equal bits.
//
// Arithmetic: S^T = K Q^T and O^T = V^T P^T by m16n8k16 instructions: the many tokens (and
// the d output channels) fill the 16-wide side, the few heads the 8-wide one.  16-bit
// caches multiply in their own type; an 8-bit cache is widened to f16 (exact), with bf16
// queries first scaled by a power of two of each head so that they fit f16: what that
// drops is below 2^-38 of the head's largest query element.  The weights P go in as two
// 16-bit parts (value and remainder), so that no rounding of P to 16 bits is left; sums and
// outputs are fp32.  The running maximum only moves when a score exceeds it by 2^4.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cstring>
#include <type_traits>

#include "vkv_page.cuh"

namespace vkv {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxBlocksPerSm = 3;
constexpr int kMaxBlocks = kMaxBlocksPerSm * kMaxCtas;
constexpr float kSlack = 4.f;  // log2: how far a score may exceed the running maximum
// The least share of a warp, tiles: a share of t tiles takes t times a tile's time and leaves
// (tiles of the unit) / t parts to join, so the best t grows with the root of the unit's tiles
// (one row of 131072 tokens, one head: 36 us with this factor, 40 with its double, 54 with 4 tiles
// throughout)
constexpr int kMinTiles = 2;
constexpr float kShareRoot = 0.045f;
// Calls of at most this many tiles per warp give each unit whole blocks (two rows of 520 tokens,
// 8 key heads of 64 channels: 8.8 us, on the line 16.7; one row of 1560 tokens 11.0 and 12.7; above
// it equal shares count for more)
constexpr int kWholeMost = 8;

struct PageAttnParams {
  int R, H, Hkv, G, page, n_pages, W, sink, window, topk;
  FastDiv by_page;
  int n_chunks;                 // chunks of query heads per key head
  int pair;                     // 1: the line's heads are pairs of key heads (see launch), else 0
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
  int* counters;  // [blocks][2]
  float* ws_ml;   // [blocks][2][2][heads of a chunk][2]: maximum, sum
  float* ws_o;    // [blocks][2][2][heads of a chunk][d]
  float* ws_first;  // [warps][8 or 16 heads][d + 4]: the parts of shares' first units
  int* err;
};

// ---------------------------------------------------------------------------------------
// instructions
// ---------------------------------------------------------------------------------------
__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const char* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t movm_t(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
// D (16x8, fp32) += A (16x16) B (16x8), 16-bit operands
template <typename M>
__device__ __forceinline__ void mma16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (std::is_same<M, __nv_bfloat16>::value) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
        "%2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
}
template <typename M>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (std::is_same<M, __nv_bfloat16>::value) {
    return pack_bf16x2(lo, hi);
  } else {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
}
template <typename M>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if constexpr (std::is_same<M, __nv_bfloat16>::value)
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
  else
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// ---------------------------------------------------------------------------------------
// sizes of a variant
// ---------------------------------------------------------------------------------------
template <int D, bool F8, int NT>
struct Shape {
  static constexpr int RB = F8 ? D : 2 * D;        // bytes of a token's row of one head
  static constexpr int CPR = RB / 16;              // 16-byte pieces of it
  // tokens per tile: 8 KB of K and V (4 KB for 64-byte rows).  16 tokens for 128-byte rows, which
  // would leave room for more warps, cost more per token than these hid (252 against 205 us, and
  // 214 us with three blocks, on 64 rows of 4096 to 12288 tokens)
  static constexpr int TT = RB == 256 ? 16 : 32;
  static constexpr int MT = TT / 16;
  // blocks per SM and stages per warp.  More warps hide each other's latencies better than
  // deeper rings (201 against 209 us for 2 blocks of 3 stages on the case above); two chunks'
  // accumulators leave registers for two blocks
  static constexpr int BLOCKS = NT == 1 ? 3 : 2;
  static constexpr int S = NT == 1 ? 2 : 3;
  static constexpr int HC = 8 * NT;                // heads of a chunk
  static constexpr int TILE = TT * RB;             // bytes of K (or V) in a stage
  static constexpr int LD = D + 4;                 // floats between a part's heads (conflict-free accumulator
                                                   // stores); D and D + 1 hold the head's maximum and sum
  static constexpr int PART = HC * LD * 4;         // bytes of a part's O
  static constexpr int WARP = S * 2 * TILE;        // bytes of a warp's ring; a last part is left in it
  static constexpr int SMEM = kWarps * WARP;
  static_assert(WARP >= PART, "a part fits the ring");
};

// Where a row's 16-byte piece lies in a tile: pieces of one column of 8 rows hit 8 bank groups.
template <int RB>
__device__ __forceinline__ uint32_t piece_at(int row, int piece) {
  if constexpr (RB >= 128)
    return (uint32_t)(row * RB + ((piece ^ (row & 7)) << 4));
  else
    return (uint32_t)(row * RB + ((piece ^ ((row >> 1) & 3)) << 4));
}

// x / y for x >= 0, y > 0; 64-bit division only where it is needed (it takes hundreds of cycles).
__device__ __forceinline__ long long quotient(long long x, long long y) {
  if (((x | y) >> 32) == 0) return (uint32_t)x / (uint32_t)y;
  return x / y;
}
// Inclusive sum over the warp's lanes.
__device__ __forceinline__ long long warp_scan(long long x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Counts one arrival and returns the arrivals before it; what the block has written (seen by
// this thread through a barrier) is visible to whoever counts after it.
__device__ __forceinline__ int arrive(int* counter) {
  int n;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(n) : "l"(counter) : "memory");
  return n;
}

struct Part {  // what a warp leaves of a cut unit; valid: te > tb
  int r, u, tb, te, tiles;
  long long unit0;  // the unit's first tile on the line
};

// Shares: the line's first `rem` shares have q + 1 tiles, the others q.
struct Shares {
  long long q, rem;
  int n;
  __device__ __forceinline__ long long begin(long long w) const { return w * q + min(w, rem); }
  // The share of tile x.  The quotient is below 2^11, so the approximate division is off by
  // one at most, which is put right; a 64-bit division would take hundreds of cycles.
  __device__ __forceinline__ int of(long long x) const {
    const long long cut = rem * (q + 1);
    int w = x < cut ? (int)__fdividef((float)x, (float)(q + 1)) : (int)(rem + (int)__fdividef((float)(x - cut), (float)q));
    w = min(w, n - 1);
    while (begin(w) > x) --w;
    while (w + 1 < n && begin(w + 1) <= x) ++w;
    return w;
  }
};

// What the joins need to know of the line, the same in all of a block's warps.
struct Line {
  Shares sh;
  int pair, unit_b0, unit_nb;  // unit_nb > 0: whole blocks per unit, of this one its first block and its blocks
};

template <int D>
struct Vec;
template <>
struct Vec<128> { using type = float4; };
template <>
struct Vec<64> { using type = float2; };

__device__ __forceinline__ void axpy(float4& a, float w, const float4 x) {
  a.x = fmaf(w, x.x, a.x); a.y = fmaf(w, x.y, a.y); a.z = fmaf(w, x.z, a.z); a.w = fmaf(w, x.w, a.w);
}
__device__ __forceinline__ void axpy(float2& a, float w, const float2 x) {
  a.x = fmaf(w, x.x, a.x); a.y = fmaf(w, x.y, a.y);
}
template <typename T>
__device__ __forceinline__ void store_out(T* dst, const float4 a, float f) {
  *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<T>(a.x * f, a.y * f), pack2<T>(a.z * f, a.w * f));
}
template <typename T>
__device__ __forceinline__ void store_out(T* dst, const float2 a, float f) {
  *reinterpret_cast<uint32_t*>(dst) = pack2<T>(a.x * f, a.y * f);
}

template <int D, typename T, bool F8, int NT>
__global__ void __launch_bounds__(kThreads, Shape<D, F8, NT>::BLOCKS) page_attn_kernel(const PageAttnParams p) {
  using Z = Shape<D, F8, NT>;
  using M = typename std::conditional<F8, __half, T>::type;  // operand type of the products
  // f16 weights use the exponents above 1: with 2^11 for the running maximum, what is below
  // f16's smallest step is below 2^-36 of it.  bf16 has the exponents below 1: with 2^-kSlack no weight
  // exceeds 1, so that values near the type's largest are not multiplied past fp32's
  constexpr float kShift = std::is_same<M, __half>::value ? 11.f : -kSlack;
  using V4 = typename Vec<D>::type;
  constexpr int VL = D / 32;  // floats of V4
  extern __shared__ __align__(256) char smem[];
  __shared__ int4 meta[kWarps][Z::S];  // of a stage: token mask, row, key head << 16 | chunk of query heads, flags
  __shared__ Part parts[2 * kWarps];
  __shared__ Line line;  // (not in registers: it is not needed while the tiles are streamed)
  __shared__ int4 pending[4];
  __shared__ int s_last[4];

  griddep_wait();  // launched ahead of the end of the stream's last kernel: see launch_ahead on its loads
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g8 = lane >> 2, t4 = lane & 3;
  // a row's visible tokens: x in [0, n) is token x (x < lo) or x + gap, or token x % page of
  // selected page x / page
  auto row_len = [&](int r) {
    const int len = p.kv_len[r];
    return len >= -1 && (long long)len <= (long long)p.W * p.page ? len : -2;
  };
  auto visible = [&](int len, int& lo, int& gap) {
    if (p.sel) {
      lo = gap = 0;
      return min(p.topk, p.by_page(len) + (p.by_page(len) * p.page < len ? 1 : 0)) * p.page;
    }
    lo = p.window > 0 ? min(p.sink, len) : len;
    gap = p.window > 0 ? max(0, len - p.window - lo) : 0;
    return len - gap;
  };
  auto row_tiles = [&](int len) {  // a row without visible tokens still gets its outputs
    if (len < 0) return 0;
    int lo, gap;
    return max(1, (visible(len, lo, gap) + Z::TT - 1) / Z::TT);
  };

  // ---- the line: its length and where this warp's share begins; every warp finds that by
  // itself (each lane adds up a run of rows), so that none waits for another
  const int per = (p.R + 31) / 32;
  const int r0 = min(p.R, lane * per), r1 = min(p.R, r0 + per);
  long long mine = 0;
  int len = -1, longest = 0;
  for (int r = r0; r < r1; ++r) {
    len = row_len(r);
    if (len == -2 && p.err && blockIdx.x == 0 && warp == 0) atomicCAS(p.err, 0, VKV_DEVERR_BAD_OFFSETS);
    const int t = row_tiles(len);
    mine += t;
    longest = max(longest, t);
  }
  long long all = mine;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
  if (all == 0) return;
  longest = __reduce_max_sync(0xFFFFFFFFu, longest);
  const int root = max(1, (int)sqrtf(kShareRoot * (float)longest)), least = max(kMinTiles, root);
  // Small calls: whole blocks per unit (of shares of `tb` / kWarps tiles at most), if the grid has
  // that many blocks
  int tb = 0, nb = 0;  // tiles of a block, or 0; blocks of the lane's rows, per unit
  {
    const int units = p.Hkv * p.n_chunks;
    const long long even = quotient(all * units + gridDim.x * kWarps - 1, (long long)gridDim.x * kWarps);
    if (even <= kWholeMost && (long long)p.R * units <= 4 * kMaxBlocks) {
      // (single tiles where a unit needs several blocks anyway: two rows of 520 tokens 9.2 and 8.8 us,
      // 42 rows of up to 456 tokens 12.6 and 11.6)
      const int s0 = max(longest > kMinTiles * kWarps ? root : least, (int)even);
#pragma unroll 1
      for (int s = s0; s <= s0 + 1 + s0 / 4; ++s) {
        nb = 0;
        if (per == 1) nb = ((int)mine + s * kWarps - 1) / (s * kWarps);
        else
          for (int r = r0; r < r1; ++r) nb += (row_tiles(row_len(r)) + s * kWarps - 1) / (s * kWarps);
        if (__reduce_add_sync(0xFFFFFFFFu, nb) * units <= (int)gridDim.x) {
          tb = s * kWarps;
          break;
        }
      }
    }
  }
  // the line's heads: key heads, or pairs of them, of which an even and an odd warp take one each
  const int pair = tb ? 0 : p.pair;
  const int heads = p.Hkv >> pair, U = heads * p.n_chunks, sub = warp & pair;
  const int kw = kWarps >> pair;  // the block's shares
  // a row's part of the line, for each of its units: tiles, or blocks
  auto extent = [&](int len) {
    const int t = row_tiles(len);
    return tb ? (t + tb - 1) / tb : t;
  };
  if (tb) mine = nb;
  long long before = warp_scan(mine, lane);
  const long long total = __shfl_sync(0xFFFFFFFFu, before, 31) * U;
  before -= mine;
  Shares sh;
  sh.q = sh.rem = sh.n = 0;
  int count = 0;                 // tiles of the warp
  long long line0 = blockIdx.x;  // where on the line the warp, or block, begins
  if (tb) {
    if (line0 >= total) return;
  } else {
    const long long n_share = min((long long)gridDim.x * kw, quotient(total + least - 1, least));
    if (line0 * kw >= n_share) return;
    sh.q = quotient(total, n_share);
    sh.rem = total - sh.q * n_share;
    sh.n = (int)n_share;
    const long long my_w = line0 * kw + (warp >> pair);
    count = my_w < n_share ? (int)(sh.q + (my_w < sh.rem ? 1 : 0)) : 0;
    line0 = sh.begin(my_w);
    if (lane == 0) {
      line.sh = sh;
      line.pair = pair;
      line.unit_nb = 0;
    }
  }
  const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * Z::WARP);
  if (lane < 2) parts[2 * warp + lane].te = 0;
  if (tb || count > 0) {
    // the row there: the lane whose rows hold it, then (long batches) the row among them
    const int src = __ffs(__ballot_sync(0xFFFFFFFFu, line0 < (before + mine) * U)) - 1;
    long long row0 = __shfl_sync(0xFFFFFFFFu, before, src) * U;
    int cr = src * per;
    if (per == 1) {
      len = __shfl_sync(0xFFFFFFFFu, len, src);
    } else {
      for (; cr < p.R; cr += 32) {
        const int l = cr + lane < p.R ? row_len(cr + lane) : -1;
        const long long t = extent(l), a = warp_scan(t, lane);
        const unsigned b = __ballot_sync(0xFFFFFFFFu, line0 < row0 + a * U);
        if (b) {
          const int x = __ffs(b) - 1;
          cr += x;
          len = __shfl_sync(0xFFFFFFFFu, l, x);
          row0 += __shfl_sync(0xFFFFFFFFu, a - t, x) * U;
          break;
        }
        row0 += __shfl_sync(0xFFFFFFFFu, a, 31) * U;
      }
    }
    int lo, gap, n_vis = visible(len, lo, gap);
    int tiles = row_tiles(len);
    const int ext = extent(len), cu = (int)quotient(line0 - row0, ext);
    int ct = (int)(line0 - row0 - (long long)cu * ext);
    if (tb) {  // the unit's tiles in equal shares to the warps of its blocks
      if (lane == 0) {
        line.pair = 0;
        line.unit_b0 = blockIdx.x - ct;
        line.unit_nb = ext;
      }
      const int q = tiles / (ext * kWarps), rem = tiles - q * ext * kWarps, w = ct * kWarps + warp;
      count = q + (w < rem ? 1 : 0);
      ct = w * q + min(w, rem);
    }
    int chead = cu / p.n_chunks, chunk = cu - chead * p.n_chunks;
    const int ct0 = ct;
    // ---- cursor: the next tile to look up
    int todo = count;  // tiles not yet looked up
    bool first = true;
    const int tok_lane = lane & (Z::TT - 1);

    int nx_page = -1, nx_off = 0, nx_r = 0, nx_hc = 0, nx_flags = 0;
    bool nx_want = false;
    // flags: 1 the share's piece of a unit begins, 2 it ends, 4 the unit begins, 8 the unit ends
    auto lookup = [&]() {
      nx_r = cr;
      const int head = (chead << pair) + sub;
      nx_hc = head << 16 | chunk;
      nx_flags = (first || ct == 0 ? 1 : 0) | (todo == 1 || ct == tiles - 1 ? 2 : 0) | (ct == 0 ? 4 : 0) |
                 (ct == tiles - 1 ? 8 : 0);
      first = false;
      const int x = ct * Z::TT + tok_lane;
      nx_want = x < n_vis;
      nx_page = -1;
      if (nx_want) {
        int j, tok;
        if (p.sel) {
          const int e = p.by_page(x);
          j = p.sel[((long long)cr * p.Hkv + head) * p.topk + e];
          nx_off = x - e * p.page;
          if (j < 0 || j >= p.W) {
            if (j != -1 && p.err) atomicCAS(p.err, 0, VKV_DEVERR_BAD_INDEX);
            nx_want = false;
          } else {
            tok = j * p.page + nx_off;
            nx_want = tok < len;
          }
        } else {
          tok = x < lo ? x : x + gap;
          j = p.by_page(tok);
          nx_off = tok - j * p.page;
        }
        if (nx_want) nx_page = p.table[cr * p.table_stride + j];
      }
      --todo;
      if (++ct == tiles) {
        ct = 0;
        if (++chunk == p.n_chunks) {
          chunk = 0;
          ++chead;
        }
        if (chead == heads && todo > 0) {
          chead = 0;
          // the next row with tiles: there is one, the line has `todo` more
          int base = cr + 1;
          while (base < p.R) {
            const int l = base + lane < p.R ? row_len(base + lane) : -1;
            const unsigned b = __ballot_sync(0xFFFFFFFFu, l >= 0);
            if (b) {
              cr = base + __ffs(b) - 1;
              break;
            }
            base += 32;
          }
          len = row_len(cr);
          n_vis = visible(len, lo, gap);
          tiles = row_tiles(len);
        }
      }
    };
    constexpr int ROWS = 32 / Z::CPR;  // rows that the warp copies at once
    const int row_b = lane / Z::CPR, piece = lane % Z::CPR;
    auto swizzled = [&](int i) {  // piece_at's offset within row i * ROWS + row_b
      return Z::RB >= 128 ? (uint32_t)((piece ^ row_b ^ ((i * ROWS) & 7)) << 4) : (uint32_t)((piece ^ ((row_b >> 1) & 3)) << 4);
    };
    auto issue = [&](int stage) {
      const bool ok = nx_want && nx_page >= 0 && nx_page < p.n_pages;
      if (nx_want && !ok && p.err) atomicCAS(p.err, 0, VKV_DEVERR_BAD_INDEX);
      const unsigned mask = __ballot_sync(0xFFFFFFFFu, ok) & (Z::TT == 32 ? 0xFFFFFFFFu : (1u << Z::TT) - 1u);
      if (lane == 0) meta[warp][stage] = make_int4((int)mask, nx_r, nx_hc, nx_flags);
      const int h = nx_hc >> 16;
      const char* kb = p.k + h * p.k_sh + piece * 16;
      const char* vb = p.v + h * p.v_sh + piece * 16;
      const uint32_t dk = ring + (uint32_t)(stage * 2 * Z::TILE) + row_b * Z::RB;
      // the lane's copies: rows i * ROWS + row_b, one 16-byte piece; a copy of 0 bytes writes
      // zeros and reads nothing, wherever its source lies
      const int page0 = __shfl_sync(0xFFFFFFFFu, nx_page, 0), off0 = __shfl_sync(0xFFFFFFFFu, nx_off, 0);
      if (__all_sync(0xFFFFFFFFu, !ok || (nx_page == page0 && nx_off == off0 + tok_lane))) {
        // consecutive rows of one page (pages of a multiple of the tile): plain strides
        const char* sk = kb + (mask & 1u ? page0 * p.k_sb + (off0 + row_b) * p.k_st : 0);
        const char* sv = vb + (mask & 1u ? page0 * p.v_sb + (off0 + row_b) * p.v_st : 0);
        const uint32_t there = mask >> row_b;
#pragma unroll
        for (int i = 0; i < Z::TT / ROWS; ++i) {
          const uint32_t at = dk + i * ROWS * Z::RB + swizzled(i);
          const int n = there >> (i * ROWS) << 4 & 16;
          cp_async16_zfill(at, sk, n);
          cp_async16_zfill(at + Z::TILE, sv, n);
          sk += ROWS * p.k_st;
          sv += ROWS * p.v_st;
        }
      } else {
        const long long ko = ok ? nx_page * p.k_sb + nx_off * p.k_st : 0, vo = ok ? nx_page * p.v_sb + nx_off * p.v_st : 0;
#pragma unroll
        for (int i = 0; i < Z::TT / ROWS; ++i) {
          const int row = i * ROWS + row_b;
          const long long rk = __shfl_sync(0xFFFFFFFFu, ko, row), rv = __shfl_sync(0xFFFFFFFFu, vo, row);
          const int n = (mask >> row) & 1u ? 16 : 0;
          const uint32_t at = dk + i * ROWS * Z::RB + swizzled(i);
          cp_async16_zfill(at, kb + rk, n);
          cp_async16_zfill(at + Z::TILE, vb + rv, n);
        }
      }
    };

    // ---- consume
    uint32_t qf[NT][D / 16][2];
    float cs[NT][2];  // log2 score per product, for heads 2 t4 and 2 t4 + 1 of each 8
    float m[NT][2], l[NT][2], acc[NT][D / 16][4];
    auto load_q = [&](int r, int h, int hc0, int n_heads) {
      const T* q = reinterpret_cast<const T*>(p.q) + r * p.q_sb + (long long)(h * p.G + hc0) * p.q_sh;
      const float c0 = p.scale_log2 * (F8 && p.ks ? p.ks[h] : 1.f);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int hd = nt * 8 + g8;
        const bool in = hd < n_heads;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          // an 8-bit row's fragment has channels 16 c + 4 t4 ..+3, a 16-bit row's 16 c + 2 t4, +1, +8, +9
          const int d0 = 16 * c + (F8 ? 4 * t4 : 2 * t4), d1 = d0 + (F8 ? 2 : 8);
          qf[nt][c][0] = in ? *reinterpret_cast<const uint32_t*>(q + hd * p.q_sh + d0) : 0u;
          qf[nt][c][1] = in ? *reinterpret_cast<const uint32_t*>(q + hd * p.q_sh + d1) : 0u;
        }
        float inv = 1.f;
        if constexpr (F8 && std::is_same<T, __nv_bfloat16>::value) {
          float big = 0.f;
#pragma unroll
          for (int c = 0; c < D / 16; ++c)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 x = unpack2<T>(qf[nt][c][e]);
              big = fmaxf(big, fmaxf(fabsf(x.x), fabsf(x.y)));
            }
          big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, 1));
          big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, 2));
          // big 2^f in [2^14, 2^15); |f| <= 126 so that both powers are normal numbers
          const int ex = (int)(__float_as_uint(big) >> 23);
          const int f = ex == 255 ? 0 : max(-113, min(126, 141 - ex));
          const float mul = __uint_as_float((uint32_t)(127 + f) << 23);
          inv = __uint_as_float((uint32_t)(127 - f) << 23);
#pragma unroll
          for (int c = 0; c < D / 16; ++c)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 x = unpack2<T>(qf[nt][c][e]);
              qf[nt][c][e] = pack2<__half>(x.x * mul, x.y * mul);
            }
        }
        const float ch = c0 * inv;
        cs[nt][0] = __shfl_sync(0xFFFFFFFFu, ch, 8 * t4);
        cs[nt][1] = __shfl_sync(0xFFFFFFFFu, ch, 8 * t4 + 4);
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[nt][c][e] = 0.f;
      }
    };
    int piece_t0 = 0, piece_n = 0;
    bool unit_begin = false;
    int stage = 0;
    // ldmatrix row addresses: K pairs (tokens 0-7, 8-15) x (piece, next piece), V the other way round
    const uint32_t k_at = piece_at<Z::RB>((lane & 7) + ((lane >> 3) & 1) * 8, lane >> 4);
    const uint32_t v_at = piece_at<Z::RB>((lane & 7) + (lane >> 4) * 8, (lane >> 3) & 1) + Z::TILE;
    // Tile i + S is looked up, tile i + S - 1 fetched and tile i used.  A fetch waits until tile i
    // has come: with more in flight the memory serves some SMs before others, and the call
    // waits for the slowest (303 against 281 us for 8 rows of 24 frames)
    int put = Z::S - 1;  // stage of the tile to fetch
#pragma unroll 1
    for (int i = -Z::S; i < count; ++i) {
      int4 mt = make_int4(0, 0, 0, 0);
      if (i >= 0) {
        __syncwarp();
        mt = meta[warp][stage];
        if (mt.w & 1) {
          const int hc0 = (mt.z & 0xFFFF) * Z::HC;
          load_q(mt.y, mt.z >> 16, hc0, min(Z::HC, p.G - hc0));
        }
        cp_async_wait<Z::S - 2>();
      }
      __syncwarp();  // the tile is here, and every lane is done with the stage before it
      if (i + Z::S - 1 >= 0 && i + Z::S - 1 < count) issue(put);
      if (todo > 0) lookup();
      cp_async_commit();
      put = put + 1 == Z::S ? 0 : put + 1;
      if (i < 0) continue;
      const unsigned mask = (unsigned)mt.x;
      const int flags = mt.w;
      if (flags & 1) {
        piece_n = 0;
        piece_t0 = i;
        unit_begin = (flags & 4) != 0;
      }
      ++piece_n;
      // piece c of every row: the swizzle and c (even) meet by exclusive or, tiles are aligned to 256 bytes
      const uint32_t sk = ring + (uint32_t)(stage * 2 * Z::TILE) + k_at, sv = ring + (uint32_t)(stage * 2 * Z::TILE) + v_at;

      // ---- scores
      float s[Z::MT][NT][4];
#pragma unroll
      for (int mt2 = 0; mt2 < Z::MT; ++mt2)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[mt2][nt][e] = 0.f;
#pragma unroll
      for (int c = 0; c < Z::CPR; c += 2) {
#pragma unroll
        for (int mt2 = 0; mt2 < Z::MT; ++mt2) {
          uint32_t a[4];
          ldsm4((sk ^ (uint32_t)(c << 4)) + mt2 * 16 * Z::RB, a);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if constexpr (F8) {
#pragma unroll
              for (int e = 0; e < 2; ++e)
                mma16816<M>(s[mt2][nt], e4m3x2_to_f16x2(a[2 * e]), e4m3x2_to_f16x2(a[2 * e + 1]),
                            e4m3x2_to_f16x2(a[2 * e] >> 16), e4m3x2_to_f16x2(a[2 * e + 1] >> 16), qf[nt][c + e][0],
                            qf[nt][c + e][1]);
            } else {
              mma16816<M>(s[mt2][nt], a[0], a[1], a[2], a[3], qf[nt][c / 2][0], qf[nt][c / 2][1]);
            }
          }
        }
      }
      // ---- weights
      const bool holes = mask != (Z::TT == 32 ? 0xFFFFFFFFu : (1u << Z::TT) - 1u);
      float top[NT][2];
      bool over = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          top[nt][e] = -INFINITY;
#pragma unroll
          for (int mt2 = 0; mt2 < Z::MT; ++mt2)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              float& x = s[mt2][nt][2 * hf + e];
              x *= cs[nt][e];
              if (holes && !(mask >> (mt2 * 16 + hf * 8 + g8) & 1u)) x = -INFINITY;
              top[nt][e] = fmaxf(top[nt][e], x);
            }
          over |= top[nt][e] > m[nt][e] + kSlack;
        }
      }
      if (__any_sync(0xFFFFFFFFu, over)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = fmaxf(top[nt][e], m[nt][e]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
            const float a = ex2_approx(m[nt][e] - (x == -INFINITY ? 0.f : x));
            m[nt][e] = x;
            l[nt][e] *= a;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              acc[nt][c][e] *= a;
              acc[nt][c][2 + e] *= a;
            }
          }
      }
      uint32_t ph[Z::MT][NT][2], pl[Z::MT][NT][2];  // B fragments: weights' values and remainders
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float b0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0] - kShift;
        const float b1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1] - kShift;
#pragma unroll
        for (int mt2 = 0; mt2 < Z::MT; ++mt2)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const float p0 = ex2_approx(s[mt2][nt][2 * hf] - b0), p1 = ex2_approx(s[mt2][nt][2 * hf + 1] - b1);
            l[nt][0] += p0;
            l[nt][1] += p1;
            const uint32_t hi = pack2<M>(p0, p1);
            const float2 b = unpack2<M>(hi);
            ph[mt2][nt][hf] = movm_t(hi);
            pl[mt2][nt][hf] = movm_t(pack2<M>(p0 - b.x, p1 - b.y));
          }
      }
      // ---- outputs
#pragma unroll
      for (int c = 0; c < Z::CPR; c += 2) {
#pragma unroll
        for (int mt2 = 0; mt2 < Z::MT; ++mt2) {
          uint32_t a[4];
          ldsm4_t((sv ^ (uint32_t)(c << 4)) + mt2 * 16 * Z::RB, a);
          if constexpr (F8) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              // bytes (token, channel): (0,0) (0,1) (1,0) (1,1) -> (0,0) (1,0) (0,1) (1,1)
              const uint32_t x = __byte_perm(a[e], 0, 0x3120), y = __byte_perm(a[2 + e], 0, 0x3120);
              const uint32_t a0 = e4m3x2_to_f16x2(x), a1 = e4m3x2_to_f16x2(x >> 16), a2 = e4m3x2_to_f16x2(y),
                             a3 = e4m3x2_to_f16x2(y >> 16);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma16816<M>(acc[nt][c + e], a0, a1, a2, a3, ph[mt2][nt][0], ph[mt2][nt][1]);
                mma16816<M>(acc[nt][c + e], a0, a1, a2, a3, pl[mt2][nt][0], pl[mt2][nt][1]);
              }
            }
          } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma16816<M>(acc[nt][c / 2], a[0], a[1], a[2], a[3], ph[mt2][nt][0], ph[mt2][nt][1]);
              mma16816<M>(acc[nt][c / 2], a[0], a[1], a[2], a[3], pl[mt2][nt][0], pl[mt2][nt][1]);
            }
          }
        }
      }
      if (flags & 2) {
        const int r = mt.y, h = mt.z >> 16, hc0 = (mt.z & 0xFFFF) * Z::HC;  // row, key head, first query head of the chunk
        const int n_heads = min(Z::HC, p.G - hc0);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) l[nt][e] += __shfl_xor_sync(0xFFFFFFFFu, l[nt][e], o);
        if (unit_begin && (flags & 8)) {  // the whole unit
          const float vs = F8 && p.vs ? p.vs[h] : 1.f;
          T* o = reinterpret_cast<T*>(p.o) + r * p.o_sb + (long long)(h * p.G + hc0) * p.o_sh;
          float* lse = p.lse + (size_t)r * p.H + h * p.G + hc0;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float f0 = l[nt][0] == 0.f ? 0.f : vs / l[nt][0], f1 = l[nt][1] == 0.f ? 0.f : vs / l[nt][1];
            const int hd = nt * 8 + g8;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              const uint32_t x = movm_t(pack2<T>(acc[nt][c][0] * f0, acc[nt][c][1] * f1));
              const uint32_t y = movm_t(pack2<T>(acc[nt][c][2] * f0, acc[nt][c][3] * f1));
              if (hd < n_heads) {
                T* dst = o + hd * p.o_sh + 16 * c;
                if constexpr (F8) {  // x: channels 4 t4, 4 t4 + 2; y: 4 t4 + 1, 4 t4 + 3
                  *reinterpret_cast<uint2*>(dst + 4 * t4) =
                      make_uint2(__byte_perm(x, y, 0x5410), __byte_perm(x, y, 0x7632));
                } else {
                  *reinterpret_cast<uint32_t*>(dst + 2 * t4) = x;
                  *reinterpret_cast<uint32_t*>(dst + 8 + 2 * t4) = y;
                }
              }
            }
            if (lane < 4) {
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (nt * 8 + 2 * lane + e < n_heads)
                  lse[nt * 8 + 2 * lane + e] =
                      l[nt][e] == 0.f ? -INFINITY : (m[nt][e] - kShift + log2f(l[nt][e])) * 0.69314718055994531f;
            }
          }
        } else {
          // a part: the share's last piece goes into this warp's ring (all of it has been read),
          // a first piece that others follow to the workspace
          const bool is_first = i + 1 == piece_n, is_last = i + 1 == count;
          const int slot = 2 * warp + (is_last ? 1 : 0);
          float* po = is_last ? reinterpret_cast<float*>(smem + warp * Z::WARP) : p.ws_first + ((long long)blockIdx.x * kWarps + warp) * (Z::HC * Z::LD);
          __syncwarp();
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const int hd = nt * 8 + 2 * t4;
#pragma unroll
            for (int c = 0; c < D / 16; ++c)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int d = 16 * c + (F8 ? 2 * g8 + (e >> 1) : g8 + (e >> 1) * 8);
                po[(hd + (e & 1)) * Z::LD + d] = acc[nt][c][e];
              }
            if (lane < 4) {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                po[(nt * 8 + 2 * lane + e) * Z::LD + D] = m[nt][e];
                po[(nt * 8 + 2 * lane + e) * Z::LD + D + 1] = l[nt][e];
              }
            }
          }
          if (lane == 0) {
            const int tl = row_tiles(row_len(r));
            const int t0 = is_first ? ct0 : 0;
            Part& pt = parts[slot];
            pt.r = r;
            pt.u = h * p.n_chunks + (mt.z & 0xFFFF);
            pt.tb = t0;
            pt.te = t0 + piece_n;
            pt.tiles = tl;
            pt.unit0 = line0 + piece_t0 - t0;
          }
        }
      }
      stage = stage + 1 == Z::S ? 0 : stage + 1;
    }
    cp_async_wait<0>();
  }
  __syncthreads();

  griddep_launch_dependents();
  // ---- join the block's parts; units that go on in other blocks meet in the workspace
  auto part_o = [&](int i) {
    return (i & 1) ? reinterpret_cast<const float*>(smem + (i >> 1) * Z::WARP)
                   : p.ws_first + ((long long)blockIdx.x * kWarps + (i >> 1)) * (Z::HC * Z::LD);
  };
  const int hcw = min(Z::HC, p.G);  // heads of a workspace part
  constexpr int HW = Z::HC / kWarps;  // heads of a warp in the joins
  auto finish = [&](int r, int head, const V4& x, float top, float sum, float vs) {
    store_out(reinterpret_cast<T*>(p.o) + r * p.o_sb + (long long)head * p.o_sh + lane * VL, x, sum == 0.f ? 0.f : vs / sum);
    if (lane == 0)
      p.lse[(size_t)r * p.H + head] =
          sum == 0.f ? -INFINITY : ((top == -INFINITY ? 0.f : top) - kShift + log2f(sum)) * 0.69314718055994531f;
  };
  const int jp = line.pair;
  // lane j holds part j (2 w: warp w's first, 2 w + 1: its last); parts of one unit are neighbours
  const int my_part = lane & (2 * kWarps - 1);
  const Part mp = parts[my_part];
  unsigned todo = __ballot_sync(0xFFFFFFFFu, lane < 2 * kWarps && mp.te > 0);
  int my_b0 = 0, my_n = 0, n_pending = 0;
  if (todo >> my_part & 1u) {
    static_assert(kWarps == 4, "2 - pair: the logarithm of the block's shares");
    my_b0 = line.unit_nb ? line.unit_b0 : line.sh.of(mp.unit0) >> (2 - jp);
    my_n = line.unit_nb ? line.unit_nb : (line.sh.of(mp.unit0 + mp.tiles - 1) >> (2 - jp)) - my_b0 + 1;
  }
#pragma unroll 1
  while (todo) {
    const int i = __ffs(todo) - 1;
    const int r = __shfl_sync(0xFFFFFFFFu, mp.r, i), u = __shfl_sync(0xFFFFFFFFu, mp.u, i);
    const unsigned grp = __ballot_sync(0xFFFFFFFFu, mp.r == r && mp.u == u) & todo;
    todo &= ~grp;
    const int t0 = __shfl_sync(0xFFFFFFFFu, mp.tb, i), tiles = __shfl_sync(0xFFFFFFFFu, mp.tiles, i);
    const int te = __shfl_sync(0xFFFFFFFFu, mp.te, 31 - __clz(grp));
    const int h = u / p.n_chunks, hc0 = (u - h * p.n_chunks) * Z::HC, n_heads = min(Z::HC, p.G - hc0);
    const bool whole = t0 == 0 && te == tiles;
    const float vs = F8 && p.vs ? p.vs[h] : 1.f;
    const size_t ws = (((size_t)(2 * blockIdx.x + (t0 == 0 ? 1 : 0)) << jp) + (h & jp)) * hcw;
    // the warps' parts of this unit (at most one each)
    const float* src[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) src[w] = part_o(2 * w + (grp >> (2 * w + 1) & 1));
    float top[HW], sum[HW];
    V4 x[HW];
#pragma unroll
    for (int k = 0; k < HW; ++k) {
      const int hd = min(warp + k * kWarps, n_heads - 1);
      float2 ml[kWarps];
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        ml[w] = grp >> (2 * w) & 3 ? *reinterpret_cast<const float2*>(src[w] + hd * Z::LD + D) : make_float2(-INFINITY, 0.f);
      top[k] = fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x));
      const float base = top[k] == -INFINITY ? 0.f : top[k];
      sum[k] = 0.f;
      std::memset(&x[k], 0, sizeof(V4));
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float e = ex2_approx(ml[w].x - base);
        sum[k] = fmaf(e, ml[w].y, sum[k]);
        if (grp >> (2 * w) & 3) axpy(x[k], e, *reinterpret_cast<const V4*>(src[w] + hd * Z::LD + lane * VL));
      }
    }
#pragma unroll
    for (int k = 0; k < HW; ++k) {
      const int hd = warp + k * kWarps;
      if (hd >= n_heads) break;
      if (whole) {
        finish(r, h * p.G + hc0 + hd, x[k], top[k], sum[k], vs);
      } else {
        *reinterpret_cast<V4*>(p.ws_o + (ws + hd) * D + lane * VL) = x[k];
        if (lane == 0) *reinterpret_cast<float2*>(p.ws_ml + (ws + hd) * 2) = make_float2(top[k], sum[k]);
      }
    }
    if (!whole) {
      const int b0 = __shfl_sync(0xFFFFFFFFu, my_b0, i), n = __shfl_sync(0xFFFFFFFFu, my_n, i);
      // row, key head << 16 | chunk, first block << pair | the head's place in its pair, blocks
      if (tid == 0) pending[n_pending] = make_int4(r, h << 16 | (u - h * p.n_chunks), b0 << jp | (h & jp), n);
      ++n_pending;  // two per head at most: what began in an earlier block, and what goes on in a later one
    }
  }
  if (n_pending == 0) return;
  // every unit's parts are on their way before any is waited for
  __syncthreads();  // the block's parts are written; the arrival passes that on
  int* counter = p.counters;  // the unit's, in its first block
  if (tid < n_pending) {
    counter += pending[tid].z;
    s_last[tid] = arrive(counter) == pending[tid].w - 1;
  }
  __syncthreads();
  if (tid < n_pending && s_last[tid]) *counter = 0;
  // The units that this block completes, a warp's heads side by side.  This code runs once per
  // block and its time is latencies, those of fetching it among them: dealing the heads of both
  // units to the warps at once, with twice the loads in flight, took 4 us longer
#pragma unroll 1
  for (int f = 0; f < n_pending; ++f) {
    if (s_last[f]) {
      const int r = pending[f].x, h = pending[f].y >> 16, hc0 = (pending[f].y & 0xFFFF) * Z::HC, n_heads = min(Z::HC, p.G - hc0);
      const int n = pending[f].w, first = pending[f].z;
      const float vs = F8 && p.vs ? p.vs[h] : 1.f;
      float top[HW], sum[HW];
      V4 x[HW];
      // part 0 lies among its block's lasts, the others among their blocks' firsts
      // loads in flight per head; fewer where a warp has four heads (37 rows of 2310 tokens, e4m3, 12
      // heads per key head: 63.3 us with 8, 59.9 with 4; one row of 131072 tokens 49.6 and 51.7)
      constexpr int kBatch = NT == 1 ? 8 : 4;
      const int b0 = first >> jp, stride = (2 * hcw) << jp;
      const size_t row1 = (size_t)(b0 + 1) * stride + (first & jp) * hcw, row0 = row1 - (hcw << jp);
      auto at = [&](int j, int hd) { return (j == 0 ? row0 : row1 + (size_t)(j - 1) * stride) + hd; };
      V4 y[HW][kBatch];
      auto load = [&](int j0) {
#pragma unroll
        for (int k = 0; k < HW; ++k)
#pragma unroll
          for (int e = 0; e < kBatch; ++e)
            if (j0 + e < n && warp + k * kWarps < n_heads)
              y[k][e] = __ldcg(reinterpret_cast<const V4*>(p.ws_o + at(j0 + e, warp + k * kWarps) * D + lane * VL));
      };
      auto ml = [&](int j, int k) {
        return j < n && warp + k * kWarps < n_heads
                   ? __ldcg(reinterpret_cast<const float2*>(p.ws_ml + at(j, warp + k * kWarps) * 2))
                   : make_float2(-INFINITY, 0.f);
      };
      float2 v[HW];
#pragma unroll
      for (int k = 0; k < HW; ++k) v[k] = ml(lane, k);
      load(0);
#pragma unroll
      for (int k = 0; k < HW; ++k) {
        top[k] = v[k].x;
        for (int j = 32 + lane; j < n; j += 32) top[k] = fmaxf(top[k], ml(j, k).x);
#pragma unroll
        for (int q = 16; q > 0; q >>= 1) top[k] = fmaxf(top[k], __shfl_xor_sync(0xFFFFFFFFu, top[k], q));
        sum[k] = 0.f;
        std::memset(&x[k], 0, sizeof(V4));
      }
#pragma unroll 1
      for (int j0 = 0; j0 < n; j0 += 32) {
        float wl[HW];
#pragma unroll
        for (int k = 0; k < HW; ++k) {
          if (j0 > 0) v[k] = ml(j0 + lane, k);
          wl[k] = ex2_approx(v[k].x - (top[k] == -INFINITY ? 0.f : top[k]));
          sum[k] = fmaf(wl[k], v[k].y, sum[k]);
        }
#pragma unroll 1
        for (int jb = 0; jb < 32 && j0 + jb < n; jb += kBatch) {
#pragma unroll
          for (int k = 0; k < HW; ++k)
#pragma unroll
            for (int e = 0; e < kBatch; ++e) {
              const float w = __shfl_sync(0xFFFFFFFFu, wl[k], jb + e);
              if (j0 + jb + e < n) axpy(x[k], w, y[k][e]);
            }
          load(j0 + jb + kBatch);
        }
      }
#pragma unroll
      for (int k = 0; k < HW; ++k) {
#pragma unroll
        for (int q = 16; q > 0; q >>= 1) sum[k] += __shfl_xor_sync(0xFFFFFFFFu, sum[k], q);
        const int hd = warp + k * kWarps;
        if (hd < n_heads) finish(r, h * p.G + hc0 + hd, x[k], top[k], sum[k], vs);
      }
    }
  }
}

// ---------------------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------------------
template <int D, typename T, bool F8, int NT>
cudaError_t launch(const PageAttnParams& p, int blocks, int n_sm, int dev, cudaStream_t st) {
  using Z = Shape<D, F8, NT>;
  auto fn = page_attn_kernel<D, T, F8, NT>;
  static std::atomic<uint64_t> ready{0};  // devices (by bit) on which the limit is raised
  if (!(ready.load(std::memory_order_acquire) >> dev & 1u)) {
    const cudaError_t rc = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, Z::SMEM);
    if (rc != cudaSuccess) return rc;
    ready.fetch_or(1ull << dev, std::memory_order_release);
  }
  return launch_ahead(fn, dim3((unsigned)std::min(blocks, Z::BLOCKS * n_sm)), dim3(kThreads), Z::SMEM, st, p);
}

template <int D, typename T, bool F8>
cudaError_t launch_nt(const PageAttnParams& p, int blocks, int n_sm, int dev, cudaStream_t st) {
  return p.G <= 8 ? launch<D, T, F8, 1>(p, blocks, n_sm, dev, st) : launch<D, T, F8, 2>(p, blocks, n_sm, dev, st);
}

template <int D>
cudaError_t launch_d(const PageAttnParams& p, int q_dtype, int kv_dtype, int blocks, int n_sm, int dev, cudaStream_t st) {
  if (kv_dtype == VKV_E4M3)
    return q_dtype == VKV_BF16 ? launch_nt<D, __nv_bfloat16, true>(p, blocks, n_sm, dev, st) : launch_nt<D, __half, true>(p, blocks, n_sm, dev, st);
  return q_dtype == VKV_BF16 ? launch_nt<D, __nv_bfloat16, false>(p, blocks, n_sm, dev, st) : launch_nt<D, __half, false>(p, blocks, n_sm, dev, st);
}

// Bytes of the counters and of one block's workspace parts.
constexpr size_t kCounterBytes = VKV_PAGE_ATTN_CLEAR_BYTES;
static_assert(2 * kMaxBlocks * sizeof(int) <= kCounterBytes, "counters");
size_t part_bytes(int G, int d) {
  const int hc = G <= 8 ? 8 : 16;
  return ((size_t)4 * std::min(G, hc) * (d + 2) + (size_t)kWarps * hc * (d + 4)) * sizeof(float);
}

}  // namespace
}  // namespace vkv

using namespace vkv;

extern "C" size_t vkv_page_attn_workspace_size(int32_t H, int32_t Hkv, int32_t d) {
  if (H < 1 || Hkv < 1 || H % Hkv || (d != 64 && d != 128)) return 0;
  const int n_sm = device_sm_count(nullptr);
  if (n_sm <= 0) return 0;
  const int blocks = std::min(kMaxBlocks, kMaxBlocksPerSm * n_sm);
  return (kCounterBytes + blocks * part_bytes(H / Hkv, d) + 255) / 256 * 256;
}

extern "C" vkv_status vkv_page_attn(const vkv_page_attn_args* a, vkv_stream_t stream) {
  if (!a) return VKV_ERR_NULL;
  if (a->d != 64 && a->d != 128) return VKV_ERR_UNSUPPORTED;
  if (a->q_dtype != VKV_BF16 && a->q_dtype != VKV_FP16) return VKV_ERR_UNSUPPORTED;
  if (a->kv_dtype != a->q_dtype && a->kv_dtype != VKV_E4M3) return VKV_ERR_UNSUPPORTED;
  if (a->R < 1 || a->R > VKV_PAGE_MAX_ROWS || a->H < 1 || a->Hkv < 1 || a->H % a->Hkv || a->page < 1 ||
      a->n_pages < 1 || a->W < 1 || a->sink < 0 || a->window < 0 || a->table_stride < a->W)
    return VKV_ERR_SHAPE;
  if (!(a->scale > 0.f) || a->scale > 2.0e38f) return VKV_ERR_SHAPE;
  if (a->sel ? (a->topk < 1 || a->window != 0) : a->topk != 0) return VKV_ERR_SHAPE;
  if ((long long)a->R * a->W > INT_MAX || (long long)a->W * a->page > INT_MAX - 64 || a->H > 4096 ||
      (long long)a->topk * a->page > INT_MAX - 64)
    return VKV_ERR_UNSUPPORTED;
  if (a->kv_dtype != VKV_E4M3 && (a->k_scale || a->v_scale)) return VKV_ERR_UNSUPPORTED;
  if (!a->q.ptr || !a->o.ptr || !a->k.ptr || !a->v.ptr || !a->table || !a->kv_len || !a->lse) return VKV_ERR_NULL;
  vkv_tensor q = a->q, o = a->o;
  q.st = o.st = 0;
  if (!page_tensor_aligned(q, a->q_dtype) || !page_tensor_aligned(o, a->q_dtype) ||
      !page_tensor_aligned(a->k, a->kv_dtype) || !page_tensor_aligned(a->v, a->kv_dtype))
    return VKV_ERR_ALIGN;
  int dev = 0;
  const int n_sm = device_sm_count(&dev);
  if (n_sm <= 0) return VKV_ERR_CUDA;
  const size_t need = vkv_page_attn_workspace_size(a->H, a->Hkv, a->d);
  if (!a->workspace || a->workspace_bytes < need) return VKV_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(a->workspace) & 255u) return VKV_ERR_ALIGN;
  PageAttnParams p;
  std::memset(&p, 0, sizeof(p));
  p.R = a->R; p.H = a->H; p.Hkv = a->Hkv; p.G = a->H / a->Hkv;
  p.page = a->page; p.n_pages = a->n_pages; p.W = a->W; p.sink = a->sink; p.window = a->window; p.topk = a->topk;
  p.by_page = fast_div(a->page);
  const int e = dtype_bytes(a->kv_dtype);
  const int hc = p.G <= 8 ? 8 : 16;
  p.n_chunks = (p.G + hc - 1) / hc;
  // Rows of 128 bytes or less, one key head's beside the next's: two warps take neighbouring
  // heads of the same tokens, so that HBM serves runs of twice the length (64 rows of 4096 to
  // 12288 tokens, e4m3, d = 128: 206 us alone, 192 in pairs).  Selected pages differ by head
  p.pair = a->d * e <= 128 && !a->sel && a->Hkv % 2 == 0 && a->k.sh == a->d && a->v.sh == a->d ? 1 : 0;
  p.scale_log2 = a->scale * 1.4426950408889634f;
  p.q = a->q.ptr; p.q_sb = a->q.sb; p.q_sh = a->q.sh;
  p.o = a->o.ptr; p.o_sb = a->o.sb; p.o_sh = a->o.sh;
  p.k = reinterpret_cast<const char*>(a->k.ptr);
  p.v = reinterpret_cast<const char*>(a->v.ptr);
  p.k_sb = a->k.sb * e; p.k_st = a->k.st * e; p.k_sh = a->k.sh * e;
  p.v_sb = a->v.sb * e; p.v_st = a->v.st * e; p.v_sh = a->v.sh * e;
  p.table = a->table; p.table_stride = a->table_stride;
  p.kv_len = a->kv_len;
  p.sel = a->sel;
  p.ks = a->k_scale; p.vs = a->v_scale;
  p.lse = a->lse;
  const int all = std::min(kMaxBlocks, kMaxBlocksPerSm * n_sm);
  p.counters = reinterpret_cast<int*>(a->workspace);
  p.ws_first = reinterpret_cast<float*>(reinterpret_cast<char*>(a->workspace) + kCounterBytes);
  p.ws_o = p.ws_first + (size_t)all * kWarps * hc * (a->d + 4);
  p.ws_ml = p.ws_o + (size_t)4 * all * std::min(p.G, hc) * a->d;
  p.err = a->err_word;
  // no more blocks than the longest rows that the table allows could fill
  const int tt = a->d * e == 256 ? 16 : 32;
  const long long most = a->sel ? std::min<long long>((long long)a->topk * a->page, (long long)a->W * a->page)
                         : a->window > 0 ? std::min<long long>((long long)a->sink + a->window, (long long)a->W * a->page)
                                         : (long long)a->W * a->page;
  const long long row_blocks = (std::max<long long>(1, (most + tt - 1) / tt) + kWarps - 1) / kWarps;
  const int blocks = (int)std::min<long long>(all, row_blocks * a->R * a->Hkv * p.n_chunks);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t rc = a->d == 128 ? launch_d<128>(p, a->q_dtype, a->kv_dtype, blocks, n_sm, dev, st)
                                     : launch_d<64>(p, a->q_dtype, a->kv_dtype, blocks, n_sm, dev, st);
  return rc == cudaSuccess ? VKV_OK : VKV_ERR_CUDA;
}
