// Parts of shared-prefix attention in tiles of 16 query rows (bf16, any head width),
// on the warp-level matrix instruction.
//
// A decoding step gives a key/value head G = H / H_kv rows of a request: its suffix
// cache is read for 4 to 16 rows, and so is the prefix of a small batch.  That is a
// memory-bound pass (16 rows do 16 operations a byte, the machine 250), and what
// costs is latency: a 128-row tcgen05 tile needs a TMEM allocation, a dozen barriers
// and 113 KB of shared memory a block, 5.6 us for a block of 64 keys (here 2.6).  m16n8k16
// products hold everything in a warp's registers instead: the rows fill its 16
// (one thread holds row lane / 4 and that + 8), the scores of 16 keys leave the
// first product in the layout in which the second takes them, and no warp waits for
// another until the end.
//
// A block computes one part for one key/value head and 16 rows.  Its 4 warps (2 for parts of up
// to 64 keys) take the part's 32-key tiles in turn, each through a ring of its own (cp.async, 16 bytes a lane,
// rows of 2 DP bytes with their 16-byte words swapped by key mod 8 so that ldmatrix reads
// without bank conflicts).  Keys past the part's end arrive as zeros, whatever the cache
// holds, and are masked.  The warps' (m, l, O) are merged in shared memory.
//
// Where a request has few keys, prefix and suffix together, one block takes them all and
// writes the output itself (`whole`): no parts, no merge, one launch.
//
// Bound by HBM where there are many keys (128 suffixes of up to 1024 keys of 8 heads of 128,
// 270 MB: 49 us, 85% of the copy rate), by latency where there are few (64 keys: 3.9 us, of
// them 2.6 a block).  16 keys a step left the matrix unit waiting for shuffles and fragments
// (1.8k cycles a warp's tile, so 1.3k for twice the keys).
//
// Weights are rounded to bf16 for the product as in the tensor-core path (half a
// step, 2^-8 relative); sums and statistics are fp32.
#include <algorithm>

#include "lvx_prefix.cuh"
#include "lvx_ptx.cuh"

namespace lvx {
namespace {

constexpr int kTile = 32;      // keys a warp takes at a time
// Warps of a block, and 32-key tiles of K or V in a warp's ring.  Parts of up to 64 keys take
// two warps with a tile each (six blocks an SM, so that many short suffixes overlap their
// latencies), the others four with a ring (two blocks an SM).
template <int DP, bool SHORT>
struct Config {
  static constexpr int warps = SHORT ? 2 : 4;
  static constexpr int slots = SHORT ? 2 : DP == 128 ? 3 : 6;
};
constexpr float kRescaleThreshold = 8.0f;   // log2 units
constexpr float kLn2 = 0.6931471805599453f;

struct RowsArgs {
  PrefixProblem p;
  int pre_tiles, suf_tiles;   // 16-row tiles of a key/value head's rows, of a request's
  int pre_items;              // blocks of prefix parts
  bool whole;
  __nv_bfloat16* out;         // whole
  float* lse;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool on) {
  // src-size 0: nothing is read, the 16 bytes become zero
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// DP: the head width padded to 64 or 128 (the columns from d on are zeros).
template <int DP, bool SHORT>
__global__ void __launch_bounds__(32 * Config<DP, SHORT>::warps, SHORT ? 6 : 2)
prefix_rows_kernel(const RowsArgs a, const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ kp,
                   const __nv_bfloat16* __restrict__ vp, const __nv_bfloat16* __restrict__ ks,
                   const __nv_bfloat16* __restrict__ vs) {
  constexpr int kRow = 2 * DP;             // bytes of a key in shared memory
  constexpr int kWords = DP / 8;           // ... in 16-byte words
  constexpr int kHalf = kTile * kRow;      // a tile of K or V
  constexpr int kWarps = Config<DP, SHORT>::warps, kThreads = 32 * kWarps, NS = Config<DP, SHORT>::slots;
  extern __shared__ __align__(128) uint8_t smem[];
  const PrefixProblem& p = a.p;

  // keys [a0, a1) of the prefix, then [b0, b1) of request b's suffix
  const bool pre = blockIdx.x < (unsigned)a.pre_items;
  int idx = blockIdx.x - (pre ? 0 : a.pre_items);
  const int row_tiles = pre ? a.pre_tiles : a.suf_tiles;
  const int r0 = idx % row_tiles * 16;
  idx /= row_tiles;
  const int g = idx % p.H_kv;
  idx /= p.H_kv;
  int part = 0, tok0 = 0, a0 = 0, a1 = 0, b0 = 0, b1 = 0, n = 0, b = 0;
  if (!pre) {
    b = a.whole ? idx : idx / p.n_suf;
    tok0 = b * p.S_Q;
  }
  const int rows = min(16, (pre ? p.B * p.S_Q : p.S_Q) * p.G - r0);

  // the queries' loads come first, the latest to be used
  constexpr int kQWords = 16 * kWords / kThreads;   // of a thread
  uint4 qw[kQWords];
#pragma unroll
  for (int x = 0; x < kQWords; ++x) {
    const int r = r0 + threadIdx.x / kWords + x * (kThreads / kWords), w = threadIdx.x % kWords;
    qw[x] = make_uint4(0, 0, 0, 0);
    if (r - r0 < rows && w * 8 < p.d)
      qw[x] = __ldg(reinterpret_cast<const uint4*>(
          q + ((size_t)(tok0 + r / p.G) * p.H + g * p.G + r % p.G) * p.d + w * 8));
  }
  if (pre) {
    part = idx;
    a0 = part * p.pre_len;
    a1 = min(a0 + p.pre_len, p.S_P);
  } else {
    const int s = a.whole ? 0 : idx % p.n_suf;
    n = suffix_keys(p, b);
    if (a.whole) {
      a1 = p.S_P;
      b1 = n;
    } else {
      part = p.n_pre + s;
      b0 = s * p.suf_len;
      b1 = min(b0 + p.suf_len, n);
    }
  }
  const __nv_bfloat16* ksb = ks + (size_t)b * p.S_cap * p.H_kv * p.d;
  const __nv_bfloat16* vsb = vs + (size_t)b * p.S_cap * p.H_kv * p.d;
  if (!a.whole) let_next_start();
  const int a_tiles = (a1 - a0 + kTile - 1) / kTile, b_tiles = b1 > b0 ? (b1 - b0 + kTile - 1) / kTile : 0;
  const int tiles = a_tiles + b_tiles;
  if (tiles == 0 && !a.whole) return;   // the merge does not read this part
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int mine = (tiles - warp + kWarps - 1) / kWarps;   // tiles warp, warp + 4, ...

  // copies: lane word w of key r, two keys (DP = 128) or four (64) a pass
  const uint32_t ring = ptx::smem_u32(smem) + warp * (NS * kHalf);
  const size_t key_stride = (size_t)p.H_kv * p.d;
  const int cw = lane % kWords, cr = lane / kWords;
  const bool in_row = cw * 8 < p.d;
  const size_t lane_at = (size_t)g * p.d + (in_row ? cw * 8 : 0);
  int put = 0, get = 0;   // slots
  auto fetch = [&](int x) {   // K_0, V_0, K_1, V_1, ... of the warp's tiles
    const int i = x >> 1;
    if (i < mine) {
      const uint32_t dst = ring + put * kHalf;
      const int t = i * kWarps + warp;
      const bool in_a = t < a_tiles;
      const __nv_bfloat16* src = in_a ? x & 1 ? vp : kp : x & 1 ? vsb : ksb;
      const int key0 = in_a ? a0 + t * kTile : b0 + (t - a_tiles) * kTile, end = in_a ? a1 : b1;
      const __nv_bfloat16* at = src + (size_t)(key0 + cr) * key_stride + lane_at;
      const int there = in_row ? end - key0 - cr : 0;   // rows x < there of this lane's are
#pragma unroll
      for (int x = 0; x < kTile; x += 32 / kWords) {
        const int r = x + cr;
        cp_async16(dst + r * kRow + ((cw ^ (r & 7)) << 4), x < there ? at : src, x < there);
        at += 32 / kWords * key_stride;
      }
    }
    cp_commit();
    put = put + 1 == NS ? 0 : put + 1;
  };
  // the ring's next tile, once it is there
  auto next = [&] {
    cp_wait<NS - 1>();
    __syncwarp();
    const uint32_t at = ring + get * kHalf;
    get = get + 1 == NS ? 0 : get + 1;
    return at;
  };
#pragma unroll
  for (int x = 0; x < NS; ++x) fetch(x);

  // the queries, 16 rows as the keys' rows lie, behind the rings; zeros past the last row
  const int r_lo = lane >> 2, quad = lane & 3;
  uint8_t* q_rows = smem + kWarps * NS * kHalf;
#pragma unroll
  for (int x = 0; x < kQWords; ++x) {
    const int r = threadIdx.x / kWords + x * (kThreads / kWords), w = threadIdx.x % kWords;
    *reinterpret_cast<uint4*>(q_rows + r * kRow + ((w ^ (r & 7)) << 4)) = qw[x];
  }
  __syncthreads();
  const uint32_t sq = ptx::smem_u32(q_rows);
  int lim[2];   // suffix keys below lim are visible to the lane's rows
#pragma unroll
  for (int hi = 0; hi < 2; ++hi) lim[hi] = min(b1, n - p.S_Q + 1 + (r0 + r_lo + 8 * hi) / p.G);
  const int lim_all = min(b1, n - p.S_Q + 1 + r0 / p.G);   // ... to every row

  float o[DP / 8][4];
#pragma unroll
  for (int n = 0; n < DP / 8; ++n)
#pragma unroll
    for (int c = 0; c < 4; ++c) o[n][c] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  const float sl2 = p.scale_log2;
  // ldmatrix rows of this lane: K takes keys (lane & 7) + 8 (lane >> 4), word (lane >> 3) & 1;
  // V keys lane & 15, word lane >> 4
  const int krow = (lane & 7) + ((lane >> 4) << 3), kword = (lane >> 3) & 1;
  const int vrow = lane & 15, vword = lane >> 4;

  for (int i = 0; i < mine; ++i) {
    const uint32_t sk = next();
    const int t = i * kWarps + warp;
    const bool in_a = t < a_tiles;
    const int key0 = in_a ? a0 + t * kTile : b0 + (t - a_tiles) * kTile;
    float s[4][4];   // n-tiles of 8 keys
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int c = 0; c < 4; ++c) s[n][c] = 0.f;
    // fragments of the next step are on their way during a step's products
    uint32_t qf[2][4], kf[2][2][4];   // q: rows lane & 15, word lane >> 4
    auto load_k = [&](int kk) {
      ldsm4(sq + vrow * kRow + (((2 * kk + vword) ^ (vrow & 7)) << 4), qf[kk & 1]);
#pragma unroll
      for (int j = 0; j < 2; ++j)
        ldsm4(sk + (16 * j + krow) * kRow + (((2 * kk + kword) ^ (krow & 7)) << 4), kf[kk & 1][j]);
    };
    load_k(0);
#pragma unroll
    for (int kk = 0; kk < DP / 16; ++kk) {
      if (kk + 1 < DP / 16) load_k(kk + 1);
#pragma unroll
      for (int n = 0; n < 4; ++n)
        mma(s[n], qf[kk & 1], kf[kk & 1][n >> 1][2 * (n & 1)], kf[kk & 1][n >> 1][2 * (n & 1) + 1]);
    }
    __syncwarp();   // every lane has read K
    fetch(2 * i + NS);
    if (key0 + kTile > (in_a ? a1 : lim_all)) {
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (key0 + n * 8 + quad * 2 + (c & 1) >= (in_a ? a1 : lim[c >> 1])) s[n][c] = -INFINITY;
    }
    float mt[2];
    bool move = false;
#pragma unroll
    for (int hi = 0; hi < 2; ++hi) {
      float x = fmaxf(s[0][2 * hi], s[0][2 * hi + 1]);
#pragma unroll
      for (int n = 1; n < 4; ++n) x = fmaxf(x, fmaxf(s[n][2 * hi], s[n][2 * hi + 1]));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
      mt[hi] = x * sl2;
      move |= mt[hi] > m[hi] + kRescaleThreshold;
    }
    if (__any_sync(0xffffffffu, move)) {
#pragma unroll
      for (int hi = 0; hi < 2; ++hi) {
        const float m_new = fmaxf(m[hi], mt[hi]);
        const float al = m_new == -INFINITY ? 1.f : ptx::ex2(m[hi] - m_new);
        m[hi] = m_new;
        l[hi] *= al;
#pragma unroll
        for (int n = 0; n < DP / 8; ++n) {
          o[n][2 * hi] *= al;
          o[n][2 * hi + 1] *= al;
        }
      }
    }
    const float mu[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
    uint32_t pf[2][4];
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int hi = 0; hi < 2; ++hi) {
        const float e0 = ptx::ex2(fmaf(s[n][2 * hi], sl2, -mu[hi]));
        const float e1 = ptx::ex2(fmaf(s[n][2 * hi + 1], sl2, -mu[hi]));
        l[hi] += e0 + e1;
        pf[n >> 1][2 * (n & 1) + hi] = ptx::pack_bf16x2(e0, e1);
      }
    const uint32_t sv = next();
    uint32_t vf[2][2][4];
    auto load_v = [&](int n) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        ldsm4_t(sv + (16 * j + vrow) * kRow + (((2 * n + vword) ^ (vrow & 7)) << 4), vf[n & 1][j]);
    };
    load_v(0);
#pragma unroll
    for (int n = 0; n < DP / 16; ++n) {
      if (n + 1 < DP / 16) load_v(n + 1);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        mma(o[2 * n], pf[j], vf[n & 1][j][0], vf[n & 1][j][1]);
        mma(o[2 * n + 1], pf[j], vf[n & 1][j][2], vf[n & 1][j][3]);
      }
    }
    __syncwarp();   // ... and V
    fetch(2 * i + 1 + NS);
  }
  cp_wait<0>();
#pragma unroll
  for (int hi = 0; hi < 2; ++hi) {
    l[hi] += __shfl_xor_sync(0xffffffffu, l[hi], 1);
    l[hi] += __shfl_xor_sync(0xffffffffu, l[hi], 2);
  }

  // merge of the warps: O [warp][16][DP + 8], then m and l [warp][16]
  __syncthreads();
  float* so = reinterpret_cast<float*>(smem);
  constexpr int kLdO = DP + 8;   // rows 8 banks apart
  float* sm = so + kWarps * 16 * kLdO;
  float* sl = sm + kWarps * 16;
#pragma unroll
  for (int hi = 0; hi < 2; ++hi) {
    const int r = r_lo + 8 * hi;
    if (quad == 0) {
      sm[warp * 16 + r] = m[hi];
      sl[warp * 16 + r] = l[hi];
    }
    if (r < rows) {
#pragma unroll
      for (int n = 0; n < DP / 8; ++n)
        *reinterpret_cast<float2*>(so + (warp * 16 + r) * kLdO + n * 8 + quad * 2) =
            make_float2(o[n][2 * hi], o[n][2 * hi + 1]);
    }
  }
  // a row's weights of the warps, its place and its log-sum-exp
  uint32_t* place = reinterpret_cast<uint32_t*>(sl + kWarps * 16);
  __syncthreads();
  const size_t all_rows = (size_t)p.B * p.S_Q * p.H;
  if (threadIdx.x < rows) {
    const int r = threadIdx.x;
    float M = -INFINITY, tot = 0.f, f[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w * 16 + r]);
    const float M0 = M == -INFINITY ? 0.f : M;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      f[w] = ptx::ex2(sm[w * 16 + r] - M0);
      tot = fmaf(f[w], sl[w * 16 + r], tot);
    }
    const float inv = tot == 0.f ? 0.f : 1.f / tot;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sm[w * 16 + r] = f[w] * inv;
    const int h = g * p.G + (r0 + r) % p.G, t = (r0 + r) / p.G;
    place[r] = (uint32_t)(tok0 + t) * p.H + h;
    const float L = tot == 0.f ? -INFINITY : (M0 + log2f(tot)) * kLn2;
    if (a.whole) a.lse[((size_t)b * p.H + h) * p.S_Q + t] = L;
    else p.l_parts[part * all_rows + place[r]] = L;
  }
  __syncthreads();
  constexpr int kVecs = DP / 4;
  const int c = threadIdx.x % kVecs;
  if (c * 4 >= p.d) return;
#pragma unroll
  for (int x0 = 0; x0 < 16; x0 += kThreads / kVecs) {
    const int r = x0 + threadIdx.x / kVecs;
    if (r >= rows) break;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = sm[w * 16 + r];
      const float4 u = *reinterpret_cast<const float4*>(so + (w * 16 + r) * kLdO + c * 4);
      x.x = fmaf(f, u.x, x.x); x.y = fmaf(f, u.y, x.y); x.z = fmaf(f, u.z, x.z); x.w = fmaf(f, u.w, x.w);
    }
    const size_t row = place[r];
    if (a.whole)
      *reinterpret_cast<uint2*>(a.out + row * p.d + c * 4) =
          make_uint2(ptx::pack_bf16x2(x.x, x.y), ptx::pack_bf16x2(x.z, x.w));
    else
      *reinterpret_cast<float4*>(p.o_parts + (part * all_rows + row) * p.d + c * 4) = x;
  }
}

template <int DP, bool SHORT>
cudaError_t launch(const RowsArgs& a, unsigned grid, const void* q, const void* kp, const void* vp,
                   const void* ks, const void* vs, cudaStream_t s) {
  using C = Config<DP, SHORT>;
  constexpr int ring = (C::warps * C::slots * kTile + 16) * 2 * DP;   // and the queries
  constexpr int merge = (C::warps * 16 * (DP + 10) + 16) * (int)sizeof(float);
  constexpr int smem = ring > merge ? ring : merge;
  cudaError_t e =
      cudaFuncSetAttribute(prefix_rows_kernel<DP, SHORT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  auto bf = [](const void* x) { return reinterpret_cast<const __nv_bfloat16*>(x); };
  prefix_rows_kernel<DP, SHORT><<<grid, 32 * C::warps, smem, s>>>(a, bf(q), bf(kp), bf(vp), bf(ks), bf(vs));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prefix_rows(const PrefixProblem& p, bool pre, bool suf, void* out, float* lse, const void* q,
                               const void* kp, const void* vp, const void* ks, const void* vs, cudaStream_t s) {
  RowsArgs a;
  a.p = p;
  a.whole = out != nullptr;
  a.out = reinterpret_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  const long long pre_tiles = ((long long)p.B * p.S_Q * p.G + 15) / 16, suf_tiles = ((long long)p.S_Q * p.G + 15) / 16;
  const long long pre_items = pre ? pre_tiles * p.n_pre * p.H_kv : 0;
  const long long items = pre_items + (suf ? suf_tiles * p.B * (a.whole ? 1 : p.n_suf) * p.H_kv : 0);
  if (items > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  a.pre_tiles = (int)pre_tiles;
  a.suf_tiles = (int)suf_tiles;
  a.pre_items = (int)pre_items;
  const unsigned n = (unsigned)items;
  const long long longest = a.whole ? (long long)p.S_P + p.S_cap
                                    : std::max(pre ? std::min(p.pre_len, p.S_P) : 0, suf ? std::min(p.suf_len, p.S_cap) : 0);
  if (longest <= kPrefixShort)
    return p.d <= 64 ? launch<64, true>(a, n, q, kp, vp, ks, vs, s) : launch<128, true>(a, n, q, kp, vp, ks, vs, s);
  return p.d <= 64 ? launch<64, false>(a, n, q, kp, vp, ks, vs, s) : launch<128, false>(a, n, q, kp, vp, ks, vs, s);
}

}  // namespace lvx
