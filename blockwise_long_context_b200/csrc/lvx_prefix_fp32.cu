// Parts of shared-prefix attention in fp32 arithmetic (fp32 inputs, and bf16 with more
// than 128 query heads a key/value head), on the CUDA cores.
//
// A block computes one part for one key/value head and up to 32 rows, 64 keys at a time.
// Its 4 warps are WR slabs of 8 rows times 4 / WR slices of 16 WR keys (WR = 1, 2 or 4,
// as few as hold the rows: with 4 to 16 rows, a decoding step's, every warp still has
// work).  A warp keeps its slab's softmax to itself:
//   S: lane (row group of 4, key 16 j + lane % 16) holds a 4 x WR tile of the scores, and
//      reads float4s of both operands; a row's maximum and sum are shuffles in 16 lanes;
//   P goes through the warp's corner of shared memory;
//   O += P V: a lane holds 4 columns of 8 rows (d > 64) or of 4 rows.
// Rows of K and V lie 68 or 132 floats apart, so that 8 lanes' float4s hit 32 banks.  The
// copies of the next K run during the product with V, those of the next V during the next
// scores (cp.async; keys past the part's end become zeros, whatever the cache holds).
// The slices' (m, l, O) are merged in shared memory.  Where a request has few keys, prefix
// and suffix together, a block takes them all and writes the output itself (`whole`).
//
// Bound: 4 rows do 2 operations a byte (the machine 11) and wait for their copies: with one
// buffer each for K and V and block-wide barriers around them, one tile of a block is on its way
// on average.  16384 keys of 8 heads of 128, 134 MB, 37 us, 55% of the copy rate.  32 rows are
// bound by fp32 multiply-adds, of which the
// two or three warps a scheduler holds keep 40% busy (128 rows x 32 heads over 2048 keys
// 154 us, 28 TFLOP/s).  Slabs of 16 rows and packed multiply-adds were no faster.
#include <type_traits>

#include "lvx_prefix.cuh"
#include "lvx_ptx.cuh"

namespace lvx {
namespace {

using namespace ptx;

constexpr int kThreads = 128;
constexpr int KT = 64;          // keys a tile
constexpr float kRescaleThreshold = 8.0f;   // log2 units
constexpr float kLn2 = 0.6931471805599453f;

struct Fp32Args {
  PrefixProblem p;
  int pre_rows, suf_rows;     // rows of a tile of prefix, suffix parts: 8, 16 or 32
  int pre_tiles, suf_tiles;   // row tiles of a key/value head
  int pre_items;              // blocks of prefix parts
  bool whole;
  void* out;                  // whole
  float* lse;
};

// One block's part: rows r0 .. r0 + nr of its key/value head (row r is head r % G of
// token tok0 + r / G), keys [a0, a1) of the prefix and [b0, b1) of request b's suffix, of
// which row r sees those below min(b1, lim0 + r / G).
template <typename T>
struct Part {
  const T *ka, *va, *kb, *vb;
  int g, b, part, tok0, r0, nr, a0, a1, b0, b1, lim0;
};

__device__ __forceinline__ void cp_async16(float* dst, const float* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_wait_but_one() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

// Keys key0 .. key0 + KT of one key/value head into dst[KT][DP + 4], zeros from kend on.
template <int DP>
__device__ __forceinline__ void load_tile(float* dst, const float* base, int key0, int kend, size_t stride, int d) {
  constexpr int W = DP / 4, STEP = kThreads / W;
  const int w = threadIdx.x % W, r0 = threadIdx.x / W;
  if (w * 4 < d) {
    const float* src = base + (size_t)(key0 + r0) * stride + w * 4;
    const int n = kend - key0 - r0;   // rows r < n of this thread's are there
    float* to = dst + r0 * (DP + 4) + w * 4;
#pragma unroll
    for (int r = 0; r < KT; r += STEP) {
      cp_async16(to + r * (DP + 4), r < n ? src : base, r < n);
      src += STEP * stride;
    }
  }
  cp_commit();
}
template <int DP>
__device__ __forceinline__ void load_tile(float* dst, const __nv_bfloat16* base, int key0, int kend, size_t stride,
                                          int d) {
  constexpr int W = DP / 8;
  const int w = threadIdx.x % W;
  if (w * 8 < d) {
#pragma unroll 4
    for (int r = threadIdx.x / W; r < KT; r += kThreads / W) {
      uint4 u = make_uint4(0, 0, 0, 0);
      if (key0 + r < kend) u = __ldg(reinterpret_cast<const uint4*>(base + (size_t)(key0 + r) * stride + w * 8));
      float4* to = reinterpret_cast<float4*>(dst + r * (DP + 4) + w * 8);
      auto lo = [](uint32_t x) { return __uint_as_float(x << 16); };
      auto hi = [](uint32_t x) { return __uint_as_float(x & 0xffff0000u); };
      to[0] = make_float4(lo(u.x), hi(u.x), lo(u.y), hi(u.y));
      to[1] = make_float4(lo(u.z), hi(u.z), lo(u.w), hi(u.w));
    }
  }
  cp_commit();
}

// The block's rows of q into dst[rows][DP + 4], zeros past the last (committed with the next tile).
template <int DP>
__device__ __forceinline__ void load_rows(float* dst, const Part<float>& t, const PrefixProblem& p, const float* q,
                                          int rows) {
  constexpr int W = DP / 4;
  const int w = threadIdx.x % W;
  if (w * 4 >= p.d) return;
#pragma unroll 4
  for (int i = threadIdx.x / W; i < rows; i += kThreads / W) {
    const int r = t.r0 + (i < t.nr ? i : 0);
    cp_async16(dst + i * (DP + 4) + w * 4,
               q + ((size_t)(t.tok0 + r / p.G) * p.H + t.g * p.G + r % p.G) * p.d + w * 4, i < t.nr);
  }
}
template <int DP>
__device__ __forceinline__ void load_rows(float* dst, const Part<__nv_bfloat16>& t, const PrefixProblem& p,
                                          const __nv_bfloat16* q, int rows) {
  constexpr int W = DP / 4;
  const int w = threadIdx.x % W;
  if (w * 4 >= p.d) return;
#pragma unroll 4
  for (int i = threadIdx.x / W; i < rows; i += kThreads / W) {
    const int r = t.r0 + (i < t.nr ? i : 0);
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(
        q + ((size_t)(t.tok0 + r / p.G) * p.H + t.g * p.G + r % p.G) * p.d + w * 4));
    const bool on = i < t.nr;
    *reinterpret_cast<float4*>(dst + i * (DP + 4) + w * 4) =
        make_float4(on ? __uint_as_float(u.x << 16) : 0.f, on ? __uint_as_float(u.x & 0xffff0000u) : 0.f,
                    on ? __uint_as_float(u.y << 16) : 0.f, on ? __uint_as_float(u.y & 0xffff0000u) : 0.f);
  }
}

template <typename T, int DP, int WR>
__device__ __forceinline__ void run_part(const PrefixProblem& p, const Part<T>& t, const Fp32Args& args,
                                         const T* __restrict__ q, float* sm) {
  constexpr int KW = 16 * WR;                // keys of a warp's slice
  constexpr int NR = DP == 128 ? 8 : 4;      // rows of a lane in the product with V
  constexpr int ld = DP + 4;   // (a constant, so that rows are constant offsets)
  const int d = p.d;
  float* sk = sm;                     // [KT][ld]; at the end O [4][8][d]
  float* sv = sk + KT * ld;           // [KT][ld]
  float* sq = sv + KT * ld;           // [8 WR][ld]
  float* sp = sq + 8 * WR * ld;      // [4][8][KW + 4]; at the end m, l [4][8]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slab = warp % WR, slice = warp / WR;
  const int rg = lane >> 4, kl = lane & 15;
  const bool busy = slab * 8 < t.nr;
  const size_t stride = (size_t)p.H_kv * d;

  // the queries first: they and K are one group of copies
  load_rows<DP>(sq, t, p, q, 8 * WR);
  const int a_tiles = (t.a1 - t.a0 + KT - 1) / KT;
  const int tiles = a_tiles + (t.b1 > t.b0 ? (t.b1 - t.b0 + KT - 1) / KT : 0);
  auto load_k = [&](int x) {
    if (x < a_tiles) load_tile<DP>(sk, t.ka, t.a0 + x * KT, t.a1, stride, d);
    else if (x < tiles) load_tile<DP>(sk, t.kb, t.b0 + (x - a_tiles) * KT, t.b1, stride, d);
    else cp_commit();
  };
  auto load_v = [&](int x) {
    if (x < a_tiles) load_tile<DP>(sv, t.va, t.a0 + x * KT, t.a1, stride, d);
    else if (x < tiles) load_tile<DP>(sv, t.vb, t.b0 + (x - a_tiles) * KT, t.b1, stride, d);
    else cp_commit();
  };
  load_k(0);
  load_v(0);
  float m[4], l[4];
  int lim[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
    lim[i] = min(t.b1, t.lim0 + (t.r0 + slab * 8 + rg * 4 + i) / p.G);
  }
  const int col = (DP == 128 ? lane : lane & 15) * 4, row = DP == 128 ? 0 : (lane >> 4) * NR;
  const bool has_col = col < d;
  float o[NR][4];
#pragma unroll
  for (int i = 0; i < NR; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) o[i][c] = 0.f;

  const float* qr = sq + (slab * 8 + rg * 4) * ld;
  const float* kr = sk + (slice * KW + kl) * ld;
  float* pw = sp + warp * 8 * (KW + 4);
  for (int x = 0; x < tiles; ++x) {
    const bool in_a = x < a_tiles;
    const int key0 = in_a ? t.a0 + x * KT : t.b0 + (x - a_tiles) * KT;
    const int left = (in_a ? t.a1 : t.b1) - key0 - slice * KW;   // keys of this warp's slice
    cp_wait_but_one();
    __syncthreads();
    float s[4][WR];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < WR; ++j) s[i][j] = 0.f;
    auto scores = [&](auto width) {   // of the first 16 `width` keys
      constexpr int N = decltype(width)::value;
#pragma unroll 2
      for (int c = 0; c < d; c += 4) {
        float4 a[4], b[N];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(qr + i * ld + c);
#pragma unroll
        for (int j = 0; j < N; ++j) b[j] = *reinterpret_cast<const float4*>(kr + 16 * j * ld + c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < N; ++j)
            s[i][j] = fmaf(a[i].w, b[j].w, fmaf(a[i].z, b[j].z, fmaf(a[i].y, b[j].y, fmaf(a[i].x, b[j].x, s[i][j]))));
      }
    };
    if (busy && left > 16) scores(std::integral_constant<int, WR>());
    else if (busy && left > 0) scores(std::integral_constant<int, 1>());
    __syncthreads();   // K is free
    load_k(x + 1);
    if (busy) {
      float mt[4];
      bool move = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        mt[i] = -INFINITY;
#pragma unroll
        for (int j = 0; j < WR; ++j) {
          const int key = key0 + slice * KW + 16 * j + kl;
          s[i][j] = key < (in_a ? t.a1 : lim[i]) ? s[i][j] * p.scale_log2 : -INFINITY;
          mt[i] = fmaxf(mt[i], s[i][j]);
        }
#pragma unroll
        for (int o16 = 8; o16 > 0; o16 >>= 1) mt[i] = fmaxf(mt[i], __shfl_xor_sync(0xffffffffu, mt[i], o16));
        move |= mt[i] > m[i] + kRescaleThreshold;
      }
      if (__any_sync(0xffffffffu, move)) {
        float al[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float m_new = fmaxf(m[i], mt[i]);
          al[i] = m_new == -INFINITY ? 1.f : exp2f(m[i] - m_new);
          m[i] = m_new;
          l[i] *= al[i];
        }
#pragma unroll
        for (int i = 0; i < NR; ++i) {   // from a lane that knows row + i
          const float f = __shfl_sync(0xffffffffu, al[i & 3], ((row + i) >> 2) * 16);
#pragma unroll
          for (int c = 0; c < 4; ++c) o[i][c] *= f;
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float mu = m[i] == -INFINITY ? 0.f : m[i];
#pragma unroll
        for (int j = 0; j < WR; ++j) {
          const float e = exp2f(s[i][j] - mu);   // a NaN score stays one
          l[i] += e;
          pw[(rg * 4 + i) * (KW + 4) + 16 * j + kl] = e;
        }
      }
    }
    cp_wait_but_one();
    __syncthreads();
    if (busy && has_col) {
      const float* vr = sv + slice * KW * ld + col;
      const int keys = min(KW, left);   // (past them the weights are 0)
#pragma unroll 2
      for (int k = 0; k < keys; k += 4) {
        float4 v[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) v[x] = *reinterpret_cast<const float4*>(vr + (k + x) * ld);
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          const float4 w = *reinterpret_cast<const float4*>(pw + (row + i) * (KW + 4) + k);
          const float f[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            o[i][0] = fmaf(f[x], v[x].x, o[i][0]);
            o[i][1] = fmaf(f[x], v[x].y, o[i][1]);
            o[i][2] = fmaf(f[x], v[x].z, o[i][2]);
            o[i][3] = fmaf(f[x], v[x].w, o[i][3]);
          }
        }
      }
    }
    __syncthreads();   // V is free
    load_v(x + 1);
  }

  // merge of the slices
  float *so = sk, *s_m = sp, *s_l = sp + 32;
  uint32_t* place = reinterpret_cast<uint32_t*>(sp + 64);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int x = 8; x > 0; x >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
    if (kl == 0) {
      s_m[warp * 8 + rg * 4 + i] = m[i];
      s_l[warp * 8 + rg * 4 + i] = l[i];
    }
  }
  if (has_col) {
#pragma unroll
    for (int i = 0; i < NR; ++i)
      *reinterpret_cast<float4*>(so + (warp * 8 + row + i) * d + col) = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
  }
  __syncthreads();
  const size_t rows = (size_t)p.B * p.S_Q * p.H;
  if (threadIdx.x < t.nr) {   // a row's weights of the slices, its place and its log-sum-exp
    const int i = threadIdx.x, r = t.r0 + i;
    float M = -INFINITY, tot = 0.f, f[4 / WR];
#pragma unroll
    for (int x = 0; x < 4 / WR; ++x) M = fmaxf(M, s_m[(x * WR + i / 8) * 8 + i % 8]);
    const float M0 = M == -INFINITY ? 0.f : M;
#pragma unroll
    for (int x = 0; x < 4 / WR; ++x) {
      const int at = (x * WR + i / 8) * 8 + i % 8;
      f[x] = exp2f(s_m[at] - M0);
      tot = fmaf(f[x], s_l[at], tot);
    }
    const float inv = tot == 0.f ? 0.f : 1.f / tot;
#pragma unroll
    for (int x = 0; x < 4 / WR; ++x) s_m[(x * WR + i / 8) * 8 + i % 8] = f[x] * inv;
    const int h = t.g * p.G + r % p.G, tok = r / p.G;
    place[i] = (uint32_t)(t.tok0 + tok) * p.H + h;
    const float L = tot == 0.f ? -INFINITY : (M0 + log2f(tot)) * kLn2;
    if (args.whole) args.lse[((size_t)t.b * p.H + h) * p.S_Q + tok] = L;
    else p.l_parts[t.part * rows + place[i]] = L;
  }
  __syncthreads();
  constexpr int kVecs = DP / 4;
  const int c = threadIdx.x % kVecs;
  if (c * 4 >= d) return;
  for (int i = threadIdx.x / kVecs; i < t.nr; i += kThreads / kVecs) {
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int x = 0; x < 4 / WR; ++x) {
      const int at = (x * WR + i / 8) * 8 + i % 8;
      const float f = s_m[at];
      const float4 u = *reinterpret_cast<const float4*>(so + at * d + c * 4);
      a.x = fmaf(f, u.x, a.x); a.y = fmaf(f, u.y, a.y); a.z = fmaf(f, u.z, a.z); a.w = fmaf(f, u.w, a.w);
    }
    const size_t to = place[i];
    if (!args.whole) {
      *reinterpret_cast<float4*>(p.o_parts + (t.part * rows + to) * d + c * 4) = a;
    } else if (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(reinterpret_cast<float*>(args.out) + to * d + c * 4) = a;
    } else {
      *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(args.out) + to * d + c * 4) =
          make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
    }
  }
}

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads, DP == 128 ? 3 : 4)
prefix_fp32_kernel(const Fp32Args a, const T* __restrict__ q, const T* __restrict__ kp, const T* __restrict__ vp,
                   const T* __restrict__ ks, const T* __restrict__ vs) {
  extern __shared__ __align__(16) float sm[];
  const PrefixProblem& p = a.p;
  Part<T> t;
  const bool pre = blockIdx.x < (unsigned)a.pre_items;
  int idx = blockIdx.x - (pre ? 0 : a.pre_items);
  const int tiles = pre ? a.pre_tiles : a.suf_tiles, rows = pre ? a.pre_rows : a.suf_rows;
  t.r0 = idx % tiles * rows;
  idx /= tiles;
  t.g = idx % p.H_kv;
  idx /= p.H_kv;
  t.part = t.tok0 = t.b = t.a0 = t.a1 = t.b0 = t.b1 = t.lim0 = 0;
  if (pre) {
    t.part = idx;
    t.a0 = idx * p.pre_len;
    t.a1 = min(t.a0 + p.pre_len, p.S_P);
  } else {
    const int s = a.whole ? 0 : idx % p.n_suf;
    t.b = a.whole ? idx : idx / p.n_suf;
    const int n = suffix_keys(p, t.b);
    t.tok0 = t.b * p.S_Q;
    t.lim0 = n - p.S_Q + 1;
    if (a.whole) {
      t.a1 = p.S_P;
      t.b1 = n;
    } else {
      t.part = p.n_pre + s;
      t.b0 = s * p.suf_len;
      t.b1 = min(t.b0 + p.suf_len, n);
    }
  }
  t.ka = kp + (size_t)t.g * p.d;
  t.va = vp + (size_t)t.g * p.d;
  t.kb = ks + ((size_t)t.b * p.S_cap * p.H_kv + t.g) * p.d;
  t.vb = vs + ((size_t)t.b * p.S_cap * p.H_kv + t.g) * p.d;
  if (!a.whole) let_next_start();
  if (t.a0 >= t.a1 && t.b0 >= t.b1 && !a.whole) return;   // the merge does not read this part
  t.nr = min(rows, (pre ? p.B * p.S_Q : p.S_Q) * p.G - t.r0);
  if (rows == 8) run_part<T, DP, 1>(p, t, a, q, sm);
  else if (rows == 16) run_part<T, DP, 2>(p, t, a, q, sm);
  else run_part<T, DP, 4>(p, t, a, q, sm);
}

template <typename T, int DP>
cudaError_t launch(const Fp32Args& a, unsigned grid, const void* q, const void* kp, const void* vp, const void* ks,
                   const void* vs, cudaStream_t s) {
  const int rows = a.pre_items ? a.pre_rows : a.suf_rows;   // (a suffix part has no more rows)
  const size_t smem = sizeof(float) * ((size_t)(2 * KT + rows) * (DP + 4) + 4 * 8 * (2 * rows + 4));
  cudaError_t e = cudaFuncSetAttribute(prefix_fp32_kernel<T, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)smem);
  if (e != cudaSuccess) return e;
  prefix_fp32_kernel<T, DP><<<grid, kThreads, smem, s>>>(a, (const T*)q, (const T*)kp, (const T*)vp, (const T*)ks,
                                                         (const T*)vs);
  return cudaGetLastError();
}

}  // namespace

int prefix_fp32_rows(long long rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : 32; }

cudaError_t launch_prefix_fp32(const PrefixProblem& p, lvx_dtype dt, void* out, float* lse, const void* q,
                               const void* kp, const void* vp, const void* ks, const void* vs, cudaStream_t s) {
  Fp32Args a;
  a.p = p;
  a.whole = out != nullptr;
  a.out = out;
  a.lse = lse;
  const long long pre_rows = (long long)p.B * p.S_Q * p.G, suf_rows = (long long)p.S_Q * p.G;
  a.pre_rows = prefix_fp32_rows(pre_rows);
  a.suf_rows = prefix_fp32_rows(suf_rows);
  const long long pre_tiles = (pre_rows + a.pre_rows - 1) / a.pre_rows;
  const long long suf_tiles = (suf_rows + a.suf_rows - 1) / a.suf_rows;
  const long long pre_items = pre_tiles * p.H_kv * p.n_pre;
  const long long items = pre_items + suf_tiles * p.H_kv * (a.whole ? 1 : p.n_suf) * p.B;
  if (items > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  a.pre_tiles = (int)pre_tiles;
  a.suf_tiles = (int)suf_tiles;
  a.pre_items = (int)pre_items;
  const unsigned n = (unsigned)items;
  if (dt == LVX_FP32)
    return p.d <= 64 ? launch<float, 64>(a, n, q, kp, vp, ks, vs, s) : launch<float, 128>(a, n, q, kp, vp, ks, vs, s);
  return p.d <= 64 ? launch<__nv_bfloat16, 64>(a, n, q, kp, vp, ks, vs, s)
                   : launch<__nv_bfloat16, 128>(a, n, q, kp, vp, ks, vs, s);
}

}  // namespace lvx
