// Shared-prefix attention: the C entry points, the cut into parts and their merge.
//
// For request b, token t of S_Q, head h with key/value head g = h / (H / H_kv), and
// n_b valid suffix keys, the visible keys are all S_P prefix keys and the suffix keys
// j <= n_b - S_Q + t (the S_Q tokens are the request's last):
//   O = sum softmax(s q.k) v,   LSE = ln sum exp(s q.k)   over them.
// The keys are cut into parts, each part's (O_i, L_i) is computed by one block for a
// tile of the rows that read the part's keys (128, 16 or up to 32, by the kernel), and
// the parts are merged by the framework's rescaling: L = M + ln sum exp(L_i - M),
// O = sum exp(L_i - L) O_i.  Requests of few keys are computed whole, without parts.
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "lvx_prefix.cuh"

namespace lvx {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ------------------------------------------------------------------ merge

template <typename T>
__device__ __forceinline__ void store4(T* dst, const float4& x) {
  if (sizeof(T) == 2) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(x.x, x.y), hi = __floats2bfloat162_rn(x.z, x.w);
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  } else {
    *reinterpret_cast<float4*>(dst) = x;
  }
}

// At most P parts (2, 4 or 8): a thread takes four columns of a row, all its parts at once,
// and computes the row's weights for itself.  No thread waits for another, so many rows of
// few parts keep their bytes coming (49280 rows of 2 parts 42 us with a warp a row).
constexpr int kFewThreads = 256;

template <typename T, int P>
__global__ void __launch_bounds__(kFewThreads)
prefix_merge_few_kernel(const PrefixProblem p, T* __restrict__ out, float* __restrict__ lse) {
  const size_t rows = (size_t)p.B * p.S_Q * p.H;
  const unsigned vecs = p.d / 4;
  const size_t at = (size_t)blockIdx.x * kFewThreads + threadIdx.x;
  const unsigned row = (unsigned)(at / vecs), c = (unsigned)(at - (size_t)row * vecs);
  if (row >= rows) return;
  const unsigned b = row / ((unsigned)p.S_Q * p.H);
  const int parts = p.n_pre + (suffix_keys(p, b) + p.suf_len - 1) / p.suf_len;
  const float* lp = p.l_parts + row;
  const float4* op = reinterpret_cast<const float4*>(p.o_parts + (size_t)row * p.d) + c;
  wait_for_previous();
  float l[P];
  float4 x[P];
#pragma unroll
  for (int i = 0; i < P; ++i) l[i] = i < parts ? load_l2(lp + i * rows) : -INFINITY;
#pragma unroll
  for (int i = 0; i < P; ++i) x[i] = i < parts ? load_l2(op + i * rows * vecs) : make_float4(0.f, 0.f, 0.f, 0.f);
  float M = l[0];
#pragma unroll
  for (int i = 1; i < P; ++i) M = fmaxf(M, l[i]);
  const float M0 = M == -INFINITY ? 0.f : M;
  float tot = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const float w = exp2f((l[i] - M0) * kLog2e);
    tot += w;
    if (w != 0.f) {   // a part of no visible key holds no numbers that count
      acc.x = fmaf(w, x[i].x, acc.x);
      acc.y = fmaf(w, x[i].y, acc.y);
      acc.z = fmaf(w, x[i].z, acc.z);
      acc.w = fmaf(w, x[i].w, acc.w);
    }
  }
  const float inv = tot == 0.f ? 0.f : 1.f / tot;
  store4(out + (size_t)row * p.d + c * 4, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
  if (c == 0) {
    const unsigned h = row % p.H, t = row / p.H % p.S_Q;
    lse[((size_t)b * p.H + h) * p.S_Q + t] = tot == 0.f ? -INFINITY : M0 + log2f(tot) * kLn2;
  }
}

// More parts: W warps a row (1, 2 or 4; a block has 4): each takes every W-th part, a float4 a lane
// and several parts a step where d < 128, then the warps' sums are added in shared
// memory.  Bound by the latency of its reads, which come from L2 (the parts were just
// written): the first eight of a lane are in flight before the maximum is known.  The
// grid is launched while the parts are still being computed and waits for them here;
// it reads them at L2 (they were not read-only while the grid ran).
constexpr int kMergeWarps = 4;
constexpr int kAhead = 8;

template <typename T, int W>
__global__ void __launch_bounds__(32 * kMergeWarps, 7)
prefix_merge_kernel(const PrefixProblem p, T* __restrict__ out, float* __restrict__ lse) {
  __shared__ float4 acc_s[kMergeWarps][32];
  __shared__ float sum_s[kMergeWarps];
  const size_t rows = (size_t)p.B * p.S_Q * p.H;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, slice = warp % W;
  const size_t row = (size_t)blockIdx.x * (kMergeWarps / W) + warp / W;
  const bool live = row < rows;
  const int b = live ? (int)(row / ((size_t)p.S_Q * p.H)) : 0;
  const int parts = live ? p.n_pre + (suffix_keys(p, b) + p.suf_len - 1) / p.suf_len : 0;
  const int vecs = p.d / 4;                       // float4s of a row
  const int subs = 32 / vecs;                     // parts a warp reads at a time
  const int sub = lane / vecs, c = lane % vecs;   // lanes past subs * vecs idle
  const int first = slice * subs + sub, step = W * subs, n = sub < subs ? parts : 0;
  const float* lp = p.l_parts + row;
  const float4* op = reinterpret_cast<const float4*>(p.o_parts + row * p.d) + c;
  const size_t ostep = rows * vecs;
  wait_for_previous();
  // L is read by all, O_i before its weight is known (weights of 0 do not touch it: a part
  // of no visible key holds no numbers that count)
  float4 x[kAhead];
  float li[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const int i = first + k * step;
    li[k] = i < n ? load_l2(lp + i * rows) : -INFINITY;
    x[k] = i < n ? load_l2(op + i * ostep) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float M = -INFINITY;
  for (int i = lane; i < parts; i += 32) M = fmaxf(M, load_l2(lp + i * rows));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float M0 = M == -INFINITY ? 0.f : M;      // no part with a key (or one with a NaN, which stays)
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float tot = 0.f;
  auto add = [&](float l, const float4& u) {
    const float w = exp2f((l - M0) * kLog2e);
    tot += w;
    if (w != 0.f) {
      acc.x = fmaf(w, u.x, acc.x);
      acc.y = fmaf(w, u.y, acc.y);
      acc.z = fmaf(w, u.z, acc.z);
      acc.w = fmaf(w, u.w, acc.w);
    }
  };
#pragma unroll
  for (int k = 0; k < kAhead; ++k) add(li[k], x[k]);
#pragma unroll 4
  for (int i = first + kAhead * step; i < n; i += step) add(load_l2(lp + i * rows), load_l2(op + i * ostep));
  acc_s[warp][lane] = acc;
  if (c != 0) tot = 0.f;   // every lane of a part counted it: one does
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
  if (lane == 0) sum_s[warp] = tot;
  if (W > 1) __syncthreads();
  else __syncwarp();
  if (live && slice == 0 && lane < vecs) {
    tot = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      tot += sum_s[warp + w];
      for (int s = 0; s < subs; ++s) {
        const float4 u = acc_s[warp + w][s * vecs + lane];
        acc.x += u.x; acc.y += u.y; acc.z += u.z; acc.w += u.w;
      }
    }
    const float inv = tot == 0.f ? 0.f : 1.f / tot;
    store4(out + row * p.d + lane * 4, make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
    if (lane == 0) {
      const int h = (int)(row % p.H), t = (int)(row / p.H % p.S_Q);
      lse[((size_t)b * p.H + h) * p.S_Q + t] = tot == 0.f ? -INFINITY : M0 + log2f(tot) * kLn2;
    }
  }
}

template <typename T>
cudaError_t merge(const PrefixProblem& p, T* out, float* lse, cudaStream_t s) {
  const long long rows = (long long)p.B * p.S_Q * p.H;
  const int parts = p.n_pre + p.n_suf;
  if (parts <= 8) {
    const unsigned grid = (unsigned)((rows * (p.d / 4) + kFewThreads - 1) / kFewThreads);
    if (parts <= 2) return launch_after(prefix_merge_few_kernel<T, 2>, grid, kFewThreads, 0, s, p, out, lse);
    if (parts <= 4) return launch_after(prefix_merge_few_kernel<T, 4>, grid, kFewThreads, 0, s, p, out, lse);
    return launch_after(prefix_merge_few_kernel<T, 8>, grid, kFewThreads, 0, s, p, out, lse);
  }
  // about eight steps a warp, unless the rows alone give the SMs work
  const int steps = parts / (128 / p.d);   // of one warp: it reads 128 / d parts at a time
  const int w = steps <= 10 || rows > 148 * 64 ? 1 : steps <= 20 ? 2 : 4;
  const unsigned grid = (unsigned)((rows * w + kMergeWarps - 1) / kMergeWarps);
  if (w == 1) return launch_after(prefix_merge_kernel<T, 1>, grid, 32 * kMergeWarps, 0, s, p, out, lse);
  if (w == 2) return launch_after(prefix_merge_kernel<T, 2>, grid, 32 * kMergeWarps, 0, s, p, out, lse);
  return launch_after(prefix_merge_kernel<T, 4>, grid, 32 * kMergeWarps, 0, s, p, out, lse);
}

}  // namespace

cudaError_t launch_prefix_merge(const PrefixProblem& p, lvx_dtype dt, void* out, float* lse, cudaStream_t s) {
  return dt == LVX_FP32 ? merge(p, (float*)out, lse, s) : merge(p, (__nv_bfloat16*)out, lse, s);
}

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

lvx_status check_prefix(int B, int H, int H_kv, int S_Q, int S_P, int S_cap, int d, lvx_dtype dt) {
  if (B < 1 || H < 1 || H_kv < 1 || S_Q < 1 || S_P < 0 || S_cap < 0 || d < 1) return LVX_ERR_INVALID_ARG;
  if (H % H_kv != 0 || S_P + (long long)S_cap < 1) return LVX_ERR_INVALID_ARG;
  if (dt != LVX_FP32 && dt != LVX_BF16) return LVX_ERR_UNSUPPORTED;
  if (d > 128 || d % 8 != 0) return LVX_ERR_UNSUPPORTED;
  // rows are grid blocks of the merge; key positions plus a tile stay below 2^31
  if ((long long)B * S_Q > (1ll << 30) / H || S_P > (1 << 30) || S_cap > (1 << 30)) return LVX_ERR_UNSUPPORTED;
  return LVX_OK;
}

// Blocks that one wave holds, the rows of one block, and its fewest keys (below them the
// block's start and its partial output weigh more than its keys); of parts of `keys` keys.
struct Shape { int wave, rows, least; };
Shape shape_of(PrefixKernel k, const PrefixProblem& p, long long rows, double keys) {
  if (k == kPrefixRows) {
    const bool small = keys <= kPrefixShort || (p.S_cap > 0 && p.S_cap <= kPrefixShort && p.S_P <= 512);
    return {small ? 148 * 6 : 148 * 2, kPrefixRowsTile, 128};
  }
  if (k == kPrefixTc) return {148 * 2, kPrefixTile / p.G * p.G, 256};
  const int r = prefix_fp32_rows(rows);
  return {148 * (p.d > 64 ? r == 8 ? 3 : 2 : 4), r, 64};
}

// Time of one block, in us, as measured: a start and an end, then its key tiles.
double block_us(PrefixKernel k, int d, double keys) {
  if (k == kPrefixTc) return 4.0 + std::ceil(keys / 64) * (d > 64 ? 0.9 : 0.55);
  if (k == kPrefixFp32) return 3.0 + std::ceil(keys / 64) * (d > 64 ? 3.5 : 2.0);
  return keys <= kPrefixShort ? 2.6 : 2.2 + std::ceil(keys / 128) * 0.75;
}
// Time of the keys' way from L2, by 16-row tiles that each read them for themselves.
double l2_us(long long tiles, double keys, int d) { return tiles * keys * 4.0 * d / 6e6; }
// Time of the merge, and of writing what it reads.
double merge_us(const PrefixProblem& p, double parts) {
  return 4.0 + parts * p.B * p.S_Q * p.H * p.d * 8.0 / 5e6;
}

// A cut of keys into n parts of len, the blocks it makes (of suffixes, those that are half
// full on average), and the time until the last one is done.
struct Cut {
  int n, len;
  double blocks, us;
};

// The prefix's parts: as many as fill one wave of blocks, or several where they fill the
// machine better.
Cut cut_prefix(PrefixKernel k, const Shape& f, const PrefixProblem& p, long long tiles) {
  const int S_P = p.S_P, d = p.d;
  const long long most = (S_P + (long long)f.least - 1) / f.least;
  Cut best = {0, 64, 0.0, 0.0};
  double least = 0.0;
  // beside short suffixes, a few hundred keys in short parts: one launch of small blocks
  const bool small = k == kPrefixRows && p.S_cap > 0 && p.S_cap <= kPrefixShort && S_P <= 512;
  for (int w = 1; S_P > 0 && w <= (small ? 1 : 4); ++w) {
    const long long n = small ? (S_P + kPrefixShort - 1) / kPrefixShort
                              : std::min(std::max(1ll, (long long)w * f.wave / tiles), most);
    const int len = (int)((S_P + n - 1) / n + 63) / 64 * 64;
    const long long parts = (S_P + (long long)len - 1) / len, blocks = tiles * parts;
    // the last wave's blocks have the machine to themselves
    const double us = (double)((blocks + f.wave - 1) / f.wave) * block_us(k, d, len) +
                      (k == kPrefixRows ? l2_us(tiles, S_P, d) : 0.0);
    const double all = us + merge_us(p, (double)parts);
    if (best.n == 0 || all < least) {
      best = {(int)parts, len, (double)blocks, us};
      least = all;
    }
  }
  return best;
}

// A suffix is cut by its capacity, as its length is on the device (blocks of parts past a
// length return at once; half of the parts are counted).  Parts of up to 512 keys by their time;
// where parts of 512 make more than four waves of blocks, longer ones until they do not: so many
// even out nothing, the blocks past the lengths cost their start, and each part takes its rows'
// output in fp32, in the workspace and in the merge (1024 tokens over 16384 + 16384 keys 500 us,
// with parts of 512 keys 750; 64 requests of up to 1309 keys in caches of 65536 46 us, 231).
Cut cut_suffix(PrefixKernel k, const Shape& f, const PrefixProblem& p, long long tiles) {
  Cut best = {0, 64, 0.0, 0.0};
  double least = 0.0;
  auto cut = [&](int len) {
    const int n = (p.S_cap + len - 1) / len;
    const double blocks = tiles * (n + 1) * 0.5;
    return Cut{n, len, blocks, std::max(1.0, blocks / f.wave) * block_us(k, p.d, std::min(len, p.S_cap))};
  };
  for (int len = 512; p.S_cap > 0 && len >= f.least; len /= 2) {
    const Cut c = cut(len);
    const double all = c.us + merge_us(p, c.n * 0.5);
    if (best.n == 0 || all < least) {
      best = c;
      least = all;
    }
  }
  for (int len = 512; 2 * len < p.S_cap && cut(len).blocks > 4.0 * f.wave; len *= 2) best = cut(2 * len);
  return best;
}

// How a call's keys are cut and who computes the parts.
struct PrefixPlan {
  PrefixProblem p;
  PrefixKernel pre, suf;
  bool whole;   // no parts: a block takes all of a request's keys (few-row or fp32 kernel)
};

PrefixPlan plan_prefix(int B, int H, int H_kv, int S_Q, int S_P, int S_cap, int d, lvx_dtype dt, float scale) {
  PrefixPlan plan;
  PrefixProblem& p = plan.p;
  p = PrefixProblem{};
  p.B = B; p.H = H; p.H_kv = H_kv; p.G = H / H_kv; p.S_Q = S_Q; p.S_P = S_P; p.S_cap = S_cap; p.d = d;
  p.scale_log2 = (scale > 0.f ? scale : 1.0f / sqrtf((float)d)) * kLog2e;
  const long long pre_rows = (long long)B * S_Q * p.G, suf_rows = (long long)S_Q * p.G;
  auto pre_cut = [&](PrefixKernel k) {
    const Shape f = shape_of(k, p, pre_rows, S_P);
    return cut_prefix(k, f, p, (pre_rows + f.rows - 1) / f.rows * H_kv);
  };
  auto suf_cut = [&](PrefixKernel k) {
    const Shape f = shape_of(k, p, suf_rows, S_cap);
    return cut_suffix(k, f, p, (suf_rows + f.rows - 1) / f.rows * H_kv * B);
  };
  Cut pre, suf;
  if (dt == LVX_FP32 || p.G > kPrefixTile) {
    plan.pre = plan.suf = kPrefixFp32;
    pre = pre_cut(kPrefixFp32);
    suf = suf_cut(kPrefixFp32);
  } else {
    const Cut pr = pre_cut(kPrefixRows), pt = pre_cut(kPrefixTc), sr = suf_cut(kPrefixRows), st = suf_cut(kPrefixTc);
    plan.pre = pr.us <= pt.us ? kPrefixRows : kPrefixTc;
    plan.suf = sr.us <= st.us ? kPrefixRows : kPrefixTc;
    pre = plan.pre == kPrefixRows ? pr : pt;
    suf = plan.suf == kPrefixRows ? sr : st;
  }
  // one launch's blocks share the machine; two kernels follow one another
  const double one = std::max({pre.us, suf.us, (pre.blocks + suf.blocks) / shape_of(plan.pre, p, suf_rows, S_cap).wave *
                                                  block_us(plan.pre, d, std::min(pre.len, 128))});
  const double parts = (plan.pre == plan.suf ? one : pre.us + suf.us) + merge_us(p, pre.n + suf.n * 0.5);
  // against whole requests
  const PrefixKernel k = plan.pre == kPrefixFp32 ? kPrefixFp32 : kPrefixRows;
  const double most = (double)S_P + S_cap, mean = S_P + S_cap * 0.5;
  const Shape f = shape_of(k, p, suf_rows, most);
  const long long blocks = (suf_rows + f.rows - 1) / f.rows * H_kv * B;
  const double whole = std::max({block_us(k, d, most), std::ceil((double)blocks / f.wave) * block_us(k, d, mean),
                                 block_us(k, d, 0) + l2_us(blocks, mean, d) * (k == kPrefixFp32 ? 2 : 1)});
  plan.whole = whole <= parts;
  if (plan.whole) pre.n = suf.n = 0;
  p.n_pre = pre.n;
  p.pre_len = pre.len;
  p.n_suf = suf.n;
  p.suf_len = suf.len;
  return plan;
}

size_t o_bytes(const PrefixProblem& p) {
  return align256((size_t)(p.n_pre + p.n_suf) * p.B * p.S_Q * p.H * p.d * sizeof(float));
}
size_t l_bytes(const PrefixProblem& p) {
  return align256((size_t)(p.n_pre + p.n_suf) * p.B * p.S_Q * p.H * sizeof(float));
}

}  // namespace
}  // namespace lvx

using namespace lvx;

extern "C" {

size_t lvx_attn_prefix_workspace(int B, int H, int H_kv, int S_Q, int S_P, int S_cap, int d, lvx_dtype dt) {
  if (check_prefix(B, H, H_kv, S_Q, S_P, S_cap, d, dt) != LVX_OK) return 0;
  const PrefixProblem p = plan_prefix(B, H, H_kv, S_Q, S_P, S_cap, d, dt, 0.f).p;
  return std::max(o_bytes(p) + l_bytes(p), (size_t)256);
}

lvx_status lvx_attn_prefix(const void* q, const void* k_prefix, const void* v_prefix, const void* k_suffix,
                           const void* v_suffix, const int32_t* suffix_len, void* out, float* lse, int B, int H,
                           int H_kv, int S_Q, int S_P, int S_cap, int d, lvx_dtype dt, float scale,
                           void* workspace, size_t ws_bytes, lvx_stream stream) {
  const lvx_status st = check_prefix(B, H, H_kv, S_Q, S_P, S_cap, d, dt);
  if (st != LVX_OK) return st;
  const void* ptrs[] = {q, out, lse, workspace};
  for (const void* ptr : ptrs)
    if (!ptr || !aligned16(ptr)) return LVX_ERR_INVALID_ARG;
  if (S_P > 0 && (!k_prefix || !v_prefix || !aligned16(k_prefix) || !aligned16(v_prefix)))
    return LVX_ERR_INVALID_ARG;
  if (S_cap > 0 && (!k_suffix || !v_suffix || !suffix_len || !aligned16(k_suffix) || !aligned16(v_suffix) ||
                    (reinterpret_cast<uintptr_t>(suffix_len) & 3u)))
    return LVX_ERR_INVALID_ARG;
  if (!(scale == scale)) return LVX_ERR_INVALID_ARG;   // NaN scale
  PrefixPlan plan = plan_prefix(B, H, H_kv, S_Q, S_P, S_cap, d, dt, scale);
  PrefixProblem& p = plan.p;
  if (ws_bytes < std::max(o_bytes(p) + l_bytes(p), (size_t)256)) return LVX_ERR_WORKSPACE;
  p.suffix_len = suffix_len;
  p.o_parts = reinterpret_cast<float*>(workspace);
  p.l_parts = reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) + o_bytes(p));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (plan.whole) {
    e = plan.pre == kPrefixFp32 ? launch_prefix_fp32(p, dt, out, lse, q, k_prefix, v_prefix, k_suffix, v_suffix, s)
                                : launch_prefix_rows(p, false, true, out, lse, q, k_prefix, v_prefix, k_suffix, v_suffix, s);
    return e == cudaSuccess ? LVX_OK : LVX_ERR_CUDA;
  }
  const bool has_pre = p.n_pre > 0, has_suf = p.n_suf > 0;
  if (plan.pre == kPrefixFp32) {   // the type and G decide it for both
    e = launch_prefix_fp32(p, dt, nullptr, nullptr, q, k_prefix, v_prefix, k_suffix, v_suffix, s);
  } else {
    const bool pre_tc = has_pre && plan.pre == kPrefixTc, suf_tc = has_suf && plan.suf == kPrefixTc;
    const bool pre_rows = has_pre && plan.pre == kPrefixRows, suf_rows = has_suf && plan.suf == kPrefixRows;
    const bool rows = pre_rows || suf_rows;
    if (rows)
      e = launch_prefix_rows(p, pre_rows, suf_rows, nullptr, nullptr, q, k_prefix, v_prefix, k_suffix, v_suffix, s);
    if (e == cudaSuccess && (pre_tc || suf_tc))
      e = launch_prefix_tc(p, pre_tc, suf_tc, rows, q, k_prefix, v_prefix, k_suffix, v_suffix, s);
  }
  if (e == cudaSuccess) e = launch_prefix_merge(p, dt, out, lse, s);
  return e == cudaSuccess ? LVX_OK : LVX_ERR_CUDA;
}

lvx_status lvx_selftest_prefix_plan(int B, int H, int H_kv, int S_Q, int S_P, int S_cap, int d, lvx_dtype dt,
                                    int plan[7]) {
  const lvx_status st = check_prefix(B, H, H_kv, S_Q, S_P, S_cap, d, dt);
  if (st != LVX_OK) return st;
  if (!plan) return LVX_ERR_INVALID_ARG;
  const PrefixPlan x = plan_prefix(B, H, H_kv, S_Q, S_P, S_cap, d, dt, 0.f);
  // whole requests: the few-row kernel in bf16, whatever the parts would have taken
  const bool rows = x.whole && x.pre != kPrefixFp32;
  const int values[7] = {rows ? kPrefixRows : x.pre, rows ? kPrefixRows : x.suf, x.p.n_pre, x.p.pre_len,
                         x.p.n_suf, x.p.suf_len, x.whole};
  std::copy(values, values + 7, plan);
  return LVX_OK;
}

}  // extern "C"
