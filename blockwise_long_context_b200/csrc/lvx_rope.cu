// Rotary positions with several axes, and the RMS norm of every query and key
// head with that rotation in the same pass (forward and backward).
//
// Rotation of head row x [d] at token r.  Pair i (of n_freq) turns by the angle
// theta_i = pos[axis_of[i]][r] * inv_freq[i]:
//   a' = a cos - b sin,   b' = b cos + a sin,
// (a, b) = (x[i], x[i + n_freq]) or, adjacent, (x[2i], x[2i + 1]).  Elements from
// 2 n_freq on pass.  The map is orthogonal: its gradient is the inverse rotation.
// Norm:  y = R (w o x h),  h = (mean x^2 + eps)^(-1/2).  With g = R^T dy, xh = x h:
//   dx = h (w o g - xh mean(w o g o xh)),   dw = sum over rows of g o xh.
//
// Angles.  A position times a frequency reaches 10^7 radians, where a 32-bit
// product has lost the turn's fraction.  The frequency is held in turns as a
// 64-bit fraction F = frac(inv_freq / 2 pi) 2^64; the low 64 bits of pos * F
// are then the angle modulo one turn (two's complement, so for negative positions too),
// off by |pos| * 2^-54 turns at most for frequencies up to 1 (F comes from a double product).
// The top 32 bits go to a float.  16-bit outputs take the special-function unit's
// sine and cosine (absolute error below 2^-20 on [-pi, pi], against the 2^-9 of
// the output's rounding); 32-bit outputs take the Taylor series of the remainder to the
// nearest quarter turn (off by 1.6 x 2^-24 at most).
//
// All three are bound by HBM: 2 (forward) or 3 (backward) streams of
// (H + H_kv) d elements a token, a few operations an element.  A group of LP lanes
// (one a 8 pairs, and a power of two for the norms) holds a head row in registers, so
// that a row's norm and the backward's dot product are shuffles inside the group.  A
// group takes up to 8 heads of one token: its cosines and sines are computed once, in
// the registers that use them, while the first rows are on their way (8 heads: one
// sine a 16 elements; a table in shared memory for a tile of tokens was slower, 58 us
// for 65536 x 8 rows of 128, because a block's loads stopped while it was filled).
// The next rows are loaded as soon as a row's registers are unpacked, so that a lane has 32 to
// 128 bytes on their way throughout.  Sums and statistics are 32-bit; outputs are rounded
// once.  Device time, bf16, heads of 128: 65536 x 8 rows rotated 46 us (88% of the copy
// rate), 32768 x 40 normed and rotated 112 (91%), their backward at 16382 tokens 100 (77 of
// traffic; instruction issue is 60% busy).
#include <algorithm>

#include "lvx_after.cuh"
#include "lvx_rope.cuh"

namespace lvx {
namespace {

constexpr int kThreads = 256;
constexpr int PP = 8;             // pairs a lane
constexpr int kMaxPairs = 128;

enum Mode { kRotate, kNormFwd, kNormBwd };

// Pair i of lane l's eight: the lanes take runs of W = 2^lw pairs in turn.  W depends on
// the type, d and n_freq alone, so that sums run in the same order whatever the strides;
// a short W spreads a warp's narrow loads over consecutive addresses.
__device__ __forceinline__ int pair_of(int i, int l, int lp, int lw) {
  return ((((i >> lw) * lp) + l) << lw) + (i & ((1 << lw) - 1));
}

// Where they lie in a row.  Chunk c holds the V <= W pairs from p0 on, as two runs of V
// elements: half-split, at p0 and p0 + n_freq; adjacent pairs and passing elements, at
// 2 p0 and 2 p0 + V.  For V > 1 the host sees to it that no chunk straddles n_freq
// (half-split) or the row's end.
template <int V, bool ADJ>
struct Place {
  int a[PP / V], b[PP / V];
  bool in[PP / V];
  __device__ __forceinline__ Place(int l, int lp, int lw, int d, int n_freq) {
#pragma unroll
    for (int c = 0; c < PP / V; ++c) {
      const int p0 = pair_of(c * V, l, lp, lw);
      in[c] = 2 * p0 < d;
      const bool split = !ADJ && p0 < n_freq;
      a[c] = split ? p0 : 2 * p0;
      b[c] = split ? p0 + n_freq : 2 * p0 + V;
    }
  }
};

// A lane's part of a head row as it lies in memory: chunk by chunk, both runs.
template <typename T, int V, bool ADJ>
struct Row {
  static constexpr int kWords = 2 * PP * (int)sizeof(T) / 4;
  static constexpr int kRun = V * (int)sizeof(T) / 4;   // words of a run (0: half a word)
  // both runs of a chunk in one access (the host sees to the alignment)
  static constexpr bool kOne = ADJ && V > 1 && kRun <= 2;
  uint32_t w[kWords];

  __device__ __forceinline__ void load(const T* p, const Place<V, ADJ>& at, bool on) {
#pragma unroll
    for (int c = 0; c < PP / V; ++c) {
      const bool get = on && at.in[c];
      if constexpr (kOne && kRun == 2) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (get) u = *reinterpret_cast<const uint4*>(p + at.a[c]);
        w[4 * c] = u.x; w[4 * c + 1] = u.y; w[4 * c + 2] = u.z; w[4 * c + 3] = u.w;
      } else if constexpr (kOne) {
        uint2 u = make_uint2(0, 0);
        if (get) u = *reinterpret_cast<const uint2*>(p + at.a[c]);
        w[2 * c] = u.x; w[2 * c + 1] = u.y;
      } else if constexpr (kRun == 4) {
        uint4 u = make_uint4(0, 0, 0, 0), v = u;
        if (get) {
          u = *reinterpret_cast<const uint4*>(p + at.a[c]);
          v = *reinterpret_cast<const uint4*>(p + at.b[c]);
        }
        w[8 * c] = u.x; w[8 * c + 1] = u.y; w[8 * c + 2] = u.z; w[8 * c + 3] = u.w;
        w[8 * c + 4] = v.x; w[8 * c + 5] = v.y; w[8 * c + 6] = v.z; w[8 * c + 7] = v.w;
      } else if constexpr (kRun == 2) {
        uint2 u = make_uint2(0, 0), v = u;
        if (get) {
          u = *reinterpret_cast<const uint2*>(p + at.a[c]);
          v = *reinterpret_cast<const uint2*>(p + at.b[c]);
        }
        w[4 * c] = u.x; w[4 * c + 1] = u.y; w[4 * c + 2] = v.x; w[4 * c + 3] = v.y;
      } else if constexpr (kRun == 1) {
        w[2 * c] = get ? *reinterpret_cast<const uint32_t*>(p + at.a[c]) : 0u;
        w[2 * c + 1] = get ? *reinterpret_cast<const uint32_t*>(p + at.b[c]) : 0u;
      } else {
        const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
        w[c] = get ? (uint32_t)h[at.a[c]] | (uint32_t)h[at.b[c]] << 16 : 0u;
      }
    }
  }
  __device__ __forceinline__ void store(T* p, const Place<V, ADJ>& at, bool on) const {
#pragma unroll
    for (int c = 0; c < PP / V; ++c) {
      if (!(on && at.in[c])) continue;
      if constexpr (kOne && kRun == 2) {
        *reinterpret_cast<uint4*>(p + at.a[c]) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
      } else if constexpr (kOne) {
        *reinterpret_cast<uint2*>(p + at.a[c]) = make_uint2(w[2 * c], w[2 * c + 1]);
      } else if constexpr (kRun == 4) {
        *reinterpret_cast<uint4*>(p + at.a[c]) = make_uint4(w[8 * c], w[8 * c + 1], w[8 * c + 2], w[8 * c + 3]);
        *reinterpret_cast<uint4*>(p + at.b[c]) = make_uint4(w[8 * c + 4], w[8 * c + 5], w[8 * c + 6], w[8 * c + 7]);
      } else if constexpr (kRun == 2) {
        *reinterpret_cast<uint2*>(p + at.a[c]) = make_uint2(w[4 * c], w[4 * c + 1]);
        *reinterpret_cast<uint2*>(p + at.b[c]) = make_uint2(w[4 * c + 2], w[4 * c + 3]);
      } else if constexpr (kRun == 1) {
        *reinterpret_cast<uint32_t*>(p + at.a[c]) = w[2 * c];
        *reinterpret_cast<uint32_t*>(p + at.b[c]) = w[2 * c + 1];
      } else {
        uint16_t* h = reinterpret_cast<uint16_t*>(p);
        h[at.a[c]] = (uint16_t)w[c];
        h[at.b[c]] = (uint16_t)(w[c] >> 16);
      }
    }
  }
  // element e of the lane's 16, in memory order
  static constexpr __device__ __forceinline__ int where(int i, bool second) {   // ... of pair i
    const int c = i / V, j = i % V;
    return c * 2 * V + (ADJ ? 2 * j + (second ? 1 : 0) : j + (second ? V : 0));
  }
  __device__ __forceinline__ float get(int e) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[e]);
    else return __uint_as_float(e & 1 ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16);
  }
  // x[0..7] first elements of the lane's pairs, x[8..15] their partners
  __device__ __forceinline__ void unpack(float (&x)[2 * PP]) const {
#pragma unroll
    for (int i = 0; i < PP; ++i) {
      x[i] = get(where(i, false));
      x[PP + i] = get(where(i, true));
    }
  }
  __device__ __forceinline__ void pack(const float (&x)[2 * PP]) {
    float u[2 * PP];
#pragma unroll
    for (int i = 0; i < PP; ++i) {
      u[where(i, false)] = x[i];
      u[where(i, true)] = x[PP + i];
    }
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (sizeof(T) == 4) {
        w[i] = __float_as_uint(u[i]);
      } else {
        const __nv_bfloat162 t = __floats2bfloat162_rn(u[2 * i], u[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&t);
      }
    }
  }
};

// Rows whose second halves start at an odd place (half-split, n_freq not a multiple of 4;
// V = 0).  Their runs are too narrow for the loads and stores (640k rows of 128 with
// n_freq = 63: 171 us), so a lane moves 16-byte words of the row as it lies, and the
// elements change lanes through the warp's corner of shared memory.
template <typename T>
struct Row<T, 0, false> {
  static constexpr int kWords = 2 * PP * (int)sizeof(T) / 4;
  static constexpr int kEach = 16 / (int)sizeof(T);   // elements of a 16-byte word
  uint4 w[kWords / 4];

  __device__ __forceinline__ void load(const T* p, int l, int lp, int d, bool on) {
#pragma unroll
    for (int c = 0; c < kWords / 4; ++c) {
      const int e = (c * lp + l) * kEach;
      w[c] = on && e < d ? *reinterpret_cast<const uint4*>(p + e) : make_uint4(0, 0, 0, 0);
    }
  }
  // corner: this row's place in shared memory
  __device__ __forceinline__ void unpack(float (&x)[2 * PP], T* corner, const Place<1, false>& at, int l, int lp,
                                         int d) const {
#pragma unroll
    for (int c = 0; c < kWords / 4; ++c) {
      const int e = (c * lp + l) * kEach;
      if (e < d) *reinterpret_cast<uint4*>(corner + e) = w[c];
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < PP; ++i) {
      x[i] = at.in[i] ? Elem<T>::to_f(corner[at.a[i]]) : 0.f;
      x[PP + i] = at.in[i] ? Elem<T>::to_f(corner[at.b[i]]) : 0.f;
    }
    __syncwarp();
  }
  static __device__ __forceinline__ void store(T* p, const float (&x)[2 * PP], T* corner, const Place<1, false>& at,
                                               int l, int lp, int d, bool on) {
#pragma unroll
    for (int i = 0; i < PP; ++i) {
      if (!at.in[i]) continue;
      corner[at.a[i]] = Elem<T>::from_f(x[i]);
      corner[at.b[i]] = Elem<T>::from_f(x[PP + i]);
    }
    __syncwarp();
#pragma unroll
    for (int c = 0; c < kWords / 4; ++c) {
      const int e = (c * lp + l) * kEach;
      if (on && e < d) *reinterpret_cast<uint4*>(p + e) = *reinterpret_cast<const uint4*>(corner + e);
    }
    __syncwarp();
  }
};

// Pair i of the lane turns by t[i] = (cos, sin) when bit i of `turns` is set; the
// others keep their values (0 * infinity would not).  all: every lane's pairs turn.
__device__ __forceinline__ void rotate(float (&x)[2 * PP], const float2 (&t)[PP], uint32_t turns, bool all) {
  if (all) {
#pragma unroll
    for (int i = 0; i < PP; ++i) {
      const float a = x[i], b = x[PP + i];
      x[i] = a * t[i].x - b * t[i].y;
      x[PP + i] = b * t[i].x + a * t[i].y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < PP; ++i) {
      const float a = x[i], b = x[PP + i];
      x[i] = turns >> i & 1 ? a * t[i].x - b * t[i].y : a;
      x[PP + i] = turns >> i & 1 ? b * t[i].x + a * t[i].y : b;
    }
  }
}

__device__ __forceinline__ float group_sum(float v, int lp) {
  for (int o = lp >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A frequency in turns, as a 64-bit fraction.
__device__ __forceinline__ uint64_t turn_fraction(float inv_freq) {
  const double f = (double)inv_freq * 0.15915494309189533577;   // 1 / (2 pi)
  return __double2ull_rd((f - floor(f)) * 18446744073709551616.0);
}

// (cos, sin) of the angle F turns times pos.
template <typename T>
__device__ __forceinline__ float2 turn_of(uint64_t F, int pos, bool back) {
  const uint32_t phase = (uint32_t)((F * (uint64_t)(int64_t)pos) >> 32);
  float2 cs;
  if (sizeof(T) == 2) {
    const float t = (float)(int)phase * 2.3283064365386963e-10f;   // turns in [-1/2, 1/2]
    cs.x = __cosf(t * 6.283185307179586f);
    cs.y = __sinf(t * 6.283185307179586f);
  } else {
    // the remainder x to the nearest quarter turn (two bits more than a float of the whole turn
    // keeps), and the Taylor series of sin 2 pi x and cos 2 pi x, which end below 2^-29 at x = 1/8
    constexpr double w = 6.283185307179586477, w2 = w * w, w4 = w2 * w2;
    const uint32_t quarter = (phase + (1u << 29)) >> 30;
    const float x = (float)(int)(phase - (quarter << 30)) * 2.3283064365386963e-10f, x2 = x * x;
    float p = fmaf((float)(w4 * w4 * w / 362880), x2, (float)(-w4 * w2 * w / 5040));
    p = fmaf(fmaf(p, x2, (float)(w4 * w / 120)), x2, (float)(-w2 * w / 6));
    const float sn = fmaf(x, (float)w, x * fmaf(x2, p, (float)(w - (float)w)));
    float q = fmaf((float)(-w4 * w4 * w2 / 3628800), x2, (float)(w4 * w4 / 40320));
    q = fmaf(fmaf(q, x2, (float)(-w4 * w2 / 720)), x2, (float)(w4 / 24));
    const float c = fmaf(x2, fmaf(x2, q, (float)(-w2 / 2)), 1.f);
    const float u = quarter & 1 ? sn : c, v = quarter & 1 ? c : sn;
    cs.x = (quarter + 1) & 2 ? -u : u;
    cs.y = quarter & 2 ? -v : v;
  }
  if (back) cs.y = -cs.y;
  return cs;
}

// Rows that a lane has on their way, and blocks that an SM is to hold at once (their
// registers are held to it).
template <typename T>
constexpr int batch(Mode m) {
  return m == kNormBwd ? 1 : sizeof(T) == 4 ? 2 : 4;
}
template <typename T, int V>
constexpr int blocks_per_sm(Mode m) {
  return m == kNormBwd && (V < 4 || sizeof(T) == 4) ? 1 : 2;
}
constexpr int kMostBlocks = 148 * 2;

template <typename T, int V, bool ADJ, Mode M>
__global__ void __launch_bounds__(kThreads, blocks_per_sm<T, V>(M))
rope_kernel(const RopeArgs a) {
  constexpr int NB = batch<T>(M), VP = V ? V : 1;
  constexpr bool kStaged = V == 0;
  __shared__ uint64_t fraction[kMaxPairs];
  __shared__ int axis[kMaxPairs];
  extern __shared__ __align__(16) unsigned char dynamic[];   // corners of V = 0; at the end dw [groups][d]
  const int side = blockIdx.x < (unsigned)a.blocks[0] ? 0 : 1;   // queries or keys
  const RopeSide s = a.side[side];
  const int block = blockIdx.x - (side ? a.blocks[0] : 0);
  const int lp = a.lanes, lane = threadIdx.x & 31, l = lane % lp;
  const int per_warp = 32 / lp, groups = kThreads / 32 * per_warp;
  const int group = threadIdx.x / 32 * per_warp + lane / lp;
  const bool idle = lane >= per_warp * lp;   // the warp's last lanes, where lp does not divide 32
  const Place<VP, ADJ> at(l, lp, a.lw, a.d, a.n_freq);
  T* corner = reinterpret_cast<T*>(dynamic) +
              (size_t)(threadIdx.x / 32 * (per_warp + 1) + lane / lp) * (a.d + 16 / sizeof(T));

  // The group's items (a token and `step` of its heads): every (blocks * groups)-th.  The loops are
  // uniform in the block, as the shuffles want it.
  const uint32_t stride = (uint32_t)a.blocks[side] * groups, first = (uint32_t)block * groups;
  const uint32_t dtok = stride / s.chunks, dchunk = stride % s.chunks;
  uint32_t tok = (first + group) / s.chunks, chunk = (first + group) % s.chunks;
  uint32_t lead = first / s.chunks, lead_chunk = first % s.chunks;
  const T *xs, *gs;
  T* ys;
  int n;   // rows of the item
  auto place = [&] {
    const bool on = tok < (uint32_t)a.rows && !idle;
    const size_t t64 = on ? tok : 0, h = (size_t)(chunk * s.step) * a.d;
    xs = reinterpret_cast<const T*>(s.x) + t64 * s.x_stride + h;
    if (M == kNormBwd) gs = reinterpret_cast<const T*>(s.dy) + t64 * s.dy_stride + h;
    ys = reinterpret_cast<T*>(s.y) + t64 * s.y_stride + h;
    n = on ? min(s.step, s.heads - (int)chunk * s.step) : 0;
  };
  auto advance = [&](uint32_t& t, uint32_t& c) {
    t += dtok;
    c += dchunk;
    if (c >= (uint32_t)s.chunks) { c -= s.chunks; ++t; }
  };
  Row<T, V, ADJ> x[NB], g[NB];
  auto fetch = [&](int j, int h) {   // row h of the item into slot j
    if constexpr (kStaged) {
      x[j].load(xs + h * a.d, l, lp, a.d, h < n);
      if (M == kNormBwd) g[j].load(gs + h * a.d, l, lp, a.d, h < n);
    } else {
      x[j].load(xs + h * a.d, at, h < n);
      if (M == kNormBwd) g[j].load(gs + h * a.d, at, h < n);
    }
  };
  auto unpack = [&](const Row<T, V, ADJ>& r, float (&v)[2 * PP]) {
    if constexpr (kStaged) r.unpack(v, corner, at, l, lp, a.d);
    else r.unpack(v);
  };
  place();
#pragma unroll
  for (int j = 0; j < NB; ++j) fetch(j, j);

  for (int e = threadIdx.x; e < lp * PP; e += kThreads) {   // lane by lane
    const int p = pair_of(e % PP, e / PP, lp, a.lw);
    const bool is = p < a.n_freq;
    const int x = is ? __ldg(a.axis_of + p) : -1;
    const float f = is ? __ldg(a.inv_freq + p) : 0.f;
    axis[e] = x >= 0 && x < a.n_axes ? x : -1;
    fraction[e] = turn_fraction(f);
  }
  Row<T, VP, ADJ> weight;   // packed: registers are what bounds the loads in flight
  float dw[2 * PP];
  if (M != kRotate) {
    float one[2 * PP];
#pragma unroll
    for (int i = 0; i < 2 * PP; ++i) { one[i] = 1.f; dw[i] = 0.f; }
    if (s.w) weight.load(reinterpret_cast<const T*>(s.w), at, true);
    else weight.pack(one);
  }
  if (M == kNormBwd) let_next_start();   // dw_sum_kernel follows
  __syncthreads();
  uint32_t turns = 0, fresh = 0;   // pairs that turn; those of another axis than the pair before
  int last = -1;
  bool all = true;
#pragma unroll
  for (int i = 0; i < PP; ++i) {
    const int x = axis[l * PP + i];
    if (x >= 0) {
      turns |= 1u << i;
      if (x != last) fresh |= 1u << i;
      last = x;
    } else if (at.in[i / VP]) {
      all = false;
    }
  }
  all = __all_sync(0xffffffffu, all);   // pairs past the row's end may turn as they like

  while (lead < (uint32_t)a.rows) {
    float2 t[PP];
    {
      int pos[PP];
#pragma unroll
      for (int i = 0; i < PP; ++i) {
        pos[i] = 0;
        if (n > 0 && (fresh >> i & 1)) pos[i] = __ldg(a.pos + (size_t)axis[l * PP + i] * a.rows + tok);
      }
#pragma unroll
      for (int i = 0; i < PP; ++i) {
        if (i > 0 && !(fresh >> i & 1)) pos[i] = pos[i - 1];
        t[i] = make_float2(1.f, 0.f);
        if (turns) t[i] = turn_of<T>(fraction[l * PP + i], pos[i], (M == kNormBwd) != (a.inverse != 0));
      }
    }
    T* const y_item = ys;
    const int n_item = n;
    advance(tok, chunk);
    advance(lead, lead_chunk);
    for (int h = 0; h < s.step; h += NB) {
      const bool end = h + NB >= s.step;
      if (end) place();   // the next item's rows follow
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        if (j > 0 && h + j >= s.step) {
          fetch(j, j);
          continue;
        }
        const bool in = h + j < n_item;
        float v[2 * PP], w[2 * PP];
        unpack(x[j], v);
        if (M == kNormBwd) {
          float y[2 * PP];
          unpack(g[j], y);
          fetch(j, end ? j : h + NB + j);
          weight.unpack(w);
          rotate(y, t, turns, all);
          // z = g x:  m = sum w z,  dw += z r,  dx = r (w g) - x r^3 m / d
          float q = 0.f, m = 0.f, z[2 * PP];
#pragma unroll
          for (int i = 0; i < 2 * PP; ++i) {
            z[i] = y[i] * v[i];
            q = fmaf(v[i], v[i], q);
            m = fmaf(w[i], z[i], m);
          }
          const float r = rsqrtf(group_sum(q, lp) * a.inv_d + a.eps);
          m = group_sum(m, lp);
          const float c = -(r * r) * (r * (m * a.inv_d)), r_in = in ? r : 0.f;
#pragma unroll
          for (int i = 0; i < 2 * PP; ++i) {
            dw[i] = fmaf(z[i], r_in, dw[i]);
            v[i] = fmaf(w[i] * y[i], r, v[i] * c);
          }
        } else {
          fetch(j, end ? j : h + NB + j);
          if (M == kNormFwd) {
            weight.unpack(w);
            float q = 0.f;
#pragma unroll
            for (int i = 0; i < 2 * PP; ++i) q = fmaf(v[i], v[i], q);
            const float r = rsqrtf(group_sum(q, lp) * a.inv_d + a.eps);
#pragma unroll
            for (int i = 0; i < 2 * PP; ++i) v[i] = v[i] * r * w[i];
          }
          rotate(v, t, turns, all);
        }
        T* to = y_item + (h + j) * a.d;
        if constexpr (kStaged) {
          Row<T, V, ADJ>::store(to, v, corner, at, l, lp, a.d, in);
        } else {
          Row<T, V, ADJ> o;
          o.pack(v);
          o.store(to, at, in);
        }
      }
    }
  }

  if (M == kNormBwd) {
    // the block's sum of dw over its groups, in a fixed order
    if (kStaged) __syncthreads();
    float* sdw = reinterpret_cast<float*>(dynamic);   // [groups][d]
    float* mine = sdw + group * a.d;
#pragma unroll
    for (int i = 0; i < PP; ++i) {
      const int c = i / VP, j = i % VP;
      if (at.in[c]) {
        mine[at.a[c] + (ADJ ? 2 * j : j)] = dw[i];
        mine[ADJ ? at.a[c] + 2 * j + 1 : at.b[c] + j] = dw[PP + i];
      }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.d; e += kThreads) {
      float t = 0.f;
      for (int k = 0; k < groups; ++k) t += sdw[k * a.d + e];
      a.dw_parts[(size_t)blockIdx.x * a.d + e] = t;
    }
  }
}

// dw[side][e] = sum over the side's blocks of their parts, in a fixed order: a
// block takes 32 columns, each of 32 warps every 32nd part.
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(32 * kSumWarps)
dw_sum_kernel(const float* parts, float* __restrict__ dw_q, float* __restrict__ dw_k, int n_q, int n_k, int d) {
  __shared__ float s[kSumWarps][32];
  const int side = blockIdx.x & 1;
  float* out = side ? dw_k : dw_q;
  const int lo = side ? n_q : 0, n = side ? n_k : n_q;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = (blockIdx.x >> 1) * 32 + lane;
  if (!out || n == 0) return;
  wait_for_previous();
  float t = 0.f;
  if (e < d) {
#pragma unroll 4
    for (int i = warp; i < n; i += kSumWarps) t += load_l2(parts + (size_t)(lo + i) * d + e);
  }
  s[warp][lane] = t;
  __syncthreads();
  if (warp == 0 && e < d) {
#pragma unroll
    for (int i = 1; i < kSumWarps; ++i) t += s[i][lane];
    out[e] = t;
  }
}

// Lanes of a group: as few as hold the row, for the norms rounded up to a power of two.
int lanes_of(int d, Mode m) {
  if (m == kRotate) return (d / 2 + PP - 1) / PP;
  return d <= 64 ? 4 : d <= 128 ? 8 : 16;
}
int groups_of(int lanes) { return kThreads / 32 * (32 / lanes); }

// Heads an item and blocks of a side, of which the machine holds `most` at once.  Eight
// heads share their angles; fewer, where the items would not fill the machine.
void plan_side(RopeArgs& a, int i, int most) {
  RopeSide& s = a.side[i];
  a.blocks[i] = 0;
  s.chunks = s.step = 1;
  if (s.heads == 0) return;
  const int groups = groups_of(a.lanes);
  int step = 8;
  while (step > 1 && (long long)a.rows * ((s.heads + step - 1) / step) < (long long)most * groups) step /= 2;
  s.chunks = (s.heads + step - 1) / step;
  s.step = (s.heads + s.chunks - 1) / s.chunks;
  a.blocks[i] = (int)std::min(((long long)a.rows * s.chunks + groups - 1) / groups, (long long)most);
}

template <typename T, int V, bool ADJ, Mode M>
cudaError_t launch(RopeArgs a, cudaStream_t s) {
  // the sides share the machine by their cost: an item's angles are worth about three rows
  constexpr int kBlocks = 148 * blocks_per_sm<T, V>(M);
  const int hq = a.side[0].heads, hk = a.side[1].heads;
  const int wq = hq + 3 * ((hq + 7) / 8), wk = hk + 3 * ((hk + 7) / 8);
  const int q = !hq ? 0 : !hk ? kBlocks : std::min(std::max(1, (int)((long long)kBlocks * wq / (wq + wk))), kBlocks - 1);
  a.lanes = lanes_of(a.d, M);
  plan_side(a, 0, q);
  plan_side(a, 1, kBlocks - q);
  size_t smem = V == 0 ? (size_t)(groups_of(a.lanes) + kThreads / 32) * (a.d * sizeof(T) + 16) : 0;
  if (M == kNormBwd) smem = std::max(smem, (size_t)groups_of(a.lanes) * a.d * sizeof(float));
  rope_kernel<T, V, ADJ, M><<<a.blocks[0] + a.blocks[1], kThreads, smem, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (M != kNormBwd || e != cudaSuccess || (!a.dw[0] && !a.dw[1])) return e;
  return launch_after(dw_sum_kernel, (a.d + 31) / 32 * 2, 32 * kSumWarps, 0, s, a.dw_parts, a.dw[0], a.dw[1],
                      a.blocks[0], a.blocks[1], a.d);
}

template <typename T, int V, Mode M>
cudaError_t launch_adj(const RopeArgs& a, bool adjacent, cudaStream_t s) {
  return adjacent ? launch<T, V, true, M>(a, s) : launch<T, V, false, M>(a, s);
}

// The widest run of elements that every row, pair chunk and pointer allows (pointers are
// 16-byte aligned: 8 bf16 or 4 fp32).
template <typename T, Mode M>
cudaError_t launch_vec(RopeArgs a, bool adjacent, cudaStream_t s) {
  long long strides = 0;
  for (const RopeSide& e : a.side)
    if (e.heads) strides |= e.x_stride | e.y_stride | (M == kNormBwd ? e.dy_stride : 0);
  const int widest = sizeof(T) == 2 ? 8 : 4, even = a.d / 2 | (adjacent ? 0 : a.n_freq);
  a.lw = 0;
  while (2 << a.lw <= widest && even % (2 << a.lw) == 0) ++a.lw;
  if (!adjacent && a.lw < 2 && strides % (16 / (int)sizeof(T)) == 0) return launch<T, 0, false, M>(a, s);
  // adjacent pairs: a chunk of 2 V elements is one run
  const long long bits = even | (!adjacent ? strides : strides % 2 ? 1 : strides / 2);
  if (sizeof(T) == 2 && bits % 8 == 0) return launch_adj<__nv_bfloat16, 8, M>(a, adjacent, s);
  if (bits % 4 == 0) return launch_adj<T, 4, M>(a, adjacent, s);
  return launch_adj<T, 1, M>(a, adjacent, s);
}

template <Mode M>
cudaError_t launch_type(const RopeArgs& a, bool adjacent, lvx_dtype dt, cudaStream_t s) {
  return dt == LVX_FP32 ? launch_vec<float, M>(a, adjacent, s) : launch_vec<__nv_bfloat16, M>(a, adjacent, s);
}

}  // namespace

// One part a block.
size_t rope_bwd_parts(int d) { return align256((size_t)kMostBlocks * d * sizeof(float)); }

cudaError_t launch_rope(RopeArgs a, RopeKind kind, bool adjacent, lvx_dtype dt, cudaStream_t s) {
  a.inv_d = 1.f / a.d;
  if (kind == kRopeNorm) return launch_type<kNormFwd>(a, adjacent, dt, s);
  if (kind == kRopeNormBwd) return launch_type<kNormBwd>(a, adjacent, dt, s);
  return launch_type<kRotate>(a, adjacent, dt, s);
}

}  // namespace lvx

using namespace lvx;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Checks shared by the three entry points; fills the rotation's part of `a`.
lvx_status set_rope(RopeArgs& a, const int32_t* pos, const float* inv_freq, const int32_t* axis_of, int rows,
                    int H, int H_kv, int d, int n_axes, int n_freq, int pairing, lvx_dtype dt) {
  if (rows < 1 || H < 0 || H_kv < 0 || H + H_kv < 1 || d < 1 || n_freq < 0) return LVX_ERR_INVALID_ARG;
  if (dt != LVX_FP32 && dt != LVX_BF16) return LVX_ERR_UNSUPPORTED;
  if (d > 256 || d % 8 != 0 || H > 65535 || H_kv > 65535) return LVX_ERR_UNSUPPORTED;
  if (n_freq > d / 2 || (pairing != LVX_PAIR_HALF && pairing != LVX_PAIR_ADJACENT)) return LVX_ERR_INVALID_ARG;
  if (n_freq > 0 && (n_axes < 1 || !pos || !inv_freq || !axis_of || !aligned4(pos) || !aligned4(inv_freq) ||
                     !aligned4(axis_of)))
    return LVX_ERR_INVALID_ARG;
  a = RopeArgs{};
  a.pos = pos; a.inv_freq = inv_freq; a.axis_of = axis_of;
  a.rows = rows; a.d = d; a.n_axes = n_axes; a.n_freq = n_freq;
  return LVX_OK;
}

// One side's tensors: null only when it has no heads, 16-byte aligned, rows that do not overlap.
lvx_status set_side(RopeSide& s, const void* x, const void* dy, void* y, const void* w, int heads, int d,
                    long long x_stride, long long dy_stride, long long y_stride, bool backward) {
  if (heads == 0) return LVX_OK;
  if (!x || !y || !aligned16(x) || !aligned16(y) || (w && !aligned16(w))) return LVX_ERR_INVALID_ARG;
  if (backward && (!dy || !aligned16(dy))) return LVX_ERR_INVALID_ARG;
  const long long least = (long long)heads * d;
  if (x_stride < least || y_stride < least || (backward && dy_stride < least)) return LVX_ERR_INVALID_ARG;
  s.x = x; s.dy = dy; s.y = y; s.w = w;
  s.x_stride = x_stride; s.dy_stride = dy_stride; s.y_stride = y_stride;
  s.heads = heads;
  return LVX_OK;
}

}  // namespace

extern "C" {

lvx_status lvx_rope_axes(const void* q, const void* k, void* q_out, void* k_out, const int32_t* pos,
                         const float* inv_freq, const int32_t* axis_of, int rows, int H, int H_kv, int d,
                         int n_axes, int n_freq, int pairing, int inverse, int64_t q_stride, int64_t k_stride,
                         int64_t q_out_stride, int64_t k_out_stride, lvx_dtype dt, lvx_stream stream) {
  RopeArgs a;
  lvx_status st = set_rope(a, pos, inv_freq, axis_of, rows, H, H_kv, d, n_axes, n_freq, pairing, dt);
  if (st != LVX_OK) return st;
  if (n_freq < 1) return LVX_ERR_INVALID_ARG;
  if ((st = set_side(a.side[0], q, nullptr, q_out, nullptr, H, d, q_stride, 0, q_out_stride, false)) != LVX_OK ||
      (st = set_side(a.side[1], k, nullptr, k_out, nullptr, H_kv, d, k_stride, 0, k_out_stride, false)) != LVX_OK)
    return st;
  a.inverse = inverse != 0;
  return launch_rope(a, kRopeOnly, pairing == LVX_PAIR_ADJACENT, dt, reinterpret_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? LVX_OK
             : LVX_ERR_CUDA;
}

lvx_status lvx_head_norm_rope(const void* q, const void* k, const void* w_q, const void* w_k, void* q_out,
                              void* k_out, const int32_t* pos, const float* inv_freq, const int32_t* axis_of,
                              int rows, int H, int H_kv, int d, int n_axes, int n_freq, int pairing, float eps,
                              int64_t q_stride, int64_t k_stride, int64_t q_out_stride, int64_t k_out_stride,
                              lvx_dtype dt, lvx_stream stream) {
  RopeArgs a;
  lvx_status st = set_rope(a, pos, inv_freq, axis_of, rows, H, H_kv, d, n_axes, n_freq, pairing, dt);
  if (st != LVX_OK) return st;
  if (!(eps >= 0.f)) return LVX_ERR_INVALID_ARG;   // NaN too
  if ((st = set_side(a.side[0], q, nullptr, q_out, w_q, H, d, q_stride, 0, q_out_stride, false)) != LVX_OK ||
      (st = set_side(a.side[1], k, nullptr, k_out, w_k, H_kv, d, k_stride, 0, k_out_stride, false)) != LVX_OK)
    return st;
  a.eps = eps;
  return launch_rope(a, kRopeNorm, pairing == LVX_PAIR_ADJACENT, dt, reinterpret_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? LVX_OK
             : LVX_ERR_CUDA;
}

size_t lvx_head_norm_rope_bwd_workspace(int d) { return d < 1 || d > 256 || d % 8 != 0 ? 0 : rope_bwd_parts(d); }

lvx_status lvx_head_norm_rope_bwd(const void* q, const void* k, const void* w_q, const void* w_k,
                                  const void* dq_out, const void* dk_out, void* dq, void* dk, float* dw_q,
                                  float* dw_k, const int32_t* pos, const float* inv_freq, const int32_t* axis_of,
                                  int rows, int H, int H_kv, int d, int n_axes, int n_freq, int pairing, float eps,
                                  int64_t q_stride, int64_t k_stride, int64_t dq_out_stride, int64_t dk_out_stride,
                                  int64_t dq_stride, int64_t dk_stride, lvx_dtype dt, void* workspace,
                                  size_t ws_bytes, lvx_stream stream) {
  RopeArgs a;
  lvx_status st = set_rope(a, pos, inv_freq, axis_of, rows, H, H_kv, d, n_axes, n_freq, pairing, dt);
  if (st != LVX_OK) return st;
  if (!(eps >= 0.f)) return LVX_ERR_INVALID_ARG;
  if ((st = set_side(a.side[0], q, dq_out, dq, w_q, H, d, q_stride, dq_out_stride, dq_stride, true)) != LVX_OK ||
      (st = set_side(a.side[1], k, dk_out, dk, w_k, H_kv, d, k_stride, dk_out_stride, dk_stride, true)) != LVX_OK)
    return st;
  if ((dw_q && !aligned16(dw_q)) || (dw_k && !aligned16(dw_k))) return LVX_ERR_INVALID_ARG;
  if (!workspace || !aligned16(workspace)) return LVX_ERR_INVALID_ARG;
  if (ws_bytes < rope_bwd_parts(d)) return LVX_ERR_WORKSPACE;
  a.eps = eps;
  a.dw_parts = reinterpret_cast<float*>(workspace);
  a.dw[0] = H ? dw_q : nullptr;
  a.dw[1] = H_kv ? dw_k : nullptr;
  return launch_rope(a, kRopeNormBwd, pairing == LVX_PAIR_ADJACENT, dt, reinterpret_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? LVX_OK
             : LVX_ERR_CUDA;
}

}  // extern "C"
