// Parts of shared-prefix attention on the tcgen05 tensor cores (bf16, fp32
// accumulation and softmax statistics).  Head widths below 64 or 128 run in tiles of
// that width: the copies' boxes reach past the row, and TMA fills the rest with zeros.
//
// One CTA computes one part (O_i, L_i) for up to 128 query rows that read the same
// keys: the G = H / H_kv query heads of a key/value head, times the tokens of all
// requests (a part of the prefix) or of one request (a part of its suffix).  The
// prefix is thus read once for 128 rows of the batch (by further row tiles from L2),
// and a row tile is full of queries where a tile per query head would hold S_Q rows.  Row i of a
// tile is head i % G of the group, token i / G: the box {64, G, tokens} of a TMA
// copy of q lands in that order.
//
// Bound: bytes, as long as the rows that share a key are fewer than about 250
// (4 d operations against 4 d bytes a key and row; 1650 TFLOP/s over 6.6 TB/s).
// So the key tiles are small (64 keys) and two CTAs share an SM: one's prologue,
// softmax and epilogue hide behind the other's loads, with 5 (d = 128) half tiles
// of 16 KB in flight for each (3 were half as slow again).  32 requests over 65536 keys of 8
// heads: 58 us with the merge, 4.6 TB/s.  With more rows the MMA pipe bounds it: 830 cycles a
// tile and SM against 696 of products (S tiles of N = 64 run at 58%); 128 requests over 32768
// keys 68 us, 1010 TFLOP/s.
//
// Roles (6 warps): warps 0-3 softmax, one thread per row; warp 4 the TMA producer
// and TMEM allocator; warp 5 the MMA issuer.
//   S_j = Q K_j^T into one of two TMEM buffers, so that S_{j+1} runs during the
//   softmax of S_j; P_j (bf16) is written over S_j; O += P_j V_j (A from TMEM).
// The running maximum moves only when it grows by more than 2^8, as in the block
// forward.  P is rounded to bf16 for the product (half a step, at most 2^-8 of each
// weight), the type in which V and the matrix unit take it; the row sum adds the
// unrounded fp32 weights.  Outputs of independent values are then off by 2.3e-3 (root mean
// square) where their own rounding alone is 1.65e-3; a second product with what is left of
// the weights brings them there and takes 115 -> 135 us for 128 requests over 32768 + 1024
// keys, 250 -> 327 for 8 x 64 tokens over 32768.
//
// Keys past a request's length.  The cache behind them may hold anything: their
// scores are replaced by -inf, and their rows of V are zeroed in shared memory
// before the product (0 * NaN is NaN).
#include <algorithm>

#include "lvx_prefix.cuh"
#include "lvx_ptx.cuh"

namespace lvx {
namespace {

using namespace ptx;

constexpr int BM = 128;        // query rows per tile (MMA M)
constexpr int BK = 64;         // keys per tile
constexpr int kThreads = 192;
constexpr float kRescaleThreshold = 8.0f;   // log2 units
constexpr float kRescaleFactor = 256.0f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr uint32_t kTmemCols = 256;   // S: SBUF x 64, O: d; two CTAs share the 512 columns

template <int D>
struct Layout {
  static constexpr uint32_t CHUNK_Q = BM * 128;   // 128 rows x 64 bf16
  static constexpr uint32_t CHUNK_K = BK * 128;
  static constexpr uint32_t Q_BYTES = BM * D * 2;
  static constexpr uint32_t SLOT = BK * D * 2;    // one K or V tile
  static constexpr int SLOTS = D == 128 ? 5 : 11;
  // K_j's slot is freed by the softmax, which sees S_j, and not by a commit: that spares the
  // issuing thread's time (d = 128, 128 requests over 32768 keys: 68 us, with the commit 71; d = 64,
  // where the softmax is the slower side: 64.5, with the commit 63)
  static constexpr bool LATE_K = D == 128;
  static constexpr int SBUF = 2;   // (three, where d = 64 leaves the columns, were no faster)
  static constexpr uint32_t OFF_RING = Q_BYTES;
  static constexpr uint32_t OFF_BAR = OFF_RING + SLOTS * SLOT;
  static constexpr uint32_t BYTES = OFF_BAR + 512;
  static constexpr uint32_t IDESC_QK = idesc_bf16_f32(BM, BK, false, false);
  static constexpr uint32_t IDESC_PV = idesc_bf16_f32(BM, D, false, true);
  static_assert(2 * (BYTES + 1024) <= 233472, "two CTAs an SM");
};

struct TcArgs {
  PrefixProblem p;
  unsigned int* err;
  int tokens;       // tokens per row tile: 128 / G
  int pre_tiles;    // row tiles over B * S_Q tokens
  int suf_tiles;    // row tiles over S_Q tokens
  int pre_items;    // CTAs of prefix parts: n_pre * H_kv * pre_tiles
  bool second;      // follows launch_prefix_rows
};

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
prefix_tc_kernel(const __grid_constant__ CUtensorMap map_qp, const __grid_constant__ CUtensorMap map_qs,
                 const __grid_constant__ CUtensorMap map_kp, const __grid_constant__ CUtensorMap map_vp,
                 const __grid_constant__ CUtensorMap map_ks, const __grid_constant__ CUtensorMap map_vs,
                 const TcArgs a) {
  using L = Layout<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const PrefixProblem& p = a.p;

  // which part, key/value head and rows
  const bool pre = blockIdx.x < (unsigned)a.pre_items;
  int idx = blockIdx.x - (pre ? 0 : a.pre_items);
  int part, g, b, tok0, n_tok, k0, kend, lim0;   // lim0: visible suffix keys of the first token
  if (pre) {
    const int rt = idx % a.pre_tiles;
    idx /= a.pre_tiles;
    g = idx % p.H_kv;
    part = idx / p.H_kv;
    b = 0;
    tok0 = rt * a.tokens;
    n_tok = min(a.tokens, p.B * p.S_Q - tok0);
    k0 = part * p.pre_len;
    kend = min(k0 + p.pre_len, p.S_P);
    lim0 = kend;
  } else {
    const int rt = idx % a.suf_tiles;
    idx /= a.suf_tiles;
    g = idx % p.H_kv;
    idx /= p.H_kv;
    const int s = idx % p.n_suf;
    b = idx / p.n_suf;
    const int n = suffix_keys(p, b);
    const int t0 = rt * a.tokens;
    tok0 = b * p.S_Q + t0;
    n_tok = min(a.tokens, p.S_Q - t0);
    part = p.n_pre + s;
    k0 = s * p.suf_len;
    kend = min(k0 + p.suf_len, n);
    lim0 = n - p.S_Q + t0 + 1;
  }
  let_next_start();
  if (a.second && blockIdx.x == gridDim.x - 1) wait_for_previous();   // see lvx_prefix.cuh
  if (k0 >= kend) return;   // the merge does not read this part
  const int T = (kend - k0 + BK - 1) / BK;

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::OFF_BAR);
  uint64_t* q_full = bars;
  uint64_t* mma_drain = bars + 1;
  uint64_t* o_done = bars + 2;    // [SBUF]: PV_j done, by the buffer of P_j
  uint64_t* s_full = bars + 5;    // [SBUF]
  uint64_t* p_full = bars + 8;    // [SBUF]
  uint64_t* full = bars + 11;             // [SLOTS]
  uint64_t* empty = full + L::SLOTS;      // [SLOTS]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 40);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int i = 0; i < L::SBUF; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_done[i], 1);
    }
    mbar_init(mma_drain, 1);
    for (int i = 0; i < L::SLOTS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    *abort_flag = 0;
    // a misplaced base would break the swizzled layout: give up before any copy
    if (smem_u32(smem) & 1023u) {
      record_error(a.err, kErrSmemAlign);
      *abort_flag = 1;
    }
    fence_barrier_init();
  }
  if (warp == 4) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tO = tmem + L::SBUF * BK;

  if (*abort_flag) {
    // nothing was started
  } else if (warp == 4) {
    if (lane == 0) {
      // ---------------------------------------------------------------- producer
      const CUtensorMap* mq = pre ? &map_qp : &map_qs;
      const CUtensorMap* mk = pre ? &map_kp : &map_ks;
      const CUtensorMap* mv = pre ? &map_vp : &map_vs;
      const int box_tokens = pre ? a.tokens : min(a.tokens, p.S_Q);
      mbar_arrive_expect_tx(q_full, (uint32_t)(box_tokens * p.G * D * 2));
      for (int c = 0; c < D / 64; ++c)
        tma_load_4d(smem + c * L::CHUNK_Q, mq, q_full, 64 * c, g * p.G, tok0, 0);
      int issued = 0, slot = 0;
      uint32_t ph = 1;
      for (int i = 0; i < 2 * T; ++i) {   // K_0, V_0, K_1, V_1, ...
        if (!mbar_wait(&empty[slot], ph, a.err, kErrTimeoutTma, abort_flag)) break;
        mbar_arrive_expect_tx(&full[slot], L::SLOT);
        uint8_t* dst = smem + L::OFF_RING + slot * L::SLOT;
        for (int c = 0; c < D / 64; ++c)
          tma_load_4d(dst + c * L::CHUNK_K, (i & 1) ? mv : mk, &full[slot], 64 * c, g, k0 + (i >> 1) * BK, b);
        issued = i + 1;
        if (++slot == L::SLOTS) { slot = 0; ph ^= 1u; }
      }
      if (*abort_flag) {
        // copies in flight must land before shared memory is released
        mbar_wait(q_full, 0, a.err, kErrTimeoutTma, nullptr);
        for (int i = issued > L::SLOTS ? issued - L::SLOTS : 0; i < issued; ++i)
          mbar_wait(&full[i % L::SLOTS], (i / L::SLOTS) & 1, a.err, kErrTimeoutTma, nullptr);
      }
    }
  } else if (warp == 5) {
    if (lane == 0) {
      // ---------------------------------------------------------------- MMA issuer
      // order, with n = SBUF - 1: S_0 .. S_{n-1}, then S_{j+n}, PV_j, ...: S_{j+n} overwrites
      // P_{j-1}, which PV_{j-1}, issued before it, reads first
      // The issuing thread bounds its CTA (8 MMAs of S took it 800 cycles, the pipe 440), so of
      // the descriptors only low words are kept, K-step offsets are constants, and the ring's
      // places are counted, not divided.
      constexpr uint32_t kHi = (1024u >> 4) | 1u << 14 | 2u << 29;   // smem_desc_sw128's high word
      const uint32_t q_lo = (smem_u32(smem) >> 4) | 1u << 16;
      const uint32_t k_lo = (smem_u32(smem + L::OFF_RING) >> 4) | 1u << 16;
      const uint32_t v_lo = (smem_u32(smem + L::OFF_RING) >> 4) | (L::CHUNK_K >> 4) << 16;
      auto desc = [](uint32_t lo) {
        uint64_t d;
        asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(kHi));
        return d;
      };
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        const bool ok = mbar_wait(bar, parity, a.err, kErrTimeoutMma, abort_flag);
        tc_fence_after();
        return ok;
      };
      int ks = 0, vs = 1;           // slots of the next K, the next V
      uint32_t kph = 0, vph = 0;    // ... and their phases
      auto step = [](int& slot, uint32_t& ph) {
        slot += 2;
        if (slot >= L::SLOTS) { slot -= L::SLOTS; ph ^= 1u; }
      };
      auto issue_s = [&](int buf) {
        if (!wait(&full[ks], kph)) return false;
        const uint32_t kd = k_lo + ks * (L::SLOT >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss(tmem + buf * BK, desc(q_lo + (kk >> 2) * (L::CHUNK_Q >> 4) + (kk & 3) * 2),
                 desc(kd + (kk >> 2) * (L::CHUNK_K >> 4) + (kk & 3) * 2), L::IDESC_QK, kk > 0);
        mma_commit(&s_full[buf]);
        if (!L::LATE_K) mma_commit(&empty[ks]);
        step(ks, kph);
        return true;
      };
      bool ok = wait(q_full, 0);
      for (int j = 0; j < L::SBUF - 1 && j < T && ok; ++j) ok = issue_s(j);
      int buf = 0, ahead = L::SBUF - 1;   // of P_j, of S_{j + SBUF - 1}
      uint32_t pph = 0;
      for (int j = 0; j < T && ok; ++j) {
        if (j + L::SBUF - 1 < T && !issue_s(ahead)) break;
        if (!wait(&full[vs], vph) || !wait(&p_full[buf], pph)) break;
        const uint32_t vd = v_lo + vs * (L::SLOT >> 4);
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk)
          mma_ts(tO, tmem + buf * BK + kk * 8, desc(vd + kk * (2048 >> 4)), L::IDESC_PV,
                 (j > 0 || kk > 0) ? 1u : 0u);
        mma_commit(&o_done[buf]);
        mma_commit(&empty[vs]);
        step(vs, vph);
        ahead = buf;
        if (++buf == L::SBUF) { buf = 0; pph ^= 1u; }
      }
      mma_commit(mma_drain);
    }
  } else {
    // ------------------------------------------------------------------ softmax
    const int row = warp * 32 + lane;
    const int tok = row / p.G;
    const bool live = tok < n_tok;
    const bool warp_live = warp * 32 < n_tok * p.G;
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    const int lim = pre ? kend : min(kend, lim0 + tok);   // keys [k0, lim) are visible
    const int lim_min = pre ? kend : min(kend, lim0);     // ... to every row
    const float sl2 = p.scale_log2;
    float m_ref = -INFINITY, l_sum = 0.f;
    bool ok = true;
    // A wait for a parity is a wait for a phase only while the phases before it are known to be
    // over and the one after it cannot be.  PV_j arrives at the barrier of its buffer: S_j seen
    // means PV_{j-SBUF} done, and PV_{j+1} waits for this warp.
    int buf = 0, last_buf = 0;           // of tile j, of the one before
    uint32_t ph = 0, last_ph = 0;
    int k_slot = 0;
    for (int j = 0; j < T; ++j) {
      const int key0 = k0 + BK * j;
      ok = __all_sync(0xffffffffu,
                      mbar_wait(&s_full[buf], ph, a.err, kErrTimeoutSoftmax, abort_flag));
      if (!ok) break;
      tc_fence_after();
      if (L::LATE_K) {
        if (threadIdx.x == 0) mbar_arrive(&empty[k_slot]);
        k_slot += 2;
        if (k_slot >= L::SLOTS) k_slot -= L::SLOTS;
      }
      if (!pre && key0 + BK > kend) {
        // the cache's rows behind the last key: zeroed, whatever they hold
        const int i = 2 * j + 1, slot = i % L::SLOTS;
        ok = __all_sync(0xffffffffu, mbar_wait(&full[slot], (i / L::SLOTS) & 1, a.err, kErrTimeoutSoftmax,
                                               abort_flag));
        if (!ok) break;
        uint8_t* v = smem + L::OFF_RING + slot * L::SLOT;
        const int r0 = kend - key0, words = (BK - r0) * 8 * (D / 64);   // 16-byte words
        for (int w = threadIdx.x; w < words; w += 128) {
          const int c = w / ((BK - r0) * 8), o = w % ((BK - r0) * 8);
          *reinterpret_cast<uint4*>(v + c * L::CHUNK_K + r0 * 128 + o * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
      }
      if (warp_live) {
        const uint32_t tS = tmem + lanes + buf * BK;
        uint32_t sr[BK];
        tmem_ld32(tS, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
        tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < BK; i += 8)   // the loads' outputs are valid from here on
          asm volatile("" : "+r"(sr[i]), "+r"(sr[i + 1]), "+r"(sr[i + 2]), "+r"(sr[i + 3]), "+r"(sr[i + 4]),
                       "+r"(sr[i + 5]), "+r"(sr[i + 6]), "+r"(sr[i + 7]));
        // P of the tile with the maximum m, over S; the sum of the weights
        auto weights = [&](float m) {
          const uint64_t sl2x2 = pk2(sl2, sl2), negm2 = pk2(-m, -m);
          uint64_t acc[2] = {pk2(0.f, 0.f), pk2(0.f, 0.f)};
#pragma unroll
          for (int c = 0; c < BK / 32; ++c) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const uint64_t x2 = ffma2(
                  pk2(__uint_as_float(sr[32 * c + 2 * i]), __uint_as_float(sr[32 * c + 2 * i + 1])), sl2x2, negm2);
              float x0, x1;
              upk2(x2, x0, x1);
              x0 = ex2(x0);
              x1 = ex2(x1);
              acc[i & 1] = fadd2(acc[i & 1], pk2(x0, x1));
              pk[i] = pack_bf16x2(x0, x1);
            }
            tmem_st16(tS + 16 * c, pk);
          }
          float a0, a1;
          upk2(fadd2(acc[0], acc[1]), a0, a1);
          return a0 + a1;
        };
        // Steady state: with the running maximum straight away, and the tile's own looked for only
        // if some weight may be above 2^8 (the sum bounds each; a NaN fails the test as well).
        bool done = false;
        if (key0 + BK <= lim_min && __all_sync(0xffffffffu, !live || m_ref != -INFINITY)) {
          const float sum = weights(m_ref == -INFINITY ? 0.f : m_ref);
          done = __all_sync(0xffffffffu, !live || sum <= kRescaleFactor);
          if (done) l_sum += sum;
        }
        if (!done) {
          tmem_wait_st();   // P is stored again below: two stores to one place keep no order of their own
          if (key0 + BK > lim_min) {
#pragma unroll
            for (int i = 0; i < BK; ++i)
              if (key0 + i >= lim) sr[i] = __float_as_uint(-INFINITY);
          }
          float m4[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            m4[c] = fmaxf(__uint_as_float(sr[16 * c]), __uint_as_float(sr[16 * c + 1]));
#pragma unroll
            for (int i = 2; i < 16; i += 2)
              m4[c] = fmax3(m4[c], __uint_as_float(sr[16 * c + i]), __uint_as_float(sr[16 * c + i + 1]));
          }
          const float m_tile = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * sl2;
          const bool resc = live && m_tile > m_ref + kRescaleThreshold;
          float alpha = 1.f;
          if (resc) {
            alpha = ex2(m_ref - m_tile);   // 0 when m_ref is -inf
            m_ref = m_tile;
            l_sum *= alpha;
          }
          if (j > 0 && __any_sync(0xffffffffu, resc)) {
            // O is at rest once PV_{j-1} is done; PV_j waits for this tile's P
            ok = __all_sync(0xffffffffu,
                            mbar_wait(&o_done[last_buf], last_ph, a.err, kErrTimeoutSoftmax, abort_flag));
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(tO + lanes + c * 32, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st32(tO + lanes + c * 32, o);
            }
          }
          l_sum += weights(m_ref == -INFINITY ? 0.f : m_ref);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[buf]);
      last_buf = buf;
      last_ph = ph;
      if (++buf == L::SBUF) { buf = 0; ph ^= 1u; }
    }
    // ---------------------------------------------------------------- epilogue
    if (ok) ok = mbar_wait(&o_done[last_buf], last_ph, a.err, kErrTimeoutEpilogue, abort_flag);
    ok = __all_sync(0xffffffffu, ok);
    tc_fence_after();
    if (ok && warp_live) {
      const bool seen = l_sum != 0.f;   // a NaN row stays one
      const float inv_l = seen ? 1.f / l_sum : 0.f;
      const size_t grow = (size_t)(tok0 + tok) * p.H + g * p.G + row % p.G;
      const size_t prow = (size_t)part * p.B * p.S_Q * p.H + grow;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(tO + lanes + c * 32, o);
        tmem_wait_ld();
        if (!live) continue;
        float4* dst = reinterpret_cast<float4*>(p.o_parts + prow * p.d + c * 32);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (c * 32 + i * 4 < p.d) dst[i] = make_float4(__uint_as_float(o[4 * i]) * inv_l, __uint_as_float(o[4 * i + 1]) * inv_l,
                               __uint_as_float(o[4 * i + 2]) * inv_l, __uint_as_float(o[4 * i + 3]) * inv_l);
      }
      if (live) p.l_parts[prow] = seen ? (m_ref + __log2f(l_sum)) * kLn2 : -INFINITY;
    }
  }

  // ------------------------------------------------------------------ teardown
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    if (!(smem_u32(smem) & 1023u)) mbar_wait(mma_drain, 0, a.err, kErrTimeoutEpilogue, nullptr);
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D>
cudaError_t launch(const PrefixProblem& p, bool pre, bool suf, bool second, const void* q, const void* kp,
                   const void* vp, const void* ks, const void* vs, cudaStream_t s) {
  using L = Layout<D>;
  TcArgs a;
  a.p = p;
  a.err = device_error_word();
  if (!a.err) return cudaErrorInvalidValue;
  a.tokens = BM / p.G;
  const long long all_tokens = (long long)p.B * p.S_Q;
  a.pre_tiles = (int)((all_tokens + a.tokens - 1) / a.tokens);
  a.suf_tiles = (p.S_Q + a.tokens - 1) / a.tokens;
  const long long pre_items = pre ? (long long)p.n_pre * p.H_kv * a.pre_tiles : 0;
  const long long items = pre_items + (suf ? (long long)p.B * p.n_suf * p.H_kv * a.suf_tiles : 0);
  if (items > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  a.pre_items = (int)pre_items;
  a.second = second;

  CUtensorMap mqp, mqs, mkp, mvp, mks, mvs;
  {
    const uint64_t dims[4] = {(uint64_t)p.d, (uint64_t)p.H, (uint64_t)all_tokens, 1};
    const uint64_t row = (uint64_t)p.H * p.d * 2;
    const uint64_t str[3] = {(uint64_t)p.d * 2, row, row * all_tokens};
    const uint32_t box_p[4] = {64, (uint32_t)p.G, (uint32_t)a.tokens, 1};
    const uint32_t box_s[4] = {64, (uint32_t)p.G, (uint32_t)std::min(a.tokens, p.S_Q), 1};
    if ((pre && !encode_tensor_map(&mqp, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, q, dims, str, box_p,
                                   CU_TENSOR_MAP_SWIZZLE_128B)) ||
        (suf && !encode_tensor_map(&mqs, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, q, dims, str, box_s,
                                   CU_TENSOR_MAP_SWIZZLE_128B)))
      return cudaErrorInvalidValue;
  }
  const uint32_t box[4] = {64, 1, BK, 1};
  auto keys = [&](CUtensorMap* m, const void* x, int len, int batch) {
    const uint64_t dims[4] = {(uint64_t)p.d, (uint64_t)p.H_kv, (uint64_t)len, (uint64_t)batch};
    const uint64_t row = (uint64_t)p.H_kv * p.d * 2;
    const uint64_t str[3] = {(uint64_t)p.d * 2, row, row * len};
    return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, x, dims, str, box,
                             CU_TENSOR_MAP_SWIZZLE_128B);
  };
  if (pre && (!keys(&mkp, kp, p.S_P, 1) || !keys(&mvp, vp, p.S_P, 1))) return cudaErrorInvalidValue;
  if (suf && (!keys(&mks, ks, p.S_cap, p.B) || !keys(&mvs, vs, p.S_cap, p.B))) return cudaErrorInvalidValue;
  if (!pre) { mqp = mqs; mkp = mks; mvp = mvs; }   // no CTA reads them
  if (!suf) { mqs = mqp; mks = mkp; mvs = mvp; }
  cudaError_t e = cudaFuncSetAttribute(prefix_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES);
  if (e != cudaSuccess) return e;
  if (second)
    return launch_after(prefix_tc_kernel<D>, (unsigned)items, kThreads, L::BYTES, s, mqp, mqs, mkp, mvp, mks, mvs, a);
  prefix_tc_kernel<D><<<(unsigned)items, kThreads, L::BYTES, s>>>(mqp, mqs, mkp, mvp, mks, mvs, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prefix_tc(const PrefixProblem& p, bool pre, bool suf, bool second, const void* q, const void* kp,
                             const void* vp, const void* ks, const void* vs, cudaStream_t s) {
  return p.d > 64 ? launch<128>(p, pre, suf, second, q, kp, vp, ks, vs, s)
                  : launch<64>(p, pre, suf, second, q, kp, vp, ks, vs, s);
}

}  // namespace lvx
