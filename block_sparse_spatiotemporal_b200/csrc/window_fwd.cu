// Causal attention with a sliding window and sinks, forward, on the
// 5th-generation tensor cores: whole sequences, chunks against a cache, and
// single tokens.  Query i of a sequence stands at position
// p = i + kv_len - q_len and sees the keys of its own unit and the window - 1
// units before it, and the first `sinks` units (see span_of).
//   s = scale q k^T, out = sum_j 2^(s'_j - m) v_j / sum_j 2^(s'_j - m),
//   s' = s log2(e), lse = ln 2 (m + log2 sum_j 2^(s'_j - m)),
// in one pass over the visible keys.  The reference m of a row is the largest
// logit of its first visible key tile; it moves (and O is rescaled) only when
// the probabilities of a later tile sum past 2^64, which fp32 sums and bf16
// probabilities hold without loss, so no step takes a row maximum.
//
// Persistent kernel, one CTA per SM, 384 threads, over items of two 128-row
// query tiles A, B that share one stream of 128-key tiles:
//   warp 0       TMA: the item's Q, then K and V tiles through one ring;
//   warp 1       MMAs: per step j and tile g, O_g += P_g(j-1) V, then
//                S_g(j) = Q_g K^T into the TMEM columns P_g(j-1) held (MMAs
//                of one thread run in issue order), so while one tile's
//                softmax runs the other tile's products keep the tensor
//                cores fed;
//   warps 4-7, 8-11   softmax of tile A, B: thread r owns row r; P is
//                written back over S as bf16 (the A operand of the PV MMA;
//                its rounding, relative 2^-9, is the step's largest error).
// Key tiles that none of a tile's rows sees are skipped for that tile, and
// only tiles that some row sees in part are masked.
//
// Few queries (at most 128 rows a KV head, the query heads of a KV head
// packed into one tile when there are fewer than 128 queries): both softmax
// groups work on the same query tile, on alternate key tiles, and the key
// tiles of an item are split over several CTAs.  Each group writes its
// normalised part and its lse to the workspace, and the last one to arrive
// (a counter per item) joins the parts in ascending order, so the result
// does not depend on which that is.
//
// TMEM (512 columns): S_A, S_B at 0, 128 (P over the first 64 of each), O_A,
// O_B at 256, 384.  Shared memory: Q 2 x 128 rows, ring of 128-key tiles, all
// in 128-byte swizzled parts of 64 dims.
#include "window.cuh"

namespace fvattn {
namespace win {

constexpr int THREADS = 384;
constexpr int SW0 = 4;                       // first softmax warp
constexpr uint32_t PART = 128 * 128;         // 64 dims of 128 rows: 16 KB
constexpr float RESCALE_SUM = 18446744073709551616.f;   // 2^64
constexpr uint32_t TMEM_COLS = 512, TM_S = 0, TM_O = 256;

template <int D> struct Cfg {
  static constexpr int PARTS = D / 64;
  static constexpr uint32_t TILE = PART * PARTS;        // 128 rows
  static constexpr int NST = D == 128 ? 5 : 10;         // ring of K and V tiles
  static constexpr uint32_t SMEM = 1024 + 2 * TILE + NST * TILE;
  static constexpr uint32_t IDESC_S = idesc_bf16_f32(128, 128, false, false);
  static constexpr uint32_t IDESC_PV = idesc_bf16_f32(128, D, false, true);
};

struct FwdCtl {
  uint64_t q_full, q_empty;
  uint64_t kv_full[10], kv_empty[10];
  uint64_t s_full[2];    // S_g of its next step written (and every earlier MMA complete)
  uint64_t p_full[2];    // P_g written (4 warps)
  uint64_t o_full[2];    // the item's last PV of tile g complete
  uint64_t o_empty[2];   // O_g read (4 warps)
  uint64_t group[2];     // softmax group t meets (4 warps), twice per item with parts
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int last[2];           // this group's part was the item's last
};
static_assert(Cfg<128>::SMEM + sizeof(FwdCtl) <= 232448 && Cfg<64>::SMEM + sizeof(FwdCtl) <= 232448, "shared memory");

// Polynomial share of the exponentials: pair i of a 32-column chunk.
#ifndef FVATTN_WIN_POLY
#define FVATTN_WIN_POLY 1000
#endif
__host__ __device__ constexpr bool poly_pair(int i) { return i % FVATTN_WIN_POLY == 1 % FVATTN_WIN_POLY && FVATTN_WIN_POLY < 1000; }

// 2^x of a pair on the FMA pipe: i = floor(x) from a round-down add of
// 1.5 * 2^23, 2^(x - i) by a degree-3 polynomial (a minimax fit in relative
// error on [0, 1), 7.5e-5, below half a bf16 step), i added to the exponent.
__device__ inline void exp2_poly2(uint64_t X, float& y0, float& y1) {
  constexpr float C0 = 0.9999252557754517f, C1 = 0.6958333253860474f, C2 = 0.22606715559959412f,
                  C3 = 0.07802474498748779f, MAGIC = 12582912.f;
  float x0, x1;
  uf2(X, x0, x1);
  x0 = fminf(fmaxf(x0, -126.f), 126.f);
  x1 = fminf(fmaxf(x1, -126.f), 126.f);
  const uint64_t C = f2(x0, x1), M = f2(MAGIC, MAGIC);
  const uint64_t Y = add2_rm(C, M);
  const uint64_t F = sub2(C, sub2(Y, M));
  uint64_t P = fma2(F, f2(C3, C3), f2(C2, C2));
  P = fma2(P, F, f2(C1, C1));
  P = fma2(P, F, f2(C0, C0));
  float p0, p1, q0, q1;
  uf2(P, p0, p1);
  uf2(Y, q0, q1);
  y0 = __uint_as_float(__float_as_uint(p0) + (__float_as_uint(q0) << 23));
  y1 = __uint_as_float(__float_as_uint(p1) + (__float_as_uint(q1) << 23));
}

// P of 32 logits as 16 bf16x2 words, their fp32 sum added to acc.
template <bool MASKED>
__device__ inline void exp_chunk(const uint32_t (&s)[32], uint64_t SL, uint64_t NM, uint32_t mask, uint32_t* pk,
                                 uint64_t (&acc)[2]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float a = __uint_as_float(s[2 * i]), b = __uint_as_float(s[2 * i + 1]);
    if (MASKED) {
      a = (mask >> (2 * i)) & 1u ? a : -INFINITY;
      b = (mask >> (2 * i + 1)) & 1u ? b : -INFINITY;
    }
    const uint64_t X = fma2(f2(a, b), SL, NM);
    float p0, p1;
    if (!MASKED && poly_pair(i)) {
      exp2_poly2(X, p0, p1);
    } else {
      float x0, x1;
      uf2(X, x0, x1);
      p0 = ex2(x0);
      p1 = ex2(x1);
    }
    acc[i & 1] = add2(acc[i & 1], f2(p0, p1));
    pk[i] = cvt_bf16x2(p0, p1);
  }
}

__device__ inline uint32_t chunk_mask(const Span& sp, int key0) {
  return bits(sp.lo - key0, sp.hi - key0) | bits(0, sp.sk - key0);
}

// Row of 128 logits at tS: P (64 words) and the sum of its values.
template <bool MASKED>
__device__ inline float exp_row(uint32_t tS, float sl2, float m, const Span& sp, int key0, uint32_t (&pk)[64]) {
  const uint64_t SL = f2(sl2, sl2), NM = f2(-m, -m);
  uint64_t acc[2] = {0ull, 0ull};
#pragma unroll
  for (int c = 0; c < 4; c += 2) {
    uint32_t s0[32], s1[32];
    tmem_ld32(tS + 32 * c, s0);
    tmem_ld32(tS + 32 * c + 32, s1);
    tmem_wait_ld();
    exp_chunk<MASKED>(s0, SL, NM, MASKED ? chunk_mask(sp, key0 + 32 * c) : 0u, pk + 16 * c, acc);
    exp_chunk<MASKED>(s1, SL, NM, MASKED ? chunk_mask(sp, key0 + 32 * c + 32) : 0u, pk + 16 * c + 16, acc);
  }
  float a, b;
  uf2(add2(acc[0], acc[1]), a, b);
  return a + b;
}

// Largest visible logit of the row (-inf: none).
__device__ inline float row_max(uint32_t tS, const Span& sp, int key0) {
  float m = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t s[32];
    tmem_ld32(tS + 32 * c, s);
    tmem_wait_ld();
    const uint32_t mask = chunk_mask(sp, key0 + 32 * c);
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if ((mask >> i) & 1u) m = fmaxf(m, __uint_as_float(s[i]));
  }
  return m;
}

// Item and its key tiles, the same for every warp.
struct Item {
  int b, hk, g0;         // batch, KV head, first query head of the tile within the KV head's (0 when packed)
  int tile;              // first 128-row query tile
  int split;
  Seq seq;
  int ns, t_lo, n;       // steps 0 .. ns - 1 are tiles 0 .., the others t_lo, t_lo + 1, ..; n steps in all
  int j0, j1;            // this split's steps
  int lo[2], hi[2], sk[2];   // of query tile g: smallest lo, largest hi and sk of its rows
  int dead_lo, dead_sk;  // keys in [dead_sk, dead_lo) are seen by no query of the sequence
  __device__ int key0(int j) const { return 128 * (j < ns ? j : t_lo + j - ns); }
};

__device__ inline Item item_of(const WinFwdArgs& a, int idx) {
  const WinGeom& g = a.g;
  Item it;
  it.split = idx % a.splits;
  idx /= a.splits;
  const int qt = idx % a.item_tiles;
  idx /= a.item_tiles;
  const int per_kv = g.G / a.pack;             // head slots of a KV head
  it.g0 = idx % per_kv;
  idx /= per_kv;
  it.hk = idx % g.Hk;
  it.b = idx / g.Hk;
  it.tile = (a.item_tiles - 1 - qt) * (a.dual ? 2 : 1);   // the longest spans first
  it.seq = seq_of(g, it.b);
  int lo = 0x7fffffff, hi = 0, sk = 0;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    it.lo[t] = it.hi[t] = it.sk[t] = 0;
    const int i0 = (it.tile + (a.dual ? t : 0)) * a.tokens;
    if (i0 >= it.seq.ql) continue;
    const int i1 = i0 + a.tokens < it.seq.ql ? i0 + a.tokens : it.seq.ql;
    const Span last = span_of(g, it.seq, i1 - 1);
    if (last.hi == 0) continue;
    const int first_pos = it.seq.ql - it.seq.kvl;          // first query that is not in front of the keys
    it.lo[t] = span_of(g, it.seq, i0 > first_pos ? i0 : first_pos).lo;
    it.hi[t] = last.hi;
    it.sk[t] = last.sk;
    lo = it.lo[t] < lo ? it.lo[t] : lo;
    hi = it.hi[t] > hi ? it.hi[t] : hi;
    sk = it.sk[t] > sk ? it.sk[t] : sk;
  }
  if (hi == 0) {
    it.ns = it.t_lo = it.n = 0;
  } else {
    const int t_hi = (hi + 127) >> 7, ns = (sk + 127) >> 7;
    it.t_lo = lo >> 7;
    it.ns = ns < it.t_lo ? ns : 0;
    if (ns >= it.t_lo) it.t_lo = sk > 0 ? 0 : it.t_lo;
    it.n = it.ns + t_hi - it.t_lo;
  }
  it.j0 = (int)((long long)it.n * it.split / a.splits);
  it.j1 = (int)((long long)it.n * (it.split + 1) / a.splits);
  const int first = it.seq.ql > it.seq.kvl ? it.seq.ql - it.seq.kvl : 0;
  const Span f = span_of(g, it.seq, first);
  it.dead_lo = f.lo;
  const long long all_sk = (long long)g.sinks * g.unit;
  it.dead_sk = all_sk < f.lo ? (int)all_sk : f.lo;
  return it;
}

// Does softmax group / accumulator t work on step j?
__device__ inline bool active(const WinFwdArgs& a, const Item& it, int t, int j) {
  const int k0 = it.key0(j);
  if (!a.dual && ((j - it.j0) & 1) != t) return false;
  return k0 < it.hi[t] && (k0 + 128 > it.lo[t] || k0 < it.sk[t]);
}

template <int D>
__global__ void __launch_bounds__(THREADS, 1)
    window_fwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                      const __grid_constant__ CUtensorMap mv, const WinFwdArgs a) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sKV = smem + 2 * C::TILE;
  __shared__ FwdCtl ctl_s;
  FwdCtl* ctl = &ctl_s;
  volatile int* abort_flag = &ctl->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WinGeom& g = a.g;
  const long long cap = a.wait_cap;

  if (threadIdx.x == 0) {
    mbar_init(&ctl->q_full, 1);
    mbar_init(&ctl->q_empty, 1);
    for (int i = 0; i < C::NST; ++i) {
      mbar_init(&ctl->kv_full[i], 1);
      mbar_init(&ctl->kv_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->s_full[i], 1);
      mbar_init(&ctl->p_full[i], 4);
      mbar_init(&ctl->o_full[i], 1);
      mbar_init(&ctl->o_empty[i], 4);
      mbar_init(&ctl->group[i], 4);
    }
    mbar_init(&ctl->drain, 1);
    ctl->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&ctl->tmem_base, TMEM_COLS);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = ctl->tmem_base;

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA
    if (lane == 0) {
      prefetch_tensormap(&mq);
      prefetch_tensormap(&mk);
      prefetch_tensormap(&mv);
      long long seq = 0;
      int k = 0, q_issued = 0;
      bool ok = true;
      for (int idx = blockIdx.x; idx < a.n_items && ok; idx += gridDim.x) {
        const Item it = item_of(a, idx);
        if (it.j0 >= it.j1) continue;
        if (k >= 1 && !mbar_wait(&ctl->q_empty, (uint32_t)(k - 1) & 1, abort_flag, a.status, cap)) break;
        ++k;
        const int tiles = a.dual ? 2 : 1;
        mbar_arrive_expect_tx(&ctl->q_full, (uint32_t)(tiles * C::PARTS * a.pack * a.tokens) * 128u);
        for (int t = 0; t < tiles; ++t)
          for (int h = 0; h < C::PARTS; ++h)
            tma_load_5d(sQ + t * C::TILE + h * PART, &mq, &ctl->q_full, 64 * h, it.g0, (it.tile + t) * a.tokens, it.hk,
                        it.b);
        ++q_issued;
        for (int j = it.j0; j < it.j1 && ok; ++j) {
          const int key0 = it.key0(j);
          for (int kv = 0; kv < 2; ++kv, ++seq) {
            const int st = (int)(seq % C::NST);
            if (seq >= C::NST &&
                !mbar_wait(&ctl->kv_empty[st], (uint32_t)(seq / C::NST - 1) & 1, abort_flag, a.status, cap)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&ctl->kv_full[st], C::TILE);
            for (int h = 0; h < C::PARTS; ++h)
              tma_load_4d(sKV + st * C::TILE + h * PART, kv ? &mv : &mk, &ctl->kv_full[st], 64 * h, key0, it.hk, it.b);
          }
        }
      }
      // every copy issued has landed before the block exits
      if (q_issued >= 1) mbar_drain(&ctl->q_full, (uint32_t)(q_issued - 1) & 1, a.status, cap);
      for (int i = 0; i < C::NST && i < seq; ++i) {
        const long long last = i + ((seq - 1 - i) / C::NST) * C::NST;
        mbar_drain(&ctl->kv_full[i], (uint32_t)(last / C::NST) & 1, a.status, cap);
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA
    long long seq = 0;               // ring number of the K tile of the item's first step
    int k = 0;
    long long cnt[2] = {0, 0};       // steps done of each tile
    int items[2] = {0, 0};           // items whose O_g was written
    bool ok = true;
    const uint32_t q_base = smem_u32(sQ), kv_base = smem_u32(sKV);
    for (int idx = blockIdx.x; idx < a.n_items && ok; idx += gridDim.x) {
      const Item it = item_of(a, idx);
      if (it.j0 >= it.j1) continue;
      if (!mbar_wait_warp(&ctl->q_full, (uint32_t)k & 1, abort_flag, a.status, cap)) break;
      ++k;
      bool first[2] = {true, true};
      for (int j = it.j0; j <= it.j1 && ok; ++j) {
        const long long sk = seq + 2ll * (j - it.j0), sv = sk - 1;     // K of step j, V of step j - 1
        const int stk = (int)(sk % C::NST), stv = (int)(sv % C::NST);
        if (j < it.j1 && !mbar_wait_warp(&ctl->kv_full[stk], (uint32_t)(sk / C::NST) & 1, abort_flag, a.status, cap)) {
          ok = false;
          break;
        }
        if (j > it.j0) {
          if (!mbar_wait_warp(&ctl->kv_full[stv], (uint32_t)(sv / C::NST) & 1, abort_flag, a.status, cap)) {
            ok = false;
            break;
          }
          // values that no query of the sequence sees may be anything: their
          // probabilities are 0, and 0 times NaN is not
          const int key0 = it.key0(j - 1);
          if (key0 + 128 > it.seq.kvl && it.seq.kvl < g.Nk)
            zero_rows(sKV + stv * C::TILE, PART, C::PARTS, it.seq.kvl - key0, 128);
          if (key0 < it.dead_lo && key0 + 128 > it.dead_sk)
            zero_rows(sKV + stv * C::TILE, PART, C::PARTS, it.dead_sk > key0 ? it.dead_sk - key0 : 0,
                      it.dead_lo - key0 < 128 ? it.dead_lo - key0 : 128);
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (j > it.j0 && active(a, it, t, j - 1)) {
            if (first[t] && items[t] >= 1 &&
                !mbar_wait_warp(&ctl->o_empty[t], (uint32_t)(items[t] - 1) & 1, abort_flag, a.status, cap)) {
              ok = false;
              break;
            }
            if (!mbar_wait_warp(&ctl->p_full[t], (uint32_t)(cnt[t] - 1) & 1, abort_flag, a.status, cap)) {
              ok = false;
              break;
            }
            tc_fence_after();
            if (elect_one()) {
              const uint64_t vd = umma_desc_sw128(kv_base + stv * C::TILE, PART, 1024);
              const uint32_t tO = tbase + TM_O + 128 * t, tP = tbase + TM_S + 128 * t;
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                mma_ts(tO, tP + 8 * kk, vd + ((kk * 2048) >> 4), C::IDESC_PV, first[t] && kk == 0 ? 0u : 1u);
            }
            __syncwarp();
            first[t] = false;
          }
          if (j < it.j1 && active(a, it, t, j)) {
            if (elect_one()) {
              const uint64_t qd = umma_desc_sw128(q_base + (a.dual ? t : 0) * C::TILE, 16, 1024);
              const uint64_t kd = umma_desc_sw128(kv_base + stk * C::TILE, 16, 1024);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = ((kk >> 2) * PART + (kk & 3) * 32) >> 4;
                mma_ss(tbase + TM_S + 128 * t, qd + off, kd + off, C::IDESC_S, kk ? 1u : 0u);
              }
              mma_commit(&ctl->s_full[t]);
            }
            __syncwarp();
            ++cnt[t];
          }
        }
        if (!ok) break;
        if (elect_one()) {
          if (j > it.j0) mma_commit(&ctl->kv_empty[stv]);
          if (j < it.j1) mma_commit(&ctl->kv_empty[stk]);
          if (j == it.j1 - 1) mma_commit(&ctl->q_empty);
          if (j == it.j1) {
            if (!first[0]) mma_commit(&ctl->o_full[0]);
            if (!first[1]) mma_commit(&ctl->o_full[1]);
          }
        }
        __syncwarp();
      }
      if (!first[0]) ++items[0];
      if (!first[1]) ++items[1];
      seq += 2ll * (it.j1 - it.j0);
    }
    // every MMA issued has completed before TMEM is freed
    if (elect_one()) {
      mma_commit(&ctl->drain);
      mbar_drain(&ctl->drain, 0, a.status, cap);
    }
    __syncwarp();
  } else if (warp >= SW0) {
    // ------------------------------------------------------------ softmax
    const int t = (warp - SW0) >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tbase + TM_S + 128 * t + lane_off, tO = tbase + TM_O + 128 * t + lane_off;
    const float sl2 = g.scale * 1.4426950408889634f;
    const int prow = a.tokens * a.pack;          // rows of a part
    long long cnt = 0;
    int items = 0;
    bool ok = true;
    for (int idx = blockIdx.x; idx < a.n_items && ok; idx += gridDim.x) {
      const Item it = item_of(a, idx);
      const int i = (it.tile + (a.dual ? t : 0)) * a.tokens + r / a.pack;     // query
      const int head = it.hk * g.G + it.g0 + r % a.pack;
      const bool valid = r < a.tokens * a.pack && i < it.seq.ql;
      // rows that are not stored count as seeing everything: no mask for them
      const Span sp = valid ? span_of(g, it.seq, i) : Span{0, 0x7fffffff, 0};
      const bool warp_on = __any_sync(0xffffffffu, valid);
      float m = -INFINITY, l = 0.f;
      bool any = false;
      for (int j = it.j0; j < it.j1; ++j) {
        if (!active(a, it, t, j)) continue;
        if (!mbar_wait(&ctl->s_full[t], (uint32_t)cnt & 1, abort_flag, a.status, cap)) {
          ok = false;
          break;
        }
        tc_fence_after();
        any = true;
        ++cnt;
        if (warp_on) {
          const int key0 = it.key0(j);
          const bool full = !valid || (key0 + 128 <= sp.hi && (key0 >= sp.lo || key0 + 128 <= sp.sk));
          const bool masked = __any_sync(0xffffffffu, !full);
          if (__any_sync(0xffffffffu, m == -INFINITY)) {
            const float mx = row_max(tS, sp, key0) * sl2;
            if (m == -INFINITY) m = mx;
          }
          uint32_t pk[64];
          const float m_use = m == -INFINITY ? 0.f : m;
          float sum = masked ? exp_row<true>(tS, sl2, m_use, sp, key0, pk) : exp_row<false>(tS, sl2, m_use, sp, key0, pk);
          const bool over = valid && !(sum <= RESCALE_SUM);
          if (__any_sync(0xffffffffu, over)) {
            // too large (or not a number): move the reference up; every MMA
            // before this S is complete, so O holds the earlier steps
            const float mx = fmaxf(row_max(tS, sp, key0) * sl2, m_use);
            const float m_new = over ? mx : m_use;
            const float alpha = ex2(m_use - m_new);
            if (over) m = m_new;
            sum = exp_row<true>(tS, sl2, m_new, sp, key0, pk);
            if (__any_sync(0xffffffffu, over && l > 0.f)) {
#pragma unroll 1
              for (int ch = 0; ch < D / 32; ++ch) {
                uint32_t o[32];
                tmem_ld32(tO + ch * 32, o);
                tmem_wait_ld();
#pragma unroll
                for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * alpha);
                tmem_st32(tO + ch * 32, o);
              }
            }
            l *= alpha;
          }
          l += sum;
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_st16(tS + 16 * c, pk + 16 * c);
          tmem_wait_st();
        }
        tc_fence_before();
        mbar_arrive_warp(&ctl->p_full[t]);
      }
      if (!ok) break;
      // ---- epilogue
      if (any) {
        if (!mbar_wait(&ctl->o_full[t], (uint32_t)items & 1, abort_flag, a.status, cap)) break;
        tc_fence_after();
        ++items;
      }
      const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
      const float lse2 = l > 0.f || l != l ? m + __log2f(l) : -INFINITY;
      const bool parts = a.parts > 1;
      const long long slot = parts ? ((long long)idx * 2 + t) * prow + r : 0;
      __nv_bfloat16* orow = static_cast<__nv_bfloat16*>(a.out) + (long long)it.b * a.o_batch +
                            (long long)head * a.o_head + (long long)i * a.o_token;
      if (warp_on) {
#pragma unroll 1
        for (int ch = 0; ch < D / 32; ++ch) {
          uint32_t o[32];
          if (any) {
            tmem_ld32(tO + ch * 32, o);
            tmem_wait_ld();
          }
          if (!any || inv == 0.f) {
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] = 0u;
          }
          if (valid) {
            if (parts) {
              float4* dst = reinterpret_cast<float4*>(a.part_o + slot * D + ch * 32);
#pragma unroll
              for (int x = 0; x < 8; ++x)
                dst[x] = make_float4(__uint_as_float(o[4 * x]) * inv, __uint_as_float(o[4 * x + 1]) * inv,
                                     __uint_as_float(o[4 * x + 2]) * inv, __uint_as_float(o[4 * x + 3]) * inv);
            } else {
              uint32_t w[16];
#pragma unroll
              for (int x = 0; x < 16; ++x)
                w[x] = cvt_bf16x2(__uint_as_float(o[2 * x]) * inv, __uint_as_float(o[2 * x + 1]) * inv);
              uint4* dst = reinterpret_cast<uint4*>(orow + ch * 32);
#pragma unroll
              for (int x = 0; x < 4; ++x) dst[x] = make_uint4(w[4 * x], w[4 * x + 1], w[4 * x + 2], w[4 * x + 3]);
            }
          }
        }
        if (valid) {
          if (parts)
            a.part_lse[slot] = lse2;
          else
            a.lse[((long long)it.b * g.H + head) * g.Nq + i] = lse2 * 0.6931471805599453f;
        }
      }
      if (any) {
        tc_fence_before();
        mbar_arrive_warp(&ctl->o_empty[t]);
      }
      if (parts) {
        // the group that completes the query tile's parts joins them
        __threadfence();
        mbar_arrive_warp(&ctl->group[t]);
        if (!mbar_wait(&ctl->group[t], 0u, abort_flag, a.status, cap)) break;
        const int base = idx - it.split;               // split 0 of this item
        if (r == 0)
          ctl->last[t] = atomicAdd(a.counters + (a.dual ? base / a.splits * 2 + t : base / a.splits), 1) == a.parts - 1;
        mbar_arrive_warp(&ctl->group[t]);
        if (!mbar_wait(&ctl->group[t], 1u, abort_flag, a.status, cap)) break;
        if (ctl->last[t]) {
          __threadfence();
          const int rows_tok = it.seq.ql - (it.tile + (a.dual ? t : 0)) * a.tokens;
          const int rows = (rows_tok < a.tokens ? rows_tok : a.tokens) * a.pack;
          constexpr int TPR = D / 4;                   // threads per row, four dims each
          const int sub = r / TPR, d0 = (r % TPR) * 4;
          for (int row = sub; row < rows; row += 128 / TPR) {
            float M = -INFINITY;
            for (int p = 0; p < a.parts; ++p) {
              const long long sl = a.dual ? ((long long)(base + p) * 2 + t) * 128 + row
                                          : ((long long)(base + (p >> 1)) * 2 + (p & 1)) * prow + row;
              M = fmaxf(M, __ldcg(a.part_lse + sl));
            }
            const float M_use = M == -INFINITY ? 0.f : M;
            float L = 0.f;
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
            for (int p = 0; p < a.parts; ++p) {
              const long long sl = a.dual ? ((long long)(base + p) * 2 + t) * 128 + row
                                          : ((long long)(base + (p >> 1)) * 2 + (p & 1)) * prow + row;
              const float w = ex2(__ldcg(a.part_lse + sl) - M_use);
              const float4 v = __ldcg(reinterpret_cast<const float4*>(a.part_o + sl * D + d0));
              L += w;
              acc[0] = fmaf(w, v.x, acc[0]);
              acc[1] = fmaf(w, v.y, acc[1]);
              acc[2] = fmaf(w, v.z, acc[2]);
              acc[3] = fmaf(w, v.w, acc[3]);
            }
            const float li = L > 0.f || L != L ? 1.f / L : 0.f;
            const int qi = (it.tile + (a.dual ? t : 0)) * a.tokens + row / a.pack;
            const int hd = it.hk * g.G + it.g0 + row % a.pack;
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + (long long)it.b * a.o_batch +
                                 (long long)hd * a.o_head + (long long)qi * a.o_token + d0;
            *reinterpret_cast<uint2*>(dst) =
                make_uint2(cvt_bf16x2(acc[0] * li, acc[1] * li), cvt_bf16x2(acc[2] * li, acc[3] * li));
            if (r % TPR == 0)
              a.lse[((long long)it.b * g.H + hd) * g.Nq + qi] =
                  li == 0.f ? -INFINITY : (M_use + __log2f(L)) * 0.6931471805599453f;
          }
        }
      }
    }
  }

  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, TMEM_COLS);
  }
}

template <int D>
cudaError_t launch_fwd(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const WinFwdArgs& a,
                       int num_sms, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(window_fwd_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)Cfg<D>::SMEM);
  if (e != cudaSuccess) return e;
  const int grid = a.n_items < num_sms ? a.n_items : num_sms;
  window_fwd_kernel<D><<<grid, THREADS, Cfg<D>::SMEM, s>>>(mq, mk, mv, a);
  return cudaGetLastError();
}

}  // namespace win

cudaError_t launch_window_fwd(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const WinFwdArgs& a,
                              int num_sms, cudaStream_t s) {
  return a.g.D == 128 ? win::launch_fwd<128>(mq, mk, mv, a, num_sms, s) : win::launch_fwd<64>(mq, mk, mv, a, num_sms, s);
}

}  // namespace fvattn
