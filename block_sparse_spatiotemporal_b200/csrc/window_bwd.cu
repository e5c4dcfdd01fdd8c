// Backward of the sliding-window attention (see window_fwd.cu for who sees
// whom).  With s = scale q k^T, p = exp(s - lse) over the visible pairs:
//   dv = p^T dout,  dp = dout v^T,  ds = p (dp - rowsum(dout * out)),
//   dq = scale ds k,  dk = scale ds^T q,
// dk and dv summed over the query heads that share a KV head.
//
// Two persistent tcgen05 kernels share one template, so no gradient needs
// atomics and every run gives the same bits:
//   * key-stationary (KV = true): a work item is 128 keys of a KV head (128
//     TMEM lanes); it walks the queries that see any of them, head after
//     head, 64 a step, and accumulates dV += P^T dO and dK += dS^T Q in TMEM;
//   * query-stationary (KV = false): a work item is 128 queries of a head; it
//     walks the keys they see, 64 a step, and accumulates dQ += dS K.
// S and dP are computed in both: 7 products of the matrix units where one
// kernel with atomic sums would do 5; what that buys is the fixed order.
// Warp 0 takes the CTA's next item from a counter, decodes it once and
// publishes it in a ring (every warp decoding its own, items dealt out in
// turn: 1,311 against 1,161 us at 12 heads, 16,384 tokens in frames of 1,024,
// window 3 + 1, one call at a time behind a flush of L2), and loads the tiles
// by TMA.
// Per step two warps issue S = X0 Y0^T and dP = X1 Y1^T (X stationary: K, V
// or Q, dO; Y moving) into one of NB TMEM buffers, eight warps (two per TMEM
// lane quarter, half the columns each) turn them into P and dS and write both
// back into the same columns as bf16 (off by up to 2^-8 of it: the operands
// of the next products), and a fourth warp's accumulating MMAs read them from
// TMEM as the A operand.  The moving tiles are used twice: K-major for the
// scores, MN-major for the accumulations.
// Where one tile's steps would outlast the others' (the tile of the sinks,
// which every query sees; few KV heads under many query heads) they are split:
// each part writes fp32 sums to the workspace, and the last one to arrive adds
// them in ascending order (2 x 14 heads over 2 KV heads, 1,531 tokens, window
// 300: 197 us unsplit).
#include <utility>

#include "window.cuh"

namespace fvattn {
namespace wb {

using namespace win;

constexpr int THREADS = 384;          // warp 0 TMA, warps 1-3 MMA, warps 4..11 compute + epilogue
constexpr int CW0 = 4;
constexpr int CTHREADS = 256;
constexpr uint32_t SPART = 128 * 128; // 64 dims of the 128 stationary rows: 16 KB
constexpr uint32_t MPART = 64 * 128;  // 64 dims of the 64 moving rows: 8 KB
constexpr uint32_t TMEM_COLS = 512;

template <int D> struct Sh {
  static constexpr int PARTS = D / 64;
  static constexpr int MST = D == 128 ? 4 : 8;      // moving stages
  static constexpr uint32_t STENSOR = SPART * PARTS, MTENSOR = MPART * PARTS;
  static constexpr uint32_t STAT_BYTES = 2 * STENSOR, MOV_BYTES = 2 * MTENSOR;
  static constexpr uint32_t SMEM = 1024 + STAT_BYTES + MST * MOV_BYTES;
  static constexpr uint32_t IDESC_S = idesc_bf16_f32(128, 64, false, false);
  static constexpr uint32_t IDESC_ACC = idesc_bf16_f32(128, D, false, true);
};
constexpr int MAXST = 8;
// NB score buffers: S buffer b at columns 64 b, dP buffer b at 64 (NB + b),
// then the accumulators.
template <bool KV> struct Tm {
  static constexpr int NB = KV ? 2 : 3;
  static constexpr uint32_t S = 0, DP = 64 * NB, ACC0 = 128 * NB, ACC1 = ACC0 + 128;
  static_assert(ACC0 + (KV ? 256 : 128) <= TMEM_COLS, "TMEM columns");
};
constexpr int MAXNB = 3;

constexpr int ITEMS = 2;      // items published ahead

// A work item and its steps.
template <bool KV> struct Item {
  int idx;               // -1: the CTA has no further item
  int b, hk, h;          // h: query head (query-stationary)
  int row0;              // first stationary row (key or query)
  Seq seq;
  int lo, n_per, n;      // KV: first query tile, tiles per head, steps (n_per * G)
  int j0, j1;            // this part's steps
  int part, parts, cell; // KV: part of the tile's steps; number of its (batch, KV head, tile)
  int ns, t_lo;          // else: as in the forward, key tiles of 64
  int dead_lo, dead_sk;
  // first moving row of step j, and (KV) its query head
  __device__ int moving(int j) const { return KV ? 64 * (lo + j % n_per) : 64 * (j < ns ? j : t_lo + j - ns); }
  __device__ int head(const WinGeom& g, int j) const { return KV ? hk * g.G + j / n_per : h; }
};

template <bool KV> __device__ inline Item<KV> item_of(const WinBwdArgs& a, int idx) {
  const WinGeom& g = a.g;
  Item<KV> it{};
  it.idx = idx;
  if (KV) {
    // the tiles with sinks first: every later query sees them
    const int heavy = a.heavy_tiles * g.B * g.Hk * a.heavy_parts;
    int tile, bh;
    if (idx < heavy) {
      it.parts = a.heavy_parts;
      it.part = idx % it.parts;
      idx /= it.parts;
      tile = idx % a.heavy_tiles;
      bh = idx / a.heavy_tiles;
    } else {
      idx -= heavy;
      it.parts = a.parts;
      it.part = idx % it.parts;
      idx /= it.parts;
      const int rest = a.tiles - a.heavy_tiles;
      tile = a.heavy_tiles + idx % rest;
      bh = idx / rest;
    }
    it.cell = bh * a.tiles + tile;
    it.b = bh / g.Hk;
    it.hk = bh % g.Hk;
    it.row0 = 128 * tile;
    it.seq = seq_of(g, it.b);
    const int j1 = it.row0 + 128 < it.seq.kvl ? it.row0 + 128 : it.seq.kvl;
    it.n_per = it.n = 0;
    if (it.row0 < j1) {
      const int off = it.seq.kvl - it.seq.ql;              // position of query 0
      int lo = it.row0 / g.unit * g.unit - off;
      lo = lo < 0 ? 0 : lo;
      long long hi = it.seq.ql;
      if (g.window > 0 && it.row0 / g.unit >= g.sinks) {
        const long long end = ((long long)(j1 - 1) / g.unit + g.window) * g.unit - off;
        hi = end < hi ? end : hi;
      }
      if (lo < hi) {
        it.lo = lo >> 6;
        it.n_per = (int)((hi + 63) >> 6) - it.lo;
        it.n = it.n_per * g.G;
      }
    }
    it.j0 = (int)((long long)it.n * it.part / it.parts);
    it.j1 = (int)((long long)it.n * (it.part + 1) / it.parts);
  } else {
    const int tile = a.tiles - 1 - idx % a.tiles;
    idx /= a.tiles;
    it.h = idx % g.H;
    it.b = idx / g.H;
    it.hk = it.h / g.G;
    it.row0 = 128 * tile;
    it.seq = seq_of(g, it.b);
    const int i1 = it.row0 + 128 < it.seq.ql ? it.row0 + 128 : it.seq.ql;
    if (it.row0 < i1) {
      const Span last = span_of(g, it.seq, i1 - 1);
      if (last.hi > 0) {
        const int first_pos = it.seq.ql - it.seq.kvl;
        const int lo = span_of(g, it.seq, it.row0 > first_pos ? it.row0 : first_pos).lo;
        const int t_hi = (last.hi + 63) >> 6, ns = (last.sk + 63) >> 6;
        it.t_lo = lo >> 6;
        it.ns = ns < it.t_lo ? ns : 0;
        if (ns >= it.t_lo) it.t_lo = last.sk > 0 ? 0 : it.t_lo;
        it.n = it.ns + t_hi - it.t_lo;
      }
    }
    const int first = it.seq.ql > it.seq.kvl ? it.seq.ql - it.seq.kvl : 0;
    const Span f = span_of(g, it.seq, first);
    it.dead_lo = f.lo;
    const long long all_sk = (long long)g.sinks * g.unit;
    it.dead_sk = all_sk < f.lo ? (int)all_sk : f.lo;
    it.parts = 1;
    it.j1 = it.n;
  }
  return it;
}

template <bool KV> struct Ctl {
  uint64_t item_full[ITEMS], item_empty[ITEMS];   // 3 MMA and 8 compute warps read an item
  uint64_t stat_full, stat_empty;
  uint64_t mov_full[MAXST], mov_empty[MAXST];
  uint64_t s_full[MAXNB];    // S and dP of step c in buffer c % NB (two commits)
  uint64_t p_full[MAXNB];    // P / dS of step c written back (8 warps)
  uint64_t step_done[MAXNB]; // the accumulating MMAs of step c, which read buffer c % NB, complete
  uint64_t acc_full;         // the item's accumulators complete
  uint64_t acc_empty;        // the epilogue read them (8 warps)
  uint64_t meet;             // the compute warps meet (8 warps)
  uint64_t drain;
  alignas(16) float lse2[MAXST][64];     // key-stationary only: lse * log2(e) of the step's queries
  alignas(16) float dd[MAXST][64];       //   and their rowsum(dout * out)
  Item<KV> item[ITEMS];
  uint32_t tmem_base;
  int abort;
  int last;                  // this part was its tile's last
};
static_assert(Sh<128>::SMEM + sizeof(Ctl<true>) <= 232448 && Sh<64>::SMEM + sizeof(Ctl<true>) <= 232448, "shared memory");

// A kernel launched with launch_after may start while the one in front of it
// in the stream still runs, once every block of that one called
// start_following() or ended; wait_preceding() returns when that one is
// complete and its writes are visible.
__device__ inline void start_following() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ inline void wait_preceding() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_after(bool early, void (*kernel)(P...), int grid, int threads, uint32_t smem, cudaStream_t s,
                         A&&... args) {
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(grid);
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  c.attrs = &at;
  c.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&c, kernel, std::forward<A>(args)...);
}

// K-major operand of 64-dim parts `part` bytes apart, K step kk.
__device__ inline uint64_t kdesc(uint32_t base, uint32_t part, int kk) {
  return umma_desc_sw128(base + (kk >> 2) * part + (kk & 3) * 32, 16, 1024);
}

template <int D, bool KV>
__global__ void __launch_bounds__(THREADS, 1)
    window_bwd_kernel(const __grid_constant__ CUtensorMap ms0, const __grid_constant__ CUtensorMap ms1,
                      const __grid_constant__ CUtensorMap mm0, const __grid_constant__ CUtensorMap mm1,
                      const WinBwdArgs a) {
  using C = Sh<D>;
  constexpr int NB = Tm<KV>::NB, MST = C::MST;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sStat = smem;                         // X0 then X1
  uint8_t* sMov = smem + C::STAT_BYTES;          // per stage: Y0 then Y1
  __shared__ Ctl<KV> ctl_s;
  Ctl<KV>* ctl = &ctl_s;
  volatile int* abort_flag = &ctl->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WinGeom& g = a.g;
  const long long cap = a.wait_cap;

  if (threadIdx.x == 0) {
    for (int i = 0; i < ITEMS; ++i) {
      mbar_init(&ctl->item_full[i], 1);
      mbar_init(&ctl->item_empty[i], 3 + CTHREADS / 32);
    }
    mbar_init(&ctl->stat_full, 1);
    mbar_init(&ctl->stat_empty, 2);              // one commit per score warp
    for (int i = 0; i < MST; ++i) {
      mbar_init(&ctl->mov_full[i], KV ? 32 : 1);
      mbar_init(&ctl->mov_empty[i], 1);
    }
    for (int i = 0; i < MAXNB; ++i) {
      mbar_init(&ctl->s_full[i], 2);
      mbar_init(&ctl->p_full[i], CTHREADS / 32);
      mbar_init(&ctl->step_done[i], 1);
    }
    mbar_init(&ctl->acc_full, 1);
    mbar_init(&ctl->acc_empty, CTHREADS / 32);
    mbar_init(&ctl->meet, CTHREADS / 32);
    mbar_init(&ctl->drain, 3);                   // final commit of each MMA warp
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
  // The query-stationary kernel needs nothing of the key-stationary one in
  // front of it and starts on the SMs that one leaves (2 x 14 heads over 2,
  // 1,531 tokens: 80 -> 63 us; 12 heads, 16,384 tokens: 1,157 -> 1,140 us, one
  // call at a time behind a flush of L2);
  // what prep wrote is complete then, since every block of that one has waited
  // for it, and is read past L1.  It ends after that one, so that whatever
  // follows in the stream does too.
  if (KV) {
    wait_preceding();
    start_following();
  }

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA
    const bool leader = lane == 0;
    if (leader) {
      prefetch_tensormap(&ms0);
      prefetch_tensormap(&ms1);
      prefetch_tensormap(&mm0);
      prefetch_tensormap(&mm1);
    }
    long long gs = 0;       // moving steps loaded
    int k = 0;
    bool ok = true;
    int idx = blockIdx.x;   // then the next one from a counter
    for (int n = 0; ok; ++n) {
      const int ib = n % ITEMS;
      if (n >= ITEMS &&
          !mbar_wait_warp(&ctl->item_empty[ib], (uint32_t)(n / ITEMS - 1) & 1, abort_flag, a.status, cap))
        break;
      if (leader) {
        if (idx < a.n_items) {
          ctl->item[ib] = item_of<KV>(a, idx);
          idx = gridDim.x + atomicAdd(a.next_item, 1);
        } else {
          ctl->item[ib].idx = -1;
        }
        mbar_arrive(&ctl->item_full[ib]);
      }
      __syncwarp();
      const Item<KV> it = ctl->item[ib];     // overwritten only when this warp comes round again
      if (it.idx < 0) break;
      if (it.j0 == it.j1) continue;
      if (leader) {
        if (k >= 1) ok = mbar_wait(&ctl->stat_empty, (uint32_t)(k - 1) & 1, abort_flag, a.status, cap);
        if (ok) {
          const int hs = KV ? it.hk : it.h;
          mbar_arrive_expect_tx(&ctl->stat_full, C::STAT_BYTES);
          for (int p = 0; p < C::PARTS; ++p) {
            tma_load_4d(sStat + p * SPART, &ms0, &ctl->stat_full, 64 * p, it.row0, hs, it.b);
            tma_load_4d(sStat + C::STENSOR + p * SPART, &ms1, &ctl->stat_full, 64 * p, it.row0, hs, it.b);
          }
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      ++k;
      for (int j = it.j0; j < it.j1 && ok; ++j, ++gs) {
        const int st = (int)(gs % MST);
        const int m0 = it.moving(j), hm = KV ? it.head(g, j) : it.hk;
        if (leader && gs >= MST)
          ok = mbar_wait(&ctl->mov_empty[st], (uint32_t)((gs / MST) - 1) & 1, abort_flag, a.status, cap);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        if (KV) {
          const long long row = ((long long)it.b * g.H + hm) * g.Nq + m0;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int i = lane + 32 * u;
            const bool in = m0 + i < it.seq.ql;
            ctl->lse2[st][i] = in ? a.lse2[row + i] : 0.f;
            ctl->dd[st][i] = in ? a.dd[row + i] : 0.f;
          }
        }
        if (leader) {
          mbar_arrive_expect_tx(&ctl->mov_full[st], C::MOV_BYTES);
          uint8_t* dst = sMov + st * C::MOV_BYTES;
          for (int p = 0; p < C::PARTS; ++p) {
            tma_load_4d(dst + p * MPART, &mm0, &ctl->mov_full[st], 64 * p, m0, hm, it.b);
            tma_load_4d(dst + C::MTENSOR + p * MPART, &mm1, &ctl->mov_full[st], 64 * p, m0, hm, it.b);
          }
        } else if (KV) {
          mbar_arrive(&ctl->mov_full[st]);
        }
      }
    }
    // every copy issued has landed before the block exits
    if (leader) {
      if (k >= 1) mbar_drain(&ctl->stat_full, (uint32_t)(k - 1) & 1, a.status, cap);
      for (int i = 0; i < MST && i < gs; ++i) {
        const long long last = i + ((gs - 1 - i) / MST) * MST;
        mbar_drain(&ctl->mov_full[i], (uint32_t)(last / MST) & 1, a.status, cap);
      }
    }
  } else if (warp == 1 || warp == 2) {
    // ------------------------------------------------------- MMA: scores
    // Warp 1 issues S = X0 Y0^T, warp 2 dP = X1 Y1^T.  Step c goes to buffer
    // c % NB once the accumulations of step c - NB, which read it, are
    // complete; the stationary tiles are released after the item's last score.
    const bool is_s = warp == 1;
    long long c = 0;
    int k = 0;
    bool ok = true;
    const uint32_t x = smem_u32(sStat) + (is_s ? 0u : C::STENSOR);
    const uint32_t tdst = tbase + (is_s ? Tm<KV>::S : Tm<KV>::DP);
    for (int m = 0; ok; ++m) {
      const int ib = m % ITEMS;
      if (!mbar_wait_warp(&ctl->item_full[ib], (uint32_t)(m / ITEMS) & 1, abort_flag, a.status, cap)) break;
      const int idx = ctl->item[ib].idx, n = ctl->item[ib].j1 - ctl->item[ib].j0;
      mbar_arrive_warp(&ctl->item_empty[ib]);
      if (idx < 0) break;
      if (n == 0) continue;
      if (!mbar_wait_warp(&ctl->stat_full, (uint32_t)k & 1, abort_flag, a.status, cap)) break;
      ++k;
      for (int j = 0; j < n; ++j, ++c) {
        const int st = (int)(c % MST), b = (int)(c % NB);
        if (!mbar_wait_warp(&ctl->mov_full[st], (uint32_t)(c / MST) & 1, abort_flag, a.status, cap) ||
            (c >= NB &&
             !mbar_wait_warp(&ctl->step_done[b], (uint32_t)((c - NB) / NB) & 1, abort_flag, a.status, cap))) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          const uint32_t y = smem_u32(sMov + st * C::MOV_BYTES) + (is_s ? 0u : C::MTENSOR);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ss(tdst + 64 * b, kdesc(x, SPART, kk), kdesc(y, MPART, kk), C::IDESC_S, kk ? 1u : 0u);
          mma_commit(&ctl->s_full[b]);
          if (j == n - 1) mma_commit(&ctl->stat_empty);
        }
        __syncwarp();
      }
    }
    // every MMA issued has completed before TMEM is freed
    if (elect_one()) {
      mma_commit(&ctl->drain);
      mbar_drain(&ctl->drain, 0, a.status, cap);
    }
    __syncwarp();
  } else if (warp == 3) {
    // ------------------------------------------------- MMA: accumulations
    long long c = 0;
    int k = 0;
    bool ok = true;
    for (int m = 0; ok; ++m) {
      const int ib = m % ITEMS;
      if (!mbar_wait_warp(&ctl->item_full[ib], (uint32_t)(m / ITEMS) & 1, abort_flag, a.status, cap)) break;
      const Item<KV> it = ctl->item[ib];
      mbar_arrive_warp(&ctl->item_empty[ib]);
      if (it.idx < 0) break;
      if (it.j0 == it.j1) continue;
      if (k >= 1 && !mbar_wait_warp(&ctl->acc_empty, (uint32_t)(k - 1) & 1, abort_flag, a.status, cap)) break;
      ++k;
      for (int j = it.j0; j < it.j1; ++j, ++c) {
        const int b = (int)(c % NB), st = (int)(c % MST);
        if (!mbar_wait_warp(&ctl->p_full[b], (uint32_t)(c / NB) & 1, abort_flag, a.status, cap)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // Rows behind the sequence (and keys that nobody sees) may be
        // anything: their P and dS are 0, and 0 times NaN is not.  S and dP of
        // the step are complete, so nothing else reads the tile.
        uint8_t* mov = sMov + st * C::MOV_BYTES;
        const int m0 = it.moving(j);
        if (KV) {
          if (m0 + 64 > it.seq.ql && it.seq.ql < g.Nq) {
            zero_rows(mov, MPART, C::PARTS, it.seq.ql - m0, 64);
            zero_rows(mov + C::MTENSOR, MPART, C::PARTS, it.seq.ql - m0, 64);
          }
        } else {
          if (m0 + 64 > it.seq.kvl && it.seq.kvl < g.Nk) zero_rows(mov, MPART, C::PARTS, it.seq.kvl - m0, 64);
          if (m0 < it.dead_lo && m0 + 64 > it.dead_sk)
            zero_rows(mov, MPART, C::PARTS, it.dead_sk > m0 ? it.dead_sk - m0 : 0,
                      it.dead_lo - m0 < 64 ? it.dead_lo - m0 : 64);
        }
        if (elect_one()) {
          // 16 moving rows = 2048 bytes of the MN-major operand per K step; P / dS of moving rows
          // 16 kk .. 16 kk + 15 in TMEM columns 32 (kk / 2) + 8 (kk % 2) .. + 7 of the buffer
          // (bf16 pairs; each 32-row half packed at the start of its own 32 columns)
          const uint32_t y0 = smem_u32(mov), y1 = y0 + C::MTENSOR;
          const uint64_t b0 = umma_desc_sw128(y0, MPART, 1024), b1 = umma_desc_sw128(y1, MPART, 1024);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint32_t acc = (j == it.j0 && kk == 0) ? 0u : 1u;
            const uint32_t col = 64 * b + 32 * (kk >> 1) + 8 * (kk & 1);
            if (KV)
              mma_ts(tbase + Tm<KV>::ACC1, tbase + Tm<KV>::S + col, b1 + ((kk * 2048) >> 4), C::IDESC_ACC, acc);  // dV
            mma_ts(tbase + Tm<KV>::ACC0, tbase + Tm<KV>::DP + col, b0 + ((kk * 2048) >> 4), C::IDESC_ACC, acc);   // dK, dQ
          }
          mma_commit(&ctl->mov_empty[st]);
          mma_commit(&ctl->step_done[b]);
          if (j == it.j1 - 1) mma_commit(&ctl->acc_full);
        }
        __syncwarp();
      }
    }
    if (elect_one()) {
      mma_commit(&ctl->drain);
      mbar_drain(&ctl->drain, 0, a.status, cap);
    }
    __syncwarp();
  } else if (warp >= CW0) {
    // ------------------------------------------------- P, dS and epilogue
    // warps 4..7 take moving columns 0..31 of every step and the first half
    // of the accumulator columns, warps 8..11 the other halves
    const int q4 = warp & 3;
    const int part = (warp - CW0) >> 2;
    const int r = q4 * 32 + lane;                 // TMEM lane = stationary row
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const float sl2 = g.scale * 1.4426950408889634f;
    long long c = 0;
    int k = 0;
    uint32_t meets = 0;
    for (int m = 0;; ++m) {
      const int ib = m % ITEMS;
      if (!mbar_wait_warp(&ctl->item_full[ib], (uint32_t)(m / ITEMS) & 1, abort_flag, a.status, cap)) break;
      const Item<KV> it = ctl->item[ib];
      mbar_arrive_warp(&ctl->item_empty[ib]);
      const int idx = it.idx;
      if (idx < 0) break;
      const int row = it.row0 + r;
      const bool valid = row < (KV ? it.seq.kvl : it.seq.ql);
      // moving rows this row meets: KV: queries [lo, hi); else keys [lo, hi) and [0, sk)
      Span sp{0, 0, 0};
      float lr = 0.f, dr = 0.f;
      const bool steps = it.j0 < it.j1;
      if (valid && steps) {
        if (KV) {
          const int off = it.seq.kvl - it.seq.ql, u = row / g.unit;
          sp.lo = u * g.unit - off;
          sp.hi = it.seq.ql;
          if (g.window > 0 && u >= g.sinks) {
            const long long end = ((long long)u + g.window) * g.unit - off;
            sp.hi = end < sp.hi ? (int)end : sp.hi;
          }
        } else {
          sp = span_of(g, it.seq, row);
          const long long at = ((long long)it.b * g.H + it.h) * g.Nq + row;
          lr = __ldcg(a.lse2 + at);
          dr = __ldcg(a.dd + at);
        }
      }
      for (int j = it.j0; j < it.j1; ++j, ++c) {
        const int b = (int)(c % NB), st = (int)(c % MST);
        mbar_wait_step(&ctl->s_full[b], (uint32_t)(c / NB) & 1, abort_flag, a.status, cap);
        tc_fence_after();
        const int m0 = it.moving(j) + 32 * part;  // this warp's columns
        const uint32_t mask = bits(sp.lo - m0, sp.hi - m0) | (KV ? 0u : bits(0, sp.sk - m0));
        const bool masked = __any_sync(0xffffffffu, mask != 0xffffffffu);
        const uint32_t tS = tbase + Tm<KV>::S + 64 * b + lane_off + 32 * part;
        const uint32_t tD = tbase + Tm<KV>::DP + 64 * b + lane_off + 32 * part;
        uint32_t pk[16], dk[16];
        uint32_t s[32], dp[32];
        tmem_ld32(tS, s);
        tmem_ld32(tD, dp);
        tmem_wait_ld();
        const uint64_t SL = both(sl2);
        const float4* l4 = reinterpret_cast<const float4*>(&ctl->lse2[st][32 * part]);
        const float4* d4 = reinterpret_cast<const float4*>(&ctl->dd[st][32 * part]);
        float x[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) {              // four columns at a time: p = 2^(s' - lse2)
          uint64_t n0, n1;
          if (KV) {
            const float4 l = l4[i];
            n0 = f2(-l.x, -l.y);
            n1 = f2(-l.z, -l.w);
          } else {
            n0 = n1 = both(-lr);
          }
          uf2(fma2(f2(__uint_as_float(s[4 * i]), __uint_as_float(s[4 * i + 1])), SL, n0), x[4 * i], x[4 * i + 1]);
          uf2(fma2(f2(__uint_as_float(s[4 * i + 2]), __uint_as_float(s[4 * i + 3])), SL, n1), x[4 * i + 2], x[4 * i + 3]);
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = ex2(x[i]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {              // ds = p (dp - dd)
          uint64_t n0, n1;
          if (KV) {
            const float4 d = d4[i];
            n0 = f2(d.x, d.y);
            n1 = f2(d.z, d.w);
          } else {
            n0 = n1 = both(dr);
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int c2 = 4 * i + 2 * u;
            float a0, a1;
            uf2(mul2(f2(x[c2], x[c2 + 1]),
                     sub2(f2(__uint_as_float(dp[c2]), __uint_as_float(dp[c2 + 1])), u ? n1 : n0)), a0, a1);
            pk[2 * i + u] = cvt_bf16x2(x[c2], x[c2 + 1]);
            dk[2 * i + u] = cvt_bf16x2(a0, a1);
          }
        }
        if (masked) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint32_t keep = ((mask >> (2 * i)) & 1u ? 0xFFFFu : 0u) | ((mask >> (2 * i + 1)) & 1u ? 0xFFFF0000u : 0u);
            pk[i] &= keep;
            dk[i] &= keep;
          }
        }
        // packed into the first 16 of the 32 columns this warp read (the other
        // warp of the lane quarter reads and writes only its own 32)
        if (KV) tmem_st16(tS, pk);
        tmem_st16(tD, dk);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive_warp(&ctl->p_full[b]);
      }
      // ---- epilogue: accumulators to bf16 rows, or to this part's place in the workspace
      if (steps) {
        mbar_wait_step(&ctl->acc_full, (uint32_t)k & 1, abort_flag, a.status, cap);
        ++k;
        tc_fence_after();
      }
      const bool whole = !KV || it.parts == 1;
#pragma unroll 1
      for (int o = 0; o < (KV ? 2 : 1); ++o) {
        const uint32_t tacc = tbase + (o == 0 ? Tm<KV>::ACC0 : Tm<KV>::ACC1) + lane_off;
        const float mul = o == 0 ? g.scale : 1.f;      // dq, dk carry the softmax scale; dv does not
        const WinOut& out = o == 0 ? a.out0 : a.out1;
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(out.data) + (long long)it.b * out.batch +
                             (long long)(KV ? it.hk : it.h) * out.head + (long long)row * out.token;
        float* pdst = whole ? nullptr : a.part + (((long long)idx * 2 + o) * 128 + r) * D;
#pragma unroll 1
        for (int ch = part * (D / 64); ch < (part + 1) * (D / 64); ++ch) {
          uint32_t v[32];
          if (steps) {
            tmem_ld32(tacc + 32 * ch, v);
            tmem_wait_ld();
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = steps ? __float_as_uint(__uint_as_float(v[i]) * mul) : 0u;
          if (!whole) {
            uint4* d4 = reinterpret_cast<uint4*>(pdst + 32 * ch);
#pragma unroll
            for (int i = 0; i < 8; ++i) d4[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          } else if (valid) {
            uint4* d4 = reinterpret_cast<uint4*>(dst + 32 * ch);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t w[4];
#pragma unroll
              for (int u = 0; u < 4; ++u)
                w[u] = cvt_bf16x2(__uint_as_float(v[8 * i + 2 * u]), __uint_as_float(v[8 * i + 2 * u + 1]));
              d4[i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
      }
      if (steps) {
        tc_fence_before();
        mbar_arrive_warp(&ctl->acc_empty);
      }
      if (!whole) {
        // the last of the tile's parts to arrive adds them in ascending order
        __threadfence();
        mbar_arrive_warp(&ctl->meet);
        mbar_wait_step(&ctl->meet, meets++ & 1, abort_flag, a.status, cap);
        if (threadIdx.x == CW0 * 32) ctl->last = atomicAdd(a.counters + it.cell, 1) == it.parts - 1;
        mbar_arrive_warp(&ctl->meet);
        mbar_wait_step(&ctl->meet, meets++ & 1, abort_flag, a.status, cap);
        if (ctl->last) {
          __threadfence();
          const float* src = a.part + (long long)(idx - it.part) * 2 * 128 * D;
          const long long step = 2ll * 128 * D;
          const int rows = it.seq.kvl - it.row0;             // rows past 128 or the sequence's end are not there
          constexpr int NE = 4;                              // values asked for before one is used
#pragma unroll 1
          for (int e0 = threadIdx.x - CW0 * 32; e0 < 2 * 128 * D / 4; e0 += NE * CTHREADS) {
            float acc[NE][4] = {};
#pragma unroll 1
            for (int p = 0; p < it.parts; p += 2) {
              float4 v[2][NE];
#pragma unroll
              for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < NE; ++e)
                  v[u][e] = p + u < it.parts
                                ? __ldcg(reinterpret_cast<const float4*>(src + (p + u) * step) + e0 + e * CTHREADS)
                                : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
              for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < NE; ++e) {
                  acc[e][0] += v[u][e].x;
                  acc[e][1] += v[u][e].y;
                  acc[e][2] += v[u][e].z;
                  acc[e][3] += v[u][e].w;
                }
            }
#pragma unroll
            for (int e = 0; e < NE; ++e) {
              const int at = e0 + e * CTHREADS;
              const int o = at / (32 * D), rr = at / (D / 4) % 128, d0 = at % (D / 4) * 4;
              if (rr >= rows) continue;
              const WinOut& out = o == 0 ? a.out0 : a.out1;
              __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(out.data) + (long long)it.b * out.batch +
                                   (long long)it.hk * out.head + (long long)(it.row0 + rr) * out.token + d0;
              *reinterpret_cast<uint2*>(dst) =
                  make_uint2(cvt_bf16x2(acc[e][0], acc[e][1]), cvt_bf16x2(acc[e][2], acc[e][3]));
            }
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
  if (!KV) wait_preceding();
}

// rowsum(dout * out) in fp32 and lse * log2(e), D / 8 threads a row; and the
// `zeroed` words at `words` set to 0.
template <int D>
__global__ void __launch_bounds__(256)
    window_prep_kernel(const WinGeom g, const WinOut out, const WinOut dout, const float* __restrict__ lse,
                       float* __restrict__ lse2, float* __restrict__ dd, int* words, long long zeroed) {
  start_following();
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < zeroed; i += (long long)gridDim.x * 256) words[i] = 0;
  constexpr int T = D / 8;
  const long long at = ((long long)blockIdx.x * 256 + threadIdx.x) / T;
  const int part = threadIdx.x % T;
  const long long rows = (long long)g.B * g.H * g.Nq;
  float acc = 0.f;
  bool on = at < rows;
  if (on) {
    const int i = (int)(at % g.Nq);
    const long long bh = at / g.Nq;
    const int h = (int)(bh % g.H), b = (int)(bh / g.H);
    on = i < seq_of(g, b).ql;
    if (on) {
      const uint4 o4 = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(out.data) + b * out.batch +
                                                       h * out.head + i * out.token + part * 8);
      const uint4 g4 = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(dout.data) + b * dout.batch +
                                                       h * dout.head + i * dout.token + part * 8);
      const __nv_bfloat162* o2 = reinterpret_cast<const __nv_bfloat162*>(&o4);
      const __nv_bfloat162* g2 = reinterpret_cast<const __nv_bfloat162*>(&g4);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 of = __bfloat1622float2(o2[k]), gf = __bfloat1622float2(g2[k]);
        acc = fmaf(of.x, gf.x, acc);
        acc = fmaf(of.y, gf.y, acc);
      }
    }
  }
#pragma unroll
  for (int o = T / 2; o >= 1; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if (on && part == 0) {
    dd[at] = acc;
    lse2[at] = lse[at] * 1.4426950408889634f;
  }
}

template <int D, bool KV>
cudaError_t launch_v(const CUtensorMap& s0, const CUtensorMap& s1, const CUtensorMap& m0, const CUtensorMap& m1,
                     const WinBwdArgs& a, bool early, int num_sms, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(window_bwd_kernel<D, KV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)Sh<D>::SMEM);
  if (e != cudaSuccess) return e;
  const int grid = a.n_items < num_sms ? a.n_items : num_sms;
  return launch_after(early, window_bwd_kernel<D, KV>, grid, THREADS, Sh<D>::SMEM, s, s0, s1, m0, m1, a);
}

}  // namespace wb

cudaError_t launch_window_prep(const WinGeom& g, const WinOut& out, const WinOut& dout, const float* lse, float* lse2,
                               float* dd, int* words, long long zeroed, cudaStream_t s) {
  const long long threads = (long long)g.B * g.H * g.Nq * (g.D / 8);
  const unsigned blocks = (unsigned)((threads + 255) / 256);
  if (g.D == 128)
    wb::window_prep_kernel<128><<<blocks, 256, 0, s>>>(g, out, dout, lse, lse2, dd, words, zeroed);
  else
    wb::window_prep_kernel<64><<<blocks, 256, 0, s>>>(g, out, dout, lse, lse2, dd, words, zeroed);
  return cudaGetLastError();
}

cudaError_t launch_window_bwd(const CUtensorMap& s0, const CUtensorMap& s1, const CUtensorMap& m0,
                              const CUtensorMap& m1, const WinBwdArgs& a, bool key_stationary, bool early,
                              int num_sms, cudaStream_t s) {
  if (a.g.D == 128)
    return key_stationary ? wb::launch_v<128, true>(s0, s1, m0, m1, a, early, num_sms, s)
                          : wb::launch_v<128, false>(s0, s1, m0, m1, a, early, num_sms, s);
  return key_stationary ? wb::launch_v<64, true>(s0, s1, m0, m1, a, early, num_sms, s)
                        : wb::launch_v<64, false>(s0, s1, m0, m1, a, early, num_sms, s);
}

}  // namespace fvattn
