// Causal attention with a sliding window and sinks, forward, on the
// 5th-generation tensor cores: whole sequences, chunks against a cache, and
// single tokens.  Query i of a sequence stands at position
// p = i + kv_len - q_len and sees the keys of its own unit and the window - 1
// units before it, and the first `sinks` units (see span_of).
//   s = scale q k^T, out = sum_j 2^(s'_j - m) v_j / sum_j 2^(s'_j - m),
//   s' = s log2(e), lse = ln 2 (m + log2 sum_j 2^(s'_j - m)),
// in one pass over the visible keys.  The reference m of a row stands 40 above
// the largest logit of its first visible key tile; it moves (and O is rescaled)
// only when the probabilities of a later tile sum past 2^24, which fp32 sums
// and bf16 probabilities hold without loss, so no step takes a row maximum.
//
// Persistent kernel, one CTA per SM, 384 threads, over items of two 128-row
// query tiles A, B that share one stream of 128-key tiles:
//   warp 0       TMA: takes the CTA's next item from a counter, publishes it
//                in a ring in shared memory (the other warps would each spend
//                3,000 clocks on its divisions), loads its Q and its K and V
//                tiles, these through one ring;
//   warp 1       MMAs, for tile A and then tile B of every step:
//                O_g += P_g(j-1) V, then S_g(j) = Q_g K^T into the TMEM
//                columns P_g(j-1) held (MMAs of one thread run in issue
//                order; handing P over in halves of 64 keys, for an earlier
//                start, cost more in fences than it won: 227 against 211 us
//                at 2 x 32 heads, 4,099 tokens, window 1,024).  The
//                fixed order keeps the tiles half a step apart, so that one's
//                products run during the other's softmax; with a warp of its
//                own for each tile both fell into step, exponentials against
//                exponentials, and a step took 5,260 clocks instead of 4,200;
//   warps 4-7, 8-11   softmax of tile A, B: thread r owns row r; P is
//                written back over S as bf16 (the A operand of the PV MMA;
//                its rounding, relative 2^-8, is the step's largest error).
// Key tiles that none of a tile's rows sees are skipped for that tile, and
// only tiles that some row sees in part are masked.  Output rows go through
// shared memory so that a store writes whole 128-byte lines (a thread storing
// its own row took 6,400 clocks an item).
//
// Few queries (at most 128 rows a KV head, the query heads of a KV head
// packed into one tile when there are fewer than 128 queries): both softmax
// groups work on the same query tile, on alternate key tiles, and the key
// tiles of an item are split over several CTAs.  Up to 32 (64) rows are held
// four times (twice), 32 (64) lanes apart, and each copy's warps work on a
// quarter (half) of every tile's keys, the rest of its P being 0: one warp
// over all 128 keys took 4,800 clocks a tile where K and V take 2,800 to
// read.  Bound by the reading of K and V, this form has tensor time to spare
// and gives P a second bf16 for what the first one rounds away (a second PV
// product).  Each copy of each group writes its normalised part and its lse to
// the workspace; whoever completes an item's parts (a counter per item) joins
// them in ascending order, so the result does not depend on who that is.
// Warp 1 issues the S of every step and warp 2 its PV, so that neither waits
// for the other's operands; with up to 32 rows warp 3 counts and joins the
// parts, beside the next item's steps (32 sequences of up to 32,768 keys,
// 32 / 8 heads, window 8,192: 231 -> 221 us), with more rows a softmax group.
//
// TMEM (512 columns): S_A, S_B at 0, 128, O_A, O_B at 256, 384.  P goes over
// the first 64 columns of S, or, with its second bf16, each 32 keys' two parts
// over their own columns.  Shared memory: Q 2 x
// 128 rows, ring of 128-key tiles, all in 128-byte swizzled parts of 64 dims;
// 4 KB a softmax warp for the output.
#include "window.cuh"

namespace fvattn {
namespace win {

constexpr int THREADS = 384;
constexpr int SW0 = 4;                       // first softmax warp
constexpr uint32_t PART = 128 * 128;         // 64 dims of 128 rows: 16 KB
// A row's reference stands 2^HEAD above the largest logit it was taken from,
// and a step's probabilities (of 128 keys; few queries: of 32) may sum to
// RESCALE_SUM before it moves: logits may rise by 64 in base 2, so moves are
// rare (without the head and with sums up to 2^24, logits of a spread of 10
// took 316 us where this takes 212, at 2 x 32 heads, 4,099 tokens, window
// 1,024), and O, sums of probabilities times V over up to 2^21 steps, stays in
// fp32 for |v| up to 2^80 (at most 2^21 2^26 2^80) and down to 2^-80 (2^-40
// 2^-80 and 2^-6 of it are normal numbers).
constexpr float HEAD = 40.f, HEAD_MUL = 1099511627776.f;   // 2^40
constexpr float RESCALE_SUM = 16777216.f;    // 2^24
constexpr uint32_t TMEM_COLS = 512, TM_S = 0, TM_O = 256;

constexpr int ITEMS = 2;                     // items published ahead
constexpr uint32_t OUT_STAGE = 32 * 128;     // 32 rows x 128 bytes a softmax warp

// The single form holds one query tile, which leaves the ring a stage more:
// what is on its way from memory is what bounds it.
template <int D, bool DUAL> struct Cfg {
  static constexpr int PARTS = D / 64, QTILES = DUAL ? 2 : 1;
  static constexpr uint32_t TILE = PART * PARTS;        // 128 rows
  static constexpr int NST = (D == 128 ? 6 : 12) - QTILES * (D == 128 ? 1 : 2);   // ring of K and V tiles
  static constexpr uint32_t SMEM = 1024 + QTILES * TILE + NST * TILE + 8 * OUT_STAGE;
  static constexpr uint32_t IDESC_S = idesc_bf16_f32(128, 128, false, false);
  static constexpr uint32_t IDESC_PV = idesc_bf16_f32(128, D, false, true);
};
constexpr int MAXST = 10;

// Item and its key tiles.
struct Item {
  int idx;               // -1: the CTA has no further item
  int b, hk, g0;         // batch, KV head, first query head of the tile within the KV head's (0 when packed)
  int tile;              // first 128-row query tile
  int split;
  Seq seq;
  int ns, t_lo, n;       // steps 0 .. ns - 1 are key tiles 0 .., the others t_lo, t_lo + 1, ..; n steps in all
  int j0, j1;            // this split's steps
  int a_lo[2], a_hi[2], a_sk[2];   // query tile g works on key tiles [a_lo, a_hi) and, below, [0, a_sk)
  int dead_lo, dead_sk;  // keys in [dead_sk, dead_lo) are seen by no query of the sequence
  __device__ int key_tile(int j) const { return j < ns ? j : t_lo + j - ns; }
};

struct FwdCtl {
  uint64_t item_full[ITEMS], item_empty[ITEMS];   // the warps behind the producer read an item
  uint64_t q_full, q_empty;
  uint64_t kv_full[MAXST], kv_empty[MAXST];
  uint64_t s_full[2];      // S_g of its next step written (and every earlier MMA of the tile complete)
  uint64_t p_full[2];      // P_g written (4 warps)
  uint64_t pv_done[2];     // single form: the PV of a step of group g complete
  uint64_t o_full[2];      // the item's last PV of tile g complete
  uint64_t o_empty[2];     // O_g read (4 warps)
  uint64_t group[2];       // softmax group t meets (4 warps)
  uint64_t ready[ITEMS];   // single form, four copies: the item's parts written (8 warps)
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int last[2];             // this group's part was the item's last
  Item item[ITEMS];
};
static_assert(Cfg<128, true>::SMEM + sizeof(FwdCtl) <= 232448 && Cfg<128, false>::SMEM + sizeof(FwdCtl) <= 232448 &&
                  Cfg<64, true>::SMEM + sizeof(FwdCtl) <= 232448 && Cfg<64, false>::SMEM + sizeof(FwdCtl) <= 232448 &&
                  Cfg<64, false>::NST <= MAXST,
              "shared memory");

// P of 32 logits as 16 bf16x2 words (and what they round away as 16 more),
// their fp32 sum added to acc.  In three sweeps: one pair after another waits
// out every instruction's latency.
template <bool MASKED, bool TWO>
__device__ inline void exp_chunk(const uint32_t (&s)[32], uint64_t SL, uint64_t NM, uint32_t mask, uint32_t* pk,
                                 uint32_t* lo, uint64_t (&acc)[2]) {
  float x[32];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float a = __uint_as_float(s[2 * i]), b = __uint_as_float(s[2 * i + 1]);
    if (MASKED) {
      a = (mask >> (2 * i)) & 1u ? a : -INFINITY;
      b = (mask >> (2 * i + 1)) & 1u ? b : -INFINITY;
    }
    uf2(fma2(f2(a, b), SL, NM), x[2 * i], x[2 * i + 1]);
  }
#pragma unroll
  for (int i = 0; i < 32; ++i) x[i] = ex2(x[i]);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    acc[i & 1] = add2(acc[i & 1], f2(x[2 * i], x[2 * i + 1]));
    const uint32_t w = cvt_bf16x2(x[2 * i], x[2 * i + 1]);
    pk[i] = w;
    if (TWO) lo[i] = cvt_bf16x2(x[2 * i] - __uint_as_float(w << 16), x[2 * i + 1] - __uint_as_float(w & 0xFFFF0000u));
  }
}

__device__ inline uint32_t chunk_mask(const Span& sp, int key0) {
  return bits(sp.lo - key0, sp.hi - key0) | bits(0, sp.sk - key0);
}

// P of a row's 128 logits, which start at tS, and their sum.  32 logits are on
// their way while 32 are worked on.
template <bool MASKED>
__device__ inline float exp_row(uint32_t tS, float sl2, float m, const Span& sp, int key0, uint32_t (&pk)[64]) {
  const uint64_t SL = f2(sl2, sl2), NM = f2(-m, -m);
  uint64_t acc[2] = {0ull, 0ull};
  uint32_t s0[32], s1[32];
  tmem_ld32(tS, s0);
  tmem_wait_ld();
  tmem_ld32(tS + 32, s1);
  exp_chunk<MASKED, false>(s0, SL, NM, MASKED ? chunk_mask(sp, key0) : 0u, pk, nullptr, acc);
  tmem_wait_ld();
  tmem_ld32(tS + 64, s0);
  exp_chunk<MASKED, false>(s1, SL, NM, MASKED ? chunk_mask(sp, key0 + 32) : 0u, pk + 16, nullptr, acc);
  tmem_wait_ld();
  tmem_ld32(tS + 96, s1);
  exp_chunk<MASKED, false>(s0, SL, NM, MASKED ? chunk_mask(sp, key0 + 64) : 0u, pk + 32, nullptr, acc);
  tmem_wait_ld();
  exp_chunk<MASKED, false>(s1, SL, NM, MASKED ? chunk_mask(sp, key0 + 96) : 0u, pk + 48, nullptr, acc);
  return sum2(add2(acc[0], acc[1]));
}

// Largest visible of a row's 32 logits at tS (-inf: none).
__device__ inline float max_chunk(uint32_t tS, const Span& sp, int key0) {
  float m = -INFINITY;
  uint32_t s[32];
  tmem_ld32(tS, s);
  tmem_wait_ld();
  const uint32_t mask = chunk_mask(sp, key0);
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if ((mask >> i) & 1u) m = fmaxf(m, __uint_as_float(s[i]));
  return m;
}

// The same of all 128.
__device__ inline float max_row(uint32_t tS, const Span& sp, int key0) {
  float m = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) m = fmaxf(m, max_chunk(tS + 32 * c, sp, key0 + 32 * c));
  return m;
}

// O of this row times alpha.
template <int D> __device__ inline void scale_o(uint32_t tO, float alpha) {
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

__device__ inline Item item_of(const WinFwdArgs& a, int idx0) {
  const WinGeom& g = a.g;
  Item it;
  it.idx = idx0;
  unsigned idx = idx0;
  it.split = idx % a.splits;
  idx /= a.splits;
  const int qt = idx % a.item_tiles;
  idx /= a.item_tiles;
  const unsigned per_kv = g.G / a.pack;        // head slots of a KV head
  it.g0 = idx % per_kv;
  idx /= per_kv;
  it.hk = idx % g.Hk;
  it.b = idx / g.Hk;
  it.tile = (a.item_tiles - 1 - qt) * (a.dual ? 2 : 1);   // the longest spans first
  it.seq = seq_of(g, it.b);
  int lo = 0x7fffffff, hi = 0, sk = 0;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    it.a_lo[t] = it.a_hi[t] = it.a_sk[t] = 0;
    const int i0 = (it.tile + (a.dual ? t : 0)) * a.tokens;
    if (i0 >= it.seq.ql) continue;
    const int i1 = i0 + a.tokens < it.seq.ql ? i0 + a.tokens : it.seq.ql;
    const Span last = span_of(g, it.seq, i1 - 1);
    if (last.hi == 0) continue;
    const int first_pos = it.seq.ql - it.seq.kvl;          // first query that is not in front of the keys
    const int lo_t = span_of(g, it.seq, i0 > first_pos ? i0 : first_pos).lo;
    it.a_lo[t] = lo_t >> 7;
    it.a_hi[t] = (last.hi + 127) >> 7;
    it.a_sk[t] = (last.sk + 127) >> 7;
    lo = lo_t < lo ? lo_t : lo;
    hi = last.hi > hi ? last.hi : hi;
    sk = last.sk > sk ? last.sk : sk;
  }
  it.ns = it.t_lo = it.n = 0;
  if (hi > 0) {
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

// The key tiles of one query tile (dual) or one group's turns (single).
template <bool DUAL> struct Turn {
  int lo, hi, sk, j0, t;
  __device__ Turn(const Item& it, int t_) : lo(it.a_lo[t_]), hi(it.a_hi[t_]), sk(it.a_sk[t_]), j0(it.j0), t(t_) {}
  __device__ bool on(int j, int key_tile) const {
    return DUAL ? key_tile < hi && (key_tile >= lo || key_tile < sk) : ((j - j0) & 1) == t;
  }
};

// Writes 128 bytes of 32 consecutive rows of one head (lane r: row r, 32 words
// in v) by a TMA store (the swizzle is the map's), which runs on while the warp
// goes on; rows past the tensor's end are not written.
__device__ inline void store_rows_tma(uint8_t* stage, const uint32_t (&v)[32], const CUtensorMap* map, int dim, int row,
                                      int head, int batch) {
  const int lane = threadIdx.x & 31;
  uint4* st = reinterpret_cast<uint4*>(stage);
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");   // the store before is read
  __syncwarp();
#pragma unroll
  for (int c = 0; c < 8; ++c)
    st[lane * 8 + (c ^ (lane & 7))] = make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(map),
                 "r"(smem_u32(stage)), "r"(dim), "r"(row), "r"(head), "r"(batch)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
}

// The same of 32 rows anywhere, to the rows' own addresses through the warp's staging: eight lanes write
// a row's line.  Chunks of 16 bytes are swizzled by the row against bank
// conflicts.
__device__ inline void store_rows(uint8_t* stage, const uint32_t (&v)[32], uint8_t* row_ptr, bool valid) {
  const int lane = threadIdx.x & 31;
  uint4* st = reinterpret_cast<uint4*>(stage);
#pragma unroll
  for (int c = 0; c < 8; ++c)
    st[lane * 8 + (c ^ (lane & 7))] = make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
  __syncwarp();
  const unsigned mask = __ballot_sync(0xffffffffu, valid);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int row = 4 * k + (lane >> 3), c = lane & 7;
    const unsigned long long p = __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row_ptr), row);
    if ((mask >> row) & 1u) reinterpret_cast<uint4*>(p)[c] = st[row * 8 + (c ^ (row & 7))];
  }
  __syncwarp();
}

// Joining the parts of `rows` rows by NT threads (r: this one's number).  What other SMs wrote is
// about 1,000 clocks away, so every step asks for several values before it
// uses one (one after another, 24 parts of 4 rows took 25,000 clocks).
template <int NT> struct JoinRows {
  const float *lse, *o;   // part 0 of row 0
  long long step;         // rows from a part to the next
  int parts, rows;

  // lse of rows rb .. re - 1, all parts, into sh [rows][parts]
  __device__ void load_lse(float* sh, int rb, int re, int r) const {
    const int n = (re - rb) * parts;
#pragma unroll 1
    for (int e0 = r; e0 < n; e0 += 4 * NT) {
      float v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int e = e0 + NT * k < n ? e0 + NT * k : e0;
        v[k] = __ldcg(lse + (e % parts) * step + rb + e / parts);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (e0 + NT * k < n) sh[e0 + NT * k] = v[k];
    }
  }
  // one row's parts to their shares 2^(lse_p - max) / sum; returns its lse (natural)
  __device__ float shares(float* sh) const {
    float M = -INFINITY, L = 0.f;
#pragma unroll 1
    for (int p = 0; p < parts; ++p) M = fmaxf(M, sh[p]);
    const float M_use = M == -INFINITY ? 0.f : M;
#pragma unroll 1
    for (int p = 0; p < parts; ++p) {
      const float w = ex2(sh[p] - M_use);
      sh[p] = w;
      L += w;
    }
    const float li = L > 0.f || L != L ? 1.f / L : 0.f;
#pragma unroll 1
    for (int p = 0; p < parts; ++p) sh[p] *= li;
    return li == 0.f ? -INFINITY : (M_use + __log2f(L)) * 0.6931471805599453f;
  }
  // NR rows x NP parts at a time: rows row, row + RPP, ..
  template <int D, int NR, int NP>
  __device__ void some(const float* sh, int rb, int re, int row, int d0, float (&acc)[NR][4]) const {
    constexpr int RPP = 4 * NT / D;
    int up[NR];
#pragma unroll
    for (int k = 0; k < NR; ++k) {
      up[k] = row + k * RPP < re ? k * RPP : 0;                // one that is not there repeats the first
      acc[k][0] = acc[k][1] = acc[k][2] = acc[k][3] = 0.f;
    }
    const float* w = sh + (row - rb) * parts;
    const float* op = o + (long long)row * D + d0;
#pragma unroll 1
    for (int p0 = 0; p0 < parts; p0 += NP) {
      float4 v[NP][NR];
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int k = 0; k < NR; ++k)
          v[p][k] = __ldcg(reinterpret_cast<const float4*>(op + ((p0 + p < parts ? p0 + p : p0) * step + up[k]) * D));
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int k = 0; k < NR; ++k) {
          const float x = p0 + p < parts ? w[up[k] * parts + p0 + p] : 0.f;
          acc[k][0] = fmaf(x, v[p][k].x, acc[k][0]);
          acc[k][1] = fmaf(x, v[p][k].y, acc[k][1]);
          acc[k][2] = fmaf(x, v[p][k].z, acc[k][2]);
          acc[k][3] = fmaf(x, v[p][k].w, acc[k][3]);
        }
    }
  }
  // out(row, first dim, four dims) for rows rb .. re - 1
  template <int D, typename F> __device__ void sum(const float* sh, int rb, int re, int r, F out) const {
    constexpr int TPR = D / 4, RPP = NT / TPR;         // threads a row, rows a pass
    const int d0 = (r % TPR) * 4;
    if (NT == 32 || re - rb <= RPP) {
#pragma unroll 1
      for (int row = rb + r / TPR; row < re; row += RPP) {
        float acc[1][4];
        some<D, 1, 8>(sh, rb, re, row, d0, acc);
        out(row, d0, acc[0]);
      }
    } else {
#pragma unroll 1
      for (int row = rb + r / TPR; row < re; row += 4 * RPP) {
        float acc[4][4];
        some<D, 4, 2>(sh, rb, re, row, d0, acc);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (row + k * RPP < re) out(row + k * RPP, d0, acc[k]);
      }
    }
  }
};

template <int D, bool DUAL>
__global__ void __launch_bounds__(THREADS, 1)
    window_fwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                      const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo,
                      const WinFwdArgs a) {
  using C = Cfg<D, DUAL>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sKV = smem + C::QTILES * C::TILE;
  uint8_t* sOut = sKV + C::NST * C::TILE;
  __shared__ FwdCtl ctl_s;
  FwdCtl* ctl = &ctl_s;
  volatile int* abort_flag = &ctl->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WinGeom& g = a.g;
  const long long cap = a.wait_cap;

  if (threadIdx.x == 0) {
    for (int i = 0; i < ITEMS; ++i) {
      mbar_init(&ctl->item_full[i], 1);
      mbar_init(&ctl->item_empty[i], DUAL ? 9 : 11);
      mbar_init(&ctl->ready[i], 8);
    }
    mbar_init(&ctl->q_full, 1);
    mbar_init(&ctl->q_empty, 1);
    for (int i = 0; i < C::NST; ++i) {
      mbar_init(&ctl->kv_full[i], 1);
      mbar_init(&ctl->kv_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->s_full[i], 1);
      mbar_init(&ctl->p_full[i], 4);
      mbar_init(&ctl->pv_done[i], 1);
      mbar_init(&ctl->o_full[i], 1);
      mbar_init(&ctl->o_empty[i], 4);
      mbar_init(&ctl->group[i], 4);
    }
    mbar_init(&ctl->drain, DUAL ? 1 : 2);         // a final commit of each MMA warp
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

  // Registers: the launch's 168 a thread (384 x 168) are 88 for these four
  // warps and 208 for the softmax's eight, whose row of logits and
  // probabilities spilled in 168.
  if (warp == 0) {
    // ---------------------------------------------------------------- TMA
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (lane == 0) {
      prefetch_tensormap(&mq);
      prefetch_tensormap(&mk);
      prefetch_tensormap(&mv);
      long long seq = 0;
      int q_issued = 0;
      bool ok = true;
      int idx = blockIdx.x;
      for (int n = 0;; ++n) {
        const int ib = n % ITEMS;
        if (n >= ITEMS && !mbar_wait(&ctl->item_empty[ib], (uint32_t)(n / ITEMS - 1) & 1, abort_flag, a.status, cap))
          break;
        if (idx >= a.n_items) {
          ctl->item[ib].idx = -1;
          mbar_arrive(&ctl->item_full[ib]);
          break;
        }
        const Item it = item_of(a, idx);
        ctl->item[ib] = it;
        mbar_arrive(&ctl->item_full[ib]);
        idx = gridDim.x + atomicAdd(a.next_item, 1);        // the one after this
        if (it.j0 >= it.j1) continue;
        if (q_issued >= 1 && !mbar_wait(&ctl->q_empty, (uint32_t)(q_issued - 1) & 1, abort_flag, a.status, cap)) break;
        const int tiles = DUAL ? 2 : 1;
        const int copies = DUAL ? 1 : a.copies;
        mbar_arrive_expect_tx(&ctl->q_full, (uint32_t)(tiles * copies * C::PARTS * a.pack * a.tokens) * 128u);
        for (int t = 0; t < tiles; ++t)
          for (int c = 0; c < copies; ++c)
            for (int h = 0; h < C::PARTS; ++h)
              tma_load_5d(sQ + t * C::TILE + h * PART + c * (PART / copies), &mq, &ctl->q_full, 64 * h, it.g0,
                          (it.tile + t) * a.tokens, it.hk, it.b);
        ++q_issued;
        for (int j = it.j0; j < it.j1 && ok; ++j) {
          const int key0 = 128 * it.key_tile(j);
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
        if (!ok) break;
      }
      // every copy issued has landed before the block exits
      if (q_issued >= 1) mbar_drain(&ctl->q_full, (uint32_t)(q_issued - 1) & 1, a.status, cap);
      for (int i = 0; i < C::NST && i < seq; ++i) {
        const long long last = i + ((seq - 1 - i) / C::NST) * C::NST;
        mbar_drain(&ctl->kv_full[i], (uint32_t)(last / C::NST) & 1, a.status, cap);
      }
    }
  } else if (DUAL && warp == 1) {
    // ------------------------------------------------------ MMAs, two tiles
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    long long seq = 0;               // ring number of the K tile of the item's first step
    int q_items = 0;                 // items with steps
    uint32_t cnt[2] = {0, 0};        // steps of each tile
    int items[2] = {0, 0};           // items whose O_t was written
    bool ok = true;
    const uint32_t q_at = uni(smem_u32(sQ)), kv_base = smem_u32(sKV), tb = uni(tbase);
    for (int n = 0; ok; ++n) {
      const int ib = n % ITEMS;
      if (!mbar_wait_warp(&ctl->item_full[ib], (uint32_t)(n / ITEMS) & 1, abort_flag, a.status, cap)) break;
      const Item& si = ctl->item[ib];
      const int idx = si.idx, j0 = si.j0, j1 = si.j1, ns = si.ns, t_lo = si.t_lo, kvl = si.seq.kvl;
      const int dead_lo = si.dead_lo, dead_sk = si.dead_sk;
      const Turn<DUAL> turn[2] = {Turn<DUAL>(si, 0), Turn<DUAL>(si, 1)};
      mbar_arrive_warp(&ctl->item_empty[ib]);
      if (idx < 0) break;
      if (j0 >= j1) continue;
      if (!mbar_wait_warp(&ctl->q_full, (uint32_t)q_items & 1, abort_flag, a.status, cap)) break;
      ++q_items;
      bool first[2] = {true, true}, prev[2] = {false, false}, done[2] = {false, false};
      int prev_key0 = 0;
      for (int j = j0; j <= j1 && ok; ++j) {
        const long long sk = seq + 2ll * (j - j0), sv = sk - 1;     // K of step j, V of step j - 1
        const int stk = (int)(sk % C::NST), stv = (int)(sv % C::NST);
        const uint32_t k_at = uni(kv_base + stk * C::TILE), v_at = uni(kv_base + stv * C::TILE);
        const int kt = j < ns ? j : t_lo + j - ns;
        auto issue_s = [&](int t) {
          if (elect_one()) {
            const uint64_t qd = umma_desc_sw128(q_at + t * C::TILE, 16, 1024);
            const uint64_t kd = umma_desc_sw128(k_at, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = ((kk >> 2) * PART + (kk & 3) * 32) >> 4;
              mma_ss(tb + TM_S + 128 * t, qd + off, kd + off, C::IDESC_S, kk ? 1u : 0u);
            }
            mma_commit(&ctl->s_full[t]);
          }
          __syncwarp();
          ++cnt[t];
        };
        if (j > j0) {
          if (!mbar_wait_warp(&ctl->kv_full[stv], (uint32_t)(sv / C::NST) & 1, abort_flag, a.status, cap)) {
            ok = false;
            break;
          }
          // values that no query of the sequence sees may be anything: their
          // probabilities are 0, and 0 times NaN is not
          if (prev_key0 + 128 > kvl && kvl < g.Nk)
            zero_rows(sKV + stv * C::TILE, PART, C::PARTS, kvl - prev_key0, 128);
          if (prev_key0 < dead_lo && prev_key0 + 128 > dead_sk)
            zero_rows(sKV + stv * C::TILE, PART, C::PARTS, dead_sk > prev_key0 ? dead_sk - prev_key0 : 0,
                      dead_lo - prev_key0 < 128 ? dead_lo - prev_key0 : 128);
        }
        if (j < j1 && !mbar_wait_warp(&ctl->kv_full[stk], (uint32_t)(sk / C::NST) & 1, abort_flag, a.status, cap)) {
          ok = false;
          break;
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const uint32_t tS = tb + TM_S + 128 * t, tO = tb + TM_O + 128 * t;
          if (prev[t]) {
            // no step of this tile from here on: its key tiles ascend, sinks first
            const bool last = j == j1 || kt >= turn[t].hi;
            if (first[t] && items[t] >= 1 &&
                !mbar_wait_warp(&ctl->o_empty[t], (uint32_t)(items[t] - 1) & 1, abort_flag, a.status, cap)) {
              ok = false;
              break;
            }
            if (!mbar_wait_warp(&ctl->p_full[t], (cnt[t] - 1) & 1, abort_flag, a.status, cap)) {
              ok = false;
              break;
            }
            tc_fence_after();
            if (elect_one()) {
              const uint64_t vd = umma_desc_sw128(v_at, PART, 1024);
#pragma unroll
              for (int kk = 0; kk < 8; ++kk) {
                mma_ts(tO, tS + 8 * kk, vd + ((kk * 2048) >> 4), C::IDESC_PV, first[t] && kk == 0 ? 0u : 1u);
              }
              if (last) mma_commit(&ctl->o_full[t]);
            }
            __syncwarp();
            first[t] = false;
            done[t] = last;
          } else if (j == j1 && !first[t] && !done[t]) {     // the rest of this split had no step for it
            if (elect_one()) mma_commit(&ctl->o_full[t]);
            __syncwarp();
          }
          prev[t] = j < j1 && turn[t].on(j, kt);
          if (prev[t]) issue_s(t);
        }
        if (!ok) break;
        if (elect_one()) {
          if (j > j0) mma_commit(&ctl->kv_empty[stv]);
          if (j < j1) mma_commit(&ctl->kv_empty[stk]);
          if (j == j1 - 1) mma_commit(&ctl->q_empty);
        }
        __syncwarp();
        prev_key0 = 128 * kt;
      }
      items[0] += !first[0];
      items[1] += !first[1];
      seq += 2ll * (j1 - j0);
    }
    // every MMA issued has completed before TMEM is freed
    if (elect_one()) {
      mma_commit(&ctl->drain);
      mbar_drain(&ctl->drain, 0, a.status, cap);
    }
    __syncwarp();
  } else if (!DUAL && (warp == 1 || warp == 2)) {
    // ------------------------------------------------- MMAs, single form
    // Warp 1 issues the S of every step as its K arrives, warp 2 the PV as its
    // P is written: bound by memory, neither waits for what the other needs.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    const bool is_s = warp == 1;
    long long seq = 0;               // ring number of the K tile of the item's first step
    int q_items = 0;
    uint32_t cnt[2] = {0, 0};        // steps of each group
    int items[2] = {0, 0};           // items whose O_t was written
    bool ok = true;
    const uint32_t q_at = uni(smem_u32(sQ)), kv_base = smem_u32(sKV), tb = uni(tbase);
    for (int n = 0; ok; ++n) {
      const int ib = n % ITEMS;
      if (!mbar_wait_warp(&ctl->item_full[ib], (uint32_t)(n / ITEMS) & 1, abort_flag, a.status, cap)) break;
      const Item& si = ctl->item[ib];
      const int idx = si.idx, j0 = si.j0, j1 = si.j1, ns = si.ns, t_lo = si.t_lo, kvl = si.seq.kvl;
      const int dead_lo = si.dead_lo, dead_sk = si.dead_sk;
      mbar_arrive_warp(&ctl->item_empty[ib]);
      if (idx < 0) break;
      if (j0 >= j1) continue;
      if (is_s && !mbar_wait_warp(&ctl->q_full, (uint32_t)q_items & 1, abort_flag, a.status, cap)) break;
      ++q_items;
      for (int j = j0; j < j1; ++j) {
        const int t = (j - j0) & 1;
        const long long at = seq + 2ll * (j - j0) + (is_s ? 0 : 1);
        const int st = (int)(at % C::NST);
        const uint32_t tile_at = uni(kv_base + st * C::TILE), tS = uni(tb + TM_S + 128 * t), tO = uni(tb + TM_O + 128 * t);
        if (!mbar_wait_warp(&ctl->kv_full[st], (uint32_t)(at / C::NST) & 1, abort_flag, a.status, cap)) {
          ok = false;
          break;
        }
        if (is_s) {
          // the group's last P, in the columns of this S, is read
          if (cnt[t] >= 1 && !mbar_wait_warp(&ctl->pv_done[t], (cnt[t] - 1) & 1, abort_flag, a.status, cap)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            const uint64_t qd = umma_desc_sw128(q_at, 16, 1024), kd = umma_desc_sw128(tile_at, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = ((kk >> 2) * PART + (kk & 3) * 32) >> 4;
              mma_ss(tS, qd + off, kd + off, C::IDESC_S, kk ? 1u : 0u);
            }
            mma_commit(&ctl->s_full[t]);
            mma_commit(&ctl->kv_empty[st]);
            if (j == j1 - 1) mma_commit(&ctl->q_empty);
          }
        } else {
          const int key0 = 128 * (j < ns ? j : t_lo + j - ns);
          if (key0 + 128 > kvl && kvl < g.Nk) zero_rows(sKV + st * C::TILE, PART, C::PARTS, kvl - key0, 128);
          if (key0 < dead_lo && key0 + 128 > dead_sk)
            zero_rows(sKV + st * C::TILE, PART, C::PARTS, dead_sk > key0 ? dead_sk - key0 : 0,
                      dead_lo - key0 < 128 ? dead_lo - key0 : 128);
          const bool first = j - j0 < 2;
          if ((first && items[t] >= 1 &&
               !mbar_wait_warp(&ctl->o_empty[t], (uint32_t)(items[t] - 1) & 1, abort_flag, a.status, cap)) ||
              !mbar_wait_warp(&ctl->p_full[t], cnt[t] & 1, abort_flag, a.status, cap)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            const uint64_t vd = umma_desc_sw128(tile_at, PART, 1024);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              const uint32_t tP = tS + 32 * (kk >> 1) + 8 * (kk & 1);
              mma_ts(tO, tP, vd + ((kk * 2048) >> 4), C::IDESC_PV, first && kk == 0 ? 0u : 1u);
              mma_ts(tO, tP + 16, vd + ((kk * 2048) >> 4), C::IDESC_PV, 1u);
            }
            mma_commit(&ctl->pv_done[t]);
            mma_commit(&ctl->kv_empty[st]);
            if (j >= j1 - 2) mma_commit(&ctl->o_full[t]);
          }
        }
        __syncwarp();
        ++cnt[t];
      }
      items[0] += 1;
      items[1] += j1 - j0 > 1;
      seq += 2ll * (j1 - j0);
    }
    if (elect_one()) {
      mma_commit(&ctl->drain);
      mbar_drain(&ctl->drain, 0, a.status, cap);
    }
    __syncwarp();
  } else if (!DUAL && warp == 3) {
    // ---------------------------------------- joins the parts of few rows
    // (a quarter of the softmax warps' time an item went into the fence, the
    // counter and the join, with the next item's K and V waiting)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    const int prow = a.tokens * a.pack;
    for (int n = 0;; ++n) {
      const int ib = n % ITEMS;
      if (!mbar_wait_warp(&ctl->item_full[ib], (uint32_t)(n / ITEMS) & 1, abort_flag, a.status, cap)) break;
      const Item& si = ctl->item[ib];
      const int idx = si.idx, split = si.split, batch = si.b, head0 = si.hk * g.G + si.g0, tok0 = si.tile * a.tokens;
      const int left = si.seq.ql - tok0;
      if (idx < 0 || a.copies < 4) {             // the groups join larger items themselves
        mbar_arrive_warp(&ctl->item_empty[ib]);
        if (idx < 0) break;
        continue;
      }
      if (!mbar_wait_warp(&ctl->ready[ib], (uint32_t)(n / ITEMS) & 1, abort_flag, a.status, cap)) break;
      const int base = idx - split;
      int last = 0;
      if (lane == 0) {
        __threadfence();
        last = atomicAdd(a.counters + base / a.splits, 1) == a.splits - 1;
      }
      last = __shfl_sync(0xffffffffu, last, 0);
      if (last) {
        __threadfence();
        const int rows = (left < a.tokens ? left : a.tokens) * a.pack;
        const JoinRows<32> jr{a.part_lse + (long long)base * 8 * prow, a.part_o + (long long)base * 8 * prow * D, prow,
                              a.parts, rows};
        float* share = reinterpret_cast<float*>(sOut);         // [batch of rows][parts]
        const int most = (int)(8 * OUT_STAGE / sizeof(float)) / a.parts;
        for (int rb = 0; rb < rows; rb += most) {
          const int re = rb + most < rows ? rb + most : rows;
          jr.load_lse(share, rb, re, lane);
          __syncwarp();
          for (int row = rb + lane; row < re; row += 32)
            a.lse[((long long)batch * g.H + head0 + row % a.pack) * g.Nq + tok0 + row / a.pack] =
                jr.shares(share + (row - rb) * a.parts);
          __syncwarp();
          jr.template sum<D>(share, rb, re, lane, [&](int rr, int d0, const float (&v)[4]) {
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + (long long)batch * a.o_batch +
                                 (long long)(head0 + rr % a.pack) * a.o_head + (long long)(tok0 + rr / a.pack) * a.o_token +
                                 d0;
            *reinterpret_cast<uint2*>(dst) = make_uint2(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]));
          });
          __syncwarp();
        }
      }
      mbar_arrive_warp(&ctl->item_empty[ib]);    // behind the join: the ready barriers stay an item apart
    }
  } else if (warp < SW0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
  } else {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int t = (warp - SW0) >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tbase + TM_S + 128 * t + lane_off, tO = tbase + TM_O + 128 * t + lane_off;
    uint8_t* stage = sOut + (warp - SW0) * OUT_STAGE;
    const float sl2 = g.scale * 1.4426950408889634f;
    const int prow = a.tokens * a.pack;          // rows of a tile
    // Single form with few rows: every 128 / copies lanes hold a copy of the
    // rows, and each copy works on its share of the tile's 32-key chunks.
    const int copies = DUAL ? 1 : a.copies;
    const int copy = r / (128 / copies), rl = r % (128 / copies);
    const uint32_t chunks = ((1u << (4 / copies)) - 1u) << (copy * (4 / copies));
    uint32_t cnt = 0, meets = 0;
    int items = 0;
    for (int n = 0;; ++n) {
      const int ib = n % ITEMS;
      if (!mbar_wait_warp(&ctl->item_full[ib], (uint32_t)(n / ITEMS) & 1, abort_flag, a.status, cap)) break;
      const Item& si = ctl->item[ib];
      const int idx = si.idx, j0 = si.j0, j1 = si.j1, ns = si.ns, t_lo = si.t_lo, split = si.split;
      const int batch = si.b, head0 = si.hk * g.G + si.g0, tok0 = (si.tile + (DUAL ? t : 0)) * a.tokens;
      const Seq seq = si.seq;
      const Turn<DUAL> turn(si, t);
      mbar_arrive_warp(&ctl->item_empty[ib]);
      if (idx < 0) break;
      const int i = tok0 + (a.pack == 1 ? rl : rl / a.pack);                  // query
      const int head = head0 + (a.pack == 1 ? 0 : rl % a.pack);
      const bool valid = rl < prow && i < seq.ql;
      // rows that are not stored count as seeing everything: no mask for them
      const Span sp = valid ? span_of(g, seq, i) : Span{0, 0x7fffffff, 0x7fffffff};
      const int hi_min = (int)__reduce_min_sync(0xffffffffu, (unsigned)sp.hi);
      const int lo_max = (int)__reduce_max_sync(0xffffffffu, (unsigned)sp.lo);
      const int sk_min = (int)__reduce_min_sync(0xffffffffu, (unsigned)sp.sk);
      const bool warp_on = __any_sync(0xffffffffu, valid);
      float m = -INFINITY, l = 0.f;
      bool any = false, unset = true;
      for (int j = j0; j < j1; ++j) {
        const int kt = j < ns ? j : t_lo + j - ns;
        if (!turn.on(j, kt)) continue;
        mbar_wait_step(&ctl->s_full[t], cnt & 1, abort_flag, a.status, cap);
        tc_fence_after();
        any = true;
        if (warp_on) {
          const int key0 = 128 * kt;
          const bool masked = !(key0 + 128 <= hi_min && (key0 >= lo_max || key0 + 128 <= sk_min));
          if constexpr (DUAL) {
            if (unset) {                         // some row has met no visible key yet
              const float mx = max_row(tS, sp, key0) * sl2;
              if (m == -INFINITY) m = mx + HEAD;
              unset = __any_sync(0xffffffffu, m == -INFINITY);
            }
            uint32_t pk[64];
            const float m_use = m == -INFINITY ? 0.f : m;
            float sum = masked ? exp_row<true>(tS, sl2, m_use, sp, key0, pk) : exp_row<false>(tS, sl2, m_use, sp, key0, pk);
            const bool over = valid && !(sum <= RESCALE_SUM);
            if (__any_sync(0xffffffffu, over)) {
              // too large (or not a number): move the reference up and do the
              // row again.  Every earlier MMA of the tile is complete (so says
              // S), so O holds the earlier steps; before an item's first PV it
              // holds nothing that is used.
              const float mx = fmaxf(max_row(tS, sp, key0) * sl2, m_use);
              const float m_new = over ? mx + HEAD : m_use;
              const float alpha = ex2(m_use - m_new);
              if (over) m = m_new;
              sum = exp_row<true>(tS, sl2, m_new, sp, key0, pk);
              scale_o<D>(tO, alpha);
              l *= alpha;
            }
            l += sum;
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_st16(tS + 16 * c, pk + 16 * c);
          } else {
            // 32 keys at a time, P as two bf16 in the columns of their logits
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              const uint32_t tC = tS + 32 * c;
              uint32_t pk[32];
              if ((chunks >> c) & 1u) {
                const int k0 = key0 + 32 * c;
                if (unset) {
                  const float mx = max_chunk(tC, sp, k0) * sl2;
                  if (m == -INFINITY) m = mx + HEAD;
                  unset = __any_sync(0xffffffffu, m == -INFINITY);
                }
                float m_use = m == -INFINITY ? 0.f : m;
                float sum;
#pragma unroll 1
                for (int again = 0;; ++again) {
                  uint32_t s[32];
                  uint64_t acc[2] = {0ull, 0ull};
                  tmem_ld32(tC, s);
                  tmem_wait_ld();
                  exp_chunk<true, true>(s, f2(sl2, sl2), f2(-m_use, -m_use), masked ? chunk_mask(sp, k0) : ~0u, pk, pk + 16,
                                        acc);
                  sum = sum2(add2(acc[0], acc[1]));
                  const bool over = again == 0 && valid && !(sum <= RESCALE_SUM);
                  if (!__any_sync(0xffffffffu, over)) break;
                  // as above; what this step already holds of P moves too
                  const float mx = fmaxf(max_chunk(tC, sp, k0) * sl2, m_use);   // by every lane: TMEM loads are the warp's
                  const float m_new = over ? mx + HEAD : m_use;
                  const float alpha = ex2(m_use - m_new);
                  if (over) m = m_new;
                  m_use = m_new;
                  // (S waited for the PV of the group's step before, so O holds it).
                  // What this step stored of P and, at an earlier move, of O is
                  // read back here: loads wait only for stores that were waited for.
                  tmem_wait_st();
                  scale_o<D>(tO, alpha);
                  l *= alpha;
#pragma unroll 1
                  for (int e = 0; e < c; ++e) {
                    if (!((chunks >> e) & 1u)) continue;
                    tmem_ld32(tS + 32 * e, s);
                    tmem_wait_ld();
#pragma unroll
                    for (int x = 0; x < 16; ++x) {
                      const float p0 = (__uint_as_float(s[x] << 16) + __uint_as_float(s[16 + x] << 16)) * alpha;
                      const float p1 = (__uint_as_float(s[x] & 0xFFFF0000u) + __uint_as_float(s[16 + x] & 0xFFFF0000u)) * alpha;
                      s[x] = cvt_bf16x2(p0, p1);
                      s[16 + x] = cvt_bf16x2(p0 - __uint_as_float(s[x] << 16), p1 - __uint_as_float(s[x] & 0xFFFF0000u));
                    }
                    tmem_st32(tS + 32 * e, s);
                  }
                }
                l += sum;
              } else {
#pragma unroll
                for (int x = 0; x < 32; ++x) pk[x] = 0u;
              }
              tmem_st32(tC, pk);
            }
          }
          tmem_wait_st();
        }
        tc_fence_before();
        mbar_arrive_warp(&ctl->p_full[t]);
        ++cnt;
      }
      // ---- epilogue
      if (any) {
        mbar_wait_step(&ctl->o_full[t], (uint32_t)items & 1, abort_flag, a.status, cap);
        tc_fence_after();
        ++items;
      }
      const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
      const float lse2 = l > 0.f || l != l ? (m - HEAD) + __log2f(l * HEAD_MUL) : -INFINITY;
      const bool parts = !DUAL || a.parts > 1;
      const long long slot = parts ? (((long long)idx * 2 + t) * copies + copy) * prow + rl : 0;
      if (warp_on) {
        uint8_t* row_ptr =
            parts ? reinterpret_cast<uint8_t*>(a.part_o + slot * D)
                  : reinterpret_cast<uint8_t*>(static_cast<__nv_bfloat16*>(a.out) + (long long)batch * a.o_batch +
                                               (long long)head * a.o_head + (long long)i * a.o_token);
#pragma unroll 1
        for (int ch = 0; ch < D / 64; ++ch) {
          uint32_t o0[32], o1[32];
          if (any) {
            tmem_ld32(tO + ch * 64, o0);
            tmem_ld32(tO + ch * 64 + 32, o1);
            tmem_wait_ld();
          }
          // (a row that saw no key holds 0 where its tile had steps)
#pragma unroll
          for (int x = 0; x < 32; ++x) {
            o0[x] = any ? __float_as_uint(__uint_as_float(o0[x]) * inv) : 0u;
            o1[x] = any ? __float_as_uint(__uint_as_float(o1[x]) * inv) : 0u;
          }
          if (!DUAL) {
            if (valid) {
#pragma unroll
              for (int x = 0; x < 8; ++x) {
                reinterpret_cast<uint4*>(row_ptr + ch * 256)[x] = make_uint4(o0[4 * x], o0[4 * x + 1], o0[4 * x + 2], o0[4 * x + 3]);
                reinterpret_cast<uint4*>(row_ptr + ch * 256 + 128)[x] = make_uint4(o1[4 * x], o1[4 * x + 1], o1[4 * x + 2], o1[4 * x + 3]);
              }
            }
          } else if (parts) {
            store_rows(stage, o0, row_ptr + ch * 256, valid);
            store_rows(stage, o1, row_ptr + ch * 256 + 128, valid);
          } else {
            uint32_t w[32];
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              w[x] = cvt_bf16x2(__uint_as_float(o0[2 * x]), __uint_as_float(o0[2 * x + 1]));
              w[16 + x] = cvt_bf16x2(__uint_as_float(o1[2 * x]), __uint_as_float(o1[2 * x + 1]));
            }
            if (ch == D / 64 - 1 && any) {       // O is in registers: the next item's first PV may overwrite it
              tc_fence_before();
              mbar_arrive_warp(&ctl->o_empty[t]);
            }
            if (a.tma_out)
              store_rows_tma(stage, w, &mo, 64 * ch, tok0 + (warp & 3) * 32, head0, batch);
            else
              store_rows(stage, w, row_ptr + ch * 128, valid);
          }
        }
        if (valid) {
          if (parts)
            a.part_lse[slot] = lse2;
          else
            a.lse[((long long)batch * g.H + head) * g.Nq + i] = lse2 * 0.6931471805599453f;
        }
      }
      if (any && (parts || !warp_on)) {
        tc_fence_before();
        mbar_arrive_warp(&ctl->o_empty[t]);
      }
      if (!DUAL && copies == 4) {
        mbar_arrive_warp(&ctl->ready[ib]);       // the joining warp takes it from here
      } else if (parts) {
        // the group that completes the query tile's parts joins them
        __threadfence();
        mbar_arrive_warp(&ctl->group[t]);
        mbar_wait_step(&ctl->group[t], meets++ & 1, abort_flag, a.status, cap);
        const int base = idx - split;                  // split 0 of this item
        if (r == 0)
          ctl->last[t] = atomicAdd(a.counters + (DUAL ? base / a.splits * 2 + t : base / a.splits), 1) == a.parts / copies - 1;
        mbar_arrive_warp(&ctl->group[t]);
        mbar_wait_step(&ctl->group[t], meets++ & 1, abort_flag, a.status, cap);
        if (ctl->last[t]) {
          __threadfence();
          const int left = seq.ql - tok0;
          const int rows = (left < a.tokens ? left : a.tokens) * a.pack;
          // part p of a row: split p of this tile, or copy p % copies of group (p / copies) % 2 of its split
          const long long row0 = (long long)base * 2 * copies * prow + (DUAL ? t * prow : 0);
          const long long step = (DUAL ? 2ll : 1ll) * prow;
          const JoinRows<128> jr{a.part_lse + row0, a.part_o + row0 * D, step, a.parts, rows};
          float* share = reinterpret_cast<float*>(sOut + t * 4 * OUT_STAGE);        // [batch of rows][parts]
          const int most = (int)(4 * OUT_STAGE / sizeof(float)) / a.parts;
          for (int rb = 0; rb < rows; rb += most) {
            const int re = rb + most < rows ? rb + most : rows;
            jr.load_lse(share, rb, re, r);
            mbar_arrive_warp(&ctl->group[t]);
            mbar_wait_step(&ctl->group[t], meets++ & 1, abort_flag, a.status, cap);
            const int row = rb + r;
            if (row < re)
              a.lse[((long long)batch * g.H + head0 + row % a.pack) * g.Nq + tok0 + row / a.pack] =
                  jr.shares(share + r * a.parts);
            mbar_arrive_warp(&ctl->group[t]);
            mbar_wait_step(&ctl->group[t], meets++ & 1, abort_flag, a.status, cap);
            jr.template sum<D>(share, rb, re, r, [&](int rr, int d0, const float (&v)[4]) {
              __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out) + (long long)batch * a.o_batch +
                                   (long long)(head0 + rr % a.pack) * a.o_head +
                                   (long long)(tok0 + rr / a.pack) * a.o_token + d0;
              *reinterpret_cast<uint2*>(dst) = make_uint2(cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3]));
            });
            mbar_arrive_warp(&ctl->group[t]);          // the shares are read
            mbar_wait_step(&ctl->group[t], meets++ & 1, abort_flag, a.status, cap);
          }
        }
      }
    }
    if (DUAL && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");   // shared memory is read
  }

  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, TMEM_COLS);
  }
}

template <int D, bool DUAL>
cudaError_t launch_fwd(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mo,
                       const WinFwdArgs& a, int num_sms, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(window_fwd_kernel<D, DUAL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)Cfg<D, DUAL>::SMEM);
  if (e != cudaSuccess) return e;
  const int grid = a.n_items < num_sms ? a.n_items : num_sms;
  window_fwd_kernel<D, DUAL><<<grid, THREADS, Cfg<D, DUAL>::SMEM, s>>>(mq, mk, mv, mo, a);
  return cudaGetLastError();
}

}  // namespace win

cudaError_t launch_window_fwd(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mo,
                              const WinFwdArgs& a, int num_sms, cudaStream_t s) {
  if (a.g.D == 128)
    return a.dual ? win::launch_fwd<128, true>(mq, mk, mv, mo, a, num_sms, s)
                  : win::launch_fwd<128, false>(mq, mk, mv, mo, a, num_sms, s);
  return a.dual ? win::launch_fwd<64, true>(mq, mk, mv, mo, a, num_sms, s)
                : win::launch_fwd<64, false>(mq, mk, mv, mo, a, num_sms, s);
}

}  // namespace fvattn
