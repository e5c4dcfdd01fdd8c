// Layer norm in front of the QKV projection, forward and backward, with an
// affine per group of consecutive rows (one group: the plain layer norm; one
// per sample or per latent frame: the timestep modulation of a DiT block).
//   mean = sum x / C, rstd = 1 / sqrt(sum (x - mean)^2 / C + eps),
//   xhat = (x - mean) rstd, y = xhat gain + bias, gain = w or 1 + w;
//   gy = dy gain, dx = rstd (gy - sum gy / C - xhat sum(gy xhat) / C),
//   dw = sum_rows dy xhat, dbias = sum_rows dy over the rows of a group.
// Bound by memory: x is read and y written once (forward), x and dy are read
// and dx written once (backward).
//
// Forward: a block takes two rows of one group at once and holds them in
// registers, 32 elements a thread in vectors of 4: gain and bias are then one
// fully coalesced 16-byte load a vector, shared by both rows and coming from
// L1.  At 33,280 x 5,120 bf16 (104 us of memory at a copy's rate) it takes 139
// us, one row a block 201, 16 elements a thread 213, vectors of 8, which read
// every other 16 bytes of the gain, 152.  Without gain and bias it takes 135:
// what keeps it from the memory's rate is that an SM holds three blocks (128
// registers a thread), which load, meet and store in turn; most stalls wait
// for loads.  Where so few rows come that the SMs hold them all at once, a row
// is spread thin (8 a thread) for the latency.
// The variance never subtracts large sums, and no rounding is larger than one
// of the row's mean |x|: a warp takes the mean of its own elements as its
// shift, and what the shift's rounding left (s) and M2 from the differences,
//   shift = sum x / n, s = sum (x - shift) / n, M2 = sum (x - shift)^2 - n s^2;
// with one barrier a row the warps are joined about A = sum n_i shift_i / C,
//   e_i = (shift_i - A) + s_i, dm = sum n_i e_i / C, mean = A + dm,
//   M2 = sum (M2_i + n_i e_i^2) - C dm^2,
// and y comes from (x - A) - dm, which keeps what an fp32 mean cannot hold.
// (A shift by the row's first element rounds every difference at that
// element's size: 8,192 wide with x[0] = 1e4 among values near 1 it cost y
// 2e-4 and the mean 5e-4 of itself.  Both take the same time within 1%.)
//
// Backward: the column sums stay in the registers of a thread, which keeps
// its columns (and their gain) for all its rows.  Blocks walk contiguous row
// ranges of equal length (persistent grid), their teams taking the rows in
// turn; rows arrive through a ring in shared memory that each thread fills
// with asynchronous copies of its own elements (no barrier: it reads only
// what it copied), and the second pass over a row reads the ring again.  The
// sums of block c over its rows of group g are added over its teams in shared
// memory and go to partial slot c + g: the ranges and the groups are both
// ascending, so every (c, g) pair that meets has a slot of its own, and a
// second kernel adds a group's slots in ascending order (no atomics, the same
// bits every run).
//
// Rows wider than 8192 elements take the wide kernels, which pass over the
// row again from L2.
#include "packed.cuh"

namespace fvattn {
namespace ln {

using namespace pk;

constexpr int MAX_C = 8192;      // widest row of the team kernels
constexpr int MAX_WARPS = 32;    // warps of a team (8 elements a thread; 8 with 32)
constexpr int MAX_TEAMS = 15;    // teams of a block: one named barrier each
constexpr int WIDE = 1024;       // threads of a wide row's block
// rows in the backward's ring, the one at work among them
template <typename T> constexpr int stages() { return sizeof(T) == 4 ? 2 : 3; }

// VEC consecutive elements as loaded.
template <typename T, int VEC> struct Raw;
template <> struct Raw<float, 4> { using type = float4; };
template <> struct Raw<float, 1> { using type = float; };
template <> struct Raw<__nv_bfloat16, 8> { using type = uint4; };
template <> struct Raw<__nv_bfloat16, 4> { using type = uint2; };
template <> struct Raw<__nv_bfloat16, 2> { using type = uint32_t; };
template <> struct Raw<__nv_bfloat16, 1> { using type = unsigned short; };

__device__ inline float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ inline float hi16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ inline void unpack(const float4& r, float* v) { v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w; }
__device__ inline void unpack(const float& r, float* v) { v[0] = r; }
__device__ inline void unpack(const uint4& r, float* v) {
  v[0] = lo16(r.x); v[1] = hi16(r.x); v[2] = lo16(r.y); v[3] = hi16(r.y);
  v[4] = lo16(r.z); v[5] = hi16(r.z); v[6] = lo16(r.w); v[7] = hi16(r.w);
}
__device__ inline void unpack(const uint2& r, float* v) { v[0] = lo16(r.x); v[1] = hi16(r.x); v[2] = lo16(r.y); v[3] = hi16(r.y); }
__device__ inline void unpack(const uint32_t& r, float* v) { v[0] = lo16(r); v[1] = hi16(r); }
__device__ inline void unpack(const unsigned short& r, float* v) { v[0] = lo16(r); }
__device__ inline uint32_t pack2(float a, float b) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ inline void pack(const float* v, float4& r) { r = make_float4(v[0], v[1], v[2], v[3]); }
__device__ inline void pack(const float* v, float& r) { r = v[0]; }
__device__ inline void pack(const float* v, uint4& r) {
  r = make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}
__device__ inline void pack(const float* v, uint2& r) { r = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3])); }
__device__ inline void pack(const float* v, uint32_t& r) { r = pack2(v[0], v[1]); }
__device__ inline void pack(const float* v, unsigned short& r) { r = (unsigned short)(pack2(v[0], 0.f) & 0xFFFFu); }

__device__ inline float to_f(float v) { return v; }
__device__ inline float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }

__device__ inline float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Meets the warps of one team of the block.
__device__ inline void team_sync(int warps, int id) {
  if (warps == 1)
    __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(1 + id), "r"(32 * warps) : "memory");
}

// 1 / sqrt(v): the approximation (2 steps of fp32 at most) and one Newton step
// (v r first: half of a variance below 2^-126 would lose its last bits).
__device__ inline float rsqrt_near(float v) {
  const float r = rsqrtf(v);
  return v > 0.f && v < INFINITY ? r * fmaf(-0.5f * (v * r), r, 1.5f) : r;
}

struct Range {
  long long r0, r1;
};
// Rows of block c of the persistent grid.
__device__ inline Range block_rows(const NormArgs& a) {
  const long long r0 = (long long)blockIdx.x * a.rows_per_block;
  const long long r1 = r0 + a.rows_per_block;
  return {r0, r1 < a.rows ? r1 : a.rows};
}

template <int BYTES>
__device__ inline void copy_async(void* dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(dst)), "l"(src), "n"(BYTES) : "memory");
}
__device__ inline void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ inline void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Which vectors of a row a thread holds: warp w of the team the 32 NV vectors
// from 32 NV w on, its lane l every 32nd of them from l on, so that a thread's
// addresses differ by constants.  FULL: the row fills every thread.  Otherwise
// a vector past the row's end stands for the row's last one, so that loads
// need no branch (one branch a vector kept the loads from being issued
// together: 33,280 x 5,120 bf16 took 240 us so), and its values are masked.
template <bool FULL> struct Place {
  int first, nvec;
  __device__ bool on(int k) const { return FULL || first + 32 * k < nvec; }
  __device__ int at(int k) const { return FULL || first + 32 * k < nvec ? first + 32 * k : nvec - 1; }
};

// The ring of one tensor's rows, a slot of its own for every vector of every
// thread.  Where a vector is a single bf16 there is no copy that small: the
// team copies the row's aligned words instead (WORDS), one element further on
// in shared memory when the row starts inside a word, and meets before it
// reads them.
template <typename T, int VEC, int EPT, bool FULL> struct Ring {
  using R = typename Raw<T, VEC>::type;
  static constexpr int NV = EPT / VEC, STAGES = stages<T>();
  static constexpr bool WORDS = sizeof(T) * VEC < 4;
  static __host__ __device__ constexpr int bytes(int team) { return EPT * (int)sizeof(T) * team + (WORDS ? 16 : 0); }
  unsigned char* base;               // the team's ring
  Place<FULL> pl;
  int team, t, C;
  __device__ unsigned char* stage(int s) const { return base + s * bytes(team); }
  __device__ void fetch(int s, const T* row) const {
    unsigned char* dst = stage(s);
    if constexpr (WORDS) {
      const int odd = (int)((reinterpret_cast<uintptr_t>(row) >> 1) & 1);
      const T* w0 = row - odd;       // aligned word that holds the row's first element
      const int n = C + odd;         // elements from there to the row's end
      for (int i = t; i < n / 2; i += team)
        if (i > 0 || odd == 0) copy_async<4>(dst + 4 * i, w0 + 2 * i);
      // elements alone in their word: the first after an odd start, the last before an odd end
      if (odd && t == 0) reinterpret_cast<unsigned short*>(dst)[1] = *reinterpret_cast<const unsigned short*>(row);
      if ((n & 1) && t == team - 1)
        reinterpret_cast<unsigned short*>(dst)[n - 1] = *reinterpret_cast<const unsigned short*>(w0 + n - 1);
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v)
        copy_async<(int)sizeof(R)>(dst + (pl.first + 32 * v) * sizeof(R), reinterpret_cast<const R*>(row) + pl.at(v));
    }
  }
  __device__ R get(int s, int v, const T* row) const {
    if constexpr (WORDS)
      return *reinterpret_cast<const R*>(stage(s) + 2 * (pl.at(v) + (int)((reinterpret_cast<uintptr_t>(row) >> 1) & 1)));
    else
      return *reinterpret_cast<const R*>(stage(s) + (pl.first + 32 * v) * sizeof(R));
  }
};

// Values a thread keeps: team, place in it.
struct Lane {
  int lane, warp, warps, team, teams, id, t;
  __device__ Lane(int warps_)
      : lane(threadIdx.x & 31), warp(threadIdx.x >> 5), warps(warps_), team(32 * warps_), teams(1), id(0),
        t((int)threadIdx.x) {
    if ((int)blockDim.x != team) {
      teams = (int)blockDim.x / team;
      id = (int)threadIdx.x / team;
      t = (int)threadIdx.x - id * team;
    }
  }
};

// The thread's elements in chunks of packed pairs: a chunk is one vector, or
// two single elements.
template <typename T, int VEC, int EPT, bool FULL> struct Chunks {
  using R = typename Raw<T, VEC>::type;
  static constexpr int CE = VEC == 1 ? 2 : VEC;      // elements of a chunk
  static constexpr int NP = CE / 2, N = EPT / CE, VC = VEC == 1 ? 2 : 1;   // vectors of a chunk
  struct Part {
    R v[VC];
  };
  Place<FULL> pl;
  // 64-bit mask of pair i's existing elements
  __device__ uint64_t mask(int k) const {
    if constexpr (FULL) return ~0ull;
    if constexpr (VEC == 1)
      return (pl.on(2 * k) ? 0xFFFFFFFFull : 0ull) | (pl.on(2 * k + 1) ? 0xFFFFFFFF00000000ull : 0ull);
    else
      return pl.on(k) ? ~0ull : 0ull;
  }
  __device__ float count() const {
    if (FULL) return (float)EPT;
    int n = 0;
#pragma unroll
    for (int v = 0; v < N * VC; ++v) n += pl.on(v) ? VEC : 0;
    return (float)n;
  }
  __device__ void load(const T* row, int k, Part& p) const {
#pragma unroll
    for (int j = 0; j < VC; ++j) p.v[j] = __ldcs(reinterpret_cast<const R*>(row) + pl.at(VC * k + j));
  }
  template <typename Rg> __device__ void get(const Rg& ring, int st, int k, const T* row, uint64_t (&d)[NP]) const {
    Part p;
#pragma unroll
    for (int j = 0; j < VC; ++j) p.v[j] = ring.get(st, VC * k + j, row);
    pairs(p, d);
  }
  static __device__ void pairs(const Part& p, uint64_t (&d)[NP]) {
    float f[CE];
#pragma unroll
    for (int j = 0; j < VC; ++j) unpack(p.v[j], f + j);
#pragma unroll
    for (int i = 0; i < NP; ++i) d[i] = f2(f[2 * i], f[2 * i + 1]);
  }
  // rounded once and written past the caches (nothing here reads it again)
  __device__ void put(T* row, int k, const uint64_t (&d)[NP]) const {
    float f[CE];
#pragma unroll
    for (int i = 0; i < NP; ++i) uf2(d[i], f[2 * i], f[2 * i + 1]);
#pragma unroll
    for (int j = 0; j < VC; ++j) {
      R pk;
      pack(f + j, pk);
      if (pl.on(VC * k + j)) __stcs(reinterpret_cast<R*>(row) + pl.first + 32 * (VC * k + j), pk);
    }
  }
  // column of element i (existing chunks only)
  __device__ int col(int k, int i) const {
    return VEC == 1 ? pl.first + 32 * (2 * k + i) : (pl.first + 32 * k) * VEC + i;
  }
  __device__ bool on(int k, int i) const { return pl.on(VEC == 1 ? 2 * k + i : k); }
  // gain or bias of chunk k (null: `none`), `add` added
  __device__ void affine(const float* p, float none, float add, int k, uint64_t (&d)[NP]) const {
    float f[CE];
    if (!p) {
#pragma unroll
      for (int i = 0; i < CE; ++i) f[i] = none;
    } else if constexpr (VEC % 4 == 0) {
#pragma unroll
      for (int i = 0; i < CE; i += 4) {
        const float4 q = __ldg(reinterpret_cast<const float4*>(p + pl.at(k) * VEC + i));
        f[i] = q.x;
        f[i + 1] = q.y;
        f[i + 2] = q.z;
        f[i + 3] = q.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < CE; ++i) f[i] = __ldg(p + (VEC == 1 ? pl.at(2 * k + i) : pl.at(k) * VEC + i));
    }
    if (!p) add = 0.f;
#pragma unroll
    for (int i = 0; i < NP; ++i) d[i] = add2(f2(f[2 * i], f[2 * i + 1]), both(add));
  }
};

// Warps of a backward block: 96 registers a thread with wide vectors (20 warps;
// 15 of 32 elements a thread took 275 us where 20 of 16 take 210), 128 with
// narrow ones, which spill below that.
template <int VEC> __host__ __device__ constexpr int bwd_warps() { return VEC >= 4 ? 20 : 16; }

// First byte behind the rings of the teams.
__host__ __device__ constexpr int ring_end(int bytes) { return (bytes + 15) & ~15; }

// RW rows of one group per team.  Block b holds the teams b TEAMS ..; a team's
// rows are rows RW k .. of its group.
template <typename T, int VEC, int EPT, int RW, bool FULL>
__global__ void __launch_bounds__(EPT == 8 ? 1024 : EPT == 16 ? 512 : 256, EPT == 32 ? 2 : 1)
    norm_fwd_kernel(const NormArgs a, const T* x, T* y) {
  using Ch = Chunks<T, VEC, EPT, FULL>;
  constexpr int N = Ch::N, NP = Ch::NP;
  __shared__ float4 red[RW][MAX_WARPS];        // a warp's shift, its residual mean, its M2, its elements
  const Lane L(a.warps);
  const Ch ch{{(L.t >> 5) * (32 * EPT / VEC) + L.lane, a.C / VEC}};
  const unsigned per_group = (unsigned)((a.rows_per_group + RW - 1) / RW);
  unsigned unit = blockIdx.x * L.teams + L.id, g = blockIdx.y;
  if (a.flat) {                      // many short groups: numbered through
    g = unit / per_group;
    unit -= g * per_group;
  }
  if (g >= (unsigned)a.groups || unit >= per_group) return;   // whole teams: the others meet on barriers of their own
  const long long in_group = (long long)unit * RW;
  const float inv_c = a.inv_c;
  const long long r0 = g * a.rows_per_group + in_group;
  bool on[RW];
#pragma unroll
  for (int k = 0; k < RW; ++k) on[k] = in_group + k < a.rows_per_group;
  uint64_t d[RW][N * NP];            // x
  float A[RW], dm[RW], m2[RW];       // mean = A + dm, and M2 about it
  {
    typename Ch::Part raw[RW][N];
#pragma unroll
    for (int k = 0; k < RW; ++k) {
      const T* row = x + (on[k] ? r0 + k : r0) * a.x_stride;
#pragma unroll
      for (int c = 0; c < N; ++c)
        ch.load(row, c, raw[k][c]);
    }
    const float n_w = FULL ? 32.f * EPT : warp_sum(ch.count()), inv_w = FULL ? 1.f / (32 * EPT) : 1.f / n_w;
    // sum of the warp's elements over their number (scaled first: no sum overflows)
    float shift[RW], s[RW];
#pragma unroll
    for (int k = 0; k < RW; ++k) {
      uint64_t s2[2] = {0ull, 0ull};
      const uint64_t I = both(inv_w);
#pragma unroll
      for (int c = 0; c < N; ++c) {
        uint64_t p[NP];
        ch.pairs(raw[k][c], p);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          d[k][c * NP + i] = p[i] & ch.mask(c);
          s2[i & 1] = fma2(d[k][c * NP + i], I, s2[i & 1]);
        }
      }
      shift[k] = sum2(add2(s2[0], s2[1]));
    }
#pragma unroll
    for (int k = 0; k < RW; ++k) shift[k] = warp_sum(shift[k]);
#pragma unroll
    for (int k = 0; k < RW; ++k) {
      uint64_t s2[2] = {0ull, 0ull}, q2[2] = {0ull, 0ull};
      const uint64_t S = both(shift[k]);
#pragma unroll
      for (int c = 0; c < N; ++c) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const uint64_t e = sub2(d[k][c * NP + i], S) & ch.mask(c);
          s2[i & 1] = add2(s2[i & 1], e);
          q2[i & 1] = fma2(e, e, q2[i & 1]);
        }
      }
      s[k] = sum2(add2(s2[0], s2[1]));
      m2[k] = sum2(add2(q2[0], q2[1]));
    }
#pragma unroll
    for (int k = 0; k < RW; ++k) {
      s[k] = warp_sum(s[k]) * inv_w;             // what the shift's rounding left of the warp's mean
      m2[k] = warp_sum(m2[k]);
      m2[k] = fmaf(-n_w * s[k], s[k], m2[k]);
    }
    if (L.warps > 1) {
      if (L.lane == 0) {
#pragma unroll
        for (int k = 0; k < RW; ++k) red[k][L.warp] = make_float4(shift[k], s[k], m2[k], n_w);
      }
      team_sync(L.warps, L.id);
      const float4(*rd)[MAX_WARPS] = red;
#pragma unroll
      for (int k = 0; k < RW; ++k) A[k] = dm[k] = m2[k] = 0.f;
      for (int i = L.id * L.warps; i < (L.id + 1) * L.warps; ++i)
#pragma unroll
        for (int k = 0; k < RW; ++k) A[k] = fmaf(rd[k][i].w * inv_c, rd[k][i].x, A[k]);
      for (int i = L.id * L.warps; i < (L.id + 1) * L.warps; ++i)
#pragma unroll
        for (int k = 0; k < RW; ++k) {
          const float4 w = rd[k][i];
          const float e = (w.x - A[k]) + w.y;    // the warp's mean from A
          dm[k] = fmaf(w.w * inv_c, e, dm[k]);
          m2[k] += fmaf(w.w * e, e, w.z);
        }
#pragma unroll
      for (int k = 0; k < RW; ++k) m2[k] = fmaf(-(float)a.C * dm[k], dm[k], m2[k]);
    } else {
#pragma unroll
      for (int k = 0; k < RW; ++k) {
        A[k] = shift[k];
        dm[k] = s[k];
      }
    }
  }
  uint64_t RS[RW], MA[RW], MR[RW];
#pragma unroll
  for (int k = 0; k < RW; ++k) {
    const float var = m2[k] < 0.f ? 0.f : m2[k] * inv_c;       // (NaN stays)
    const float rstd = rsqrt_near(var + a.eps);
    RS[k] = both(rstd);
    MA[k] = both(A[k]);
    MR[k] = both(sizeof(T) == 4 ? -dm[k] : -dm[k] * rstd);
    if (L.t == 0 && on[k]) {
      if (a.mean_out) a.mean_out[r0 + k] = dm[k] == dm[k] ? A[k] + dm[k] : A[k];   // an infinity is the mean's own
      if (a.rstd_out) a.rstd_out[r0 + k] = rstd;
    }
  }
  const float *gw = a.w ? a.w + (long long)g * a.C : nullptr, *gb = a.b ? a.b + (long long)g * a.C : nullptr;
#pragma unroll
  for (int c = 0; c < N; ++c) {
    uint64_t w[NP], b[NP], o[NP];
    ch.affine(gw, 1.f, a.gain_one, c, w);
    ch.affine(gb, 0.f, 0.f, c, b);
#pragma unroll
    for (int k = 0; k < RW; ++k) {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const uint64_t e = sub2(d[k][c * NP + i], MA[k]);
        // fp32: the difference rounded at its own size; a bf16 output does not need the operation
        const uint64_t xh = sizeof(T) == 4 ? mul2(add2(e, MR[k]), RS[k]) : fma2(e, RS[k], MR[k]);
        o[i] = fma2(xh, w[i], b[i]);
      }
      if (on[k]) ch.put(y + (r0 + k) * a.y_stride, c, o);
    }
  }
}

// dx of the block's rows and the block's column sums per group.  The second
// pass over a row reads the ring again: the sums take the registers.  There
// dx = rstd gy + (x - mean) A + B with A = -rstd^2 c2, B = -rstd c1 (c1, c2
// the two row means).  The mean is taken off before anything is scaled: with
// mean rstd in a product of its own, its rounding, 2^-24 |mean| rstd, stays in
// every xhat.
template <typename T, int VEC, int EPT, bool FULL>
__global__ void __launch_bounds__(32 * bwd_warps<VEC>(), 1)
    norm_bwd_kernel(const NormArgs a, const T* x, const T* dy, T* dx) {
  using Rg = Ring<T, VEC, EPT, FULL>;
  using Ch = Chunks<T, VEC, EPT, FULL>;
  constexpr int N = Ch::N, NP = Ch::NP, CE = Ch::CE, STAGES = Rg::STAGES;
  extern __shared__ __align__(16) unsigned char ring_smem[];
  __shared__ float2 red[2][MAX_WARPS];
  const Lane L(a.warps);
  const int team = L.team, t = L.t;
  const Place<FULL> pl{(t >> 5) * (32 * EPT / VEC) + L.lane, a.C / VEC};
  unsigned char* base = ring_smem + L.id * 2 * STAGES * Rg::bytes(L.team);
  const Rg rx{base, pl, team, t, a.C}, ry{base + STAGES * Rg::bytes(L.team), pl, team, t, a.C};
  const Ch ch{pl};
  // sums of the teams: [teams][C]
  float* sw = reinterpret_cast<float*>(ring_smem + ring_end(L.teams * 2 * STAGES * Rg::bytes(L.team)));
  const float inv_c = 1.f / (float)a.C;
  const Range rg = block_rows(a);
  const bool sums = a.partial != nullptr;
  const long long first = rg.r0 + L.id;
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) {
    if (first + s * L.teams < rg.r1) {
      rx.fetch(s, x + (first + s * L.teams) * a.x_stride);
      ry.fetch(s, dy + (first + s * L.teams) * a.y_stride);
    }
    copy_commit();
  }
  float next_mean = 0.f, next_rstd = 0.f;
  if (first < rg.r1) {
    next_mean = a.mean[first];
    next_rstd = a.rstd[first];
  }
  int st = 0, par = 0;
  long long r = first;
  for (long long s0 = rg.r0; s0 < rg.r1;) {       // the block's rows of one group
    const long long g = s0 / a.rows_per_group;
    long long s1 = (g + 1) * a.rows_per_group;
    if (s1 > rg.r1) s1 = rg.r1;
    uint64_t w[N][NP], aw[N * NP], ab[N * NP];
#pragma unroll
    for (int k = 0; k < N; ++k)
      ch.affine(a.w ? a.w + g * a.C : nullptr, 1.f, a.gain_one, k, w[k]);
#pragma unroll
    for (int i = 0; i < N * NP; ++i) aw[i] = ab[i] = 0ull;
    for (; r < s1; r += L.teams) {
      const T *xr = x + r * a.x_stride, *yr = dy + r * a.y_stride;
      if constexpr (Rg::WORDS) {
        copy_wait<STAGES - 2>();
        team_sync(L.warps, L.id);    // the rows are whole, and the stage fetched below is read by nobody
      }
      const long long ahead = r + (long long)(STAGES - 1) * L.teams;
      if (ahead < rg.r1) {
        const int sn = st == 0 ? STAGES - 1 : st - 1;
        rx.fetch(sn, x + ahead * a.x_stride);
        ry.fetch(sn, dy + ahead * a.y_stride);
      }
      copy_commit();
      const float mean = next_mean, rstd = next_rstd;
      if (r + L.teams < rg.r1) {
        next_mean = a.mean[r + L.teams];
        next_rstd = a.rstd[r + L.teams];
      }
      if constexpr (!Rg::WORDS) copy_wait<STAGES - 1>();
      uint64_t C1 = 0ull, C2 = 0ull;
      const uint64_t RS = both(rstd), MN = both(mean);
#pragma unroll
      for (int k = 0; k < N; ++k) {
          uint64_t xv[NP], gv[NP];
          ch.get(rx, st, k, xr, xv);
          ch.get(ry, st, k, yr, gv);
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            gv[i] &= ch.mask(k);                    // an absent element adds nothing
            const uint64_t xh = mul2(sub2(xv[i], MN), RS);
            aw[k * NP + i] = fma2(gv[i], xh, aw[k * NP + i]);
            ab[k * NP + i] = add2(ab[k * NP + i], gv[i]);
            const uint64_t gy = mul2(gv[i], w[k][i]);
            C1 = add2(C1, gy);
            C2 = fma2(gy, xh, C2);
          }
        }
      if (dx) {
        float c1 = warp_sum(sum2(C1)), c2 = warp_sum(sum2(C2));
        if (L.warps > 1) {
          if (L.lane == 0) red[par][L.warp] = make_float2(c1, c2);
          team_sync(L.warps, L.id);
          const float2 p = L.lane < L.warps ? red[par][L.id * L.warps + L.lane] : make_float2(0.f, 0.f);
          c1 = warp_sum(p.x);
          c2 = warp_sum(p.y);
          par ^= 1;
        }
        const uint64_t KA = both(-rstd * rstd * (c2 * inv_c)), KB = both(-rstd * (c1 * inv_c));
        T* dr = dx + r * a.x_stride;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            uint64_t xv[NP], gv[NP];
            ch.get(rx, st, k, xr, xv);
            ch.get(ry, st, k, yr, gv);
#pragma unroll
            for (int i = 0; i < NP; ++i) xv[i] = fma2(mul2(gv[i], w[k][i]), RS, fma2(sub2(xv[i], MN), KA, KB));
            ch.put(dr, k, xv);
          }
      }
      st = st == STAGES - 1 ? 0 : st + 1;
    }
    if (sums) {
      float* out = a.partial + ((long long)blockIdx.x + g) * 2 * a.C;
#pragma unroll
      for (int h = 0; h < 2; ++h, out += a.C) {
        if (L.teams > 1 && (h == 1 || s0 > rg.r0)) __syncthreads();      // the sums before are read
#pragma unroll
        for (int k = 0; k < N; ++k) {
          float f[CE];
#pragma unroll
          for (int i = 0; i < NP; ++i) uf2(h ? ab[k * NP + i] : aw[k * NP + i], f[2 * i], f[2 * i + 1]);
#pragma unroll
          for (int i = 0; i < CE; ++i)
            if (ch.on(k, i)) {
              if (L.teams > 1)
                sw[L.id * a.C + ch.col(k, i)] = f[i];
              else
                out[ch.col(k, i)] = f[i];
            }
        }
        if (L.teams > 1) {           // over the teams, in order
          __syncthreads();
          for (int c = threadIdx.x; c < a.C; c += blockDim.x) {
            float v = sw[c];
            for (int id = 1; id < L.teams; ++id) v += sw[id * a.C + c];
            out[c] = v;
          }
        }
      }
    }
    s0 = s1;
  }
}

// dw and dbias of group blockIdx.y: the partial slots of the blocks whose
// rows meet the group, in ascending order.  32 columns a block; warp k of W
// adds the slots k, k + W, ... and the W sums are added in warp order.  W is 8
// where a group has few slots and 32 where it has many, which eight warps
// would wait for one batch of loads after another (4,099 x 1,001 fp32, 148
// slots: the whole backward 25.6 us with 8, 23.9 with 32).
template <int W>
__global__ void __launch_bounds__(32 * W) norm_reduce_kernel(const NormArgs a, float* dw, float* db) {
  __shared__ float sm[2][W][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  for (long long g = blockIdx.y; g < a.groups; g += gridDim.y) {
    const long long c0 = g * a.rows_per_group / a.rows_per_block;
    const long long c1 = ((g + 1) * a.rows_per_group - 1) / a.rows_per_block;
    float sw = 0.f, sb = 0.f;
    if (col < a.C) {
#pragma unroll 4
      for (long long c = c0 + warp; c <= c1; c += W) {
        const float* p = a.partial + (c + g) * 2 * a.C + col;
        sw += p[0];
        sb += p[a.C];
      }
    }
    sm[0][warp][lane] = sw;
    sm[1][warp][lane] = sb;
    __syncthreads();
    if (warp < 2 && col < a.C) {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < W; ++k) s += sm[warp][k][lane];
      float* dst = warp == 0 ? dw : db;
      if (dst) dst[g * a.C + col] = s;
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------- wide rows
// Sums of two values over the block.
__device__ inline void block_sum2(float& a, float& b, float (*red)[32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  a = warp_sum(a);
  b = warp_sum(b);
  __syncthreads();
  if (lane == 0) {
    red[0][warp] = a;
    red[1][warp] = b;
  }
  __syncthreads();
  a = b = 0.f;
  for (int i = 0; i < WIDE / 32; ++i) {
    a += red[0][i];
    b += red[1][i];
  }
}
__device__ inline void from_f(float v, float* p) { *p = v; }
__device__ inline void from_f(float v, __nv_bfloat16* p) { *p = __float2bfloat16(v); }

template <typename T>
__global__ void __launch_bounds__(WIDE) norm_fwd_wide_kernel(const NormArgs a, const T* x, T* y) {   // y may be x
  __shared__ float red[2][32];
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* xr = x + r * a.x_stride;
    const long long g = r / a.rows_per_group;
    float s = 0.f, s1 = 0.f, s2 = 0.f;
    for (int c = threadIdx.x; c < a.C; c += WIDE) s += to_f(xr[c]);
    block_sum2(s, s1, red);
    const float m0 = s / (float)a.C;
    s1 = 0.f;
    for (int c = threadIdx.x; c < a.C; c += WIDE) {
      const float e = to_f(xr[c]) - m0;
      s1 += e;
      s2 = fmaf(e, e, s2);
    }
    block_sum2(s1, s2, red);
    const float dm = s1 / (float)a.C;
    const float var = fmaxf(s2 / (float)a.C - dm * dm, 0.f) + (s2 != s2 ? s2 : 0.f);
    const float rstd = 1.f / sqrtf(var + a.eps);
    for (int c = threadIdx.x; c < a.C; c += WIDE) {
      const float w = a.w ? a.w[g * a.C + c] + a.gain_one : 1.f;
      const float b = a.b ? a.b[g * a.C + c] : 0.f;
      from_f(fmaf((to_f(xr[c]) - m0 - dm) * rstd, w, b), y + r * a.y_stride + c);
    }
    if (threadIdx.x == 0) {
      if (a.mean_out) a.mean_out[r] = m0 + dm;
      if (a.rstd_out) a.rstd_out[r] = rstd;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(WIDE)
    norm_bwd_wide_kernel(const NormArgs a, const T* x, const T* dy, T* dx) {   // dx may be x or dy
  __shared__ float red[2][32];
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const T* xr = x + r * a.x_stride;
    const T* gr = dy + r * a.y_stride;
    const long long g = r / a.rows_per_group;
    const float mean = a.mean[r], rstd = a.rstd[r];
    float c1 = 0.f, c2 = 0.f;
    for (int c = threadIdx.x; c < a.C; c += WIDE) {
      const float gy = to_f(gr[c]) * (a.w ? a.w[g * a.C + c] + a.gain_one : 1.f);
      c1 += gy;
      c2 = fmaf(gy, (to_f(xr[c]) - mean) * rstd, c2);
    }
    block_sum2(c1, c2, red);
    c1 /= (float)a.C;
    c2 /= (float)a.C;
    for (int c = threadIdx.x; c < a.C; c += WIDE) {
      const float gy = to_f(gr[c]) * (a.w ? a.w[g * a.C + c] + a.gain_one : 1.f);
      const float xh = (to_f(xr[c]) - mean) * rstd;
      from_f(rstd * (gy - fmaf(xh, c2, c1)), dx + r * a.x_stride + c);
    }
  }
}

// Column sums of one row range (blockIdx.y) and 256 columns (blockIdx.x).
template <typename T>
__global__ void __launch_bounds__(256)
    norm_cols_wide_kernel(const NormArgs a, const T* __restrict__ x, const T* __restrict__ dy) {
  const int col = blockIdx.x * 256 + threadIdx.x;
  const long long r0 = (long long)blockIdx.y * a.rows_per_block;
  const long long r1 = r0 + a.rows_per_block < a.rows ? r0 + a.rows_per_block : a.rows;
  if (col >= a.C) return;
  for (long long s0 = r0; s0 < r1;) {
    const long long g = s0 / a.rows_per_group;
    long long s1 = (g + 1) * a.rows_per_group;
    if (s1 > r1) s1 = r1;
    float sw = 0.f, sb = 0.f;
#pragma unroll 4
    for (long long r = s0; r < s1; ++r) {
      const float d = to_f(dy[r * a.y_stride + col]);
      sw = fmaf(d, (to_f(x[r * a.x_stride + col]) - a.mean[r]) * a.rstd[r], sw);
      sb += d;
    }
    float* out = a.partial + ((long long)blockIdx.y + g) * 2 * a.C + col;
    out[0] = sw;
    out[a.C] = sb;
    s0 = s1;
  }
}

// Largest vector (elements) that divides the row and both row strides; gain
// and bias, read four at a time with vectors of four or more, have to be
// 16-byte aligned for those (their pointers need only be a float's).
template <typename T>
int vec_of(const NormArgs& a) {
  const bool quads = ((reinterpret_cast<uintptr_t>(a.w) | reinterpret_cast<uintptr_t>(a.b)) & 15) == 0;
  const int opts_b[4] = {8, 4, 2, 1}, opts_f[4] = {4, 1, 1, 1};
  for (int i = 0; i < 4; ++i) {
    const int v = sizeof(T) == 2 ? opts_b[i] : opts_f[i];
    if (a.C % v == 0 && a.x_stride % v == 0 && a.y_stride % v == 0 && (quads || v < 4)) return v;
  }
  return 1;
}

// 8 elements a thread when the SMs hold all rows at once like that.
inline bool few_rows(long long rows, int C, int num_sms) { return rows * ((C + 255) / 256) <= (long long)num_sms * 32; }

template <typename T, int VEC, int EPT, int RW>
cudaError_t fwd_v(NormArgs a, const T* x, T* y, cudaStream_t s) {
  a.warps = (a.C + 32 * EPT - 1) / (32 * EPT);
  auto kernel = a.C == 32 * EPT * a.warps ? norm_fwd_kernel<T, VEC, EPT, RW, true> : norm_fwd_kernel<T, VEC, EPT, RW, false>;
  const int teams = a.warps < 4 ? 4 / a.warps : 1;       // blocks of three warps or more
  const long long per_group = (a.rows_per_group + RW - 1) / RW;
  a.flat = a.groups > 65535 || per_group < 8 * teams;
  const long long units = a.flat ? per_group * a.groups : per_group;
  const dim3 grid((unsigned)((units + teams - 1) / teams), a.flat ? 1 : a.groups);
  kernel<<<grid, teams * 32 * a.warps, 0, s>>>(a, x, y);
  return cudaGetLastError();
}

// Elements a thread of the long forms: narrow vectors cost an address each,
// and 32 of them spill.
template <int VEC> constexpr int long_ept() { return VEC >= 4 ? 32 : 16; }

template <typename T, int VEC>
cudaError_t fwd_e(const NormArgs& a, const T* x, T* y, int num_sms, cudaStream_t s) {
  return few_rows(a.rows, a.C, num_sms) ? fwd_v<T, VEC, 8, 1>(a, x, y, s) : fwd_v<T, VEC, long_ept<VEC>(), 2>(a, x, y, s);
}

template <typename T>
cudaError_t fwd_t(const NormArgs& a, const void* x, void* y, int num_sms, cudaStream_t s) {
  const T* xp = static_cast<const T*>(x);
  T* yp = static_cast<T*>(y);
  if (a.C > MAX_C) {
    const long long blocks = a.rows < 2ll * num_sms ? a.rows : 2ll * num_sms;
    norm_fwd_wide_kernel<T><<<(unsigned)blocks, WIDE, 0, s>>>(a, xp, yp);
    return cudaGetLastError();
  }
  const int v = vec_of<T>(a);
  if constexpr (sizeof(T) == 2) {
    if (v >= 4) return fwd_e<T, 4>(a, xp, yp, num_sms, s);
    if (v == 2) return fwd_e<T, 2>(a, xp, yp, num_sms, s);
  } else {
    if (v == 4) return fwd_e<T, 4>(a, xp, yp, num_sms, s);
  }
  return fwd_e<T, 1>(a, xp, yp, num_sms, s);
}

template <typename T, int VEC>
cudaError_t bwd_v(NormArgs a, const T* x, const T* dy, T* dx, cudaStream_t s) {
  constexpr int EPT = 16, WARPS = bwd_warps<VEC>();
  using Rg = Ring<T, VEC, EPT, true>;
  a.warps = (a.C + 32 * EPT - 1) / (32 * EPT);
  auto kernel = a.C == 32 * EPT * a.warps ? norm_bwd_kernel<T, VEC, EPT, true> : norm_bwd_kernel<T, VEC, EPT, false>;
  // as many teams as the warps allow, as many as the shared memory takes, one block an SM
  int teams = WARPS / a.warps < MAX_TEAMS ? WARPS / a.warps : MAX_TEAMS;
  auto bytes = [&](int n) { return ring_end(n * 2 * Rg::STAGES * Rg::bytes(32 * a.warps)) + (n > 1 ? 4 * a.C * n : 0); };
  while (teams > 1 && bytes(teams) > 220 * 1024) --teams;
  const int smem = bytes(teams);
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const long long blocks = (a.rows + a.rows_per_block - 1) / a.rows_per_block;
  kernel<<<(unsigned)blocks, teams * 32 * a.warps, smem, s>>>(a, x, dy, dx);
  return cudaGetLastError();
}

template <typename T>
cudaError_t bwd_t(const NormArgs& a, const void* x, const void* dy, void* dx, int num_sms, cudaStream_t s) {
  const T* xp = static_cast<const T*>(x);
  const T* gp = static_cast<const T*>(dy);
  T* dp = static_cast<T*>(dx);
  if (a.C > MAX_C) {
    if (a.partial) {
      const dim3 grid((a.C + 255) / 256, (unsigned)((a.rows + a.rows_per_block - 1) / a.rows_per_block));
      norm_cols_wide_kernel<T><<<grid, 256, 0, s>>>(a, xp, gp);   // before dx, which may be x or dy
      const cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return e;
    }
    if (dp) {
      const long long blocks = a.rows < 2ll * num_sms ? a.rows : 2ll * num_sms;
      norm_bwd_wide_kernel<T><<<(unsigned)blocks, WIDE, 0, s>>>(a, xp, gp, dp);
    }
    return cudaGetLastError();
  }
  const int v = vec_of<T>(a);
  if constexpr (sizeof(T) == 2) {
    if (v == 8) return bwd_v<T, 8>(a, xp, gp, dp, s);
    if (v == 4) return bwd_v<T, 4>(a, xp, gp, dp, s);
    if (v == 2) return bwd_v<T, 2>(a, xp, gp, dp, s);
  } else {
    if (v == 4) return bwd_v<T, 4>(a, xp, gp, dp, s);
  }
  return bwd_v<T, 1>(a, xp, gp, dp, s);
}

}  // namespace ln

long long norm_bwd_blocks(long long rows) { return rows < kNormBlocks ? rows : kNormBlocks; }

cudaError_t launch_norm_fwd(const NormArgs& a, int dtype, const void* x, void* y, int num_sms, cudaStream_t s) {
  return dtype == FVATTN_BF16 ? ln::fwd_t<__nv_bfloat16>(a, x, y, num_sms, s) : ln::fwd_t<float>(a, x, y, num_sms, s);
}

cudaError_t launch_norm_bwd(const NormArgs& a, int dtype, const void* x, const void* dy, void* dx, float* dw, float* db,
                            int num_sms, cudaStream_t s) {
  cudaError_t e = dtype == FVATTN_BF16 ? ln::bwd_t<__nv_bfloat16>(a, x, dy, dx, num_sms, s)
                                       : ln::bwd_t<float>(a, x, dy, dx, num_sms, s);
  if (e != cudaSuccess || !a.partial) return e;
  const dim3 grid((a.C + 31) / 32, (unsigned)(a.groups < 65535 ? a.groups : 65535));
  if (a.rows_per_group > 32 * a.rows_per_block)
    ln::norm_reduce_kernel<32><<<grid, 1024, 0, s>>>(a, dw, db);
  else
    ln::norm_reduce_kernel<8><<<grid, 256, 0, s>>>(a, dw, db);
  return cudaGetLastError();
}

}  // namespace fvattn
