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
// A row is held in the registers of a team of up to 16 warps, 16 elements a
// thread, so the variance is a second pass over registers and not over
// memory, and a thread keeps the same columns for all its rows: gain, bias
// and the backward's column sums stay in registers too.  Blocks walk
// contiguous row ranges of equal length (persistent grid) and load the next
// row before they reduce the current one.  The column sums of block c over
// its rows of group g go to partial slot c + g: the ranges and the groups
// are both ascending, so every (c, g) pair that meets has a slot of its own,
// and a second kernel adds a group's slots in ascending order (no atomics,
// the same bits every run).  Rows wider than 16 warps hold (8192 elements)
// take the wide kernels, which pass over the row again from L2.
#include "fvattn_internal.cuh"

namespace fvattn {
namespace ln {

constexpr int EPT = 16;          // elements of a row per thread
constexpr int MAX_WARPS = 16;    // warps of a team
constexpr int MAX_C = EPT * 32 * MAX_WARPS;
constexpr int TEAMS1 = 8;        // one-warp teams per block
constexpr int WIDE = 1024;       // threads of a wide row's block

// VEC consecutive elements as loaded.
template <typename T, int VEC> struct Raw;
template <> struct Raw<float, 4> { using type = float4; };
template <> struct Raw<float, 1> { using type = float; };
template <> struct Raw<__nv_bfloat16, 8> { using type = uint4; };
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
__device__ inline void pack(const float* v, uint32_t& r) { r = pack2(v[0], v[1]); }
__device__ inline void pack(const float* v, unsigned short& r) { r = (unsigned short)(pack2(v[0], 0.f) & 0xFFFFu); }

__device__ inline float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sums of a and b over the team; red is the team's [2][MAX_WARPS] buffer,
// free again after the block's next barrier.
__device__ inline void team_sum2(float& a, float& b, float (*red)[MAX_WARPS], int warps, int warp, int lane) {
  a = warp_sum(a);
  b = warp_sum(b);
  if (warps == 1) return;
  if (lane == 0) {
    red[0][warp] = a;
    red[1][warp] = b;
  }
  __syncthreads();
  a = b = 0.f;
  for (int i = 0; i < warps; ++i) {
    a += red[0][i];
    b += red[1][i];
  }
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

// A thread's vectors of one row: vector v of thread t is number v * team + t.
template <typename T, int VEC>
__device__ inline void load_row(const T* p, int nvec, int t, int team, typename Raw<T, VEC>::type (&x)[EPT / VEC]) {
  using R = typename Raw<T, VEC>::type;
#pragma unroll
  for (int v = 0; v < EPT / VEC; ++v)
    if (v * team + t < nvec) x[v] = __ldcs(reinterpret_cast<const R*>(p) + v * team + t);
}

// The thread's columns of gain (or 1 + w) and bias of group g.
template <int VEC>
__device__ inline void load_affine(const float* p, float none, float add, long long g, int C, int nvec, int t, int team,
                                   float (&w)[EPT]) {
#pragma unroll
  for (int v = 0; v < EPT / VEC; ++v)
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      w[v * VEC + i] = p && v * team + t < nvec ? p[g * C + (v * team + t) * VEC + i] + add : none;
}

template <typename T, int VEC>
__global__ void __launch_bounds__(32 * MAX_WARPS)
    norm_fwd_kernel(const NormArgs a, const T* __restrict__ x, T* __restrict__ y) {
  using R = typename Raw<T, VEC>::type;
  constexpr int NV = EPT / VEC;
  __shared__ float red[2][2][MAX_WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int warps = a.warps, team = warps * 32, teams = (int)blockDim.x / team;
  const int t = warps == 1 ? lane : (int)threadIdx.x;
  const int nvec = a.C / VEC;
  const float inv_c = 1.f / (float)a.C;
  const Range rg = block_rows(a);
  long long r = rg.r0 + (teams > 1 ? warp : 0);
  long long cur_g = -1;
  float w[EPT], b[EPT];
  R nx[NV];
  if (r < rg.r1) load_row<T, VEC>(x + r * a.x_stride, nvec, t, team, nx);
  for (; r < rg.r1; r += teams) {
    float d[EPT];
    float s = 0.f, s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (v * team + t < nvec) {
        unpack(nx[v], d + v * VEC);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) d[v * VEC + i] = 0.f;
      }
    }
    if (r + teams < rg.r1) load_row<T, VEC>(x + (r + teams) * a.x_stride, nvec, t, team, nx);
    const long long g = r / a.rows_per_group;
    if (g != cur_g) {
      load_affine<VEC>(a.w, 1.f, a.gain_one, g, a.C, nvec, t, team, w);
      load_affine<VEC>(a.b, 0.f, 0.f, g, a.C, nvec, t, team, b);
      cur_g = g;
    }
#pragma unroll
    for (int i = 0; i < EPT; ++i) s += d[i];
    team_sum2(s, s1, red[0], warps, warp, lane);
    const float m0 = s * inv_c;
    s1 = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (v * team + t < nvec) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float e = d[v * VEC + i] - m0;
          d[v * VEC + i] = e;
          s1 += e;
          s2 = fmaf(e, e, s2);
        }
      }
    team_sum2(s1, s2, red[1], warps, warp, lane);
    // the rounding of the first mean, put right by the mean of the differences
    const float dm = s1 * inv_c;
    const float var = fmaxf(s2 * inv_c - dm * dm, 0.f) + (s2 != s2 ? s2 : 0.f);
    const float rstd = 1.f / sqrtf(var + a.eps);
    T* yr = y + r * a.y_stride;
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (v * team + t < nvec) {
        float o[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) o[i] = fmaf((d[v * VEC + i] - dm) * rstd, w[v * VEC + i], b[v * VEC + i]);
        R pk;
        pack(o, pk);
        __stcs(reinterpret_cast<R*>(yr) + v * team + t, pk);
      }
    if (t == 0) {
      if (a.mean_out) a.mean_out[r] = m0 + dm;
      if (a.rstd_out) a.rstd_out[r] = rstd;
    }
  }
}

// dx of the block's rows and the block's column sums per group.  With
// one-warp teams the block's warps interleave their rows and add their sums
// in shared memory, in warp order, when a group ends.
template <typename T, int VEC>
__global__ void __launch_bounds__(32 * MAX_WARPS)
    norm_bwd_kernel(const NormArgs a, const T* __restrict__ x, const T* __restrict__ dy, T* __restrict__ dx) {
  using R = typename Raw<T, VEC>::type;
  constexpr int NV = EPT / VEC;
  __shared__ float red[2][2][MAX_WARPS];
  __shared__ float comb[EPT * 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int warps = a.warps, team = warps * 32, teams = (int)blockDim.x / team;
  const int t = warps == 1 ? lane : (int)threadIdx.x;
  const int nvec = a.C / VEC;
  const float inv_c = 1.f / (float)a.C;
  const Range rg = block_rows(a);
  const bool sums = a.partial != nullptr;
  int par = 0;
  for (long long s0 = rg.r0; s0 < rg.r1;) {       // the block's rows of one group
    const long long g = s0 / a.rows_per_group;
    long long s1 = (g + 1) * a.rows_per_group;
    if (s1 > rg.r1) s1 = rg.r1;
    float w[EPT], aw[EPT], ab[EPT];
    load_affine<VEC>(a.w, 1.f, a.gain_one, g, a.C, nvec, t, team, w);
#pragma unroll
    for (int i = 0; i < EPT; ++i) aw[i] = ab[i] = 0.f;
    R nx[NV], ny[NV];
    long long r = s0 + (teams > 1 ? warp : 0);
    float nm = 0.f, nr = 0.f;
    if (r < s1) {
      load_row<T, VEC>(x + r * a.x_stride, nvec, t, team, nx);
      load_row<T, VEC>(dy + r * a.y_stride, nvec, t, team, ny);
      nm = a.mean[r];
      nr = a.rstd[r];
    }
    for (; r < s1; r += teams) {
      const float mean = nm, rstd = nr;
      float xh[EPT], gy[EPT];
      float c1 = 0.f, c2 = 0.f;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        if (v * team + t < nvec) {
          unpack(nx[v], xh + v * VEC);
          unpack(ny[v], gy + v * VEC);
#pragma unroll
          for (int i = v * VEC; i < (v + 1) * VEC; ++i) {
            xh[i] = (xh[i] - mean) * rstd;
            aw[i] = fmaf(gy[i], xh[i], aw[i]);
            ab[i] += gy[i];
            gy[i] *= w[i];
            c1 += gy[i];
            c2 = fmaf(gy[i], xh[i], c2);
          }
        }
      }
      if (r + teams < s1) {
        load_row<T, VEC>(x + (r + teams) * a.x_stride, nvec, t, team, nx);
        load_row<T, VEC>(dy + (r + teams) * a.y_stride, nvec, t, team, ny);
        nm = a.mean[r + teams];
        nr = a.rstd[r + teams];
      }
      if (dx) {
        team_sum2(c1, c2, red[par], warps, warp, lane);
        par ^= 1;
        c1 *= inv_c;
        c2 *= inv_c;
        T* dr = dx + r * a.x_stride;
#pragma unroll
        for (int v = 0; v < NV; ++v)
          if (v * team + t < nvec) {
            float o[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) o[i] = rstd * (gy[v * VEC + i] - fmaf(xh[v * VEC + i], c2, c1));
            R pk;
            pack(o, pk);
            __stcs(reinterpret_cast<R*>(dr) + v * team + t, pk);
          }
      }
    }
    if (sums) {
      float* out = a.partial + ((long long)blockIdx.x + g) * 2 * a.C;
      if (teams > 1) {
        for (int h = 0; h < 2; ++h) {
          for (int k = 0; k < teams; ++k) {
            if (warp == k) {
#pragma unroll
              for (int i = 0; i < EPT; ++i) {
                const float v = h ? ab[i] : aw[i];
                comb[i * 32 + lane] = k == 0 ? v : comb[i * 32 + lane] + v;
              }
            }
            __syncthreads();
          }
          if (warp == 0) {
#pragma unroll
            for (int v = 0; v < NV; ++v)
              if (v * 32 + lane < nvec) {
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                  out[(long long)h * a.C + (v * 32 + lane) * VEC + i] = comb[(v * VEC + i) * 32 + lane];
              }
          }
          __syncthreads();
        }
      } else {
#pragma unroll
        for (int v = 0; v < NV; ++v)
          if (v * team + t < nvec) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              out[(v * team + t) * VEC + i] = aw[v * VEC + i];
              out[(long long)a.C + (v * team + t) * VEC + i] = ab[v * VEC + i];
            }
          }
      }
    }
    s0 = s1;
  }
}

// dw and dbias of group blockIdx.y: the partial slots of the blocks whose
// rows meet the group, in ascending order.  32 columns a block; warp k adds
// the slots k, k + 8, ... and the eight sums are added in warp order.
__global__ void __launch_bounds__(256) norm_reduce_kernel(const NormArgs a, float* dw, float* db) {
  __shared__ float sm[2][8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;
  for (long long g = blockIdx.y; g < a.groups; g += gridDim.y) {
    const long long c0 = g * a.rows_per_group / a.rows_per_block;
    const long long c1 = ((g + 1) * a.rows_per_group - 1) / a.rows_per_block;
    float sw = 0.f, sb = 0.f;
    if (col < a.C) {
#pragma unroll 4
      for (long long c = c0 + warp; c <= c1; c += 8) {
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
      for (int k = 0; k < 8; ++k) s += sm[warp][k][lane];
      float* dst = warp == 0 ? dw : db;
      if (dst) dst[g * a.C + col] = s;
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------- wide rows
// Sums of up to three values over the block.
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
__device__ inline float to_f(float v) { return v; }
__device__ inline float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ inline void from_f(float v, float* p) { *p = v; }
__device__ inline void from_f(float v, __nv_bfloat16* p) { *p = __float2bfloat16(v); }

template <typename T>
__global__ void __launch_bounds__(WIDE) norm_fwd_wide_kernel(const NormArgs a, const T* __restrict__ x, T* __restrict__ y) {
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
    norm_bwd_wide_kernel(const NormArgs a, const T* __restrict__ x, const T* __restrict__ dy, T* __restrict__ dx) {
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

// Largest vector (elements) that divides the row and both row strides.
template <typename T>
int vec_of(const NormArgs& a) {
  const int opts_b[3] = {8, 2, 1}, opts_f[3] = {4, 1, 1};
  for (int i = 0; i < 3; ++i) {
    const int v = sizeof(T) == 2 ? opts_b[i] : opts_f[i];
    if (a.C % v == 0 && a.x_stride % v == 0 && a.y_stride % v == 0) return v;
  }
  return 1;
}

// Warps of a row's team and the block's threads.
inline void team_of(NormArgs& a, int vec, int* threads) {
  const int nvec = a.C / vec;
  const int per = 32 * (EPT / vec);
  a.warps = (nvec + per - 1) / per;
  *threads = a.warps == 1 ? 32 * TEAMS1 : 32 * a.warps;
}

template <typename K>
cudaError_t resident_blocks(K kernel, int threads, int num_sms, long long* blocks) {
  int per_sm = 0;
  const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, 0);
  *blocks = (long long)num_sms * (per_sm < 1 ? 1 : per_sm);
  return e;
}

template <typename T, int VEC>
cudaError_t fwd_v(NormArgs a, const T* x, T* y, int num_sms, cudaStream_t s) {
  int threads;
  team_of(a, VEC, &threads);
  long long blocks;
  cudaError_t e = resident_blocks(norm_fwd_kernel<T, VEC>, threads, num_sms, &blocks);
  if (e != cudaSuccess) return e;
  const long long teams = a.warps == 1 ? TEAMS1 : 1;
  const long long most = (a.rows + teams - 1) / teams;
  if (blocks > most) blocks = most;
  a.rows_per_block = (a.rows + blocks - 1) / blocks;
  blocks = (a.rows + a.rows_per_block - 1) / a.rows_per_block;
  norm_fwd_kernel<T, VEC><<<(unsigned)blocks, threads, 0, s>>>(a, x, y);
  return cudaGetLastError();
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
    if (v == 8) return fwd_v<T, 8>(a, xp, yp, num_sms, s);
    if (v == 2) return fwd_v<T, 2>(a, xp, yp, num_sms, s);
  } else {
    if (v == 4) return fwd_v<T, 4>(a, xp, yp, num_sms, s);
  }
  return fwd_v<T, 1>(a, xp, yp, num_sms, s);
}

template <typename T, int VEC>
cudaError_t bwd_v(NormArgs a, const T* x, const T* dy, T* dx, cudaStream_t s) {
  int threads;
  team_of(a, VEC, &threads);
  const long long blocks = (a.rows + a.rows_per_block - 1) / a.rows_per_block;
  norm_bwd_kernel<T, VEC><<<(unsigned)blocks, threads, 0, s>>>(a, x, dy, dx);
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
    if (v == 2) return bwd_v<T, 2>(a, xp, gp, dp, s);
  } else {
    if (v == 4) return bwd_v<T, 4>(a, xp, gp, dp, s);
  }
  return bwd_v<T, 1>(a, xp, gp, dp, s);
}

}  // namespace ln

long long norm_bwd_blocks(long long rows, int C) {
  const long long teams = C <= ln::EPT * 32 ? ln::TEAMS1 : 1;
  const long long most = (rows + teams - 1) / teams;
  return most < kNormBlocks ? most : kNormBlocks;
}

cudaError_t launch_norm_fwd(const NormArgs& a, int dtype, const void* x, void* y, int num_sms, cudaStream_t s) {
  return dtype == FVATTN_BF16 ? ln::fwd_t<__nv_bfloat16>(a, x, y, num_sms, s) : ln::fwd_t<float>(a, x, y, num_sms, s);
}

cudaError_t launch_norm_bwd(const NormArgs& a, int dtype, const void* x, const void* dy, void* dx, float* dw, float* db,
                            int num_sms, cudaStream_t s) {
  cudaError_t e = dtype == FVATTN_BF16 ? ln::bwd_t<__nv_bfloat16>(a, x, dy, dx, num_sms, s)
                                       : ln::bwd_t<float>(a, x, dy, dx, num_sms, s);
  if (e != cudaSuccess || !a.partial) return e;
  const dim3 grid((a.C + 31) / 32, (unsigned)(a.groups < 65535 ? a.groups : 65535));
  ln::norm_reduce_kernel<<<grid, 256, 0, s>>>(a, dw, db);
  return cudaGetLastError();
}

}  // namespace fvattn
