// Shared by the forward and the backward of the sliding-window attention:
// the visibility rule and tile helpers.
#pragma once

#include "packed.cuh"

namespace fvattn {
namespace win {

using namespace pk;

// Lengths of one sequence; a length outside [0, the tensor's] is cut to it.
struct Seq {
  int ql, kvl;
};
__device__ inline Seq seq_of(const WinGeom& g, int b) {
  Seq s{g.Nq, g.Nk};
  if (g.q_lens) {
    const int n = g.q_lens[b];
    s.ql = n < 0 ? 0 : n < g.Nq ? n : g.Nq;
  }
  if (g.kv_lens) {
    const int n = g.kv_lens[b];
    s.kvl = n < 0 ? 0 : n < g.Nk ? n : g.Nk;
  }
  return s;
}

// Keys that query i sees: [lo, hi) and, below lo, [0, sk).  A query in front
// of the first key (more queries than keys) sees none.
struct Span {
  int lo, hi, sk;
};
__device__ inline Span span_of(const WinGeom& g, const Seq& s, int i) {
  const int p = i + s.kvl - s.ql;
  if (p < 0) return {0, 0, 0};
  const int u = g.unit == 1 ? p : p / g.unit;
  const long long end = ((long long)u + 1) * g.unit;
  const int hi = end < s.kvl ? (int)end : s.kvl;
  const int u0 = g.window > 0 && u >= g.window ? u - g.window + 1 : 0;
  const long long sk = (long long)g.sinks * g.unit;
  return {u0 * g.unit, hi, sk < hi ? (int)sk : hi};
}

// The value of lane 0, which the compiler then knows to be the same in every
// lane: operands of the matrix instructions stay in uniform registers.
__device__ inline uint32_t uni(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

// Bits a .. b - 1 of a 32-bit word (a and b may lie outside it).
__device__ inline uint32_t bits(int a, int b) {
  a = a < 0 ? 0 : a;
  b = b > 32 ? 32 : b;
  if (a >= b) return 0u;
  return (0xFFFFFFFFu >> (32 - (b - a))) << a;
}

__device__ inline void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ inline void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// Rows r0 .. r1 - 1 of a staged tile set to zero by a converged warp.  The
// tile is D / 64 parts of `part` bytes, 128 bytes a row (a 128-byte swizzled
// row keeps its 128 bytes).  Ends with the fence that lets the MMAs see it.
__device__ inline void zero_rows(uint8_t* tile, uint32_t part, int parts, int r0, int r1) {
  const int lane = threadIdx.x & 31;
  for (int h = 0; h < parts; ++h)
    for (int i = r0 * 8 + lane; i < r1 * 8; i += 32)
      *reinterpret_cast<uint4*>(tile + h * part + i * 16) = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  __syncwarp();
}

}  // namespace win
}  // namespace fvattn
