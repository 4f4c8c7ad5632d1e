// Warp-level pieces of the chunked gated delta rule: mma.sync fragments of
// bf16 products whose fp32 operands are split into bf16 parts.
//
// An fp32 x is b1 + b2 + b3 with b1 = bf16(x), b2 = bf16(x - b1), b3 = bf16(x - b1 - b2): three
// parts keep its 24 bits, two about 16.  A product of operands with PA and PB parts sums the
// pairs whose order i + j stays below max(PA, PB): 3 products for an fp32 operand with an exact
// bf16 one, 6 for two fp32 operands (relative 2^-24), 3 for two of two parts (2^-16).
//
// Fragments of m16n8k16, lane = 4 g + c:  A holds rows g, g + 8 and k = 2c, 2c + 1, 2c + 8, 2c + 9;
// B the same k of column g; the accumulator rows g, g + 8 of columns 2c, 2c + 1.  The
// accumulators of two neighbouring column tiles are therefore an A fragment of the next product.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace infini {
namespace gd {

typedef __nv_bfloat16 bf16;

template <int P> struct AFrag {
  uint32_t r[P][4];
};
template <int P> struct BFrag {  // two column tiles: [2 t + h], k half h of tile t
  uint32_t r[P][4];
};

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Column tiles 0, 1 of d += A B.  The smallest terms first.
template <int PA, int PB> __device__ __forceinline__ void mma2(float (&d0)[4], float (&d1)[4], const AFrag<PA>& a, const BFrag<PB>& b) {
  constexpr int M = (PA > PB ? PA : PB) - 1;
#pragma unroll
  for (int o = M; o >= 0; --o)
#pragma unroll
    for (int i = 0; i < PA; ++i) {
      const int j = o - i;
      if (j < 0 || j >= PB) continue;
      mma16816(d0, a.r[i], b.r[j][0], b.r[j][1]);
      mma16816(d1, a.r[i], b.r[j][2], b.r[j][3]);
    }
}

// Column tile t of d += A B with the pairs of order above 0 (2^-8 of the result) in a sum of their
// own: the tensor cores truncate each addition to a running sum, so the fewer additions the large
// sum takes the smaller the error (the state over 512 chunks, relative: 3.6e-7 before, 2.0e-7 so),
// and the sums are independent chains.
template <int PA, int PB> __device__ __forceinline__ void mma1(float (&h)[4], float (&l)[4], const AFrag<PA>& a, const BFrag<PB>& b, int t) {
  constexpr int M = (PA > PB ? PA : PB) - 1;
  mma16816(h, a.r[0], b.r[0][2 * t], b.r[0][2 * t + 1]);
#pragma unroll
  for (int o = M; o > 0; --o)
#pragma unroll
    for (int i = 0; i < PA; ++i) {
      const int j = o - i;
      if (j >= 0 && j < PB) mma16816(l, a.r[i], b.r[j][2 * t], b.r[j][2 * t + 1]);
    }
}
// Both tiles.
template <int PA, int PB>
__device__ __forceinline__ void mma2(float (&h0)[4], float (&h1)[4], float (&l0)[4], float (&l1)[4], const AFrag<PA>& a, const BFrag<PB>& b) {
  constexpr int M = (PA > PB ? PA : PB) - 1;
  mma16816(h0, a.r[0], b.r[0][0], b.r[0][1]);
  mma16816(h1, a.r[0], b.r[0][2], b.r[0][3]);
#pragma unroll
  for (int o = M; o > 0; --o)
#pragma unroll
    for (int i = 0; i < PA; ++i) {
      const int j = o - i;
      if (j < 0 || j >= PB) continue;
      mma16816(l0, a.r[i], b.r[j][0], b.r[j][1]);
      mma16816(l1, a.r[i], b.r[j][2], b.r[j][3]);
    }
}

// Slot s of every part from the pair (x0, x1).
template <int P> __device__ __forceinline__ void split(float x0, float x1, uint32_t (&r)[P][4], int s) {
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const uint32_t h = pack_bf16x2(x0, x1);
    r[p][s] = h;
    if (p + 1 < P) {
      x0 -= bf16_lo(h);
      x1 -= bf16_hi(h);
    }
  }
}
// A fragment of a k-step from its two accumulator tiles.
template <int P> __device__ __forceinline__ AFrag<P> from_acc(const float (&lo)[4], const float (&hi)[4]) {
  AFrag<P> a;
  split<P>(lo[0], lo[1], a.r, 0);
  split<P>(lo[2], lo[3], a.r, 1);
  split<P>(hi[0], hi[1], a.r, 2);
  split<P>(hi[2], hi[3], a.r, 3);
  return a;
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], const bf16* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_u32(p)));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], const bf16* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_u32(p)));
}

// B[k][n] = m[n][k] (k contiguous), columns n0 .. n0 + 15.
template <int P> __device__ __forceinline__ BFrag<P> load_b_k(const bf16* m, int ld, int n0, int k0, int lane) {
  static_assert(P == 1, "bf16 is exact in one part");
  BFrag<P> b;
  ldsm4(b.r[0], m + (n0 + (lane >> 4) * 8 + (lane & 7)) * ld + k0 + ((lane >> 3) & 1) * 8);
  return b;
}
template <int P> __device__ __forceinline__ BFrag<P> load_b_k(const float* m, int ld, int n0, int k0, int lane) {
  BFrag<P> b;
  const float* p = m + (n0 + (lane >> 2)) * ld + k0 + 2 * (lane & 3);
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float2 x = *reinterpret_cast<const float2*>(p + 8 * t * ld + 8 * h);
      split<P>(x.x, x.y, b.r, 2 * t + h);
    }
  return b;
}
// ... columns of the tiles ta and tb (8 each)
__device__ __forceinline__ BFrag<1> load_b_k2(const bf16* m, int ld, int ta, int tb, int k0, int lane) {
  BFrag<1> b;
  ldsm4(b.r[0], m + ((lane < 16 ? ta : tb) * 8 + (lane & 7)) * ld + k0 + (lane & 8));
  return b;
}
__device__ __forceinline__ BFrag<3> load_b_k2(const float* m, int ld, int ta, int tb, int k0, int lane) {
  BFrag<3> b;
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float2 x = *reinterpret_cast<const float2*>(m + ((t ? tb : ta) * 8 + (lane >> 2)) * ld + k0 + 2 * (lane & 3) + 8 * h);
      split<3>(x.x, x.y, b.r, 2 * t + h);
    }
  return b;
}
// B[k][n] = m[k][n] (n contiguous).
template <int P> __device__ __forceinline__ BFrag<P> load_b_n(const bf16* m, int ld, int k0, int n0, int lane) {
  static_assert(P == 1, "bf16 is exact in one part");
  BFrag<P> b;
  ldsm4t(b.r[0], m + (k0 + ((lane >> 3) & 1) * 8 + (lane & 7)) * ld + n0 + (lane >> 4) * 8);
  return b;
}
template <int P> __device__ __forceinline__ BFrag<P> load_b_n(const float* m, int ld, int k0, int n0, int lane) {
  BFrag<P> b;
  const float* p = m + (k0 + 2 * (lane & 3)) * ld + n0 + (lane >> 2);
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int h = 0; h < 2; ++h) split<P>(p[8 * h * ld + 8 * t], p[(8 * h + 1) * ld + 8 * t], b.r, 2 * t + h);
  return b;
}
// A[m][k] = x[m][k] (k contiguous).
template <int P> __device__ __forceinline__ AFrag<P> load_a_k(const bf16* x, int ld, int m0, int k0, int lane) {
  static_assert(P == 1, "bf16 is exact in one part");
  AFrag<P> a;
  ldsm4(a.r[0], x + (m0 + ((lane >> 3) & 1) * 8 + (lane & 7)) * ld + k0 + (lane >> 4) * 8);
  return a;
}
// ... of an fp32 operand, rows g and g + 8 times s0 and s1
template <int P>
__device__ __forceinline__ AFrag<P> load_a_k(const float* x, int ld, int m0, int k0, int lane, float s0 = 1.f, float s1 = 1.f) {
  AFrag<P> a;
  const float* p = x + (m0 + (lane >> 2)) * ld + k0 + 2 * (lane & 3);
#pragma unroll
  for (int kh = 0; kh < 2; ++kh)
#pragma unroll
    for (int rh = 0; rh < 2; ++rh) {
      const float2 v = *reinterpret_cast<const float2*>(p + 8 * rh * ld + 8 * kh);
      const float s = rh ? s1 : s0;
      split<P>(s * v.x, s * v.y, a.r, rh + 2 * kh);
    }
  return a;
}
// A[m][k] = x[k][m] (m contiguous).
template <int P> __device__ __forceinline__ AFrag<P> load_a_m(const bf16* x, int ld, int k0, int m0, int lane) {
  static_assert(P == 1, "bf16 is exact in one part");
  AFrag<P> a;
  ldsm4t(a.r[0], x + (k0 + (lane >> 4) * 8 + (lane & 7)) * ld + m0 + ((lane >> 3) & 1) * 8);
  return a;
}
template <int P> __device__ __forceinline__ AFrag<P> load_a_m(const float* x, int ld, int k0, int m0, int lane) {
  AFrag<P> a;
  const float* p = x + (k0 + 2 * (lane & 3)) * ld + m0 + (lane >> 2);
#pragma unroll
  for (int kh = 0; kh < 2; ++kh)
#pragma unroll
    for (int rh = 0; rh < 2; ++rh) split<P>(p[8 * kh * ld + 8 * rh], p[(8 * kh + 1) * ld + 8 * rh], a.r, rh + 2 * kh);
  return a;
}
// ... with k times s[k] (s at k0), in P parts
template <int P> __device__ __forceinline__ AFrag<P> load_a_m_scaled(const bf16* x, int ld, int k0, int m0, int lane, const float* s, float f) {
  const AFrag<1> e = load_a_m<1>(x, ld, k0, m0, lane);
  AFrag<P> a;
#pragma unroll
  for (int kh = 0; kh < 2; ++kh) {
    const float2 w = *reinterpret_cast<const float2*>(s + 8 * kh + 2 * (lane & 3));
#pragma unroll
    for (int rh = 0; rh < 2; ++rh) {
      const uint32_t u = e.r[0][rh + 2 * kh];
      split<P>(bf16_lo(u) * (f * w.x), bf16_hi(u) * (f * w.y), a.r, rh + 2 * kh);
    }
  }
  return a;
}
template <int P> __device__ __forceinline__ AFrag<P> load_a_m_scaled(const float* x, int ld, int k0, int m0, int lane, const float* s, float f) {
  AFrag<P> a;
  const float* p = x + (k0 + 2 * (lane & 3)) * ld + m0 + (lane >> 2);
#pragma unroll
  for (int kh = 0; kh < 2; ++kh) {
    const float2 w = *reinterpret_cast<const float2*>(s + 8 * kh + 2 * (lane & 3));
#pragma unroll
    for (int rh = 0; rh < 2; ++rh)
      split<P>(p[8 * kh * ld + 8 * rh] * (f * w.x), p[(8 * kh + 1) * ld + 8 * rh] * (f * w.y), a.r, rh + 2 * kh);
  }
  return a;
}

// Fragments of a matrix kept as P planes of bf16 parts, `plane` elements apart.
template <int P> __device__ __forceinline__ BFrag<P> load_b_k(const bf16* m, int plane, int ld, int n0, int k0, int lane) {
  BFrag<P> b;
  const bf16* x = m + (n0 + (lane >> 4) * 8 + (lane & 7)) * ld + k0 + ((lane >> 3) & 1) * 8;
#pragma unroll
  for (int p = 0; p < P; ++p) ldsm4(b.r[p], x + p * plane);
  return b;
}
template <int P> __device__ __forceinline__ BFrag<P> load_b_n(const bf16* m, int plane, int ld, int k0, int n0, int lane) {
  BFrag<P> b;
  const bf16* x = m + (k0 + ((lane >> 3) & 1) * 8 + (lane & 7)) * ld + n0 + (lane >> 4) * 8;
#pragma unroll
  for (int p = 0; p < P; ++p) ldsm4t(b.r[p], x + p * plane);
  return b;
}
template <int P> __device__ __forceinline__ AFrag<P> load_a_k(const bf16* m, int plane, int ld, int m0, int k0, int lane) {
  AFrag<P> a;
  const bf16* x = m + (m0 + ((lane >> 3) & 1) * 8 + (lane & 7)) * ld + k0 + (lane >> 4) * 8;
#pragma unroll
  for (int p = 0; p < P; ++p) ldsm4(a.r[p], x + p * plane);
  return a;
}
template <int P> __device__ __forceinline__ AFrag<P> load_a_m(const bf16* m, int plane, int ld, int k0, int m0, int lane) {
  AFrag<P> a;
  const bf16* x = m + (k0 + (lane >> 4) * 8 + (lane & 7)) * ld + m0 + ((lane >> 3) & 1) * 8;
#pragma unroll
  for (int p = 0; p < P; ++p) ldsm4t(a.r[p], x + p * plane);
  return a;
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {  // an 8 x 8 block of 16-bit elements
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// B[k][n] = x[k][n] from the accumulator tiles of x: rows k = 16, columns the tiles' 2 x 8.
template <int P> __device__ __forceinline__ BFrag<P> b_from_acc(const float4& t0, const float4& t1) {
  BFrag<P> b;
  split<P>(t0.x, t0.y, b.r, 0);
  split<P>(t0.z, t0.w, b.r, 1);
  split<P>(t1.x, t1.y, b.r, 2);
  split<P>(t1.z, t1.w, b.r, 3);
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int i = 0; i < 4; ++i) b.r[p][i] = transpose8(b.r[p][i]);
  return b;
}
// A fragments to and from shared memory as they are: [part][lane], 16 bytes each
template <int P> __device__ __forceinline__ void put_frag(uint4* dst, const AFrag<P>& a, int lane) {
#pragma unroll
  for (int p = 0; p < P; ++p) dst[p * 32 + lane] = make_uint4(a.r[p][0], a.r[p][1], a.r[p][2], a.r[p][3]);
}
// ... the half of k step t / 2 that accumulator tile t is
template <int P> __device__ __forceinline__ void put_tile(uint4* dst, const float (&x)[4], int t, int lane) {
  uint32_t r[P][4];
  split<P>(x[0], x[1], r, 0);
  split<P>(x[2], x[3], r, 1);
#pragma unroll
  for (int p = 0; p < P; ++p) reinterpret_cast<uint2*>(dst + p * 32 + lane)[t & 1] = make_uint2(r[p][0], r[p][1]);
}
// A [16 columns x 8 tokens] accumulator tile (rows = columns of m) from, and rounded to, 8 rows of m from x.
__device__ __forceinline__ void load_tile_t(float (&d)[4], const float* m, int ld, int lane) {
  const float* p = m + 2 * (lane & 3) * ld + (lane >> 2);
  d[0] = p[0];
  d[1] = p[ld];
  d[2] = p[8];
  d[3] = p[ld + 8];
}
__device__ __forceinline__ void load_tile_t(float (&d)[4], const bf16* m, int ld, int lane) {
  uint32_t a, b;
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];"
               : "=r"(a), "=r"(b)
               : "r"(smem_u32(m + (lane & 7) * ld + (lane & 8))));
  d[0] = bf16_lo(a);
  d[1] = bf16_hi(a);
  d[2] = bf16_lo(b);
  d[3] = bf16_hi(b);
}
__device__ __forceinline__ void store_tile_t(float* m, int ld, const float (&d)[4], int lane) {
  float* p = m + 2 * (lane & 3) * ld + (lane >> 2);
  p[0] = d[0];
  p[ld] = d[1];
  p[8] = d[2];
  p[ld + 8] = d[3];
}
__device__ __forceinline__ void store_tile_t(bf16* m, int ld, const float (&d)[4], int lane) {
  asm volatile("stmatrix.sync.aligned.m8n8.x2.trans.shared.b16 [%0], {%1, %2};" ::"r"(smem_u32(m + (lane & 7) * ld + (lane & 8))),
               "r"(pack_bf16x2(d[0], d[1])), "r"(pack_bf16x2(d[2], d[3]))
               : "memory");
}
// ... in three parts, each a plane
__device__ __forceinline__ void store_parts_t(bf16* m, int plane, int ld, const float (&d)[4], int lane) {
  uint32_t r[3][4];
  split<3>(d[0], d[1], r, 0);
  split<3>(d[2], d[3], r, 1);
#pragma unroll
  for (int p = 0; p < 3; ++p)
    asm volatile("stmatrix.sync.aligned.m8n8.x2.trans.shared.b16 [%0], {%1, %2};" ::"r"(smem_u32(m + p * plane + (lane & 7) * ld + (lane & 8))),
                 "r"(r[p][0]), "r"(r[p][1])
                 : "memory");
}
template <int P> __device__ __forceinline__ AFrag<P> get_frag(const uint4* src, int lane) {
  AFrag<P> a;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const uint4 x = src[p * 32 + lane];
    a.r[p][0] = x.x; a.r[p][1] = x.y; a.r[p][2] = x.z; a.r[p][3] = x.w;
  }
  return a;
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool in) {
  const int n = in ? 16 : 0;  // the rest is written as zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Rows 0 .. 63 of `cols` (a multiple of 16 bytes) elements into shared memory, zeros where the
// row is at or past n or the column at or past d.  vec: rows start on 16 bytes and d is a
// multiple of them; then the copy is asynchronous.
template <typename T>
__device__ __forceinline__ void load_rows(T* dst, int ld, const T* src, long long stride, int n, int d, int cols, bool vec,
                                          int tid, int nthr) {
  constexpr int V = 16 / sizeof(T);
  if (vec) {
    const int sh = __ffs(cols / V) - 1;  // cols / V is a power of 2, nthr a multiple of it
    const int x = (tid & (cols / V - 1)) * V, r0 = tid >> sh, rows = nthr >> sh;
    const T* p = src + r0 * stride + x;
    T* to = dst + r0 * ld + x;
    const long long step = rows * stride;
#pragma unroll 4
    for (int r = r0; r < 64; r += rows, p += step, to += rows * ld) {
      const bool in = r < n && x < d;
      cp_async16(to, in ? p : src, in);
    }
  } else {
    for (int i = tid; i < 64 * cols; i += nthr) {
      const int r = i / cols, x = i % cols;
      dst[r * ld + x] = (r < n && x < d) ? src[r * stride + x] : from_f32<T>(0.f);
    }
  }
}

}  // namespace gd
}  // namespace infini
