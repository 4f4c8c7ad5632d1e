// Gated delta rule, token by token (CUDA cores, fp32):
//   S' = e^g S,  u = beta (v - S'^T k),  S = S' + k u^T,  o = scale S^T q.
// With both products taken on the old state, kS = S^T k and qS = S^T q, a token is one pass and
// one reduction: u = beta (v - e^g kS), o = scale (e^g qS + (q.k) u).
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace infini {
namespace gd {

constexpr int kMaxHead = 128;

struct RecurArgs {
  const void* q;
  const void* k;
  const void* v;
  const float* g;
  const float* beta;
  float* S;
  void* out;
  const int* lens;   // [B] or nullptr
  const int* slots;  // [B] or nullptr: row b
  long long qs[3], ks[3], vs[3], os[3], gs[3], bs[3];
  long long L, pool;
  int B, H, group, dk, dv;
  float scale;
};

constexpr int kRecurThreads = 128;
constexpr int kRecurCols = 16;  // value columns per block

// HBM-bound for a serving batch: 192 requests x 32 heads of 128 x 128, 805 MB of state in and out, in
// 164 us (75 % of the copy rate); one request of 8 heads 2.5 us, another token 0.6 us.  A thread per
// column with all 128 rows in registers needs no reduction but 255 registers: 217 us.
// One block: 16 value columns of one (b, h).  Thread (rg, cg) holds rows rg + 32 i and columns
// 4 cg .. 4 cg + 3 of the state in registers for the whole call.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kRecurThreads) recur_kernel(const RecurArgs a) {
  __shared__ float sk[2][kMaxHead], sq[2][kMaxHead];
  __shared__ float red[2][4][4][9];
  __shared__ int next_b;
  const int tid = threadIdx.x, cg = tid & 3, rg = tid >> 2, warp = tid >> 5;
  const int h = blockIdx.y, col = blockIdx.x * kRecurCols + cg * 4;
  int b = blockIdx.z;
  const long long row = a.slots ? a.slots[b] : b;
  if (row < 0 || row >= a.pool) return;  // a padded request
  float* Sp = a.S + (row * a.H + h) * a.dk * a.dv;
  float s[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = rg + 32 * i;
    if (VEC && r < a.dk && col < a.dv) {
      const float4 x = *reinterpret_cast<const float4*>(Sp + (long long)r * a.dv + col);
      s[i][0] = x.x; s[i][1] = x.y; s[i][2] = x.z; s[i][3] = x.w;
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) s[i][c] = (!VEC && r < a.dk && col + c < a.dv) ? Sp[(long long)r * a.dv + col + c] : 0.f;
    }
  }
  if (a.slots) {
    // the first request that names a slot takes the others of it too, in order
    int before = 0;
    for (int i = tid; i < b; i += kRecurThreads) before |= a.slots[i] == row;
    if (__syncthreads_or(before)) return;
  }
  const int hk = h / a.group;
  for (;;) {
    const long long len = a.lens ? min(max((long long)a.lens[b], 0LL), a.L) : a.L;
    const T* q = static_cast<const T*>(a.q) + b * a.qs[0] + hk * a.qs[1];
    const T* k = static_cast<const T*>(a.k) + b * a.ks[0] + hk * a.ks[1];
    const T* v = static_cast<const T*>(a.v) + b * a.vs[0] + h * a.vs[1];
    const float* g = a.g + b * a.gs[0] + h * a.gs[1];
    const float* be = a.beta + b * a.bs[0] + h * a.bs[1];
    T* o = static_cast<T*>(a.out) + b * a.os[0] + h * a.os[1];
    for (long long t = 0; t < len; ++t) {
      const int p = t & 1;
      sk[p][tid] = tid < a.dk ? to_f32(k[t * a.ks[2] + tid]) : 0.f;
      sq[p][tid] = tid < a.dk ? to_f32(q[t * a.qs[2] + tid]) : 0.f;
      const float decay = expf(g[t * a.gs[2]]), beta = be[t * a.bs[2]];
      float vv[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) vv[c] = col + c < a.dv ? to_f32(v[t * a.vs[2] + col + c]) : 0.f;
      __syncthreads();
      if (decay == 0.f)  // cleared, and 0 * s would not be 0 of a state that is not finite
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) s[i][c] = 0.f;
      float x[9] = {};  // kS and qS of four columns, q.k
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float kr = sk[p][rg + 32 * i], qr = sq[p][rg + 32 * i];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          x[c] = fmaf(kr, s[i][c], x[c]);
          x[4 + c] = fmaf(qr, s[i][c], x[4 + c]);
        }
        x[8] = fmaf(kr, qr, x[8]);
      }
#pragma unroll
      for (int off = 4; off < 32; off <<= 1)
#pragma unroll
        for (int n = 0; n < 9; ++n) x[n] += __shfl_xor_sync(0xffffffffu, x[n], off);
      if ((tid & 31) < 4)
#pragma unroll
        for (int n = 0; n < 9; ++n) red[p][warp][cg][n] = x[n];
      __syncthreads();
#pragma unroll
      for (int n = 0; n < 9; ++n) x[n] = (red[p][0][cg][n] + red[p][1][cg][n]) + (red[p][2][cg][n] + red[p][3][cg][n]);
      float u[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) u[c] = beta * (vv[c] - decay * x[c]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float kr = sk[p][rg + 32 * i];
#pragma unroll
        for (int c = 0; c < 4; ++c) s[i][c] = fmaf(kr, u[c], decay * s[i][c]);
      }
      if (rg == 0)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (col + c < a.dv) o[t * a.os[2] + col + c] = from_f32<T>(a.scale * fmaf(x[8], u[c], decay * x[4 + c]));
    }
    if (!a.slots) break;
    __syncthreads();
    if (tid == 0) next_b = a.B;
    __syncthreads();
    for (int i = b + 1 + tid; i < a.B; i += kRecurThreads)
      if (a.slots[i] == row) {
        atomicMin(&next_b, i);
        break;
      }
    __syncthreads();
    b = next_b;
    if (b >= a.B) break;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = rg + 32 * i;
    if (r >= a.dk) continue;
    if (VEC) {
      if (col < a.dv) *reinterpret_cast<float4*>(Sp + (long long)r * a.dv + col) = make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (col + c < a.dv) Sp[(long long)r * a.dv + col + c] = s[i][c];
    }
  }
}

}  // namespace gd
}  // namespace infini
