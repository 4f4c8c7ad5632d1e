// Gated delta rule over chunks of 64 tokens.
//
// With G the running sum of the log decays inside a chunk, gamma_i = e^G_i, rho_i = e^(G_last - G_i),
// Gamma = e^G_last and S the state before the chunk, the recurrence of 64 tokens is
//   (I + A) U = X,   A_ij = beta_i e^(G_i - G_j) k_i.k_j (i > j),   X = beta (V - gamma (K S))
//   O  = scale (gamma (Q S) + P U),   P_ij = e^(G_i - G_j) q_i.k_j (i >= j)
//   S' = Gamma S + K^T (rho U)
// prep_kernel computes T = (I + A)^-1 and P of every chunk in parallel; state_pass (forward_kernel)
// passes the state from chunk to chunk.  Only differences G_i - G_j with i >= j enter an exponential, so
// nothing overflows that the recurrence itself does not.  G is summed in 64 bits (a difference of
// two sums near -100 would have lost 1e-5 in 32), from max(g, -1e4): e^-1e4 is 0 in fp32, and
// differences stay finite where g is -inf.  A token whose own decay is 0 clears the state, one that
// is not finite too: gamma is -0 (not 0) from that token on and Gamma in its chunk, and state_pass
// selects there where 0 * S would not be 0.
//
// Gradients, with d denoting the loss's derivative and dS' that of the state after the chunk:
//   dU = scale P^T dO + rho (K dS'),  dX = T^T dU,  dV = beta dX,  dA = -dX U^T,  dP = scale dO U^T
//   dQ = (dP e^(G_i-G_j)) K + scale gamma dO S^T
//   dK = (dP e^..)^T Q + (M + M^T) K - beta gamma dX S^T + rho U dS'^T,  M_ij = beta_i e^(G_i-G_j) dA_ij
//   dbeta_i = dX_i.(V - gamma K S)_i + sum_j dA_ij e^(G_i-G_j) k_i.k_j
//   dG collects every exponent's derivative; dg_t = sum_(i >= t) dG_i
//   dS = Gamma dS' + scale Q^T (gamma dO) - K^T (beta gamma dX)
// bwd_state_pass (both_kernel, beside state_pass) passes dS from chunk to chunk, grad_kernel or
// grad_bf16_kernel does the rest for all chunks in parallel from the stored states and state
// gradients.
//
// Every product runs on mma.sync with fp32 operands split into bf16 parts (gd_frag.cuh).  A group
// of KS warps owns 16 columns of the state, transposed (rows = value columns): each warp holds
// DK / KS rows of S in its accumulators and works on 64 / KS tokens of a chunk, so that K S, T X,
// P U and the update of S follow one another with fragments that pass through shared memory
// unchanged (KS 4) or stay in registers (KS 1).
#pragma once

#include "gd_frag.cuh"

namespace infini {
namespace gd {

constexpr int kC = 64;             // tokens per chunk
constexpr int kTri = 10 * 256;     // elements of a lower triangular 64 x 64 matrix: 16 x 16 blocks r >= c at r (r + 1) / 2 + c, swizzled (tri_at)
constexpr int kVec = 256;          // floats per chunk: gamma[64], rho[64], beta[64], Gamma; the sign of gamma, Gamma: cleared
constexpr int kLdT = 68;           // leading dimension of 64 x 64 fp32 matrices in shared memory
constexpr int kMaxWarps = 8;
constexpr float kMinLog = -1e4f;

template <typename T, int DK> struct Dims {
  static constexpr int kLdK = DK + 16 / (int)sizeof(T);  // rows shifted by 4 banks
  static constexpr int kIn = sizeof(T) == 2 ? 1 : 3;     // parts of an input element
  // Parts of an fp32 factor of a result that is rounded to T.  For bf16 two: the error against 64 bits is that of the
  // rounding, 1.66e-3, with two parts and with three (the results differ from the fp32 formulas' by 1.2e-4 and 4e-5),
  // and three cost a tenth (B 4, H 32, L 4096: 684 us instead of 619; B 2, H 8, L 2048: 119 instead of 103).
  static constexpr int kOut = sizeof(T) == 2 ? 2 : 3;
};

struct ChunkArgs {
  const void* q;
  const void* k;
  const void* v;
  const float* g;
  const float* beta;
  const void* d_out;
  const int* lens;
  long long qs[3], ks[3], vs[3], os[3], gs[3], bs[3];  // os: out, or d_out
  long long L;
  int B, H, Hk, group, dk, dv;
  float scale;
  bool vec_k, vec_v, vec_o;  // 16-byte rows of q and k, of v, of out / d_out
  // chunks c0 .. c0 + nc - 1 of every row are worked on; workspaces hold those
  int c0, nc;
  int groups;  // state kernels: groups of 16 value columns per block (a power of 2)
  int blocks;  // ... blocks per (b, h) and segment
  int stages;  // ... chunks in shared memory, 1 or 2
  int first_loader;  // ... the threads from this one on copy the next chunk
  bf16* T;       // [B H][nc][3][kTri]: the three bf16 parts
  bf16* P;       // [B H][nc][parts][kTri]
  float* vec;    // [B H][nc][kVec]
  float2* G;     // [B H][nc][64]: high and low part
  float4* snap;  // [B H][nc][nw][DK / 8][32]: states before the chunks (accumulator order)
  float4* dsnap; // the same of the gradients of the states after them
  // With few (b, h) a row's chunks are split into nseg segments of seg chunks that run side by side
  int seg, nseg;
  float4* segS;  // [B H][nseg][nw][DK / 8][32]: the state before a segment
  float4* segD;  // [B H][nseg][nw][DK / 8][32]: the gradient of the state after it
  float4* segA;  // [B H][nseg][DK / 16][DK / 8][32]: A with S_after = A S_before + B, 16 columns of it per strip; the first
                 // segment has none, and there float i says whether segment i clears the state
  float* S;      // forward: [B, H, dk, dv], read and written
  void* out;
  const float* S0;  // bwd: initial values, may be null (zero)
  const float* dS;  // bwd: gradient of the final state, may be null
  float* dS0;       // bwd: gradient of the initial state, may be null
  void* dq;
  void* dkk;
  void* dvv;
  float* dg;
  float* dbeta;
  bool vec_dq, vec_dv;  // pairs of dq and dk, 16-byte rows of dv can be written whole
  // grad, group > 1: dq and dk of one key head from its value heads, [B Hk][nc][2][64][DK] running sums of one block
  // that takes them in turn, or (split) [B H][nc][2][64][DK] a block's own, which sum_heads_kernel adds
  bool split;
  float* acc;
};

// A sum of log decays as two floats, and e^(a - b) of two such sums where `in`, else 0.  The
// difference of the high parts rounds at 2^-24 of itself and the low parts hold what they lack, so
// this is as good as a difference in 64 bits, whose conversions cost 6000 of 17000 cycles of a
// chunk's preparation; no branch, so that the exponentials overlap.
__device__ __forceinline__ float2 halves(double x) {
  const float hi = (float)x;
  return make_float2(hi, (float)(x - hi));
}
__device__ __forceinline__ float decay(float2 a, float2 b, bool in) {
  const float e = expf(in ? (a.x - b.x) + (a.y - b.y) : 0.f);
  return in ? e : 0.f;
}

__device__ __forceinline__ long long row_len(const ChunkArgs& a, int b) {
  return a.lens ? min(max((long long)a.lens[b], 0LL), a.L) : a.L;
}
// valid tokens of chunk c (absolute) of a row of n tokens
__device__ __forceinline__ int chunk_len(long long n, long long c) { return (int)min(max(n - c * kC, 0LL), (long long)kC); }
__device__ __forceinline__ int tri_block(int r, int c) { return r * (r + 1) / 2 + c; }

// Element (r, c) of a 16 x 16 block: 16-byte halves of a row change places every 4 rows, so that 8
// rows of a half lie in different banks.
__device__ __forceinline__ int tri_at(int r, int c) { return r * 16 + ((((c >> 3) ^ (r >> 2)) & 1) << 3) + (c & 7); }
// B[k][n] = m[n][k] of block (rb, cb): n its rows, k its columns; B[k][n] = m[k][n]: the other way.
template <int P> __device__ __forceinline__ BFrag<P> load_tri_k(const bf16* m, int rb, int cb, int lane) {
  BFrag<P> b;
  const bf16* x = m + tri_block(rb, cb) * 256 + tri_at((lane >> 4) * 8 + (lane & 7), lane & 8);
#pragma unroll
  for (int p = 0; p < P; ++p) ldsm4(b.r[p], x + p * kTri);
  return b;
}
template <int P> __device__ __forceinline__ BFrag<P> load_tri_n(const bf16* m, int rb, int cb, int lane) {
  BFrag<P> b;
  const bf16* x = m + tri_block(rb, cb) * 256 + tri_at((lane & 8) + (lane & 7), (lane >> 4) * 8);
#pragma unroll
  for (int p = 0; p < P; ++p) ldsm4t(b.r[p], x + p * kTri);
  return b;
}
// ... of the 8-wide tiles ta and tb at k step kk, as B[k][n] = m[n][k] (blocks kk <= t / 2) and B[k][n] =
// m[k][n] (kk >= t / 2); what a tile gets outside these blocks is not used.
template <int P> __device__ __forceinline__ BFrag<P> load_tri_k2(const bf16* m, int ta, int tb, int kk, int lane) {
  BFrag<P> b;
  const int t = lane < 16 ? ta : tb, rb = t >> 1;
  const bf16* x = m + tri_block(rb, min(kk, rb)) * 256 + tri_at((t & 1) * 8 + (lane & 7), lane & 8);
#pragma unroll
  for (int p = 0; p < P; ++p) ldsm4(b.r[p], x + p * kTri);
  return b;
}
template <int P> __device__ __forceinline__ BFrag<P> load_tri_n2(const bf16* m, int ta, int tb, int kk, int lane) {
  BFrag<P> b;
  const int t = lane < 16 ? ta : tb, cb = t >> 1;
  const bf16* x = m + tri_block(max(kk, cb), cb) * 256 + tri_at(lane & 15, (t & 1) * 8);
#pragma unroll
  for (int p = 0; p < P; ++p) ldsm4t(b.r[p], x + p * kTri);
  return b;
}
// A[m][k] = m[m][k] of block (rb, cb), and A[m][k] = m[k][m].
template <int P> __device__ __forceinline__ AFrag<P> load_tri_a_k(const bf16* m, int rb, int cb, int lane) {
  AFrag<P> a;
  const bf16* x = m + tri_block(rb, cb) * 256 + tri_at((lane & 8) + (lane & 7), (lane >> 4) * 8);
#pragma unroll
  for (int p = 0; p < P; ++p) ldsm4(a.r[p], x + p * kTri);
  return a;
}
template <int P> __device__ __forceinline__ AFrag<P> load_tri_a_m(const bf16* m, int rb, int cb, int lane) {
  AFrag<P> a;
  const bf16* x = m + tri_block(rb, cb) * 256 + tri_at((lane >> 4) * 8 + (lane & 7), lane & 8);
#pragma unroll
  for (int p = 0; p < P; ++p) ldsm4t(a.r[p], x + p * kTri);
  return a;
}
// A matrix of three parts as fp32 [64][kLdT].
__device__ __forceinline__ void load_tri_f32(float* dst, const bf16* src, int tid, int nthr) {
  for (int i = tid; i < kTri; i += nthr) {
    const int blk = i >> 8, r = blk >= 6 ? 3 : blk >= 3 ? 2 : blk >= 1 ? 1 : 0, c = blk - r * (r + 1) / 2;
    const bf16* x = src + blk * 256 + tri_at((i >> 4) & 15, i & 15);
    dst[(16 * r + ((i >> 4) & 15)) * kLdT + 16 * c + (i & 15)] = (to_f32(x[2 * kTri]) + to_f32(x[kTri])) + to_f32(x[0]);
  }
}
// The parts of (x0, x1), elements at and at + 1 of planes `plane` apart.
template <int P> __device__ __forceinline__ void put_parts(bf16* dst, int plane, float x0, float x1) {
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const uint32_t h = pack_bf16x2(x0, x1);
    *reinterpret_cast<uint32_t*>(dst + p * plane) = h;
    x0 -= bf16_lo(h);
    x1 -= bf16_hi(h);
  }
}

// ------------------------------------------------------------------ prep
template <typename T, int DK> struct PrepSmem {
  union {
    struct {
      T k[kC * Dims<T, DK>::kLdK];
      T q[kC * Dims<T, DK>::kLdK];
    };
    float R[kC * kLdT];  // T, once the products are done
  };
  float A[kC * kLdT];
  float2 G[kC];
  float beta[kC];
};

// Blocks at distance D below the diagonal: T_rc = -T_rr (sum_(c <= m < r) A_rm T_mc), r = c + D; warp c
// computes its block, into R and in parts into T.  (Scalar products by all threads: 256 fused
// multiply-adds and as many shared loads a thread, 4000 of 17000 cycles.)
template <int D> __device__ __forceinline__ void invert_level(const float* A, float* R, bf16* T, int warp, int lane) {
  const int c = warp, r = c + D, g = lane >> 2, c2 = 2 * (lane & 3);
  if (c < 4 - D) {
    float hi[2][4] = {}, lo[2][4] = {};
#pragma unroll
    for (int m = 0; m < D; ++m)
      mma2(hi[0], hi[1], lo[0], lo[1], load_a_k<3>(A, kLdT, 16 * r, 16 * (c + m), lane), load_b_n<3>(R, kLdT, 16 * (c + m), 16 * c, lane));
    float4 e[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) e[t] = make_float4(hi[t][0] + lo[t][0], hi[t][1] + lo[t][1], hi[t][2] + lo[t][2], hi[t][3] + lo[t][3]);
    const BFrag<3> fe = b_from_acc<3>(e[0], e[1]);
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int x = 0; x < 4; ++x) hi[t][x] = lo[t][x] = 0.f;
    mma2(hi[0], hi[1], lo[0], lo[1], load_a_k<3>(R, kLdT, 16 * r, 16 * r, lane), fe);
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float x0 = -(hi[t][2 * h] + lo[t][2 * h]), x1 = -(hi[t][2 * h + 1] + lo[t][2 * h + 1]);
        const int i = g + 8 * h, j = 8 * t + c2;
        if (D < 3) *reinterpret_cast<float2*>(R + (16 * r + i) * kLdT + 16 * c + j) = make_float2(x0, x1);
        put_parts<3>(T + tri_block(r, c) * 256 + tri_at(i, j), kTri, x0, x1);
      }
  }
  if (D < 3) __syncthreads();
}

// PP: parts of P that are stored
template <typename T, int DK, int PP> __global__ void __launch_bounds__(256) prep_kernel(const ChunkArgs a) {
  constexpr int LD = Dims<T, DK>::kLdK, PI = Dims<T, DK>::kIn;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  PrepSmem<T, DK>& s = *reinterpret_cast<PrepSmem<T, DK>*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c2 = 2 * (lane & 3);
  const int b = blockIdx.z, h = blockIdx.y, hk = h / a.group;
  const long long c = a.c0 + (int)blockIdx.x;
  const int n = chunk_len(row_len(a, b), c);
  if (n == 0) return;
  const long long t0 = c * kC;
  const T* q = static_cast<const T*>(a.q) + b * a.qs[0] + hk * a.qs[1] + t0 * a.qs[2];
  const T* k = static_cast<const T*>(a.k) + b * a.ks[0] + hk * a.ks[1] + t0 * a.ks[2];
  load_rows<T>(s.k, LD, k, a.ks[2], n, a.dk, DK, a.vec_k, tid, 256);
  load_rows<T>(s.q, LD, q, a.qs[2], n, a.dk, DK, a.vec_k, tid, 256);
  cp_async_commit();
  const long long at = ((long long)b * a.H + h) * a.nc + blockIdx.x;
  if (warp == 0) {
    const float* gp = a.g + b * a.gs[0] + h * a.gs[1] + t0 * a.gs[2];
    const float* bp = a.beta + b * a.bs[0] + h * a.bs[1] + t0 * a.bs[2];
    double x[2];
    float be[2];
    unsigned clear[2];  // bit l: token 2 l + i clears the state
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = 2 * lane + i;
      const float gt = t < n ? gp[t * a.gs[2]] : 0.f;
      x[i] = gt < kMinLog ? kMinLog : gt;
      clear[i] = __ballot_sync(0xffffffffu, expf(gt) == 0.f);
      be[i] = t < n ? bp[t * a.bs[2]] : 0.f;
    }
    double sum = x[0] + x[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += y;
    }
    const double G0 = sum - x[1], G1 = sum, last = __shfl_sync(0xffffffffu, sum, 31);
    const float2 two[2] = {halves(G0), halves(G1)};
    s.G[2 * lane] = two[0];
    s.G[2 * lane + 1] = two[1];
    s.beta[2 * lane] = be[0];
    s.beta[2 * lane + 1] = be[1];
    *reinterpret_cast<float4*>(a.G + at * kC + 2 * lane) = make_float4(two[0].x, two[0].y, two[1].x, two[1].y);
    float* v = a.vec + at * kVec;
    const unsigned before = (1u << lane) - 1, upto = (2u << lane) - 1;
    const bool c0 = (clear[0] & upto) | (clear[1] & before), c1 = (clear[0] | clear[1]) & upto;
    *reinterpret_cast<float2*>(v + 2 * lane) = make_float2(c0 ? -0.f : expf((float)G0), c1 ? -0.f : expf((float)G1));
    *reinterpret_cast<float2*>(v + 64 + 2 * lane) = make_float2(expf((float)(last - G0)), expf((float)(last - G1)));
    *reinterpret_cast<float2*>(v + 128 + 2 * lane) = make_float2(be[0], be[1]);
    if (lane == 0) v[192] = clear[0] | clear[1] ? -0.f : expf((float)last);
  }
  cp_async_wait<0>();
  __syncthreads();
  // warps 0-3: K K^T, warps 4-7: Q K^T, 16 rows each, column blocks up to the diagonal.  The low orders of fp32 inputs
  // in sums of their own: 48 truncated additions to one left 7e-7 of the outputs and gradients that come from T and P,
  // 8 leave 2e-7 (one product has the same error from K S; the time is the same).
  const int rb = warp & 3, m0 = 16 * rb;
  const bool is_q = warp >= 4;
  float acc[4][2][4] = {}, lo[4][2][4] = {};
  for (int kk = 0; kk < DK / 16; ++kk) {
    const AFrag<PI> fa = load_a_k<PI>(is_q ? s.q : s.k, LD, m0, 16 * kk, lane);
#pragma unroll
    for (int cb = 0; cb < 4; ++cb)
      if (cb <= rb)
        mma2(acc[cb][0], acc[cb][1], lo[cb][0], lo[cb][1], fa, load_b_k<PI>(s.k, LD, 16 * cb, 16 * kk, lane));
  }
#pragma unroll
  for (int cb = 0; cb < 4; ++cb)
    if (cb <= rb)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2) {
          const int i = m0 + g + 8 * e2, j = 16 * cb + 8 * t + c2;
          float x[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const bool in = is_q ? i >= j + e : i > j + e;
            x[e] = (acc[cb][t][2 * e2 + e] + lo[cb][t][2 * e2 + e]) * decay(s.G[i], s.G[j + e], in) * (is_q ? 1.f : s.beta[i]);
          }
          if (is_q)
            put_parts<PP>(a.P + at * PP * kTri + tri_block(rb, cb) * 256 + tri_at(g + 8 * e2, 8 * t + c2), kTri, x[0], x[1]);
          else
            *reinterpret_cast<float2*>(s.A + i * kLdT + j) = make_float2(x[0], x[1]);
        }
  __syncthreads();
  // T = (I + A)^-1, lower triangular with a unit diagonal.  Diagonal blocks: column j of block d
  // by forward substitution, one thread each.
  if (tid < 64) {
    const int d = tid >> 4, j = tid & 15;
    const float* Ad = s.A + 16 * d * kLdT + 16 * d;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float y = i == j ? 1.f : 0.f;
#pragma unroll
      for (int m = 0; m < i; ++m) y = fmaf(-Ad[i * kLdT + m], x[m], y);
      x[i] = i >= j ? y : 0.f;
      s.R[(16 * d + i) * kLdT + 16 * d + j] = x[i];
    }
  }
  __syncthreads();
  bf16* T_out = a.T + at * 3 * kTri;
  {  // the diagonal blocks' parts
    const int d = tid >> 6, i = (tid >> 2) & 15, j = (tid & 3) * 4;
    const float4 x = *reinterpret_cast<const float4*>(s.R + (16 * d + i) * kLdT + 16 * d + j);
    bf16* to = T_out + tri_block(d, d) * 256 + tri_at(i, j);
    put_parts<3>(to, kTri, x.x, x.y);
    put_parts<3>(to + 2, kTri, x.z, x.w);
  }
  invert_level<1>(s.A, s.R, T_out, warp, lane);
  invert_level<2>(s.A, s.R, T_out, warp, lane);
  invert_level<3>(s.A, s.R, T_out, warp, lane);
}

// ------------------------------------------------------------------ state
constexpr int kMaxGroups = 4;
template <typename T, int DK, int PP> struct Stage {
  T k[kC * Dims<T, DK>::kLdK];
  T q[kC * Dims<T, DK>::kLdK];
  bf16 Tm[3 * kTri];
  bf16 P[PP * kTri];
  float vec[kVec];
  // then [64][ldv] of T: the block's value columns of v (then of out) or d_out
};
// Fragments that the warps of a group exchange (KS > 1): of S, of X (dU), of rho U (dX) and of U.
template <int DK, int PO> struct Exchange {
  uint4 S[DK / 16][3][32];
  uint4 X[4][3][32];
  uint4 W[4][3][32];
  uint4 U[4][PO][32];
};
template <typename T> __host__ __device__ constexpr int strip_ld(int groups) { return 16 * groups + 16 / (int)sizeof(T); }
template <typename T, int DK, int PP> __host__ __device__ constexpr size_t stage_bytes(int groups) {
  return sizeof(Stage<T, DK, PP>) + kC * strip_ld<T>(groups) * sizeof(T);
}

// A chunk's operands into a stage, by the threads `tid` of `nthr`.
struct Fetch {
  const void *k, *q, *x;  // the chunk's first rows; q may be null
  long long ks, qs, xs;   // row strides
  int n, dk, w;           // rows, elements of a row of k and q, of x
  bool vec_k, vec_x;
  const bf16 *T, *P;      // P may be null
  const float* vec;
};
template <typename T, int DK, int PP>
__device__ __forceinline__ void fetch_chunk(Stage<T, DK, PP>& s, const Fetch& f, int ldx, int cols, int tid, int nthr) {
  constexpr int LD = Dims<T, DK>::kLdK;
  load_rows<T>(s.k, LD, static_cast<const T*>(f.k), f.ks, f.n, f.dk, DK, f.vec_k, tid, nthr);
  if (f.q) load_rows<T>(s.q, LD, static_cast<const T*>(f.q), f.qs, f.n, f.dk, DK, f.vec_k, tid, nthr);
  load_rows<T>(reinterpret_cast<T*>(&s + 1), ldx, static_cast<const T*>(f.x), f.xs, f.n, f.w, cols, f.vec_x, tid, nthr);
#pragma unroll 4
  for (int i = tid; i < 3 * kTri / 8; i += nthr) cp_async16(s.Tm + 8 * i, f.T + 8 * i, true);
  if (f.P)
#pragma unroll 4
    for (int i = tid; i < PP * kTri / 8; i += nthr) cp_async16(s.P + 8 * i, f.P + 8 * i, true);
  for (int i = tid; i < kVec / 4; i += nthr) cp_async16(s.vec + 4 * i, f.vec + 4 * i, true);
  cp_async_commit();
}

// Rows r0 .. r0 + 8 N - 1 of 16 columns from v0 of a [dk, dv] matrix, transposed.
template <int N> __device__ __forceinline__ void state_load(float (&S)[N][4], const float* p, int r0, int v0, int dk, int dv, int lane) {
  const int g = lane >> 2, c2 = 2 * (lane & 3);
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = r0 + 8 * n + c2 + (e & 1), x = v0 + g + 8 * (e >> 1);
      S[n][e] = (p && r < dk && x < dv) ? p[(long long)r * dv + x] : 0.f;
    }
}
template <int N> __device__ __forceinline__ void state_store(const float (&S)[N][4], float* p, int r0, int v0, int dk, int dv, int lane) {
  const int g = lane >> 2, c2 = 2 * (lane & 3);
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = r0 + 8 * n + c2 + (e & 1), x = v0 + g + 8 * (e >> 1);
      if (r < dk && x < dv) p[(long long)r * dv + x] = S[n][e];
    }
}
template <int N> __device__ __forceinline__ void state_get(float (&S)[N][4], const float4* p) {
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const float4 x = p[n * 32];
    S[n][0] = x.x; S[n][1] = x.y; S[n][2] = x.z; S[n][3] = x.w;
  }
}
template <int N> __device__ __forceinline__ void state_snap(const float (&S)[N][4], float4* p) {
#pragma unroll
  for (int n = 0; n < N; ++n) p[n * 32] = make_float4(S[n][0], S[n][1], S[n][2], S[n][3]);
}

// What a group's warps hold and how they meet.
template <int KS> __device__ __forceinline__ void group_sync(int group) {
  if constexpr (KS > 1)
    named_bar_sync(1 + group, 32 * KS);
  else
    __syncwarp();
}

// The passes, forward (state_pass) and backward (bwd_state_pass).  What bounds them is the chain
// K S -> X -> U -> S of each chunk on the tensor cores: per chunk and 16 value columns of a 128-row
// state 692 products of 16 x 8 x 16 with outputs (192 K S, 128 Q S, 120 T X, 60 P U, 192 K^T U; blocks
// above the diagonal are skipped), 8 cycles each on one of four sub-cores.  KS 1: 128 (b, h) x
// 64 chunks in 520 us, the tensor pipe 48 % of the time active; two blocks to an SM, so that one's
// loads and conversions run beside the other's products (one block of eight warps: 650 us, its warps
// all do the same at the same time).  KS 4: 8 (b, h) x 512 chunks in 1170 us, 2.3 us a chunk, of
// which products are 0.7 us; one warp per sub-core leaves every latency open.  Warps that only copy
// took the copies (3500 of 7300 cycles) off that chain; a bulk copy per row by one warp cost more
// (2.2 times the whole pass), for the row count of such copies.

// What a pass over the chunks of a segment leaves behind.
enum Pass {
  kPassOut,   // outputs, and S after the row's last chunk
  kPassSnap,  // the states before the chunks, for the gradients
  kPassSeg    // segS: the state after the segment, from S where it is the first and from 0 in the others; segA:
              // what the segment makes of each unit vector (value columns past nw: v = 0, S = I)
};

// One block: `groups` x 16 value columns of one segment of one (b, h).
template <typename T, int DK, int KS, int MODE, int PP>
__device__ __forceinline__ void state_pass(const ChunkArgs& a, int vblock, int seg, int h, int b) {
  constexpr bool OUT = MODE == kPassOut;
  constexpr int LD = Dims<T, DK>::kLdK, PI = Dims<T, DK>::kIn, PO = Dims<T, DK>::kOut;
  constexpr int NB = 4 / KS, ND = DK / KS / 8;  // token blocks and state tiles of a warp
  typedef Stage<T, DK, PP> St;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  const int tid = threadIdx.x, nthr = blockDim.x, warp = tid >> 5, lane = tid & 31, c2 = 2 * (lane & 3);
  const int group = warp / KS, ks = warp % KS, ldv = strip_ld<T>(a.groups), nw = (a.dv + 15) >> 4;
  const int wg = vblock * a.groups + group;  // 16 columns from v0
  const int v0 = 16 * wg, vb = 16 * vblock * a.groups, vs = 16 * group;
  const int hk = h / a.group;
  const size_t stage = stage_bytes<T, DK, PP>(a.groups);
  Exchange<DK, PO>& ex = reinterpret_cast<Exchange<DK, PO>*>(smem_raw + a.stages * stage)[KS > 1 ? group : 0];
  const long long len = row_len(a, b), bh = (long long)b * a.H + h;
  const int all = (int)min((long long)a.nc, max(0LL, (len + kC - 1) / kC - a.c0));  // the row's chunks
  const int first = seg * a.seg, nc = min(a.seg, all - first);
  if (nc <= 0 || (MODE == kPassSeg && first + nc == all)) return;  // nothing follows a row's last segment
  const T* q = static_cast<const T*>(a.q) + b * a.qs[0] + hk * a.qs[1];
  const T* k = static_cast<const T*>(a.k) + b * a.ks[0] + hk * a.ks[1];
  const T* v = static_cast<const T*>(a.v) + b * a.vs[0] + h * a.vs[1] + vb;
  T* out = OUT ? static_cast<T*>(a.out) + b * a.os[0] + h * a.os[1] + vb : nullptr;
  const int w_in = min(16 * a.groups, a.dv - vb);
  auto fetch = [&](int i) {
    if (tid < a.first_loader) return;
    const long long t0 = ((long long)a.c0 + first + i) * kC, at = bh * a.nc + first + i;
    const Fetch f = {k + t0 * a.ks[2], OUT ? q + t0 * a.qs[2] : nullptr, v + t0 * a.vs[2], a.ks[2], a.qs[2], a.vs[2],
                     chunk_len(len, (long long)a.c0 + first + i), a.dk, w_in, a.vec_k, a.vec_v, a.T + at * 3 * kTri,
                     OUT ? a.P + at * PP * kTri : nullptr, a.vec + at * kVec};
    fetch_chunk<T, DK, PP>(*reinterpret_cast<St*>(smem_raw + (a.stages == 2 ? i & 1 : 0) * stage), f, ldv, 16 * a.groups,
                           tid - a.first_loader, nthr - a.first_loader);
  };
  const bool unit = MODE == kPassSeg && wg >= nw;  // columns of the identity
  const bool live = group < a.groups && wg < nw + (MODE == kPassSeg && seg > 0 ? DK / 16 : 0);
  // a warp's tiles of 8 tokens: all of them (KS 1), or tiles ks and 7 - ks, so that the triangular products balance
  auto tile = [&](int x, int y) { return KS == 1 ? 2 * x + y : y ? 7 - ks : ks; };
  float S[ND][4];
  float4* before = a.segS + (((bh * a.nseg + seg) * nw + wg) * (DK / 8) + ks * ND) * 32 + lane;
  if (MODE != kPassSeg && a.nseg > 1 && nc < all) {
    if (live) state_get<ND>(S, before);
  } else {
    const float* from = MODE == kPassSeg && seg > 0 ? nullptr : a.S ? a.S : a.S0;
    state_load<ND>(S, from ? from + bh * a.dk * a.dv : nullptr, ks * DK / KS, v0, a.dk, a.dv, lane);
    if (unit) {
#pragma unroll
      for (int n = 0; n < ND; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          S[n][e] = ks * DK / KS + 8 * n + c2 + (e & 1) == 16 * (wg - nw) + (lane >> 2) + 8 * (e >> 1) ? 1.f : 0.f;
    } else if (MODE == kPassSeg && seg == 0 && live) {
      state_snap<ND>(S, before);
    }
  }
  bool cleared = false;  // by a token of the segment
  fetch(0);
  for (int i = 0; i < nc; ++i) {
    if constexpr (KS > 1)
      if (live)
#pragma unroll
        for (int kk = 0; kk < ND / 2; ++kk)
          put_frag<3>(ex.S[ks * (ND / 2) + kk][0], from_acc<3>(S[2 * kk], S[2 * kk + 1]), lane);
    cp_async_wait<0>();
    __syncthreads();
    if (a.stages == 2 && i + 1 < nc) fetch(i + 1);
    St& s = *reinterpret_cast<St*>(smem_raw + (a.stages == 2 ? i & 1 : 0) * stage);
    T* sv = reinterpret_cast<T*>(&s + 1);
    auto vec2 = [&](int which, int t) { return *reinterpret_cast<const float2*>(s.vec + 64 * which + 8 * t + c2); };
    const float full = s.vec[192];
    if (MODE == kPassSeg) cleared |= __float_as_uint(full) >> 31;
    if (live) {
      if (MODE == kPassSnap) state_snap<ND>(S, a.snap + (((bh * a.nc + first + i) * nw + wg) * (DK / 8) + ks * ND) * 32 + lane);
      // R^T = S^T K^T, Y^T = S^T Q^T
      float R[NB][2][4] = {}, Y[NB][2][4] = {}, lo[NB][2][4] = {};
      float yl[NB][2][4] = {};  // low order sums of Y, where it is not rounded to bf16 in the end
#pragma unroll
      for (int kk = 0; kk < DK / 16; ++kk) {
        AFrag<3> fs;
        if constexpr (KS > 1)
          fs = get_frag<3>(ex.S[kk][0], lane);
        else
          fs = from_acc<3>(S[2 * kk], S[2 * kk + 1]);
#pragma unroll
        for (int x = 0; x < NB; ++x) {
          mma2(R[x][0], R[x][1], lo[x][0], lo[x][1], fs, load_b_k2(s.k, LD, tile(x, 0), tile(x, 1), 16 * kk, lane));
          if (OUT) {
            AFrag<PO> fo;
#pragma unroll
            for (int p = 0; p < PO; ++p)
#pragma unroll
              for (int y = 0; y < 4; ++y) fo.r[p][y] = fs.r[p][y];
            const auto fq = load_b_k2(s.q, LD, tile(x, 0), tile(x, 1), 16 * kk, lane);
            if constexpr (PI > 1)
              mma2(Y[x][0], Y[x][1], yl[x][0], yl[x][1], fo, fq);
            else
              mma2(Y[x][0], Y[x][1], fo, fq);
          }
        }
      }
      if (__builtin_expect(__float_as_uint(full) >> 31, 0)) {
        // A token of the chunk clears the state: a column of S that is not finite (every product with it is not) ends
        // there.  The tokens before it have no answer; as zeros they leave nothing behind the clear, as they should.
#pragma unroll
        for (int x = 0; x < NB; ++x)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float2 gam = vec2(0, tile(x, y));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float gm = e & 1 ? gam.y : gam.x;
              const bool after = __float_as_uint(gm) >> 31;
              if (!isfinite(gm * (R[x][y][e] + lo[x][y][e]))) {
                R[x][y][e] = lo[x][y][e] = 0.f;
                if (OUT && !after) Y[x][y][e] = __int_as_float(0x7fffffff);
              }
              if (OUT && after && !isfinite(Y[x][y][e] + yl[x][y][e])) Y[x][y][e] = yl[x][y][e] = 0.f;
            }
          }
#pragma unroll
        for (int x = 0; x < ND; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) S[x][e] = 0.f;
      }
      // X^T = beta (V^T - gamma R^T), in R's place
#pragma unroll
      for (int x = 0; x < NB; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int t = tile(x, y);
          const float2 gam = vec2(0, t), be = vec2(2, t);
          float v[4];
          load_tile_t(v, sv + 8 * t * ldv + vs, ldv, lane);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            R[x][y][e] = (e & 1 ? be.y : be.x) * (v[e] - (e & 1 ? gam.y : gam.x) * (R[x][y][e] + lo[x][y][e]));
            lo[x][y][e] = 0.f;
          }
          if constexpr (KS > 1) put_tile<3>(ex.X[t >> 1][0], R[x][y], t, lane);
        }
      if constexpr (KS > 1) group_sync<KS>(group);
      // U^T = X^T T^T
      float U[NB][2][4] = {};
      if constexpr (KS > 1) {  // every fragment first: the loads overlap, only the products branch
        AFrag<3> fx[4];
        BFrag<3> ft[4];
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          fx[kk] = get_frag<3>(ex.X[kk][0], lane);
          ft[kk] = load_tri_k2<3>(s.Tm, tile(0, 0), tile(0, 1), kk, lane);
        }
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          if (kk <= tile(0, 0) >> 1)
            mma2(U[0][0], U[0][1], lo[0][0], lo[0][1], fx[kk], ft[kk]);
          else if (kk <= tile(0, 1) >> 1)
            mma1(U[0][1], lo[0][1], fx[kk], ft[kk], 1);
        }
      } else {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const AFrag<3> fx = from_acc<3>(R[kk][0], R[kk][1]);
#pragma unroll
          for (int x = kk; x < NB; ++x) mma2(U[x][0], U[x][1], lo[x][0], lo[x][1], fx, load_tri_k<3>(s.Tm, x, kk, lane));
        }
      }
      AFrag<3> fw[4];   // rho U
      AFrag<PO> fu[4];  // U
#pragma unroll
      for (int x = 0; x < NB; ++x) {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int t = tile(x, y);
#pragma unroll
          for (int e = 0; e < 4; ++e) U[x][y][e] += lo[x][y][e];
          if constexpr (OUT && KS > 1) put_tile<PO>(ex.U[t >> 1][0], U[x][y], t, lane);
        }
        if constexpr (OUT && KS == 1) fu[x] = from_acc<PO>(U[x][0], U[x][1]);
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int t = tile(x, y);
          const float2 rho = vec2(1, t);
#pragma unroll
          for (int e = 0; e < 4; ++e) U[x][y][e] *= e & 1 ? rho.y : rho.x;
          if constexpr (KS > 1) put_tile<3>(ex.W[t >> 1][0], U[x][y], t, lane);
        }
        if constexpr (KS == 1) fw[x] = from_acc<3>(U[x][0], U[x][1]);
      }
      if constexpr (KS > 1) {
        group_sync<KS>(group);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) fw[kk] = get_frag<3>(ex.W[kk][0], lane);
      }
      if (OUT) {
        // O^T = scale (gamma Y^T + U^T P^T)
#pragma unroll
        for (int x = 0; x < NB; ++x)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float2 gam = vec2(0, tile(x, y));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              Y[x][y][e] = (e & 1 ? gam.y : gam.x) * (PI > 1 ? Y[x][y][e] + yl[x][y][e] : Y[x][y][e]);
              yl[x][y][e] = 0.f;
            }
          }
        if constexpr (KS > 1) {
          BFrag<PO> fp[4];
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            fu[kk] = get_frag<PO>(ex.U[kk][0], lane);
            fp[kk] = load_tri_k2<PO>(s.P, tile(0, 0), tile(0, 1), kk, lane);
          }
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            if (kk <= tile(0, 0) >> 1)
              mma2(Y[0][0], Y[0][1], yl[0][0], yl[0][1], fu[kk], fp[kk]);
            else if (kk <= tile(0, 1) >> 1)
              mma1(Y[0][1], yl[0][1], fu[kk], fp[kk], 1);
          }
        } else {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int x = kk; x < NB; ++x) {
              if constexpr (PI > 1)
                mma2(Y[x][0], Y[x][1], yl[x][0], yl[x][1], fu[kk], load_tri_k<PO>(s.P, x, kk, lane));
              else
                mma2(Y[x][0], Y[x][1], fu[kk], load_tri_k<PO>(s.P, x, kk, lane));
            }
        }
        __syncwarp();  // every lane has taken its v
        const int n = chunk_len(len, (long long)a.c0 + first + i), w = min(16, a.dv - v0);
        T* o = out + ((long long)a.c0 + first + i) * kC * a.os[2] + vs;
#pragma unroll
        for (int x = 0; x < NB; ++x)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
#pragma unroll
            for (int e = 0; e < 4; ++e) Y[x][y][e] = a.scale * (KS > 1 || PI > 1 ? Y[x][y][e] + yl[x][y][e] : Y[x][y][e]);
            store_tile_t(sv + 8 * tile(x, y) * ldv + vs, ldv, Y[x][y], lane);
          }
        __syncwarp();
        auto token = [&](int r) { return KS == 1 ? r : 8 * tile(0, r >> 3) + (r & 7); };  // of the warp's row r
        if (a.vec_o) {
          constexpr int V = 16 / sizeof(T), per = 16 / V;
#pragma unroll
          for (int x = lane; x < 16 * NB * per; x += 32) {
            const int t = token(x / per), y = (x % per) * V;
            if (t < n && y < w) *reinterpret_cast<uint4*>(o + t * a.os[2] + y) = *reinterpret_cast<const uint4*>(sv + t * ldv + vs + y);
          }
        } else {
          for (int x = lane; x < 16 * NB * 16; x += 32) {
            const int t = token(x >> 4), y = x & 15;
            if (t < n && y < w) o[t * a.os[2] + y] = sv[t * ldv + vs + y];
          }
        }
      }
      // S^T = Gamma S^T + (rho U)^T K
#pragma unroll
      for (int np = 0; np < ND / 2; ++np) {
        float hi[2][4] = {}, lw[2][4] = {};
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma2(hi[0], hi[1], lw[0], lw[1], fw[kk], load_b_n<PI>(s.k, LD, 16 * kk, ks * (DK / KS) + 16 * np, lane));
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int e = 0; e < 4; ++e) S[2 * np + y][e] = fmaf(full, S[2 * np + y][e], hi[y][e] + lw[y][e]);
      }
    }
    if (a.stages == 1) {
      __syncthreads();
      if (i + 1 < nc) fetch(i + 1);
    }
  }
  if (OUT && live && first + nc == all) state_store<ND>(S, a.S + bh * a.dk * a.dv, ks * DK / KS, v0, a.dk, a.dv, lane);
  if (MODE == kPassSeg && live) {
    if (unit && wg == nw && ks == 0 && lane == 0)  // in segment 0's place, which no segment takes
      reinterpret_cast<float*>(a.segA + bh * a.nseg * (DK / 16) * (DK / 8) * 32)[seg] = cleared ? 1.f : 0.f;
    if (unit)
      state_snap<ND>(S, a.segA + (((bh * a.nseg + seg) * (DK / 16) + wg - nw) * (DK / 8) + ks * ND) * 32 + lane);
    else if (seg + 1 < a.nseg)
      state_snap<ND>(S, before + (long long)nw * (DK / 8) * 32);
  }
}

// The gradient of the state from a segment's last chunk to its first.  SEG: from dS where it is the
// row's last and from 0 in the others, to segD of the segment before.
template <typename T, int DK, int KS, bool SEG>
__device__ __forceinline__ void bwd_state_pass(const ChunkArgs& a, int vblock, int seg, int h, int b) {
  constexpr int LD = Dims<T, DK>::kLdK, PI = Dims<T, DK>::kIn, PO = Dims<T, DK>::kOut;
  constexpr int NB = 4 / KS, ND = DK / KS / 8;
  typedef Stage<T, DK, 3> St;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  const int tid = threadIdx.x, nthr = blockDim.x, warp = tid >> 5, lane = tid & 31, c2 = 2 * (lane & 3);
  const int group = warp / KS, ks = warp % KS, ldv = strip_ld<T>(a.groups), nw = (a.dv + 15) >> 4;
  const int wg = vblock * a.groups + group;
  const int v0 = 16 * wg, vb = 16 * vblock * a.groups, vs = 16 * group;
  const int hk = h / a.group;
  const size_t stage = stage_bytes<T, DK, 3>(a.groups);
  Exchange<DK, PO>& ex = reinterpret_cast<Exchange<DK, PO>*>(smem_raw + a.stages * stage)[KS > 1 ? group : 0];
  const long long len = row_len(a, b), bh = (long long)b * a.H + h;
  const int all = (int)min((long long)a.nc, (len + kC - 1) / kC);  // the row's chunks
  const int first = seg * a.seg, nc = min(a.seg, all - first);
  if (SEG ? nc <= 0 || seg == 0 : nc <= 0 && seg > 0) return;
  const T* q = static_cast<const T*>(a.q) + b * a.qs[0] + hk * a.qs[1];
  const T* k = static_cast<const T*>(a.k) + b * a.ks[0] + hk * a.ks[1];
  const T* d_out = static_cast<const T*>(a.d_out) + b * a.os[0] + h * a.os[1] + vb;
  const int w_in = min(16 * a.groups, a.dv - vb);
  auto fetch = [&](int i) {
    if (tid < a.first_loader) return;
    const long long t0 = (long long)(first + i) * kC, at = bh * a.nc + first + i;
    const Fetch f = {k + t0 * a.ks[2], q + t0 * a.qs[2], d_out + t0 * a.os[2], a.ks[2], a.qs[2], a.os[2], chunk_len(len, first + i),
                     a.dk, w_in, a.vec_k, a.vec_o, a.T + at * 3 * kTri, a.P + at * 3 * kTri, a.vec + at * kVec};
    fetch_chunk<T, DK, 3>(*reinterpret_cast<St*>(smem_raw + (a.stages == 2 ? i & 1 : 0) * stage), f, ldv, 16 * a.groups,
                          tid - a.first_loader, nthr - a.first_loader);
  };
  const bool live = group < a.groups && wg < nw;
  auto tile = [&](int x, int y) { return KS == 1 ? 2 * x + y : y ? 7 - ks : ks; };
  float S[ND][4];
  const bool last = first + nc >= all;
  float4* after = a.segD + (((bh * a.nseg + seg) * nw + wg) * (DK / 8) + ks * ND) * 32 + lane;
  if (!SEG && !last) {
    if (live) state_get<ND>(S, after);
  } else {
    state_load<ND>(S, a.dS && last ? a.dS + bh * a.dk * a.dv : nullptr, ks * DK / KS, v0, a.dk, a.dv, lane);
  }
  if (nc > 0) fetch(nc - 1);
  for (int i = nc - 1; i >= 0; --i) {
    if constexpr (KS > 1)
      if (live)
#pragma unroll
        for (int kk = 0; kk < ND / 2; ++kk)
          put_frag<3>(ex.S[ks * (ND / 2) + kk][0], from_acc<3>(S[2 * kk], S[2 * kk + 1]), lane);
    cp_async_wait<0>();
    __syncthreads();
    if (a.stages == 2 && i > 0) fetch(i - 1);
    St& s = *reinterpret_cast<St*>(smem_raw + (a.stages == 2 ? i & 1 : 0) * stage);
    const T* sd = reinterpret_cast<const T*>(&s + 1);
    auto vec2 = [&](int which, int t) { return *reinterpret_cast<const float2*>(s.vec + 64 * which + 8 * t + c2); };
    if (live) {
      if (!SEG) state_snap<ND>(S, a.dsnap + (((bh * a.nc + first + i) * nw + wg) * (DK / 8) + ks * ND) * 32 + lane);
      // dU^T = scale dO^T P + rho (dS^T K^T)
      float U[NB][2][4] = {}, W[NB][2][4] = {}, lo[NB][2][4] = {}, lw[NB][2][4] = {};
#pragma unroll
      for (int kk = 0; kk < DK / 16; ++kk) {
        AFrag<3> fs;
        if constexpr (KS > 1)
          fs = get_frag<3>(ex.S[kk][0], lane);
        else
          fs = from_acc<3>(S[2 * kk], S[2 * kk + 1]);
#pragma unroll
        for (int x = 0; x < NB; ++x)
          mma2(W[x][0], W[x][1], lw[x][0], lw[x][1], fs, load_b_k2(s.k, LD, tile(x, 0), tile(x, 1), 16 * kk, lane));
      }
      if constexpr (KS > 1) {  // every fragment first: the loads overlap, only the products branch
        AFrag<PI> fd[4];
        BFrag<3> fp[4];
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          fd[kk] = load_a_m<PI>(sd, ldv, 16 * kk, vs, lane);
          fp[kk] = load_tri_n2<3>(s.P, tile(0, 0), tile(0, 1), kk, lane);
        }
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          if (kk >= tile(0, 1) >> 1)
            mma2(U[0][0], U[0][1], lo[0][0], lo[0][1], fd[kk], fp[kk]);
          else if (kk >= tile(0, 0) >> 1)
            mma1(U[0][0], lo[0][0], fd[kk], fp[kk], 0);
        }
      } else {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const AFrag<PI> fd = load_a_m<PI>(sd, ldv, 16 * kk, vs, lane);
#pragma unroll
          for (int x = 0; x <= kk; ++x)
            if (x < NB) mma2(U[x][0], U[x][1], lo[x][0], lo[x][1], fd, load_tri_n<3>(s.P, kk, x, lane));
        }
      }
#pragma unroll
      for (int x = 0; x < NB; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int t = tile(x, y);
          const float2 rho = vec2(1, t);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            U[x][y][e] = a.scale * (U[x][y][e] + lo[x][y][e]) + (e & 1 ? rho.y : rho.x) * (W[x][y][e] + lw[x][y][e]);
            W[x][y][e] = lo[x][y][e] = 0.f;
          }
          if constexpr (KS > 1) put_tile<3>(ex.X[t >> 1][0], U[x][y], t, lane);
        }
      if constexpr (KS > 1) group_sync<KS>(group);
      // dX^T = dU^T T, then -beta gamma dX^T
      if constexpr (KS > 1) {
        AFrag<3> fx[4];
        BFrag<3> ft[4];
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          fx[kk] = get_frag<3>(ex.X[kk][0], lane);
          ft[kk] = load_tri_n2<3>(s.Tm, tile(0, 0), tile(0, 1), kk, lane);
        }
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          if (kk >= tile(0, 1) >> 1)
            mma2(W[0][0], W[0][1], lo[0][0], lo[0][1], fx[kk], ft[kk]);
          else if (kk >= tile(0, 0) >> 1)
            mma1(W[0][0], lo[0][0], fx[kk], ft[kk], 0);
        }
      } else {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const AFrag<3> fx = from_acc<3>(U[kk][0], U[kk][1]);
#pragma unroll
          for (int x = 0; x <= kk; ++x)
            if (x < NB) mma2(W[x][0], W[x][1], lo[x][0], lo[x][1], fx, load_tri_n<3>(s.Tm, kk, x, lane));
        }
      }
      AFrag<3> fw[4];
#pragma unroll
      for (int x = 0; x < NB; ++x) {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int t = tile(x, y);
          const float2 gam = vec2(0, t), be = vec2(2, t);
          const float f[2] = {-be.x * gam.x, -be.y * gam.y};
#pragma unroll
          for (int e = 0; e < 4; ++e) W[x][y][e] = f[e & 1] * (W[x][y][e] + lo[x][y][e]);
          if constexpr (KS > 1) put_tile<3>(ex.W[t >> 1][0], W[x][y], t, lane);
        }
        if constexpr (KS == 1) fw[x] = from_acc<3>(W[x][0], W[x][1]);
      }
      AFrag<3> fd[4];
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) fd[kk] = load_a_m_scaled<3>(sd, ldv, 16 * kk, vs, lane, s.vec + 16 * kk, a.scale);
      if constexpr (KS > 1) {
        group_sync<KS>(group);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) fw[kk] = get_frag<3>(ex.W[kk][0], lane);
      }
      const float full = s.vec[192];
#pragma unroll
      for (int np = 0; np < ND / 2; ++np) {
        float hi[2][4] = {}, l2[2][4] = {};
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          mma2(hi[0], hi[1], l2[0], l2[1], fw[kk], load_b_n<PI>(s.k, LD, 16 * kk, ks * (DK / KS) + 16 * np, lane));
          mma2(hi[0], hi[1], l2[0], l2[1], fd[kk], load_b_n<PI>(s.q, LD, 16 * kk, ks * (DK / KS) + 16 * np, lane));
        }
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int e = 0; e < 4; ++e) S[2 * np + y][e] = fmaf(full, S[2 * np + y][e], hi[y][e] + l2[y][e]);
      }
    }
    if (a.stages == 1) {
      __syncthreads();
      if (i > 0) fetch(i - 1);
    }
  }
  if (SEG && live) state_snap<ND>(S, after - (long long)nw * (DK / 8) * 32);
  if (!SEG && a.dS0 && seg == 0 && live) state_store<ND>(S, a.dS0 + bh * a.dk * a.dv, ks * DK / KS, v0, a.dk, a.dv, lane);
}

// Threads at most: two (KS 4) or four (KS 1) groups and four copying warps.
constexpr int state_threads(int KS) { return KS == 4 ? 384 : 256; }

// Blocks: gridDim.x = segments x blocks per segment.
template <typename T, int DK, int KS, int MODE> __global__ void __launch_bounds__(state_threads(KS)) forward_kernel(const ChunkArgs a) {
  state_pass<T, DK, KS, MODE, Dims<T, DK>::kOut>(a, blockIdx.x % a.blocks, blockIdx.x / a.blocks, blockIdx.y, blockIdx.z);
}
// The two passes of the backward do not depend on each other: the first half of the grid (z) runs the
// states forward, the second their gradients backward.  (Neighbouring blocks of the two on one SM
// evict each other's instructions: "no instruction" was a fifth of the stalls at 128 (b, h).)
template <typename T, int DK, int KS, bool SEG> __global__ void __launch_bounds__(state_threads(KS)) both_kernel(const ChunkArgs a) {
  const int vblock = blockIdx.x % a.blocks, seg = blockIdx.x / a.blocks;
  if ((int)blockIdx.z >= a.B)
    bwd_state_pass<T, DK, KS, SEG>(a, vblock, seg, blockIdx.y, blockIdx.z - a.B);
  else
    state_pass<T, DK, KS, SEG ? kPassSeg : kPassSnap, 3>(a, vblock, seg, blockIdx.y, blockIdx.z);
}

// The states between segments from what each makes of a zero state (in segS, segD) and of the unit
// vectors: S_(i+1) = A_i S_i + B_i; odd blocks (backward): D_(i-1) = A_i^T D_i + C_i.  A block: 16
// value columns of one (b, h), four warps with DK / 4 key rows each.
template <int DK> __global__ void __launch_bounds__(128) combine_kernel(const ChunkArgs a, int both) {
  constexpr int ND = DK / 32, NS = DK / 16;
  __shared__ uint4 ex[NS][3][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = (a.dv + 15) >> 4;
  const bool back = both && (blockIdx.x & 1);
  const int wg = both ? blockIdx.x >> 1 : blockIdx.x;
  const long long bh = (long long)blockIdx.z * a.H + blockIdx.y, len = row_len(a, blockIdx.z);
  const int all = (int)min((long long)a.nc, max(0LL, (len + kC - 1) / kC - a.c0)), n = (all + a.seg - 1) / a.seg;  // live segments
  if (n < 3) return;
  const long long step = (long long)nw * (DK / 8) * 32;
  float4* at = (back ? a.segD : a.segS) + ((bh * a.nseg * nw + wg) * (DK / 8) + warp * ND) * 32 + lane;
  const float4* A = a.segA + bh * a.nseg * NS * (DK / 8) * 32 + lane;
  float S[ND][4];
  state_get<ND>(S, at + (back ? n - 2 : 1) * step);
  // forward: the segments (32 at most) that clear the state
  const unsigned clears = __ballot_sync(0xffffffffu, !back && lane > 0 && lane < n - 1 && reinterpret_cast<const float*>(A - lane)[lane] != 0.f);
  for (int k = 1; k < n - 1; ++k) {
    const int i = back ? n - 1 - k : k;  // the segment that is passed
    if (clears >> i & 1) {  // A_i = 0, and S_i may not be finite
      state_get<ND>(S, at + (i + 1) * step);
      continue;
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < ND / 2; ++x) put_frag<3>(ex[warp * (ND / 2) + x][0], from_acc<3>(S[2 * x], S[2 * x + 1]), lane);
    __syncthreads();
    const float4* Ai = A + (long long)i * NS * (DK / 8) * 32;
    float4* to = at + (back ? i - 1 : i + 1) * step;
    float hi[ND][4], lo[ND][4] = {};
    state_get<ND>(hi, to);
#pragma unroll 2
    for (int kk = 0; kk < NS; ++kk) {
      const AFrag<3> f = get_frag<3>(ex[kk][0], lane);
#pragma unroll
      for (int x = 0; x < ND / 2; ++x) {
        const int np = warp * (ND / 2) + x;
        BFrag<3> m;
        if (!back) {  // B[k = column of A][n = its row]
          m = b_from_acc<3>(Ai[(kk * (DK / 8) + 2 * np) * 32], Ai[(kk * (DK / 8) + 2 * np + 1) * 32]);
        } else {  // B[k = row of A][n = its column]
          const float4 t0 = Ai[(np * (DK / 8) + 2 * kk) * 32], t1 = Ai[(np * (DK / 8) + 2 * kk + 1) * 32];
          split<3>(t0.x, t0.y, m.r, 0);
          split<3>(t1.x, t1.y, m.r, 1);
          split<3>(t0.z, t0.w, m.r, 2);
          split<3>(t1.z, t1.w, m.r, 3);
        }
        mma2(hi[2 * x], hi[2 * x + 1], lo[2 * x], lo[2 * x + 1], f, m);
      }
    }
#pragma unroll
    for (int x = 0; x < ND; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) S[x][e] = hi[x][e] + lo[x][e];
    state_snap<ND>(S, to);
  }
}

// ------------------------------------------------------------------ gradients
constexpr int kLdU = 132;
template <typename T, int DK> struct GradSmem {
  T k[kC * Dims<T, DK>::kLdK];
  T q[kC * Dims<T, DK>::kLdK];
  T d[kC * Dims<T, 128>::kLdK];  // d_out
  float U[kC * kLdU];
  float X[kC * kLdU];  // dX
  float Tm[kC * kLdT];  // T, then M + M^T
  float P[kC * kLdT];   // P, then N = dP e^(G_i - G_j)
  float vec[kVec];
  float2 G[kC];
  float tok[kMaxWarps][3][kC];
  float rowP[kC], rowA[kC], rowB[kC];
  float col[kMaxWarps][kC];
  float sdot[kMaxWarps];
};

// Sum over the rows of a warp's [16 x 64] fragment: token values x[2 n + e] to dst[64].
__device__ __forceinline__ void sum_rows(float (&x)[16], float* dst, int lane) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[i], o);
  if (lane < 4)
#pragma unroll
    for (int i = 0; i < 16; ++i) dst[8 * (i >> 1) + 2 * lane + (i & 1)] = x[i];
}

// dg_t = sum over i >= t of x_i, the exponents' derivatives but for G_last - G_i's, and over i < t of these, e_i (all of
// them count for G_last).  Two sums, and none of them a difference: e of the last token is as large as dv is whatever the
// decays, dg e^g of that.  Tokens 2 lane, 2 lane + 1; `sum` is that of the x from 2 lane + 1 on, `before` that of the e
// before 2 lane.
__device__ __forceinline__ void decay_sums(const double (&x)[2], const double (&e)[2], double& sum, double& before, int lane) {
  sum = x[0] + x[1];
  before = e[0] + e[1];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_down_sync(0xffffffffu, sum, o), z = __shfl_up_sync(0xffffffffu, before, o);
    if (lane + o < 32) sum += y;
    if (lane >= o) before += z;
  }
  const double y = __shfl_down_sync(0xffffffffu, sum, 1), z = __shfl_up_sync(0xffffffffu, before, 1);
  sum = (lane < 31 ? y : 0.) + x[1];
  before = lane > 0 ? z : 0.;
}

// B fragment [k = value column][n = key row] of the state whose accumulator-order copy of the
// 16 value columns is p.
template <int P> __device__ __forceinline__ BFrag<P> load_b_state(const float* p, int n0, int lane) {
  BFrag<P> b;
  const int g = lane >> 2, c = lane & 3;
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float* x = p + (((n0 >> 3) + t) * 32 + (2 * c) * 4 + (g >> 1)) * 4 + 2 * h + (g & 1);
      split<P>(x[0], x[16], b.r, 2 * t + h);
    }
  return b;
}

template <typename T, int DK> __global__ void __launch_bounds__(256) grad_kernel(const ChunkArgs a) {
  constexpr int LD = Dims<T, DK>::kLdK, LDD = Dims<T, 128>::kLdK, PI = Dims<T, DK>::kIn, PO = Dims<T, DK>::kOut;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  GradSmem<T, DK>& s = *reinterpret_cast<GradSmem<T, DK>*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c2 = 2 * (lane & 3);
  const int b = blockIdx.z, hk = a.split ? blockIdx.y / a.group : blockIdx.y, nw = (a.dv + 15) >> 4;
  const int h0 = a.split ? blockIdx.y : hk * a.group, heads = a.split ? 1 : a.group;
  const int i0 = blockIdx.x;
  const long long t0 = (long long)i0 * kC;
  const int n = chunk_len(row_len(a, b), i0);
  const int rows = chunk_len(a.L, i0);  // rows of the tensors in this chunk
  T* dq = static_cast<T*>(a.dq) + (((long long)b * a.Hk + hk) * a.L + t0) * a.dk;
  T* dkk = static_cast<T*>(a.dkk) + (((long long)b * a.Hk + hk) * a.L + t0) * a.dk;
  const T zero = from_f32<T>(0.f);
  if (n == 0) {  // padding only
    for (int x = tid; x < rows * a.dk && !a.split; x += 256) dq[x] = dkk[x] = zero;
    for (int h = h0; h < h0 + heads; ++h) {
      const long long r0 = ((long long)b * a.H + h) * a.L + t0;
      for (int x = tid; x < rows * a.dv; x += 256) static_cast<T*>(a.dvv)[r0 * a.dv + x] = zero;
      if (tid < rows) a.dg[r0 + tid] = a.dbeta[r0 + tid] = 0.f;
    }
    return;
  }
  load_rows<T>(s.k, LD, static_cast<const T*>(a.k) + b * a.ks[0] + hk * a.ks[1] + t0 * a.ks[2], a.ks[2], n, a.dk, DK, a.vec_k, tid, 256);
  load_rows<T>(s.q, LD, static_cast<const T*>(a.q) + b * a.qs[0] + hk * a.qs[1] + t0 * a.qs[2], a.qs[2], n, a.dk, DK, a.vec_k, tid, 256);
  for (int hi = 0; hi < heads; ++hi) {
    const int h = h0 + hi;
    const long long bh = (long long)b * a.H + h, at = bh * a.nc + i0, r0 = bh * a.L + t0;
    load_rows<T>(s.d, LDD, static_cast<const T*>(a.d_out) + b * a.os[0] + h * a.os[1] + t0 * a.os[2], a.os[2], n, a.dv, 128, a.vec_o, tid, 256);
    load_tri_f32(s.Tm, a.T + at * 3 * kTri, tid, 256);
    load_tri_f32(s.P, a.P + at * 3 * kTri, tid, 256);
    if (tid < kVec / 4) cp_async16(s.vec + 4 * tid, a.vec + at * kVec + 4 * tid, true);
    if (tid < kC / 2) cp_async16(s.G + 2 * tid, a.G + at * kC + 2 * tid, true);
    cp_async_commit();
    cp_async_wait<0>();
    __syncthreads();
    const float4* snap = a.snap + at * nw * (DK / 8) * 32;
    const float4* dsnap = a.dsnap + at * nw * (DK / 8) * 32;
    // ---- 1: U, dX and the sums over value columns; 16 value columns per warp
    if (warp < nw) {
      float R[8][4] = {}, Y[8][4] = {}, W[8][4] = {}, dot = 0.f;
      const float4* ps = snap + warp * (DK / 8) * 32 + lane;
      const float4* pd = dsnap + warp * (DK / 8) * 32 + lane;
      // two token halves, so that the low order sums find room
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float rl[4][4] = {}, yl[4][4] = {}, wl[4][4] = {};
#pragma unroll 2
        for (int kk = 0; kk < DK / 16; ++kk) {
          const float4 s0 = ps[2 * kk * 32], s1 = ps[(2 * kk + 1) * 32], d0 = pd[2 * kk * 32], d1 = pd[(2 * kk + 1) * 32];
          if (half == 0)
            dot += s0.x * d0.x + s0.y * d0.y + s0.z * d0.z + s0.w * d0.w + s1.x * d1.x + s1.y * d1.y + s1.z * d1.z + s1.w * d1.w;
          const float sa[4] = {s0.x, s0.y, s0.z, s0.w}, sb[4] = {s1.x, s1.y, s1.z, s1.w};
          const float da[4] = {d0.x, d0.y, d0.z, d0.w}, db[4] = {d1.x, d1.y, d1.z, d1.w};
          const AFrag<3> fs = from_acc<3>(sa, sb), fd = from_acc<3>(da, db);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int np = 2 * half + x;
            const BFrag<PI> bk = load_b_k<PI>(s.k, LD, 16 * np, 16 * kk, lane);
            mma2(R[2 * np], R[2 * np + 1], rl[2 * x], rl[2 * x + 1], fs, bk);
            mma2(W[2 * np], W[2 * np + 1], wl[2 * x], wl[2 * x + 1], fd, bk);
            mma2(Y[2 * np], Y[2 * np + 1], yl[2 * x], yl[2 * x + 1], fs, load_b_k<PI>(s.q, LD, 16 * np, 16 * kk, lane));
          }
        }
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            R[4 * half + x][e] += rl[x][e];
            Y[4 * half + x][e] += yl[x][e];
            W[4 * half + x][e] += wl[x][e];
          }
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      if (lane == 0) s.sdot[warp] = dot;
      const T* v = static_cast<const T*>(a.v) + b * a.vs[0] + h * a.vs[1] + t0 * a.vs[2] + 16 * warp;
      const int w = a.dv - 16 * warp;
      // a_i = scale gamma dO.Y; then Y = V - gamma R (the error the write corrects), R stays K S
      float sum_a[16];
#pragma unroll
      for (int x = 0; x < 8; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int t = 8 * x + c2 + e;
          sum_a[2 * x + e] = a.scale * s.vec[t] *
                             (to_f32(s.d[t * LDD + 16 * warp + g]) * Y[x][e] + to_f32(s.d[t * LDD + 16 * warp + g + 8]) * Y[x][2 + e]);
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float vv = (t < n && g + 8 * r < w) ? to_f32(v[t * a.vs[2] + g + 8 * r]) : 0.f;
            Y[x][2 * r + e] = vv - s.vec[t] * R[x][2 * r + e];
          }
        }
      float U[8][4] = {}, lo[8][4] = {};
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        float xa[4], xb[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          xa[e] = s.vec[128 + 16 * kk + c2 + (e & 1)] * Y[2 * kk][e];
          xb[e] = s.vec[128 + 16 * kk + 8 + c2 + (e & 1)] * Y[2 * kk + 1][e];
        }
        const AFrag<3> fx = from_acc<3>(xa, xb);
#pragma unroll
        for (int np = 0; np < 4; ++np)
          if (np >= kk) mma2(U[2 * np], U[2 * np + 1], lo[2 * np], lo[2 * np + 1], fx, load_b_k<3>(s.Tm, kLdT, 16 * np, 16 * kk, lane));
      }
      float sum_e[16];
#pragma unroll
      for (int x = 0; x < 8; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int t = 8 * x + c2 + e;
          U[x][e] += lo[x][e];
          U[x][2 + e] += lo[x][2 + e];
          lo[x][e] = lo[x][2 + e] = 0.f;
          sum_e[2 * x + e] = s.vec[64 + t] * (W[x][e] * U[x][e] + W[x][2 + e] * U[x][2 + e]);
          s.U[t * kLdU + 16 * warp + g] = U[x][e];
          s.U[t * kLdU + 16 * warp + g + 8] = U[x][2 + e];
          U[x][e] = U[x][2 + e] = 0.f;
        }
      sum_rows(sum_e, s.tok[warp][1], lane);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        const AFrag<PI> fd = load_a_m<PI>(s.d, LDD, 16 * kk, 16 * warp, lane);
#pragma unroll
        for (int np = 0; np < 4; ++np)
          if (np <= kk) mma2(U[2 * np], U[2 * np + 1], lo[2 * np], lo[2 * np + 1], fd, load_b_n<3>(s.P, kLdT, 16 * kk, 16 * np, lane));
      }
#pragma unroll
      for (int x = 0; x < 8; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          U[x][e] = a.scale * (U[x][e] + lo[x][e]) + s.vec[64 + 8 * x + c2 + (e & 1)] * W[x][e];
          W[x][e] = lo[x][e] = 0.f;
        }
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        const AFrag<3> fu = from_acc<3>(U[2 * kk], U[2 * kk + 1]);
#pragma unroll
        for (int np = 0; np < 4; ++np)
          if (np <= kk) mma2(W[2 * np], W[2 * np + 1], lo[2 * np], lo[2 * np + 1], fu, load_b_n<3>(s.Tm, kLdT, 16 * kk, 16 * np, lane));
      }
      float sum_b[16];
#pragma unroll
      for (int x = 0; x < 8; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int t = 8 * x + c2 + e;
          W[x][e] += lo[x][e];
          W[x][2 + e] += lo[x][2 + e];
          sum_a[2 * x + e] -= s.vec[128 + t] * s.vec[t] * (W[x][e] * R[x][e] + W[x][2 + e] * R[x][2 + e]);
          sum_b[2 * x + e] = W[x][e] * Y[x][e] + W[x][2 + e] * Y[x][2 + e];
          s.X[t * kLdU + 16 * warp + g] = W[x][e];
          s.X[t * kLdU + 16 * warp + g + 8] = W[x][2 + e];
        }
      sum_rows(sum_a, s.tok[warp][0], lane);
      sum_rows(sum_b, s.tok[warp][2], lane);
    }
    __syncthreads();
    // ---- 2: dP (warps 0-3) and dA (warps 4-7), 16 rows each; dV
    {
      T* dv = static_cast<T*>(a.dvv) + r0 * a.dv;
      for (int x = tid; x < rows * a.dv; x += 256) {
        const int t = x / a.dv, y = x % a.dv;
        dv[x] = t < n ? from_f32<T>(s.vec[128 + t] * s.X[t * kLdU + y]) : zero;
      }
      const int rb = warp & 3, m0 = 16 * rb;
      const bool is_a = warp >= 4;
      float acc[4][2][4] = {}, kk2[4][2][4] = {}, lo[4][2][4] = {};
      if (is_a) {
        for (int kk = 0; kk < DK / 16; ++kk) {
          const AFrag<PI> fk = load_a_k<PI>(s.k, LD, m0, 16 * kk, lane);
#pragma unroll
          for (int cb = 0; cb < 4; ++cb)
            if (cb <= rb) mma2(kk2[cb][0], kk2[cb][1], lo[cb][0], lo[cb][1], fk, load_b_k<PI>(s.k, LD, 16 * cb, 16 * kk, lane));
        }
#pragma unroll
        for (int cb = 0; cb < 4; ++cb)
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              kk2[cb][t][e] += lo[cb][t][e];
              lo[cb][t][e] = 0.f;
            }
      }
      for (int kk = 0; kk < nw; ++kk) {
        AFrag<3> fx;
        AFrag<PI> fd;
        if (is_a)
          fx = load_a_k<3>(s.X, kLdU, m0, 16 * kk, lane);
        else
          fd = load_a_k<PI>(s.d, LDD, m0, 16 * kk, lane);
#pragma unroll
        for (int cb = 0; cb < 4; ++cb)
          if (cb <= rb) {
            const BFrag<3> fu = load_b_k<3>(s.U, kLdU, 16 * cb, 16 * kk, lane);
            if (is_a)
              mma2(acc[cb][0], acc[cb][1], lo[cb][0], lo[cb][1], fx, fu);
            else
              mma2(acc[cb][0], acc[cb][1], lo[cb][0], lo[cb][1], fd, fu);
          }
      }
      float row[2] = {}, rowb[2] = {};
#pragma unroll
      for (int cb = 0; cb < 4; ++cb)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          float col[2] = {};
          const int j = 16 * cb + 8 * t + c2;
          if (cb <= rb)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int i = m0 + g + 8 * (e >> 1), jj = j + (e & 1);
              const float x = acc[cb][t][e] + lo[cb][t][e];
              if (is_a) {
                const float dec = decay(s.G[i], s.G[jj], i > jj), be = s.vec[128 + i];
                const float ab = -x * dec * kk2[cb][t][e];
                rowb[e >> 1] += ab;
                row[e >> 1] += be * ab;
                col[e & 1] += be * ab;
                const float m = -x * be * dec;
                if (i >= jj) s.Tm[i * kLdT + jj] = m;
                if (i > jj) s.Tm[jj * kLdT + i] = m;
              } else {
                const float dp = a.scale * x, y = i > jj ? dp * s.P[i * kLdT + jj] : 0.f;
                row[e >> 1] += y;
                col[e & 1] += y;
                s.P[i * kLdT + jj] = dp * decay(s.G[i], s.G[jj], i >= jj);
              }
            }
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            col[0] += __shfl_xor_sync(0xffffffffu, col[0], o);
            col[1] += __shfl_xor_sync(0xffffffffu, col[1], o);
          }
          if (lane < 4) {
            s.col[warp][j] = col[0];
            s.col[warp][j + 1] = col[1];
          }
        }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          row[r] += __shfl_xor_sync(0xffffffffu, row[r], o);
          rowb[r] += __shfl_xor_sync(0xffffffffu, rowb[r], o);
        }
      if ((lane & 3) == 0)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          (is_a ? s.rowA : s.rowP)[m0 + g + 8 * r] = row[r];
          if (is_a) s.rowB[m0 + g + 8 * r] = rowb[r];
        }
    }
    __syncthreads();
    // ---- 3: dg, dbeta (warp 0, two tokens a lane); dQ and dK, 16 key columns per warp
    if (warp == 0) {
      double x[2], ev2[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = 2 * lane + i;
        float av = 0.f, ev = 0.f, bv = 0.f, cv = 0.f;
        for (int w = 0; w < nw; ++w) {
          av += s.tok[w][0][t];
          ev += s.tok[w][1][t];
          bv += s.tok[w][2][t];
        }
        for (int w = 0; w < 8; ++w) cv += s.col[w][t];
        x[i] = (double)av + s.rowP[t] + s.rowA[t] - cv;
        ev2[i] = ev;
        if (t < rows) a.dbeta[r0 + t] = t < n ? bv + s.rowB[t] : 0.f;
      }
      float dot = 0.f;
      for (int w = 0; w < nw; ++w) dot += s.sdot[w];
      if (lane == 31) x[1] += (double)s.vec[192] * dot;
      double sum, before;
      decay_sums(x, ev2, sum, before, lane);
      if (2 * lane < rows) a.dg[r0 + 2 * lane] = 2 * lane < n ? (float)(sum + x[0] + before) : 0.f;
      if (2 * lane + 1 < rows) a.dg[r0 + 2 * lane + 1] = 2 * lane + 1 < n ? (float)(sum + before + ev2[0]) : 0.f;
    }
    if (warp < DK / 16) {
      const int n0 = 16 * warp;
      float Q[4][2][4] = {}, K[4][2][4] = {}, ql[4][2][4] = {}, kl[4][2][4] = {};
      for (int kw = 0; kw < nw; ++kw) {
        const BFrag<PO> fs = load_b_state<PO>(reinterpret_cast<const float*>(snap + kw * (DK / 8) * 32), n0, lane);
        const BFrag<PO> fd = load_b_state<PO>(reinterpret_cast<const float*>(dsnap + kw * (DK / 8) * 32), n0, lane);
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
          const int t = 16 * mt + g;
          mma2(Q[mt][0], Q[mt][1], ql[mt][0], ql[mt][1], load_a_k<PI>(s.d, LDD, 16 * mt, 16 * kw, lane), fs);
          mma2(K[mt][0], K[mt][1], kl[mt][0], kl[mt][1],
               load_a_k<PO>(s.X, kLdU, 16 * mt, 16 * kw, lane, -s.vec[128 + t] * s.vec[t], -s.vec[136 + t] * s.vec[t + 8]), fs);
          mma2(K[mt][0], K[mt][1], kl[mt][0], kl[mt][1], load_a_k<PO>(s.U, kLdU, 16 * mt, 16 * kw, lane, s.vec[64 + t], s.vec[72 + t]), fd);
        }
      }
#pragma unroll
      for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            Q[mt][t][e] = (Q[mt][t][e] + ql[mt][t][e]) * (a.scale * s.vec[16 * mt + g + 8 * (e >> 1)]);
            ql[mt][t][e] = 0.f;
          }
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        const BFrag<PI> bk = load_b_n<PI>(s.k, LD, 16 * kk, n0, lane), bq = load_b_n<PI>(s.q, LD, 16 * kk, n0, lane);
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
          if (kk <= mt) mma2(Q[mt][0], Q[mt][1], ql[mt][0], ql[mt][1], load_a_k<PO>(s.P, kLdT, 16 * mt, 16 * kk, lane), bk);
          mma2(K[mt][0], K[mt][1], kl[mt][0], kl[mt][1], load_a_k<PO>(s.Tm, kLdT, 16 * mt, 16 * kk, lane), bk);
          if (kk >= mt) mma2(K[mt][0], K[mt][1], kl[mt][0], kl[mt][1], load_a_m<PO>(s.P, kLdT, 16 * kk, 16 * mt, lane), bq);
        }
      }
      float* acc = a.acc + ((a.split ? bh : (long long)b * a.Hk + hk) * a.nc + i0) * 2 * kC * DK;
#pragma unroll
      for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int tk = 16 * mt + g + 8 * r, x = n0 + 8 * t + c2;
            float2 yq = make_float2(Q[mt][t][2 * r] + ql[mt][t][2 * r], Q[mt][t][2 * r + 1] + ql[mt][t][2 * r + 1]);
            float2 yk = make_float2(K[mt][t][2 * r] + kl[mt][t][2 * r], K[mt][t][2 * r + 1] + kl[mt][t][2 * r + 1]);
            if (a.group > 1) {  // the same thread holds this element for every value head of the key head
              float2* pq = reinterpret_cast<float2*>(acc + tk * DK + x);
              float2* pk = reinterpret_cast<float2*>(acc + (kC + tk) * DK + x);
              if (hi > 0) {
                const float2 oq = *pq, ok = *pk;
                yq.x += oq.x; yq.y += oq.y; yk.x += ok.x; yk.y += ok.y;
              }
              if (a.split || hi + 1 < a.group) {
                *pq = yq;
                *pk = yk;
                continue;
              }
            }
            if (tk < rows) {
              const long long o = (long long)tk * a.dk + x;
              const bool in = tk < n;
              if (x < a.dk) {
                dq[o] = in ? from_f32<T>(yq.x) : zero;
                dkk[o] = in ? from_f32<T>(yk.x) : zero;
              }
              if (x + 1 < a.dk) {
                dq[o + 1] = in ? from_f32<T>(yq.y) : zero;
                dkk[o + 1] = in ? from_f32<T>(yk.y) : zero;
              }
            }
          }
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ gradients, bf16
// Bound by the tensor pipe and what feeds it: 26 thousand cycles of products in 54 thousand per chunk
// and (b, h) (pipe active 48 %), at one block of 16 warps an SM for its 217 KB of operands.  4096
// chunks in 934 us; with 8 warps that split the operands at each use 1770 us.  Products of order 2^-8
// and below have sums of their own wherever dg and dbeta come from them (all orders in one sum: 902 us,
// but dg and dbeta, relative to 64 bits, 4.9e-7 and 7.3e-7 instead of 3.0e-7 and 3.0e-7, which is what
// the formulas in fp32 give); the sums of K S and Q S and those of K dS' one after the other, so that
// they find room.
// The same with 16 warps and every fp32 operand split once, where it is made: U and dX as three
// planes [64][kLdG], T and P as they come, M + M^T and N as two.  Two warps share 16 value columns
// (then 16 key columns): token blocks 0 and 3, or 1 and 2, so that the triangular products balance.
constexpr int kLdG = 136, kPlaneG = kC * kLdG, kLdM = 72, kPlaneM = kC * kLdM;
template <int DK> struct GradSmemB {
  bf16 k[kC * (DK + 8)];
  bf16 q[kC * (DK + 8)];
  bf16 d[kPlaneG];      // d_out
  bf16 U[3 * kPlaneG];
  bf16 X[3 * kPlaneG];  // X, then dU, in fragments [strip][4][3][32] x 16 bytes; then dX
  bf16 Tm[3 * kTri];
  bf16 P[3 * kTri];     // P, then N in the first two planes
  bf16 M[2 * kPlaneM];  // v [64][kLdG], then M + M^T
  float vec[kVec];
  float2 G[kC];
  float tok[8][3][kC];
  float rowP[10][16], colP[10][16], rowA[10][16], colA[10][16], rowB[10][16];
  float sdot[16];
};

// Token sums of a warp's two blocks: x[block][tile][e] over the 16 value columns, to dst[64].
__device__ __forceinline__ void sum_tokens(float (&x)[2][2][2], float* dst, int b0, int b1, int lane) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) x[i][t][e] += __shfl_xor_sync(0xffffffffu, x[i][t][e], o);
  if (lane < 4)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int t = 0; t < 2; ++t)
        *reinterpret_cast<float2*>(dst + 16 * (i ? b1 : b0) + 8 * t + 2 * lane) = make_float2(x[i][t][0], x[i][t][1]);
}

template <int DK> __global__ void __launch_bounds__(512) grad_bf16_kernel(const ChunkArgs a) {
  constexpr int LD = DK + 8;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  GradSmemB<DK>& s = *reinterpret_cast<GradSmemB<DK>*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c2 = 2 * (lane & 3);
  const int b = blockIdx.z, hk = a.split ? blockIdx.y / a.group : blockIdx.y, nw = (a.dv + 15) >> 4;
  const int h0 = a.split ? blockIdx.y : hk * a.group, heads = a.split ? 1 : a.group;
  const int i0 = blockIdx.x;
  const long long t0 = (long long)i0 * kC;
  const int n = chunk_len(row_len(a, b), i0);
  const int rows = chunk_len(a.L, i0);  // rows of the tensors in this chunk
  bf16* dq = static_cast<bf16*>(a.dq) + (((long long)b * a.Hk + hk) * a.L + t0) * a.dk;
  bf16* dkk = static_cast<bf16*>(a.dkk) + (((long long)b * a.Hk + hk) * a.L + t0) * a.dk;
  const bf16 zero = from_f32<bf16>(0.f);
  if (n == 0) {  // padding only
    for (int x = tid; x < rows * a.dk && !a.split; x += 512) dq[x] = dkk[x] = zero;
    for (int h = h0; h < h0 + heads; ++h) {
      const long long r0 = ((long long)b * a.H + h) * a.L + t0;
      for (int x = tid; x < rows * a.dv; x += 512) static_cast<bf16*>(a.dvv)[r0 * a.dv + x] = zero;
      if (tid < rows) a.dg[r0 + tid] = a.dbeta[r0 + tid] = 0.f;
    }
    return;
  }
  const int strip = warp >> 1, half = warp & 1;
  const int blks[2] = {half ? 1 : 0, half ? 2 : 3};
  load_rows<bf16>(s.k, LD, static_cast<const bf16*>(a.k) + b * a.ks[0] + hk * a.ks[1] + t0 * a.ks[2], a.ks[2], n, a.dk, DK, a.vec_k, tid, 512);
  load_rows<bf16>(s.q, LD, static_cast<const bf16*>(a.q) + b * a.qs[0] + hk * a.qs[1] + t0 * a.qs[2], a.qs[2], n, a.dk, DK, a.vec_k, tid, 512);
  for (int hi = 0; hi < heads; ++hi) {
    const int h = h0 + hi;
    const long long bh = (long long)b * a.H + h, at = bh * a.nc + i0, r0 = bh * a.L + t0;
    load_rows<bf16>(s.d, kLdG, static_cast<const bf16*>(a.d_out) + b * a.os[0] + h * a.os[1] + t0 * a.os[2], a.os[2], n, a.dv, 128, a.vec_o, tid, 512);
    load_rows<bf16>(s.M, kLdG, static_cast<const bf16*>(a.v) + b * a.vs[0] + h * a.vs[1] + t0 * a.vs[2], a.vs[2], n, a.dv, 128, a.vec_v, tid, 512);
    for (int i = tid; i < 3 * kTri / 8; i += 512) {
      cp_async16(s.Tm + 8 * i, a.T + at * 3 * kTri + 8 * i, true);
      cp_async16(s.P + 8 * i, a.P + at * 3 * kTri + 8 * i, true);
    }
    if (tid < kVec / 4) cp_async16(s.vec + 4 * tid, a.vec + at * kVec + 4 * tid, true);
    if (tid < kC / 2) cp_async16(s.G + 2 * tid, a.G + at * kC + 2 * tid, true);
    cp_async_commit();
    const float4* snap = a.snap + at * nw * (DK / 8) * 32;
    const float4* dsnap = a.dsnap + at * nw * (DK / 8) * 32;
    cp_async_wait<0>();
    __syncthreads();
    float W[2][2][4] = {};
    // ---- 1: U, dX and the sums over value columns; 16 value columns and two token blocks per warp
    if (strip < nw) {
      float R[2][2][4] = {}, Y[2][2][4] = {}, dot = 0.f;
      const float4* ps = snap + strip * (DK / 8) * 32 + lane;
      const float4* pd = dsnap + strip * (DK / 8) * 32 + lane;
      {
        float rl[2][2][4] = {}, yl[2][2][4] = {};
        float4 s0 = ps[0], s1 = ps[32];
#pragma unroll 1
        for (int kk = 0; kk < DK / 16; ++kk) {
          const float sa[4] = {s0.x, s0.y, s0.z, s0.w}, sb[4] = {s1.x, s1.y, s1.z, s1.w};
          const AFrag<3> fs = from_acc<3>(sa, sb);
          if (kk + 1 < DK / 16) {
            s0 = ps[(2 * kk + 2) * 32];
            s1 = ps[(2 * kk + 3) * 32];
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            mma2(R[x][0], R[x][1], rl[x][0], rl[x][1], fs, load_b_k<1>(s.k, LD, 16 * blks[x], 16 * kk, lane));
            mma2(Y[x][0], Y[x][1], yl[x][0], yl[x][1], fs, load_b_k<1>(s.q, LD, 16 * blks[x], 16 * kk, lane));
          }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              R[x][t][e] += rl[x][t][e];
              Y[x][t][e] += yl[x][t][e];
            }
      }
      float lo[2][2][4] = {};
      {
        // two steps' loads in flight; S.dS' of every other step in each of the strip's two warps
        float4 d[2][2], m[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          d[i][0] = pd[2 * i * 32];
          d[i][1] = pd[(2 * i + 1) * 32];
          m[i] = ps[(2 * half + i) * 32];
        }
#pragma unroll 1
        for (int k2 = 0; k2 < DK / 32; ++k2) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int kk = 2 * k2 + i;
            const float4 d0 = d[i][0], d1 = d[i][1];
            const float da[4] = {d0.x, d0.y, d0.z, d0.w}, db[4] = {d1.x, d1.y, d1.z, d1.w};
            const AFrag<3> fd = from_acc<3>(da, db);
            if (i == half)
              dot += m[0].x * d0.x + m[0].y * d0.y + m[0].z * d0.z + m[0].w * d0.w + m[1].x * d1.x + m[1].y * d1.y + m[1].z * d1.z + m[1].w * d1.w;
            if (k2 + 1 < DK / 32) {
              d[i][0] = pd[(2 * kk + 4) * 32];
              d[i][1] = pd[(2 * kk + 5) * 32];
            }
#pragma unroll
            for (int x = 0; x < 2; ++x)
              mma2(W[x][0], W[x][1], lo[x][0], lo[x][1], fd, load_b_k<1>(s.k, LD, 16 * blks[x], 16 * kk, lane));
          }
          if (k2 + 1 < DK / 32)
#pragma unroll
            for (int i = 0; i < 2; ++i) m[i] = ps[(4 * k2 + 4 + 2 * half + i) * 32];
        }
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              W[x][t][e] += lo[x][t][e];
              lo[x][t][e] = 0.f;
            }
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      if (lane == 0) s.sdot[warp] = dot;
      uint4* frag = reinterpret_cast<uint4*>(s.X) + strip * 4 * 3 * 32;
      const int v0 = 16 * strip + g;
      // sum_a = scale gamma dO.Y; then Y = V - gamma R (the error the write corrects), R stays K S
      float sum_a[2][2][2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float xa[2][4];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int tk = 16 * blks[x] + 8 * t + c2 + e;
            const float gam = s.vec[tk], be = s.vec[128 + tk];
            sum_a[x][t][e] = a.scale * gam * (to_f32(s.d[tk * kLdG + v0]) * Y[x][t][e] + to_f32(s.d[tk * kLdG + v0 + 8]) * Y[x][t][2 + e]);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              Y[x][t][2 * r + e] = to_f32(s.M[tk * kLdG + v0 + 8 * r]) - gam * R[x][t][2 * r + e];
              xa[t][2 * r + e] = be * Y[x][t][2 * r + e];
            }
          }
        put_frag<3>(frag + blks[x] * 96, from_acc<3>(xa[0], xa[1]), lane);
      }
      named_bar_sync(1 + strip, 64);
      float U[2][2][4] = {};
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        if (kk > blks[1]) break;
        const AFrag<3> fx = get_frag<3>(frag + kk * 96, lane);
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if (kk <= blks[x]) mma2(U[x][0], U[x][1], lo[x][0], lo[x][1], fx, load_tri_k<3>(s.Tm, blks[x], kk, lane));
      }
      float sum[2][2][2];
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            U[x][t][e] += lo[x][t][e];
            lo[x][t][e] = 0.f;
          }
          store_parts_t(s.U + (16 * blks[x] + 8 * t) * kLdG + 16 * strip, kPlaneG, kLdG, U[x][t], lane);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int tk = 16 * blks[x] + 8 * t + c2 + e;
            sum[x][t][e] = s.vec[64 + tk] * (W[x][t][e] * U[x][t][e] + W[x][t][2 + e] * U[x][t][2 + e]);
            U[x][t][e] = U[x][t][2 + e] = 0.f;
          }
        }
      sum_tokens(sum, s.tok[strip][1], blks[0], blks[1], lane);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        if (kk < blks[0]) continue;
        const AFrag<1> fd = load_a_m<1>(s.d, kLdG, 16 * kk, 16 * strip, lane);
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if (kk >= blks[x]) mma2(U[x][0], U[x][1], lo[x][0], lo[x][1], fd, load_tri_n<3>(s.P, kk, blks[x], lane));
      }
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            U[x][t][e] = a.scale * (U[x][t][e] + lo[x][t][e]) + s.vec[64 + 16 * blks[x] + 8 * t + c2 + (e & 1)] * W[x][t][e];
            W[x][t][e] = lo[x][t][e] = 0.f;
          }
      named_bar_sync(1 + strip, 64);  // both warps have taken X
#pragma unroll
      for (int x = 0; x < 2; ++x) put_frag<3>(frag + blks[x] * 96, from_acc<3>(U[x][0], U[x][1]), lane);
      named_bar_sync(1 + strip, 64);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        if (kk < blks[0]) continue;
        const AFrag<3> fu = get_frag<3>(frag + kk * 96, lane);
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if (kk >= blks[x]) mma2(W[x][0], W[x][1], lo[x][0], lo[x][1], fu, load_tri_n<3>(s.Tm, kk, blks[x], lane));
      }
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int tk = 16 * blks[x] + 8 * t + c2 + e;
            W[x][t][e] += lo[x][t][e];
            W[x][t][2 + e] += lo[x][t][2 + e];
            sum_a[x][t][e] -= s.vec[128 + tk] * s.vec[tk] * (W[x][t][e] * R[x][t][e] + W[x][t][2 + e] * R[x][t][2 + e]);
            sum[x][t][e] = W[x][t][e] * Y[x][t][e] + W[x][t][2 + e] * Y[x][t][2 + e];
          }
      sum_tokens(sum_a, s.tok[strip][0], blks[0], blks[1], lane);
      sum_tokens(sum, s.tok[strip][2], blks[0], blks[1], lane);
    }
    __syncthreads();  // every fragment has been read: dX takes their place
    if (strip < nw)
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int t = 0; t < 2; ++t) store_parts_t(s.X + (16 * blks[x] + 8 * t) * kLdG + 16 * strip, kPlaneG, kLdG, W[x][t], lane);
    __syncthreads();
    // ---- 2: a 16 x 16 block of dA in each of warps 0-9, one or two of dP in the others; dV
    {
      bf16* dv = static_cast<bf16*>(a.dvv) + r0 * a.dv;
      for (int x = tid; x < kC * 16; x += 512) {
        const int t = x >> 4, y = (x & 15) * 8;
        if (t >= rows || y >= a.dv) continue;
        const float be = s.vec[128 + t];
        const uint4 u0 = *reinterpret_cast<const uint4*>(s.X + t * kLdG + y);
        const uint4 u1 = *reinterpret_cast<const uint4*>(s.X + kPlaneG + t * kLdG + y);
        const uint32_t p0[4] = {u0.x, u0.y, u0.z, u0.w}, p1[4] = {u1.x, u1.y, u1.z, u1.w};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          o[i] = t < n ? pack_bf16x2(be * (bf16_lo(p0[i]) + bf16_lo(p1[i])), be * (bf16_hi(p0[i]) + bf16_hi(p1[i]))) : 0u;
        if (a.dv % 8 == 0 && a.vec_dv) {
          *reinterpret_cast<uint4*>(dv + (long long)t * a.dv + y) = make_uint4(o[0], o[1], o[2], o[3]);
        } else {
          const bf16* w = reinterpret_cast<const bf16*>(o);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (y + i < a.dv) dv[(long long)t * a.dv + y + i] = w[i];
        }
      }
      const bool is_a = warp < 10;
      for (int blk = is_a ? warp : warp - 10; blk < 10; blk += is_a ? 10 : 6) {
        const int rb = blk >= 6 ? 3 : blk >= 3 ? 2 : blk >= 1 ? 1 : 0, cb = blk - rb * (rb + 1) / 2;
        float acc[2][4] = {}, lo[2][4] = {}, kk2[2][4] = {};
#pragma unroll 1
        for (int kk = 0; kk < nw; ++kk) {
          const BFrag<3> fu = load_b_k<3>(s.U, kPlaneG, kLdG, 16 * cb, 16 * kk, lane);
          if (is_a)
            mma2(acc[0], acc[1], lo[0], lo[1], load_a_k<3>(s.X, kPlaneG, kLdG, 16 * rb, 16 * kk, lane), fu);
          else
            mma2(acc[0], acc[1], lo[0], lo[1], load_a_k<1>(s.d, kLdG, 16 * rb, 16 * kk, lane), fu);
        }
        if (is_a)
#pragma unroll
          for (int kk = 0; kk < DK / 16; ++kk)
            mma2(kk2[0], kk2[1], load_a_k<1>(s.k, LD, 16 * rb, 16 * kk, lane), load_b_k<1>(s.k, LD, 16 * cb, 16 * kk, lane));
        float row[2] = {}, rowb[2] = {};
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          float col[2] = {};
          const int jl = 8 * t + c2, j = 16 * cb + jl;
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int il = g + 8 * r, i = 16 * rb + il;
            float m[2], dec[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              m[e] = acc[t][2 * r + e] + lo[t][2 * r + e];
              dec[e] = decay(s.G[i], s.G[j + e], is_a ? i > j + e : i >= j + e);
            }
            if (is_a) {
              const float be = s.vec[128 + i];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float ab = -m[e] * dec[e] * kk2[t][2 * r + e];
                rowb[r] += ab;
                row[r] += be * ab;
                col[e] += be * ab;
                m[e] *= -be * dec[e];
              }
#pragma unroll
              for (int p = 0; p < 2; ++p) {
                const uint32_t w = pack_bf16x2(m[0], m[1]);
                bf16* M = s.M + p * kPlaneM;
                // the pair lies on one side of the diagonal or across it
                if (i > j + 1) *reinterpret_cast<uint32_t*>(M + i * kLdM + j) = w;
                else if (i >= j) M[i * kLdM + j] = from_f32<bf16>(m[0]);
                if (i == j + 1) M[i * kLdM + j + 1] = zero;
                if (i > j) M[j * kLdM + i] = __ushort_as_bfloat16((unsigned short)(w & 0xffffu));
                if (i > j + 1) M[(j + 1) * kLdM + i] = __ushort_as_bfloat16((unsigned short)(w >> 16));
                m[0] -= bf16_lo(w);
                m[1] -= bf16_hi(w);
              }
            } else {
              bf16* P = s.P + blk * 256 + tri_at(il, jl);
              const uint32_t p0 = *reinterpret_cast<const uint32_t*>(P), p1 = *reinterpret_cast<const uint32_t*>(P + kTri),
                             p2 = *reinterpret_cast<const uint32_t*>(P + 2 * kTri);
              const float pe[2] = {(bf16_lo(p2) + bf16_lo(p1)) + bf16_lo(p0), (bf16_hi(p2) + bf16_hi(p1)) + bf16_hi(p0)};
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float dp = a.scale * m[e], y = i > j + e && dec[e] != 0.f ? dp * pe[e] : 0.f;
                row[r] += y;
                col[e] += y;
                m[e] = dp * dec[e];
              }
              put_parts<2>(P, kTri, m[0], m[1]);
            }
          }
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            col[0] += __shfl_xor_sync(0xffffffffu, col[0], o);
            col[1] += __shfl_xor_sync(0xffffffffu, col[1], o);
          }
          if (lane < 4) {
            (is_a ? s.colA : s.colP)[blk][jl] = col[0];
            (is_a ? s.colA : s.colP)[blk][jl + 1] = col[1];
          }
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            row[r] += __shfl_xor_sync(0xffffffffu, row[r], o);
            rowb[r] += __shfl_xor_sync(0xffffffffu, rowb[r], o);
          }
        if ((lane & 3) == 0)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            (is_a ? s.rowA : s.rowP)[blk][g + 8 * r] = row[r];
            if (is_a) s.rowB[blk][g + 8 * r] = rowb[r];
          }
      }
    }
    __syncthreads();
    // ---- 3: dg, dbeta (warp 15, two tokens a lane); dQ and dK, 16 key columns and 32 tokens per warp
    if (warp == 15) {
      double x[2], ev2[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int t = 2 * lane + i, tb = t >> 4, tl = t & 15;
        float av = 0.f, ev = 0.f, bv = 0.f, pos = 0.f, neg = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) {  // every load in flight; what lies behind nw is not added
          const float x0 = s.tok[w][0][t], x1 = s.tok[w][1][t], x2 = s.tok[w][2][t];
          av += w < nw ? x0 : 0.f;
          ev += w < nw ? x1 : 0.f;
          bv += w < nw ? x2 : 0.f;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int above = tri_block(tb, min(c, tb)), below = tri_block(max(c, tb), tb);
          const float x0 = s.rowP[above][tl] + s.rowA[above][tl], x1 = s.rowB[above][tl], x2 = s.colP[below][tl] + s.colA[below][tl];
          pos += c <= tb ? x0 : 0.f;
          bv += c <= tb ? x1 : 0.f;
          neg += c >= tb ? x2 : 0.f;
        }
        x[i] = (double)av + pos - neg;
        ev2[i] = ev;
        if (t < rows) a.dbeta[r0 + t] = t < n ? bv : 0.f;
      }
      float dot = 0.f;
      for (int w = 0; w < 2 * nw; ++w) dot += s.sdot[w];
      if (lane == 31) x[1] += (double)s.vec[192] * dot;
      double sum, before;
      decay_sums(x, ev2, sum, before, lane);
      if (2 * lane < rows) a.dg[r0 + 2 * lane] = 2 * lane < n ? (float)(sum + x[0] + before) : 0.f;
      if (2 * lane + 1 < rows) a.dg[r0 + 2 * lane + 1] = 2 * lane + 1 < n ? (float)(sum + before + ev2[0]) : 0.f;
    }
    if (strip < DK / 16) {
      const int n0 = 16 * strip;
      float Q[2][2][4] = {}, K[2][2][4] = {}, V[2][2][4] = {};
      const float4* ps = snap + 2 * strip * 32 + lane;
      const float4* pd = dsnap + 2 * strip * 32 + lane;
#pragma unroll 2
      for (int kw = 0; kw < nw; ++kw) {
        const BFrag<2> fs = b_from_acc<2>(ps[kw * (DK / 8) * 32], ps[kw * (DK / 8) * 32 + 32]);
        const BFrag<2> fd = b_from_acc<2>(pd[kw * (DK / 8) * 32], pd[kw * (DK / 8) * 32 + 32]);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int m0 = 32 * half + 16 * x;
          mma2(Q[x][0], Q[x][1], load_a_k<1>(s.d, kLdG, m0, 16 * kw, lane), fs);
          mma2(K[x][0], K[x][1], load_a_k<2>(s.X, kPlaneG, kLdG, m0, 16 * kw, lane), fs);
          mma2(V[x][0], V[x][1], load_a_k<2>(s.U, kPlaneG, kLdG, m0, 16 * kw, lane), fd);
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int tk = 32 * half + 16 * x + g + 8 * r;
          const float gam = s.vec[tk], be = s.vec[128 + tk], rho = s.vec[64 + tk];
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 2 * r; e < 2 * r + 2; ++e) {
              Q[x][t][e] *= a.scale * gam;
              K[x][t][e] = rho * V[x][t][e] - be * gam * K[x][t][e];
            }
        }
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        const BFrag<1> bk = load_b_n<1>(s.k, LD, 16 * kk, n0, lane), bq = load_b_n<1>(s.q, LD, 16 * kk, n0, lane);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int mt = 2 * half + x;
          if (kk <= mt) mma2(Q[x][0], Q[x][1], load_tri_a_k<2>(s.P, mt, kk, lane), bk);
          mma2(K[x][0], K[x][1], load_a_k<2>(s.M, kPlaneM, kLdM, 16 * mt, 16 * kk, lane), bk);
          if (kk >= mt) mma2(K[x][0], K[x][1], load_tri_a_m<2>(s.P, kk, mt, lane), bq);
        }
      }
      float* acc = a.acc + ((a.split ? bh : (long long)b * a.Hk + hk) * a.nc + i0) * 2 * kC * DK;
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int tk = 32 * half + 16 * x + g + 8 * r, col = n0 + 8 * t + c2;
            float2 yq = make_float2(Q[x][t][2 * r], Q[x][t][2 * r + 1]), yk = make_float2(K[x][t][2 * r], K[x][t][2 * r + 1]);
            if (a.group > 1) {  // the same thread holds this element for every value head of the key head
              float2* pq = reinterpret_cast<float2*>(acc + tk * DK + col);
              float2* pk = reinterpret_cast<float2*>(acc + (kC + tk) * DK + col);
              if (hi > 0) {
                const float2 oq = *pq, ok = *pk;
                yq.x += oq.x; yq.y += oq.y; yk.x += ok.x; yk.y += ok.y;
              }
              if (a.split || hi + 1 < a.group) {
                *pq = yq;
                *pk = yk;
                continue;
              }
            }
            if (tk < rows) {
              const long long o = (long long)tk * a.dk + col;
              if (tk >= n) yq = yk = make_float2(0.f, 0.f);
              if (a.vec_dq && col < a.dk) {
                *reinterpret_cast<uint32_t*>(dq + o) = pack_bf16x2(yq.x, yq.y);
                *reinterpret_cast<uint32_t*>(dkk + o) = pack_bf16x2(yk.x, yk.y);
              } else {
                if (col < a.dk) {
                  dq[o] = from_f32<bf16>(yq.x);
                  dkk[o] = from_f32<bf16>(yk.x);
                }
                if (col + 1 < a.dk) {
                  dq[o + 1] = from_f32<bf16>(yq.y);
                  dkk[o + 1] = from_f32<bf16>(yk.y);
                }
              }
            }
          }
    }
    __syncthreads();
  }
}

// dq and dk of a chunk from the value heads' own, in their order (split).
template <typename T, int DK> __global__ void __launch_bounds__(256) sum_heads_kernel(const ChunkArgs a) {
  const int b = blockIdx.z, hk = blockIdx.y, i0 = blockIdx.x;
  const long long t0 = (long long)i0 * kC;
  const int n = chunk_len(row_len(a, b), i0), rows = chunk_len(a.L, i0);
  const long long out = (((long long)b * a.Hk + hk) * a.L + t0) * a.dk;
  const float* acc = a.acc + (((long long)b * a.H + hk * a.group) * a.nc + i0) * 2 * kC * DK;
#pragma unroll 2
  for (int x = threadIdx.x; x < rows * (DK / 4); x += 256) {
    const int t = x / (DK / 4), c = x % (DK / 4) * 4;
    float4 q = make_float4(0.f, 0.f, 0.f, 0.f), k = q;
    if (t < n)
#pragma unroll 4
      for (int hi = 0; hi < a.group; ++hi) {
        const float* p = acc + (long long)hi * a.nc * 2 * kC * DK + t * DK + c;
        const float4 u = *reinterpret_cast<const float4*>(p), w = *reinterpret_cast<const float4*>(p + kC * DK);
        q.x += u.x; q.y += u.y; q.z += u.z; q.w += u.w;
        k.x += w.x; k.y += w.y; k.z += w.z; k.w += w.w;
      }
    const float qs[4] = {q.x, q.y, q.z, q.w}, ks[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (c + e < a.dk) {
        static_cast<T*>(a.dq)[out + (long long)t * a.dk + c + e] = from_f32<T>(qs[e]);
        static_cast<T*>(a.dkk)[out + (long long)t * a.dk + c + e] = from_f32<T>(ks[e]);
      }
  }
}

}  // namespace gd
}  // namespace infini
