// Layer normalisation over the last dimension of contiguous rows, forward and backward.
//
//   xhat = (x - mean) rstd,  mean = sum x / D,  rstd = 1 / sqrt(sum (x - mean)^2 / D + eps)
//   y    = xhat * weight + bias
//   h = dy * weight:  dx = rstd (h - sum h / D - xhat * sum(h xhat) / D)
//   dweight = sum over rows of dy xhat,  dbias = sum over rows of dy
//
// HBM-bound: the forward reads x and writes y once, the backward reads x and dy and writes dx
// once.  A row lives in the registers of TPR threads (NV vectors of VEC elements each), so the
// variance is the two-pass sum of squared distances from the mean (a one-pass sum of squares
// loses it where |mean| is far above the spread), and the backward takes the statistics from the
// row again instead of reading them.  All arithmetic and sums in fp32; y, dx and the weight
// gradients are rounded once, to their tensors' types.
//
// Measured (bf16, of a 6544 GB/s copy): forward 32768 x 4096 98 us (84 %), 32768 x 1024 30 us (69 %);
// backward 32768 x 4096 177 us (69 %), 32768 x 1024 55 us with its reduction (56 %; the issue slots
// are 58 % busy with fp32 arithmetic and shuffles).  Odd rows: 32768 x 1025 57 and 111 us.
#include <cuda_bf16.h>

#include <algorithm>

#include "../../include/infini_attn.h"
#include "common.cuh"
#include "host.h"

namespace infini {
namespace ln {

constexpr int kMaxD = 16384;

template <int VEC> struct Floats { float v[VEC]; };
// VEC consecutive elements as they lie in memory (16-byte aligned when VEC > 1).
template <typename T, int VEC> struct Raw;
template <> struct Raw<__nv_bfloat16, 8> { uint4 u; };
template <> struct Raw<float, 4> { float4 u; };
template <> struct Raw<__nv_bfloat16, 1> { __nv_bfloat16 u; };
template <> struct Raw<float, 1> { float u; };

template <int VEC, typename T> __device__ __forceinline__ Raw<T, VEC> load_raw(const T* p) {
  return *reinterpret_cast<const Raw<T, VEC>*>(p);
}
// Elements lo .. hi - 1 of a vector, zeros around them (kept in registers: no array is indexed).
template <int VEC> __device__ __forceinline__ Raw<__nv_bfloat16, VEC> load_edge(const __nv_bfloat16* p, int lo, int hi) {
  const unsigned short* u = reinterpret_cast<const unsigned short*>(p);
  uint32_t w[4] = {};
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    uint32_t x = 0;
    if (i >= lo && i < hi) x = u[i];
    w[i / 2] |= x << (16 * (i % 2));
  }
  Raw<__nv_bfloat16, VEC> r;
  r.u = make_uint4(w[0], w[1], w[2], w[3]);
  return r;
}
template <int VEC> __device__ __forceinline__ Raw<float, VEC> load_edge(const float* p, int lo, int hi) {
  float x[4] = {};
#pragma unroll
  for (int i = 0; i < VEC; ++i)
    if (i >= lo && i < hi) x[i] = p[i];
  Raw<float, VEC> r;
  r.u = make_float4(x[0], x[1], x[2], x[3]);
  return r;
}
template <typename T, int VEC> __device__ __forceinline__ Floats<VEC> floats(const Raw<T, VEC>& r) {
  Floats<VEC> f;
  if constexpr (VEC == 8) {
    const uint32_t w[4] = {r.u.x, r.u.y, r.u.z, r.u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f.v[2 * i] = bf16_lo(w[i]);
      f.v[2 * i + 1] = bf16_hi(w[i]);
    }
  } else if constexpr (VEC == 4) {
    f = {{r.u.x, r.u.y, r.u.z, r.u.w}};
  } else {
    f.v[0] = to_f32(r.u);
  }
  return f;
}
template <int VEC> __device__ __forceinline__ void store_vec(__nv_bfloat16* p, const Floats<VEC>& f) {
  if constexpr (VEC == 8) {
    uint4 u;
    u.x = pack_bf16x2(f.v[0], f.v[1]);
    u.y = pack_bf16x2(f.v[2], f.v[3]);
    u.z = pack_bf16x2(f.v[4], f.v[5]);
    u.w = pack_bf16x2(f.v[6], f.v[7]);
    *reinterpret_cast<uint4*>(p) = u;
  } else {
    *p = __float2bfloat16_rn(f.v[0]);
  }
}
template <int VEC> __device__ __forceinline__ void store_vec(float* p, const Floats<VEC>& f) {
  if constexpr (VEC == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(f.v[0], f.v[1], f.v[2], f.v[3]);
  } else {
    *p = f.v[0];
  }
}
// weight / bias elements, bf16 or fp32
template <int VEC> __device__ __forceinline__ Floats<VEC> load_weight(const void* p, bool f32, long long at) {
  Floats<VEC> f;
  if (f32) {
    const float* w = static_cast<const float*>(p) + at;
    if constexpr (VEC == 8) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const Floats<4> h = floats(load_raw<4>(w + 4 * i));
#pragma unroll
        for (int e = 0; e < 4; ++e) f.v[4 * i + e] = h.v[e];
      }
    } else {
      f = floats(load_raw<VEC>(w));
    }
  } else {
    const __nv_bfloat16* w = static_cast<const __nv_bfloat16*>(p) + at;
    if constexpr (VEC == 8)
      f = floats(load_raw<8>(w));
    else
#pragma unroll
      for (int e = 0; e < VEC; ++e) f.v[e] = to_f32(w[e]);
  }
  return f;
}

// Sums of N values over the TPR threads of a row, the same in all of them.  Above a warp the
// warps' sums meet in shared memory; `red` holds one slot set per call in flight.
template <int TPR, int N> __device__ __forceinline__ void row_sum(float (&x)[N], float* red, int sub) {
  constexpr int W = TPR < 32 ? TPR : 32;
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1)
#pragma unroll
    for (int n = 0; n < N; ++n) x[n] += __shfl_xor_sync(0xffffffffu, x[n], o);
  if constexpr (TPR > 32) {
    constexpr int NW = TPR / 32;
    const int warp = (threadIdx.x / 32) % NW;
    float* slot = red + sub * NW * N;
    if (threadIdx.x % 32 == 0)
#pragma unroll
      for (int n = 0; n < N; ++n) slot[warp * N + n] = x[n];
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) x[n] = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w)
#pragma unroll
      for (int n = 0; n < N; ++n) x[n] += slot[w * N + n];
  }
}


struct Args {
  const void* x;
  const void* weight;
  const void* bias;  // nullptr: none
  const void* dy;
  void* y;         // forward: y; backward: dx
  float* partial;  // backward: [gridDim.x][2][D]
  long long rows;
  int D;
  float eps;
  bool w32;       // weight and bias are fp32
  int shift;      // elements by which x, dy and y lie behind a multiple of 16 bytes
  bool has_bias;  // backward: dbias is wanted
};

// Threads per block: rows of at most a warp share a block of 128, wider rows have a block each.
template <int TPR> constexpr int kBlockThreads = TPR < 128 ? 128 : TPR;
// Elements per thread up to which the weights stay in registers for all the rows of a block.
// (Re-read for each row they cost four times the row itself from L2: 146 us at 32768 x 4096 bf16.)
constexpr int kKeep = 24;

// Column of element 0 of a thread's vector v.  SHIFT: rows do not start on 16 bytes; a row's vectors
// then are those of memory, the first starting `off` elements before the row, so that all but the
// first and the last are still loaded and stored whole.  A thread's rows are a multiple of VEC
// apart: off, and with it the columns it holds, is the same for all of them.
template <int VEC, int TPR> __device__ __forceinline__ int column(int v, int lane, int off) { return (v * TPR + lane) * VEC - off; }

// A thread's part of row `row`.  SHIFT: a row's first and last vector hold elements of its neighbours too, which
// inside() leaves out where they are used; only at the tensor's own ends are elements loaded one by one (putting a
// vector together there waits for its loads, and with it the whole prefetch).
template <typename T, int VEC, int TPR, int NV, bool SHIFT>
__device__ __forceinline__ void load_row(Raw<T, VEC> (&r)[NV], const void* x, long long row, const Args& a, int lane, int off) {
  const T* p = static_cast<const T*>(x) + row * a.D;
  const bool active = row < a.rows;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int at = column<VEC, TPR>(v, lane, off);
    r[v] = Raw<T, VEC>{};
    if (!active || at >= a.D) continue;
    if constexpr (SHIFT)
      if (row * a.D + at < 0 || row * a.D + at + VEC > a.rows * a.D) {
        r[v] = load_edge<VEC>(p + at, -at, a.D - at);
        continue;
      }
    r[v] = load_raw<VEC>(p + at);
  }
}
template <bool SHIFT> __device__ __forceinline__ bool inside(int at, int e, int D) { return SHIFT ? at + e >= 0 && at + e < D : at < D; }
template <int VEC, int TPR, bool SHIFT, typename T> __device__ __forceinline__ void store_part(T* p, int at, int D, const Floats<VEC>& o) {
  if constexpr (SHIFT) {
    if (at >= 0 && at + VEC <= D) {
      store_vec<VEC>(p + at, o);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (at + i >= 0 && at + i < D) p[at + i] = from_f32<T>(o.v[i]);
    }
  } else {
    store_vec<VEC>(p + at, o);
  }
}
template <int VEC, bool SHIFT> __device__ __forceinline__ Floats<VEC> weight_part(const void* p, bool f32, int at, int D) {
  Floats<VEC> w = {};
  if constexpr (SHIFT) {
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (at + i >= 0 && at + i < D) w.v[i] = f32 ? static_cast<const float*>(p)[at + i] : to_f32(static_cast<const __nv_bfloat16*>(p)[at + i]);
  } else {
    if (at < D) w = load_weight<VEC>(p, f32, at);
  }
  return w;
}
// xs: the row's elements less their mean, 0 outside the row; returns the variance.
template <typename T, int VEC, int TPR, int NV, bool SHIFT>
__device__ __forceinline__ float centre(const Raw<T, VEC> (&r)[NV], int lane, int D, int off, float (&xs)[NV][VEC], float* red, int sub, int red_stride) {
  float s[1] = {0.f};
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const Floats<VEC> f = floats(r[v]);
    const int at = column<VEC, TPR>(v, lane, off);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      xs[v][e] = !SHIFT || inside<SHIFT>(at, e, D) ? f.v[e] : 0.f;
      s[0] += xs[v][e];
    }
  }
  row_sum<TPR>(s, red, sub);
  const float mean = s[0] / (float)D;
  float q[1] = {0.f};
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int at = column<VEC, TPR>(v, lane, off);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      xs[v][e] = inside<SHIFT>(at, e, D) ? xs[v][e] - mean : 0.f;
      q[0] = fmaf(xs[v][e], xs[v][e], q[0]);
    }
  }
  row_sum<TPR>(q, red + red_stride, sub);
  return q[0] / (float)D;
}

template <typename T, int VEC, int TPR, int NV, bool SHIFT>
__global__ void __launch_bounds__(kBlockThreads<TPR>) ln_forward_kernel(const Args a) {
  constexpr int TH = kBlockThreads<TPR>, RPB = TH / TPR, NW = TPR > 32 ? TPR / 32 : 1;
  constexpr bool KEEP = NV * VEC <= kKeep;
  __shared__ float red[2 * RPB * NW];
  const int sub = threadIdx.x / TPR, lane = threadIdx.x % TPR;
  const long long step = (long long)gridDim.x * RPB;
  long long row = (long long)blockIdx.x * RPB + sub;
  const int off = SHIFT ? (int)((a.shift + row * a.D) % VEC) : 0;
  Raw<T, VEC> next[NV];
  load_row<T, VEC, TPR, NV, SHIFT>(next, a.x, row, a, lane, off);
  Floats<VEC> w[KEEP ? NV : 1], b[KEEP ? NV : 1];
  if constexpr (KEEP)
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int at = column<VEC, TPR>(v, lane, off);
      w[v] = weight_part<VEC, SHIFT>(a.weight, a.w32, at, a.D);
      b[v] = {};
      if (a.bias) b[v] = weight_part<VEC, SHIFT>(a.bias, a.w32, at, a.D);
    }
  for (long long base = (long long)blockIdx.x * RPB; base < a.rows; base += step, row += step) {
    const bool active = row < a.rows;
    Raw<T, VEC> cur[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) cur[v] = next[v];
    load_row<T, VEC, TPR, NV, SHIFT>(next, a.x, row + step, a, lane, off);
    float xs[NV][VEC];
    const float var = centre<T, VEC, TPR, NV, SHIFT>(cur, lane, a.D, off, xs, red, sub, RPB * NW);
    const float rstd = 1.f / sqrtf(var + a.eps);
    if (!active) continue;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int at = column<VEC, TPR>(v, lane, off);
      if (at < a.D) {
        Floats<VEC> wv, bv = {}, o;
        if constexpr (KEEP) {
          wv = w[v];
          bv = b[v];
        } else {
          wv = weight_part<VEC, SHIFT>(a.weight, a.w32, at, a.D);
          if (a.bias) bv = weight_part<VEC, SHIFT>(a.bias, a.w32, at, a.D);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) o.v[e] = fmaf(xs[v][e] * rstd, wv.v[e], bv.v[e]);
        store_part<VEC, TPR, SHIFT>(static_cast<T*>(a.y) + row * a.D, at, a.D, o);
      }
    }
  }
}

template <typename T, int VEC, int TPR, int NV, bool SHIFT>
__global__ void __launch_bounds__(kBlockThreads<TPR>) ln_backward_kernel(const Args a) {
  constexpr int TH = kBlockThreads<TPR>, RPB = TH / TPR, NW = TPR > 32 ? TPR / 32 : 1, E = NV * VEC;
  constexpr bool KEEP = E <= kKeep;
  __shared__ float red[4 * RPB * NW];  // statistics, then the two sums of a row
  extern __shared__ float acc[];       // RPB > 1: [2][D], the block's sums over its rows in flight
  const int sub = threadIdx.x / TPR, lane = threadIdx.x % TPR;
  const long long step = (long long)gridDim.x * RPB;
  long long row = (long long)blockIdx.x * RPB + sub;
  const int off = SHIFT ? (int)((a.shift + row * a.D) % VEC) : 0;
  Raw<T, VEC> nx[NV], nd[NV];
  load_row<T, VEC, TPR, NV, SHIFT>(nx, a.x, row, a, lane, off);
  load_row<T, VEC, TPR, NV, SHIFT>(nd, a.dy, row, a, lane, off);
  Floats<VEC> w[KEEP ? NV : 1];
  if constexpr (KEEP)
#pragma unroll
    for (int v = 0; v < NV; ++v) w[v] = weight_part<VEC, SHIFT>(a.weight, a.w32, column<VEC, TPR>(v, lane, off), a.D);
  float dw[NV][VEC] = {}, db[NV][VEC] = {};
  for (long long base = (long long)blockIdx.x * RPB; base < a.rows; base += step, row += step) {
    const bool active = row < a.rows;
    Raw<T, VEC> cx[NV], cd[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      cx[v] = nx[v];
      cd[v] = nd[v];
    }
    load_row<T, VEC, TPR, NV, SHIFT>(nx, a.x, row + step, a, lane, off);
    load_row<T, VEC, TPR, NV, SHIFT>(nd, a.dy, row + step, a, lane, off);
    float xs[NV][VEC];
    const float var = centre<T, VEC, TPR, NV, SHIFT>(cx, lane, a.D, off, xs, red, sub, RPB * NW);
    const float rstd = active ? 1.f / sqrtf(var + a.eps) : 0.f;  // 0 * (1 / 0) of a place without a row would reach dw
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int at = column<VEC, TPR>(v, lane, off);
      Floats<VEC> d = floats(cd[v]), wv;
      if constexpr (KEEP)
        wv = w[v];
      else
        wv = weight_part<VEC, SHIFT>(a.weight, a.w32, at, a.D);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        if (SHIFT && !inside<SHIFT>(at, e, a.D)) d.v[e] = 0.f;
        xs[v][e] *= rstd;
        dw[v][e] = fmaf(d.v[e], xs[v][e], dw[v][e]);
        db[v][e] += d.v[e];
        const float h = d.v[e] * wv.v[e];
        s[0] += h;
        s[1] = fmaf(h, xs[v][e], s[1]);
      }
    }
    row_sum<TPR>(s, red + 2 * RPB * NW, sub);
    const float m0 = s[0] / (float)a.D, m1 = s[1] / (float)a.D;
    if (active) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int at = column<VEC, TPR>(v, lane, off);
        if (at < a.D) {
          const Floats<VEC> d = floats(cd[v]);
          Floats<VEC> wv, o;
          if constexpr (KEEP)
            wv = w[v];
          else
            wv = weight_part<VEC, SHIFT>(a.weight, a.w32, at, a.D);
#pragma unroll
          for (int e = 0; e < VEC; ++e) o.v[e] = rstd * (d.v[e] * wv.v[e] - m0 - xs[v][e] * m1);
          store_part<VEC, TPR, SHIFT>(static_cast<T*>(a.y) + row * a.D, at, a.D, o);
        }
      }
    }
  }
  // the block's sum over its RPB rows in flight, in their order, column by column
  float* pw = a.partial + (long long)blockIdx.x * 2 * a.D;
  for (int r = 0; r < RPB; ++r) {
    if (sub == r)
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const int at = column<VEC, TPR>(v, lane, off) + e;
          if (at < 0 || at >= a.D) continue;
          float x = dw[v][e], y = db[v][e];
          if constexpr (RPB > 1) {
            if (r > 0) {
              x += acc[at];
              y += acc[a.D + at];
            }
            if (r + 1 < RPB) {
              acc[at] = x;
              acc[a.D + at] = y;
              continue;
            }
          }
          pw[at] = x;
          pw[a.D + at] = y;
        }
    if constexpr (RPB > 1) __syncthreads();
  }
}

// dweight, dbias: the sum of the blocks' partials, in their order (32 columns per block; 32
// interleaved ranges of blocks, then those 32 sums).
__global__ void __launch_bounds__(1024) ln_reduce_kernel(const float* partial, int parts, int D, void* dw, void* db, bool w32) {
  __shared__ float s[32][33];
  const int x = threadIdx.x % 32, col = blockIdx.x * 32 + x, r = threadIdx.x / 32;
  const bool is_b = blockIdx.y == 1;
  float y = 0.f;
  if (col < D)
#pragma unroll 4
    for (int p = r; p < parts; p += 32) y += partial[((long long)p * 2 + is_b) * D + col];
  s[r][x] = y;
  __syncthreads();
  // warp r sums column r
  float t = s[x][r];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  const int c = blockIdx.x * 32 + r;
  if (x == 0 && c < D) {
    void* out = is_b ? db : dw;
    if (w32)
      static_cast<float*>(out)[c] = t;
    else
      static_cast<__nv_bfloat16*>(out)[c] = __float2bfloat16_rn(t);
  }
}

// Blocks of the row loops.  Forward: as many as are resident (one per row at most).  Backward: every
// block leaves a partial of 2 D sums, so no more than keep them small beside the rows.
int backward_blocks(long long rows, int rpb) {
  return (int)std::min<long long>((rows + rpb - 1) / rpb, 4LL * kSms);
}

template <typename F> int resident_blocks(F* kernel, int threads, size_t smem) {
  int n = 0;
  return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem) == cudaSuccess && n > 0 ? n * kSms : kSms;
}

// A multiple of VEC rows between a thread's rows (SHIFT).
int whole_blocks(long long most, long long blocks, int rpb, int vec) {
  if (most <= blocks) return (int)most;
  const int unit = std::max(1, vec / rpb);
  return (int)(blocks / unit * unit);
}

template <typename T, int VEC, int TPR, int NV, bool SHIFT> int launch(const Args& a, bool bwd, cudaStream_t st, int* parts) {
  constexpr int TH = kBlockThreads<TPR>, RPB = TH / TPR;
  const long long most = (a.rows + RPB - 1) / RPB;
  if (!bwd) {
    static const int resident = resident_blocks(ln_forward_kernel<T, VEC, TPR, NV, SHIFT>, TH, 0);
    LaunchScope scope(kPhasePre, st);
    ln_forward_kernel<T, VEC, TPR, NV, SHIFT><<<whole_blocks(most, resident, RPB, VEC), TH, 0, st>>>(a);
  } else {
    const size_t smem = RPB > 1 ? (size_t)2 * a.D * 4 : 0;
    static const int resident = resident_blocks(ln_backward_kernel<T, VEC, TPR, NV, SHIFT>, TH, RPB > 1 ? (size_t)2 * TPR * NV * VEC * 4 : 0);
    *parts = whole_blocks(most, std::min<long long>(backward_blocks(a.rows, RPB), resident), RPB, VEC);
    LaunchScope scope(kPhaseBwd, st);
    ln_backward_kernel<T, VEC, TPR, NV, SHIFT><<<*parts, TH, smem, st>>>(a);
  }
  return launch_status();
}

// Threads per row and vectors per thread by the number of vectors of a row; a multiple of 16 bytes
// to a row or (SHIFT) not.  VEC 1 where x, dy and y lie on different 16-byte grids.
template <typename T, int V, bool SHIFT> int dispatch_rows(const Args& a, bool bwd, cudaStream_t st, int* parts) {
  const int n = SHIFT ? (a.D + 2 * (V - 1)) / V : a.D / V;
  if (n <= 8) return launch<T, V, 8, 1, SHIFT>(a, bwd, st, parts);
  if (n <= 16) return launch<T, V, 16, 1, SHIFT>(a, bwd, st, parts);
  if (n <= 32) return launch<T, V, 32, 1, SHIFT>(a, bwd, st, parts);
  if (n <= 64) return launch<T, V, 32, 2, SHIFT>(a, bwd, st, parts);
  if (n <= 96) return launch<T, V, 32, 3, SHIFT>(a, bwd, st, parts);
  if (n <= 128) return launch<T, V, 64, 2, SHIFT>(a, bwd, st, parts);
  if (n <= 192) return launch<T, V, 64, 3, SHIFT>(a, bwd, st, parts);
  if (n <= 256) return launch<T, V, 128, 2, SHIFT>(a, bwd, st, parts);
  if (n <= 384) return launch<T, V, 128, 3, SHIFT>(a, bwd, st, parts);
  if (n <= 512) return launch<T, V, 256, 2, SHIFT>(a, bwd, st, parts);
  if (n <= 768) return launch<T, V, 256, 3, SHIFT>(a, bwd, st, parts);
  if (n <= 1024) return launch<T, V, 512, 2, SHIFT>(a, bwd, st, parts);
  if (n <= 1536) return launch<T, V, 512, 3, SHIFT>(a, bwd, st, parts);
  if (n <= 2048) return launch<T, V, 1024, 2, SHIFT>(a, bwd, st, parts);
  return launch<T, V, 1024, V == 8 ? 3 : SHIFT ? 5 : 4, SHIFT>(a, bwd, st, parts);
}
template <typename T> int dispatch(const Args& a, bool vec, bool bwd, cudaStream_t st, int* parts) {
  constexpr int V = 16 / sizeof(T);
  if (vec && a.shift == 0 && a.D % V == 0) return dispatch_rows<T, V, false>(a, bwd, st, parts);
  if (vec) return dispatch_rows<T, V, true>(a, bwd, st, parts);
  if (a.D <= 128) return launch<T, 1, 32, 4, false>(a, bwd, st, parts);
  if (a.D <= 1024) return launch<T, 1, 128, 8, false>(a, bwd, st, parts);
  return launch<T, 1, 1024, 16, false>(a, bwd, st, parts);
}

int past16(const void* p) { return (int)(reinterpret_cast<uintptr_t>(p) % 16); }

int check(long long rows, int D, float eps, int mode) {
  if (rows <= 0 || D <= 0 || !(eps >= 0.f) || isinf(eps)) return INFINI_ERR_INVALID_ARG;
  if ((mode & ~(INFINI_F32 | INFINI_WEIGHT_F32)) != 0 || D > kMaxD || rows > (1LL << 40) / D) return INFINI_ERR_UNSUPPORTED;
  return INFINI_OK;
}

}  // namespace ln
}  // namespace infini

using namespace infini;

extern "C" {

int infini_attn_layer_norm_forward(const void* x, const void* weight, const void* bias, void* y, long long rows, int D,
                                   float eps, int mode, cudaStream_t stream) {
  if (!x || !weight || !y) return INFINI_ERR_INVALID_ARG;
  int rc = ln::check(rows, D, eps, mode);
  if (rc != INFINI_OK) return rc;
  const size_t es = (mode & INFINI_F32) ? 4 : 2, ws = (mode & INFINI_WEIGHT_F32) ? 4 : 2;
  const size_t n = (size_t)rows * D * es, nw = (size_t)D * ws;
  if (ranges_overlap(y, n, weight, nw) || (bias && ranges_overlap(y, n, bias, nw)) ||
      (x != y && ranges_overlap(y, n, x, n)))
    return INFINI_ERR_INVALID_ARG;
  rc = check_device(false);
  if (rc != INFINI_OK) return rc;
  ln::Args a = {};
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.y = y;
  a.rows = rows;
  a.D = D;
  a.eps = eps;
  a.w32 = (mode & INFINI_WEIGHT_F32) != 0;
  a.shift = ln::past16(x) / (int)es;
  // whole vectors of the weights only where rows are whole vectors too
  const bool vec = ln::past16(x) == ln::past16(y) && (a.shift != 0 || D % (16 / es) != 0 || (ln::past16(weight) == 0 && ln::past16(bias) == 0));
  return (mode & INFINI_F32) ? ln::dispatch<float>(a, vec, false, stream, nullptr)
                             : ln::dispatch<__nv_bfloat16>(a, vec, false, stream, nullptr);
}

size_t infini_attn_layer_norm_backward_workspace_size(long long rows, int D) {
  if (ln::check(rows, D, 0.f, 0) != INFINI_OK) return 0;
  return align_up((size_t)ln::backward_blocks(rows, 1) * 2 * D * 4);
}

int infini_attn_layer_norm_backward(const void* x, const void* weight, const void* dy, void* dx, void* dweight,
                                    void* dbias, long long rows, int D, float eps, int mode, void* workspace,
                                    size_t workspace_bytes, cudaStream_t stream) {
  if (!x || !weight || !dy || !dx || !dweight) return INFINI_ERR_INVALID_ARG;
  int rc = ln::check(rows, D, eps, mode);
  if (rc != INFINI_OK) return rc;
  const size_t es = (mode & INFINI_F32) ? 4 : 2, wsz = (mode & INFINI_WEIGHT_F32) ? 4 : 2;
  const size_t n = (size_t)rows * D * es, nw = (size_t)D * wsz;
  const void* outs[3] = {dx, dweight, dbias};
  const size_t outn[3] = {n, nw, nw};
  const void* ins[3] = {x, dy, weight};
  const size_t inn[3] = {n, n, nw};
  for (int i = 0; i < 3; ++i) {
    if (!outs[i]) continue;
    for (int j = 0; j < 3; ++j)  // dx may take dy's or x's place exactly
      if (ranges_overlap(outs[i], outn[i], ins[j], inn[j]) && !(i == 0 && j < 2 && outs[i] == ins[j]))
        return INFINI_ERR_INVALID_ARG;
    for (int j = i + 1; j < 3; ++j)
      if (outs[j] && ranges_overlap(outs[i], outn[i], outs[j], outn[j])) return INFINI_ERR_INVALID_ARG;
  }
  const size_t need = infini_attn_layer_norm_backward_workspace_size(rows, D);
  if (workspace && (workspace_bytes < need || reinterpret_cast<uintptr_t>(workspace) % kAlign != 0))
    return INFINI_ERR_WORKSPACE;
  rc = check_device(false);
  if (rc != INFINI_OK) return rc;
  void* w = workspace;
  if (!w && !ws_alloc(&w, need, stream)) return INFINI_ERR_WORKSPACE;
  ln::Args a = {};
  a.x = x;
  a.weight = weight;
  a.dy = dy;
  a.y = dx;
  a.partial = static_cast<float*>(w);
  a.rows = rows;
  a.D = D;
  a.eps = eps;
  a.w32 = (mode & INFINI_WEIGHT_F32) != 0;
  a.shift = ln::past16(x) / (int)es;
  const bool vec = ln::past16(x) == ln::past16(dy) && ln::past16(x) == ln::past16(dx) &&
                   (a.shift != 0 || D % (16 / es) != 0 || ln::past16(weight) == 0);
  int parts = 0;
  rc = (mode & INFINI_F32) ? ln::dispatch<float>(a, vec, true, stream, &parts)
                           : ln::dispatch<__nv_bfloat16>(a, vec, true, stream, &parts);
  if (rc == INFINI_OK) {
    LaunchScope scope(kPhaseBwd, stream);
    ln::ln_reduce_kernel<<<dim3((D + 31) / 32, dbias ? 2 : 1), 1024, 0, stream>>>(a.partial, parts, D, dweight, dbias, a.w32);
    rc = launch_status();
  }
  if (!workspace && cudaFreeAsync(w, stream) != cudaSuccess && rc == INFINI_OK) rc = INFINI_ERR_WORKSPACE;
  return rc;
}

}  // extern "C"
