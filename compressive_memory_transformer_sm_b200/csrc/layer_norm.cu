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
  bool has_bias;  // backward: dbias is wanted
};

// Threads per block: rows of at most a warp share a block of 128, wider rows have a block each.
template <int TPR> constexpr int kBlockThreads = TPR < 128 ? 128 : TPR;
// Elements per thread up to which the weights stay in registers for all the rows of a block.
// (Re-read for each row they cost four times the row itself from L2: 146 us at 32768 x 4096 bf16.)
constexpr int kKeep = 16;

// A thread's part of row `row`; zeros behind the row's end.
template <typename T, int VEC, int TPR, int NV>
__device__ __forceinline__ void load_row(Raw<T, VEC> (&r)[NV], const void* x, long long row, bool active, int lane, int D) {
  const T* p = static_cast<const T*>(x) + row * D;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int at = (v * TPR + lane) * VEC;
    r[v] = Raw<T, VEC>{};
    if (active && at < D) r[v] = load_raw<VEC>(p + at);
  }
}
template <int VEC, int TPR, int NV>
__device__ __forceinline__ void load_weights(Floats<VEC> (&w)[NV], const void* p, bool f32, int lane, int D) {
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int at = (v * TPR + lane) * VEC;
    w[v] = {};
    if (p && at < D) w[v] = load_weight<VEC>(p, f32, at);
  }
}
// xs: the row's elements less their mean, 0 behind its end; returns the variance.
template <typename T, int VEC, int TPR, int NV>
__device__ __forceinline__ float centre(const Raw<T, VEC> (&r)[NV], int lane, int D, float (&xs)[NV][VEC], float* red, int sub, int red_stride) {
  float s[1] = {0.f};
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const Floats<VEC> f = floats(r[v]);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      xs[v][e] = f.v[e];
      s[0] += f.v[e];
    }
  }
  row_sum<TPR>(s, red, sub);
  const float mean = s[0] / (float)D;
  float q[1] = {0.f};
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const bool in = (v * TPR + lane) * VEC < D;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      xs[v][e] = in ? xs[v][e] - mean : 0.f;
      q[0] = fmaf(xs[v][e], xs[v][e], q[0]);
    }
  }
  row_sum<TPR>(q, red + red_stride, sub);
  return q[0] / (float)D;
}

template <typename T, int VEC, int TPR, int NV>
__global__ void __launch_bounds__(kBlockThreads<TPR>) ln_forward_kernel(const Args a) {
  constexpr int TH = kBlockThreads<TPR>, RPB = TH / TPR, NW = TPR > 32 ? TPR / 32 : 1;
  constexpr bool KEEP = NV * VEC <= kKeep;
  __shared__ float red[2 * RPB * NW];
  const int sub = threadIdx.x / TPR, lane = threadIdx.x % TPR;
  const long long step = (long long)gridDim.x * RPB;
  long long row = (long long)blockIdx.x * RPB + sub;
  Raw<T, VEC> next[NV];
  load_row<T, VEC, TPR, NV>(next, a.x, row, row < a.rows, lane, a.D);
  Floats<VEC> w[KEEP ? NV : 1], b[KEEP ? NV : 1];
  if constexpr (KEEP) {
    load_weights<VEC, TPR, NV>(w, a.weight, a.w32, lane, a.D);
    load_weights<VEC, TPR, NV>(b, a.bias, a.w32, lane, a.D);
  }
  for (long long base = (long long)blockIdx.x * RPB; base < a.rows; base += step, row += step) {
    const bool active = row < a.rows;
    Raw<T, VEC> cur[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) cur[v] = next[v];
    load_row<T, VEC, TPR, NV>(next, a.x, row + step, row + step < a.rows, lane, a.D);
    float xs[NV][VEC];
    const float var = centre<T, VEC, TPR, NV>(cur, lane, a.D, xs, red, sub, RPB * NW);
    const float rstd = 1.f / sqrtf(var + a.eps);
    if (!active) continue;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int at = (v * TPR + lane) * VEC;
      if (at < a.D) {
        Floats<VEC> wv, bv = {}, o;
        if constexpr (KEEP) {
          wv = w[v];
          bv = b[v];
        } else {
          wv = load_weight<VEC>(a.weight, a.w32, at);
          if (a.bias) bv = load_weight<VEC>(a.bias, a.w32, at);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) o.v[e] = fmaf(xs[v][e] * rstd, wv.v[e], bv.v[e]);
        store_vec<VEC>(static_cast<T*>(a.y) + row * a.D + at, o);
      }
    }
  }
}

template <typename T, int VEC, int TPR, int NV>
__global__ void __launch_bounds__(kBlockThreads<TPR>) ln_backward_kernel(const Args a) {
  constexpr int TH = kBlockThreads<TPR>, RPB = TH / TPR, NW = TPR > 32 ? TPR / 32 : 1, E = NV * VEC;
  constexpr bool KEEP = E <= kKeep;
  // statistics of the two sums of a row, then (RPB > 1) the rows' accumulators of the block
  __shared__ float red[4 * RPB * NW];
  extern __shared__ float acc[];  // [RPB > 1 ? TPR * E * 2 : 0]
  const int sub = threadIdx.x / TPR, lane = threadIdx.x % TPR;
  const long long step = (long long)gridDim.x * RPB;
  long long row = (long long)blockIdx.x * RPB + sub;
  Raw<T, VEC> nx[NV], nd[NV];
  load_row<T, VEC, TPR, NV>(nx, a.x, row, row < a.rows, lane, a.D);
  load_row<T, VEC, TPR, NV>(nd, a.dy, row, row < a.rows, lane, a.D);
  Floats<VEC> w[KEEP ? NV : 1];
  if constexpr (KEEP) load_weights<VEC, TPR, NV>(w, a.weight, a.w32, lane, a.D);
  float dw[NV][VEC] = {}, db[NV][VEC] = {};
  for (long long base = (long long)blockIdx.x * RPB; base < a.rows; base += step, row += step) {
    const bool active = row < a.rows;
    Raw<T, VEC> cx[NV], cd[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      cx[v] = nx[v];
      cd[v] = nd[v];
    }
    load_row<T, VEC, TPR, NV>(nx, a.x, row + step, row + step < a.rows, lane, a.D);
    load_row<T, VEC, TPR, NV>(nd, a.dy, row + step, row + step < a.rows, lane, a.D);
    float xs[NV][VEC];
    const float var = centre<T, VEC, TPR, NV>(cx, lane, a.D, xs, red, sub, RPB * NW);
    const float rstd = 1.f / sqrtf(var + a.eps);
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int at = (v * TPR + lane) * VEC;
      const Floats<VEC> d = floats(cd[v]);
      Floats<VEC> wv = {};
      if constexpr (KEEP)
        wv = w[v];
      else if (at < a.D)
        wv = load_weight<VEC>(a.weight, a.w32, at);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
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
        const int at = (v * TPR + lane) * VEC;
        if (at < a.D) {
          const Floats<VEC> d = floats(cd[v]);
          Floats<VEC> wv, o;
          if constexpr (KEEP)
            wv = w[v];
          else
            wv = load_weight<VEC>(a.weight, a.w32, at);
#pragma unroll
          for (int e = 0; e < VEC; ++e) o.v[e] = rstd * (d.v[e] * wv.v[e] - m0 - xs[v][e] * m1);
          store_vec<VEC>(static_cast<T*>(a.y) + row * a.D + at, o);
        }
      }
    }
  }
  // the block's sum over its RPB rows in flight, in their order
  if constexpr (RPB > 1) {
    for (int r = RPB - 1; r > 0; --r) {
      __syncthreads();
      if (sub == r)
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            acc[(v * VEC + e) * TPR + lane] = dw[v][e];
            acc[(E + v * VEC + e) * TPR + lane] = db[v][e];
          }
      __syncthreads();
      if (sub == r - 1)
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            dw[v][e] += acc[(v * VEC + e) * TPR + lane];
            db[v][e] += acc[(E + v * VEC + e) * TPR + lane];
          }
    }
  }
  if (sub == 0) {
    float* pw = a.partial + (long long)blockIdx.x * 2 * a.D;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int at = (v * TPR + lane) * VEC + e;
        if (at < a.D) {
          pw[at] = dw[v][e];
          pw[a.D + at] = db[v][e];
        }
      }
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

template <typename T, int VEC, int TPR, int NV> int launch(const Args& a, bool bwd, cudaStream_t st, int* parts) {
  constexpr int TH = kBlockThreads<TPR>, RPB = TH / TPR;
  const long long most = (a.rows + RPB - 1) / RPB;
  if (!bwd) {
    static const int resident = resident_blocks(ln_forward_kernel<T, VEC, TPR, NV>, TH, 0);
    LaunchScope scope(kPhasePre, st);
    ln_forward_kernel<T, VEC, TPR, NV><<<(int)std::min<long long>(most, resident), TH, 0, st>>>(a);
  } else {
    const size_t smem = RPB > 1 ? (size_t)TPR * NV * VEC * 2 * 4 : 0;
    static const int resident = resident_blocks(ln_backward_kernel<T, VEC, TPR, NV>, TH, smem);
    *parts = (int)std::min<long long>(backward_blocks(a.rows, RPB), resident);
    LaunchScope scope(kPhaseBwd, st);
    ln_backward_kernel<T, VEC, TPR, NV><<<*parts, TH, smem, st>>>(a);
  }
  return launch_status();
}

// Threads per row and vectors per thread by the number of vectors of a row.  Scalars (VEC = 1)
// where D is not a multiple of 16 bytes or a pointer is not aligned to them.
template <typename T> int dispatch(const Args& a, bool vec, bool bwd, cudaStream_t st, int* parts) {
  constexpr int V = 16 / sizeof(T);
  const int n = vec ? a.D / V : a.D;
  if (vec) {
    if (n <= 8) return launch<T, V, 8, 1>(a, bwd, st, parts);
    if (n <= 16) return launch<T, V, 16, 1>(a, bwd, st, parts);
    if (n <= 32) return launch<T, V, 32, 1>(a, bwd, st, parts);
    if (n <= 64) return launch<T, V, 32, 2>(a, bwd, st, parts);
    if (n <= 128) return launch<T, V, 64, 2>(a, bwd, st, parts);
    if (n <= 256) return launch<T, V, 128, 2>(a, bwd, st, parts);
    if (n <= 512) return launch<T, V, 256, 2>(a, bwd, st, parts);
    if (n <= 1024) return launch<T, V, 512, 2>(a, bwd, st, parts);
    if (n <= 2048) return launch<T, V, 1024, 2>(a, bwd, st, parts);
    return launch<T, V, 1024, 4>(a, bwd, st, parts);
  }
  if (n <= 128) return launch<T, 1, 32, 4>(a, bwd, st, parts);
  if (n <= 512) return launch<T, 1, 128, 4>(a, bwd, st, parts);
  if (n <= 2048) return launch<T, 1, 256, 8>(a, bwd, st, parts);
  if (n <= 8192) return launch<T, 1, 1024, 8>(a, bwd, st, parts);
  return launch<T, 1, 1024, 16>(a, bwd, st, parts);
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

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
  const bool vec = D % (16 / es) == 0 && ln::aligned16(x) && ln::aligned16(y) && ln::aligned16(weight) &&
                   (!bias || ln::aligned16(bias));
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
  const bool vec = D % (16 / es) == 0 && ln::aligned16(x) && ln::aligned16(dy) && ln::aligned16(dx) && ln::aligned16(weight);
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
