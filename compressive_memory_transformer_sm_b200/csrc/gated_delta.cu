// Host side of the gated delta rule: infini_attn_gated_delta_forward, _step, _backward.
#include <math.h>
#include <string.h>

#include <algorithm>

#include "../../include/infini_attn.h"
#include "common.cuh"
#include "gated_delta.cuh"
#include "gd_chunk.cuh"
#include "host.h"

namespace infini {
namespace gd {
namespace {

// Strides of (B, heads, L) of a contiguous [B, heads, L, d] tensor where none are given.
void fill_strides(long long st[3], int heads, long long L, int d) {
  if (st[0] == 0 && st[1] == 0 && st[2] == 0) {
    st[2] = d;
    st[1] = L * d;
    st[0] = (long long)heads * L * d;
  }
}

bool fits(const long long st[3], int B, int heads, long long L) {
  // offsets of the last row stay far inside 64 bits
  const long long lim = 1LL << 60;
  return st[0] >= 0 && st[1] >= 0 && st[2] >= 0 && (B == 1 || st[0] <= lim / B) && (heads == 1 || st[1] <= lim / heads) &&
         (L == 1 || st[2] <= lim / L);
}

size_t extent(const long long st[3], int B, int heads, long long L, int d, size_t es) {
  return (size_t)((B - 1) * st[0] + (heads - 1) * st[1] + (L - 1) * st[2] + d) * es;
}

// Whether no two rows of a written tensor share an element.
bool rows_apart(const long long st[3], int B, int heads, long long L, int d) {
  std::pair<long long, long long> dim[3] = {{st[0], B}, {st[1], heads}, {st[2], L}};
  std::sort(dim, dim + 3);
  long long reach = d;
  for (const auto& x : dim) {
    if (x.second == 1) continue;
    if (x.first < reach) return false;
    reach = x.first * (x.second - 1) + reach;
  }
  return true;
}

struct Shape {
  int B, H, Hk, dk, dv, mode;
  long long L;
};

int check_shape(const Shape& s) {
  if (s.B <= 0 || s.H <= 0 || s.Hk <= 0 || s.L <= 0 || s.dk <= 0 || s.dv <= 0 || s.H % s.Hk != 0) return INFINI_ERR_INVALID_ARG;
  if ((s.mode & ~INFINI_F32) != 0 || s.dk > kMaxHead || s.dv > kMaxHead) return INFINI_ERR_UNSUPPORTED;
  if (s.B > 65535 || s.H > 65535 || s.L > (1LL << 31) - 1 || (long long)s.B * s.H > (1LL << 30) / 64) return INFINI_ERR_UNSUPPORTED;
  return INFINI_OK;
}

bool space_ok(const void* ws, size_t bytes, size_t need) {
  return !ws || (bytes >= need && reinterpret_cast<uintptr_t>(ws) % kAlign == 0);
}

int launch_recur(const RecurArgs& a, bool f32, cudaStream_t st) {
  const bool vec = a.dv % 4 == 0 && reinterpret_cast<uintptr_t>(a.S) % 16 == 0;
  const dim3 grid((a.dv + kRecurCols - 1) / kRecurCols, a.H, a.B);
  LaunchScope scope(kPhaseUpdate, st);
  if (f32)
    vec ? recur_kernel<float, true><<<grid, kRecurThreads, 0, st>>>(a) : recur_kernel<float, false><<<grid, kRecurThreads, 0, st>>>(a);
  else
    vec ? recur_kernel<__nv_bfloat16, true><<<grid, kRecurThreads, 0, st>>>(a)
        : recur_kernel<__nv_bfloat16, false><<<grid, kRecurThreads, 0, st>>>(a);
  return launch_status();
}

// Whether rows of d elements can be read and written 16 bytes at a time.
bool rows_vec(const void* p, const long long st[3], int d, size_t es) {
  const long long v = 16 / (long long)es;
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && d % v == 0 && st[0] % v == 0 && st[1] % v == 0 && st[2] % v == 0;
}

// ---------------------------------------------------------------- chunked
int padded_dk(int dk) { return dk <= 64 ? 64 : 128; }
int col_warps(int dv) { return (dv + 15) / 16; }

int out_parts(int mode) { return (mode & INFINI_F32) ? 3 : 2; }

// Microseconds of a pass with outputs of `strips` groups of 16 columns over n chunks, as measured (128 x 128 bf16): a
// strip per SM 2.3 a chunk, two 3.8, four 5.3, and from there 9.2 per thousand strips.
double pass_time(double strips, double n) {
  return n * (strips <= kSms ? 2.3 : strips <= 2 * kSms ? 3.8 : std::max(5.3, 0.0092 * strips));
}
// Chunks per segment.  Segments run side by side, but all of them twice, and the first time with the unit vectors'
// columns too: it pays where few (b, h) leave most SMs without work.  Measured at B 1, H 8, 512 chunks: forward 1174 us
// in one piece, 820 in segments of 64; both passes of the backward, which fill the SMs better, 1403 and 1789.  For fp32 and
// 64-row states the same model: whole calls in one piece and as it chooses, fp32 128 x 128, 8 heads x 32768 tokens 3399
// and 2859, 1 x 4096 402 and 148; 64 x 64, 8 x 32768 1072 and 394 (bf16), 1729 and 771 (fp32), 16 x 16384 953 and 717;
// backward fp32 128 x 128, 3 x 16384 2236 and 2194, 64 x 64, 8 x 8192 904 and 922 (the one of 44 where it lost).
int segment_chunks(const Shape& s, long long chunks, bool bwd) {
  const double strips = (double)s.B * s.H * col_warps(s.dv), unit = (double)s.B * s.H * padded_dk(s.dk) / 16;
  const double whole = bwd ? 1.2 * pass_time(2 * strips, (double)chunks) : pass_time(strips, (double)chunks);
  double best = 0.9 * whole;
  long long seg = chunks;
  for (long long n = 3; n <= 32 && chunks / n >= 4; ++n) {
    const double each = (double)((chunks + n - 1) / n);
    const double again = bwd ? 1.2 * pass_time(2 * n * strips, each) : pass_time(n * strips, each);
    const double first = (bwd ? 1.2 : 0.9) * pass_time((n - 1) * (bwd ? 2 * strips + unit : strips + unit), each);
    const double t = first + again + 5.5 * n + 10.;
    if (t < best) {
      best = t;
      seg = (chunks + n - 1) / n;
    }
  }
  return (int)seg;
}

// Workspace of nc chunks of every (b, h).
struct ChunkSpace {
  size_t T, P, vec, G, snap, dsnap, acc, segS, segD, segA, bytes;
  int seg;
  bool split;
  ChunkSpace(const Shape& s, long long nc, bool bwd) {
    const size_t n = (size_t)s.B * s.H * nc, state = (size_t)col_warps(s.dv) * padded_dk(s.dk) * 16 * 4;
    size_t at = 0;
    auto take = [&](size_t bytes) {
      const size_t was = at;
      at += align_up(bytes);
      return was;
    };
    T = take(n * 3 * kTri * 2);
    P = take(n * (bwd ? 3 : out_parts(s.mode)) * kTri * 2);
    vec = take(n * kVec * 4);
    G = take(n * kC * 8);
    snap = take(bwd ? n * state : 0);
    dsnap = take(bwd ? n * state : 0);
    // Few chunks: a block per value head (B 3, H 24, 6 key heads, L 20: the four heads of 18 blocks in turn take 159 us
    // of the backward, side by side 80; with a block per SM and more already, the sum only costs).
    split = bwd && s.H > s.Hk && (long long)s.B * s.Hk * nc < kSms;
    acc = take(bwd && s.H > s.Hk ? (size_t)s.B * (split ? s.H : s.Hk) * nc * 2 * kC * padded_dk(s.dk) * 4 : 0);
    seg = segment_chunks(s, nc, bwd);
    const size_t nseg = (nc + seg - 1) / seg, m = nseg > 1 ? (size_t)s.B * s.H * nseg : 0;
    segS = take(m * state);
    segD = take(bwd ? m * state : 0);
    segA = take(m * padded_dk(s.dk) * padded_dk(s.dk) * 4);
    bytes = at;
  }
  void place(ChunkArgs& a, void* ws) const {
    char* w = static_cast<char*>(ws);
    a.T = reinterpret_cast<bf16*>(w + T);
    a.P = reinterpret_cast<bf16*>(w + P);
    a.vec = reinterpret_cast<float*>(w + vec);
    a.G = reinterpret_cast<float2*>(w + G);
    a.snap = reinterpret_cast<float4*>(w + snap);
    a.dsnap = reinterpret_cast<float4*>(w + dsnap);
    a.acc = reinterpret_cast<float*>(w + acc);
    a.segS = reinterpret_cast<float4*>(w + segS);
    a.segD = reinterpret_cast<float4*>(w + segD);
    a.segA = reinterpret_cast<float4*>(w + segA);
    a.seg = seg;
    a.split = split;
  }
};

constexpr int kMaxSmem = 232448;  // per block

// The forward works through a long sequence in slabs of chunks, so that its workspace stays below this.
constexpr size_t kSlabBytes = size_t(1) << 30;
long long all_chunks(const Shape& s) { return (s.L + kC - 1) / kC; }
long long slab_chunks(const Shape& s) {
  const size_t one = (size_t)s.B * s.H * ((3 + out_parts(s.mode)) * kTri * 2 + kVec * 4 + kC * 8);
  return std::max<long long>(1, std::min<long long>(all_chunks(s), (long long)(kSlabBytes / one)));
}

// The dynamic shared-memory limit is an attribute of a function in the current context: raised to all there is once for
// every context (and thread).
template <typename... A> int launch_chunk(void (*kernel)(A...), dim3 grid, int threads, size_t smem, int phase, const ChunkArgs& a,
                                          unsigned long long* raised, cudaStream_t st) {
  const unsigned long long ctx = current_context_id();
  if (ctx == 0 || *raised != ctx) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e != cudaSuccess) return note_cuda_error(e);
    *raised = ctx;
  }
  LaunchScope scope(phase, st);
  kernel<<<grid, threads, smem, st>>>(a);
  return launch_status();
}
// (kernel, grid, threads, shared memory, phase, arguments, stream), with the kernel's own note of the context
#define GD_LAUNCH(kernel, grid, threads, smem, phase, a, st)              \
  [&] {                                                                   \
    static thread_local unsigned long long raised = 0;                    \
    return launch_chunk(kernel, grid, threads, smem, phase, a, &raised, st); \
  }()

// Shape of a state block.  KS 4: four warps to 16 value columns, for the shortest time per chunk; KS 1: one warp, less
// exchange, for the most chunks per SM.  As few groups per block as keep the blocks within one per SM.
struct StatePlan {
  int KS, groups, stages, blocks, threads, first_loader;
  size_t smem;
};
template <typename T, int DK, int PP> StatePlan state_plan(int nw, long long heads) {
  StatePlan p = {};
  p.KS = heads * nw <= 2 * kSms ? 4 : 1;
  const int most = p.KS == 4 ? 2 : kMaxGroups;
  p.groups = 1;
  while (p.groups < most && p.groups < nw && heads * ((nw + p.groups - 1) / p.groups) > kSms) p.groups *= 2;
  p.blocks = (nw + p.groups - 1) / p.groups;
  const size_t one = stage_bytes<T, DK, PP>(p.groups), ex = p.KS == 4 ? p.groups * sizeof(Exchange<DK, Dims<T, DK>::kOut>) : 0;
  const bool alone = heads * p.blocks <= kSms;  // a block per SM: two stages, and four warps that only copy
  p.stages = alone && 2 * one + ex <= (size_t)kMaxSmem ? 2 : 1;
  p.smem = p.stages * one + ex;
  p.first_loader = alone ? std::max(128, 32 * p.KS * p.groups) : 0;
  p.threads = alone ? p.first_loader + 128 : 32 * p.KS * p.groups;
  return p;
}

void take_plan(ChunkArgs& a, const StatePlan& p) {
  a.groups = p.groups;
  a.stages = p.stages;
  a.blocks = p.blocks;
  a.first_loader = p.first_loader;
}

template <typename T, int DK, int PP> int run_prep(const ChunkArgs& a, cudaStream_t st) {
  return GD_LAUNCH((prep_kernel<T, DK, PP>), dim3(a.nc, a.H, a.B), 256, sizeof(PrepSmem<T, DK>), kPhaseUpdate, a, st);
}
template <typename T, int DK, int MODE> int run_forward(ChunkArgs a, int segments, int strips, cudaStream_t st) {
  const StatePlan p = state_plan<T, DK, Dims<T, DK>::kOut>(strips, (long long)a.B * a.H * segments);
  take_plan(a, p);
  const dim3 grid(p.blocks * segments, a.H, a.B);
  return p.KS == 4 ? GD_LAUNCH((forward_kernel<T, DK, 4, MODE>), grid, p.threads, p.smem, kPhaseState, a, st)
                   : GD_LAUNCH((forward_kernel<T, DK, 1, MODE>), grid, p.threads, p.smem, kPhaseState, a, st);
}
template <typename T, int DK, bool SEG> int run_both(ChunkArgs a, int strips, cudaStream_t st) {
  const StatePlan p = state_plan<T, DK, 3>(strips, 2LL * a.B * a.H * a.nseg);
  take_plan(a, p);
  const dim3 grid(p.blocks * a.nseg, a.H, 2 * a.B);
  return p.KS == 4 ? GD_LAUNCH((both_kernel<T, DK, 4, SEG>), grid, p.threads, p.smem, kPhaseBwd, a, st)
                   : GD_LAUNCH((both_kernel<T, DK, 1, SEG>), grid, p.threads, p.smem, kPhaseBwd, a, st);
}
template <int DK> int run_combine(const ChunkArgs& a, int both, cudaStream_t st) {
  if (a.nseg < 3) return INFINI_OK;
  LaunchScope scope(kPhaseState, st);
  combine_kernel<DK><<<dim3((1 + both) * col_warps(a.dv), a.H, a.B), 128, 0, st>>>(a, both);
  return launch_status();
}
template <typename T, int DK> int chunk_forward(ChunkArgs a, long long chunks, long long slab, cudaStream_t st) {
  const int nw = col_warps(a.dv);
  for (long long c = 0; c < chunks; c += slab) {
    a.c0 = (int)c;
    a.nc = (int)std::min(slab, chunks - c);
    a.nseg = (a.nc + a.seg - 1) / a.seg;
    int rc = run_prep<T, DK, Dims<T, DK>::kOut>(a, st);
    if (rc == INFINI_OK && a.nseg > 1) {
      rc = run_forward<T, DK, kPassSeg>(a, a.nseg - 1, nw + DK / 16, st);
      if (rc == INFINI_OK) rc = run_combine<DK>(a, 0, st);
    }
    if (rc == INFINI_OK) rc = run_forward<T, DK, kPassOut>(a, a.nseg, nw, st);
    if (rc != INFINI_OK) return rc;
  }
  return INFINI_OK;
}
template <typename T, int DK> int chunk_backward(ChunkArgs a, cudaStream_t st) {
  const int nw = col_warps(a.dv);
  a.nseg = (a.nc + a.seg - 1) / a.seg;
  int rc = run_prep<T, DK, 3>(a, st);
  if (rc == INFINI_OK && a.nseg > 1) {
    rc = run_both<T, DK, true>(a, nw + DK / 16, st);
    if (rc == INFINI_OK) rc = run_combine<DK>(a, 1, st);
  }
  if (rc == INFINI_OK) rc = run_both<T, DK, false>(a, nw, st);
  if (rc != INFINI_OK) return rc;
  const dim3 chunks(a.nc, a.split ? a.H : a.Hk, a.B);
  if constexpr (sizeof(T) == 2)
    rc = GD_LAUNCH((grad_bf16_kernel<DK>), chunks, 512, sizeof(GradSmemB<DK>), kPhaseBwd, a, st);
  else
    rc = GD_LAUNCH((grad_kernel<T, DK>), chunks, 256, sizeof(GradSmem<T, DK>), kPhaseBwd, a, st);
  if (rc != INFINI_OK || !a.split) return rc;
  LaunchScope scope(kPhaseBwd, st);
  sum_heads_kernel<T, DK><<<dim3(a.nc, a.Hk, a.B), 256, 0, st>>>(a);
  return launch_status();
}

// Sequences of fewer tokens than this go token by token (128 x 128, microseconds, tokens against a chunk of 64: bf16, 8
// heads, 20 tokens 13.4 / 13.8; 128 heads, 10 tokens 20.5 / 22.6, 16 tokens 30.7 / 22.6; fp32, 8 heads, 31 tokens
// 19.3 / 22.2; 128 heads 57 / 72).  The switch lies between the 8 and the 128 heads that were measured.
long long chunk_from(const Shape& s) {
  if (s.mode & INFINI_F32) return 36;
  return (long long)s.B * s.H <= kSms / 4 ? 20 : 11;
}

int forward(infini_attn_gated_delta_params p) {
  if (!p.q || !p.k || !p.v || !p.g || !p.beta || !p.S || !p.out) return INFINI_ERR_INVALID_ARG;
  int rc = check_shape({p.B, p.H, p.Hk, p.dk, p.dv, p.mode, p.L});
  if (rc != INFINI_OK) return rc;
  fill_strides(p.q_stride, p.Hk, p.L, p.dk);
  fill_strides(p.k_stride, p.Hk, p.L, p.dk);
  fill_strides(p.v_stride, p.H, p.L, p.dv);
  fill_strides(p.o_stride, p.H, p.L, p.dv);
  fill_strides(p.g_stride, p.H, p.L, 1);
  fill_strides(p.beta_stride, p.H, p.L, 1);
  if (!fits(p.q_stride, p.B, p.Hk, p.L) || !fits(p.k_stride, p.B, p.Hk, p.L) || !fits(p.v_stride, p.B, p.H, p.L) ||
      !fits(p.o_stride, p.B, p.H, p.L) || !fits(p.g_stride, p.B, p.H, p.L) || !fits(p.beta_stride, p.B, p.H, p.L) ||
      !rows_apart(p.o_stride, p.B, p.H, p.L, p.dv))
    return INFINI_ERR_INVALID_ARG;
  const bool f32 = (p.mode & INFINI_F32) != 0;
  const size_t es = f32 ? 4 : 2;
  struct Range {
    const void* p;
    size_t n;
  };
  const size_t nS = (size_t)p.B * p.H * p.dk * p.dv * 4;
  const Range out{p.out, extent(p.o_stride, p.B, p.H, p.L, p.dv, es)}, S{p.S, nS};
  const Range ins[6] = {{p.q, extent(p.q_stride, p.B, p.Hk, p.L, p.dk, es)}, {p.k, extent(p.k_stride, p.B, p.Hk, p.L, p.dk, es)},
                        {p.v, extent(p.v_stride, p.B, p.H, p.L, p.dv, es)},  {p.g, extent(p.g_stride, p.B, p.H, p.L, 1, 4)},
                        {p.beta, extent(p.beta_stride, p.B, p.H, p.L, 1, 4)}, {p.lens, p.lens ? (size_t)p.B * 4 : 0}};
  for (const Range& x : ins)
    if (x.p && (ranges_overlap(out.p, out.n, x.p, x.n) || ranges_overlap(S.p, S.n, x.p, x.n))) return INFINI_ERR_INVALID_ARG;
  if (ranges_overlap(out.p, out.n, S.p, S.n)) return INFINI_ERR_INVALID_ARG;
  if (!space_ok(p.workspace, p.workspace_bytes, infini_attn_gated_delta_workspace_size(&p))) return INFINI_ERR_WORKSPACE;
  rc = check_device(false);
  if (rc != INFINI_OK) return rc;
  const Shape shape{p.B, p.H, p.Hk, p.dk, p.dv, p.mode, p.L};
  const float scale = p.scale != 0.f ? p.scale : 1.f / sqrtf((float)p.dk);
  if (p.L >= chunk_from(shape)) {
    const long long slab = slab_chunks(shape);
    const ChunkSpace space(shape, slab, false);
    void* w = p.workspace;
    if (!w && !ws_alloc(&w, space.bytes, p.stream)) return INFINI_ERR_WORKSPACE;
    ChunkArgs a = {};
    a.q = p.q; a.k = p.k; a.v = p.v; a.g = p.g; a.beta = p.beta; a.lens = p.lens; a.S = p.S; a.out = p.out;
    memcpy(a.qs, p.q_stride, sizeof(a.qs));
    memcpy(a.ks, p.k_stride, sizeof(a.ks));
    memcpy(a.vs, p.v_stride, sizeof(a.vs));
    memcpy(a.os, p.o_stride, sizeof(a.os));
    memcpy(a.gs, p.g_stride, sizeof(a.gs));
    memcpy(a.bs, p.beta_stride, sizeof(a.bs));
    a.L = p.L; a.B = p.B; a.H = p.H; a.Hk = p.Hk; a.group = p.H / p.Hk; a.dk = p.dk; a.dv = p.dv; a.scale = scale;
    a.vec_k = rows_vec(p.q, p.q_stride, p.dk, es) && rows_vec(p.k, p.k_stride, p.dk, es);
    a.vec_v = rows_vec(p.v, p.v_stride, p.dv, es);
    a.vec_o = rows_vec(p.out, p.o_stride, p.dv, es);
    space.place(a, w);
    const bool wide = padded_dk(p.dk) == 128;
    const long long n = all_chunks(shape);
    rc = f32 ? wide ? chunk_forward<float, 128>(a, n, slab, p.stream) : chunk_forward<float, 64>(a, n, slab, p.stream)
             : wide ? chunk_forward<bf16, 128>(a, n, slab, p.stream) : chunk_forward<bf16, 64>(a, n, slab, p.stream);
    if (!p.workspace && cudaFreeAsync(w, p.stream) != cudaSuccess && rc == INFINI_OK) rc = INFINI_ERR_WORKSPACE;
    return rc;
  }
  RecurArgs a = {};
  a.q = p.q; a.k = p.k; a.v = p.v; a.g = p.g; a.beta = p.beta; a.S = p.S; a.out = p.out; a.lens = p.lens;
  memcpy(a.qs, p.q_stride, sizeof(a.qs));
  memcpy(a.ks, p.k_stride, sizeof(a.ks));
  memcpy(a.vs, p.v_stride, sizeof(a.vs));
  memcpy(a.os, p.o_stride, sizeof(a.os));
  memcpy(a.gs, p.g_stride, sizeof(a.gs));
  memcpy(a.bs, p.beta_stride, sizeof(a.bs));
  a.L = p.L; a.pool = p.B; a.B = p.B; a.H = p.H; a.group = p.H / p.Hk; a.dk = p.dk; a.dv = p.dv;
  a.scale = scale;
  return launch_recur(a, f32, p.stream);
}

int backward(infini_attn_gated_delta_backward_params p) {
  if (!p.q || !p.k || !p.v || !p.g || !p.beta || !p.d_out || !p.dq || !p.dk_out || !p.dv_out || !p.dg || !p.dbeta)
    return INFINI_ERR_INVALID_ARG;
  const Shape shape{p.B, p.H, p.Hk, p.dk, p.dv, p.mode, p.L};
  int rc = check_shape(shape);
  if (rc != INFINI_OK) return rc;
  fill_strides(p.q_stride, p.Hk, p.L, p.dk);
  fill_strides(p.k_stride, p.Hk, p.L, p.dk);
  fill_strides(p.v_stride, p.H, p.L, p.dv);
  fill_strides(p.d_out_stride, p.H, p.L, p.dv);
  fill_strides(p.g_stride, p.H, p.L, 1);
  fill_strides(p.beta_stride, p.H, p.L, 1);
  if (!fits(p.q_stride, p.B, p.Hk, p.L) || !fits(p.k_stride, p.B, p.Hk, p.L) || !fits(p.v_stride, p.B, p.H, p.L) ||
      !fits(p.d_out_stride, p.B, p.H, p.L) || !fits(p.g_stride, p.B, p.H, p.L) || !fits(p.beta_stride, p.B, p.H, p.L))
    return INFINI_ERR_INVALID_ARG;
  if (p.B > 32767) return INFINI_ERR_UNSUPPORTED;  // two grid rows per batch row
  const bool f32 = (p.mode & INFINI_F32) != 0;
  const size_t es = f32 ? 4 : 2, tok = (size_t)p.B * p.L, nS = (size_t)p.B * p.H * p.dk * p.dv * 4;
  struct Range {
    const void* p;
    size_t n;
  };
  const Range ins[9] = {{p.q, extent(p.q_stride, p.B, p.Hk, p.L, p.dk, es)}, {p.k, extent(p.k_stride, p.B, p.Hk, p.L, p.dk, es)},
                        {p.v, extent(p.v_stride, p.B, p.H, p.L, p.dv, es)},  {p.d_out, extent(p.d_out_stride, p.B, p.H, p.L, p.dv, es)},
                        {p.g, extent(p.g_stride, p.B, p.H, p.L, 1, 4)},      {p.beta, extent(p.beta_stride, p.B, p.H, p.L, 1, 4)},
                        {p.S0, p.S0 ? nS : 0}, {p.dS_L, p.dS_L ? nS : 0},    {p.lens, p.lens ? (size_t)p.B * 4 : 0}};
  const Range outs[6] = {{p.dq, tok * p.Hk * p.dk * es}, {p.dk_out, tok * p.Hk * p.dk * es}, {p.dv_out, tok * p.H * p.dv * es},
                         {p.dg, tok * p.H * 4},          {p.dbeta, tok * p.H * 4},           {p.dS0, p.dS0 ? nS : 0}};
  for (int i = 0; i < 6; ++i) {
    for (const Range& x : ins)
      if (x.p && outs[i].p && ranges_overlap(outs[i].p, outs[i].n, x.p, x.n)) return INFINI_ERR_INVALID_ARG;
    for (int j = i + 1; j < 6; ++j)
      if (outs[i].p && outs[j].p && ranges_overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return INFINI_ERR_INVALID_ARG;
  }
  const long long n = all_chunks(shape);
  const ChunkSpace space(shape, n, true);
  if (!space_ok(p.workspace, p.workspace_bytes, space.bytes)) return INFINI_ERR_WORKSPACE;
  rc = check_device(false);
  if (rc != INFINI_OK) return rc;
  void* w = p.workspace;
  if (!w && !ws_alloc(&w, space.bytes, p.stream)) return INFINI_ERR_WORKSPACE;
  ChunkArgs a = {};
  a.q = p.q; a.k = p.k; a.v = p.v; a.g = p.g; a.beta = p.beta; a.lens = p.lens; a.d_out = p.d_out; a.S0 = p.S0; a.dS = p.dS_L;
  a.dq = p.dq; a.dkk = p.dk_out; a.dvv = p.dv_out; a.dg = p.dg; a.dbeta = p.dbeta; a.dS0 = p.dS0;
  memcpy(a.qs, p.q_stride, sizeof(a.qs));
  memcpy(a.ks, p.k_stride, sizeof(a.ks));
  memcpy(a.vs, p.v_stride, sizeof(a.vs));
  memcpy(a.os, p.d_out_stride, sizeof(a.os));
  memcpy(a.gs, p.g_stride, sizeof(a.gs));
  memcpy(a.bs, p.beta_stride, sizeof(a.bs));
  a.L = p.L; a.B = p.B; a.H = p.H; a.Hk = p.Hk; a.group = p.H / p.Hk; a.dk = p.dk; a.dv = p.dv;
  a.scale = p.scale != 0.f ? p.scale : 1.f / sqrtf((float)p.dk);
  a.vec_k = rows_vec(p.q, p.q_stride, p.dk, es) && rows_vec(p.k, p.k_stride, p.dk, es);
  a.vec_v = rows_vec(p.v, p.v_stride, p.dv, es);
  a.vec_o = rows_vec(p.d_out, p.d_out_stride, p.dv, es);
  auto aligned = [](const void* x, int to) { return reinterpret_cast<uintptr_t>(x) % to == 0; };
  a.vec_dq = p.dk % 2 == 0 && aligned(p.dq, 4) && aligned(p.dk_out, 4);
  a.vec_dv = p.dv % 8 == 0 && aligned(p.dv_out, 16);
  a.nc = (int)n;
  space.place(a, w);
  const bool wide = padded_dk(p.dk) == 128;
  rc = f32 ? wide ? chunk_backward<float, 128>(a, p.stream) : chunk_backward<float, 64>(a, p.stream)
           : wide ? chunk_backward<bf16, 128>(a, p.stream) : chunk_backward<bf16, 64>(a, p.stream);
  if (!p.workspace && cudaFreeAsync(w, p.stream) != cudaSuccess && rc == INFINI_OK) rc = INFINI_ERR_WORKSPACE;
  return rc;
}

int step(const infini_attn_gated_delta_step_params& p) {
  if (!p.q || !p.k || !p.v || !p.g || !p.beta || !p.S || !p.out) return INFINI_ERR_INVALID_ARG;
  int rc = check_shape({p.B, p.H, p.Hk, p.dk, p.dv, p.mode, 1});
  if (rc != INFINI_OK) return rc;
  if (p.pool <= 0 || (!p.slots && p.pool < p.B)) return INFINI_ERR_INVALID_ARG;
  if (p.pool > (1LL << 50) / ((long long)p.H * p.dk * p.dv)) return INFINI_ERR_UNSUPPORTED;
  RecurArgs a = {};
  auto take = [](long long dst[3], const long long src[2], int heads, int d) {
    dst[0] = src[0];
    dst[1] = src[1];
    if (dst[0] == 0 && dst[1] == 0) {
      dst[1] = d;
      dst[0] = (long long)heads * d;
    }
  };
  take(a.qs, p.q_stride, p.Hk, p.dk);
  take(a.ks, p.k_stride, p.Hk, p.dk);
  take(a.vs, p.v_stride, p.H, p.dv);
  take(a.os, p.o_stride, p.H, p.dv);
  take(a.gs, p.g_stride, p.H, 1);
  take(a.bs, p.beta_stride, p.H, 1);
  if (!fits(a.qs, p.B, p.Hk, 1) || !fits(a.ks, p.B, p.Hk, 1) || !fits(a.vs, p.B, p.H, 1) || !fits(a.os, p.B, p.H, 1) ||
      !fits(a.gs, p.B, p.H, 1) || !fits(a.bs, p.B, p.H, 1) || !rows_apart(a.os, p.B, p.H, 1, p.dv))
    return INFINI_ERR_INVALID_ARG;
  const bool f32 = (p.mode & INFINI_F32) != 0;
  const size_t es = f32 ? 4 : 2, nS = (size_t)p.pool * p.H * p.dk * p.dv * 4;
  const size_t no = extent(a.os, p.B, p.H, 1, p.dv, es);
  const struct {
    const void* p;
    size_t n;
  } ins[6] = {{p.q, extent(a.qs, p.B, p.Hk, 1, p.dk, es)}, {p.k, extent(a.ks, p.B, p.Hk, 1, p.dk, es)},
              {p.v, extent(a.vs, p.B, p.H, 1, p.dv, es)},  {p.g, extent(a.gs, p.B, p.H, 1, 1, 4)},
              {p.beta, extent(a.bs, p.B, p.H, 1, 1, 4)},   {p.slots, p.slots ? (size_t)p.B * 4 : 0}};
  for (const auto& x : ins)
    if (x.p && (ranges_overlap(p.out, no, x.p, x.n) || ranges_overlap(p.S, nS, x.p, x.n))) return INFINI_ERR_INVALID_ARG;
  if (ranges_overlap(p.out, no, p.S, nS)) return INFINI_ERR_INVALID_ARG;
  rc = check_device(false);
  if (rc != INFINI_OK) return rc;
  a.q = p.q; a.k = p.k; a.v = p.v; a.g = p.g; a.beta = p.beta; a.S = p.S; a.out = p.out; a.slots = p.slots;
  a.L = 1; a.pool = p.pool; a.B = p.B; a.H = p.H; a.group = p.H / p.Hk; a.dk = p.dk; a.dv = p.dv;
  a.scale = p.scale != 0.f ? p.scale : 1.f / sqrtf((float)p.dk);
  return launch_recur(a, f32, p.stream);
}

}  // namespace
}  // namespace gd

}  // namespace infini

using namespace infini;

extern "C" {

int infini_attn_gated_delta_forward(const infini_attn_gated_delta_params* p) {
  return p ? gd::forward(*p) : INFINI_ERR_INVALID_ARG;
}

size_t infini_attn_gated_delta_workspace_size(const infini_attn_gated_delta_params* p) {
  if (!p) return 0;
  const gd::Shape s{p->B, p->H, p->Hk, p->dk, p->dv, p->mode, p->L};
  if (gd::check_shape(s) != INFINI_OK || p->L < gd::chunk_from(s)) return 0;
  return gd::ChunkSpace(s, gd::slab_chunks(s), false).bytes;
}

int infini_attn_gated_delta_backward(const infini_attn_gated_delta_backward_params* p) {
  return p ? gd::backward(*p) : INFINI_ERR_INVALID_ARG;
}

size_t infini_attn_gated_delta_backward_workspace_size(const infini_attn_gated_delta_backward_params* p) {
  if (!p) return 0;
  const gd::Shape s{p->B, p->H, p->Hk, p->dk, p->dv, p->mode, p->L};
  return gd::check_shape(s) == INFINI_OK ? gd::ChunkSpace(s, gd::all_chunks(s), true).bytes : 0;
}

int infini_attn_gated_delta_step(const infini_attn_gated_delta_step_params* p) {
  return p ? gd::step(*p) : INFINI_ERR_INVALID_ARG;
}

size_t infini_attn_gated_delta_params_size(int which) {
  return which == 0   ? sizeof(infini_attn_gated_delta_params)
         : which == 1 ? sizeof(infini_attn_gated_delta_step_params)
         : which == 2 ? sizeof(infini_attn_gated_delta_backward_params)
                      : 0;
}

}  // extern "C"
