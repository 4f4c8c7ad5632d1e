// Host side of the gated delta rule: infini_attn_gated_delta_forward, _step.
#include <math.h>
#include <string.h>

#include <algorithm>

#include "../../include/infini_attn.h"
#include "common.cuh"
#include "gated_delta.cuh"
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
  rc = check_device(false);
  if (rc != INFINI_OK) return rc;
  RecurArgs a = {};
  a.q = p.q; a.k = p.k; a.v = p.v; a.g = p.g; a.beta = p.beta; a.S = p.S; a.out = p.out; a.lens = p.lens;
  memcpy(a.qs, p.q_stride, sizeof(a.qs));
  memcpy(a.ks, p.k_stride, sizeof(a.ks));
  memcpy(a.vs, p.v_stride, sizeof(a.vs));
  memcpy(a.os, p.o_stride, sizeof(a.os));
  memcpy(a.gs, p.g_stride, sizeof(a.gs));
  memcpy(a.bs, p.beta_stride, sizeof(a.bs));
  a.L = p.L; a.pool = p.B; a.B = p.B; a.H = p.H; a.group = p.H / p.Hk; a.dk = p.dk; a.dv = p.dv;
  a.scale = p.scale != 0.f ? p.scale : 1.f / sqrtf((float)p.dk);
  return launch_recur(a, f32, p.stream);
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
  (void)p;
  return 0;
}

int infini_attn_gated_delta_step(const infini_attn_gated_delta_step_params* p) {
  return p ? gd::step(*p) : INFINI_ERR_INVALID_ARG;
}

size_t infini_attn_gated_delta_params_size(int which) {
  return which == 0 ? sizeof(infini_attn_gated_delta_params) : which == 1 ? sizeof(infini_attn_gated_delta_step_params) : 0;
}

}  // extern "C"
