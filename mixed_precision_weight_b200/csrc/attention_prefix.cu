// KV-BSS decode attention over the 8-bit paged cache (Spark card, "2. KV-BSS:
// Key-Value Binding Softmax Sharpening"), for one query token per sequence
// with grouped-query heads, over an optional prefix that all sequences share
// and each sequence's own keys:
//   s_l = (q . k_l) tau / sqrt(d),  m = max_l s_l,
//   p_l = exp(s_l - m) if s_l >= m - haze else 0,  out = sum_l p_l v_l / sum_l p_l
// with k_l = ks_l kc_l and v_l = vs_l vc_l.  The haze threshold needs the final
// maximum before any weight is known, so the logits are formed in a first pass.
//   pfx_logits  one CTA per (page, KV head, sequence): a warp per key
//   pfx_out     one CTA per (query head, sequence): maximum, weights, sum p v
#include "common.cuh"
#include "kernels.h"

namespace dvssq {

struct PfxParams {
  const uint16_t *q;
  long long q_bs, q_hs;
  const int8_t *k, *v;
  const uint16_t *ks, *vs;
  const int32_t *table, *ptable, *lens;
  void *out;
  int out_bf16;
  float *logit;                  // [B][Hq][PL + ctx]
  int B, Hq, H, G, W, n_pages, ctx, prefix, ppages;
  float scale, haze;
};

__device__ __forceinline__ int pfx_len(const PfxParams &p, int b) {
  const int n = p.lens[b];
  if (n < 0 || n > p.ctx) set_error(kErrBadIndex);
  return max(0, min(n, p.ctx));
}

template <int D>
__global__ void __launch_bounds__(128) pfx_logits_kernel(const PfxParams p) {
  constexpr int VPL = D / 32;
  const int w = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool pre = w < p.ppages;
  const int own = w - p.ppages, keys = pre ? p.prefix - 64 * w : pfx_len(p, b) - 64 * own;
  if (keys <= 0) return;
  const int page = pre ? p.ptable[w] : p.table[(size_t)b * p.W + own];
  const bool ok = page >= 0 && page < p.n_pages;
  if (!ok) set_error(kErrBadIndex);
  const size_t ph = (size_t)(ok ? page : 0) * p.H + h;
  for (int i = warp; i < min(keys, 64); i += 4) {
    const float ks = bf16_bits_to_f32(p.ks[ph * 64 + i]);
    float kf[VPL];
    for (int u = 0; u < VPL; ++u) kf[u] = (float)p.k[(ph * 64 + i) * D + lane * VPL + u];
    for (int g = 0; g < p.G; ++g) {
      const uint16_t *q = p.q + b * p.q_bs + (h * p.G + g) * p.q_hs + lane * VPL;
      float s = 0.f;
      for (int u = 0; u < VPL; ++u) s = fmaf(bf16_bits_to_f32(q[u]), kf[u], s);
      for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (lane == 0)
        p.logit[((size_t)b * p.Hq + h * p.G + g) * (64 * p.ppages + p.ctx) + 64 * w + i] =
            ok ? s * ks * p.scale : -INFINITY;
    }
  }
}

template <int D>
__global__ void __launch_bounds__(D) pfx_out_kernel(const PfxParams p) {
  __shared__ float red[32], wt[64];
  const int hq = blockIdx.x, b = blockIdx.y, h = hq / p.G, tid = threadIdx.x;
  const int len = pfx_len(p, b), n = 64 * p.ppages + len;
  const float *lg = p.logit + ((size_t)b * p.Hq + hq) * (64 * p.ppages + p.ctx);
  auto live = [&](int i) { return i < p.prefix || i >= 64 * p.ppages; };
  float m = -INFINITY;
  for (int i = tid; i < n; i += D)
    if (live(i)) m = fmaxf(m, lg[i]);
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((tid & 31) == 0) red[tid >> 5] = m;
  __syncthreads();
  m = -INFINITY;
  for (int i = 0; i < D / 32; ++i) m = fmaxf(m, red[i]);
  float acc = 0.f, sum = 0.f;
  for (int w = 0; 64 * w < n; ++w) {
    const bool pre = w < p.ppages;
    const int page = pre ? p.ptable[w] : p.table[(size_t)b * p.W + w - p.ppages];
    if (page < 0 || page >= p.n_pages) continue;
    const size_t ph = (size_t)page * p.H + h;
    __syncthreads();
    if (tid < 64) {
      const int i = 64 * w + tid;
      const float s = i < n && live(i) ? lg[i] : -INFINITY;
      wt[tid] = s == -INFINITY || (p.haze > 0.f && s < m - p.haze) ? 0.f : expf(s - m);
    }
    __syncthreads();
    for (int i = 0; i < 64; ++i)
      if (wt[i] != 0.f) {
        sum += wt[i];
        acc = fmaf(wt[i] * bf16_bits_to_f32(p.vs[ph * 64 + i]), (float)p.v[(ph * D + tid) * 64 + i], acc);
      }
  }
  const float o = sum == 0.f ? 0.f : acc / sum;
  const size_t at = ((size_t)b * p.Hq + hq) * D + tid;
  if (p.out_bf16) static_cast<uint16_t *>(p.out)[at] = f32_to_bf16_rn_bits(o);
  else static_cast<float *>(p.out)[at] = o;
}

size_t pfx_workspace_bytes(const Q8Shape &s) {
  return (size_t)s.B * s.Hq * (((s.prefix + 63) & ~63) + (size_t)s.ctx) * 4 + 256;
}

cudaError_t launch_prefix_attention(const Q8Args &a, cudaStream_t st, Launcher &L) {
  PfxParams p{};
  p.q = a.q; p.q_bs = a.q_bs; p.q_hs = a.q_hs;
  p.k = a.pool.k; p.v = a.pool.v; p.ks = a.pool.ks; p.vs = a.pool.vs;
  p.table = a.pool.table; p.ptable = a.ptable; p.lens = a.lens;
  p.out = a.out; p.out_bf16 = a.out_bf16;
  p.logit = static_cast<float *>(a.workspace);
  p.B = a.s.B; p.Hq = a.s.Hq; p.H = a.s.Hkv; p.G = a.s.Hq / a.s.Hkv; p.W = a.pool.W;
  p.n_pages = a.pool.n_pages; p.ctx = a.s.ctx; p.prefix = a.s.prefix; p.ppages = (a.s.prefix + 63) / 64;
  p.scale = a.tau / sqrtf((float)a.s.D);
  p.haze = a.haze;
  const dim3 gl((unsigned)(p.ppages + (p.ctx + 63) / 64), (unsigned)p.H, (unsigned)p.B);
  const dim3 go((unsigned)p.Hq, (unsigned)p.B);
  cudaError_t e;
#define PFX_CASE(D_)                                                                              \
  if (a.s.D == D_) {                                                                             \
    if ((e = L.launch("pfx_logits", pfx_logits_kernel<D_>, gl, dim3(128), 0, st, false, p)) !=     \
        cudaSuccess)                                                                             \
      return e;                                                                                  \
    return L.launch("pfx_out", pfx_out_kernel<D_>, go, dim3(D_), 0, st, false, p);                 \
  }
  PFX_CASE(64) PFX_CASE(128) PFX_CASE(256)
#undef PFX_CASE
  return cudaErrorInvalidValue;
}

}  // namespace dvssq
