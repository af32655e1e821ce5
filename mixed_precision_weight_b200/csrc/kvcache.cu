// The 8-bit KV cache: quantising K and V rows as they are written into its
// pages (dvssq_kv_append) and reading rows back as BF16 (dvssq_kv_read).
//
// A row x of one token and KV head (d values) is held like a row of the
// salient INT8 tier (Spark card, Tier A: clip(round(W / s)) with one scale per
// row):
//   s = RN_bf16(max|x| / 127),  c_i = clip(rint(x_i / s), -127, 127)  (c = 0 where s = 0)
// and stands for c s.  x_i / s is the correctly rounded quotient, so that the
// codes are those of exact arithmetic: x and s have 8 significant bits each,
// and a quotient that is not a tie lies at least 1/510 from one.
//
// Pages of 64 tokens; within a page the K codes of a head are [64][d] and the
// V codes are transposed, [d][64]: the attention contracts K over d and V over
// the tokens, and either way the contracted axis is contiguous.
//
// One CTA per (run of one sequence's rows inside one page, KV head, K or V):
// a run's rows are consecutive positions, so the transposed V bytes go out as
// words.  Work is HBM-bound: 2 d bytes of BF16 and d + 2 bytes of codes and
// scale per row.
#include "common.cuh"
#include "kernels.h"

namespace dvssq {

constexpr int kKvThreads = 256;
constexpr int kKvWarps = kKvThreads / 32;

// Which rows of the flat token axis belong to which sequence and position.
struct KvIndex {
  const int32_t *cu;      // [B + 1] first row of each sequence; nullptr: one row per sequence
  const int32_t *start;   // [B] position of each sequence's first row
  const int32_t *table;   // [B][W]
  int B, W, n_pages;
  long long T;            // rows
};

// One run: rows [row0, row0 + n) at slots [slot0, slot0 + n) of page `page`.
struct KvRun {
  long long row0;
  int slot0, n, page;
};

// Item -> run.  Sequence b owns the items [cu[b] / 64 + 2 b, cu[b+1] / 64 +
// 2 (b+1)): n rows touch at most n / 64 + 2 pages, so that range covers them
// without a prefix sum, and a warp-wide search over cu finds b.  Rows outside
// [0, T), positions outside the table and pages outside the pool are skipped
// and flagged.  Whole warps call this; false: nothing to do.
__device__ __forceinline__ bool kv_find_run(const KvIndex &ix, int item, KvRun &r) {
  const int lane = threadIdx.x & 31;
  int b = item, j = 0;
  long long row0 = item, n = 1;
  if (ix.cu != nullptr) {
    int lo = 0, hi = ix.B;
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32, idx = lo + step * (lane + 1);
      const bool le = idx < hi && (ix.cu[idx] >> 6) + 2 * idx <= item;
      lo += step * __popc(__ballot_sync(0xffffffffu, le));
      hi = min(hi, lo + step);
    }
    b = lo;
    row0 = ix.cu[b];
    n = (long long)ix.cu[b + 1] - row0;
    j = item - ((int)(row0 >> 6) + 2 * b);
    if (j < 0 || n <= 0) return false;
  }
  bool bad = false;
  if (row0 < 0 || row0 + n > ix.T) {
    bad = true;
    if (row0 < 0) return set_error(kErrBadIndex), false;
    n = ix.T - row0;
    if (n <= 0) return set_error(kErrBadIndex), false;
  }
  const long long pos = ix.start[b];
  if (pos < 0) return set_error(kErrBadIndex), false;
  const long long p = (pos >> 6) + j;
  const long long a = max(pos, 64 * p), z = min(pos + n, 64 * (p + 1));
  if (a >= z) {
    if (bad) set_error(kErrBadIndex);
    return false;
  }
  if (p >= ix.W) return set_error(kErrBadIndex), false;
  r.page = ix.table[(size_t)b * ix.W + p];
  if (r.page < 0 || r.page >= ix.n_pages) return set_error(kErrBadIndex), false;
  if (bad) set_error(kErrBadIndex);
  r.row0 = row0 + (a - pos);
  r.slot0 = (int)(a - 64 * p);
  r.n = (int)(z - a);
  return true;
}

struct KvAppendParams {
  KvIndex ix;
  const uint16_t *src[2];          // K, V rows
  long long ts[2], hs[2];          // token and head strides in elements
  int8_t *k, *v;
  uint16_t *ks, *vs;
  int H;
};

// VPL consecutive BF16 values of one lane as packed pairs
template <int VPL>
struct KvRaw {
  uint32_t w[VPL / 2];
};
template <int VPL>
__device__ __forceinline__ KvRaw<VPL> kv_load(const uint16_t *src) {
  KvRaw<VPL> r;
  if constexpr (VPL == 8) {
    const uint4 u = __ldg(reinterpret_cast<const uint4 *>(src));
    r.w[0] = u.x; r.w[1] = u.y; r.w[2] = u.z; r.w[3] = u.w;
  } else if constexpr (VPL == 4) {
    const uint2 u = __ldg(reinterpret_cast<const uint2 *>(src));
    r.w[0] = u.x; r.w[1] = u.y;
  } else {
    r.w[0] = __ldg(reinterpret_cast<const uint32_t *>(src));
  }
  return r;
}

// x / s rounded to nearest: the reciprocal's quotient with one residual step,
// exact for these 8-bit significands; the plain division where the residual
// could fall below the normal range.
__device__ __forceinline__ int kv_code(float x, float s, float rs, bool plain) {
  float y;
  if (plain) {
    y = __fdiv_rn(x, s);
  } else {
    y = x * rs;
    y = fmaf(fmaf(-y, s, x), rs, y);
  }
  return max(-127, min(127, __float2int_rn(y)));
}

// One row held by a warp -> its scale (BF16 bits) and this lane's VPL codes as bytes.
template <int VPL>
__device__ __forceinline__ uint32_t kv_quantise(const KvRaw<VPL> &raw, uint32_t *codes) {
  // the largest magnitude by its bits: a NaN or an infinity stays the largest
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < VPL / 2; ++i)
    m = max(m, max(raw.w[i] & 0x7FFFu, (raw.w[i] >> 16) & 0x7FFFu));
  m = __reduce_max_sync(0xffffffffu, m);
  uint32_t sb;
  if (m >= 0x7F80u) sb = 0x7FC0u;      // the row reads back as NaN
  else sb = f32_to_bf16_rn_bits(__fdiv_rn(bf16_bits_to_f32(m), 127.0f));
  const float s = bf16_bits_to_f32(sb);
#pragma unroll
  for (int i = 0; i < (VPL + 3) / 4; ++i) codes[i] = 0;
  if (m < 0x7F80u && sb != 0) {
    const bool plain = s < 1e-27f;
    const float rs = plain ? 0.0f : __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const uint32_t h = i & 1 ? raw.w[i / 2] >> 16 : raw.w[i / 2] & 0xFFFFu;
      const int c = kv_code(bf16_bits_to_f32(h), s, rs, plain);
      codes[i / 4] |= ((uint32_t)c & 0xFFu) << (8 * (i & 3));
    }
  }
  return sb;
}

template <int VPL>
__device__ __forceinline__ void kv_store_codes(int8_t *dst, const uint32_t *c) {
  if constexpr (VPL == 8) *reinterpret_cast<uint2 *>(dst) = make_uint2(c[0], c[1]);
  else if constexpr (VPL == 4) *reinterpret_cast<uint32_t *>(dst) = c[0];
  else *reinterpret_cast<uint16_t *>(dst) = (uint16_t)c[0];
}

template <int D>
__global__ void __launch_bounds__(kKvThreads) kv_append_kernel(const KvAppendParams p) {
  constexpr int VPL = D / 32;
  constexpr int U = 4;                        // rows in flight per warp
  __shared__ __align__(16) int8_t tile[64][D + 4];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.y, which = blockIdx.z;
  KvRun r;
  if (!kv_find_run(p.ix, blockIdx.x, r)) return;
  const uint16_t *src = p.src[which] + r.row0 * p.ts[which] + h * p.hs[which] + lane * VPL;
  const size_t ph = (size_t)r.page * p.H + h;
  uint16_t *scales = (which ? p.vs : p.ks) + ph * 64 + r.slot0;
  int8_t *kdst = p.k + (ph * 64 + r.slot0) * D + lane * VPL;
  for (int i0 = warp; i0 < r.n; i0 += U * kKvWarps) {
    KvRaw<VPL> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u * kKvWarps < r.n)
        raw[u] = kv_load<VPL>(src + (long long)(i0 + u * kKvWarps) * p.ts[which]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kKvWarps;
      if (i >= r.n) break;
      uint32_t codes[(VPL + 3) / 4];
      const uint32_t sb = kv_quantise<VPL>(raw[u], codes);
      if (lane == 0) scales[i] = (uint16_t)sb;
      if (which == 0) kv_store_codes<VPL>(kdst + (size_t)i * D, codes);
      else if constexpr (VPL == 8) {
        uint32_t *t = reinterpret_cast<uint32_t *>(&tile[r.slot0 + i][lane * VPL]);
        t[0] = codes[0];
        t[1] = codes[1];
      } else {
        kv_store_codes<VPL>(&tile[r.slot0 + i][lane * VPL], codes);
      }
    }
  }
  if (which == 0) return;
  __syncthreads();
  // V transposed: word w of dimension dd holds slots 4 w .. 4 w + 3; only the
  // run's own bytes are written
  const int s0 = r.slot0, s1 = r.slot0 + r.n;
  const int w0 = s0 >> 2, nw = ((s1 + 3) >> 2) - w0;
  int8_t *vdst = p.v + ph * 64 * D;
  for (int i = tid; i < nw * D; i += kKvThreads) {
    const int dd = i / nw, w = w0 + i - dd * nw, t0 = 4 * w;
    int8_t *dst = vdst + dd * 64 + t0;
    if (t0 >= s0 && t0 + 4 <= s1) {
      const uint32_t a = (uint8_t)tile[t0][dd], b = (uint8_t)tile[t0 + 1][dd],
                     c = (uint8_t)tile[t0 + 2][dd], d = (uint8_t)tile[t0 + 3][dd];
      *reinterpret_cast<uint32_t *>(dst) = a | (b << 8) | (c << 16) | (d << 24);
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (t0 + u >= s0 && t0 + u < s1) dst[u] = tile[t0 + u][dd];
    }
  }
}

struct KvReadParams {
  KvIndex ix;
  const int8_t *k, *v;
  const uint16_t *ks, *vs;
  uint16_t *out[2];                // K, V rows [T][H][d]
  int H;
};

__device__ __forceinline__ uint32_t kv_value2(int c0, int c1, float s) {
  return (uint32_t)f32_to_bf16_rn_bits((float)c0 * s) |
         ((uint32_t)f32_to_bf16_rn_bits((float)c1 * s) << 16);
}

template <int D>
__global__ void __launch_bounds__(kKvThreads) kv_read_kernel(const KvReadParams p) {
  constexpr int VPL = D / 32;
  __shared__ __align__(16) uint32_t tile[D][17];     // V words: slots 4 w .. 4 w + 3 of dimension dd
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.y, which = blockIdx.z;
  KvRun r;
  if (!kv_find_run(p.ix, blockIdx.x, r)) return;
  const size_t ph = (size_t)r.page * p.H + h;
  uint16_t *dst = p.out[which] + ((size_t)r.row0 * p.H + h) * D;
  const size_t ts = (size_t)p.H * D;
  if (which == 0) {
    const int8_t *src = p.k + (ph * 64 + r.slot0) * D + lane * VPL;
#pragma unroll 4
    for (int i = warp; i < r.n; i += kKvWarps) {
      const float s = bf16_bits_to_f32(p.ks[ph * 64 + r.slot0 + i]);
      uint16_t *o = dst + i * ts + lane * VPL;
      if constexpr (VPL == 8) {
        const uint2 c = __ldg(reinterpret_cast<const uint2 *>(src + (size_t)i * D));
        const char4 a = *reinterpret_cast<const char4 *>(&c.x), b = *reinterpret_cast<const char4 *>(&c.y);
        *reinterpret_cast<uint4 *>(o) = make_uint4(kv_value2(a.x, a.y, s), kv_value2(a.z, a.w, s),
                                                   kv_value2(b.x, b.y, s), kv_value2(b.z, b.w, s));
      } else if constexpr (VPL == 4) {
        const char4 a = __ldg(reinterpret_cast<const char4 *>(src + (size_t)i * D));
        *reinterpret_cast<uint2 *>(o) = make_uint2(kv_value2(a.x, a.y, s), kv_value2(a.z, a.w, s));
      } else {
        const char2 a = __ldg(reinterpret_cast<const char2 *>(src + (size_t)i * D));
        *reinterpret_cast<uint32_t *>(o) = kv_value2(a.x, a.y, s);
      }
    }
    return;
  }
  const int s0 = r.slot0, s1 = r.slot0 + r.n;
  const int w0 = s0 >> 2, nw = ((s1 + 3) >> 2) - w0;
  const uint32_t *src = reinterpret_cast<const uint32_t *>(p.v + ph * 64 * D);
  for (int i = tid; i < nw * D; i += kKvThreads) {
    const int dd = i / nw, w = i - dd * nw;
    tile[dd][w] = __ldg(src + dd * 16 + w0 + w);
  }
  __syncthreads();
  // a warp takes four slots at a time, a lane two dimensions of each 64
  for (int w = warp; w < nw; w += kKvWarps) {
    const int t0 = 4 * (w0 + w);
    float s[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      s[u] = t0 + u >= s0 && t0 + u < s1 ? bf16_bits_to_f32(p.vs[ph * 64 + t0 + u]) : 0.0f;
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
      const int dd = 64 * j + 2 * lane;
      const uint32_t a = tile[dd][w], b = tile[dd + 1][w];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (t0 + u >= s0 && t0 + u < s1)
          *reinterpret_cast<uint32_t *>(dst + (size_t)(t0 + u - s0) * ts + dd) =
              kv_value2((int)(int8_t)(a >> (8 * u)), (int)(int8_t)(b >> (8 * u)), s[u]);
    }
  }
}

namespace {
KvIndex kv_index(const KvPool &c, const int32_t *start, const int32_t *cu, long long T) {
  KvIndex ix;
  ix.cu = cu; ix.start = start; ix.table = c.table;
  ix.B = c.B; ix.W = c.W; ix.n_pages = c.n_pages; ix.T = T;
  return ix;
}
unsigned kv_items(const KvIndex &ix) {
  return (unsigned)(ix.cu == nullptr ? ix.B : ix.T / 64 + 2 * (long long)ix.B);
}
}  // namespace

cudaError_t launch_kv_append(const KvPool &c, const uint16_t *k, const uint16_t *v,
                             const long long *strides, long long T, const int32_t *start,
                             const int32_t *cu, cudaStream_t st, Launcher &L) {
  KvAppendParams p;
  p.ix = kv_index(c, start, cu, T);
  p.src[0] = k; p.src[1] = v;
  p.ts[0] = strides[0]; p.hs[0] = strides[1]; p.ts[1] = strides[2]; p.hs[1] = strides[3];
  p.k = c.k; p.v = c.v; p.ks = c.ks; p.vs = c.vs; p.H = c.H;
  const dim3 grid(kv_items(p.ix), (unsigned)c.H, 2), block(kKvThreads);
  if (c.D == 256) return L.launch("kv_append", kv_append_kernel<256>, grid, block, 0, st, false, p);
  if (c.D == 128) return L.launch("kv_append", kv_append_kernel<128>, grid, block, 0, st, false, p);
  return L.launch("kv_append", kv_append_kernel<64>, grid, block, 0, st, false, p);
}

cudaError_t launch_kv_read(const KvPool &c, uint16_t *k, uint16_t *v, long long T,
                           const int32_t *start, const int32_t *cu, cudaStream_t st, Launcher &L) {
  KvReadParams p;
  p.ix = kv_index(c, start, cu, T);
  p.k = c.k; p.v = c.v; p.ks = c.ks; p.vs = c.vs; p.H = c.H;
  p.out[0] = k; p.out[1] = v;
  const dim3 grid(kv_items(p.ix), (unsigned)c.H, 2), block(kKvThreads);
  if (c.D == 256) return L.launch("kv_read", kv_read_kernel<256>, grid, block, 0, st, false, p);
  if (c.D == 128) return L.launch("kv_read", kv_read_kernel<128>, grid, block, 0, st, false, p);
  return L.launch("kv_read", kv_read_kernel<64>, grid, block, 0, st, false, p);
}

}  // namespace dvssq
