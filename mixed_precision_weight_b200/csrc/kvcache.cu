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
// words.  Bound by HBM where it is large: 2 d bytes of BF16 and d + 2 bytes of
// codes and scale per row.  Measured in a graph: 4096 rows of 4 heads of 256, K and V,
// written and read back in 17.1 us (50 MB, from and to the L2); 28 K such rows read back in
// 33.0 us (174 MB, floor 26.6 at copy bandwidth); single tokens at launch latency
// (3 us each).
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
// without a prefix sum, and a warp-wide search over cu finds b (its last round reads
// the start positions along, so that a call on up to 31 sequences waits for two
// loads before its rows: these and the page's id).  Rows at and past T, sequences that
// begin before row 0, positions outside the table and pages outside the pool are
// skipped and flagged.  Whole warps call this; false: nothing to do.
__device__ __forceinline__ bool kv_find_run(const KvIndex &ix, int item, KvRun &r) {
  const int lane = threadIdx.x & 31;
  int b = item, j = 0;
  long long row0 = item, n = 1, pos;
  if (ix.cu != nullptr) {
    int lo = 0, hi = ix.B;
    while (hi - lo > 31) {
      const int step = (hi - lo + 31) / 32, idx = lo + step * (lane + 1);
      const bool le = idx < hi && (ix.cu[idx] >> 6) + 2 * idx <= item;
      lo += step * __popc(__ballot_sync(0xffffffffu, le));
      hi = min(hi, lo + step);
    }
    const int idx = lo + lane;
    const int first = idx <= ix.B ? ix.cu[idx] : 0, at = idx < ix.B ? ix.start[idx] : 0;
    const uint32_t le = __ballot_sync(0xffffffffu, idx < hi && (first >> 6) + 2 * idx <= item);
    const int k = __ffs(~le) - 1;              // candidates before the first that lies behind
    if (k <= 0) return false;
    b = lo + k - 1;
    row0 = __shfl_sync(0xffffffffu, first, k - 1);
    n = (long long)__shfl_sync(0xffffffffu, first, k) - row0;
    pos = __shfl_sync(0xffffffffu, at, k - 1);
    j = item - ((int)(row0 >> 6) + 2 * b);
    if (j < 0 || n <= 0) return false;
  } else {
    pos = ix.start[b];
  }
  bool bad = false;
  if (row0 < 0 || row0 + n > ix.T) {
    bad = true;
    if (row0 < 0) return set_index_error(), false;
    n = ix.T - row0;
    if (n <= 0) return set_index_error(), false;
  }
  const long long p = (pos >> 6) + j;
  const long long a = max(pos, 64 * p), z = min(pos + n, 64 * (p + 1));
  if (a >= z) {
    if (bad) set_index_error();
    return false;
  }
  if (p < 0 || p >= ix.W) return set_index_error(), false;
  r.page = ix.table[(size_t)b * ix.W + p];
  if (r.page < 0 || r.page >= ix.n_pages) return set_index_error(), false;
  if (bad) set_index_error();
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

// One row held by a warp -> its scale (BF16 bits) and this lane's VPL codes as bytes.
// x / s is the reciprocal's quotient with one residual step (Markstein's correction:
// q + r (x - q s) by two FMAs), exact for these 8-bit significands, and no larger than
// 127 (1 + 2^-8), so that rounding needs no clamp; adding 1.5 2^23 rounds it to the
// nearest integer, ties to even, and leaves the code in the low byte.  Two values at a
// time (packed FP32).  Where the residual could fall below the normal range (s < 1e-27):
// the plain division, and a clamp, because the scale itself may be a subnormal.
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
  if (m >= 0x7F80u || sb == 0) return sb;
  float2 y[VPL / 2];
  if (s >= 1e-27f) {
    const float rs = __frcp_rn(s);
    const float2 r2 = make_float2(rs, rs), n2 = make_float2(-s, -s), magic = make_float2(12582912.0f, 12582912.0f);
#pragma unroll
    for (int i = 0; i < VPL / 2; ++i) {
      const float2 x = make_float2(__uint_as_float(raw.w[i] << 16), __uint_as_float(raw.w[i] & 0xFFFF0000u));
      const float2 q = mat_mul2(x, r2);
      y[i] = mat_add2(mat_fma2(mat_fma2(q, n2, x), r2, q), magic);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL / 2; ++i) {
      const float a = __fdiv_rn(__uint_as_float(raw.w[i] << 16), s);
      const float b = __fdiv_rn(__uint_as_float(raw.w[i] & 0xFFFF0000u), s);
      y[i] = make_float2(fmaxf(-127.f, fminf(127.f, a)) + 12582912.0f, fmaxf(-127.f, fminf(127.f, b)) + 12582912.0f);
    }
  }
#pragma unroll
  for (int i = 0; i < VPL / 2; ++i) {
    const uint32_t two = __byte_perm(__float_as_uint(y[i].x), __float_as_uint(y[i].y), 0x0040);
    codes[i / 2] |= i & 1 ? two << 16 : two & 0xFFFFu;
  }
  return sb;
}

template <int VPL>
__device__ __forceinline__ void kv_store_codes(int8_t *dst, const uint32_t *c) {
  if constexpr (VPL == 8) *reinterpret_cast<uint2 *>(dst) = make_uint2(c[0], c[1]);
  else if constexpr (VPL == 4) *reinterpret_cast<uint32_t *>(dst) = c[0];
  else *reinterpret_cast<uint16_t *>(dst) = (uint16_t)c[0];
}

// 4 x 4 bytes transposed: word i of the result holds byte i of each input word.
__device__ __forceinline__ void kv_transpose4(const uint32_t a[4], uint32_t o[4]) {
  const uint32_t x = __byte_perm(a[0], a[1], 0x5140), y = __byte_perm(a[2], a[3], 0x5140);   // bytes 0, 1
  const uint32_t z = __byte_perm(a[0], a[1], 0x7362), w = __byte_perm(a[2], a[3], 0x7362);   // bytes 2, 3
  o[0] = __byte_perm(x, y, 0x5410);
  o[1] = __byte_perm(x, y, 0x7632);
  o[2] = __byte_perm(z, w, 0x5410);
  o[3] = __byte_perm(z, w, 0x7632);
}

// A warp takes aligned groups of four slots, both its groups' rows in flight at
// once.  A lane then holds the same dimensions of four neighbouring tokens: for V,
// four-byte words of the transposed page after a byte transposition in registers.
// They go through shared memory (word w of a row at w ^ (row / VPL mod 16), two-way
// conflicts at most) so that whole rows of 64 bytes are written.
template <int D>
__global__ void __launch_bounds__(kKvThreads) kv_append_kernel(const KvAppendParams p) {
  constexpr int VPL = D / 32, NC = (VPL + 3) / 4;
  constexpr int NG = 16 / kKvWarps;           // slot groups per warp
  __shared__ uint32_t tile[D][16];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.y, which = blockIdx.z;
  KvRun r;
  if (!kv_find_run(p.ix, blockIdx.x, r)) return;
  const int s0 = r.slot0, s1 = r.slot0 + r.n;
  const long long ts = which ? p.ts[1] : p.ts[0], hs = which ? p.hs[1] : p.hs[0];
  const uint16_t *src = (which ? p.src[1] : p.src[0]) + (r.row0 - s0) * ts + h * hs + lane * VPL;
  const size_t ph = (size_t)r.page * p.H + h;
  uint16_t *scales = (which ? p.vs : p.ks) + ph * 64;
  int8_t *kdst = p.k + ph * 64 * D + lane * VPL;
  KvRaw<VPL> raw[NG][4];
#pragma unroll
  for (int q = 0; q < NG; ++q)
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int slot = 4 * (warp + kKvWarps * q) + u;
      if (slot >= s0 && slot < s1) raw[q][u] = kv_load<VPL>(src + slot * ts);
    }
#pragma unroll
  for (int q = 0; q < NG; ++q) {
    const int w = warp + kKvWarps * q;        // slots 4 w .. 4 w + 3
    if (4 * w >= s1 || 4 * w + 4 <= s0) continue;
    uint32_t codes[4][NC];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int slot = 4 * w + u;
      if (slot >= s0 && slot < s1) {
        const uint32_t sb = kv_quantise<VPL>(raw[q][u], codes[u]);
        if (lane == 0) scales[slot] = (uint16_t)sb;
        if (which == 0) kv_store_codes<VPL>(kdst + (size_t)slot * D, codes[u]);
      } else {
#pragma unroll
        for (int i = 0; i < NC; ++i) codes[u][i] = 0;
      }
    }
    if (which == 1) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const uint32_t a[4] = {codes[0][i], codes[1][i], codes[2][i], codes[3][i]};
        uint32_t o[4];
        kv_transpose4(a, o);
#pragma unroll
        for (int u = 0; u < (VPL < 4 ? VPL : 4); ++u) tile[lane * VPL + 4 * i + u][w ^ (lane & 15)] = o[u];
      }
    }
  }
  if (which == 0) return;
  __syncthreads();
  uint32_t *vdst = reinterpret_cast<uint32_t *>(p.v + ph * 64 * D);
#pragma unroll 4
  for (int i = tid; i < 16 * D; i += kKvThreads) {
    const int dd = i >> 4, w = i & 15, t0 = 4 * w;
    if (t0 >= s1 || t0 + 4 <= s0) continue;
    const uint32_t x = tile[dd][w ^ ((dd / VPL) & 15)];
    if (t0 >= s0 && t0 + 4 <= s1) {
      vdst[i] = x;
    } else {                                  // a run's ragged end: its own bytes only
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (t0 + u >= s0 && t0 + u < s1) reinterpret_cast<uint8_t *>(vdst + i)[u] = (uint8_t)(x >> (8 * u));
    }
  }
}

// Constants of the code conversion, passed as a kernel parameter: the compiler keeps
// them in registers, and each mask-and-set below is one instruction (as literals
// they took two, and the integer pipe bounds the conversion).
struct KvBits {
  uint32_t low7, sign, one2, nzero2;
};
constexpr KvBits kKvBits = {0x007F007Fu, 0x00800080u, 0x3F803F80u, 0x80008000u};

struct KvReadParams {
  KvIndex ix;
  const int8_t *k, *v;
  const uint16_t *ks, *vs;
  uint16_t *out[2];                // K, V rows [T][H][d]
  int H;
  KvBits bits;
};

// a b + c on BF16 pairs, rounded once
__device__ __forceinline__ uint32_t bf16x2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// Bytes 0, 2 (even) or 1, 3 (odd, x already shifted right by 8) of x as a BF16
// pair: 128 + (low 7 bits), minus 128 or, with the sign bit, 256; all exact.
__device__ __forceinline__ uint32_t kv_bf16_pair(uint32_t x, const KvBits &k) {
  return bf16x2_fma((x & k.low7) | 0x43004300u, k.one2, (x & k.sign) | 0xC300C300u);
}

// D threads, four 16-byte pieces of the page each.
//   K: a piece is 16 dimensions of one row: 32 contiguous bytes out, which two lanes write
//      whole, one piece each per store (28 K rows: 33 us; as two half sectors 35; the same
//      trade for V, 16-byte stores for its 8-byte ones, was slower: 36).
//   V: a warp takes 32 dimensions; a lane 4 of them (one piece each) x 16 tokens, so that
//      after a transposition of the BF16 results in registers every token's 4
//      dimensions are 8 contiguous bytes and 8 lanes fill 64.  No shared memory.
template <int D>
__global__ void __launch_bounds__(D) kv_read_kernel(const KvReadParams p) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.y, which = blockIdx.z;
  KvRun r;
  if (!kv_find_run(p.ix, blockIdx.x, r)) return;
  const size_t ph = (size_t)r.page * p.H + h;
  const int s0 = r.slot0, s1 = r.slot0 + r.n;
  // a code pair times a scale pair: one rounding of the exact product
  auto times = [&](uint32_t codes, uint32_t s) { return bf16x2_fma(kv_bf16_pair(codes, p.bits), s, p.bits.nzero2); };
  const long long ts = (long long)p.H * D;
  uint16_t *dst = (which ? p.out[1] : p.out[0]) + (r.row0 - s0) * ts + (long long)h * D;   // slot t at dst + t ts
  if (which == 0) {
    constexpr int CPR = D / 16;
    const int8_t *src = p.k + ph * 64 * D;
    uint4 c[4];
    uint32_t s[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int row = (tid + D * x) / CPR;
      c[x] = make_uint4(0, 0, 0, 0);
      s[x] = 0;
      if (row >= s0 && row < s1) {
        c[x] = __ldg(reinterpret_cast<const uint4 *>(src) + tid + D * x);
        s[x] = p.ks[ph * 64 + row] * 0x10001u;
      }
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int row = (tid + D * x) / CPR, ch = (tid + D * x) % CPR;
      const uint32_t w[4] = {c[x].x, c[x].y, c[x].z, c[x].w};
      uint32_t o[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t e = times(w[i], s[x]), f = times(w[i] >> 8, s[x]);
        o[2 * i] = __byte_perm(e, f, 0x5410);
        o[2 * i + 1] = __byte_perm(e, f, 0x7632);
      }
      // a pair of lanes holds two pieces of 32 bytes; each store writes one of them whole
      const bool odd = lane & 1;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? o[i] : o[4 + i], 1);
        if (odd) o[i] = got; else o[4 + i] = got;
      }
      if (row < s0 || row >= s1) continue;
      uint4 *out = reinterpret_cast<uint4 *>(dst + row * ts + 16 * (ch & ~1)) + odd;
      out[0] = make_uint4(o[0], o[1], o[2], o[3]);
      out[2] = make_uint4(o[4], o[5], o[6], o[7]);
    }
    return;
  }
  const int d0 = 32 * warp + 4 * (lane >> 2), t0 = 16 * (lane & 3);
  if (t0 >= s1 || t0 + 16 <= s0) return;
  uint4 c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = __ldg(reinterpret_cast<const uint4 *>(p.v + (ph * D + d0 + i) * 64 + t0));
  const uint4 sa = *reinterpret_cast<const uint4 *>(p.vs + ph * 64 + t0);
  const uint4 sb = *reinterpret_cast<const uint4 *>(p.vs + ph * 64 + t0 + 8);
  const uint32_t sc[8] = {sa.x, sa.y, sa.z, sa.w, sb.x, sb.y, sb.z, sb.w};
#pragma unroll
  for (int g = 0; g < 4; ++g) {              // tokens t0 + 4 g .. + 3
    const uint32_t s02 = __byte_perm(sc[2 * g], sc[2 * g + 1], 0x5410);
    const uint32_t s13 = __byte_perm(sc[2 * g], sc[2 * g + 1], 0x7632);
    uint32_t e[4], o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x = g == 0 ? c[i].x : g == 1 ? c[i].y : g == 2 ? c[i].z : c[i].w;
      e[i] = times(x, s02);       // tokens 0 and 2 of dimension d0 + i
      o[i] = times(x >> 8, s13);  // tokens 1 and 3
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int t = t0 + 4 * g + u;
      if (t < s0 || t >= s1) continue;
      const uint32_t sel = u < 2 ? 0x5410 : 0x7632;
      *reinterpret_cast<uint2 *>(dst + t * ts + d0) =
          u & 1 ? make_uint2(__byte_perm(o[0], o[1], sel), __byte_perm(o[2], o[3], sel))
                : make_uint2(__byte_perm(e[0], e[1], sel), __byte_perm(e[2], e[3], sel));
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
  p.bits = kKvBits;
  const dim3 grid(kv_items(p.ix), (unsigned)c.H, 2), block((unsigned)c.D);
  if (c.D == 256) return L.launch("kv_read", kv_read_kernel<256>, grid, block, 0, st, false, p);
  if (c.D == 128) return L.launch("kv_read", kv_read_kernel<128>, grid, block, 0, st, false, p);
  return L.launch("kv_read", kv_read_kernel<64>, grid, block, 0, st, false, p);
}

}  // namespace dvssq
