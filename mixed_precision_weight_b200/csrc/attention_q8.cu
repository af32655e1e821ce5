// KV-BSS decode attention over the 8-bit paged cache (Spark card, "2. KV-BSS:
// Key-Value Binding Softmax Sharpening"), for one query token per sequence
// with grouped-query heads (G query heads share a KV head):
//   s_l = (q . k_l) tau / sqrt(d),  m = max_l s_l,
//   p_l = exp(s_l - m) if s_l >= m - haze else 0,  out = sum_l p_l v_l / sum_l p_l
// with k_l = ks_l kc_l and v_l = vs_l vc_l.  The haze threshold needs the final
// maximum before any weight is known, so the context is walked twice, K then V,
// each byte read once (HBM-bound: 2 (d + 2) bytes per key and KV head):
//   q8_logits  logits of the keys, FP32, and each item's maximum per head
//   q8_pv      weights from the final maximum, and each item's sum of p v; the V
//              codes of a page whose 64 keys all fell below the threshold are
//              never read
//   q8_merge   the items' partials added in order, divided, stored
// An item is a run of pages of one sequence and one KV head.  The lengths live
// on the device, so every CTA derives the same plan from them: pages per item
// such that the items fill whole rounds of the grid.
// Contexts up to 64 pages (q8_cluster) take one launch instead (q8_short: a CTA, or a cluster of
// them, per sequence and KV head).
//
// Measured, 4 sequences of up to 32768 keys, 16/4 heads of 256 (190 MB of keys and
// values, 29 us at copy bandwidth; the L2 keeps part of them from call to call): 44 us in a
// graph, of which logits 18 (5.3 TB/s), P V 21 (4.5 TB/s), merge 3.  Neither pass
// saturates anything: four CTAs of 128 threads per SM (120 registers hold the pages in
// flight) issue on 19 and 37 % of the cycles and wait for their rows, after a prologue (plan,
// page ids, query or maxima) of about 3 us.
#include "common.cuh"
#include "kernels.h"

namespace dvssq {

constexpr int kQ8Threads = 128;
constexpr int kQ8MaxPages = 16;        // pages per item at most
constexpr int kQ8Sms = 148;            // B200; any value gives the same results

// n-tiles of 4 heads x 2 limbs that cover G heads
__host__ __device__ constexpr int q8_tiles(int G) { return G <= 4 ? 1 : G <= 8 ? 2 : 4; }
// resident CTAs per SM the kernels are compiled for (registers: query fragments
// and accumulators grow with the tiles)
__host__ __device__ constexpr int q8_occ(int NT) { return NT == 1 ? 4 : NT == 2 ? 3 : 2; }

struct Q8Params {
  const uint16_t *q;
  long long q_bs, q_hs;
  const int8_t *k, *v;
  const uint16_t *ks, *vs;
  const int32_t *table, *lens;
  void *out;
  int out_bf16;
  float *logit;                  // [B][H][ctxp][4 NT]
  float *smax;                   // [B][H][pages][4][4 NT]: maxima of each page's 16-key strips
  float *cmax, *psum;            // [items][4 NT]
  float *pacc;                   // [items][G][D]
  int *off;                      // [B + 1] first item of each sequence (per KV head)
  // a shared prefix (splits > 0), rows = B G per KV head: every split's row maxima
  // [splits][H][rows] and largest value scale [splits][H], their maxima with the own
  // keys' [B][Hq] and [H], which this part's kernels write, and the splits' partial sums
  const float *pmax, *psv;
  float *mfin, *svfin;
  const float *po, *pl;
  int splits, rows;
  int single;                    // one item per sequence and KV head, whatever its length
  int cluster;                   // CTAs per sequence and KV head of the one-launch form
  const int32_t *ptable;         // and a prefix that it takes as the sequences' first keys:
  int prefix, pp;                // its pages, keys and their number
  int B, Hq, H, G, W, n_pages, ctx, ctxp, target;
  float scale2;                  // tau / sqrt(d) log2 e: logits are held in units of log2 e
  float haze2;                   // -haze log2 e; -inf: no truncation
  KvBits bits;
};

__device__ __forceinline__ int q8_len(const Q8Params &p, int b) {
  const int n = p.lens[b];
  if (n < 0 || n > p.ctx) set_index_error();
  return max(0, min(n, p.ctx));
}

// The plan, the same in every CTA: off[b] = items of the sequences before b (per KV
// head) in shared memory.  A sequence gets ceil(pages / c) items of even shares.  N
// page-heads over r rounds of `target` CTAs, r the fewest for at most kQ8MaxPages pages
// per item; there are up to N / c + B H items, and c is chosen for those to fit the
// rounds (a few items over a round would double the time: 20 us instead of 13 for the
// logits of 32 sequences of up to 8000 keys).
__device__ __forceinline__ void q8_plan(const Q8Params &p, int *off) {
  __shared__ int part[kQ8Threads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = (p.B + kQ8Threads - 1) / kQ8Threads;
  const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  uint32_t sum = 0;
  for (int b = b0; b < b1; ++b) {
    const int n = p.pp + ((q8_len(p, b) + 63) >> 6);
    off[b] = n;                              // this thread's entries: pages first, then offsets
    sum += n;
  }
  sum = __reduce_add_sync(0xffffffffu, sum);
  if (lane == 0) part[warp] = (int)sum;
  __syncthreads();
  uint32_t N = 0;                            // the host bounds it below 2^31
#pragma unroll
  for (int i = 0; i < kQ8Threads / 32; ++i) N += (uint32_t)part[i];
  N *= (uint32_t)p.H;
  const uint32_t round = (uint32_t)p.target * kQ8MaxPages, heads = (uint32_t)p.B * (uint32_t)p.H;
  const uint32_t slots = p.target * max(1u, (N + round - 1) / round), least = slots - slots / 4;
  const uint32_t room = slots > heads ? max(slots - heads, least) : least;
  const int c = (int)min((uint32_t)kQ8MaxPages, max(1u, (N + room - 1) / room));
  int items = 0;
  for (int b = b0; b < b1; ++b) items += (off[b] + c - 1) / c;
  int scan = items;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += t;
  }
  __syncthreads();
  if (lane == 31) part[warp] = scan;
  __syncthreads();
  int base = scan - items;
  for (int i = 0; i < warp; ++i) base += part[i];
  for (int b = b0; b < b1; ++b) {
    const int n = (off[b] + c - 1) / c;
    off[b] = base;
    base += n;
  }
  if (b1 == p.B && b0 < b1) off[p.B] = base;
  __syncthreads();
}

// Sequence of item u (the last b with off[b] <= u and items of its own)
__device__ __forceinline__ int q8_find(const int *off, int B, int u) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= u) lo = mid; else hi = mid;
  }
  return lo;
}

// D(16x8, s32) += A(16x32, s8, row) * B(32x8, s8, col)
__device__ __forceinline__ void mma_s8(int c[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                       uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// D(16x8, f32) += A(16x16, bf16, row) * B(16x8, bf16, col)
__device__ __forceinline__ void mma_bf16(float c[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 q8_ldg(const int8_t *p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}
__device__ __forceinline__ uint32_t word(const uint4 &u, int i) {
  return i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w;
}

// One query head as limbs: 16-bit integers of step 2^(e - 14), e the exponent of
// the head's largest magnitude: exact for BF16 values of the top 8 binades (but for
// +255/128 2^e, one unit more than two signed bytes hold), off by half a unit at most
// below; hi and lo rows of bytes.  Two limbs because four heads of two fill the eight
// columns of a product.  A whole warp.
template <int D>
__device__ __forceinline__ void q8_limbs(const uint16_t *q, int8_t *hi, int8_t *lo, float *step) {
  constexpr int VPL = D / 32;
  const int lane = threadIdx.x & 31;
  const KvRaw<VPL> raw = kv_load<VPL>(q + lane * VPL);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < VPL / 2; ++i) m = max(m, max(raw.w[i] & 0x7FFFu, (raw.w[i] >> 16) & 0x7FFFu));
  m = __reduce_max_sync(0xffffffffu, m);
  const bool finite = m < 0x7F80u;
  // times 2^(14 - e) in two exact steps (14 - e is 140 at most)
  const int e = max((int)(m >> 7) - 127, -126), up = min(14 - e, 100), rest = 14 - e - up;
  const float f0 = __int_as_float((127 + up) << 23), f1 = __int_as_float((127 + rest) << 23);
  uint32_t ph[(VPL + 3) / 4], pl[(VPL + 3) / 4];
#pragma unroll
  for (int i = 0; i < (VPL + 3) / 4; ++i) ph[i] = pl[i] = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const uint32_t bits = i & 1 ? raw.w[i / 2] >> 16 : raw.w[i / 2] & 0xFFFFu;
    // the clamp only meets +255/128 2^e, one unit above hi = lo = 127
    const int x = finite ? min(__float2int_rn(bf16_bits_to_f32(bits) * f0 * f1), 32639) : 0;
    const int l = ((x + 128) & 255) - 128;
    pl[i / 4] |= ((uint32_t)l & 0xFFu) << (8 * (i & 3));
    ph[i / 4] |= ((uint32_t)((x - l) >> 8) & 0xFFu) << (8 * (i & 3));
  }
  kv_store_codes<VPL>(hi + lane * VPL, ph);
  kv_store_codes<VPL>(lo + lane * VPL, pl);
  if (lane == 0)
    *step = finite ? __int_as_float((127 - up) << 23) * __int_as_float((127 - rest) << 23)
                   : __uint_as_float(0x7FC00000u);
}

// What the two contractions of a run of pages work on, one CTA of four warps.
template <int D, int NT>
struct Q8Shared {
  __align__(16) int8_t limbs[8 * NT][D + 16];
  float step[4 * NT];
  float m[4 * NT];                           // maxima of the heads
  float warp[kQ8Threads / 32][4 * NT];
  int page[kQ8MaxPages], live[kQ8MaxPages];  // ids, and keys that count, of the run's pages
  int list[kQ8MaxPages];
  uint32_t kept;                             // pages with a key above the threshold
};

__device__ __forceinline__ float max_nan(float a, float b) {   // a NaN wins
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Ids and live keys of a run's pages [p0, p0 + np) of sequence b, which has len keys of its
// own; a page outside the pool has none.
template <int D, int NT>
__device__ __forceinline__ void q8_pages(const Q8Params &p, Q8Shared<D, NT> &sm, int b, int len, int p0, int np) {
  if (threadIdx.x < np) {
    const int at = p0 + threadIdx.x, w = at - p.pp;
    int x = w < 0 ? p.ptable[at] : p.table[(size_t)b * p.W + w];
    int n = w < 0 ? p.prefix - 64 * at : len - 64 * w;
    if (x < 0 || x >= p.n_pages) {
      set_index_error();
      x = -1;
      n = 0;
    }
    sm.page[threadIdx.x] = x;
    sm.live[threadIdx.x] = n;
  }
}

// Logits (in units of log2 e) of the run's keys, put(key of the run, head, value), the
// maximum of each page's strip of 16 keys, put_max(page, strip, head, value; NaN
// where the strip has one), and in sm.warp those over the run (NaN passed over).  The
// first pages' rows are on their way before the query is
// prepared; `fresh`: the query's limbs and fragments are not those held.
template <int D, int NT, class Put, class PutMax>
__device__ __forceinline__ void q8_logits_run(const Q8Params &p, Q8Shared<D, NT> &sm, int b, int h,
                                              int np, bool fresh, uint32_t (&qf)[NT][D / 64][4],
                                              float (&step)[NT], Put put, PutMax put_max) {
  constexpr int DB = D / 64;                 // 64-byte blocks of a K row
  constexpr int DEPTH = 8 / DB;              // pages in flight per warp
  constexpr int GP = 4 * NT;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tig = lane & 3;
  // warp w: keys 16 w .. 16 w + 15 of every page
  const int key = 16 * warp + g;
  uint4 buf[DEPTH][DB][2];
  uint16_t sc[DEPTH][2];
  auto issue = [&](int pp, uint4 (*dst)[2], uint16_t *s) {
    const size_t ph = (size_t)max(0, sm.page[pp]) * p.H + h;
    const int8_t *src = p.k + (ph * 64 + key) * D + 16 * tig;
#pragma unroll
    for (int j = 0; j < DB; ++j) {
      dst[j][0] = q8_ldg(src + 64 * j);
      dst[j][1] = q8_ldg(src + 8 * D + 64 * j);
    }
    s[0] = __ldg(p.ks + ph * 64 + key);
    s[1] = __ldg(p.ks + ph * 64 + key + 8);
  };
#pragma unroll
  for (int d = 0; d < DEPTH; ++d)
    if (d < np) issue(d, buf[d], sc[d]);
  if (fresh) {
    for (int i = warp; i < GP; i += kQ8Threads / 32) {
      int8_t *hi = sm.limbs[2 * i], *lo = sm.limbs[2 * i + 1];
      if (i < p.G) {
        q8_limbs<D>(p.q + b * p.q_bs + (long long)(h * p.G + i) * p.q_hs, hi, lo, &sm.step[i]);
      } else {
        for (int j = lane; j < D; j += 32) hi[j] = lo[j] = 0;
        if (lane == 0) sm.step[i] = 0.f;
      }
    }
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < DB; ++j) {
        const uint4 w = *reinterpret_cast<const uint4 *>(&sm.limbs[8 * nt + g][64 * j + 16 * tig]);
        qf[nt][j][0] = w.x; qf[nt][j][1] = w.y; qf[nt][j][2] = w.z; qf[nt][j][3] = w.w;
      }
      step[nt] = sm.step[4 * nt + tig] * p.scale2;
    }
  }
  float mx[NT];                              // lane tig of every quad: head 4 nt + tig
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) mx[nt] = -INFINITY;
  for (int pb = 0; pb < np; pb += DEPTH) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      const int pp = pb + d;
      if (pp >= np) break;
      int acc[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[nt][i] = 0;
#pragma unroll
      for (int j = 0; j < DB; ++j)
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma_s8(acc[nt], word(buf[d][j][0], 2 * s), word(buf[d][j][1], 2 * s),
                   word(buf[d][j][0], 2 * s + 1), word(buf[d][j][1], 2 * s + 1), qf[nt][j][2 * s],
                   qf[nt][j][2 * s + 1]);
      const float k0 = bf16_bits_to_f32(sc[d][0]), k1 = bf16_bits_to_f32(sc[d][1]);
      const int live = sm.live[pp];
      if (pp + DEPTH < np) issue(pp + DEPTH, buf[d], sc[d]);
      const int at = 64 * pp + key;
      const bool v0 = key < live, v1 = key + 8 < live;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        // 256 hi + lo in exact integers, rounded once to FP32.  The two scales first: their
        // product lies near the logit, the sum times either may pass FP32's range
        const float l0 = v0 ? (float)(acc[nt][0] * 256 + acc[nt][1]) * (k0 * step[nt]) : -INFINITY;
        const float l1 = v1 ? (float)(acc[nt][2] * 256 + acc[nt][3]) * (k1 * step[nt]) : -INFINITY;
        put(at, 4 * nt + tig, l0);
        put(at + 8, 4 * nt + tig, l1);
        float m = max_nan(l0, l1);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (lane < 4) put_max(pp, warp, 4 * nt + lane, m);
        mx[nt] = fmaxf(mx[nt], m);
      }
    }
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
    if (lane < 4) sm.warp[warp][4 * nt + lane] = mx[nt];
  __syncthreads();
}

// The maximum of head `tid` over the warps of the CTA (tid < 4 NT).
template <int D, int NT>
__device__ __forceinline__ float q8_warps_max(const Q8Shared<D, NT> &sm) {
  float m = sm.warp[0][threadIdx.x];
#pragma unroll
  for (int w = 1; w < kQ8Threads / 32; ++w) m = fmaxf(m, sm.warp[w][threadIdx.x]);
  return m;
}

template <int D, int NT>
__global__ void __launch_bounds__(kQ8Threads, q8_occ(NT)) q8_logits_kernel(const Q8Params p) {
  constexpr int GP = 4 * NT;
  extern __shared__ int off[];
  __shared__ Q8Shared<D, NT> sm;
  const int tid = threadIdx.x;
  pdl_launch_dependents();
  q8_plan(p, off);
  if (blockIdx.x == 0)
    for (int b = tid; b <= p.B; b += kQ8Threads) p.off[b] = off[b];
  const uint32_t total = (uint32_t)off[p.B] * (uint32_t)p.H;
  int held = -1;                             // the (sequence, KV head) whose query is held
  uint32_t qf[NT][D / 64][4];
  float step[NT];
  for (uint32_t item = blockIdx.x; item < total; item += gridDim.x) {
    const int u = (int)(item / (uint32_t)p.H), h = (int)(item - (uint32_t)u * p.H);
    const int b = q8_find(off, p.B, u), len = q8_len(p, b);
    const int pages = p.pp + ((len + 63) >> 6), own = off[b + 1] - off[b];
    const int c = (pages + own - 1) / own;   // even shares of the sequence's pages
    const int p0 = (u - off[b]) * c, np = min(c, pages - p0);
    __syncthreads();                         // the previous item's shared memory is free
    q8_pages(p, sm, b, len, p0, np);
    __syncthreads();
    float *lg = p.logit + ((size_t)(b * p.H + h) * p.ctxp + 64 * p0) * GP;
    float *lm = p.smax + ((size_t)(b * p.H + h) * (p.ctxp >> 6) + p0) * 4 * GP;
    q8_logits_run<D, NT>(p, sm, b, h, np, held != b * p.H + h, qf, step,
                         [&](int key, int head, float v) { lg[key * GP + head] = v; },
                         [&](int page, int strip, int head, float v) { lm[(4 * page + strip) * GP + head] = v; });
    held = b * p.H + h;
    if (tid < GP) p.cmax[(size_t)item * GP + tid] = q8_warps_max(sm);
  }
}

// Weights of a page: [column][64 keys] of BF16, rows padded by 16 bytes so that a
// fragment's loads (8 columns x 4 key groups) meet every bank once.  The keys
// of each group of four are kept in the order 0, 2, 1, 3: a code word's even and
// odd bytes are then the fragment's pairs.
constexpr int kQ8WRow = 72;

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// What a head's maximum is subtracted as: a sequence without a finite logit subtracts
// nothing (its NaN logits stay NaN), and the heads that pad a tile lie below every
// threshold.
__device__ __forceinline__ float q8_reference(float m, bool padding) {
  return padding ? INFINITY : m == -INFINITY ? 0.f : m;
}

// The run's pages with a key at or above the threshold (lm: its strips' maxima, global
// or shared; references in sm.m), in order, into sm.list; returns their number.
template <int D, int NT>
__device__ __forceinline__ int q8_kept_pages(const Q8Params &p, Q8Shared<D, NT> &sm, int np, const float *lm) {
  constexpr int GP = 4 * NT;
  const int tid = threadIdx.x;
  if (tid == 0) sm.kept = 0;
  __syncthreads();
  uint32_t kept = 0;
#pragma unroll 4
  for (int i = tid; i < np * 4 * GP; i += kQ8Threads)
    if (!(lm[i] - sm.m[i % GP] < p.haze2)) kept |= 1u << (i / (4 * GP));
  kept = __reduce_or_sync(0xffffffffu, kept);
  if ((tid & 31) == 0 && kept) atomicOr(&sm.kept, kept);
  __syncthreads();
  kept = sm.kept;
  if (tid < np && (kept >> tid & 1)) sm.list[__popc(kept & ((1u << tid) - 1))] = tid;
  __syncthreads();
  return __popc(kept);
}

// Weights of the n kept pages from the run's logits (lg [key][4 NT], global or shared) and
// the references sm.m: two BF16 limbs of exp2(s - m) vs per head, and in sm.warp the
// sums of the exponentials per warp.  Warp w takes kept pages w, w + 4, ..; a lane two
// keys of a group of four.
template <int D, int NT>
__device__ __forceinline__ void q8_weights_run(const Q8Params &p, Q8Shared<D, NT> &sm,
                                               uint16_t (*wt)[8 * NT][kQ8WRow], int h, int n,
                                               const float *lg) {
  constexpr int GP = 4 * NT, NW = kQ8Threads / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float sum[GP], m[GP];
#pragma unroll
  for (int i = 0; i < GP; ++i) {
    sum[i] = 0.f;
    m[i] = sm.m[i];
  }
  const float haze2 = p.haze2;               // -inf where the truncation is off
  const int key = 4 * (lane >> 1) + (lane & 1);
#pragma unroll 2
  for (int x = warp; x < n; x += NW) {
    const int pp = sm.list[x];
    const size_t ph = (size_t)max(0, sm.page[pp]) * p.H + h;
    float s[2][GP], vs[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const float *src = lg + (64 * pp + key + 2 * t) * GP;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const float4 f = *reinterpret_cast<const float4 *>(src + 4 * i);
        s[t][4 * i] = f.x - m[4 * i]; s[t][4 * i + 1] = f.y - m[4 * i + 1];
        s[t][4 * i + 2] = f.z - m[4 * i + 2]; s[t][4 * i + 3] = f.w - m[4 * i + 3];
      }
      vs[t] = bf16_bits_to_f32(p.vs[ph * 64 + key + 2 * t]);
    }
#pragma unroll
    for (int i = 0; i < GP; ++i) {
      // (a NaN logit is kept)
      const float e0 = s[0][i] < haze2 ? 0.f : ex2_approx(s[0][i]);
      const float e1 = s[1][i] < haze2 ? 0.f : ex2_approx(s[1][i]);
      sum[i] += e0 + e1;
      // a key without weight adds nothing whatever its value scale holds
      const float w0 = e0 == 0.f ? 0.f : e0 * vs[0], w1 = e1 == 0.f ? 0.f : e1 * vs[1];
      const __nv_bfloat162 hi = __floats2bfloat162_rn(w0, w1);
      const uint32_t hb = *reinterpret_cast<const uint32_t *>(&hi);
      const __nv_bfloat162 lo =
          __floats2bfloat162_rn(w0 - __uint_as_float(hb << 16), w1 - __uint_as_float(hb & 0xFFFF0000u));
      *reinterpret_cast<uint32_t *>(&wt[x][2 * i][2 * lane]) = hb;
      *reinterpret_cast<uint32_t *>(&wt[x][2 * i + 1][2 * lane]) = *reinterpret_cast<const uint32_t *>(&lo);
    }
  }
#pragma unroll
  for (int i = 0; i < GP; ++i) {
#pragma unroll
    for (int o = 16; o; o >>= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
    if (lane == 0) sm.warp[warp][i] = sum[i];
  }
  __syncthreads();
}

// The sum of the exponentials of head `tid` over the warps of the CTA (tid < 4 NT).
template <int D, int NT>
__device__ __forceinline__ float q8_warps_sum(const Q8Shared<D, NT> &sm, int i) {
  float s = sm.warp[0][i];
#pragma unroll
  for (int w = 1; w < kQ8Threads / 32; ++w) s += sm.warp[w][i];
  return s;
}

// Sum of the weights times V over the run's n kept pages; put(head, dimension, value)
// for every head below G.  Warp w: rows (D / 4) w .. of V^T.  The first pages' rows are
// on their way before the weights are formed.
template <int D, int NT, class Put>
__device__ __forceinline__ void q8_pv_run(const Q8Params &p, Q8Shared<D, NT> &sm,
                                          uint16_t (*wt)[8 * NT][kQ8WRow], int h, int n, const float *lg,
                                          Put put) {
  constexpr int MT = D / 64;                 // 16-row tiles of V^T per warp
  constexpr int DEPTH = 8 / MT;              // pages in flight per warp
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
  const KvBits bits = p.bits;
  const int row = 16 * MT * warp + g;
  uint4 buf[DEPTH][MT][2];
  auto issue = [&](int x, uint4 (*dst)[2]) {
    const size_t ph = (size_t)max(0, sm.page[sm.list[x]]) * p.H + h;
    const int8_t *src = p.v + (ph * D + row) * 64 + 16 * tig;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      dst[i][0] = q8_ldg(src + 16 * i * 64);
      dst[i][1] = q8_ldg(src + (16 * i + 8) * 64);
    }
  };
#pragma unroll
  for (int d = 0; d < DEPTH; ++d)
    if (d < n) issue(d, buf[d]);
  q8_weights_run<D, NT>(p, sm, wt, h, n, lg);
  float acc[MT][NT][4];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][nt][j] = 0.f;
  for (int xb = 0; xb < n; xb += DEPTH) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      const int x = xb + d;
      if (x >= n) break;
      const uint16_t (*w)[kQ8WRow] = wt[x];
      uint32_t bw[NT][8];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint4 a = *reinterpret_cast<const uint4 *>(&w[8 * nt + g][16 * tig]);
        const uint4 e = *reinterpret_cast<const uint4 *>(&w[8 * nt + g][16 * tig + 8]);
        bw[nt][0] = a.x; bw[nt][1] = a.y; bw[nt][2] = a.z; bw[nt][3] = a.w;
        bw[nt][4] = e.x; bw[nt][5] = e.y; bw[nt][6] = e.z; bw[nt][7] = e.w;
      }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const uint32_t r0 = word(buf[d][i][0], s), r1 = word(buf[d][i][1], s);
          const uint32_t a0 = kv_bf16_pair(r0, bits), a2 = kv_bf16_pair(r0 >> 8, bits);
          const uint32_t a1 = kv_bf16_pair(r1, bits), a3 = kv_bf16_pair(r1 >> 8, bits);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma_bf16(acc[i][nt], a0, a1, a2, a3, bw[nt][2 * s], bw[nt][2 * s + 1]);
        }
      if (x + DEPTH < n) issue(x + DEPTH, buf[d]);
    }
  }
  // columns 2 tig and 2 tig + 1 are the limbs of one head
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int head = 4 * nt + tig;
    if (head < p.G) {
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        put(head, row + 16 * i, acc[i][nt][0] + acc[i][nt][1]);
        put(head, row + 16 * i + 8, acc[i][nt][2] + acc[i][nt][3]);
      }
    }
  }
}

// The references sm.m from every thread's share m of the maximum of head tid mod 4 NT,
// and with a prefix from its splits' maxima too; those go to mfin.  All threads.
template <int D, int NT>
__device__ __forceinline__ void q8_final_max(const Q8Params &p, Q8Shared<D, NT> &sm, float *s_red, int b,
                                             int h, float m) {
  constexpr int GP = 4 * NT;
  const int tid = threadIdx.x, i = tid % GP;
  if (p.splits > 0 && i < p.G) {
    const float *src = p.pmax + (size_t)h * p.rows + b * p.G + i;
#pragma unroll 4
    for (int t = tid / GP; t < p.splits; t += kQ8Threads / GP) m = fmaxf(m, src[(size_t)t * p.H * p.rows]);
  }
  s_red[tid] = m;
  __syncthreads();
  if (tid < GP) {
    for (int t = tid + GP; t < kQ8Threads; t += GP) m = fmaxf(m, s_red[t]);
    sm.m[tid] = q8_reference(m, tid >= p.G);
    if (p.splits > 0 && tid < p.G) p.mfin[(size_t)b * p.Hq + h * p.G + tid] = m;
  }
  __syncthreads();
}

// The largest value scale of the prefix for each KV head, over its splits.
__device__ __forceinline__ void q8_final_scale(const Q8Params &p) {
  const int lane = threadIdx.x & 31;
  for (int h = threadIdx.x >> 5; h < p.H; h += kQ8Threads / 32) {
    float m = 0.f;
#pragma unroll 4
    for (int t = lane; t < p.splits; t += 32) m = fmaxf(m, p.psv[(size_t)t * p.H + h]);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) p.svfin[h] = m;
  }
}

template <int D, int NT>
__global__ void __launch_bounds__(kQ8Threads, q8_occ(NT)) q8_pv_kernel(const Q8Params p) {
  constexpr int GP = 4 * NT;
  extern __shared__ __align__(16) uint8_t q8_dsm[];
  uint16_t (*wt)[8 * NT][kQ8WRow] = reinterpret_cast<uint16_t (*)[8 * NT][kQ8WRow]>(q8_dsm);
  int *off = reinterpret_cast<int *>(q8_dsm + sizeof(uint16_t) * kQ8MaxPages * 8 * NT * kQ8WRow);
  __shared__ Q8Shared<D, NT> sm;
  __shared__ float s_red[kQ8Threads];
  const int tid = threadIdx.x;
  pdl_launch_dependents();
  q8_plan(p, off);
  const uint32_t total = (uint32_t)off[p.B] * (uint32_t)p.H;
  pdl_wait();                                // the logits and maxima of q8_logits
  if (p.splits > 0) {
    if (blockIdx.x == 0) q8_final_scale(p);
    // sequences without own keys have no item: their maxima are the prefix's
    for (uint32_t i = blockIdx.x; i < (uint32_t)p.B * p.H; i += gridDim.x) {
      const int b = i / (uint32_t)p.H, h = i - (uint32_t)b * p.H;
      if (off[b] == off[b + 1]) q8_final_max<D, NT>(p, sm, s_red, b, h, -INFINITY);
    }
  }
  for (uint32_t item = blockIdx.x; item < total; item += gridDim.x) {
    const int u = (int)(item / (uint32_t)p.H), h = (int)(item - (uint32_t)u * p.H);
    const int b = q8_find(off, p.B, u), len = q8_len(p, b);
    const int pages = p.pp + ((len + 63) >> 6), own = off[b + 1] - off[b];
    const int c = (pages + own - 1) / own;   // even shares of the sequence's pages
    const int p0 = (u - off[b]) * c, np = min(c, pages - p0);
    __syncthreads();                         // the previous item's shared memory is free
    q8_pages(p, sm, b, len, p0, np);
    // the final maximum of each head over the sequence's items
    {
      const int i = tid % GP;
      float m = -INFINITY;
      for (int t = off[b] + tid / GP; t < off[b + 1]; t += kQ8Threads / GP)
        m = fmaxf(m, p.cmax[((size_t)t * p.H + h) * GP + i]);
      q8_final_max<D, NT>(p, sm, s_red, b, h, m);
    }
    const size_t first = (size_t)(b * p.H + h) * p.ctxp + 64 * p0;   // the run's first key
    const int n = q8_kept_pages<D, NT>(p, sm, np, p.smax + first / 16 * GP);
    float *dst = p.pacc + (size_t)item * p.G * D;
    q8_pv_run<D, NT>(p, sm, wt, h, n, p.logit + first * GP,
                     [&](int head, int d, float v) { dst[head * D + d] = v; });
    if (tid < GP) p.psum[(size_t)item * GP + tid] = q8_warps_sum(sm, tid);
  }
}

// One launch: a CTA takes all keys of one sequence and KV head, or a cluster of p.cluster
// CTAs does, an even share of its pages each (at most kQ8MaxPages); the logits stay
// in shared memory.  The cluster's CTAs read each other's maxima there, and at the end
// each a share of the outputs of all partial sums, added in order.
// Prefix: the own keys behind a shared prefix that the prefix kernels take: one CTA, a partial
// sum for q8_merge; the logits are formed beside the prefix's maximum pass.
template <int D, int NT, bool Prefix>
__global__ void __launch_bounds__(kQ8Threads, q8_occ(NT)) q8_short_kernel(const Q8Params p) {
  constexpr int GP = 4 * NT;
  extern __shared__ __align__(16) uint8_t q8_dsm[];
  const int C = Prefix ? 1 : p.cluster, pages = ((p.ctxp >> 6) + C - 1) / C;
  uint16_t (*wt)[8 * NT][kQ8WRow] = reinterpret_cast<uint16_t (*)[8 * NT][kQ8WRow]>(q8_dsm);
  float *lg = reinterpret_cast<float *>(q8_dsm + sizeof(uint16_t) * pages * 8 * NT * kQ8WRow);
  float *lm = lg + 64 * pages * GP;
  float *part = lm + 4 * pages * GP;         // [G][D], of a cluster
  __shared__ Q8Shared<D, NT> sm;
  __shared__ float s_red[kQ8Threads];
  __shared__ float s_max[GP], s_sum[GP];     // read by the cluster
  const int tid = threadIdx.x, h = blockIdx.x, rank = blockIdx.y, b = blockIdx.z;
  const int len = q8_len(p, b), all = p.pp + ((len + 63) >> 6);
  const int c = (all + C - 1) / C, p0 = min(rank * c, all), np = min(c, all - p0);
  if constexpr (Prefix) pdl_launch_dependents();
  const size_t at = ((size_t)b * p.Hq + h * p.G) * D;
  auto store = [&](int i, float v) {
    if (p.out_bf16) static_cast<uint16_t *>(p.out)[at + i] = f32_to_bf16_rn_bits(v);
    else static_cast<float *>(p.out)[at + i] = v;
  };
  if (!Prefix && C == 1 && np == 0) {        // no key: zeros
    for (int i = tid; i < p.G * D; i += kQ8Threads) store(i, 0.f);
    return;
  }
  q8_pages(p, sm, b, len, p0, np);
  __syncthreads();
  uint32_t qf[NT][D / 64][4];
  float step[NT];
  q8_logits_run<D, NT>(p, sm, b, h, np, true, qf, step,
                       [&](int key, int head, float v) { lg[key * GP + head] = v; },
                       [&](int page, int strip, int head, float v) { lm[(4 * page + strip) * GP + head] = v; });
  if constexpr (Prefix) {
    pdl_wait();                              // the prefix's maxima
    if (h == 0 && b == 0) q8_final_scale(p);
    q8_final_max<D, NT>(p, sm, s_red, b, h, tid < GP ? q8_warps_max(sm) : -INFINITY);
  } else {
    float m = tid < GP ? q8_warps_max(sm) : -INFINITY;
    if (C > 1) {
      if (tid < GP) s_max[tid] = m;
      cluster_sync();
      if (tid < GP)
        for (int r = 0; r < C; ++r) m = fmaxf(m, ld_cluster_f32(cluster_map(smem_u32(&s_max[tid]), r)));
    }
    if (tid < GP) sm.m[tid] = q8_reference(m, tid >= p.G);
    __syncthreads();
  }
  const int n = q8_kept_pages<D, NT>(p, sm, np, lm);
  if constexpr (Prefix) {
    const size_t item = (size_t)b * p.H + h;
    float *dst = p.pacc + item * p.G * D;
    q8_pv_run<D, NT>(p, sm, wt, h, n, lg, [&](int head, int d, float v) { dst[head * D + d] = v; });
    if (tid < GP) p.psum[item * GP + tid] = q8_warps_sum(sm, tid);
  } else if (C == 1) {
    q8_pv_run<D, NT>(p, sm, wt, h, n, lg, [&](int head, int d, float v) {
      const float sum = q8_warps_sum(sm, head);
      store(head * D + d, sum == 0.f ? 0.f : v / sum);
    });
  } else {
    q8_pv_run<D, NT>(p, sm, wt, h, n, lg, [&](int head, int d, float v) { part[head * D + d] = v; });
    if (tid < GP) s_sum[tid] = q8_warps_sum(sm, tid);
    cluster_sync();
    for (int i = rank * kQ8Threads + tid; i < p.G * D; i += C * kQ8Threads) {
      float v = 0.f, sum = 0.f;
#pragma unroll 4
      for (int r = 0; r < C; ++r) {
        sum += ld_cluster_f32(cluster_map(smem_u32(&s_sum[i / D]), r));
        v += ld_cluster_f32(cluster_map(smem_u32(&part[i]), r));
      }
      store(i, sum == 0.f ? 0.f : v / sum);
    }
    cluster_sync();                          // the others have read this CTA's share
  }
}

// out of one query head: the partials of the sequence's items, then those of the
// prefix's splits, added in order (thread group j the j-th share of them),
// divided by the sum of the weights.
// NV vectors of 4 dimensions per CTA: 16 where there are few rows (a long axis of
// partials in 16 shares), else all of them (1024 rows of 256 with 19 partials each: 11 us
// against 18).
template <int D, int NV>
__global__ void __launch_bounds__(256) q8_merge_kernel(const Q8Params p, int GP) {
  constexpr int J = 256 / NV;
  __shared__ float4 s_acc[J][NV];
  __shared__ float s_sum[J];
  const int hq = blockIdx.x, b = blockIdx.y, h = hq / p.G, i = hq - h * p.G;
  const int v = NV * blockIdx.z + threadIdx.x % NV, j = threadIdx.x / NV;
  pdl_wait();
  const int t0 = p.single ? b : p.off[b], own = p.single ? 1 : p.off[b + 1] - t0, nt = own + p.splits;
  const int a = (int)((long long)nt * j / J), z = (int)((long long)nt * (j + 1) / J);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
#pragma unroll 4
  for (int t = a; t < z; ++t) {
    const long long item = (long long)(t0 + t) * p.H + h;
    const long long row = ((long long)(t - own) * p.H + h) * p.rows + (long long)b * p.G + i;
    const float *src = t < own ? p.pacc + (item * p.G + i) * D : p.po + row * D;
    const float4 x = *reinterpret_cast<const float4 *>(src + 4 * v);
    sum += t < own ? p.psum[item * GP + i] : p.pl[row];
    acc.x += x.x; acc.y += x.y; acc.z += x.z; acc.w += x.w;
  }
  s_acc[j][threadIdx.x % NV] = acc;
  if (threadIdx.x % NV == 0) s_sum[j] = sum;
  __syncthreads();
  if (j != 0) return;
#pragma unroll
  for (int t = 1; t < J; ++t) {
    const float4 x = s_acc[t][threadIdx.x];
    acc.x += x.x; acc.y += x.y; acc.z += x.z; acc.w += x.w;
    sum += s_sum[t];
  }
  if (sum == 0.f) acc = make_float4(0.f, 0.f, 0.f, 0.f);   // no key: zeros
  else { acc.x /= sum; acc.y /= sum; acc.z /= sum; acc.w /= sum; }
  const size_t at = ((size_t)b * p.Hq + hq) * D + 4 * v;
  if (p.out_bf16) {
    uint2 o;
    o.x = f32_to_bf16_rn_bits(acc.x) | (uint32_t)f32_to_bf16_rn_bits(acc.y) << 16;
    o.y = f32_to_bf16_rn_bits(acc.z) | (uint32_t)f32_to_bf16_rn_bits(acc.w) << 16;
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + at) = o;
  } else {
    *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) = acc;
  }
}

namespace {
int q8_pages_max(const Q8Shape &s);
struct Q8Layout {
  size_t logit, smax, cmax, psum, pacc, off, total;
  int target;
  long long items;               // bound on the items of one call
};
// Items: sum_b ceil(pages_b / c) H <= N / c + B H <= target r + B H.
Q8Layout q8_layout(const Q8Shape &s) {
  Q8Layout y{};
  const int G = s.Hq / s.Hkv, NT = q8_tiles(G);
  const long long pages = q8_pages_max(s);
  y.target = kQ8Sms * q8_occ(NT);
  const long long N = pages * s.B * s.Hkv, round = (long long)y.target * kQ8MaxPages;
  y.items = std::min(N, y.target * ((N + round - 1) / round) + (long long)s.B * s.Hkv);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += (bytes + 255) & ~(size_t)255;
    return o;
  };
  y.logit = take((size_t)s.B * s.Hkv * pages * 64 * 4 * NT * 4);
  y.smax = take((size_t)s.B * s.Hkv * pages * 4 * 4 * NT * 4);
  y.cmax = take((size_t)y.items * 4 * NT * 4);
  y.psum = take((size_t)y.items * 4 * NT * 4);
  y.pacc = take((size_t)y.items * G * s.D * 4);
  y.off = take((size_t)(s.B + 1) * 4);
  y.total = at;
  return y;
}

size_t q8_pv_smem(int NT, int B) {
  return sizeof(uint16_t) * kQ8MaxPages * 8 * NT * kQ8WRow + (size_t)(B + 1) * 4;
}

// CTAs per sequence and KV head of the one-launch form, 0: three launches.  Up to 16 pages
// one CTA; a cluster where that leaves SMs idle and there is enough to share.  Up to 64
// pages the largest cluster that fits the resident CTAs, as long as a CTA gets at most 8
// pages (16 of 64 dimensions, whose CTA needs less time per page); up to 32 pages 4 CTAs
// also past that, unless 9 to 16 query heads leave room for one CTA per SM.  Beyond, three
// launches spread ragged lengths better, but for few rows of 64 dimensions.  Measured in us (16/4 heads of 256; one launch with
// 1 / 2 / 4 / 8 CTAs, three launches):
//   1 x 100 keys 5.5 / 7.5 / 6.5 / 6.5, 9.6        16 x 4096   - / - / 34 / 28, 36
//   1 x 1024     17.8 / 13.3 / 9.2 / 7.5, 10.2     1 x 8192    - / - / - / 19.8, 17.1
//   16 x 1024    17.8 / 13.7 / 11.3 / 11.3, 18.1   64 x 1024   32 / 29 / 33 / 41, 36
//   16 x <= 2048 - / 21.5 / 15.6 / 12.4, 17.5      148 x 1024  51 / 57 / 68 / 86, 64
// 148 x 4096 of 16/2 heads of 128: - / - / 100 / 100, 87; of 8/8 heads of 64: - / - / 152 / 187, 186;
// 4 x 8192 of those - / - / - / 13.7, 18.4.
int q8_cluster(const Q8Shape &s, int pages) {
  const int NT = q8_tiles(s.Hq / s.Hkv), slots = kQ8Sms * q8_occ(NT), rows = s.B * s.Hkv;
  if (pages > 64) return s.D == 64 && pages <= 8 * kQ8MaxPages && 8 * rows <= slots ? 8 : 0;
  const bool few = pages <= kQ8MaxPages;
  int C = 1;
  if (!few || (pages * s.D > 512 && 4 * rows <= slots))
    while (C < 8 && 2 * C * rows <= slots && pages > C) C *= 2;
  if (few) return C;
  if (s.D == 64) C = std::max(C, pages <= 32 ? 2 : 4);
  else if (pages <= 32 && NT <= 2) C = std::max(C, 4);
  return pages <= C * (s.D == 64 ? kQ8MaxPages : 8) ? C : 0;
}
// Whether a prefix is taken as the first keys of each sequence, which reads it once per
// sequence (from the L2 after the first) but without the prefix kernels' four launches and
// preparation of Q.  Measured in us, these kernels / the prefix kernels, by page visits
// (sequences x KV heads x pages of the prefix):
//   16/4 heads of 256: 4 x 512 keys (128 visits) 7.9 / 18, 16 x 3000 (3008) 19 / 29,
//   4 x 16000 (4000) 28 / 33, 8 x 9000 (4512) 30 / 29, 48 x 1900 (5760) 34 / 29;
//   16/2 of 128: 24 x 5001 (3792) 24 / 25, 48 x 3000 (4512) 27 / 26; 8/8 of 64: 24 x 1900
//   (5760) 15 / 20, 24 x 3000 (9024) 24 / 21; 32/2 of 256: 16 x 5001 (2528) 34 / 36,
//   48 x 1900 (2880) 38 / 38, 8 x 16000 (4000) 46 / 38.
// The rule is a compromise: it counts visits, not a page's bytes, and of 64 dimensions the
// joined form is ahead up to about 8000 visits (2 x 32768 keys 25 / 47), which it leaves.
bool q8_joins(const Q8Shape &s) {
  const long long rows = (long long)s.B * s.Hkv, pages = (s.prefix + 63) / 64;
  return s.prefix > 0 && rows * pages <= (s.Hq / s.Hkv <= 8 ? 4096 : 2400) &&
         rows * (pages + (s.ctx + 63) / 64) <= INT32_MAX;
}
// Pages of a sequence at most, as these kernels take it.
int q8_pages_max(const Q8Shape &s) {
  return (s.ctx + 63) / 64 + (q8_joins(s) ? (s.prefix + 63) / 64 : 0);
}
// Whether the (own) keys of a sequence take one launch.
bool q8_is_short(const Q8Shape &s) {
  if (s.prefix > 0 && !q8_joins(s)) return (s.ctx + 63) / 64 <= kQ8MaxPages;
  return q8_cluster(s, q8_pages_max(s)) > 0;
}
size_t q8_short_smem(int NT, int pages, int part) {
  return (size_t)pages * (sizeof(uint16_t) * 8 * NT * kQ8WRow + (64 + 4) * 4 * NT * sizeof(float)) + part * sizeof(float);
}

template <int D, int NT>
cudaError_t q8_run_short(const Q8Params &p, cudaStream_t st, Launcher &L) {
  const int C = p.splits > 0 ? 1 : p.cluster;
  const dim3 grid((unsigned)p.H, (unsigned)C, (unsigned)p.B), block(kQ8Threads);
  const size_t smem = q8_short_smem(NT, (p.ctxp / 64 + C - 1) / C, C > 1 ? p.G * D : 0);
  if (p.splits > 0)
    return L.launch("q8_short", q8_short_kernel<D, NT, true>, grid, block, smem, st, true, p);
  return L.launch_ex("q8_short", q8_short_kernel<D, NT, false>, grid, block, smem, st, false, C > 1 ? C : 0, p);
}

template <int D>
cudaError_t q8_run_merge(const Q8Params &p, int GP, cudaStream_t st, Launcher &L) {
  if (p.B * p.Hq < 2 * kQ8Sms)
    return L.launch("q8_merge", q8_merge_kernel<D, 16>, dim3((unsigned)p.Hq, (unsigned)p.B, D / 64),
                    dim3(256), 0, st, true, p, GP);
  return L.launch("q8_merge", q8_merge_kernel<D, D / 4>, dim3((unsigned)p.Hq, (unsigned)p.B),
                  dim3(256), 0, st, true, p, GP);
}

template <int D, int NT>
cudaError_t q8_run(const Q8Params &p, long long items, cudaStream_t st, Launcher &L) {
  const dim3 grid((unsigned)std::min<long long>(items, p.target)), block(kQ8Threads);
  cudaError_t e = L.launch("q8_logits", q8_logits_kernel<D, NT>, grid, block, (size_t)(p.B + 1) * 4,
                           st, false, p);
  if (e != cudaSuccess) return e;
  e = L.launch("q8_pv", q8_pv_kernel<D, NT>, grid, block, q8_pv_smem(NT, p.B), st, true, p);
  if (e != cudaSuccess) return e;
  return q8_run_merge<D>(p, 4 * NT, st, L);
}
}  // namespace

size_t q8_workspace_bytes(const Q8Shape &s) { return q8_is_short(s) ? 0 : q8_layout(s).total; }

cudaError_t prepare_q8_kernels() {
  cudaError_t e = cudaSuccess;
  auto set = [&](const void *k, int NT) {
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)q8_pv_smem(NT, 4096));
  };
  auto set_short = [&](const void *k, int NT) {
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)q8_short_smem(NT, kQ8MaxPages, 4 * NT * 256));
  };
  set_short((const void *)q8_short_kernel<64, 1, false>, 1);
  set_short((const void *)q8_short_kernel<64, 1, true>, 1);
  set_short((const void *)q8_short_kernel<64, 2, false>, 2);
  set_short((const void *)q8_short_kernel<64, 2, true>, 2);
  set_short((const void *)q8_short_kernel<64, 4, false>, 4);
  set_short((const void *)q8_short_kernel<64, 4, true>, 4);
  set_short((const void *)q8_short_kernel<128, 1, false>, 1);
  set_short((const void *)q8_short_kernel<128, 1, true>, 1);
  set_short((const void *)q8_short_kernel<128, 2, false>, 2);
  set_short((const void *)q8_short_kernel<128, 2, true>, 2);
  set_short((const void *)q8_short_kernel<128, 4, false>, 4);
  set_short((const void *)q8_short_kernel<128, 4, true>, 4);
  set_short((const void *)q8_short_kernel<256, 1, false>, 1);
  set_short((const void *)q8_short_kernel<256, 1, true>, 1);
  set_short((const void *)q8_short_kernel<256, 2, false>, 2);
  set_short((const void *)q8_short_kernel<256, 2, true>, 2);
  set_short((const void *)q8_short_kernel<256, 4, false>, 4);
  set_short((const void *)q8_short_kernel<256, 4, true>, 4);
  set((const void *)q8_pv_kernel<64, 1>, 1);
  set((const void *)q8_pv_kernel<64, 2>, 2);
  set((const void *)q8_pv_kernel<64, 4>, 4);
  set((const void *)q8_pv_kernel<128, 1>, 1);
  set((const void *)q8_pv_kernel<128, 2>, 2);
  set((const void *)q8_pv_kernel<128, 4>, 4);
  set((const void *)q8_pv_kernel<256, 1>, 1);
  set((const void *)q8_pv_kernel<256, 2>, 2);
  set((const void *)q8_pv_kernel<256, 4>, 4);
  return e;
}

namespace {
Q8Params q8_params(const Q8Args &a, const Q8Layout &y) {
  char *ws = static_cast<char *>(a.workspace);
  Q8Params p{};
  p.q = a.q; p.q_bs = a.q_bs; p.q_hs = a.q_hs;
  p.k = a.pool.k; p.v = a.pool.v; p.ks = a.pool.ks; p.vs = a.pool.vs;
  p.table = a.pool.table; p.lens = a.lens;
  p.out = a.out; p.out_bf16 = a.out_bf16;
  p.logit = reinterpret_cast<float *>(ws + y.logit);
  p.smax = reinterpret_cast<float *>(ws + y.smax);
  p.cmax = reinterpret_cast<float *>(ws + y.cmax);
  p.psum = reinterpret_cast<float *>(ws + y.psum);
  p.pacc = reinterpret_cast<float *>(ws + y.pacc);
  p.off = reinterpret_cast<int *>(ws + y.off);
  p.B = a.s.B; p.Hq = a.s.Hq; p.H = a.s.Hkv; p.G = a.s.Hq / a.s.Hkv; p.W = a.pool.W;
  p.n_pages = a.pool.n_pages; p.ctx = a.s.ctx; p.ctxp = (a.s.ctx + 63) / 64 * 64;
  p.target = y.target;
  p.scale2 = (float)((double)a.tau / sqrt((double)a.s.D) * 1.4426950408889634);
  p.bits = kKvBits;
  p.haze2 = a.haze > 0.f ? -a.haze * 1.44269504f : -INFINITY;
  return p;
}
}  // namespace

cudaError_t launch_q8_attention(const Q8Args &a, cudaStream_t st, Launcher &L) {
  const Q8Layout y = q8_layout(a.s);
  Q8Params p = q8_params(a, y);
  p.ctxp = 64 * q8_pages_max(a.s);
  p.cluster = q8_cluster(a.s, p.ctxp / 64);
  if (a.s.prefix > 0) {
    p.ptable = a.ptable; p.prefix = a.s.prefix; p.pp = (a.s.prefix + 63) / 64;
  }
  const bool once = p.cluster > 0;
  const int NT = q8_tiles(p.G);
#define Q8_CASE(D_, N_) \
  if (a.s.D == D_ && NT == N_)                            \
    return once ? q8_run_short<D_, N_>(p, st, L) : q8_run<D_, N_>(p, y.items, st, L);
  Q8_CASE(64, 1) Q8_CASE(64, 2) Q8_CASE(64, 4)
  Q8_CASE(128, 1) Q8_CASE(128, 2) Q8_CASE(128, 4)
  Q8_CASE(256, 1) Q8_CASE(256, 2) Q8_CASE(256, 4)
#undef Q8_CASE
  return cudaErrorInvalidValue;
}

}  // namespace dvssq
