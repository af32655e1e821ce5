// KV-BSS decode attention of a batch over a prefix that all its sequences share
// (dvssq_bss_attention_prefix), on the 5th-generation tensor cores.  The
// B G queries of a KV head are the rows of one matrix, so the prefix is a pair
// of dense products instead of B walks over it:
//   S = Q K^T,   w = exp(S - m) vs (zero below the haze threshold),   O = w V
// The haze threshold needs each row's final maximum first, so Q K^T runs twice:
//   pfx_max   S and each split's row maxima, and its largest value scale per KV head
//   pfx_pv    S again (K comes from L2 now), the weights, and a split's O
// (A prefix of few page visits is taken by those kernels as well: q8_joins.)
// Each sequence's own keys go through q8_short, or q8_logits and q8_pv, as without a
// prefix; those form the maxima over prefix and own keys between the two passes,
// and q8_merge adds the items' and the splits' partials in order.
//
// A CTA holds 128 rows of Q and walks a split of the prefix page by page (64
// keys).  Converting warpgroups bring pages from global memory through registers,
// where the 8-bit codes become FP16, into a ring of 128-byte-swizzled tiles (a
// warpgroup per page in turn, in the order the products take them); one warp
// issues the MMAs; warps 0-7 turn S into weights (a thread per row, a warpgroup per
// half of the page's keys).  Q lies in tensor memory and the weights overwrite
// their S there, so that both products read one operand only from shared memory
// (staging the raw codes there too was slower).  Q K^T of page j + 1 is issued
// before w V of page j.
//
// Measured, 64 sequences of 16/4 heads of 256 over 32768 keys (34.5 GFLOP and 88 MB: floor
// 21 us of tensor rate, 31 with the second Q K^T): 85 us in a graph, of which maximum pass
// 24, weight pass 46, own keys and merge the rest.  A page takes about 2300 cycles in the
// weight pass against 1024 of products: the converting warps' loads, conversions and
// shared-memory stores bound it (the load-store pipe is busy 50 % of the time, the
// schedulers 56 %, the tensor pipe 37 %).
//
// Number formats: a code is exact in FP16 (1024 + u from a byte permutation,
// minus 1152), and so is a query scaled by a power of two to 2^14 .. 2^15 (BF16
// has 8 significant bits; values 2^29 below the row's largest vanish), so S is
// FP32-grade.  A weight is rounded once to FP16 (2^-11 relative), scaled by
// 2^(14 - e) with 2^e at or above the head's largest vs: the rounding holds
// down to e^-19 of the largest weight, and what underflows is below 2^-38 of it
// (largest value scales from 2^-86; below, the weights lose bits).
#include "common.cuh"
#include "kernels.h"

namespace dvssq {

constexpr int kPfxConv = 3;              // converting warpgroups
constexpr int kPfxThreads = (3 + kPfxConv) * 128;   // two of weights and one that issues beside them
constexpr int kPfxMma = 4 * (2 + kPfxConv);         // the issuing warp

struct PfxParams {
  Q8Params q8;
  const int32_t *ptable;
  int prefix, pages, splits, rows;          // rows = B G per KV head
  float *pmax;                   // [splits][H][rows] row maxima
  float *psv;                    // [splits][H] largest finite value scales
  float *po;                     // [splits][H][rows][D]
  float *pl;                     // [splits][H][rows]
  uint32_t magic;                // 0x64646464
  float nzero;                   // -0
};

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t r[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

// Waits for the thread's tensor-memory loads; the values pass through, so that no
// use of them can be placed before the wait.
__device__ __forceinline__ void tmem_ld_wait32(uint32_t r[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                 "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]),
                 "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29])
               :
               : "memory");
  asm volatile("" : "+r"(r[30]), "+r"(r[31]) : : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t r[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
      :
      : "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
        "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
        "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
        "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t r[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
               :
               : "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
                 "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// D[tmem] (+)= A[tmem] * B[smem desc], kind::f16 (A: two FP16 per 32-bit column).
// The whole warp runs the issuing code and one lane (`lead`) is predicated in: the
// operands then live in uniform registers (a branch on the lane cost 100 cycles
// per product issued).
__device__ __forceinline__ void tc_mma_f16_ta(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem,
                                              uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 e, %5, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void tc_commit_lead(uint32_t lead, uint64_t *bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_u32(bar)),
      "r"(lead)
      : "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(r));
  return r;
}

// 16 codes -> 16 FP16 values in order, as two 16-byte chunks.  `magic` is 0x64646464, a
// kernel parameter: as a literal beside the selector it is not held in a register.
__device__ __forceinline__ void pfx_f16(const uint4 &c, uint32_t magic, uint4 &lo, uint4 &hi) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t o[8];
  const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u = w[i] ^ 0x80808080u;
    uint32_t a = __byte_perm(u, magic, 0x4140), b = __byte_perm(u, magic, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<__half2 *>(&a), bias);
    const __half2 y = __hsub2(*reinterpret_cast<__half2 *>(&b), bias);
    o[2 * i] = *reinterpret_cast<const uint32_t *>(&x);
    o[2 * i + 1] = *reinterpret_cast<const uint32_t *>(&y);
  }
  lo = make_uint4(o[0], o[1], o[2], o[3]);
  hi = make_uint4(o[4], o[5], o[6], o[7]);
}

// mbar_wait with the limit at hand: read once per thread, because a wait that has to
// read it wakes up late by that load's latency.
__device__ __forceinline__ bool pfx_wait(uint64_t *bar, uint32_t parity, long long limit) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (clock64() - t0 > limit) {
      set_error(kErrWaitMbarrier);
      return false;
    }
  }
  return true;
}

// A row's 32 products of half a page: their largest logit S (ks r2) (a NaN is passed over).
// The two scales first: their product lies near the logit, S times either may pass FP32's range.
// Whole: all the page's keys are live; else the half's first nv are.
template <bool Whole>
__device__ __forceinline__ float pfx_half_max(const uint32_t *s, const float *ks, int nv, float r2) {
  const float2 rr = make_float2(r2, r2);
  float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    const float4 a = *reinterpret_cast<const float4 *>(ks + i);
    const float2 x = mat_mul2(make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), mat_mul2(make_float2(a.x, a.y), rr));
    const float2 y = mat_mul2(make_float2(__uint_as_float(s[i + 2]), __uint_as_float(s[i + 3])), mat_mul2(make_float2(a.z, a.w), rr));
    if (Whole || i < nv) m0 = fmaxf(m0, x.x);
    if (Whole || i + 1 < nv) m0 = fmaxf(m0, x.y);
    if (Whole || i + 2 < nv) m1 = fmaxf(m1, y.x);
    if (Whole || i + 3 < nv) m1 = fmaxf(m1, y.y);
  }
  return fmaxf(m0, m1);
}

// A row's weights of a quarter of a page (16 keys), FP16 pairs exp2(t - m) (vs up), and
// the sum of the exponentials.  t = S (ks r2) is rounded as the maximum pass rounds it, and
// only then does m come off: the largest key's difference is zero, however large the logits
// are (fused into one operation it is the product's rounding error, which passes any
// threshold and FP16's range in turn).  The second product is a packed FMA with `nzero`,
// -0 from a kernel parameter: a packed multiplication before a packed addition is compiled
// into one FMA, .rn or not.  `up`, the power of two that brings the weights into
// FP16's range, goes with the value scale, so that the sum needs none.
// Whole: all the page's keys are live and no value scale is a NaN.  The two
// bodies are apart so that each is one straight block for the scheduler: with the
// choice inside the loop 64 keys took 2700 cycles instead of 1700.
template <bool Whole>
__device__ __forceinline__ float2 pfx_weights16(const uint32_t *s, const float *ks, const float *vs,
                                                   int nv, float r2, float m, float haze2, float up, float nzero,
                                                   uint32_t *w) {
  const float2 rr = make_float2(r2, r2), nm = make_float2(-m, -m), uu = make_float2(up, up);
  const float2 nz = make_float2(nzero, nzero);
  float2 sum = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    const float4 a = *reinterpret_cast<const float4 *>(ks + i);
    const float4 v = *reinterpret_cast<const float4 *>(vs + i);
    const float2 vx = mat_mul2(make_float2(v.x, v.y), uu), vy = mat_mul2(make_float2(v.z, v.w), uu);
    const float2 x = mat_add2(mat_fma2(make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), mat_mul2(make_float2(a.x, a.y), rr), nz), nm);
    const float2 y = mat_add2(mat_fma2(make_float2(__uint_as_float(s[i + 2]), __uint_as_float(s[i + 3])), mat_mul2(make_float2(a.z, a.w), rr), nz), nm);
    float2 ex = make_float2(ex2_approx(x.x), ex2_approx(x.y));
    float2 ey = make_float2(ex2_approx(y.x), ex2_approx(y.y));
    float2 wx, wy;
    // below the haze threshold: dropped (a NaN logit is kept)
    if (x.x < haze2) ex.x = 0.f;
    if (x.y < haze2) ex.y = 0.f;
    if (y.x < haze2) ey.x = 0.f;
    if (y.y < haze2) ey.y = 0.f;
    if (Whole) {
      wx = mat_mul2(ex, vx);
      wy = mat_mul2(ey, vy);
    } else {
      // keys past the prefix's end weigh nothing, and the value scale of a key
      // without weight is not looked at
      if (i >= nv) ex.x = 0.f;
      if (i + 1 >= nv) ex.y = 0.f;
      if (i + 2 >= nv) ey.x = 0.f;
      if (i + 3 >= nv) ey.y = 0.f;
      wx = make_float2(ex.x == 0.f ? 0.f : ex.x * vx.x, ex.y == 0.f ? 0.f : ex.y * vx.y);
      wy = make_float2(ey.x == 0.f ? 0.f : ey.x * vy.x, ey.y == 0.f ? 0.f : ey.y * vy.y);
    }
    sum = mat_add2(sum, mat_add2(ex, ey));
    const __half2 ox = __floats2half2_rn(wx.x, wx.y), oy = __floats2half2_rn(wy.x, wy.y);
    w[i / 2] = *reinterpret_cast<const uint32_t *>(&ox);
    w[i / 2 + 1] = *reinterpret_cast<const uint32_t *>(&oy);
  }
  return sum;
}

template <int D, bool PV>
struct PfxSmem {
  static constexpr int DB = D / 64;
  static constexpr int R = 6;                            // FP16 pages
  static constexpr int kSlot = D * 128;                  // FP16: K [DB][64 rows][128 B] or V [D rows][128 B]
  static constexpr int kQRow = 2 * D + 16;               // a staged row of Q (in the FP16 ring, before it fills)
  static constexpr int sa = R * kSlot;                   // float [4][64]: key scales
  static constexpr int sv = sa + 4 * 64 * 4;             // float [4][64]: value scales
  static constexpr int step = sv + 4 * 64 * 4;           // float [128]
  static constexpr int nv = step + 128 * 4;              // int [4][2]: live keys, NaN value scales
  static constexpr int svm = nv + 32;                    // uint32 [12]: largest value scales of the converting warps
  static constexpr int bar = svm + 48;
  static constexpr int bytes = bar + (2 * R + 16) * 8 + 16;
  static_assert(128 * kQRow <= (R - kPfxConv) * kSlot && 8 * 32 * 36 * 4 <= R * kSlot, "staging fits the ring");
  static_assert(bytes <= 232448, "shared memory of one CTA");
  // tensor memory columns: O, then Q, then the S buffers (64 columns each)
  static constexpr int NS = PV ? 2 : 4;
  static constexpr int tq = PV ? 256 : 0;
  static constexpr int ts = tq + 128;
};

template <int D, bool PV>
__global__ void __launch_bounds__(kPfxThreads, 1) pfx_kernel(const PfxParams p) {
  using L = PfxSmem<D, PV>;
  constexpr int DB = L::DB, VPL = D / 32, NS = L::NS, R = L::R;
  extern __shared__ __align__(1024) uint8_t pfx_sm[];
  uint64_t *bar = reinterpret_cast<uint64_t *>(pfx_sm + L::bar);
  uint64_t *full = bar, *empty = bar + R, *s_full = bar + 2 * R, *s_empty = s_full + 4,
           *sc_full = s_empty + 4, *w_full = sc_full + 4, *o_full = w_full + 2, *q_full = o_full + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(q_full + 1);
  float (*s_a)[64] = reinterpret_cast<float (*)[64]>(pfx_sm + L::sa);
  float (*s_v)[64] = reinterpret_cast<float (*)[64]>(pfx_sm + L::sv);
  float *s_step = reinterpret_cast<float *>(pfx_sm + L::step);
  uint32_t *s_svm = reinterpret_cast<uint32_t *>(pfx_sm + L::svm);
  int (*s_nv)[2] = reinterpret_cast<int (*)[2]>(pfx_sm + L::nv);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, wg = warp >> 2;
  const int split = blockIdx.x, h = blockIdx.y, rt = blockIdx.z;
  const int H = p.q8.H, G = p.q8.G;
  const int j0 = (int)((long long)p.pages * split / p.splits);
  const int n = (int)((long long)p.pages * (split + 1) / p.splits) - j0;
  if ((smem_u32(pfx_sm) & 1023) != 0) {      // the swizzled tiles need it; the segment's alignment gives it
    if (tid == 0) set_error(kErrBadShape);
    return;
  }
  // jobs in the order of the products: K(0), then K(j + 1), V(j), .., V(n - 1)
  const int jobs = PV ? 2 * n : n;
  auto is_k = [&](int t) { return !PV || t == 0 || ((t & 1) && t < 2 * n - 1); };
  auto page_of = [&](int t) { return !PV ? t : t == 2 * n - 1 ? n - 1 : is_k(t) ? (t + 1) >> 1 : (t >> 1) - 1; };
  if (tid == 0) {
    for (int s = 0; s < R; ++s) {
      mbar_init(&full[s], 4);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&s_empty[s], 8);
      mbar_init(&sc_full[s], 4);
    }
    mbar_init(&w_full[0], 8);
    mbar_init(&w_full[1], 8);
    mbar_init(o_full, 1);
    mbar_init(q_full, 8);
    fence_mbarrier_init();
  }
  if (warp == kPfxMma) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // tensor memory is held: a dependent grid that wants it may be launched now
  pdl_launch_dependents();
  const uint32_t tmem = *tmem_slot;
  const long long limit = wait_limit();
  bool ok = true;
  // Q by the warpgroups that do not convert (those fetch their first pages meanwhile): a
  // warp per row, all its rows in flight; row r of the tile is query head h G + r % G of
  // sequence r / G.  Staged as FP16 rows in the ring's last slots, then into tensor
  // memory.
  if (wg < 2 || wg == 2 + kPfxConv) {
    constexpr int NW = 12, NR = (128 + NW - 1) / NW;
    uint8_t *stage = pfx_sm + kPfxConv * L::kSlot;
    const int w = wg < 2 ? warp : warp - 4 * kPfxConv;
    KvRaw<VPL> raw[NR];
    uint32_t m[NR];
#pragma unroll
    for (int u = 0; u < NR; ++u) {
      const int r = w + NW * u, rr = rt * 128 + r;
#pragma unroll
      for (int i = 0; i < VPL / 2; ++i) raw[u].w[i] = 0;
      if (r < 128 && rr < p.rows) {
        const int b = rr / G;
        raw[u] = kv_load<VPL>(p.q8.q + b * p.q8.q_bs + (long long)(h * G + rr - b * G) * p.q8.q_hs + lane * VPL);
      }
    }
    // (no branch between the rows, so that their reductions overlap)
#pragma unroll
    for (int u = 0; u < NR; ++u) {
      m[u] = 0;
#pragma unroll
      for (int i = 0; i < VPL / 2; ++i) m[u] = max(m[u], max(raw[u].w[i] & 0x7FFFu, (raw[u].w[i] >> 16) & 0x7FFFu));
      m[u] = __reduce_max_sync(0xffffffffu, m[u]);
    }
#pragma unroll
    for (int u = 0; u < NR; ++u) {
      const int r = w + NW * u;
      const bool finite = m[u] < 0x7F80u, in = r < 128;
      // times 2^(14 - e) in two exact steps (14 - e is 140 at most); the step undoes it
      const int e = max((int)(m[u] >> 7) - 127, -126), up = min(14 - e, 100), rest = 14 - e - up;
      const float f0 = __int_as_float((127 + up) << 23), f1 = __int_as_float((127 + rest) << 23);
      const float step = __int_as_float((127 - up) << 23) * __int_as_float((127 - rest) << 23);
      uint8_t *dst = stage + r * L::kQRow + 2 * lane * VPL;
#pragma unroll
      for (int i = 0; i < VPL / 2; ++i) {
        const __half2 x = __floats2half2_rn(bf16_bits_to_f32(raw[u].w[i] & 0xFFFFu) * f0 * f1,
                                            bf16_bits_to_f32(raw[u].w[i] >> 16) * f0 * f1);
        if (in) *reinterpret_cast<uint32_t *>(dst + 4 * i) = finite ? *reinterpret_cast<const uint32_t *>(&x) : 0u;
      }
      if (in && lane == 0) s_step[r] = finite ? step : __uint_as_float(0x7FC00000u);
    }
    asm volatile("bar.sync 3, 384;" ::: "memory");
    if (wg < 2) {
#pragma unroll 1
      for (int j = wg; j < DB; j += 2) {             // a warpgroup every other block of 64 dimensions
        uint32_t x[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint4 v = *reinterpret_cast<const uint4 *>(stage + (tid & 127) * L::kQRow + 128 * j + 16 * i);
          x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
        }
        tmem_st32(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + L::tq + 32 * j, x);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);            // Q is in place and its stage is free
    }
  }

  if (wg < 2) {
    // ------------------------------- weights -------------------------------
    const int row = tid & 127, rr = rt * 128 + row;
    const bool live = rr < p.rows;
    const int b = live ? rr / G : 0, hq = h * G + (live ? rr - b * G : 0);
    const float r2 = s_step[row] * p.q8.scale2;      // logit (in units of log2 e) = S (ks r2)
    const uint32_t lane_base = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
    float mx = -INFINITY, m = 0.f, up = 1.f;
    float2 sum = make_float2(0.f, 0.f);
    int shift = 0;
    if constexpr (PV) {
      pdl_wait();                                    // the row maxima, over the prefix and the own keys
      m = q8_reference(*(volatile float *)&p.q8.mfin[(size_t)b * p.q8.Hq + hq], false);
      // value scales times 2^shift: the largest lies in [2^13, 2^14)
      const float sv = *(volatile float *)&p.q8.svfin[h];
      if (sv > 0.f) {
        int e;
        frexpf(sv, &e);                              // vs < 2^e
        shift = min(14 - e, 100);                    // (taken back, FP16's smallest stays normal in FP32)
      }
      up = ldexpf(1.0f, shift);
    }
    for (int j = 0; j < n && ok; ++j) {
      const int sb = j & 3, ss = j % NS;
      const bool got = pfx_wait(&sc_full[sb], (j >> 2) & 1, limit) && pfx_wait(&s_full[ss], (j / NS) & 1, limit);
      // a warp gives up as one: the tensor-memory loads are warp-wide
      if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
      tc_fence_after();
      const int nv = s_nv[sb][0], live_keys = nv - 32 * wg;
      const uint32_t src = lane_base + L::ts + 64 * ss + 32 * wg;
      const float *ks = s_a[sb] + 32 * wg, *vs = s_v[sb] + 32 * wg;
      uint32_t s[32];
      tmem_ld32(src, s);
      tmem_ld_wait32(s);
      if constexpr (!PV) {
        if (nv == 64) mx = fmaxf(mx, pfx_half_max<true>(s, ks, live_keys, r2));
        else mx = fmaxf(mx, pfx_half_max<false>(s, ks, live_keys, r2));
      } else {
        const bool whole = nv == 64 && s_nv[sb][1] == 0;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t w[8];
          if (whole)
            sum = mat_add2(sum, pfx_weights16<true>(s + 16 * c, ks + 16 * c, vs + 16 * c, 16, r2, m, p.q8.haze2, up, p.nzero, w));
          else
            sum = mat_add2(sum, pfx_weights16<false>(s + 16 * c, ks + 16 * c, vs + 16 * c, live_keys - 16 * c, r2, m, p.q8.haze2, up, p.nzero, w));
          tmem_st8(src + 8 * c, w);                  // over this thread's S
        }
        tmem_st_wait();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&s_empty[sb]);
        if constexpr (PV) mbar_arrive(&w_full[ss]);
      }
    }
    if constexpr (!PV) {
      // the two warpgroups' halves of the row (every thread has read its step: all S are done)
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (wg == 1) s_step[row] = mx;
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (wg == 0 && live) p.pmax[((size_t)split * H + h) * p.rows + rr] = fmaxf(mx, s_step[row]);
    } else {
      if (!__all_sync(0xffffffffu, ok && pfx_wait(o_full, 0, limit))) ok = false;
      tc_fence_after();
      const float back = ldexpf(1.0f, -shift);
      const size_t at = ((size_t)split * H + h) * p.rows;
      // the two warpgroups' sums of the row (every thread has read its step by now:
      // the last weights were waited for)
      if (wg == 1) s_step[row] = sum.x + sum.y;
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (wg == 0 && live) p.pl[at + rr] = sum.x + sum.y + s_step[row];
      // each warpgroup half of the columns, 32 x 32 blocks through shared memory (the
      // ring, free now): whole 128-byte lines out
      float (*st)[36] = reinterpret_cast<float (*)[36]>(pfx_sm + warp * 32 * 36 * 4);
      const int sub = lane >> 3, c4 = (lane & 7) * 4, first = rt * 128 + 32 * (warp & 3) + sub;
      const int rows = ok ? p.rows - first : 0;      // of this lane's rows first + 4 i: those below
      float *out = p.po + (at + first) * D + c4;
#pragma unroll 1
      for (int cc = 0; cc < D / 64; ++cc) {
        const int col = wg * (D / 2) + 32 * cc;
        uint32_t o[32];
        tmem_ld32(lane_base + col, o);
        tmem_ld_wait32(o);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 32; i += 4)
          *reinterpret_cast<float4 *>(&st[lane][i]) =
              make_float4(__uint_as_float(o[i]) * back, __uint_as_float(o[i + 1]) * back,
                          __uint_as_float(o[i + 2]) * back, __uint_as_float(o[i + 3]) * back);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (4 * i < rows)
            *reinterpret_cast<float4 *>(out + 4 * i * D + col) =
                *reinterpret_cast<const float4 *>(&st[4 * i + sub][c4]);
        }
      }
    }
    tc_fence_before();
  } else if (wg < 2 + kPfxConv) {
    // --------------------------- codes to FP16 tiles ---------------------------
    const int kt = tid & 127;
    constexpr int NL = D / 32;                       // 16-byte pieces per thread and page
    // FP16 pieces 2 c and 2 c + 1 of a tile's row, c = kt mod 4: eight lanes (two rows)
    // meet the eight 16-byte columns.  K: piece x is in row kt / 4 + 32 (x mod 2) of the
    // 64-dimension block x / 2; V: in row kt / 4 + 32 x; the same place of the tile.
    const int rw = kt >> 2;
    const uint32_t c0 = rw * 128 + ((((kt & 3) * 2) ^ (rw & 7)) << 4);
    const uint32_t c1 = rw * 128 + ((((kt & 3) * 2 + 1) ^ (rw & 7)) << 4);
    uint32_t svm = 0;
    // a job's codes (and a K page's scales) into registers; page ids one job ahead
    uint4 r[NL];
    uint32_t ks = 0, vs = 0;
    int nv = 0, ahead = 0;
    auto page_id = [&](int t) { return t < jobs ? p.ptable[j0 + page_of(t)] : 0; };
    auto fetch = [&](int t) {
      const bool k = is_k(t);
      int page = ahead;
      ahead = page_id(t + kPfxConv);
      nv = min(64, p.prefix - 64 * (j0 + page_of(t)));
      if (page < 0 || page >= p.q8.n_pages) {        // its keys weigh nothing
        set_index_error();
        page = nv = 0;
      }
      const size_t ph = (size_t)page * H + h;
      if (k) {
        const int8_t *src = p.q8.k + ph * 64 * D + rw * D + (kt & 3) * 16;
#pragma unroll
        for (int x = 0; x < NL; ++x) r[x] = q8_ldg(src + (x & 1) * 32 * D + (x >> 1) * 64);
        ks = p.q8.ks[ph * 64 + (kt & 63)];
        vs = p.q8.vs[ph * 64 + (kt & 63)];
      } else {
        const int8_t *src = p.q8.v + ph * 64 * D + kt * 16;
#pragma unroll
        for (int x = 0; x < NL; ++x) r[x] = q8_ldg(src + x * 2048);
      }
    };
    int t = wg - 2;
    ahead = page_id(t);
    if (t < jobs) fetch(t);
    for (; t < jobs && ok; t += kPfxConv) {
      const int slot = t % R, j = page_of(t), sb = j & 3;
      const bool k = is_k(t);
      bool got = true;
      if (t >= R) got = pfx_wait(&empty[slot], ((t / R) - 1) & 1, limit);
      else if (t >= kPfxConv) got = pfx_wait(q_full, 0, limit);   // the ring's last slots staged Q
      // the weights of page j - 4 are done with this slot of scales
      if (k && j >= 4) got = got && pfx_wait(&s_empty[sb], ((j >> 2) - 1) & 1, limit);
      if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
      uint8_t *dst = pfx_sm + slot * L::kSlot;
#pragma unroll
      for (int x = 0; x < NL; ++x) {
        uint4 lo, hi;
        pfx_f16(r[x], p.magic, lo, hi);
        *reinterpret_cast<uint4 *>(dst + c0 + x * 32 * 128) = lo;
        *reinterpret_cast<uint4 *>(dst + c1 + x * 32 * 128) = hi;
      }
      if (k) {
        if ((kt & 63) < nv && vs < 0x7F80u) svm = max(svm, vs);
        const bool nan = __any_sync(0xffffffffu, vs >= 0x7F80u);
        if (kt < 64) {
          s_a[sb][kt] = bf16_bits_to_f32(ks);
          s_v[sb][kt] = bf16_bits_to_f32(vs);
        }
        if (kt == 0) s_nv[sb][0] = nv;
        if (kt == 0 || kt == 32) reinterpret_cast<uint16_t *>(&s_nv[sb][1])[kt >> 5] = nan;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&full[slot]);
        if (k) mbar_arrive(&sc_full[sb]);
      }
      // behind the fence, which would wait for these loads as well
      if (t + kPfxConv < jobs) fetch(t + kPfxConv);
    }
    if constexpr (!PV) {
      // over the converting warpgroups
      __syncwarp();
      svm = __reduce_max_sync(0xffffffffu, svm);
      if (lane == 0) s_svm[warp - 8] = svm;
      asm volatile("bar.sync 2, %0;" ::"n"(kPfxConv * 128) : "memory");
      if (tid == 256 && rt == 0) {
        for (int i = 1; i < 4 * kPfxConv; ++i) svm = max(svm, s_svm[i]);
        p.psv[(size_t)split * H + h] = bf16_bits_to_f32(svm);
      }
    }
  } else {
    if (warp == kPfxMma) {
      // ------------------------------- MMA issuer -------------------------------
      constexpr uint32_t id_s = umma_idesc_f16(128, 64), id_o = umma_idesc_f16(128, D);
      const uint32_t lead = elect_one();
      const uint64_t desc = umma_desc_sw128(smem_u32(pfx_sm));   // addresses below 256 KB: sums do not carry
      int t = 0, slot = 0, par = 0;                  // the ring's jobs, in the loaders' order
      auto next = [&] {
        ++t;
        if (++slot == R) { slot = 0; par ^= 1; }
      };
      auto qk = [&](int j) {
        const int ss = j % NS;
        bool got = pfx_wait(&full[slot], par, limit);
        if (!PV && j >= NS) got = got && pfx_wait(&s_empty[ss], ((j / NS) - 1) & 1, limit);
        // S j - 2 holds the weights of w V j - 2: that product has to be done
        if (PV && j >= 2) {
          const int tv = 2 * (j - 1);                // its V's job
          got = got && pfx_wait(&empty[tv % R], (tv / R) & 1, limit);
        }
        if (!__all_sync(0xffffffffu, got)) return false;
        tc_fence_after();
        const uint32_t acc = tmem + L::ts + 64 * ss;
        const uint64_t kb = desc + (uint64_t)(slot * (L::kSlot >> 4));
#pragma unroll
        for (int i = 0; i < DB; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma_f16_ta(lead, acc, tmem + L::tq + 32 * i + 8 * k, kb + (uint64_t)(i * 512 + 2 * k),
                          id_s, i > 0 || k > 0);
        tc_commit_lead(lead, &empty[slot]);
        tc_commit_lead(lead, &s_full[ss]);
        next();
        return true;
      };
      auto wv = [&](int j) {
        const int ss = j % NS;
        const bool got = pfx_wait(&w_full[ss], (j / NS) & 1, limit) && pfx_wait(&full[slot], par, limit);
        if (!__all_sync(0xffffffffu, got)) return false;
        tc_fence_after();
        const uint64_t vb = desc + (uint64_t)(slot * (L::kSlot >> 4));
#pragma unroll
        for (int k = 0; k < 4; ++k)                  // keys 0-31 lie over S columns 0 .., keys 32-63 over 32 ..
          tc_mma_f16_ta(lead, tmem, tmem + L::ts + 64 * ss + 8 * k + (k < 2 ? 0 : 16), vb + (uint64_t)(2 * k), id_o,
                        j > 0 || k > 0);
        tc_commit_lead(lead, &empty[slot]);
        next();
        return true;
      };
      ok = __all_sync(0xffffffffu, pfx_wait(q_full, 0, limit));
      tc_fence_after();
      ok = ok && qk(0);
      for (int j = 0; j < n && ok; ++j) {
        if (j + 1 < n) ok = qk(j + 1);
        if constexpr (PV) ok = ok && wv(j);
      }
      if (PV || !ok) tc_commit_lead(lead, o_full);
      if (!ok) pfx_wait(o_full, 0, limit);           // nothing is in flight when the memory goes
    }
  }
  // what follows waits for this grid only: it ends after the one before it
  if constexpr (!PV) pdl_wait();
  tc_fence_before();
  __syncthreads();
  if (warp == kPfxMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

namespace {
struct PfxLayout {
  Q8Layout q8;
  size_t pmax, psv, mfin, svfin, po, pl, total;
  int pages, splits, rows, row_tiles;
};
PfxLayout pfx_layout(const Q8Shape &s) {
  PfxLayout y{};
  y.q8 = q8_layout(s);
  y.pages = (s.prefix + 63) / 64;
  y.rows = s.B * (s.Hq / s.Hkv);
  y.row_tiles = (y.rows + 127) / 128;
  // one CTA per SM: the splits that fill one round of the SMs
  y.splits = std::max(1, std::min(y.pages, kQ8Sms / (y.row_tiles * s.Hkv)));
  size_t at = y.q8.total;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += (bytes + 255) & ~(size_t)255;
    return o;
  };
  y.pmax = take((size_t)y.splits * s.Hkv * y.rows * 4);
  y.psv = take((size_t)y.splits * s.Hkv * 4);
  y.mfin = take((size_t)s.B * s.Hq * 4);
  y.svfin = take((size_t)s.Hkv * 4);
  y.po = take((size_t)y.splits * s.Hkv * y.rows * s.D * 4);
  y.pl = take((size_t)y.splits * s.Hkv * y.rows * 4);
  y.total = at;
  return y;
}

template <int D, int NT>
cudaError_t pfx_run(const PfxParams &p, const PfxLayout &y, cudaStream_t st, Launcher &L) {
  // The first launch waits for the stream; the later ones are programmatic dependents.
  // Each waits for its predecessor before it ends, so that one wait covers all before.
  const dim3 block(kQ8Threads), grid((unsigned)std::min<long long>(y.q8.items, p.q8.target));
  const dim3 pg((unsigned)y.splits, (unsigned)p.q8.H, (unsigned)y.row_tiles);
  const bool once = p.q8.single;
  cudaError_t e = cudaSuccess;
  if (!once)
    e = L.launch("q8_logits", q8_logits_kernel<D, NT>, grid, block, (size_t)(p.q8.B + 1) * 4, st,
                 false, p.q8);
  if (e != cudaSuccess) return e;
  e = L.launch("pfx_max", pfx_kernel<D, false>, pg, dim3(kPfxThreads), PfxSmem<D, false>::bytes, st,
               !once, p);
  if (e != cudaSuccess) return e;
  e = once ? q8_run_short<D, NT>(p.q8, st, L)
           : L.launch("q8_pv", q8_pv_kernel<D, NT>, grid, block, q8_pv_smem(NT, p.q8.B), st, true, p.q8);
  if (e != cudaSuccess) return e;
  e = L.launch("pfx_pv", pfx_kernel<D, true>, pg, dim3(kPfxThreads), PfxSmem<D, true>::bytes, st,
               true, p);
  if (e != cudaSuccess) return e;
  return q8_run_merge<D>(p.q8, 4 * NT, st, L);
}
}  // namespace

size_t pfx_workspace_bytes(const Q8Shape &s) { return q8_joins(s) ? q8_workspace_bytes(s) : pfx_layout(s).total; }

cudaError_t prepare_prefix_kernels() {
  cudaError_t e = cudaSuccess;
  auto set = [&](const void *k, int bytes) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  };
  set((const void *)pfx_kernel<64, false>, PfxSmem<64, false>::bytes);
  set((const void *)pfx_kernel<64, true>, PfxSmem<64, true>::bytes);
  set((const void *)pfx_kernel<128, false>, PfxSmem<128, false>::bytes);
  set((const void *)pfx_kernel<128, true>, PfxSmem<128, true>::bytes);
  set((const void *)pfx_kernel<256, false>, PfxSmem<256, false>::bytes);
  set((const void *)pfx_kernel<256, true>, PfxSmem<256, true>::bytes);
  return e;
}

cudaError_t launch_prefix_attention(const Q8Args &a, cudaStream_t st, Launcher &L) {
  if (q8_joins(a.s)) return launch_q8_attention(a, st, L);
  const PfxLayout y = pfx_layout(a.s);
  char *ws = static_cast<char *>(a.workspace);
  PfxParams p{};
  p.q8 = q8_params(a, y.q8);
  p.ptable = a.ptable;
  p.magic = 0x64646464u;
  p.nzero = -0.0f;
  p.prefix = a.s.prefix; p.pages = y.pages; p.splits = y.splits; p.rows = y.rows;
  p.pmax = reinterpret_cast<float *>(ws + y.pmax);
  p.psv = reinterpret_cast<float *>(ws + y.psv);
  p.po = reinterpret_cast<float *>(ws + y.po);
  p.pl = reinterpret_cast<float *>(ws + y.pl);
  p.q8.pmax = p.pmax; p.q8.psv = p.psv; p.q8.po = p.po; p.q8.pl = p.pl;
  p.q8.mfin = reinterpret_cast<float *>(ws + y.mfin);
  p.q8.svfin = reinterpret_cast<float *>(ws + y.svfin);
  p.q8.splits = y.splits; p.q8.rows = y.rows;
  p.q8.single = q8_is_short(a.s);
  const int NT = q8_tiles(p.q8.G);
#define PFX_CASE(D_, N_) \
  if (a.s.D == D_ && NT == N_) return pfx_run<D_, N_>(p, y, st, L);
  PFX_CASE(64, 1) PFX_CASE(64, 2) PFX_CASE(64, 4)
  PFX_CASE(128, 1) PFX_CASE(128, 2) PFX_CASE(128, 4)
  PFX_CASE(256, 1) PFX_CASE(256, 2) PFX_CASE(256, 4)
#undef PFX_CASE
  return cudaErrorInvalidValue;
}

}  // namespace dvssq
