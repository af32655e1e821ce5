// KV-BSS decode attention of a batch over a prefix that all its sequences share
// (dvssq_bss_attention_prefix), on the 5th-generation tensor cores.  The
// B G queries of a KV head are the rows of one matrix, so the prefix is a pair
// of dense products instead of B walks over it:
//   S = Q K^T,   w = exp(S - m) vs (zero below the haze threshold),   O = w V
// The haze threshold needs each row's final maximum first, so Q K^T runs twice:
//   pfx_max   S and its row maxima (an atomic maximum: any order, one result),
//             and the largest value scale of each KV head
//   pfx_pv    S again (K comes from L2 now), the weights, and a split's O
// Each sequence's own keys go through q8_logits and q8_pv as without a prefix,
// and q8_merge adds the items' and the splits' partials in order.
//
// A CTA holds 128 rows of Q and walks a split of the prefix in steps of two
// pages (128 keys).  Warps 0-7 turn S into weights (a warpgroup per page of the
// step, a thread per row), warps 8-11 bring K and warps 12-15 V from global
// memory through registers, where the 8-bit codes become FP16, into
// 128-byte-swizzled shared memory, and one thread issues the MMAs.  S is
// double-buffered in tensor memory; Q K^T of step i + 1 is issued before w V of
// step i, so that the weights of a step are formed behind the next product.
//
// Number formats: a code is exact in FP16 (1024 + u from a byte permutation,
// minus 1152), and so is a query scaled by a power of two to 2^14 .. 2^15 (BF16
// has 8 significant bits; values 2^29 below the row's largest vanish), so S is
// FP32-grade.  A weight is rounded once to FP16 (2^-12 relative), scaled by
// 2^(14 - e) with 2^e at or above the head's largest vs: the rounding holds
// down to e^-19 of the largest weight, and what underflows is below 2^-38 of it.
#include "common.cuh"
#include "kernels.h"

namespace dvssq {

constexpr int kPfxThreads = 17 * 32;
constexpr int kPfxSoft = 256;            // threads of the weight warps
constexpr float kLog2e = 1.44269504088896341f;

struct PfxParams {
  Q8Params q8;
  const int32_t *ptable;
  int prefix, pages, steps, splits, rows;   // rows = B G per KV head
  uint32_t *mrow;                // [B][Hq] row maxima, order-preserving bits
  uint32_t *svmax;               // [H] largest finite value scale (bits)
  float *po;                     // [splits][H][rows][D]
  float *pl;                     // [splits][H][rows]
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

// 16 codes -> 16 FP16 values in order, as two 16-byte chunks
__device__ __forceinline__ void pfx_f16(const uint4 &c, uint4 &lo, uint4 &hi) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t o[8];
  const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u = w[i] ^ 0x80808080u;
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<__half2 *>(&a), bias);
    const __half2 y = __hsub2(*reinterpret_cast<__half2 *>(&b), bias);
    o[2 * i] = *reinterpret_cast<const uint32_t *>(&x);
    o[2 * i + 1] = *reinterpret_cast<const uint32_t *>(&y);
  }
  lo = make_uint4(o[0], o[1], o[2], o[3]);
  hi = make_uint4(o[4], o[5], o[6], o[7]);
}

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int D, bool PV>
struct PfxSmem {
  static constexpr int DB = D / 64;
  static constexpr int NK = !PV || D < 256 ? 2 : 1;      // K slots (128 keys each)
  static constexpr int kTile = 128 * 128;                // 128 rows of 128 bytes
  static constexpr int kV = D * 128;                     // one page of V
  static constexpr int q = 0;
  static constexpr int k = q + DB * kTile;
  static constexpr int v = k + NK * DB * kTile;
  static constexpr int w = v + (PV ? 2 * kV : 0);
  static constexpr int sc = w + (PV ? 2 * kTile : 0);    // float2 [2][128]: key and value scales
  static constexpr int step = sc + 2 * 128 * 8;          // float [128]
  static constexpr int nv = step + 128 * 4;              // int [2][2]: live keys of each page
  static constexpr int bar = nv + 16;
  static constexpr int bytes = bar + 20 * 8 + 16;
};

template <int D, bool PV>
__global__ void __launch_bounds__(kPfxThreads, 1) pfx_kernel(const PfxParams p) {
  using L = PfxSmem<D, PV>;
  constexpr int DB = L::DB, NK = L::NK;
  extern __shared__ __align__(1024) uint8_t pfx_sm[];
  uint64_t *bar = reinterpret_cast<uint64_t *>(pfx_sm + L::bar);
  uint64_t *k_full = bar, *k_empty = bar + 2, *s_full = bar + 4, *s_empty = bar + 6,
           *sc_full = bar + 8, *v_full = bar + 10, *v_empty = bar + 12, *w_full = bar + 14,
           *w_empty = bar + 15, *o_full = bar + 16;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bar + 20);
  float2 (*sc)[128] = reinterpret_cast<float2 (*)[128]>(pfx_sm + L::sc);
  float *s_step = reinterpret_cast<float *>(pfx_sm + L::step);
  int (*s_nv)[2] = reinterpret_cast<int (*)[2]>(pfx_sm + L::nv);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int split = blockIdx.x, h = blockIdx.y, rt = blockIdx.z;
  const int H = p.q8.H, G = p.q8.G;
  const int i0 = (int)((long long)p.steps * split / p.splits);
  const int n = (int)((long long)p.steps * (split + 1) / p.splits) - i0;
  if ((smem_u32(pfx_sm) & 1023) != 0) {      // the swizzled tiles need it; the segment's alignment gives it
    if (tid == 0) set_error(kErrBadShape);
    return;
  }
  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&k_full[s], 4);
      mbar_init(&k_empty[s], 1);
      mbar_init(&s_full[s], 1);
      mbar_init(&s_empty[s], 8);
      mbar_init(&sc_full[s], 4);
      mbar_init(&v_full[s], 4);
      mbar_init(&v_empty[s], 1);
    }
    mbar_init(w_full, 8);
    mbar_init(w_empty, 1);
    mbar_init(o_full, 1);
    fence_mbarrier_init();
  }
  if (warp == 16) {
    tmem_alloc(tmem_slot, PV ? 512 : 256);
    tmem_relinquish();
  }
  // Q: a warp per row; row r of the tile is query head h G + r % G of sequence r / G
  for (int r = warp; r < 128; r += 17) {
    constexpr int VPL = D / 32;
    const int rr = rt * 128 + r;
    uint32_t bits[VPL], m = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) bits[i] = 0;
    if (rr < p.rows) {
      const int b = rr / G;
      const uint16_t *src = p.q8.q + b * p.q8.q_bs + (long long)(h * G + rr - b * G) * p.q8.q_hs + lane * VPL;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        bits[i] = src[i];
        m = max(m, bits[i] & 0x7FFFu);
      }
    }
    m = __reduce_max_sync(0xffffffffu, m);
    const int e = max((int)(m >> 7) - 127, -126);
    uint16_t f[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      f[i] = m >= 0x7F80u ? 0 : __half_as_ushort(__float2half_rn(ldexpf(bf16_bits_to_f32(bits[i]), 14 - e)));
    const int dim = lane * VPL, kb = dim >> 6, c = (dim & 63) >> 3;
    uint16_t *dst = reinterpret_cast<uint16_t *>(pfx_sm + L::q + kb * L::kTile + r * 128 + ((c ^ (r & 7)) << 4)) + (dim & 7);
#pragma unroll
    for (int i = 0; i < VPL; i += 2)
      *reinterpret_cast<uint32_t *>(dst + i) = f[i] | (uint32_t)f[i + 1] << 16;
    if (lane == 0) s_step[r] = m >= 0x7F80u ? __uint_as_float(0x7FC00000u) : ldexpf(1.0f, e - 14);
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // tensor memory is held: a dependent grid that wants it may be launched now
  pdl_launch_dependents();
  const uint32_t tmem = *tmem_slot;
  bool ok = true;

  if (warp < 8) {
    // ------------------------------- weights -------------------------------
    const int quarter = warp & 3, half = warp >> 2, row = 32 * quarter + lane, rr = rt * 128 + row;
    const bool live = rr < p.rows;
    const int b = live ? rr / G : 0, hq = h * G + (live ? rr - b * G : 0);
    const float r1 = s_step[row] * p.q8.scale;       // logit = S ks r1
    const uint32_t lane_base = tmem + ((uint32_t)(32 * quarter) << 16);
    float mx = -INFINITY, sum = 0.f, x0 = 0.f, floor2 = -INFINITY;
    int shift = 0;
    if constexpr (PV) {
      pdl_wait();                                    // the row maxima, of the prefix and of the items
      float m = from_order_bits(*(volatile uint32_t *)&p.mrow[(size_t)b * p.q8.Hq + hq]);
      const int gp = 4 * q8_tiles(G);
      for (int t = p.q8.off[b]; t < p.q8.off[b + 1]; ++t)
        m = fmaxf(m, p.q8.cmax[((long long)t * H + h) * gp + hq - h * G]);
      // weights times 2^shift: the largest vs 2^shift lies in (2^13, 2^14]
      const uint32_t sv = p.svmax[h];
      if (sv != 0) {
        int e;
        frexpf(__uint_as_float(sv), &e);             // vs < 2^e
        shift = 14 - e;
      }
      if (m > -INFINITY) {
        x0 = (float)shift - m * kLog2e;              // exponent of a weight: S ks r1 log2e + x0
        if (p.q8.haze > 0.f) floor2 = (float)shift - p.q8.haze * kLog2e;
      }
    }
    const float r2 = r1 * kLog2e;
    for (int i = 0; i < n && ok; ++i) {
      const int sb = i & 1, par = (i >> 1) & 1;
      bool got = mbar_wait(&sc_full[sb], par) && mbar_wait(&s_full[sb], par);
      if constexpr (PV)
        if (i > 0) got = got && mbar_wait(w_empty, (i - 1) & 1);
      // a warp gives up as one: the tensor-memory loads are warp-wide
      if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
      tc_fence_after();
      const int nv = s_nv[sb][half];
      const float2 *scale = sc[sb] + 64 * half;
      const uint32_t src = lane_base + (PV ? 256 : 0) + 128 * sb + 64 * half;
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        uint32_t s[32];
        tmem_ld32(src + 32 * cc, s);
        tmem_ld_wait();
        if constexpr (!PV) {
          float f[32];
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float4 a = *reinterpret_cast<const float4 *>(&scale[32 * cc + j]);
            f[j] = __uint_as_float(s[j]) * a.x;
            f[j + 1] = __uint_as_float(s[j + 1]) * a.z;
          }
          if (nv == 64) {
#pragma unroll
            for (int j = 0; j < 32; ++j) mx = fmaxf(mx, f[j]);
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (32 * cc + j < nv) mx = fmaxf(mx, f[j]);
          }
        } else {
          uint32_t w[16];
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float4 a = *reinterpret_cast<const float4 *>(&scale[32 * cc + j]);
            const float x = fmaf(__uint_as_float(s[j]) * a.x, r2, x0);
            const float y = fmaf(__uint_as_float(s[j + 1]) * a.z, r2, x0);
            // a NaN logit is kept; a dropped key's value scale is not looked at
            const bool kx = !(x < floor2) && (nv == 64 || 32 * cc + j < nv);
            const bool ky = !(y < floor2) && (nv == 64 || 32 * cc + j + 1 < nv);
            const float ex = kx ? ex2_approx(x) : 0.f, ey = ky ? ex2_approx(y) : 0.f;
            sum += ex;
            sum += ey;
            const __half2 o = __floats2half2_rn(kx ? ex * a.y : 0.f, ky ? ey * a.w : 0.f);
            w[j / 2] = *reinterpret_cast<const uint32_t *>(&o);
          }
          uint8_t *dst = pfx_sm + L::w + half * L::kTile + row * 128;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint4 *>(dst + (((4 * cc + j) ^ (row & 7)) << 4)) =
                make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
        }
      }
      if constexpr (PV) fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&s_empty[sb]);
        if constexpr (PV) mbar_arrive(w_full);
      }
    }
    if constexpr (!PV) {
      pdl_wait();                                    // the row maxima were cleared by q8_logits
      const float m = mx * r1;
      if (live && m == m) atomicMax(&p.mrow[(size_t)b * p.q8.Hq + hq], order_bits(m));
    } else {
      if (ok && !mbar_wait(o_full, 0)) ok = false;
      tc_fence_after();
      const float back = ldexpf(1.0f, -shift);
      const size_t at = ((size_t)split * H + h) * p.rows + rr;
#pragma unroll 1
      for (int cc = 0; cc < D / 64; ++cc) {
        uint32_t o[32];
        const int col = half * (D / 2) + 32 * cc;
        tmem_ld32(lane_base + col, o);
        tmem_ld_wait();
        if (live && ok) {
#pragma unroll
          for (int j = 0; j < 32; j += 4)
            *reinterpret_cast<float4 *>(p.po + at * D + col + j) =
                make_float4(__uint_as_float(o[j]) * back, __uint_as_float(o[j + 1]) * back,
                            __uint_as_float(o[j + 2]) * back, __uint_as_float(o[j + 3]) * back);
        }
      }
      tc_fence_before();
      // the two halves' sums of the row
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (half == 1) s_step[row] = sum;
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (half == 0 && live) p.pl[at] = (sum + s_step[row]) * back;
    }
  } else if (warp < 12) {
    // -------------------------------- K and scales --------------------------------
    const int kt = tid - 256;
    constexpr int NL = D / 16;                       // 16-byte loads per thread and step
    uint32_t sv = 0;
    int page[2], nv[2];
    uint4 r[NL];
    uint16_t ks, vs;
    auto fetch = [&](int i) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int w = 2 * (i0 + i) + x;
        page[x] = w < p.pages ? p.ptable[w] : 0;
        nv[x] = w < p.pages ? min(64, p.prefix - 64 * w) : 0;
        if (page[x] < 0 || page[x] >= p.q8.n_pages) {
          set_error(kErrBadIndex);
          page[x] = nv[x] = 0;
        }
      }
#pragma unroll
      for (int x = 0; x < NL; ++x) {
        const size_t ph = (size_t)page[x >= NL / 2] * H + h;
        r[x] = q8_ldg(p.q8.k + ph * 64 * D + (size_t)(kt + 128 * (x % (NL / 2))) * 16);
      }
      const size_t ph = (size_t)page[kt >> 6] * H + h;
      ks = p.q8.ks[ph * 64 + (kt & 63)];
      vs = p.q8.vs[ph * 64 + (kt & 63)];
    };
    if (n > 0) fetch(0);
    for (int i = 0; i < n && ok; ++i) {
      const int slot = i % NK, sb = i & 1;
      if (i >= NK && !mbar_wait(&k_empty[slot], ((i / NK) - 1) & 1)) { ok = false; break; }
      uint8_t *dst = pfx_sm + L::k + slot * DB * L::kTile;
#pragma unroll
      for (int x = 0; x < NL; ++x) {
        const int at = kt + 128 * (x % (NL / 2)), rw = at / NL + (x >= NL / 2 ? 64 : 0), ch = at % NL;
        uint4 lo, hi;
        pfx_f16(r[x], lo, hi);
        // chunks 2 c and 2 c + 1 of row rw; lanes 4-7 store the odd one first, so that
        // eight lanes meet the eight chunk columns
        const int c = (ch & 3) * 2, odd = (ch >> 2) & 1;
        uint8_t *base = dst + (ch >> 2) * L::kTile + rw * 128;
        *reinterpret_cast<uint4 *>(base + (((c + odd) ^ (rw & 7)) << 4)) = odd ? hi : lo;
        *reinterpret_cast<uint4 *>(base + (((c + 1 - odd) ^ (rw & 7)) << 4)) = odd ? lo : hi;
      }
      // the weights of step i - 2 are done with this slot of scales
      if (i >= 2 && !mbar_wait(&s_empty[sb], ((i >> 1) - 1) & 1)) { ok = false; break; }
      const bool alive = (kt & 63) < nv[kt >> 6];
      sc[sb][kt] = make_float2(bf16_bits_to_f32(ks), bf16_bits_to_f32(vs));
      if (alive && vs < 0x7F80u) sv = max(sv, (uint32_t)vs);
      if ((kt & 63) == 0) s_nv[sb][kt >> 6] = nv[kt >> 6];
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&k_full[slot]);
        mbar_arrive(&sc_full[sb]);
      }
      if (i + 1 < n) fetch(i + 1);
    }
    if constexpr (!PV) {
      pdl_wait();                                    // svmax was cleared by q8_logits
      sv = __reduce_max_sync(0xffffffffu, sv);
      if (lane == 0 && sv != 0) atomicMax(&p.svmax[h], sv << 16);
    }
  } else if (warp < 16) {
    // ------------------------------------ V ------------------------------------
    if constexpr (PV) {
      const int vt = tid - 384;
      constexpr int NL = D / 32;
      uint4 r[NL];
      auto fetch = [&](int j) {                      // j = 2 (step) + page of the step
        const int w = 2 * i0 + j;
        int page = w < p.pages ? p.ptable[w] : 0;
        if (page < 0 || page >= p.q8.n_pages) page = 0;
        const int8_t *src = p.q8.v + ((size_t)page * H + h) * 64 * D + vt * 16;
#pragma unroll
        for (int x = 0; x < NL; ++x) r[x] = q8_ldg(src + x * 2048);
      };
      if (n > 0) fetch(0);
      for (int j = 0; j < 2 * n && ok; ++j) {
        const int slot = j & 1;
        if (j >= 2 && !mbar_wait(&v_empty[slot], ((j >> 1) - 1) & 1)) { ok = false; break; }
        uint8_t *dst = pfx_sm + L::v + slot * L::kV;
#pragma unroll
        for (int x = 0; x < NL; ++x) {
          const int at = vt + 128 * x, rw = at >> 2, c = (at & 3) * 2;
          uint4 lo, hi;
          pfx_f16(r[x], lo, hi);
          *reinterpret_cast<uint4 *>(dst + rw * 128 + ((c ^ (rw & 7)) << 4)) = lo;
          *reinterpret_cast<uint4 *>(dst + rw * 128 + (((c + 1) ^ (rw & 7)) << 4)) = hi;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_full[slot]);
        if (j + 1 < 2 * n) fetch(j + 1);
      }
    }
  } else if (lane == 0) {
    // ------------------------------- MMA issuer -------------------------------
    constexpr uint32_t id_s = umma_idesc_f16(128, 128), id_o = umma_idesc_f16(128, D);
    const uint32_t q0 = smem_u32(pfx_sm + L::q), k0 = smem_u32(pfx_sm + L::k);
    const uint32_t v0 = smem_u32(pfx_sm + L::v), w0 = smem_u32(pfx_sm + L::w);
    auto weights_v = [&](int i) {
      if (!mbar_wait(w_full, i & 1)) return false;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (!mbar_wait(&v_full[x], i & 1)) return false;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < 4; ++k)
          tc_mma_f16(tmem, umma_desc_sw128(w0 + x * L::kTile + 32 * k),
                     umma_desc_sw128(v0 + x * L::kV + 32 * k), id_o, i > 0 || x > 0 || k > 0);
        tc_commit(&v_empty[x]);
      }
      tc_commit(w_empty);
      return true;
    };
    for (int i = 0; i < n && ok; ++i) {
      const int slot = i % NK, sb = i & 1;
      if (!mbar_wait(&k_full[slot], (i / NK) & 1)) { ok = false; break; }
      if (i >= 2 && !mbar_wait(&s_empty[sb], ((i >> 1) - 1) & 1)) { ok = false; break; }
      tc_fence_after();
      const uint32_t acc = tmem + (PV ? 256 : 0) + 128 * sb, kb = k0 + slot * DB * L::kTile;
#pragma unroll
      for (int j = 0; j < DB; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          tc_mma_f16(acc, umma_desc_sw128(q0 + j * L::kTile + 32 * k),
                     umma_desc_sw128(kb + j * L::kTile + 32 * k), id_s, j > 0 || k > 0);
      tc_commit(&k_empty[slot]);
      tc_commit(&s_full[sb]);
      if constexpr (PV)
        if (i > 0 && !weights_v(i - 1)) { ok = false; break; }
    }
    if constexpr (PV) {
      if (ok && n > 0) ok = weights_v(n - 1);
      tc_commit(o_full);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 16) {
    tc_fence_after();
    tmem_dealloc(tmem, PV ? 512 : 256);
  }
}

namespace {
struct PfxLayout {
  Q8Layout q8;
  size_t mrow, svmax, po, pl, total;
  int pages, steps, splits, rows, row_tiles;
};
PfxLayout pfx_layout(const Q8Shape &s) {
  PfxLayout y{};
  y.q8 = q8_layout(s);
  y.pages = (s.prefix + 63) / 64;
  y.steps = (y.pages + 1) / 2;
  y.rows = s.B * (s.Hq / s.Hkv);
  y.row_tiles = (y.rows + 127) / 128;
  // one CTA per SM: the splits that fill one round of the SMs
  y.splits = std::max(1, std::min(y.steps, kQ8Sms / (y.row_tiles * s.Hkv)));
  size_t at = y.q8.total;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += (bytes + 255) & ~(size_t)255;
    return o;
  };
  y.mrow = take((size_t)s.B * s.Hq * 4);
  y.svmax = take((size_t)s.Hkv * 4);
  y.po = take((size_t)y.splits * s.Hkv * y.rows * s.D * 4);
  y.pl = take((size_t)y.splits * s.Hkv * y.rows * 4);
  y.total = at;
  return y;
}

template <int D, int NT>
cudaError_t pfx_run(const PfxParams &p, const PfxLayout &y, cudaStream_t st, Launcher &L) {
  const dim3 block(kQ8Threads), grid((unsigned)std::min<long long>(y.q8.items, p.q8.target));
  const dim3 pg((unsigned)y.splits, (unsigned)p.q8.H, (unsigned)y.row_tiles);
  cudaError_t e = L.launch("q8_logits", q8_logits_kernel<D, NT>, grid, block,
                           (size_t)(p.q8.B + 1) * 4, st, false, p.q8);
  if (e != cudaSuccess) return e;
  e = L.launch("pfx_max", pfx_kernel<D, false>, pg, dim3(kPfxThreads), PfxSmem<D, false>::bytes, st,
               true, p);
  if (e != cudaSuccess) return e;
  e = L.launch("q8_pv", q8_pv_kernel<D, NT>, grid, block, q8_pv_smem(NT, p.q8.B), st, true, p.q8);
  if (e != cudaSuccess) return e;
  e = L.launch("pfx_pv", pfx_kernel<D, true>, pg, dim3(kPfxThreads), PfxSmem<D, true>::bytes, st,
               true, p);
  if (e != cudaSuccess) return e;
  return L.launch("q8_merge", q8_merge_kernel<D>, dim3((unsigned)p.q8.Hq, (unsigned)p.q8.B),
                  dim3(256), 0, st, true, p.q8, 4 * NT);
}
}  // namespace

size_t pfx_workspace_bytes(const Q8Shape &s) { return pfx_layout(s).total; }

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
  const PfxLayout y = pfx_layout(a.s);
  char *ws = static_cast<char *>(a.workspace);
  PfxParams p{};
  p.q8 = q8_params(a, y.q8);
  p.ptable = a.ptable;
  p.prefix = a.s.prefix; p.pages = y.pages; p.steps = y.steps; p.splits = y.splits; p.rows = y.rows;
  p.mrow = reinterpret_cast<uint32_t *>(ws + y.mrow);
  p.svmax = reinterpret_cast<uint32_t *>(ws + y.svmax);
  p.po = reinterpret_cast<float *>(ws + y.po);
  p.pl = reinterpret_cast<float *>(ws + y.pl);
  p.q8.mrow = p.mrow; p.q8.svmax = p.svmax; p.q8.po = p.po; p.q8.pl = p.pl;
  p.q8.splits = y.splits; p.q8.rows = y.rows;
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
