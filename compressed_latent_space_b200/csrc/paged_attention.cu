// Attention of new tokens over the paged cache (16-bit pages, or 4-bit codes with a scale and a
// zero per vector), for any number of new tokens per sequence and ragged lengths.
//
// Row r = i G + (h - g G) of sequence b and key/value head g is token i's query head h; its
// token sits at position len - n + i and sees the keys up to there.  Rows are taken R = 8 NT at
// a time; a work item is (sequence, head, row tile) and its units are the tiles of KT keys that
// its last row sees.
//
// Mathematics, 4 bits (k_j = ks_j n_j + kz_j, v_j = vs_j u_j + vz_j with codes n, u in 0..15):
//   s_j = c (q . k_j) = (c ks_j) (q . n_j) + kz_j (c sum q)
//   o   = sum_j p_j v_j = sum_j (p_j vs_j) u_j + sum_j p_j vz_j
// so the tensor cores multiply by the bare codes and the scales are applied to one score per
// (key, row) instead of d~ channels.  A code needs no conversion either: n in the low bits of a
// float16 is the subnormal n 2^-24, and four bits further up n 2^-20, so `word & 0x000f000f` and
// `word & 0x00f000f0` are pairs of operands, exact, and the powers of two go into the queries
// (those that meet the second kind are scaled by 1/16) and into the result.
//
// Both products are m16n8k16 with the keys (resp. the channels) on the 16 side and eight rows on
// the 8 side: S^T = K Q^T and O^T = V^T P^T.  That way the usual 1 to 8 query heads of a group
// fill the tile (16-row tiles of heads would be half empty), and both operands A come straight
// out of row-major rows: the order of channels within a product is free as long as Q's is the
// same, so a lane reads consecutive channels of a key; the order of keys within P V is free as
// long as P's is the same, so a lane reads keys t, t+4, t+8, t+12 at consecutive channels.
// S^T leaves the product with rows in lanes' columns; movmatrix turns the probabilities into the
// second product's operand.
//
// Softmax: running maximum per row, moved only when a score passes it by more than 8 (in log2
// units), so p <= 2^8; sums in float32.  4 bits: p vs is rounded to float16 after a power of two
// nrm (per warp, following the largest vs met) has brought vs under 2^7: 11 bits of each weight
// whatever the values' scale.  16-bit pages: p itself in float16, or, for bfloat16 pages, as two
// bfloat16 terms (one would keep 8 bits).  q . n: the queries in float16 times a power of two
// that brings the warp's largest to 2^14 (exact but for elements 2^28 below it).
//
// Split: units of all items in one line, cut into equal runs, one per warp; a warp walks its run
// through a private ring of asynchronous copies, without any barrier.  Any mix of lengths is
// balanced, and one long sequence uses the whole machine.  A run that covers an item writes its
// rows; pieces of an item go to the workspace (a warp leaves at most two) and the merge kernel
// adds them in order, so results do not depend on timing.
#include "paged.cuh"

namespace cca {
namespace {

constexpr int kWarps = 4;        // warps per CTA
constexpr int kStages = 3;       // tiles per warp's ring, kStages - 1 in flight
constexpr float kLazy = 8.f;     // the running maximum moves when a score passes it by this much

struct AttnParams {
  PagedBatch batch;
  Rows q, o;
  __nv_bfloat16 *o_lo;           // with o.dtype == kRowsSplit
  const uint8_t *k, *v;
  const uint2 *scales;
  const int *table;
  int *status;
  int *pre;                      // [B + 1] units before each sequence (written by CTA 0)
  float *part_o;                 // [2 warps][R][D]
  float2 *part_ml;               // [2 warps][R]
  int max_pages, n_pages, page_log2, Hkv, G, warps;
  float scale_log2;
};

template <int D, int BITS>
struct Shape {
  static constexpr int ROWB = BITS == 4 ? D / 2 : 2 * D;      // bytes of a cached row
  static constexpr int KT = (BITS == 16 && D == 128) ? 32 : 64;  // keys per tile
  static constexpr int KB = KT / 16;
  static constexpr int TILE = KT * (2 * ROWB + (BITS == 4 ? 8 : 0));
  static constexpr size_t SMEM = static_cast<size_t>(kWarps) * kStages * TILE;
};

// 16-byte piece `c` of row `r` of a 16-bit tile, in pieces from the tile's start: an XOR order
// in which both the key reads (rows g and their neighbours 4 on, consecutive pieces) and the
// value reads (four rows, one piece) of eight lanes fall into different banks.
template <int D>
__device__ __forceinline__ int piece16(int r, int c) {
  if constexpr (D == 64) return r * 8 + (c ^ (((r & 3) << 1) | ((r >> 2) & 1)));
  else if constexpr (D == 128)
    return r * 16 + ((c ^ ((c >> 3) << 1)) ^ (((r & 1) << 2) | ((r >> 1) & 1)) ^ ((r >> 2) & 1));
  else if constexpr (D == 32)
    return (r * 4 + (c ^ (((r >> 1) & 1) << 1))) ^ (((r >> 2) & 1) << 2);
  else
    return (r * 2 + c) ^ (((r >> 2) & 1) << 2);
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
// n consecutive words (1, 2, 4 or a multiple of 4) of a lane
template <int N>
__device__ __forceinline__ void lds_words(uint32_t a, uint32_t *w) {
  if constexpr (N == 1) {
    w[0] = lds32(a);
  } else if constexpr (N == 2) {
    const uint2 u = lds64(a);
    w[0] = u.x;
    w[1] = u.y;
  } else {
    static_assert(N % 4 == 0, "");
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint4 u = lds128(a + 4 * i);
      w[i] = u.x;
      w[i + 1] = u.y;
      w[i + 2] = u.z;
      w[i + 3] = u.w;
    }
  }
}
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Keys tiles that rows up to (row tile rt) of a sequence see; one even where there is none, so
// that some warp writes the rows.
__device__ __forceinline__ int tiles_of(const PagedSeq &s, int rt, int R, int G, int kt_log2) {
  const int last = min(s.n - 1, (rt * R + R - 1) / G);
  const int keys = max(0, min(s.len, s.len - s.n + last + 1));
  return max(1, (keys + (1 << kt_log2) - 1) >> kt_log2);
}
__device__ __forceinline__ int row_tiles(const PagedSeq &s, int R, int G) {
  return (s.n * G + R - 1) / R;
}
__device__ __forceinline__ int units_per_head(const PagedSeq &s, int R, int G, int kt_log2) {
  const int rts = row_tiles(s, R, G);
  int u = 0;
  for (int rt = 0; rt < rts; ++rt) u += tiles_of(s, rt, R, G, kt_log2);
  return u;
}

template <int D, int BITS, int NT, bool QBF16, bool PBF16>
struct Core {
  using S = Shape<D, BITS>;
  static constexpr int KS = D / 16, MT = D / 16, KB = S::KB;
  // tensor-core element types: the queries and 16-bit keys in the pages' type, codes in float16
  static constexpr bool BF_QK = BITS == 16 && PBF16;

  uint32_t qf[NT][KS][2];
  float qz[NT][2];               // scale_log2 * sum of the row's query (4 bits)
  float ksf;                     // factor of a raw score into log2 units
  float m[NT][2], l[NT][2], z[NT][2];
  float o[MT][NT][4];
  float nrm;

  __device__ __forceinline__ void mma_qk(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    if constexpr (BF_QK) mma_bf16_16816(d, a, b);
    else mma_f16_16816(d, a, b);
  }

  // queries of rows [r0, r0 + R) (zero past `rows`) as B fragments
  __device__ __forceinline__ void load_q(const AttnParams &p, const PagedSeq &s, int b, int h,
                                         int r0, int rows, int g, int t) {
    constexpr int E = D / 4;                         // channels [t E, t E + E) of row g
    float mxq = 0.f;
    uint32_t w[NT][E / 2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = r0 + nt * 8 + g;
#pragma unroll
      for (int i = 0; i < E / 2; ++i) w[nt][i] = 0u;
      if (r < rows) {
        const int tok = r / p.G, hh = h * p.G + r % p.G;
        const size_t off = row_offset(p.q, p.batch.cu != nullptr, s, b, tok, hh) + t * E;
        const uint32_t *src = reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(p.q.ptr) + off);
        if constexpr (E == 4) {
          const uint2 u = *reinterpret_cast<const uint2 *>(src);
          w[nt][0] = u.x;
          w[nt][1] = u.y;
        } else {
#pragma unroll
          for (int i = 0; i < E / 2; i += 4) {
            const uint4 u = *reinterpret_cast<const uint4 *>(src + i);
            w[nt][i] = u.x;
            w[nt][i + 1] = u.y;
            w[nt][i + 2] = u.z;
            w[nt][i + 3] = u.w;
          }
        }
      }
    }
    if constexpr (BITS == 16) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          qf[nt][ks][0] = w[nt][2 * ks];
          qf[nt][ks][1] = w[nt][2 * ks + 1];
        }
      ksf = p.scale_log2;
    } else {
      auto val = [&](int nt, int i) {
        const uint32_t x = w[nt][i >> 1];
        const uint32_t hx = (i & 1) ? x >> 16 : x & 0xffffu;
        if constexpr (QBF16) return __uint_as_float(hx << 16);
        else return __half2float(__ushort_as_half(static_cast<unsigned short>(hx)));
      };
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const float x = val(nt, i);
          mxq = fmaxf(mxq, fabsf(x));
          sum += x;
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        qz[nt][0] = __shfl_sync(0xffffffffu, sum, 8 * t) * p.scale_log2;
        qz[nt][1] = __shfl_sync(0xffffffffu, sum, 8 * t + 4) * p.scale_log2;
      }
#pragma unroll
      for (int off = 1; off < 32; off <<= 1)
        mxq = fmaxf(mxq, __shfl_xor_sync(0xffffffffu, mxq, off));
      // 2^(14 - floor(log2 mxq)), the exponent kept within what the inverse below can hold
      int e = static_cast<int>((__float_as_uint(mxq) >> 23) & 255u) - 127;
      e = max(-100, min(100, e));
      const float f = __uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23);
      ksf = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(24 - 14 + e + 127) << 23);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if constexpr (D == 16) {
          qf[nt][0][0] = pack_f16x2(val(nt, 0) * f, val(nt, 1) * f * 0.0625f);
          qf[nt][0][1] = pack_f16x2(val(nt, 2) * f, val(nt, 3) * f * 0.0625f);
        } else {
#pragma unroll
          for (int i = 0; i < E / 8; ++i) {
            const float f16 = f * 0.0625f;
            qf[nt][2 * i][0] = pack_f16x2(val(nt, 8 * i) * f, val(nt, 8 * i + 4) * f);
            qf[nt][2 * i][1] = pack_f16x2(val(nt, 8 * i + 1) * f16, val(nt, 8 * i + 5) * f16);
            qf[nt][2 * i + 1][0] = pack_f16x2(val(nt, 8 * i + 2) * f, val(nt, 8 * i + 6) * f);
            qf[nt][2 * i + 1][1] = pack_f16x2(val(nt, 8 * i + 3) * f16, val(nt, 8 * i + 7) * f16);
          }
        }
      }
    }
  }

  __device__ __forceinline__ void reset() {
    nrm = __uint_as_float(227u << 23);               // 2^100: the first scale met brings it down
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[nt][e] = -INFINITY;
        l[nt][e] = z[nt][e] = 0.f;
      }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) o[mt][nt][0] = o[mt][nt][1] = o[mt][nt][2] = o[mt][nt][3] = 0.f;
  }

  // A fragments of 16 keys (MMA row g = key kp, row g + 8 = key kp + 8 of the block)
  __device__ __forceinline__ void load_k(uint32_t base, int blk, int kp, int t, uint32_t (&a)[KS][4]) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int key = blk * 16 + kp + 8 * half;
      if constexpr (BITS == 4 && D == 16) {
        uint32_t w = lds16(base + key * 8 + t * 2);
        w |= w << 16;
        a[0][half] = w & 0x00f0000fu;
        a[0][2 + half] = (w >> 8) & 0x00f0000fu;
      } else if constexpr (BITS == 4) {
        uint32_t w[D / 32];
        lds_words<D / 32>(base + key * S::ROWB + t * (D / 8), w);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          a[2 * i][half] = w[i] & 0x000f000fu;
          a[2 * i][2 + half] = w[i] & 0x00f000f0u;
          const uint32_t u = w[i] >> 8;
          a[2 * i + 1][half] = u & 0x000f000fu;
          a[2 * i + 1][2 + half] = u & 0x00f000f0u;
        }
      } else if constexpr (D == 16) {
        const uint2 u = lds64(base + piece16<D>(key, t >> 1) * 16 + (t & 1) * 8);
        a[0][half] = u.x;
        a[0][2 + half] = u.y;
      } else {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {           // 16-byte pieces of the lane's D / 4 channels
          const uint4 u = lds128(base + piece16<D>(key, t * (D / 32) + i) * 16);
          a[2 * i][half] = u.x;
          a[2 * i][2 + half] = u.y;
          a[2 * i + 1][half] = u.z;
          a[2 * i + 1][2 + half] = u.w;
        }
      }
    }
  }

  // A fragments of V^T: lane g's channels [g D/8, ..), channel 2 mt in MMA row g and 2 mt + 1 in
  // row g + 8 of product mt; keys t, t + 4, t + 8, t + 12 of the block
  __device__ __forceinline__ void load_v(uint32_t base, int blk, int g, int t, uint32_t (&a)[MT][4]) {
    const int k0 = blk * 16 + t;
    if constexpr (BITS == 4) {
      constexpr int W = D == 128 ? 2 : 1;
      uint32_t w[4][W];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t at = base + (k0 + 4 * i) * S::ROWB + g * (D / 16);
        if constexpr (D == 128) lds_words<2>(at, w[i]);
        else if constexpr (D == 64) w[i][0] = lds32(at);
        else if constexpr (D == 32) w[i][0] = lds16(at);
        else w[i][0] = lds8(at);
      }
#pragma unroll
      for (int pr = 0; pr < 2; ++pr) {               // key pairs (t, t+4), (t+8, t+12)
#pragma unroll
        for (int x = 0; x < W; ++x) {
          const uint32_t lo = __byte_perm(w[2 * pr][x], w[2 * pr + 1][x], 0x5410);
          a[x * 4][2 * pr] = lo & 0x000f000fu;
          a[x * 4][2 * pr + 1] = lo & 0x00f000f0u;
          if constexpr (D >= 32) {
            a[x * 4 + 1][2 * pr] = (lo >> 8) & 0x000f000fu;
            a[x * 4 + 1][2 * pr + 1] = (lo >> 8) & 0x00f000f0u;
          }
          if constexpr (D >= 64) {
            const uint32_t hi = __byte_perm(w[2 * pr][x], w[2 * pr + 1][x], 0x7632);
            a[x * 4 + 2][2 * pr] = hi & 0x000f000fu;
            a[x * 4 + 2][2 * pr + 1] = hi & 0x00f000f0u;
            a[x * 4 + 3][2 * pr] = (hi >> 8) & 0x000f000fu;
            a[x * 4 + 3][2 * pr + 1] = (hi >> 8) & 0x00f000f0u;
          }
        }
      }
    } else {
      constexpr int W = D / 16;                      // words of a lane's D / 8 channels
#pragma unroll
      for (int pr = 0; pr < 2; ++pr) {
        uint32_t x[W], y[W];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int key = k0 + 8 * pr + 4 * e;
          uint32_t(&w)[W] = e ? y : x;
          if constexpr (W == 1) {
            w[0] = lds32(base + piece16<D>(key, g >> 2) * 16 + (g & 3) * 4);
          } else if constexpr (W == 2) {
            const uint2 u = lds64(base + piece16<D>(key, g >> 1) * 16 + (g & 1) * 8);
            w[0] = u.x;
            w[1] = u.y;
          } else {
#pragma unroll
            for (int i = 0; i < W; i += 4) lds_words<4>(base + piece16<D>(key, g * (W / 4) + i / 4) * 16, w + i);
          }
        }
#pragma unroll
        for (int i = 0; i < W; ++i) {                // word i = channels 2 i, 2 i + 1
          a[i][2 * pr] = __byte_perm(x[i], y[i], 0x5410);
          a[i][2 * pr + 1] = __byte_perm(x[i], y[i], 0x7632);
        }
      }
    }
  }

  // One tile of KT keys from key `key0` on.  lim[nt][e]: keys that row 2 t + e of n-tile nt
  // sees; MASK where some row does not see the whole tile.
  template <bool MASK>
  __device__ __forceinline__ void tile(uint32_t kbase, uint32_t vbase, uint32_t sbase, int key0,
                                       const int (&lim)[NT][2], int len, int lane) {
    const int g = lane >> 2, t = lane & 3;
    const int kp = (g >> 1) + 4 * (g & 1);           // the key of MMA row g within its block
    float c[KB][NT][4];
    float2 kzs[KB][2], vzs[KB][2];                   // (scale, zero) of the lane's keys
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      uint32_t a[KS][4];
      load_k(kbase, kb, kp, t, a);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) c[kb][nt][0] = c[kb][nt][1] = c[kb][nt][2] = c[kb][nt][3] = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_qk(c[kb][nt], a[ks], qf[nt][ks]);
      if constexpr (BITS == 4) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int key = kb * 16 + kp + 8 * e;
          const uint2 u = lds64(sbase + key * 8);
          kzs[kb][e] = __half22float2(*reinterpret_cast<const __half2 *>(&u.x));
          vzs[kb][e] = __half22float2(*reinterpret_cast<const __half2 *>(&u.y));
          kzs[kb][e].x *= ksf;
          if (MASK && key0 + key >= len) vzs[kb][e] = make_float2(0.f, 0.f);  // no such key
        }
      }
    }
    auto score = [&](int kb, int nt, int e, float mm) {   // log2 units, less mm
      const int half = e >> 1, col = e & 1;
      if constexpr (BITS == 4)
        return fmaf(c[kb][nt][e], kzs[kb][half].x, fmaf(kzs[kb][half].y, qz[nt][col], -mm));
      else
        return fmaf(c[kb][nt][e], ksf, -mm);
    };
    auto seen = [&](int kb, int nt, int e) {
      return key0 + kb * 16 + kp + 8 * (e >> 1) < lim[nt][e & 1];
    };
    float top = -INFINITY;
    float mv[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) mv[nt][e] = m[nt][e];
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = score(kb, nt, e, m[nt][e & 1]);
          if (MASK && !seen(kb, nt, e)) x = -INFINITY;
          top = fmaxf(top, x);
        }
    bool grow = top > kLazy;
    float vmax = 0.f;
    if constexpr (BITS == 4) {
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) vmax = fmaxf(vmax, fmaxf(vzs[kb][0].x, vzs[kb][1].x));
      grow = grow || vmax * nrm > 128.f;
    }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int col = 0; col < 2; ++col) {
          float mx = mv[nt][col];
#pragma unroll
          for (int kb = 0; kb < KB; ++kb)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const int e = 2 * half + col;
              float x = score(kb, nt, e, 0.f);
              if (MASK && !seen(kb, nt, e)) x = -INFINITY;
              mx = fmaxf(mx, x);
            }
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          const float al = mv[nt][col] == -INFINITY ? 0.f : ex2(mv[nt][col] - mx);
          m[nt][col] = mx;
          l[nt][col] *= al;
          z[nt][col] *= al;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            o[mt][nt][col] *= al;
            o[mt][nt][2 + col] *= al;
          }
        }
      if constexpr (BITS == 4) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1)
          vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, off));
        if (vmax * nrm > 128.f) {                    // warp-uniform: lanes of one g agree already
          const int e = static_cast<int>((__float_as_uint(vmax) >> 23) & 255u) - 127;
          const float nn = __uint_as_float(static_cast<uint32_t>(6 - e + 127) << 23);
          const float f = nn / nrm;
          nrm = nn;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e4 = 0; e4 < 4; ++e4) o[mt][nt][e4] *= f;
        }
      }
    }
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      uint32_t pb[NT][2], pl[NT][2];
      float vn[2] = {0.f, 0.f};
      if constexpr (BITS == 4) {
        vn[0] = vzs[kb][0].x * nrm;
        vn[1] = vzs[kb][1].x * nrm;
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool on = !MASK || seen(kb, nt, e);
          const float pr = on ? ex2(score(kb, nt, e, m[nt][e & 1])) : 0.f;
          l[nt][e & 1] += pr;
          if constexpr (BITS == 4) {
            w[e] = on ? pr * vn[e >> 1] : 0.f;       // a masked key's scale may be anything
            z[nt][e & 1] = on ? fmaf(pr, vzs[kb][e >> 1].y, z[nt][e & 1]) : z[nt][e & 1];
          } else {
            w[e] = pr;
          }
        }
        if constexpr (BITS == 16 && PBF16) {
          uint32_t h0, l0, h1, l1;
          split_bf16x2(make_float2(w[0], w[1]), h0, l0);
          split_bf16x2(make_float2(w[2], w[3]), h1, l1);
          pb[nt][0] = movmatrix_t(h0);
          pb[nt][1] = movmatrix_t(h1);
          pl[nt][0] = movmatrix_t(l0);
          pl[nt][1] = movmatrix_t(l1);
        } else {
          pb[nt][0] = movmatrix_t(pack_f16x2(w[0], w[1]));
          pb[nt][1] = movmatrix_t(pack_f16x2(w[2], w[3]));
        }
      }
      uint32_t a[MT][4];
      load_v(vbase, kb, g, t, a);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if constexpr (BITS == 16 && PBF16) {
            mma_bf16_16816(o[mt][nt], a[mt], pb[nt]);
            mma_bf16_16816(o[mt][nt], a[mt], pl[nt]);
          } else {
            mma_f16_16816(o[mt][nt], a[mt], pb[nt]);
          }
        }
    }
  }

  // l and z over the lanes of a row; o in the values' units, the zeros' share added
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], off);
          if constexpr (BITS == 4) z[nt][e] += __shfl_xor_sync(0xffffffffu, z[nt][e], off);
        }
    if constexpr (BITS == 4) {
      const float f0 = 16777216.f / nrm, f1 = 1048576.f / nrm;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[mt][nt][e] = fmaf(o[mt][nt][e], e < 2 ? f0 : f1, z[nt][e & 1]);
    }
  }
};

// N consecutive output channels of one row
template <int N>
__device__ __forceinline__ void store_row(const Rows &o, __nv_bfloat16 *o_lo, size_t off,
                                          const float (&v)[N]) {
  if (o.dtype == CCA_F32) {
    float *d = static_cast<float *>(o.ptr) + off;
#pragma unroll
    for (int i = 0; i < N; i += 2) *reinterpret_cast<float2 *>(d + i) = make_float2(v[i], v[i + 1]);
  } else if (o.dtype == CCA_F16) {
    uint32_t *d = reinterpret_cast<uint32_t *>(static_cast<__half *>(o.ptr) + off);
#pragma unroll
    for (int i = 0; i < N; i += 2) d[i / 2] = pack_f16x2(v[i], v[i + 1]);
  } else {
    uint32_t *d = reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(o.ptr) + off);
    uint32_t *dl = reinterpret_cast<uint32_t *>(o_lo + off);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      uint32_t hi, lo;
      split_bf16x2(make_float2(v[i], v[i + 1]), hi, lo);
      d[i / 2] = hi;
      if (o.dtype == kRowsSplit) dl[i / 2] = lo;
    }
  }
}

template <int D, int BITS, int NT, bool QBF16, bool PBF16>
__global__ void __launch_bounds__(32 * kWarps) paged_attention_kernel(const __grid_constant__ AttnParams p) {
  using C = Core<D, BITS, NT, QBF16, PBF16>;
  using S = Shape<D, BITS>;
  constexpr int R = 8 * NT, KT = S::KT, KTL = KT == 64 ? 6 : 5, ROWB = S::ROWB;
  extern __shared__ __align__(128) uint8_t smem[];
  int *pre = reinterpret_cast<int *>(smem + S::SMEM);          // [B + 1]
  __shared__ int warp_sum[kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  pdl_launch_dependents();
  pdl_wait();
  // units before each sequence: thread i sums a run of sequences, then a scan over the threads
  const int B = p.batch.B;
  {
    const int per = (B + 32 * kWarps - 1) / (32 * kWarps);
    const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
    int sum = 0;
    for (int b = b0; b < b1; ++b) {
      const int u = p.Hkv * units_per_head(paged_seq(p.batch, b, p.status), R, p.G, KTL);
      pre[b + 1] = u;
      sum += u;
    }
    int inc = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc, off);
      if (lane >= off) inc += x;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    int run = inc - sum;
    for (int w = 0; w < warp; ++w) run += warp_sum[w];
    if (tid == 0) pre[0] = 0;
    for (int b = b0; b < b1; ++b) {
      run += pre[b + 1];
      pre[b + 1] = run;
    }
    __syncthreads();
    if (blockIdx.x == 0)
      for (int b = tid; b <= B; b += 32 * kWarps) p.pre[b] = pre[b];
  }
  const int total = pre[B];
  const int w = blockIdx.x * kWarps + warp;
  const int upw = (total + p.warps - 1) / p.warps;
  int u = min(static_cast<long long>(total), static_cast<long long>(w) * upw);
  const int uend = min(total, u + upw);
  const uint32_t ring = smem_u32(smem) + warp * kStages * S::TILE;
  uint8_t *ring_p = smem + warp * kStages * S::TILE;
  const uint64_t pol = l2_evict_first_policy();
  (void)pol;

  while (u < uend) {
    int b;
    {
      int lo = 0, hi = B;                            // the last b with pre[b] <= u
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= u) lo = mid;
        else hi = mid;
      }
      b = lo;
    }
    const PagedSeq s = paged_seq(p.batch, b, p.status);
    const int per_head = (pre[b + 1] - pre[b]) / p.Hkv;
    const int h = (u - pre[b]) / per_head;
    int t0 = (u - pre[b]) % per_head, rt = 0, T;
    while (t0 >= (T = tiles_of(s, rt, R, p.G, KTL))) {
      t0 -= T;
      ++rt;
    }
    const int t1 = min(T, t0 + (uend - u));
    u += t1 - t0;
    const int rows = s.n * p.G, r0 = rt * R;

    // ---- copies of tile `i` into its slot; the next tile's pages are looked up one tile ahead
    auto look = [&](int i) {                         // lane kb < KB: first row of block kb, or -1
      const int key = i * KT + lane * 16;
      int row = -1;
      if (lane < S::KB && i < t1 && key < s.len) {
        const int page = paged_page(p.table, p.max_pages, p.n_pages, b, key >> p.page_log2, p.status);
        if (page >= 0)
          row = ((page * p.Hkv + h) << p.page_log2) + (key & ((1 << p.page_log2) - 1));
      }
      return row;
    };
    int next = look(t0);
    auto issue = [&](int i, int slot) {
      if (i < t1) {
        const int rows16 = next;
        next = look(i + 1);
        uint8_t *kd = ring_p + slot * S::TILE, *vd = kd + KT * ROWB, *sd = vd + KT * ROWB;
#pragma unroll
        for (int j = 0; j < KT * ROWB / 512; ++j) {
          const int cidx = j * 32 + lane, blk = cidx / ROWB, cb = cidx % ROWB;
          const int row = __shfl_sync(0xffffffffu, rows16, blk);
          bool ok = row >= 0;
          int dst = cidx;
          if constexpr (BITS == 16) {
            constexpr int CPR = D / 8;
            const int key = cidx / CPR;
            ok = ok && i * KT + key < s.len;         // nothing of a row without a token is used
            dst = piece16<D>(key, cidx % CPR);
          }
          const size_t src = static_cast<size_t>(max(row, 0)) * ROWB + cb * 16;
          cp_async16_zfill(kd + dst * 16, p.k + src, ok);
          cp_async16_zfill(vd + dst * 16, p.v + src, ok);
        }
        if constexpr (BITS == 4) {
          const int row = __shfl_sync(0xffffffffu, rows16, lane >> 3);
          cp_async16_zfill(sd + lane * 16, p.scales + static_cast<size_t>(max(row, 0)) + (lane & 7) * 2,
                           row >= 0);
        }
      }
      cp_async_commit();
    };
    __syncwarp();                                    // the ring's last readers are done
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(t0 + i, i);

    C core;
    core.reset();
    core.load_q(p, s, b, h, r0, rows, g, t);
    int lim[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int tok = min(s.n - 1, (r0 + nt * 8 + 2 * t + e) / p.G);
        lim[nt][e] = min(s.len, s.len - s.n + tok + 1);
      }
    const int first_lim = min(s.len, s.len - s.n + r0 / p.G + 1);   // of the tile's first row

    int slot = 0;
    for (int i = t0; i < t1; ++i) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      __syncwarp();
      issue(i + kStages - 1, slot == 0 ? kStages - 1 : slot - 1);
      const uint32_t kb = ring + slot * S::TILE, vb = kb + KT * ROWB, sb = vb + KT * ROWB;
      if ((i + 1) * KT <= first_lim) core.template tile<false>(kb, vb, sb, i * KT, lim, s.len, lane);
      else core.template tile<true>(kb, vb, sb, i * KT, lim, s.len, lane);
      slot = slot == kStages - 1 ? 0 : slot + 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    core.finish();

    const bool whole = t0 == 0 && t1 == T;
    constexpr int N = D / 8;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rr = nt * 8 + 2 * t + e, r = r0 + rr;
        if (r >= rows) continue;
        float v[N];
#pragma unroll
        for (int mt = 0; mt < C::MT; ++mt) {
          v[2 * mt] = core.o[mt][nt][e];
          v[2 * mt + 1] = core.o[mt][nt][2 + e];
        }
        if (whole) {
          const float inv = core.l[nt][e] == 0.f ? 0.f : 1.f / core.l[nt][e];
#pragma unroll
          for (int x = 0; x < N; ++x) v[x] = core.l[nt][e] == 0.f ? 0.f : v[x] * inv;
          store_row<N>(p.o, p.o_lo,
                       row_offset(p.o, p.batch.cu != nullptr, s, b, r / p.G, h * p.G + r % p.G) + g * N, v);
        } else {
          const size_t at = (static_cast<size_t>(w) * 2 + (t0 == 0 ? 1 : 0)) * R + rr;
          float *d = p.part_o + at * D + g * N;
#pragma unroll
          for (int x = 0; x < N; x += 2) *reinterpret_cast<float2 *>(d + x) = make_float2(v[x], v[x + 1]);
          if (g == 0) p.part_ml[at] = make_float2(core.m[nt][e], core.l[nt][e]);
        }
      }
  }
}

// Joins the pieces of the items that more than one warp worked on.  One CTA per (row of a tile,
// head, sequence): D / 4 lanes hold the row's channels, the CTA's lane groups take pieces in turn
// and are added in a fixed order.
template <int D, int NT, int KTL>
__global__ void __launch_bounds__(128) paged_merge_kernel(const __grid_constant__ AttnParams p) {
  constexpr int R = 8 * NT, LN = D / 4, GR = 128 / LN;
  __shared__ float so[GR][D];
  __shared__ float2 sml[GR];
  const int rr = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int grp = threadIdx.x / LN, ln = threadIdx.x % LN;
  pdl_launch_dependents();
  pdl_wait();
  const PagedSeq s = paged_seq(p.batch, b, nullptr);
  const int rows = s.n * p.G, rts = row_tiles(s, R, p.G);
  if (rr >= rows) return;
  const int total = p.pre[p.batch.B], upw = (total + p.warps - 1) / p.warps;
  int u0 = p.pre[b] + h * ((p.pre[b + 1] - p.pre[b]) / p.Hkv);
  for (int rt = 0; rt < rts; ++rt) {
    const int T = tiles_of(s, rt, R, p.G, KTL);
    const int w0 = u0 / upw, w1 = (u0 + T - 1) / upw, r = rt * R + rr;
    u0 += T;
    if (w0 == w1 || r >= rows) continue;
    float m = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w = w0 + grp; w <= w1; w += GR) {
      const size_t at = (static_cast<size_t>(w) * 2 + (w == w0 ? 1 : 0)) * R + rr;
      const float2 ml = p.part_ml[at];
      const float4 v = *reinterpret_cast<const float4 *>(p.part_o + at * D + ln * 4);
      if (ml.y == 0.f && ml.x == -INFINITY) continue;      // no visible key in this piece
      const float mn = fmaxf(m, ml.x);
      const float fa = m == -INFINITY ? 0.f : ex2(m - mn), fb = ex2(ml.x - mn);
      m = mn;
      l = l * fa + ml.y * fb;
      acc.x = acc.x * fa + v.x * fb;
      acc.y = acc.y * fa + v.y * fb;
      acc.z = acc.z * fa + v.z * fb;
      acc.w = acc.w * fa + v.w * fb;
    }
    __syncthreads();
    *reinterpret_cast<float4 *>(&so[grp][ln * 4]) = acc;
    if (ln == 0) sml[grp] = make_float2(m, l);
    __syncthreads();
    if (threadIdx.x < LN) {
      float M = -INFINITY, L = 0.f;
      for (int i = 0; i < GR; ++i) M = fmaxf(M, sml[i].x);
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      for (int i = 0; i < GR; ++i) {
        if (sml[i].x == -INFINITY && sml[i].y == 0.f) continue;
        const float f = ex2(sml[i].x - M);
        L = fmaf(sml[i].y, f, L);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = fmaf(so[i][ln * 4 + j], f, v[j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = L == 0.f ? 0.f : v[j] / L;
      store_row<4>(p.o, p.o_lo,
                   row_offset(p.o, p.batch.cu != nullptr, s, b, r / p.G, h * p.G + r % p.G) + ln * 4, v);
    }
  }
}

inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Row tiles of 8, 16 or 32 rows by the rows of an average sequence: a tile's keys are read and
// unpacked once for all its rows.  16 at d~ = 128, where 32 rows' accumulators would not fit the
// registers.
int pick_nt(const PagedArgs &a) {
  const long long per = (static_cast<long long>(a.tokens) + a.B - 1) / a.B * (a.H / a.Hkv);
  if (per <= 8) return 1;
  if (per <= 16 || a.D == 128) return 2;
  return 4;
}

int key_tile_log2(const PagedArgs &a) { return a.bits == 16 && a.D == 128 ? 5 : 6; }

// Warps of a launch: as many CTAs as fit the device at once by shared memory (227 KB an SM; the
// registers allow as many), but no more than the units there can be.
int plan_ctas(const PagedArgs &a) {
  const int rowb = a.bits == 4 ? a.D / 2 : 2 * a.D, kt = 1 << key_tile_log2(a);
  const size_t smem = static_cast<size_t>(kWarps) * kStages * kt * (2 * rowb + (a.bits == 4 ? 8 : 0)) +
                      (a.B + 1) * 4 + 1024;
  const int nt = pick_nt(a);
  const int by_regs = nt == 1 ? 4 : (nt == 2 ? 3 : 2);
  long long per_sm = (227 * 1024) / static_cast<long long>(smem);
  if (per_sm > by_regs) per_sm = by_regs;
  if (per_sm < 1) per_sm = 1;
  const long long units = paged_attention_units(a);
  long long ctas = per_sm * num_sms();
  if (ctas > (units + kWarps - 1) / kWarps) ctas = (units + kWarps - 1) / kWarps;
  return static_cast<int>(ctas < 1 ? 1 : ctas);
}

struct AttnLayout {
  size_t pre, ml, o, total;
};
AttnLayout attn_layout(const PagedArgs &a, int ctas) {
  AttnLayout L;
  const size_t rows = static_cast<size_t>(ctas) * kWarps * 2 * 8 * pick_nt(a);
  L.pre = 0;
  L.ml = align256(static_cast<size_t>(a.B + 1) * 4);
  L.o = L.ml + align256(rows * 8);
  L.total = L.o + align256(rows * a.D * 4);
  return L;
}

template <int D, int BITS, int NT, bool QBF16, bool PBF16>
cudaError_t launch(const PagedArgs &a, const AttnParams &p, int ctas, cudaStream_t st) {
  const size_t smem = Shape<D, BITS>::SMEM + static_cast<size_t>(a.B + 1) * 4;
  cudaError_t e = ensure_dyn_smem<paged_attention_kernel<D, BITS, NT, QBF16, PBF16>>(smem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(paged_attention_kernel<D, BITS, NT, QBF16, PBF16>, dim3(ctas), dim3(32 * kWarps),
                 smem, st, p);
  if (e != cudaSuccess) return e;
  const long long rows = static_cast<long long>(a.tokens) * p.G;
  const unsigned gx = static_cast<unsigned>(rows < 8 * NT ? rows : 8 * NT);
  return launch_pdl(paged_merge_kernel<D, NT, Shape<D, BITS>::KT == 64 ? 6 : 5>,
                    dim3(gx, a.Hkv, a.B), dim3(128), 0, st, p);
}

template <int D, int NT>
cudaError_t launch_typed(const PagedArgs &a, const AttnParams &p, int ctas, cudaStream_t st) {
  if (a.bits == 16) {
    if (a.page_f16) return launch<D, 16, NT, false, false>(a, p, ctas, st);
    return launch<D, 16, NT, true, true>(a, p, ctas, st);
  }
  if (a.q.dtype == CCA_F16) return launch<D, 4, NT, false, false>(a, p, ctas, st);
  return launch<D, 4, NT, true, false>(a, p, ctas, st);
}

template <int D>
cudaError_t launch_rows(const PagedArgs &a, const AttnParams &p, int ctas, cudaStream_t st) {
  switch (pick_nt(a)) {
    case 1: return launch_typed<D, 1>(a, p, ctas, st);
    case 2: return launch_typed<D, 2>(a, p, ctas, st);
    default:
      if constexpr (D < 128) return launch_typed<D, 4>(a, p, ctas, st);
      return cudaErrorInvalidValue;
  }
}

}  // namespace

long long paged_attention_units(const PagedArgs &a) {
  const long long R = 8 * pick_nt(a), G = a.H / a.Hkv;
  const long long cap = static_cast<long long>(a.max_pages) << a.page_log2;
  const long long tiles = (cap >> key_tile_log2(a)) + 1;
  const long long row_tiles = a.tokens * G / R + a.B;
  return row_tiles * tiles * a.Hkv;
}

size_t paged_attention_workspace(const PagedArgs &a) { return attn_layout(a, plan_ctas(a)).total; }

cudaError_t paged_attention(const PagedArgs &a, cudaStream_t st) {
  if (a.tokens == 0) return cudaSuccess;
  const int ctas = plan_ctas(a);
  const AttnLayout L = attn_layout(a, ctas);
  char *ws = static_cast<char *>(a.workspace);
  AttnParams p;
  p.batch.lengths = a.lengths;
  p.batch.cu = a.cu;
  p.batch.B = a.B;
  p.batch.tokens = a.tokens;
  p.batch.len_add = a.len_add;
  p.batch.cap = a.max_pages << a.page_log2;
  p.q = a.q;
  p.o = a.qo;
  p.o_lo = static_cast<__nv_bfloat16 *>(a.o_lo);
  p.k = static_cast<const uint8_t *>(a.k);
  p.v = static_cast<const uint8_t *>(a.v);
  p.scales = static_cast<const uint2 *>(a.scales);
  p.table = a.table;
  p.status = a.status;
  p.pre = reinterpret_cast<int *>(ws + L.pre);
  p.part_ml = reinterpret_cast<float2 *>(ws + L.ml);
  p.part_o = reinterpret_cast<float *>(ws + L.o);
  p.max_pages = a.max_pages;
  p.n_pages = a.n_pages;
  p.page_log2 = a.page_log2;
  p.Hkv = a.Hkv;
  p.G = a.H / a.Hkv;
  p.warps = ctas * kWarps;
  p.scale_log2 = static_cast<float>(a.scale * 1.4426950408889634);
  switch (a.D) {
    case 16: return launch_rows<16>(a, p, ctas, st);
    case 32: return launch_rows<32>(a, p, ctas, st);
    case 64: return launch_rows<64>(a, p, ctas, st);
    case 128: return launch_rows<128>(a, p, ctas, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace cca
