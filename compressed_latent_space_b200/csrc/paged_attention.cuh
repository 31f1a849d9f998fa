// What the paged attention kernels share: their parameters, the line of work units they split, the
// output rows, and the kernel that joins pieces (paged_attention.cu, paged_attention_tc.cu).
#pragma once

#include "paged.cuh"

namespace cca {
namespace {

// x / d for x >= 0 and a quotient below 2^20, rd = 1 / d to 2 ulp: the float quotient is off by one
// at most.
__device__ __forceinline__ float rcp(int d) { return __fdividef(1.f, __int2float_rn(d)); }
__device__ __forceinline__ int div(int x, int d, float rd) {
  int q = __float2int_rz(__int2float_rn(x) * rd);
  const int r = x - q * d;
  if (r < 0) --q;
  else if (r >= d) ++q;
  return q;
}

struct AttnParams {
  PagedBatch batch;
  Rows q, o;
  __nv_bfloat16 *o_lo;           // with o.dtype == kRowsSplit
  const uint8_t *k, *v;
  const uint2 *scales;
  const int *table;
  int *status;
  int *plan;                     // [B + 3]: units before each sequence, run length, item padding
  float *spill;                  // [warps][R D + 2 R]
  float *part_o;                 // [2 CTAs][R][D]
  float2 *part_ml;               // [2 CTAs][R]
  int max_pages, n_pages, page_log2, Hkv, G, warps;
  FastDiv by_g, by_hkv, by_warps;
  int whole;                     // > 0: items are never split, none has more tiles than this
  int direct;                    // ... and every sequence has one row tile: no plan is needed
  FastDiv by_seq;                // units of a sequence then
  float scale_log2;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Whether the sequences have more rows between them than the call.  Ranges that all run forwards
// in [0, tokens] cannot (each begins where the one before ends), so only a batch with an odd one is
// counted.
__device__ __noinline__ bool paged_overlap(const PagedBatch &p) {
  long long n = 0;
  for (int b = 0; b < p.B; ++b) n += paged_seq(p, b, nullptr).n;
  return n > p.tokens;
}

// Tiles of keys that the rows of row tile rt see; one even where there is none, so that some
// warp writes the rows.
template <int KT>
__device__ __forceinline__ int tiles_of(const PagedSeq &s, int rt, int R, const FastDiv &by_g) {
  const int last = min(s.n - 1, div(rt * R + R - 1, by_g));
  const int keys = max(0, min(s.len, s.len - s.n + last + 1));
  return max(1, (keys + KT - 1) / KT);
}
__device__ __forceinline__ int row_tiles(const PagedSeq &s, int R, int G) {
  return (s.n * G + R - 1) / R;
}
// Units of an item on the line.
__device__ __forceinline__ int padded(int tiles, int pad, float rpad) {
  return div(tiles + pad - 1, pad, rpad) * pad;
}
// Where row r of (sequence b, head h) goes in the output.
__device__ __forceinline__ size_t out_offset(const AttnParams &p, const PagedSeq &s, int b, int h, int r) {
  const int tok = div(r, p.by_g);
  return row_offset(p.o, p.batch.cu != nullptr, s, b, tok, h * p.G + r - tok * p.G);
}

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

// (m, l, acc) joined with another piece of the same row.  A piece without a visible key has l = 0
// and no maximum.
__device__ __forceinline__ void join(float &m, float &l, float4 &acc, float m2, float l2, const float4 &v) {
  if (l2 == 0.f) return;
  const float mn = l == 0.f ? m2 : fmaxf(m, m2);
  const float fa = l == 0.f ? 0.f : ex2(m - mn), fb = ex2(m2 - mn);
  m = mn;
  l = l * fa + l2 * fb;
  acc.x = acc.x * fa + v.x * fb;
  acc.y = acc.y * fa + v.y * fb;
  acc.z = acc.z * fa + v.z * fb;
  acc.w = acc.w * fa + v.w * fb;
}

// Rows that a warp of the merge takes: several where a tile has very many.
constexpr int merge_rows(int R) { return R >= 128 ? 8 : 1; }

// Joins the pieces of the items that more than one CTA (of RUNS runs) worked on: WPR warps per
// (row of a tile, head, sequence).  D / 4 lanes hold the row's channels; the lane groups take pieces
// in turn and are added in a fixed order.  4 us at 64 x 8192 tokens (256 items of 2 or 3 pieces):
// three dependent loads and the launch; 10 us behind the tensor-core kernel, whose pieces are 64 KB.
template <int D, int R, int KT, int RUNS, int WPR>
__global__ void __launch_bounds__(128) paged_merge_kernel(const __grid_constant__ AttnParams p, int rows_max) {
  constexpr int LN = D / 4, GW = 32 / LN, GR = GW * WPR, UN = 4;   // UN pieces in flight per group
  constexpr int RPW = WPR == 1 ? merge_rows(R) : 1;  // rows of a warp
  __shared__ float so[WPR == 4 ? 4 : 1][D];
  __shared__ float2 sml[4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int unit = WPR == 4 ? blockIdx.x : blockIdx.x * 4 + warp, per = (rows_max + RPW - 1) / RPW;
  const int h = unit / per, rr0 = (unit - h * per) * RPW, b = blockIdx.y;
  const int ln = lane % LN, grp = (WPR == 4 ? warp * GW : 0) + lane / LN;
  // (the attention kernel lets this one start once its own predecessors are done, so lengths and
  // cu_seqlens are final; what the attention writes is read behind the wait)
  const PagedSeq s = paged_seq(p.batch, b, nullptr);
  const int rows = s.n * p.G, rts = row_tiles(s, R, p.G);
  pdl_wait();
  pdl_launch_dependents();
  if (h >= p.Hkv || rr0 >= rows) return;
  const int p0 = p.plan[b], p1 = p.plan[b + 1], upw = p.plan[p.batch.B + 1], pad = p.plan[p.batch.B + 2];
  if (p0 == p1) return;                              // overlapping sequences: nothing was computed
  const float rpad = rcp(pad), rrun = rcp(upw * RUNS);
  int u0 = p0 + h * div(p1 - p0, p.by_hkv);
  for (int rt = 0; rt < rts; ++rt) {
    const int T = tiles_of<KT>(s, rt, R, p.by_g), first = u0;
    u0 += padded(T, pad, rpad);
    if (rt % gridDim.z != blockIdx.z) continue;
    // the CTAs with its first and last tile
    const int ca = div(first, upw * RUNS, rrun), cz = div(first + T - 1, upw * RUNS, rrun);
    if (ca == cz) continue;
#pragma unroll 1
    for (int q = 0; q < RPW; ++q) {
      const int rr = rr0 + q, r = rt * R + rr;
      if (rr >= R || r >= rows) break;
      float m = 0.f, l = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int c0 = ca + grp; c0 <= cz; c0 += UN * GR) {
        float2 ml[UN];
        float4 v[UN];
#pragma unroll
        for (int i = 0; i < UN; ++i) {
          const int c = c0 + i * GR;
          const size_t at = (static_cast<size_t>(min(c, cz)) * 2 + (c == ca ? 1 : 0)) * R + rr;
          ml[i] = c <= cz ? p.part_ml[at] : make_float2(0.f, 0.f);
          v[i] = c <= cz ? *reinterpret_cast<const float4 *>(p.part_o + at * D + ln * 4)
                         : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int i = 0; i < UN; ++i) join(m, l, acc, ml[i].x, ml[i].y, v[i]);
      }
      __syncwarp();
#pragma unroll
      for (int off = LN; off < 32; off <<= 1) {      // the warp's groups, lower first
        const float m2 = __shfl_down_sync(0xffffffffu, m, off), l2 = __shfl_down_sync(0xffffffffu, l, off);
        float4 v;
        v.x = __shfl_down_sync(0xffffffffu, acc.x, off);
        v.y = __shfl_down_sync(0xffffffffu, acc.y, off);
        v.z = __shfl_down_sync(0xffffffffu, acc.z, off);
        v.w = __shfl_down_sync(0xffffffffu, acc.w, off);
        join(m, l, acc, m2, l2, v);
      }
      if constexpr (WPR == 4) {
        __syncthreads();
        if (lane < LN) *reinterpret_cast<float4 *>(&so[warp][ln * 4]) = acc;
        if (lane == 0) sml[warp] = make_float2(m, l);
        __syncthreads();
        if (warp == 0 && lane < LN)
#pragma unroll
          for (int i = 1; i < 4; ++i)
            join(m, l, acc, sml[i].x, sml[i].y, *reinterpret_cast<const float4 *>(&so[i][ln * 4]));
      }
      if ((WPR == 1 || warp == 0) && lane < LN) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const float v[4] = {l == 0.f ? 0.f : acc.x * inv, l == 0.f ? 0.f : acc.y * inv,
                            l == 0.f ? 0.f : acc.z * inv, l == 0.f ? 0.f : acc.w * inv};
        store_row<4>(p.o, p.o_lo, out_offset(p, s, b, h, r) + ln * 4, v);
      }
    }
  }
}

// CTAs (grid z) that share a sequence's row tiles in the merge: an average sequence's, up to 16.
inline unsigned merge_depth(const PagedArgs &a, int R) {
  const long long tiles = (static_cast<long long>(a.tokens) / a.B * (a.H / a.Hkv) + R - 1) / R;
  return static_cast<unsigned>(tiles < 1 ? 1 : (tiles < 16 ? tiles : 16));
}

inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

}  // namespace
}  // namespace cca
