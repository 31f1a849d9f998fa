// The paged latent cache's writer and reader: keys and values of new tokens appended to their
// sequences' pages with the rotary embedding applied on the way (16 bits, or 4 bits with a scale
// and a zero for each vector), and cached rows read back dense.
//
// 4 bits, per (token, key/value head) vector x of d channels, keys after the rotation:
//   lo = min x, hi = max x;  zero = f16(lo), scale = f16((hi - lo) / 15)
//   n_j = clamp(round_half_even((x_j - zero) / scale), 0, 15)   (0 where scale is 0)
//   held value = scale n_j + zero, off by at most scale / 2 and the two roundings to float16.
// The codes are chosen against the rounded scale and zero, so their rounding costs nothing more
// than the range's ends.  Every step is the IEEE one (division, no contraction), so the same
// input gives the same codes everywhere.
//
// Both kernels move each byte once; HBM bounds them at long prompts and launch latency at single
// tokens.
#include "paged.cuh"

namespace cca {
namespace {

struct AppendParams {
  PagedBatch batch;
  Rows q, qo, nk, nv;
  uint8_t *k, *v;
  __half2 *scales;
  const int *table;
  int *status;
  int max_pages, n_pages, page_log2, Hkv, HQ, page_f16;
  bool rotate;
  float turn_hi[64], turn_lo[64];   // RoPE frequencies in turns, hi + lo (rope_turns_host)
};

// One thread takes channels [8 l, 8 l + 8) and their rotation partners d/2 above of one
// (token, head) row, so a row is D / 16 neighbouring lanes: 16-byte loads of 16-bit inputs, the
// rotation inside the thread, and the extremes of a 4-bit row over at most 8 lanes.
// HQ query heads (rotated into qo), then Hkv keys, then Hkv values per token.
template <int D, int BITS>
__global__ void __launch_bounds__(256) paged_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int LPR = D / 16, HALF = D / 2;
  __shared__ float thi[HALF], tlo[HALF];
  for (int i = threadIdx.x; i < HALF; i += blockDim.x) {
    thi[i] = p.turn_hi[i];
    tlo[i] = p.turn_lo[i];
  }
  __syncthreads();
  pdl_launch_dependents();
  pdl_wait();
  const int heads = p.HQ + 2 * p.Hkv;
  const long long rows = static_cast<long long>(p.batch.tokens) * heads;
  const long long idx = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  const long long row = idx / LPR;
  const int c0 = static_cast<int>(idx % LPR) * 8;
  bool live = row < rows;
  const int token = live ? static_cast<int>(row / heads) : 0;
  const int hh = live ? static_cast<int>(row % heads) : 0;
  // the token's sequence: the last b with cu[b] <= token
  const bool packed = p.batch.cu != nullptr;
  int b;
  if (packed) {
    int lo = 0, hi = p.batch.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.batch.cu[mid] <= token) lo = mid;
      else hi = mid;
    }
    b = lo;
  } else {
    b = token / (p.batch.tokens / p.batch.B);
  }
  const PagedSeq s = paged_seq(p.batch, b, p.status);
  const int i = token - s.t0;
  const int pos = s.len - s.n + i;
  live = live && i >= 0 && i < s.n && pos >= 0 && s.len > 0;

  const bool is_q = hh < p.HQ, is_k = !is_q && hh < p.HQ + p.Hkv;
  const int h = is_q ? hh : (is_k ? hh - p.HQ : hh - p.HQ - p.Hkv);
  float lo8[8], hi8[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) lo8[j] = hi8[j] = 0.f;
  if (live) {
    const Rows &src = is_q ? p.q : (is_k ? p.nk : p.nv);
    const size_t off = row_offset(src, packed, s, b, i, h) + c0;
    load8_as(src.ptr, off, src.dtype, lo8);
    load8_as(src.ptr, off + HALF, src.dtype, hi8);
    if (p.rotate && (is_q || is_k)) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float c, sn;
        rope_cos_sin_turns(pos, thi[c0 + j], tlo[c0 + j], c, sn);
        const float a = lo8[j], bb = hi8[j];
        lo8[j] = a * c - bb * sn;
        hi8[j] = a * sn + bb * c;
      }
    }
  }
  if (is_q) {
    if (live) {
      const size_t off = row_offset(p.qo, packed, s, b, i, h) + c0;
      store8_as(p.qo.ptr, off, p.qo.dtype, lo8);
      store8_as(p.qo.ptr, off + HALF, p.qo.dtype, hi8);
    }
  }
  int page = -1;
  if (live && !is_q)
    page = paged_page(p.table, p.max_pages, p.n_pages, b, pos >> p.page_log2, p.status);
  const size_t slot =
      ((static_cast<size_t>(page < 0 ? 0 : page) * p.Hkv + h) << p.page_log2) + (pos & ((1 << p.page_log2) - 1));
  if constexpr (BITS == 16) {
    if (page >= 0) {
      uint8_t *pages = is_k ? p.k : p.v;
      const int dt = p.page_f16 ? CCA_F16 : CCA_BF16;
      if (p.page_f16) {
        float m = 0.f;                               // a NaN or a value beyond float16
        bool bad = false;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          m = fmaxf(m, fmaxf(fabsf(lo8[j]), fabsf(hi8[j])));
          bad = bad || isnan(lo8[j]) || isnan(hi8[j]);
        }
        if (bad || m > kF16Max) report(p.status, DEV_RANGE);
      }
      store8_as(pages, slot * D + c0, dt, lo8);
      store8_as(pages, slot * D + c0 + HALF, dt, hi8);
    }
  } else {
    float mn = lo8[0], mx = lo8[0], nan = 0.f;       // nan: 0, or NaN when an element is not finite
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      mn = fminf(mn, fminf(lo8[j], hi8[j]));
      mx = fmaxf(mx, fmaxf(lo8[j], hi8[j]));
      nan += __fmul_rn(lo8[j], 0.f) + __fmul_rn(hi8[j], 0.f);
    }
#pragma unroll
    for (int off = 1; off < LPR; off <<= 1) {
      mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, off));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      nan += __shfl_xor_sync(0xffffffffu, nan, off);
    }
    __half zh = __float2half_rn(mn);
    __half sh = __float2half_rn(__fdiv_rn(__fsub_rn(mx, mn), 15.f));
    const bool bad = nan != 0.f || __hisinf(zh) || __hisinf(sh);
    if (bad) {                                       // the whole vector reads back as NaN
      zh = __ushort_as_half(0x7fff);
      sh = __ushort_as_half(0x7fff);
    }
    const float z = __half2float(zh), sc = __half2float(sh);
    if (page >= 0) {
      if (bad) report(p.status, DEV_RANGE);
      uint32_t wl = 0, wh = 0;
      if (!bad && sc > 0.f) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float nl = rintf(__fdiv_rn(__fsub_rn(lo8[j], z), sc));
          const float nh = rintf(__fdiv_rn(__fsub_rn(hi8[j], z), sc));
          wl |= static_cast<uint32_t>(fminf(fmaxf(nl, 0.f), 15.f)) << (4 * j);
          wh |= static_cast<uint32_t>(fminf(fmaxf(nh, 0.f), 15.f)) << (4 * j);
        }
      }
      uint8_t *dst = (is_k ? p.k : p.v) + slot * (D / 2) + c0 / 2;
      *reinterpret_cast<uint32_t *>(dst) = wl;
      *reinterpret_cast<uint32_t *>(dst + HALF / 2) = wh;
      if (c0 == 0) p.scales[slot * 2 + (is_k ? 0 : 1)] = __halves2half2(sh, zh);
    }
  }
}

template <int D, int BITS>
cudaError_t launch_append(const PagedArgs &a, const AppendParams &p, cudaStream_t st) {
  const long long threads = static_cast<long long>(a.tokens) * (p.HQ + 2 * a.Hkv) * (D / 16);
  const long long blocks = (threads + 255) / 256;
  return launch_pdl(paged_append_kernel<D, BITS>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0,
                    st, p);
}

// ------------------------------------------------------------------ gather
struct GatherParams {
  PagedBatch batch;
  Rows nk, nv;
  const uint8_t *k, *v;
  const __half2 *scales;
  const int *table;
  int *status;
  int max_pages, n_pages, page_log2, Hkv, page_f16;
};

// Eight channels of one (token, head, key or value) per thread; the CTAs of sequence blockIdx.y
// walk its tokens in strides, so the grid needs no length.
template <int D, int BITS>
__global__ void __launch_bounds__(256) paged_gather_kernel(const __grid_constant__ GatherParams p) {
  constexpr int CPR = D / 8;
  const int b = blockIdx.y;
  pdl_launch_dependents();
  pdl_wait();
  const PagedSeq s = paged_seq(p.batch, b, p.status);
  const bool packed = p.batch.cu != nullptr;
  const int n = min(s.len, s.n);
  const int per_token = 2 * p.Hkv * CPR;
  const long long total = static_cast<long long>(n) * per_token;
  const long long stride = static_cast<long long>(gridDim.x) * blockDim.x;
  for (long long e = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; e < total;
       e += stride) {
    const int i = static_cast<int>(e / per_token), r = static_cast<int>(e % per_token);
    const int which = r / (p.Hkv * CPR), h = r / CPR % p.Hkv, c0 = r % CPR * 8;
    const int page = paged_page(p.table, p.max_pages, p.n_pages, b, i >> p.page_log2, p.status);
    float v8[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v8[j] = 0.f;
    if (page >= 0) {
      const size_t slot = ((static_cast<size_t>(page) * p.Hkv + h) << p.page_log2) +
                          (i & ((1 << p.page_log2) - 1));
      const uint8_t *pages = which ? p.v : p.k;
      if constexpr (BITS == 16) {
        load8_as(pages, slot * D + c0, p.page_f16 ? CCA_F16 : CCA_BF16, v8);
      } else {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(pages + slot * (D / 2) + c0 / 2);
        const float2 sz = __half22float2(p.scales[slot * 2 + which]);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v8[j] = __fadd_rn(__fmul_rn(static_cast<float>((w >> (4 * j)) & 15u), sz.x), sz.y);
      }
    }
    const Rows &dst = which ? p.nv : p.nk;
    store8_as(dst.ptr, row_offset(dst, packed, s, b, i, h) + c0, dst.dtype, v8);
  }
}

template <int D, int BITS>
cudaError_t launch_gather(const PagedArgs &a, const GatherParams &p, cudaStream_t st) {
  // enough CTAs of a sequence to cover its share of the rows, at most 8 per SM in all
  const long long per_seq = (static_cast<long long>(a.tokens) + a.B - 1) / a.B;
  const long long want = (per_seq * 2 * a.Hkv * (D / 8) + 255) / 256;
  const long long most = 8LL * num_sms() / a.B + 1;
  const unsigned gx = static_cast<unsigned>(want < most ? (want < 1 ? 1 : want) : most);
  return launch_pdl(paged_gather_kernel<D, BITS>, dim3(gx, a.B), dim3(256), 0, st, p);
}

PagedBatch batch_of(const PagedArgs &a) {
  PagedBatch b;
  b.lengths = a.lengths;
  b.cu = a.cu;
  b.B = a.B;
  b.tokens = a.tokens;
  b.len_add = a.len_add;
  b.cap = a.max_pages << a.page_log2;
  return b;
}

}  // namespace

cudaError_t paged_append(const PagedArgs &a, cudaStream_t st) {
  if (a.tokens == 0) return cudaSuccess;
  AppendParams p;
  p.batch = batch_of(a);
  p.q = a.q;
  p.qo = a.qo;
  p.nk = a.nk;
  p.nv = a.nv;
  p.k = static_cast<uint8_t *>(a.k);
  p.v = static_cast<uint8_t *>(a.v);
  p.scales = static_cast<__half2 *>(a.scales);
  p.table = a.table;
  p.status = a.status;
  p.max_pages = a.max_pages;
  p.n_pages = a.n_pages;
  p.page_log2 = a.page_log2;
  p.Hkv = a.Hkv;
  p.HQ = a.q.ptr ? a.H : 0;
  p.page_f16 = a.page_f16;
  p.rotate = a.rope_base > 0.f;
  rope_turns_host(a.D, p.rotate ? a.rope_base : 2.0, p.turn_hi, p.turn_lo, 64);
#define CCA_APPEND(DD)                                                                  \
  if (a.D == DD)                                                                        \
    return a.bits == 4 ? launch_append<DD, 4>(a, p, st) : launch_append<DD, 16>(a, p, st);
  CCA_APPEND(16)
  CCA_APPEND(32)
  CCA_APPEND(64)
  CCA_APPEND(128)
#undef CCA_APPEND
  return cudaErrorInvalidValue;
}

cudaError_t paged_gather(const PagedArgs &a, cudaStream_t st) {
  if (a.tokens == 0) return cudaSuccess;
  GatherParams p;
  p.batch = batch_of(a);
  p.nk = a.nk;
  p.nv = a.nv;
  p.k = static_cast<const uint8_t *>(a.k);
  p.v = static_cast<const uint8_t *>(a.v);
  p.scales = static_cast<const __half2 *>(a.scales);
  p.table = a.table;
  p.status = a.status;
  p.max_pages = a.max_pages;
  p.n_pages = a.n_pages;
  p.page_log2 = a.page_log2;
  p.Hkv = a.Hkv;
  p.page_f16 = a.page_f16;
#define CCA_GATHER(DD)                                                                  \
  if (a.D == DD)                                                                        \
    return a.bits == 4 ? launch_gather<DD, 4>(a, p, st) : launch_gather<DD, 16>(a, p, st);
  CCA_GATHER(16)
  CCA_GATHER(32)
  CCA_GATHER(64)
  CCA_GATHER(128)
#undef CCA_GATHER
  return cudaErrorInvalidValue;
}

}  // namespace cca
