// cache_kernel.cuh -- quantising keys and values as they are written into the pages of a
// cache, and reading them back in 16 bits.
//
// A row x (one token of one head) is held as 8-bit codes and one fp32 scale:
//   amax = max |x_e|,  scale = fl(amax / TOP),  code_e = nearest(x_e TOP / amax), ties to even,
// TOP = 127 (int8) or 448 (e4m3, its largest value); a row of zeros has scale 0 and codes 0,
// a row with an element that is not finite has scale NaN, so all of it reads back as NaN.
// The code is the one nearest to the exact ratio: x_e TOP is exact in fp32 (11 bits by 7)
// and a ratio that is no tie lies at least 2^-19 of itself from one, so an fp32 quotient that
// is exact for short ratios and near for the others falls on the right side of it: the product
// with the row's reciprocal (off by 2^-22), corrected once by its residual (Markstein's step of a division by
// multiplication, 1990), is off by 2^-45 before its last rounding. (Dividing by the ROUNDED scale turns ties to one side; a full division
// for each element cost 14 us where the row's reciprocal and two more products cost 6: 1560 tokens of
// 12 heads of 128.)
// Read back: fl16(code_e scale), one rounding.
//
// Memory bound: every row is read once and written once. A block serves 2^k consecutive tokens
// over all heads, keys and values; where each token lives (sequence, page) is found once and
// kept in shared memory. Rows go token fastest, so that neighbouring lanes read neighbouring
// rows of a page, and a row's token, head and kind are shifts and masks of its number. A lane
// holds pieces of 8 elements (one 16-byte access of 16-bit data): one piece when writing, where the
// row's maximum takes shuffles and the quotients registers, two when reading. 75600 e4m3 tokens of 24 heads of 128
// are read back in 240 us (1.41 GB, 5.8 TB/s; the card's copy runs at 6.55); 1560 int8 tokens of 12 heads
// are written in 7.3 us and read back in 4.6 (activity records), which is mostly launch, the way from token to page
// and, when writing, three turns whose rows are loaded one turn after the other.
#pragma once

#include "dense_common.cuh"
#include "rows_kernel.cuh"

namespace solattn {

struct CacheArgs {
  void *k, *v;  // pages
  float *k_scale, *v_scale;
  long long k_row, k_head, k_seq, v_row, v_head, v_seq;  // strides of the pages, in elements
  void *new_k, *new_v;                                   // 16-bit rows: read (write call) or written (read call)
  long long nk_tok, nk_head, nv_tok, nv_head;
  const int *table, *cu, *len;
  int width, page, page_shift, num_pages, B, Hkv, n, total, Lmax, token_shift;  // n: of calls without cu (there are none)
  int *status;
};

template <class QT>
__device__ __forceinline__ float to_float(uint32_t w, int hi);
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(uint32_t w, int hi) {
  return __uint_as_float(hi ? (w & 0xffff0000u) : (w << 16));
}
template <>
__device__ __forceinline__ float to_float<__half>(uint32_t w, int hi) {
  const __half2 h = *reinterpret_cast<const __half2 *>(&w);
  return hi ? __high2float(h) : __low2float(h);
}

// The larger of two magnitudes; NaN wins.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

constexpr int kCacheThreads = 256;
constexpr int kCacheCu = 1024;  // sequence bounds that are searched in shared memory
// Pieces of 8 elements of a lane, and rows of a block at a time (the most tokens that a block serves).
template <int D, bool WRITE>
struct CacheShape {
  static constexpr int PC = WRITE ? 1 : 2;
  static constexpr int LPR = D / (8 * PC);
  static constexpr int RPB = kCacheThreads / LPR;
  static constexpr int U = WRITE ? 2 : 8;  // rows of a lane in flight (reading a 75600-token cache: 2, 4, 8 rows 248, 253, 240 us)
};

// WRITE: rows into the pages; else rows out of them.
template <class QT, int KIND, int D, bool WRITE>
__global__ void __launch_bounds__(kCacheThreads) cache_kernel(const __grid_constant__ CacheArgs a) {
  using C = CacheShape<D, WRITE>;
  constexpr int PC = C::PC, LPR = C::LPR, U = C::U;
  __shared__ int s_page[C::RPB], s_row[C::RPB], s_cu[kCacheCu];
  const int t0 = blockIdx.x << a.token_shift;
  const int nt = min(1 << a.token_shift, a.total - t0);
  const int lane = threadIdx.x % LPR, g = threadIdx.x / LPR;
  // A thread keeps its token; its rows are (head, key or value) pairs hk = hk0 + i * step.
  const int t = g & ((1 << a.token_shift) - 1);
  const int hk0 = g >> a.token_shift, step = C::RPB >> a.token_shift, n_hk = 2 * a.Hkv;
  const bool live = t < nt;
  QT *new_k = static_cast<QT *>(a.new_k) + static_cast<long long>(t0 + t) * a.nk_tok + lane * 8;
  QT *new_v = static_cast<QT *>(a.new_v) + static_cast<long long>(t0 + t) * a.nv_tok + lane * 8;
  auto new_row = [&](int hk) { return (hk & 1) ? new_v + (hk >> 1) * a.nv_head : new_k + (hk >> 1) * a.nk_head; };
  uint4 x[U][PC];
  // Source rows of a written turn: their place does not wait for the pages.
  auto load_rows = [&](int hb) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int hk = hb + hk0 + u * step;
      x[u][0] = live && hk < n_hk ? *reinterpret_cast<const uint4 *>(new_row(hk)) : make_uint4(0, 0, 0, 0);
    }
  };
  if constexpr (WRITE) load_rows(0);
  const bool in_smem = a.B < kCacheCu;
  if (in_smem) {
    for (int i = threadIdx.x; i <= a.B; i += kCacheThreads) s_cu[i] = first_row(a, __ldg(a.cu + i));
    __syncthreads();
  }
  if (blockIdx.x == 0 && threadIdx.x >= kCacheThreads - 32) check_lengths(a);
  if (static_cast<int>(threadIdx.x) < nt) {
    const int tt = t0 + threadIdx.x;
    auto cu = [&](int i) { return in_smem ? s_cu[i] : first_row(a, __ldg(a.cu + i)); };
    // last sequence that begins at or before the token: cu is ascending (where it is not, a sequence that holds
    // the token, or none)
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cu(mid) <= tt) lo = mid;
      else hi = mid;
    }
    const int end = cu(lo + 1);
    int page = -1, row = 0;
    if (tt >= cu(lo) && tt < end) {  // rows in front of the first and behind the last sequence are left alone
      const int pos = keys_of(a, lo) - (end - tt);
      bool ok = pos >= 0;  // and below Lmax, as the length is
      if (ok) {
        page = __ldg(a.table + static_cast<size_t>(lo) * a.width + (pos >> a.page_shift));
        ok = static_cast<unsigned>(page) < static_cast<unsigned>(a.num_pages);
      }
      if (!ok) {
        page = -1;
        atomicCAS(a.status, 0, kStatusTable);
      }
      row = pos & (a.page - 1);
      if (!SOLATTN_DCHECK_STATUS(page < a.num_pages && lo < a.B && tt < a.total && pos < a.Lmax, a.status)) page = -1;
    }
    s_page[threadIdx.x] = page;
    s_row[threadIdx.x] = row;
  }
  __syncthreads();
  const int page = live ? s_page[t] : -1;
  const int prow = page >= 0 ? s_row[t] : 0;
  constexpr int ES = KIND == kKind16 ? 2 : 1;
  uint8_t *k_row = static_cast<uint8_t *>(a.k) + (max(page, 0) * a.k_seq + prow * a.k_row + lane * 8) * ES;
  uint8_t *v_row = static_cast<uint8_t *>(a.v) + (max(page, 0) * a.v_seq + prow * a.v_row + lane * 8) * ES;
  const long long sc_row = static_cast<long long>(max(page, 0)) * a.Hkv * a.page + prow;
  auto page_row = [&](int hk) { return (hk & 1) ? v_row + (hk >> 1) * a.v_head * ES : k_row + (hk >> 1) * a.k_head * ES; };
  auto scale_at = [&](int hk) { return ((hk & 1) ? a.v_scale : a.k_scale) + sc_row + (hk >> 1) * a.page; };
  // Every lane of a warp runs every turn (the maxima use whole-warp shuffles).
  for (int hb = 0; hb < n_hk; hb += step * U) {
    if constexpr (WRITE) {
      if (hb > 0) load_rows(hb);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int hk = hb + hk0 + u * step;
        const bool ok = page >= 0 && hk < n_hk;
        if constexpr (KIND == kKind16) {
          if (ok) *reinterpret_cast<uint4 *>(page_row(hk)) = x[u][0];
        } else {
          const uint32_t w[4] = {x[u][0].x, x[u][0].y, x[u][0].z, x[u][0].w};
          constexpr float TOP = KIND == kKindInt8 ? 127.f : 448.f;
          float amax = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) amax = max_nan(amax, fabsf(to_float<QT>(w[e >> 1], e & 1)));
#pragma unroll
          for (int o = LPR / 2; o; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          const bool finite = amax < CUDART_INF_F;  // false for NaN
          // x TOP and the quotient keep clear of overflow and of subnormals: rows of very
          // large or very small elements are moved by a power of two first (exact, or below
          // half a code: elements that it flushes are under 2^-20 of the largest)
          float mul = TOP, den = amax;
          if (amax > 0x1p100f) mul = TOP * 0x1p-30f, den = amax * 0x1p-30f;
          if (amax < 0x1p-100f) mul = TOP * 0x1p60f, den = amax * 0x1p60f;
          if (!finite || amax == 0.f) mul = 0.f, den = 1.f;
          const float inv = __frcp_rn(den);
          auto quotient = [&](float y) {
            const float num = y * mul, q = num * inv;
            return finite ? fmaf(fmaf(-q, den, num), inv, q) : 0.f;
          };
          uint32_t out[2] = {0, 0};
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const float c0 = quotient(to_float<QT>(w[e >> 1], 0)), c1 = quotient(to_float<QT>(w[e >> 1], 1));
            uint32_t two;
            if constexpr (KIND == kKindInt8) {
              two = (static_cast<uint32_t>(__float2int_rn(c0)) & 0xffu) | ((static_cast<uint32_t>(__float2int_rn(c1)) & 0xffu) << 8);
            } else {
              uint16_t r;
              asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(c1), "f"(c0));
              two = r;
            }
            out[e >> 2] |= two << (16 * ((e >> 1) & 1));
          }
          if (ok) {
            *reinterpret_cast<uint2 *>(page_row(hk)) = make_uint2(out[0], out[1]);
            if (lane == 0) *scale_at(hk) = finite ? __fdiv_rn(amax, TOP) : CUDART_NAN_F;
          }
        }
      }
    } else if (page >= 0) {
      [[maybe_unused]] uint2 cd[U][PC];
      [[maybe_unused]] float sc[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int hk = hb + hk0 + u * step;
        if (hk < n_hk) {
          const uint8_t *src = page_row(hk);
#pragma unroll
          for (int c = 0; c < PC; ++c) {
            if constexpr (KIND == kKind16) x[u][c] = ld_stream16(src + c * (D / PC) * 2);
            else cd[u][c] = ld_stream8(src + c * (D / PC));
          }
          if constexpr (KIND != kKind16) sc[u] = __ldg(scale_at(hk));
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int hk = hb + hk0 + u * step;
        if (hk < n_hk) {
          QT *dst = new_row(hk);
#pragma unroll
          for (int c = 0; c < PC; ++c) {
            uint4 r = x[u][c];
            if constexpr (KIND != kKind16) {
              uint32_t o[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                // two codes: bytes 0, 1 or 2, 3 of a word
                const uint32_t word = code_word<KIND>(e < 2 ? cd[u][c].x : cd[u][c].y);
                const uint32_t h2 = (e & 1) ? codes_f16x2<KIND, 1>(word) : codes_f16x2<KIND, 0>(word);
                o[e] = pack16<QT>(to_float<__half>(h2, 0) * sc[u], to_float<__half>(h2, 1) * sc[u]);
              }
              r = make_uint4(o[0], o[1], o[2], o[3]);
            }
            *reinterpret_cast<uint4 *>(dst + c * (D / PC)) = r;
          }
        }
      }
    }
  }
}

}  // namespace solattn
