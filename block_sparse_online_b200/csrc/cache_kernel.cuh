// cache_kernel.cuh -- quantising keys and values as they are written into the pages of a
// cache, and reading them back in 16 bits.
//
// A row x (one token of one head) is held as 8-bit codes and one fp32 scale:
//   amax = max |x_e|,  scale = fl(amax / TOP),  code_e = nearest(x_e TOP / amax), ties to even,
// TOP = 127 (int8) or 448 (e4m3, its largest value); a row of zeros has scale 0 and codes 0,
// a row with an element that is not finite has scale NaN, so all of it reads back as NaN.
// The code is the one nearest to the exact ratio: x_e TOP is exact in fp32 (11 bits by 7)
// and a ratio that is no tie lies at least 2^-19 of itself from one, so the correctly
// rounded fp32 quotient falls on the right side of it. (Dividing by the ROUNDED scale does
// not: for amax / TOP inexact it turns ties to one side.)
// Read back: fl16(code_e scale), one rounding.
//
// Memory bound: every row is read once and written once. D / 8 lanes hold a row, 8 elements
// (one 16-byte access of 16-bit data) each, and reduce |x| with shuffles. A block serves
// `tokens` consecutive tokens over all heads, keys and values; where each of them lives
// (sequence, page) is found once and kept in shared memory.
#pragma once

#include "dense_common.cuh"

namespace solattn {

struct CacheArgs {
  void *k, *v;  // pages
  float *k_scale, *v_scale;
  long long k_row, k_head, k_seq, v_row, v_head, v_seq;  // strides of the pages, in elements
  void *new_k, *new_v;                                   // 16-bit rows: read (write call) or written (read call)
  long long nk_tok, nk_head, nv_tok, nv_head;
  const int *table, *cu, *len;
  int width, page, page_shift, num_pages, B, Hkv, total, tokens;
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
constexpr int kCacheTokens = 32;  // most tokens of a block

// WRITE: rows into the pages; else rows out of them.
template <class QT, int KIND, int D, bool WRITE>
__global__ void __launch_bounds__(kCacheThreads) cache_kernel(const CacheArgs a) {
  constexpr int LPR = D / 8;                    // lanes of a row
  constexpr int RPB = kCacheThreads / LPR;      // rows of a block at a time
  constexpr int U = 4;                          // rows of a lane in flight
  __shared__ int s_page[kCacheTokens], s_row[kCacheTokens];
  const int t0 = blockIdx.x * a.tokens;
  const int nt = min(a.tokens, a.total - t0);
  if (static_cast<int>(threadIdx.x) < nt) {
    const int t = t0 + threadIdx.x;
    // last sequence that begins at or before t: cu is ascending
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(a.cu + mid) <= t) lo = mid;
      else hi = mid;
    }
    const int end = __ldg(a.cu + lo + 1);
    int page = -1, row = 0;
    if (t >= __ldg(a.cu + lo) && t < end) {  // rows in front of the first and behind the last sequence are left alone
      const int pos = __ldg(a.len + lo) - (end - t);
      bool ok = pos >= 0 && (pos >> a.page_shift) < a.width;
      if (ok) {
        page = __ldg(a.table + static_cast<size_t>(lo) * a.width + (pos >> a.page_shift));
        ok = static_cast<unsigned>(page) < static_cast<unsigned>(a.num_pages);
      }
      if (!ok) {
        page = -1;
        atomicCAS(a.status, 0, kStatusTable);
      }
      row = pos & (a.page - 1);
    }
    s_page[threadIdx.x] = page;
    s_row[threadIdx.x] = row;
  }
  __syncthreads();
  const int lane = threadIdx.x % LPR;
  const int rows = nt * a.Hkv * 2;  // (token, head, key or value), value fastest
  for (int base = 0; base < rows; base += RPB * U) {
    const int i0 = base + threadIdx.x / LPR;
    uint4 x[U];
    uint2 cd[U];
    float sc[U];
    // Every lane of a warp runs every turn (the maxima use whole-warp shuffles).
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * RPB;
      const int kv = i & 1, ht = i >> 1, t = min(ht / a.Hkv, nt - 1), h = ht % a.Hkv;
      const int page = i < rows ? s_page[t] : -1;
      x[u] = make_uint4(0, 0, 0, 0);
      cd[u] = make_uint2(0, 0);
      sc[u] = 0.f;
      if (page >= 0) {
        if constexpr (WRITE) {
          const QT *src = static_cast<const QT *>(kv ? a.new_v : a.new_k) +
                          static_cast<long long>(t0 + t) * (kv ? a.nv_tok : a.nk_tok) + h * (kv ? a.nv_head : a.nk_head);
          x[u] = *reinterpret_cast<const uint4 *>(src + lane * 8);
        } else {
          const long long at = page * (kv ? a.v_seq : a.k_seq) + h * (kv ? a.v_head : a.k_head) +
                               s_row[t] * (kv ? a.v_row : a.k_row) + lane * 8;
          if constexpr (KIND == kKind16) {
            x[u] = *reinterpret_cast<const uint4 *>(static_cast<const QT *>(kv ? a.v : a.k) + at);
          } else {
            cd[u] = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(kv ? a.v : a.k) + at);
            sc[u] = (kv ? a.v_scale : a.k_scale)[(static_cast<size_t>(page) * a.Hkv + h) * a.page + s_row[t]];
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * RPB;
      const int kv = i & 1, ht = i >> 1, t = min(ht / a.Hkv, nt - 1), h = ht % a.Hkv;
      const int page = i < rows ? s_page[t] : -1;
      const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      if constexpr (WRITE) {
        const long long at = page * (kv ? a.v_seq : a.k_seq) + h * (kv ? a.v_head : a.k_head) +
                             s_row[t] * (kv ? a.v_row : a.k_row) + lane * 8;
        if constexpr (KIND == kKind16) {
          if (page >= 0) *reinterpret_cast<uint4 *>(static_cast<QT *>(kv ? a.v : a.k) + at) = x[u];
        } else {
          constexpr float TOP = KIND == kKindInt8 ? 127.f : 448.f;
          float y[8], amax = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            y[e] = to_float<QT>(w[e >> 1], e & 1);
            amax = max_nan(amax, fabsf(y[e]));
          }
#pragma unroll
          for (int o = LPR / 2; o; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          const bool finite = amax < CUDART_INF_F;  // false for NaN
          float scale = finite ? __fdiv_rn(amax, TOP) : CUDART_NAN_F;
          // x TOP and the quotient keep clear of overflow and of subnormals: rows of very
          // large or very small elements are moved by a power of two first (exact, or below
          // half a code: elements that it flushes are under 2^-20 of the largest)
          float mul = TOP, den = amax;
          if (amax > 0x1p100f) mul = TOP * 0x1p-30f, den = amax * 0x1p-30f;
          if (amax < 0x1p-100f) mul = TOP * 0x1p60f, den = amax * 0x1p60f;
          if (!finite || amax == 0.f) mul = 0.f, den = 1.f;
          uint32_t out[2] = {0, 0};
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            float c0 = finite ? __fdiv_rn(y[e] * mul, den) : 0.f, c1 = finite ? __fdiv_rn(y[e + 1] * mul, den) : 0.f;
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
          if (page >= 0) {
            *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(kv ? a.v : a.k) + at) = make_uint2(out[0], out[1]);
            if (lane == 0) (kv ? a.v_scale : a.k_scale)[(static_cast<size_t>(page) * a.Hkv + h) * a.page + s_row[t]] = scale;
          }
        }
      } else if (page >= 0) {
        QT *dst = static_cast<QT *>(kv ? a.new_v : a.new_k) + static_cast<long long>(t0 + t) * (kv ? a.nv_tok : a.nk_tok) +
                  h * (kv ? a.nv_head : a.nk_head) + lane * 8;
        uint4 r = x[u];
        if constexpr (KIND != kKind16) {
          float y[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t code = ((e < 4 ? cd[u].x : cd[u].y) >> (8 * (e & 3))) & 0xffu;
            if constexpr (KIND == kKindInt8) {
              y[e] = static_cast<float>(static_cast<int>(static_cast<int8_t>(code)));
            } else {
              uint32_t h2;
              asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(code)));
              y[e] = to_float<__half>(h2, 0);
            }
            y[e] *= sc[u];
          }
          r = make_uint4(pack16<QT>(y[0], y[1]), pack16<QT>(y[2], y[3]), pack16<QT>(y[4], y[5]), pack16<QT>(y[6], y[7]));
        }
        *reinterpret_cast<uint4 *>(dst) = r;
      }
    }
  }
}

}  // namespace solattn
