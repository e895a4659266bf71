// rows_kernel.cuh -- dense attention for few query rows of a key head (single tokens, short
// chunks, a handful of queries): every key and value is read once, straight into registers.
//
// A block of four warps walks its range of the work line; a tile is 8 NT rows. Each warp
// takes 16 keys at a time, with its own running maximum, sum and output per row; the block
// joins the four at the end of a segment. Both products run on m16n8k16 tensor
// instructions with the KEYS (or the output columns) in the 16-row operand and the query
// rows in the 8-column one, so eight rows fill an instruction:
//   S^T = K Q^T   the lane's K registers are 16-byte pieces of two key rows as they lie in
//                 memory; a dot product does not mind the order of its terms, so Q is laid
//                 out once in the order that those pieces give.
//   O^T = V^T P^T the lane loads pieces of four key rows and pairs the keys of each column
//                 with byte permutes; P^T comes from S^T by an 8x8 transpose in registers.
// No shared memory, no barrier and no copy stands between a key's load and its use, and the
// next keys are in flight meanwhile.
//
// Softmax: a row's reference maximum moves only when a score exceeds it by more than 8 (in
// log2 units), so the usual step has one vote in place of the shuffles of a maximum, and
// P <= 2^8. P is rounded to the 16-bit type of the product: off by at most 2^-8 (bf16) or 2^-11
// (fp16) of each value, independently from key to key, which adds about as much to the result's
// error as the output's own rounding. Maxima, sums and O stay in 32 bits.
//
// 8-bit caches: codes are expanded to fp16 (exact: int8 has 8 bits, e4m3 four and a range
// that fp16 holds). A key's scale multiplies its score in 32 bits. A value's scale s_j multiplies its
// probability before that is rounded, and the row's reference is the maximum of x_j + log2 |s_j| over the keys
// that the row sees, not of the scores x_j: then the products 2^(x_j - m) s_j are at most 2^8 and the largest is at least 1,
// for caches of any magnitude (2^-100 to 2^100) and scales of any spread, and a product is off by 2^-11 of itself or,
// below 2^-14 of the largest, by at most 2^-25 of that. Keys that a row does not see, or that have
// no weight, take no bits from the others. The sum of weights is kept in 32 bits in the same units, which reach from 2^-100 to
// 2^100: where the reference moves by more than a factor holds, the sum takes the factor's root twice.
// Queries in bf16 become fp16 after a division of each row by a power of two that brings its largest element to
// [2^14, 2^15): exact down to 2^-31 of that element.
//
// Bound by memory: at 32 sequences of 1 to 16384 keys, 4 key heads of 128, bf16, one token each, it reads
// 551 MB in 84 us (6.5 TB/s). In e4m3 at 118800 keys of 24 heads (753 MB) it takes 135 us (5.6 TB/s): half the
// bytes for each key leave half the bytes in flight, and more blocks per SM cost spills. Measured and not kept:
// the next values loaded before the next scores (155 us there), four blocks per SM (156 us).
#pragma once

#include "dense_common.cuh"

namespace solattn {

template <class T>
struct Type16;
template <>
struct Type16<__nv_bfloat16> {
  static __device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
};
template <>
struct Type16<__half> {
  static __device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
};

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(x));
  return d;
}
// Loads of keys and values: read once by this SM, so they do not stay in its L1.
__device__ __forceinline__ uint4 ld_stream16(const void *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ld_stream8(const void *p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

// Two 8-bit codes (bytes 0 and 1 of t after the caller's permute) as two fp16, exactly.
template <int KIND, int HI>
__device__ __forceinline__ uint32_t codes_f16x2(uint32_t t) {
  uint32_t d;
  if constexpr (KIND == kKindE4m3) {
    // hardware conversion of two e4m3 codes
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(static_cast<uint16_t>(HI ? (t >> 16) : (t & 0xffffu))));
  } else {
    // t holds code + 128 as unsigned bytes: 1024 + byte is the fp16 with bits 0x6400 | byte
    const uint32_t w = prmt(t, 0x64646464u, HI ? 0x4342u : 0x4140u);
    const __half2 v = __hsub2(*reinterpret_cast<const __half2 *>(&w), __half2half2(__float2half(1152.f)));
    d = *reinterpret_cast<const uint32_t *>(&v);
  }
  return d;
}
// Codes as the conversion wants them: int8 moved to unsigned by flipping the sign bits.
template <int KIND>
__device__ __forceinline__ uint32_t code_word(uint32_t x) {
  return KIND == kKindInt8 ? x ^ 0x80808080u : x;
}

// log2 of a value scale's magnitude, for the reference of a row: cut to +-100, which a scale of 0, and one beyond, takes.
__device__ __forceinline__ float log2_scale(float x) { return fminf(fmaxf(__log2f(fabsf(x)), -100.f), 100.f); }

constexpr int kRowsWarps = 4;
constexpr float kRowsSlack = 8.0f;  // log2 units the reference maximum may lag

// Blocks of an SM, as registers allow: 168 of a thread with eight rows, 254 with sixteen. (The 16-bit kernel for d = 128 and
// eight rows stores 32 to 72 bytes of a thread to local memory at that; four blocks for the 8-bit kinds
// spill more: 156 against 142 us at 118800 e4m3 keys of 24 heads.)
constexpr int rows_blocks(int nt) { return nt == 1 ? 3 : 2; }

template <class QT, int KIND, int D, int NT, bool PAGED>
struct RowsCfg {
  static constexpr int ROWS = 8 * NT;
  static constexpr int KW = KIND == kKind16 ? D / 8 : D / 16;  // 32-bit words of a key row per lane
  static constexpr int VW = KIND == kKind16 ? D / 16 : D / 32; // words of a value row per lane (D / 8 elements)
  static constexpr int KS = D / 16;                            // k steps of S = m tiles of O
};

// Merge buffers of a block: per warp and row, maximum, sum and output.
template <int ROWS, int D>
struct RowsSmem {
  float m[kRowsWarps][ROWS], l[kRowsWarps][ROWS];
  alignas(16) float o[kRowsWarps][ROWS][D + 4];
};

template <class QT, int KIND, int D, int NT, bool PAGED>
__global__ void __launch_bounds__(kRowsWarps * 32, rows_blocks(NT)) rows_kernel(const __grid_constant__ DenseArgs a, int min_units, int whole_items) {
  using C = RowsCfg<QT, KIND, D, NT, PAGED>;
  using T = RowTiles<C::ROWS>;
  using MT = typename std::conditional<KIND == kKind16, QT, __half>::type;  // operands' type
  constexpr int ES = KIND == kKind16 ? 2 : 1;                               // bytes of a cached element
  __shared__ RowsSmem<C::ROWS, D> sm;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  pdl_launch_dependents();
  if (blockIdx.x == 0 && warp == 0) check_lengths(a);
  Cursor<T> cur;
  int4 rec = make_int4(0, 0, 0, 0);
  for (bool more = cur.begin(a, blockIdx.x, gridDim.x, min_units, whole_items); more; more = cur.step(a)) {
    const Seq s = cur.s;
    const int b = cur.b, h = cur.h, t = cur.t;
    // ---- queries of the tile, in the order of the keys' pieces
    uint32_t qf[NT][C::KS][2];
    float qscale[NT][2];  // scale of rows 2c, 2c + 1 (log2 units)
    int lim[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      int tok, gg;
      const bool ok = T::row(a, s.n, t, nt * 8 + g, tok, gg) &&
                      SOLATTN_DCHECK_STATUS(row_inside(a, b, s.tok0 + tok, h * a.G + gg), a.status);
      const QT *src = static_cast<const QT *>(a.q) + b * a.q_batch + static_cast<long long>(s.tok0 + tok) * a.q_tok +
                      static_cast<long long>(h * a.G + gg) * a.q_head;
      uint32_t w[D / 8];
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        // 16-bit keys: piece i holds d = 32 i + 8 c ..+7. 8-bit: piece i / 2 holds d = 64 (i / 2) + 16 c ..+15.
        const int d0 = KIND == kKind16 ? 32 * i + 8 * c : 64 * (i >> 1) + 16 * c + 8 * (i & 1);
        const uint4 v = ok ? __ldg(reinterpret_cast<const uint4 *>(src + d0)) : make_uint4(0, 0, 0, 0);
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
      }
      float down = 1.f;  // what the row was divided by
      if constexpr (KIND != kKind16 && std::is_same<QT, __nv_bfloat16>::value) {
        uint32_t big = 0;  // largest magnitude of the row, as bf16 bits
#pragma unroll
        for (int i = 0; i < D / 8; ++i) big = max(big, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
        big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
        const int ex = static_cast<int>(big >> 7);  // biased exponent
        // up = 2^(14 - e), down = 2^(e - 14) with e = ex - 127, kept to normal numbers
        const int sh = (ex == 0 || ex == 255) ? 0 : min(max(141 - ex, -126), 126);
        const float up = __int_as_float((127 + sh) << 23);
        down = __int_as_float((127 - sh) << 23);
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
          w[i] = pack_f16x2(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xffff0000u) * up);
      }
#pragma unroll
      for (int i = 0; i < C::KS; ++i) qf[nt][i][0] = w[2 * i], qf[nt][i][1] = w[2 * i + 1];
      // row g's factor sits in lanes 4 g ..; this lane's scores belong to rows 2c and 2c + 1
      qscale[nt][0] = __shfl_sync(0xffffffffu, down, 8 * c) * a.scale_log2;
      qscale[nt][1] = __shfl_sync(0xffffffffu, down, 8 * c + 4) * a.scale_log2;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const bool r_ok = T::row(a, s.n, t, nt * 8 + 2 * c + e, tok, gg);
        lim[nt][e] = r_ok ? key_limit(a, s, tok) : 0;
      }
    }
    const int klim = key_limit(a, s, T::last_token(a, s.n, t));  // keys that some row sees
    const int kmin = key_limit(a, s, (t * C::ROWS) / a.G);       // keys that every row sees
    const int gend = min(cur.u1 * (kUnitKeys / 16), (klim + 15) >> 4);

    float m[NT][2], l[NT][2], o[NT][C::KS][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -CUDART_INF_F;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int i = 0; i < C::KS; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
    }
    const uint8_t *kbase = static_cast<const uint8_t *>(a.k) + h * a.k_head * ES;
    const uint8_t *vbase = static_cast<const uint8_t *>(a.v) + h * a.v_head * ES;
    // Page of a group of 16 keys (contiguous keys: the batch index); -1: not to be read.
    auto locate = [&](int gr) -> int {
      if (gr >= gend) return -1;
      if constexpr (PAGED) return page_of(a, b, gr * 16);
      return b;
    };
    uint32_t kr[2][C::KW];
    float ksc[2], vsc[2];
    auto load_k = [&](int gr, int id) {
      const int j = PAGED ? (gr * 16) & (a.page - 1) : gr * 16;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int key = gr * 16 + g + 8 * e;
        const bool ok = id >= 0 && key < klim && SOLATTN_DCHECK_STATUS(key_inside(a, id, j + g + 8 * e), a.status);
        const uint8_t *p = kbase + (id * a.k_seq + static_cast<long long>(j + g + 8 * e) * a.k_row) * ES + c * 16;
#pragma unroll
        for (int i = 0; i < C::KW / 4; ++i) {
          const uint4 x = ok ? ld_stream16(p + i * 64) : make_uint4(0, 0, 0, 0);
          kr[e][4 * i] = x.x, kr[e][4 * i + 1] = x.y, kr[e][4 * i + 2] = x.z, kr[e][4 * i + 3] = x.w;
        }
        if constexpr (KIND != kKind16) {
          const size_t at = (static_cast<size_t>(ok ? id : 0) * a.Hkv + h) * a.page + j + g + 8 * e;
          ksc[e] = ok ? __ldg(a.k_scale + at) : 0.f;
          vsc[e] = ok ? __ldg(a.v_scale + at) : 0.f;
        }
      }
    };
    uint32_t vr[4][C::VW];
    auto load_v = [&](int gr, int id) {
      const int j = PAGED ? (gr * 16) & (a.page - 1) : gr * 16;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int kk = 2 * c + (e & 1) + 8 * (e >> 1);  // keys 2c, 2c+1, 2c+8, 2c+9
        const bool ok = id >= 0 && gr * 16 + kk < klim && SOLATTN_DCHECK_STATUS(key_inside(a, id, j + kk), a.status);
        const uint8_t *p = vbase + (id * a.v_seq + static_cast<long long>(j + kk) * a.v_row) * ES;
        if constexpr (C::VW == 8) {  // 16 bits, d = 128: two pieces 64 columns apart
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint4 x = ok ? ld_stream16(p + g * 16 + i * 128) : make_uint4(0, 0, 0, 0);
            vr[e][4 * i] = x.x, vr[e][4 * i + 1] = x.y, vr[e][4 * i + 2] = x.z, vr[e][4 * i + 3] = x.w;
          }
        } else if constexpr (C::VW == 4) {
          const uint4 x = ok ? ld_stream16(p + g * 16) : make_uint4(0, 0, 0, 0);
          vr[e][0] = x.x, vr[e][1] = x.y, vr[e][2] = x.z, vr[e][3] = x.w;
        } else {
          const uint2 x = ok ? ld_stream8(p + g * 8) : make_uint2(0, 0);
          vr[e][0] = x.x, vr[e][1] = x.y;
        }
      }
    };

    int gr = cur.u0 * (kUnitKeys / 16) + warp;
    int id = locate(gr), id_next = locate(gr + kRowsWarps);
    if (gr < gend) load_k(gr, id);
    for (; gr < gend; gr += kRowsWarps) {
      load_v(gr, id);
      // ---- S^T = K Q^T
      float sc[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
      if constexpr (KIND == kKind16) {
#pragma unroll
        for (int i = 0; i < C::KS; ++i)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            Type16<MT>::mma(sc[nt], kr[0][2 * i], kr[1][2 * i], kr[0][2 * i + 1], kr[1][2 * i + 1], qf[nt][i][0],
                            qf[nt][i][1]);
      } else {
#pragma unroll
        for (int i = 0; i < C::KS; ++i) {
          const uint32_t x0 = code_word<KIND>(kr[0][i]), x1 = code_word<KIND>(kr[1][i]);
          const uint32_t a0 = codes_f16x2<KIND, 0>(x0), a2 = codes_f16x2<KIND, 1>(x0);
          const uint32_t a1 = codes_f16x2<KIND, 0>(x1), a3 = codes_f16x2<KIND, 1>(x1);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) Type16<MT>::mma(sc[nt], a0, a1, a2, a3, qf[nt][i][0], qf[nt][i][1]);
        }
      }
      const float ks0 = ksc[0], ks1 = ksc[1], vs0 = vsc[0], vs1 = vsc[1];
      const int gr0 = gr;
      if (gr + kRowsWarps < gend) load_k(gr + kRowsWarps, id_next);
      id = id_next;
      id_next = locate(gr + 2 * kRowsWarps);
      // ---- scores in log2 units, masked
      bool grow = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float f = qscale[nt][e & 1];
          if constexpr (KIND != kKind16) f *= (e >> 1) ? ks1 : ks0;
          sc[nt][e] *= f;
        }
      }
      if (gr0 * 16 + 16 > kmin) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (gr0 * 16 + g + 8 * (e >> 1) >= lim[nt][e & 1]) sc[nt][e] = -CUDART_INF_F;
      }
      float lv0 = 0.f, lv1 = 0.f;
      if constexpr (KIND != kKind16) lv0 = log2_scale(vs0), lv1 = log2_scale(vs1);
      auto top = [&](int nt, int e) { return fmaxf(sc[nt][e] + lv0, sc[nt][e + 2] + lv1); };
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) grow |= top(nt, e) > m[nt][e] + kRowsSlack;
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float al[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = top(nt, e);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            al[e] = 1.f;
            if (mx > m[nt][e] + kRowsSlack) {
              if (m[nt][e] != -CUDART_INF_F) al[e] = ex2_approx(0.5f * (m[nt][e] - mx));
              m[nt][e] = mx;
            }
            l[nt][e] = l[nt][e] * al[e] * al[e];  // (the square may be below 2^-126 where l is above 2^100)
            al[e] *= al[e];
          }
#pragma unroll
          for (int i = 0; i < C::KS; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nt][i][e] *= al[e & 1];
        }
      }
      // ---- P^T, to the layout of the second product
      uint32_t pb[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float m0 = m[nt][0] == -CUDART_INF_F ? 0.f : m[nt][0], m1 = m[nt][1] == -CUDART_INF_F ? 0.f : m[nt][1];
        float p0 = ex2_approx(sc[nt][0] - m0), p1 = ex2_approx(sc[nt][1] - m1);
        float p2 = ex2_approx(sc[nt][2] - m0), p3 = ex2_approx(sc[nt][3] - m1);
        l[nt][0] += p0 + p2;
        l[nt][1] += p1 + p3;
        if constexpr (KIND != kKind16) p0 *= vs0, p1 *= vs0, p2 *= vs1, p3 *= vs1;
        pb[nt][0] = transpose8(pack16<MT>(p0, p1));
        pb[nt][1] = transpose8(pack16<MT>(p2, p3));
      }
      // ---- O^T += V^T P^T; m tile i, row g and row g + 8 are the columns col(i, 0) and col(i, 1) below
#pragma unroll
      for (int i = 0; i < C::KS; ++i) {
        uint32_t a0, a1, a2, a3;
        if constexpr (KIND == kKind16) {
          if constexpr (D == 128) {
            const uint32_t sel = (i & 1) ? 0x7632u : 0x5410u;
            a0 = prmt(vr[0][i >> 1], vr[1][i >> 1], sel);
            a1 = prmt(vr[0][4 + (i >> 1)], vr[1][4 + (i >> 1)], sel);
            a2 = prmt(vr[2][i >> 1], vr[3][i >> 1], sel);
            a3 = prmt(vr[2][4 + (i >> 1)], vr[3][4 + (i >> 1)], sel);
          } else {
            a0 = prmt(vr[0][i], vr[1][i], 0x5410u);
            a1 = prmt(vr[0][i], vr[1][i], 0x7632u);
            a2 = prmt(vr[2][i], vr[3][i], 0x5410u);
            a3 = prmt(vr[2][i], vr[3][i], 0x7632u);
          }
        } else {
          // bytes 2 (i & 1), 2 (i & 1) + 1 of word i / 2, paired over the two keys
          const uint32_t sel = (i & 1) ? 0x7362u : 0x5140u;
          const uint32_t x = code_word<KIND>(prmt(vr[0][i >> 1], vr[1][i >> 1], sel));
          const uint32_t y = code_word<KIND>(prmt(vr[2][i >> 1], vr[3][i >> 1], sel));
          a0 = codes_f16x2<KIND, 0>(x), a1 = codes_f16x2<KIND, 1>(x);
          a2 = codes_f16x2<KIND, 0>(y), a3 = codes_f16x2<KIND, 1>(y);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) Type16<MT>::mma(o[nt][i], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
      }
    }

    // ---- join the warps
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = l[nt][e];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        if (g == 0) {
          sm.m[warp][nt * 8 + 2 * c + e] = m[nt][e];
          sm.l[warp][nt * 8 + 2 * c + e] = x;
        }
      }
#pragma unroll
      for (int i = 0; i < C::KS; ++i) {
        // columns of m tile i: 16-bit d = 128 pairs columns 64 apart, the others neighbours
        const int d0 = (KIND == kKind16 && D == 128) ? g * 8 + i : g * (D / 8) + 2 * i;
        const int d1 = (KIND == kKind16 && D == 128) ? d0 + 64 : d0 + 1;
        sm.o[warp][nt * 8 + 2 * c][d0] = o[nt][i][0];
        sm.o[warp][nt * 8 + 2 * c + 1][d0] = o[nt][i][1];
        sm.o[warp][nt * 8 + 2 * c][d1] = o[nt][i][2];
        sm.o[warp][nt * 8 + 2 * c + 1][d1] = o[nt][i][3];
      }
    }
    __syncthreads();
    constexpr int TPR = D / 4;
    const int e = threadIdx.x % TPR;
    const int slot = cur.slot(blockIdx.x);
    for (int r = threadIdx.x / TPR; r < C::ROWS; r += kRowsWarps * 32 / TPR) {
      int tok, gg;
      if (!T::row(a, s.n, t, r, tok, gg)) continue;
      if (!SOLATTN_DCHECK_STATUS(row_inside(a, b, s.tok0 + tok, h * a.G + gg) && slot_inside(slot, gridDim.x), a.status)) continue;
      float mm = -CUDART_INF_F;
#pragma unroll
      for (int w = 0; w < kRowsWarps; ++w) mm = fmaxf(mm, sm.m[w][r]);
      const float ms = mm == -CUDART_INF_F ? 0.f : mm;
      float ll = 0.f, x0 = 0.f, x1 = 0.f, x2 = 0.f, x3 = 0.f;
#pragma unroll
      for (int w = 0; w < kRowsWarps; ++w) {
        const float root = ex2_approx(0.5f * (sm.m[w][r] - ms)), f = root * root;
        ll = fmaf(root, root * sm.l[w][r], ll);
        const float4 y = *reinterpret_cast<const float4 *>(&sm.o[w][r][4 * e]);
        x0 = fmaf(f, y.x, x0);
        x1 = fmaf(f, y.y, x1);
        x2 = fmaf(f, y.z, x2);
        x3 = fmaf(f, y.w, x3);
      }
      if (cur.partial()) {
        if (e == 0) {
          a.part_ml[static_cast<size_t>(slot) * 2 * C::ROWS + r] = mm;
          a.part_ml[static_cast<size_t>(slot) * 2 * C::ROWS + C::ROWS + r] = ll;
        }
        *reinterpret_cast<float4 *>(a.part_o + (static_cast<size_t>(slot) * C::ROWS + r) * D + 4 * e) =
            make_float4(x0, x1, x2, x3);
      } else {
        const float inv = ll == 0.f ? 0.f : 1.f / ll;  // a row that sees no key is zero
        QT *dst = static_cast<QT *>(a.out) + b * a.o_batch + static_cast<long long>(s.tok0 + tok) * a.o_tok +
                  static_cast<long long>(h * a.G + gg) * a.o_head + 4 * e;
        *reinterpret_cast<uint2 *>(dst) = make_uint2(pack16<QT>(x0 * inv, x1 * inv), pack16<QT>(x2 * inv, x3 * inv));
      }
    }
    if (cur.partial() && cur.u0 == 0) rec = cur.record(blockIdx.x);
    __syncthreads();  // the buffers serve the next segment
  }
  if (threadIdx.x == 0) a.desc[blockIdx.x] = rec;
}

}  // namespace solattn
