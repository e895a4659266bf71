// tile_kernel.cuh -- dense attention for many query rows of a key head: tcgen05 with the
// accumulators in tensor memory.
//
// A block per SM walks its range of the work line. A tile is 256 query rows, two halves of
// 128; K and V come in units of 128 keys and serve both halves, so a key tile crosses L2
// once per 256 rows. Roles, by warp:
//   warp 0       16-bit keys: TMA producer. Q halves into three buffers (the next item's first half
//                lands while this item runs), K and V units into a ring.
//   warps 1, 3   MMA issuers, one thread for each half: S = Q K^T into tensor memory, O += P V with
//                P read from tensor memory. They take turns through a shared counter, as the
//                issuers of the sparse kernel do, so the tensor core works on one half while the
//                other half's softmax runs.
//   warp 2       owns the TMEM allocation; walks the block's range of the line and publishes its
//                segments (one tile's run of units) to the other roles, a few ahead.
//   warps 4-11   softmax, one warpgroup for each half, one row per thread. Where a sequence ends inside a
//                unit they zero the value rows behind the end, which may hold anything (0 times NaN is NaN).
//   warps 12-15  8-bit keys only: read codes from the pages, expand them to fp16 into the ring (and the
//                queries, scaled, into their buffers), one unit ahead in registers.
// S and P of a half share their columns: S(u+1) is computed after P V(u) has read P(u).
//
// Softmax: once a row has a reference maximum a unit is exponentiated against it without taking the row
// maximum; a row sum <= 2^15 shows that no value is large, otherwise (or for a row's first
// unit) the maximum is taken and the unit done again. P is rounded to the 16-bit type of the
// keys (bf16: half a step of 2^-9 on average; independent from key to key, so the output's
// own rounding is what remains; fp16 for 8-bit caches). The reference, sums and O are in 32 bits.
// One pair of exponentials in kTilePolyEvery goes through the polynomial on the FMA pipe;
// a unit that is done again uses the special-function unit only, which hands NaN through.
//
// Causal and ragged ends: columns at or behind a row's limit are replaced by -infinity; the
// products of a unit stop at the last 16 keys that some row of the tile sees.
#pragma once

#include "dense_common.cuh"
#include "rows_kernel.cuh"

namespace solattn {

constexpr float kTileSlack = 8.0f;         // log2 units the reference may lag a unit's maximum
constexpr float kTileSumLimit = 32768.0f;  // row sum that shows every value <= 2^15
constexpr uint32_t kTilePolyMask = 0x80u;  // pairs (mod 8) on the polynomial

template <class QT_, int KIND_, int D_, bool PAGED_>
struct TileCfg {
  using QT = QT_;
  static constexpr int KIND = KIND_, D = D_;
  static constexpr bool PAGED = PAGED_;
  static constexpr bool BITS8 = KIND != kKind16;
  using MT = typename std::conditional<BITS8, __half, QT>::type;  // operands' type
  static constexpr int PANELS = D / 64;
  static constexpr int HALF_BYTES = 128 * D * 2;  // a half's queries, or a unit of K or V
  // 224 KB of tiles at d = 128: 3 + 4 (16-bit), 2 + 4 (8-bit, which also keeps scales)
  static constexpr int NQ = BITS8 ? 2 : 3;
  static constexpr int NSLOT = D == 128 ? 4 : 8;
  static constexpr int NSC = 4;  // units whose scales are kept
  static constexpr int COLS = 128 + D;  // tensor memory columns of a half: S (and P), O
  static constexpr int TMEM_COLS = 2 * COLS <= 256 ? 256 : 512;
  static constexpr int THREADS = BITS8 ? 512 : 384;
  // Register shares: within what the block is launched with (384 x 168, 512 x 128).
  static constexpr int CTRL_REGS = BITS8 ? 80 : 104;
  static constexpr int CONV_REGS = 112;
  static constexpr int SOFTMAX_REGS = BITS8 ? 160 : 200;
  static_assert(BITS8 ? 128 * CTRL_REGS + 128 * CONV_REGS + 256 * SOFTMAX_REGS <= 512 * 128
                      : 128 * CTRL_REGS + 256 * SOFTMAX_REGS <= 384 * 168, "register split");
  static constexpr bool FP16 = std::is_same<MT, __half>::value;
  static constexpr uint32_t IDESC_PV = idesc_16bit_f32(128, D, true, FP16);
};

constexpr int kSegs = 4;  // segments published ahead

// A segment of the block's range: units u0 .. u1 - 1 of one tile.
struct Segment {
  int n, u0, klim, L;   // units (0: no more work), first unit, keys that some row sees, keys
  int tok, end;         // the tile's first query row in Q and out, and its sequence's end there
  int b, h, lim0;       // lim0: keys that the tile's first token sees
  int part;             // workspace slot of a partial result, or -1
};

template <class C>
struct TileCtl {
  Segment seg[kSegs];
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  uint64_t full[C::NSLOT], empty[C::NSLOT];
  uint64_t q_full[C::NQ], q_empty[C::NQ];
  uint64_t s_full[2], p_full[2], o_full[2], o_empty[2];
  uint64_t conv;  // the converter's four warps
  uint64_t mma_done[2];
  uint32_t turn;
  uint32_t tmem_base;
  int abort_flag;
  float wmax[2][4];              // converter: largest value scale per warp
  alignas(16) float ks[C::BITS8 ? C::NSC : 1][C::BITS8 ? 128 : 4];  // key scales (x log2(e) / sqrt d)
  alignas(16) float vs[C::BITS8 ? C::NSC : 1][C::BITS8 ? 128 : 4];  // value scales over the reference
  float vgrow[C::NSC], vref[C::NSC];  // factor of O when the reference grew, and the reference
  alignas(16) float qdown[C::BITS8 ? C::NQ : 1][C::BITS8 ? 128 : 4];  // what a query row was divided by
};

template <class C>
constexpr size_t tile_smem_bytes() {
  return 1024 + static_cast<size_t>(C::NQ + C::NSLOT) * C::HALF_BYTES + sizeof(TileCtl<C>);
}

__device__ __forceinline__ void tma_load_4d_hint(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1,
                                                 int c2, int c3, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tma_load_5d_hint(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1,
                                                 int c2, int c3, int c4, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2], %8;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void tile_abort(int *abort_flag, int *status) {
  atomicCAS(status, 0, -4);  // SOLATTN_ETIMEOUT
  *reinterpret_cast<volatile int *>(abort_flag) = 1;
}

// Extra arguments of the tile kernel.
struct TileArgs {
  int k_b, k_h, v_b, v_h;  // 0: the batch (head) stride is zero, and so is the coordinate
  int min_units, whole_items;
};

// Steps of 16 keys that a unit's products need: some row of the tile sees a key in each.
__device__ __forceinline__ int unit_steps(int klim, int u) { return min(8, max(1, (klim - u * kUnitKeys + 15) >> 4)); }
// Whether value rows of the unit's last step lie behind the sequence's end.
__device__ __forceinline__ bool unit_ragged(int L, int klim, int u) {
  return L < u * kUnitKeys + 16 * unit_steps(klim, u);
}

// ------------------------------------------------------------------ segments

template <class C>
__device__ void tile_scheduler(TileCtl<C> &sc, const DenseArgs &a, const TileArgs &x, int lane) {
  Cursor<TokenTiles> cur;
  bool more = cur.begin(a, blockIdx.x, gridDim.x, x.min_units, x.whole_items);
  if (lane != 0) return;
  int4 rec = make_int4(0, 0, 0, 0);
  for (uint32_t i = 0;; ++i) {
    const int sl = i % kSegs;
    if (!mbar_wait(&sc.seg_empty[sl], ((i / kSegs) & 1) ^ 1, a.timeout_ns, &sc.abort_flag)) {
      tile_abort(&sc.abort_flag, a.status);
      break;
    }
    Segment g{};
    if (more) {
      const Seq &s = cur.s;
      g.n = cur.u1 - cur.u0;
      g.u0 = cur.u0;
      g.klim = key_limit(a, s, TokenTiles::last_token(a, s.n, cur.t));
      g.L = s.L;
      g.tok = s.tok0 + cur.t * a.tile_tokens;
      g.end = s.tok0 + s.n;
      g.b = cur.b;
      g.h = cur.h;
      // causal: token i of the tile sees lim0 + i keys (cut to 0 .. L)
      g.lim0 = a.causal ? s.L - s.n + cur.t * a.tile_tokens + 1 : s.L;
      g.part = cur.partial() ? cur.slot(blockIdx.x) : -1;
      if (cur.partial() && cur.u0 == 0) rec = cur.record(blockIdx.x);
    }
    sc.seg[sl] = g;
    mbar_arrive(&sc.seg_full[sl]);
    if (!more) break;
    more = cur.step(a);
  }
  a.desc[blockIdx.x] = *reinterpret_cast<volatile int *>(&sc.abort_flag) ? make_int4(0, 0, 0, 0) : rec;
}

// A role's walk over the segments.
template <class C>
struct SegmentReader {
  uint32_t i = 0;
  // The next segment, or null at the end (or when a wait gave up: ok is cleared).
  __device__ __forceinline__ const Segment *next(TileCtl<C> &sc, const DenseArgs &a, bool &ok) {
    const int sl = i % kSegs;
    if (!mbar_wait(&sc.seg_full[sl], (i / kSegs) & 1, a.timeout_ns, &sc.abort_flag)) {
      ok = false;
      return nullptr;
    }
    ++i;
    return sc.seg[sl].n ? &sc.seg[sl] : nullptr;
  }
  __device__ __forceinline__ const Segment *next_warp(TileCtl<C> &sc, const DenseArgs &a, bool &ok) {
    const int sl = i % kSegs;
    if (!__all_sync(0xffffffffu, mbar_wait(&sc.seg_full[sl], (i / kSegs) & 1, a.timeout_ns, &sc.abort_flag))) {
      ok = false;
      return nullptr;
    }
    ++i;
    return sc.seg[sl].n ? &sc.seg[sl] : nullptr;
  }
  __device__ __forceinline__ void done(TileCtl<C> &sc) { mbar_arrive(&sc.seg_empty[(i - 1) % kSegs]); }
};

// Token (from the tile's first) and head of the group of row r of a half; whether the row is used.
__device__ __forceinline__ bool half_row(const DenseArgs &a, const Segment &g, int w, int r, int &tok, int &hg) {
  const int half = a.tile_tokens >> 1;
  const int i = r / a.G;
  hg = r - i * a.G;
  tok = w * half + i;
  return i < half && g.tok + tok < g.end;
}

// ------------------------------------------------------------------ TMA producer (16-bit keys)

template <class C>
__device__ void tile_producer(TileCtl<C> &sc, const DenseArgs &a, const TileArgs &x, uint8_t *q_smem, uint8_t *ring, const CUtensorMap *tm_q, const CUtensorMap *tm_k, const CUtensorMap *tm_v) {
  const volatile int *ab = &sc.abort_flag;
  const uint64_t pol_stream = l2_policy_evict_first(), pol_reuse = l2_policy_evict_last();
  const int half = a.tile_tokens >> 1;
  const uint32_t q_bytes = static_cast<uint32_t>(half) * a.G * 128;  // of a panel
  uint32_t kv = 0, qi = 0;
  bool ok = true;
  SegmentReader<C> rd;
  while (const Segment *g = ok ? rd.next(sc, a, ok) : nullptr) {
    const int b = g->b, h = g->h, L = g->L, tok0 = g->tok, u0 = g->u0, u1 = u0 + g->n;
    rd.done(sc);
    auto load_q = [&](int w) {
      const int sl = qi % C::NQ;
      if (!mbar_wait(&sc.q_empty[sl], ((qi / C::NQ) & 1) ^ 1, a.timeout_ns, ab)) return false;
      mbar_arrive_expect_tx(&sc.q_full[sl], q_bytes * C::PANELS);
      const int tok = tok0 + w * half;
#pragma unroll
      for (int pn = 0; pn < C::PANELS; ++pn)
        tma_load_5d_hint(smem_u32(q_smem + sl * C::HALF_BYTES + pn * (128 * 128)), tm_q, smem_u32(&sc.q_full[sl]), pn * 64, 0,
                         tok, h, a.cu ? 0 : b, pol_stream);
      ++qi;
      return true;
    };
    auto load_kv = [&](int u, bool is_v) {
      const int sl = kv % C::NSLOT;
      if (!mbar_wait(&sc.empty[sl], ((kv / C::NSLOT) & 1) ^ 1, a.timeout_ns, ab)) return false;
      mbar_arrive_expect_tx(&sc.full[sl], C::HALF_BYTES);
      const CUtensorMap *map = is_v ? tm_v : tm_k;
      uint8_t *dst = ring + sl * C::HALF_BYTES;
      if constexpr (C::PAGED) {
        for (int r = 0; r < kUnitKeys; r += a.page) {
          const int j = u * kUnitKeys + r;
          // keys behind the end, and bad table entries, lie outside the map: they read as zeros
          int id = -1;
          if (j < L) id = page_of(a, b, j);
          if (id < 0) id = a.num_pages;
#pragma unroll
          for (int pn = 0; pn < C::PANELS; ++pn)
            tma_load_4d_hint(smem_u32(dst + pn * (128 * 128) + r * 128), map, smem_u32(&sc.full[sl]), pn * 64, 0, h, id, pol_reuse);
        }
      } else {
#pragma unroll
        for (int pn = 0; pn < C::PANELS; ++pn)
          tma_load_4d_hint(smem_u32(dst + pn * (128 * 128)), map, smem_u32(&sc.full[sl]), pn * 64, u * kUnitKeys,
                           h * (is_v ? x.v_h : x.k_h), b * (is_v ? x.v_b : x.k_b), pol_reuse);
      }
      ++kv;
      return true;
    };
    ok = load_q(0) && load_kv(u0, false) && load_q(1);
    for (int u = u0; u < u1 && ok; ++u) {
      ok = load_kv(u, true);
      if (ok && u + 1 < u1) ok = load_kv(u + 1, false);
    }
  }
  if (!ok) tile_abort(&sc.abort_flag, a.status);
  // No copy may outlive the block: wait (bounded) for the last fill of every buffer.
  const int zero = 0;
  for (uint32_t f = kv > C::NSLOT ? kv - C::NSLOT : 0; f < kv; ++f)
    mbar_wait(&sc.full[f % C::NSLOT], (f / C::NSLOT) & 1, a.timeout_ns, &zero);
  for (uint32_t f = qi > C::NQ ? qi - C::NQ : 0; f < qi; ++f)
    mbar_wait(&sc.q_full[f % C::NQ], (f / C::NQ) & 1, a.timeout_ns, &zero);
}

// ------------------------------------------------------------------ converter (8-bit keys)

// Byte offset of 16-byte chunk ch (0 .. D/8 - 1) of row r in a tile of 128-byte-swizzled panels.
__device__ __forceinline__ uint32_t swz(int r, int ch) {
  return static_cast<uint32_t>((ch >> 3) * (128 * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
}

template <class C>
__device__ void tile_converter(TileCtl<C> &sc, const DenseArgs &a, uint8_t *q_smem, uint8_t *ring) {
  constexpr int D = C::D, LPR = D / 16;    // lanes of a row of codes
  constexpr int RPP = 128 / LPR;           // rows of a pass of the four warps
  constexpr int NP = 128 / RPP;            // passes of a unit
  const volatile int *ab = &sc.abort_flag;
  const int tid = threadIdx.x & 127, warp = tid >> 5, lane = tid & 31;
  const int rl = tid / LPR, pc = tid % LPR;
  uint32_t kv = 0, qi = 0, tile = 0;
  bool ok = true;
  auto wait = [&](uint64_t *bar, uint32_t par) {
    bool w = mbar_wait(bar, par, a.timeout_ns, ab);
    w = __all_sync(0xffffffffu, w);
    if (!w) ok = false;
    return w;
  };
  uint4 cd[NP];
  float ksc, vsc;
  // Codes of a unit's keys or values into registers.
  auto fetch = [&](const Segment &c, int u, bool is_v) {
    const uint8_t *base = static_cast<const uint8_t *>(is_v ? a.v : a.k) + c.h * (is_v ? a.v_head : a.k_head) + pc * 16;
    const long long row = is_v ? a.v_row : a.k_row, seq = is_v ? a.v_seq : a.k_seq;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int j = u * kUnitKeys + i * RPP + rl;
      int id = -1;
      if (j < c.L) id = page_of(a, c.b, j);
      cd[i] = id >= 0 ? ld_stream16(base + id * seq + (j & (a.page - 1)) * row) : make_uint4(0, 0, 0, 0);
    }
  };
  // The scales of a unit: thread t takes key t.
  auto fetch_scales = [&](const Segment &c, int u) {
    const int j = u * kUnitKeys + tid;
    int id = -1;
    if (j < c.L) id = page_of(a, c.b, j);
    const size_t at = (static_cast<size_t>(max(id, 0)) * a.Hkv + c.h) * a.page + (j & (a.page - 1));
    ksc = id >= 0 ? __ldg(a.k_scale + at) : 0.f;
    vsc = id >= 0 ? __ldg(a.v_scale + at) : 0.f;
  };
  auto expand = [&](uint8_t *dst) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int r = i * RPP + rl;
      uint32_t w[8];
      const uint32_t cw[4] = {cd[i].x, cd[i].y, cd[i].z, cd[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t t = code_word<C::KIND>(cw[e]);
        w[2 * e] = codes_f16x2<C::KIND, 0>(t);
        w[2 * e + 1] = codes_f16x2<C::KIND, 1>(t);
      }
      // lanes of the two panels write their two chunks in opposite order: no bank conflict
      const bool swap = pc >= 4;
      const uint32_t first = swz(r, 2 * pc + (swap ? 1 : 0)), second = swz(r, 2 * pc + (swap ? 0 : 1));
      const uint4 lo = make_uint4(w[0], w[1], w[2], w[3]), hi = make_uint4(w[4], w[5], w[6], w[7]);
      *reinterpret_cast<uint4 *>(dst + first) = swap ? hi : lo;
      *reinterpret_cast<uint4 *>(dst + second) = swap ? lo : hi;
    }
  };
  auto publish = [&](uint64_t *bar) {
    fence_proxy_async();
    mbar_arrive(bar);  // 128 arrivals
  };
  SegmentReader<C> rd;
  const Segment *g = rd.next_warp(sc, a, ok);
  if (g) {
    fetch(*g, g->u0, false);
    fetch_scales(*g, g->u0);
  }
  while (g) {
    // ---- queries of both halves, a row per thread, scaled to fp16
    for (int w = 0; w < 2 && ok; ++w) {
      const int sl = qi % C::NQ;
      if (!wait(&sc.q_empty[sl], ((qi / C::NQ) & 1) ^ 1)) break;
      int tok, hg;
      const bool row_ok = half_row(a, *g, w, tid, tok, hg);
      const typename C::QT *src = static_cast<const typename C::QT *>(a.q) + static_cast<long long>(g->tok + tok) * a.q_tok +
                                  static_cast<long long>(g->h * a.G + hg) * a.q_head;
      uint8_t *dst = q_smem + sl * C::HALF_BYTES;
      float down = 1.f, up = 1.f;
      if constexpr (std::is_same<typename C::QT, __nv_bfloat16>::value) {
        uint32_t big = 0;
#pragma unroll 4
        for (int i = 0; i < D / 8; ++i) {
          const uint4 v = row_ok ? __ldg(reinterpret_cast<const uint4 *>(src) + i) : make_uint4(0, 0, 0, 0);
          const uint32_t vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) big = max(big, max(vv[e] & 0x7fffu, (vv[e] >> 16) & 0x7fffu));
        }
        const int ex = static_cast<int>(big >> 7);
        const int sh = (ex == 0 || ex == 255) ? 0 : min(max(141 - ex, -126), 126);
        up = __int_as_float((127 + sh) << 23);
        down = __int_as_float((127 - sh) << 23);
      }
#pragma unroll 4
      for (int i = 0; i < D / 8; ++i) {
        uint4 v = row_ok ? __ldg(reinterpret_cast<const uint4 *>(src) + i) : make_uint4(0, 0, 0, 0);
        if constexpr (std::is_same<typename C::QT, __nv_bfloat16>::value) {
          v.x = pack_f16x2(__uint_as_float(v.x << 16) * up, __uint_as_float(v.x & 0xffff0000u) * up);
          v.y = pack_f16x2(__uint_as_float(v.y << 16) * up, __uint_as_float(v.y & 0xffff0000u) * up);
          v.z = pack_f16x2(__uint_as_float(v.z << 16) * up, __uint_as_float(v.z & 0xffff0000u) * up);
          v.w = pack_f16x2(__uint_as_float(v.w << 16) * up, __uint_as_float(v.w & 0xffff0000u) * up);
        }
        *reinterpret_cast<uint4 *>(dst + swz(tid, i)) = v;
      }
      sc.qdown[sl][tid] = down;
      publish(&sc.q_full[sl]);
      ++qi;
    }
    if (!ok) break;
    // ---- units: K u, then V u, each with the next piece's codes on their way
    float vref = 0.f;
    const Segment *nxt = nullptr;
    const int u1 = g->u0 + g->n;
    for (int u = g->u0; u < u1 && ok; ++u) {
      int sl = kv % C::NSLOT;
      if (!wait(&sc.empty[sl], ((kv / C::NSLOT) & 1) ^ 1)) break;
      // scales: the reference is a power of two >= the largest value scale so far (2^-100 .. 2^100)
      float mx = vsc;
#pragma unroll
      for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      if (lane == 0) {
        sc.wmax[tile & 1][warp] = mx;
        mbar_arrive(&sc.conv);
      }
      if (!wait(&sc.conv, tile & 1)) break;
      mx = fmaxf(fmaxf(sc.wmax[tile & 1][0], sc.wmax[tile & 1][1]), fmaxf(sc.wmax[tile & 1][2], sc.wmax[tile & 1][3]));
      float growth = 1.f;
      if (mx > vref) {
        const int ex = min(max((__float_as_int(mx) >> 23) + 1, 27), 227);
        const float vnew = __int_as_float(ex << 23);
        growth = vref * __int_as_float((254 - ex) << 23);
        vref = vnew;
      }
      const int ss = tile % C::NSC;
      sc.ks[ss][tid] = ksc * a.scale_log2;
      sc.vs[ss][tid] = vref > 0.f ? vsc * __int_as_float((254 << 23) - __float_as_int(vref)) : vsc;
      if (tid == 0) sc.vgrow[ss] = growth, sc.vref[ss] = vref;
      ++tile;
      expand(ring + sl * C::HALF_BYTES);
      fetch(*g, u, true);
      publish(&sc.full[sl]);
      ++kv;
      sl = kv % C::NSLOT;
      if (!wait(&sc.empty[sl], ((kv / C::NSLOT) & 1) ^ 1)) break;
      expand(ring + sl * C::HALF_BYTES);
      if (u + 1 < u1) {
        fetch(*g, u + 1, false);
        fetch_scales(*g, u + 1);
      } else {
        rd.done(sc);
        nxt = rd.next_warp(sc, a, ok);
        if (nxt) {
          fetch(*nxt, nxt->u0, false);
          fetch_scales(*nxt, nxt->u0);
        }
      }
      publish(&sc.full[sl]);
      ++kv;
    }
    if (!ok) break;
    g = nxt;
  }
  if (!ok && lane == 0) tile_abort(&sc.abort_flag, a.status);
}

// ------------------------------------------------------------------ MMA issuers

template <class C>
__device__ void tile_mma(TileCtl<C> &sc, const DenseArgs &a, uint32_t tmem, uint8_t *q_smem, uint8_t *ring, int w) {
  const volatile int *ab = &sc.abort_flag;
  volatile uint32_t *turn = &sc.turn;
  const uint64_t q_desc0 = smem_desc_sw128(smem_u32(q_smem), 16, 1024);
  const uint64_t k_desc0 = smem_desc_sw128(smem_u32(ring), 16, 1024);
  const uint64_t v_desc0 = smem_desc_sw128(smem_u32(ring), 128 * 128, 1024);
  constexpr uint32_t kUnits = C::HALF_BYTES / 16;
  const uint32_t s_tmem = tmem + w * C::COLS, o_tmem = s_tmem + 128;
  uint32_t kv = 0, qi = 0, p_ph = 0, g = 0, o_ph = 0;
  bool ok = true;
  auto wait = [&](uint64_t *bar, uint32_t par) {
    if (!ok) return false;
    if (!mbar_wait(bar, par, a.timeout_ns, ab)) ok = false;
    else tc_fence_after_sync();
    return ok;
  };
  auto take = [&](uint32_t target) {
    if (*turn == target) return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t it = 1;; ++it) {
      if (*turn == target) return true;
      if ((it & 255u) == 0u && (*ab || global_timer_ns() - t0 > a.timeout_ns)) {
        ok = false;
        return false;
      }
    }
  };
  SegmentReader<C> rd;
  while (const Segment *sg = ok ? rd.next(sc, a, ok) : nullptr) {
    const int n = sg->n, klim = sg->klim, u0 = sg->u0;
    rd.done(sc);
    const uint32_t qe = qi + w;
    qi += 2;
    if (!wait(&sc.q_full[qe % C::NQ], (qe / C::NQ) & 1)) break;
    const uint64_t q_desc = q_desc0 + (qe % C::NQ) * kUnits;
    auto issue_qk = [&](int i) {
      const uint64_t kd = k_desc0 + ((kv + 2 * i) % C::NSLOT) * kUnits;
      const uint32_t idesc = idesc_16bit_f32(128, 16 * unit_steps(klim, u0 + i), false, C::FP16);
#pragma unroll
      for (int kk = 0; kk < C::D / 16; ++kk) {
        const uint64_t off = static_cast<uint64_t>((kk >> 2) * (128 * 128 / 16) + (kk & 3) * 2);
        mma_bf16_ss(s_tmem, q_desc + off, kd + off, idesc, kk > 0 ? 1u : 0u);
      }
      tc_commit(&sc.s_full[w]);
    };
    auto wait_entry = [&](uint32_t e) { return wait(&sc.full[e % C::NSLOT], (e / C::NSLOT) & 1); };
    if (!wait_entry(kv) || !take(g + w)) break;
    issue_qk(0);
    *turn = g + w + 1;
    for (int i = 0; i < n && ok; ++i) {
      if (!wait_entry(kv + 2 * i + 1)) break;
      if (i + 1 < n && !wait_entry(kv + 2 * i + 2)) break;
      if (i == 0 && !wait(&sc.o_empty[w], o_ph ^ 1)) break;
      if (!wait(&sc.p_full[w], p_ph)) break;
      p_ph ^= 1;
      const uint32_t my = g + 2 + 2 * i + w;
      if (!take(my)) break;
      const uint64_t vd = v_desc0 + ((kv + 2 * i + 1) % C::NSLOT) * kUnits;
      const int steps = unit_steps(klim, u0 + i);
      if (steps == 8) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_bf16_ts(o_tmem, s_tmem + kk * 8, vd + static_cast<uint64_t>(kk * (16 * 128 / 16)), C::IDESC_PV, (i > 0 || kk > 0) ? 1u : 0u);
      } else {
        for (int kk = 0; kk < steps; ++kk)
          mma_bf16_ts(o_tmem, s_tmem + kk * 8, vd + static_cast<uint64_t>(kk * (16 * 128 / 16)), C::IDESC_PV, (i > 0 || kk > 0) ? 1u : 0u);
      }
      if (i + 1 < n) issue_qk(i + 1);
      else tc_commit(&sc.o_full[w]);
      *turn = my + 1;
    }
    if (!ok) break;
    o_ph ^= 1;
    kv += 2 * n;
    g += 2 + 2 * n;
  }
  if (!ok) tile_abort(&sc.abort_flag, a.status);
  // Every tcgen05 operation issued here must finish before TMEM is released.
  const int zero = 0;
  tc_commit(&sc.mma_done[w]);
  mbar_wait(&sc.mma_done[w], 0, a.timeout_ns, &zero);
}

// ------------------------------------------------------------------ softmax and epilogue

template <class C>
__device__ void tile_softmax(TileCtl<C> &sc, const DenseArgs &a, uint32_t tmem, uint8_t *q_smem, uint8_t *ring, int w, int warp,
                             int lane) {
  constexpr int D = C::D;
  using QT = typename C::QT;
  using MT = typename C::MT;
  const volatile int *ab = &sc.abort_flag;
  const int wq = warp & 3, row = wq * 32 + lane;
  const uint32_t s_addr = tmem + (static_cast<uint32_t>(wq * 32) << 16) + w * C::COLS;
  const uint32_t o_addr = s_addr + 128;
  const bool leader = (threadIdx.x & 127) == 0;
  const uint64_t pol_out = l2_policy_evict_first();
  uint32_t kv = 0, qi = 0, tile = 0, s_ph = 0, o_ph = 0;
  bool ok = true;
  auto wait = [&](uint64_t *bar, uint32_t par) {
    bool x = mbar_wait(bar, par, a.timeout_ns, ab);
    x = __all_sync(0xffffffffu, x);
    if (!x) ok = false;
    else tc_fence_after_sync();
    return x;
  };
  auto release = [&](uint32_t e) { mbar_arrive(&sc.empty[e % C::NSLOT]); };
  SegmentReader<C> rd;
  while (const Segment *sg = ok ? rd.next_warp(sc, a, ok) : nullptr) {
    const int n = sg->n;
    int lim;
    {
      int tok, hg;
      const bool row_ok = half_row(a, *sg, w, row, tok, hg);
      lim = row_ok ? (a.causal ? min(max(sg->lim0 + tok, 0), sg->L) : sg->L) : sg->klim;
    }
    const uint32_t qe = qi + w;
    qi += 2;
    float m_ref = -CUDART_INF_F, l = 0.f, vref = 0.f, down = 1.f;
    for (int i = 0; i < n; ++i, ++tile) {
      if (!wait(&sc.s_full[w], s_ph)) break;
      s_ph ^= 1;
      if constexpr (C::BITS8) {  // the converter's scales (complete: the product above used the same buffers)
        const uint32_t ke = kv + 2 * i;
        if (!wait(&sc.full[ke % C::NSLOT], (ke / C::NSLOT) & 1)) break;
        if (i == 0) {
          if (!wait(&sc.q_full[qe % C::NQ], (qe / C::NQ) & 1)) break;
          down = sc.qdown[qe % C::NQ][row];
        }
      }
      // The group that produced this S is complete: K of this unit and V of the one before have
      // been read by this half, and after the last S its queries.
      if (leader) {
        release(kv + 2 * i);
        if (i > 0) release(kv + 2 * i - 1);
      }
      // (a complete tile keeps its queries' buffer for its output)
      if (i == n - 1 && sg->part >= 0 && lane == 0) mbar_arrive(&sc.q_empty[qe % C::NQ]);
      const int base = (sg->u0 + i) * kUnitKeys, klim = sg->klim;
      const int left = lim - base;  // keys of this unit that the row sees
      const bool plain = __all_sync(0xffffffffu, left >= kUnitKeys);
      const int nch = (16 * unit_steps(klim, sg->u0 + i) + 31) >> 5;  // 32-column chunks in use
      float alpha = 1.f, lsum = 0.f;
      const int ss = tile % C::NSC;
      // Exponentials of one 32-column chunk (v: scores) against -neg_m, to P; row sums into acc.
      auto exp_chunk = [&](const uint32_t *v, int c, uint64_t scp, uint64_t nmp, uint64_t(&acc)[4], auto poly_tag) {
        constexpr bool POLY = decltype(poly_tag)::value;
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const uint64_t xx = fma2(f2(u2f_(v[2 * e]), u2f_(v[2 * e + 1])), scp, nmp);
          float x0, x1, p0, p1;
          f2_split(xx, x0, x1);
          if (POLY && ((kTilePolyMask >> (e % 8)) & 1u)) {
            exp2_poly_nan_x2(x0, x1, p0, p1);
          } else {
            p0 = ex2_approx(x0);
            p1 = ex2_approx(x1);
          }
          acc[e & 3] = add2(acc[e & 3], f2(p0, p1));
          if constexpr (C::BITS8) {
            const float2 vv = *reinterpret_cast<const float2 *>(&sc.vs[ss][c * 32 + 2 * e]);
            p0 *= vv.x, p1 *= vv.y;
          }
          pk[e] = pack16<MT>(p0, p1);
        }
        tmem_st16(s_addr + c * 16, pk);
      };
      auto total = [&](const uint64_t(&acc)[4]) {
        float t0, t1, t2, t3, t4, t5, t6, t7;
        f2_split(acc[0], t0, t1);
        f2_split(acc[1], t2, t3);
        f2_split(acc[2], t4, t5);
        f2_split(acc[3], t6, t7);
        return ((t0 + t1) + (t2 + t3)) + ((t4 + t5) + (t6 + t7));
      };
      if constexpr (!C::BITS8) {
        // The row in registers: P overwrites S, and a unit may have to be done again.
        uint32_t x[128];
        auto run = [&](auto full_tag) {
          constexpr bool FULL = decltype(full_tag)::value;  // all four chunks, no masks
          auto exp_all = [&](float neg_m, auto poly_tag) {
            const uint64_t scp = f2(a.scale_log2, a.scale_log2), nmp = f2(neg_m, neg_m);
            uint64_t acc[4] = {f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (FULL || c < nch) exp_chunk(x + c * 32, c, scp, nmp, acc, poly_tag);
            return total(acc);
          };
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (FULL || c < nch) tmem_ld32(s_addr + c * 32, *reinterpret_cast<uint32_t(*)[32]>(x + c * 32));
          tmem_wait_ld();
          reg_fence<128>(x);
          if (!FULL) {
#pragma unroll
            for (int e = 0; e < 128; ++e)
              if (e >= left) x[e] = __float_as_uint(-CUDART_INF_F);
          }
          if (__all_sync(0xffffffffu, m_ref != -CUDART_INF_F)) {
            lsum = exp_all(-m_ref, std::true_type{});
            if (__all_sync(0xffffffffu, lsum <= kTileSumLimit)) return;
            tmem_wait_st();
          }
          const float mx = max_tree_bits<128>(x) * a.scale_log2;
          if (mx > m_ref + kTileSlack) {
            if (m_ref != -CUDART_INF_F) alpha = ex2_approx(m_ref - mx);
            m_ref = mx;
          }
          lsum = exp_all(m_ref == -CUDART_INF_F ? 0.f : -m_ref, std::false_type{});
        };
        if (plain) run(std::true_type{});
        else run(std::false_type{});
      } else {
        // The scales leave no room for the row: it is read twice, a chunk at a time, for its maximum
        // (NaN wins and takes the row) and for the exponentials. P of chunk c overwrites columns of
        // chunk c / 2, which has been read.
        auto load = [&](int c, uint32_t(&v)[32]) {
          tmem_ld32(s_addr + c * 32, v);
          tmem_wait_ld();
          reg_fence32(v);
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 kk = *reinterpret_cast<const float4 *>(&sc.ks[ss][c * 32 + e]);
            v[e] = __float_as_uint(u2f_(v[e]) * kk.x);
            v[e + 1] = __float_as_uint(u2f_(v[e + 1]) * kk.y);
            v[e + 2] = __float_as_uint(u2f_(v[e + 2]) * kk.z);
            v[e + 3] = __float_as_uint(u2f_(v[e + 3]) * kk.w);
          }
          if (!plain) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (c * 32 + e >= left) v[e] = __float_as_uint(-CUDART_INF_F);
          }
        };
        float mx = -CUDART_INF_F;
#pragma unroll 1
        for (int c = 0; c < nch; ++c) {
          uint32_t v[32];
          load(c, v);
          float m0 = mx, m1 = mx;
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            m0 = fmax3_nan(m0, u2f_(v[e]), u2f_(v[e + 1]));
            m1 = fmax3_nan(m1, u2f_(v[e + 2]), u2f_(v[e + 3]));
          }
          mx = fmax3_nan(mx, m0, m1);
        }
        mx *= down;
        if (!(mx <= m_ref + kTileSlack)) {
          if (m_ref != -CUDART_INF_F) alpha = ex2_approx(m_ref - mx);
          m_ref = mx;
        }
        const float neg_m = m_ref == -CUDART_INF_F ? 0.f : -m_ref;
        const uint64_t scp = f2(down, down), nmp = f2(neg_m, neg_m);
        uint64_t acc[4] = {f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll 1
        for (int c = 0; c < nch; ++c) {
          uint32_t v[32];
          load(c, v);
          exp_chunk(v, c, scp, nmp, acc, std::true_type{});
        }
        lsum = total(acc);
      }
      l = l * alpha + lsum;
      if constexpr (C::BITS8) {
        alpha *= sc.vgrow[ss];
        vref = sc.vref[ss];
      }
      if (i > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
        // P V of the unit before has completed (its commit was this S's), so O can be rescaled.
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(o_addr + c * 32, o);
          tmem_wait_ld();
          reg_fence32(o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(u2f_(o[e]) * alpha);
          tmem_st32(o_addr + c * 32, o);
        }
      }
      if (!C::BITS8 && i == n - 1 && unit_ragged(sg->L, klim, sg->u0 + i)) {
        // both halves write the same zeros, each before its own product
        const uint32_t ve = kv + 2 * i + 1;
        if (!wait(&sc.full[ve % C::NSLOT], (ve / C::NSLOT) & 1)) break;
        uint8_t *v = ring + (ve % C::NSLOT) * C::HALF_BYTES;
        const int r0 = max(sg->L - base, 0), r1 = 16 * unit_steps(klim, sg->u0 + i);
        for (int e = row; e < (r1 - r0) * 8 * C::PANELS; e += 128) {
          const int r = r0 + e / (8 * C::PANELS), ch = e % (8 * C::PANELS);
          *reinterpret_cast<uint4 *>(v + (ch >> 3) * (128 * 128) + r * 128 + (ch & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async();
      }
      tmem_wait_st();
      tc_fence_before_sync();
      mbar_arrive(&sc.p_full[w]);
    }
    if (!ok) break;
    // ---- the last P V of this half is done: write its rows
    if (!wait(&sc.o_full[w], o_ph)) break;
    o_ph ^= 1;
    if (leader) release(kv + 2 * n - 1);
    kv += 2 * n;
    const float vm = C::BITS8 ? vref : 1.f;
    if (sg->part >= 0) {
      // Partial result, [slot][half][column / 4][row][4]: a warp's stores are contiguous.
      const size_t slot = sg->part;
      float *dst = a.part_o + (slot * 2 + w) * (128 * D) + row * 4;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(o_addr + c * 32, o);
        tmem_wait_ld();
        reg_fence32(o);
#pragma unroll
        for (int e = 0; e < 32; e += 4)
          *reinterpret_cast<float4 *>(dst + (c * 8 + e / 4) * (128 * 4)) =
              make_float4(u2f_(o[e]) * vm, u2f_(o[e + 1]) * vm, u2f_(o[e + 2]) * vm, u2f_(o[e + 3]) * vm);
      }
      a.part_ml[slot * 512 + w * 128 + row] = m_ref;
      a.part_ml[slot * 512 + 256 + w * 128 + row] = l;
    } else {
      // Complete rows: through this half's query buffer (every product with it is done), so that
      // a warp writes whole rows: its 32 rows one by one would touch 32 lines with every
      // store (measured: 3300 cycles a half, and the stores held up the barriers behind them).
      const float inv = l == 0.f ? 0.f : vm / l;  // a row that sees no key is zero
      uint8_t *buf = q_smem + (qe % C::NQ) * C::HALF_BYTES;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(o_addr + c * 32, o);
        tmem_wait_ld();
        reg_fence32(o);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t pk[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) pk[k] = pack16<QT>(u2f_(o[8 * e + 2 * k]) * inv, u2f_(o[8 * e + 2 * k + 1]) * inv);
          *reinterpret_cast<uint4 *>(buf + swz(row, c * 4 + e)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
      }
      tc_fence_before_sync();
      mbar_arrive(&sc.o_empty[w]);
      int tok, hg;
      const bool row_ok = half_row(a, *sg, w, row, tok, hg);
      unsigned long long dst = reinterpret_cast<unsigned long long>(
          static_cast<QT *>(a.out) + sg->b * a.o_batch + static_cast<long long>(sg->tok + tok) * a.o_tok +
          static_cast<long long>(sg->h * a.G + hg) * a.o_head);
      if (!row_ok) dst = 0;
      __syncwarp();
      constexpr int LPR = D / 8, RPI = 32 / LPR;  // lanes of a row, rows of a store
      const int ch = lane % LPR;
#pragma unroll 4
      for (int r = 0; r < 32; r += RPI) {
        const int rr = r + lane / LPR;
        const unsigned long long p = __shfl_sync(0xffffffffu, dst, rr);
        const uint4 v = *reinterpret_cast<const uint4 *>(buf + swz(wq * 32 + rr, ch));
        if (p) st_global_v4_hint(reinterpret_cast<uint4 *>(p) + ch, v.x, v.y, v.z, v.w, pol_out);
      }
      // The next copy into the buffer is ordered behind these reads.
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sc.q_empty[qe % C::NQ]);
      rd.done(sc);
      continue;
    }
    tc_fence_before_sync();
    mbar_arrive(&sc.o_empty[w]);
    rd.done(sc);
  }
  if (!ok && lane == 0) tile_abort(&sc.abort_flag, a.status);
}

// ------------------------------------------------------------------ kernel

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    tile_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ DenseArgs a, const __grid_constant__ TileArgs x) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *q_smem = base;
  uint8_t *ring = base + C::NQ * C::HALF_BYTES;
  TileCtl<C> &sc = *reinterpret_cast<TileCtl<C> *>(ring + C::NSLOT * C::HALF_BYTES);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    const int fillers = C::BITS8 ? 128 : 1;  // converter threads, or the producer's expected bytes
    for (int i = 0; i < C::NSLOT; ++i) {
      mbar_init(&sc.full[i], fillers);
      mbar_init(&sc.empty[i], 2);  // one arrival per half
    }
    for (int i = 0; i < C::NQ; ++i) {
      mbar_init(&sc.q_full[i], fillers);
      mbar_init(&sc.q_empty[i], 4);  // the half's softmax warps
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(&sc.s_full[w], 1);
      mbar_init(&sc.p_full[w], 128);
      mbar_init(&sc.o_full[w], 1);
      mbar_init(&sc.o_empty[w], 128);
      mbar_init(&sc.mma_done[w], 1);
    }
    mbar_init(&sc.conv, 4);
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(&sc.seg_full[i], 1);
      mbar_init(&sc.seg_empty[i], (C::BITS8 ? 128 : 1) + 2 + 256);  // producer or converter, issuers, softmax
    }
    sc.turn = 0;
    sc.abort_flag = 0;
    fence_mbar_init();
    if (!C::BITS8) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
  }
  if constexpr (!C::BITS8) {
    // Rows behind a half's whole tokens are never copied: zeros, so that their scores are finite.
    const int r0 = (a.tile_tokens >> 1) * a.G, per = (128 - r0) * 8;
    for (int i = threadIdx.x; i < per * C::PANELS * C::NQ; i += C::THREADS) {
      const int pn = i / per, e = i - pn * per;  // panels of the buffers follow one another
      *reinterpret_cast<uint4 *>(q_smem + pn * (128 * 128) + (r0 * 8 + e) * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async();
  }
  if (warp == 2) {
    tmem_alloc(&sc.tmem_base, C::TMEM_COLS);
    tmem_relinquish();
    if (blockIdx.x == 0) check_lengths(a);
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = sc.tmem_base;
  if (warp < 4) regs_dec<C::CTRL_REGS>();
  else if (warp < 12) regs_inc<C::SOFTMAX_REGS>();
  else if constexpr (C::BITS8) regs_dec<C::CONV_REGS>();
  if (warp < 4) {
    if (warp == 0) {
      if constexpr (!C::BITS8) {
        if (lane == 0) tile_producer<C>(sc, a, x, q_smem, ring, &tm_q, &tm_k, &tm_v);
      }
    } else if (warp == 2) {
      tile_scheduler<C>(sc, a, x, lane);
    } else if (lane == 0) {
      tile_mma<C>(sc, a, tmem, q_smem, ring, warp == 1 ? 0 : 1);
    }
  } else if (warp < 12) {
    tile_softmax<C>(sc, a, tmem, q_smem, ring, (warp - 4) >> 2, warp, lane);
  } else if constexpr (C::BITS8) {
    tile_converter<C>(sc, a, q_smem, ring);
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 2) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

}  // namespace solattn
