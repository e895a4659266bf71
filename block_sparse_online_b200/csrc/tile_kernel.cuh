// tile_kernel.cuh -- dense attention for many query rows of a key head: tcgen05 with the
// accumulators in tensor memory.
//
// A block per SM walks its range of the work line. A tile is 256 query rows, two halves of
// 128; K and V come in units of 128 keys and serve both halves, so a key tile crosses L2
// once per 256 rows. Roles, by warp:
//   warp 0       16-bit keys: TMA producer. Q halves into three buffers (the next item's first half
//                lands while this item runs), K and V units into a ring.
//   warps 1, 3   MMA issuers, one for each half: S = Q K^T into tensor memory, O += P V with
//                P read from tensor memory. They take turns through a shared counter, so the tensor core
//                works on one half while the other half's softmax runs.
//   warp 2       owns the TMEM allocation; walks the block's range of the line and publishes its
//                segments (one tile's run of units) to the other roles, a few ahead.
//   warps 4-11   softmax, one warpgroup for each half, one row per thread. Where a sequence ends inside a step they
//                zero the value rows behind the end, which may hold anything (0 times NaN is NaN).
//   last 4 warps 8-bit keys only: read codes from the pages, expand them to fp16 into the ring (and the
//                queries, scaled, into their buffers), one unit ahead in registers.
// A step is 64 keys. Each half has two buffers of S (P takes the place of its S): Q K^T of step j + 2
// follows P V of step j, so while a warpgroup exponentiates step j + 1 the tensor core works on its steps
// j and j + 2. With one buffer of 128 keys instead, S, softmax and P V form one chain of 3500 to 3700 cycles a
// unit for both halves, of which the tensor core works 2130.
//
// Softmax: once a row has a reference maximum a step is exponentiated against it without taking the row
// maximum; a row sum <= 2^15 shows that no value is large, otherwise (or for a row's first step, or a masked
// one) the maximum is taken (a NaN wins it) and the step done again. P is rounded to the 16-bit type of the
// keys, fp16 for 8-bit caches: off by at most 2^-8 (bf16) or 2^-11 of each value, independently from key to
// key, which adds about as much to the result's error as the output's own rounding. The reference, sums and
// O are in 32 bits. Two pairs of exponentials in eight go through the polynomial on the FMA pipe. 8-bit caches:
// the reference is that of x + log2 |value scale|, as in the rows kernel; that no product of P and a scale is
// large is shown by the row sum times the unit's largest scale.
//
// What bounds it, measured at 1560 tokens x 32760 keys x 12 heads of 128 in bf16 (320 to 400 us, 800 to 980
// TFLOP/s; the card's power limit moves it): the tensor core's instructions. A step's 8 products of 64 columns
// take 85 cycles each where 128 columns take 67, so a step costs both halves 1900 cycles, the
// softmax 1700. Measured and not kept: one S buffer of 128 columns with two warpgroups a half by columns
// (387 us), two warpgroups a half by steps (400 us), output by TMA stores (no gain, and the queries'
// buffer comes back late), a deeper queue of queries for a shallower ring of keys (558 us). Short rows of
// keys (one or two steps) are bound by a tile's fixed 5500 cycles: queries in, first maximum, rows out.
// 8-bit caches add the expansion of the codes, which is what bounds them (520 to 550 us for the same in int8; every tile
// expands its keys again, and the softmax warps store 52 to 88 bytes of a thread for want of registers).
//
// Causal and ragged ends: columns at or behind a row's limit are replaced by -infinity; the
// products of a unit stop at the last 16 keys that some row of the tile sees.
#pragma once

#include "dense_common.cuh"
#include "rows_kernel.cuh"

namespace solattn {

constexpr float kTileSlack = 8.0f;         // log2 units the reference may lag a unit's maximum
constexpr float kTileSumLimit = 32768.0f;  // row sum that shows every value <= 2^15
// Pairs (mod 8) on the polynomial: at 1560 x 32760 none 416, one 384, two 359, three 390 us.
constexpr uint32_t kTilePolyMask = 0x88u;

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
  static constexpr int NSLOT = D == 128 ? 4 : 8;  // even: K in the even slots, V in the odd ones
  // Units whose scales are kept. A unit's slot of K is free as soon as its last S is there, while the softmax still
  // reads its scales: the converter may be NSLOT / 2 units ahead of the last unit that is done with.
  static constexpr int NSC = NSLOT / 2 + 2;
  static constexpr int COLS = 128 + D;  // tensor memory columns of a half: O, two buffers of S (and P)
  static constexpr int TMEM_COLS = 512;
  static constexpr int THREADS = BITS8 ? 512 : 384;
  // Register shares: within what the block is launched with.
  static constexpr int LAUNCH_REGS = BITS8 ? 128 : 168;
  static constexpr int CTRL_REGS = BITS8 ? 72 : 104;
  static constexpr int CONV_REGS = 136;
  static constexpr int SOFTMAX_REGS = BITS8 ? 152 : 200;
  static_assert(CTRL_REGS < LAUNCH_REGS && (!BITS8 || CONV_REGS > LAUNCH_REGS) && SOFTMAX_REGS > LAUNCH_REGS,
                "control warps give registers up, the others take them");
  static_assert(128 * CTRL_REGS + 256 * SOFTMAX_REGS + (BITS8 ? 128 * CONV_REGS : 0) <= THREADS * LAUNCH_REGS,
                "register split");
  static constexpr bool ROW_SCALE = BITS8 && !std::is_same<QT, __half>::value;  // bf16 queries multiply as fp16, far rows by a factor of their own
  static constexpr bool FP16 = std::is_same<MT, __half>::value;
  static constexpr uint32_t IDESC_PV = idesc_16bit_f32(128, D, true, FP16);
};

constexpr int kStatusTimeoutTile = -4;  // SOLATTN_ETIMEOUT
constexpr int kStepKeys = 64;  // keys of a step: a unit is two (the last may be one)
constexpr int kSegs = 4;  // segments published ahead

// A segment of the block's range: units u0 .. u1 - 1 of one tile.
struct Segment {
  int n, ns, u0, klim, L;  // units (0: no more work), steps, first unit, keys that some row sees, keys
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
  uint64_t s_full[2][2], p_full[2][2];  // by half, and buffer of S
  uint64_t o_pre[2], o_full[2], o_empty[2];  // the tile's last product but one, its last, and O read
  uint64_t conv;  // the converter's four warps
  uint64_t mma_done[2];
  uint32_t turn;
  uint32_t tmem_base;
  int abort_flag;
  alignas(16) float ks[C::BITS8 ? C::NSC : 1][C::BITS8 ? 128 : 4];  // key scales (x log2(e) / sqrt d)
  alignas(16) float vs[C::BITS8 ? C::NSC : 1][C::BITS8 ? 128 : 4];  // value scales
  alignas(16) float lv[C::BITS8 ? C::NSC : 1][C::BITS8 ? 128 : 4];  // their log2_scale()
  alignas(16) float wmax[C::NSC][4];  // largest magnitude of the value scales, by the converter's warps
  uint32_t qmax[2][4];           // converter: largest query of a tile per warp (bf16 bits); tiles alternate
  int qrel[C::NQ][C::BITS8 ? 128 : 1];  // bf16 queries as fp16: log2 of what a row was divided by over the tile's
};

template <class C>
constexpr size_t tile_smem_bytes() {
  return static_cast<size_t>(C::NQ + C::NSLOT) * C::HALF_BYTES + sizeof(TileCtl<C>);
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
  atomicCAS(status, 0, kStatusTimeoutTile);
  *reinterpret_cast<volatile int *>(abort_flag) = 1;
}

// Extra arguments of the tile kernel.
struct TileArgs {
  int k_b, k_h, v_b, v_h;  // 0: the batch (head) stride is zero, and so is the coordinate
  int min_units, whole_items;
};

// Slices of 16 keys that the products of the step at key `base` need: some row of the tile sees
// a key in each.
__device__ __forceinline__ int step_slices(int klim, int base) { return min(4, max(1, (klim - base + 15) >> 4)); }

// ------------------------------------------------------------------ segments

template <class C>
__device__ void tile_scheduler(TileCtl<C> &sc, const DenseArgs &a, const TileArgs &x, int lane) {
  Cursor<TokenTiles> cur;
  bool more = cur.begin(a, blockIdx.x, gridDim.x, x.min_units, x.whole_items);
  if (lane != 0) return;
  int4 rec = make_int4(0, 0, 0, 0);
  for (uint32_t i = 0;; ++i) {
    const int sl = i % kSegs;
    if (!mbar_sleep(&sc.seg_empty[sl], ((i / kSegs) & 1) ^ 1, a.timeout_ns, &sc.abort_flag)) {
      tile_abort(&sc.abort_flag, a.status);
      break;
    }
    Segment g{};
    if (more) {
      const Seq &s = cur.s;
      g.n = cur.u1 - cur.u0;
      g.u0 = cur.u0;
      g.klim = key_limit(a, s, TokenTiles::last_token(a, s.n, cur.t));
      g.ns = 2 * g.n - (g.klim - (cur.u1 - 1) * kUnitKeys <= kStepKeys ? 1 : 0);
      g.L = s.L;
      g.tok = s.tok0 + cur.t * a.tile_tokens;
      g.end = s.tok0 + s.n;
      g.b = cur.b;
      g.h = cur.h;
      // causal: token i of the tile sees lim0 + i keys (cut to 0 .. L)
      g.lim0 = a.causal ? s.L - s.n + cur.t * a.tile_tokens + 1 : s.L;
      g.part = cur.partial() ? cur.slot(blockIdx.x) : -1;
      if (cur.partial() && cur.u0 == 0) rec = cur.record(blockIdx.x);
      if (!SOLATTN_DCHECK(g.n > 0 && g.u0 >= 0 && (g.u0 + g.n - 1) * kUnitKeys <= a.Lmax && g.klim <= g.L && row_inside(a, g.b, g.tok, g.h * a.G) &&
                              g.end <= (a.cu ? a.total : a.n) && (g.part < 0 || slot_inside(g.part, gridDim.x)),
                          &sc.abort_flag, a.status))
        break;
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
  // The next segment, or null at the end (or when a wait gave up: ok is cleared). The whole warp calls it.
  __device__ __forceinline__ const Segment *next(TileCtl<C> &sc, const DenseArgs &a, bool &ok) {
    const int sl = i % kSegs;
    if (!__all_sync(0xffffffffu, mbar_sleep(&sc.seg_full[sl], (i / kSegs) & 1, a.timeout_ns, &sc.abort_flag))) {
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

// The whole warp walks along: lane 0 keeps the barriers, and the copies of a buffer (one a panel, or a
// panel and page) are issued by as many lanes at once. Pages are looked up a unit ahead, one by each of those lanes: with
// pages of 16 tokens a single thread's 16 lookups and 32 copies took longer than the unit's products.
template <class C>
__device__ void tile_producer(TileCtl<C> &sc, const DenseArgs &a, const TileArgs &x, uint8_t *q_smem, uint8_t *ring,
                              const CUtensorMap *tm_q, const CUtensorMap *tm_k, const CUtensorMap *tm_v, int lane) {
  const volatile int *ab = &sc.abort_flag;
  const uint64_t pol_stream = l2_policy_evict_first(), pol_reuse = l2_policy_evict_last();
  const int half = a.tile_tokens >> 1;
  const uint32_t q_bytes = static_cast<uint32_t>(half) * a.G * 128;  // of a panel
  const int boxes = C::PAGED ? kUnitKeys >> a.page_shift : 1;        // of a panel of a unit
  const int box = lane % boxes, pn = lane / boxes;                   // this lane's copy of a unit's K or V
  const bool mine = pn < C::PANELS;
  uint32_t kv = 0, qi = 0;
  bool ok = true;
  auto wait = [&](uint64_t *bar, uint32_t par) { return __all_sync(0xffffffffu, mbar_sleep(bar, par, a.timeout_ns, ab)); };
  SegmentReader<C> rd;
  while (const Segment *g = ok ? rd.next(sc, a, ok) : nullptr) {
    const int b = g->b, h = g->h, L = g->L, tok0 = g->tok, u0 = g->u0, u1 = u0 + g->n;
    __syncwarp();
    if (lane == 0) rd.done(sc);
    auto load_q = [&](int w) {
      const int sl = qi % C::NQ;
      if (!wait(&sc.q_empty[sl], ((qi / C::NQ) & 1) ^ 1)) return false;
      if (lane == 0) mbar_arrive_expect_tx(&sc.q_full[sl], q_bytes * C::PANELS);
      __syncwarp();
      if (lane < C::PANELS)
        tma_load_5d_hint(smem_u32(q_smem + sl * C::HALF_BYTES + lane * (128 * 128)), tm_q, smem_u32(&sc.q_full[sl]), lane * 64, 0,
                         tok0 + w * half, h, a.cu ? 0 : b, pol_stream);
      ++qi;
      return true;
    };
    // Page of this lane's box of unit u. Keys behind the end, and bad table entries, lie outside the map: they
    // read as zeros.
    auto page_at = [&](int u) {
      const int j = u * kUnitKeys + (box << a.page_shift);
      int id = -1;
      if (mine && u < u1 && j < L) id = page_of(a, b, j);
      return id < 0 ? a.num_pages : id;
    };
    auto load_kv = [&](int u, bool is_v, int page) {
      const int sl = kv % C::NSLOT;
      if (!wait(&sc.empty[sl], ((kv / C::NSLOT) & 1) ^ 1)) return false;
      if (lane == 0) mbar_arrive_expect_tx(&sc.full[sl], C::HALF_BYTES);
      __syncwarp();
      if (mine) {
        const CUtensorMap *map = is_v ? tm_v : tm_k;
        uint8_t *dst = ring + sl * C::HALF_BYTES + pn * (128 * 128);
        if constexpr (C::PAGED)
          tma_load_4d_hint(smem_u32(dst + (box << a.page_shift) * 128), map, smem_u32(&sc.full[sl]), pn * 64, 0, h, page, pol_reuse);
        else
          tma_load_4d_hint(smem_u32(dst), map, smem_u32(&sc.full[sl]), pn * 64, u * kUnitKeys, h * (is_v ? x.v_h : x.k_h),
                           b * (is_v ? x.v_b : x.k_b), pol_reuse);
      }
      ++kv;
      return true;
    };
    int page = 0, next = 0;
    if constexpr (C::PAGED) {
      page = page_at(u0);
      next = page_at(u0 + 1);
    }
    ok = load_q(0) && load_kv(u0, false, page) && load_q(1);
    for (int u = u0; u < u1 && ok; ++u) {
      ok = load_kv(u, true, page);
      page = next;
      if (ok && u + 1 < u1) ok = load_kv(u + 1, false, page);
      if constexpr (C::PAGED) next = page_at(u + 2);
    }
  }
  if (!ok && lane == 0) tile_abort(&sc.abort_flag, a.status);
  // No copy may outlive the block: wait (bounded) for the last fill of every buffer.
  const int zero = 0;
  for (uint32_t f = kv > C::NSLOT ? kv - C::NSLOT : 0; f < kv; ++f)
    mbar_sleep(&sc.full[f % C::NSLOT], (f / C::NSLOT) & 1, a.timeout_ns, &zero);
  for (uint32_t f = qi > C::NQ ? qi - C::NQ : 0; f < qi; ++f)
    mbar_sleep(&sc.q_full[f % C::NQ], (f / C::NQ) & 1, a.timeout_ns, &zero);
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
  uint32_t kv = 0, qi = 0, tile = 0, item = 0;
  bool ok = true;
  auto wait = [&](uint64_t *bar, uint32_t par) {
    bool w = mbar_sleep(bar, par, a.timeout_ns, ab);
    w = __all_sync(0xffffffffu, w);
    if (!w) ok = false;
    return w;
  };
  uint4 ck[NP], cv[NP];  // codes of the next unit's keys and values
  float ksc, vsc;
  // Table entries of a unit: lane g holds that of its keys 16 (g % 8) .. + 15 (a page has 16 tokens at least), or -2
  // behind the sequence's end. Read a unit ahead of the codes, and looked at only then.
  auto fetch_entries = [&](const Segment &c, int u) {
    const int j = u * kUnitKeys + (lane & 7) * 16;
    return j < c.L && SOLATTN_DCHECK(j < a.Lmax, &sc.abort_flag, a.status) ? __ldg(a.table + static_cast<size_t>(c.b) * a.width + (j >> a.page_shift)) : -2;
  };
  // The pages they name; -1 for none (an entry that names no page of the cache is recorded).
  auto pages_of = [&](int entry) {
    if (static_cast<unsigned>(entry) < static_cast<unsigned>(a.num_pages)) return entry;
    if (entry != -2) atomicCAS(a.status, 0, kStatusTable);
    return -1;
  };
  // Codes of a unit's keys or values into registers, zeros where there is no key.
  auto fetch = [&](const Segment &c, int u, int pages, bool is_v, uint4(&cd)[NP]) {
    const uint8_t *base = static_cast<const uint8_t *>(is_v ? a.v : a.k) + c.h * (is_v ? a.v_head : a.k_head) + pc * 16;
    const long long row = is_v ? a.v_row : a.k_row, seq = is_v ? a.v_seq : a.k_seq;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int j = u * kUnitKeys + i * RPP + rl;
      const int id = __shfl_sync(0xffffffffu, pages, (i * RPP + rl) >> 4);
      cd[i] = id >= 0 && j < c.L && SOLATTN_DCHECK(key_inside(a, id, j & (a.page - 1)), &sc.abort_flag, a.status) ? ld_stream16(base + id * seq + (j & (a.page - 1)) * row) : make_uint4(0, 0, 0, 0);
    }
  };
  // The scales of a unit: thread t takes key t.
  auto fetch_scales = [&](const Segment &c, int u, int pages) {
    const int j = u * kUnitKeys + tid;
    const int id = __shfl_sync(0xffffffffu, pages, tid >> 4);
    const bool in = id >= 0 && j < c.L && SOLATTN_DCHECK(key_inside(a, id, j & (a.page - 1)), &sc.abort_flag, a.status);
    const size_t at = (static_cast<size_t>(max(id, 0)) * a.Hkv + c.h) * a.page + (j & (a.page - 1));
    ksc = in ? __ldg(a.k_scale + at) : 0.f;
    vsc = in ? __ldg(a.v_scale + at) : 0.f;
  };
  auto expand = [&](uint8_t *dst, const uint4(&cd)[NP]) {
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
  const Segment *g = rd.next(sc, a, ok);
  if (g) {
    const int pages = pages_of(fetch_entries(*g, g->u0));
    fetch(*g, g->u0, pages, false, ck);
    fetch_scales(*g, g->u0, pages);
    fetch(*g, g->u0, pages, true, cv);
  }
  while (g) {
    // ---- queries of both halves, a row of each per thread. bf16 queries become fp16 after a division by a power of
    // two, which brings the tile's largest finite element to [2^14, 2^15): elements down to 2^-31 of that are exact,
    // and a smaller one is off by 2^-39 of it. The factor goes into the key scales. A row whose own largest element lies
    // more than 2^16 below the tile's (another token's, or head's, is that much larger) would lose bits and then
    // all of them: it is divided by a power of two of its own, and the softmax, which takes its slow path for the warp,
    // multiplies its scores by the ratio. (A factor for every row in every step: 540 us against 532 for an int8 chunk of 1560 tokens over 32760 keys.)
    const typename C::QT *src[2];
    bool row_ok[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      int tok, hg;
      row_ok[w] = half_row(a, *g, w, tid, tok, hg) &&
                  SOLATTN_DCHECK(row_inside(a, g->b, g->tok + tok, g->h * a.G + hg), &sc.abort_flag, a.status);
      src[w] = static_cast<const typename C::QT *>(a.q) + static_cast<long long>(g->tok + tok) * a.q_tok +
               static_cast<long long>(g->h * a.G + hg) * a.q_head;
    }
    float up[2] = {1.f, 1.f}, down = 1.f;
    int rel[2] = {0, 0};
    if constexpr (C::ROW_SCALE) {
      uint32_t big[2] = {0, 0};
#pragma unroll
      for (int w = 0; w < 2; ++w) {
#pragma unroll 2
        for (int i = 0; i < D / 8; ++i) {
          const uint4 v = row_ok[w] ? __ldg(reinterpret_cast<const uint4 *>(src[w]) + i) : make_uint4(0, 0, 0, 0);
          const uint32_t vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t lo = vv[e] & 0x7fffu, hi = (vv[e] >> 16) & 0x7fffu;
            big[w] = max(big[w], max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
          }
        }
      }
      const uint32_t most = __reduce_max_sync(0xffffffffu, max(big[0], big[1]));
      if (lane == 0) {
        sc.qmax[item & 1][warp] = most;
        mbar_arrive(&sc.conv);
      }
      if (!wait(&sc.conv, item & 1)) break;
      const uint32_t *qm = sc.qmax[item & 1];
      ++item;
      const auto shift = [](int ex) { return ex == 0 ? 0 : min(max(141 - ex, -126), 126); };  // ex: biased exponent
      const int ex = static_cast<int>(max(max(qm[0], qm[1]), max(qm[2], qm[3])) >> 7), sh = shift(ex);
      down = __int_as_float((127 - sh) << 23);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const int own = static_cast<int>(big[w] >> 7);
        const int sw = own == 0 || own + 16 >= ex ? sh : shift(own);
        up[w] = __int_as_float((127 + sw) << 23);
        rel[w] = sh - sw;
      }
    }
    for (int w = 0; w < 2 && ok; ++w) {
      const int sl = qi % C::NQ;
      if (!wait(&sc.q_empty[sl], ((qi / C::NQ) & 1) ^ 1)) break;
      uint8_t *dst = q_smem + sl * C::HALF_BYTES;
#pragma unroll 2
      for (int i = 0; i < D / 8; ++i) {
        uint4 v = row_ok[w] ? __ldg(reinterpret_cast<const uint4 *>(src[w]) + i) : make_uint4(0, 0, 0, 0);
        if constexpr (std::is_same<typename C::QT, __nv_bfloat16>::value) {
          const float f = up[w];
          v.x = pack_f16x2(__uint_as_float(v.x << 16) * f, __uint_as_float(v.x & 0xffff0000u) * f);
          v.y = pack_f16x2(__uint_as_float(v.y << 16) * f, __uint_as_float(v.y & 0xffff0000u) * f);
          v.z = pack_f16x2(__uint_as_float(v.z << 16) * f, __uint_as_float(v.z & 0xffff0000u) * f);
          v.w = pack_f16x2(__uint_as_float(v.w << 16) * f, __uint_as_float(v.w & 0xffff0000u) * f);
        }
        *reinterpret_cast<uint4 *>(dst + swz(tid, i)) = v;
      }
      sc.qrel[sl][tid] = rel[w];
      publish(&sc.q_full[sl]);
      ++qi;
    }
    if (!ok) break;
    const float kmul = a.scale_log2 * down;
    // ---- units: K u, then V u, each with the next piece's codes on their way
    const Segment *nxt = nullptr;
    const int u1 = g->u0 + g->n;
    for (int u = g->u0; u < u1 && ok; ++u) {
      // what the registers hold next: the following unit, of this segment or of the next one
      const Segment *f = g;
      int fu = u + 1;
      if (fu == u1) {
        rd.done(sc);
        f = nxt = rd.next(sc, a, ok);
        if (f) fu = f->u0;
      }
      const int entries = f ? fetch_entries(*f, fu) : -2;
      int sl = kv % C::NSLOT;
      if (!wait(&sc.empty[sl], ((kv / C::NSLOT) & 1) ^ 1)) break;
      const int ss = tile % C::NSC;
      float mx = fabsf(vsc);  // (a scale may be negative)
#pragma unroll
      for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      if (lane == 0) sc.wmax[ss][warp] = mx;
      sc.ks[ss][tid] = ksc * kmul;
      sc.vs[ss][tid] = vsc;
      sc.lv[ss][tid] = log2_scale(vsc);
      ++tile;
      expand(ring + sl * C::HALF_BYTES, ck);
      publish(&sc.full[sl]);
      ++kv;
      const int pages = pages_of(entries);
      if (f) {
        fetch(*f, fu, pages, false, ck);
        fetch_scales(*f, fu, pages);
      }
      sl = kv % C::NSLOT;
      if (!wait(&sc.empty[sl], ((kv / C::NSLOT) & 1) ^ 1)) break;
      expand(ring + sl * C::HALF_BYTES, cv);
      publish(&sc.full[sl]);
      ++kv;
      if (f) fetch(*f, fu, pages, true, cv);
    }
    if (!ok) break;
    g = nxt;
  }
  if (!ok && lane == 0) tile_abort(&sc.abort_flag, a.status);
}

// ------------------------------------------------------------------ MMA issuers

// Groups of one half: S(0) and S(1), then P V(j) with S(j + 2) behind it. Halves alternate group by group.
// The whole warp walks through the loop and one lane issues: descriptors then live in uniform registers,
// where a lone thread pays several moves for each of them (measured: 80 cycles an instruction under the
// softmax warps' load, of which the tensor core needs 32 to 64).
template <class C>
__device__ void tile_mma(TileCtl<C> &sc, const DenseArgs &a, uint32_t tmem, uint8_t *q_smem, uint8_t *ring, int w) {
  const volatile int *ab = &sc.abort_flag;
  volatile uint32_t *turn = &sc.turn;
  const uint64_t q_desc0 = smem_desc_sw128(smem_u32(q_smem), 16, 1024);
  const uint64_t k_desc0 = smem_desc_sw128(smem_u32(ring), 16, 1024);
  const uint64_t v_desc0 = smem_desc_sw128(smem_u32(ring), 128 * 128, 1024);
  constexpr uint32_t kUnits = C::HALF_BYTES / 16;
  constexpr uint32_t kStepUnits = kStepKeys * 128 / 16;  // from one step's keys to the next in a unit
  const uint32_t o_tmem = tmem + w * C::COLS, s_tmem = o_tmem + C::D;
  uint32_t kv = 0, qi = 0, p_ph = 0, g = 0, o_ph = 0;  // p_ph: bit b is the phase of buffer b
  bool ok = true;
  const uint32_t lead = elect_one();
  auto wait = [&](uint64_t *bar, uint32_t par) {
    ok = __all_sync(0xffffffffu, mbar_sleep(bar, par, a.timeout_ns, ab));
    tc_fence_after_sync();
    return ok;
  };
  auto take = [&](uint32_t target) {
    if (__all_sync(0xffffffffu, *turn == target)) return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t it = 1;; ++it) {
      if (__all_sync(0xffffffffu, *turn == target)) return true;
      if ((it & 255u) == 0u && __any_sync(0xffffffffu, *ab || global_timer_ns() - t0 > a.timeout_ns)) {
        ok = false;
        return false;
      }
    }
  };
  auto pass = [&](uint32_t next) {
    if (lead) *turn = next;
    __syncwarp();
  };
  SegmentReader<C> rd;
  while (const Segment *sg = ok ? rd.next(sc, a, ok) : nullptr) {
    // (a broadcast tells the compiler that the values are the same in every lane)
    const int n = __shfl_sync(0xffffffffu, sg->n, 0), ns = __shfl_sync(0xffffffffu, sg->ns, 0);
    const int klim = __shfl_sync(0xffffffffu, sg->klim, 0), base = __shfl_sync(0xffffffffu, sg->u0, 0) * kUnitKeys;
    __syncwarp();
    if (lead) rd.done(sc);
    const uint32_t qe = qi + w;
    qi += 2;
    if (!wait(&sc.q_full[qe % C::NQ], (qe / C::NQ) & 1)) break;
    const uint64_t q_desc = q_desc0 + (qe % C::NQ) * kUnits;
    auto issue_qk = [&](int j) {
      const uint64_t kd = k_desc0 + ((kv + (j & ~1)) % C::NSLOT) * kUnits + (j & 1) * kStepUnits;
      const uint32_t idesc = idesc_16bit_f32(128, 16 * step_slices(klim, base + j * kStepKeys), false, C::FP16);
#pragma unroll
      for (int kk = 0; kk < C::D / 16; ++kk) {
        const uint64_t off = static_cast<uint64_t>((kk >> 2) * (128 * 128 / 16) + (kk & 3) * 2);
        mma_ss_if(lead, s_tmem + (j & 1) * kStepKeys, q_desc + off, kd + off, idesc, kk > 0 ? 1u : 0u);
      }
    };
    auto wait_entry = [&](uint32_t e) { return wait(&sc.full[e % C::NSLOT], (e / C::NSLOT) & 1); };
    if (!wait_entry(kv) || !take(g + w)) break;
    issue_qk(0);
    tc_commit_if(lead, &sc.s_full[w][0]);
    if (ns > 1) {
      issue_qk(1);
      tc_commit_if(lead, &sc.s_full[w][1]);
    }
    pass(g + w + 1);
    for (int j = 0; j < ns && ok; ++j) {
      const int b = j & 1;
      if (b == 0) {
        if (!wait_entry(kv + j + 1)) break;                    // V of the step's unit
        if (j + 2 < ns && !wait_entry(kv + j + 2)) break;      // K of the next unit
      }
      if (j == 0 && !wait(&sc.o_empty[w], o_ph ^ 1)) break;
      if (!wait(&sc.p_full[w][b], (p_ph >> b) & 1)) break;
      p_ph ^= 1u << b;
      const uint32_t my = g + 2 + 2 * j + w;
      if (!take(my)) break;
      const uint64_t vd = v_desc0 + ((kv + (j & ~1) + 1) % C::NSLOT) * kUnits + b * kStepUnits;
      const uint32_t p_tmem = s_tmem + b * kStepKeys;
      const int slices = step_slices(klim, base + j * kStepKeys);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        if (kk < slices)
          mma_ts_if(lead, o_tmem, p_tmem + kk * 8, vd + static_cast<uint64_t>(kk * (16 * 128 / 16)), C::IDESC_PV, (j > 0 || kk > 0) ? 1u : 0u);
      pass(my + 1);  // the other issuer wakes while this one is still at S(j + 2)
      if (j + 2 < ns) issue_qk(j + 2);
      // S(j + 2), or the end of one of the last two P V. These have barriers of their own: the next tile's S may
      // follow at once, and a second phase of one barrier could pass before the first is seen.
      tc_commit_if(lead, j + 2 < ns ? &sc.s_full[w][b] : j + 1 < ns ? &sc.o_pre[w] : &sc.o_full[w]);
    }
    if (!ok) break;
    o_ph ^= 1;
    kv += 2 * n;
    g += 2 + 2 * ns;
  }
  if (!ok && lead) tile_abort(&sc.abort_flag, a.status);
  // Every tcgen05 operation issued here must finish before TMEM is released.
  const int zero = 0;
  tc_commit_if(lead, &sc.mma_done[w]);
  mbar_sleep(&sc.mma_done[w], 0, a.timeout_ns, &zero);
}

// ------------------------------------------------------------------ softmax and epilogue

// w: half of the tile.
template <class C>
__device__ void tile_softmax(TileCtl<C> &sc, const DenseArgs &a, uint32_t tmem, uint8_t *q_smem, uint8_t *ring,
                             int w, int warp, int lane) {
  constexpr int D = C::D;
  using QT = typename C::QT;
  using MT = typename C::MT;
  const volatile int *ab = &sc.abort_flag;
  const int wq = warp & 3, row = wq * 32 + lane;
  const uint32_t o_addr = tmem + (static_cast<uint32_t>(wq * 32) << 16) + w * C::COLS;
  const bool leader = row == 0;  // of its warpgroup
  const uint64_t pol_out = l2_policy_evict_first();
  uint32_t kv = 0, qi = 0, tile = 0;
  uint32_t s_n[2] = {0, 0}, pre_n = 0, o_n = 0;  // phases of the S, o_pre and o_full barriers before this segment
  bool ok = true;
  auto wait = [&](uint64_t *bar, uint32_t par) {
    bool x = mbar_sleep(bar, par & 1, a.timeout_ns, ab);
    x = __all_sync(0xffffffffu, x);
    if (!x) ok = false;
    else tc_fence_after_sync();
    return x;
  };
  auto release = [&](uint32_t e) { mbar_arrive(&sc.empty[e % C::NSLOT]); };
  // The row's token (from the tile's first) and head of the group.
  const int half = a.tile_tokens >> 1, my_i = row / a.G, my_hg = row - my_i * a.G, my_tok = w * half + my_i;
  auto row_in = [&](const Segment &g) { return my_i < half && g.tok + my_tok < g.end; };
  SegmentReader<C> rd;
  while (const Segment *sg = ok ? rd.next(sc, a, ok) : nullptr) {
    const int n = sg->n, ns = sg->ns;
    const int lim = row_in(*sg) ? (a.causal ? min(max(sg->lim0 + my_tok, 0), sg->L) : sg->L) : sg->klim;
    const uint32_t qe = qi + w;
    qi += 2;
    float m_ref = -CUDART_INF_F, l = 0.f;
    bool own_scale = false;  // some row of the warp has a factor of its own
    if constexpr (C::ROW_SCALE) {
      if (!wait(&sc.q_full[qe % C::NQ], qe / C::NQ)) break;
      own_scale = __any_sync(0xffffffffu, sc.qrel[qe % C::NQ][row] != 0);
    }
    for (int j = 0; j < ns; ++j) {
      const int b = j & 1;
      if (!wait(&sc.s_full[w][b], s_n[b] + (j >> 1))) break;
      if constexpr (C::BITS8) {  // the converter's scales (complete: the product above used the same buffers)
        const uint32_t ke = kv + (j & ~1);
        if (!wait(&sc.full[ke % C::NSLOT], ke / C::NSLOT)) break;
      }
      const uint32_t s_addr = o_addr + D + b * kStepKeys;
      uint32_t x[kStepKeys];
      tmem_ld32(s_addr, *reinterpret_cast<uint32_t(*)[32]>(x));
      tmem_ld32(s_addr + 32, *reinterpret_cast<uint32_t(*)[32]>(x + 32));
      // The group that produced this S is complete, so this half has done with K of the unit (after its
      // last step), with V of the unit that ended two steps ago, and after the last S with its queries.
      // (8-bit keys: each warp speaks for itself about K, whose barrier it has just waited on: once the slot is refilled
      // that wait could no longer tell the phases apart)
      if ((C::BITS8 ? lane == 0 : leader) && (b == 1 || j == ns - 1)) release(kv + (j & ~1));
      if (leader && b == 1 && j >= 3) release(kv + j - 2);
      const int base = sg->u0 * kUnitKeys + j * kStepKeys;
      const int left = lim - base;  // keys of this step that the row sees
      float grow = 1.f, lsum = 0.f;  // root of the factor of O and l
      const float *kscale = C::BITS8 ? &sc.ks[(tile + (j >> 1)) % C::NSC][b * kStepKeys] : nullptr;
      const float *vscale = C::BITS8 ? &sc.vs[(tile + (j >> 1)) % C::NSC][b * kStepKeys] : nullptr;
      const float *lscale = C::BITS8 ? &sc.lv[(tile + (j >> 1)) % C::NSC][b * kStepKeys] : nullptr;
      // P = 2^(x f - m) of 32-column chunk c; f: the logit scale, a key's own scale, or 1 (PRE: x is
      // scaled already).
      auto exp_chunk = [&](int c, float neg_m, uint64_t(&acc)[2], auto pre_tag) {
        constexpr bool PRE = decltype(pre_tag)::value;
        const uint64_t nmp = f2(neg_m, neg_m);
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          [[maybe_unused]] float4 kk, vv;
          if constexpr (C::BITS8 && !PRE) kk = *reinterpret_cast<const float4 *>(kscale + c * 32 + 2 * e);
          if constexpr (C::BITS8) vv = *reinterpret_cast<const float4 *>(vscale + c * 32 + 2 * e);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const uint64_t v = f2(u2f_(x[c * 32 + 2 * (e + t)]), u2f_(x[c * 32 + 2 * (e + t) + 1]));
            uint64_t xx;
            if constexpr (PRE) xx = add2(v, nmp);
            else if constexpr (C::BITS8) xx = fma2(v, t ? f2(kk.z, kk.w) : f2(kk.x, kk.y), nmp);
            else xx = fma2(v, f2(a.scale_log2, a.scale_log2), nmp);
            float x0, x1, p0, p1;
            f2_split(xx, x0, x1);
            if (((kTilePolyMask >> ((e + t) % 8)) & 1u) != 0u) {
              exp2_poly_nan_x2(x0, x1, p0, p1);
            } else {
              p0 = ex2_approx(x0);
              p1 = ex2_approx(x1);
            }
            acc[t] = add2(acc[t], f2(p0, p1));
            if constexpr (C::BITS8) {
              p0 *= t ? vv.z : vv.x;
              p1 *= t ? vv.w : vv.y;
            }
            pk[e + t] = pack16<MT>(p0, p1);
          }
        }
        tmem_st16(s_addr + c * 16, pk);
      };
      auto total = [&](const uint64_t(&acc)[2]) {
        float t0, t1, t2, t3;
        f2_split(acc[0], t0, t1);
        f2_split(acc[1], t2, t3);
        return (t0 + t1) + (t2 + t3);
      };
      auto exp_fast = [&]() {
        uint64_t acc[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < 2; ++c) exp_chunk(c, -m_ref, acc, std::false_type{});
        lsum = total(acc);
        float most = lsum;  // of the probabilities that were packed
        if constexpr (C::BITS8) {
          const float4 w = *reinterpret_cast<const float4 *>(sc.wmax[(tile + (j >> 1)) % C::NSC]);
          most *= fmaxf(fmaxf(fmaxf(w.x, w.y), fmaxf(w.z, w.w)), 0x1p-85f);  // (and the sum itself is <= 2^100)
        }
        return __all_sync(0xffffffffu, most <= kTileSumLimit);
      };
      const bool plain = __all_sync(0xffffffffu, left >= kStepKeys);
      bool done = false;
      tmem_wait_ld();
      reg_fence<kStepKeys>(x);
      if (plain && !own_scale && __all_sync(0xffffffffu, m_ref != -CUDART_INF_F)) {
        done = exp_fast();
        if (!done) tmem_wait_st();
      }
      if (!done) {
        // With the row maximum (a NaN wins and takes the row): a row's first step, masked steps, and large values.
        [[maybe_unused]] float f1 = 1.f, g1 = 1.f;
        if constexpr (C::ROW_SCALE) {  // (two factors: their product may be below 2^-126)
          const int rel = sc.qrel[qe % C::NQ][row];
          f1 = __int_as_float((127 + (rel >> 1)) << 23);
          g1 = __int_as_float((127 + rel - (rel >> 1)) << 23);
        }
#pragma unroll
        for (int e = 0; e < kStepKeys; ++e) {
          float f = a.scale_log2;
          if constexpr (C::ROW_SCALE) f = kscale[e] * f1 * g1;
          else if constexpr (C::BITS8) f = kscale[e];
          x[e] = e < left ? __float_as_uint(u2f_(x[e]) * f) : __float_as_uint(-CUDART_INF_F);
        }
        float mxs[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
        for (int e = 0; e < kStepKeys; e += 2) {
          float z0 = u2f_(x[e]), z1 = u2f_(x[e + 1]);
          if constexpr (C::BITS8) z0 += lscale[e], z1 += lscale[e + 1];
          mxs[(e >> 1) & 3] = fmax3_nan(mxs[(e >> 1) & 3], z0, z1);
        }
        const float mx = fmax3_nan(mxs[0], mxs[1], fmax3_nan(mxs[2], mxs[3], mxs[3]));
        if (!(mx <= m_ref + kTileSlack)) {
          if (m_ref != -CUDART_INF_F) grow = ex2_approx(0.5f * (m_ref - mx));
          m_ref = mx;
        }
        const float ms = m_ref == -CUDART_INF_F ? 0.f : m_ref;
        uint64_t acc[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < 2; ++c)
          exp_chunk(c, -ms, acc, std::true_type{});
        // A maximum of +infinity or NaN makes the row NaN whatever the polynomial made of infinity - infinity; where no
        // key has weight the sum is 0, not the polynomial's least values.
        lsum = m_ref == -CUDART_INF_F ? 0.f : total(acc) + (ms - ms);
      }
      l = l * grow * grow + lsum;  // (the square may be below 2^-126 where l is above 2^100)
      if (j > 0 && __any_sync(0xffffffffu, grow != 1.f)) {
        const float alpha = grow * grow;
        // O is at rest once P V of the step before has completed: its commit is that of S(j + 1), if there is one.
        if (!(j + 1 < ns ? wait(&sc.s_full[w][b ^ 1], s_n[b ^ 1] + ((j + 1) >> 1)) : wait(&sc.o_pre[w], pre_n))) break;
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
      if (!C::BITS8 && j == ns - 1 && sg->L < base + 16 * step_slices(sg->klim, base)) {
        // The sequence ends inside this step. Both halves write the same zeros, each before its own product.
        const uint32_t ve = kv + (j & ~1) + 1;
        if (!wait(&sc.full[ve % C::NSLOT], ve / C::NSLOT)) break;
        uint8_t *v = ring + (ve % C::NSLOT) * C::HALF_BYTES + b * (kStepKeys * 128);
        const int r0 = max(sg->L - base, 0), r1 = 16 * step_slices(sg->klim, base);
        for (int e = row; e < (r1 - r0) * 8 * C::PANELS; e += 128) {
          const int r = r0 + e / (8 * C::PANELS), ch = e % (8 * C::PANELS);
          *reinterpret_cast<uint4 *>(v + (ch >> 3) * (128 * 128) + r * 128 + (ch & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async();
      }
      tmem_wait_st();
      tc_fence_before_sync();
      mbar_arrive(&sc.p_full[w][b]);
    }
    if (!ok) break;
    tile += n;
    // ---- the last P V of this half (and with it all before) is done: write its rows
    if (ns > 1 && !wait(&sc.o_pre[w], pre_n)) break;
    if (!wait(&sc.o_full[w], o_n)) break;
    pre_n += ns > 1 ? 1 : 0;
    ++o_n;
    s_n[0] += (ns + 1) >> 1;
    s_n[1] += ns >> 1;
    if (sg->part >= 0 && lane == 0) mbar_arrive(&sc.q_empty[qe % C::NQ]);  // (a complete tile's output goes through it)
    if (leader) {
      // values not returned yet: the steps released those of units before (last odd step - 1) / 2
      const int last = (ns - 1) & 1 ? ns - 1 : ns - 2;  // last odd step, or -1
      for (int i = last >= 3 ? (last - 1) / 2 : 0; i < n; ++i) release(kv + 2 * i + 1);
    }
    kv += 2 * n;
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
              make_float4(u2f_(o[e]), u2f_(o[e + 1]), u2f_(o[e + 2]), u2f_(o[e + 3]));
      }
      a.part_ml[slot * 512 + w * 128 + row] = m_ref;
      a.part_ml[slot * 512 + 256 + w * 128 + row] = l;
      tc_fence_before_sync();
      mbar_arrive(&sc.o_empty[w]);
    } else {
      // Complete rows: through this half's query buffer (every product with it is done), so that
      // a warp writes whole lines: its 32 rows one by one would touch 32 lines with every
      // store (measured: 3300 cycles a half, and the stores held up the barriers behind them).
      const float inv = l == 0.f ? 0.f : 1.f / l;  // a row that sees no key is zero
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
          // (rows behind the half's whole tokens stay zeros: no copy ever fills them)
          if (my_i < half) *reinterpret_cast<uint4 *>(buf + swz(row, c * 4 + e)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
      }
      tc_fence_before_sync();
      mbar_arrive(&sc.o_empty[w]);
      unsigned long long dst = reinterpret_cast<unsigned long long>(
          static_cast<QT *>(a.out) + sg->b * a.o_batch + static_cast<long long>(sg->tok + my_tok) * a.o_tok +
          static_cast<long long>(sg->h * a.G + my_hg) * a.o_head);
      if (!row_in(*sg) || !SOLATTN_DCHECK(row_inside(a, sg->b, sg->tok + my_tok, sg->h * a.G + my_hg), &sc.abort_flag, a.status)) dst = 0;
      __syncwarp();
      constexpr int LPR = D / 8, RPI = 32 / LPR;  // lanes of a row, rows of a store
      const int ch = lane % LPR;
#pragma unroll 8
      for (int r = 0; r < 32; r += RPI) {
        const int rr = r + lane / LPR;
        const unsigned long long ptr = __shfl_sync(0xffffffffu, dst, rr);
        const uint4 v = *reinterpret_cast<const uint4 *>(buf + swz(wq * 32 + rr, ch));
        if (ptr) st_global_v4_hint(reinterpret_cast<uint4 *>(ptr) + ch, v.x, v.y, v.z, v.w, pol_out);
      }
      // The next copy into the buffer is ordered behind these reads.
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sc.q_empty[qe % C::NQ]);
    }
    rd.done(sc);
  }
  if (!ok && lane == 0) tile_abort(&sc.abort_flag, a.status);
}

// ------------------------------------------------------------------ kernel

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    tile_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ DenseArgs a, const __grid_constant__ TileArgs x) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // The swizzled tiles need 1024-byte alignment, which the start of a block's shared memory has.
  uint8_t *base = smem_raw;
  if (smem_u32(smem_raw) & 1023u) {
    if (threadIdx.x == 0) {
      atomicCAS(a.status, 0, kStatusTimeoutTile);
      a.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
    }
    return;
  }
  uint8_t *q_smem = base;
  uint8_t *ring = base + C::NQ * C::HALF_BYTES;
  TileCtl<C> &sc = *reinterpret_cast<TileCtl<C> *>(ring + C::NSLOT * C::HALF_BYTES);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    const int fillers = C::BITS8 ? 128 : 1;  // converter threads, or the producer's expected bytes
    for (int i = 0; i < C::NSLOT; ++i) {
      mbar_init(&sc.full[i], fillers);
      mbar_init(&sc.empty[i], C::BITS8 && i % 2 == 0 ? 8 : 2);  // an arrival per half, or (K in the even slots) per softmax warp
    }
    for (int i = 0; i < C::NQ; ++i) {
      mbar_init(&sc.q_full[i], fillers);
      mbar_init(&sc.q_empty[i], 4);  // the half's softmax warps
    }
    for (int w = 0; w < 2; ++w) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(&sc.s_full[w][b], 1);
        mbar_init(&sc.p_full[w][b], 128);
      }
      mbar_init(&sc.o_pre[w], 1);
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
    // Rows behind a half's whole tokens are never copied and never written again: zeros, so that their scores are finite
    // (a NaN among them would send its warp down the slow softmax path with every tile).
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
  else if constexpr (C::BITS8) regs_inc<C::CONV_REGS>();
  if (warp < 4) {
    if (warp == 0) {
      if constexpr (!C::BITS8) {
        tile_producer<C>(sc, a, x, q_smem, ring, &tm_q, &tm_k, &tm_v, lane);
      }
    } else if (warp == 2) {
      tile_scheduler<C>(sc, a, x, lane);
    } else {
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
