// dense_common.cuh -- what the dense attention kernels share: the description of a call,
// the schedule of its work over the blocks of a launch, and the kernel that joins rows
// whose keys were split over several blocks.
//
// A call attends B sequences: sequence b has n_b query tokens and L_b keys, and every key
// head serves G query heads. The rows of one (sequence, key head) are its (token, query
// head of the group) pairs, token-major, so shared key heads fill a tile's rows and every
// key is read once for all of them. The rows are cut into tiles; the keys into units of 128.
//
// Schedule. The units of all (sequence, key head, row tile) items, in that order, each item's behind a few
// places that stand for its fixed cost (queries in, rows out), form one
// line of W places, which the P blocks of the launch share evenly: block c takes places
// [c W / P, (c + 1) W / P). Lengths live on the device, so the line is laid out there: each
// warp scans the sequences' work once at its start (B values, 32 at a time). A block whose
// range begins or ends inside an item leaves an unnormalised partial result (row maximum,
// row sum, 32-bit output) in the workspace, and a second launch joins each split item's
// parts in the order of the blocks, so results do not depend on timing. With many more
// items than blocks the split would only add that traffic: then a block takes the items
// that BEGIN in its range, whole.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include "debug_check.cuh"
#include "ptx_sm100.cuh"

namespace solattn {

constexpr int kStatusTable = -7;  // a page table entry or a length is out of range
constexpr int kUnitKeys = 128;    // keys of one unit of work

// Kinds of cached rows.
constexpr int kKind16 = 0, kKindInt8 = 1, kKindE4m3 = 2;

struct DenseArgs {
  const void *q;
  void *out;
  long long q_tok, q_head, q_batch;  // strides in elements
  long long o_tok, o_head, o_batch;
  // Keys and values: rows of a (batch, head) of a tensor, or of a (page, head) of the cache.
  const void *k, *v;
  long long k_row, k_head, k_seq, v_row, v_head, v_seq;  // strides in elements
  const float *k_scale, *v_scale;  // [page][head][row], 8-bit caches
  const int *table;                // [B][width], or null: contiguous keys
  int width, page, page_shift, num_pages;
  const int *cu;   // [B + 1] first query row of each sequence, or null: n rows each
  const int *len;  // [B] keys of each sequence, or null: Lmax
  int B, Hkv, G, n, total, Lmax, causal;
  float scale_log2;  // log2(e) / sqrt(d)
  int tile_tokens;   // tile kernel: query tokens of a tile (rows kernel: unused)
  int4 *desc;        // [P] {parts, b, h, t} of the item that block c begins and others end
  float *part_ml;    // [2 P][2][rows]
  float *part_o;     // [2 P][rows][d]
  int *status;
  unsigned long long timeout_ns;
};

struct Seq {
  int n, L, tok0;
};

// What the debug build checks before an access: a row of the queries or the output, a key's place (page or batch, row in it),
// a partial result's slot.
__device__ __forceinline__ bool row_inside(const DenseArgs &a, int b, int tok, int head) {
  return b >= 0 && b < a.B && tok >= 0 && tok < (a.cu ? a.total : a.n) && head >= 0 && head < a.Hkv * a.G;
}
__device__ __forceinline__ bool key_inside(const DenseArgs &a, int at, int row) {
  return at >= 0 && at < (a.table ? a.num_pages : a.B) && row >= 0 && row < (a.table ? a.page : a.Lmax);
}
__device__ __forceinline__ bool slot_inside(int slot, int blocks) { return slot >= 0 && slot < 2 * blocks; }

// Query tokens, keys and first query row of sequence b. Values outside the call's buffers
// are cut to them, so that no access depends on unchecked device data. The cache calls (CacheArgs)
// cut them the same way: what a call writes is what the attention over it assumes.
template <class A>
__device__ __forceinline__ int first_row(const A &a, int cu) { return min(max(cu, 0), a.total); }
template <class A>
__device__ __forceinline__ int keys_of(const A &a, int b) {
  return a.len ? min(max(__ldg(a.len + b), 0), a.Lmax) : a.Lmax;
}
template <class A>
__device__ __forceinline__ Seq seq_of(const A &a, int b) {
  Seq s;
  if (a.cu) {
    const int lo = first_row(a, __ldg(a.cu + b));
    const int hi = max(first_row(a, __ldg(a.cu + b + 1)), lo);
    s.tok0 = lo;
    s.n = hi - lo;
  } else {
    s.tok0 = 0;
    s.n = a.n;
  }
  s.L = keys_of(a, b);
  return s;
}

// Keys that query token i of a sequence sees: all of them, or those up to its own position.
__device__ __forceinline__ int key_limit(const DenseArgs &a, const Seq &s, int tok) {
  if (!a.causal) return s.L;
  return min(max(s.L - s.n + tok + 1, 0), s.L);
}

// Rows kernel: a tile is RT consecutive rows, whatever tokens they belong to.
template <int RT_>
struct RowTiles {
  static constexpr int RT = RT_;
  static constexpr int COST = 1;  // an item's fixed cost in units
  static __device__ __forceinline__ int tiles(const DenseArgs &a, int n) { return (n * a.G + RT - 1) / RT; }
  static __device__ __forceinline__ int last_token(const DenseArgs &a, int n, int t) {
    return (min(n * a.G, (t + 1) * RT) - 1) / a.G;
  }
  static __device__ __forceinline__ bool row(const DenseArgs &a, int n, int t, int r, int &tok, int &g) {
    const int x = t * RT + r;
    tok = x / a.G;
    g = x - tok * a.G;
    return x < n * a.G;
  }
};

// Tile kernel: two halves of 128 rows, each tile_tokens / 2 whole tokens (the rows behind
// the last whole token of a half are empty), as a box copy of (heads of the group, tokens) lays them.
struct TokenTiles {
  static constexpr int RT = 256;
  // A tile costs about 5500 cycles and 3700 a unit. (Without it blocks of many short items finish last: a
  // batch of prompts of 0 to 256 keys lost 15 % to that.)
  static constexpr int COST = 2;
  static __device__ __forceinline__ int tiles(const DenseArgs &a, int n) {
    return (n + a.tile_tokens - 1) / a.tile_tokens;
  }
  static __device__ __forceinline__ int last_token(const DenseArgs &a, int n, int t) {
    return min(n, (t + 1) * a.tile_tokens) - 1;
  }
  static __device__ __forceinline__ bool row(const DenseArgs &a, int n, int t, int r, int &tok, int &g) {
    const int half = a.tile_tokens >> 1, rr = r & 127;
    const int i = rr / a.G;
    g = rr - i * a.G;
    tok = t * a.tile_tokens + (r >> 7) * half + i;
    return i < half && tok < n;
  }
};

template <class T>
__device__ __forceinline__ int item_units(const DenseArgs &a, const Seq &s, int t) {
  return max(1, (key_limit(a, s, T::last_token(a, s.n, t)) + kUnitKeys - 1) / kUnitKeys);
}

// Places of one key head of sequence b.
template <class T>
__device__ __forceinline__ long long head_places(const DenseArgs &a, const Seq &s) {
  const int tiles = T::tiles(a, s.n);
  if (!a.causal) return static_cast<long long>(tiles) * (T::COST + max(1, (s.L + kUnitKeys - 1) / kUnitKeys));
  long long w = 0;
  for (int t = 0; t < tiles; ++t) w += T::COST + item_units<T>(a, s, t);
  return w;
}

// A block's walk over its range of the line. Every thread of the warp calls begin(); after
// it the cursor is the same in every lane and step() needs no other lane.
template <class T>
struct Cursor {
  long long x, x1, W;  // next place, end of the range, length of the line
  int P;               // blocks that share the line
  bool whole;
  Seq s;
  int b, h, t, tiles, units, o0, o1, u0, u1;  // o0, o1: the segment's places in its item; u0, u1: its units

  __device__ __forceinline__ long long bound(int c) const { return W * c / P; }

  // min_units: a block's share is at least so many units where the items alone do not fill
  // the launch. whole_items: with at least so many items per block, items are not split.
  __device__ __forceinline__ bool begin(const DenseArgs &a, int c, int blocks, int min_units, int whole_items) {
    const int lane = threadIdx.x & 31;
    long long w_all = 0, items = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      long long w = 0, it = 0;
      if (b0 + lane < a.B) {
        const Seq q = seq_of(a, b0 + lane);
        w = head_places<T>(a, q) * a.Hkv;
        it = static_cast<long long>(T::tiles(a, q.n)) * a.Hkv;
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        w += __shfl_xor_sync(0xffffffffu, w, o);
        it += __shfl_xor_sync(0xffffffffu, it, o);
      }
      w_all += w;
      items += it;
    }
    W = w_all;
    whole = items >= static_cast<long long>(whole_items) * blocks;
    const long long want = max(items, (W + min_units - 1) / min_units);
    P = static_cast<int>(min(static_cast<long long>(blocks), max(want, 1ll)));
    if (c >= P || W == 0) return false;
    x = bound(c);
    x1 = bound(c + 1);
    if (x >= x1) return false;
    long long before = 0, rem = 0;
    int found = -1;
    for (int b0 = 0; b0 < a.B && found < 0; b0 += 32) {
      long long w = 0;
      if (b0 + lane < a.B) w = head_places<T>(a, seq_of(a, b0 + lane)) * a.Hkv;
      long long incl = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, before + incl > x);
      if (hit) {
        const int l = __ffs(hit) - 1;
        found = b0 + l;
        rem = x - before - __shfl_sync(0xffffffffu, incl - w, l);
      } else {
        before += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    b = found;
    s = seq_of(a, b);
    tiles = T::tiles(a, s.n);
    const long long per_head = head_places<T>(a, s);
    h = static_cast<int>(rem / per_head);
    rem -= per_head * h;
    t = 0;
    if (!a.causal) {
      units = item_units<T>(a, s, 0);
      t = static_cast<int>(rem / (T::COST + units));
      rem -= static_cast<long long>(T::COST + units) * t;
    } else {
      for (;; ++t) {
        units = item_units<T>(a, s, t);
        if (rem < T::COST + units) break;
        rem -= T::COST + units;
      }
    }
    o0 = static_cast<int>(rem);
    if (whole && o0 > 0) {  // the item begins in an earlier block's range
      x += T::COST + units - o0;
      next_item(a);
      if (x >= x1 || b >= a.B) return false;
    }
    return set_end();
  }

  // False where the range ends before the item's first unit: the next block then takes the item.
  __device__ __forceinline__ bool set_end() {
    const int span = T::COST + units;
    o1 = whole ? span : static_cast<int>(min(static_cast<long long>(span), o0 + (x1 - x)));
    u0 = max(0, o0 - T::COST);
    u1 = max(0, o1 - T::COST);
    return u1 > 0;
  }

  __device__ __forceinline__ void next_item(const DenseArgs &a) {
    o0 = 0;
    if (++t == tiles) {
      t = 0;
      if (++h == a.Hkv) {
        h = 0;
        tiles = 0;
        while (tiles == 0 && ++b < a.B) {
          s = seq_of(a, b);
          tiles = T::tiles(a, s.n);
        }
        if (b >= a.B) return;
      }
    }
    units = item_units<T>(a, s, t);
  }

  // The next segment of the range; false at its end.
  __device__ __forceinline__ bool step(const DenseArgs &a) {
    x += o1 - o0;
    if (x >= x1) return false;
    next_item(a);
    if (b >= a.B) return false;
    return set_end();
  }

  __device__ __forceinline__ bool partial() const { return u0 > 0 || u1 < units; }
  __device__ __forceinline__ int slot(int c) const { return 2 * c + (u0 > 0 ? 0 : 1); }
  // The record of an item that this block begins and other blocks end.
  __device__ __forceinline__ int4 record(int c) const {
    int e = c;
    while (bound(e + 1) < x - o0 + T::COST + units) ++e;
    return make_int4(e - c + 1, b, h, t);
  }
};

// Physical page of key position j (a multiple of 16) of sequence b, or -1 (recorded) where
// the table names no page of the cache: such keys read as zeros.
__device__ __forceinline__ int page_of(const DenseArgs &a, int b, int j) {
  if (!SOLATTN_DCHECK_STATUS(b >= 0 && b < a.B && j >= 0 && j < a.Lmax, a.status)) return -1;
  const int id = __ldg(a.table + static_cast<size_t>(b) * a.width + (j >> a.page_shift));
  if (static_cast<unsigned>(id) < static_cast<unsigned>(a.num_pages)) return id;
  atomicCAS(a.status, 0, kStatusTable);
  return -1;
}

// Lengths that seq_of had to cut are recorded once per call, by one warp of block 0.
template <class A>
__device__ __forceinline__ void check_lengths(const A &a) {
  for (int b = threadIdx.x & 31; b < a.B; b += 32) {
    bool bad = false;
    if (a.cu) bad = a.cu[b] < 0 || a.cu[b + 1] < a.cu[b] || a.cu[b + 1] > a.total;
    if (a.len) bad |= a.len[b] < 0 || a.len[b] > a.Lmax;
    if (a.cu && !bad) {  // the new tokens are the sequence's last
      const Seq s = seq_of(a, b);
      bad = s.L < s.n;
    }
    if (bad) atomicCAS(a.status, 0, kStatusTable);
  }
}

template <class QT>
__device__ __forceinline__ uint32_t pack16(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack16<__nv_bfloat16>(float lo, float hi) { return pack_bf16x2(lo, hi); }
template <>
__device__ __forceinline__ uint32_t pack16<__half>(float lo, float hi) { return pack_f16x2(lo, hi); }

__device__ __forceinline__ float u2f_(uint32_t x) { return __uint_as_float(x); }

__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Joins the parts of each split item: o = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i with
// m the largest m_i (l_i times the root of its factor twice: see the rows kernel on 8-bit caches), in the order of the blocks that wrote them. Grid (P, row chunks): the
// blocks of column c take the item that block c of the attention launch begins, if others
// end it; most have none. Reads 4 (d + 2) bytes a row and part. Launched as a programmatic
// dependent: it is resident when the attention ends, which saves the gap between launches.
template <class T, class QT, int D, int ROWS>
__global__ void __launch_bounds__(256) join_kernel(const DenseArgs a) {
  pdl_wait();
  const int c = blockIdx.x;
  const int4 rec = a.desc[c];
  const int parts = rec.x;
  if (parts == 0) return;
  if (!SOLATTN_DCHECK_STATUS(parts > 0 && c + parts <= static_cast<int>(gridDim.x) && rec.y >= 0 && rec.y < a.B, a.status)) return;
  const Seq s = seq_of(a, rec.y);
  if constexpr (T::RT == TokenTiles::RT) {
    // Parts lie column group by column group: a warp reads 32 rows of a group of 4 columns
    // at a time and the results turn through shared memory, so that rows are written whole.
    __shared__ alignas(16) uint2 out[ROWS][D / 4 + 1];
    static_assert(ROWS % 32 == 0 && 128 % ROWS == 0, "rows of a warp share a half");
    for (int i = threadIdx.x; i < ROWS * (D / 4); i += 256) {
      const int rl = i % ROWS, e = i / ROWS, r = blockIdx.y * ROWS + rl;
      float m = -CUDART_INF_F;
      for (int p = 0; p < parts; ++p) m = fmaxf(m, a.part_ml[static_cast<size_t>(p == 0 ? 2 * c + 1 : 2 * (c + p)) * 512 + r]);
      float l = 0.f, o0 = 0.f, o1 = 0.f, o2 = 0.f, o3 = 0.f;
      const float ms = m == -CUDART_INF_F ? 0.f : m;
      for (int p = 0; p < parts; ++p) {
        const size_t sl = p == 0 ? 2 * c + 1 : 2 * (c + p);
        const float root = ex2_approx(0.5f * (a.part_ml[sl * 512 + r] - ms)), w = root * root;
        l = fmaf(root, root * a.part_ml[sl * 512 + 256 + r], l);
        const float4 x = *reinterpret_cast<const float4 *>(a.part_o + ((sl * 2 + (r >> 7)) * (D / 4) + e) * 512 + (r & 127) * 4);
        o0 = fmaf(w, x.x, o0);
        o1 = fmaf(w, x.y, o1);
        o2 = fmaf(w, x.z, o2);
        o3 = fmaf(w, x.w, o3);
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;  // a row that sees no key is zero
      out[rl][e] = make_uint2(pack16<QT>(o0 * inv, o1 * inv), pack16<QT>(o2 * inv, o3 * inv));
    }
    __syncthreads();
    for (int i = threadIdx.x; i < ROWS * (D / 4); i += 256) {
      const int rl = i / (D / 4), e = i % (D / 4);
      int tok, g;
      if (!T::row(a, s.n, rec.w, blockIdx.y * ROWS + rl, tok, g)) continue;
      if (!SOLATTN_DCHECK_STATUS(row_inside(a, rec.y, s.tok0 + tok, rec.z * a.G + g), a.status)) continue;
      QT *dst = static_cast<QT *>(a.out) + rec.y * a.o_batch + static_cast<long long>(s.tok0 + tok) * a.o_tok +
                static_cast<long long>(rec.z * a.G + g) * a.o_head + 4 * e;
      *reinterpret_cast<uint2 *>(dst) = out[rl][e];
    }
    return;
  }
  // A warp for each row: lane p reads the maximum and sum of part p, then every lane adds up its columns, several
  // parts in flight (one part after the other cost 600 cycles for each of them).
  constexpr int CPL = D / 32;  // columns of a lane
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = warp; i < ROWS; i += 8) {
    const int r = blockIdx.y * ROWS + i;
    int tok, g;
    if (!T::row(a, s.n, rec.w, r, tok, g)) continue;
    if (!SOLATTN_DCHECK_STATUS(row_inside(a, rec.y, s.tok0 + tok, rec.z * a.G + g), a.status)) continue;
    float m = -CUDART_INF_F, l = 0.f, o[CPL];
#pragma unroll
    for (int e = 0; e < CPL; ++e) o[e] = 0.f;
    for (int p0 = 0; p0 < parts; p0 += 32) {
      const int p = p0 + lane;
      const size_t sl = p == 0 ? 2 * c + 1 : 2 * (c + p);
      const bool in = p < parts;
      const float mp = in ? a.part_ml[sl * 2 * T::RT + r] : -CUDART_INF_F;
      float lp = in ? a.part_ml[sl * 2 * T::RT + T::RT + r] : 0.f;
      float mx = mp;
#pragma unroll
      for (int off = 16; off; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      const float mn = fmaxf(m, mx), ms = mn == -CUDART_INF_F ? 0.f : mn;
      const float old_root = ex2_approx(0.5f * (m - ms)), root = ex2_approx(0.5f * (mp - ms));  // (0 for -infinity)
      const float old = old_root * old_root, w = root * root;
      lp = lp * root * root;
#pragma unroll
      for (int off = 16; off; off >>= 1) lp += __shfl_xor_sync(0xffffffffu, lp, off);
      l = fmaf(l * old_root, old_root, lp);
#pragma unroll
      for (int e = 0; e < CPL; ++e) o[e] *= old;
      m = mn;
      const int np = min(32, parts - p0);
#pragma unroll 8
      for (int q = 0; q < np; ++q) {
        const float wq = __shfl_sync(0xffffffffu, w, q);
        const size_t sq = p0 + q == 0 ? 2 * c + 1 : 2 * (c + p0 + q);
        const float *src = a.part_o + (sq * T::RT + r) * D + CPL * lane;
        if constexpr (CPL == 4) {
          const float4 x = *reinterpret_cast<const float4 *>(src);
          o[0] = fmaf(wq, x.x, o[0]);
          o[1] = fmaf(wq, x.y, o[1]);
          o[2] = fmaf(wq, x.z, o[2]);
          o[3] = fmaf(wq, x.w, o[3]);
        } else {
          const float2 x = *reinterpret_cast<const float2 *>(src);
          o[0] = fmaf(wq, x.x, o[0]);
          o[1] = fmaf(wq, x.y, o[1]);
        }
      }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;  // a row that sees no key is zero
    QT *dst = static_cast<QT *>(a.out) + rec.y * a.o_batch + static_cast<long long>(s.tok0 + tok) * a.o_tok +
              static_cast<long long>(rec.z * a.G + g) * a.o_head + CPL * lane;
    if constexpr (CPL == 4)
      *reinterpret_cast<uint2 *>(dst) = make_uint2(pack16<QT>(o[0] * inv, o[1] * inv), pack16<QT>(o[2] * inv, o[3] * inv));
    else
      *reinterpret_cast<uint32_t *>(dst) = pack16<QT>(o[0] * inv, o[1] * inv);
  }
}

}  // namespace solattn
