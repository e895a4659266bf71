// dense_api.cu -- host side of the dense attention entry points and of the cache: argument
// checks, choice of kernel, launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "cache_kernel.cuh"
#include "dense_common.cuh"
#include "host_common.h"
#include "rows_kernel.cuh"
#include "solattn.h"
#include "tile_kernel.cuh"

namespace {

using namespace solattn;

constexpr size_t kHeader = 256;  // [4]: status word
// Limit of a wait on the device. Some last as long as a block's work on one tile (the next queries' buffer, a place for the next
// segment): 10 us more for each unit of keys that a sequence may have, where a unit takes 1 to 4.
constexpr unsigned long long kTimeoutNs = 2000000000ull, kTimeoutUnitNs = 10000ull;
constexpr int kMaxSms = 160;     // blocks per SM slot that the workspace provides for
constexpr int kRowsBlocks1 = rows_blocks(1) * kMaxSms, kRowsBlocks2 = rows_blocks(2) * kMaxSms;

// Workspace: header, one record per block, then maxima and sums, then outputs of the parts.
struct DenseWs {
  size_t desc, ml, o, total;
};
DenseWs dense_ws(int d) {
  // the larger of the kernels' needs: two parts per block
  const size_t rows = 2 * static_cast<size_t>(kMaxSms) * TokenTiles::RT;
  static_assert(kRowsBlocks1 * 8 <= kMaxSms * TokenTiles::RT && kRowsBlocks2 * 16 <= kMaxSms * TokenTiles::RT, "part rows");
  DenseWs w;
  w.desc = kHeader;
  w.ml = w.desc + align_up(sizeof(int4) * kRowsBlocks1, kAlign);
  w.o = w.ml + align_up(rows * 2 * sizeof(float), kAlign);
  w.total = w.o + align_up(rows * d * sizeof(float), kAlign);
  return w;
}

bool heads_ok(int H, int Hkv) { return H >= 1 && Hkv >= 1 && H % Hkv == 0; }

// Strides of a view that the kernels can follow: 16-byte steps, and for an output no step of zero.
bool view_ok(const solattn_view *x, int elem, bool output, int64_t nb, int64_t nh, int64_t nn) {
  if (!x || !x->ptr || !aligned(x->ptr, 16)) return false;
  const int64_t step = 16 / elem;
  const int64_t st[3] = {x->stride_b, x->stride_h, x->stride_n};
  const int64_t ext[3] = {nb, nh, nn};
  for (int i = 0; i < 3; ++i) {
    if (ext[i] <= 1) continue;
    if (st[i] < 0 || st[i] % step != 0 || (output && st[i] == 0)) return false;
  }
  return true;
}

int check_device(std::initializer_list<const void *> ptrs, DeviceInfo *di) {
  if (device_info(di) != SOLATTN_OK) return SOLATTN_ECUDA;
  if (di->major != 10) return SOLATTN_EUNSUPPORTED;
  if (di->devices == 1) return SOLATTN_OK;  // no other GPU for a pointer to belong to
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SOLATTN_ECUDA;
  for (const void *p : ptrs)
    if (p && foreign_device_pointer(p, dev)) return SOLATTN_EINVAL;
  return SOLATTN_OK;
}

int check_cache(const solattn_cache *c) {
  if (!c) return SOLATTN_EINVAL;
  if (c->num_pages < 1 || c->Hkv < 1) return SOLATTN_EINVAL;
  if (c->kind < SOLATTN_CACHE_16 || c->kind > SOLATTN_CACHE_E4M3) return SOLATTN_EINVAL;
  if (c->d != 64 && c->d != 128) return SOLATTN_EUNSUPPORTED;
  if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) return SOLATTN_EUNSUPPORTED;
  const int elem = c->kind == SOLATTN_CACHE_16 ? 2 : 1;
  if (!view_ok(&c->k, elem, true, c->num_pages, c->Hkv, c->page) || !view_ok(&c->v, elem, true, c->num_pages, c->Hkv, c->page))
    return SOLATTN_EINVAL;
  if (c->kind != SOLATTN_CACHE_16 &&
      (!c->k_scale || !c->v_scale || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4)))
    return SOLATTN_EINVAL;
  return SOLATTN_OK;
}

int check_seqs(const solattn_seqs *s, int page) {
  if (!s || s->B < 1 || s->total < 0 || s->width < 1) return SOLATTN_EINVAL;
  if (!s->table || !s->cu || !s->len) return SOLATTN_EINVAL;
  if (!aligned(s->table, 4) || !aligned(s->cu, 4) || !aligned(s->len, 4)) return SOLATTN_EINVAL;
  if (static_cast<long long>(s->width) * page > (1ll << 30)) return SOLATTN_EUNSUPPORTED;  // positions are 32-bit
  return SOLATTN_OK;
}

int page_shift(int page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7; }

// A launch that may begin while the launch before it ends (its kernel waits for the data).
template <class K, class... Args>
bool launch(K kernel, dim3 grid, dim3 block, cudaStream_t st, bool dependent, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess;
}

// Items of a call with at least 6 times as many as blocks are not split: the uneven share of the last
// items costs less than the parts' traffic.
constexpr int kWholeItems = 6;

// Whether some item may be split over blocks. It is not where no item has more units than the least
// share of a block, nor where a uniform call has items enough; then nothing needs joining.
template <class T>
bool may_split(const DenseArgs &a, int blocks, int min_units) {
  if (a.Lmax <= min_units * kUnitKeys) return false;
  if (a.cu) return true;  // the host does not know the lengths
  const long long per_head = T::RT == TokenTiles::RT ? (a.n + a.tile_tokens - 1) / a.tile_tokens
                                                     : (static_cast<long long>(a.n) * a.G + T::RT - 1) / T::RT;
  return per_head * a.B * a.Hkv < static_cast<long long>(kWholeItems) * blocks;
}

template <class QT, int KIND, int D, int NT, bool PAGED>
int launch_rows(const DenseArgs &a, int sms, cudaStream_t st) {
  using T = RowTiles<8 * NT>;
  const int blocks = rows_blocks(NT) * sms;
  // A block's share is at least two units (256 keys) when the items alone do not fill the launch.
  constexpr int min_units = 2;
  const bool split = may_split<T>(a, blocks, min_units);
  if (!launch(rows_kernel<QT, KIND, D, NT, PAGED>, blocks, kRowsWarps * 32, st, false, a, min_units, split ? kWholeItems : 0))
    return SOLATTN_ECUDA;
  if (split && !launch(join_kernel<T, QT, D, T::RT>, blocks, 256, st, true, a)) return SOLATTN_ECUDA;
  return SOLATTN_OK;
}

// 16-bit tensor maps. Queries: (d, head of the group, token, key head, batch), boxes of 64 x G x tokens of
// a half. Keys and values: (d, row, head, batch or page), boxes of 64 x rows. A dimension of stride zero has
// extent one. Everything outside reads as zeros.
int encode(CUtensorMap *map, int dtype, int rank, const void *ptr, const cuuint64_t *dims, const long long *strides, const cuuint32_t *box) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return SOLATTN_ECUDA;
  cuuint64_t dm[5], st[4];
  cuuint32_t one[5] = {1, 1, 1, 1, 1};
  for (int i = 0; i < rank; ++i) dm[i] = dims[i];
  for (int i = 1; i < rank; ++i) {
    if (dm[i] > 1 && strides[i] == 0) dm[i] = 1;
    st[i - 1] = dm[i] > 1 ? static_cast<cuuint64_t>(strides[i]) * 2 : 16;
  }
  const CUresult r = enc(map, dtype == SOLATTN_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank,
                         const_cast<void *>(ptr), dm, st, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? SOLATTN_OK : SOLATTN_ECUDA;
}

// Whether the tile kernel can take the call: its copies need a token step in Q, K and V that is not
// zero, strides below 2^40 bytes, and a group of heads that fits half a tile.
bool tile_fits(const DenseArgs &a, int kind) {
  if (a.G > 128 || a.Lmax == 0) return false;
  if (kind != SOLATTN_CACHE_16) return true;  // no tensor maps
  const long long most = 1ll << 39;
  const long long st[] = {a.q_tok, a.q_head * a.G, a.q_batch, a.k_row, a.k_head, a.k_seq, a.v_row, a.v_head, a.v_seq};
  for (long long x : st)
    if (x >= most) return false;
  if (a.q_tok == 0 && (a.cu ? a.total : a.n) > 1) return false;
  if (a.q_head == 0 && a.G * a.Hkv > 1) return false;
  if (!a.cu && a.q_batch == 0 && a.B > 1) return false;
  if (!a.table && a.Lmax > 1 && (a.k_row == 0 || a.v_row == 0)) return false;
  return true;
}

template <class QT, int KIND, int D, bool PAGED>
int launch_tiles(DenseArgs a, int dtype, int sms, cudaStream_t st) {
  using C = TileCfg<QT, KIND, D, PAGED>;
  constexpr size_t smem = tile_smem_bytes<C>();
  static_assert(smem <= 232448, "shared memory");
  auto kern = tile_kernel<C>;
  static bool attr_set[64] = {};  // per device; guarded by g_mu
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SOLATTN_ECUDA;
  {
    std::lock_guard<std::mutex> lk(g_mu);
    if (!attr_set[dev]) {
      if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
        return SOLATTN_ECUDA;
      attr_set[dev] = true;
    }
  }
  const int half = 128 / a.G;
  a.tile_tokens = 2 * half;
  TileArgs x{};
  // The uneven share of whole items is at most one item per block: below 1/6 of a block's work. A part
  // costs about as much as two units of keys: a block's share of a split item is at least four.
  x.min_units = 4;
  const bool split = may_split<TokenTiles>(a, sms, x.min_units);
  x.whole_items = split ? kWholeItems : 0;
  CUtensorMap mq{}, mk{}, mv{};
  if constexpr (!C::BITS8) {
    const cuuint64_t ntok = a.cu ? a.total : a.n;
    const cuuint64_t qd[5] = {D, static_cast<cuuint64_t>(a.G), ntok, static_cast<cuuint64_t>(a.Hkv),
                              static_cast<cuuint64_t>(a.cu ? 1 : a.B)};
    const cuuint32_t qb[5] = {64, static_cast<cuuint32_t>(a.G), static_cast<cuuint32_t>(half), 1, 1};
    const long long qs[5] = {1, a.q_head, a.q_tok, a.q_head * a.G, a.q_batch};
    const cuuint64_t kd[4] = {D, static_cast<cuuint64_t>(PAGED ? a.page : a.Lmax), static_cast<cuuint64_t>(a.Hkv),
                              static_cast<cuuint64_t>(PAGED ? a.num_pages : a.B)};
    const long long ks[4] = {1, a.k_row, a.k_head, a.k_seq}, vs[4] = {1, a.v_row, a.v_head, a.v_seq};
    const cuuint32_t kb[4] = {64, static_cast<cuuint32_t>(PAGED ? a.page : kUnitKeys), 1, 1};
    if (encode(&mq, dtype, 5, a.q, qd, qs, qb) != SOLATTN_OK || encode(&mk, dtype, 4, a.k, kd, ks, kb) != SOLATTN_OK ||
        encode(&mv, dtype, 4, a.v, kd, vs, kb) != SOLATTN_OK)
      return SOLATTN_ECUDA;
    x.k_b = a.k_seq != 0, x.k_h = a.k_head != 0, x.v_b = a.v_seq != 0, x.v_h = a.v_head != 0;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(sms);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  if (cudaLaunchKernelEx(&cfg, kern, mq, mk, mv, a, x) != cudaSuccess) return SOLATTN_ECUDA;
  if (split && !launch(join_kernel<TokenTiles, QT, D, 32>, dim3(sms, TokenTiles::RT / 32), 256, st, true, a)) return SOLATTN_ECUDA;
  return SOLATTN_OK;
}

// Which kernel is sooner done, by what each costs (us, d = 128): a start, a share for each item of a block, a share for
// each unit of keys, and the join of split items. Fitted to, rows kernel against tile kernel (B, Hkv, Nq, Nk):
// (1, 8, 256, 256) 10.4 against 11.9, (1, 8, 1024, 256) 17.2 : 12.3, (1, 8, 2048, 512) 49.6 : 16.4, (2, 8, 32, 4096) 23.3 :
// 33.2, (1, 8, 128, 2048) 22.4 : 25.3, (4, 16, 1024, 128) 70.4 : 16.4, (1, 1, 100, 4096) 21.6 : 30.7. Over a cache the
// longest sequence that the table could name stands for all of them.
bool tiles_faster(const DenseArgs &a, int sms) {
  const int tile_tokens = 2 * (128 / a.G);
  auto estimate = [&](double per_head, double blocks, double least, double start, double item, double unit, double join) {
    const double items = per_head * a.Hkv, units = a.Lmax > 32 ? a.Lmax / 128.0 : 0.25;
    const double share = items * units / blocks, floor = units < least ? units : least;
    return start + item * (items > blocks ? items / blocks : 1.0) + unit * (share > floor ? share : floor) +
           (items < blocks && units > least ? join : 0.0);
  };
  const double n = a.cu ? a.total : a.n, copies = a.cu ? 1 : a.B;
  auto ceil_div = [](double x, double y) { return std::ceil(x / y); };
  double row_tiles = copies * ceil_div(n * a.G, 16), tiles = copies * ceil_div(n, tile_tokens);
  if (a.cu) {  // every sequence has a tile of its own
    row_tiles = row_tiles > a.B ? row_tiles : a.B;
    tiles = tiles > a.B ? tiles : a.B;
  }
  return estimate(tiles, sms, 4, 6.0, 2.9, 1.95, 5.0) < estimate(row_tiles, 2.0 * sms, 2, 5.0, 2.2, 2.4, 3.0);
}

template <class QT, int KIND, int D, bool PAGED>
int dispatch_rows(const DenseArgs &a, int dtype, int rows, int sms, cudaStream_t st) {
  constexpr int kind = KIND == kKind16 ? SOLATTN_CACHE_16 : KIND == kKindInt8 ? SOLATTN_CACHE_INT8 : SOLATTN_CACHE_E4M3;
  if (rows > 16 && tile_fits(a, kind) && tiles_faster(a, sms)) return launch_tiles<QT, KIND, D, PAGED>(a, dtype, sms, st);
  return rows <= 8 ? launch_rows<QT, KIND, D, 1, PAGED>(a, sms, st) : launch_rows<QT, KIND, D, 2, PAGED>(a, sms, st);
}

template <class QT, int D>
int dispatch_kind(const DenseArgs &a, int dtype, int kind, int rows, int sms, cudaStream_t st) {
  if (!a.table) return dispatch_rows<QT, kKind16, D, false>(a, dtype, rows, sms, st);
  if (kind == SOLATTN_CACHE_16) return dispatch_rows<QT, kKind16, D, true>(a, dtype, rows, sms, st);
  if (kind == SOLATTN_CACHE_INT8) return dispatch_rows<QT, kKindInt8, D, true>(a, dtype, rows, sms, st);
  return dispatch_rows<QT, kKindE4m3, D, true>(a, dtype, rows, sms, st);
}

int dispatch_dense(const DenseArgs &a, int d, int dtype, int kind, int rows, int sms, cudaStream_t st) {
  if (dtype == SOLATTN_BF16)
    return d == 128 ? dispatch_kind<__nv_bfloat16, 128>(a, dtype, kind, rows, sms, st) : dispatch_kind<__nv_bfloat16, 64>(a, dtype, kind, rows, sms, st);
  return d == 128 ? dispatch_kind<__half, 128>(a, dtype, kind, rows, sms, st) : dispatch_kind<__half, 64>(a, dtype, kind, rows, sms, st);
}

void set_workspace(DenseArgs *a, void *workspace, int d) {
  const DenseWs wl = dense_ws(d);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  a->status = reinterpret_cast<int *>(ws + 4);
  a->desc = reinterpret_cast<int4 *>(ws + wl.desc);
  a->part_ml = reinterpret_cast<float *>(ws + wl.ml);
  a->part_o = reinterpret_cast<float *>(ws + wl.o);
  a->timeout_ns = kTimeoutNs + kTimeoutUnitNs * static_cast<unsigned long long>(a->Lmax / kUnitKeys);
  a->scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(d));
}

int check_cross(int B, int H, int Hkv, int Nq, int Nk, int d) {
  if (B < 1 || Nq < 0 || Nk < 0 || !heads_ok(H, Hkv)) return SOLATTN_EINVAL;
  if (d != 64 && d != 128) return SOLATTN_EUNSUPPORTED;
  // row and key indices are 32-bit
  if (static_cast<long long>(Nq) * (H / Hkv) > (1ll << 30) || Nk > (1 << 30) || static_cast<long long>(B) * H > (1ll << 30))
    return SOLATTN_EUNSUPPORTED;
  return SOLATTN_OK;
}

int check_paged(int B, int H, int Hkv, int total, int d) {
  if (B < 1 || total < 0 || !heads_ok(H, Hkv)) return SOLATTN_EINVAL;
  if (d != 64 && d != 128) return SOLATTN_EUNSUPPORTED;
  if (static_cast<long long>(total) * (H / Hkv) > (1ll << 30) || static_cast<long long>(B) * H > (1ll << 30))
    return SOLATTN_EUNSUPPORTED;
  return SOLATTN_OK;
}

template <class QT, int KIND, int D>
bool launch_cache(const CacheArgs &a, bool write, int blocks, cudaStream_t st) {
  return write ? launch(cache_kernel<QT, KIND, D, true>, blocks, kCacheThreads, st, false, a)
               : launch(cache_kernel<QT, KIND, D, false>, blocks, kCacheThreads, st, false, a);
}
template <class QT, int D>
bool dispatch_cache(const CacheArgs &a, int kind, bool write, int blocks, cudaStream_t st) {
  if (kind == SOLATTN_CACHE_16) return launch_cache<QT, kKind16, D>(a, write, blocks, st);
  if (kind == SOLATTN_CACHE_INT8) return launch_cache<QT, kKindInt8, D>(a, write, blocks, st);
  return launch_cache<QT, kKindE4m3, D>(a, write, blocks, st);
}

int cache_impl(const solattn_cache *cache, const solattn_view *nk, const solattn_view *nv, const solattn_seqs *s,
               int dtype, void *status, void *stream, bool write) {
  const int rc = check_cache(cache);
  if (rc != SOLATTN_OK) return rc;
  const int rs = check_seqs(s, cache->page);
  if (rs != SOLATTN_OK) return rs;
  if (dtype != SOLATTN_BF16 && dtype != SOLATTN_FP16) return SOLATTN_EINVAL;
  if (static_cast<long long>(s->total) * cache->Hkv > (1ll << 30)) return SOLATTN_EUNSUPPORTED;
  if (!status || !aligned(status, kAlign)) return SOLATTN_EWORKSPACE;
  if (s->total == 0) return SOLATTN_OK;
  if (!view_ok(nk, 2, !write, 1, cache->Hkv, s->total) || !view_ok(nv, 2, !write, 1, cache->Hkv, s->total)) return SOLATTN_EINVAL;
  DeviceInfo di;
  const int rd = check_device({cache->k.ptr, cache->v.ptr, cache->k_scale, cache->v_scale, nk->ptr, nv->ptr, s->table, s->cu,
                               s->len, status}, &di);
  if (rd != SOLATTN_OK) return rd;
  CacheArgs a{};
  a.k = cache->k.ptr, a.v = cache->v.ptr, a.k_scale = cache->k_scale, a.v_scale = cache->v_scale;
  a.k_row = cache->k.stride_n, a.k_head = cache->k.stride_h, a.k_seq = cache->k.stride_b;
  a.v_row = cache->v.stride_n, a.v_head = cache->v.stride_h, a.v_seq = cache->v.stride_b;
  a.new_k = nk->ptr, a.new_v = nv->ptr;
  a.nk_tok = nk->stride_n, a.nk_head = nk->stride_h, a.nv_tok = nv->stride_n, a.nv_head = nv->stride_h;
  a.table = s->table, a.cu = s->cu, a.len = s->len;
  a.width = s->width, a.page = cache->page, a.page_shift = page_shift(cache->page), a.num_pages = cache->num_pages;
  a.B = s->B, a.Hkv = cache->Hkv, a.total = s->total, a.Lmax = s->width * cache->page;
  a.status = reinterpret_cast<int *>(static_cast<uint8_t *>(status) + 4);
  // Tokens of a block: the power of two that leaves two blocks per SM, at most its rows at a time (1560 tokens of
  // 12 heads written and read: 14.5 us with two, 18.6 with four or one, 20.9 with eight).
  const int most = cache->d == 128 ? (write ? CacheShape<128, true>::RPB : CacheShape<128, false>::RPB)
                                   : (write ? CacheShape<64, true>::RPB : CacheShape<64, false>::RPB);
  while (2 << a.token_shift <= most && (s->total >> (a.token_shift + 1)) >= 2 * di.sms) ++a.token_shift;
  const int blocks = (s->total + (1 << a.token_shift) - 1) >> a.token_shift;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  NvtxRange r(write ? "solattn cache append" : "solattn cache read");
  bool ok;
  if (dtype == SOLATTN_BF16)
    ok = cache->d == 128 ? dispatch_cache<__nv_bfloat16, 128>(a, cache->kind, write, blocks, st)
                         : dispatch_cache<__nv_bfloat16, 64>(a, cache->kind, write, blocks, st);
  else
    ok = cache->d == 128 ? dispatch_cache<__half, 128>(a, cache->kind, write, blocks, st)
                         : dispatch_cache<__half, 64>(a, cache->kind, write, blocks, st);
  return ok ? SOLATTN_OK : SOLATTN_ECUDA;
}

}  // namespace

extern "C" {

size_t solattn_cross_workspace_size(int B, int H, int Hkv, int Nq, int Nk, int d) {
  return check_cross(B, H, Hkv, Nq, Nk, d) == SOLATTN_OK ? dense_ws(d).total : 0;
}

size_t solattn_paged_workspace_size(int B, int H, int Hkv, int total, int d) {
  return check_paged(B, H, Hkv, total, d) == SOLATTN_OK ? dense_ws(d).total : 0;
}

int solattn_cross(const solattn_view *q, const solattn_view *k, const solattn_view *v, const solattn_view *out,
                  const int32_t *key_len, int B, int H, int Hkv, int Nq, int Nk, int d, int dtype, void *workspace,
                  size_t ws_bytes, void *stream) {
  if (!q || !k || !v || !out) return SOLATTN_EINVAL;
  const int rc = check_cross(B, H, Hkv, Nq, Nk, d);
  if (rc != SOLATTN_OK) return rc;
  if (dtype != SOLATTN_BF16 && dtype != SOLATTN_FP16) return SOLATTN_EINVAL;
  if (key_len && !aligned(key_len, 4)) return SOLATTN_EINVAL;
  if (Nq > 0 && (!view_ok(q, 2, false, B, H, Nq) || !view_ok(out, 2, true, B, H, Nq))) return SOLATTN_EINVAL;
  if (Nk > 0 && (!view_ok(k, 2, false, B, Hkv, Nk) || !view_ok(v, 2, false, B, Hkv, Nk))) return SOLATTN_EINVAL;
  if (!workspace || !aligned(workspace, kAlign) || ws_bytes < dense_ws(d).total) return SOLATTN_EWORKSPACE;
  if (Nq == 0) return SOLATTN_OK;
  DeviceInfo di;
  const int rd = check_device({q->ptr, k->ptr, v->ptr, out->ptr, key_len, workspace}, &di);
  if (rd != SOLATTN_OK) return rd;
  DenseArgs a{};
  a.q = q->ptr, a.q_tok = q->stride_n, a.q_head = q->stride_h, a.q_batch = q->stride_b;
  a.out = out->ptr, a.o_tok = out->stride_n, a.o_head = out->stride_h, a.o_batch = out->stride_b;
  a.k = k->ptr, a.k_row = k->stride_n, a.k_head = k->stride_h, a.k_seq = k->stride_b;
  a.v = v->ptr, a.v_row = v->stride_n, a.v_head = v->stride_h, a.v_seq = v->stride_b;
  a.len = key_len;
  a.B = B, a.Hkv = Hkv, a.G = H / Hkv, a.n = Nq, a.total = Nq, a.Lmax = Nk;
  set_workspace(&a, workspace, d);
  NvtxRange r("solattn cross attention");
  const long long rows = static_cast<long long>(Nq) * a.G;
  return dispatch_dense(a, d, dtype, SOLATTN_CACHE_16, static_cast<int>(rows), di.sms < kMaxSms ? di.sms : kMaxSms,
                        static_cast<cudaStream_t>(stream));
}

int solattn_paged_forward(const solattn_view *q, const solattn_view *out, const solattn_cache *cache,
                          const solattn_seqs *seqs, int H, int max_new, int causal, int dtype, void *workspace,
                          size_t ws_bytes, void *stream) {
  if (!q || !out) return SOLATTN_EINVAL;
  const int rc = check_cache(cache);
  if (rc != SOLATTN_OK) return rc;
  const int rs = check_seqs(seqs, cache->page);
  if (rs != SOLATTN_OK) return rs;
  const int rp = check_paged(seqs->B, H, cache->Hkv, seqs->total, cache->d);
  if (rp != SOLATTN_OK) return rp;
  if (dtype != SOLATTN_BF16 && dtype != SOLATTN_FP16) return SOLATTN_EINVAL;
  if (max_new < 0 || (causal != 0 && causal != 1)) return SOLATTN_EINVAL;
  const int d = cache->d;
  if (!workspace || !aligned(workspace, kAlign) || ws_bytes < dense_ws(d).total) return SOLATTN_EWORKSPACE;
  if (seqs->total == 0) return SOLATTN_OK;
  if (!view_ok(q, 2, false, 1, H, seqs->total) || !view_ok(out, 2, true, 1, H, seqs->total)) return SOLATTN_EINVAL;
  DeviceInfo di;
  const int rd = check_device({q->ptr, out->ptr, cache->k.ptr, cache->v.ptr, cache->k_scale, cache->v_scale, seqs->table,
                               seqs->cu, seqs->len, workspace}, &di);
  if (rd != SOLATTN_OK) return rd;
  DenseArgs a{};
  a.q = q->ptr, a.q_tok = q->stride_n, a.q_head = q->stride_h;
  a.out = out->ptr, a.o_tok = out->stride_n, a.o_head = out->stride_h;
  a.k = cache->k.ptr, a.k_row = cache->k.stride_n, a.k_head = cache->k.stride_h, a.k_seq = cache->k.stride_b;
  a.v = cache->v.ptr, a.v_row = cache->v.stride_n, a.v_head = cache->v.stride_h, a.v_seq = cache->v.stride_b;
  a.k_scale = cache->k_scale, a.v_scale = cache->v_scale;
  a.table = seqs->table, a.width = seqs->width, a.page = cache->page, a.page_shift = page_shift(cache->page);
  a.num_pages = cache->num_pages;
  a.cu = seqs->cu, a.len = seqs->len;
  a.B = seqs->B, a.Hkv = cache->Hkv, a.G = H / cache->Hkv, a.n = 0, a.total = seqs->total;
  a.Lmax = seqs->width * cache->page, a.causal = causal;
  set_workspace(&a, workspace, d);
  NvtxRange r("solattn paged attention");
  const int n = max_new < seqs->total ? max_new : seqs->total;
  return dispatch_dense(a, d, dtype, cache->kind, n * a.G, di.sms < kMaxSms ? di.sms : kMaxSms, static_cast<cudaStream_t>(stream));
}

int solattn_cache_append(const solattn_cache *cache, const solattn_view *new_k, const solattn_view *new_v,
                         const solattn_seqs *seqs, int dtype, void *status, void *stream) {
  return cache_impl(cache, new_k, new_v, seqs, dtype, status, stream, true);
}

int solattn_cache_read(const solattn_cache *cache, const solattn_seqs *seqs, const solattn_view *k_out,
                       const solattn_view *v_out, int dtype, void *status, void *stream) {
  return cache_impl(cache, k_out, v_out, seqs, dtype, status, stream, false);
}

}  // extern "C"
