// C-ABI entry points of the paged key/value cache: host-side argument checks,
// workspace and kernel choice. Every check runs before anything is enqueued.
#include <cmath>

#include "paged.cuh"

namespace gdn {
namespace {

bool aligned(const void* p, uintptr_t to) {
  return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0;
}

// Places (less new tokens and a window, too) and tensor-map extents stay in 32
// bits, strides in the 40 bits of a tensor map.
constexpr long long kMaxPlaces = 1ll << 30;
constexpr long long kMaxStride = 1ll << 38;

bool stride_ok(int64_t s) { return s >= 0 && s % 8 == 0 && s < kMaxStride; }

// Whether rows of `wa` elements `sa` apart from a on and rows of `wb` elements
// `sb` apart from b on share memory (both 16-bit, `rows` of each; yes, too, where
// their strides differ and only their ends lie apart).
bool rows_overlap(const void* a, int64_t sa, int64_t wa, const void* b,
                  int64_t sb, int64_t wb, long long rows) {
  const auto x = static_cast<long long>(reinterpret_cast<uintptr_t>(a) / 2);
  const auto y = static_cast<long long>(reinterpret_cast<uintptr_t>(b) / 2);
  if (x + (rows - 1) * sa + wa <= y || y + (rows - 1) * sb + wb <= x) return false;
  if (sa != sb) return true;
  const long long off = ((y - x) % sa + sa) % sa;
  return off < wa || off + wb > sa;
}

int check_cache(const gdn_paged_cache_t* c, int B) {
  // (arrays of no sequences have no address)
  if (!c || !c->k || !c->v || (B > 0 && (!c->page_table || !c->kv_lens)))
    return GDN_ERR_INVALID_ARG;
  if (c->num_pages <= 0 || c->max_pages <= 0 || c->heads <= 0 ||
      c->table_stride < c->max_pages)
    return GDN_ERR_INVALID_ARG;
  if (c->dtype != GDN_DTYPE_BF16 && c->dtype != GDN_DTYPE_F16)
    return GDN_ERR_UNSUPPORTED;
  if (c->d != 64 && c->d != 128) return GDN_ERR_UNSUPPORTED;
  const int ps = c->page_size;
  if (ps < 16 || ps > 256 || (ps & (ps - 1))) return GDN_ERR_UNSUPPORTED;
  if ((long long)c->max_pages * ps > kMaxPlaces) return GDN_ERR_UNSUPPORTED;
  const int64_t strides[] = {c->k_page, c->k_head, c->k_token,
                             c->v_page, c->v_head, c->v_token};
  for (int64_t s : strides)
    if (!stride_ok(s)) return GDN_ERR_INVALID_ARG;
  // neighbours along an axis may not overlap
  if (c->k_token < c->d || c->v_token < c->d ||
      (c->heads > 1 && (c->k_head < c->d || c->v_head < c->d)) ||
      (c->num_pages > 1 && (c->k_page < c->d || c->v_page < c->d)))
    return GDN_ERR_INVALID_ARG;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->page_table, 4) ||
      !aligned(c->kv_lens, 4))
    return GDN_ERR_MISALIGNED;
  return GDN_OK;
}

int check_batch(const int32_t* cu, int B, int T, int Hq, int hkv) {
  if (B < 0 || T < 0 || Hq <= 0 || (cu && B == 0)) return GDN_ERR_INVALID_ARG;
  if (cu && !aligned(cu, 4)) return GDN_ERR_MISALIGNED;
  const long long tokens = cu ? (long long)T : (long long)B * T;
  if (tokens > kMaxPlaces || tokens * Hq >= (1ll << 40) ||
      (long long)B * hkv >= (1ll << 31) || tokens + B >= (1ll << 31))
    return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

PagedView view(const gdn_paged_cache_t* c) {
  PagedView v{};
  v.k = c->k; v.v = c->v;
  v.k_page = c->k_page; v.k_head = c->k_head; v.k_token = c->k_token;
  v.v_page = c->v_page; v.v_head = c->v_head; v.v_token = c->v_token;
  v.table = c->page_table; v.table_stride = c->table_stride;
  v.kv_lens = c->kv_lens;
  v.num_pages = c->num_pages; v.max_pages = c->max_pages; v.hkv = c->heads;
  while ((1 << v.page_shift) < c->page_size) ++v.page_shift;
  return v;
}

}  // namespace
}  // namespace gdn

extern "C" int gdn_paged_append(
    const void* q, int64_t q_stride, const void* k, int64_t k_stride,
    const void* v, int64_t v_stride, void* q_out, int64_t q_out_stride,
    const float* rope, int rope_rows, int rot, const int32_t* positions,
    int axes, const int32_t* sections, int interleaved,
    const gdn_paged_cache_t* cache, const int32_t* cu_seqlens, int B, int T,
    int Hq, gdn_stream_t stream) {
  using namespace gdn;
  int rc = check_cache(cache, B);
  if (rc != GDN_OK) return rc;
  rc = check_batch(cu_seqlens, B, T, q ? Hq : 1, cache->heads);
  if (rc != GDN_OK) return rc;
  if (rot < 0 || rot > cache->d || axes < 1 || axes > 4)
    return GDN_ERR_INVALID_ARG;
  if (rot % 16) return GDN_ERR_UNSUPPORTED;
  if (rot > 0 && (!rope || rope_rows <= 0)) return GDN_ERR_INVALID_ARG;
  if (rot == 0 && positions) return GDN_ERR_INVALID_ARG;
  PagedAppendParams p{};
  if (axes > 1) {
    if (!positions || !sections) return GDN_ERR_INVALID_ARG;
    long long end = 0;
    for (int a = 0; a < 4; ++a) {
      if (a < axes) {
        if (sections[a] < 0 || sections[a] > rot) return GDN_ERR_INVALID_ARG;
        end += sections[a];
      }
      p.section_end[a] = (int)end;
    }
    if (end != rot / 2) return GDN_ERR_INVALID_ARG;
  }
  const long long tokens = cu_seqlens ? (long long)T : (long long)B * T;
  if (tokens == 0) return GDN_OK;
  if (!k || !v || (q && !q_out)) return GDN_ERR_INVALID_ARG;
  const int64_t strides[] = {k_stride, v_stride};
  for (int64_t s : strides)
    if (!stride_ok(s) || s < (int64_t)cache->heads * cache->d)
      return GDN_ERR_INVALID_ARG;
  if (q && (!stride_ok(q_stride) || !stride_ok(q_out_stride) ||
            q_stride < (int64_t)Hq * cache->d ||
            q_out_stride < (int64_t)Hq * cache->d))
    return GDN_ERR_INVALID_ARG;
  const void* ptrs[] = {q, k, v, q_out, rope};
  for (const void* x : ptrs)
    if (x && !aligned(x, 16)) return GDN_ERR_MISALIGNED;
  if (positions && !aligned(positions, 4)) return GDN_ERR_MISALIGNED;
  // in place only row for row
  const int64_t wq = (int64_t)Hq * cache->d, wkv = (int64_t)cache->heads * cache->d;
  if (q && ((!(q == q_out && q_stride == q_out_stride) &&
             rows_overlap(q, q_stride, wq, q_out, q_out_stride, wq, tokens)) ||
            rows_overlap(k, k_stride, wkv, q_out, q_out_stride, wq, tokens) ||
            rows_overlap(v, v_stride, wkv, q_out, q_out_stride, wq, tokens)))
    return GDN_ERR_INVALID_ARG;
  if ((rc = device_status_ptr(&p.status)) != GDN_OK) return rc;
  p.c = view(cache);
  p.q = q; p.k = k; p.v = v; p.q_out = q_out;
  p.q_row = q_stride; p.k_row = k_stride; p.v_row = v_stride;
  p.q_out_row = q_out_stride;
  p.rope = rope; p.positions = positions;
  p.rope_rows = rope_rows; p.rot = rot; p.axes = axes;
  p.interleaved = interleaved ? 1 : 0;
  p.cu = cu_seqlens; p.tokens = tokens; p.N = B; p.T = T; p.hq = Hq;
  const cudaError_t e =
      launch_paged_append(p, cache->d, cache->dtype == GDN_DTYPE_BF16, stream);
  return count_launches(e, 1) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

extern "C" int gdn_paged_attn(const void* q, int64_t q_stride,
                              const gdn_paged_cache_t* cache,
                              const int32_t* cu_seqlens, int B, int T, int Hq,
                              float scale, int causal, int window, void* out,
                              float* lse, int path, gdn_stream_t stream) {
  using namespace gdn;
  int rc = check_cache(cache, B);
  if (rc != GDN_OK) return rc;
  rc = check_batch(cu_seqlens, B, T, Hq, cache->heads);
  if (rc != GDN_OK) return rc;
  if (!(scale > 0.f) || !std::isfinite(scale) || window < 0 ||
      path < GDN_PAGED_AUTO || path > GDN_PAGED_TILES)
    return GDN_ERR_INVALID_ARG;
  if (Hq % cache->heads) return GDN_ERR_INVALID_ARG;
  if (Hq / cache->heads > 128) return GDN_ERR_UNSUPPORTED;
  const long long tokens = cu_seqlens ? (long long)T : (long long)B * T;
  if (tokens == 0) return GDN_OK;
  if (!q || !out) return GDN_ERR_INVALID_ARG;
  if (!stride_ok(q_stride) || q_stride < (int64_t)Hq * cache->d)
    return GDN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4))
    return GDN_ERR_MISALIGNED;
  const int64_t wq = (int64_t)Hq * cache->d;
  if (rows_overlap(q, q_stride, wq, out, wq, wq, tokens))
    return GDN_ERR_INVALID_ARG;
  PagedAttnParams p{};
  if ((rc = device_status_ptr(&p.status)) != GDN_OK) return rc;
  p.c = view(cache);
  p.q = q; p.q_row = q_stride; p.out = out; p.lse = lse; p.cu = cu_seqlens;
  p.N = B; p.T = T; p.hq = Hq; p.group = Hq / cache->heads;
  p.causal = causal ? 1 : 0;
  p.window = window < kMaxPlaces ? window : (int)kMaxPlaces;
  p.scale_log2 = scale * 1.4426950408889634f;

  // Up to 16 rows per key head stream the cache through the small products of
  // paged_rows.cu, more go to the tensor-core tiles (32 sequences of 4096
  // keys, 4 key heads: 16 rows 58.6 us against 64.5 us, 24 rows, a second
  // block of them, 80 us against 65 us; 64-wide heads 37 against 53 and 56
  // against 54; sequences alike). A packed batch of few rows on the average may
  // hold longer sequences all the same: each kernel takes its own (127 single
  // tokens after 500 to 2000 keys and a prompt of 300, 32 heads, 8 key heads:
  // 142 us, 175 on the tiles, 139 in two calls). One of many rows on the average
  // takes the tiles for its single tokens, too (63 after 500 to 4000 keys and a
  // chunk of 2048: 179 us, 170 in two calls; 31 after 200 to 1000 and 1024: 56
  // us, 63 in two calls). A call that the few-row kernel splits (a short cache)
  // goes there with any number of rows: one launch and no tensor-core tiles to
  // fill (one user, 5 tokens of 32 heads, 4 key heads, 1024 keys 10 us against
  // 15, 32 tokens 13 against 19; 128 tokens, 512 keys 14 against 19).
  const int split = path == GDN_PAGED_TILES ? 0 : paged_rows_split(p);
  const long long mean = (long long)T * p.group;  // rows (packed: times B)
  const bool few = mean <= 16ll * (cu_seqlens ? B : 1);
  const bool rows =
      path == GDN_PAGED_ROWS || (path == GDN_PAGED_AUTO && (few || split));
  const bool tiles =
      path == GDN_PAGED_TILES ||
      (path == GDN_PAGED_AUTO && !split && (!few || (cu_seqlens && T > 1)));
  p.rows_min = rows && tiles ? 16 : 0;
  p.rows_max = rows && tiles ? 16 : (1ll << 40);
  const bool bf16 = cache->dtype == GDN_DTYPE_BF16;
  const int d = cache->d, ps = cache->page_size;
  auto cache_map = [&](CUtensorMap* m, bool v, int box) {
    return v ? make_paged_map(m, cache->v, bf16, d, ps, cache->heads,
                              cache->num_pages, cache->v_token, cache->v_head,
                              cache->v_page, box, 1)
             : make_paged_map(m, cache->k, bf16, d, ps, cache->heads,
                              cache->num_pages, cache->k_token, cache->k_head,
                              cache->k_page, box, 1);
  };
  int launches = 0;
  auto run = [&](bool use_tiles) {
    const int box = use_tiles ? paged_tiles_box(ps) : paged_rows_box(ps);
    CUtensorMap tq, tk, tv;
    if (!cache_map(&tk, false, box) || !cache_map(&tv, true, box) ||
        (use_tiles && !make_paged_map(&tq, q, bf16, d, Hq, tokens, 1, d,
                                      q_stride, d, p.group, 128 / p.group)))
      return cudaErrorUnknown;
    p.split = use_tiles ? 0 : split;
    if (p.split)
      return launch_paged_rows(p, d, bf16, tk, tv, stream, &launches);
    void* ws = nullptr;
    cudaError_t e =
        paged_workspace(&ws, use_tiles ? paged_tiles_workspace_bytes(p, d)
                                       : paged_rows_workspace_bytes(d),
                        stream);
    if (e != cudaSuccess) return e;
    if (use_tiles) {
      paged_tiles_bind_workspace(p, ws, d);
      e = launch_paged_tiles(p, d, bf16, tq, tk, tv, stream, &launches);
    } else {
      paged_rows_bind_workspace(p, ws, d);
      e = launch_paged_rows(p, d, bf16, tk, tv, stream, &launches);
    }
    const cudaError_t f = cudaFreeAsync(ws, stream);
    return e == cudaSuccess ? f : e;
  };
  cudaError_t e = cudaSuccess;
  if (rows) e = run(false);
  if (tiles && e == cudaSuccess) e = run(true);
  count_launches(cudaSuccess, launches);
  return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
