// Attention of few query rows over a paged cache (one decode token, a few
// drafted ones; any number over a short cache): softmax(scale q K^T + mask) V,
// one pass over the keys with a running reference maximum and sum per row.
//
// Rows. The query heads of a key head share its keys, so the query tokens x
// group heads of one (sequence, key head) are the rows of one problem: row r
// is token r / group, head r % group of the group. Blocks of 16 rows.
//
// Bound: HBM. Every key and value is read once, 4 D bytes a key and head,
// for 4 D flops a row: far below the tensor cores' rate at 16 rows, so
// legacy m16n8k16 products (16 rows are their row tile; tcgen05's smallest is
// 64) are enough and the whole design is about keeping copies in flight.
//
// Split. The tiles of 64 keys of all (sequence, row block, key head) items
// form one list that is cut into equal runs, one per resident CTA, so a batch
// of ragged lengths and a single long sequence both fill the machine and the
// host needs to know no length. A run that holds a whole item writes its
// output; the pieces of a cut item (row maxima, sums and unnormalised
// outputs in fp32) go to the workspace and paged_merge.cu joins them in
// the order of the runs, so results do not depend on timing.
//
// Short caches. Where the page table cannot hold many keys and the items leave
// CTAs over, an item gets a cluster of 1 to 8 CTAs instead, a fixed share of its
// tiles each, which join their pieces in shared memory: one launch, no
// workspace. (An instance of its own: with the join in it the other one takes
// 2 us longer, 185 us against 182 for 64 sequences of up to 8192 keys.)
//
// A CTA: a producer warp that looks pages up and issues TMA copies (64
// columns by up to 64 tokens a box, 128-byte swizzle) into a ring of key and
// value tiles, and four consumer warps that each take 16 keys of every tile
// with their own maxima, sums and accumulators, joined in shared memory once
// per item. Values of keys outside the sequence are zeroed in shared memory
// before they are multiplied: the tail of a page may hold anything.
#include <type_traits>

#include "paged.cuh"
#include "tc_ptx.cuh"

namespace gdn {

using namespace tc;

namespace {

constexpr int TK = 64;       // keys per tile
constexpr int kConsumers = 4;
constexpr int kThreads = (kConsumers + 1) * 32;

constexpr int ROWS = 16;     // rows per block
constexpr int kCtasPerSm = 2;
// Split calls: up to 8 CTAs an item, where the table holds up to 512 keys for
// each of them; 320 where single tokens leave a quarter of the CTAs idle, which
// the even cut would use. (More rows than one block go to the tiles otherwise:
// 40 rows, 4 key heads, 4096 keys 14.5 us against 23.8.) Single tokens, 8 key
// heads, D = 128, us in a graph and (one call after the other, where the cut's
// second launch and workspace show on the host) split against cut:
//   one user     64 keys 5.8 (10.1) against 7.1 (13.4), 2048 11.2 (11.3) against
//                10.2 (14.0), 3072 12.5 (12.7) against 10.7 (14.6), 4096 14.0
//                (14.2) against 11.0 (14.6)
//   two users    2048 keys 12.3 (12.5) against 10.4 (15.3), 3072 13.8 (13.9)
//                against 11.2 (13.6)
//   four users   (256 of 304 CTAs) 4096 keys 16.1 (16.3) against 16.7 (16.8)
//   32 users     (one CTA an item) 512 keys 12.4 (12.7) against 16.8 (17.1)
constexpr int kMaxSplit = 8;
constexpr int kSplitKeys = 512;
constexpr int kSplitKeysIdle = 320;

template <int D>
struct Shape {
  static constexpr int kTile = TK * D * 2;  // bytes of a key (or value) tile
  // 96 KB in flight per CTA, two CTAs per SM
  static constexpr int kStages = 96 * 1024 / (2 * kTile);
  static constexpr int kRed = ROWS * D * 4;
  static constexpr int kMisc = 4 * kStages * 8;  // barriers, for two passes
  static constexpr int kSmem = 1024 + kStages * 2 * kTile + kRed + kMisc;
  // [kStages] full, [kStages] empty; the same for a second pass
  static __device__ __forceinline__ uint64_t* barriers(char* sm) {
    return reinterpret_cast<uint64_t*>(sm + kStages * 2 * kTile + kRed);
  }
  static __device__ __forceinline__ void init(uint64_t* bars) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars[s], 1);
      mbar_init(&bars[kStages + s], kConsumers);
    }
  }
};

// ---- the work list -------------------------------------------------------------
struct Seq {
  int q0, len, kv;
  int tile0, tiles;  // key tiles [tile0, tile0 + tiles)
  int blocks;        // row blocks
  bool ordered;      // its offsets in a packed batch are
};

__device__ __forceinline__ Seq seq_work(const PagedAttnParams& p, int n) {
  const PagedSeq s = paged_seq(p.c, p.cu, p.T, n, p.status);
  Seq w;
  w.q0 = s.q0;
  w.len = s.len;
  w.kv = s.kv;
  w.ordered = s.ordered;
  const long long n_rows = (long long)s.len * p.group;
  w.blocks = n_rows <= p.rows_max ? (int)((n_rows + ROWS - 1) / ROWS) : 0;
  int lo = 0;
  if (p.window > 0) lo = max(0, s.kv - s.len - p.window + 1);
  w.tile0 = min(lo, max(s.kv - 1, 0)) / TK;
  // an item without a single key still has its rows to write
  w.tiles = max(1, (s.kv + TK - 1) / TK - w.tile0);
  return w;
}

template <bool SPLIT>
__device__ __forceinline__ long long seq_units(const PagedAttnParams& p,
                                               const Seq& s) {
  return (long long)s.blocks * (SPLIT ? p.split : s.tiles) * p.c.hkv;
}

// One run [w, w_end) of the list, walked item by item.
struct Walk {
  long long w, w_end;
  long long base;  // first unit of sequence n
  int n;
  Seq s;
};

struct Segment {
  int n, head, block;
  int t0, t1;            // tiles of the item in this run
  bool starts, ends;     // holds the item's first / last tile
  long long item_end;    // unit past the item's last
};

template <bool SPLIT>
__device__ __forceinline__ bool next_segment(const PagedAttnParams& p, Walk& k,
                                             Segment& g) {
  if (k.w >= k.w_end) return false;
  long long units = seq_units<SPLIT>(p, k.s);
  while (k.w >= k.base + units) {  // (sequences without rows have no units)
    k.base += units;
    if (++k.n >= p.N) return false;
    k.s = seq_work(p, k.n);
    units = seq_units<SPLIT>(p, k.s);
  }
  const long long off = k.w - k.base;
  const int tiles = SPLIT ? p.split : k.s.tiles;  // units of an item
  const long long item = off / tiles;
  g.n = k.n;
  g.head = (int)(item % p.c.hkv);
  g.block = (int)(item / p.c.hkv);
  g.t0 = (int)(off - item * tiles);
  g.item_end = k.base + (item + 1) * tiles;
  const long long end = g.item_end < k.w_end ? g.item_end : k.w_end;
  g.t1 = g.t0 + (int)(end - k.w);
  if (SPLIT) {  // part t0 of an item
    g.t1 = (int)((long long)k.s.tiles * (g.t0 + 1) / p.split);
    g.t0 = (int)((long long)k.s.tiles * g.t0 / p.split);
  }
  g.starts = g.t0 == 0;
  g.ends = g.t1 == k.s.tiles;
  k.w = end;
  return true;
}

// ---- warp-level products ---------------------------------------------------------
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile(
      "ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile(
      "ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4],
                                         uint32_t b0, uint32_t b1,
                                         __nv_bfloat16) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4],
                                         uint32_t b0, uint32_t b1, __half) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte offset of 16-byte chunk c (0 .. D/8 - 1) of token row r in a tile:
// blocks of 64 columns, each TK rows of 128 swizzled bytes.
__device__ __forceinline__ uint32_t tile_off(int r, int c) {
  return (uint32_t)((c >> 3) * (TK * 128)) + sw128(r, c & 7);
}

__device__ __forceinline__ float4 ld_cluster(uint32_t addr) {
  float4 x;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
               : "r"(addr)
               : "memory");
  return x;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float x;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(addr) : "memory");
  return x;
}

// The parts of an item (unnormalised outputs `red` as fragments of the
// products, maxima M, sums L) lie in the shared memory of the cluster's CTAs.
// Each warp joins its share of the columns, in the order of the CTAs.
template <typename E, int D>
__device__ __noinline__ void join_cluster(const PagedAttnParams& p, const Seq& s,
                                          const Segment& g, float* red, float* M,
                                          float* L) {
  const int lane = threadIdx.x % 32, g8 = lane / 4, t4 = lane % 4;
  const int nrows = min(s.len * p.group - g.block * ROWS, ROWS);
  float f[2][kMaxSplit], inv[2];
  long long to[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = h * 8 + g8, row = g.block * ROWS + r, tok = row / p.group;
    float m[kMaxSplit], l[kMaxSplit], top = kNegInf, sum = 0.f;
#pragma unroll
    for (int c = 0; c < kMaxSplit; ++c) {
      m[c] = kNegInf;
      l[c] = 0.f;
      if (c < p.split) {
        m[c] = ld_cluster_f32(map_to_cta(&M[r], c));
        l[c] = ld_cluster_f32(map_to_cta(&L[r], c));
      }
    }
#pragma unroll
    for (int c = 0; c < kMaxSplit; ++c) top = fmaxf(top, m[c]);
#pragma unroll
    for (int c = 0; c < kMaxSplit; ++c) {
      f[h][c] = l[c] != 0.f ? factor(m[c], top) : 0.f;
      sum += l[c] * f[h][c];
    }
    const int x = s.kv - s.len + tok;
    const int hi = p.causal ? min(x + 1, s.kv) : s.kv;
    const int lo = p.window > 0 ? max(0, x - p.window + 1) : 0;
    inv[h] = hi <= lo ? 0.f : 1.f / sum;
    to[h] = r < nrows ? (s.q0 + (long long)tok) * p.hq + g.head * p.group +
                            row % p.group
                      : -1;
    if (p.lse && to[h] >= 0 && t4 == 0 && threadIdx.x < 32 &&
        cluster_ctarank() == 0)
      p.lse[to[h]] = row_lse(top, sum);
  }
  for (int j = cluster_ctarank() * kConsumers + threadIdx.x / 32; j < D / 8;
       j += p.split * kConsumers) {
    float4 x[kMaxSplit];
#pragma unroll
    for (int c = 0; c < kMaxSplit; ++c)
      if (c < p.split) x[c] = ld_cluster(map_to_cta(&red[(j * 32 + lane) * 4], c));
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int c = 0; c < kMaxSplit; ++c) {  // (factor 0: a part that saw nothing)
      if (c < p.split && f[0][c] != 0.f) {
        y.x += x[c].x * f[0][c];
        y.y += x[c].y * f[0][c];
      }
      if (c < p.split && f[1][c] != 0.f) {
        y.z += x[c].z * f[1][c];
        y.w += x[c].w * f[1][c];
      }
    }
    uint32_t* const out = static_cast<uint32_t*>(p.out);
    if (to[0] >= 0)
      out[to[0] * (D / 2) + j * 4 + t4] = pack2<E>(y.x * inv[0], y.y * inv[0]);
    if (to[1] >= 0)
      out[to[1] * (D / 2) + j * 4 + t4] = pack2<E>(y.z * inv[1], y.w * inv[1]);
  }
}

// What the warps of a CTA share beside the tiles.
struct Shared {
  float m[kConsumers][ROWS], l[kConsumers][ROWS];  // warps' maxima and sums
  float M[ROWS], L[ROWS];                          // the item's
  long long sum[kThreads / 32];
  long long base, total;  // first unit of sequence n, where the run begins; units
  long long per;          // units of a run
  int n, abort;
  int redo;               // a result may hold what its row does not see
};

// A CTA's run. CAREFUL: with a look through the values of tiles that some row
// sees in part. Leaves the last segment in g and its sequence in walk.
template <typename E, int D, bool SPLIT, bool CAREFUL>
__device__ __forceinline__ void serve(const PagedAttnParams& p,
                                      const CUtensorMap& tk,
                                      const CUtensorMap& tv, int box,
                                      char* sm, Shared& c, Walk& walk,
                                      Segment& g) {
  using S = Shape<D>;
  constexpr int KS = D / 16;
  float* const red = reinterpret_cast<float*>(sm + S::kStages * 2 * S::kTile);
  uint64_t* const full = S::barriers(sm) + (CAREFUL ? 2 * S::kStages : 0);
  uint64_t* const empty = full + S::kStages;
  volatile int* const abort_flag = &c.abort;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (warp == kConsumers) {
    // ---- producer ------------------------------------------------------------
    const int page = 1 << p.c.page_shift;
    const int boxes = TK / box;                 // boxes of rows per tile
    constexpr int HALVES = D / 64;
    const int per_tile = boxes * HALVES * 2;    // copies per tile: <= 16
    const int b = lane / (HALVES * 2), hf = (lane / 2) % HALVES, kv = lane & 1;
    int it = 0;
    bool ok = true;
    while (ok && next_segment<SPLIT>(p, walk, g)) {
      const int32_t* table = p.c.table + (long long)g.n * p.c.table_stride;
      // keys that any row may see
      int lo = 0;
      if (p.window > 0) lo = max(0, walk.s.kv - walk.s.len - p.window + 1);
      for (int t = g.t0; t < g.t1; ++t, ++it) {
        const int key = (walk.s.tile0 + t) * TK + b * box;
        const bool need = lane < per_tile && key < walk.s.kv && key + box > lo;
        int pid = 0;
        if (need) {
          pid = table[key >> p.c.page_shift];
          if (pid < 0 || pid >= p.c.num_pages) {
            record_status(p.status, GDN_ERR_INVALID_ARG);
            pid = p.c.num_pages;  // past the pool: the copy fills zeros
          }
        }
        const int st = it % S::kStages;
        if (it >= S::kStages)
          ok = warp_wait(&empty[st], (it / S::kStages - 1) & 1, abort_flag);
        if (!ok) break;
        const int copies = __popc(__ballot_sync(0xffffffffu, need));
        if (lane == 0)
          mbar_arrive_expect_tx(&full[st], (uint32_t)copies * box * 128);
        __syncwarp();
        if (need) {
          char* dst = sm + st * 2 * S::kTile + kv * S::kTile +
                      hf * (TK * 128) + b * box * 128;
          tma_load_4d(dst, kv ? &tv : &tk, &full[st], hf * 64,
                      key & (page - 1), g.head, pid);
        }
      }
    }
  } else {
    // ---- consumers -----------------------------------------------------------
    const int g8 = lane / 4, t4 = lane % 4;
    const int mat = lane >> 3, r8 = lane & 7;
    const int kb = warp * 16;
    int it = 0;
    // (after a wait gave up the warps still walk the list, without waiting,
    // so that every named barrier finds all of them)
    bool ok = true;
    while (next_segment<SPLIT>(p, walk, g)) {
      const int rows_left = walk.s.len * p.group - g.block * ROWS;
      const int nrows = min(rows_left, ROWS);
      // queries (rows past the last are zero), row limits
      uint32_t qf[KS][4];
      int hi[2], lo[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = h * 8 + g8;
        const int row = g.block * ROWS + min(r, nrows - 1);
        const int tok = row / p.group;
        const int x = walk.s.kv - walk.s.len + tok;
        hi[h] = p.causal ? min(x + 1, walk.s.kv) : walk.s.kv;
        lo[h] = p.window > 0 ? max(0, x - p.window + 1) : 0;
        const E* q = static_cast<const E*>(p.q) +
                     (walk.s.q0 + (long long)tok) * p.q_row +
                     (long long)(g.head * p.group + row % p.group) * D;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          qf[ks][h] = qf[ks][2 + h] = 0u;
          if (r < nrows) {
            qf[ks][h] =
                *reinterpret_cast<const uint32_t*>(q + ks * 16 + 2 * t4);
            qf[ks][2 + h] =
                *reinterpret_cast<const uint32_t*>(q + ks * 16 + 8 + 2 * t4);
          }
        }
      }
      // keys [free_lo, free_hi) are seen by every row of the block; keys
      // outside [any_lo, kv) by none
      const int x0 = walk.s.kv - walk.s.len + g.block * ROWS / p.group;
      const int x1 = walk.s.kv - walk.s.len +
                     (g.block * ROWS + nrows - 1) / p.group;
      const int free_hi = p.causal ? min(x0 + 1, walk.s.kv) : walk.s.kv;
      const int free_lo = p.window > 0 ? x1 - p.window + 1 : 0;
      int any_lo = 0;
      if (p.window > 0)
        any_lo = max(0, walk.s.kv - walk.s.len - p.window + 1);

      float acc[D / 8][4];
      float mx[2], sum[2];
      mx[0] = mx[1] = kNegInf;
      sum[0] = sum[1] = 0.f;
#pragma unroll
      for (int j = 0; j < D / 8; ++j)
        acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;

      for (int t = g.t0; ok && t < g.t1; ++t, ++it) {
        const int st = it % S::kStages;
        ok = warp_wait(&full[st], (it / S::kStages) & 1, abort_flag);
        if (!ok) break;
        const int key0 = (walk.s.tile0 + t) * TK + kb;
        char* ks_ = sm + st * 2 * S::kTile;
        char* vs_ = ks_ + S::kTile;
        // a warp whose 16 keys nobody sees has nothing to do
        if (key0 < walk.s.kv && key0 + 16 > any_lo) {
          if (key0 + 16 > walk.s.kv || key0 < any_lo) {
            // zero the values of keys outside the sequence (or before every
            // row's window): their weights are 0, and 0 * NaN is NaN
            for (int i = lane; i < 16 * (D / 8); i += 32) {
              const int r = i / (D / 8), key = key0 + r;
              if (key >= walk.s.kv || key < any_lo)
                *reinterpret_cast<uint4*>(vs_ + tile_off(kb + r, i % (D / 8))) =
                    make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async();  // before the next copy into this stage
            __syncwarp();
          }
          float s[2][4];
#pragma unroll
          for (int j = 0; j < 2; ++j)
            s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
          const uint32_t ka = smem_u32(ks_), va = smem_u32(vs_);
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            uint32_t bfr[4];
            ldsm4(ka + tile_off(kb + (mat >> 1) * 8 + r8, 2 * ks + (mat & 1)),
                  bfr);
            mma16816(s[0], qf[ks], bfr[0], bfr[1], E());
            mma16816(s[1], qf[ks], bfr[2], bfr[3], E());
          }
          const bool masked = key0 < free_lo || key0 + 16 > free_hi;
          bool grow = false;
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float x = __fmul_rn(s[j][e], p.scale_log2);  // (see kFar)
              if (masked) {
                const int key = key0 + j * 8 + 2 * t4 + (e & 1);
                if (key >= hi[e >> 1] || key < lo[e >> 1]) x = kNegInf;
              }
              s[j][e] = x;
              grow = grow || !(x <= mx[e >> 1] + kSlack + kLift<E>);  // (NaN too)
            }
          if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float top = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]),
                                fmaxf(s[1][2 * h], s[1][2 * h + 1]));
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
              const float now = fmaxf(mx[h], top - kLift<E>);
              const float f = factor(mx[h], now);
              mx[h] = now;
              sum[h] *= f;
#pragma unroll
              for (int j = 0; j < D / 8; ++j) {
                acc[j][2 * h] *= f;
                acc[j][2 * h + 1] *= f;
              }
            }
          }
          uint32_t pf[4];
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float ref = mx[h] == kNegInf ? 0.f : mx[h];
              const float a = ex2(s[j][2 * h] - ref);
              const float b = ex2(s[j][2 * h + 1] - ref);
              sum[h] += a + b;
              pf[2 * j + h] = pack2<E>(a, b);
            }
          bool by_key = false;
          if (CAREFUL && masked) {
            // look through the values of the warp's keys
            uint32_t z = 0;
            for (int i = lane; i < 16 * (D / 8); i += 32)
              z = probe8<E>(*reinterpret_cast<const uint4*>(
                                vs_ + tile_off(kb + i / (D / 8), i % (D / 8))),
                            z);
            by_key = __any_sync(0xffffffffu, probe_hit(z));
          }
          if (by_key) {
#pragma unroll 1
            for (int key = 0; key < 16; ++key) {
              const int from = (lane & ~3) | (key >> 1 & 3);
              float w[2];
              bool sees[2];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float2 x = unpack2(
                    __shfl_sync(0xffffffffu, key < 8 ? pf[h] : pf[2 + h], from),
                    E());
                w[h] = key & 1 ? x.y : x.x;
                sees[h] = key0 + key < hi[h] && key0 + key >= lo[h];
              }
#pragma unroll
              for (int j = 0; j < D / 8; ++j) {
                const float2 x = unpack2(
                    *reinterpret_cast<const uint32_t*>(
                        vs_ + tile_off(kb + key, j) + t4 * 4),
                    E());
#pragma unroll
                for (int h = 0; h < 2; ++h)
                  if (sees[h]) {
                    acc[j][2 * h] = fmaf(w[h], x.x, acc[j][2 * h]);
                    acc[j][2 * h + 1] = fmaf(w[h], x.y, acc[j][2 * h + 1]);
                  }
              }
              __syncwarp();
            }
          } else {
#pragma unroll
            for (int j = 0; j < D / 16; ++j) {
              uint32_t bfr[4];
              ldsm4_t(va + tile_off(kb + (mat & 1) * 8 + r8, 2 * j + (mat >> 1)),
                      bfr);
              mma16816(acc[2 * j], pf, bfr[0], bfr[1], E());
              mma16816(acc[2 * j + 1], pf, bfr[2], bfr[3], E());
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
      }

      // ---- join the four warps -------------------------------------------------
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float l = sum[h];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (t4 == 0) {
          c.m[warp][h * 8 + g8] = mx[h];
          c.l[warp][h * 8 + g8] = l;
        }
      }
      named_bar(1, kConsumers * 32);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = h * 8 + g8;
        float top = kNegInf;
#pragma unroll
        for (int w = 0; w < kConsumers; ++w)
          top = fmaxf(top, c.m[w][r]);
        float l = 0.f;
#pragma unroll
        for (int w = 0; w < kConsumers; ++w)
          l += c.l[w][r] * factor(c.m[w][r], top);
        const float f = factor(mx[h], top);
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          acc[j][2 * h] *= f;
          acc[j][2 * h + 1] *= f;
        }
        if (warp == 0 && t4 == 0) {
          c.M[r] = top;
          c.L[r] = l;
        }
      }
      // turns: 3 -> 2, 1 -> (after) 0, 2 -> 0 through one buffer, in a fixed
      // order
#pragma unroll 1
      for (int turn = 0; turn < 3; ++turn) {
        const int from = 3 - turn, to = turn == 0 ? 2 : turn == 1 ? 1 : 0;
        if (warp == from) {
#pragma unroll
          for (int j = 0; j < D / 8; ++j)
            reinterpret_cast<float4*>(red)[j * 32 + lane] =
                make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
        }
        named_bar(1, kConsumers * 32);
        if (warp == to) {
#pragma unroll
          for (int j = 0; j < D / 8; ++j) {
            const float4 x = reinterpret_cast<float4*>(red)[j * 32 + lane];
            acc[j][0] += x.x;
            acc[j][1] += x.y;
            acc[j][2] += x.z;
            acc[j][3] += x.w;
          }
        }
        named_bar(1, kConsumers * 32);
      }
      const bool whole = g.starts && g.ends;
      if (warp == 0) {
        float4* const mine = reinterpret_cast<float4*>(red);
        // rows that are not finite and do not see all that was multiplied
        if (!CAREFUL) {
          const int key0 = (walk.s.tile0 + g.t0) * TK;
          const int key1 = min((walk.s.tile0 + g.t1) * TK, walk.s.kv);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r = h * 8 + g8;
            float z = 0.f;
#pragma unroll
            for (int j = 0; j < D / 8; ++j)
              z = fmaf(acc[j][2 * h + 1], 0.f, fmaf(acc[j][2 * h], 0.f, z));
            if (r < nrows && c.L[r] != 0.f && !(z == 0.f) &&
                (hi[h] < key1 || lo[h] > max(key0, any_lo)))
              c.redo = 1;
          }
        }
        const int slot = 2 * blockIdx.x + (g.starts ? 1 : 0);
        if (SPLIT && p.split > 1) {  // joined over the cluster below
#pragma unroll
          for (int j = 0; j < D / 8; ++j)
            mine[j * 32 + lane] =
                make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = h * 8 + g8;
          if (r >= nrows || (SPLIT && p.split > 1)) continue;
          const float top = c.M[r], l = c.L[r];
          if (whole) {
            const int row = g.block * ROWS + r;
            const long long tok = walk.s.q0 + (long long)(row / p.group);
            const int head = g.head * p.group + row % p.group;
            const float inv = 1.f / l;
            E* o = static_cast<E*>(p.out) + (tok * p.hq + head) * D;
#pragma unroll
            for (int j = 0; j < D / 8; ++j)  // (a row that sees nothing: 0)
              *reinterpret_cast<uint32_t*>(o + j * 8 + 2 * t4) =
                  hi[h] <= lo[h]
                      ? 0u
                      : pack2<E>(acc[j][2 * h] * inv,
                                      acc[j][2 * h + 1] * inv);
            if (p.lse && t4 == 0) p.lse[tok * p.hq + head] = row_lse(top, l);
          } else {
            float* o = p.part_o + ((long long)slot * ROWS + r) * D;
#pragma unroll
            for (int j = 0; j < D / 8; ++j)
              *reinterpret_cast<float2*>(o + j * 8 + 2 * t4) =
                  make_float2(acc[j][2 * h], acc[j][2 * h + 1]);
            if (t4 == 0)
              *reinterpret_cast<float2*>(
                  p.part_ml + ((long long)slot * ROWS + r) * 2) =
                  make_float2(top, l);
          }
        }
        if (!SPLIT && g.starts && !g.ends && lane == 0) {
          const int last = (int)((g.item_end - 1) / c.per);
          p.meta[2 * blockIdx.x] = make_int4(g.n, g.head, g.block, last);
          p.meta[2 * blockIdx.x + 1] =
              make_int4(walk.s.q0, walk.s.len, walk.s.kv, 0);
        }
      }
      named_bar(1, kConsumers * 32);
    }
  }
}

// The run once more, with barriers as at the start.
template <typename E, int D, bool SPLIT>
__device__ __noinline__ void serve_again(const PagedAttnParams& p,
                                         const CUtensorMap& tk,
                                         const CUtensorMap& tv, int box, char* sm,
                                         Shared& c) {
  using S = Shape<D>;
  if (threadIdx.x == 0) {
    S::init(S::barriers(sm) + 2 * S::kStages);
    fence_mbar_init();
  }
  __syncthreads();
  Walk walk;
  walk.w = c.per * blockIdx.x;
  walk.w_end = min(walk.w + c.per, c.total);
  walk.n = c.n;
  walk.base = c.base;
  walk.s = seq_work(p, c.n);
  Segment g;
  serve<E, D, SPLIT, true>(p, tk, tv, box, sm, c, walk, g);
  __syncthreads();
}

template <typename E, int D, bool SPLIT>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    paged_rows_kernel(const __grid_constant__ PagedAttnParams p,
                      const __grid_constant__ CUtensorMap tk,
                      const __grid_constant__ CUtensorMap tv, int box) {
  using S = Shape<D>;
  extern __shared__ char smem_raw[];
  char* sm = reinterpret_cast<char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  __shared__ Shared c;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  if (tid == 0) {
    c.abort = c.redo = 0;
    c.n = p.N;
    S::init(S::barriers(sm));
    fence_mbar_init();
    prefetch_tmap(&tk);
    prefetch_tmap(&tv);
  }
  griddep_wait();  // nothing above touches what earlier kernels write

  // where this CTA's run lies: thread t sums the sequences [t * per, ...)
  const int per_t = (p.N + kThreads - 1) / kThreads;
  const int n_lo = min(p.N, tid * per_t), n_hi = min(p.N, n_lo + per_t);
  long long mine = 0;
  bool bad = false;
  for (int n = n_lo; n < n_hi; ++n) {
    const Seq s = seq_work(p, n);
    mine += seq_units<SPLIT>(p, s);
    bad = bad || !s.ordered;
  }
  long long scan = mine;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const long long up = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += up;
  }
  if (lane == 31) c.sum[warp] = scan;
  const bool skip = __syncthreads_or(bad);
  long long total = 0, before = scan - mine;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) before += c.sum[i];
    total += c.sum[i];
  }
  if (skip) total = 0;
  // (a split call has a block for every part)
  const long long per =
      SPLIT ? 1 : (total + gridDim.x - 1) / gridDim.x;
  Walk walk;
  walk.w = per * blockIdx.x;
  walk.w_end = walk.w + per < total ? walk.w + per : total;
  if (walk.w < walk.w_end && mine > 0 && walk.w >= before &&
      walk.w < before + mine) {
    long long base = before;
    int n = n_lo;
    for (; n < n_hi; ++n) {
      const long long u = seq_units<SPLIT>(p, seq_work(p, n));
      if (walk.w < base + u) break;
      base += u;
    }
    c.n = n;
    c.base = base;
    c.total = total;
    c.per = per;
  }
  __syncthreads();
  walk.n = c.n;
  walk.base = c.base;
  if (tid == 0 && !SPLIT) p.meta[2 * blockIdx.x] = make_int4(-1, 0, 0, 0);
  if (walk.n >= p.N) return;  // no work for this CTA
  walk.s = seq_work(p, walk.n);

  Segment g;
  serve<E, D, SPLIT, false>(p, tk, tv, box, sm, c, walk, g);
  __syncthreads();
  if (c.redo && !c.abort)
    serve_again<E, D, SPLIT>(p, tk, tv, box, sm, c);
  if (SPLIT && p.split > 1) {
    // ---- join the cluster's parts of the item ----------------------------------
    cluster_sync();
    if (warp < kConsumers)
      join_cluster<E, D>(
          p, walk.s, g,
          reinterpret_cast<float*>(sm + S::kStages * 2 * S::kTile), c.M, c.L);
    __syncwarp();
    cluster_sync();  // (the others may still read this one's)
  }
  if (tid == 0 && c.abort) {
    record_status(p.status, GDN_ERR_TIMEOUT);
    wait_out_copies();
  }
}

// Items that a call can have.
long long item_bound(const PagedAttnParams& p) {
  const long long rows = (long long)p.T * p.group;
  return (p.cu ? rows / ROWS + p.N : (rows + ROWS - 1) / ROWS * p.N) * p.c.hkv;
}

int rows_grid() { return paged_sm_count() * kCtasPerSm; }

template <typename E, int D, bool SPLIT>
cudaError_t launch_shape(const PagedAttnParams& p, const CUtensorMap& tk,
                         const CUtensorMap& tv, cudaStream_t stream,
                         int* launches) {
  using S = Shape<D>;
  static_assert(S::kSmem <= 227 * 1024 / kCtasPerSm, "shared memory");
  auto kern = paged_rows_kernel<E, D, SPLIT>;
  static std::atomic<unsigned long long> allowed{0};
  cudaError_t e = paged_allow_smem(kern, S::kSmem, allowed);
  if (e != cudaSuccess) return e;
  const int grid = SPLIT ? (int)item_bound(p) * p.split : rows_grid();
  const int t = timing_start(GDN_KERNEL_PAGED_ROWS, stream);
  e = paged_launch_clusters(kern, SPLIT ? p.split : 1, dim3(grid), kThreads,
                            S::kSmem, stream, p, tk, tv,
                            paged_rows_box(1 << p.c.page_shift));
  timing_stop(t, stream, e);
  if (e != cudaSuccess) return e;
  ++*launches;
  if (SPLIT) return e;
  return launch_paged_merge(p, D, std::is_same<E, __nv_bfloat16>::value, grid,
                            ROWS, stream, launches);
}

template <typename E, int D>
cudaError_t launch_either(const PagedAttnParams& p, const CUtensorMap& tk,
                          const CUtensorMap& tv, cudaStream_t stream,
                          int* launches) {
  return p.split ? launch_shape<E, D, true>(p, tk, tv, stream, launches)
                 : launch_shape<E, D, false>(p, tk, tv, stream, launches);
}

}  // namespace

int paged_rows_box(int page_size) { return page_size < TK ? page_size : TK; }

int paged_rows_split(const PagedAttnParams& p) {
  const long long keys = (long long)p.c.max_pages << p.c.page_shift;
  const bool few = (long long)p.T * p.group <= (long long)ROWS * (p.cu ? p.N : 1);
  for (int s = kMaxSplit; s > 0; s /= 2) {
    const long long ctas = item_bound(p) * s;
    if (ctas > rows_grid() || (s > 1 && keys <= TK * (s / 2))) continue;
    const bool idle = few && 4 * ctas < 3ll * rows_grid();
    return keys <= (long long)(idle ? kSplitKeysIdle : kSplitKeys) * s ? s : 0;
  }
  return 0;
}

size_t paged_rows_workspace_bytes(int d) {
  const size_t grid = rows_grid();
  return grid * 2 * sizeof(int4) + grid * 2 * ROWS * (2 + d) * sizeof(float);
}

void paged_rows_bind_workspace(PagedAttnParams& p, void* ws, int d) {
  const size_t grid = rows_grid();
  p.meta = static_cast<int4*>(ws);
  p.part_o = reinterpret_cast<float*>(p.meta + 2 * grid);
  p.part_ml = p.part_o + grid * 2 * ROWS * d;
}

cudaError_t launch_paged_rows(const PagedAttnParams& p, int d, bool bf16,
                              const CUtensorMap& tk, const CUtensorMap& tv,
                              cudaStream_t stream, int* launches) {
  if (bf16)
    return d == 128
               ? launch_either<__nv_bfloat16, 128>(p, tk, tv, stream, launches)
               : launch_either<__nv_bfloat16, 64>(p, tk, tv, stream, launches);
  return d == 128 ? launch_either<__half, 128>(p, tk, tv, stream, launches)
                  : launch_either<__half, 64>(p, tk, tv, stream, launches);
}

}  // namespace gdn
