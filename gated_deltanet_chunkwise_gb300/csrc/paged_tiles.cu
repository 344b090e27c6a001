// Attention of many query rows over a paged cache (a chunk of a prompt, a few
// drafted tokens): softmax(scale q K^T + mask) V on tcgen05 with the
// accumulators in TMEM.
//
// Rows. The query heads of a key head share its keys, so rows are (token,
// head of the group) pairs: a 128-row tile holds the group for 128 / group
// (rounded down) consecutive tokens. A CTA works on two such tiles against the
// same 128-key tiles, so that every key tile is read once for 256 rows and one
// tile's softmax runs while the tensor core serves the other.
//
// Per key tile j and row tile t (TMEM columns 128 t: S, 256 + D t: O):
//   S = Q K(j)^T     128 x 128, A and B from shared memory
//   P = 2^(S c - m)  one thread a row: S to registers, the row's maximum and
//                    sum there, P (16-bit) back over S in two halves
//   O += P V(j)      A from TMEM, B = V as it lies (N-major)
// Two 128 x 128 fp32 S and two 128 x 128 O fill TMEM's 512 columns, so P goes
// over S and S(j + 1) waits for O += P(j) V(j): the chain softmax -> products
// -> softmax of one row tile is what the other one's work has to cover. (S in
// steps of 64 keys with P beside it decouples the two, but a product of 64
// keys costs as much as one of 128, 85 cycles, bound by the reads of Q: 840 us
// for the case below.) The first half of P goes to work while the second is
// computed (722 -> 671 us).
//
// The reference m (for fp16 2^7 below the maximum) follows the running maximum
// only when a score passes it by more than 2^8 (weights stay below 2^8, fp16
// ones below 2^15; sums and O are fp32), so O, which lives in TMEM, is rarely
// rescaled, and the softmax warps do it themselves: S(j + 1)'s barrier already
// says that O += P(j) V(j) is complete. Weights are rounded to 16 bits for their
// product (2^-9 on the average, as the output is); sums take them unrounded.
//
// Bound: the tensor core, 4 D flops a visible (row, key) pair: 2048 tokens of
// 16 heads against 65536 keys, D = 128 (1.08 TFLOP) take 672 us, 1.6 PFLOP/s,
// and 720 to 740 us called over and over (power-capped). Of a step's 2850 cycles
// the products take 2340. The exponentials (one a pair, 32 a cycle and SM) take
// 1024 beside them. Short items are bound by what they cost once: 3 us to find
// a run's place and 4 us to the first scores, 2 us a change of item, 3 us for
// the last one's output.
//
// Split. The key tiles of all (tile pair, key head) items form one list that
// is cut into equal runs, one per SM (causal items have the tiles that they
// see), so ragged batches, few long items and many short ones fill the machine
// alike. A run that holds a whole item writes its output; pieces of a cut item
// go to the workspace in fp32 and paged_merge.cu joins them in the order
// of the runs. A run that may have spoilt a result (see paged.cuh on hidden
// values) is handed out a second time.
//
// Warps: 0-3 and 4-7 the softmax and epilogue of row tiles 0 and 1 (their TMEM
// lanes), 8 looks pages up and issues TMA copies into a ring of key and value
// tiles, 9 hands out the run's segments and loads their queries, 10 and 11
// issue the products of row tiles 0 and 1.
#include <type_traits>

#include "paged.cuh"
#include "tc_ptx.cuh"

namespace gdn {

using namespace tc;

namespace {

constexpr int TK = 128;  // keys per tile
constexpr int TM = 128;  // rows per tile
constexpr int kThreads = 384;  // three warpgroups, as setmaxnreg wants them
constexpr uint32_t kTmemCols = 512;
// What an item costs beside its key tiles (queries, first scores, output), in
// key tiles, for the even cut of the list: 2 against 1, 3 and 5 changes mixed
// and short prompts by 4 % at most, long ones not at all.
constexpr int kItemCost = 2;
constexpr int kLengthsStaged = 8192;  // sequences whose lengths fit the ring
constexpr int kSegs = 4;       // segments handed out ahead
constexpr int kSegReaders = 11;  // 8 softmax warps, producer, 2 of products

template <int D>
struct Shape {
  static constexpr int kHalves = D / 64;
  static constexpr int kQ = TM * D * 2;     // bytes of a query tile
  static constexpr int kTile = TK * D * 2;  // bytes of a key or value tile
  // 64 KB of queries, 128 KB of keys and values at D = 128, 32 KB (4 for each
  // softmax warp) on the way of results to memory
  static constexpr int kRing = 128 * 1024 / kTile;
  static constexpr int kStage = 8 * 4096;
  static constexpr int kMisc = 1536;
  static constexpr int kSmem = 1024 + 2 * kQ + kRing * kTile + kStage + kMisc;
};
static_assert(Shape<128>::kSmem <= 227 * 1024, "shared memory");
static_assert(Shape<64>::kRing * 16 + 192 <= 512, "barriers");

// ---- the work list -----------------------------------------------------------
struct Slot {
  int n, block;      // sequence, tile pair of it
  int q0, len, kv;   // the sequence
  int tok;           // first token (within the new ones)
  int ntok[2];       // tokens of each row tile
  int b[2], e[2];    // key tiles each row tile needs (b == e: none)
  int lo, hi;        // keys outside [lo, hi) are seen by no row
  int tile0, tiles;  // key tiles of the item; tiles >= 1 unless it has no rows
};

__device__ __forceinline__ int seq_first_slot(const PagedAttnParams& p, int n,
                                              int tt) {
  // packed: floor(cu[n] / 2 tt) + n grows by at least the sequence's pairs
  return p.cu[n] / (2 * tt) + n;
}

__device__ __forceinline__ Slot slot_work(const PagedAttnParams& p, int n,
                                          int block, int tt) {
  const PagedSeq s = paged_seq(p.c, p.cu, p.T, n, p.status);
  Slot w;
  w.n = n;
  w.block = block;
  w.q0 = s.q0;
  w.len = s.len;
  w.kv = s.kv;
  w.tok = block * 2 * tt;
  w.tiles = 0;
  w.tile0 = 0;
  w.lo = w.hi = 0;
#pragma unroll
  for (int t = 0; t < 2; ++t) w.ntok[t] = w.b[t] = w.e[t] = 0;
  if (w.tok < 0 || w.tok >= s.len ||
      (long long)s.len * p.group <= p.rows_min)
    return w;
  const int left = s.len - w.tok;
  bool any = false;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    w.ntok[t] = max(0, min(tt, left - t * tt));
    const int x0 = s.kv - s.len + w.tok + t * tt;
    const int x1 = x0 + w.ntok[t] - 1;
    const int hi = p.causal ? min(s.kv, x1 + 1) : s.kv;
    const int lo = p.window > 0 ? max(0, x0 - p.window + 1) : 0;
    if (w.ntok[t] > 0 && hi > lo) {
      w.b[t] = lo / TK;
      w.e[t] = (hi + TK - 1) / TK;
      w.lo = any ? min(w.lo, lo) : lo;
      w.hi = any ? max(w.hi, hi) : hi;
      any = true;
    }
  }
  if (any) {
    w.tile0 = w.lo / TK;
    w.tiles = (w.hi + TK - 1) / TK - w.tile0;
  } else {
    w.tiles = 1;  // nothing to see, but rows to write
  }
  return w;
}

// Slots of the call: dense ones are (sequence, pair), packed ones lie at
// seq_first_slot with a few unused between sequences. (Fewer than 2^31: a slot
// holds at least one of the call's tokens or is a sequence's spare one.)
__device__ __forceinline__ int pairs_per_sequence(const PagedAttnParams& p,
                                                  int tt) {
  return (p.T + 2 * tt - 1) / (2 * tt);
}

__device__ __forceinline__ int slot_count(const PagedAttnParams& p, int tt) {
  return p.cu ? p.T / (2 * tt) + p.N : p.N * pairs_per_sequence(p, tt);
}

// A place in the slots, stepped one by one.
struct Place {
  int slot, n, first;  // first: the sequence's first slot
};

__device__ __forceinline__ Place place_of(const PagedAttnParams& p, int slot,
                                          int tt) {
  Place x;
  x.slot = slot;
  if (!p.cu) {
    const int pairs = pairs_per_sequence(p, tt);
    x.n = slot / pairs;
    x.first = x.n * pairs;
    return x;
  }
  int lo = 0, hi = p.N - 1;  // the last n with seq_first_slot(n) <= slot
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (seq_first_slot(p, mid, tt) <= slot)
      lo = mid;
    else
      hi = mid - 1;
  }
  x.n = lo;
  x.first = seq_first_slot(p, lo, tt);
  return x;
}

__device__ __forceinline__ void step(const PagedAttnParams& p, Place& x,
                                     int tt) {
  ++x.slot;
  if (!p.cu) {
    const int pairs = pairs_per_sequence(p, tt);
    if (x.slot - x.first == pairs) {
      x.first = x.slot;
      ++x.n;
    }
    return;
  }
  while (x.n + 1 < p.N) {
    const int first = seq_first_slot(p, x.n + 1, tt);
    if (first > x.slot) break;
    ++x.n;
    x.first = first;
  }
}

__device__ __forceinline__ Slot slot_at(const PagedAttnParams& p,
                                        const Place& x, int tt) {
  // (negative where tokens before the first sequence would be: no rows)
  return slot_work(p, x.n, x.slot - x.first, tt);
}

// Units of the list that a slot takes: each head's item counts its key tiles
// and, before them, kItemCost units that stand for its fixed cost.
__device__ __forceinline__ int item_units(const Slot& s) {
  return s.tiles > 0 ? s.tiles + kItemCost : 0;
}

// One run [w, w_end) of the list, walked item by item.
struct Walk {
  long long w, w_end, base;  // base: first unit of the slot at `at`
  Place at;
  int slots;
  Slot s;
};

// A run's share of one item, as the scheduler hands it to the other warps.
struct Segment {
  int n, block, head;     // n < 0: no more
  int q0, before, tok;    // sequence's first token; its keys before the new
                          // ones (negative: fewer keys than new tokens); the
                          // item's first token
  int kv, lo, hi;
  int ntok[2];
  int s0, s1;             // key tiles of this run (absolute); none: s0 == s1
  int first[2], last[2];  // each row tile's share of them
  int starts, ends;       // holds the item's first / last tile
  int last_run;           // the run that holds the item's last tile
  int careful;            // a second time
};

__device__ __forceinline__ bool next_segment(const PagedAttnParams& p, int tt,
                                             long long per, Walk& k,
                                             Segment& g) {
  int t0, t1;
  long long item_end;
  do {
    if (k.w >= k.w_end) return false;
    long long units = item_units(k.s);
    while (k.w >= k.base + units * p.c.hkv) {
      k.base += units * p.c.hkv;
      step(p, k.at, tt);
      if (k.at.slot >= k.slots) return false;
      k.s = slot_at(p, k.at, tt);
      units = item_units(k.s);
    }
    const long long off = k.w - k.base;
    // (off is below the slot's units, 2^32 for any cache that fits the card)
    g.head = off >> 32 ? (int)(off / units)
                       : (int)((uint32_t)off / (uint32_t)units);
    item_end = k.base + (g.head + 1) * units;
    const long long end = item_end < k.w_end ? item_end : k.w_end;
    const int u0 = (int)(off - g.head * units);
    t0 = max(0, u0 - kItemCost);
    t1 = max(0, u0 + (int)(end - k.w) - kItemCost);
    k.w = end;
  } while (t0 == t1);  // a run that ends within the fixed cost
  g.n = k.s.n;
  g.block = k.s.block;
  g.q0 = k.s.q0;
  g.before = k.s.kv - k.s.len;
  g.tok = k.s.tok;
  g.kv = k.s.kv;
  g.lo = k.s.lo;
  g.hi = k.s.hi;
  g.starts = t0 == 0;
  g.ends = t1 == k.s.tiles;
  g.last_run = (int)((item_end - 1) / per);
  g.s0 = k.s.tile0 + t0;
  g.s1 = k.s.tile0 + t1;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    g.ntok[t] = k.s.ntok[t];
    g.first[t] = max(g.s0, k.s.b[t]);
    g.last[t] = max(g.first[t], min(g.s1, k.s.e[t]));
  }
  // an item that sees nothing has no steps
  if (g.first[0] == g.last[0] && g.first[1] == g.last[1]) g.s1 = g.s0;
  return true;
}

// A value that is the same in every lane, told to the compiler.
__device__ __forceinline__ int uniform(int x) {
  return __shfl_sync(0xffffffffu, x, 0);
}

// True in one thread of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

// Pairs of fp32 values in 64-bit registers: one instruction for two.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// (NaN operands are passed over, as by fmaxf)
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Largest of 32 scores: four chains of three-operand maxima.
__device__ __forceinline__ float max32(const float (&s)[32]) {
  float m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = max3(s[i], s[i + 4], s[i + 8]);
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = max3(m[i], s[i + 12], s[i + 16]);
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = max3(m[i], s[i + 20], s[i + 24]);
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = fmaxf(m[i], s[i + 28]);
  return max3(fmaxf(m[0], m[1]), m[2], m[3]);
}
// Scores of columns outside [lo, hi) become -inf; s holds columns from `at`.
// (One bit a column, which turns into predicates several at a time, instead
// of two comparisons a column: a quarter of the code and 1000 cycles less for a
// masked tile.)
__device__ __forceinline__ void mask32(float (&s)[32], int lo, int hi, int at) {
  const int a = min(max(lo - at, 0), 32), b = min(max(hi - at, 0), 32);
  const uint32_t bits = (uint32_t)((1ull << b) - 1ull) &
                        ~(uint32_t)((1ull << a) - 1ull);
#pragma unroll
  for (int i = 0; i < 32; ++i) s[i] = (bits >> i) & 1u ? s[i] : -INFINITY;
}

// Position in the ring of key and value tiles and the parity of its phase,
// stepped without divisions: the warps that use it run one thread's worth of
// instructions per tile on the critical path.
template <int R>
struct Ring {
  uint32_t slot = 0, parity = 0;
  __device__ __forceinline__ Ring next() const {
    Ring r;
    const bool wrap = slot + 1 == R;
    r.slot = wrap ? 0 : slot + 1;
    r.parity = wrap ? parity ^ 1u : parity;
    return r;
  }
};

// Instruction descriptor: 16-bit A and B of the element type, fp32 D.
template <typename E>
__host__ __device__ constexpr uint32_t idesc_of(int N, bool b_mn);
template <>
__host__ __device__ constexpr uint32_t idesc_of<__nv_bfloat16>(int N, bool b_mn) {
  return idesc_bf16(128, N, false, b_mn);
}
template <>
__host__ __device__ constexpr uint32_t idesc_of<__half>(int N, bool b_mn) {
  return idesc_bf16(128, N, false, b_mn) & ~((1u << 7) | (1u << 10));
}

// For tiles that hold a value which is not finite and hidden from some row: O +
// P V of one key tile and a row a lane, key by key, over the keys [lo, hi) that
// the row sees, with the weights that lie in TMEM at t_p for the product. The
// tensor core makes its product all the same and spoils O, so the row is kept in
// `out` and put back when that is done. (Some 60 us a tile.)
template <typename E, int D>
__device__ __noinline__ void add_by_key(uint32_t t_p, uint32_t t_o, const char* v,
                                        int lo, int hi, bool fresh, float* out) {
#pragma unroll 1
  for (int col = 0; col < D; col += 16) {
    float o[16];
    tmem_ld16(t_o + col, o);
    tmem_ld_wait();
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] = fresh ? 0.f : o[e];
    const char* const half = v + (col / 64) * (TK * 128);
#pragma unroll 1
    for (int k0 = 0; k0 < TK; k0 += 32) {
      float p[16];  // pairs of weights
      tmem_ld16(t_p + k0 / 2, p);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const int key = k0 + i;
        const float2 w2 = unpack2(__float_as_uint(p[i / 2]), E());
        const float w = i & 1 ? w2.y : w2.x;
        const bool sees = key >= lo && key < hi;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint4 x = *reinterpret_cast<const uint4*>(
              half + sw128(key, (col % 64) / 8 + c));
          const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 y = unpack2(u[e], E());
            float* const a = o + c * 8 + 2 * e;
            a[0] = sees ? fmaf(w, y.x, a[0]) : a[0];
            a[1] = sees ? fmaf(w, y.y, a[1]) : a[1];
          }
        }
      }
      __syncwarp();
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) out[col + e] = o[e];
  }
}

// A kept row back to O.
template <int D>
__device__ __noinline__ void put_row(uint32_t t_o, const float* row) {
#pragma unroll 1
  for (int col = 0; col < D; col += 16) {
    uint32_t u[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(row[col + e]);
    tmem_st16(t_o + col, u);
  }
  tmem_st_wait();
}

// The softmax of a segment's key tiles the second time, for row tile t (a row a
// thread): as in the kernel (to the order of its additions), but plainly, with
// the care that scores beyond kFar want and a look through the values of tiles
// that some row sees in part. (`at`
// counts the row tile's steps so far, `outs` its outputs, `probes` the steps made
// here; pos: key tiles before the segment.)
struct RowSums {
  float ref, sum;
  bool ok;
};
template <typename E, int D>
__device__ __noinline__ RowSums careful_keys(const PagedAttnParams& p,
                                             const Segment& g, char* kv,
                                             uint64_t* bars, uint64_t* kv_full,
                                             volatile uint32_t* by_key,
                                             volatile int* abort_flag, int t,
                                             uint32_t t_s, uint32_t t_o, int pos,
                                             uint32_t at, uint32_t outs,
                                             uint32_t probes) {
  using S = Shape<D>;
  uint64_t *s_full = bars + 4 + t, *p_full = bars + 6 + 2 * t,
           *o_full = bars + 10 + t, *probed = bars + 22 + t;
  const int r = threadIdx.x & 127, lane = threadIdx.x % 32;
  const int tt = 128 / p.group;
  const int x = g.before + g.tok + t * tt + r / p.group;
  const int hi = p.causal ? min(x + 1, g.kv) : g.kv;
  const int lo = p.window > 0 ? max(0, x - p.window + 1) : 0;
  const bool valid = r < g.ntok[t] * p.group;
  // keys [free_lo, free_hi) are seen by every row of the tile
  const int x0 = g.before + g.tok + t * tt;
  const int free_hi = p.causal ? min(x0 + 1, g.kv) : g.kv;
  const int free_lo = p.window > 0 ? x0 + g.ntok[t] - p.window : 0;
  const int first = g.first[t], last = g.last[t];
  RowSums y{kNegInf, 0.f, false};
#pragma unroll 1
  for (int j = first; j < last; ++j) {
    if (!warp_wait(s_full, at & 1, abort_flag)) return y;
    tc_fence_after();
    ++at;
    const uint32_t v = 2u * (uint32_t)(pos + j - g.s0) + 1u, slot = v % S::kRing;
    if (!warp_wait(&kv_full[slot], (v / S::kRing) & 1, abort_flag)) return y;
    char* const values = kv + slot * S::kTile;
    const int key0 = j * TK, key = key0 + r;
    uint32_t z = 0;
#pragma unroll 1
    for (int i = 0; i < S::kHalves * 8; ++i) {  // (lanes in different banks)
      uint4* const x16 = reinterpret_cast<uint4*>(
          values + (i / 8) * (TK * 128) + r * 128 + (i + lane) % 8 * 16);
      if (key >= g.hi || key < g.lo)
        *x16 = make_uint4(0u, 0u, 0u, 0u);  // seen by no row
      else if (key0 < free_lo || key0 + TK > free_hi)
        z = probe8<E>(*x16, z);
    }
    fence_proxy_async();
    if (probe_hit(z)) by_key[t] = at;
    __syncwarp();
    if (lane == 0) mbar_arrive(probed);
    if (!warp_wait(probed, probes++ & 1, abort_flag)) return y;
    const bool spoilt = by_key[t] == at;
    float top = kNegInf;
#pragma unroll 1
    for (int i = 0; i < TK; i += 32) {
      float s[32];
      tmem_ld32(t_s + i, s);
      tmem_ld_wait();
      mask32(s, lo - key0, hi - key0, i);
      top = fmaxf(top, max32(s));
    }
    top *= p.scale_log2;
    if (__any_sync(0xffffffffu, valid && top > y.ref + kSlack + kLift<E>)) {
      const float now = fmaxf(y.ref, top - kLift<E>);
      const float f = factor(y.ref, now);
      y.ref = now;
      y.sum *= f;
#pragma unroll 1
      for (int i = 0; j > first && i < D; i += 16) {
        float o[16];
        tmem_ld16(t_o + i, o);
        tmem_ld_wait();
        uint32_t u[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(o[e] * f);
        tmem_st16(t_o + i, u);
      }
    }
    const float m = y.ref == kNegInf ? 0.f : y.ref;
    const bool far = __any_sync(0xffffffffu, valid && fabsf(y.ref) >= kFar &&
                                                 y.ref != kNegInf);
    uint64_t part[2] = {0, 0};  // (the kernel's order of additions)
#pragma unroll 1
    for (int i = 0; i < TK; i += 32) {  // (weights over scores read already)
      float s[32];
      tmem_ld32(t_s + i, s);
      tmem_ld_wait();
      mask32(s, lo - key0, hi - key0, i);
      uint32_t u[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float a = ex2(far ? __fmul_rn(s[2 * e], p.scale_log2) - m
                                : fmaf(s[2 * e], p.scale_log2, -m));
        const float b = ex2(far ? __fmul_rn(s[2 * e + 1], p.scale_log2) - m
                                : fmaf(s[2 * e + 1], p.scale_log2, -m));
        part[e & 1] = add2(part[e & 1], pair(a, b));
        u[e] = pack2<E>(a, b);
      }
      tmem_st16(t_s + i / 2, u);
    }
    float even, odd;
    unpair(add2(part[0], part[1]), even, odd);
    y.sum += even + odd;
    tmem_st_wait();
    float o[D];
    if (spoilt)
      add_by_key<E, D>(t_s, t_o, values, lo - key0, hi - key0, j == first, o);
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(p_full);
      mbar_arrive(p_full + 1);
    }
    if (spoilt) {
      if (!(j + 1 < last ? warp_wait(s_full, at & 1, abort_flag)
                         : warp_wait(o_full, outs & 1, abort_flag)))
        return y;
      tc_fence_after();
      put_row<D>(t_o, o);
    }
  }
  y.ok = true;
  return y;
}

template <typename E, int D>
__global__ void __launch_bounds__(kThreads, 1)
    paged_tiles_kernel(const __grid_constant__ PagedAttnParams p,
                       const __grid_constant__ CUtensorMap tq,
                       const __grid_constant__ CUtensorMap tk,
                       const __grid_constant__ CUtensorMap tv, int box) {
  using S = Shape<D>;
  extern __shared__ char smem_raw[];
  char* sm = reinterpret_cast<char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  char* sm_q = sm;
  char* sm_kv = sm + 2 * S::kQ;
  char* sm_out = sm_kv + S::kRing * S::kTile;
  char* misc = sm_out + S::kStage;
  uint64_t* bars = reinterpret_cast<uint64_t*>(misc);
  uint64_t* q_full = bars;        // [2]
  uint64_t* q_empty = bars + 2;   // [2]
  uint64_t* s_full = bars + 4;    // [2]
  uint64_t* p_full = bars + 6;    // [2][2], halves of a tile's weights
  uint64_t* o_full = bars + 10;   // [2]
  uint64_t* o_free = bars + 12;   // [2]
  uint64_t* seg_full = bars + 14;   // [kSegs]
  uint64_t* seg_empty = bars + 18;  // [kSegs]
  uint64_t* probed = bars + 22;     // [2]
  uint64_t* kv_full = bars + 24;
  uint64_t* kv_empty = kv_full + S::kRing;
  long long* s_sum = reinterpret_cast<long long*>(misc + 512);  // [12]
  long long* s_base = s_sum + 12;
  Place* s_place = reinterpret_cast<Place*>(misc + 624);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(misc + 640);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 644);
  int* s_n = reinterpret_cast<int*>(misc + 648);
  // a result may hold what its row does not see, or its scores are beyond kFar
  volatile int* redo = reinterpret_cast<volatile int*>(misc + 652);
  // [2]: the row tile's last step that its softmax warps made key by key
  volatile uint32_t* by_key = reinterpret_cast<volatile uint32_t*>(misc + 656);
  // [8]: the softmax warp is at the first half of a step
  volatile uint32_t* busy = reinterpret_cast<volatile uint32_t*>(misc + 664);
  Segment* s_seg = reinterpret_cast<Segment*>(misc + 696);  // [kSegs]
  static_assert(696 + kSegs * sizeof(Segment) <= S::kMisc, "segments");

  const int tid = threadIdx.x, lane = tid % 32;
  const int warp = uniform(tid / 32);
  const int tt = 128 / p.group;  // tokens per row tile
  const int hkv = p.c.hkv;

  if (tid < (int)(kv_full - bars) + 2 * S::kRing) {
    // barriers, a thread each: all count one arrival but these
    uint64_t* const bar = bars + tid;
    uint32_t count = 1;
    if (bar >= kv_empty)
      count = 2;
    else if ((bar >= p_full && bar < o_full) || (bar >= o_free && bar < seg_full) ||
             (bar >= probed && bar < kv_full))
      count = 4;
    else if (bar >= seg_empty && bar < probed)
      count = kSegReaders;
    mbar_init(bar, count);
    fence_mbar_init();
  }
  if (tid == 0) {
    *abort_flag = 0;
    *s_n = -1;
    *redo = 0;
    by_key[0] = by_key[1] = 0;
    for (int i = 0; i < 8; ++i) busy[i] = 0;
    prefetch_tmap(&tq);
    prefetch_tmap(&tk);
    prefetch_tmap(&tv);
  }
  griddep_wait();  // nothing above touches what earlier kernels write
  // (TMEM too only now: a block of the last kernel may still be to allocate
  // its own, and this one would hold it until that kernel ends)
  if (warp == 9) {
    tmem_alloc(s_tmem, kTmemCols);
    tmem_relinquish();
  }
  if (tid == 0) p.meta[2 * blockIdx.x] = make_int4(-1, 0, 0, 0);

  // The sequences' lengths in shared memory (where keys and values come
  // later) while the run's place is sought: one trip to memory instead of one
  // per probe.
  PagedAttnParams ps = p;
  const bool staged = p.N <= kLengthsStaged;
  int32_t* lens = reinterpret_cast<int32_t*>(sm_kv);
  int32_t* cu = lens + kLengthsStaged;
  if (staged)
    for (int i = tid; i < p.N; i += kThreads) lens[i] = p.c.kv_lens[i];
  bool bad = false;
  if (p.cu)
    for (int i = tid; i < p.N; i += kThreads) {
      const int b = p.cu[i], e = p.cu[i + 1];
      bad = bad || !ordered_pair(b, e, p.T);
      if (staged) {
        cu[i] = b;
        if (i + 1 == p.N) cu[p.N] = e;
      }
    }
  if (bad) record_status(p.status, GDN_ERR_INVALID_ARG);
  const bool skip = __syncthreads_or(bad);
  if (staged) {
    ps.c.kv_lens = lens;
    if (p.cu) ps.cu = cu;
  }

  // where this CTA's run lies: thread t sums slots [t * per_t, ...). (The slots
  // of a packed batch follow its offsets, so they have to be in order.)
  const int slots = skip ? 0 : slot_count(p, tt);
  const int per_t = (slots + kThreads - 1) / kThreads;
  const int lo_s = (int)min((long long)slots, (long long)tid * per_t);
  const int hi_s = min(slots, lo_s + per_t);
  long long mine = 0;
  Place my{};
  if (lo_s < hi_s) {
    my = place_of(ps, lo_s, tt);
    for (Place x = my; x.slot < hi_s; step(ps, x, tt))
      mine += (long long)item_units(slot_at(ps, x, tt)) * hkv;
  }
  long long scan = mine;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const long long up = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += up;
  }
  if (lane == 31) s_sum[warp] = scan;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  long long total = 0, before = scan - mine;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) before += s_sum[i];
    total += s_sum[i];
  }
  const long long per = (total + gridDim.x - 1) / gridDim.x;
  const long long w0 = per * blockIdx.x;
  const long long w1 = w0 + per < total ? w0 + per : total;
  if (w0 < w1 && mine > 0 && w0 >= before && w0 < before + mine) {
    long long base = before;
    Place x = my;
    for (; x.slot < hi_s; step(ps, x, tt)) {
      const long long u = (long long)item_units(slot_at(ps, x, tt)) * hkv;
      if (w0 < base + u) break;
      base += u;
    }
    *s_base = base;
    *s_place = x;
    *s_n = x.n;
  }
  fence_proxy_async();  // (the staged lengths, before copies land there)
  __syncthreads();
  const uint32_t tmem = *s_tmem;
  const uint32_t tmem_u = (uint32_t)uniform((int)tmem);
  const bool work = *s_n >= 0;

  // 168 registers a thread at launch: the softmax warps hold 128 scores each
  // and take 216, the third warpgroup gives 96 back ((216 + 216 + 72) * 128 =
  // 168 * 384)
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (work && warp == 9) {
      // ---- scheduler: hands the run's segments out, loads their queries ----------
      if (lane == 0) {
        uint32_t loads[2] = {0, 0};
        int i = 0;  // segments handed out
        bool ok = true;
        // a second time if a result of the first may hold hidden values
        for (int pass = 0; pass < 2; ++pass) {
          Walk walk;
          walk.slots = slots;
          walk.w = w0;
          walk.w_end = w1;
          walk.base = *s_base;
          walk.at = *s_place;
          walk.s = slot_at(p, walk.at, tt);
          for (; ok; ++i) {
            if (i >= kSegs)
              ok = fast_wait(&seg_empty[i % kSegs], (i / kSegs - 1) & 1,
                             abort_flag);
            Segment g;
            if (!ok || !next_segment(p, tt, per, walk, g)) break;
            g.careful = pass;
            s_seg[i % kSegs] = g;
            mbar_arrive(&seg_full[i % kSegs]);
            if (g.s0 == g.s1) continue;
            // its queries, a row tile's once the last scores of that row tile
            // are done with theirs
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (!ok || g.first[t] >= g.last[t]) continue;
              if (loads[t] > 0)
                ok = fast_wait(&q_empty[t], (loads[t] - 1) & 1, abort_flag);
              if (!ok) continue;
              ++loads[t];
              mbar_arrive_expect_tx(&q_full[t], S::kHalves * tt * p.group * 128);
#pragma unroll
              for (int h = 0; h < S::kHalves; ++h)
                tma_load_4d(sm_q + t * S::kQ + h * (TM * 128), &tq, &q_full[t],
                            h * 64, g.head * p.group, g.q0 + g.tok + t * tt, 0);
            }
          }
          if (!ok || i == 0 ||
              !fast_wait(&seg_empty[(i - 1) % kSegs], ((i - 1) / kSegs) & 1,
                         abort_flag) ||
              !*redo)
            break;
        }
        if (ok) {
          s_seg[i % kSegs].n = -1;
          mbar_arrive(&seg_full[i % kSegs]);
        }
      }
      __syncwarp();
    } else if (work && warp == 8) {
      // ---- producer ------------------------------------------------------------
      const int page = 1 << p.c.page_shift;
      const int boxes = TK / box;                    // <= 8
      const int per_tile = boxes * S::kHalves;       // copies of a tile: <= 16
      const int l16 = lane & 15, b = l16 / S::kHalves, hf = l16 % S::kHalves;
      const bool is_v = lane >= 16;
      Ring<S::kRing> at;  // of the next tile
      bool refill = false;  // the ring has been full once
      bool ok = true;
      for (int i = 0; ok; ++i) {
        const Segment& g = s_seg[i % kSegs];
        ok = warp_wait(&seg_full[i % kSegs], (i / kSegs) & 1, abort_flag);
        if (!ok) break;
        const int n = g.n, s0 = g.s0, s1 = g.s1, lo = g.lo, hi = g.hi;
        const int head = g.head;
        __syncwarp();
        if (lane == 0) mbar_arrive(&seg_empty[i % kSegs]);
        if (n < 0) break;
        const int32_t* table = p.c.table + (long long)n * p.c.table_stride;
        // this lane's page of key tile j: looked up a tile ahead
        auto lookup = [&](int j) {
          const int key = j * TK + b * box;
          if (l16 >= per_tile || j >= s1 || key >= hi || key + box <= lo)
            return -1;
          const int pid = table[key >> p.c.page_shift];
          if (pid >= 0 && pid < p.c.num_pages) return pid;
          record_status(p.status, GDN_ERR_INVALID_ARG);
          return p.c.num_pages;  // past the pool: the copy fills zeros
        };
        int pid = lookup(s0);
        for (int j = s0; ok && j < s1; ++j) {
          const int next = lookup(j + 1);
          const uint32_t bytes =
              (uint32_t)__popc(__ballot_sync(0xffffffffu, pid >= 0) & 0xffffu) *
              box * 128;
          const int row = (j * TK + b * box) & (page - 1);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const uint32_t st = at.slot;
            if (refill) ok = warp_wait(&kv_empty[st], at.parity ^ 1u, abort_flag);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(&kv_full[st], bytes);
            __syncwarp();
            if (pid >= 0 && is_v == (kv == 1))
              tma_load_4d(sm_kv + st * S::kTile + hf * (TK * 128) + b * box * 128,
                          kv ? &tv : &tk, &kv_full[st], hf * 64, row, head, pid);
            at = at.next();
            refill = refill || at.slot == 0;
          }
          pid = next;
        }
      }
    } else if (work) {
      // ---- products --------------------------------------------------------------
      // One warp per row tile, so that one's waits overlap the other's
      // products. The whole warp walks the loop and one elected thread issues:
      // the operands of tcgen05.mma are warp-uniform registers, which values
      // of a divergent branch have to be moved into one by one (90 cycles a
      // product with the loop inside `if (lane == 0)`, 60 like this). A wait
      // costs 90 cycles even when its barrier is ready (and as much again for
      // every other barrier that lanes of the warp poll with it), so what is
      // ready early is waited for early.
      const int t = warp - 10;
      constexpr uint32_t iqk = idesc_of<E>(TK, false);
      constexpr uint32_t ipv = idesc_of<E>(D, true);
      using Pos = Ring<S::kRing>;
      Pos at;  // of the segment's current key tile
      uint32_t seg = 0, step = 0, outs = 0;
      bool ok = true;
      const uint64_t qd = sdesc(smem_u32(sm_q) + t * S::kQ, 0, 1024);
      const uint64_t kd = sdesc(smem_u32(sm_kv), 0, 1024);
      const uint64_t vd = sdesc(smem_u32(sm_kv), TK * 128, 1024);
      const uint32_t t_s = tmem_u + t * 128, t_o = tmem_u + 256 + t * D;
      auto qk = [&](const Pos& x) {
        const uint64_t ks = kd + x.slot * (uint32_t)(S::kTile >> 4);
#pragma unroll
        for (int h = 0; h < S::kHalves; ++h)
          mma_bf16_run<4>(t_s, qd + h * (TM * 128 >> 4), 32,
                          ks + h * (TK * 128 >> 4), 32, iqk, h > 0);
        mma_commit(&s_full[t]);
      };
      for (int i = 0; ok; ++i) {
        ok = warp_wait(&seg_full[i % kSegs], (i / kSegs) & 1, abort_flag);
        if (!ok) break;
        const Segment& g = s_seg[i % kSegs];
        const int n = uniform(g.n), s0 = uniform(g.s0), s1 = uniform(g.s1);
        const int first = uniform(g.first[t]), last = uniform(g.last[t]);
        if (lane == 0) mbar_arrive(&seg_empty[i % kSegs]);
        if (n < 0) break;
        if (s0 == s1) continue;
        if (first < last) ok = warp_wait(&q_full[t], seg++ & 1, abort_flag);
        ok = ok && warp_wait(&kv_full[at.slot], at.parity, abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          if (first <= s0 && s0 < last) {
            qk(at);
            if (s0 + 1 == last) mma_commit(&q_empty[t]);
          }
          mma_commit(&kv_empty[at.slot]);
        }
        __syncwarp();
        for (int j = s0; j < s1; ++j) {
          const bool next = j + 1 < s1;
          const bool pv = first <= j && j < last;
          const Pos v = at.next(), k = v.next();
          // (what is ready long before the weights is waited for first: a wait
          // on a barrier that is ready costs 90 cycles)
          ok = warp_wait(&kv_full[v.slot], v.parity, abort_flag) &&
               (!next || warp_wait(&kv_full[k.slot], k.parity, abort_flag));
          // the last item's outputs have been read
          if (pv && j == first && outs++ > 0)
            ok = ok && warp_wait(&o_free[t], outs & 1, abort_flag);
          const uint64_t vs = vd + v.slot * (uint32_t)(S::kTile >> 4);
          if (pv) {
            // the first half's weights go to work while the second half's are
            // being computed
            ok = ok && warp_wait(&p_full[2 * t], step, abort_flag);
            if (!ok) break;
            tc_fence_after();
            if (elect_one())
              mma_bf16_ta_run<TK / 32>(t_o, t_s, vs, 2048, ipv, j > first);
            __syncwarp();
            ok = warp_wait(&p_full[2 * t + 1], step, abort_flag);
            step ^= 1u;
          }
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            if (pv) {
              mma_bf16_ta_run<TK / 32>(t_o, t_s + TK / 4,
                                       vs + (TK / 2 * 128 >> 4), 2048, ipv,
                                       true);
              if (j + 1 == last) mma_commit(&o_full[t]);
            }
            if (next && first <= j + 1 && j + 1 < last) {
              qk(k);
              if (j + 2 == last) mma_commit(&q_empty[t]);
            }
            mma_commit(&kv_empty[v.slot]);
            if (next) mma_commit(&kv_empty[k.slot]);
          }
          __syncwarp();
          at = v.next();
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    if (work) {
      // ---- softmax and epilogue ------------------------------------------------
      const int t = warp / 4;
      const int r = tid & 127;  // row of the tile, TMEM lane
      const uint32_t t_lane = tmem + ((uint32_t)(warp & 3) << 21);
      const uint32_t t_s = t_lane + t * 128, t_o = t_lane + 256 + t * D;
      const float c = p.scale_log2;
      int pos = 0;  // key tiles (of any item) before this segment's
      int steps = 0, outs = 0;  // of this row tile, over all segments
      int probes = 0;
      bool ok = true;
      const int rt = r / p.group, rh = r - rt * p.group;
      for (int i_seg = 0; ok; ++i_seg) {
        const Segment& g = s_seg[i_seg % kSegs];
        ok = warp_wait(&seg_full[i_seg % kSegs], (i_seg / kSegs) & 1, abort_flag);
        if (!ok || g.n < 0) break;
        const bool valid = r < g.ntok[t] * p.group;
        const int x0 = g.before + g.tok + t * tt;
        const int x = x0 + rt, kv = g.kv;
        const int hi = p.causal ? min(x + 1, kv) : kv;
        const int lo = p.window > 0 ? max(0, x - p.window + 1) : 0;
        // keys [free_lo, free_hi) are seen by every row of the tile, keys
        // outside [any_lo, any_hi) by none of the item
        const int free_hi = p.causal ? min(x0 + 1, kv) : kv;
        const int free_lo = p.window > 0 ? x0 + g.ntok[t] - p.window : 0;
        const int any_lo = g.lo, any_hi = g.hi;
        const int s0 = g.s0, first = g.first[t], last = g.last[t];
        const int looks = g.first[1 - t] < g.last[1 - t] ? 8 : 0;
        float ref = kNegInf, sum = 0.f;
        int begin = first;
        if (g.careful) {
          const RowSums y = careful_keys<E, D>(p, g, sm_kv, bars, kv_full, by_key,
                                               abort_flag, t, t_s, t_o, pos, steps,
                                               outs, probes);
          ok = y.ok;
          if (!ok) break;
          ref = y.ref;
          sum = y.sum;
          steps += last - first;
          probes += last - first;
          begin = last;
        }
        for (int j = begin; j < last; ++j) {
          ok = warp_wait(&s_full[t], steps & 1, abort_flag);
          if (!ok) break;
          tc_fence_after();
          // (S(j) follows O += P(j - 1) V(j - 1): O may be rescaled)
          ++steps;
          const int key0 = j * TK;
          // the second half's load is in flight behind the first half's maximum
          float x[4][32];
          const bool masked = key0 < free_lo || key0 + TK > free_hi;
          const int see_lo = lo - key0, see_hi = hi - key0;
          tmem_ld32(t_s, x[0]);
          tmem_ld32(t_s + 32, x[1]);
          // Let the other row tile's warp of this scheduler finish its first
          // half (some 40 cycles a look, and then on in any case). The row tiles
          // fall into step with each other otherwise: their exponentials share
          // the scheduler, then the tensor core waits (2048 tokens over 65536
          // keys 725 us, 880 without the looks). Not before masked tiles, where
          // looks cost more than they give, nor where the other row tile has no
          // keys (4 drafted tokens of 8 heads over 3000 to 9000 keys, D = 64:
          // 39.8 us, 41.0 with).
#pragma unroll 1
          for (int i = 0; !masked && i < looks && busy[warp ^ 4] != 0; ++i) {
          }
          __syncwarp();
          if (lane == 0) busy[warp] = 1;
          tmem_ld_wait();
          tmem_ld32(t_s + 64, x[2]);
          tmem_ld32(t_s + 96, x[3]);
          if (masked) {
            mask32(x[0], see_lo, see_hi, 0);
            mask32(x[1], see_lo, see_hi, 32);
          }
          float top = fmaxf(max32(x[0]), max32(x[1]));
          tmem_ld_wait();
          if (masked) {
            mask32(x[2], see_lo, see_hi, 64);
            mask32(x[3], see_lo, see_hi, 96);
          }
          top = max3(top, max32(x[2]), max32(x[3])) * c;
          if (key0 + TK > any_hi || key0 < any_lo) {
            // zero the values of keys that no row sees: their weights are 0,
            // and 0 * NaN is NaN
            const uint32_t v = 2u * (uint32_t)(pos + j - s0) + 1u;
            const uint32_t slot = v % S::kRing;
            ok = warp_wait(&kv_full[slot], (v / S::kRing) & 1, abort_flag);
            if (!ok) break;
            const int key = key0 + r;
            if (key >= any_hi || key < any_lo) {
              char* row = sm_kv + slot * S::kTile + r * 128;
#pragma unroll
              for (int i = 0; i < S::kHalves * 8; ++i)
                *reinterpret_cast<uint4*>(row + (i / 8) * (TK * 128) +
                                          (i % 8) * 16) =
                    make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async();
          }
          const bool grow = valid && top > ref + kSlack + kLift<E>;
          if (__any_sync(0xffffffffu, grow)) {
            const float now = fmaxf(ref, top - kLift<E>);
            const float f = factor(ref, now);
            ref = now;
            sum *= f;
            if (valid && now != kNegInf && fabsf(now) >= kFar) *redo = 1;
            if (j > first) {
#pragma unroll 1
              for (int i = 0; i < D; i += 16) {
                float o[16];
                tmem_ld16(t_o + i, o);
                tmem_ld_wait();
                uint32_t u[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(o[e] * f);
                tmem_st16(t_o + i, u);
              }
            }
          }
          // (a long row's sum gets one addition per tile)
          const float m = ref == kNegInf ? 0.f : ref;
          const uint64_t c2 = pair(c, c), m2 = pair(-m, -m);
          uint64_t part[2] = {0, 0};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t u[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float a, b;
              unpair(fma2(pair(x[i][2 * e], x[i][2 * e + 1]), c2, m2), a, b);
              a = ex2(a);
              b = ex2(b);
              part[e & 1] = add2(part[e & 1], pair(a, b));
              u[e] = pack2<E>(a, b);
            }
            tmem_st16(t_s + i * 16, u);
            if (i == 1) {
              tmem_st_wait();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) {
                mbar_arrive(&p_full[2 * t]);
                busy[warp] = 0;
              }
            }
          }
          float pa, pb;
          unpair(add2(part[0], part[1]), pa, pb);
          sum += pa + pb;
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[2 * t + 1]);
        }
        if (!ok) break;
        const bool some = first < last;
        pos += g.s1 - s0;

        // ---- this run's piece of the item ------------------------------------------
        if (some) {
          ok = warp_wait(&o_full[t], outs & 1, abort_flag);
          if (!ok) break;
          ++outs;
          tc_fence_after();
        }
        const bool whole = g.starts && g.ends;
        const long long tok = g.q0 + (long long)(g.tok + t * tt + rt);
        const int head = g.head * p.group + rh;
        const long long piece =
            (long long)(2 * blockIdx.x + (g.starts ? 1 : 0)) *
                (2 * tt * p.group) +
            t * tt * p.group + r;
        if (valid) {
          if (!whole)
            *reinterpret_cast<float2*>(p.part_ml + piece * 2) =
                make_float2(ref, sum);
          else if (p.lse)
            p.lse[tok * p.hq + head] = row_lse(ref, sum);
        }
        // Rows leave through 4 KB of shared memory per warp, 128 bytes of each
        // row at a time: a lane's own row would put every store of the warp in
        // 32 lines of memory instead of 4.
        char* stage = sm_out + warp * 4096;
        char* const dst = whole ? static_cast<char*>(p.out)
                                : reinterpret_cast<char*>(p.part_o);
        const long long row_off =
            !valid || (!whole && !some) ? -1
            : whole                     ? (tok * p.hq + head) * (D * 2)
                                        : piece * (D * 4);
        const bool none = !some || (whole && hi <= lo);  // sees nothing: 0
        const float scale = 1.f / sum;
        const int chunks = whole ? D / 64 : D / 32;
        uint32_t odd = 0;  // a column of the row is not finite
#pragma unroll 1
        for (int i = 0; i < chunks; ++i) {
          uint32_t u[32];
          if (!some) {
            // (no TMEM to read)
          } else if (whole) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float o[32];
              tmem_ld32(t_o + i * 64 + h * 32, o);
              tmem_ld_wait();
              odd |= nonfinite(o);
#pragma unroll
              for (int e = 0; e < 16; ++e)
                u[h * 16 + e] = pack2<E>(o[2 * e] * scale, o[2 * e + 1] * scale);
            }
          } else {
            float o[32];
            tmem_ld32(t_o + i * 32, o);
            tmem_ld_wait();
            odd |= nonfinite(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(o[e]);
          }
          if (none) {
#pragma unroll
            for (int e = 0; e < 32; ++e) u[e] = 0u;
          }
          if (some && i + 1 == chunks) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&o_free[t]);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<uint4*>(stage + sw128(lane, e)) =
                make_uint4(u[4 * e], u[4 * e + 1], u[4 * e + 2], u[4 * e + 3]);
          __syncwarp();
          uint4 y[8];
          long long off[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int from = e * 4 + lane / 8;
            off[e] = __shfl_sync(0xffffffffu, row_off, from);
            y[e] = *reinterpret_cast<const uint4*>(stage + sw128(from, lane & 7));
          }
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (off[e] >= 0)
              *reinterpret_cast<uint4*>(dst + off[e] + i * 128 +
                                        (lane & 7) * 16) = y[e];
          __syncwarp();
        }
        // a row that is not finite and does not see all that was multiplied
        const int low = max(lo, first * TK), high = min(hi, last * TK);
        const bool bad = valid && !none && odd != 0 &&
                         (low > max(any_lo, first * TK) ||
                          high < min(any_hi, last * TK));
        if (bad) *redo = 1;
        if (tid == 0 && g.starts && !g.ends) {
          p.meta[2 * blockIdx.x] =
              make_int4(g.n, g.head, g.block, g.last_run);
          p.meta[2 * blockIdx.x + 1] =
              make_int4(g.q0, kv - g.before, kv, 0);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&seg_empty[i_seg % kSegs]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    if (tid == 0) record_status(p.status, GDN_ERR_TIMEOUT);
    wait_out_copies();
    __syncthreads();
  }
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <typename E, int D>
cudaError_t launch_shape(const PagedAttnParams& p, const CUtensorMap& tq,
                         const CUtensorMap& tk, const CUtensorMap& tv,
                         cudaStream_t stream, int* launches) {
  using S = Shape<D>;
  auto kern = paged_tiles_kernel<E, D>;
  static std::atomic<unsigned long long> allowed{0};
  cudaError_t e = paged_allow_smem(kern, S::kSmem, allowed);
  if (e != cudaSuccess) return e;
  const int grid = paged_sm_count();
  const int t = timing_start(GDN_KERNEL_PAGED_TILES, stream);
  e = paged_launch(kern, dim3(grid), kThreads, S::kSmem, stream, p, tq, tk, tv,
                   paged_tiles_box(1 << p.c.page_shift));
  timing_stop(t, stream, e);
  if (e != cudaSuccess) return e;
  ++*launches;
  return launch_paged_merge(p, D, std::is_same<E, __nv_bfloat16>::value, grid,
                            2 * (128 / p.group) * p.group, stream, launches);
}

}  // namespace

int paged_tiles_box(int page_size) { return page_size < TK ? page_size : TK; }

size_t paged_tiles_workspace_bytes(const PagedAttnParams& p, int d) {
  const size_t grid = paged_sm_count(), rows = 2 * (128 / p.group) * p.group;
  return grid * 2 * sizeof(int4) + grid * 2 * rows * (2 + d) * sizeof(float);
}

void paged_tiles_bind_workspace(PagedAttnParams& p, void* ws, int d) {
  const size_t grid = paged_sm_count(), rows = 2 * (128 / p.group) * p.group;
  p.meta = static_cast<int4*>(ws);
  p.part_o = reinterpret_cast<float*>(p.meta + 2 * grid);
  p.part_ml = p.part_o + grid * 2 * rows * d;
}

cudaError_t launch_paged_tiles(const PagedAttnParams& p, int d, bool bf16,
                               const CUtensorMap& tq, const CUtensorMap& tk,
                               const CUtensorMap& tv, cudaStream_t stream,
                               int* launches) {
  if (bf16)
    return d == 128
               ? launch_shape<__nv_bfloat16, 128>(p, tq, tk, tv, stream, launches)
               : launch_shape<__nv_bfloat16, 64>(p, tq, tk, tv, stream, launches);
  return d == 128 ? launch_shape<__half, 128>(p, tq, tk, tv, stream, launches)
                  : launch_shape<__half, 64>(p, tq, tk, tv, stream, launches);
}

}  // namespace gdn
