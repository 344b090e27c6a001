// Appending new tokens to the paged cache, with the position rotation of
// queries and keys on the way.
//
// Pair i of a head (elements i and i + rot/2, or 2i and 2i + 1 when
// interleaved) turns by the angle whose cosine and sine stand at columns i
// and rot/2 + i of row p of the table:
//   (a, b) -> (a cos - b sin, b cos + a sin)
// with p the token's place in its sequence, or its given position on the
// axis that owns pair i. Elements past `rot` are copied. Arithmetic is fp32
// on the 16-bit inputs, rounded once.
//
// Bound: HBM. 4 (hq + 2 hkv) D bytes a token are unavoidable, one read and
// one write of every element.
//
// Layout of the work: a warp serves one token (or a share of its heads when
// there are few tokens), so the search for the token's sequence and its page
// lookup are warp-uniform and need no shared memory. A lane owns two 16-byte
// vectors of a head (the two halves of 8 pairs) and walks over the heads with
// the cosines and sines of its pairs in registers, so the table is read once
// per token and lane, not once per head. Three head rows are loaded before the
// first is stored: 15,100 tokens of 32 + 2 * 8 heads of 128 (379 MB) take 58 us
// a call one after the other, 6.5 TB/s (between events around each launch, which
// add 4 us: 62 us, two rows 68 us, six 63 us).
#include "paged.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kBatch = 3;

// The sequence that owns packed token t: the number of ends cu[1..N] that are
// <= t, found 32 probes at a time (two steps serve 1024 sequences).
__device__ __forceinline__ int find_sequence(const int32_t* cu, int N, int t,
                                             int lane) {
  int lo = 0, span = N;  // the answer lies in [lo, lo + span]
  while (span > 0) {
    const int step = (span + 31) / 32;
    const int at = lo + (lane + 1) * step;  // 1-based end index
    const bool below = at <= lo + span && cu[at] <= t;
    const int hits = __popc(__ballot_sync(0xffffffffu, below));
    lo += hits * step;
    span = min(step - 1, max(0, N - lo));
  }
  return lo;
}

template <typename E, int D>
__global__ void __launch_bounds__(kThreads)
    paged_append_kernel(const __grid_constant__ PagedAppendParams p,
                        int warps_per_token) {
  constexpr int LPR = D / 16;    // lanes per head row
  constexpr int RPW = 32 / LPR;  // head rows per warp step
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const long long tok = (long long)blockIdx.x * (kWarps / warps_per_token) +
                        warp / warps_per_token;
  tc::griddep_launch_dependents();
  tc::griddep_wait();
  // offsets that decrease or leave the batch, which a token may not meet
  if (p.cu && blockIdx.x == 0)
    for (int j = threadIdx.x; j < p.N; j += kThreads)
      if (!ordered_pair(p.cu[j], p.cu[j + 1], p.T))
        record_status(p.status, GDN_ERR_INVALID_ARG);
  if (tok >= p.tokens) return;
  int n;
  if (p.cu) {
    n = find_sequence(p.cu, p.N, (int)tok, lane);
    if (n >= p.N) return;  // past the last sequence: belongs to none
  } else {
    n = (int)(tok / p.T);
  }
  const PagedSeq s = paged_seq(p.c, p.cu, p.T, n, p.status);
  if (!s.ok) return;
  const int i = (int)tok - s.q0;
  const int x = s.kv - s.len + i;
  // before the first sequence: belongs to none (or between offsets that
  // decrease, recorded above)
  if (i < 0 || i >= s.len) return;
  if (x < 0) {
    record_status(p.status, GDN_ERR_INVALID_ARG);
    return;
  }
  const int page = p.c.table[(long long)n * p.c.table_stride +
                             (x >> p.c.page_shift)];
  if (page < 0 || page >= p.c.num_pages) {
    record_status(p.status, GDN_ERR_INVALID_ARG);
    return;
  }
  const int slot = x & ((1 << p.c.page_shift) - 1);

  // this lane's two vectors of a head row, and its pairs' cosines and sines
  const int c = lane % LPR, half = p.rot / 2;
  const bool turns = c * 16 < p.rot;
  const int e0 = turns && !p.interleaved ? c * 8 : c * 16;
  const int e1 = turns && !p.interleaved ? half + c * 8 : c * 16 + 8;
  int row[4] = {x, x, x, x};
  if (p.rot > 0) {
    bool bad = false;
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      if (p.positions && a < p.axes) row[a] = p.positions[a * p.tokens + tok];
      bad = bad || (a < p.axes && (row[a] < 0 || row[a] >= p.rope_rows));
    }
    if (bad) {
      record_status(p.status, GDN_ERR_INVALID_ARG);
      return;
    }
  }
  float cs[8], sn[8];
  if (turns && p.axes == 1) {
    const float4* r = reinterpret_cast<const float4*>(
        p.rope + (long long)row[0] * p.rot + c * 8);
    const float4 f = r[0], g = r[1], u = r[half / 4], w = r[half / 4 + 1];
    cs[0] = f.x; cs[1] = f.y; cs[2] = f.z; cs[3] = f.w;
    cs[4] = g.x; cs[5] = g.y; cs[6] = g.z; cs[7] = g.w;
    sn[0] = u.x; sn[1] = u.y; sn[2] = u.z; sn[3] = u.w;
    sn[4] = w.x; sn[5] = w.y; sn[6] = w.z; sn[7] = w.w;
  } else if (turns) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int pair = c * 8 + e;
      const int at = pair < p.section_end[0]   ? row[0]
                     : pair < p.section_end[1] ? row[1]
                     : pair < p.section_end[2] ? row[2]
                                               : row[3];
      cs[e] = p.rope[(long long)at * p.rot + pair];
      sn[e] = p.rope[(long long)at * p.rot + half + pair];
    }
  }

  const E* qs = static_cast<const E*>(p.q) + tok * p.q_row;
  const E* ks = static_cast<const E*>(p.k) + tok * p.k_row;
  const E* vs = static_cast<const E*>(p.v) + tok * p.v_row;
  E* qd = static_cast<E*>(p.q_out) + tok * p.q_out_row;
  E* kd = static_cast<E*>(p.c.k) + page * p.c.k_page + slot * p.c.k_token;
  E* vd = static_cast<E*>(p.c.v) + page * p.c.v_page + slot * p.c.v_token;
  const int nq = p.q ? p.hq : 0, nk = nq + p.c.hkv, rows = nk + p.c.hkv;
  const int step = warps_per_token * RPW;
  // all loads of a batch before its first store (which the compiler may not
  // move a later load across)
  for (int r0 = (warp % warps_per_token) * RPW + lane / LPR; r0 < rows;
       r0 += kBatch * step) {
    uint4 a[kBatch], b[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = r0 + i * step;
      if (r < rows) {
        const E* src = r < nq   ? qs + (long long)r * D
                       : r < nk ? ks + (long long)(r - nq) * D
                                : vs + (long long)(r - nk) * D;
        a[i] = *reinterpret_cast<const uint4*>(src + e0);
        b[i] = *reinterpret_cast<const uint4*>(src + e1);
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int r = r0 + i * step;
      if (r >= rows) break;
      if (turns && r < nk) {
        uint32_t* ua = reinterpret_cast<uint32_t*>(&a[i]);
        uint32_t* ub = reinterpret_cast<uint32_t*>(&b[i]);
        if (p.interleaved) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = unpack2(ua[e], E()), g = unpack2(ub[e], E());
            ua[e] = pack2<E>(f.x * cs[e] - f.y * sn[e], f.y * cs[e] + f.x * sn[e]);
            ub[e] = pack2<E>(g.x * cs[4 + e] - g.y * sn[4 + e],
                             g.y * cs[4 + e] + g.x * sn[4 + e]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = unpack2(ua[e], E()), g = unpack2(ub[e], E());
            ua[e] = pack2<E>(f.x * cs[2 * e] - g.x * sn[2 * e],
                             f.y * cs[2 * e + 1] - g.y * sn[2 * e + 1]);
            ub[e] = pack2<E>(g.x * cs[2 * e] + f.x * sn[2 * e],
                             g.y * cs[2 * e + 1] + f.y * sn[2 * e + 1]);
          }
        }
      }
      E* dst = r < nq   ? qd + (long long)r * D
               : r < nk ? kd + (r - nq) * p.c.k_head
                        : vd + (r - nk) * p.c.v_head;
      *reinterpret_cast<uint4*>(dst + e0) = a[i];
      *reinterpret_cast<uint4*>(dst + e1) = b[i];
    }
  }
}

template <typename E>
cudaError_t launch_elem(const PagedAppendParams& p, int d, cudaStream_t stream) {
  // Few tokens: the warps of a block share one, so that the heads move in
  // parallel (4 warps a token up to 512 tokens, 2 up to 1024). 4096 tokens of
  // 48 heads take 15.2 us with one warp each and 16.3 us with two, 256 tokens
  // 8.7 us with four.
  int wpt = kWarps;
  while (wpt > 1 && p.tokens * wpt > 2048) wpt /= 2;
  const int per = kWarps / wpt;
  const unsigned grid = (unsigned)((p.tokens + per - 1) / per);
  const int t = timing_start(GDN_KERNEL_PAGED_APPEND, stream);
  const cudaError_t e =
      paged_launch(d == 128 ? paged_append_kernel<E, 128>
                            : paged_append_kernel<E, 64>,
                   dim3(grid), kThreads, 0, stream, p, wpt);
  timing_stop(t, stream, e);
  return e;
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendParams& p, int d, bool bf16,
                                cudaStream_t stream) {
  return bf16 ? launch_elem<__nv_bfloat16>(p, d, stream)
              : launch_elem<__half>(p, d, stream);
}

}  // namespace gdn
