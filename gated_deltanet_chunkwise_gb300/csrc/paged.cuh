// Shared by the paged key/value cache kernels: the cache as kernels see it,
// the per-sequence lengths, and small helpers for 16-bit elements.
//
// Places. Sequence n holds kv_lens[n] keys, its new tokens the last ones: new
// token i stands at place x = kv_lens[n] - new_n + i, in page page_table[n]
// [x / page_size], row x % page_size. A place below zero (more new tokens
// than keys) sees nothing.
#pragma once

#include <atomic>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gdn_internal.cuh"
#include "tc_ptx.cuh"

namespace gdn {

// A 16-bit paged cache after host validation (strides in elements).
struct PagedView {
  void* k;
  void* v;
  long long k_page, k_head, k_token;
  long long v_page, v_head, v_token;
  const int32_t* table;  // [N, max_pages], rows table_stride apart
  long long table_stride;
  const int32_t* kv_lens;  // [N]
  int num_pages, page_shift, max_pages, hkv;
};

struct PagedAppendParams {
  PagedView c;
  const void* q;      // [tokens, hq, D], rows q_row elements apart; may be null
  const void* k;
  const void* v;
  void* q_out;
  long long q_row, k_row, v_row, q_out_row;
  const float* rope;  // [rope_rows, rot]: cosines, then sines
  const int32_t* positions;  // [axes, tokens] or null (the places themselves)
  int rope_rows, rot, axes, interleaved;
  int section_end[4];  // first rotated pair past each axis
  const int32_t* cu;
  long long tokens;
  int N, T, hq;
  int* status;
};

struct PagedAttnParams {
  PagedView c;
  const void* q;
  long long q_row;
  void* out;         // [tokens, hq, D] contiguous
  float* lse;        // [tokens, hq] or null
  const int32_t* cu;
  int N, T, hq, group;
  int causal, window;
  float scale_log2;  // scale * log2(e)
  // The few-row kernel serves sequences of up to rows_max rows, the tile
  // kernel those of more than rows_min.
  long long rows_min, rows_max;
  int split;  // the few-row kernel's CTAs per item; 0: the list is cut evenly
  // cut items: run i has two pieces of `rows` rows, 2 i (an item begun by an
  // earlier run) and 2 i + 1 (an item that a later run ends)
  float* part_o;   // [pieces, rows, D] unnormalised outputs
  float* part_ml;  // [pieces, rows, 2] reference maxima (log2) and sums
  int4* meta;      // [runs][2] of the item begun in the run and cut: sequence,
                   // key head, row block, last run that holds some of it
                   // (sequence -1: none); the sequence's first token, new
                   // tokens and keys
  int* status;
};

// New tokens [q0, q0 + len) of a sequence and its keys; ok false (recorded)
// when the lengths are inconsistent with the batch or the page table, ordered
// false when it is the batch's offsets that decrease or leave it.
struct PagedSeq {
  int q0, len, kv;
  bool ok, ordered;
};

// Offsets of a packed batch that do not decrease and stay inside of it: checked
// pair by pair. (Both attention kernels look at all pairs and write nothing if
// one is wrong: how sequences that overlap share rows has no answer.)
__device__ __forceinline__ bool ordered_pair(int b, int e, int T) {
  return b >= 0 && e >= b && e <= T;
}

__device__ __forceinline__ PagedSeq paged_seq(const PagedView& c,
                                              const int32_t* cu, int T, int n,
                                              int* status) {
  PagedSeq s;
  s.kv = c.kv_lens[n];
  s.ok = s.ordered = true;
  if (cu) {
    const int b = cu[n], e = cu[n + 1];
    s.q0 = b;
    s.len = e - b;
    s.ok = s.ordered = ordered_pair(b, e, T);
  } else {
    s.q0 = n * T;
    s.len = T;
  }
  if (s.kv < 0 || (long long)s.kv > ((long long)c.max_pages << c.page_shift))
    s.ok = false;
  if (!s.ok) {
    record_status(status, GDN_ERR_INVALID_ARG);
    s.len = 0;
    s.kv = 0;
  }
  return s;
}

// ---- 16-bit element types ----------------------------------------------------
__device__ __forceinline__ float2 unpack2(uint32_t u, __nv_bfloat16) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
}
__device__ __forceinline__ float2 unpack2(uint32_t u, __half) {
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kNegInf = -INFINITY;
// The reference maximum moves only when a score passes it by more than this
// (in powers of two): weights stay below 2^8, exact in fp32 sums and with
// the same relative rounding as 16-bit factors, and the accumulators are
// rarely rescaled.
constexpr float kSlack = 8.f;
// The reference stands this far (in powers of two) below the maximum that it
// was taken from. bf16 weights have fp32's range; fp16's normal ones end at
// 2^-14 and their last at 2^-25, so a weight of 1 for the largest score would
// round the many small ones of a long cache behind one dominant key away or up
// (an attention sink, the others 17 below it in natural logarithms, 100000 keys:
// their part of the output is off by a quarter), while the sum takes them as they
// are. With 2^7 for the largest score weights stay below 2^15, inside the type,
// and reach down to 2^-32 of it.
template <typename E>
constexpr float kLift = 0.f;
template <>
constexpr float kLift<__half> = 7.f;
// From here on a score's product with the scale is rounded before the reference
// is taken off it, as the reference was: the two differ by up to half a unit of
// the last place otherwise, which 2^ of turns into infinity where scores pass
// 2^31 (fp16: 2^25). (In the tile kernel such a run is made a second time.)
constexpr float kFar = 1048576.f;
// What weights relative to `was` are multiplied by to be relative to `now`.
// With no score above -inf yet the reference is 0: the sums are 0 then, or
// NaN if a score was NaN, which stays one.
__device__ __forceinline__ float factor(float was, float now) {
  return now == kNegInf ? 1.f : ex2(was - now);
}
// Natural log of the sum of a row's exponentials; -inf for a row that sees
// nothing (l = 0).
__device__ __forceinline__ float row_lse(float top, float l) {
  if (l == 0.f) return kNegInf;
  return ((top == kNegInf ? 0.f : top) + log2f(l)) * 0.69314718055994531f;
}

// A TMA copy from a four-dimensional tensor.
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map,
                                            uint64_t* bar, int x, int y, int z,
                                            int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::"
      "bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(tc::smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(tc::smem_u32(bar))
      : "memory");
}

// Waits for the phase with the given parity, at first without reading the
// timer that bounds the wait: a read of it takes longer than most waits here,
// and the thread that polls is on the critical path of a whole tile.
__device__ __forceinline__ bool fast_wait(uint64_t* bar, uint32_t parity,
                                          volatile int* abort_flag) {
#pragma unroll 1
  for (int i = 0; i < 32; ++i)
    if (tc::mbar_try_wait(bar, parity)) return true;
  return tc::mbar_wait(bar, parity, abort_flag);
}

// A wait by a whole warp, with one answer for all of it: lanes that gave up
// and lanes that did not would meet at different warp-wide instructions.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity,
                                          volatile int* abort_flag) {
  return __all_sync(0xffffffffu, fast_wait(bar, parity, abort_flag));
}

// After a wait gave up: time for copies in flight to land before the CTA's
// shared memory is given back (2 ms, thousands of memory round trips).
__device__ __forceinline__ void wait_out_copies() {
  const uint64_t t0 = tc::globaltimer_ns();
  for (int i = 0; i < 1000000 && tc::globaltimer_ns() - t0 < 2000000ull; ++i) {
  }
}

// Hidden values. The products that the kernels make of whole tiles multiply the
// values of keys that a row does not see by a weight of 0, which an infinity or
// a NaN among them survives. A CTA that finds a result which is not finite in a
// row that does not see all that was multiplied makes its run once more, with a
// look through the tiles that some row sees in part: if one holds such a value,
// its weights are multiplied key by key, each row's with the keys that it sees
// and no others. So ordinary calls pay for a look at their results only; one
// hidden infinity makes 2048 tokens over 65536 keys take 2.4 ms instead of 0.7,
// and the cost of a tile made key by key does not grow with the cache.

// 1 if any of the values is infinite or NaN.
__device__ __forceinline__ uint32_t nonfinite(const float (&x)[32]) {
  float z[2] = {};
#pragma unroll
  for (int i = 0; i < 32; ++i) z[i & 1] = fmaf(x[i], 0.f, z[i & 1]);
  return z[0] + z[1] == 0.f ? 0u : 1u;
}

// (0, 0), of either sign, as long as all the elements seen are finite.
__device__ __forceinline__ uint32_t probe2(uint32_t u, uint32_t acc, __nv_bfloat16) {
  const __nv_bfloat162 z = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&u),
                                   __floats2bfloat162_rn(0.f, 0.f),
                                   *reinterpret_cast<const __nv_bfloat162*>(&acc));
  return *reinterpret_cast<const uint32_t*>(&z);
}
__device__ __forceinline__ uint32_t probe2(uint32_t u, uint32_t acc, __half) {
  const __half2 z = __hfma2(*reinterpret_cast<const __half2*>(&u),
                            __floats2half2_rn(0.f, 0.f),
                            *reinterpret_cast<const __half2*>(&acc));
  return *reinterpret_cast<const uint32_t*>(&z);
}
template <typename E>
__device__ __forceinline__ uint32_t probe8(uint4 v, uint32_t acc) {
  return probe2(v.w, probe2(v.z, probe2(v.y, probe2(v.x, acc, E()), E()), E()),
                E());
}
__device__ __forceinline__ bool probe_hit(uint32_t acc) {
  return (acc & 0x7fff7fffu) != 0;
}

// ---- host side ------------------------------------------------------------------
cudaError_t launch_paged_append(const PagedAppendParams& p, int d, bool bf16,
                                cudaStream_t stream);
// Tensor map of a 16-bit tensor, dims (d, n1, n2, n3) with the strides in
// elements, boxes of (64, b1, b2, 1) with the 128-byte swizzle.
bool make_paged_map(CUtensorMap* map, const void* ptr, bool bf16, int d,
                    long long n1, long long n2, long long n3, long long s1,
                    long long s2, long long s3, int b1, int b2);
int paged_sm_count();
// Current device, or -1.
int paged_device();
// Stream-ordered workspace (released with cudaFreeAsync) from a pool of the
// library's own that keeps its memory: the device's default pool returns it
// at every synchronisation, and a call after one then takes 250 us.
cudaError_t paged_workspace(void** ws, size_t bytes, cudaStream_t stream);
// A launch whose blocks may take their places before the stream's last kernel
// has ended; the kernel waits for it (griddep_wait) before it reads or writes
// anything global. The first in clusters of `cluster` blocks.
template <typename... P, typename... A>
cudaError_t paged_launch_clusters(void (*kernel)(P...), int cluster, dim3 grid,
                                  int threads, int smem, cudaStream_t stream,
                                  A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}
template <typename... P, typename... A>
cudaError_t paged_launch(void (*kernel)(P...), dim3 grid, int threads, int smem,
                         cudaStream_t stream, A... args) {
  return paged_launch_clusters(kernel, 1, grid, threads, smem, stream, args...);
}
// Opts a kernel in to `bytes` of shared memory, once per device.
template <typename K>
cudaError_t paged_allow_smem(K kernel, int bytes, std::atomic<unsigned long long>& done) {
  const int dev = paged_device();
  if (dev < 0) return cudaErrorInvalidDevice;
  const unsigned long long bit = 1ull << dev;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(
      kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit);
  return e;
}
// The kernel for few query rows per key head (paged_rows.cu); key and value
// maps have boxes of paged_rows_box tokens.
int paged_rows_box(int page_size);
// CTAs per item where it needs neither workspace nor a launch to join pieces,
// else 0.
int paged_rows_split(const PagedAttnParams& p);
size_t paged_rows_workspace_bytes(int d);
void paged_rows_bind_workspace(PagedAttnParams& p, void* ws, int d);
cudaError_t launch_paged_rows(const PagedAttnParams& p, int d, bool bf16,
                              const CUtensorMap& tk, const CUtensorMap& tv,
                              cudaStream_t stream, int* launches);
// The tensor-core kernel for many rows (paged_tiles.cu); the query map has
// boxes of (64, group, 128 / group).
int paged_tiles_box(int page_size);
size_t paged_tiles_workspace_bytes(const PagedAttnParams& p, int d);
void paged_tiles_bind_workspace(PagedAttnParams& p, void* ws, int d);
cudaError_t launch_paged_tiles(const PagedAttnParams& p, int d, bool bf16,
                               const CUtensorMap& tq, const CUtensorMap& tk,
                               const CUtensorMap& tv, cudaStream_t stream,
                               int* launches);
// Joins the pieces of the items that `runs` runs cut (paged_merge.cu).
cudaError_t launch_paged_merge(const PagedAttnParams& p, int d, bool bf16,
                               int runs, int rows, cudaStream_t stream,
                               int* launches);

}  // namespace gdn
