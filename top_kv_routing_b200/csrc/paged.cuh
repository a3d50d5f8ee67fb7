// Paged batches (host-side interfaces between paged.cu and its kernels, and the device
// helpers they share; not part of the ABI).
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "common.cuh"
#include "msa_paged.h"

namespace paged {

constexpr int kD = 128;
constexpr int kMaxSeqs = MSA_PAGED_MAX_SEQS;

// Arguments of one msa_shared_attend call, checked.
struct Attend {
  const __nv_bfloat16* q;          // [L][T][H*G][128]
  __nv_bfloat16* out;              // [L][T][H*G][128]
  const int32_t* q_offsets;        // [B + 1]
  const int32_t* seq_len;          // [B]
  const int32_t* group_offsets;    // [NG + 1]
  const __nv_bfloat16* mem_kv;     // [NG][L][2][H][M_max][128]
  const int32_t* mem_len;          // [NG][L]
  const __nv_bfloat16* pages;      // [L][NP][2][H][page][128]
  const int32_t* page_table;       // [B][max_pages]
  int T, B, NG, L, H, G, M_max, NP, log2_page, max_pages;
  float qscale;                    // softmax scale x log2(e)
  unsigned char* ws;
  int32_t* dev_err;
};

// ---- the row kernel (paged_rows.cu): 8 or 16 rows of one sequence per warp, mma.sync
constexpr int kRowWarps = 8;       // warps per CTA
constexpr int kRowCtas = 160;      // CTAs the workspace is laid out for (one per SM)
constexpr int kRowWorkers = kRowCtas * kRowWarps;

// Workspace: arrival counters (zero between calls, at the same place for every size), then
// two piece slots per worker.
constexpr size_t kWsCounters = 0;
constexpr size_t kWsSplits = kRowWorkers * sizeof(int32_t);  // key splits that the memory kernel chose
constexpr size_t kWsOrder = kWsSplits + 128;  // the sequences in the block form's order
constexpr size_t kWsStat = kWsOrder + kMaxSeqs * sizeof(int32_t);
constexpr size_t kWsPart = kWsStat + (size_t)2 * kRowWorkers * 16 * sizeof(float2);
constexpr size_t kWsEnd = kWsPart + (size_t)2 * kRowWorkers * 16 * kD * sizeof(float);

// memory_splits > 0: the memory part was computed by the memory kernel (with at most that many
// key splits), otherwise the row kernel walks the memory itself.
cudaError_t launch_rows(const Attend& a, int memory_splits, cudaStream_t s);

// ---- the memory kernel (paged_tc.cu): all rows of a group at once, tcgen05.  Its output, per
// partial slot and row (layer, token, query head): the unnormalised output (of every 16
// dims in the order 0 1 8 9, 2 3 10 11, 4 5 12 13, 6 7 14 15, the row kernel's), then (after all
// of them) the row's maximum (log2 domain) and sum.  A group of at most one row tile (128 / G
// tokens) has 2 x splits slots, others `splits`.
constexpr size_t kWsMemory = kWsEnd;
// Rows x splits are bounded by what two waves of one pair of row tiles per SM hold.
constexpr int64_t kSplitRows = 2 * 148 * 256;
constexpr int kMaxSplits = 64;
inline int memory_splits(int64_t rows) {
  return (int)(rows >= kSplitRows ? 1 : kSplitRows / rows < kMaxSplits ? kSplitRows / rows : kMaxSplits);
}
__host__ __device__ inline size_t memory_part_bytes(int64_t rows, int splits) {
  return (size_t)rows * 2 * splits * kD * sizeof(float);
}
inline size_t memory_bytes(int64_t rows, int splits) {
  return memory_part_bytes(rows, splits) + (size_t)rows * 2 * splits * sizeof(float2);
}
cudaError_t launch_memory(const Attend& a, int max_splits, cudaStream_t s);
// The same kernel's block form: memory and pages of long blocks of new tokens, the whole result.
cudaError_t launch_blocks(const Attend& a, cudaStream_t s);

// Lets a kernel use `bytes` of dynamic shared memory on the current device; `done` remembers the
// devices on which it may (the call costs a microsecond of every launch otherwise).
inline cudaError_t allow_shared_memory(const void* kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0ull;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// ---- device helpers

// 2^x by the hardware approximation (relative error about 2^-22, 2^-inf = 0).
__device__ __forceinline__ float ex2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Launched as a programmatic dependent: nothing an earlier kernel writes is read before this.
__device__ __forceinline__ void wait_for_earlier_kernels() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_kernel_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Asks L2 for the i-th 128 bytes of an array (no value is read, so it may run ahead of earlier
// kernels).
__device__ __forceinline__ void prefetch_line(const void* p, int64_t bytes, int64_t i) {
  if (i * 128 < bytes) asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(p) + i * 128));
}

// The tokens [lo, lo + n) of sequence b; n = 0 and false where the offsets are unusable.
__device__ __forceinline__ bool sequence_tokens(const int32_t* __restrict__ off, int b, int T, int& lo, int& n) {
  lo = off[b];
  const int hi = off[b + 1];
  const bool ok = lo >= 0 && hi >= lo && hi <= T;
  n = ok ? hi - lo : 0;
  return ok;
}

// The packed tokens [lo, lo + n) of group g (whose offsets are usable); false where the
// sequences' offsets are not.
__device__ __forceinline__ bool group_tokens(const Attend& a, int g, int& lo, int& n) {
  lo = a.q_offsets[a.group_offsets[g]];
  const int hi = a.q_offsets[a.group_offsets[g + 1]];
  const bool ok = lo >= 0 && hi >= lo && hi <= a.T;
  n = ok ? hi - lo : 0;
  return ok;
}

// The last b in [0, B) with off[b] <= t, by a 32-way search over the (non-decreasing) offsets
// (the sequence of token t, the group of sequence t); -1 when off[0] > t.  Always in [-1, B),
// whatever the offsets hold.
__device__ __forceinline__ int find_last(const int32_t* __restrict__ off, int B, int t, int lane) {
  int lo = 0, n = B;
  bool any = false;
  while (true) {
    const int step = (n + 31) >> 5;
    const int idx = lo + lane * step;
    const bool le = idx < lo + n && off[idx] <= t;
    const unsigned m = __ballot_sync(0xffffffffu, le);
    if (m == 0u) return any ? lo : -1;  // (later rounds: off[lo] <= t was seen, so m != 0)
    const int c = 31 - __clz(m);
    any = true;
    n = min(step, lo + n - (lo + c * step));
    lo += c * step;
    if (step == 1) return lo;
  }
}

// The sequence of token t, whose tokens are then [lo, lo + n), -1 for none (the lanes of a warp
// together): by the search above, and one after the other where that finds none, since an unusable
// offset may have misled it (the last usable sequence that holds t).
__device__ __forceinline__ int sequence_of(const int32_t* __restrict__ off, int B, int T, int t, int lane, int& lo,
                                           int& n) {
  const int b = find_last(off, B, t, lane);
  if (b >= 0 && sequence_tokens(off, b, T, lo, n) && t < lo + n) return b;  // (lo <= t by the search)
  int found = -1;
  for (int b0 = 0; b0 < B; b0 += 32) {
    int first, count;
    const bool holds = b0 + lane < B && sequence_tokens(off, b0 + lane, T, first, count) && t >= first && t < first + count;
    const unsigned m = __ballot_sync(0xffffffffu, holds);
    if (m) found = b0 + 31 - __clz(m);
  }
  if (found >= 0) sequence_tokens(off, found, T, lo, n);
  return found;
}

// Whether group g's offsets are usable.
__device__ __forceinline__ bool group_usable(const Attend& a, int g) {
  const int s = a.group_offsets[g], e = a.group_offsets[g + 1];
  return s >= 0 && e >= s && e <= a.B;
}

// The last usable group that holds sequence b, -1 for none (the lanes of a warp together).  Apart
// from the kernels' code: only unusable offsets lead here.
static __device__ __noinline__ int last_group_of(const Attend& a, int b, int lane) {
  int found = -1;
  for (int g0 = 0; g0 < a.NG; g0 += 32) {
    const int g = g0 + lane;
    const bool holds = g < a.NG && group_usable(a, g) && a.group_offsets[g] <= b && b < a.group_offsets[g + 1];
    const unsigned m = __ballot_sync(0xffffffffu, holds);
    if (m) found = g0 + 31 - __clz(m);
  }
  return found;
}

}  // namespace paged
