// Shared-memory attention of a paged batch on the tcgen05 tensor cores, 256 rows a CTA, in two
// forms (msa_paged.h defines the result):
//   memory form  the packed tokens of a group (all of its sequences' new tokens) x the G query
//                heads of key head h are the MMA's rows, so every tile of the group's memory is
//                read once per 256 rows whatever the number of sequences.  (Where offsets are
//                unusable, the tokens of each sequence by themselves.)  A unit is (group,
//                layer, key head, pair of row tiles, key split); its result per row and split,
//                the unnormalised fp32 output, its maximum and its sum, is joined with the
//                sequence's own pages by the row kernel (paged_rows.cu).
//   block form   for long blocks of new tokens: a unit is (sequence, layer, key head, pair of
//                row tiles of its tokens) over the memory and then the sequence's pages, causal,
//                and writes the output itself.
//
// Follows "MSA端到端可训练记忆模型完整开源，支持亿级Token上下文", section 架构 (softmax over the
// selected memory joined to the local K/V), and the MSA paper reading notes, section
// 推理全流程.
//
// Persistent CTAs (one per SM) of 384 threads walk the units:
//   warp 9               TMA: 128-key tiles of K and V in the order the MMAs use them, through a
//                        ring of 32 KB slots (memory tiles as 64-row boxes, page tiles as one
//                        box per page, a lane each);
//   warp 8, one thread   MMA issue for two streams a and b: S = Q K^T (queries from shared
//                        memory, M = N = 128), O += P V (weights from tensor memory, written
//                        over their scores; V read MN-major from its rows).  PV_a(j), S_a(j+1),
//                        PV_b(j), S_b(j+1), ...: while one stream's softmax runs, the tensor
//                        cores work for the other.  A PV starts on the weights of the first 64
//                        keys while the softmax computes those of the others.  Each pair of PV
//                        and S is one command word, so that little but the MMAs themselves is
//                        left to the thread (working them out itself took it as long again);
//   warp 10              writes the commands as the tiles land, and prepares value tiles before
//                        their PV: rows past the last valid one, which may hold anything, are
//                        zeroed, and values that are not finite taken out where some rows must
//                        not see them;
//   warp 11              works out the units ahead of everyone else (a ring of kUnits), and loads
//                        their query rows (4D boxes);
//   warps 0..3, 4..7     the softmax of stream a and of stream b: a thread per row, with the
//                        registers that warps 8..11 give up.  A running maximum that is raised
//                        (and O rescaled in tensor memory) only when a score exceeds it by more
//                        than 2^8; weights exp2(s - m) rounded to bf16 (the MMA's operand type;
//                        the row sum takes them unrounded).
// Streams a and b are the two row tiles of the pair over the same keys.  A group of at most
// one row tile gives both streams the same rows and each half of the unit's keys instead.
//
// S_x(j + 1) is issued after PV_x(j), so its completion also says that O_x is stable: the
// softmax rescales it without another wait.  Key rows past the last valid one are zeroed in
// shared memory before the PV that reads them (they may hold anything).  Every wait is
// bounded (2 s, and 60 s where a wait may last a whole unit); a timeout sets MSA_DEVERR_TIMEOUT and
// the CTA drains and frees its TMEM.
//
// Measured on one B200: 256 rows x 8 key heads x 16,384 keys of a wide batch (137 GFLOP) in 140 us,
// the tensor pipe 63 % active, 128 units on 148 SMs; a tile pair takes 3,100 cycles against 2,048
// of MMA, because a stream's softmax (1,024 cycles of exponentials on the MUFU alone), its PV and
// its next scores follow one another and two outputs leave tensor memory no second score buffer.
// Short units wait for instruction fetch: the softmax has one body and the other roles loops.
#include <cuda.h>

#include <algorithm>

#include "paged.cuh"
#include "tc_common.cuh"

namespace paged {
namespace {
using namespace tc;

constexpr int kRows = 128;
constexpr int kTile = 128;                // keys of a tile
constexpr int kBox = 64;                  // keys of a TMA box
constexpr int kHalf = 64;                 // dims of a 128-byte swizzled row
constexpr int kHalfBytes = kTile * 128;   // 16 KB: 128 rows x 64 dims
constexpr int kSlotBytes = 2 * kHalfBytes;  // one K or V tile, or one query tile
constexpr int kSlots = 5;
constexpr int kCommands = 16;             // (10 at most wait: two a tile of the ring)
constexpr int kUnits = 4;                 // units worked out ahead
constexpr int kWarpsTc = 12;              // 0..7 softmax, 8 MMA, 9 TMA, 10 value tiles, 11 units
constexpr int kThreadsTc = kWarpsTc * 32;
// registers: 168 a thread at launch; 128 x 72 + 256 x 216 = 384 x 168
constexpr int kRegsIssue = 72, kRegsSoftmax = 216;
static_assert(128 * kRegsIssue + 256 * kRegsSoftmax <= kThreadsTc * 168, "register split");
constexpr int kMmaWarp = 8, kTmaWarp = 9, kValueWarp = 10;
constexpr uint32_t kTmemCols = 512;       // S_a | S_b | O_a | O_b
constexpr uint32_t kColS = 0, kColO = 256;
constexpr float kHeadroom = 8.0f;         // log2 growth of a row's maximum tolerated before rescaling

constexpr unsigned long long kUnitWaitNs = 60000000000ull;  // (a failure within a unit is noticed by a shorter wait)
constexpr int kOrdered = 512;             // most sequences that are put in order
constexpr int kBadRing = 8;               // tiles whose page masks are kept (more than are in flight)

// One unit as every role sees it.
struct Unit {
  int e, l, h;               // entry, layer, key head
  int tok[2], n_tok[2];      // each stream's tokens
  int t0[2], t1[2];          // each stream's key tiles [t0, t1)
  int M, mt;                 // memory rows and tiles (the page tiles follow)
  int n_loc;                 // page rows that some row sees
  int lim0;                  // page rows that the first token sees (token i: i more, up to len)
  int len;                   // page rows (clamped)
  bool shared;               // the streams read the same key tiles
  int64_t kv_row;            // row of key 0 in the memory tensor; values H * M_max further
  int slot[2];               // partial slot
  int poison;                // block form: values that are not finite were taken out of its tiles
};

// Shared variables.  An entry is a group (memory form as a rule) or a sequence.
constexpr int kBlocks = kMaxSeqs / 32;
static_assert(kBlocks <= 32, "a lane per block of entries");
struct TablesTc {
  int scan[kBlocks + 1];   // row-tile pairs of the entries before each 32
  int most;                // memory form: most key tiles of any (group, layer)
  int splits;
  uint32_t tmem;
  int abort;
  uint32_t commands[kCommands];
  Unit units[kUnits];      // unit u of this CTA in place u % kUnits
  uint32_t bad[kBadRing];  // block form: per tile, its 16-row pieces without a usable page
};

// A command of the MMA thread: for stream `kStreamB`, O += P V over a value tile and then the
// scores over a key tile (either may be missing).
enum : uint32_t {
  kStreamB = 1u,
  kWeigh = 2u,        // PV: 16-key steps in bits 12..15, ring slot in bits 16..18
  kFirst = 4u,        // the unit's first PV of the stream (O starts from it)
  kFreeV = 8u,        // the tile's last use
  kOutput = 16u,      // O is complete
  kScore = 32u,       // scores: ring slot in bits 20..22
  kAwaitQ = 64u,      // the unit's first scores of the stream: its queries have to land
  kFreeK = 128u,      // the tile's last use
  kFreeQ = 256u,      // the queries' last use
  kEnd = 512u,
};

constexpr int kOffQ = 0;
constexpr int kOffRing = 2 * kSlotBytes;
constexpr int kOffBars = kOffRing + kSlots * kSlotBytes;
constexpr int kOffTables = kOffBars + 384;
constexpr int kSmemTc = kOffTables + (int)sizeof(TablesTc) + 1024;  // (+ alignment of the dynamic base)
static_assert(kSmemTc <= 227 * 1024, "shared memory");

__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// D (TMEM) += A (TMEM, K-major, 2 bf16 per column) x B (shared-memory descriptor).
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 4D tiled TMA load (no multicast): [128 / G tokens][G heads][64 dims] of one layer's queries.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z,
                                            int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
      "[%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}
__device__ __forceinline__ void tma_prefetch_4d(const CUtensorMap* map, int x, int y, int z, int w) {
  asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}
__device__ __forceinline__ void tma_load_rows(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}

// 32 bytes, in one store where the buffer they belong to starts at a multiple of 32 (all offsets
// within it are), in two where it keeps only the 16 bytes that `out` and the workspace have to.
// The wide stores take 298 us over the 18 layers of 8 questions, the others 318.
__device__ __forceinline__ void st_global_32(void* p, bool wide, const uint32_t (&x)[8]) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x[0]), "r"(x[1]),
                 "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
  } else {
    uint4* dst = static_cast<uint4*>(p);
    dst[0] = make_uint4(x[0], x[1], x[2], x[3]);
    dst[1] = make_uint4(x[4], x[5], x[6], x[7]);
  }
}

// Packed pairs of fp32 (two registers).
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// the largest of three, NaN if any is
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The first page row of the 16-row pieces that some row of the pair does not see in full: from
// there on values that are not finite are taken out of the tiles.
__device__ __forceinline__ int first_partial(const Unit& x) { return max(0, x.lim0) & ~15; }

// Adds the values that were taken out, as far as this row sees them, to its stored output.
__device__ __noinline__ void add_not_finite(const Attend& a, const Unit& x, int seen, __nv_bfloat16* out) {
  const int page = 1 << a.log2_page;
  for (int k = first_partial(x); k < seen; ++k) {
    const int id = a.page_table[(int64_t)x.e * a.max_pages + (k >> a.log2_page)];
    if (id < 0 || id >= a.NP) continue;
    const int64_t row = ((((((int64_t)x.l * a.NP + id) * 2 + 1) * a.H + x.h)) << a.log2_page) + (k & (page - 1));
    for (int e = 0; e < kD; ++e) {
      const float v = __bfloat162float(a.pages[row * kD + e]);
      if (!(fabsf(v) < INFINITY)) out[e] = __float2bfloat16(__bfloat162float(out[e]) + v);
    }
  }
}

template <int G, bool BLOCK>
__global__ void __launch_bounds__(kThreadsTc, 1)
    tile_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kv,
                const __grid_constant__ CUtensorMap tm_pages, const __grid_constant__ Attend a, int max_splits) {
  constexpr int kTok = kRows / G;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  TablesTc& tb = *reinterpret_cast<TablesTc*>(smem + kOffTables);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBars);
  uint64_t* full = bars;                 // [kSlots] tile landed
  uint64_t* empty = bars + kSlots;       // [kSlots] tile read by its MMAs and passed by warp 10
  uint64_t* q_full = bars + 2 * kSlots;  // [2] the stream's queries landed
  uint64_t* q_empty = q_full + 2;        // [2] read by the stream's last score MMA of the unit
  uint64_t* s_ready = q_empty + 2;       // [2] scores in tensor memory (and the stream's PV before them done)
  uint64_t* p_ready = s_ready + 2;       // [2][2] weights of keys 0..63, 64..127 in tensor memory (4 warps)
  uint64_t* o_done = p_ready + 4;        // [2] the stream's last PV of the unit done
  uint64_t* c_full = o_done + 2;         // [kCommands] command written
  uint64_t* u_full = c_full + kCommands; // [kUnits] unit worked out
  uint64_t* u_empty = u_full + kUnits;   // [kUnits] not needed any more (TMA, commands, 8 softmax warps)
  uint64_t* drain = u_empty + kUnits;
  volatile int* abort_flag = &tb.abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sbase = smem_u32(smem);
  const int Hq = a.H * G, LH = a.L * a.H;

  if (tid == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 2);
    }
    for (int s = 0; s < kCommands; ++s) mbar_init(smem_u32(&c_full[s]), 1);
    for (int s = 0; s < kUnits; ++s) {
      mbar_init(smem_u32(&u_full[s]), 1);
      mbar_init(smem_u32(&u_empty[s]), 10);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(smem_u32(&q_full[x]), 1);
      mbar_init(smem_u32(&q_empty[x]), 1);
      mbar_init(smem_u32(&s_ready[x]), 1);
      mbar_init(smem_u32(&p_ready[2 * x]), 4);
      mbar_init(smem_u32(&p_ready[2 * x + 1]), 4);
      mbar_init(smem_u32(&o_done[x]), 1);
    }
    mbar_init(smem_u32(drain), 1);
    tb.abort = 0;
    tb.most = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async_smem();
  }
  if (warp == kMmaWarp) {
    tmem_alloc<false>(smem_u32(&tb.tmem), kTmemCols);
    tmem_relinquish<false>();
  }
  __syncthreads();  // (the shared variables are zeroed)
  wait_for_earlier_kernels();
  let_next_kernel_start();

  // ---- the batch: row-tile pairs, most key tiles
  // (memory form: by group as a rule, by sequence where offsets are unusable: groups may overlap then,
  // and a group's first and last offset may be the unusable ones)
  bool by_sequence = BLOCK;
  const int64_t cap = (int64_t)a.max_pages << a.log2_page;
  // what the batch needs is asked for at once: memory lengths, offsets of groups, tokens
  const bool check = !BLOCK && tid < a.B;
  const int lo_first = check ? a.q_offsets[tid] : 0, hi_first = check ? a.q_offsets[tid + 1] : 0;
  int most = 0;
  for (int i = tid; i < a.NG * a.L; i += kThreadsTc) most = max(most, a.mem_len[i]);
  bool ok_here = true;  // the group offsets are usable (memory form: and the sequences')
  for (int g = tid; g < a.NG; g += kThreadsTc) {
    const int s = a.group_offsets[g], e = a.group_offsets[g + 1];
    ok_here &= s >= 0 && e >= s && e <= a.B;
  }
  ok_here &= lo_first >= 0 && hi_first >= lo_first && hi_first <= a.T;
  for (int b = tid + kThreadsTc; b < a.B && !BLOCK; b += kThreadsTc) {
    int lo, n;
    ok_here &= sequence_tokens(a.q_offsets, b, a.T, lo, n);
  }
  auto pairs_of = [](int n) -> int { return (n + 2 * kTok - 1) / (2 * kTok); };
  int32_t* order = reinterpret_cast<int32_t*>(a.ws + kWsOrder);  // (every CTA writes the same)
  if (BLOCK) {
    // the sequences by their keys, the most first (in the place of the tiles, not needed yet);
    // beyond kOrdered of them the comparisons would cost more than the order gives
    int* size = reinterpret_cast<int*>(smem + kOffRing);
    for (int e = tid; e < a.B; e += kThreadsTc) {
      const int len = a.seq_len[e];
      int lo, n, from = 0, to = a.NG;  // the group: from <= it < to (whatever the offsets hold)
      if (!sequence_tokens(a.q_offsets, e, a.T, lo, n) && blockIdx.x == 0)
        msa::set_err(a.dev_err, MSA_DEVERR_BAD_OFFSETS);
      if (blockIdx.x == 0 && n > 0 && len > cap) msa::set_err(a.dev_err, MSA_DEVERR_LOCAL_FULL);
      while (to - from > 1) {
        const int mid = (from + to) >> 1;
        if (a.group_offsets[mid] <= e) from = mid; else to = mid;
      }
      int keys = (int)min((int64_t)max(len, 0), cap) / kTile;
      if (a.NG > 0 && a.group_offsets[from] <= e && e < a.group_offsets[from + 1])
        keys += max(0, min(a.M_max, a.mem_len[(int64_t)from * a.L])) / kTile;
      size[e] = n > 0 ? keys : -1;
    }
    __syncthreads();
    for (int e = tid; e < a.B; e += kThreadsTc) {
      const int own = size[e];
      int rank = a.B > kOrdered ? e : 0;
      for (int f = 0; f < a.B && a.B <= kOrdered; ++f) rank += size[f] > own || (size[f] == own && f < e);
      order[rank] = e;
    }
    fence_async_smem();  // (the tiles come through the async proxy)
    __syncthreads();
  }
  // tokens of entry e (block form: the e-th sequence in order); none where they are unusable
  auto entry_tokens = [&](int e, int& lo, int& n) {
    lo = n = 0;
    if (by_sequence)
      sequence_tokens(a.q_offsets, BLOCK ? order[e] : e, a.T, lo, n);
    else if (group_usable(a, e))
      group_tokens(a, e, lo, n);
  };
  int n_entries, n_blocks;
  auto count_pairs = [&]() {
    n_entries = by_sequence ? a.B : a.NG;
    n_blocks = (n_entries + 31) / 32;
    for (int k = warp; k < n_blocks; k += kWarpsTc) {
      const int e = 32 * k + lane;
      int lo = 0, n = 0;
      if (e < n_entries) entry_tokens(e, lo, n);
      const int sum = __reduce_add_sync(0xffffffffu, pairs_of(n));
      if (lane == 0) tb.scan[k] = sum;
    }
  };
  count_pairs();
  if (most > a.M_max) {
    if (blockIdx.x == 0) msa::set_err(a.dev_err, MSA_DEVERR_CAPACITY);
    most = a.M_max;
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0) atomicMax(&tb.most, (most + kTile - 1) / kTile);
  tc_fence_before();
  const bool offsets_ok = __syncthreads_and(ok_here);
  tc_fence_after();
  if (!offsets_ok && blockIdx.x == 0 && tid == 0) msa::set_err(a.dev_err, MSA_DEVERR_BAD_OFFSETS);
  if (!BLOCK && !offsets_ok) {
    by_sequence = true;
    count_pairs();
    __syncthreads();
  }
  if (warp == 0) {  // sums before each block, and the split
    const int v = lane < n_blocks ? tb.scan[lane] : 0;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    tb.scan[lane] = inc - v;
    if (lane == 31) tb.scan[32] = inc;
    int best = 1;
    if (!BLOCK) {
      // the split that finishes first, a unit costing its tiles and about two more: a lane for
      // every 32nd number of splits
      const int64_t units = (int64_t)__shfl_sync(0xffffffffu, inc, 31) * LH;
      const uint32_t most_tiles = max(1, tb.most);
      float cost = INFINITY;
      for (int s = lane + 1; s <= max_splits && s <= (int)most_tiles; s += 32) {
        const float waves = ceilf((float)(units * s) / (float)gridDim.x);
        const float c = waves * (float)((most_tiles + s - 1) / s + 2);
        if (c < cost) {
          cost = c;
          best = s;
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float c = __shfl_xor_sync(0xffffffffu, cost, o);
        const int b = __shfl_xor_sync(0xffffffffu, best, o);
        if (c < cost || (c == cost && b < best)) {
          cost = c;
          best = b;
        }
      }
      if (lane == 0 && blockIdx.x == 0) *reinterpret_cast<int*>(a.ws + kWsSplits) = best;
    }
    if (lane == 0) tb.splits = best;
  }
  __syncthreads();
  const int pairs = tb.scan[kBlocks];
  const int splits = tb.splits;
  const uint32_t tmem_base = tb.tmem;
  const int64_t n_units = (int64_t)pairs * LH * splits;

  // Unit un of this CTA: in the block form every other round over the CTAs goes backwards, so that
  // units which get smaller along the line even out.
  auto unit_number = [&](int un) -> int64_t {
    return (int64_t)un * gridDim.x + (BLOCK && (un & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
  };
  // the unit (the lanes of one warp together)
  auto unit_at = [&](int64_t u) -> Unit {
    Unit x;
    // memory form: pairs run fastest (CTAs at work together read the same keys); block form:
    // (layer, key head) runs fastest, then the pairs of a sequence
    const int64_t rest = BLOCK ? u / LH : u / pairs;
    const int pair = BLOCK ? (int)rest : (int)(u - rest * pairs);
    const int s = BLOCK ? 0 : (int)(rest % splits);
    const int lh = BLOCK ? (int)(u - rest * LH) : (int)(rest / splits);
    x.l = lh / a.H;
    x.h = lh - x.l * a.H;
    // the entry: its block of 32, then a scan over the block
    const int k = 31 - __clz(__ballot_sync(0xffffffffu, lane < n_blocks && tb.scan[lane] <= pair));
    const int e = 32 * k + lane;
    int lo = 0, n = 0;
    if (e < n_entries) entry_tokens(e, lo, n);
    int before = pairs_of(n);
    const int own_pairs = before;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += y;
    }
    before += tb.scan[k] - own_pairs;
    const int from = 31 - __clz(__ballot_sync(0xffffffffu, e < n_entries && before <= pair));
    x.e = BLOCK ? order[32 * k + from] : 32 * k + from;
    lo = __shfl_sync(0xffffffffu, lo, from);
    n = __shfl_sync(0xffffffffu, n, from);
    const int at = (pair - __shfl_sync(0xffffffffu, before, from)) * 2 * kTok;
    int g = x.e;
    if (by_sequence && offsets_ok) {
      g = a.NG > 0 ? find_last(a.group_offsets, a.NG, x.e, lane) : -1;
      if (g >= 0 && x.e >= a.group_offsets[g + 1]) g = -1;
    } else if (by_sequence) {
      g = last_group_of(a, x.e, lane);
    }
    const int64_t gl = (int64_t)g * a.L + x.l;
    x.M = g < 0 ? 0 : max(0, min(a.M_max, __ldg(a.mem_len + gl)));
    x.kv_row = (gl * 2 * a.H + x.h) * a.M_max;
    x.mt = (x.M + kTile - 1) / kTile;
    x.tok[0] = lo + at;
    x.n_tok[0] = min(kTok, n - at);
    x.n_loc = x.lim0 = x.len = 0;
    x.slot[0] = x.slot[1] = s;
    x.poison = 0;
    x.shared = BLOCK || n > kTok;
    if (BLOCK) {
      x.tok[1] = x.tok[0] + kTok;
      x.n_tok[1] = max(0, min(kTok, n - at - kTok));
      const int len = max(a.seq_len[x.e], 0);
      x.len = (int)min((int64_t)len, cap);
      x.lim0 = len - n + at + 1;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int seen = max(0, min(x.lim0 + x.n_tok[0] - 1 + i * x.n_tok[1], x.len));
        x.t0[i] = 0;
        x.t1[i] = x.n_tok[i] > 0 ? x.mt + (seen + kTile - 1) / kTile : 0;
        x.n_loc = max(x.n_loc, seen);
      }
    } else if (x.shared) {
      const int per = (x.mt + splits - 1) / splits;
      x.tok[1] = x.tok[0] + kTok;
      x.n_tok[1] = max(0, min(kTok, n - at - kTok));
      x.t0[0] = x.t0[1] = min(x.mt, s * per);
      x.t1[0] = min(x.mt, s * per + per);
      x.t1[1] = x.n_tok[1] > 0 ? x.t1[0] : x.t0[1];  // (no rows: no tiles)
    } else {
      const int per = (x.mt + 2 * splits - 1) / (2 * splits);
      x.tok[1] = x.tok[0];
      x.n_tok[1] = x.n_tok[0];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x.slot[i] = 2 * s + i;
        x.t0[i] = min(x.mt, x.slot[i] * per);
        x.t1[i] = min(x.mt, x.slot[i] * per + per);
      }
    }
    return x;
  };
  // valid keys of a tile (for the pair: a single row may see fewer)
  auto valid_keys = [&](const Unit& x, int tile) -> int {
    return !BLOCK || tile < x.mt ? min(kTile, x.M - tile * kTile) : min(kTile, x.n_loc - (tile - x.mt) * kTile);
  };

  // a value tile that warp 10 prepares: rows past the last valid one within a 16-key step, or a
  // page tile that some rows of the pair do not see in full
  auto prepared = [&](const Unit& x, int tile) -> bool {
    return (valid_keys(x, tile) & 15) != 0 || (BLOCK && tile >= x.mt && (tile - x.mt + 1) * kTile > x.lim0);
  };
  // unit un of this CTA (every lane of the caller's warp, or its one thread, waits)
  auto unit_wait = [&](int un) -> bool { return mbar_wait(smem_u32(&u_full[un % kUnits]), (un / kUnits) & 1u, abort_flag, kUnitWaitNs); };

  // (setmaxnreg in each role's own branch: the compiler allocates what follows by it)
  if (warp == kTmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    // ---- loads: the warp walks together (a lane per page box), lane 0 arms and waits
    if (lane == 0) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_kv)) : "memory");
      if (BLOCK) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_pages)) : "memory");
    }
    bool ok = true;
    uint32_t it = 0;                // ring position
    uint32_t tiles = 0;             // key tiles of the block form so far
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity, abort_flag))) ok = false;
      return ok;
    };
    // page ids of 512 consecutive rows of a sequence, a lane per 16 rows
    int ids_e = -1, ids_win = -1, ids = 0;
    const int log2_box = min(6, a.log2_page);  // rows of a page box: the page, at most 64
    auto load = [&](const Unit& x, int tile, bool is_v) {
      if (!ok) return;
      const int slot = it % kSlots;
      if (!wait(&empty[slot], ((it / kSlots) & 1u) ^ 1u)) return;
      ++it;
      const uint32_t bar = smem_u32(&full[slot]);
      const uint32_t dst = sbase + kOffRing + slot * kSlotBytes;
      const int valid = valid_keys(x, tile);
      if (!BLOCK || tile < x.mt) {
        if (lane == 0) {
          const int boxes = valid > kBox ? 2 : 1;
          const int row = (int)(x.kv_row + (is_v ? (int64_t)a.H * a.M_max : 0) + tile * kTile);
          if (BLOCK && !is_v) tb.bad[tiles % kBadRing] = 0u;
          mbar_arrive_expect_tx(bar, boxes * 2 * kBox * 128);
          for (int b = 0; b < boxes; ++b) {
            tma_load_rows(dst + b * kBox * 128, &tm_kv, bar, 0, row + b * kBox);
            tma_load_rows(dst + kHalfBytes + b * kBox * 128, &tm_kv, bar, kHalf, row + b * kBox);
          }
        }
      } else {
        const int key0 = (tile - x.mt) * kTile;
        if (ids_e != x.e || ids_win != (key0 >> 9)) {
          ids_e = x.e;
          ids_win = key0 >> 9;
          const int row = (ids_win << 9) + lane * 16;
          ids = row < x.len ? __ldg(a.page_table + (int64_t)x.e * a.max_pages + (row >> a.log2_page)) : 0;
        }
        const int boxes = (valid + (1 << log2_box) - 1) >> log2_box;
        // lane b < boxes: rows [b << log2_box, ...) of the tile
        const int id = __shfl_sync(0xffffffffu, ids, ((key0 & 511) >> 4) + ((lane << log2_box) >> 4 & 7));
        const bool use = lane < boxes;
        const bool bad = use && (id < 0 || id >= a.NP);
        const uint32_t bads = __ballot_sync(0xffffffffu, bad);
        if (lane == 0) {
          if (!is_v) {
            uint32_t mask = 0u;
            for (int b = 0; b < boxes; ++b)
              if ((bads >> b) & 1u) mask |= ((1u << (1 << (log2_box - 4))) - 1u) << (b << (log2_box - 4));
            tb.bad[tiles % kBadRing] = mask;
            if (bads) msa::set_err(a.dev_err, MSA_DEVERR_BAD_PAGE);
          }
          mbar_arrive_expect_tx(bar, (uint32_t)boxes * 2u * (128u << log2_box));
        }
        __syncwarp();
        if (use) {
          // (a bad page's box starts past the tensor's end and reads as zeros)
          const int64_t first = ((((int64_t)x.l * a.NP + id) * 2 + (is_v ? 1 : 0)) * a.H + x.h) << a.log2_page;
          const int64_t past = ((int64_t)a.L * a.NP * 2 * a.H) << a.log2_page;
          const int row = (int)(bad ? past : first + ((key0 + (lane << log2_box)) & ((1 << a.log2_page) - 1)));
          const uint32_t to = dst + (uint32_t)(lane << log2_box) * 128u;
          tma_load_rows(to, &tm_pages, bar, 0, row);
          tma_load_rows(to + kHalfBytes, &tm_pages, bar, kHalf, row);
        }
      }
      if (BLOCK && !is_v) ++tiles;
      __syncwarp();
    };
    int un = 0;
    for (; unit_number(un) < n_units && ok; ++un) {
      if (!__all_sync(0xffffffffu, unit_wait(un))) {
        ok = false;
        break;
      }
      const Unit& x = tb.units[un % kUnits];
      const int n0 = x.t1[0] - x.t0[0], n1 = x.t1[1] - x.t0[1];
      // tile j of stream b is loaded for it alone
      auto own_b = [&](int j) { return j < n1 && (!x.shared || j >= n0); };
      // the first key tiles (j = -1), then per j value tile j and key tile j + 1 of either stream
#pragma unroll 1
      for (int i = -2; i < 2 * max(n0, n1) && ok; ++i) {
        const int st = i & 1, j = i >> 1;
        auto own = [&](int k) { return st == 0 ? k < n0 : own_b(k); };
#pragma unroll 1
        for (int v = 1; v >= 0; --v) {
          const int k = v ? j : j + 1;
          if (k >= 0 && own(k)) load(x, x.t0[st] + k, v != 0);
        }
      }
      if (lane == 0) mbar_arrive(smem_u32(&u_empty[un % kUnits]));
      __syncwarp();
    }
    if (!ok) {
      // wait (bounded) for the copies in flight: the last kSlots loads
      if (lane == 0) {
        *abort_flag = 1;
        msa::set_err(a.dev_err, MSA_DEVERR_TIMEOUT);
        for (uint32_t p = it > kSlots ? it - kSlots : 0; p < it; ++p)
          mbar_drain(smem_u32(&full[p % kSlots]), (p / kSlots) & 1u);
      }
      __syncwarp();
    }
  } else if (warp == kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    if (elect_one()) {
      // one thread waits and issues.  Descriptors: the low words carry the address (and the
      // leading offset), the high words are the same for all tiles of a kind.
      constexpr uint32_t idesc_s = idesc_make(kRows, kTile, false);
      constexpr uint32_t idesc_pv = idesc_make_bmn(kRows, kD);
      const uint64_t rows_desc = sw128_desc(sbase + kOffRing), q_desc = sw128_desc(sbase + kOffQ);
      const uint64_t cols_desc = sw128_desc_mn(sbase + kOffRing, kHalfBytes, 1024);
      bool ok = true, issued = false;
      uint32_t qn = 0, pn = 0;       // parities of the query and weight tiles used, a bit per stream
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = ok && mbar_wait(smem_u32(bar), parity & 1u, abort_flag);
      };
#pragma unroll 1
      for (uint32_t i = 0;; ++i) {
        wait(&c_full[i % kCommands], i / kCommands);
        if (!ok) break;
        const uint32_t w = *const_cast<volatile uint32_t*>(&tb.commands[i % kCommands]);
        if (w & kEnd) break;
        const uint32_t st = w & kStreamB;
        const uint32_t s_cols = tmem_base + kColS + st * kTile;
        if (w & kWeigh) {
          const int n_ks = (w >> 12) & 15;
          const uint32_t slot = (w >> 16) & 7u, o_cols = tmem_base + kColO + st * kTile;
          const uint64_t vt = cols_desc + (uint64_t)(slot * (kSlotBytes >> 4));
          const uint32_t acc = w & kFirst ? 0u : 1u;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            wait(&p_ready[2 * st + h], pn >> st);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int ks = 4 * h; ks < 4 * h + 4; ++ks)
              if (ks < n_ks) umma_ts(o_cols, s_cols + 8 * ks, vt + ks * (2048 >> 4), idesc_pv, ks > 0 ? 1u : acc);
          }
          if (!ok) break;
          pn ^= 1u << st;
          if (w & kOutput) umma_commit<false>(smem_u32(&o_done[st]));
          if (w & kFreeV) umma_commit<false>(smem_u32(&empty[slot]));
        }
        if (w & kScore) {
          if (w & kAwaitQ) {
            wait(&q_full[st], qn >> st);
            if (!ok) break;
            qn ^= 1u << st;
          }
          const uint32_t slot = (w >> 20) & 7u;
          const uint64_t kt = rows_desc + (uint64_t)(slot * (kSlotBytes >> 4)), qt = q_desc + (uint64_t)(st * (kSlotBytes >> 4));
#pragma unroll
          for (int ks = 0; ks < kD / 16; ++ks) {
            const uint64_t on = ((ks >> 2) * kHalfBytes + (ks & 3) * 32) >> 4;
            umma<false, false>(s_cols, qt + on, kt + on, idesc_s, ks > 0 ? 1u : 0u);
          }
          umma_commit<false>(smem_u32(&s_ready[st]));
          if (w & kFreeK) umma_commit<false>(smem_u32(&empty[slot]));
          if (w & kFreeQ) umma_commit<false>(smem_u32(&q_empty[st]));
          issued = true;
        }
      }
      if (!ok) {
        *abort_flag = 1;
        msa::set_err(a.dev_err, MSA_DEVERR_TIMEOUT);
        if (issued) {
          umma_commit<false>(smem_u32(drain));
          mbar_drain(smem_u32(drain), 0u);
        }
      }
    }
    __syncwarp();
  } else if (warp < kMmaWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // ---- softmax: stream st, thread = row (TMEM lane)
    const int st = warp >> 2, r = tid & (kRows - 1);
    const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem_base + lane_addr + kColS + (uint32_t)(st * kTile);
    const uint32_t o_col = tmem_base + lane_addr + kColO + (uint32_t)(st * kTile);
    float* part = reinterpret_cast<float*>(a.ws + kWsMemory);
    const int64_t all_rows = (int64_t)a.L * a.T * Hq;
    float2* stat = reinterpret_cast<float2*>(a.ws + kWsMemory + memory_part_bytes(all_rows, max_splits));
    const bool wide = ((BLOCK ? reinterpret_cast<uintptr_t>(a.out) : reinterpret_cast<uintptr_t>(part)) & 31u) == 0;
    const f32x2 scale2 = pack2(a.qscale, a.qscale);
    uint32_t sn = 0, on = 0;  // score tiles and units so far
    uint32_t tiles = 0;       // key tiles of the pairs before (block form)
    bool ok = true;
    for (int un = 0; unit_number(un) < n_units && ok; ++un) {
      if (!__all_sync(0xffffffffu, unit_wait(un))) {
        ok = false;
        break;
      }
      const Unit& x = tb.units[un % kUnits];
      const int t0 = x.t0[st], n = x.t1[st] - t0, M = x.M, mt = x.mt;
      const int tk = r / G;                     // this row's token in its row tile
      const bool mine = tk < x.n_tok[st];
      const int64_t row = x.slot[st] * all_rows + ((int64_t)x.l * a.T + x.tok[st] + tk) * Hq + x.h * G + r % G;
      // page rows that this row sees
      const int seen = BLOCK ? max(0, min(x.lim0 + st * kTok + tk, x.len)) : 0;
      const uint32_t tiles_after = tiles + (BLOCK ? max(x.t1[0], x.t1[1]) : 0);
      const bool any_row = (r & ~31) / G < x.n_tok[st];  // (else the warp only passes its tiles on)
      float m = -INFINITY;
      float sum = 0.f;
      for (int j = 0; j < n; ++j) {
        if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&s_ready[st]), sn & 1u, abort_flag, kUnitWaitNs))) {
          ok = false;
          break;
        }
        ++sn;
        if (!any_row) {
          if (lane < 2) mbar_arrive(smem_u32(&p_ready[2 * st + lane]));
          continue;
        }
        tc_fence_after();
        uint32_t sv[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(s_col + 32 * c, sv[c]);
        tmem_wait_ld();
        const bool page = BLOCK && t0 + j >= mt;
        const int valid = page ? seen - (t0 + j - mt) * kTile : M - (t0 + j) * kTile;
        const uint32_t bad = BLOCK ? *const_cast<volatile uint32_t*>(&tb.bad[(tiles + j) % kBadRing]) : 0u;
        if (!__all_sync(0xffffffffu, valid >= kTile && bad == 0u)) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            // a bit per key that is seen: below the limit, and its page usable
            const int n_seen = valid - 32 * c;
            uint32_t keep = n_seen >= 32 ? 0xFFFFFFFFu : n_seen <= 0 ? 0u : (1u << n_seen) - 1u;
            if (BLOCK) keep &= ~(((bad >> (2 * c)) & 1u) * 0xFFFFu | ((bad >> (2 * c + 1)) & 1u) * 0xFFFF0000u);
#pragma unroll
            for (int e = 0; e < 32; ++e) sv[c][e] = (keep >> e) & 1u ? sv[c][e] : 0xFF800000u;
          }
        }
        float mx[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          mx[c] = max3(__uint_as_float(sv[c][0]), __uint_as_float(sv[c][1]), __uint_as_float(sv[c][2]));
#pragma unroll
          for (int e = 3; e < 31; e += 2)
            mx[c] = max3(mx[c], __uint_as_float(sv[c][e]), __uint_as_float(sv[c][e + 1]));
          mx[c] = max3(mx[c], __uint_as_float(sv[c][31]), __uint_as_float(sv[c][31]));
        }
        const float top = max3(max3(mx[0], mx[1], mx[2]), mx[3], mx[3]) * a.qscale;  // (qscale > 0; NaN kept)
        const bool need = top > m + kHeadroom;
        if (__any_sync(0xffffffffu, need)) {
          const float alpha = need ? ex2_ftz(m - top) : 1.f;  // 0 while m is still -inf
          if (need) m = top;
          if (j > 0) {  // (PV(j - 1) is done: its commit came before this tile's scores)
            sum *= alpha;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t o[32];
              tmem_ld32(o_col + 32 * c, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st32(o_col + 32 * c, o);
            }
          }
        }
        const float base = m == -INFINITY ? 0.f : m;
        const f32x2 base2 = pack2(-base, -base);
        f32x2 add[2] = {0ull, 0ull};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pw[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const uint32_t s0 = sv[2 * c + (e >> 4)][2 * (e & 15)], s1 = sv[2 * c + (e >> 4)][2 * (e & 15) + 1];
            float p0, p1;
            unpack2(fma2(pack2(__uint_as_float(s0), __uint_as_float(s1)), scale2, base2), p0, p1);
            p0 = ex2_ftz(p0);
            p1 = ex2_ftz(p1);
            add[e & 1] = add2(add[e & 1], pack2(p0, p1));
            pw[e] = msa::float2_to_bf16x2(p0, p1);
          }
          tmem_st32(s_col + 32 * c, pw);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&p_ready[2 * st + c]));
        }
        float s0, s1;
        unpack2(add2(add[0], add[1]), s0, s1);
        sum += s0 + s1;
      }
      tiles = tiles_after;
      if (!ok) break;
      const float inv = sum == 0.f ? 0.f : 1.f / sum;  // (no key seen: output 0; a NaN sum is kept)
      if (n > 0) {
        if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&o_done[st]), on & 1u, abort_flag))) {
          ok = false;
          break;
        }
        ++on;
        tc_fence_after();
      }
      const bool poisoned = BLOCK && *const_cast<volatile int*>(&tb.units[un % kUnits].poison) != 0;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t o[32];
        if (n > 0) {
          tmem_ld32(o_col + 32 * c, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
        if (mine && BLOCK) {
          __nv_bfloat16* dst = a.out + row * kD + 32 * c;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t w[8];
#pragma unroll
            for (int v = 0; v < 8; ++v)
              w[v] = msa::float2_to_bf16x2(__uint_as_float(o[16 * e + 2 * v]) * inv, __uint_as_float(o[16 * e + 2 * v + 1]) * inv);
            st_global_32(dst + 16 * e, wide, w);
          }
        } else if (mine && n > 0) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // (the row kernel's order: of every 16 dims, 0 1 8 9, 2 3 10 11, 4 5 12 13, 6 7 14 15)
            const int d = 16 * (e >> 1) + 4 * (e & 1);
            const uint32_t w[8] = {o[d], o[d + 1], o[d + 8], o[d + 9], o[d + 2], o[d + 3], o[d + 10], o[d + 11]};
            st_global_32(part + row * kD + 32 * c + 8 * e, wide, w);
          }
        }
      }
      if (BLOCK && mine && poisoned) add_not_finite(a, x, seen, a.out + row * kD);
      tc_fence_before();  // (O is read: the next unit's first PV may overwrite it)
      if (!BLOCK && mine) stat[row] = make_float2(m, sum);  // (no tiles: -inf and 0)
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&u_empty[un % kUnits]));
    }
    if (!ok) {
      *abort_flag = 1;
      if (lane == 0) msa::set_err(a.dev_err, MSA_DEVERR_TIMEOUT);
    }
  } else if (warp == kValueWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    // ---- commands and value tiles.  The warp passes every tile of the ring in order (and no slot is filled
    // again before), so that the phases it waits for are never ambiguous.
    bool ok = true;
    uint32_t it = 0, cn = 0;  // ring position, commands so far
    auto prepare = [&](const Unit& x, int tile, uint32_t vt, int un) {
      const int valid = valid_keys(x, tile), rows = (valid + 15) & ~15;
      for (int i = lane; i < (rows - valid) * 16; i += 32) {
        const int row = valid + (i >> 4), c16 = i & 15;
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vt + (uint32_t)((c16 >> 3) * kHalfBytes + row * 128 +
                                                                             (((c16 & 7) ^ (row & 7)) << 4))),
                     "r"(0u)
                     : "memory");
      }
      __syncwarp();
      // Values that are not finite must not reach the rows that do not see them (0 x inf is NaN):
      // they are taken out, and the unit's rows add what they see of them at the end.
      // (One pass that only looks, 16 rows at a time, and as a rule finds nothing: adding a
      // step to an exponent of all ones carries into the sign's place.)
      if (BLOCK && tile >= x.mt) {
        for (int i0 = max(0, first_partial(x) - (tile - x.mt) * kTile); i0 < rows; i0 += 16) {
          uint32_t w[8][4], found = 0u;
          const uint32_t from = vt + (uint32_t)(i0 * 128 + lane * 16);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[e][0]), "=r"(w[e][1]), "=r"(w[e][2]), "=r"(w[e][3])
                         : "r"(from + (uint32_t)((e >> 2) * kHalfBytes + (e & 3) * 512))
                         : "memory");
#pragma unroll
          for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int v = 0; v < 4; ++v) found |= ((w[e][v] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
          if (__any_sync(0xffffffffu, found != 0u)) {
            for (int e = 0; e < 8; ++e)
              for (int v = 0; v < 4; ++v) {
                const uint32_t to = from + (uint32_t)((e >> 2) * kHalfBytes + (e & 3) * 512 + v * 4);
                uint32_t y;
                asm volatile("ld.shared.b32 %0, [%1];" : "=r"(y) : "r"(to) : "memory");
                if ((y & 0x7F80u) == 0x7F80u) y &= 0xFFFF0000u;
                if ((y & 0x7F800000u) == 0x7F800000u) y &= 0x0000FFFFu;
                asm volatile("st.shared.b32 [%0], %1;" ::"r"(to), "r"(y) : "memory");
              }
            if (lane == 0) *const_cast<volatile int*>(&tb.units[un % kUnits].poison) = 1;
          }
        }
      }
      __threadfence_block();
      fence_async_smem();
      __syncwarp();
    };
    auto command = [&](uint32_t w) {
      if (!ok) return;
      if (lane == 0) {
        *const_cast<volatile uint32_t*>(&tb.commands[cn % kCommands]) = w;
        mbar_arrive(smem_u32(&c_full[cn % kCommands]));
      }
      ++cn;
    };
    auto pass = [&](const Unit& x, int tile, bool is_v, int un) {
      if (!ok) return;
      if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&full[it % kSlots]), (it / kSlots) & 1u, abort_flag))) {
        ok = false;
        return;
      }
      if (is_v && prepared(x, tile)) prepare(x, tile, sbase + kOffRing + (it % kSlots) * kSlotBytes, un);
      if (lane == 0) mbar_arrive(smem_u32(&empty[it % kSlots]));
      __syncwarp();
      ++it;
    };
    int un = 0;
    for (; unit_number(un) < n_units && ok; ++un) {
      if (!__all_sync(0xffffffffu, unit_wait(un))) {
        ok = false;
        break;
      }
      const Unit& x = tb.units[un % kUnits];
      const int n0 = x.t1[0] - x.t0[0], n1 = x.t1[1] - x.t0[1];
      const bool shared = x.shared;
      uint32_t ka = 0, va = 0;  // slots of stream a's key and value tile
#pragma unroll 1
      for (int i = -2; i < 2 * max(n0, n1) && ok; ++i) {  // (the order of the loads)
        const int st = i & 1, j = i >> 1;
        const int n = st ? n1 : n0, n_other = st ? n0 : n1;
        if (j >= n) continue;
        uint32_t w = (uint32_t)st;
#pragma unroll 1
        for (int v = 1; v >= 0; --v) {  // value tile j, key tile j + 1
          const int k = v ? j : j + 1;
          if (k < 0 || k >= n) continue;
          const bool with = shared && k < n_other;  // both streams use the tile
          uint32_t slot = v ? va : ka;
          if (st == 0 || !with) {
            slot = it % kSlots;
            pass(x, x.t0[st] + k, v != 0, un);
          }
          if (st == 0) (v ? va : ka) = slot;
          const bool last_use = st == 1 || !with;
          if (v)
            w |= kWeigh | (k == 0 ? kFirst : 0u) | (k + 1 == n ? kOutput : 0u) | (last_use ? kFreeV : 0u) |
                 (uint32_t)((valid_keys(x, x.t0[st] + k) + 15) >> 4) << 12 | slot << 16;
          else
            w |= kScore | (k == 0 ? kAwaitQ : 0u) | (k + 1 == n ? kFreeQ : 0u) | (last_use ? kFreeK : 0u) | slot << 20;
        }
        if (w & (kWeigh | kScore)) command(w);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&u_empty[un % kUnits]));
    }
    command(kEnd);
    if (!ok && lane == 0) {
      *abort_flag = 1;
      msa::set_err(a.dev_err, MSA_DEVERR_TIMEOUT);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    // ---- units, each worked out before the queries of the one before it are loaded
    if (lane == 0) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_q)) : "memory");
    bool ok = true;
    uint32_t qn[2] = {0, 0};  // query tiles loaded per stream
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity, abort_flag, kUnitWaitNs))) ok = false;
      return ok;
    };
    auto load_q = [&](const Unit& x, int st) {
      if (!ok || x.t1[st] <= x.t0[st]) return;
      if (!wait(&q_empty[st], (qn[st] & 1u) ^ 1u)) return;
      ++qn[st];
      if (lane == 0) {
        const uint32_t bar = smem_u32(&q_full[st]);
        const uint32_t dst = sbase + kOffQ + st * kSlotBytes;
        mbar_arrive_expect_tx(bar, kSlotBytes);
        tma_load_4d(dst, &tm_q, bar, 0, x.h * G, x.tok[st], x.l);
        tma_load_4d(dst + kHalfBytes, &tm_q, bar, kHalf, x.h * G, x.tok[st], x.l);
      }
      __syncwarp();
    };
    for (int un = 0; ok; ++un) {
      const int64_t u = unit_number(un);
      if (u < n_units) {
        const Unit x = unit_at(u);
        if (!wait(&u_empty[un % kUnits], ((un / kUnits) & 1u) ^ 1u)) break;
        if (lane == 0) {
          tb.units[un % kUnits] = x;
          mbar_arrive(smem_u32(&u_full[un % kUnits]));
          // its queries into L2, so that they arrive soon once their place is free
          for (int st = 0; st < 2; ++st)
            if (x.t1[st] > x.t0[st] && (st == 0 || x.shared)) {
              tma_prefetch_4d(&tm_q, 0, x.h * G, x.tok[st], x.l);
              tma_prefetch_4d(&tm_q, kHalf, x.h * G, x.tok[st], x.l);
            }
        }
        __syncwarp();
      }
      if (un > 0) {  // (its place is not taken again before this warp has come by)
        const Unit& x = tb.units[(un - 1) % kUnits];
        load_q(x, 0);
        load_q(x, 1);
      }
      if (u >= n_units) break;
    }
    if (!ok) {
      if (lane == 0) {
        *abort_flag = 1;
        msa::set_err(a.dev_err, MSA_DEVERR_TIMEOUT);
        for (int st = 0; st < 2; ++st)
          if (qn[st] > 0) mbar_drain(smem_u32(&q_full[st]), (qn[st] - 1) & 1u);
      }
      __syncwarp();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc<false>(tmem_base, kTmemCols);
  }
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static const EncodeTiledFn fn = []() -> EncodeTiledFn {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult qr;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &qr) == cudaSuccess &&
        qr == cudaDriverEntryPointSuccess)
      return reinterpret_cast<EncodeTiledFn>(p);
    return nullptr;
  }();
  return fn;
}

// bf16 rows of 128 elements, box [box_rows][64 elements], 128-byte swizzle; rows past the end
// read as zero
bool make_kv_map(CUtensorMap* m, const void* base, uint64_t rows, int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)kD, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)kD * 2};
  const cuuint32_t box[2] = {(cuuint32_t)kHalf, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// bf16 [L][T][Hq][128], box [128 / G tokens][G heads][64 dims]; coordinates (dim, head, token, layer)
bool make_q_map(CUtensorMap* m, const void* base, int Hq, int T, int L, int G) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)kD, (cuuint64_t)Hq, (cuuint64_t)T, (cuuint64_t)L};
  const cuuint64_t strides[3] = {(cuuint64_t)kD * 2, (cuuint64_t)Hq * kD * 2, (cuuint64_t)T * Hq * kD * 2};
  const cuuint32_t box[4] = {(cuuint32_t)kHalf, (cuuint32_t)G, (cuuint32_t)(kRows / G), 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int G, bool BLOCK>
cudaError_t launch_tiles_t(const Attend& a, int max_splits, cudaStream_t s) {
  CUtensorMap tm_q, tm_kv, tm_pages;
  if (!make_q_map(&tm_q, a.q, a.H * G, a.T, a.L, G)) return cudaErrorInvalidValue;
  tm_kv = tm_pages = tm_q;  // (whichever is not read)
  if (a.NG > 0 && !make_kv_map(&tm_kv, a.mem_kv, (uint64_t)a.NG * a.L * 2 * a.H * a.M_max, kBox))
    return cudaErrorInvalidValue;
  if (BLOCK && !make_kv_map(&tm_pages, a.pages, ((uint64_t)a.L * a.NP * 2 * a.H) << a.log2_page,
                            std::min(kBox, 1 << a.log2_page)))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_shared_memory(reinterpret_cast<const void*>(tile_kernel<G, BLOCK>), kSmemTc, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(msa::sm_count(), 1, 1);
  cfg.blockDim = dim3(kThreadsTc, 1, 1);
  cfg.dynamicSmemBytes = kSmemTc;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tile_kernel<G, BLOCK>, tm_q, tm_kv, tm_pages, a, max_splits);
}

}  // namespace

cudaError_t launch_memory(const Attend& a, int max_splits, cudaStream_t s) {
  switch (a.G) {
    case 1: return launch_tiles_t<1, false>(a, max_splits, s);
    case 2: return launch_tiles_t<2, false>(a, max_splits, s);
    case 4: return launch_tiles_t<4, false>(a, max_splits, s);
    default: return launch_tiles_t<8, false>(a, max_splits, s);
  }
}

cudaError_t launch_blocks(const Attend& a, cudaStream_t s) {
  switch (a.G) {
    case 1: return launch_tiles_t<1, true>(a, 1, s);
    case 2: return launch_tiles_t<2, true>(a, 1, s);
    case 4: return launch_tiles_t<4, true>(a, 1, s);
    default: return launch_tiles_t<8, true>(a, 1, s);
  }
}

}  // namespace paged
