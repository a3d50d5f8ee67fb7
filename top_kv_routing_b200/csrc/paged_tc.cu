// Shared-memory attention of a paged batch on the tcgen05 tensor cores: the memory part, all
// new tokens of a group at once.
//
// Follows "MSA端到端可训练记忆模型完整开源，支持亿级Token上下文", section 架构 (softmax over the
// selected memory joined to the local K/V), and the MSA paper reading notes, section
// 推理全流程.
//
// The packed tokens of a group (all of its sequences' new tokens) x the G query heads of key
// head h are the MMA's rows, 128 a row tile, so every tile of keys is read once per 256 rows
// whatever the number of sequences.  A unit is (group, layer, key head, pair of row tiles,
// key split).  Persistent CTAs (one per SM) of 320 threads walk the units:
//   warp 9 (one thread)  TMA: the unit's query rows (4D box), then 128-key tiles of K and V in
//                        the order the MMAs use them, through a ring of 32 KB slots;
//   warp 8               MMA issue for two streams a and b: S = Q K^T (queries from shared
//                        memory, M = N = 128), O += P V (weights from tensor memory, written
//                        over their scores; V read MN-major from its rows).  PV_a(j), S_a(j+1),
//                        PV_b(j), S_b(j+1), ...: while one stream's softmax runs, the tensor
//                        cores work for the other;
//   warps 0..3, 4..7     the softmax of stream a and of stream b: a thread per row.  A running
//                        maximum that is raised (and O rescaled in tensor memory) only when a
//                        score exceeds it by more than 2^8; weights exp2(s - m) rounded to
//                        bf16 (the MMA's operand type; the row sum takes them unrounded).
// Streams a and b are the two row tiles of the pair over the same keys.  A group of at most
// one row tile gives both streams the same rows and each half of the unit's keys instead.
// Output: per row and key split the unnormalised fp32 output, its maximum and its sum, which
// the row kernel (paged_rows.cu) joins with the sequence's own pages.
//
// S_x(j + 1) is issued after PV_x(j), so its completion also says that O_x is stable: the
// softmax rescales it without another wait.  Key rows past the memory's length are zeroed in
// shared memory before the PV that reads them (they may hold anything).  Every wait is
// bounded (2 s); a timeout sets MSA_DEVERR_TIMEOUT and the CTA drains and frees its TMEM.
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
constexpr int kSlots = 4;
constexpr int kWarpsTc = 10;
constexpr int kThreadsTc = kWarpsTc * 32;
constexpr int kMmaWarp = 8, kTmaWarp = 9;
constexpr uint32_t kTmemCols = 512;       // S_a | S_b | O_a | O_b
constexpr uint32_t kColS = 0, kColO = 256;
constexpr float kHeadroom = 8.0f;         // log2 growth of a row's maximum tolerated before rescaling

struct TablesTc {
  int scan[kMaxSeqs + 1];  // row-tile pairs of the groups before g
  int lo[kMaxSeqs];        // first token
  int n[kMaxSeqs];         // tokens
  int warp_sum[kWarpsTc];
  int most;                // most key tiles of any (group, layer)
  int splits;
  uint32_t tmem;
  int abort;
};

constexpr int kOffQ = 0;
constexpr int kOffRing = 2 * kSlotBytes;
constexpr int kOffBars = kOffRing + kSlots * kSlotBytes;
constexpr int kOffTables = kOffBars + 256;
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
__device__ __forceinline__ void tma_load_rows(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}

__device__ __forceinline__ void st_global_v8(float* p, const float (&x)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(x[0]), "f"(x[1]), "f"(x[2]),
               "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
               : "memory");
}

// One unit as every role sees it.
struct Unit {
  int l, h;
  int tok[2], n_tok[2];      // each stream's tokens
  int t0[2], t1[2];          // each stream's key tiles [t0, t1)
  int M;                     // memory rows
  bool shared;               // the streams read the same key tiles
  int64_t kv_row;            // row of key 0 in the memory tensor; values H * M_max further
  int slot[2];               // partial slot
};

template <int G>
__global__ void __launch_bounds__(kThreadsTc, 1)
    memory_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kv,
                  const __grid_constant__ Attend a, int max_splits) {
  constexpr int kTok = kRows / G;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  TablesTc& tb = *reinterpret_cast<TablesTc*>(smem + kOffTables);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBars);
  uint64_t* full = bars;                 // [kSlots] tile landed
  uint64_t* empty = bars + kSlots;       // [kSlots] tile read by its MMAs
  uint64_t* q_full = bars + 2 * kSlots;  // [2] the stream's queries landed
  uint64_t* q_empty = q_full + 2;        // [2] read by the stream's last score MMA of the unit
  uint64_t* s_ready = q_empty + 2;       // [2] scores in tensor memory (and the stream's PV before them done)
  uint64_t* p_ready = s_ready + 2;       // [2] weights in tensor memory (4 warps)
  uint64_t* o_done = p_ready + 2;        // [2] the stream's last PV of the unit done
  uint64_t* drain = o_done + 2;
  volatile int* abort_flag = &tb.abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sbase = smem_u32(smem);
  const int Hq = a.H * G, LH = a.L * a.H;

  if (tid == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(smem_u32(&q_full[x]), 1);
      mbar_init(smem_u32(&q_empty[x]), 1);
      mbar_init(smem_u32(&s_ready[x]), 1);
      mbar_init(smem_u32(&p_ready[x]), 4);
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
  wait_for_earlier_kernels();
  let_next_kernel_start();

  // ---- tables: tokens and row-tile pairs of every group
  const bool groups_ok = group_offsets_usable(a, tid, kThreadsTc);  // (a barrier for all threads)
  if (!groups_ok && blockIdx.x == 0 && tid == 0) msa::set_err(a.dev_err, MSA_DEVERR_BAD_OFFSETS);
  {
    constexpr int kPer = (kMaxSeqs + kThreadsTc - 1) / kThreadsTc;
    int v[kPer], sum = 0, most = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int g = tid * kPer + i;
      v[i] = sum;
      if (g < a.NG) {
        int lo, n;
        if (!groups_ok || !group_tokens(a, g, lo, n)) n = 0;
        tb.lo[g] = lo;
        tb.n[g] = n;
        sum += (n + 2 * kTok - 1) / (2 * kTok);
      }
    }
    for (int i = tid; i < a.NG * a.L; i += kThreadsTc) most = max(most, a.mem_len[i]);
    if (most > a.M_max) {
      if (blockIdx.x == 0) msa::set_err(a.dev_err, MSA_DEVERR_CAPACITY);
      most = a.M_max;
    }
    most = __reduce_max_sync(0xffffffffu, most);
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) tb.warp_sum[warp] = inc;
    if (lane == 0) atomicMax(&tb.most, (most + kTile - 1) / kTile);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    int base = inc - sum;
    for (int w = 0; w < warp; ++w) base += tb.warp_sum[w];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int g = tid * kPer + i;
      if (g < a.NG) tb.scan[g] = base + v[i];
    }
    if (tid == kThreadsTc - 1) tb.scan[a.NG] = base + sum;
  }
  __syncthreads();
  const int pairs = tb.scan[a.NG];
  if (tid == 0) {
    // the split that finishes first, a unit costing its tiles and about two more
    const int64_t units = (int64_t)pairs * LH;
    int best = 1;
    int64_t cost = INT64_MAX;
    for (int s = 1; s <= max_splits && s <= max(1, tb.most); ++s) {
      const int64_t c = (units * s + gridDim.x - 1) / gridDim.x * ((tb.most + s - 1) / s + 2);
      if (c < cost) {
        cost = c;
        best = s;
      }
    }
    tb.splits = best;
    if (blockIdx.x == 0) *reinterpret_cast<int*>(a.ws + kWsSplits) = best;
  }
  __syncthreads();
  const int splits = tb.splits;
  const uint32_t tmem_base = tb.tmem;
  const int64_t n_units = (int64_t)pairs * LH * splits;

  auto unit_at = [&](int64_t u) -> Unit {
    Unit x;
    const int pair = (int)(u % pairs);
    const int64_t rest = u / pairs;
    const int s = (int)(rest % splits), lh = (int)(rest / splits);
    x.l = lh / a.H;
    x.h = lh - x.l * a.H;
    int lo = 0, hi = a.NG;  // scan[lo] <= pair < scan[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tb.scan[mid] <= pair) lo = mid; else hi = mid;
    }
    const int64_t gl = (int64_t)lo * a.L + x.l;
    x.M = max(0, min(a.M_max, __ldg(a.mem_len + gl)));
    x.kv_row = (gl * 2 * a.H + x.h) * a.M_max;
    const int nt = (x.M + kTile - 1) / kTile;
    const int at = (pair - tb.scan[lo]) * 2 * kTok, n = tb.n[lo];
    x.shared = n > kTok;
    x.tok[0] = tb.lo[lo] + at;
    x.n_tok[0] = min(kTok, n - at);
    if (x.shared) {
      const int per = (nt + splits - 1) / splits;
      x.tok[1] = x.tok[0] + kTok;
      x.n_tok[1] = max(0, min(kTok, n - at - kTok));
      x.t0[0] = x.t0[1] = min(nt, s * per);
      x.t1[0] = min(nt, s * per + per);
      x.t1[1] = x.n_tok[1] > 0 ? x.t1[0] : x.t0[1];  // (no rows: no tiles)
      x.slot[0] = x.slot[1] = s;
    } else {
      const int per = (nt + 2 * splits - 1) / (2 * splits);
      x.tok[1] = x.tok[0];
      x.n_tok[1] = x.n_tok[0];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        x.slot[i] = 2 * s + i;
        x.t0[i] = min(nt, x.slot[i] * per);
        x.t1[i] = min(nt, x.slot[i] * per + per);
      }
    }
    return x;
  };

  if (warp == kTmaWarp) {
    if (lane == 0) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_q)) : "memory");
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_kv)) : "memory");
      bool ok = true;
      uint32_t it = 0;                 // ring position
      int armed[kSlots], q_armed[2] = {-1, -1};
#pragma unroll
      for (int s = 0; s < kSlots; ++s) armed[s] = -1;
      uint32_t qn[2] = {0, 0};         // query tiles loaded per stream
      auto load = [&](const Unit& x, int tile, bool is_v) {
        if (!ok) return;
        const int slot = it % kSlots;
        const uint32_t ph = (it / kSlots) & 1u;
        if (!mbar_wait(smem_u32(&empty[slot]), ph ^ 1u, abort_flag)) {
          ok = false;
          return;
        }
        const int key0 = tile * kTile;
        const int boxes = x.M - key0 > kBox ? 2 : 1;
        const uint32_t bar = smem_u32(&full[slot]);
        const uint32_t dst = sbase + kOffRing + slot * kSlotBytes;
        const int row = (int)(x.kv_row + (is_v ? (int64_t)a.H * a.M_max : 0) + key0);
        mbar_arrive_expect_tx(bar, boxes * 2 * kBox * 128);
        for (int b = 0; b < boxes; ++b) {
          tma_load_rows(dst + b * kBox * 128, &tm_kv, bar, 0, row + b * kBox);
          tma_load_rows(dst + kHalfBytes + b * kBox * 128, &tm_kv, bar, kHalf, row + b * kBox);
        }
        armed[slot] = (int)ph;
        ++it;
      };
      auto load_q = [&](const Unit& x, int st) {
        if (!ok) return;
        if (!mbar_wait(smem_u32(&q_empty[st]), (qn[st] & 1u) ^ 1u, abort_flag)) {
          ok = false;
          return;
        }
        const uint32_t bar = smem_u32(&q_full[st]);
        const uint32_t dst = sbase + kOffQ + st * kSlotBytes;
        mbar_arrive_expect_tx(bar, kSlotBytes);
        tma_load_4d(dst, &tm_q, bar, 0, x.h * G, x.tok[st], x.l);
        tma_load_4d(dst + kHalfBytes, &tm_q, bar, kHalf, x.h * G, x.tok[st], x.l);
        q_armed[st] = (int)(qn[st] & 1u);
        ++qn[st];
      };
      for (int64_t u = blockIdx.x; u < n_units && ok; u += gridDim.x) {
        const Unit x = unit_at(u);
        const int n0 = x.t1[0] - x.t0[0], n1 = x.t1[1] - x.t0[1];
        if (n0 > 0) {
          load_q(x, 0);
          load(x, x.t0[0], false);
        }
        if (n1 > 0) {
          load_q(x, 1);
          if (!x.shared) load(x, x.t0[1], false);
        }
        for (int j = 0; j < max(n0, n1) && ok; ++j) {
          if (j < n0) {
            load(x, x.t0[0] + j, true);
            if (j + 1 < n0) load(x, x.t0[0] + j + 1, false);
          }
          if (!x.shared && j < n1) {
            load(x, x.t0[1] + j, true);
            if (j + 1 < n1) load(x, x.t0[1] + j + 1, false);
          }
        }
      }
      if (!ok) {
        *abort_flag = 1;
        msa::set_err(a.dev_err, MSA_DEVERR_TIMEOUT);
        for (int s = 0; s < kSlots; ++s)
          if (armed[s] >= 0) mbar_drain(smem_u32(&full[s]), (uint32_t)armed[s]);
        for (int st = 0; st < 2; ++st)
          if (q_armed[st] >= 0) mbar_drain(smem_u32(&q_full[st]), (uint32_t)q_armed[st]);
      }
    }
  } else if (warp == kMmaWarp) {
    // the warp waits together, one elected lane issues
    const bool leader = elect_one();
    constexpr uint32_t idesc_s = idesc_make(kRows, kTile, false);
    constexpr uint32_t idesc_pv = idesc_make_bmn(kRows, kD);
    bool ok = true, issued = false;
    uint32_t it = 0;               // ring position of the next tile
    uint32_t qn[2] = {0, 0};       // query tiles used per stream
    uint32_t pn[2] = {0, 0};       // weight tiles used per stream
    uint32_t kpos = 0, vpos = 0;   // (shared) ring positions of stream a's current K and V
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity, abort_flag))) ok = false;
      if (ok) tc_fence_after();
      return ok;
    };
    // scores of stream st over its key tile in ring position `pos`; `release`: the tile's last use
    auto score = [&](int st, uint32_t pos, bool release, bool last) {
      if (!ok) return;
      if (!wait(&full[pos % kSlots], (pos / kSlots) & 1u)) return;
      if (leader) {
        const uint32_t kt = sbase + kOffRing + (pos % kSlots) * kSlotBytes;
        const uint32_t qt = sbase + kOffQ + st * kSlotBytes;
        const uint32_t d = tmem_base + kColS + (uint32_t)(st * kTile);
#pragma unroll
        for (int ks = 0; ks < kD / 16; ++ks) {
          const uint32_t off = (uint32_t)((ks >> 2) * kHalfBytes);
          umma<false, false>(d, sw128_desc(qt + off) + (uint64_t)(2 * (ks & 3)),
                             sw128_desc(kt + off) + (uint64_t)(2 * (ks & 3)), idesc_s, ks > 0 ? 1u : 0u);
        }
        umma_commit<false>(smem_u32(&s_ready[st]));
        if (release) umma_commit<false>(smem_u32(&empty[pos % kSlots]));
        if (last) umma_commit<false>(smem_u32(&q_empty[st]));
      }
      issued = true;
      __syncwarp();
    };
    auto weigh = [&](int st, uint32_t pos, int valid, bool first, bool release, bool last) {
      if (!ok) return;
      if (!wait(&p_ready[st], pn[st] & 1u)) return;
      ++pn[st];
      if (!wait(&full[pos % kSlots], (pos / kSlots) & 1u)) return;
      const uint32_t vt = sbase + kOffRing + (pos % kSlots) * kSlotBytes;
      const int n_ks = min(kTile, valid + 15) / 16;  // 16-key steps
      if (valid < n_ks * 16) {  // rows past the memory's end may hold anything
        for (int i = lane; i < (n_ks * 16 - valid) * 16; i += 32) {
          const int row = valid + (i >> 4), c16 = i & 15;
          asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vt + (uint32_t)((c16 >> 3) * kHalfBytes + row * 128 +
                                                                               (((c16 & 7) ^ (row & 7)) << 4))),
                       "r"(0u)
                       : "memory");
        }
        fence_async_smem();
        __syncwarp();
      }
      if (leader) {
        const uint32_t p = tmem_base + kColS + (uint32_t)(st * kTile);
        const uint32_t d = tmem_base + kColO + (uint32_t)(st * kTile);
        for (int ks = 0; ks < n_ks; ++ks)
          umma_ts(d, p + (uint32_t)(8 * ks), sw128_desc_mn(vt + (uint32_t)(ks * 2048), kHalfBytes, 1024), idesc_pv,
                  (!first || ks > 0) ? 1u : 0u);
        if (release) umma_commit<false>(smem_u32(&empty[pos % kSlots]));
        if (last) umma_commit<false>(smem_u32(&o_done[st]));
      }
      __syncwarp();
    };
    for (int64_t u = blockIdx.x; u < n_units && ok; u += gridDim.x) {
      const Unit x = unit_at(u);
      const int n0 = x.t1[0] - x.t0[0], n1 = x.t1[1] - x.t0[1];
      const bool both = x.shared && n1 > 0;  // stream b reads stream a's tiles
      auto valid = [&](int tile) { return min(kTile, x.M - tile * kTile); };
      auto q_wait = [&](int st) {
        if (ok && wait(&q_full[st], qn[st] & 1u)) ++qn[st];
      };
      if (n0 > 0) {
        q_wait(0);
        kpos = it++;
        score(0, kpos, !both, n0 == 1);
      }
      if (n1 > 0) {
        q_wait(1);
        const uint32_t pos = x.shared ? kpos : it++;
        score(1, pos, true, n1 == 1);
      }
      for (int j = 0; j < max(n0, n1) && ok; ++j) {
        if (j < n0) {
          vpos = it++;
          weigh(0, vpos, valid(x.t0[0] + j), j == 0, !both, j + 1 == n0);
          if (j + 1 < n0) {
            kpos = it++;
            score(0, kpos, !both, j + 2 == n0);
          }
        }
        if (j < n1) {
          const uint32_t pv = x.shared ? vpos : it++;
          weigh(1, pv, valid(x.t0[1] + j), j == 0, true, j + 1 == n1);
          if (j + 1 < n1) {
            const uint32_t pk = x.shared ? kpos : it++;
            score(1, pk, true, j + 2 == n1);
          }
        }
      }
    }
    if (!ok) {
      if (lane == 0) {
        *abort_flag = 1;
        msa::set_err(a.dev_err, MSA_DEVERR_TIMEOUT);
      }
      if (issued) {
        if (leader) umma_commit<false>(smem_u32(drain));
        __syncwarp();
        mbar_drain(smem_u32(drain), 0u);
      }
    }
  } else {
    // ---- softmax: stream st, thread = row (TMEM lane)
    const int st = warp >> 2, r = tid & (kRows - 1);
    const uint32_t lane_addr = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem_base + lane_addr + kColS + (uint32_t)(st * kTile);
    const uint32_t o_col = tmem_base + lane_addr + kColO + (uint32_t)(st * kTile);
    float* part = reinterpret_cast<float*>(a.ws + kWsMemory);
    const int64_t all_rows = (int64_t)a.L * a.T * Hq;
    float2* stat = reinterpret_cast<float2*>(a.ws + kWsMemory + memory_part_bytes(all_rows, max_splits));
    uint32_t sn = 0, on = 0;  // score tiles and units so far
    bool ok = true;
    for (int64_t u = blockIdx.x; u < n_units && ok; u += gridDim.x) {
      const Unit x = unit_at(u);
      const int t0 = x.t0[st], n = x.t1[st] - t0;
      const bool mine = r / G < x.n_tok[st];
      const int64_t row = x.slot[st] * all_rows + ((int64_t)x.l * a.T + x.tok[st] + r / G) * Hq + x.h * G + r % G;
      float m = -INFINITY, sum = 0.f;
      for (int j = 0; j < n; ++j) {
        if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&s_ready[st]), sn & 1u, abort_flag))) {
          ok = false;
          break;
        }
        ++sn;
        tc_fence_after();
        uint32_t sv[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(s_col + 32 * c, sv[c]);
        tmem_wait_ld();
        const int valid = x.M - (t0 + j) * kTile;
        if (valid < kTile) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (32 * c + e >= valid) sv[c][e] = 0xFF800000u;
        }
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int e = 0; e < 32; ++e) mx = fmaxf(mx, __uint_as_float(sv[c][e]));
        mx *= a.qscale;  // (qscale > 0)
        const bool need = mx > m + kHeadroom;
        if (__any_sync(0xffffffffu, need)) {
          const float alpha = need ? ex2_ftz(m - mx) : 1.f;  // 0 while m is still -inf
          if (need) m = mx;
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
        float add[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pw[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const uint32_t s0 = sv[2 * c + (e >> 4)][2 * (e & 15)], s1 = sv[2 * c + (e >> 4)][2 * (e & 15) + 1];
            const float p0 = ex2_ftz(fmaf(__uint_as_float(s0), a.qscale, -base));
            const float p1 = ex2_ftz(fmaf(__uint_as_float(s1), a.qscale, -base));
            add[2 * (e & 1)] += p0;
            add[2 * (e & 1) + 1] += p1;
            pw[e] = msa::float2_to_bf16x2(p0, p1);
          }
          tmem_st32(s_col + 32 * c, pw);
        }
        sum += (add[0] + add[1]) + (add[2] + add[3]);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&p_ready[st]));
      }
      if (!ok) break;
      if (n > 0) {
        if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&o_done[st]), on & 1u, abort_flag))) {
          ok = false;
          break;
        }
        ++on;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32];
          tmem_ld32(o_col + 32 * c, o);
          tmem_wait_ld();
          if (mine) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float w[8];
#pragma unroll
              for (int v = 0; v < 8; ++v) w[v] = __uint_as_float(o[8 * e + v]);
              st_global_v8(part + row * kD + 32 * c + 8 * e, w);
            }
          }
        }
        tc_fence_before();  // (O is read: the next unit's first PV may overwrite it)
      }
      if (mine) stat[row] = make_float2(m, sum);  // (no tiles: -inf and 0)
    }
    if (!ok) {
      *abort_flag = 1;
      if (lane == 0) msa::set_err(a.dev_err, MSA_DEVERR_TIMEOUT);
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

// bf16 rows of 128 elements, box [64 rows][64 elements], 128-byte swizzle; rows past the end
// read as zero
bool make_kv_map(CUtensorMap* m, const void* base, uint64_t rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)kD, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)kD * 2};
  const cuuint32_t box[2] = {(cuuint32_t)kHalf, (cuuint32_t)kBox};
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

template <int G>
cudaError_t launch_memory_t(const Attend& a, int max_splits, cudaStream_t s) {
  CUtensorMap tm_q, tm_kv;
  if (!make_q_map(&tm_q, a.q, a.H * G, a.T, a.L, G) ||
      !make_kv_map(&tm_kv, a.mem_kv, (uint64_t)a.NG * a.L * 2 * a.H * a.M_max))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(memory_kernel<G>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemTc);
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
  return cudaLaunchKernelEx(&cfg, memory_kernel<G>, tm_q, tm_kv, a, max_splits);
}

}  // namespace

cudaError_t launch_memory(const Attend& a, int max_splits, cudaStream_t s) {
  switch (a.G) {
    case 1: return launch_memory_t<1>(a, max_splits, s);
    case 2: return launch_memory_t<2>(a, max_splits, s);
    case 4: return launch_memory_t<4>(a, max_splits, s);
    default: return launch_memory_t<8>(a, max_splits, s);
  }
}

}  // namespace paged
