// Shared-memory attention of a paged batch, few rows at a time: what msa_shared_attend
// defines (msa_paged.h), on mma.sync.
//
// Follows "MSA端到端可训练记忆模型完整开源，支持亿级Token上下文", section 架构 (softmax over the
// selected memory joined to the local K/V), and the MSA paper reading notes, section
// 推理全流程.
//
// A unit is up to R (8 or 16) rows, R / G consecutive new tokens x the G query heads of key
// head h, of one sequence and layer, against all keys they can see: the group's memory rows,
// then the sequence's page rows.  Its keys are cut into tiles of 16.  All tiles of all units,
// in the order (sequence, layer, key head, row tile, key tile), form one line that is cut
// into equal pieces, one per warp of the grid (one 8-warp CTA per SM), so that ragged lengths
// do not leave SMs idle and a single long sequence is spread over all of them.  A unit takes
// six tiles more on the line than it has (its queries, join and output cost about that; nine where
// the memory kernel's results are joined too).
//
// Each warp streams its tiles through its own 3-stage cp.async ring in shared memory (16 K
// rows and 16 V rows a stage, 16-byte chunks XOR-swizzled by row so ldmatrix is
// conflict-free), running on from unit to unit.  Per tile: S = Q K^T and O += P V as
// m16n8k16 (bf16 in, fp32 accumulate).  The queries are exact bf16 operands.  With R = 8 the
// weights are split into a bf16 value and a bf16 residual (about 16 bits), which rides in the
// MMA's spare rows; with R = 16 they are rounded to bf16 (half a step, 2^-8 of each, as in the
// tile kernel), since a residual would double the PV's MMAs.  Online softmax per row in the log2
// domain, the running maximum raised (and O rescaled) only when a score exceeds it by 2^8.
//
// A unit that lies inside one warp's piece is written out at its end.  A unit cut between
// warps leaves (max, sum, unnormalised output) per piece in the workspace; the last warp to
// arrive (a counter that it resets) joins the pieces in their order along the line, so the
// result does not depend on the order of arrival.
//
// Measured on one B200: 128 answers of 215 page rows on average, 18 layers, 32 / 8 heads: 2.0 GB of
// pages in 345 us (5.9 TB/s, 0.9 of the copy rate); one token over 256 + 320 keys, 18 layers (42
// MB): 18 us.  With many tiles a warp HBM bounds it; with few the chain of a launch does (tables,
// page ids, first keys, joins), and otherwise the warps' own latencies: 420 instructions a tile at
// two warps a scheduler take about 1,750 cycles.
#include <algorithm>

#include "attn_common.cuh"
#include "paged.cuh"

namespace paged {
namespace {
using namespace attn;

constexpr int kThreads = kRowWarps * 32;
constexpr int kTileKeys = 16;
constexpr int kStages = 3;
constexpr int kRowBytes = kD * 2;
constexpr int kStageBytes = 2 * kTileKeys * kRowBytes;  // 16 K rows, then 16 V rows
constexpr int kRingBytes = kRowWarps * kStages * kStageBytes;
constexpr int kMinTiles = 2;  // tiles per warp below which a unit is not cut further
constexpr float kHeadroom = 8.0f; // log2 growth of a row's maximum tolerated before rescaling

// The tables of the batch in shared memory.
struct Tables {
  int64_t scan[kMaxSeqs + 1];  // tiles of sequences before b, in units of one (layer, key head)
  int tok0[kMaxSeqs + 1];      // first token (the offsets as given)
  int n[kMaxSeqs];             // new tokens
  int len[kMaxSeqs];           // rows with the new tokens, as given
  int grp[kMaxSeqs];           // group, or -1
  int gmt[kMaxSeqs];           // memory tiles of a group's longest layer (PART: partial slots per split)
  int goff[kMaxSeqs + 1];      // group offsets
  int64_t warp_sum[kRowWarps];
  int by_sequence;             // PART: the memory kernel took each sequence's tokens by themselves
};

// Whether this lane's eighth of a warp's 16 bf16 rows at `st` holds an infinity or a NaN.
__device__ __forceinline__ bool not_finite(uint32_t st, int lane) {
  bool bad = false;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    uint32_t w[4];
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(st + (u * 32 + lane) * 16));
#pragma unroll
    for (int e = 0; e < 4; ++e)
      bad |= (w[e] & 0x7F80u) == 0x7F80u || (w[e] & 0x7F800000u) == 0x7F800000u;
  }
  return bad;
}

// 16-byte global -> shared copy
__device__ __forceinline__ void cp_async16_full(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}

// PART: the memory part comes from the memory kernel's partial results.
template <int G, int NR, bool PART>
__global__ void __launch_bounds__(kThreads, 1)
    rows_kernel(const __grid_constant__ Attend a, int max_splits) {
  constexpr int R = 8 * NR;       // rows of a unit
  constexpr int kTok = R / G;     // tokens of a unit
  constexpr int kUnitTicks = PART ? 9 : 6;  // what a unit costs beyond its tiles (queries in, joins, output), in tiles
  extern __shared__ __align__(128) unsigned char smem_raw[];
  Tables& tb = *reinterpret_cast<Tables*>(smem_raw + kRingBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int Hq = a.H * G, LH = a.L * a.H;
  const int page_mask = (1 << a.log2_page) - 1;
  const int64_t cap = (int64_t)a.max_pages << a.log2_page;

  // With PART this kernel follows the memory kernel, which lets it start once every one of its
  // CTAs has seen all earlier kernels complete: only the memory kernel itself is still to be
  // waited for, before its results are read (and before this kernel ends, so that whoever
  // waits for this one has waited for both).
  if (!PART) wait_for_earlier_kernels();
  let_next_kernel_start();

  // ---- tables (a thread's first entries of all they read are on their way at once)
  const int g_first = a.NG > 0 && tid <= a.NG ? a.group_offsets[tid] : 0;
  int lo_first = 0, hi_first = 0, len_first = 0;
  if (tid < a.B) {
    lo_first = a.q_offsets[tid];
    hi_first = a.q_offsets[tid + 1];
    len_first = a.seq_len[tid];
  }
  int ml[2];  // memory rows of (group, layer)
  if (!PART) {
#pragma unroll
    for (int i = 0; i < 2; ++i) ml[i] = tid + i * kThreads < a.NG * a.L ? a.mem_len[tid + i * kThreads] : 0;
  }
  for (int g = tid; g <= a.NG; g += kThreads) {
    tb.goff[g] = g == tid ? g_first : a.group_offsets[g];
    if (g < a.NG) tb.gmt[g] = 0;
  }
  bool ok = true;  // all offsets are usable
  for (int b = tid; b < a.B; b += kThreads) {
    const int lo = b == tid ? lo_first : a.q_offsets[b], hi = b == tid ? hi_first : a.q_offsets[b + 1];
    const int len = b == tid ? len_first : a.seq_len[b];
    const bool usable = lo >= 0 && hi >= lo && hi <= a.T;
    const int n = usable ? hi - lo : 0;
    ok &= usable;
    if (blockIdx.x == 0 && n > 0 && len > cap) msa::set_err(a.dev_err, MSA_DEVERR_LOCAL_FULL);
    tb.tok0[b] = lo;
    if (b == a.B - 1) tb.tok0[a.B] = hi;
    tb.n[b] = n;
    tb.len[b] = len;
    tb.grp[b] = -1;
  }
  __syncthreads();
  for (int g = tid; g < a.NG; g += kThreads) {
    const int s = tb.goff[g], e = tb.goff[g + 1];
    ok &= s >= 0 && e >= s && e <= a.B;
  }
  if (!PART) {
    for (int i = tid; i < a.NG * a.L; i += kThreads) {
      int m = i == tid ? ml[0] : i == tid + kThreads ? ml[1] : a.mem_len[i];
      if (m > a.M_max) {
        if (blockIdx.x == 0) msa::set_err(a.dev_err, MSA_DEVERR_CAPACITY);
        m = a.M_max;
      }
      if (m > 0) atomicMax(&tb.gmt[i / a.L], (m + kTileKeys - 1) / kTileKeys);
    }
  }
  const bool offsets_ok = __syncthreads_and(ok);
  if (!offsets_ok && blockIdx.x == 0 && tid == 0) msa::set_err(a.dev_err, MSA_DEVERR_BAD_OFFSETS);
  if (tid == 0) tb.by_sequence = !offsets_ok;
  for (int gr = warp; gr < a.NG; gr += kRowWarps) {
    const int s = tb.goff[gr], e = tb.goff[gr + 1];
    if (!offsets_ok) {
      // each usable group by itself; of several that hold a sequence the last (in every CTA: the
      // pieces of the line have to agree)
      for (int b = s + lane; s >= 0 && e <= a.B && b < e; b += 32) atomicMax(&tb.grp[b], gr);
    } else if (PART) {
      for (int b = s + lane; b < e; b += 32) tb.grp[b] = gr;
      // partial slots per split: two where the group's rows fit one row tile
      if (lane == 0) tb.gmt[gr] = tb.tok0[e] - tb.tok0[s] <= 128 / G ? 2 : 1;
    } else {
      for (int b = s + lane; b < e; b += 32) tb.grp[b] = gr;
    }
  }
  __syncthreads();
  // tiles of sequence b per (layer, key head): row tiles x key tiles (at least one, so that a
  // unit without any key still writes its zeros)
  auto memory_tiles = [&](int b) -> int { return PART || tb.grp[b] < 0 ? 0 : tb.gmt[tb.grp[b]]; };
  auto key_tiles = [&](int b, int mt) -> int {
    const int64_t len = min((int64_t)max(tb.len[b], 0), cap);
    return max(1, mt + (int)((len + kTileKeys - 1) / kTileKeys));
  };
  auto row_tiles = [&](int b) -> int { return (tb.n[b] + kTok - 1) / kTok; };
  {
    constexpr int kPer = kMaxSeqs / kThreads;
    int64_t v[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = tid * kPer + i;
      v[i] = sum;
      if (b < a.B) {
        sum += (int64_t)row_tiles(b) * (key_tiles(b, memory_tiles(b)) + kUnitTicks);
      }
    }
    int64_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) tb.warp_sum[warp] = inc;
    __syncthreads();
    int64_t base = inc - sum;
    for (int w = 0; w < warp; ++w) base += tb.warp_sum[w];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = tid * kPer + i;
      if (b < a.B) tb.scan[b] = base + v[i];
    }
    if (tid == kThreads - 1) tb.scan[a.B] = base + sum;
  }
  __syncthreads();

  // ---- this warp's piece of the line
  const int workers = gridDim.x * kRowWarps;
  const int worker = blockIdx.x * kRowWarps + warp;
  const int64_t total = tb.scan[a.B] * LH;
  // (64-bit divisions cost hundreds of cycles before the first load)
  auto divide = [](int64_t x, int64_t y) -> int64_t {
    return (uint64_t)(x | y) >> 32 ? x / y : (int64_t)((uint32_t)x / (uint32_t)y);
  };
  const int64_t per = max((int64_t)kMinTiles, divide(total + workers - 1, workers));
  const int64_t w0 = worker * per, w1 = min(total, w0 + per);
  if (w0 >= w1) {
    if (PART) wait_for_earlier_kernels();
    return;
  }

  struct Cursor {
    int b, lh, rt, j;       // sequence, layer x H + key head, row tile, key tile
    int RT, nt, mt;         // row tiles, key tiles, memory tiles of the sequence
    int l, h, M;            // layer, key head, the group's memory rows in this layer
    int len, cut;           // page rows (clamped), rows minus new tokens (token 0 sees row `cut`)
  };
  auto set_layer = [&](Cursor& c) {
    c.l = c.lh / a.H;
    c.h = c.lh - c.l * a.H;
    c.M = 0;
    if (!PART && c.mt > 0) c.M = max(0, min(a.M_max, a.mem_len[(int64_t)tb.grp[c.b] * a.L + c.l]));
  };
  auto set_sequence = [&](Cursor& c) {
    c.RT = row_tiles(c.b);
    c.mt = memory_tiles(c.b);
    c.nt = key_tiles(c.b, c.mt);
    c.len = (int)min((int64_t)max(tb.len[c.b], 0), cap);
    c.cut = max(tb.len[c.b], 0) - tb.n[c.b];
  };
  // the unit after this one (the caller stays within the line)
  auto next_unit = [&](Cursor& c) {
    c.j = 0;
    if (++c.rt < c.RT) return;
    c.rt = 0;
    if (++c.lh < LH) {
      set_layer(c);
      return;
    }
    c.lh = 0;
    do ++c.b; while (c.b < a.B && tb.n[c.b] == 0);
    if (c.b >= a.B) {  // (past the line's end: nothing is read through this cursor again)
      c.b = a.B - 1;
      return;
    }
    set_sequence(c);
    set_layer(c);
  };
  Cursor c;
  int64_t at = w0;  // the position of cursor c on the line
  {
    int lo = 0, hi = a.B;  // scan[lo] * LH <= w0 < scan[hi] * LH
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tb.scan[mid] * LH <= w0) lo = mid; else hi = mid;
    }
    c.b = lo;
    set_sequence(c);
    const int64_t rem = w0 - tb.scan[lo] * LH, unit = c.nt + kUnitTicks, each = c.RT * unit;
    c.lh = (int)divide(rem, each);
    const int64_t in = rem - c.lh * each;
    c.rt = (int)divide(in, unit);
    c.j = (int)(in - (int64_t)c.rt * unit);
    set_layer(c);
    if (c.j >= c.nt) {  // behind the unit's last tile
      at += unit - c.j;
      next_unit(c);
    }
  }
  Cursor pc = c;  // the loads run ahead of the arithmetic
  int64_t pat = at;

  const uint32_t my_ring = smem_u32(smem_raw) + warp * (kStages * kStageBytes);
  // page ids of 32 consecutive tiles of a sequence, one per lane
  int ids_b = -1, ids_win = -1, ids = 0;
  uint32_t bad = 0u;  // stages whose page id is unusable

  // where this lane's 16 bytes of rows 2 u and 2 u + 1 go, beyond u x 512 bytes (u modulo 4)
  uint32_t to[4];
#pragma unroll
  for (int q = 0; q < 4; ++q)
    to[q] = (lane >> 4) * kRowBytes + (((lane & 15) ^ ((2 * q + (lane >> 4)) & 7)) << 4);

  auto issue = [&](int i) {
    const int stage = i % kStages;
    const __nv_bfloat16 *kp, *vp;
    int rows;
    bad &= ~(1u << stage);
    if (!PART && pc.j < pc.mt) {
      const int64_t row = (((int64_t)tb.grp[pc.b] * a.L + pc.l) * 2 * a.H + pc.h) * a.M_max + pc.j * kTileKeys;
      kp = a.mem_kv + row * kD;
      vp = kp + (int64_t)a.H * a.M_max * kD;
      rows = pc.M - pc.j * kTileKeys;
    } else {
      const int jj = pc.j - pc.mt;
      if (ids_b != pc.b || ids_win != (jj >> 5)) {
        ids_b = pc.b;
        ids_win = jj >> 5;
        const int64_t row = (int64_t)((ids_win << 5) + lane) * kTileKeys;
        ids = row < pc.len ? a.page_table[(int64_t)pc.b * a.max_pages + (row >> a.log2_page)] : 0;
      }
      const int id = __shfl_sync(0xffffffffu, ids, jj & 31);
      rows = pc.len - jj * kTileKeys;
      if (id < 0 || id >= a.NP) {
        if (rows > 0) {
          bad |= 1u << stage;
          if (lane == 0) msa::set_err(a.dev_err, MSA_DEVERR_BAD_PAGE);
        }
        rows = 0;
        kp = vp = a.pages;
      } else {
        const int64_t row =
            ((((int64_t)pc.l * a.NP + id) * 2 * a.H + pc.h) << a.log2_page) + ((jj * kTileKeys) & page_mask);
        kp = a.pages + row * kD;
        vp = kp + ((int64_t)a.H << a.log2_page) * kD;
      }
    }
    // instruction u: rows 2 u and 2 u + 1 of the keys, then of the values (a half warp each)
    const uint32_t st = my_ring + stage * kStageBytes;
    const __nv_bfloat16 *ks = kp + lane * 8, *vs = vp + lane * 8;
    if (rows >= kTileKeys) {
#pragma unroll
      for (int u = 0; u < 8; ++u) cp_async16_full(st + to[u & 3] + u * 512, ks + u * 256);
#pragma unroll
      for (int u = 0; u < 8; ++u) cp_async16_full(st + to[u & 3] + (u + 8) * 512, vs + u * 256);
    } else {
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const bool ok = 2 * u + (lane >> 4) < rows;
        cp_async16(st + to[u & 3] + u * 512, ok ? ks + u * 256 : kp, ok ? 16u : 0u);
        cp_async16(st + to[u & 3] + (u + 8) * 512, ok ? vs + u * 256 : vp, ok ? 16u : 0u);
      }
    }
    ++pat;
    if (++pc.j == pc.nt) {
      pat += kUnitTicks;
      next_unit(pc);
    }
  };

#pragma unroll
  for (int p = 0; p < kStages; ++p) {
    if (pat < w1) issue(p);
    cp_async_commit();
  }

  uint32_t qa[8][2 * NR];
  float o[16][4];
  float m[NR], lsum[NR];
  int lim[NR];  // the last page row that this thread's rows see
  bool fresh = true, memory_done = false;
  int64_t u0 = at - c.j;  // the unit's first tile on the line

  // a row's token within the sequence, and its place among the rows of q and out
  auto row_token = [&](int r) -> int { return c.rt * kTok + r / G; };
  auto row_at = [&](int r) -> int64_t {
    return (((int64_t)c.l * a.T + tb.tok0[c.b] + row_token(r)) * Hq + c.h * G + r % G) * kD;
  };

  for (int i = 0; at < w1; ++i) {
    if (fresh) {  // a new unit: its queries (row g in words 0 and 1 of the A fragment, row g + 8)
      fresh = false;
#pragma unroll
      for (int v = 0; v < NR; ++v) {
        const int r = g + 8 * v;
        const bool ok = row_token(r) < tb.n[c.b];
        const __nv_bfloat16* qp = a.q + (ok ? row_at(r) : 0) + 2 * t;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          qa[ks][2 * v] = ok ? *reinterpret_cast<const uint32_t*>(qp + 16 * ks) : 0u;
          qa[ks][2 * v + 1] = ok ? *reinterpret_cast<const uint32_t*>(qp + 16 * ks + 8) : 0u;
        }
        lim[v] = min(c.cut + row_token(r), c.len - 1);
        m[v] = -INFINITY;
        lsum[v] = 0.f;
      }
#pragma unroll
      for (int n = 0; n < 16; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    }
    cp_async_wait<kStages - 1>();  // (3 + i groups committed: tile i has landed)
    __syncwarp();
    const int stage = i % kStages;
    const uint32_t st = my_ring + stage * kStageBytes;
    const bool mem = !PART && c.j < c.mt;
    // keys of this tile below `top` are seen: the same for all rows of a memory tile
    const int key0 = mem ? c.j * kTileKeys : (c.j - c.mt) * kTileKeys;
    int top[NR];
    int most = 0;
#pragma unroll
    for (int v = 0; v < NR; ++v) {
      top[v] = mem ? c.M - key0 : ((bad >> stage) & 1u) ? 0 : lim[v] + 1 - key0;
      most = max(most, top[v]);
    }
    if (__any_sync(0xffffffffu, most > 0)) {
      // two accumulators per 8-key half (even / odd k-steps) keep the MMA chains short
      float s[2][2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int u = 0; u < 2; ++u) s[j][u][0] = s[j][u][1] = s[j][u][2] = s[j][u][3] = 0.f;
      }
#pragma unroll
      for (int ks2 = 0; ks2 < 4; ++ks2) {
        uint32_t a0[4], a1[4];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          a0[2 * w] = qa[2 * ks2][w];
          a0[2 * w + 1] = NR == 2 ? qa[2 * ks2][NR * 2 - 2 + w] : 0u;
          a1[2 * w] = qa[2 * ks2 + 1][w];
          a1[2 * w + 1] = NR == 2 ? qa[2 * ks2 + 1][NR * 2 - 2 + w] : 0u;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int row = 8 * j + (lane & 7);
          const int chunk = 4 * ks2 + (lane >> 3);
          uint32_t b0, b1, b2, b3;
          ldsm_x4(st + row * kRowBytes + ((chunk ^ (row & 7)) << 4), b0, b1, b2, b3);
          mma_bf16(s[j][0], a0, b0, b1);
          mma_bf16(s[j][1], a1, b2, b3);
        }
      }
      float pr[NR][4];
      float alpha[NR];
      bool rescale = false;
#pragma unroll
      for (int v = 0; v < NR; ++v) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int key = 8 * j + 2 * t + e;
            pr[v][2 * j + e] = key < top[v] ? (s[j][0][2 * v + e] + s[j][1][2 * v + e]) * a.qscale : -INFINITY;
          }
        }
        float mx = fmaxf(fmaxf(pr[v][0], pr[v][1]), fmaxf(pr[v][2], pr[v][3]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float m_new = mx > m[v] + kHeadroom ? mx : m[v];
        const float base = m_new == -INFINITY ? 0.f : m_new;  // (a row that has seen no key yet)
        alpha[v] = m_new == m[v] ? 1.f : ex2_ftz(m[v] - base);  // 0 while m is still -inf
#pragma unroll
        for (int u = 0; u < 4; ++u) pr[v][u] = ex2_ftz(pr[v][u] - base);
        lsum[v] = fmaf(lsum[v], alpha[v], (pr[v][0] + pr[v][1]) + (pr[v][2] + pr[v][3]));
        m[v] = m_new;
        rescale |= alpha[v] != 1.f;
      }
      if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll
        for (int n = 0; n < 16; ++n) {
          o[n][0] *= alpha[0];
          o[n][1] *= alpha[0];
          o[n][2] *= alpha[NR - 1];
          o[n][3] *= alpha[NR - 1];
        }
      }
      // A fragments of the weights: {row g keys 2t.., row g + 8 keys 2t.., the same for keys + 8}
      uint32_t pa[4];
      if (NR == 1) {  // residuals in rows 8..15
        split_pair(pr[0][0], pr[0][1], pa[0], pa[1]);
        split_pair(pr[0][2], pr[0][3], pa[2], pa[3]);
      } else {
        pa[0] = msa::float2_to_bf16x2(pr[0][0], pr[0][1]);
        pa[1] = msa::float2_to_bf16x2(pr[NR - 1][0], pr[NR - 1][1]);
        pa[2] = msa::float2_to_bf16x2(pr[0][2], pr[0][3]);
        pa[3] = msa::float2_to_bf16x2(pr[NR - 1][2], pr[NR - 1][3]);
      }
      const int vrow = kTileKeys + (lane & 7) + 8 * ((lane >> 3) & 1);
      // O += P V, in the rows of token `only` alone if that is >= 0
      auto add_pv = [&](int only) {
        const bool r0 = only < 0 || g / G == only;
        const bool r1 = only < 0 || (NR == 2 ? (g + 8) / G == only : r0);  // (NR = 1: row g's residuals)
#pragma unroll
        for (int i2 = 0; i2 < 8; ++i2) {
          const int chunk = 2 * i2 + (lane >> 4);
          uint32_t v[4];
          ldsm_x4_t(st + vrow * kRowBytes + ((chunk ^ (vrow & 7)) << 4), v[0], v[1], v[2], v[3]);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            float(&d)[4] = o[2 * i2 + u];
            float x[4] = {d[0], d[1], d[2], d[3]};
            mma_bf16(x, pa, v[2 * u], v[2 * u + 1]);
            d[0] = r0 ? x[0] : d[0];
            d[1] = r0 ? x[1] : d[1];
            d[2] = r1 ? x[2] : d[2];
            d[3] = r1 ? x[3] : d[3];
          }
        }
      };
      // a tile with rows that the unit's first token does not see (later new tokens): a value
      // that is not finite must not reach the rows that do not see it (0 x inf is NaN)
      const int n_tok = min(kTok, tb.n[c.b] - c.rt * kTok);
      bool poison = false;
      if (!mem && c.cut + c.rt * kTok < min(key0 + kTileKeys, c.len) - 1)
        poison = __any_sync(0xffffffffu, not_finite(st + kTileKeys * kRowBytes, lane));
      if (!poison) {
        add_pv(-1);
      } else {
        // one token at a time, the last first, clearing the value rows that it does not see
        for (int tk = n_tok - 1; tk >= 0; --tk) {
          const int seen = min(c.cut + c.rt * kTok + tk, c.len - 1) + 1 - key0;
          for (int r = max(seen, 0); r < kTileKeys; ++r)
            if (lane < 16)
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};\n" ::"r"(st + (kTileKeys + r) * kRowBytes + lane * 16),
                           "r"(0u)
                           : "memory");
          __syncwarp();
          add_pv(tk);
          __syncwarp();
        }
      }
    }
    __syncwarp();  // every lane is done with the stage: refill it with tile i + 3
    if (pat < w1) issue(i + kStages);
    cp_async_commit();

    const bool unit_end = c.j + 1 == c.nt;
    ++at;
    if (unit_end || at == w1) {
      // ---- the unit (or this piece of it) is done
      float sum[NR];
#pragma unroll
      for (int v = 0; v < NR; ++v) {
        sum[v] = lsum[v];
        sum[v] += __shfl_xor_sync(0xffffffffu, sum[v], 1);
        sum[v] += __shfl_xor_sync(0xffffffffu, sum[v], 2);
      }
      if (NR == 1) {
        // (an infinite value times a residual of zero or below zero would make the row's infinity a NaN)
#pragma unroll
        for (int n = 0; n < 16; ++n) {
          o[n][0] += fabsf(o[n][0]) < INFINITY ? o[n][2] : 0.f;
          o[n][1] += fabsf(o[n][1]) < INFINITY ? o[n][3] : 0.f;
        }
      }
      // Joins `n` partial results (place(i, r): of row r the i-th one's index) to what the rows
      // hold.  With fewer than eight rows several of the eight quads of lanes share a row: of its
      // `share` quads, number `mine` takes the places mine, mine + share, ...
      const int valid = min(kTok, tb.n[c.b] - c.rt * kTok) * G;
      const int vr = valid > 4 ? 8 : valid > 2 ? 4 : valid;
      const int share = 8 / vr, mine = g / vr;
      auto join = [&](int n_places, const float2* stat, const float* part, auto place) {
#pragma unroll
        for (int v = 0; v < NR; ++v) {
          if (v > 0 && valid <= 8) break;
          const int r = (g & (vr - 1)) + 8 * v;
          const int n_mine = r < valid ? n_places : 0;
          float top = __shfl_sync(0xffffffffu, m[v], ((g & (vr - 1)) << 2) | t);
          for (int s = mine * 4 + t; s < n_mine; s += 4 * share) top = fmaxf(top, __ldcg(&stat[place(s, r)]).x);
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          for (int o2 = 4 * vr; o2 < 32; o2 <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o2));
          const float base = top == -INFINITY ? 0.f : top;
          const float own = ex2_ftz(m[v] - base);
          sum[v] = mine == 0 ? sum[v] * own : 0.f;
#pragma unroll
          for (int n = 0; n < 16; ++n) {
            o[n][2 * v] = mine == 0 ? o[n][2 * v] * own : 0.f;
            o[n][2 * v + 1] = mine == 0 ? o[n][2 * v + 1] * own : 0.f;
          }
          m[v] = top;
#pragma unroll 2
          for (int s = mine; s < n_mine; s += share) {
            const int64_t at_s = place(s, r);
            const float2 ml = __ldcg(&stat[at_s]);
            const bool use = ml.y != 0.f;  // (where no key was seen the output may not be written)
            const float f = use ? ex2_ftz(ml.x - base) : 0.f;
            float4 x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
              x[k] = use ? __ldcg(reinterpret_cast<const float4*>(part + at_s * kD + 16 * k + 4 * t)) : make_float4(0.f, 0.f, 0.f, 0.f);
            sum[v] = fmaf(f, ml.y, sum[v]);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              o[2 * k][2 * v] = fmaf(f, x[k].x, o[2 * k][2 * v]);
              o[2 * k][2 * v + 1] = fmaf(f, x[k].y, o[2 * k][2 * v + 1]);
              o[2 * k + 1][2 * v] = fmaf(f, x[k].z, o[2 * k + 1][2 * v]);
              o[2 * k + 1][2 * v + 1] = fmaf(f, x[k].w, o[2 * k + 1][2 * v + 1]);
            }
          }
          for (int o2 = 4 * vr; o2 < 32; o2 <<= 1) {
            sum[v] += __shfl_xor_sync(0xffffffffu, sum[v], o2);
#pragma unroll
            for (int n = 0; n < 16; ++n) {
              o[n][2 * v] += __shfl_xor_sync(0xffffffffu, o[n][2 * v], o2);
              o[n][2 * v + 1] += __shfl_xor_sync(0xffffffffu, o[n][2 * v + 1], o2);
            }
          }
        }
      };
      bool write = true;
      const int64_t u1 = u0 + c.nt;
      if (u0 < w0 || u1 > w1) {
        // a cut unit: pieces belong to workers first .. last; the piece at a worker's start
        // (a unit begun before it) goes to slot 2 w, the one it begins to slot 2 w + 1
        const int first = (int)divide(u0, per), last = (int)divide(u1 - 1, per);
        float2* stat = reinterpret_cast<float2*>(a.ws + kWsStat);
        float* part = reinterpret_cast<float*>(a.ws + kWsPart);
        int* counter = reinterpret_cast<int*>(a.ws + kWsCounters) + first;
        const int64_t slot = 2 * (int64_t)worker + (u0 < w0 ? 0 : 1);
#pragma unroll
        for (int v = 0; v < NR; ++v) {
          const int r = g + 8 * v;
          if (r < valid) {
            float* dst = part + (slot * 16 + r) * kD + 4 * t;  // (the order that `join` reads)
#pragma unroll
            for (int k = 0; k < 8; ++k)
              __stcg(reinterpret_cast<float4*>(dst + 16 * k),
                     make_float4(o[2 * k][2 * v], o[2 * k][2 * v + 1], o[2 * k + 1][2 * v], o[2 * k + 1][2 * v + 1]));
            if (t == 0) __stcg(&stat[slot * 16 + r], make_float2(m[v], sum[v]));
          }
        }
        __threadfence();
        __syncwarp();
        int old = 0;
        if (lane == 0) old = atomicAdd(counter, 1);
        old = __shfl_sync(0xffffffffu, old, 0);
        write = old == last - first;
        if (write) {
          __threadfence();
          if (lane == 0) *counter = 0;  // ready for the next call
#pragma unroll
          for (int v = 0; v < NR; ++v) {
            m[v] = -INFINITY;
            sum[v] = 0.f;
#pragma unroll
            for (int n = 0; n < 16; ++n) o[n][2 * v] = o[n][2 * v + 1] = 0.f;
          }
          join(last - first + 1, stat, part, [&](int i, int r) -> int64_t { return (2 * (int64_t)(first + i) + (i == 0)) * 16 + r; });
        }
      }
      if (PART && write && tb.grp[c.b] >= 0) {
        // join the memory part: its slots in order, then this sequence's rows
        if (!memory_done) {
          wait_for_earlier_kernels();
          memory_done = true;
        }
        const int per_split = tb.by_sequence ? (tb.n[c.b] <= 128 / G ? 2 : 1) : tb.gmt[tb.grp[c.b]];
        const int slots = __ldcg(reinterpret_cast<const int*>(a.ws + kWsSplits)) * per_split;
        const int64_t all_rows = (int64_t)a.L * a.T * Hq;
        join(slots, reinterpret_cast<const float2*>(a.ws + kWsMemory + memory_part_bytes(all_rows, max_splits)),
             reinterpret_cast<const float*>(a.ws + kWsMemory),
             [&](int s, int r) -> int64_t { return s * all_rows + row_at(r) / kD; });
      }
      if (write) {
#pragma unroll
        for (int v = 0; v < NR; ++v) {
          const int r = g + 8 * v;
          if (row_token(r) < tb.n[c.b]) {
            // (no key seen: sum 0, output 0; a NaN sum is kept)
            const float inv = sum[v] == 0.f ? 0.f : 1.f / sum[v];
            __nv_bfloat16* dst = a.out + row_at(r) + 2 * t;
#pragma unroll
            for (int n = 0; n < 16; ++n)
              *reinterpret_cast<uint32_t*>(dst + 8 * n) =
                  msa::float2_to_bf16x2(o[n][2 * v] * inv, o[n][2 * v + 1] * inv);
          }
        }
      }
      at += kUnitTicks;  // (past w1 where the piece ends within the unit)
      if (at < w1) {
        u0 = at;
        next_unit(c);
        fresh = true;
      }
    } else {
      ++c.j;
    }
  }
  cp_async_wait<0>();
  if (PART && !memory_done) wait_for_earlier_kernels();
}

template <int G, int NR, bool PART>
cudaError_t launch_rows_t(const Attend& a, int memory_splits, cudaStream_t s) {
  constexpr int kSmem = kRingBytes + (int)sizeof(Tables);
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_shared_memory(reinterpret_cast<const void*>(rows_kernel<G, NR, PART>), kSmem, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(std::min(msa::sm_count(), kRowCtas), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rows_kernel<G, NR, PART>, a, memory_splits);
}

// Eight rows where the sequences have at most eight on average (their weights' residuals then
// cost no MMA of their own), sixteen otherwise.
template <int G>
cudaError_t launch_rows_g(const Attend& a, int memory_splits, cudaStream_t s) {
  const bool few = (int64_t)a.T * a.G <= 8 * (int64_t)a.B;
  if (memory_splits > 0) return few ? launch_rows_t<G, 1, true>(a, memory_splits, s) : launch_rows_t<G, 2, true>(a, memory_splits, s);
  return few ? launch_rows_t<G, 1, false>(a, 0, s) : launch_rows_t<G, 2, false>(a, 0, s);
}

}  // namespace

cudaError_t launch_rows(const Attend& a, int memory_splits, cudaStream_t s) {
  switch (a.G) {
    case 1: return launch_rows_g<1>(a, memory_splits, s);
    case 2: return launch_rows_g<2>(a, memory_splits, s);
    case 4: return launch_rows_g<4>(a, memory_splits, s);
    default: return launch_rows_g<8>(a, memory_splits, s);
  }
}

}  // namespace paged
