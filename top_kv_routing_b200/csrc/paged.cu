// Paged batches: the append kernel and the entry points (the attention kernels are in
// paged_rows.cu).
//
// Follows "MSA端到端可训练记忆模型完整开源，支持亿级Token上下文", section 架构 (全局 RoPE: positions
// offset by k; local K/V joined to the selected memory), and the MSA paper reading notes,
// section 推理全流程 (the local KV grows while the memory stays fixed).
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "msa_paged.h"
#include "paged.cuh"

MSA_DEFINE_LAST_ERROR(msa_paged_last_error)

namespace {
using namespace paged;

constexpr int kHalf = 64;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kSharedRows = 16;
constexpr int kBlockRows = 64;
constexpr int64_t kMaxTensorRows = 0x7fffffff - 128;  // (TMA row coordinates are 32-bit)

// Which kernels a batch takes, by its average rows (tokens x G) per sequence and group (the
// split of the tokens over the sequences is known to the device alone; any split is computed
// correctly by every form).
struct Plan {
  enum Form { kRowsOnly, kMemory, kBlocks } form;
  int splits;  // memory form: most key splits
};
Plan plan_of(int64_t T, int64_t B, int64_t NG, int64_t L, int64_t Hq, int64_t H) {
  const int64_t G = Hq / H;
  // Blocks of new tokens that fill half a row tile: memory and pages in one walk.
  if (T * G >= kBlockRows * B) return {Plan::kBlocks, 0};
  // The memory once for a whole group, on the tensor cores, where its sequences share enough
  // rows; a group of one or two answers reads it sooner within the row kernel.
  if (NG > 0 && T * G > kSharedRows * NG) return {Plan::kMemory, memory_splits(L * T * Hq)};
  return {Plan::kRowsOnly, 0};
}

static thread_local int32_t g_launches = 0;

// RoPE frequencies in fixed point: step[j] = round(2^64 theta^(-2j/128) / (2 pi)), the
// rotation of frequency j per position in units of 2^-64 turns; the angle of position p is
// p * step[j] mod 2^64 turns (integer arithmetic: exact range reduction at any position).
struct RopeFreq {
  unsigned long long step[kHalf];
};

// The table of the thread's last theta (64 long double exponentials cost several
// microseconds of host time, as much as a one-token launch).
const RopeFreq& rope_freq(float theta) {
  static thread_local float last = 0.f;
  static thread_local RopeFreq rf;
  if (theta != last) {
    const long double log2_theta = log2l((long double)theta);
    for (int j = 0; j < kHalf; ++j) {
      const long double turns = exp2l(-2.0L * j / kD * log2_theta) / (2.0L * 3.14159265358979323846264338L);
      rf.step[j] = (unsigned long long)llroundl(ldexpl(turns, 64));
    }
    last = theta;
  }
  return rf;
}

// ---------------------------------------------------------------------------- append
// CTA (token tile, layer): warp w < TOK finds its token's sequence (a 32-way search of the
// offsets), its page slot, and the 64 angles of its position; then eight threads per head
// row rotate (query and key heads) or copy (value heads) 8 + 8 elements each.  The first
// rows are loaded before the position is known.  Bound by HBM: every byte moves once.
constexpr int kAppendThreads = 256;

struct AppendArgs {
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  const int32_t* off;
  int T, B, Hq, H;
  __nv_bfloat16* pages;
  int NP, log2_page;
  const int32_t* table;
  int max_pages;
  const int32_t* seq_len;
  const int32_t* pos_offset;
  int rope_pos_offset;
  __nv_bfloat16* q_rot;
  int32_t* dev_err;
  RopeFreq rf;
};

struct Eight {
  float x[8];
};
__device__ __forceinline__ Eight load8(const __nv_bfloat16* p) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  Eight r;
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = msa::bf16x2_to_float2(u[e]);
    r.x[2 * e] = f.x;
    r.x[2 * e + 1] = f.y;
  }
  return r;
}
__device__ __forceinline__ Eight load8(const float* p) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  return Eight{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const Eight& r) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(msa::float2_to_bf16x2(r.x[0], r.x[1]), msa::float2_to_bf16x2(r.x[2], r.x[3]),
                 msa::float2_to_bf16x2(r.x[4], r.x[5]), msa::float2_to_bf16x2(r.x[6], r.x[7]));
}

template <typename In, int TOK>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendArgs a) {
  __shared__ float2 s_cs[TOK][kHalf];
  __shared__ int64_t s_row[TOK];   // element offset of the token's row in key head 0, or -1
  __shared__ int s_own[TOK];       // the token belongs to a sequence
  const int l = blockIdx.y, t0 = blockIdx.x * TOK;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  wait_for_earlier_kernels();
  let_next_kernel_start();
  const int heads = a.Hq + 2 * a.H;
  const int items = heads * 8;
  const int p = tid & 7;  // dims 8p .. 8p + 7 and 64 + 8p .. (kAppendThreads is a multiple of 8)

  // row `idx / 8` of token t: a query, key or value head
  auto source = [&](int t, int head) -> const In* {
    const int64_t row = (int64_t)l * a.T + t;
    if (head < a.Hq) return static_cast<const In*>(a.q) + row * a.q_stride + head * kD;
    if (head < a.Hq + a.H) return static_cast<const In*>(a.k) + row * a.k_stride + (head - a.Hq) * kD;
    return static_cast<const In*>(a.v) + row * a.v_stride + (head - a.Hq - a.H) * kD;
  };
  // with no queries to rotate the walk starts at the keys
  const int first = a.q_rot ? 0 : a.Hq * 8;
  int idx = first + tid, ti = 0;
  auto wrap = [&]() {
    while (idx >= items && ti < TOK) {
      idx -= items - first;
      ++ti;
    }
  };
  wrap();
  Eight lo, hi;
  const bool have = ti < TOK && t0 + ti < a.T;
  if (have) {
    const In* src = source(t0 + ti, idx >> 3);
    lo = load8(src + 8 * p);
    hi = load8(src + kHalf + 8 * p);
  }
  if (warp < TOK) {
    const int t = t0 + warp;
    int b = t < a.T ? find_last(a.off, a.B, t, lane) : -1;
    int b0 = 0, n = 0;
    if (b >= 0 && (!sequence_tokens(a.off, b, a.T, b0, n) || t < b0 || t >= b0 + n)) b = -1;
    int64_t row = -1;
    if (b >= 0) {
      const long long r = (long long)a.seq_len[b] - n + (t - b0);
      const long long pos = (long long)a.rope_pos_offset + (a.pos_offset ? (long long)a.pos_offset[b] : 0ll) + r;
      uint32_t err = 0u;
      if (r < 0) {
        err = MSA_DEVERR_BAD_OFFSETS;
      } else if ((r >> a.log2_page) >= a.max_pages) {
        err = MSA_DEVERR_LOCAL_FULL;
      } else {
        const int page = a.table[(int64_t)b * a.max_pages + (r >> a.log2_page)];
        if (page < 0 || page >= a.NP) {
          err = MSA_DEVERR_BAD_PAGE;
        } else {
          row = ((((int64_t)l * a.NP + page) * 2 * a.H) << a.log2_page) + (r & ((1ll << a.log2_page) - 1));
          row *= kD;
        }
      }
      if (err && lane == 0 && l == 0) msa::set_err(a.dev_err, err);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = lane + 32 * e;
        // the top 32 bits of the angle, read as signed, are angle / pi in [-1, 1) x 2^31
        const int top = (int)(((unsigned long long)pos * a.rf.step[j]) >> 32);
        float sn, c;
        sincospif((float)top * 4.656612873077392578125e-10f, &sn, &c);
        s_cs[warp][j] = make_float2(c, sn);
      }
    }
    if (lane == 0) {
      s_row[warp] = row;
      s_own[warp] = b >= 0;
    }
  } else if (blockIdx.x == 0 && l == 0) {
    // the first CTA's other warps check all offsets
    for (int b = tid - 32 * TOK; b < a.B; b += kAppendThreads - 32 * TOK) {
      int b0, n;
      if (!sequence_tokens(a.off, b, a.T, b0, n)) msa::set_err(a.dev_err, MSA_DEVERR_BAD_OFFSETS);
    }
  }
  __syncthreads();
  bool loaded = have;
  while (ti < TOK && t0 + ti < a.T) {
    const int head = idx >> 3;
    if (s_own[ti]) {
      if (!loaded) {
        const In* src = source(t0 + ti, head);
        lo = load8(src + 8 * p);
        hi = load8(src + kHalf + 8 * p);
      }
      if (head < a.Hq + a.H) {
        Eight rl, rh;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 c = s_cs[ti][8 * p + e];
          rl.x[e] = lo.x[e] * c.x - hi.x[e] * c.y;
          rh.x[e] = hi.x[e] * c.x + lo.x[e] * c.y;
        }
        lo = rl;
        hi = rh;
      }
      __nv_bfloat16* dst = nullptr;
      if (head < a.Hq) {
        dst = a.q_rot + (((int64_t)l * a.T + t0 + ti) * a.Hq + head) * kD;
      } else if (s_row[ti] >= 0) {  // key heads, then value heads: consecutive [page][128] blocks
        dst = a.pages + s_row[ti] + ((int64_t)(head - a.Hq) << a.log2_page) * kD;
      }
      if (dst) {
        store8(dst + 8 * p, lo);
        store8(dst + kHalf + 8 * p, hi);
      }
    }
    loaded = false;
    idx += kAppendThreads;
    wrap();
  }
}

// ---------------------------------------------------------------------------- host side

msa_status check_device() {
  const int arch = msa::current_device_is_sm100(nullptr);
  if (arch < 0) return msa_fail(MSA_ERR_CUDA, "no CUDA device");
  if (arch == 0) return msa_fail(MSA_ERR_UNSUPPORTED, "device is not sm_100");
  return MSA_OK;
}

int log2_of_page(int page_size) {
  for (int k = 4; k <= 8; ++k)
    if (page_size == 1 << k) return k;
  return -1;
}

msa_status check_heads(int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim) {
  if (head_dim != kD) return msa_fail(MSA_ERR_INVALID_ARG, "head_dim must be 128");
  if (n_kv_heads < 1 || n_kv_heads > 16 || n_q_heads < 1 || n_q_heads % n_kv_heads != 0)
    return msa_fail(MSA_ERR_INVALID_ARG, "n_q_heads must be a multiple of n_kv_heads (<= 16)");
  const int G = n_q_heads / n_kv_heads;
  if (G != 1 && G != 2 && G != 4 && G != 8) return msa_fail(MSA_ERR_INVALID_ARG, "n_q_heads / n_kv_heads in {1,2,4,8}");
  return MSA_OK;
}

msa_status check_batch(int32_t n_tokens, int32_t n_seqs, int32_t n_layers) {
  if (n_tokens < 1 || n_seqs < 1 || n_layers < 1 || n_layers > 65535)
    return msa_fail(MSA_ERR_INVALID_ARG, "bad counts (n_tokens, n_seqs >= 1, 1 <= n_layers <= 65535)");
  if (n_seqs > kMaxSeqs) return msa_fail(MSA_ERR_INVALID_ARG, "n_seqs must be <= %d", kMaxSeqs);
  return MSA_OK;
}

msa_status check_pages(const void* kv_pages, int32_t n_pages, int32_t page_size, const int32_t* page_table,
                       int32_t max_pages) {
  if (!kv_pages || !page_table) return msa_fail(MSA_ERR_INVALID_ARG, "null pointer");
  if (log2_of_page(page_size) < 0) return msa_fail(MSA_ERR_INVALID_ARG, "page_size must be 16, 32, 64, 128 or 256");
  if (n_pages < 1 || max_pages < 1) return msa_fail(MSA_ERR_INVALID_ARG, "n_pages and max_pages must be >= 1");
  if ((int64_t)max_pages * page_size > 0x7fffffffll)
    return msa_fail(MSA_ERR_INVALID_ARG, "max_pages * page_size must fit 31 bits");
  if (!msa::aligned16(kv_pages)) return msa_fail(MSA_ERR_INVALID_ARG, "kv_pages must be 16-byte aligned");
  return MSA_OK;
}

template <typename In>
cudaError_t launch_append(const AppendArgs& a, int n_layers, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kAppendThreads, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(a.T, n_layers, 1);
  return cudaLaunchKernelEx(&cfg, append_kernel<In, 1>, a);
}

}  // namespace

extern "C" msa_status msa_paged_append(const void* q, const void* k_new, const void* v_new, msa_dtype in_dtype,
                                       int64_t q_stride, int64_t k_stride, int64_t v_stride,
                                       const int32_t* q_offsets, int32_t n_tokens, int32_t n_seqs, int32_t n_layers,
                                       int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim, void* kv_pages,
                                       int32_t n_pages, int32_t page_size, const int32_t* page_table,
                                       int32_t max_pages, const int32_t* seq_len, const int32_t* pos_offset,
                                       int32_t rope_pos_offset, float rope_theta, void* q_rot, int32_t* dev_err,
                                       msa_stream_t stream) {
  if (!k_new || !v_new || !q_offsets || !seq_len || (q == nullptr) != (q_rot == nullptr))
    return msa_fail(MSA_ERR_INVALID_ARG, "null pointer (q and q_rot go together)");
  msa_status st = check_heads(n_q_heads, n_kv_heads, head_dim);
  if (st == MSA_OK) st = check_batch(n_tokens, n_seqs, n_layers);
  if (st == MSA_OK) st = check_pages(kv_pages, n_pages, page_size, page_table, max_pages);
  if (st != MSA_OK) return st;
  if (in_dtype != MSA_BF16 && in_dtype != MSA_F32)
    return msa_fail(MSA_ERR_UNSUPPORTED, "in_dtype must be MSA_BF16 or MSA_F32");
  if (!(rope_theta > 1.0f) || !(rope_theta < INFINITY))
    return msa_fail(MSA_ERR_INVALID_ARG, "rope_theta must be > 1 and finite");
  if (!msa::aligned16(q) || !msa::aligned16(k_new) || !msa::aligned16(v_new) || !msa::aligned16(q_rot))
    return msa_fail(MSA_ERR_INVALID_ARG, "16-byte alignment (q, k_new, v_new, q_rot)");
  AppendArgs a;
  a.q_stride = q_stride == 0 ? (int64_t)n_q_heads * kD : q_stride;
  a.k_stride = k_stride == 0 ? (int64_t)n_kv_heads * kD : k_stride;
  a.v_stride = v_stride == 0 ? (int64_t)n_kv_heads * kD : v_stride;
  const int64_t unit = in_dtype == MSA_F32 ? 4 : 8;  // elements in 16 bytes
  if (a.q_stride < (int64_t)n_q_heads * kD || a.k_stride < (int64_t)n_kv_heads * kD ||
      a.v_stride < (int64_t)n_kv_heads * kD || a.q_stride % unit || a.k_stride % unit || a.v_stride % unit)
    return msa_fail(MSA_ERR_INVALID_ARG, "strides must be >= heads * head_dim and multiples of 16 bytes");
  st = check_device();
  if (st != MSA_OK) return st;
  a.q = q;
  a.k = k_new;
  a.v = v_new;
  a.off = q_offsets;
  a.T = n_tokens;
  a.B = n_seqs;
  a.Hq = n_q_heads;
  a.H = n_kv_heads;
  a.pages = static_cast<__nv_bfloat16*>(kv_pages);
  a.NP = n_pages;
  a.log2_page = log2_of_page(page_size);
  a.table = page_table;
  a.max_pages = max_pages;
  a.seq_len = seq_len;
  a.pos_offset = pos_offset;
  a.rope_pos_offset = rope_pos_offset;
  a.q_rot = static_cast<__nv_bfloat16*>(q_rot);
  a.dev_err = dev_err;
  a.rf = rope_freq(rope_theta);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  MSA_CUDA_TRY((in_dtype == MSA_F32 ? launch_append<float>(a, n_layers, s)
                                    : launch_append<__nv_bfloat16>(a, n_layers, s)));
  g_launches = 1;
  return msa_ok();
}

extern "C" msa_status msa_shared_attend_workspace_size(int32_t n_tokens, int32_t n_seqs, int32_t n_groups,
                                                       int32_t n_layers, int32_t n_q_heads, int32_t n_kv_heads,
                                                       size_t* bytes) {
  if (!bytes) return msa_fail(MSA_ERR_INVALID_ARG, "null pointer");
  msa_status st = check_heads(n_q_heads, n_kv_heads, kD);
  if (st == MSA_OK) st = check_batch(n_tokens, n_seqs, n_layers);
  if (st != MSA_OK) return st;
  if (n_groups < 0 || n_groups > n_seqs) return msa_fail(MSA_ERR_INVALID_ARG, "n_groups must be in [0, n_seqs]");
  const Plan plan = plan_of(n_tokens, n_seqs, n_groups, n_layers, n_q_heads, n_kv_heads);
  const int64_t rows = (int64_t)n_layers * n_tokens * n_q_heads;
  *bytes = kWsEnd + (plan.form == Plan::kMemory ? memory_bytes(rows, plan.splits) : 0);
  return msa_ok();
}

extern "C" msa_status msa_shared_attend(const void* q, const int32_t* q_offsets, int32_t n_tokens, int32_t n_seqs,
                                        int32_t n_layers, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                                        const void* mem_kv, const int32_t* mem_len, int32_t max_mem_chunks,
                                        const int32_t* group_offsets, int32_t n_groups, const void* kv_pages,
                                        int32_t n_pages, int32_t page_size, const int32_t* page_table,
                                        int32_t max_pages, const int32_t* seq_len, float softmax_scale, void* out,
                                        void* workspace, size_t workspace_bytes, int32_t* dev_err,
                                        msa_stream_t stream) {
  if (!q || !q_offsets || !seq_len || !out || !workspace) return msa_fail(MSA_ERR_INVALID_ARG, "null pointer");
  msa_status st = check_heads(n_q_heads, n_kv_heads, head_dim);
  if (st == MSA_OK) st = check_batch(n_tokens, n_seqs, n_layers);
  if (st == MSA_OK) st = check_pages(kv_pages, n_pages, page_size, page_table, max_pages);
  if (st != MSA_OK) return st;
  if (n_groups < 0 || n_groups > n_seqs) return msa_fail(MSA_ERR_INVALID_ARG, "n_groups must be in [0, n_seqs]");
  if (n_groups > 0 && (!mem_kv || !mem_len || !group_offsets || max_mem_chunks < 1))
    return msa_fail(MSA_ERR_INVALID_ARG, "n_groups > 0 needs mem_kv, mem_len, group_offsets and max_mem_chunks >= 1");
  if (!(softmax_scale > 0.f) || !(softmax_scale < INFINITY))
    return msa_fail(MSA_ERR_INVALID_ARG, "softmax_scale must be > 0 and finite");
  if (!msa::aligned16(q) || !msa::aligned16(mem_kv) || !msa::aligned16(out) || !msa::aligned16(workspace))
    return msa_fail(MSA_ERR_INVALID_ARG, "16-byte alignment (q, mem_kv, out, workspace)");
  size_t need = 0;
  st = msa_shared_attend_workspace_size(n_tokens, n_seqs, n_groups, n_layers, n_q_heads, n_kv_heads, &need);
  if (st != MSA_OK) return st;
  if (workspace_bytes < need)
    return msa_fail(MSA_ERR_CAPACITY, "workspace too small (%zu < %zu)", workspace_bytes, need);
  st = check_device();
  if (st != MSA_OK) return st;
  Attend a;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.out = static_cast<__nv_bfloat16*>(out);
  a.q_offsets = q_offsets;
  a.seq_len = seq_len;
  a.group_offsets = group_offsets;
  a.mem_kv = static_cast<const __nv_bfloat16*>(mem_kv);
  a.mem_len = mem_len;
  a.pages = static_cast<const __nv_bfloat16*>(kv_pages);
  a.page_table = page_table;
  a.T = n_tokens;
  a.B = n_seqs;
  a.NG = n_groups;
  a.L = n_layers;
  a.H = n_kv_heads;
  a.G = n_q_heads / n_kv_heads;
  a.M_max = n_groups > 0 ? max_mem_chunks : 0;
  a.NP = n_pages;
  a.log2_page = log2_of_page(page_size);
  a.max_pages = max_pages;
  a.qscale = softmax_scale * kLog2e;
  a.ws = static_cast<unsigned char*>(workspace);
  a.dev_err = dev_err;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const Plan plan = plan_of(n_tokens, n_seqs, n_groups, n_layers, n_q_heads, n_kv_heads);
  const int64_t mem_rows = (int64_t)n_groups * n_layers * 2 * n_kv_heads * a.M_max;
  const int64_t page_rows = ((int64_t)n_layers * n_pages * 2 * n_kv_heads) << a.log2_page;
  if (plan.form != Plan::kRowsOnly && (mem_rows > kMaxTensorRows || (plan.form == Plan::kBlocks && page_rows > kMaxTensorRows)))
    return msa_fail(MSA_ERR_CAPACITY, "mem_kv or kv_pages beyond 2^31 rows of 128 elements");
  if (plan.form == Plan::kBlocks) {
    MSA_CUDA_TRY(launch_blocks(a, s));
  } else {
    if (plan.form == Plan::kMemory) MSA_CUDA_TRY(launch_memory(a, plan.splits, s));
    MSA_CUDA_TRY(launch_rows(a, plan.splits, s));
  }
  g_launches = plan.form == Plan::kMemory ? 2 : 1;
  return msa_ok();
}

extern "C" int32_t msa_paged_last_launch_count(void) { return g_launches; }
