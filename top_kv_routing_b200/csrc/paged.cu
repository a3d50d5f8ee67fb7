// Paged batches: the append kernel, the choice of the attention kernels and the entry points (those
// kernels are in paged_rows.cu and paged_tc.cu).
//
// Follows "MSA端到端可训练记忆模型完整开源，支持亿级Token上下文", section 架构 (全局 RoPE: positions
// offset by k; local K/V joined to the selected memory), and the MSA paper reading notes,
// section 推理全流程 (the local KV grows while the memory stays fixed).
#include <math.h>

#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "msa_paged.h"
#include "paged.cuh"

MSA_DEFINE_LAST_ERROR(msa_paged_last_error)

namespace {
using namespace paged;

constexpr int kHalf = 64;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int64_t kMaxTensorRows = 0x7fffffff - 128;  // (TMA row coordinates are 32-bit)

// Which kernels a batch takes (the split of the tokens over the sequences is known to the device
// alone; any split is computed correctly by every form):
//   kRows    the row kernel walks memory and pages of 8 or 16 rows (tokens x G) of a sequence;
//   kMemory  the memory once for all rows of a group, on the tensor cores, cut into pieces where
//            there are few of them, then the row kernel over the pages;
//   kBlocks  memory and pages of 256 rows of a sequence on the tensor cores.
struct Plan {
  enum Form { kRows, kMemory, kBlocks } form;
  int splits;  // memory form: most key splits
};

// Whether a batch may take the memory form (its workspace follows from the sizes alone): groups
// of more than eight rows, in short blocks or in few units.
bool memory_form_open(int64_t T, int64_t B, int64_t NG, int64_t L, int64_t G, int64_t H) {
  return NG > 0 && T * G > 8 * NG && (T * G < 64 * B || std::max(B, T * G / 256) * L * H < 148);
}

// The form that takes least, estimated in cycles of a B200's 148 SMs from measured ones: 220 per
// (16 keys, row tile) of the row kernel with all warps at work, six of them for a row tile's own
// costs and ten where the memory's results are joined to it; 3,100 per 128 keys and 5,000 per unit
// of the tensor-core kernel; 20,000 for each kernel of the first two forms to start and end, 15,000
// for the third.  Of 228 batches of all sizes in buffers of just the lengths in use, timed in every
// form that they may take, 223 got a form within 12 % of the best, 1 % from it on average.  Both
// sides of the borders (us, 32 / 8 heads, cold): 16 answers over 256 + 300 keys, one layer: rows 20,
// blocks 22, memory 27; 18 layers: rows 94, memory 100 (taken), blocks 164; 128 answers in 16 groups
// over 400 + 215 keys, 18 layers: memory 451, rows 843, blocks 1,350; 40 sequences of 8 tokens over
// 500 + 250 keys, 6 layers: memory 150, rows 174, blocks 180; of 12 tokens: blocks 186, memory 209
// (taken), rows 258; of 15: blocks 186, memory 266, rows 328.
//
// The lengths are the largest ones that the buffers allow (those in use are known to the device
// alone), so room in the buffers moves the choice although it costs no form anything: over 256 + 300
// keys in a memory of 2,048 rows and a table of 4,096, 4 sequences of 8 tokens and 4 layers take the
// memory form, 44 against 21 of blocks; 16 of one token and one layer the memory form, 27 against
// 20 of rows; 37 of 5 tokens over 1,000 + 500 keys with a table of 32,768 rows blocks, 192 against
// 143 of memory.
Plan plan_of(int64_t T, int64_t B, int64_t NG, int64_t L, int64_t Hq, int64_t H, int64_t mem_rows, int64_t page_rows) {
  const double G = (double)(Hq / H), rows = (double)T * G, units = (double)L * H, sms = 148;
  const double M = NG > 0 ? (double)mem_rows : 0., P = (double)page_rows;
  const double start = 20000, start_blocks = 15000, tile = 3100, unit = 5000, row_tile = 220;
  const double R = rows <= 8. * B ? 8 : 16, row_tiles = B * std::ceil(rows / B / R);
  const double pairs = std::max((double)B, rows / 256);
  auto rows_cost = [&](double keys, double own) { return start + units * row_tiles * (keys / 16 + own) * row_tile / sms; };
  Plan best = {Plan::kRows, 0};
  double cost = rows_cost(M + P, 6);
  if (memory_form_open(T, B, NG, L, Hq / H, H)) {
    const double c =
        start + units * std::max((double)NG, rows / 256) * (std::ceil(M / 128) * tile + unit) / sms + rows_cost(P, 10);
    if (c < cost) {
      cost = c;
      best = {Plan::kMemory, memory_splits(L * T * Hq)};
    }
  }
  const double waves = std::max(std::ceil(units * B / sms), units * pairs / sms);
  if (start_blocks + waves * ((std::ceil(M / 128) + std::ceil(P / 128)) * tile + unit) < cost) best = {Plan::kBlocks, 0};
  return best;
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
// CTA (token, run of layers): warp 0 finds the token's sequence (a 32-way search of the offsets),
// its page slot and the 64 angles of its position, once for all layers of the run; then eight
// threads per head row rotate (query and key heads) or copy (value heads) 8 + 8 elements each.
// The first rows are loaded before the position is known and the next before the ones at hand are
// stored.  Bound by HBM: every byte moves once (2.7 GB of long texts in 420 us, 0.99 of the copy
// rate; one token 3.3 us in a graph).
constexpr int kAppendThreads = 256;
constexpr int kAppendCtas = 148 * 7;  // runs of layers are as long as leaves so many CTAs (five fit an SM at once)

struct AppendArgs {
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  const int32_t* off;
  int T, B, L, Hq, H;
  int run;  // layers of a CTA
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

// Eight elements as they lie in memory, and as floats.
template <typename In>
struct Eight {
  uint4 w[sizeof(In) / 2];
};
template <typename In>
__device__ __forceinline__ Eight<In> load8(const In* p) {
  Eight<In> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(In) / 2; ++i)
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.w[i].x), "=r"(r.w[i].y), "=r"(r.w[i].z), "=r"(r.w[i].w)
                 : "l"(reinterpret_cast<const uint4*>(p) + i));
  return r;
}
__device__ __forceinline__ void floats(const Eight<__nv_bfloat16>& r, float (&x)[8]) {
  const uint32_t u[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = msa::bf16x2_to_float2(u[e]);
    x[2 * e] = f.x;
    x[2 * e + 1] = f.y;
  }
}
__device__ __forceinline__ void floats(const Eight<float>& r, float (&x)[8]) {
  const uint32_t u[8] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w, r.w[1].x, r.w[1].y, r.w[1].z, r.w[1].w};
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(u[e]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  // (streaming: what does not fit L2 leaves it first; 5 % of a large call)
  __stcs(reinterpret_cast<uint4*>(p),
         make_uint4(msa::float2_to_bf16x2(x[0], x[1]), msa::float2_to_bf16x2(x[2], x[3]),
                    msa::float2_to_bf16x2(x[4], x[5]), msa::float2_to_bf16x2(x[6], x[7])));
}

template <typename In>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendArgs a) {
  __shared__ float2 s_cs[kHalf];
  __shared__ int64_t s_row;  // element offset of the token's row in layer 0's key head 0, or -1
  __shared__ int s_own;      // the token belongs to a sequence
  const int t = blockIdx.x, l0 = blockIdx.y * a.run, nl = min(a.run, a.L - l0);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // (what the search below reads one after the other: asked of L2 at once)
  prefetch_line(a.off, (a.B + 1) * 4ll, tid);
  prefetch_line(a.seq_len, a.B * 4ll, tid);
  if (a.pos_offset) prefetch_line(a.pos_offset, a.B * 4ll, tid);
  prefetch_line(a.table, (int64_t)a.B * a.max_pages * 4, tid);
  wait_for_earlier_kernels();
  let_next_kernel_start();
  const int p = tid & 7;  // dims 8p .. 8p + 7 and 64 + 8p .. (kAppendThreads is a multiple of 8)
  // this thread's rows: `head` of layer l0 + li (with no queries to rotate from the first key head on)
  const int first = a.q_rot ? 0 : a.Hq, heads = a.Hq + 2 * a.H;
  struct At {
    int li, head;
  };
  auto wrap = [&](At x) -> At {
    while (x.head >= heads && x.li < nl) {
      x.head -= heads - first;
      ++x.li;
    }
    return x;
  };
  struct Row {
    Eight<In> lo, hi;
  };
  auto load = [&](const At& x) -> Row {
    const int64_t row = (int64_t)(l0 + x.li) * a.T + t;
    const In* src;
    if (x.head < a.Hq)
      src = static_cast<const In*>(a.q) + row * a.q_stride + x.head * kD;
    else if (x.head < a.Hq + a.H)
      src = static_cast<const In*>(a.k) + row * a.k_stride + (x.head - a.Hq) * kD;
    else
      src = static_cast<const In*>(a.v) + row * a.v_stride + (x.head - a.Hq - a.H) * kD;
    return Row{load8(src + 8 * p), load8(src + kHalf + 8 * p)};
  };
  auto next = [&](const At& x) -> At { return wrap(At{x.li, x.head + kAppendThreads / 8}); };
  At x = wrap(At{0, first + (tid >> 3)});
  Row r;
  if (x.li < nl) r = load(x);
  if (warp == 0) {
    int b0 = 0, n = 0;
    const int b = sequence_of(a.off, a.B, a.T, t, lane, b0, n);
    int64_t row = -1;
    if (b >= 0) {
      const long long i = (long long)a.seq_len[b] - n + (t - b0);
      const long long pos = (long long)a.rope_pos_offset + (a.pos_offset ? (long long)a.pos_offset[b] : 0ll) + i;
      uint32_t err = 0u;
      if (i < 0) {
        err = MSA_DEVERR_BAD_OFFSETS;
      } else if ((i >> a.log2_page) >= a.max_pages) {
        err = MSA_DEVERR_LOCAL_FULL;
      } else {
        const int page = a.table[(int64_t)b * a.max_pages + (i >> a.log2_page)];
        if (page < 0 || page >= a.NP)
          err = MSA_DEVERR_BAD_PAGE;
        else
          row = ((((int64_t)page * 2 * a.H) << a.log2_page) + (i & ((1ll << a.log2_page) - 1))) * kD;
      }
      if (err && lane == 0 && l0 == 0) msa::set_err(a.dev_err, err);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = lane + 32 * e;
        // the top 32 bits of the angle, read as signed, are angle / pi in [-1, 1) x 2^31
        const int top = (int)(((unsigned long long)pos * a.rf.step[j]) >> 32);
        float sn, c;
        sincospif((float)top * 4.656612873077392578125e-10f, &sn, &c);
        s_cs[j] = make_float2(c, sn);
      }
    }
    if (lane == 0) {
      s_row = row;
      s_own = b >= 0;
    }
  } else if (blockIdx.x == 0 && l0 == 0) {
    // the first CTA's other warps check all offsets
    for (int b = tid - 32; b < a.B; b += kAppendThreads - 32) {
      int b0, n;
      if (!sequence_tokens(a.off, b, a.T, b0, n)) msa::set_err(a.dev_err, MSA_DEVERR_BAD_OFFSETS);
    }
  }
  __syncthreads();
  if (!s_own) return;
  const int64_t row = s_row;
  while (x.li < nl) {
    const At y = next(x);
    Row ahead;
    if (y.li < nl) ahead = load(y);
    float lo[8], hi[8];
    floats(r.lo, lo);
    floats(r.hi, hi);
    if (x.head < a.Hq + a.H) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 c = s_cs[8 * p + e];
        const float rl = lo[e] * c.x - hi[e] * c.y;
        hi[e] = hi[e] * c.x + lo[e] * c.y;
        lo[e] = rl;
      }
    }
    __nv_bfloat16* dst = nullptr;
    const int64_t l = l0 + x.li;
    if (x.head < a.Hq) {
      dst = a.q_rot + ((l * a.T + t) * a.Hq + x.head) * kD;
    } else if (row >= 0) {  // key heads, then value heads: consecutive [page][128] blocks
      dst = a.pages + row + (((l * a.NP * 2 * a.H + (x.head - a.Hq)) << a.log2_page) * kD);
    }
    if (dst) {
      store8(dst + 8 * p, lo);
      store8(dst + kHalf + 8 * p, hi);
    }
    x = y;
    r = ahead;
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
cudaError_t launch_append(const AppendArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kAppendThreads, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(a.T, (a.L + a.run - 1) / a.run, 1);
  return cudaLaunchKernelEx(&cfg, append_kernel<In>, a);
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
  a.L = n_layers;
  a.run = (int)std::min<int64_t>(n_layers, std::max<int64_t>(1, (int64_t)n_tokens * n_layers / kAppendCtas));
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
  MSA_CUDA_TRY((in_dtype == MSA_F32 ? launch_append<float>(a, s) : launch_append<__nv_bfloat16>(a, s)));
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
  const int64_t rows = (int64_t)n_layers * n_tokens * n_q_heads;
  const bool memory = memory_form_open(n_tokens, n_seqs, n_groups, n_layers, n_q_heads / n_kv_heads, n_kv_heads);
  *bytes = kWsEnd + (memory ? memory_bytes(rows, memory_splits(rows)) : 0);
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
  const Plan plan = plan_of(n_tokens, n_seqs, n_groups, n_layers, n_q_heads, n_kv_heads, a.M_max,
                            (int64_t)max_pages * page_size);
  const int64_t mem_rows = (int64_t)n_groups * n_layers * 2 * n_kv_heads * a.M_max;
  const int64_t page_rows = ((int64_t)n_layers * n_pages * 2 * n_kv_heads) << a.log2_page;
  if (plan.form != Plan::kRows && (mem_rows > kMaxTensorRows || (plan.form == Plan::kBlocks && page_rows > kMaxTensorRows)))
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
