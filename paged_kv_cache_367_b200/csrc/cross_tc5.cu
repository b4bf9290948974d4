// paged_cross_attention: every query row attends over all cached tokens of its
// sequence (no causal mask), on the tcgen05 kernel of prefill_tc5.cuh.
//
//   out[r] = sum_t softmax_t(scale q_r . K[t]) V[t],  t = 0 .. L - 1
//
// Many rows are bound by the tensor cores (4 head_dim flops per row, head and
// token; 256 rows share each K/V chunk), few by the read of K and V. The launch is
// cut to size on the host:
//  * up to 128 rows (queries x heads of the group) per (sequence, KV head) take the
//    one-tile form of the tcgen05 kernel, with the rows in the tile four times (up to
//    32) or twice (up to 64), each copy taking a part of every chunk's tokens: rows
//    are M there, and a few of them would leave one thread in many to take the
//    exponentials;
//  * up to 16 rows over many tokens take the one-token decode's kernel (decode_tc.cu);
//  * where there are too few (sequence, KV head, tile) units for the GPU, the
//    cached tokens are cut into pieces of the same length, each a work item whose
//    rows go to the workspace normalised, in fp32, with their base-2 log-sum-exp;
//    a second kernel joins the pieces of a row in token order.
// Measured on B200: 8 x 250-1,000 queries of 64/8 heads of 128 over 2,100-4,096 tokens
// 634 us (948 TFLOP/s; 682 under the power cap); 2 x 7 queries of 32/8 heads over
// 60,000-65,536 E4M3 tokens 86 us (0.47 of the HBM rate: a chain of widening, S, softmax
// and PV of 1,250 clocks per 64-token chunk); 64 x 1 query over 16-2,048 tokens 62 us
// (0.75); 8 x 5 queries of 16 heads of 64 over 1,500 tokens 17 us; one query over 4,096
// tokens 13 us; 16 x 10, 16 and 32 queries of 32/8 heads over 2,000-4,096 tokens (two
// copies of the rows, two, one) 56, 59 and 61 us; 2 x 300 of them over 8,192, 80 units
// uncut on 148 SMs, 157 us (513 TFLOP/s).
//
// Items are handed out through cluster launch control (a CTA per item in the grid;
// running CTAs take over those not yet launched), so a call keeps no counter in
// memory: calls, and replays of captured calls, may overlap if their outputs and
// workspaces do not.
#include <math.h>

#include "prefill_tc5.cuh"
#include "schedule.cuh"

namespace pkv {

cudaError_t launch_cross_few(const DecodeParams& prm, int q_dtype, int cache_dtype, int num_sms,
                             cudaStream_t stream);
int num_sms_of_current_device(int* out);

namespace pf {
namespace {

// kWarps warps per (token, head) row, each taking every kWarps-th of its parts
// (pieces x copies): out = sum_k w_k o_k / sum_k w_k, w_k = 2^(lse_k - max lse);
// zeros for a sequence without tokens. A part of log-sum-exp -inf (no token of it has
// a weight) drops out; a NaN one makes the row NaN, as do parts that are all -inf. A
// warp has eight parts in flight, their log-sum-exps and rows together (a running
// maximum rescales the sums), so a row of up to eight costs one memory latency; a row
// of more is given a block of its own (one warp for each of 448 rows of 296 parts took
// 60 us). A programmatic dependent launch: the main kernel triggers it only by its CTAs'
// ends, so what overlaps is the launch and the search for the row with the last CTAs'
// writes becoming visible.
constexpr int kJoinWarps = 8;
template <typename OT, int D, int kWarps>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const PrefillParams p) {
  constexpr int V = D / 32, kBatch = 8;  // columns per lane, parts in flight
  __shared__ float sums[kWarps > 1 ? kWarps : 1][D + 2];
  const int seq = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int q1 = min(max(__ldg(p.query_start + seq + 1), 0), p.num_q_tokens);
  const int q0 = max(min(max(__ldg(p.query_start + seq), 0), q1), q1 - p.max_q_len);
  const int64_t r = kWarps > 1 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * kJoinWarps + warp;
  if (r >= (int64_t)(q1 - q0) * p.num_heads) return;  // kWarps > 1: the whole block
  const int64_t row = (int64_t)q0 * p.num_heads + r, rows = (int64_t)p.num_q_tokens * p.num_heads;
  const int L = min(__ldg(p.seq_lens + seq), p.len_cap);
  const int n = L > 0 ? ((L - 1) / p.piece_len + 1) * p.copies : 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float m = -INFINITY, acc[V], den = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.f;
  for (int k0 = kWarps > 1 ? warp : 0; k0 < n; k0 += kWarps * kBatch) {
    float lse[kBatch], o[kBatch][V], mx = m;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int64_t k = k0 + i * kWarps;
      lse[i] = -INFINITY;
#pragma unroll
      for (int v = 0; v < V; ++v) o[i][v] = 0.f;
      if (k < n) {
        lse[i] = __ldcg(p.ws_lse + k * rows + row);
        const float* src = p.ws_o + (k * rows + row) * D + lane * V;
        if constexpr (V == 4) {
          const float4 x = __ldcg(reinterpret_cast<const float4*>(src));
          o[i][0] = x.x, o[i][1] = x.y, o[i][2] = x.z, o[i][3] = x.w;
        } else {
          const float2 x = __ldcg(reinterpret_cast<const float2*>(src));
          o[i][0] = x.x, o[i][1] = x.y;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) mx = fmaxf(mx, lse[i]);  // a NaN is passed over here ..
    const float sub = mx == -INFINITY ? 0.f : mx;
    const float keep = fast_exp2(m - sub);
    m = mx;
    den *= keep;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] *= keep;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const float w = fast_exp2(lse[i] - sub);  // .. and reaches the sums here
      den += w;
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] = fmaf(w, o[i][v], acc[v]);
    }
  }
  if constexpr (kWarps > 1) {
#pragma unroll
    for (int v = 0; v < V; ++v) sums[warp][lane * V + v] = acc[v];
    if (lane == 0) {
      sums[warp][D] = den;
      sums[warp][D + 1] = m;
    }
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int x = 1; x < kWarps; ++x) m = fmaxf(m, sums[x][D + 1]);
    const float mx = m == -INFINITY ? 0.f : m;
    den = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.f;
#pragma unroll
    for (int x = 0; x < kWarps; ++x) {
      const float w = fast_exp2(sums[x][D + 1] - mx);
      den = fmaf(w, sums[x][D], den);
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] = fmaf(w, sums[x][lane * V + v], acc[v]);
    }
  }
  const float inv = n > 0 ? 1.f / den : 0.f;  // den 0: 0 * inf
  OT* dst = static_cast<OT*>(p.out) + row * D + lane * V;
  float a, b;
  if constexpr (V == 4) {
    uint2 w;
    w.x = Mma<OT>::pack(acc[0] * inv, acc[1] * inv, a, b);
    w.y = Mma<OT>::pack(acc[2] * inv, acc[3] * inv, a, b);
    *reinterpret_cast<uint2*>(dst) = w;
  } else {
    *reinterpret_cast<uint32_t*>(dst) = Mma<OT>::pack(acc[0] * inv, acc[1] * inv, a, b);
  }
}

constexpr int kSms = 148;

// How a call is cut: on tcgen05, tiles of rows per (sequence, KV head) and pieces of
// the tokens; with few rows over many tokens, at multiples of kFewPart tokens by the
// decode's split. kFewChunks is the number of 64-token chunks (sequences x KV heads x
// length bound) from which the decode's kernel is the faster one: its set-up and
// in-kernel joins take 15 us, and then it streams at 0.8-0.9 of the HBM rate, the
// one-tile kernel at 0.6-0.8 (one token, head_dim 128: 16 x 8 heads x 500 tokens 24.6
// us against 15.1, x 2,048 29.3 against 31.9, x 8,000 59.7 against 68.1; 64 x 8 heads
// x 2,048 94 against 104; at head_dim 64 the one-tile kernel wins, 83 us against 94).
constexpr int kFewRows = 16, kFewPart = 128;
constexpr int64_t kFewChunks = 4096;
constexpr int64_t kMaxPartBytes = 160 << 20;
struct Cut {
  bool few, one_tile;
  int copies;  // of the rows, in the one-tile kernel
  int64_t tiles, items;
  int pieces, piece_len;
  // Of the partial rows, of them and their log-sum-exps, and of the whole
  // workspace (few rows: with the split's counters at the end).
  size_t o_bytes, lse_end, bytes;
};

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

Cut cut_for(int64_t num_seqs, int64_t num_q_tokens, int64_t max_q_len, int64_t num_heads,
            int64_t num_kv_heads, int64_t head_dim, int64_t max_seq_len, int cache_dtype) {
  Cut c = {};
  const int64_t g = num_heads / num_kv_heads, rows = max_q_len * g;
  const int64_t chunks = (max_seq_len + kChunk - 1) / kChunk;
  c.few = rows <= kFewRows && head_dim == 128 && num_seqs * num_kv_heads * chunks >= kFewChunks;
  if (c.few) {
    if (max_seq_len > kFewPart) {
      const size_t part_rows = (size_t)2 * kMaxRanges * (size_t)rows;
      c.o_bytes = align256(part_rows * (size_t)head_dim * 4);
      c.lse_end = align256(c.o_bytes + part_rows * 4);
      c.bytes = align256(c.lse_end + sizeof(int32_t) * (size_t)(num_seqs * num_kv_heads + 1));
    }
    return c;
  }
  c.one_tile = rows <= Roles<kCrossOneTile>::kCtaRows;
  // Parts (pieces x copies) of each query row that the workspace holds at most.
  const int64_t part_bytes = std::max<int64_t>(num_q_tokens * num_heads * (head_dim + 1) * 4, 1);
  const int64_t most_parts = std::max<int64_t>(kMaxPartBytes / part_bytes, 1);
  c.copies = rows <= 32 ? 4 : rows <= 64 ? 2 : 1;
  while (c.copies > most_parts) c.copies /= 2;
  const int64_t cta_rows = c.one_tile ? Roles<kCrossOneTile>::kCtaRows : Roles<kCross>::kCtaRows;
  c.tiles = (rows + cta_rows - 1) / cta_rows;
  const int64_t units = std::max<int64_t>(num_seqs * num_kv_heads * c.tiles, 1);
  // Pieces: enough to fill the GPU in one go; or, with one tile, up to four times as
  // many where the items, handed out as CTAs become free, then even out unequal
  // lengths. Times in chunks, for lengths from half of the bound to the bound; an item
  // costs 4 + 16 / copies chunks beside its own (6 us at four copies, more with more
  // rows). Measured: 4 sequences of 10,000-20,000 tokens, 8 KV heads, 65 us in one go,
  // 54 by this rule; 2 of 60,000-65,536 87 us in one go (kept), 104 in four; 16 of
  // 2,000-4,096 with 64 rows 59 (kept) and 67. Two tiles: an item's partial rows cost
  // more than that gives (4 x 300 queries over 2,500-5,000 tokens: 117 us whole, 130
  // in two pieces).
  const int64_t slots =
      c.copies > 1 && head_dim == 64 && cache_dtype != PKV_FP8_E4M3 ? 2 * kSms : kSms;
  const int64_t most = std::max<int64_t>(most_parts / c.copies, 1);
  int64_t pieces = std::max<int64_t>(1, std::min({slots / units, chunks / 2, most}));
  if (c.one_tile) {
    const double item_cost = 4 + 16.0 / c.copies, mean = 0.75;
    double least = units * pieces <= slots ? (double)chunks / pieces + item_cost : 1e300;
    for (int times2 = 3; times2 <= 8; ++times2) {  // items: 1.5, 2, .. 4 times the slots
      const int64_t n = std::min(times2 * slots / (2 * units), std::min(chunks / 8, most));
      if (n < 1 || units * n <= slots) continue;
      const double item = (double)chunks / n + item_cost;
      const double cost = mean * units * n / slots * item + item / 2;
      if (cost < least) least = cost, pieces = n;
    }
  }
  const int64_t piece_chunks = std::max<int64_t>((chunks + pieces - 1) / pieces, 1);
  c.pieces = (int)std::max<int64_t>((chunks + piece_chunks - 1) / piece_chunks, 1);
  // Unsplit, the piece is as long as any sequence.
  c.piece_len = c.pieces == 1 ? INT32_MAX : (int)(piece_chunks * kChunk);
  c.items = units * c.pieces;
  if (c.pieces > 1 || c.copies > 1) {
    const size_t part_rows = (size_t)(c.pieces * c.copies) * (size_t)num_q_tokens * (size_t)num_heads;
    c.o_bytes = align256(part_rows * (size_t)head_dim * 4);
    c.bytes = c.lse_end = align256(c.o_bytes + part_rows * 4);
  }
  return c;
}

template <typename OT, int D, bool QT, bool F8, int KIND, int REP>
cudaError_t launch_cross(const PrefillParams& p, const CUtensorMap& mk, const CUtensorMap& mv,
                         const CUtensorMap& mq, const Cut& c, int num_seqs, cudaStream_t stream) {
  using C = Cfg5<D, F8, KIND>;
  auto kernel = prefill_tc5_kernel<OT, D, QT, F8, KIND, REP>;
  static std::atomic<int> opted_in[64];  // the shared-memory opt-in, once per device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!opted_in[dev].load(std::memory_order_relaxed)) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    opted_in[dev].store(1, std::memory_order_relaxed);
  }
  kernel<<<(unsigned)c.items, C::kThreads, C::kSmem, stream>>>(
      p, mk, mv, mq, num_seqs, (int)c.tiles, (int)c.items, nullptr);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || c.bytes == 0) return e;
  const int64_t rows = (int64_t)p.max_q_len * p.num_heads;
  const bool block = c.pieces * c.copies > kJoinWarps;  // a block per row
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(block ? rows : (rows + kJoinWarps - 1) / kJoinWarps), (unsigned)num_seqs);
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return block ? cudaLaunchKernelEx(&cfg, join_kernel<OT, D, kJoinWarps>, p)
               : cudaLaunchKernelEx(&cfg, join_kernel<OT, D, 1>, p);
}

template <typename OT, int D, bool F8>
cudaError_t launch_f8(PrefillParams p, const CUtensorMap& mk, const CUtensorMap& mv, const Cut& c,
                      int num_seqs, cudaStream_t stream) {
  constexpr bool kBf16 = std::is_same<OT, __nv_bfloat16>::value;
  CUtensorMap mq;
  if (c.one_tile) {
    // By TMA where whole tokens fill a copy, unless a bf16 query is rounded to f16.
    p.q_map = !(F8 && kBf16) && encode_q_map(&mq, p, D, kBf16, kRows / c.copies);
    const CUtensorMap& m = p.q_map ? mq : mk;  // mk: no query map
    if (c.copies == 4)
      return launch_cross<OT, D, false, F8, kCrossOneTile, 4>(p, mk, mv, m, c, num_seqs, stream);
    if (c.copies == 2)
      return launch_cross<OT, D, false, F8, kCrossOneTile, 2>(p, mk, mv, m, c, num_seqs, stream);
    return launch_cross<OT, D, false, F8, kCrossOneTile, 1>(p, mk, mv, m, c, num_seqs, stream);
  }
  if (encode_q_map(&mq, p, D, kBf16))
    return launch_cross<OT, D, true, F8, kCross, 1>(p, mk, mv, mq, c, num_seqs, stream);
  return launch_cross<OT, D, false, F8, kCross, 1>(p, mk, mv, mk, c, num_seqs, stream);
}

template <typename OT, int D>
cudaError_t launch_d(const PrefillParams& p, const CUtensorMap& mk, const CUtensorMap& mv, bool f8,
                     const Cut& c, int num_seqs, cudaStream_t stream) {
  return f8 ? launch_f8<OT, D, true>(p, mk, mv, c, num_seqs, stream)
            : launch_f8<OT, D, false>(p, mk, mv, c, num_seqs, stream);
}

bool sizes_ok(int num_seqs, int num_q_tokens, int max_q_len, int num_heads, int num_kv_heads,
              int max_seq_len) {
  return num_seqs >= 0 && num_q_tokens >= 0 && max_q_len >= 0 && num_heads > 0 &&
         num_kv_heads > 0 && num_heads % num_kv_heads == 0 && max_seq_len >= 0 &&
         num_seqs <= 65535 && num_kv_heads <= 65535 && num_heads <= (1 << 20);
}

}  // namespace
}  // namespace pf

int cross_status_flag(bool clear, int* value) {
  using pf::g_pf5_status;
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_pf5_status, sizeof(int)) != cudaSuccess) return -1;
  if (clear && v) {
    const int zero = 0;
    if (cudaMemcpyToSymbol(g_pf5_status, &zero, sizeof(int)) != cudaSuccess) return -1;
  }
  *value = v;
  return 0;
}

}  // namespace pkv

using namespace pkv;

extern "C" {

size_t paged_cross_attention_workspace_size(int num_seqs, int num_q_tokens, int max_q_len,
                                            int num_heads, int num_kv_heads, int head_dim,
                                            int max_seq_len, int cache_dtype) {
  if (!pf::sizes_ok(num_seqs, num_q_tokens, max_q_len, num_heads, num_kv_heads, max_seq_len) ||
      (head_dim != 64 && head_dim != 128) ||
      (cache_dtype != PKV_F16 && cache_dtype != PKV_BF16 && cache_dtype != PKV_FP8_E4M3))
    return 0;
  if (num_seqs == 0 || num_q_tokens == 0 || max_q_len == 0) return 0;
  return pf::cut_for(num_seqs, num_q_tokens, std::min(max_q_len, num_q_tokens), num_heads,
                     num_kv_heads, head_dim, max_seq_len, cache_dtype)
      .bytes;
}

int paged_cross_attention(void* out, const void* query, const void* k_cache, const void* v_cache,
                          const int32_t* block_table, const int32_t* seq_lens,
                          const int32_t* query_start, int num_seqs, int num_q_tokens,
                          int max_q_len, int num_heads, int num_kv_heads, int head_dim,
                          int block_size, int max_blocks_per_seq, int64_t num_blocks,
                          int max_seq_len, float scale, int q_dtype, int cache_dtype,
                          const float* k_scale, const float* v_scale, void* workspace,
                          size_t workspace_bytes, void* stream) {
  if (!pf::sizes_ok(num_seqs, num_q_tokens, max_q_len, num_heads, num_kv_heads, max_seq_len) ||
      num_blocks <= 0 || num_blocks > INT32_MAX || max_blocks_per_seq <= 0 || !isfinite(scale) ||
      !(scale > 0.f))
    return PKV_ERR_SHAPE;
  if (head_dim != 64 && head_dim != 128) return PKV_ERR_UNSUPPORTED;
  if (block_size != 8 && block_size != 16 && block_size != 32) return PKV_ERR_UNSUPPORTED;
  if ((q_dtype != PKV_BF16 && q_dtype != PKV_F16) ||
      (cache_dtype != q_dtype && cache_dtype != PKV_FP8_E4M3))
    return PKV_ERR_DTYPE;
  const bool f8 = cache_dtype == PKV_FP8_E4M3, bf16 = q_dtype == PKV_BF16;
  if (num_seqs == 0 || num_q_tokens == 0 || max_q_len == 0) return PKV_OK;
  if (!out || !query || !k_cache || !v_cache || !block_table || !seq_lens || !query_start)
    return PKV_ERR_NULL;
  if (f8 && (!k_scale || !v_scale)) return PKV_ERR_NULL;
  if (((uintptr_t)out | (uintptr_t)query | (uintptr_t)k_cache | (uintptr_t)v_cache) & 15u ||
      ((uintptr_t)block_table | (uintptr_t)seq_lens | (uintptr_t)query_start) & 3u ||
      (f8 && ((uintptr_t)k_scale | (uintptr_t)v_scale) & 3u))
    return PKV_ERR_ALIGN;
  const int q_len = std::min(max_q_len, num_q_tokens);
  const pf::Cut c = pf::cut_for(num_seqs, num_q_tokens, q_len, num_heads, num_kv_heads, head_dim,
                                max_seq_len, cache_dtype);
  if (c.items > INT32_MAX / 2) return PKV_ERR_SHAPE;
  if (c.bytes > 0) {
    if (!workspace || workspace_bytes < c.bytes) return PKV_ERR_WORKSPACE;
    if ((uintptr_t)workspace & 255u) return PKV_ERR_ALIGN;
  }
  char* const wsb = static_cast<char*>(workspace);
  const int len_cap = (int)std::min<int64_t>((int64_t)max_blocks_per_seq * block_size, max_seq_len);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (c.few) {
    int sms = 0;
    if (num_sms_of_current_device(&sms) != PKV_OK) return PKV_ERR_CUDA;
    DecodeParams d = {};
    d.out = out;
    d.query = query;
    d.k_cache = k_cache;
    d.v_cache = v_cache;
    d.block_table = block_table;
    d.seq_lens = seq_lens;
    d.num_seqs = num_seqs;
    d.num_heads = num_heads;
    d.num_kv_heads = num_kv_heads;
    d.head_dim = head_dim;
    d.block_size = block_size;
    d.max_blocks_per_seq = max_blocks_per_seq;
    d.num_blocks = num_blocks;
    d.len_cap = len_cap;
    d.part = c.bytes ? pf::kFewPart : 0;
    d.unit_cost = 24;  // as the decode charges them
    d.unit_round = 64;
    d.score_scale = scale * kLog2e;
    d.k_scale = k_scale;
    d.v_scale = v_scale;
    d.query_start = query_start;
    d.num_q_tokens = num_q_tokens;
    d.max_q_len = q_len;
    d.rows = q_len * (num_heads / num_kv_heads);
    if (c.bytes) {
      d.ws_o = reinterpret_cast<float*>(wsb);
      d.ws_lse = reinterpret_cast<float*>(wsb + c.o_bytes);
      d.ws_done = reinterpret_cast<int*>(wsb + c.lse_end);
      if (cudaMemsetAsync(d.ws_done, 0, c.bytes - c.lse_end, st) != cudaSuccess)
        return PKV_ERR_CUDA;
    }
    return launch_cross_few(d, q_dtype, cache_dtype, sms, st) == cudaSuccess ? PKV_OK
                                                                             : PKV_ERR_CUDA;
  }
  const CUtensorMapDataType dt = f8     ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                 : bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                        : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const int e = f8 ? 1 : 2;
  CUtensorMap mk, mv;
  if (!tcx::encode_pool_map(&mk, k_cache, dt, e, head_dim, block_size, num_kv_heads, num_blocks,
                            true) ||
      !tcx::encode_pool_map(&mv, v_cache, dt, e, head_dim, block_size, num_kv_heads, num_blocks,
                            true))
    return PKV_ERR_CUDA;
  pf::PrefillParams p = {};
  p.out = out;
  p.query = query;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.query_start = query_start;
  p.num_heads = num_heads;
  p.num_kv_heads = num_kv_heads;
  p.block_size = block_size;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.num_q_tokens = num_q_tokens;
  p.max_q_len = q_len;
  p.num_blocks = (int)num_blocks;
  p.score_scale = scale * kLog2e;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.len_cap = len_cap;
  p.pieces = c.pieces;
  p.piece_len = c.piece_len;
  p.copies = c.copies;
  p.ws_o = reinterpret_cast<float*>(wsb);
  p.ws_lse = c.bytes ? reinterpret_cast<float*>(wsb + c.o_bytes) : nullptr;
  const bool d128 = head_dim == 128;
  const cudaError_t err =
      bf16 ? (d128 ? pf::launch_d<__nv_bfloat16, 128>(p, mk, mv, f8, c, num_seqs, st)
                   : pf::launch_d<__nv_bfloat16, 64>(p, mk, mv, f8, c, num_seqs, st))
           : (d128 ? pf::launch_d<__half, 128>(p, mk, mv, f8, c, num_seqs, st)
                   : pf::launch_d<__half, 64>(p, mk, mv, f8, c, num_seqs, st));
  return err == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // extern "C"
