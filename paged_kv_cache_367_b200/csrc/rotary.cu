// Rotary positions: queries and keys rotated by their positions (pkv_rotary), and
// the same rotation on the way into the paged cache (paged_kv_append_rotary).
//
// A row x of head_dim elements has its first rot_dim elements taken as rot_dim / 2
// pairs (x_a, x_b) — elements (i, i + rot_dim / 2), or (2i, 2i + 1) with the
// interleaved layout — and pair i at position p becomes, with t = p * inv_freq[i]
// and m the magnitude,
//   y_a = m (x_a cos t - x_b sin t),   y_b = m (x_b cos t + x_a sin t);
// the rest of the row passes through. The transposed rotation (sin negated) is
// the gradient of the call with respect to x.
//
// The angle: at position 10^6 an fp32 product p * f is already 0.03 radians off,
// so the turns p * f / 2 pi are formed and reduced to [-1/2, 1/2] in fp64 (three
// operations per pair and token, shared by all heads of the token), and sine and
// cosine are taken of the fp32 remainder in units of pi, where the argument
// reduction is exact. Products and sums are fp32, rounded once on the store (to
// E4M3 directly from fp32 for an FP8 cache, not by way of the source type).
//
// Bound by HBM: one read and one write of each row. Work is laid out flat over
// (token, head) rows, heads of the token being q, then k, then v: a block takes
// consecutive rows, so one token's heads spread over several blocks in a decode
// step (latency) and a block spans several tokens of narrow models; either way it
// computes the cosines and sines of its few tokens once, into shared memory. A
// thread owns both members of the pairs it rotates (VEC of each), so a call in
// place needs no exchange; its loads of all U tasks are issued before the
// trigonometry, whose latency they cover.
//
// Measured on B200 (of the measured copy rate): 8,191 tokens of 40 + 40 heads of 128
// in f16 52.7 us (0.97), 4,096 tokens of 32 + 8 heads of 64 in fp32 16.2 us (0.79; 0.99
// at 8,192 tokens of heads of 128); 8,192 tokens of 64 / 8 heads appended to a bf16
// cache 52.8 us (0.97), to an E4M3 one 57.0 (0.85: issue slots 67% busy); one token
// 1.7-2.1 us, 128 tokens 2.5-2.9. Where rot_dim / 2 or a stride is no multiple of 4 the
// whole row goes element by element: 8,192 tokens of 32 + 32 heads of 80 in bf16 take
// 100 us with 20 rotated (0.26), 30 with 80.
#include <math.h>

#include "common.cuh"

namespace pkv {
namespace rot {
namespace {

enum { kRotate = 0, kAppend = 1, kAppendFp8 = 2 };
constexpr int kThreads = 256;
// Heads of q, k and v together: what the divisions by Div and the 12 bits of a
// head below hold.
constexpr int kMaxHeads = 4096;
constexpr uint32_t kNoRow = ~0u;

// Two 16-bit elements in a word, low one first.
template <typename T> __device__ __forceinline__ float2 pair_to_f32(uint32_t w);
template <> __device__ __forceinline__ float2 pair_to_f32<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <> __device__ __forceinline__ float2 pair_to_f32<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <typename T> __device__ __forceinline__ uint32_t pair_from_f32(float x, float y);
template <> __device__ __forceinline__ uint32_t pair_from_f32<__nv_bfloat16>(float x, float y) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <> __device__ __forceinline__ uint32_t pair_from_f32<__half>(float x, float y) {
  const __half2 v = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Division by a small number known at launch: n / d = the high word of
// n * ceil(2^32 / d), exact while n * d < 2^32.
struct Div {
  uint32_t d, m;
  __host__ static Div by(uint32_t d) { return {d, (uint32_t)(((1ull << 32) + d - 1) / d)}; }
  __device__ __forceinline__ int div(int n) const { return d == 1 ? n : (int)__umulhi(n, m); }
};

struct RotaryParams {
  const void* src[3];     // query, key, value rows (value: append only)
  int64_t src_stride[3];  // elements from token to token
  void* dst[3];           // q_out, then k_out / K pool, V pool
  int64_t dst_stride[2];  // of q_out and k_out (no pool)
  int end[3];             // heads of the flat row order below which a row is q, k, v
  const int64_t* positions;
  const double* inv_freq;
  const int64_t* slot_mapping;  // append only
  const float* scale[2];        // k_scale, v_scale of an E4M3 pool
  int64_t num_slots;
  int64_t rows;           // num_tokens * end[2]
  float magnitude;        // m
  float sin_sign;         // -1: transposed
  int head_dim, rot_dim, tasks, rows_per_pass;
  // Of n < heads + 768 rows (3 passes of 256), < 256 threads, < 6,144 table entries.
  Div by_heads, by_tasks, by_half;
  int early;              // dependent kernels may start: only the pools are written
};

// VEC elements of T as raw words (one 16-bit element when VEC is 1).
template <typename T, int VEC>
struct Raw {
  static constexpr int kBytes = VEC * (int)sizeof(T);
  static constexpr int kWords = kBytes >= 4 ? kBytes / 4 : 1;
  uint32_t w[kWords];

  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kBytes % 16 == 0) {
#pragma unroll
      for (int k = 0; k < kWords; k += 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(p) + k);
        w[k] = v.x, w[k + 1] = v.y, w[k + 2] = v.z, w[k + 3] = v.w;
      }
    } else if constexpr (kBytes == 8) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x, w[1] = v.y;
    } else if constexpr (kBytes == 4) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (kBytes % 16 == 0) {
#pragma unroll
      for (int k = 0; k < kWords; k += 4)
        *reinterpret_cast<uint4*>(reinterpret_cast<uint32_t*>(p) + k) =
            make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]);
    } else if constexpr (kBytes == 8) {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else if constexpr (kBytes == 4) {
      *reinterpret_cast<uint32_t*>(p) = w[0];
    } else {
      *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
    }
  }
  __device__ __forceinline__ void get(float (&x)[VEC]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) x[i] = __uint_as_float(w[i]);
    } else if constexpr (VEC == 1) {
      const uint16_t h = (uint16_t)w[0];
      x[0] = Elem<T>::to_f32(*reinterpret_cast<const T*>(&h));
    } else {
#pragma unroll
      for (int i = 0; i < VEC; i += 2) {
        const float2 f = pair_to_f32<T>(w[i / 2]);
        x[i] = f.x, x[i + 1] = f.y;
      }
    }
  }
  __device__ __forceinline__ void set(const float (&x)[VEC]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) w[i] = __float_as_uint(x[i]);
    } else if constexpr (VEC == 1) {
      const T h = from_f32<T>(x[0]);
      w[0] = *reinterpret_cast<const uint16_t*>(&h);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; i += 2) w[i / 2] = pair_from_f32<T>(x[i], x[i + 1]);
    }
  }
};

// Division by an E4M3 pool's scale s, correctly rounded as paged_kv_append's is,
// with the reciprocal r taken once: q = x r is off by two steps at most, the
// remainder x - q s is exact in a fused multiply-add, and q + (x - q s) r rounds
// to the quotient (Markstein, IBM J. Res. Dev. 34, 1990). Before that x and s are
// multiplied by z = 1, or by a power of two that brings s into [2^-60, 2^60]
// (where that takes x out of fp32's range, the code is 448 or 0 anyway; a scale of
// zero or infinity becomes 1 with z infinite or 0), and x is held to
// |x| <= 1024 |s| (code 448 from 464 |s| on; NaN stays), so that nothing after
// overflows. The quotient takes q's sign, which a zero's remainder loses. Two
// elements at a time; dividing where it is rare that s needs it, on a branch of
// its own, cost more than all of this (64 q, 8 k/v heads of 128, 8192 tokens: 60.4 us
// against 57.0).
struct E4m3Scale {
  float s, r, z, most;
  __device__ __forceinline__ explicit E4m3Scale(float scale) {
    const float a = fabsf(scale);
    z = a < 0x1p-60f ? 0x1p100f : a > 0x1p60f ? 0x1p-100f : 1.f;
    s = scale * z;
    if (a == 0.f || a == INFINITY) {
      z = a == 0.f ? INFINITY : 0.f;
      s = copysignf(1.f, scale);
    }
    r = 1.f / s;
    most = 1024.f * fabsf(s);
  }
  __device__ __forceinline__ void divide2(float x, float y, float& qx, float& qy) const {
    asm("{\n .reg .b64 v, q, e, rr, ss, zz;\n .reg .f32 a, b, c, d;\n"
        " mov.b64 v, {%2, %3};\n mov.b64 zz, {%7, %7};\n mul.rn.f32x2 v, v, zz;\n"
        " mov.b64 {a, b}, v;\n"
        " min.NaN.xorsign.abs.f32 a, a, %6;\n min.NaN.xorsign.abs.f32 b, b, %6;\n"
        " mov.b64 v, {a, b};\n mov.b64 rr, {%4, %4};\n mov.b64 ss, {%5, %5};\n"
        " mul.rn.f32x2 q, v, rr;\n mov.b64 {c, d}, q;\n"
        " fma.rn.f32x2 e, q, ss, v;\n fma.rn.f32x2 q, e, rr, q;\n"
        " mov.b64 {a, b}, q;\n copysign.f32 %0, c, a;\n copysign.f32 %1, d, b;\n}"
        : "=f"(qx), "=f"(qy)
        : "f"(x), "f"(y), "f"(r), "f"(-s), "f"(most), "f"(z));
  }
  template <int VEC>
  __device__ __forceinline__ void store(uint8_t* p, const float (&x)[VEC]) const {
    float q[VEC];
#pragma unroll
    for (int i = 0; i < VEC; i += 2) {
      float odd;  // VEC 1: the same element twice
      divide2(x[i], x[VEC > 1 ? i + 1 : i], q[i], VEC > 1 ? q[(i + 1) % VEC] : odd);
    }
    if constexpr (VEC == 1) {
      *p = __nv_cvt_float_to_fp8(q[0], __NV_SATFINITE, __NV_E4M3);
    } else {
      uint32_t w[VEC / 4];
#pragma unroll
      for (int i = 0; i < VEC; i += 4)
        w[i / 4] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(q[i], q[i + 1]), __NV_SATFINITE,
                                                      __NV_E4M3) |
                   (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(q[i + 2], q[i + 3]),
                                                      __NV_SATFINITE, __NV_E4M3) << 16;
      if constexpr (VEC == 8)
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
      else
        *reinterpret_cast<uint32_t*>(p) = w[0];
    }
  }
};

template <int VEC>
__device__ __forceinline__ void load_table(const float* p, float (&x)[VEC]) {
  if constexpr (VEC % 4 == 0) {
#pragma unroll
    for (int k = 0; k < VEC; k += 4) {
      const float4 v = *reinterpret_cast<const float4*>(p + k);
      x[k] = v.x, x[k + 1] = v.y, x[k + 2] = v.z, x[k + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < VEC; ++k) x[k] = p[k];
  }
}

// Rotates VEC pairs in place: (a[i], b[i]), or side by side, (a[2i], a[2i + 1])
// and then (b[2i], b[2i + 1]).
template <bool INTER, int VEC>
__device__ __forceinline__ void rotate_pairs(float (&a)[VEC], float (&b)[VEC], const float* cosines,
                                             const float* sines) {
  float co[VEC], si[VEC];
  load_table<VEC>(cosines, co);
  load_table<VEC>(sines, si);
  if constexpr (INTER && VEC > 1) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      float& xa = i < VEC / 2 ? a[2 * i % VEC] : b[2 * i % VEC];
      float& xb = i < VEC / 2 ? a[2 * i % VEC + 1] : b[2 * i % VEC + 1];
      const float va = xa, vb = xb;
      xa = fmaf(va, co[i], -(vb * si[i]));
      xb = fmaf(vb, co[i], va * si[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const float va = a[i], vb = b[i];
      a[i] = fmaf(va, co[i], -(vb * si[i]));
      b[i] = fmaf(vb, co[i], va * si[i]);
    }
  }
}

// A row is tasks = head_dim / (2 VEC) tasks (rounded up) of two vectors: the
// rotated ones hold both members of VEC pairs, the others neighbouring vectors
// past rot_dim; of a value row, task c holds vectors c and c + tasks.
template <typename T, int MODE, bool INTER, int VEC, int U>
__global__ void __launch_bounds__(kThreads, 4) rotary_kernel(const RotaryParams p) {
  extern __shared__ float table[];  // cosines [tokens][rot_dim / 2], then sines
  if (MODE != kRotate && p.early) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int heads = p.end[2], D = p.head_dim, half = p.rot_dim / 2;
  const int nrot = half / VEC;
  const int rin = p.by_tasks.div(threadIdx.x), c = threadIdx.x - rin * p.tasks;
  const int64_t r0 = (int64_t)blockIdx.x * (p.rows_per_pass * U);
  const int64_t t0 = p.rows <= UINT32_MAX ? (int64_t)((uint32_t)r0 / (uint32_t)heads) : r0 / heads;
  const int h0 = (int)(r0 - t0 * heads);
  const int block_rows = (int)min((int64_t)p.rows_per_pass * U, p.rows - r0);
  const int tokens = p.by_heads.div(h0 + block_rows - 1) + 1;

  // Elements of a vector of the row: first and second of a rotated row's task.
  const bool rotates = c < nrot;
  const int oa = rotates && !INTER ? c * VEC : 2 * c * VEC;  // rot_dim is 2 nrot VEC
  const int ob = rotates && !INTER ? oa + half : oa + VEC;
  // The loads of this thread's tasks, and where they lie: the token's place in
  // the block (below 4 * kThreads), the head of q, k or v, and which of the three.
  Raw<T, VEC> x0[U], x1[U];
  uint32_t where[U];
  int64_t slot[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int r = rin + u * p.rows_per_pass;
    where[u] = kNoRow;
    if (rin >= p.rows_per_pass || r >= block_rows) continue;
    const int tok = p.by_heads.div(h0 + r), h = h0 + r - tok * heads;
    const int kind = h < p.end[0] ? 0 : h < p.end[1] ? 1 : 2;
    const int head = h - (kind == 0 ? 0 : p.end[kind - 1]);
    where[u] = (uint32_t)(tok << 16 | head << 2 | kind);
    const int64_t t = t0 + tok;
    const T* src =
        static_cast<const T*>(p.src[kind]) + t * p.src_stride[kind] + (int64_t)head * D;
    if (MODE != kRotate) slot[u] = __ldg(p.slot_mapping + t);
    if (MODE != kRotate && kind == 2) {
      x0[u].load(src + c * VEC);
      if ((c + p.tasks) * VEC < D) x1[u].load(src + (c + p.tasks) * VEC);
    } else {
      x0[u].load(src + oa);
      if (ob < D) x1[u].load(src + ob);
    }
  }

  const E4m3Scale k8(MODE == kAppendFp8 ? __ldg(p.scale[0]) : 1.f);
  const E4m3Scale v8(MODE == kAppendFp8 ? __ldg(p.scale[1]) : 1.f);

  float* const sines = table + tokens * half;
  for (int e = threadIdx.x; e < tokens * half; e += kThreads) {
    const int tk = p.by_half.div(e), i = e - tk * half;
    const double turns = (double)__ldg(p.positions + t0 + tk) * __ldg(p.inv_freq + i) *
                         0.15915494309189533577;  // 1 / (2 pi)
    float s, co;
    sincospif(2.f * (float)(turns - rint(turns)), &s, &co);
    table[e] = co * p.magnitude;
    sines[e] = s * p.magnitude * p.sin_sign;
  }
  __syncthreads();

#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (where[u] == kNoRow) continue;
    const int tok = (int)(where[u] >> 16), head = (int)(where[u] >> 2) & (kMaxHeads - 1);
    const int kind = (int)(where[u] & 3);
    const bool value = MODE != kRotate && kind == 2;
    const bool turn = rotates && !value;
    const int o0 = value ? c * VEC : oa, o1 = value ? (c + p.tasks) * VEC : ob;
    const bool two = o1 < D;
    int64_t off;
    if (MODE != kRotate && kind > 0) {
      if (slot[u] < 0 || slot[u] >= p.num_slots) continue;  // padding
      off = (slot[u] * (p.end[1] - p.end[0]) + head) * D;
    } else {
      off = (t0 + tok) * p.dst_stride[kind & 1] + (int64_t)head * D;
    }
    float a[VEC], b[VEC];
    if (turn || (MODE == kAppendFp8 && kind > 0)) {
      x0[u].get(a);
      x1[u].get(b);
    }
    if (turn) {
      const float* cosines = table + tok * half + c * VEC;
      rotate_pairs<INTER, VEC>(a, b, cosines, cosines + tokens * half);
    }
    if (MODE == kAppendFp8 && kind > 0) {
      uint8_t* dst = static_cast<uint8_t*>(p.dst[kind]) + off;
      const E4m3Scale& to = value ? v8 : k8;
      to.store(dst + o0, a);
      if (two) to.store(dst + o1, b);
    } else {  // what is not rotated keeps its bits
      T* dst = static_cast<T*>(p.dst[kind]) + off;
      if (turn) {
        x0[u].set(a);
        x1[u].set(b);
      }
      x0[u].store(dst + o0);
      if (two) x1[u].store(dst + o1);
    }
  }
}

template <typename T, int MODE, bool INTER, int VEC>
cudaError_t launch_vec(RotaryParams p, cudaStream_t stream) {
  const int D = p.head_dim, r = p.rot_dim;
  p.tasks = (D / VEC + 1) / 2;
  p.rows_per_pass = kThreads / p.tasks;
  p.by_heads = Div::by(p.end[2]);
  p.by_tasks = Div::by(p.tasks);
  p.by_half = Div::by(r / 2);
  const int64_t passes = ceil_div64(p.rows, p.rows_per_pass);
  auto launch = [&](auto kernel, int u) -> cudaError_t {
    const int64_t block_rows = (int64_t)p.rows_per_pass * u;
    const int64_t blocks = ceil_div64(p.rows, block_rows);
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    // Tokens that a block's rows can touch, times a cosine and a sine per pair.
    const int64_t tokens = (block_rows - 1 + p.end[2] - 1) / p.end[2] + 1;
    const size_t smem = (size_t)tokens * r * sizeof(float);
    kernel<<<(unsigned)blocks, kThreads, smem, stream>>>(p);
    return cudaGetLastError();
  };
  // One task per thread until the blocks fill the GPU a few times over, then as
  // many as 64 registers hold the loads of: at four blocks per SM three of 16-bit
  // types (64 q, 8 k/v heads of 128, 8192 tokens: 48.1 us; two take 51.9) and two of
  // fp32 (32/8 heads: 51.9 us; three take 65.8).
  constexpr int kU = sizeof(T) == 4 ? 2 : 3;
  // The table: at most a token per row, kThreads / tasks rows a pass, tasks >= head_dim /
  // (2 VEC), rot_dim <= head_dim. One head of 16, 32 or 512 elements fills all of it.
  static_assert(kThreads * 2 * VEC * kU * sizeof(float) <= 48 << 10, "table without opt-in");
  if (passes <= 148 * 8) return launch(rotary_kernel<T, MODE, INTER, VEC, 1>, 1);
  return launch(rotary_kernel<T, MODE, INTER, VEC, kU>, kU);
}

template <typename T, int MODE, bool INTER>
cudaError_t launch_inter(const RotaryParams& p, cudaStream_t stream) {
  // The widest vector whose pairs, tails and strides all fall on its multiples.
  int64_t all = p.head_dim | p.rot_dim / 2;
  if (p.rows > p.end[2])  // one token has no stride
    all |= p.src_stride[0] | p.src_stride[1] | p.src_stride[2] | p.dst_stride[0] | p.dst_stride[1];
  if ((all & 7) == 0) return launch_vec<T, MODE, INTER, 8>(p, stream);
  if ((all & 3) == 0) return launch_vec<T, MODE, INTER, 4>(p, stream);
  return launch_vec<T, MODE, INTER, 1>(p, stream);
}

template <int MODE>
cudaError_t launch(const RotaryParams& p, int dtype, bool interleaved, cudaStream_t stream) {
  switch (dtype) {
    case PKV_F32:
      return interleaved ? launch_inter<float, MODE, true>(p, stream)
                         : launch_inter<float, MODE, false>(p, stream);
    case PKV_F16:
      return interleaved ? launch_inter<__half, MODE, true>(p, stream)
                         : launch_inter<__half, MODE, false>(p, stream);
    case PKV_BF16:
      return interleaved ? launch_inter<__nv_bfloat16, MODE, true>(p, stream)
                         : launch_inter<__nv_bfloat16, MODE, false>(p, stream);
    default:
      return cudaErrorInvalidValue;
  }
}

constexpr int kMaxHeadDim = 2 * kThreads;  // a row's tasks fit one block

// What the calls have in common: sizes, strides of the given tensors, pointers.
int check(const RotaryParams& p, int num_tokens, int64_t num_heads, int64_t num_kv_heads,
          int dtype, unsigned flags, unsigned allowed) {
  const int64_t D = p.head_dim;
  if (num_tokens < 0 || num_heads < 0 || num_kv_heads < 0 || D <= 0 || D % 8 != 0 ||
      p.rot_dim <= 0 || p.rot_dim % 2 != 0 || p.rot_dim > D || !isfinite(p.magnitude) ||
      (flags & ~allowed))
    return PKV_ERR_SHAPE;
  if (num_heads + 2 * num_kv_heads > kMaxHeads) return PKV_ERR_SHAPE;
  if (D > kMaxHeadDim) return PKV_ERR_UNSUPPORTED;
  if (dtype != PKV_F32 && dtype != PKV_F16 && dtype != PKV_BF16) return PKV_ERR_DTYPE;
  for (int64_t s : p.src_stride)
    if (s < 0) return PKV_ERR_SHAPE;
  // Written rows of different tokens must not overlap.
  if (num_tokens > 1 && ((num_heads > 0 && p.dst_stride[0] < num_heads * D) ||
                         (p.dst[1] && p.dst_stride[1] < num_kv_heads * D)))
    return PKV_ERR_SHAPE;
  for (int i = 0; i < 2; ++i)  // in place: row for row
    if (p.dst[i] && p.dst[i] == p.src[i] && num_tokens > 1 && p.dst_stride[i] != p.src_stride[i])
      return PKV_ERR_SHAPE;
  return PKV_OK;
}

bool aligned(const void* q, uintptr_t to) { return ((uintptr_t)q & (to - 1)) == 0; }

}  // namespace
}  // namespace rot
}  // namespace pkv

using namespace pkv;

extern "C" {

int pkv_rotary_inv_freq(double* inv_freq, float* magnitude, int rot_dim, double base, int scaling,
                        double factor, double trained_len, double low, double high) {
  if (!inv_freq || !magnitude) return PKV_ERR_NULL;
  if (rot_dim <= 0 || rot_dim % 2 != 0 || rot_dim > rot::kMaxHeadDim) return PKV_ERR_SHAPE;
  if (!(base > 1.0) || !isfinite(base)) return PKV_ERR_SHAPE;
  const bool bands = scaling == PKV_ROTARY_SCALE_RAMP || scaling == PKV_ROTARY_SCALE_BANDED;
  if (scaling != PKV_ROTARY_SCALE_NONE && (!(factor > 0.0) || !isfinite(factor)))
    return PKV_ERR_SHAPE;
  if (bands && (!(trained_len > 0.0) || !isfinite(trained_len) || !(low > 0.0) || !(high > low) ||
                !isfinite(high)))
    return PKV_ERR_SHAPE;
  const double r = rot_dim, two_pi = 6.283185307179586477;
  double b = base, ramp_lo = 0, ramp_hi = 0;
  float m = 1.f;
  switch (scaling) {
    case PKV_ROTARY_SCALE_NONE:
    case PKV_ROTARY_SCALE_LINEAR:
    case PKV_ROTARY_SCALE_BANDED:
      break;
    case PKV_ROTARY_SCALE_BASE:
      if (rot_dim <= 2) return PKV_ERR_SHAPE;
      b = base * pow(factor, r / (r - 2.0));
      if (!(b > 0.0) || !isfinite(b)) return PKV_ERR_SHAPE;
      break;
    case PKV_ROTARY_SCALE_RAMP: {
      // The pair index at which a pair makes `turns` turns over trained_len.
      auto index = [&](double turns) {
        return r * log(trained_len / (turns * two_pi)) / (2.0 * log(base));
      };
      ramp_lo = fmax(floor(index(high)), 0.0);
      ramp_hi = fmin(ceil(index(low)), r - 1.0);
      m = (float)(factor > 1.0 ? 0.1 * log(factor) + 1.0 : 1.0);
      break;
    }
    default:
      return PKV_ERR_UNSUPPORTED;
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    const double f = pow(b, -2.0 * i / r);
    double share = 0.0;  // of the frequency divided by the factor
    if (scaling == PKV_ROTARY_SCALE_LINEAR)
      share = 1.0;
    else if (scaling == PKV_ROTARY_SCALE_RAMP)
      share = fmin(fmax((i - ramp_lo) / fmax(ramp_hi - ramp_lo, 1e-3), 0.0), 1.0);
    else if (scaling == PKV_ROTARY_SCALE_BANDED)
      share = 1.0 - fmin(fmax((trained_len * f / two_pi - low) / (high - low), 0.0), 1.0);
    inv_freq[i] = share > 0.0 ? f * (share / factor + (1.0 - share)) : f;
  }
  *magnitude = m;
  return PKV_OK;
}

int pkv_rotary(void* q_out, const void* query, void* k_out, const void* key,
               const int64_t* positions, const double* inv_freq, float magnitude, int num_tokens,
               int num_heads, int num_kv_heads, int head_dim, int rot_dim, int64_t q_stride,
               int64_t q_out_stride, int64_t k_stride, int64_t k_out_stride, int dtype,
               unsigned flags, void* stream) {
  rot::RotaryParams p = {};
  p.src[0] = query, p.src[1] = key;
  p.dst[0] = q_out, p.dst[1] = k_out;
  p.src_stride[0] = q_stride, p.src_stride[1] = k_stride;
  p.dst_stride[0] = q_out_stride, p.dst_stride[1] = k_out_stride;
  p.head_dim = head_dim, p.rot_dim = rot_dim;
  p.magnitude = magnitude;
  const int st = rot::check(p, num_tokens, num_heads, num_kv_heads, dtype, flags,
                            PKV_ROTARY_INTERLEAVED | PKV_ROTARY_TRANSPOSED);
  if (st != PKV_OK) return st;
  if (num_tokens == 0 || num_heads + num_kv_heads == 0) return PKV_OK;
  if (!positions || !inv_freq || (num_heads > 0 && (!q_out || !query)) ||
      (num_kv_heads > 0 && (!k_out || !key)))
    return PKV_ERR_NULL;
  if (!rot::aligned(q_out, 16) || !rot::aligned(query, 16) || !rot::aligned(k_out, 16) ||
      !rot::aligned(key, 16) || !rot::aligned(positions, 8) || !rot::aligned(inv_freq, 8))
    return PKV_ERR_ALIGN;
  p.end[0] = num_heads, p.end[1] = p.end[2] = num_heads + num_kv_heads;
  p.positions = positions, p.inv_freq = inv_freq;
  p.rows = (int64_t)num_tokens * p.end[2];
  p.sin_sign = flags & PKV_ROTARY_TRANSPOSED ? -1.f : 1.f;
  return rot::launch<rot::kRotate>(p, dtype, flags & PKV_ROTARY_INTERLEAVED,
                                   (cudaStream_t)stream) == cudaSuccess
             ? PKV_OK
             : PKV_ERR_CUDA;
}

int paged_kv_append_rotary(void* q_out, const void* query, const void* key, const void* value,
                           void* k_cache, void* v_cache, const int64_t* slot_mapping,
                           const int64_t* positions, const double* inv_freq, float magnitude,
                           int num_tokens, int num_heads, int num_kv_heads, int head_dim,
                           int rot_dim, int block_size, int64_t num_blocks, int64_t q_stride,
                           int64_t q_out_stride, int64_t k_stride, int64_t v_stride,
                           int src_dtype, int cache_dtype, const float* k_scale,
                           const float* v_scale, unsigned flags, void* stream) {
  rot::RotaryParams p = {};
  p.src[0] = query, p.src[1] = key, p.src[2] = value;
  p.dst[0] = q_out;
  p.src_stride[0] = q_stride, p.src_stride[1] = k_stride, p.src_stride[2] = v_stride;
  p.dst_stride[0] = q_out_stride;
  p.head_dim = head_dim, p.rot_dim = rot_dim;
  p.magnitude = magnitude;
  const int st = rot::check(p, num_tokens, num_heads, num_kv_heads, src_dtype, flags,
                            PKV_ROTARY_INTERLEAVED);
  if (st != PKV_OK) return st;
  if (num_kv_heads == 0 || block_size <= 0 || num_blocks <= 0 ||
      num_blocks > INT64_MAX / block_size)
    return PKV_ERR_SHAPE;
  if (cache_dtype != src_dtype && cache_dtype != PKV_FP8_E4M3) return PKV_ERR_DTYPE;
  const bool fp8 = cache_dtype == PKV_FP8_E4M3;
  if (num_tokens == 0) return PKV_OK;
  if (!key || !value || !k_cache || !v_cache || !slot_mapping || !positions || !inv_freq ||
      (num_heads > 0 && (!q_out || !query)) || (fp8 && (!k_scale || !v_scale)))
    return PKV_ERR_NULL;
  if (!rot::aligned(q_out, 16) || !rot::aligned(query, 16) || !rot::aligned(key, 16) ||
      !rot::aligned(value, 16) || !rot::aligned(k_cache, 16) || !rot::aligned(v_cache, 16) ||
      !rot::aligned(slot_mapping, 8) || !rot::aligned(positions, 8) ||
      !rot::aligned(inv_freq, 8) ||
      (fp8 && (!rot::aligned(k_scale, 4) || !rot::aligned(v_scale, 4))))
    return PKV_ERR_ALIGN;
  p.dst[1] = k_cache, p.dst[2] = v_cache;
  p.end[0] = num_heads, p.end[1] = num_heads + num_kv_heads, p.end[2] = p.end[1] + num_kv_heads;
  p.positions = positions, p.inv_freq = inv_freq, p.slot_mapping = slot_mapping;
  p.scale[0] = k_scale, p.scale[1] = v_scale;
  p.num_slots = num_blocks * (int64_t)block_size;
  p.rows = (int64_t)num_tokens * p.end[2];
  p.sin_sign = 1.f;
  p.early = num_heads == 0;
  const bool inter = flags & PKV_ROTARY_INTERLEAVED;
  const cudaError_t e = fp8 ? rot::launch<rot::kAppendFp8>(p, src_dtype, inter, (cudaStream_t)stream)
                            : rot::launch<rot::kAppend>(p, src_dtype, inter, (cudaStream_t)stream);
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // extern "C"
