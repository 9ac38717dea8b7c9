// Rows of activations (or of weights) to 8-bit integers with one scale each,
// and the dispatch that does it on the way.
//
//   s = max_j |x_j| / 127 (fp32)      q_j = x_j / s, to nearest, ties to even
//
// The rounding is decided on the exact quotient, so q is a function of x
// alone and not of how a reciprocal rounds. t = x c + 1.5 2^23 in one fma
// rounds to an integer, with c within a few steps (2^-24 each) of 1 / s; that
// is x / s rounded unless x / s lies that close to a border m / 2, m odd.
// - fp32: the remainder x - t s is exact in one fma (t s and x agree to a step,
//   so their difference fits 24 bits); where its double reaches s the element
//   is rounded again with care.
// - bf16: with integer significands below 2^8, x = X 2^i, max = M 2^(i+k), and
//   Q = 127 x / max = 127 X / (M 2^k) is m / 2 or at least 1 / (2 M 2^k) >=
//   2^-9 2^-k away from it, where all the errors (of c, and of s against
//   max / 127) come to less than 2^-15 2^-k. Only where Q is m / 2 itself does the
//   side count, and there x / s lies below m / 2 if s was rounded up, above if
//   down: c is taken strictly below or above 127 / max accordingly (and is
//   exact where s is), and no element needs a check.
// Bound by HBM: it reads each element once and writes one byte for it. On a B200,
// bf16, buffers in turn so that none is in L2: 10240 x 4096 in 23.6 us (5.3 TB/s,
// 81% of a copy's rate; with fp32's remainder check for bf16 too 31.9), 131072 x
// 1024 in 72 us (5.6 TB/s, 85%). Odd columns (or rows off 16-byte boundaries) go
// element by element: 32768 x 1001 in 66 us, x 1000 in 22.
//
// "Expert choice routing" (aicassindra.com), "The math": X_in[e] = P[e] X. A
// permutation of rows commutes with a scale per row, so the dispatch gathers
// bytes and scales instead of activations.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "block_internal.h"
#include "device_common.cuh"

namespace moe {
namespace {

// ---- VEC consecutive elements: 16 bytes read (VEC > 1), VEC bytes written ----
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <typename T, int VEC>
struct QChunk;
template <>
struct QChunk<__nv_bfloat16, 8> {
  uint4 r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    r = __ldcs(reinterpret_cast<const uint4*>(p));
  }
  __device__ __forceinline__ void zero() { r = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ float get(int i) const {
    const uint32_t w = i < 2 ? r.x : i < 4 ? r.y : i < 6 ? r.z : r.w;
    return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
  }
  // the largest magnitude; NaN where there is one
  __device__ __forceinline__ float most() const {
    auto h = [](uint32_t w) { return __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w)); };
    const __nv_bfloat162 m =
        __hmax2_nan(__hmax2_nan(h(r.x), h(r.y)), __hmax2_nan(h(r.z), h(r.w)));
    return max_nan(__low2float(m), __high2float(m));
  }
};
template <>
struct QChunk<float, 4> {
  float4 r;
  __device__ __forceinline__ void load(const float* p) {
    r = __ldcs(reinterpret_cast<const float4*>(p));
  }
  __device__ __forceinline__ void zero() { r = make_float4(0, 0, 0, 0); }
  __device__ __forceinline__ float get(int i) const {
    return i == 0 ? r.x : i == 1 ? r.y : i == 2 ? r.z : r.w;
  }
  __device__ __forceinline__ float most() const {
    return max_nan(max_nan(fabsf(r.x), fabsf(r.y)), max_nan(fabsf(r.z), fabsf(r.w)));
  }
};
template <>
struct QChunk<__nv_bfloat16, 1> {
  uint16_t r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    r = *reinterpret_cast<const uint16_t*>(p);
  }
  __device__ __forceinline__ void zero() { r = 0; }
  __device__ __forceinline__ float get(int) const { return bf16_to_f32(r); }
  __device__ __forceinline__ float most() const { return fabsf(get(0)); }
};
template <>
struct QChunk<float, 1> {
  float r;
  __device__ __forceinline__ void load(const float* p) { r = *p; }
  __device__ __forceinline__ void zero() { r = 0.0f; }
  __device__ __forceinline__ float get(int) const { return r; }
  __device__ __forceinline__ float most() const { return fabsf(r); }
};

// Magnitudes, a NaN above all, compare as their bit patterns.
__device__ __forceinline__ uint32_t warp_most(float v) {
  return __reduce_max_sync(~0u, __float_as_uint(v) & 0x7fffffffu);
}

enum { ROW_PLAIN, ROW_DEAD, ROW_TINY };
struct RowScale {
  float s, c;
  // DEAD: a row of zeros, or one that is not finite: all q are 0.
  // TINY: 1 / s may not be a normal number, the quotient is taken by division
  int kind;
};

template <typename T>
__device__ __forceinline__ RowScale row_scale(uint32_t most) {
  RowScale r;
  const bool finite = most < 0x7f800000u;
  const float max = __uint_as_float(most);
  r.s = finite ? __fdiv_rn(max, 127.0f) : __uint_as_float(0x7fffffffu);
  r.kind = !finite || r.s == 0.0f ? ROW_DEAD : r.s < 0x1p-100f ? ROW_TINY : ROW_PLAIN;
  r.c = 0.0f;
  if (r.kind == ROW_PLAIN) {
    if (sizeof(T) == 2) {
      const float over = __fmaf_rn(127.0f, r.s, -max);  // exact: s was rounded up or down
      const float c = __fdiv_rn(127.0f, max);           // two steps off it is past 127 / max
      r.c = over == 0.0f ? c : __int_as_float(__float_as_int(c) + (over > 0.0f ? -2 : 2));
    } else {
      r.c = __fdiv_rn(1.0f, r.s);
    }
  }
  return r;
}

constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: adding it rounds to an integer

// x / s to the nearest integer, ties to even, from a candidate t at most one off
__device__ __forceinline__ float fix_round(float x, float t, float s) {
  const float r2 = 2.0f * fmaf(-t, s, x);
  const float odd = t - 2.0f * floorf(t * 0.5f);
  if (r2 > s || (r2 == s && odd != 0.0f)) t += 1.0f;
  else if (r2 < -s || (r2 == -s && odd != 0.0f)) t -= 1.0f;
  return t;
}

// The rows that the fast path leaves: dead ones, and those of a tiny scale (a
// few steps coarse as a denormal, so that the quotient may pass 127).
template <typename T, int VEC>
__device__ __noinline__ uint64_t quantize_slow(const QChunk<T, VEC> c, float s, int kind) {
  uint64_t out = 0;
  if (kind == ROW_DEAD) return 0;
  for (int j = 0; j < VEC; ++j) {
    const float x = c.get(j);
    const float t = fix_round(x, rintf(__fdiv_rn(x, s)), s);
    out |= (uint64_t)(uint8_t)(int8_t)(int)fminf(fmaxf(t, -127.0f), 127.0f) << (8 * j);
  }
  return out;
}

// VEC bytes: the low bytes of x c + kMagic (|t| <= 127, as |x| <= 127 s (1 + 2^-24)).
template <typename T, int VEC>
__device__ __forceinline__ uint64_t quantize(const QChunk<T, VEC>& c, const RowScale& k) {
  if (k.kind != ROW_PLAIN) return quantize_slow<T, VEC>(c, k.s, k.kind);
  uint32_t b[VEC];
  float far = 0.0f;
  if constexpr (VEC == 1) {
    const float v = __fmaf_rn(c.get(0), k.c, kMagic);
    b[0] = __float_as_uint(v);
    if (sizeof(T) == 4) far = fabsf(__fmaf_rn(kMagic - v, k.s, c.get(0)));
  } else {
    const float2 cc = make_float2(k.c, k.c), s = make_float2(k.s, k.s);
#pragma unroll
    for (int j = 0; j < VEC; j += 2) {
      const float2 x = make_float2(c.get(j), c.get(j + 1));
      const float2 v = __ffma2_rn(x, cc, make_float2(kMagic, kMagic));
      b[j] = __float_as_uint(v.x);
      b[j + 1] = __float_as_uint(v.y);
      if constexpr (sizeof(T) == 4) {
        // (kMagic - v is exact)
        const float2 r = __ffma2_rn(
            __ffma2_rn(v, make_float2(-1.0f, -1.0f), make_float2(kMagic, kMagic)), s, x);
        far = fmaxf(far, fmaxf(fabsf(r.x), fabsf(r.y)));
      }
    }
  }
  if (sizeof(T) == 4 && 2.0f * far >= k.s) {
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      b[j] = __float_as_uint(fix_round(c.get(j), __uint_as_float(b[j]) - kMagic, k.s) + kMagic);
  }
  if constexpr (VEC == 1) {
    return b[0] & 0xff;
  } else {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < VEC; j += 4)
      w[j / 4] = __byte_perm(__byte_perm(b[j], b[j + 1], 0x0040),
                             __byte_perm(b[j + 2], b[j + 3], 0x0040), 0x5410);
    return (uint64_t)w[1] << 32 | w[0];
  }
}

template <int VEC>
__device__ __forceinline__ void store_bytes(int8_t* p, uint64_t v) {
  if constexpr (VEC == 8) *reinterpret_cast<uint64_t*>(p) = v;
  else if constexpr (VEC == 4) *reinterpret_cast<uint32_t*>(p) = (uint32_t)v;
  else *p = (int8_t)v;
}

// ---------------------------------------------------------------------------
// quantise rows
// ---------------------------------------------------------------------------
struct QuantArgs {
  const void* x;
  int8_t* q;
  float* scale;
  long long rows;
  int cols;
  const int32_t *starts, *counts;
  int groups;
};

constexpr int kQWarps = 8;

// The rows of the groups, in order, in one contiguous run for each row owner
// (a warp, or with BLOCK the whole block). A row stays in registers between
// the maximum and the rounding, and the next one is loaded meanwhile. ITEMS ==
// 0: a row longer than the registers of a block is read twice.
template <typename T, int VEC, int ITEMS, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 1024 : 32 * kQWarps) quantize_kernel(const QuantArgs a) {
  __shared__ int start[MOE_I8_MAX_GROUPS];
  __shared__ long long prefix[MOE_I8_MAX_GROUPS + 1];  // rows of the groups before g
  __shared__ uint32_t red[2][32];
  pdl_wait();
  if (gridDim.x <= kBlockSms) pdl_trigger();
  const int lane = threadIdx.x & 31;
  long long total = a.rows;
  if (a.starts) {
    for (int g = threadIdx.x; g < a.groups; g += blockDim.x) {
      const int s0 = a.starts[g];
      const long long room = s0 < 0 ? 0 : a.rows - s0;  // a group outside the buffers is cut
      start[g] = s0;
      prefix[g + 1] = max(0LL, min((long long)a.counts[g], room));
    }
    __syncthreads();
    if (threadIdx.x < 32) {  // running sum, 32 groups at a time
      long long run = 0;
      for (int g0 = 0; g0 < a.groups; g0 += 32) {
        const int g = g0 + lane;
        long long v = g < a.groups ? prefix[g + 1] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long u = __shfl_up_sync(~0u, v, o);
          if (lane >= o) v += u;
        }
        if (g < a.groups) prefix[g + 1] = run + v;
        run += __shfl_sync(~0u, v, 31);
      }
      if (lane == 0) prefix[0] = 0;
    }
    __syncthreads();
    total = prefix[a.groups];
  }
  const int owners = BLOCK ? gridDim.x : gridDim.x * kQWarps;
  const int owner = BLOCK ? blockIdx.x : blockIdx.x * kQWarps + (threadIdx.x >> 5);
  const int tid = BLOCK ? threadIdx.x : lane;
  const int threads = BLOCK ? blockDim.x : 32;
  const int chunks = a.cols / VEC;
  const long long first = total * owner / owners, last = total * (owner + 1) / owners;
  if (first >= last) return;
  // the row being loaded, and the rows left after it in its group
  int g = 0;
  long long row = first, left = last - first - 1;
  if (a.starts) {
    int hi = a.groups - 1;
    while (g < hi) {
      const int mid = (g + hi + 1) >> 1;
      if (prefix[mid] <= first) g = mid; else hi = mid - 1;
    }
    row = start[g] + (first - prefix[g]);
    left = prefix[g + 1] - first - 1;
  }
  QChunk<T, VEC> ahead[ITEMS > 0 ? ITEMS : 1];
  const T* x = static_cast<const T*>(a.x) + (size_t)row * a.cols + (size_t)tid * VEC;
  auto fetch = [&]() {
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      ahead[k].zero();
      if (k * threads + tid < chunks) ahead[k].load(x + (size_t)k * threads * VEC);
    }
  };
  fetch();
  for (int i = (int)(last - first); i > 0; --i) {
    int8_t* q = a.q + (size_t)row * a.cols + (size_t)tid * VEC;
    float* scale = a.scale + row;
    QChunk<T, VEC> c[ITEMS > 0 ? ITEMS : 1];
    float m = 0.0f;
    if constexpr (ITEMS > 0) {
#pragma unroll
      for (int k = 0; k < ITEMS; ++k) c[k] = ahead[k];
    } else {
      for (int p = tid; p < chunks; p += threads) {
        c[0].load(x + (size_t)(p - tid) * VEC);
        m = max_nan(m, c[0].most());
      }
    }
    const T* now = x;
    if (i > 1) {
      if (left > 0) {
        --left;
        ++row;
        x += a.cols;
      } else {  // the next group that has a row
        do ++g;
        while (prefix[g + 1] == prefix[g]);
        row = start[g];
        left = prefix[g + 1] - prefix[g] - 1;
        x = static_cast<const T*>(a.x) + (size_t)row * a.cols + (size_t)tid * VEC;
      }
      fetch();
    }
    if constexpr (ITEMS > 0) {
#pragma unroll
      for (int k = 0; k < ITEMS; ++k) m = max_nan(m, c[k].most());
    }
    uint32_t most = warp_most(m);
    if (BLOCK) {
      if (lane == 0) red[i & 1][threadIdx.x >> 5] = most;
      __syncthreads();
      most = __reduce_max_sync(~0u, lane < (int)(blockDim.x >> 5) ? red[i & 1][lane] : 0u);
    }
    const RowScale k = row_scale<T>(most);
    if (tid == 0) *scale = k.s;
    if constexpr (ITEMS > 0) {
#pragma unroll
      for (int j = 0; j < ITEMS; ++j)
        if (j * threads + tid < chunks)
          store_bytes<VEC>(q + (size_t)j * threads * VEC, quantize<T, VEC>(c[j], k));
    } else {
      for (int p = tid; p < chunks; p += threads) {
        c[0].load(now + (size_t)(p - tid) * VEC);
        store_bytes<VEC>(q + (size_t)(p - tid) * VEC, quantize<T, VEC>(c[0], k));
      }
    }
  }
}

template <typename T, int VEC, int ITEMS, bool BLOCK>
cudaError_t run_quant(const QuantArgs& a, int threads, cudaStream_t s) {
  // resident blocks: 1,024 threads an SM, in up to 16 blocks
  const long long per_block = BLOCK ? 1 : kQWarps;
  const int resident = 1024 / threads > 16 ? 16 : 1024 / threads;
  long long grid = (a.rows + per_block - 1) / per_block;
  if (grid > (long long)kBlockSms * resident) grid = (long long)kBlockSms * resident;
  return launch_pdl(quantize_kernel<T, VEC, ITEMS, BLOCK>, dim3((unsigned)grid), dim3(threads), 0,
                    s, a);
}

// A warp a row while a lane holds up to 2 vectors (4 of fp32), then a block a row
// with up to 4 vectors a thread. 131072 rows, us, warp against block: bf16 512
// columns 37.9 / 50.8 (with room for 4 vectors a lane 54.0), 1024 columns, 4 vectors,
// 78.7 / 71.8; fp32 256 columns 32.9 / 48.5, 512 columns, 4 vectors, 58.4 / 64.1.
template <typename T, int VEC>
cudaError_t launch_quant(const QuantArgs& a, cudaStream_t s) {
  const int chunks = a.cols / VEC;
  if (chunks <= 32) return run_quant<T, VEC, 1, false>(a, 32 * kQWarps, s);
  if (chunks <= 32 * 2) return run_quant<T, VEC, 2, false>(a, 32 * kQWarps, s);
  if (VEC < 8 && chunks <= 32 * 4) return run_quant<T, VEC, 4, false>(a, 32 * kQWarps, s);
  if (chunks <= 1024 * 4)
    return run_quant<T, VEC, 4, true>(a, ((chunks + 3) / 4 + 31) / 32 * 32, s);
  return run_quant<T, VEC, 0, true>(a, 1024, s);
}

// ---------------------------------------------------------------------------
// dispatch of quantised rows: one block a token
// ---------------------------------------------------------------------------
struct DispatchI8 {
  const void* X;
  const int32_t *tok_row, *offsets, *counts_in;
  int8_t* q;
  float* scale;
  int32_t *starts, *counts;
  int n, d, E, n_shared, slots, shared_base, n_pad;
};

template <typename T, int VEC, int ITEMS>
__global__ void __launch_bounds__(1024) dispatch_i8_kernel(const DispatchI8 a) {
  __shared__ uint32_t red[32];
  __shared__ int dst[MOE_MAX_EXPERTS + MOE_MAX_SHARED];
  pdl_wait();
  if (gridDim.x <= kBlockSms) pdl_trigger();
  const int tid = threadIdx.x, threads = blockDim.x, lane = tid & 31;
  if (blockIdx.x == 0) {
    for (int g = tid; g < a.E + a.n_shared; g += threads) {
      a.starts[g] = g < a.E ? a.offsets[g] : a.shared_base + (g - a.E) * a.n_pad;
      a.counts[g] = g < a.E ? a.counts_in[g] : a.n;
    }
  }
  const int t = blockIdx.x;
  const int targets = a.slots + a.n_shared;
  for (int j = tid; j < targets; j += threads) {
    int r;
    if (j < a.slots) {
      r = a.tok_row[(size_t)t * a.slots + j];
      if (r >= a.shared_base) r = -1;  // (outside the routed rows)
    } else {
      r = a.shared_base + (j - a.slots) * a.n_pad + t;
    }
    dst[j] = r;
  }
  const T* x = static_cast<const T*>(a.X) + (size_t)t * a.d;
  const int chunks = a.d / VEC;
  QChunk<T, VEC> c[ITEMS > 0 ? ITEMS : 1];
  float m = 0.0f;
  if constexpr (ITEMS > 0) {
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      const int p = k * threads + tid;
      c[k].zero();
      if (p < chunks) c[k].load(x + (size_t)p * VEC);
    }
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) m = max_nan(m, c[k].most());
  } else {
    for (int p = tid; p < chunks; p += threads) {
      c[0].load(x + (size_t)p * VEC);
      m = max_nan(m, c[0].most());
    }
  }
  uint32_t most = warp_most(m);
  if (lane == 0) red[tid >> 5] = most;
  __syncthreads();
  most = __reduce_max_sync(~0u, lane < threads / 32 ? red[lane] : 0u);
  const RowScale k = row_scale<T>(most);
  for (int j = tid; j < targets; j += threads)
    if (dst[j] >= 0) a.scale[dst[j]] = k.s;
  auto put = [&](int p, uint64_t bytes) {
    for (int j = 0; j < targets; ++j)
      if (dst[j] >= 0) store_bytes<VEC>(a.q + (size_t)dst[j] * a.d + (size_t)p * VEC, bytes);
  };
  if constexpr (ITEMS > 0) {
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
      const int p = j * threads + tid;
      if (p < chunks) put(p, quantize<T, VEC>(c[j], k));
    }
  } else {
    for (int p = tid; p < chunks; p += threads) {
      c[0].load(x + (size_t)p * VEC);
      put(p, quantize<T, VEC>(c[0], k));
    }
  }
}

template <typename T, int VEC>
cudaError_t launch_dispatch(const DispatchI8& a, cudaStream_t s) {
  const int chunks = a.d / VEC;
  if (chunks <= 4 * 1024) {
    const int threads = ((chunks + 3) / 4 + 31) / 32 * 32;
    return launch_pdl(dispatch_i8_kernel<T, VEC, 4>, dim3(a.n), dim3(threads), 0, s, a);
  }
  return launch_pdl(dispatch_i8_kernel<T, VEC, 0>, dim3(a.n), dim3(1024), 0, s, a);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_quantize_rows(long long rows, int cols, moe_dtype dtype, const void* x, int8_t* q,
                             float* scale, const int32_t* starts, const int32_t* counts,
                             int groups, moe_stream_t stream) {
  if (rows < 0 || cols < 1 || (dtype != MOE_F32 && dtype != MOE_BF16)) return MOE_ERR_INVALID_ARG;
  if ((starts != nullptr) != (counts != nullptr)) return MOE_ERR_INVALID_ARG;
  if (starts && (groups < 1 || groups > MOE_I8_MAX_GROUPS || rows > 0x7fffffff))
    return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!x || !q || !scale) return MOE_ERR_INVALID_ARG;
  const uintptr_t xa = reinterpret_cast<uintptr_t>(x);
  if ((xa & (dtype == MOE_BF16 ? 1 : 3)) || (reinterpret_cast<uintptr_t>(scale) & 3))
    return MOE_ERR_INVALID_ARG;
  QuantArgs a{x, q, scale, rows, cols, starts, counts, starts ? groups : 0};
  // vectors: rows on 16-byte boundaries, their bytes on as many as a vector has
  const int vec = dtype == MOE_BF16 ? 8 : 4;
  const bool wide =
      cols % vec == 0 && aligned16(x) && reinterpret_cast<uintptr_t>(q) % vec == 0;
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e;
  if (dtype == MOE_BF16)
    e = wide ? launch_quant<__nv_bfloat16, 8>(a, s) : launch_quant<__nv_bfloat16, 1>(a, s);
  else
    e = wide ? launch_quant<float, 4>(a, s) : launch_quant<float, 1>(a, s);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_dispatch_i8(const moe_dispatch_i8_config* c, const void* X,
                           const moe_route_out* route, int8_t* q, float* scale, int32_t* starts,
                           int32_t* counts, moe_stream_t stream) {
  if (!c || c->n < 1 || c->d < 16 || c->d % 16 || c->E < 1 || c->slots < 1) return MOE_ERR_INVALID_ARG;
  if (c->n_shared < 0 || c->n_shared > MOE_MAX_SHARED || c->rows < 1 || c->shared_row_base < 0)
    return MOE_ERR_INVALID_ARG;
  if (c->dtype != MOE_F32 && c->dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (c->E > MOE_MAX_EXPERTS || c->slots > MOE_MAX_EXPERTS) return MOE_ERR_UNSUPPORTED;
  const long long n_pad = ((long long)c->n + MOE_ROW_ALIGN - 1) / MOE_ROW_ALIGN * MOE_ROW_ALIGN;
  if (c->shared_row_base + c->n_shared * n_pad > c->rows) return MOE_ERR_INVALID_ARG;
  if (!X || !route || !route->tok_row || !route->offsets || !route->counts || !q || !scale ||
      !starts || !counts)
    return MOE_ERR_INVALID_ARG;
  if (!aligned16(X) || !aligned16(q)) return MOE_ERR_INVALID_ARG;
  DispatchI8 a{};
  a.X = X;
  a.tok_row = route->tok_row;
  a.offsets = route->offsets;
  a.counts_in = route->counts;
  a.q = q;
  a.scale = scale;
  a.starts = starts;
  a.counts = counts;
  a.n = c->n;
  a.d = c->d;
  a.E = c->E;
  a.n_shared = c->n_shared;
  a.slots = c->slots;
  a.shared_base = c->shared_row_base;
  a.n_pad = (int)n_pad;
  cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = c->dtype == MOE_BF16 ? launch_dispatch<__nv_bfloat16, 8>(a, s)
                                             : launch_dispatch<float, 4>(a, s);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
