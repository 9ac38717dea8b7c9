// Rows of activations (or of weights) to 8-bit integers with one scale each,
// and the dispatch that does it on the way.
//
//   s = max_j |x_j| / 127 (fp32)      q_j = x_j / s, to nearest, ties to even
//
// The rounding is decided on the exact quotient, so q is a function of x
// alone and not of how a reciprocal rounds: t = rint(x (1/s)) is at most one
// step off, the remainder x - t s is exact in one fma (t s and x agree to a
// step, so their difference fits 24 bits), and comparing its double with s
// says whether the neighbour is nearer. Few elements come that close to a
// border; the others pay one fma and one compare. Bound by HBM: it reads each
// element once and writes one byte for it.
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

// ---- VEC consecutive elements: 16 bytes read, VEC bytes written ------------
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
};
template <>
struct QChunk<__nv_bfloat16, 1> {
  uint16_t r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    r = *reinterpret_cast<const uint16_t*>(p);
  }
  __device__ __forceinline__ void zero() { r = 0; }
  __device__ __forceinline__ float get(int) const { return bf16_to_f32(r); }
};
template <>
struct QChunk<float, 1> {
  float r;
  __device__ __forceinline__ void load(const float* p) { r = *p; }
  __device__ __forceinline__ void zero() { r = 0.0f; }
  __device__ __forceinline__ float get(int) const { return r; }
};

// The largest magnitude, with every NaN above every number: magnitudes
// compare as their bit patterns.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

struct RowScale {
  float s, inv;
  bool plain;  // inv is a normal number: x * inv is within two roundings of x / s
  bool dead;   // a row of zeros, or one that is not finite: all q are 0
};

__device__ __forceinline__ RowScale row_scale(uint32_t most) {
  RowScale r;
  const float a = __uint_as_float(most);
  r.dead = most == 0 || most >= 0x7f800000u;
  r.s = most >= 0x7f800000u ? __uint_as_float(0x7fffffffu) : __fdiv_rn(a, 127.0f);
  if (!r.dead && r.s == 0.0f) r.dead = true;  // below the smallest fp32 step
  r.plain = r.s >= 0x1p-100f;
  r.inv = r.plain ? 1.0f / r.s : 0.0f;
  return r;
}

// round(x / s) given a candidate t at most one off
__device__ __noinline__ float fix_round(float x, float t, float s) {
  const float r2 = 2.0f * fmaf(-t, s, x);
  const float odd = t - 2.0f * floorf(t * 0.5f);
  if (r2 > s || (r2 == s && odd != 0.0f)) t += 1.0f;
  else if (r2 < -s || (r2 == -s && odd != 0.0f)) t -= 1.0f;
  return t;
}

constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: adding it rounds to an integer

template <typename T, int VEC>
__device__ __forceinline__ void quantize(const QChunk<T, VEC>& c, const RowScale& k, int* q) {
  float t[VEC];
  bool near = false;
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    const float x = c.get(j);
    t[j] = k.plain ? __fadd_rn(__fadd_rn(x * k.inv, kMagic), -kMagic)
                   : rintf(__fdiv_rn(x, k.s));
    near |= fabsf(2.0f * fmaf(-t[j], k.s, x)) >= k.s;
  }
  if (near) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) t[j] = fix_round(c.get(j), t[j], k.s);
  }
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    // (a denormal scale is a few steps coarse: the quotient may pass 127)
    const float v = fminf(fmaxf(t[j], -127.0f), 127.0f);
    q[j] = k.dead ? 0 : (__float_as_int(__fadd_rn(v, kMagic)) & 0xff);
  }
}

template <int VEC>
__device__ __forceinline__ uint64_t pack_bytes(const int* q) {
  uint32_t lo = 0, hi = 0;
#pragma unroll
  for (int j = 0; j < VEC; ++j) {
    if (j < 4) lo |= (uint32_t)q[j] << (8 * j);
    else hi |= (uint32_t)q[j] << (8 * (j - 4));
  }
  return (uint64_t)hi << 32 | lo;
}

template <int VEC>
__device__ __forceinline__ void store_bytes(int8_t* p, uint64_t v) {
  if constexpr (VEC == 8) *reinterpret_cast<uint64_t*>(p) = v;
  else if constexpr (VEC == 4) *reinterpret_cast<uint32_t*>(p) = (uint32_t)v;
  else *p = (int8_t)v;
}

__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(~0u, v); }

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

// Rows of the groups, in order, dealt out to row owners (a warp, or with
// BLOCK the whole block) in a grid-wide stride; each keeps its row in
// registers between the maximum and the rounding. ITEMS == 0: a row longer
// than the registers of a block is read twice.
template <typename T, int VEC, int ITEMS, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 1024 : 32 * kQWarps) quantize_kernel(const QuantArgs a) {
  __shared__ int start[MOE_I8_MAX_GROUPS];
  __shared__ long long prefix[MOE_I8_MAX_GROUPS + 1];  // rows of the groups before g
  __shared__ uint32_t red[2][32];
  pdl_wait();
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
  int flip = 0;
  for (long long i = owner; i < total; i += owners) {
    long long row = i;
    if (a.starts) {
      int lo = 0, hi = a.groups - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= i) lo = mid; else hi = mid - 1;
      }
      row = start[lo] + (i - prefix[lo]);
    }
    const T* x = static_cast<const T*>(a.x) + (size_t)row * a.cols;
    int8_t* q = a.q + (size_t)row * a.cols;
    QChunk<T, VEC> c[ITEMS > 0 ? ITEMS : 1];
    uint32_t most = 0;
    if constexpr (ITEMS > 0) {
#pragma unroll
      for (int k = 0; k < ITEMS; ++k) {
        const int p = k * threads + tid;
        c[k].zero();
        if (p < chunks) c[k].load(x + (size_t)p * VEC);
      }
#pragma unroll
      for (int k = 0; k < ITEMS; ++k)
#pragma unroll
        for (int j = 0; j < VEC; ++j) most = max(most, magnitude(c[k].get(j)));
    } else {
      for (int p = tid; p < chunks; p += threads) {
        c[0].load(x + (size_t)p * VEC);
#pragma unroll
        for (int j = 0; j < VEC; ++j) most = max(most, magnitude(c[0].get(j)));
      }
    }
    most = warp_max(most);
    if (BLOCK) {
      if (lane == 0) red[flip][threadIdx.x >> 5] = most;
      __syncthreads();
      most = warp_max(lane < (int)(blockDim.x >> 5) ? red[flip][lane] : 0u);
      flip ^= 1;
    }
    const RowScale k = row_scale(most);
    if (tid == 0) a.scale[row] = k.s;
    int v[VEC];
    if constexpr (ITEMS > 0) {
#pragma unroll
      for (int m = 0; m < ITEMS; ++m) {
        const int p = m * threads + tid;
        if (p < chunks) {
          quantize<T, VEC>(c[m], k, v);
          store_bytes<VEC>(q + (size_t)p * VEC, pack_bytes<VEC>(v));
        }
      }
    } else {
      for (int p = tid; p < chunks; p += threads) {
        c[0].load(x + (size_t)p * VEC);
        quantize<T, VEC>(c[0], k, v);
        store_bytes<VEC>(q + (size_t)p * VEC, pack_bytes<VEC>(v));
      }
    }
  }
}

template <typename T, int VEC, int ITEMS, bool BLOCK>
cudaError_t run_quant(const QuantArgs& a, int threads, cudaStream_t s) {
  // resident blocks: up to 2,048 threads an SM, the rows dealt out in a stride
  const long long per_block = BLOCK ? 1 : kQWarps;
  const int resident = BLOCK ? (2048 / threads < 8 ? 2048 / threads : 8) : 8;
  long long grid = (a.rows + per_block - 1) / per_block;
  if (grid > (long long)kBlockSms * resident) grid = (long long)kBlockSms * resident;
  return launch_pdl(quantize_kernel<T, VEC, ITEMS, BLOCK>, dim3((unsigned)grid), dim3(threads), 0,
                    s, a);
}

// A warp a row while a lane holds at most 32 bf16 (16 fp32) elements, then a
// block a row with up to 4 vectors a thread.
template <typename T, int VEC>
cudaError_t launch_quant(const QuantArgs& a, cudaStream_t s) {
  const int chunks = a.cols / VEC;
  constexpr int I4 = 4;
  if (chunks <= 32 * I4) return run_quant<T, VEC, I4, false>(a, 32 * kQWarps, s);
  if (chunks <= 1024 * I4) {
    const int threads = ((chunks + I4 - 1) / I4 + 31) / 32 * 32;
    return run_quant<T, VEC, I4, true>(a, threads, s);
  }
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
  uint32_t most = 0;
  if constexpr (ITEMS > 0) {
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      const int p = k * threads + tid;
      c[k].zero();
      if (p < chunks) c[k].load(x + (size_t)p * VEC);
    }
#pragma unroll
    for (int k = 0; k < ITEMS; ++k)
#pragma unroll
      for (int j = 0; j < VEC; ++j) most = max(most, magnitude(c[k].get(j)));
  } else {
    for (int p = tid; p < chunks; p += threads) {
      c[0].load(x + (size_t)p * VEC);
#pragma unroll
      for (int j = 0; j < VEC; ++j) most = max(most, magnitude(c[0].get(j)));
    }
  }
  most = warp_max(most);
  if (lane == 0) red[tid >> 5] = most;
  __syncthreads();
  most = warp_max(lane < threads / 32 ? red[lane] : 0u);
  const RowScale k = row_scale(most);
  for (int j = tid; j < targets; j += threads)
    if (dst[j] >= 0) a.scale[dst[j]] = k.s;
  int v[VEC];
  auto put = [&](int p, uint64_t bytes) {
    for (int j = 0; j < targets; ++j)
      if (dst[j] >= 0) store_bytes<VEC>(a.q + (size_t)dst[j] * a.d + (size_t)p * VEC, bytes);
  };
  if constexpr (ITEMS > 0) {
#pragma unroll
    for (int m = 0; m < ITEMS; ++m) {
      const int p = m * threads + tid;
      if (p < chunks) {
        quantize<T, VEC>(c[m], k, v);
        put(p, pack_bytes<VEC>(v));
      }
    }
  } else {
    for (int p = tid; p < chunks; p += threads) {
      c[0].load(x + (size_t)p * VEC);
      quantize<T, VEC>(c[0], k, v);
      put(p, pack_bytes<VEC>(v));
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
