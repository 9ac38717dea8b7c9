// Global norm of many gradient tensors, and their clipping.
//
//   norm = (sum_i sum_j g_ij^2)^1/2      c = min(1, max_norm / (norm + 1e-6))
//   out_i = c g_i
//
// Two passes over the data, since c needs every element: two reads and a write,
// where the floor is one of each. Each tensor is cut into equal tiles of up to
// 8,192 elements; the norm pass deals them out to its blocks in turn, and the
// scaling pass takes them from the last one backwards, beginning with what the
// norm pass read last (small lists still lie in L2 whole). Both passes are bound
// by HBM. On a B200, 806 MB of bf16 gradients: 118 us for the norm (the copy
// rate), 361 us with the clip, where two reads and a write take 369 us at the copy
// rate; a scaling pass of resident blocks that walk many tiles took 40 us more
// (its accesses lie further apart).
//
// Squares: eight neighbours are summed in fp32 when the largest of them lies
// in [2^-50, 2^50] (or all are 0), where neither the squares nor their sum
// can leave the fp32 range and what underflows is below 2^-40 of the sum;
// otherwise they are squared in fp64. Everything above eight elements is
// fp64. Partial sums are per block, in tile order, and each scaling block
// adds all of them in the same fixed order: no atomics, the same norm in
// every block and every run.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "block_internal.h"
#include "device_common.cuh"

namespace moe {
namespace {

constexpr int kTile = 8192;       // most elements of a tile
constexpr int kClipThreads = 256;
constexpr int kClipBlocks = kBlockSms * 6;  // most blocks of a launch (6 resident on an SM)
constexpr int kUnroll = 4;        // vectors in flight a thread

struct GradTensor {
  const void* g;
  void* o;
  long long n;
  int tile0;    // tiles of the tensors before it (of this launch)
  int tile_bf;  // elements of a tile (a multiple of 64), 1 in the low bit for bf16
};
__host__ __device__ inline int tile_count(long long n) { return (int)((n + kTile - 1) / kTile); }

// The tensors of one launch travel in its parameters: 4 KB of them hold what
// one layer has, the largest parameter block (32,764 bytes) what an unstacked
// expert list has (5 tensors in it: 14.3 us a clip, one after another, against
// 11.4; a long list in blocks of 120 would be two launches for each).
template <int CAP>
struct GradBatch {
  GradTensor t[CAP];
  int count, tiles;
};
constexpr int kSmallBatch = 120, kLargeBatch = 1000;
static_assert(sizeof(GradBatch<kSmallBatch>) <= 4000, "one 4 KB parameter block");
static_assert(sizeof(GradBatch<kLargeBatch>) <= 32700, "the largest parameter block");

template <int CAP>
__device__ __forceinline__ int find_tensor(const GradBatch<CAP>& b, int tile) {
  if (CAP == kLargeBatch) {
    // long lists are mostly of like tensors, found at once (768 of 25 k elements:
    // 21.5 against 25.5 us a clip)
    const int i = (int)((float)tile * b.count / b.tiles);
    if (i < b.count && b.t[i].tile0 <= tile && (i + 1 == b.count || b.t[i + 1].tile0 > tile))
      return i;
  }
  int lo = 0, hi = b.count - 1;  // the last tensor with tile0 <= tile (empty ones have no tile)
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (b.t[mid].tile0 <= tile) lo = mid; else hi = mid - 1;
  }
  return lo;
}

template <typename T>
struct Vec16;  // a 16-byte vector of T
template <>
struct Vec16<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4& r, float* v) {
    v[0] = __uint_as_float(r.x);
    v[1] = __uint_as_float(r.y);
    v[2] = __uint_as_float(r.z);
    v[3] = __uint_as_float(r.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* v) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                      __float_as_uint(v[3]));
  }
};
template <>
struct Vec16<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4& r, float* v) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* v) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
  }
};

template <int N>
__device__ __forceinline__ double square_sum(const float* v) {
  float s = 0.0f, m = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    s = fmaf(v[i], v[i], s);
    m = fmaxf(m, fabsf(v[i]));  // (a NaN reaches s)
  }
  if (m == 0.0f || (m >= 0x1p-50f && m <= 0x1p50f)) return (double)s;
  double t = 0.0;
#pragma unroll
  for (int i = 0; i < N; ++i) t = fma((double)v[i], (double)v[i], t);
  return t;
}

// Elements [0, n) from p on: the vectors between the first and the last
// 16-byte boundary, and what lies before and behind them one by one.
template <typename T>
__device__ __forceinline__ void split16(const T* p, int n, int& head, int& vecs) {
  constexpr int N = Vec16<T>::N;
  const int mis = (int)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
  head = min((N - mis) % N, n);
  vecs = (n - head) / N;
}

template <typename T>
__device__ __forceinline__ double tile_squares(const T* p, int n) {
  constexpr int N = Vec16<T>::N;
  int head, vecs;
  split16(p, n, head, vecs);
  double acc = 0.0;
  const uint4* q = reinterpret_cast<const uint4*>(p + head);
  for (int i = threadIdx.x; i < vecs; i += kClipThreads * kUnroll) {
    uint4 r[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k)
      r[k] = i + k * kClipThreads < vecs ? q[i + k * kClipThreads] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      float v[N];
      Vec16<T>::unpack(r[k], v);
      acc += square_sum<N>(v);
    }
  }
  const int tail = head + vecs * N;
  const int loose = head + n - tail;  // < 2 N
  if ((int)threadIdx.x < loose) {
    const int i = (int)threadIdx.x;
    const float v = (float)p[i < head ? i : tail + i - head];
    acc += square_sum<1>(&v);
  }
  return acc;
}

__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = red[0];
#pragma unroll
  for (int i = 1; i < kClipThreads / 32; ++i) s += red[i];
  return s;
}

// partial[blockIdx.x] = the sum of squares of the block's tiles
template <int CAP>
__global__ void __launch_bounds__(kClipThreads, 6)
    grad_squares_kernel(const __grid_constant__ GradBatch<CAP> b, double* partial) {
  __shared__ double red[kClipThreads / 32];
  pdl_wait();
  double acc = 0.0;
  for (int tile = blockIdx.x; tile < b.tiles; tile += gridDim.x) {
    const GradTensor& t = b.t[find_tensor(b, tile)];
    const int size = t.tile_bf & ~1;
    const long long at = (long long)(tile - t.tile0) * size;
    const int n = (int)min((long long)size, t.n - at);
    acc += (t.tile_bf & 1) ? tile_squares(static_cast<const __nv_bfloat16*>(t.g) + at, n)
                  : tile_squares(static_cast<const float*>(t.g) + at, n);
  }
  acc = block_sum(acc, red);
  if (threadIdx.x == 0) partial[blockIdx.x] = acc;
}

// every block adds the partial sums in the same order
__device__ __forceinline__ double total_norm(const double* partial, int count, double* red) {
  double s = 0.0;
  for (int i = threadIdx.x; i < count; i += kClipThreads) s += partial[i];
  return sqrt(block_sum(s, red));
}

__global__ void __launch_bounds__(kClipThreads)
    grad_norm_kernel(const double* partial, int count, float* norm) {
  __shared__ double red[kClipThreads / 32];
  pdl_wait();
  const double r = total_norm(partial, count, red);
  if (threadIdx.x == 0) norm[0] = (float)r;
}

template <typename T>
__device__ __forceinline__ void tile_scale(const T* p, T* o, int n, float c) {
  constexpr int N = Vec16<T>::N;
  int head, vecs;
  split16(p, n, head, vecs);
  // a copy that is not aligned alike is written element by element
  if ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(o)) & 15) {
    for (int i = threadIdx.x; i < n; i += kClipThreads) o[i] = (T)((float)p[i] * c);
    return;
  }
  const uint4* q = reinterpret_cast<const uint4*>(p + head);
  uint4* w = reinterpret_cast<uint4*>(o + head);
  for (int i = threadIdx.x; i < vecs; i += kClipThreads * kUnroll) {
    uint4 r[kUnroll];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k)
      if (i + k * kClipThreads < vecs) r[k] = q[i + k * kClipThreads];
#pragma unroll
    for (int k = 0; k < kUnroll; ++k) {
      if (i + k * kClipThreads < vecs) {
        float v[N];
        Vec16<T>::unpack(r[k], v);
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] *= c;
        w[i + k * kClipThreads] = Vec16<T>::pack(v);
      }
    }
  }
  const int tail = head + vecs * N;
  const int loose = head + n - tail;
  if ((int)threadIdx.x < loose) {
    const int j = (int)threadIdx.x < head ? threadIdx.x : tail + threadIdx.x - head;
    o[j] = (T)((float)p[j] * c);
  }
}

template <int CAP>
__global__ void __launch_bounds__(kClipThreads, 6)
    grad_scale_kernel(const __grid_constant__ GradBatch<CAP> b, const double* partial, int count,
                      float max_norm, float* norm, int write_norm) {
  __shared__ double red[kClipThreads / 32];
  pdl_wait();
  // the factor is of the norm as it is returned, +inf above the largest fp32
  const float r = (float)total_norm(partial, count, red);
  const double k = (double)max_norm / ((double)r + 1e-6);
  const float c = isnan(r) ? r : (float)(k < 1.0 ? k : 1.0);  // (no limit: 1, of inf too)
  if (write_norm && blockIdx.x == 0 && threadIdx.x == 0) {
    norm[0] = r;
    norm[1] = c;
  }
  for (int tile = b.tiles - 1 - (int)blockIdx.x; tile >= 0; tile -= gridDim.x) {
    const GradTensor& t = b.t[find_tensor(b, tile)];
    if (c == 1.0f && t.g == t.o) continue;
    const int size = t.tile_bf & ~1;
    const long long at = (long long)(tile - t.tile0) * size;
    const int n = (int)min((long long)size, t.n - at);
    if (t.tile_bf & 1)
      tile_scale(static_cast<const __nv_bfloat16*>(t.g) + at, static_cast<__nv_bfloat16*>(t.o) + at,
                 n, c);
    else
      tile_scale(static_cast<const float*>(t.g) + at, static_cast<float*>(t.o) + at, n, c);
  }
}

int batches(int count) { return count <= kSmallBatch ? 1 : (count + kLargeBatch - 1) / kLargeBatch; }

size_t clip_bytes(int count) { return (size_t)batches(count) * kClipBlocks * sizeof(double); }

moe_status check_tensors(const moe_grad_tensor* t, int count, bool outs) {
  if (count < 0 || (count > 0 && !t)) return MOE_ERR_INVALID_ARG;
  long long tiles = 0;
  for (int i = 0; i < count; ++i) {
    if (t[i].numel < 0 || (t[i].dtype != MOE_F32 && t[i].dtype != MOE_BF16))
      return MOE_ERR_INVALID_ARG;
    if (t[i].numel == 0) continue;
    const uintptr_t mask = t[i].dtype == MOE_BF16 ? 1 : 3;
    if (!t[i].grad || (reinterpret_cast<uintptr_t>(t[i].grad) & mask)) return MOE_ERR_INVALID_ARG;
    if (outs && (!t[i].out || (reinterpret_cast<uintptr_t>(t[i].out) & mask)))
      return MOE_ERR_INVALID_ARG;
    if (t[i].numel > (1LL << 42)) return MOE_ERR_UNSUPPORTED;
    tiles += tile_count(t[i].numel);
    if (tiles > 0x7fffffff) return MOE_ERR_UNSUPPORTED;
  }
  return MOE_OK;
}

// the tensors with elements of [first, first + CAP)
template <int CAP>
void fill(GradBatch<CAP>& b, const moe_grad_tensor* t, int first, int count) {
  b.count = 0;
  b.tiles = 0;
  for (int i = first; i < count && i < first + CAP; ++i) {
    if (t[i].numel == 0) continue;
    GradTensor& g = b.t[b.count++];
    g.g = t[i].grad;
    g.o = t[i].out;
    g.n = t[i].numel;
    g.tile0 = b.tiles;
    const long long tiles = tile_count(g.n);
    g.tile_bf = (int)(((g.n + tiles - 1) / tiles + 63) / 64 * 64) | (t[i].dtype == MOE_BF16);
    b.tiles += (int)tiles;
  }
}

int clip_grid(int tiles) { return tiles < kClipBlocks ? tiles : kClipBlocks; }
// The scaling pass: a tile a block where there are many (see above); up to a few
// rounds, which L2 mostly holds, resident blocks save their start (38 MB: 15.7
// against 17.0 us).
int scale_grid(int tiles) { return tiles > 4 * kClipBlocks ? tiles : clip_grid(tiles); }

template <int CAP>
moe_status run_clip(const moe_grad_tensor* t, int count, bool scale, float max_norm, float* norm,
                    double* partial, cudaStream_t s) {
  GradBatch<CAP> b;  // (32 KB at most, on the host's stack)
  int used = 0;
  for (int first = 0; first < count; first += CAP) {
    fill(b, t, first, count);
    if (b.tiles == 0) continue;
    const int grid = clip_grid(b.tiles);
    if (launch_pdl(grad_squares_kernel<CAP>, dim3(grid), dim3(kClipThreads), 0, s, b,
                   partial + used) != cudaSuccess)
      return MOE_ERR_CUDA;
    used += grid;
  }
  if (!scale) {
    return launch_pdl(grad_norm_kernel, dim3(1), dim3(kClipThreads), 0, s,
                      (const double*)partial, used, norm) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
  }
  // the last tensors first: L2 holds them
  int write = 1;
  for (int first = count > 0 ? (count - 1) / CAP * CAP : 0; first >= 0; first -= CAP) {
    fill(b, t, first, count);
    if (b.tiles == 0 && !(write && first == 0)) continue;
    const int grid = b.tiles ? scale_grid(b.tiles) : 1;
    if (launch_pdl(grad_scale_kernel<CAP>, dim3(grid), dim3(kClipThreads), 0, s, b,
                   (const double*)partial, used, max_norm, norm, write) != cudaSuccess)
      return MOE_ERR_CUDA;
    write = 0;
  }
  return MOE_OK;
}

moe_status clip_impl(const moe_grad_tensor* t, int count, bool scale, float max_norm, float* norm,
                     void* ws, size_t ws_bytes, cudaStream_t s) {
  moe_status st = check_tensors(t, count, scale);
  if (st != MOE_OK) return st;
  if (!norm || (reinterpret_cast<uintptr_t>(norm) & 3)) return MOE_ERR_INVALID_ARG;
  if ((st = check_block_ws(ws, ws_bytes, clip_bytes(count))) != MOE_OK) return st;
  double* partial = static_cast<double*>(ws);
  return count <= kSmallBatch
             ? run_clip<kSmallBatch>(t, count, scale, max_norm, norm, partial, s)
             : run_clip<kLargeBatch>(t, count, scale, max_norm, norm, partial, s);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_grad_workspace_size(int count, size_t* bytes) {
  if (count < 0) return MOE_ERR_INVALID_ARG;
  if (bytes) *bytes = clip_bytes(count);
  return MOE_OK;
}

moe_status moe_grad_norm(const moe_grad_tensor* tensors, int count, float* norm, void* ws,
                         size_t ws_bytes, moe_stream_t stream) {
  return clip_impl(tensors, count, false, 0.0f, norm, ws, ws_bytes, (cudaStream_t)stream);
}

moe_status moe_grad_clip(const moe_grad_tensor* tensors, int count, float max_norm, float* norm,
                         void* ws, size_t ws_bytes, moe_stream_t stream) {
  if (!(max_norm >= 0.0f)) return MOE_ERR_INVALID_ARG;
  return clip_impl(tensors, count, true, max_norm, norm, ws, ws_bytes, (cudaStream_t)stream);
}

}  // extern "C"
