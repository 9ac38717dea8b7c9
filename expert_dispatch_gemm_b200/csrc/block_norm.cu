// Residual norms around a block, forward and backward.
//
// "Expert choice routing" (aicassindra.com), "The math": the layer's output is
// a scatter_add into zeros, and what the layer did not touch rides on the
// residual, which the caller adds. Here it is added, between the two norms:
//
//   r1 = (mean y^2 + eps)^-1/2      v   = y r1 (w1 + off)
//   out = a x + b g v
//   r2 = (mean out^2 + eps)^-1/2    h   = out r2 (w2 + off)
//
// Backward, with u = out r2 and yr = y r1 (both of unit mean square, so that
// d(norm)/dv = r (I - u u^T / d)), q = dh (w2 + off) and c = b g (w1 + off) yr:
//   D  = dout + r2 (q - u mean(q u))      dx = a D
//   dg = sum b D v                        dw1 = sum b g D yr,  dw2 = sum dh u
//   dy = r1 (b g D (w1 + off) - yr m),    m = mean(D c)
// m needs D, which needs mean(q u); expanding D gives m from sums that one
// pass over the row collects together,
//   m = (sum (dout + r2 q) c - r2 mean(q u) sum u c) / d,
// so a row takes one block reduction (of three sums), not two in sequence. All of
// it is computed from u and yr, never from y with powers of r1: yr is about 1
// whatever y and eps are, where r1^3 leaves fp32's range for |y| above 4e12, and
// for rows of zeros with eps below 2e-26.
//
// The forward moves 4 n d elements (x, y, out, h), the backward 6 n d: both are
// to be bound by HBM, which leaves about 20 instructions an element. So
// - a block (worker) owns a contiguous range of rows, and a thread the same 8
//   columns (16 above d = 8192) of each: weights, the gate's product with them
//   and the sums over tokens stay in its registers (of 16 columns, in the backward,
//   as far as 64 hold them: 500 to 700 bytes a thread are spilled and read again);
// - arithmetic is on packed fp32 pairs;
// - the next rows' chunks come into shared memory by cp.async while a row is
//   computed; each thread reads back only what it copied itself, so no barrier
//   guards the ring, and the only barriers are those of the row sums.
// On a B200, replayed from a graph: forward, n 8192, d 7168 bf16, 81 to 83 us
// (5.7 TB/s, 87 to 89% of a copy's rate; without the ring and the packed pairs
// 112); backward, n 16384, d 2048 bf16, one gate row, 70 to 73 us (5.6 TB/s, 84 to
// 88%), n 8192, d 7168 153 to 157 us (69 to 70%: one worker an SM, whose warps wait
// for each other at every row), n 2048, d 16384 165 us (37%: spills); the pre-norm's
// own, n 8192, d 7168, 222 us (32%: the general instance below, which spills too).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <initializer_list>

#include "block_internal.h"
#include "device_common.cuh"

namespace moe {
namespace {

__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

__device__ __forceinline__ uint32_t smem32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// BYTES (4, 8, 16), or (n = 0) zeros, from global into shared memory
template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, uint32_t n) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
                 : "memory");
  else if constexpr (BYTES >= 4)
    asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(n),
                 "n"(BYTES < 4 ? 4 : BYTES)
                 : "memory");
}
__device__ __forceinline__ uint32_t load_smem4(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ uint4 load_smem16(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "r"(a)
               : "memory");
  return r;
}

// A thread's EPT elements of a row, as pairs: EPT / VEC chunks of VEC
// neighbours, chunk c of the row at thread c % threads, so that an access of
// the warp is one run of 16-byte vectors, or, for rows that do not start on
// 16-byte boundaries, of 4-byte ones (two bf16 or one fp32), or of single bf16.
// Columns past d are zeros.
template <typename T, int VEC, int EPT>
struct Cols {
  static constexpr int ITEMS = EPT / VEC, BYTES = VEC * (int)sizeof(T);
  int tid, threads, chunks;

  __device__ __forceinline__ bool has(int i) const { return i * threads + tid < chunks; }
  __device__ __forceinline__ int at(int i) const { return (i * threads + tid) * VEC; }

  static __device__ __forceinline__ void unpack(float2* o, const uint4& r) {
    if constexpr (sizeof(T) == 4) {
      o[0] = make_float2(__uint_as_float(r.x), __uint_as_float(r.y));
      o[1] = make_float2(__uint_as_float(r.z), __uint_as_float(r.w));
    } else {
      const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o[j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
    }
  }
  // from a staged row whose first byte is at shared address `a` (columns past
  // d were zeroed there)
  __device__ __forceinline__ void load_smem(float2* v, uint32_t a) const {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const uint32_t at = a + (uint32_t)(i * threads + tid) * BYTES;
      if constexpr (BYTES == 16) unpack(v + i * (VEC / 2), load_smem16(at));
      else if constexpr (BYTES == 4) put(v, i, load_smem4(at));
    }
  }
  __device__ __forceinline__ void load(float2* v, const T* row) const {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      if constexpr (BYTES == 16) {
        unpack(v + i * (VEC / 2), has(i) ? __ldcs(reinterpret_cast<const uint4*>(row + at(i)))
                                         : make_uint4(0, 0, 0, 0));
      } else if constexpr (BYTES == 4) {
        put(v, i, has(i) ? *reinterpret_cast<const uint32_t*>(row + at(i)) : 0u);
      } else {
        const float x = has(i) ? (float)row[at(i)] : 0.0f;
        if (i & 1) v[i / 2].y = x; else v[i / 2].x = x;
      }
    }
  }
  __device__ __forceinline__ void store(T* row, const float2* v) const {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      if (!has(i)) continue;
      if constexpr (BYTES == 16) {
        const float2* o = v + i * (VEC / 2);
        if constexpr (sizeof(T) == 4)
          *reinterpret_cast<float4*>(row + at(i)) = make_float4(o[0].x, o[0].y, o[1].x, o[1].y);
        else
          *reinterpret_cast<uint4*>(row + at(i)) =
              make_uint4(pack_bf16x2(o[0].x, o[0].y), pack_bf16x2(o[1].x, o[1].y),
                         pack_bf16x2(o[2].x, o[2].y), pack_bf16x2(o[3].x, o[3].y));
      } else if constexpr (VEC == 2) {
        *reinterpret_cast<uint32_t*>(row + at(i)) = pack_bf16x2(v[i].x, v[i].y);
      } else {
        row[at(i)] = (T)((i & 1) ? v[i / 2].y : v[i / 2].x);
      }
    }
  }
  // chunk i of 4 bytes: a pair of bf16, or half a pair of fp32
  static __device__ __forceinline__ void put(float2* v, int i, uint32_t w) {
    if constexpr (VEC == 2) {
      v[i] = make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    } else {
      if (i & 1) v[i / 2].y = __uint_as_float(w); else v[i / 2].x = __uint_as_float(w);
    }
  }
  // fp32 rows of the same columns (weights, sums), element by element aligned
  // as the vectors need it
  __device__ __forceinline__ void load_f32(float2* v, const float* row) const {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      if constexpr (VEC == 1) {
        const float x = has(i) ? row[at(i)] : 0.0f;
        if (i & 1) v[i / 2].y = x; else v[i / 2].x = x;
      } else if constexpr (VEC == 2) {
        v[i] = has(i) ? make_float2(row[at(i)], row[at(i) + 1]) : make_float2(0, 0);
      } else {
#pragma unroll
        for (int j = 0; j < VEC; j += 4) {
          float4 w = make_float4(0, 0, 0, 0);
          if (has(i)) w = *reinterpret_cast<const float4*>(row + at(i) + j);
          v[(i * VEC + j) / 2] = make_float2(w.x, w.y);
          v[(i * VEC + j) / 2 + 1] = make_float2(w.z, w.w);
        }
      }
    }
  }
  __device__ __forceinline__ void store_f32(float* row, const float2* v) const {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      if (!has(i)) continue;
      if constexpr (VEC == 1) {
        row[at(i)] = (i & 1) ? v[i / 2].y : v[i / 2].x;
      } else if constexpr (VEC == 2) {
        row[at(i)] = v[i].x;
        row[at(i) + 1] = v[i].y;
      } else {
#pragma unroll
        for (int j = 0; j < VEC; j += 4) {
          const float2 a = v[(i * VEC + j) / 2], b = v[(i * VEC + j) / 2 + 1];
          *reinterpret_cast<float4*>(row + at(i) + j) = make_float4(a.x, a.y, b.x, b.y);
        }
      }
    }
  }
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// the oldest row of a ring of `stages` has arrived
__device__ __forceinline__ void cp_async_wait_row(int stages) {
  if (stages >= 4) cp_async_wait<3>();
  else if (stages == 3) cp_async_wait<2>();
  else if (stages == 2) cp_async_wait<1>();
  else cp_async_wait<0>();
}
constexpr int kMaxStages = 4;

// Shared addresses of a ring's next stage to fill and to read.
struct Ring {
  uint32_t first, bytes, end, fill, read;
  __device__ __forceinline__ Ring(const void* smem, uint32_t stage_bytes, int stages)
      : first(smem32(smem)), bytes(stage_bytes), end(first + stage_bytes * stages), fill(first),
        read(first) {}
  __device__ __forceinline__ void filled() { fill = fill + bytes == end ? first : fill + bytes; }
  __device__ __forceinline__ void done() { read = read + bytes == end ? first : read + bytes; }
};

__host__ __device__ __forceinline__ int worker_row(int w, int n, int workers) {
  return (int)((long long)w * n / workers);
}
// the worker that holds row r
__host__ __device__ __forceinline__ int row_worker(int r, int n, int workers) {
  return (int)((((long long)r + 1) * workers - 1) / n);
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
// Gate rows of few tokens travel through the forward's ring with the others (one
// copy for each row, from L2 after the first; 53.7 against 56.7 us at n 16384, d
// 2048, 3 tokens a gate row); rows of more tokens are loaded when they begin.
constexpr int kStagedGateTokens = 8;
__host__ __device__ __forceinline__ bool gate_staged(const void* gate, int tokens) {
  return gate && tokens > 0 && tokens <= kStagedGateTokens;
}

struct NormFwd {
  const void *x, *y, *gate;
  const float *w_post, *w_next;
  void *out, *h;
  float *rstd_post, *rstd_next;
  int n, d, gate_tokens, workers, stages, slots;
  float eps, off, a, b;
  long long gate_stride;
};

// The sum of v over the block: within the warps, then over their sums in
// `red`, which nothing else may use until the block's next barrier but one.
__device__ __forceinline__ float block_sum(float v, float* red, int warps) {
  v = warp_sum(v);
  if (warps == 1) return v;
  const int lane = threadIdx.x & 31;
  if (lane == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum(lane < warps ? red[lane] : 0.0f);
}

// rows until the gate row of row r ends (a gate without groups never does)
__device__ __forceinline__ int gate_rows_left(const void* gate, int tokens, int r) {
  return gate && tokens ? tokens - r % tokens : 0x7fffffff;
}

template <typename T, int VEC, int EPT, bool STAGED>
__global__ void __launch_bounds__(1024) norm_fwd_kernel(const NormFwd p) {
  extern __shared__ __align__(16) unsigned char nsm[];
  __shared__ float red[2][2][32];
  pdl_wait();
  constexpr int P = EPT / 2;
  const Cols<T, VEC, EPT> cols{(int)threadIdx.x, (int)blockDim.x, p.d / VEC};
  const int warps = blockDim.x >> 5;
  const int r0 = worker_row(blockIdx.x, p.n, p.workers);
  const int r1 = worker_row(blockIdx.x + 1, p.n, p.workers);
  const bool has_y = p.y, post = p.w_post, next = p.h;
  // this worker's rows; the filling pointers run ahead of `at` (elements)
  const size_t base = (size_t)r0 * p.d;
  const T* x = static_cast<const T*>(p.x) + base;
  const T* y = static_cast<const T*>(p.y) + base;
  T* out = static_cast<T*>(p.out) + base;
  T* h = static_cast<T*>(p.h) + base;
  const T* gate = static_cast<const T*>(p.gate);
  if (gate && p.gate_tokens) gate += (long long)(r0 / p.gate_tokens) * p.gate_stride;
  const bool gate_each = gate_staged(gate, p.gate_tokens);
  const uint32_t pitch = (uint32_t)blockDim.x * EPT * sizeof(T);  // of a staged row
  Ring ring(nsm, p.slots * pitch, p.stages);
  const float inv_d = 1.0f / (float)p.d;
  size_t fill_at = 0;
  const T* fill_gate = gate;
  int to_fill = r1 - r0;
  int fill_left = gate_each ? p.gate_tokens - r0 % p.gate_tokens : 0;
  auto issue = [&]() {
    if constexpr (STAGED) {
      if (to_fill > 0) {
        --to_fill;
#pragma unroll
        for (int i = 0; i < cols.ITEMS; ++i) {
          constexpr int B = Cols<T, VEC, EPT>::BYTES;
          const uint32_t n = cols.has(i) ? B : 0;
          const int c = n ? cols.at(i) : 0;
          const uint32_t dst = ring.fill + (uint32_t)(i * cols.threads + cols.tid) * B;
          cp_async<B>(dst, x + fill_at + c, n);
          if (has_y) cp_async<B>(dst + pitch, y + fill_at + c, n);
          if (gate_each) cp_async<B>(dst + 2 * pitch, fill_gate + c, n);
        }
        fill_at += p.d;
        if (gate_each && --fill_left == 0) {
          fill_gate += p.gate_stride;
          fill_left = p.gate_tokens;
        }
        ring.filled();
      }
      cp_async_commit();
    }
  };
  for (int q = 0; q < p.stages - 1; ++q) issue();
  float2 cw[P], wn[P];  // b gate (w_post + off); w_next + off
  if (next) {
    cols.load_f32(wn, p.w_next);
#pragma unroll
    for (int e = 0; e < P; ++e) wn[e] = add2(wn[e], both(p.off));
  }
  int left = 0;  // rows for which cw holds
  size_t at = 0;
  for (int r = r0; r < r1; ++r, at += p.d) {
    issue();
    if (STAGED) cp_async_wait_row(p.stages);
    float2 o[P];
    if (has_y) {
      if (left == 0) {
        if (post) {
          cols.load_f32(cw, p.w_post);
#pragma unroll
          for (int e = 0; e < P; ++e) cw[e] = mul2(add2(cw[e], both(p.off)), both(p.b));
        } else {
#pragma unroll
          for (int e = 0; e < P; ++e) cw[e] = both(p.b);
        }
        if (gate) {
          float2 g[P];
          if (STAGED && gate_each) cols.load_smem(g, ring.read + 2 * pitch);
          else cols.load(g, gate);
          gate += p.gate_stride;
#pragma unroll
          for (int e = 0; e < P; ++e) cw[e] = mul2(cw[e], g[e]);
        }
        left = gate_rows_left(p.gate, p.gate_tokens, r);
      }
      --left;
      float2 v[P];
      if (STAGED) cols.load_smem(v, ring.read + pitch);
      else cols.load(v, y + at), cols.load(o, x + at);
      float rp = 1.0f;
      if (post) {
        float2 s = both(0.0f);
#pragma unroll
        for (int e = 0; e < P; ++e) s = fma2(v[e], v[e], s);
        const float ss = block_sum(s.x + s.y, red[r & 1][0], warps);
        rp = rsqrtf(ss * inv_d + p.eps);
        if (p.rstd_post && threadIdx.x == 0) p.rstd_post[r] = rp;
      }
      if (STAGED) cols.load_smem(o, ring.read);
#pragma unroll
      for (int e = 0; e < P; ++e)
        o[e] = fma2(mul2(v[e], cw[e]), both(rp), mul2(o[e], both(p.a)));
      cols.store(out + at, o);
    } else if (STAGED) {
      cols.load_smem(o, ring.read);
    } else {
      cols.load(o, x + at);
    }
    if (next) {
      float2 s = both(0.0f);
#pragma unroll
      for (int e = 0; e < P; ++e) s = fma2(o[e], o[e], s);
      const float ss = block_sum(s.x + s.y, red[r & 1][1], warps);
      const float rn = rsqrtf(ss * inv_d + p.eps);
      if (p.rstd_next && threadIdx.x == 0) p.rstd_next[r] = rn;
#pragma unroll
      for (int e = 0; e < P; ++e) o[e] = mul2(mul2(o[e], both(rn)), wn[e]);
      cols.store(h + at, o);
    }
    ring.done();
  }
}

// ---- work split --------------------------------------------------------------
// Threads a worker: 8 columns each up to d = 8192, 16 above.
int norm_threads(int d) { return ((d <= 8192 ? (d + 7) / 8 : (d + 15) / 16) + 31) / 32 * 32; }
// shared memory for one worker's ring where `per_sm` of them share an SM
size_t ring_budget(int per_sm) { return (size_t)(224 * 1024) / per_sm - 2048; }

int fwd_workers_per_sm(int d) {
  const int k = 1024 / norm_threads(d);
  return k < 1 ? 1 : k > 16 ? 16 : k;
}

template <typename T, int VEC, int EPT, bool STAGED>
cudaError_t run_fwd(const NormFwd& p, size_t smem, cudaStream_t s) {
  auto kern = norm_fwd_kernel<T, VEC, EPT, STAGED>;
  if (smem > 32 * 1024) {  // (48 KB with the static part need no leave)
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_all_smem(kern, done);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kern, dim3(p.workers), dim3(norm_threads(p.d)), smem, s, p);
}

// bytes: what every row of every operand starts on a boundary of (16, 4, or
// less), the chunk that a thread takes
template <typename T>
cudaError_t launch_fwd(NormFwd& p, int bytes, cudaStream_t s) {
  constexpr int V16 = 16 / sizeof(T), V4 = 2;
  const int per_sm = fwd_workers_per_sm(p.d);
  const long long most = (long long)kBlockSms * per_sm;
  p.workers = (int)(p.n < most ? p.n : most);
  p.slots = gate_staged(p.gate, p.gate_tokens) ? 3 : p.y ? 2 : 1;
  const size_t row = (size_t)norm_threads(p.d) * (p.d > 8192 ? 16 : 8) * sizeof(T);
  const size_t fit = ring_budget(per_sm) / (p.slots * row);
  const int deep = (p.n + p.workers - 1) / p.workers;  // no more stages than rows
  p.stages = fit > kMaxStages ? kMaxStages : (int)fit;
  if (p.stages > deep) p.stages = deep;
  // (fp32 rows off 16-byte boundaries: single loads, not staged; 96 against 118 us
  // at n 32768, d 1002. bf16 pairs: staged, 67 against 124 us; so is the backward)
  if (bytes < 4 || (bytes < 16 && sizeof(T) == 4) || p.stages < 1) {
    p.stages = 1;
    return p.d > 8192 ? run_fwd<T, 1, 16, false>(p, 0, s) : run_fwd<T, 1, 8, false>(p, 0, s);
  }
  const size_t smem = p.stages * p.slots * row;
  if constexpr (sizeof(T) == 2)
    if (bytes < 16)
      return p.d > 8192 ? run_fwd<T, V4, 16, true>(p, smem, s)
                        : run_fwd<T, V4, 8, true>(p, smem, s);
  return p.d > 8192 ? run_fwd<T, V16, 16, true>(p, smem, s) : run_fwd<T, V16, 8, true>(p, smem, s);
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
struct NormBwd {
  const void *dout, *dh, *out, *y, *gate;
  const float *w_post, *w_next, *rstd_post, *rstd_next;
  void *dx, *dy, *dgate;
  float *dw_post, *dw_next;
  // partial sums [blocks][pitch] of dw_post, dw_next and, with one gate row
  // for all tokens, of dgate; with more gate rows [workers][pitch] of the
  // rows that a worker holds a part of: the one that began in an earlier
  // worker (head) and the one that goes on in a later one (tail)
  float *part_post, *part_next, *part_gate, *part_head, *part_tail;
  int pitch;
  int n, d, gate_tokens, workers, blocks, stages, slots;
  uint32_t ring_bytes;  // of a worker
  float off, a, b;
  long long gate_stride;
};

// Three sums over a worker at once. Within a warp, halves of the lanes first
// trade values so that each lane carries one sum (18 instructions instead of
// 30); the warps' sums then meet in `red` as one 16-byte vector a warp.
__device__ __forceinline__ float sum3_lanes(float a, float b, float c, int lane) {
  const bool h16 = lane & 16, h8 = lane & 8;
  float k0 = h16 ? c : a, k1 = h16 ? 0.0f : b;
  k0 += __shfl_xor_sync(0xffffffffu, h16 ? a : c, 16);
  k1 += __shfl_xor_sync(0xffffffffu, h16 ? b : 0.0f, 16);
  float k = h8 ? k1 : k0;
  k += __shfl_xor_sync(0xffffffffu, h8 ? k0 : k1, 8);
  k += __shfl_xor_sync(0xffffffffu, k, 4);
  k += __shfl_xor_sync(0xffffffffu, k, 2);
  k += __shfl_xor_sync(0xffffffffu, k, 1);
  return k;  // lanes 0-7: a, 8-15: b, 16-23: c
}
// (red: the worker's, one entry a warp; a worker's barrier is its own)
__device__ __forceinline__ void worker_sum3(float& a, float& b, float& c, float4* red, int warps) {
  const int lane = threadIdx.x & 31;
  float k = sum3_lanes(a, b, c, lane);
  if (warps > 1) {
    if ((lane & 7) == 0) reinterpret_cast<float*>(red + (threadIdx.x >> 5))[lane >> 3] = k;
    asm volatile("bar.sync %0, %1;" ::"r"(threadIdx.y + 1), "r"(warps * 32) : "memory");
    const float4 v = lane < warps ? red[lane] : make_float4(0, 0, 0, 0);
    k = sum3_lanes(v.x, v.y, v.z, lane);
  }
  a = __shfl_sync(0xffffffffu, k, 0);
  b = __shfl_sync(0xffffffffu, k, 8);
  c = __shfl_sync(0xffffffffu, k, 16);
}

// A block holds blockDim.y workers of blockDim.x threads, each with rows, ring
// and barrier of its own; at the end their sums meet in shared memory, so that
// a block leaves one partial row.
// Sums over tokens: dw_next in registers over all of the worker's rows; the
// gate's and dw_post share one, A = sum D yr over the rows of one gate row,
// of which they are dgate = b (w_post + off) A and dw_post += b gate A, taken
// when the gate row or the range ends (where rows of several gates meet in a
// range, dw_post's running sum waits in shared memory between). With 64
// registers a thread the next norm's weights are read from shared memory, not
// kept: what the compiler spilled instead missed the small L1 that the rings
// leave (182 against 151 us at n 8192, d 7168, 1,024 tokens a gate row).
template <typename T, int VEC, int EPT, bool STAGED, int MAXT, bool ALL>
__global__ void __launch_bounds__(MAXT) norm_bwd_kernel(const NormBwd p) {
  extern __shared__ __align__(16) unsigned char nsm[];
  __shared__ float4 red[2][32];
  pdl_wait();
  constexpr int P = EPT / 2;
  // with 64 registers a thread, y is read again for the second half of a row,
  // and the next norm's weights for each row
  constexpr int KEEP = MAXT <= 768;
  const Cols<T, VEC, EPT> cols{(int)threadIdx.x, (int)blockDim.x, p.d / VEC};
  const int warps = blockDim.x >> 5;
  const int group = threadIdx.y, groups = blockDim.y;
  const int w = blockIdx.x * groups + group;
  const int r0 = w < p.workers ? worker_row(w, p.n, p.workers) : p.n;
  const int r1 = w < p.workers ? worker_row(w + 1, p.n, p.workers) : p.n;
  // ALL: every optional part but the gate is there, known when compiled (it
  // saves the registers of the other kernel's flags)
  const bool has_y = ALL || p.y, post = ALL || p.w_post, next = ALL || p.dh,
             has_dout = ALL || p.dout;
  const bool gate_all = p.gate && p.gate_tokens == 0, gate_each = p.gate && p.gate_tokens == 1,
             gate_rows = p.gate && p.gate_tokens > 0;
  // (addresses are made from the parameters and one offset: registers are short)
  auto in = [](const void* q, size_t at) { return static_cast<const T*>(q) + at; };
  auto to = [](void* q, size_t at) { return static_cast<T*>(q) + at; };
  const float inv_d = 1.0f / (float)p.d;
  // the workers' rings; each takes its worker's sums of dw_next, of the one gate
  // row and of dw_post at the end; then, [columns] of fp32 a worker each, the
  // running sums of dw_post and the next norm's weights
  const uint32_t pitch = (uint32_t)blockDim.x * EPT * sizeof(T);
  const uint32_t fpitch = (uint32_t)blockDim.x * EPT;
  unsigned char* mine = nsm + (size_t)group * p.ring_bytes;
  Ring ring(mine, p.slots * pitch, p.stages);
  const bool running = post && gate_rows;
  // (addresses of what is used seldom are made where it is)
  auto ring_end = [&](int which) {
    return reinterpret_cast<float*>(nsm + (size_t)group * p.ring_bytes) + which * fpitch;
  };
  auto extra = [&](int which) {
    return reinterpret_cast<float*>(nsm + (size_t)groups * p.ring_bytes) +
           (size_t)(which * groups + group) * fpitch;
  };
  const int at_gate = next ? 1 : 0, at_post = at_gate + (gate_all ? 1 : 0);
  // offsets of a stage's rows, in this order where present: dh, out, y, dout, gate
  const uint32_t s_y = next ? 2 * pitch : 0, s_dout = s_y + (has_y ? pitch : 0),
                 s_gate = s_dout + (has_dout ? pitch : 0);
  auto issue = [&](int r) {
    if constexpr (STAGED) {
      if (r < r1) {
        const size_t row = (size_t)r * p.d;
#pragma unroll
        for (int i = 0; i < cols.ITEMS; ++i) {
          constexpr int B = Cols<T, VEC, EPT>::BYTES;
          const uint32_t n = cols.has(i) ? B : 0;
          const int c = n ? cols.at(i) : 0;
          const uint32_t dst = ring.fill + (uint32_t)(i * cols.threads + cols.tid) * B;
          if (next) {
            cp_async<B>(dst, in(p.dh, row + c), n);
            cp_async<B>(dst + pitch, in(p.out, row + c), n);
          }
          if (has_y) cp_async<B>(dst + s_y, in(p.y, row + c), n);
          if (has_dout) cp_async<B>(dst + s_dout, in(p.dout, row + c), n);
          if (gate_each) cp_async<B>(dst + s_gate, in(p.gate, r * p.gate_stride + c), n);
        }
        ring.filled();
      }
      cp_async_commit();
    }
  };
  for (int q = 0; q < p.stages - 1; ++q) issue(r0 + q);
  float2 cw[P], wn[P], acc_n[P], A[P];
#pragma unroll
  for (int e = 0; e < P; ++e) cw[e] = wn[e] = acc_n[e] = A[e] = both(0.0f);
  if (next) {
    cols.load_f32(wn, p.w_next);
#pragma unroll
    for (int e = 0; e < P; ++e) wn[e] = add2(wn[e], both(p.off));
  }
  if (!KEEP && EPT == 8 && next) cols.store_f32(extra(running ? 1 : 0), wn);
  if (running) cols.store_f32(extra(0), A);
  // w_post + off (1 without)
  auto post_weights = [&](float2* v) {
    if (post) {
      cols.load_f32(v, p.w_post);
#pragma unroll
      for (int e = 0; e < P; ++e) v[e] = add2(v[e], both(p.off));
    } else {
#pragma unroll
      for (int e = 0; e < P; ++e) v[e] = both(1.0f);
    }
  };
  auto gate_row = [&](float2* v, int r) {
    if (STAGED && gate_each) cols.load_smem(v, ring.read + s_gate);
    else cols.load(v, in(p.gate, p.gate_tokens ? r / p.gate_tokens * p.gate_stride : 0));
  };
  int left = 0;
  float rp_ahead = post && r0 < r1 ? p.rstd_post[r0] : 1.0f;
  float rn_ahead = next && r0 < r1 ? p.rstd_next[r0] : 0.0f;
  for (int r = r0; r < r1; ++r) {
    issue(r + p.stages - 1);
    const size_t at = (size_t)r * p.d;
    const float rp = rp_ahead, rn = rn_ahead;
    if (r + 1 < r1) {
      if (post) rp_ahead = p.rstd_post[r + 1];
      if (next) rn_ahead = p.rstd_next[r + 1];
    }
    if (STAGED) cp_async_wait_row(p.stages);
    if (left == 0 && has_y) {
      post_weights(cw);
#pragma unroll
      for (int e = 0; e < P; ++e) cw[e] = mul2(cw[e], both(p.b));
      if (p.gate) {
        float2 g[P];
        gate_row(g, r);
#pragma unroll
        for (int e = 0; e < P; ++e) cw[e] = mul2(cw[e], g[e]);
      }
      left = gate_rows_left(p.gate, p.gate_tokens, r);
    }
    --left;
    // t = dout + r2 q, u = out r2; D = t - r2 mean(q u) u
    float2 t[P], u[P], v[P];
    if (has_dout) {
      if (STAGED) cols.load_smem(t, ring.read + s_dout);
      else cols.load(t, in(p.dout, at));
    } else {
#pragma unroll
      for (int e = 0; e < P; ++e) t[e] = both(0.0f);
    }
    float k1 = 0.0f, k2 = 0.0f;
    if (next) {
      if (STAGED) cols.load_smem(u, ring.read + pitch), cols.load_smem(v, ring.read);
      else cols.load(u, in(p.out, at)), cols.load(v, in(p.dh, at));
      float2 s1 = both(0.0f);
      if constexpr (!KEEP) {
        if constexpr (EPT == 8) {
          cols.load_f32(wn, extra(running ? 1 : 0));
        } else {  // (shared memory is short here)
          cols.load_f32(wn, p.w_next);
#pragma unroll
          for (int e = 0; e < P; ++e) wn[e] = add2(wn[e], both(p.off));
        }
      }
#pragma unroll
      for (int e = 0; e < P; ++e) {
        u[e] = mul2(u[e], both(rn));
        acc_n[e] = fma2(v[e], u[e], acc_n[e]);
        v[e] = mul2(v[e], wn[e]);
        s1 = fma2(v[e], u[e], s1);
        t[e] = fma2(v[e], both(rn), t[e]);
      }
      k1 = s1.x + s1.y;
    } else {
#pragma unroll
      for (int e = 0; e < P; ++e) u[e] = both(0.0f);
    }
    auto load_y = [&]() {
      if (STAGED) cols.load_smem(v, ring.read + s_y);
      else cols.load(v, in(p.y, at));
    };
    if (has_y) {
      load_y();
      if (post) {
#pragma unroll
        for (int e = 0; e < P; ++e) v[e] = mul2(v[e], both(rp));  // yr
      }
    }
    if (next || post) {
      float2 s2 = both(0.0f), s3 = both(0.0f);
      if (post) {
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const float2 c = mul2(v[e], cw[e]);
          s2 = fma2(t[e], c, s2);
          s3 = fma2(u[e], c, s3);
        }
      }
      float a2 = s2.x + s2.y, a3 = s3.x + s3.y;
      // two buffers: a warp may still read row r's while row r + 1 is written
      worker_sum3(k1, a2, a3, red[r & 1] + group * warps, warps);
      k1 *= rn * inv_d;                  // r2 mean(q u)
      k2 = (a2 - k1 * a3) * inv_d * rp;  // r1 mean(D c)
      if (has_y && !KEEP) load_y();
    }
#pragma unroll
    for (int e = 0; e < P; ++e) {
      t[e] = fma2(u[e], both(-k1), t[e]);  // D
      u[e] = mul2(t[e], both(p.a));
    }
    cols.store(to(p.dx, at), u);
    if (has_y) {
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const float2 yr = KEEP || !post ? v[e] : mul2(v[e], both(rp));
        A[e] = fma2(t[e], yr, A[e]);
        u[e] = mul2(t[e], cw[e]);
        if (post) u[e] = fma2(u[e], both(rp), mul2(yr, both(-k2)));
      }
      cols.store(to(p.dy, at), u);
      if (gate_rows && (left == 0 || r + 1 == r1)) {
        // the gate row, or the worker's range, ends
        float2 g[P], wp[P];
        gate_row(g, r);
        post_weights(wp);
#pragma unroll
        for (int e = 0; e < P; ++e) {
          A[e] = mul2(A[e], both(p.b));
          wp[e] = mul2(wp[e], A[e]);
        }
        const int gi = r / p.gate_tokens;
        const long long first = (long long)gi * p.gate_tokens;
        const long long last = min(first + p.gate_tokens, (long long)p.n);
        if (first < r0)
          cols.store_f32(p.part_head + (size_t)w * p.pitch, wp);
        else if (last > r1)
          cols.store_f32(p.part_tail + (size_t)w * p.pitch, wp);
        else
          cols.store(static_cast<T*>(p.dgate) + (long long)gi * p.gate_stride, wp);
        if (running) {
          cols.load_f32(wp, extra(0));
#pragma unroll
          for (int e = 0; e < P; ++e) wp[e] = fma2(g[e], A[e], wp[e]);
          cols.store_f32(extra(0), wp);
        }
#pragma unroll
        for (int e = 0; e < P; ++e) A[e] = both(0.0f);
      }
    }
    ring.done();
  }
  // The ring takes the sums only when no thread reads rows from it any more: a
  // thread's columns of fp32 lie where other threads' chunks did.
  __syncthreads();
  if (next) cols.store_f32(ring_end(0), acc_n);
  if (has_y && !gate_rows) {
    float2 v[P];
#pragma unroll
    for (int e = 0; e < P; ++e) A[e] = mul2(A[e], both(p.b));
    if (gate_all) {
      post_weights(v);
#pragma unroll
      for (int e = 0; e < P; ++e) v[e] = mul2(v[e], A[e]);
      cols.store_f32(ring_end(at_gate), v);
      cols.load(v, in(p.gate, 0));
#pragma unroll
      for (int e = 0; e < P; ++e) A[e] = mul2(v[e], A[e]);
    }
    if (post) cols.store_f32(ring_end(at_post), A);
  }
  __syncthreads();
  // the workers' sums, in their order
  const bool alone = p.blocks == 1;
  const size_t ring_f = p.ring_bytes / 4;
  const float* ends = reinterpret_cast<const float*>(nsm);
  const float* sums = reinterpret_cast<const float*>(nsm + (size_t)groups * p.ring_bytes);
  const size_t row = alone ? 0 : (size_t)blockIdx.x * p.pitch;
  for (int c = group * blockDim.x + threadIdx.x; c < p.d; c += groups * blockDim.x) {
    float a = 0.0f, b = 0.0f, g = 0.0f;
    for (int k = 0; k < groups; ++k) {
      if (running) a += sums[(size_t)k * fpitch + c];
      else if (post) a += ends[k * ring_f + at_post * fpitch + c];
      if (next) b += ends[k * ring_f + c];
      if (gate_all) g += ends[k * ring_f + at_gate * fpitch + c];
    }
    if (post) (alone ? p.dw_post : p.part_post + row)[c] = a;
    if (next) (alone ? p.dw_next : p.part_next + row)[c] = b;
    if (gate_all) {
      if (alone) static_cast<T*>(p.dgate)[c] = (T)g;
      else p.part_gate[row + c] = g;
    }
  }
}

// Joins the partial sums in order: 128 columns a block, 32 slices of the
// partial rows, then the slices. blockIdx.y: dw_post, dw_next, then the gate: its
// one row, or the rows that more than one worker holds, found by row (fewer
// rows than workers) or by the worker that they begin in. Rows that span a few
// workers only are a slice's work each, 32 to a block (n 16384, d 2048, 3 tokens
// a gate row: the whole backward 106 us, with a block for each 200).
struct NormReduce {
  NormBwd b;
  int by_group;
  int slice_rows;  // a gate row a slice
};
constexpr int kRedSlices = 32;

template <typename T>
__global__ void __launch_bounds__(32 * kRedSlices) norm_reduce_kernel(const NormReduce q) {
  __shared__ float4 part[kRedSlices][32];
  pdl_wait();
  const NormBwd& p = q.b;
  const int job = blockIdx.y;
  const float* first_src;  // partial row w_lo
  const float* src;        // the others': src + w * pitch
  int w_lo = 0, w_hi = p.blocks;  // partial rows w_lo .. w_hi - 1
  long long group = 0;
  bool mine = true;  // (with a slice a row, a slice may have none)
  const bool slices = job >= 2 && q.slice_rows;
  if (job == 0) {
    if (!p.w_post) return;
    first_src = src = p.part_post;
  } else if (job == 1) {
    if (!p.w_next) return;
    first_src = src = p.part_next;
  } else if (p.gate_tokens == 0) {
    first_src = src = p.part_gate;
  } else {
    const long long tokens = p.gate_tokens;
    const long long rows = (p.n + tokens - 1) / tokens;
    const long long nth = slices ? (long long)(job - 2) * kRedSlices + threadIdx.y : job - 2;
    mine = nth < (q.by_group ? rows : p.workers);
    if (mine) {
      if (q.by_group) {
        group = nth;
      } else {
        const int end = worker_row((int)nth + 1, p.n, p.workers);
        mine = end != worker_row((int)nth, p.n, p.workers);
        group = (end - 1) / tokens;
      }
      const long long first = group * tokens, last = min(first + tokens, (long long)p.n);
      w_lo = row_worker((int)first, p.n, p.workers);
      w_hi = row_worker((int)last - 1, p.n, p.workers) + 1;
      if (!q.by_group && w_lo != nth) mine = false;  // it began earlier
      if (w_hi - w_lo == 1) mine = false;            // one worker holds it: already written
    }
    if (!slices && !mine) return;
    src = p.part_head;
    first_src = p.part_tail + (size_t)w_lo * p.pitch;
  }
  const int col = (blockIdx.x * 32 + threadIdx.x) * 4;
  float4 s = make_float4(0, 0, 0, 0);
  if (col < p.pitch && mine) {
#pragma unroll 4
    for (int w = w_lo + (slices ? 0 : threadIdx.y); w < w_hi; w += slices ? 1 : kRedSlices) {
      const float* row = w == w_lo ? first_src : src + (size_t)w * p.pitch;
      const float4 v = *reinterpret_cast<const float4*>(row + col);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
  }
  auto put = [&](const float4& r) {
    const float v[4] = {r.x, r.y, r.z, r.w};
    for (int j = 0; j < 4; ++j) {
      if (col + j >= p.d) break;
      if (job == 0) p.dw_post[col + j] = v[j];
      else if (job == 1) p.dw_next[col + j] = v[j];
      else static_cast<T*>(p.dgate)[group * p.gate_stride + col + j] = T(v[j]);
    }
  };
  if (slices) {
    if (mine) put(s);
    return;
  }
  part[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y) return;
  for (int i = 1; i < kRedSlices; ++i) {
    const float4 v = part[i][threadIdx.x];
    s.x += v.x;
    s.y += v.y;
    s.z += v.z;
    s.w += v.w;
  }
  put(s);
}

// ---- work split of the backward ---------------------------------------------
// One block an SM with as many workers as its registers hold (80 a thread up to
// 256 threads a worker, 64 above), fewer where there are not enough rows for
// all: two rows each at least, as one would only add partial sums to join (n
// 1000, d 1024: 9.1 against 9.8 us), or one while not even half of the workers get
// one (n 64, d 7168: 12.1 against 13.8 us).
int bwd_groups(int d) {
  const int t = norm_threads(d);
  const int k = (t <= 256 ? 768 : 1024) / t;
  return k < 1 ? 1 : k > 12 ? 12 : k;
}
struct BwdSplit {
  int workers, groups, blocks;
};
BwdSplit bwd_split(int n, int d) {
  const long long most = (long long)kBlockSms * bwd_groups(d);
  const long long want = 2LL * n <= most ? n : ((long long)n + 1) / 2;
  BwdSplit s;
  s.workers = (int)(want < most ? want : most);
  s.groups = (s.workers + kBlockSms - 1) / kBlockSms;
  if (s.groups < 1) s.groups = 1;
  s.blocks = (s.workers + s.groups - 1) / s.groups;
  return s;
}
int bwd_pitch(int d) { return (d + 31) / 32 * 32; }

template <typename T, int VEC, int EPT, bool STAGED, int MAXT, bool ALL = false>
cudaError_t run_bwd(const NormBwd& p, int groups, size_t smem, cudaStream_t s) {
  if constexpr (STAGED && !ALL)
    if (p.y && p.w_post && p.dh && p.dout)
      return run_bwd<T, VEC, EPT, STAGED, MAXT, true>(p, groups, smem, s);
  auto kern = norm_bwd_kernel<T, VEC, EPT, STAGED, MAXT, ALL>;
  if (smem > 32 * 1024) {  // (48 KB with the static part need no leave)
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_all_smem(kern, done);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kern, dim3(p.blocks), dim3(norm_threads(p.d), groups), smem, s, p);
}

template <typename T>
cudaError_t launch_bwd(NormBwd& p, int groups, int bytes, cudaStream_t s) {
  constexpr int V16 = 16 / sizeof(T), V4 = 4 / sizeof(T);
  const size_t cols = (size_t)norm_threads(p.d) * (p.d > 8192 ? 16 : 8);
  const size_t row = cols * sizeof(T);
  const bool gate_all = p.gate && p.gate_tokens == 0;
  const bool running = p.w_post && p.gate && p.gate_tokens;
  const bool few = norm_threads(p.d) <= 256 && bytes >= 4;  // 80 registers a thread, not 64
  const size_t sums = cols * 4 * ((running ? 1 : 0) + (p.w_next && !few && p.d <= 8192 ? 1 : 0));
  const size_t ends =
      cols * 4 * ((p.w_next ? 1 : 0) + (gate_all ? 1 : 0) + (p.w_post && !running ? 1 : 0));
  p.slots = (p.dh ? 2 : 0) + (p.y ? 1 : 0) + (p.dout ? 1 : 0) +
            (p.gate && p.gate_tokens == 1 ? 1 : 0);
  const size_t budget = ring_budget(groups);
  const size_t fit = budget > sums ? (budget - sums) / (p.slots * row) : 0;
  const int deep = (p.n + p.workers - 1) / p.workers;
  p.stages = fit > kMaxStages ? kMaxStages : (int)fit;
  if (p.stages > deep) p.stages = deep;
  // Where no stage fits beside the workers that the split gives a block, the rows go
  // through single loads, whatever their alignment: fp32 with a gate row for each
  // token, n 4096, d 4096 189 us against 103 at d 3840 and 144 at d 4160, where one fits.
  const bool staged = bytes >= 4 && p.stages >= 1 && ends + sums <= budget;
  if (!staged) p.stages = 1;
  const size_t ring = staged ? p.stages * p.slots * row : 0;
  p.ring_bytes = (uint32_t)(ring > ends ? ring : ends);
  const size_t smem = groups * (p.ring_bytes + sums);
  if (!staged)
    return p.d > 8192 ? run_bwd<T, 1, 16, false, 1024>(p, groups, smem, s)
                      : run_bwd<T, 1, 8, false, 1024>(p, groups, smem, s);
  if (bytes < 16) {
    if (p.d > 8192) return run_bwd<T, V4, 16, true, 1024>(p, groups, smem, s);
    return few ? run_bwd<T, V4, 8, true, 768>(p, groups, smem, s)
               : run_bwd<T, V4, 8, true, 1024>(p, groups, smem, s);
  }
  if (p.d > 8192) return run_bwd<T, V16, 16, true, 1024>(p, groups, smem, s);
  return few ? run_bwd<T, V16, 8, true, 768>(p, groups, smem, s)
             : run_bwd<T, V16, 8, true, 1024>(p, groups, smem, s);
}

moe_status norm_check(const moe_norm_config* c) {
  if (!c || c->n < 0 || c->d < 1) return MOE_ERR_INVALID_ARG;
  if (c->dtype != MOE_F32 && c->dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (!(c->eps > 0.0f) || c->gate_tokens < 0 || c->gate_stride < c->d) return MOE_ERR_INVALID_ARG;
  if (!(c->eps < 3.0e38f)) return MOE_ERR_INVALID_ARG;
  if (c->d > MOE_NORM_MAX_D || c->n > (1 << 30)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int gate_rows(const moe_norm_config* c) {
  return c->gate_tokens ? (int)(((long long)c->n + c->gate_tokens - 1) / c->gate_tokens) : 1;
}

// The boundary that every row of every operand starts on: 16 bytes (the fp32
// weights' too), 4, or an element's 2.
int row_bytes_of(const moe_norm_config* c, bool gate, std::initializer_list<const void*> rows,
                 std::initializer_list<const void*> weights) {
  const long long elt = c->dtype == MOE_BF16 ? 2 : 4;
  uintptr_t all = (uintptr_t)(c->d * elt) | (gate ? (uintptr_t)(c->gate_stride * elt) : 0);
  for (const void* q : rows) all |= reinterpret_cast<uintptr_t>(q);
  uintptr_t w = 0;
  for (const void* q : weights) w |= reinterpret_cast<uintptr_t>(q);
  if (all % 16 == 0 && w % 16 == 0) return 16;
  return all % 4 == 0 ? 4 : 2;
}

bool element_aligned(const moe_norm_config* c, std::initializer_list<const void*> ptrs) {
  const uintptr_t mask = c->dtype == MOE_BF16 ? 1 : 3;
  for (const void* q : ptrs)
    if (reinterpret_cast<uintptr_t>(q) & mask) return false;
  return true;
}

bool f32_aligned(std::initializer_list<const void*> ptrs) {
  for (const void* q : ptrs)
    if (reinterpret_cast<uintptr_t>(q) & 3) return false;
  return true;
}

moe_status forward_impl(const moe_norm_config* c, const NormFwd& q, cudaStream_t s) {
  NormFwd p = q;
  p.n = c->n;
  p.d = c->d;
  p.gate_tokens = c->gate_tokens;
  p.gate_stride = c->gate_stride;
  p.eps = c->eps;
  p.off = c->weight_offset;
  if (!element_aligned(c, {p.x, p.y, p.gate, p.out, p.h}) ||
      !f32_aligned({p.w_post, p.w_next, p.rstd_post, p.rstd_next}))
    return MOE_ERR_INVALID_ARG;
  const int bytes = row_bytes_of(c, p.gate != nullptr, {p.x, p.y, p.gate, p.out, p.h},
                                 {p.w_post, p.w_next});
  const cudaError_t e = c->dtype == MOE_BF16 ? launch_fwd<__nv_bfloat16>(p, bytes, s)
                                             : launch_fwd<float>(p, bytes, s);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// Partial rows: dw_post, dw_next and the one gate row a block, or two of the
// gate rows a worker.
size_t backward_bytes(const moe_norm_config* c) {
  const BwdSplit k = bwd_split(c->n, c->d);
  const size_t rows =
      c->gate_tokens ? 2 * (size_t)k.blocks + 2 * (size_t)k.workers : 3 * (size_t)k.blocks;
  const size_t b = rows * bwd_pitch(c->d) * sizeof(float);
  return b < 256 ? 256 : b;
}

// No tokens: their tensors may have no address; the sums over them are zeros
// (with one gate row for all tokens, its gradient is one of them).
moe_status backward_of_none(const moe_norm_config* c, const float* w_post, float* dw_post,
                            const void* gate, void* dgate, const float* w_next, float* dw_next,
                            const void* ws, size_t ws_bytes, cudaStream_t s) {
  const size_t elt = c->dtype == MOE_BF16 ? 2 : 4;
  const bool g = gate && c->gate_tokens == 0;
  if ((w_post && !dw_post) || (w_next && !dw_next) || (g && !dgate)) return MOE_ERR_INVALID_ARG;
  if (!f32_aligned({dw_post, dw_next}) || (g && !element_aligned(c, {dgate})))
    return MOE_ERR_INVALID_ARG;
  const moe_status st = check_block_ws(ws, ws_bytes, backward_bytes(c));
  if (st != MOE_OK) return st;
  if (w_post && cudaMemsetAsync(dw_post, 0, (size_t)c->d * 4, s) != cudaSuccess)
    return MOE_ERR_CUDA;
  if (w_next && cudaMemsetAsync(dw_next, 0, (size_t)c->d * 4, s) != cudaSuccess)
    return MOE_ERR_CUDA;
  if (g && cudaMemsetAsync(dgate, 0, c->d * elt, s) != cudaSuccess) return MOE_ERR_CUDA;
  return MOE_OK;
}

moe_status backward_impl(const moe_norm_config* c, const NormBwd& q, void* ws, size_t ws_bytes,
                         cudaStream_t s) {
  moe_status st = check_block_ws(ws, ws_bytes, backward_bytes(c));
  if (st != MOE_OK) return st;
  NormBwd p = q;
  p.n = c->n;
  p.d = c->d;
  p.gate_tokens = c->gate_tokens;
  p.gate_stride = c->gate_stride;
  p.off = c->weight_offset;
  if (!element_aligned(c, {p.dout, p.dh, p.out, p.y, p.gate, p.dx, p.dy, p.dgate}) ||
      !f32_aligned({p.w_post, p.w_next, p.rstd_post, p.rstd_next, p.dw_post, p.dw_next}))
    return MOE_ERR_INVALID_ARG;
  const BwdSplit k = bwd_split(c->n, c->d);
  p.workers = k.workers;
  p.blocks = k.blocks;
  p.pitch = bwd_pitch(c->d);
  p.part_post = static_cast<float*>(ws);
  p.part_next = p.part_post + (size_t)k.blocks * p.pitch;
  p.part_gate = p.part_head = p.part_next + (size_t)k.blocks * p.pitch;
  p.part_tail = p.part_head + (size_t)k.workers * p.pitch;
  const int bytes =
      row_bytes_of(c, p.gate != nullptr, {p.dout, p.dh, p.out, p.y, p.gate, p.dx, p.dy, p.dgate},
                   {p.w_post, p.w_next});
  cudaError_t e = c->dtype == MOE_BF16 ? launch_bwd<__nv_bfloat16>(p, k.groups, bytes, s)
                                       : launch_bwd<float>(p, k.groups, bytes, s);
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  const bool shared_rows = p.gate && p.gate_tokens > 1;  // gate rows of several workers
  if (p.blocks == 1 && (!shared_rows || p.workers == 1)) return MOE_OK;
  NormReduce r{p, 0, 0};
  if (p.blocks == 1) r.b.w_post = r.b.w_next = nullptr;  // (written already)
  int jobs = 2;
  if (shared_rows) {
    const int rows = gate_rows(c);
    r.by_group = rows <= p.workers;
    const int each = r.by_group ? rows : p.workers;
    r.slice_rows = (long long)p.gate_tokens * p.workers <= 4LL * p.n;
    jobs += r.slice_rows ? (each + kRedSlices - 1) / kRedSlices : each;
  } else if (p.gate && p.gate_tokens == 0) {
    ++jobs;
  }
  const dim3 grid((p.pitch + 127) / 128, jobs), block(32, kRedSlices);
  e = c->dtype == MOE_BF16 ? launch_pdl(norm_reduce_kernel<__nv_bfloat16>, grid, block, 0, s, r)
                           : launch_pdl(norm_reduce_kernel<float>, grid, block, 0, s, r);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_norm_validate(const moe_norm_config* cfg) { return norm_check(cfg); }

moe_status moe_norm_workspace_size(const moe_norm_config* cfg, size_t* bytes) {
  moe_status st = norm_check(cfg);
  if (st != MOE_OK) return st;
  if (bytes) *bytes = backward_bytes(cfg);
  return MOE_OK;
}

moe_status moe_norm_forward(const moe_norm_config* cfg, const void* x, const float* w, void* h,
                            float* rstd, moe_stream_t stream) {
  moe_status st = norm_check(cfg);
  if (st != MOE_OK) return st;
  if (cfg->n == 0) return MOE_OK;
  if (!x || !w || !h) return MOE_ERR_INVALID_ARG;
  NormFwd p{};
  p.x = x;
  p.w_next = w;
  p.h = h;
  p.rstd_next = rstd;
  return forward_impl(cfg, p, (cudaStream_t)stream);
}

moe_status moe_norm_backward(const moe_norm_config* cfg, const void* dres, const void* dh,
                             const void* x, const float* w, const float* rstd, void* dx,
                             float* dw, void* ws, size_t ws_bytes, moe_stream_t stream) {
  moe_status st = norm_check(cfg);
  if (st != MOE_OK) return st;
  if (cfg->n == 0)
    return backward_of_none(cfg, nullptr, nullptr, nullptr, nullptr, w, dw, ws, ws_bytes,
                            (cudaStream_t)stream);
  if (!dh || !x || !w || !rstd || !dx || !dw) return MOE_ERR_INVALID_ARG;
  NormBwd p{};
  p.dout = dres;
  p.dh = dh;
  p.out = x;
  p.w_next = w;
  p.rstd_next = rstd;
  p.dx = dx;
  p.dw_next = dw;
  p.a = 1.0f;
  return backward_impl(cfg, p, ws, ws_bytes, (cudaStream_t)stream);
}

moe_status moe_residual_norm_forward(const moe_norm_config* cfg, const void* x, const void* y,
                                     const float* w_post, const void* gate, const float* w_next,
                                     void* out, void* h, float* rstd_post, float* rstd_next,
                                     moe_stream_t stream) {
  moe_status st = norm_check(cfg);
  if (st != MOE_OK) return st;
  if (cfg->n == 0) return MOE_OK;
  if (!x || !y || !out || (h != nullptr) != (w_next != nullptr) || (h && h == out))
    return MOE_ERR_INVALID_ARG;
  NormFwd p{};
  p.x = x;
  p.y = y;
  p.gate = gate;
  p.w_post = w_post;
  p.w_next = w_next;
  p.out = out;
  p.h = h;
  p.rstd_post = rstd_post;
  p.rstd_next = rstd_next;
  p.a = cfg->res_scale;
  p.b = cfg->block_scale;
  return forward_impl(cfg, p, (cudaStream_t)stream);
}

moe_status moe_residual_norm_backward(const moe_norm_config* cfg, const void* dout,
                                      const void* dh, const void* out, const void* y,
                                      const float* w_post, const void* gate, const float* w_next,
                                      const float* rstd_post, const float* rstd_next, void* dx,
                                      void* dy, float* dw_post, void* dgate, float* dw_next,
                                      void* ws, size_t ws_bytes, moe_stream_t stream) {
  moe_status st = norm_check(cfg);
  if (st != MOE_OK) return st;
  if (cfg->n == 0)
    return backward_of_none(cfg, w_post, dw_post, gate, dgate, w_next, dw_next, ws, ws_bytes,
                            (cudaStream_t)stream);
  if ((!dout && !dh) || !y || !dx || !dy || dx == dy) return MOE_ERR_INVALID_ARG;
  if ((dh != nullptr) != (w_next != nullptr)) return MOE_ERR_INVALID_ARG;
  if (dh && (!out || !rstd_next || !dw_next)) return MOE_ERR_INVALID_ARG;
  if (w_post && (!rstd_post || !dw_post)) return MOE_ERR_INVALID_ARG;
  if (gate && !dgate) return MOE_ERR_INVALID_ARG;
  NormBwd p{};
  p.dout = dout;
  p.dh = dh;
  p.out = dh ? out : nullptr;
  p.y = y;
  p.gate = gate;
  p.w_post = w_post;
  p.w_next = w_next;
  p.rstd_post = rstd_post;
  p.rstd_next = rstd_next;
  p.dx = dx;
  p.dy = dy;
  p.dgate = dgate;
  p.dw_post = dw_post;
  p.dw_next = dw_next;
  p.a = cfg->res_scale;
  p.b = cfg->block_scale;
  return backward_impl(cfg, p, ws, ws_bytes, (cudaStream_t)stream);
}

}  // extern "C"
