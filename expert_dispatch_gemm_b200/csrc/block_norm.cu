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
// so a row takes one block reduction (of three sums), not two in sequence.
//
// All four kernels are bound by HBM: the forward moves 4 n d elements (x, y,
// out, h), the backward 6 n d.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <initializer_list>

#include "block_internal.h"
#include "device_common.cuh"

namespace moe {
namespace {

// ---- VEC consecutive elements of a row ------------------------------------
template <typename T, int VEC>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16, 8> {
  uint4 r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    r = __ldcs(reinterpret_cast<const uint4*>(p));
  }
  __device__ __forceinline__ void load_smem(const void* p) {
    r = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void zero() { r = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ float get(int i) const {
    const uint32_t w = i < 2 ? r.x : i < 4 ? r.y : i < 6 ? r.z : r.w;
    return __uint_as_float((i & 1) ? (w & 0xffff0000u) : (w << 16));
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* v) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                              pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
};
template <>
struct Chunk<float, 4> {
  float4 r;
  __device__ __forceinline__ void load(const float* p) {
    r = __ldcs(reinterpret_cast<const float4*>(p));
  }
  __device__ __forceinline__ void load_smem(const void* p) {
    r = *reinterpret_cast<const float4*>(p);
  }
  __device__ __forceinline__ void zero() { r = make_float4(0, 0, 0, 0); }
  __device__ __forceinline__ float get(int i) const {
    return i == 0 ? r.x : i == 1 ? r.y : i == 2 ? r.z : r.w;
  }
  static __device__ __forceinline__ void store(float* p, const float* v) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
};
template <>
struct Chunk<__nv_bfloat16, 1> {
  uint16_t r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    r = *reinterpret_cast<const uint16_t*>(p);
  }
  __device__ __forceinline__ void load_smem(const void* p) {
    r = *reinterpret_cast<const uint16_t*>(p);
  }
  __device__ __forceinline__ void zero() { r = 0; }
  __device__ __forceinline__ float get(int) const { return bf16_to_f32(r); }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* v) {
    *p = __float2bfloat16_rn(v[0]);
  }
};
template <>
struct Chunk<float, 1> {
  float r;
  __device__ __forceinline__ void load(const float* p) { r = *p; }
  __device__ __forceinline__ void load_smem(const void* p) {
    r = *reinterpret_cast<const float*>(p);
  }
  __device__ __forceinline__ void zero() { r = 0.0f; }
  __device__ __forceinline__ float get(int) const { return r; }
  static __device__ __forceinline__ void store(float* p, const float* v) { *p = v[0]; }
};

// VEC fp32 weights (read by every row: they stay in L1)
template <int VEC>
__device__ __forceinline__ void load_weights(float* w, const float* p, float off) {
  if constexpr (VEC == 1) {
    w[0] = __ldg(p) + off;
  } else {
#pragma unroll
    for (int i = 0; i < VEC; i += 4) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(p + i));
      w[i] = v.x + off;
      w[i + 1] = v.y + off;
      w[i + 2] = v.z + off;
      w[i + 3] = v.w + off;
    }
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over the threads of a row: the warp, or (block rows) all of the block's
// warps through `red` [32], which the caller does not reuse before another
// block barrier.
__device__ __forceinline__ float row_sum(float v, float* red, bool block_row) {
  v = warp_sum(v);
  if (!block_row) return v;
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (lane == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum(lane < warps ? red[lane] : 0.0f);
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
struct NormFwd {
  const void *x, *y, *gate;
  const float *w_post, *w_next;
  void *out, *h;
  float *rstd_post, *rstd_next;
  int n, d, gate_tokens;
  float eps, off, a, b;
  long long gate_stride;
};

// A row belongs to one warp (blockDim = 32 x rows: narrow rows) or to the
// whole block (blockDim = threads x 1). Each thread keeps ITEMS chunks of
// x and y in registers from the one read to the writes, chunk c of the row at
// thread c % threads, so that every access is one coalesced 16-byte vector.
template <typename T, int VEC, int ITEMS, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_fwd_kernel(const NormFwd p) {
  __shared__ float red[2][32];
  pdl_wait();
  const int row = blockIdx.x * blockDim.y + threadIdx.y;
  if (row >= p.n) return;  // (warp rows only: no barrier follows)
  const bool block_row = blockDim.x > 32;
  const int tid = threadIdx.x, threads = blockDim.x;
  const int chunks = p.d / VEC;
  const size_t base = (size_t)row * p.d;
  const T* x = static_cast<const T*>(p.x) + base;
  const T* y = p.y ? static_cast<const T*>(p.y) + base : nullptr;
  using C = Chunk<T, VEC>;
  C cx[ITEMS], cy[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int c = i * threads + tid;
    cx[i].zero();
    cy[i].zero();
    if (c < chunks) {
      if (y) cy[i].load(y + c * VEC);
      cx[i].load(x + c * VEC);
    }
  }
  float o[ITEMS * VEC];
  float ss = 0.0f;
  if (y) {
    float r1 = 1.0f;
    if (p.w_post) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < ITEMS; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) s = fmaf(cy[i].get(j), cy[i].get(j), s);
      s = row_sum(s, red[0], block_row);
      r1 = rsqrtf(s / (float)p.d + p.eps);
      if (p.rstd_post && tid == 0) p.rstd_post[row] = r1;
    }
    const T* gate = nullptr;
    if (p.gate)
      gate = static_cast<const T*>(p.gate) +
             (p.gate_tokens ? (long long)(row / p.gate_tokens) * p.gate_stride : 0);
    T* out = static_cast<T*>(p.out) + base;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = i * threads + tid;
      if (c < chunks) {
        float w[VEC];
        C g;
        if (p.w_post) load_weights<VEC>(w, p.w_post + c * VEC, p.off);
        if (gate) g.load(gate + c * VEC);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          float v = cy[i].get(j);
          if (p.w_post) v = v * r1 * w[j];
          if (gate) v *= g.get(j);
          o[i * VEC + j] = fmaf(p.a, cx[i].get(j), p.b * v);
        }
        C::store(out + c * VEC, o + i * VEC);
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[i * VEC + j] = 0.0f;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) o[i * VEC + j] = cx[i].get(j);
  }
  if (!p.h) return;
#pragma unroll
  for (int i = 0; i < ITEMS * VEC; ++i) ss = fmaf(o[i], o[i], ss);
  ss = row_sum(ss, red[1], block_row);
  const float r2 = rsqrtf(ss / (float)p.d + p.eps);
  if (p.rstd_next && tid == 0) p.rstd_next[row] = r2;
  T* h = static_cast<T*>(p.h) + base;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int c = i * threads + tid;
    if (c < chunks) {
      float w[VEC];
      load_weights<VEC>(w, p.w_next + c * VEC, p.off);
#pragma unroll
      for (int j = 0; j < VEC; ++j) o[i * VEC + j] = o[i * VEC + j] * r2 * w[j];
      C::store(h + c * VEC, o + i * VEC);
    }
  }
}

template <typename T, int VEC, int ITEMS, int MAXT>
cudaError_t run_fwd(const NormFwd& p, dim3 grid, dim3 block, cudaStream_t s) {
  return launch_pdl(norm_fwd_kernel<T, VEC, ITEMS, MAXT>, grid, block, 0, s, p);
}

// Narrow rows (up to 32 elements a lane with vectors, 8 without): a warp
// each, four to a block. Wider ones: a block each, with 16 elements a thread
// (32 where 1024 threads would not reach).
template <typename T, int VEC>
cudaError_t launch_fwd(const NormFwd& p, cudaStream_t s) {
  constexpr int E16 = VEC == 1 ? 16 : 16 / VEC;  // chunks a thread for 16 elements
  constexpr int E8 = VEC == 1 ? 8 : 8 / VEC;
  const int chunks = p.d / VEC;
  constexpr int kRows = 4;
  const dim3 wgrid((p.n + kRows - 1) / kRows), wblock(32, kRows);
  if (chunks <= 32 * E8) return run_fwd<T, VEC, E8, 128>(p, wgrid, wblock, s);
  if (VEC > 1 && chunks <= 32 * E16) return run_fwd<T, VEC, E16, 128>(p, wgrid, wblock, s);
  const int threads = ((chunks + E16 - 1) / E16 + 31) / 32 * 32;
  return run_fwd<T, VEC, E16, 1024>(p, dim3(p.n), dim3(threads), s);
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
struct NormBwd {
  const void *dout, *dh, *out, *y, *gate;
  const float *w_post, *w_next, *rstd_post, *rstd_next;
  void *dx, *dy, *dgate;
  float *dw_post, *dw_next;  // final sums (workers == 1)
  // partial sums: [workers][pitch] each; a worker's incomplete gate groups
  // are the one that began in an earlier worker (head) and the one that goes
  // on in a later one (tail)
  float *part_post, *part_next, *part_head, *part_tail;
  int pitch;
  int n, d, gate_tokens, workers, stages, slots;
  float off, a, b;
  long long gate_stride;
};

__host__ __device__ __forceinline__ int worker_row(int w, int n, int workers) {
  return (int)((long long)w * n / workers);
}
// the worker that holds row r
__host__ __device__ __forceinline__ int row_worker(int r, int n, int workers) {
  return (int)((((long long)r + 1) * workers - 1) / n);
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// One worker (block) owns a contiguous range of rows and walks it row by row;
// a thread owns the same ITEMS chunks of columns in every row, so the sums
// over tokens (dw_post, dw_next, dgate) stay in its registers until the range
// or the gate's token group ends. STAGED: the next rows' chunks are on their
// way into shared memory by cp.async while this one is computed; each thread
// reads back only what it copied itself, so no barrier guards the ring.
template <typename T, int VEC, int ITEMS, bool STAGED, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_bwd_kernel(const NormBwd p) {
  extern __shared__ __align__(16) unsigned char nsm[];
  __shared__ float red[2][3][32];
  pdl_wait();
  using C = Chunk<T, VEC>;
  const int tid = threadIdx.x, threads = blockDim.x, lane = tid & 31, warps = threads >> 5;
  const int chunks = p.d / VEC;
  const int w = blockIdx.x;
  const int r0 = worker_row(w, p.n, p.workers), r1 = worker_row(w + 1, p.n, p.workers);
  const T* dout = static_cast<const T*>(p.dout);
  const T* dh = static_cast<const T*>(p.dh);
  const T* out = static_cast<const T*>(p.out);
  const T* y = static_cast<const T*>(p.y);
  const T* gate = static_cast<const T*>(p.gate);
  const float inv_d = 1.0f / (float)p.d;
  const size_t row_bytes = (size_t)p.d * sizeof(T);
  auto gate_row = [&](int r) {
    return gate + (p.gate_tokens ? (long long)(r / p.gate_tokens) * p.gate_stride : 0);
  };
  auto issue = [&](int r) {
    if (STAGED && r < r1) {
      unsigned char* st = nsm + (size_t)((r - r0) % p.stages) * p.slots * row_bytes;
      const T* gr = gate ? gate_row(r) : nullptr;
      const size_t base = (size_t)r * p.d;
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        const int c = i * threads + tid;
        if (c < chunks) {
          unsigned char* dst = st + (size_t)c * 16;
          if (dh) {
            cp_async16(dst, dh + base + c * VEC), dst += row_bytes;
            cp_async16(dst, out + base + c * VEC), dst += row_bytes;
          }
          if (y) cp_async16(dst, y + base + c * VEC), dst += row_bytes;
          if (dout) cp_async16(dst, dout + base + c * VEC), dst += row_bytes;
          if (gr) cp_async16(dst, gr + c * VEC);
        }
      }
    }
    if (STAGED) cp_async_commit();
  };

  float wp[ITEMS * VEC], wn[ITEMS * VEC];
  float acc_p[ITEMS * VEC], acc_n[ITEMS * VEC], acc_g[ITEMS * VEC];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int c = i * threads + tid;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      wp[i * VEC + j] = 1.0f;
      wn[i * VEC + j] = 0.0f;
      acc_p[i * VEC + j] = acc_n[i * VEC + j] = acc_g[i * VEC + j] = 0.0f;
    }
    if (c < chunks) {
      if (p.w_post) load_weights<VEC>(wp + i * VEC, p.w_post + c * VEC, p.off);
      if (p.w_next) load_weights<VEC>(wn + i * VEC, p.w_next + c * VEC, p.off);
    }
  }
  for (int q = 0; q < p.stages - 1; ++q) issue(r0 + q);
  for (int r = r0; r < r1; ++r) {
    issue(r + p.stages - 1);
    const size_t base = (size_t)r * p.d;
    const float rp = p.w_post ? p.rstd_post[r] : 1.0f;
    const float rn = dh ? p.rstd_next[r] : 0.0f;
    if (STAGED) {
      if (p.stages == 1) cp_async_wait<0>();
      else if (p.stages == 2) cp_async_wait<1>();
      else cp_async_wait<2>();
    }
    const unsigned char* st = nsm + (size_t)((r - r0) % p.stages) * p.slots * row_bytes;
    const T* gr = gate ? gate_row(r) : nullptr;
    auto fetch = [&](int c, C& a_dh, C& a_out, C& a_y, C& a_dout, C& a_g) {
      if (STAGED) {
        const unsigned char* src = st + (size_t)c * 16;
        if (dh) {
          a_dh.load_smem(src), src += row_bytes;
          a_out.load_smem(src), src += row_bytes;
        }
        if (y) a_y.load_smem(src), src += row_bytes;
        if (dout) a_dout.load_smem(src), src += row_bytes;
        if (gate) a_g.load_smem(src);
      } else {
        if (dh) {
          a_dh.load(dh + base + c * VEC);
          a_out.load(out + base + c * VEC);
        }
        if (y) a_y.load(y + base + c * VEC);
        if (dout) a_dout.load(dout + base + c * VEC);
        if (gate) a_g.load(gr + c * VEC);
      }
    };
    // the three sums: q u, (dout + r2 q) c, u c
    float s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
    if (dh || p.w_post) {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        const int c = i * threads + tid;
        if (c < chunks) {
          C a_dh, a_out, a_y, a_dout, a_g;
          a_dh.zero();
          a_out.zero();
          a_y.zero();
          a_dout.zero();
          fetch(c, a_dh, a_out, a_y, a_dout, a_g);
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const int e = i * VEC + j;
            const float u = a_out.get(j) * rn;
            const float q = a_dh.get(j) * wn[e];
            float cc = a_y.get(j) * rp * wp[e];
            if (gate) cc *= a_g.get(j);
            s1 = fmaf(q, u, s1);
            s2 = fmaf(fmaf(rn, q, a_dout.get(j)), cc, s2);
            s3 = fmaf(u, cc, s3);
            acc_n[e] = fmaf(a_dh.get(j), u, acc_n[e]);
          }
        }
      }
      s1 = warp_sum(s1);
      s2 = warp_sum(s2);
      s3 = warp_sum(s3);
      if (warps > 1) {
        // two buffers: a warp may still read row r's while row r + 1 is written
        float(*rd)[32] = red[r & 1];
        if (lane == 0) {
          rd[0][tid >> 5] = s1;
          rd[1][tid >> 5] = s2;
          rd[2][tid >> 5] = s3;
        }
        __syncthreads();
        s1 = warp_sum(lane < warps ? rd[0][lane] : 0.0f);
        s2 = warp_sum(lane < warps ? rd[1][lane] : 0.0f);
        s3 = warp_sum(lane < warps ? rd[2][lane] : 0.0f);
      }
    }
    const float k1 = rn * s1 * inv_d;                  // r2 mean(q u)
    const float m = p.b * (s2 - k1 * s3) * inv_d;      // mean(D c)
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = i * threads + tid;
      if (c < chunks) {
        C a_dh, a_out, a_y, a_dout, a_g;
        a_dh.zero();
        a_out.zero();
        a_y.zero();
        a_dout.zero();
        fetch(c, a_dh, a_out, a_y, a_dout, a_g);
        float vx[VEC], vy[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const int e = i * VEC + j;
          const float u = a_out.get(j) * rn;
          const float q = a_dh.get(j) * wn[e];
          const float D = fmaf(rn, q, a_dout.get(j)) - k1 * u;
          vx[j] = p.a * D;
          const float yr = a_y.get(j) * rp;
          const float dz = p.b * D;
          const float dv = gate ? dz * a_g.get(j) : dz;
          acc_g[e] = fmaf(dz, yr * wp[e], acc_g[e]);
          acc_p[e] = fmaf(dv, yr, acc_p[e]);
          vy[j] = p.w_post ? rp * (dv * wp[e] - yr * m) : dv;
        }
        C::store(static_cast<T*>(p.dx) + base + c * VEC, vx);
        if (y) C::store(static_cast<T*>(p.dy) + base + c * VEC, vy);
      }
    }
    if (gate && (r + 1 == r1 || (p.gate_tokens && (r + 1) % p.gate_tokens == 0))) {
      const int g = p.gate_tokens ? r / p.gate_tokens : 0;
      const long long first = (long long)g * p.gate_tokens;
      const long long last = p.gate_tokens ? min(first + p.gate_tokens, (long long)p.n) : p.n;
      float* part = nullptr;
      if (first < r0) part = p.part_head + (size_t)w * p.pitch;
      else if (last > r1) part = p.part_tail + (size_t)w * p.pitch;
      T* dg = static_cast<T*>(p.dgate) + (long long)g * p.gate_stride;
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        const int c = i * threads + tid;
        if (c < chunks) {
          if (part) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) part[c * VEC + j] = acc_g[i * VEC + j];
          } else {
            C::store(dg + c * VEC, acc_g + i * VEC);
          }
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) acc_g[i * VEC + j] = 0.0f;
      }
    }
  }
  const bool alone = p.workers == 1;
  float* dst_p = alone ? p.dw_post : p.part_post + (size_t)w * p.pitch;
  float* dst_n = alone ? p.dw_next : p.part_next + (size_t)w * p.pitch;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int c = i * threads + tid;
    if (c < chunks) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        if (p.w_post) dst_p[c * VEC + j] = acc_p[i * VEC + j];
        if (p.w_next) dst_n[c * VEC + j] = acc_n[i * VEC + j];
      }
    }
  }
}

// Joins the workers' partial sums in worker order: 128 columns a block, 8
// slices of the workers, then the slices in order. blockIdx.y: dw_post,
// dw_next, then the gate groups that more than one worker holds, found by
// group (fewer groups than workers) or by the worker that they begin in.
struct NormReduce {
  NormBwd b;
  int by_group;
};
constexpr int kRedSlices = 8;

template <typename T>
__global__ void __launch_bounds__(32 * kRedSlices) norm_reduce_kernel(const NormReduce q) {
  __shared__ float4 part[kRedSlices][32];
  pdl_wait();
  const NormBwd& p = q.b;
  const int job = blockIdx.y;
  const float* first_src;  // worker w_lo's partial row
  const float* src;        // the others': src + w * pitch
  int w_lo = 0, w_hi = p.workers;  // workers w_lo .. w_hi - 1
  long long group = 0;
  if (job == 0) {
    if (!p.w_post) return;
    src = p.part_post;
    first_src = src;
  } else if (job == 1) {
    if (!p.w_next) return;
    src = p.part_next;
    first_src = src;
  } else {
    const int T0 = p.gate_tokens;
    long long first, last;
    if (q.by_group) {
      group = job - 2;
    } else {
      const int end = worker_row(job - 2 + 1, p.n, p.workers);
      if (end == worker_row(job - 2, p.n, p.workers)) return;
      group = (end - 1) / T0;  // (T0 > 0 here)
    }
    first = group * T0;
    last = T0 ? min(first + T0, (long long)p.n) : p.n;
    w_lo = row_worker((int)first, p.n, p.workers);
    w_hi = row_worker((int)last - 1, p.n, p.workers) + 1;
    if (!q.by_group && w_lo != job - 2) return;  // it began earlier
    if (w_hi - w_lo == 1) return;                // one worker holds it: already written
    src = p.part_head;
    first_src = p.part_tail + (size_t)w_lo * p.pitch;
  }
  const int col = (blockIdx.x * 32 + threadIdx.x) * 4;
  float4 s = make_float4(0, 0, 0, 0);
  if (col < p.pitch) {
    for (int w = w_lo + threadIdx.y; w < w_hi; w += kRedSlices) {
      const float* row = w == w_lo ? first_src : src + (size_t)w * p.pitch;
      const float4 v = *reinterpret_cast<const float4*>(row + col);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
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
  const float v[4] = {s.x, s.y, s.z, s.w};
  for (int j = 0; j < 4; ++j) {
    if (col + j >= p.d) break;
    if (job == 0) p.dw_post[col + j] = v[j];
    else if (job == 1) p.dw_next[col + j] = v[j];
    else static_cast<T*>(p.dgate)[group * p.gate_stride + col + j] = T(v[j]);
  }
}

// ---- work split of the backward --------------------------------------------
// Threads a worker: 8 elements each up to d = 8192, 16 above. Workers: about
// 1024 threads an SM, and at least two rows each (fewer rows would only add
// partial sums to join).
constexpr int kBwdMinRows = 2;
int bwd_threads(int d) { return ((d <= 8192 ? (d + 7) / 8 : (d + 15) / 16) + 31) / 32 * 32; }
int bwd_workers_per_sm(int d) {
  const int k = 1024 / bwd_threads(d);
  return k < 1 ? 1 : k > 12 ? 12 : k;
}
int bwd_workers(int n, int d) {
  const long long most = (long long)kBlockSms * bwd_workers_per_sm(d);
  const long long want = (n + kBwdMinRows - 1) / kBwdMinRows;
  return (int)(want < most ? want : most);
}
int bwd_pitch(int d) { return (d + 31) / 32 * 32; }

template <typename T, int VEC, int ITEMS, bool STAGED, int MAXT>
cudaError_t run_bwd(const NormBwd& p, int threads, size_t smem, cudaStream_t s) {
  auto kern = norm_bwd_kernel<T, VEC, ITEMS, STAGED, MAXT>;
  if (smem > 0) {
    cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kern, dim3(p.workers), dim3(threads), smem, s, p);
}

template <typename T, int VEC>
cudaError_t launch_bwd(NormBwd& p, bool vec, cudaStream_t s) {
  const int threads = bwd_threads(p.d);
  const size_t row = (size_t)p.d * sizeof(T);
  p.slots = (p.dh ? 2 : 0) + (p.y ? 1 : 0) + (p.dout ? 1 : 0) + (p.gate ? 1 : 0);
  const size_t budget = (size_t)220 * 1024 / bwd_workers_per_sm(p.d) - 1024;
  size_t st = budget / (p.slots * row);
  p.stages = st > 3 ? 3 : (int)st;
  const bool wide = p.d > 8192;
  if (!vec || p.stages < 1) {
    p.stages = 1;
    if (wide) return run_bwd<T, 1, 16, false, 1024>(p, threads, 0, s);
    return run_bwd<T, 1, 8, false, 1024>(p, threads, 0, s);
  }
  const size_t smem = p.stages * p.slots * row;
  if (wide) return run_bwd<T, VEC, 16 / VEC, true, 1024>(p, threads, smem, s);
  if (threads > 512) return run_bwd<T, VEC, 8 / VEC, true, 1024>(p, threads, smem, s);
  return run_bwd<T, VEC, 8 / VEC, true, 512>(p, threads, smem, s);
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

// 16-byte vectors: every row of every operand starts on a 16-byte boundary
bool vectors(const moe_norm_config* c, bool gate, std::initializer_list<const void*> ptrs) {
  const int vec = c->dtype == MOE_BF16 ? 8 : 4;
  if (c->d % vec) return false;
  if (gate && c->gate_stride % vec) return false;
  for (const void* q : ptrs)
    if (!aligned16(q)) return false;
  return true;
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
  const bool vec =
      vectors(c, p.gate != nullptr, {p.x, p.y, p.gate, p.out, p.h, p.w_post, p.w_next});
  cudaError_t e;
  if (c->dtype == MOE_BF16)
    e = vec ? launch_fwd<__nv_bfloat16, 8>(p, s) : launch_fwd<__nv_bfloat16, 1>(p, s);
  else
    e = vec ? launch_fwd<float, 4>(p, s) : launch_fwd<float, 1>(p, s);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t backward_bytes(const moe_norm_config* c) {
  const size_t b = (size_t)4 * bwd_workers(c->n, c->d) * bwd_pitch(c->d) * sizeof(float);
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
  p.workers = bwd_workers(c->n, c->d);
  p.pitch = bwd_pitch(c->d);
  const size_t each = (size_t)p.workers * p.pitch;
  p.part_post = static_cast<float*>(ws);
  p.part_next = p.part_post + each;
  p.part_head = p.part_next + each;
  p.part_tail = p.part_head + each;
  const bool vec = vectors(c, p.gate != nullptr,
                           {p.dout, p.dh, p.out, p.y, p.gate, p.dx, p.dy, p.dgate, p.w_post,
                            p.w_next});
  cudaError_t e = c->dtype == MOE_BF16 ? launch_bwd<__nv_bfloat16, 8>(p, vec, s)
                                       : launch_bwd<float, 4>(p, vec, s);
  if (e != cudaSuccess) return MOE_ERR_CUDA;
  if (p.workers == 1) return MOE_OK;
  NormReduce r{p, 0};
  int jobs = 2;
  if (p.gate && p.gate_tokens != 1) {
    const int groups = gate_rows(c);
    r.by_group = groups <= p.workers;
    jobs += r.by_group ? groups : p.workers;
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
