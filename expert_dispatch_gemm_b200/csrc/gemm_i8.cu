// Grouped products in 8-bit integers on the tensor cores, with a scale for
// each token and each output channel:
//
//   u[r,o] = x_scale[r] w_scale[g,o] sum_j xq[r,j] w[g,o,j]
//   out    = act(u), or silu(u) v (SwiGLU, v from a second weight)
//
// "Expert choice routing" (aicassindra.com), "The math": Expert_e on dense
// per-expert batches. The weights are the M side, as in the bf16 weights-as-M
// products: a group's tokens are the N side of the MMA and need no padding to
// 128 rows, so the same kernel serves one decoded token (where it streams the
// active experts' weights once, half the bytes of bf16) and long prompts. An
// accumulator lane is an output channel and its columns are tokens: the
// channel's scale is a register, the tokens' scales are read from shared
// memory, and the int32 sums (exact: |q| <= 127 and K <= 65,536) become fp32
// once, in the epilogue.
//
// CTA pairs (cta_group::2), tcgen05.mma kind::i8, K = 32 a step. A tile is
// (group, 256 channels, up to 256 of the group's rows): each CTA loads its 128
// channels as A and half of the rows as B by TMA, 128 bytes of K a stage
// (128-byte swizzle); K past the end and rows past the buffers arrive as
// zeros. A step of 32 bytes takes N / 2 cycles of the tensor pipe, as a bf16
// step of 16 elements does, and one thread issues a step in about 95 cycles,
// so two threads issue, on accumulators of their own:
// - i8_pair_kernel: two tile streams, each with its own producer, ring and
//   256-column accumulator; while one stream's epilogue drains, the other
//   keeps the pipe busy.
//     warps 0 / 2 producers, 1 / 3 issuers, 4-19 epilogue (eight a stream)
// - i8_swiglu_pair_kernel: one stream, W1 and W3 rows as two A operands of a
//   stage, u and v into two accumulators that meet in one epilogue thread.
//     warp 0 producer, 1 / 2 issuers, 4-19 epilogue
// On a B200 (8-bit rate: twice the measured bf16 rate, 3.3 POP/s; uniform random
// bytes): k 14336, 1,280 rows a group 3.0 POP/s (91%); SwiGLU, k 4096, 813 to 827 us
// for 10,240 rows and 14,336 units (88 to 89%; its epilogue is not overlapped);
// k 1024, 2,048 rows a group, 262 us for 131,072 rows and 2,048 channels (64%: the
// SMs' path to L2, see the epilogue); 16 rows a group of 32, k 7168, SwiGLU 2048,
// 148 to 154 us (94 to 97% of the HBM rate).
// Every mbarrier wait is bounded; on a timeout a role records the error, its
// copies and MMAs in flight are waited for (bounded), TMEM is freed and the
// kernel returns.
#include <cuda.h>
#include <cuda_bf16.h>
#include <math.h>

#include <atomic>

#include "block_internal.h"
#include "device_common.cuh"
#include "sm100.cuh"

namespace moe {
namespace {

constexpr int kBK = 128;                    // bytes (= elements) of K a stage
constexpr int kStep = 32;                   // K of one MMA
constexpr int kWBytes = 128 * kBK;          // this CTA's 128 channels
constexpr int kXBytes = 128 * kBK;          // up to 128 rows
constexpr int kMaxTok = 256;                // rows of a tile (MMA N)
constexpr int kTokUnit = 32;                // N is a multiple of this (M = 256 pairs)
constexpr int kEpiWarps = 16;
constexpr int kThreads = 32 * (4 + kEpiWarps);
constexpr int kTmemCols = 512;
constexpr uint64_t kWaitNs = 2000000000ull;  // 2 s

constexpr int kStreams = 2, kStagesS = 3, kStageBytesS = kWBytes + kXBytes;  // 3 x 32 KB each
constexpr int kStagesU = 4, kStageBytesU = 2 * kWBytes + kXBytes;            // 4 x 48 KB

enum { A_NONE = MOE_I8_NONE, A_RELU = MOE_I8_RELU, A_GELU = MOE_I8_GELU, A_SWIGLU = MOE_I8_SWIGLU };

struct I8Params {
  const int32_t *starts, *counts;  // NULL: one group of all rows
  const float *x_scale, *w_scale, *w3_scale;
  int groups, rows, K, n_out, mt_tiles;
  int parts;  // of K, in the split kernel
  void* out;
  int* err;
};

struct GroupTable {
  int start[MOE_I8_MAX_GROUPS];
  int count[MOE_I8_MAX_GROUPS];
  int tiles[MOE_I8_MAX_GROUPS + 1];  // tiles of the groups before g
};

struct StreamState {
  uint64_t full[kStreams][kStagesS];
  uint64_t empty[kStreams][kStagesS];
  uint64_t tfull[kStreams];
  uint64_t tempty[kStreams];
  uint64_t drain[kStreams];
  uint32_t tmem_base;
  volatile int abort_flag;
  GroupTable g;
};

struct UpState {
  uint64_t full[kStagesU];
  uint64_t empty[kStagesU];  // released by both issuers' commits
  uint64_t tfull;            // both issuers' last commits of a tile
  uint64_t tempty;           // both CTAs' epilogues
  uint64_t drain[2];
  uint32_t tmem_base;
  volatile int abort_flag;
  GroupTable g;
};

template <bool CLUSTER, class State>
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, State* st, int* err,
                                     int code) {
  auto probe = [&]() {
    return CLUSTER ? sm100::mbar_try_wait_cluster(bar, parity) : sm100::mbar_try_wait(bar, parity);
  };
  // the clock is read from the 64th probe on: reading it takes longer than
  // most waits have left
  uint64_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (probe()) return true;
    if ((it & 63u) == 0) {
      if (st->abort_flag) return false;
      const uint64_t now = global_timer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > kWaitNs) {
        st->abort_flag = 1;
        report_error(err, code);
        return false;
      }
    }
  }
}

// wait (bounded) for the copies of the last `pending` stages before `stage`
template <int STAGES>
__device__ __forceinline__ void settle(uint64_t* full, int stage, uint32_t phase, int pending) {
  for (int i = 0; i < pending; ++i) {
    if (--stage < 0) {
      stage = STAGES - 1;
      phase ^= 1u;
    }
    const uint64_t t0 = global_timer_ns();
    while (!sm100::mbar_try_wait(&full[stage], phase) && global_timer_ns() - t0 < kWaitNs) {
    }
  }
}

// Groups into shared memory, cut to the rows that the buffers have.
__device__ __forceinline__ void load_groups(GroupTable& g, const I8Params& p, int tid) {
  for (int i = tid; i < p.groups; i += kThreads) {
    const int s = p.starts ? p.starts[i] : 0;
    const int c = p.starts ? p.counts[i] : p.rows;
    const int room = s < 0 || s > p.rows ? 0 : p.rows - s;
    if (s < 0 || c < 0 || c > room) bad_index(p.err, kSiteI8Groups);
    g.start[i] = s;
    g.count[i] = max(0, min(c, room));
  }
  __syncthreads();
  if (tid < 32) {  // running sum of the tiles, 32 groups at a time
    int run = 0;
    for (int g0 = 0; g0 < p.groups; g0 += 32) {
      const int i = g0 + tid;
      int v = i < p.groups ? (g.count[i] + kMaxTok - 1) / kMaxTok * p.mt_tiles : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(~0u, v, o);
        if (tid >= o) v += u;
      }
      if (i < p.groups) g.tiles[i + 1] = run + v;
      run += __shfl_sync(~0u, v, 31);
    }
    if (tid == 0) g.tiles[0] = 0;
  }
}

struct Tile {
  int group, m0;  // first channel of the pair within the group
  int row;        // first row
  int valid;      // rows
  int n;          // MMA N: valid rounded up to kTokUnit
};

// Tile order: group by group, 256 channels by 256, the rows' chunks innermost
// (pairs that run together share a weight tile). A group's rows are split
// into ceil(count / 256) chunks of 32-row units, equal to a unit.
__device__ __forceinline__ Tile decode(int tile, const I8Params& p, const GroupTable& g) {
  int lo = 0, hi = p.groups - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (g.tiles[mid] <= tile) lo = mid; else hi = mid - 1;
  }
  Tile t;
  const int count = g.count[lo];
  const int chunks = max((count + kMaxTok - 1) / kMaxTok, 1);
  const int local = tile - g.tiles[lo];
  const int chunk = local % chunks;
  const int units = (count + kTokUnit - 1) / kTokUnit;
  const int each = units / chunks, more = units % chunks;  // the first `more` have one more
  const int first = (chunk * each + min(chunk, more)) * kTokUnit;
  const int last = min(first + (each + (chunk < more)) * kTokUnit, count);
  t.group = lo;
  t.m0 = local / chunks * 256;
  t.row = g.start[lo] + first;
  t.valid = last - first;
  t.n = (t.valid + kTokUnit - 1) / kTokUnit * kTokUnit;
  return t;
}

// A CTA's rows of the tile (N / 2, a multiple of 16): boxes of 64 and 16 rows at
// 1 KB-aligned offsets, whole 8-row atoms of the swizzle. (Each more box size
// would be one more tensor map for the host to encode a call.)
constexpr int kBoxes = 2;
struct RowMaps {
  CUtensorMap m[kBoxes];  // boxes of 16 and 64 rows
};
__device__ __forceinline__ void load_rows(unsigned char* dst, const RowMaps& x, uint32_t bar,
                                          int k, int row, int rows) {
  int off = 0;
  for (; off + 64 <= rows; off += 64)
    sm100::tma_load_2d_pair(dst + off * kBK, &x.m[1], bar, k, row + off);
  for (; off < rows; off += 16)
    sm100::tma_load_2d_pair(dst + off * kBK, &x.m[0], bar, k, row + off);
}

template <int ACT>
__device__ __forceinline__ float activate(float v) {
  if (ACT == A_RELU) return v < 0.0f ? 0.0f : v;
  if (ACT == A_GELU) return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
  return v;
}
// silu(u) v with e = exp(-|u|): u / (1 + e), times e where u < 0. exp(-u) would
// pass fp32's range at u = -88.7, where the value is 1e-37 v, and from -87.3 on the
// fast division by it gives zero. (131,072 rows, k 1024, 1,024 units: 270 us, with
// exp(-u) 266.)
// (bf16 outputs take the fast exponential and division: their errors, a few fp32
// steps, are far below the output's; the exact division alone took as long as
// the rest of the epilogue)
template <typename OUT>
__device__ __forceinline__ float silu_times(float u, float v) {
  const float e = sizeof(OUT) == 2 ? __expf(-fabsf(u)) : expf(-fabsf(u));
  const float n = u < 0.0f ? u * e : u;
  return (sizeof(OUT) == 2 ? __fdividef(n, 1.0f + e) : n * __frcp_rn(1.0f + e)) * v;
}

// Epilogue of bf16 outputs. A lane of the accumulator is a channel, a row of
// the output is a column of it, so a tile has to be transposed on its way out.
// The accumulator is read as MMA fragments (two neighbouring rows of a channel
// in a thread): they are scaled as pairs, converted as pairs and stored as 8 x
// 8 blocks, transposed by stmatrix, into the warp's staging buffer of 16 rows x
// 32 channels, which leaves as one TMA store (rows past the group's last: as
// 16-byte stores of the others). Two warps take turns at the 32-row groups of
// each TMEM lane quadrant. The buffer is laid out in the 64-byte swizzle,
// in which the eight 16-byte pieces of a block lie in different banks. (k 1024,
// 131,072 rows, 2,048 channels: 267 us; with 16-byte stores instead of the TMA's
// 292, without any store 222, without an epilogue 184.)
struct Staging {
  unsigned char v[16 * 64];  // [16 rows][32 channels] bf16, swizzled
};
struct Scales {
  float x[kMaxTok / 2];  // of the rows of a tile that the warp takes: 32 of 64
};
__device__ __forceinline__ uint32_t swizzled(int row, int piece) {
  return row * 64 + ((piece ^ ((row >> 1) & 3)) << 4);
}

// Sums times the channel's scale, then the rows': the scales' own product may
// leave fp32's range where the result does not.
__device__ __forceinline__ float2 scaled(uint32_t a, uint32_t b, float2 xs, float ws) {
  return __fmul2_rn(
      __fmul2_rn(make_float2((float)(int)a, (float)(int)b), make_float2(ws, ws)), xs);
}
__device__ __forceinline__ float scaled(uint32_t a, float xs, float ws) {
  return (float)(int)a * ws * xs;
}

// The 8 x 8 blocks r[j][k] (rows 8 j .., channels 8 k ..) of rows cc .. cc + 15 of
// the tile to the output, through the staging buffer.
__device__ __forceinline__ void write_rows(Staging* s, const CUtensorMap* to, const I8Params& p,
                                           const Tile& t, int cc, int col0, int lane,
                                           const uint32_t (&r)[2][4]) {
  if (lane == 0) sm100::bulk_wait_read_all();  // the last store has read the buffer
  __syncwarp();
  const uint32_t at = sm100::smem_addr(s->v) + swizzled(lane & 7, lane >> 3);
#pragma unroll
  for (int j = 0; j < 2; ++j) sm100::stmatrix_x4_trans(at + j * 512, r[j]);
  if (cc + 16 <= t.valid) {
    sm100::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0 && col0 < p.n_out) {
      sm100::tma_store_2d(to, col0, t.row + cc, s->v);
      sm100::bulk_commit_group();
    }
  } else {
    __syncwarp();
    __nv_bfloat16* out =
        static_cast<__nv_bfloat16*>(p.out) + (size_t)(t.row + cc) * p.n_out + col0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int i = k * 8 + (lane >> 2), c = lane & 3;
      const uint4 v = *reinterpret_cast<const uint4*>(s->v + swizzled(i, c));
      if (cc + i < t.valid && col0 + c * 8 < p.n_out)
        *reinterpret_cast<uint4*>(out + (size_t)i * p.n_out + c * 8) = v;
    }
  }
}

// the scales of the tile's rows 64 k + 32 half + [0, 32), before the tile is there
__device__ __forceinline__ void stage_scales(Scales* s, const I8Params& p, const Tile& t,
                                             int half, int lane) {
  __syncwarp();
#pragma unroll
  for (int k = 0; k < kMaxTok / 64; ++k) {
    const int j = 64 * k + 32 * half + lane;
    if (64 * k < t.n) s->x[32 * k + lane] = j < t.valid ? p.x_scale[t.row + j] : 0.0f;
  }
  __syncwarp();
}
__device__ __forceinline__ const float* scales_at(const Scales* s, int cc) {
  return s->x + (cc >> 6) * 32 + (cc & 31);  // of row cc of the tile
}

// the scales of a thread's channels lane / 4 + 8 k of the warp's 32 from col0 on
__device__ __forceinline__ void channel_scales(float (&ws)[4], const float* scale,
                                               const I8Params& p, const Tile& t, int col0,
                                               int lane) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int c = col0 + (lane >> 2) + 8 * k;
    ws[k] = c < p.n_out ? scale[(size_t)t.group * p.n_out + c] : 0.0f;
  }
}

// 16 rows x 32 channels of the tile from the accumulator's fragments `lo`
// (lanes 0-15 of the quadrant) and `hi` (16-31)
template <int ACT>
__device__ __forceinline__ void finish(uint32_t (&r)[2][4], const uint32_t (&lo)[8],
                                       const uint32_t (&hi)[8], const float* xs,
                                       const float (&ws)[4], int lane) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float2 x = *reinterpret_cast<const float2*>(xs + 8 * j + 2 * (lane & 3));
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t* v = (k < 2 ? lo : hi) + 4 * j + 2 * (k & 1);
      const float2 u = scaled(v[0], v[1], x, ws[k]);
      r[j][k] = pack_bf16x2(activate<ACT>(u.x), activate<ACT>(u.y));
    }
  }
}
__device__ __forceinline__ void finish_gated(uint32_t (&r)[2][4], const uint32_t (&ulo)[8],
                                             const uint32_t (&uhi)[8], const uint32_t (&vlo)[8],
                                             const uint32_t (&vhi)[8], const float* xs,
                                             const float (&ws1)[4], const float (&ws3)[4],
                                             int lane) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float2 x = *reinterpret_cast<const float2*>(xs + 8 * j + 2 * (lane & 3));
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int at = 4 * j + 2 * (k & 1);
      const uint32_t *uu = (k < 2 ? ulo : uhi) + at, *vv = (k < 2 ? vlo : vhi) + at;
      const float2 u = scaled(uu[0], uu[1], x, ws1[k]);
      const float2 v = scaled(vv[0], vv[1], x, ws3[k]);
      r[j][k] = pack_bf16x2(silu_times<__nv_bfloat16>(u.x, v.x),
                            silu_times<__nv_bfloat16>(u.y, v.y));
    }
  }
}

// fp32 outputs: a lane keeps its channel, and the warp writes the 128
// consecutive bytes of a row's 32 channels: value(i, x_scale of row i)
template <int ROWS, class F>
__device__ __forceinline__ void emit_f32(const Scales* s, const I8Params& p, const Tile& t,
                                         int cc, int col0, int lane, const F& value) {
  float* out = static_cast<float*>(p.out) + (size_t)(t.row + cc) * p.n_out + col0;
  const bool real = col0 + lane < p.n_out;
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const float r = value(i, scales_at(s, cc)[i]);
    if (real && cc + i < t.valid) out[(size_t)i * p.n_out + lane] = r;
  }
}

template <typename OUT, int ACT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    i8_pair_kernel(const __grid_constant__ RowMaps tx, const __grid_constant__ CUtensorMap tw,
                   const __grid_constant__ CUtensorMap to, const I8Params p) {
  extern __shared__ __align__(1024) unsigned char ism[];
  unsigned char* base = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(ism) + 1023) & ~uintptr_t(1023));
  constexpr int kRing = kStreams * kStagesS * kStageBytesS;
  Staging* staging = reinterpret_cast<Staging*>(base + kRing);
  Scales* scales = reinterpret_cast<Scales*>(staging + kEpiWarps);
  StreamState* st = reinterpret_cast<StreamState*>(scales + kEpiWarps);
  auto sW = [&](int sx, int j) { return base + (sx * kStagesS + j) * kStageBytesS; };
  auto sX = [&](int sx, int j) { return sW(sx, j) + kWBytes; };

  const uint32_t rank = sm100::cluster_ctarank();
  const bool leader = rank == 0;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int sx = 0; sx < kStreams; ++sx) {
      for (int j = 0; j < kStagesS; ++j) {
        sm100::mbar_init(&st->full[sx][j], 1);
        sm100::mbar_init(&st->empty[sx][j], 1);
      }
      sm100::mbar_init(&st->tfull[sx], 1);
      sm100::mbar_init(&st->tempty[sx], 2 * 32 * (kEpiWarps / kStreams));
      sm100::mbar_init(&st->drain[sx], 1);
    }
    st->abort_flag = 0;
    sm100::fence_mbar_init();
  }
  if (warp == 0 && lane < kBoxes) sm100::tma_prefetch_desc(&tx.m[lane]);
  if (warp == 0 && lane == kBoxes) sm100::tma_prefetch_desc(&tw);
  if (warp == 1) {
    sm100::tmem_alloc_pair(&st->tmem_base, kTmemCols);
    sm100::tmem_relinquish_pair();
  }
  pdl_wait();
  load_groups(st->g, p, tid);
  sm100::tc_fence_before();
  __syncthreads();
  sm100::cluster_sync();  // both CTAs' barriers exist before any remote arrive
  sm100::tc_fence_after();
  const uint32_t tmem = st->tmem_base;

  const int total = st->g.tiles[p.groups];
  const int KB = (p.K + kBK - 1) / kBK;
  const int pair_id = blockIdx.x >> 1, num_pairs = gridDim.x >> 1;
  // the pair's tiles are pair_id + i * num_pairs; stream sx takes i = sx, sx + 2, ...
  const int sx = warp < 4 ? (warp >> 1) : (warp - 4) / (kEpiWarps / kStreams);
  const int first = pair_id + sx * num_pairs, step = kStreams * num_pairs;

  if (warp < 4 && (warp & 1) == 0) {
    if (lane == 0) {  // producer of stream sx
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = first; ok && tile < total; tile += step) {
        const Tile t = decode(tile, p, st->g);
        const int half = t.n / 2;
        const uint32_t bytes = kWBytes + (uint32_t)half * kBK;
        const int wrow = t.group * p.n_out + t.m0 + (int)rank * 128;
        const int xrow = t.row + (int)rank * half;
        for (int kb = 0; kb < KB; ++kb) {
          if (!wait<false>(&st->empty[sx][stage], phase ^ 1u, st, p.err, kErrGemmTimeout | 0x61)) {
            ok = false;
            break;
          }
          const uint32_t fl = sm100::mapa_shared(sm100::smem_addr(&st->full[sx][stage]), 0);
          if (leader) sm100::mbar_arrive_expect_tx(&st->full[sx][stage], 2 * bytes);
          sm100::tma_load_2d_pair(sW(sx, stage), &tw, fl, kb * kBK, wrow);
          load_rows(sX(sx, stage), tx, fl, kb * kBK, xrow, half);
          ++issued;
          if (++stage == kStagesS) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok && leader) settle<kStagesS>(st->full[sx], stage, phase, min(issued, kStagesS));
    }
  } else if (warp < 4) {
    if (lane == 0 && leader) {  // issuer of stream sx
      int stage = 0, local = 0;
      uint32_t phase = 0;
      bool ok = true;
      const uint32_t d_tmem = tmem + (uint32_t)(sx * 256);
      for (int tile = first; ok && tile < total; tile += step, ++local) {
        const Tile t = decode(tile, p, st->g);
        if (!wait<true>(&st->tempty[sx], ((uint32_t)local & 1u) ^ 1u, st, p.err,
                        kErrGemmTimeout | 0x62)) {
          ok = false;
          break;
        }
        sm100::tc_fence_after();
        const uint32_t idesc = sm100::idesc_i8_s32(256, t.n);
        for (int kb = 0; kb < KB; ++kb) {
          if (!wait<false>(&st->full[sx][stage], phase, st, p.err, kErrGemmTimeout | 0x63)) {
            ok = false;
            break;
          }
          sm100::tc_fence_after();
          const uint64_t da = sm100::sw128_kmajor_desc(sm100::smem_addr(sW(sx, stage)));
          const uint64_t db = sm100::sw128_kmajor_desc(sm100::smem_addr(sX(sx, stage)));
#pragma unroll
          for (int k = 0; k < kBK / kStep; ++k)
            sm100::umma_i8_pair(d_tmem, da + 2 * k, db + 2 * k, idesc, (kb | k) != 0);
          sm100::umma_commit_pair_mc(&st->empty[sx][stage], 0x3);
          if (++stage == kStagesS) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        sm100::umma_commit_pair_mc(&st->tfull[sx], 0x3);
      }
      sm100::umma_commit_pair_mc(&st->drain[sx], 0x1);
      const uint64_t t0 = global_timer_ns();
      while (!sm100::mbar_try_wait(&st->drain[sx], 0) && global_timer_ns() - t0 < kWaitNs) {
      }
    }
  } else {
    // epilogue of stream sx: warps q = warp % 4 own lanes (channels) 32q..32q+31,
    // two of them for alternate 32-row groups of the tile
    const int q = warp & 3, half = ((warp - 4) >> 2) & 1;
    Staging* stg = staging + (warp - 4);
    Scales* xsc = scales + (warp - 4);
    int local = 0;
    for (int tile = first; tile < total; tile += step, ++local) {
      const Tile t = decode(tile, p, st->g);
      const int col0 = t.m0 + (int)rank * 128 + 32 * q;
      float ws[4];
      if constexpr (sizeof(OUT) == 2) {
        channel_scales(ws, p.w_scale, p, t, col0, lane);
      } else {
        ws[0] = col0 + lane < p.n_out ? p.w_scale[(size_t)t.group * p.n_out + col0 + lane] : 0.0f;
      }
      stage_scales(xsc, p, t, half, lane);
      if (!wait<true>(&st->tfull[sx], (uint32_t)local & 1u, st, p.err, kErrGemmTimeout | 0x64))
        break;
      sm100::tc_fence_after();
      const uint32_t tbase = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(sx * 256);
      if constexpr (sizeof(OUT) == 2) {
        // the next 16 rows are on their way from TMEM while these are written
        uint32_t lo[2][8], hi[2][8], r[2][4];
        auto fetch = [&](int b, int cc) {
          sm100::tmem_ld_16x256b_x2(tbase + cc, lo[b]);
          sm100::tmem_ld_16x256b_x2(tbase + (16u << 16) + cc, hi[b]);
        };
        auto give = [&](int b, int cc) {
          finish<ACT>(r, lo[b], hi[b], scales_at(xsc, cc), ws, lane);
          write_rows(stg, &to, p, t, cc, col0, lane, r);
        };
        if (32 * half < t.valid) fetch(0, 32 * half);
#pragma unroll 1
        for (int cc = 32 * half; cc < t.valid; cc += 64) {
          sm100::tmem_ld_wait();
          const bool more = cc + 16 < t.valid;
          if (more) fetch(1, cc + 16);
          give(0, cc);
          if (!more) break;
          sm100::tmem_ld_wait();
          if (cc + 64 < t.valid) fetch(0, cc + 64);
          give(1, cc + 16);
        }
      } else {
#pragma unroll 1
        for (int cc = 32 * half; cc < t.valid; cc += 64) {
          uint32_t v[32];
          sm100::tmem_ld_32x32b_x32(tbase + cc, v);
          sm100::tmem_ld_wait();
          emit_f32<32>(xsc, p, t, cc, col0, lane, [&](int i, float xs) {
            return activate<ACT>(scaled(v[i], xs, ws[0]));
          });
        }
      }
      sm100::tc_fence_before();
      sm100::mbar_arrive_cluster(sm100::mapa_shared(sm100::smem_addr(&st->tempty[sx]), 0));
    }
    if (lane == 0) sm100::bulk_wait_read_all();
  }
  sm100::tc_fence_before();
  __syncthreads();
  sm100::cluster_sync();  // no CTA leaves while its peer may still signal it
  if (warp == 1) {
    sm100::tc_fence_after();
    sm100::tmem_dealloc_pair(tmem, kTmemCols);
  }
}

template <typename OUT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    i8_swiglu_pair_kernel(const __grid_constant__ RowMaps tx,
                          const __grid_constant__ CUtensorMap tw,
                          const __grid_constant__ CUtensorMap tw3,
                          const __grid_constant__ CUtensorMap to, const I8Params p) {
  extern __shared__ __align__(1024) unsigned char ism[];
  unsigned char* base = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(ism) + 1023) & ~uintptr_t(1023));
  constexpr int kRing = kStagesU * kStageBytesU;
  Staging* staging = reinterpret_cast<Staging*>(base + kRing);
  Scales* scales = reinterpret_cast<Scales*>(staging + kEpiWarps);
  UpState* st = reinterpret_cast<UpState*>(scales + kEpiWarps);
  auto sW = [&](int j, int which) { return base + j * kStageBytesU + which * kWBytes; };
  auto sX = [&](int j) { return base + j * kStageBytesU + 2 * kWBytes; };

  const uint32_t rank = sm100::cluster_ctarank();
  const bool leader = rank == 0;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int j = 0; j < kStagesU; ++j) {
      sm100::mbar_init(&st->full[j], 1);
      sm100::mbar_init(&st->empty[j], 2);
    }
    sm100::mbar_init(&st->tfull, 2);
    sm100::mbar_init(&st->tempty, 2 * 32 * kEpiWarps);
    sm100::mbar_init(&st->drain[0], 1);
    sm100::mbar_init(&st->drain[1], 1);
    st->abort_flag = 0;
    sm100::fence_mbar_init();
  }
  if (warp == 0 && lane < kBoxes) sm100::tma_prefetch_desc(&tx.m[lane]);
  if (warp == 0 && lane == kBoxes) sm100::tma_prefetch_desc(&tw);
  if (warp == 0 && lane == kBoxes + 1) sm100::tma_prefetch_desc(&tw3);
  if (warp == 1) {
    sm100::tmem_alloc_pair(&st->tmem_base, kTmemCols);
    sm100::tmem_relinquish_pair();
  }
  pdl_wait();
  load_groups(st->g, p, tid);
  sm100::tc_fence_before();
  __syncthreads();
  sm100::cluster_sync();
  sm100::tc_fence_after();
  const uint32_t tmem = st->tmem_base;

  const int total = st->g.tiles[p.groups];
  const int KB = (p.K + kBK - 1) / kBK;
  const int pair_id = blockIdx.x >> 1, num_pairs = gridDim.x >> 1;

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = pair_id; ok && tile < total; tile += num_pairs) {
        const Tile t = decode(tile, p, st->g);
        const int half = t.n / 2;
        const uint32_t bytes = 2 * kWBytes + (uint32_t)half * kBK;
        const int wrow = t.group * p.n_out + t.m0 + (int)rank * 128;
        const int xrow = t.row + (int)rank * half;
        for (int kb = 0; kb < KB; ++kb) {
          if (!wait<false>(&st->empty[stage], phase ^ 1u, st, p.err, kErrGemmTimeout | 0x71)) {
            ok = false;
            break;
          }
          const uint32_t fl = sm100::mapa_shared(sm100::smem_addr(&st->full[stage]), 0);
          if (leader) sm100::mbar_arrive_expect_tx(&st->full[stage], 2 * bytes);
          sm100::tma_load_2d_pair(sW(stage, 0), &tw, fl, kb * kBK, wrow);
          sm100::tma_load_2d_pair(sW(stage, 1), &tw3, fl, kb * kBK, wrow);
          load_rows(sX(stage), tx, fl, kb * kBK, xrow, half);
          ++issued;
          if (++stage == kStagesU) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok && leader) settle<kStagesU>(st->full, stage, phase, min(issued, kStagesU));
    }
  } else if (warp == 1 || warp == 2) {
    // issuer `which`: W1 products into columns [0, 256), W3's into [256, 512)
    if (lane == 0 && leader) {
      const int which = warp - 1;
      const uint32_t d_tmem = tmem + (uint32_t)(which * 256);
      int stage = 0, local = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = pair_id; ok && tile < total; tile += num_pairs, ++local) {
        const Tile t = decode(tile, p, st->g);
        if (!wait<true>(&st->tempty, ((uint32_t)local & 1u) ^ 1u, st, p.err,
                        kErrGemmTimeout | 0x72)) {
          ok = false;
          break;
        }
        sm100::tc_fence_after();
        const uint32_t idesc = sm100::idesc_i8_s32(256, t.n);
        for (int kb = 0; kb < KB; ++kb) {
          if (!wait<false>(&st->full[stage], phase, st, p.err, kErrGemmTimeout | 0x73)) {
            ok = false;
            break;
          }
          sm100::tc_fence_after();
          const uint64_t da = sm100::sw128_kmajor_desc(sm100::smem_addr(sW(stage, which)));
          const uint64_t db = sm100::sw128_kmajor_desc(sm100::smem_addr(sX(stage)));
#pragma unroll
          for (int k = 0; k < kBK / kStep; ++k)
            sm100::umma_i8_pair(d_tmem, da + 2 * k, db + 2 * k, idesc, (kb | k) != 0);
          sm100::umma_commit_pair_mc(&st->empty[stage], 0x3);
          if (++stage == kStagesU) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        sm100::umma_commit_pair_mc(&st->tfull, 0x3);
      }
      sm100::umma_commit_pair_mc(&st->drain[which], 0x1);
      const uint64_t t0 = global_timer_ns();
      while (!sm100::mbar_try_wait(&st->drain[which], 0) && global_timer_ns() - t0 < kWaitNs) {
      }
    }
  } else if (warp >= 4) {
    // epilogue: warps q = warp % 4 own lanes 32q..32q+31, four of them: two for
    // alternate 32-row groups, and of each group two for 16 rows each; u in columns
    // [0, 256), v in [256, 512)
    const int q = warp & 3;
    const int half = ((warp - 4) >> 2) & 1, sub = (warp - 4) >> 3;
    Staging* stg = staging + (warp - 4);
    Scales* xsc = scales + (warp - 4);
    int local = 0;
    for (int tile = pair_id; tile < total; tile += num_pairs, ++local) {
      const Tile t = decode(tile, p, st->g);
      const int col0 = t.m0 + (int)rank * 128 + 32 * q;
      float ws1[4], ws3[4];
      if constexpr (sizeof(OUT) == 2) {
        channel_scales(ws1, p.w_scale, p, t, col0, lane);
        channel_scales(ws3, p.w3_scale, p, t, col0, lane);
      } else {
        const bool real = col0 + lane < p.n_out;  // (a tile may pass the last channel)
        const size_t wi = (size_t)t.group * p.n_out + col0 + lane;
        ws1[0] = real ? p.w_scale[wi] : 0.0f;
        ws3[0] = real ? p.w3_scale[wi] : 0.0f;
      }
      stage_scales(xsc, p, t, half, lane);
      if (!wait<true>(&st->tfull, (uint32_t)local & 1u, st, p.err, kErrGemmTimeout | 0x74)) break;
      sm100::tc_fence_after();
      const uint32_t tbase = tmem + ((uint32_t)(q * 32) << 16);
#pragma unroll 1
      for (int cc = 32 * half; cc + 16 * sub < t.valid; cc += 64) {
        if constexpr (sizeof(OUT) == 2) {
          uint32_t ulo[8], uhi[8], vlo[8], vhi[8], r[2][4];
          const int at = cc + 16 * sub;
          const uint32_t c = tbase + at;
          sm100::tmem_ld_16x256b_x2(c, ulo);
          sm100::tmem_ld_16x256b_x2(c + (16u << 16), uhi);
          sm100::tmem_ld_16x256b_x2(c + 256u, vlo);
          sm100::tmem_ld_16x256b_x2(c + 256u + (16u << 16), vhi);
          sm100::tmem_ld_wait();
          finish_gated(r, ulo, uhi, vlo, vhi, scales_at(xsc, at), ws1, ws3, lane);
          write_rows(stg, &to, p, t, at, col0, lane, r);
        } else {
          uint32_t u[16], v[16];
          const int at = cc + 16 * sub;
          sm100::tmem_ld_32x32b_x16(tbase + at, u);
          sm100::tmem_ld_32x32b_x16(tbase + 256u + at, v);
          sm100::tmem_ld_wait();
          emit_f32<16>(xsc, p, t, at, col0, lane, [&](int i, float xs) {
            return silu_times<OUT>(scaled(u[i], xs, ws1[0]), scaled(v[i], xs, ws3[0]));
          });
        }
      }
      sm100::tc_fence_before();
      sm100::mbar_arrive_cluster(sm100::mapa_shared(sm100::smem_addr(&st->tempty), 0));
    }
    if (lane == 0) sm100::bulk_wait_read_all();
  }
  sm100::tc_fence_before();
  __syncthreads();
  sm100::cluster_sync();
  if (warp == 1) {
    sm100::tc_fence_after();
    sm100::tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// Few tiles (one decoded token, a small expert): the reduction split over the
// pairs of a cluster, so that the weights stream through more SMs. One tile a
// cluster; pair i of S takes K blocks [KB i / S, KB (i + 1) / S), with the whole
// shared memory as its ring. The int32 sums are exact, so any split gives the
// same result: the tile's 32-row chunks are dealt out to the pairs, each CTA
// sends its sums of the others' chunks into their rings (free by then) through
// distributed shared memory, adds what it received to its own, and writes. One
// row, weights from HBM: k 2048, 7,168 channels (28 tiles, 2 parts) 9.3 us, unsplit
// 10.7; k 7168, 2,048 channels (8 tiles, 4 parts) 11.7 us, unsplit 25.3. The
// smallest product of all takes 5.6. (The tiles are the host's bound from the rows of
// the buffers. A layer's buffers have room for 127 rows of padding an expert, which
// keeps its products above the limit; calls with one or a few groups come here.)
// ---------------------------------------------------------------------------
constexpr int kSplitRing = 192 * 1024;
constexpr int kSplitStages = 6;  // of 32 KB; SwiGLU 4 of 48 KB
struct SplitState {
  uint64_t full[kSplitStages];
  uint64_t empty[kSplitStages];
  uint64_t tfull;
  uint64_t drain[2];
  uint32_t tmem_base;
  volatile int abort_flag;
  GroupTable g;
};

__device__ __forceinline__ void send16(uint32_t to, const uint32_t* v) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3])
               : "memory");
}

template <typename OUT, int ACT>
__global__ void __launch_bounds__(kThreads, 1)
    i8_split_kernel(const __grid_constant__ RowMaps tx, const __grid_constant__ CUtensorMap tw,
                    const __grid_constant__ CUtensorMap tw3,
                    const __grid_constant__ CUtensorMap to, const I8Params p) {
  constexpr int SIDES = ACT == A_SWIGLU ? 2 : 1;
  constexpr int STAGE = SIDES * kWBytes + kXBytes, STAGES = kSplitRing / STAGE;
  constexpr int UNIT = 16 * 32 * 4;  // bytes of a warp's 16 rows x 32 channels of sums
  extern __shared__ __align__(1024) unsigned char ism[];
  unsigned char* base = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(ism) + 1023) & ~uintptr_t(1023));
  Staging* staging = reinterpret_cast<Staging*>(base + kSplitRing);
  Scales* scales = reinterpret_cast<Scales*>(staging + kEpiWarps);
  SplitState* st = reinterpret_cast<SplitState*>(scales + kEpiWarps);
  auto sW = [&](int j, int side) { return base + j * STAGE + side * kWBytes; };
  auto sX = [&](int j) { return base + j * STAGE + SIDES * kWBytes; };

  const uint32_t cta = sm100::cluster_ctarank();
  const uint32_t rank = cta & 1, lead = cta & ~1u;
  const bool leader = rank == 0;
  const uint16_t pair_mask = (uint16_t)(0x3u << lead);
  const int part = (int)(cta >> 1), parts = p.parts;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int j = 0; j < STAGES; ++j) {
      sm100::mbar_init(&st->full[j], 1);
      sm100::mbar_init(&st->empty[j], SIDES);
    }
    sm100::mbar_init(&st->tfull, SIDES);
    sm100::mbar_init(&st->drain[0], 1);
    sm100::mbar_init(&st->drain[1], 1);
    st->abort_flag = 0;
    sm100::fence_mbar_init();
  }
  if (warp == 0 && lane < kBoxes) sm100::tma_prefetch_desc(&tx.m[lane]);
  if (warp == 0 && lane == kBoxes) sm100::tma_prefetch_desc(&tw);
  if (SIDES == 2 && warp == 0 && lane == kBoxes + 1) sm100::tma_prefetch_desc(&tw3);
  if (warp == 1) {
    sm100::tmem_alloc_pair(&st->tmem_base, SIDES * 256);
    sm100::tmem_relinquish_pair();
  }
  const int tile = blockIdx.x / (2 * parts);
  const int all = (p.K + kBK - 1) / kBK;
  const int from = all * part / parts, end = all * (part + 1) / parts;
  // One group and one chunk of rows: the tile's weights are known before the
  // previous kernel is done, and start on their way to L2 (where what that
  // kernel may still write to them would arrive too).
  if (p.groups == 1 && p.rows <= kMaxTok && warp == 3) {
    for (int kb = from + lane; kb < end; kb += 32) {
      sm100::tma_prefetch_2d(&tw, kb * kBK, tile * 256 + (int)rank * 128);
      if (SIDES == 2) sm100::tma_prefetch_2d(&tw3, kb * kBK, tile * 256 + (int)rank * 128);
    }
  }
  pdl_wait();
  load_groups(st->g, p, tid);
  sm100::tc_fence_before();
  __syncthreads();
  sm100::cluster_sync();
  sm100::tc_fence_after();
  const uint32_t tmem = st->tmem_base;

  const bool live = tile < st->g.tiles[p.groups];  // (the same in the whole cluster)
  const Tile t = live ? decode(tile, p, st->g) : Tile{0, 0, 0, 0, 0};
  const int kb0 = from, kb1 = live ? end : from;
  // epilogue warps: quadrant q; units of 16 rows, unit u = 2 chunk + half, by warp set
  const int q = warp & 3, set = (warp - 4) >> 2;
  const int units = (t.valid + 15) / 16;
  const int col0 = t.m0 + (int)rank * 128 + 32 * q;
  Scales* xsc = scales + (warp - 4);
  float ws1[4], ws3[4];

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      const int half = t.n / 2;
      const uint32_t bytes = SIDES * kWBytes + (uint32_t)half * kBK;
      const int wrow = t.group * p.n_out + t.m0 + (int)rank * 128;
      const int xrow = t.row + (int)rank * half;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!wait<false>(&st->empty[stage], phase ^ 1u, st, p.err, kErrGemmTimeout | 0x81)) {
          ok = false;
          break;
        }
        const uint32_t fl = sm100::mapa_shared(sm100::smem_addr(&st->full[stage]), lead);
        if (leader) sm100::mbar_arrive_expect_tx(&st->full[stage], 2 * bytes);
        sm100::tma_load_2d_pair(sW(stage, 0), &tw, fl, kb * kBK, wrow);
        if (SIDES == 2) sm100::tma_load_2d_pair(sW(stage, 1), &tw3, fl, kb * kBK, wrow);
        load_rows(sX(stage), tx, fl, kb * kBK, xrow, half);
        ++issued;
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok && leader) settle<STAGES>(st->full, stage, phase, min(issued, STAGES));
    }
  } else if (warp == 1 || (SIDES == 2 && warp == 2)) {
    if (lane == 0 && leader && live) {
      const int side = warp - 1;
      const uint32_t d_tmem = tmem + (uint32_t)(side * 256);
      const uint32_t idesc = sm100::idesc_i8_s32(256, t.n);
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!wait<false>(&st->full[stage], phase, st, p.err, kErrGemmTimeout | 0x83)) {
          ok = false;
          break;
        }
        sm100::tc_fence_after();
        const uint64_t da = sm100::sw128_kmajor_desc(sm100::smem_addr(sW(stage, side)));
        const uint64_t db = sm100::sw128_kmajor_desc(sm100::smem_addr(sX(stage)));
#pragma unroll
        for (int k = 0; k < kBK / kStep; ++k)
          sm100::umma_i8_pair(d_tmem, da + 2 * k, db + 2 * k, idesc, kb != kb0 || k != 0);
        sm100::umma_commit_pair_mc(&st->empty[stage], pair_mask);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (ok) sm100::umma_commit_pair_mc(&st->tfull, pair_mask);
      sm100::umma_commit_pair_mc(&st->drain[side], (uint16_t)(1u << cta));
      const uint64_t t0 = global_timer_ns();
      while (!sm100::mbar_try_wait(&st->drain[side], 0) && global_timer_ns() - t0 < kWaitNs) {
      }
    }
  } else if (warp >= 4 && live) {
    // the scales of this warp's units, then the pair's sums
    for (int u = set, k = 0; u < units; u += 4, ++k) {
      const int j = 16 * u + lane;
      if (lane < 16) xsc->x[16 * k + lane] = j < t.valid ? p.x_scale[t.row + j] : 0.0f;
    }
    channel_scales(ws1, p.w_scale, p, t, col0, lane);
    if (SIDES == 2) channel_scales(ws3, p.w3_scale, p, t, col0, lane);
    wait<true>(&st->tfull, 0, st, p.err, kErrGemmTimeout | 0x84);
  }
  sm100::tc_fence_before();
  __syncthreads();
  sm100::cluster_sync();  // every pair's MMAs are done with its ring
  sm100::tc_fence_after();
  const uint32_t tbase = tmem + ((uint32_t)(q * 32) << 16);
  // where a sender's unit lies in the ring of the CTA that finishes it
  auto slot = [&](int u, int sender, int owner, int side) {
    const int nth = sender < owner ? sender : sender - 1;
    const int mine = (u >> 1) / parts;  // of the owner's chunks
    return (uint32_t)(((((mine * (parts - 1) + nth) * SIDES + side) * 2 + (u & 1)) * 4 + q) * UNIT);
  };
  auto fetch = [&](int u, int side, uint32_t (&lo)[8], uint32_t (&hi)[8]) {
    const uint32_t c = tbase + (uint32_t)(side * 256 + 16 * u);
    sm100::tmem_ld_16x256b_x2(c, lo);
    sm100::tmem_ld_16x256b_x2(c + (16u << 16), hi);
  };
  if (warp >= 4) {
    for (int u = set; u < units; u += 4) {
      const int owner = (u >> 1) % parts;
      if (owner == part) continue;
#pragma unroll
      for (int side = 0; side < SIDES; ++side) {
        uint32_t lo[8], hi[8];
        fetch(u, side, lo, hi);
        sm100::tmem_ld_wait();
        const uint32_t at = sm100::mapa_shared(sm100::smem_addr(base) + slot(u, part, owner, side),
                                               2 * owner + rank) + lane * 16;
        send16(at, lo);
        send16(at + 512, lo + 4);
        send16(at + 1024, hi);
        send16(at + 1536, hi + 4);
      }
    }
  }
  __syncwarp();
  sm100::tc_fence_before();
  sm100::cluster_sync();  // what was sent has arrived
  sm100::tc_fence_after();
  if (warp >= 4) {
    for (int u = set, k = 0; u < units; u += 4, ++k) {
      if ((u >> 1) % parts != part) continue;
      uint32_t lo[SIDES][8], hi[SIDES][8];
#pragma unroll
      for (int side = 0; side < SIDES; ++side) fetch(u, side, lo[side], hi[side]);
      sm100::tmem_ld_wait();
      for (int other = 0; other < parts; ++other) {
        if (other == part) continue;
#pragma unroll
        for (int side = 0; side < SIDES; ++side) {
          const uint4* r = reinterpret_cast<const uint4*>(base + slot(u, other, part, side)) + lane;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 v = r[32 * i];
            uint32_t* d = (i < 2 ? lo[side] : hi[side]) + 4 * (i & 1);
            d[0] += v.x;
            d[1] += v.y;
            d[2] += v.z;
            d[3] += v.w;
          }
        }
      }
      const float* xs = xsc->x + 16 * k;
      if constexpr (sizeof(OUT) == 2) {
        uint32_t r[2][4];
        if constexpr (SIDES == 2) finish_gated(r, lo[0], hi[0], lo[1], hi[1], xs, ws1, ws3, lane);
        else finish<ACT>(r, lo[0], hi[0], xs, ws1, lane);
        write_rows(staging + (warp - 4), &to, p, t, 16 * u, col0, lane, r);
      } else {
        // (few rows: the fragments' rows are written as they lie)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int k4 = 0; k4 < 4; ++k4)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int at = 4 * j + 2 * (k4 & 1) + e, i = 8 * j + 2 * (lane & 3) + e;
              const int c = col0 + (lane >> 2) + 8 * k4;
              const float a = scaled((k4 < 2 ? lo[0] : hi[0])[at], xs[i], ws1[k4]);
              float v;
              if constexpr (SIDES == 2)
                v = silu_times<OUT>(a, scaled((k4 < 2 ? lo[1] : hi[1])[at], xs[i], ws3[k4]));
              else
                v = activate<ACT>(a);
              if (16 * u + i < t.valid && c < p.n_out)
                static_cast<OUT*>(p.out)[(size_t)(t.row + 16 * u + i) * p.n_out + c] = v;
            }
      }
    }
    if (lane == 0) sm100::bulk_wait_read_all();
  }
  sm100::tc_fence_before();
  __syncthreads();
  sm100::cluster_sync();
  if (warp == 1) {
    sm100::tc_fence_after();
    sm100::tmem_dealloc_pair(tmem, SIDES * 256);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static std::atomic<EncodeTiledFn> cached{nullptr};
  EncodeTiledFn f = cached.load();
  if (f) return f;
  void* q = nullptr;
  cudaDriverEntryPointQueryResult r;
  if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &q, cudaEnableDefault, &r) !=
          cudaSuccess ||
      r != cudaDriverEntryPointSuccess)
    return nullptr;
  f = reinterpret_cast<EncodeTiledFn>(q);
  cached.store(f);
  return f;
}

// [rows, cols] bytes, boxes of 128 columns, 128-byte swizzle; out of range = 0
bool byte_map(CUtensorMap* m, const void* ptr, long long rows, long long cols, int box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t gdim[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t gstride[1] = {(cuuint64_t)cols};
  const cuuint32_t box[2] = {(cuuint32_t)kBK, (cuuint32_t)box_rows};
  const cuuint32_t estride[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), gdim, gstride, box,
            estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// the output [rows, cols] bf16 for stores of 16 rows x 32 columns, 64-byte swizzle
bool out_map(CUtensorMap* m, void* ptr, long long rows, long long cols) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t gdim[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t gstride[1] = {(cuuint64_t)cols * 2};
  const cuuint32_t box[2] = {32, 16}, estride[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, ptr, gdim, gstride, box, estride,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class State>
constexpr size_t smem_bytes(int ring) {
  return (size_t)ring + kEpiWarps * (sizeof(Staging) + sizeof(Scales)) + sizeof(State) + 1024;
}

template <auto kern, class... Args>
cudaError_t launch_i8(int pairs, size_t bytes, cudaStream_t s, const Args&... args) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_all_smem(kern, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(2 * pairs), dim3(kThreads), bytes, s, args...);
}

// `tiles` clusters of 2 * parts CTAs
template <auto kern, class... Args>
cudaError_t launch_split(int tiles, int parts, size_t bytes, cudaStream_t s, const Args&... args) {
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_all_smem(kern, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * parts * tiles);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2 * parts;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

template <typename OUT, int ACT>
cudaError_t run_act(const RowMaps& x, const CUtensorMap& w, const CUtensorMap& w3,
                    const CUtensorMap& o, const I8Params& p, int tiles, cudaStream_t s) {
  constexpr size_t stream_bytes = smem_bytes<StreamState>(kStreams * kStagesS * kStageBytesS);
  constexpr size_t up_bytes = smem_bytes<UpState>(kStagesU * kStageBytesU);
  constexpr size_t split_bytes = smem_bytes<SplitState>(kSplitRing);
  static_assert(stream_bytes <= 232448 && up_bytes <= 232448 && split_bytes <= 232448,
                "227 KB of shared memory");
  if (p.parts > 1)
    return launch_split<i8_split_kernel<OUT, ACT>>(tiles, p.parts, split_bytes, s, x, w, w3, o, p);
  const int pairs = tiles < kBlockSms / 2 ? tiles : kBlockSms / 2;
  if constexpr (ACT == A_SWIGLU)
    return launch_i8<i8_swiglu_pair_kernel<OUT>>(pairs, up_bytes, s, x, w, w3, o, p);
  else
    return launch_i8<i8_pair_kernel<OUT, ACT>>(pairs, stream_bytes, s, x, w, o, p);
}

template <typename OUT>
cudaError_t run_gemm(const RowMaps& x, const CUtensorMap& w, const CUtensorMap& w3,
                     const CUtensorMap& o, int act, const I8Params& p, int tiles,
                     cudaStream_t s) {
  switch (act) {
    case MOE_I8_SWIGLU: return run_act<OUT, A_SWIGLU>(x, w, w3, o, p, tiles, s);
    case MOE_I8_RELU: return run_act<OUT, A_RELU>(x, w, w3, o, p, tiles, s);
    case MOE_I8_GELU: return run_act<OUT, A_GELU>(x, w, w3, o, p, tiles, s);
    default: return run_act<OUT, A_NONE>(x, w, w3, o, p, tiles, s);
  }
}

moe_status i8_check(const moe_gemm_i8_config* c) {
  if (!c || c->groups < 1 || c->rows < 0 || c->k < 1 || c->n_out < 1) return MOE_ERR_INVALID_ARG;
  if (c->dtype != MOE_F32 && c->dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (c->act != MOE_I8_NONE && c->act != MOE_I8_RELU && c->act != MOE_I8_GELU &&
      c->act != MOE_I8_SWIGLU)
    return MOE_ERR_INVALID_ARG;
  if (c->groups > MOE_I8_MAX_GROUPS || c->k % 16 || c->k > MOE_I8_MAX_K || c->n_out % 16)
    return MOE_ERR_UNSUPPORTED;
  if (c->rows > (1 << 30) || (long long)c->groups * c->n_out > (1LL << 30))
    return MOE_ERR_UNSUPPORTED;
  // tile numbers are 32-bit
  const long long tiles = ((long long)c->rows / kMaxTok + c->groups + 1) * (c->n_out / 256 + 1);
  if (tiles > (1LL << 30)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_gemm_i8_validate(const moe_gemm_i8_config* cfg) { return i8_check(cfg); }

moe_status moe_gemm_i8_workspace_size(const moe_gemm_i8_config* cfg, size_t* bytes) {
  moe_status st = i8_check(cfg);
  if (st != MOE_OK) return st;
  if (bytes) *bytes = MOE_WS_ERROR_BYTES;
  return MOE_OK;
}

moe_status moe_gemm_i8(const moe_gemm_i8_config* cfg, const int8_t* xq, const float* x_scale,
                       const int32_t* starts, const int32_t* counts, const int8_t* w,
                       const float* w_scale, const int8_t* w3, const float* w3_scale, void* out,
                       void* ws, size_t ws_bytes, moe_stream_t stream) {
  moe_status st = i8_check(cfg);
  if (st != MOE_OK) return st;
  if ((starts != nullptr) != (counts != nullptr)) return MOE_ERR_INVALID_ARG;
  if (!starts && cfg->groups != 1) return MOE_ERR_INVALID_ARG;
  if (!w || !w_scale) return MOE_ERR_INVALID_ARG;
  const bool swiglu = cfg->act == MOE_I8_SWIGLU;
  if (swiglu != (w3 != nullptr) || swiglu != (w3_scale != nullptr)) return MOE_ERR_INVALID_ARG;
  if ((st = check_block_ws(ws, ws_bytes, MOE_WS_ERROR_BYTES)) != MOE_OK) return st;
  if (cfg->rows == 0) return MOE_OK;
  if (!xq || !x_scale || !out) return MOE_ERR_INVALID_ARG;
  if (!aligned16(xq) || !aligned16(w) || !aligned16(w3) || !aligned16(out))
    return MOE_ERR_INVALID_ARG;
  RowMaps x;
  for (int b = 0; b < kBoxes; ++b)
    if (!byte_map(&x.m[b], xq, cfg->rows, cfg->k, b ? 64 : 16)) return MOE_ERR_CUDA;
  CUtensorMap mw, mw3;
  const long long wrows = (long long)cfg->groups * cfg->n_out;
  if (!byte_map(&mw, w, wrows, cfg->k, 128)) return MOE_ERR_CUDA;
  mw3 = mw;
  if (swiglu && !byte_map(&mw3, w3, wrows, cfg->k, 128)) return MOE_ERR_CUDA;
  // (fp32 outputs are not stored through it)
  CUtensorMap mo = mw;
  if (cfg->dtype == MOE_BF16 && !out_map(&mo, out, cfg->rows, cfg->n_out)) return MOE_ERR_CUDA;
  I8Params p{};
  p.starts = starts;
  p.counts = counts;
  p.x_scale = x_scale;
  p.w_scale = w_scale;
  p.w3_scale = w3_scale;
  p.groups = cfg->groups;
  p.rows = cfg->rows;
  p.K = cfg->k;
  p.n_out = cfg->n_out;
  p.mt_tiles = (cfg->n_out + 255) / 256;
  p.out = out;
  p.err = static_cast<int*>(ws);
  // A bound on the tiles. Few of them leave most SMs idle: a long K is then split
  // over the pairs of a cluster, as far as all clusters are resident at once:
  // they do not fill every GPC, and a second round costs more than the split
  // saves. Measured, one row, weights from HBM, us in 1 / 2 / 4 parts:
  //   k 7168, 15 tiles 25.5 / 16.2 / 12.8, 16 tiles 25.7 / 16.2 / 23.1;
  //   k 4096, 33 tiles 17.0 / 13.4 / 27.6, 34 tiles 17.1 / 23.3 / 27.7
  // (the limits keep one or so in hand). A short K loses to the two barriers of the
  // cluster and the exchange: 8 tiles, k 1024 6.8 / 7.7 / 7.6, k 2048 9.4 / 8.7 / 8.1;
  // SwiGLU exchanges twice the sums: 32 tiles, k 2048 11.8 / 12.6, k 4096 18.7 / 18.6.
  const long long tiles =
      ((long long)cfg->rows + (kMaxTok - 1LL) * cfg->groups) / kMaxTok * p.mt_tiles;
  const int kblocks = (cfg->k + kBK - 1) / kBK;
  p.parts = tiles <= 14 && kblocks >= 16                  ? 4
            : tiles <= 32 && kblocks >= (swiglu ? 32 : 16) ? 2
                                                           : 1;
  cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = cfg->dtype == MOE_BF16
                            ? run_gemm<__nv_bfloat16>(x, mw, mw3, mo, cfg->act, p, (int)tiles, s)
                            : run_gemm<float>(x, mw, mw3, mo, cfg->act, p, (int)tiles, s);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
