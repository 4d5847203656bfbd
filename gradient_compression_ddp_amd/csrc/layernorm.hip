// Layer norm's forward and backward passes (gc_layernorm_forward, gc_layernorm_backward),
// with the 8-bit checkpoint packed by the one and read by the other, and the reduction of
// the weight's and bias's gradients.
//
// A row belongs to a team of threads that keeps it in registers between the statistics and
// the use, so HBM sees each element once: 64, 256 or 512 threads with one to four
// chunks of 8 columns each, the smallest team that covers the row (up to 16384 columns).
// Teams walk down the rows with the weights in registers and the next row's loads in flight.
// The forward pass and the widest backward rows keep a row as it was loaded and convert it at each use: for
// 16-bit types half the registers of its fp32 values.
// Wider rows take the looped kernels at the end of this file, which re-read the row.
//
// Bound by HBM.  Measured over 16384 x 4096 in bf16, one call repeated on four sets of inputs (a copy of that size: 5.3
// TB/s): forward 46 us, 5.8 TB/s; with x packed 66 us, 5.1 TB/s; backward with dw and db from the checkpoint 67 to 75 us, 4.5
// to 5.0 TB/s, from x 80 us, 5.0 TB/s.  The backward pass falls short of the copy by its two row sums, a barrier each row, and
// by joining dw and db (5 us).  Rows of 20000 (looped), 4096 of them: forward 116 us, backward 157 from the checkpoint and 180
// from x, 2.6 to 2.8 TB/s of bytes counted once, since they read the row three times and twice.
//
// Statistics: mean first, then the sum of squared deviations from it, both over registers,
// so nothing cancels when the mean is large against the deviation.
#include <hip/hip_runtime.h>

#include "ckpt_core.hpp"
#include "gc_train.h"
#include "internal.hpp"
#include "train_internal.hpp"

namespace gc {
namespace {

constexpr int kMaxTeamCols = 16384;

// Sum over a wave; every lane ends with it.
__device__ __forceinline__ float wave_sum(float v) { return seg_tree_sum_c<6>(v); }

// Sum over a team of TEAM threads (the whole block when TEAM > 64).  s: one float per wave,
// not read or written by the previous team_sum of the same block.
template <int TEAM>
__device__ __forceinline__ float team_sum(float v, float* s) {
  v = wave_sum(v);
  if constexpr (TEAM > kWave) {
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    v = s[0];
#pragma unroll
    for (int i = 1; i < TEAM / kWave; ++i) v += s[i];
  }
  return v;
}

template <bool WHOLE, typename W>
__device__ __forceinline__ void load_weight(const W* w, int64_t col, int n, int64_t cols, float none, float v[8]) {
  if (w) {
    Raw8<W> r = raw8w<W, WHOLE>(w + col, n, cols);
    tail8<W, WHOLE>(r, n, cols);
    get8<W>(r, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = none;
  }
}

// Packs one chunk of a row; the four lanes of a block of 32 call it together.
template <typename T>
__device__ __forceinline__ void pack_chunk(const float v[8], int8_t* codes, uint8_t* exps, int64_t row, int64_t ldc, int chunk) {
  const Packed8 c = pack8<T>(v);
  const int64_t at = row * (ldc / kChunk) + chunk;
  reinterpret_cast<u32x2*>(codes)[at] = u32x2{c.lo, c.hi};
  if ((chunk & 3) == 0) exps[at >> 2] = (uint8_t)c.e;
}

__device__ __forceinline__ int left_of(int64_t cols, int chunk) {
  const int64_t l = cols - (int64_t)chunk * kChunk;
  return l > kChunk ? kChunk : (int)l;
}

template <typename T, typename W, bool WHOLE, int TEAM, int NV>
__global__ __launch_bounds__(TEAM < 256 ? 256 : TEAM) void k_ln_forward(LnFwdArgs a) {
  constexpr int BT = TEAM < 256 ? 256 : TEAM, RPB = BT / TEAM;
  __shared__ float s_mean[BT / kWave], s_var[BT / kWave];
  const int lane = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
  const int64_t ldc = (a.cols + kBlockCols - 1) / kBlockCols * kBlockCols;
  const int chunks = (int)(ldc / kChunk);
  float w[NV][8], b[NV][8];
  int n[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    n[j] = left_of(a.cols, lane + j * TEAM);
    load_weight<WHOLE>(static_cast<const W*>(a.w), (int64_t)(lane + j * TEAM) * kChunk, n[j], a.cols, 1.0f, w[j]);
    load_weight<WHOLE>(static_cast<const W*>(a.b), (int64_t)(lane + j * TEAM) * kChunk, n[j], a.cols, 0.0f, b[j]);
  }
  const float cols = (float)a.cols;
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t row = (int64_t)blockIdx.x * RPB + team;
  Raw8<T> raw[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j)
    raw[j] = raw8w<T, WHOLE>(static_cast<const T*>(a.x) + (row < a.rows ? row : 0) * a.ldx + (lane + j * TEAM) * kChunk, row < a.rows ? n[j] : 0, a.cols);
  // TEAM > 64 has one team per block, so the barriers below are reached by every thread
  for (; row < a.rows; row += step) {
    Raw8<T> cur[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) cur[j] = raw[j];
    const int64_t next = row + step;
    if (next < a.rows) {
#pragma unroll
      for (int j = 0; j < NV; ++j) raw[j] = raw8w<T, WHOLE>(static_cast<const T*>(a.x) + next * a.ldx + (lane + j * TEAM) * kChunk, n[j], a.cols);
    }
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float x[8];
      tail8<T, WHOLE>(cur[j], n[j], a.cols);
      get8<T>(cur[j], x);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += x[i];
    }
    const float mean = team_sum<TEAM>(sum, s_mean) / cols;
    float sq = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float x[8];
      if constexpr (sizeof(T) == 2) forget<T>(cur[j]);
      get8<T>(cur[j], x);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = i < n[j] ? x[i] - mean : 0.0f;
        sq = __builtin_fmaf(d, d, sq);
      }
    }
    const float var = team_sum<TEAM>(sq, s_var) / cols;
    const float rstd = 1.0f / __builtin_sqrtf(var + a.eps);
    if (lane == 0) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int chunk = lane + j * TEAM;
      if (chunk >= chunks) continue;      // the same for the four lanes of a block of 32
      float x[8], y[8];
      if constexpr (sizeof(T) == 2) forget<T>(cur[j]);
      get8<T>(cur[j], x);
      if (a.x_codes) pack_chunk<T>(x, a.x_codes, a.x_exps, row, ldc, chunk);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = __builtin_fmaf((x[i] - mean) * rstd, w[j][i], b[j][i]);
      store8n<T, WHOLE>(static_cast<T*>(a.y) + row * a.ldy + (int64_t)chunk * kChunk, n[j], y);
      if (a.y_codes) {
        round8<T>(y);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = i < n[j] ? y[i] : 0.0f;
        pack_chunk<T>(y, a.y_codes, a.y_exps, row, ldc, chunk);
      }
    }
  }
}

// One chunk of the kept input, in flight.
template <typename T, bool CK, bool WHOLE>
struct Kept;
template <typename T, bool WHOLE>
struct Kept<T, false, WHOLE> {
  Raw8<T> r;
  __device__ __forceinline__ void load(const LnBwdArgs& a, int64_t row, int64_t, int chunk, int n) {
    r = raw8w<T, WHOLE>(static_cast<const T*>(a.x) + row * a.ldx + (int64_t)chunk * kChunk, n, a.cols);
  }
  __device__ __forceinline__ void settle(int n, int64_t cols) { tail8<T, WHOLE>(r, n, cols); }    // before the first get
  __device__ __forceinline__ void get(float v[8]) const { get8<T>(r, v); }
  __device__ __forceinline__ void half(int h, float v[4]) const { get4<T>(r, h, v); }
  __device__ __forceinline__ void drop() {
    if constexpr (sizeof(T) == 2) forget<T>(r);
  }
};
template <typename T, bool WHOLE>
struct Kept<T, true, WHOLE> {
  u32x2 c;
  uint32_t e;
  __device__ __forceinline__ void load(const LnBwdArgs& a, int64_t row, int64_t ldc, int chunk, int n) {
    c = u32x2{0u, 0u};
    e = 7u;
    if (n <= 0) return;
    const int64_t at = row * (ldc / kChunk) + chunk;
    c = reinterpret_cast<const u32x2*>(a.x_codes)[at];
    e = a.x_exps[at >> 2];
  }
  __device__ __forceinline__ void settle(int, int64_t) {}
  __device__ __forceinline__ void get(float v[8]) const { decode8(c[0], c[1], ckpt_step(e), v); }
  __device__ __forceinline__ void half(int h, float v[4]) const { decode4(c[h], ckpt_step(e), v); }
  __device__ __forceinline__ void drop() { asm volatile("" : "+v"(c), "+v"(e)); }
};

// Threads of a backward block, one block per CU.  Teams of 64 and 256 share a block, which joins their sums of
// dw and db in LDS: 256 blocks leave 256 partial sums (512 blocks took 4 to 5 us longer at any width, for the second
// half's traffic).
constexpr int kBwdThreads = 512;

// The row's two sums cross the team once per row (one barrier, two LDS slots in turn).  dw
// and db are summed per thread over its team's rows, joined over the block's teams, and
// written as this block's row of `part`: [gridDim.x][2][pcols].
//
// Columns past the row's end load as zeros, and count from 0 instead of the mean: their t and xh are 0, and so is what
// they add to any sum.  (-mean * rstd can pass the largest number, and 0 * Inf would reach the whole row.)
template <typename T, typename W, bool CK, bool WHOLE, int TEAM, int NV>
__global__ __launch_bounds__(kBwdThreads) void k_ln_backward(LnBwdArgs a, float* part, int64_t pcols) {
  constexpr int BT = kBwdThreads, RPB = BT / TEAM, TW = TEAM / kWave, SPAN = NV * TEAM * kChunk;
  constexpr bool KEEP = NV <= 2;       // the row's fp32 values stay from its sums to dx; else they are converted again
  constexpr bool AHEAD = NV <= 2 || (NV == 3 && sizeof(T) == 2);   // the next row's loads in flight, where their registers fit
  __shared__ float s_sum[2][2][BT / kWave];
  // the weights while rows are read (one copy for the block), the teams' sums at the end
  __shared__ __attribute__((aligned(16))) float s_acc[RPB > 1 ? RPB * 2 * SPAN : SPAN];
  const int lane = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
  const int64_t ldc = (a.cols + kBlockCols - 1) / kBlockCols * kBlockCols;
  float dw[NV][8], db[NV][8];
  int n[NV];
  f32x4* s_w = reinterpret_cast<f32x4*>(s_acc);        // [chunk j][half][lane]: 16 bytes a lane side by side
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    n[j] = left_of(a.cols, lane + j * TEAM);
    if (team == 0) {
      float w[8];
      load_weight<WHOLE>(static_cast<const W*>(a.w), (int64_t)(lane + j * TEAM) * kChunk, n[j], a.cols, 1.0f, w);
      s_w[(2 * j) * TEAM + lane] = f32x4{w[0], w[1], w[2], w[3]};
      s_w[(2 * j + 1) * TEAM + lane] = f32x4{w[4], w[5], w[6], w[7]};
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[j][i] = db[j][i] = 0.0f;
  }
  __syncthreads();
  const auto weight = [&](int j, int h) { return s_w[(2 * j + h) * TEAM + lane]; };
  const auto centre = [&](float mean, int j, int c) { return (WHOLE ? 0 : c) < n[j] ? mean : 0.0f; };   // of column c of chunk j
  const float cols = (float)a.cols;
  const int64_t step = (int64_t)gridDim.x * RPB;
  struct Row {
    Raw8<T> dy[NV];
    Kept<T, CK, WHOLE> kept[NV];
    float mean, rstd;
  };
  const auto fetch = [&](Row& r, int64_t row) {
    const bool on = row < a.rows;
    const int64_t at = on ? row : 0;
    r.mean = on ? a.mean[at] : 0.0f;
    r.rstd = on ? a.rstd[at] : 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int chunk = lane + j * TEAM, m = on ? n[j] : 0;
      r.dy[j] = raw8w<T, WHOLE>(static_cast<const T*>(a.dy) + at * a.lddy + (int64_t)chunk * kChunk, m, a.cols);
      r.kept[j].load(a, at, ldc, chunk, m);
    }
  };
  Row next;
  if constexpr (AHEAD) fetch(next, (int64_t)blockIdx.x * RPB + team);
  int slot = 0;
  // every team of the block runs the same number of rounds; a team past the end adds zeros
  for (int64_t first = (int64_t)blockIdx.x * RPB; first < a.rows; first += step) {
    const int64_t row = first + team;
    Row cur;
    if constexpr (AHEAD) {
      cur = next;
      if (first + step < a.rows) fetch(next, row + step);
    } else {
      fetch(cur, row);
    }
    const float mean = cur.mean, rstd = cur.rstd;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int m = row < a.rows ? n[j] : 0;
      tail8<T, WHOLE>(cur.dy[j], m, a.cols);
      cur.kept[j].settle(m, a.cols);
    }
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4 w = weight(j, h);
        float d[4], x[4];
        get4<T>(cur.dy[j], h, d);
        cur.kept[j].half(h, x);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float xh = (x[i] - centre(mean, j, 4 * h + i)) * rstd, t = d[i] * w[i];
          dw[j][4 * h + i] = __builtin_fmaf(d[i], xh, dw[j][4 * h + i]);
          db[j][4 * h + i] += d[i];
          s1 += t;
          s2 = __builtin_fmaf(t, xh, s2);
        }
        if constexpr (!KEEP) __builtin_amdgcn_sched_barrier(0);     // four columns' values at a time
      }
    }
    s1 = wave_sum(s1);
    s2 = wave_sum(s2);
    if constexpr (TEAM > kWave) {
      if ((threadIdx.x & 63) == 0) {
        s_sum[slot][0][threadIdx.x >> 6] = s1;
        s_sum[slot][1][threadIdx.x >> 6] = s2;
      }
      __syncthreads();
      s1 = s_sum[slot][0][team * TW];
      s2 = s_sum[slot][1][team * TW];
#pragma unroll
      for (int i = 1; i < TW; ++i) {
        s1 += s_sum[slot][0][team * TW + i];
        s2 += s_sum[slot][1][team * TW + i];
      }
      slot ^= 1;
    }
    s1 /= cols;
    s2 /= cols;
    if (row < a.rows) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float out[8];
        if constexpr (!KEEP) {
          asm volatile("" ::: "memory");     // the weights are read again, too
          if constexpr (sizeof(T) == 2) forget<T>(cur.dy[j]);
          cur.kept[j].drop();
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const f32x4 w = weight(j, h);
          float d[4], x[4];
          get4<T>(cur.dy[j], h, d);
          cur.kept[j].half(h, x);
#pragma unroll
          for (int i = 0; i < 4; ++i) out[4 * h + i] = rstd * __builtin_fmaf(-((x[i] - centre(mean, j, 4 * h + i)) * rstd), s2, __builtin_fmaf(d[i], w[i], -s1));
          if constexpr (!KEEP) __builtin_amdgcn_sched_barrier(0);
        }
        store8n<T, WHOLE>(static_cast<T*>(a.dx) + row * a.lddx + (int64_t)(lane + j * TEAM) * kChunk, n[j], out);
        if constexpr (!KEEP) __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  if (!part) return;
  // the only block of a launch writes dw and db themselves
  const bool alone = gridDim.x == 1;
  float* out = part + (int64_t)blockIdx.x * 2 * pcols;
  if constexpr (RPB == 1) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t col = (int64_t)(lane + j * TEAM) * kChunk;
      if (n[j] <= 0) continue;
      if (alone) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (i < n[j] && a.dw) a.dw[col + i] = a.accumulate ? a.dw[col + i] + dw[j][i] : dw[j][i];
          if (i < n[j] && a.db) a.db[col + i] = a.accumulate ? a.db[col + i] + db[j][i] : db[j][i];
        }
      } else {                           // pcols is a multiple of 8: a whole chunk is written
        store8(out + col, dw[j]);
        store8(out + pcols + col, db[j]);
      }
    }
  } else {
    __syncthreads();                     // the weights are no longer read
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float* s = s_acc + team * 2 * SPAN + (lane + j * TEAM) * kChunk;
      store8(s, dw[j]);
      store8(s + SPAN, db[j]);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * SPAN; c += BT) {
      const int col = c % SPAN;
      if (col >= (alone ? a.cols : pcols)) continue;
      float sum = s_acc[c];
#pragma unroll
      for (int k = 1; k < RPB; ++k) sum += s_acc[k * 2 * SPAN + c];     // the teams in order
      if (alone) {
        float* d = c < SPAN ? a.dw : a.db;
        if (d) d[col] = a.accumulate ? d[col] + sum : sum;
      } else {
        out[(c / SPAN) * pcols + col] = sum;
      }
    }
  }
}

// dw and db from the partial sums: 32 columns x 16 slices of the partials a block at a time, each
// slice summed in order, the slices then in order.
constexpr int kSlices = 16;
__global__ __launch_bounds__(32 * kSlices) void k_ln_join(const float* part, int parts, int64_t pcols, int64_t cols,
                                                 float* dw, float* db, int accumulate) {
  __shared__ float s[kSlices][32];
  const int c = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int which = blockIdx.y;
  float* out = which ? db : dw;
  for (int64_t first = (int64_t)blockIdx.x * 32; first < cols; first += (int64_t)gridDim.x * 32) {
    const int64_t col = first + c;
    float sum = 0.0f;
    if (col < cols) {
      const float* p = part + which * pcols + col;
#pragma unroll 4
      for (int i = slice; i < parts; i += kSlices) sum += p[(int64_t)i * 2 * pcols];
    }
    s[slice][c] = sum;
    __syncthreads();
    if (slice == 0 && col < cols && out) {
#pragma unroll
      for (int i = 1; i < kSlices; ++i) sum += s[i][c];
      out[col] = accumulate ? out[col] + sum : sum;
    }
    __syncthreads();
  }
}

// ---- rows wider than a team holds ------------------------------------------------------

constexpr int kWideThreads = 1024;

template <typename T, typename W>
__global__ __launch_bounds__(kWideThreads) void k_ln_forward_wide(LnFwdArgs a) {
  __shared__ float s_mean[kWideThreads / kWave], s_var[kWideThreads / kWave];
  const int64_t ldc = (a.cols + kBlockCols - 1) / kBlockCols * kBlockCols;
  const int chunks = (int)(ldc / kChunk);
  const float cols = (float)a.cols;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    float v[8], sum = 0.0f, sq = 0.0f;
    for (int c = threadIdx.x; c < chunks; c += kWideThreads) {
      load8n(x + (int64_t)c * kChunk, left_of(a.cols, c), a.cols, v);
      float part = 0.0f;                 // chunk by chunk: a long row's sum stays a short chain of short sums
#pragma unroll
      for (int i = 0; i < 8; ++i) part += v[i];
      sum += part;
    }
    const float mean = team_sum<kWideThreads>(sum, s_mean) / cols;
    for (int c = threadIdx.x; c < chunks; c += kWideThreads) {
      const int n = left_of(a.cols, c);
      load8n(x + (int64_t)c * kChunk, n, a.cols, v);
      float part = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = i < n ? v[i] - mean : 0.0f;
        part = __builtin_fmaf(d, d, part);
      }
      sq += part;
    }
    const float var = team_sum<kWideThreads>(sq, s_var) / cols;
    const float rstd = 1.0f / __builtin_sqrtf(var + a.eps);
    if (threadIdx.x == 0) {
      a.mean[row] = mean;
      a.rstd[row] = rstd;
    }
    for (int c = threadIdx.x; c < chunks; c += kWideThreads) {
      const int n = left_of(a.cols, c);
      float w[8], b[8];
      load8n(x + (int64_t)c * kChunk, n, a.cols, v);
      load_weight<false>(static_cast<const W*>(a.w), (int64_t)c * kChunk, n, a.cols, 1.0f, w);
      load_weight<false>(static_cast<const W*>(a.b), (int64_t)c * kChunk, n, a.cols, 0.0f, b);
      if (a.x_codes) pack_chunk<T>(v, a.x_codes, a.x_exps, row, ldc, c);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __builtin_fmaf((v[i] - mean) * rstd, w[i], b[i]);
      store8n(static_cast<T*>(a.y) + row * a.ldy + (int64_t)c * kChunk, n, v);
      if (a.y_codes) {
        round8<T>(v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? v[i] : 0.0f;
        pack_chunk<T>(v, a.y_codes, a.y_exps, row, ldc, c);
      }
    }
  }
}

// The two row means of the backward pass, means[row] = (sum t, sum t * xh) / cols.
template <typename T, typename W, bool CK>
__global__ __launch_bounds__(kWideThreads) void k_ln_means_wide(LnBwdArgs a, float2* means) {
  __shared__ float s_one[kWideThreads / kWave], s_two[kWideThreads / kWave];
  const int64_t ldc = (a.cols + kBlockCols - 1) / kBlockCols * kBlockCols;
  const int chunks = (int)(ldc / kChunk);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float mean = a.mean[row], rstd = a.rstd[row];
    float s1 = 0.0f, s2 = 0.0f;
    for (int c = threadIdx.x; c < chunks; c += kWideThreads) {
      const int n = left_of(a.cols, c);
      float w[8], d[8], x[8];
      Kept<T, CK, false> k;
      k.load(a, row, ldc, c, n);
      load8n(static_cast<const T*>(a.dy) + row * a.lddy + (int64_t)c * kChunk, n, a.cols, d);
      load_weight<false>(static_cast<const W*>(a.w), (int64_t)c * kChunk, n, a.cols, 1.0f, w);
      k.settle(n, a.cols);
      k.get(x);
      float p1 = 0.0f, p2 = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float t = i < n ? d[i] * w[i] : 0.0f, xh = i < n ? (x[i] - mean) * rstd : 0.0f;
        p1 += t;
        p2 = __builtin_fmaf(t, xh, p2);
      }
      s1 += p1;
      s2 += p2;
    }
    const float c = (float)a.cols;
    s1 = team_sum<kWideThreads>(s1, s_one) / c;
    s2 = team_sum<kWideThreads>(s2, s_two) / c;
    if (threadIdx.x == 0) means[row] = float2{s1, s2};
  }
}

// dx and the partial sums over strips of 2048 columns: blockIdx.x the strip, blockIdx.y the
// share of the rows.
template <typename T, typename W, bool CK>
__global__ __launch_bounds__(256) void k_ln_backward_wide(LnBwdArgs a, const float2* means, float* part, int64_t pcols) {
  const int64_t ldc = (a.cols + kBlockCols - 1) / kBlockCols * kBlockCols;
  const int chunk = blockIdx.x * 256 + threadIdx.x;
  const int n = left_of(a.cols, chunk);
  if (n <= 0) return;
  float w[8], dw[8], db[8];
  load_weight<false>(static_cast<const W*>(a.w), (int64_t)chunk * kChunk, n, a.cols, 1.0f, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[i] = db[i] = 0.0f;
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const float mean = a.mean[row], rstd = a.rstd[row];
    const float2 m = means[row];
    float d[8], x[8];
    Kept<T, CK, false> k;
    k.load(a, row, ldc, chunk, n);
    load8n(static_cast<const T*>(a.dy) + row * a.lddy + (int64_t)chunk * kChunk, n, a.cols, d);
    k.settle(n, a.cols);
    k.get(x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float xh = (x[i] - mean) * rstd;
      dw[i] = __builtin_fmaf(d[i], xh, dw[i]);
      db[i] += d[i];
      d[i] = rstd * __builtin_fmaf(-xh, m.y, d[i] * w[i] - m.x);
    }
    store8n(static_cast<T*>(a.dx) + row * a.lddx + (int64_t)chunk * kChunk, n, d);
  }
  if (!part) return;
  float* out = part + (int64_t)blockIdx.y * 2 * pcols + (int64_t)chunk * kChunk;
  store8(out, dw);
  store8(out + pcols, db);
}

// ---- host ---------------------------------------------------------------------------------

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct TeamShape {
  int team, nv;
};
TeamShape shape_for(int64_t cols) {
  if (cols <= 512) return {64, 1};
  if (cols <= 1024) return {64, 2};
  if (cols <= 2048) return {256, 1};
  if (cols <= 4096) return {256, 2};
  if (cols <= 8192) return {512, 2};
  if (cols <= 12288) return {512, 3};
  return {512, 4};
}

// Blocks of the backward pass, which is also the number of partial sums: up to one per CU.  One block as long
// as its teams have no more than four rows each, since it needs no joining launch (32 x 1024: 13.5 us a call, not 16).
// Beyond, a team gets one row, teams of 512 two: a row more in a team is one more wait on memory, a block more
// is 8 bytes a column written and read.  In us, kernel and join, with one row, two and four:
//   bf16  1001 x 1023: 9.6, 10.8, 14.6    256 x 4096: 10.8, 10.7, 14.4    128 x 16000: 18.7, 17.2, 19.3
//   fp32  1001 x 1023: 10.2, 11.4, 15.5   256 x 4096: 11.8, 11.8, 16.0    256 x 8192: 17.2, 15.2, 16.6
int64_t backward_parts(int64_t rows, int64_t cols) {
  if (cols > kMaxTeamCols) {
    const int64_t strips = ceil_div(cols, 256 * kChunk), most = ceil_div(2048, strips);
    const int64_t want = ceil_div(rows, 8);
    return want < most ? want : most;
  }
  const TeamShape t = shape_for(cols);
  const int64_t teams = kBwdThreads / t.team;
  if (rows <= 4 * teams) return 1;
  const int64_t want = ceil_div(rows, t.team == 512 ? 2 * teams : teams), most = 256;
  return want < most ? want : most;
}
int64_t part_cols(int64_t cols) { return ceil_div(cols, kBlockCols) * kBlockCols; }

template <typename T, typename W, int TEAM, int NV>
hipError_t forward_team(const LnFwdArgs& a, hipStream_t s) {
  constexpr int BT = TEAM < 256 ? 256 : TEAM, RPB = BT / TEAM;
  const int64_t want = ceil_div(a.rows, RPB), most = (int64_t)device_cu_count() * (2048 / BT);
  const unsigned g = (unsigned)(want < most ? want : most);
  if (a.cols % kChunk == 0) k_ln_forward<T, W, true, TEAM, NV><<<g, BT, 0, s>>>(a);
  else k_ln_forward<T, W, false, TEAM, NV><<<g, BT, 0, s>>>(a);
  return hipGetLastError();
}

template <typename T, typename W>
hipError_t forward_w(const LnFwdArgs& a, hipStream_t s) {
  if (a.cols > kMaxTeamCols) {
    const int64_t most = (int64_t)device_cu_count() * 2;
    k_ln_forward_wide<T, W><<<(unsigned)(a.rows < most ? a.rows : most), kWideThreads, 0, s>>>(a);
    return hipGetLastError();
  }
  const TeamShape t = shape_for(a.cols);
  if (t.team == 64) return t.nv == 1 ? forward_team<T, W, 64, 1>(a, s) : forward_team<T, W, 64, 2>(a, s);
  if (t.team == 256) return t.nv == 1 ? forward_team<T, W, 256, 1>(a, s) : forward_team<T, W, 256, 2>(a, s);
  if (t.nv == 2) return forward_team<T, W, 512, 2>(a, s);
  return t.nv == 3 ? forward_team<T, W, 512, 3>(a, s) : forward_team<T, W, 512, 4>(a, s);
}

template <typename T, typename W, bool CK, int TEAM, int NV>
hipError_t backward_team(const LnBwdArgs& a, float* part, int64_t pcols, hipStream_t s) {
  constexpr int BT = kBwdThreads;
  const unsigned g = (unsigned)backward_parts(a.rows, a.cols);
  if (a.cols % kChunk == 0) k_ln_backward<T, W, CK, true, TEAM, NV><<<g, BT, 0, s>>>(a, part, pcols);
  else k_ln_backward<T, W, CK, false, TEAM, NV><<<g, BT, 0, s>>>(a, part, pcols);
  return hipGetLastError();
}

template <typename T, typename W, bool CK>
hipError_t backward_ck(const LnBwdArgs& a, hipStream_t s) {
  const int64_t pcols = part_cols(a.cols);
  // a dimension holds fewer than 2^32 threads: columns past 2^27 take further turns
  const int64_t groups = ceil_div(a.cols, 32);
  const dim3 join((unsigned)(groups < (int64_t(1) << 22) ? groups : (int64_t(1) << 22)), 2);
  if (a.rows == 0) {                       // nothing to sum: the sums are cleared
    k_ln_join<<<join, 32 * kSlices, 0, s>>>(nullptr, 0, pcols, a.cols, a.dw, a.db, a.accumulate);
    return hipGetLastError();
  }
  const TeamShape t = shape_for(a.cols);
  const int64_t parts = backward_parts(a.rows, a.cols);
  float* part = a.dw || a.db ? static_cast<float*>(a.ws) : nullptr;
  hipError_t e;
  if (a.cols > kMaxTeamCols) {
    float2* means = reinterpret_cast<float2*>(static_cast<char*>(a.ws) + align256((size_t)parts * 2 * pcols * 4));
    const int64_t most = (int64_t)device_cu_count() * 2;
    k_ln_means_wide<T, W, CK><<<(unsigned)(a.rows < most ? a.rows : most), kWideThreads, 0, s>>>(a, means);
    const dim3 grid((unsigned)ceil_div(a.cols, 256 * kChunk), (unsigned)parts);
    k_ln_backward_wide<T, W, CK><<<grid, 256, 0, s>>>(a, means, part, pcols);
    e = hipGetLastError();
  } else if (t.team == 64) {
    e = t.nv == 1 ? backward_team<T, W, CK, 64, 1>(a, part, pcols, s) : backward_team<T, W, CK, 64, 2>(a, part, pcols, s);
  } else if (t.team == 256) {
    e = t.nv == 1 ? backward_team<T, W, CK, 256, 1>(a, part, pcols, s) : backward_team<T, W, CK, 256, 2>(a, part, pcols, s);
  } else if (t.nv == 2) {
    e = backward_team<T, W, CK, 512, 2>(a, part, pcols, s);
  } else {
    e = t.nv == 3 ? backward_team<T, W, CK, 512, 3>(a, part, pcols, s) : backward_team<T, W, CK, 512, 4>(a, part, pcols, s);
  }
  if (e != hipSuccess || !part || (parts == 1 && a.cols <= kMaxTeamCols)) return e;
  k_ln_join<<<join, 32 * kSlices, 0, s>>>(part, (int)parts, pcols, a.cols, a.dw, a.db, a.accumulate);
  return hipGetLastError();
}

template <typename T, typename W>
hipError_t backward_w(const LnBwdArgs& a, hipStream_t s) {
  return a.x ? backward_ck<T, W, false>(a, s) : backward_ck<T, W, true>(a, s);
}

}  // namespace

size_t layernorm_backward_workspace(int64_t rows, int64_t cols) {
  if (rows == 0 || cols == 0) return 0;
  const size_t parts = align256((size_t)backward_parts(rows, cols) * 2 * (size_t)part_cols(cols) * 4);
  return parts + (cols > kMaxTeamCols ? align256((size_t)rows * 8) : 0);
}

hipError_t launch_layernorm_forward(int dtype, int wdtype, const LnFwdArgs& a, hipStream_t s) {
  if (dtype == GC_F32) return forward_w<float, float>(a, s);
  if (dtype == GC_F16) return wdtype == GC_F32 ? forward_w<f16, float>(a, s) : forward_w<f16, f16>(a, s);
  return wdtype == GC_F32 ? forward_w<bf16, float>(a, s) : forward_w<bf16, bf16>(a, s);
}

hipError_t launch_layernorm_backward(int dtype, int wdtype, const LnBwdArgs& a, hipStream_t s) {
  if (dtype == GC_F32) return backward_w<float, float>(a, s);
  if (dtype == GC_F16) return wdtype == GC_F32 ? backward_w<f16, float>(a, s) : backward_w<f16, f16>(a, s);
  return wdtype == GC_F32 ? backward_w<bf16, float>(a, s) : backward_w<bf16, bf16>(a, s);
}

}  // namespace gc
