// The 8-bit checkpoint by itself, and the MLP activation's forward and backward passes
// around it (gc_ckpt_pack, gc_ckpt_unpack, gc_act_forward, gc_act_backward).
//
// All four are one pass over the matrix in chunks of 8 columns (ckpt_core.hpp), bound by HBM; two chunks of a
// thread are in flight at a time.  Measured over 8192 x 11008 in bf16, one call repeated on three sets of inputs (a copy of
// that size: 5.3 TB/s): pack 43 us, 6.4 TB/s; unpack 43 us, 6.3 TB/s; the GELU forward with x packed 79 to 87 us, 5.2 to 5.7
// TB/s, with x and y packed 98 us, 5.6 TB/s; its backward from the checkpoint 79 us, 5.7 TB/s, from x 95 us, 5.7 TB/s.  SiLU
// and tanh-GELU take 79 to 80 us both ways; fp32 takes 143 to 146 us, and 184 us back from x.  (Pack and unpack in turn take 52
// and 39: the one writes back what the other left in the last-level cache, the other reads its checkpoint there.)  Rows of 1000
// in fp16 (no multiple of 32, so with ragged ends): 3.8 to 5 TB/s.  Small calls are a launch: 2.5 to 4 us on the card.
#include <hip/hip_runtime.h>

#include "ckpt_core.hpp"
#include "gc_train.h"
#include "train_internal.hpp"

namespace gc {
namespace {

constexpr int kThreads = 256;
constexpr int kNone = -1;

// ---------------------------------------------------------------------------------
// The activations, in fp32.  No tail is a difference of larger numbers, so each keeps its relative precision but for the
// rounding of its exponent, which grows with the exponent's size.
//
// GELU.  With z = |x| and Q(z) = 1 - Phi(z) = exp(-z^2/2) * R(t), t = 1 / (1 + 0.23 z): R is
// the scaled complementary error function, smooth in t, fitted here by a polynomial of degree
// 8 with a relative error of 4.8e-8 for z in [0, 14.5].  Phi(x) is Q(z) for x < 0 and 1 - Q(z) otherwise, and
// f'(x) = Phi(x) + x * exp(-x^2/2) / sqrt(2 pi) takes the same exponential.  Q is good to 5e-7 relative up to z = 2; beyond,
// the exponent z^2/2 is rounded twice at its own size, 2^-24 of it each: 2e-6 at z = 5, 8e-6 at z = 11.  That is what
// rounding z itself once costs, and results of 16 bits do not see it.  Past z = 13.2 the hardware's exp2 gives 0:
// x Q(z) and f', which are below 2^-122 there, are 0.
//
// The tanh form is x * p with p = 1 / (1 + exp(-u)), u = 2 sqrt(2/pi) (x + 0.044715 x^3), and
// f' = p + x p (1 - p) u'.  Past |x| = 11.5, p is 0 or 1 and p (1 - p) is 0 in fp32, so x is limited there before
// its cube can overflow.  SiLU is x * p with u = x, f' = p (1 + x (1 - p)); the limit there is 131.  A limit drops a NaN,
// which comes back with the factor x, or by a test.
// ---------------------------------------------------------------------------------
__device__ __forceinline__ float exp2_hw(float a) { return __builtin_amdgcn_exp2f(a); }
__device__ __forceinline__ float rcp_hw(float a) { return __builtin_amdgcn_rcpf(a); }

__device__ __forceinline__ float gelu_tail(float z, float e) {   // Q(z), e = exp(-z^2/2)
  const float t = rcp_hw(__builtin_fmaf(0.23f, z, 1.0f));
  float r = -0.0784842595f;
  r = __builtin_fmaf(r, t, 0.290499419f);
  r = __builtin_fmaf(r, t, -0.278312027f);
  r = __builtin_fmaf(r, t, 0.301696599f);
  r = __builtin_fmaf(r, t, -0.0330849327f);
  r = __builtin_fmaf(r, t, 0.1195895f);
  r = __builtin_fmaf(r, t, 0.0857419595f);
  r = __builtin_fmaf(r, t, 0.0923816785f);
  r = __builtin_fmaf(r, t, -2.79725336e-05f);
  return r * e;
}

constexpr float kLog2e = 1.44269504f;

// 1 / (1 + exp(-u)).  The hardware's exp2 and reciprocal flush results below 2^-126, where f' still multiplies p by some
// hundreds: far out they work on 2^-64 (1 + exp(-u)) instead, and the last product, which does not flush, scales back.
// Only there: the shift rounds the exponent at its own size of 64, 2e-6 of p, where u itself is small (p was
// off by up to 1.4e-6 for |u| < 1 with the shift everywhere).  Past -40 the shifted
// exponent is the smaller one.
//
// The reciprocal takes one Newton step, which leaves it off by about half a step instead of a whole one: with the
// hardware's own, SiLU of 5.9375 in bf16, 1.6 units of 2^-24 from the middle between two results, came out as the other
// one.  The step must meet no Inf: u is at least -131, where p is 0 already.
__device__ __forceinline__ float sigmoid(float u) {
  const bool far = u < -40.0f;
  const float k = far ? 5.42101086e-20f : 1.0f;              // 2^-64
  const float d = k + exp2_hw(__builtin_fmaf(u, -kLog2e, far ? -64.0f : 0.0f));
  const float r = rcp_hw(d);
  return k * __builtin_fmaf(__builtin_fmaf(-d, r, 1.0f), r, r);
}

__device__ __forceinline__ float silu_arg(float x) { return __builtin_amdgcn_fmed3f(x, -131.0f, 131.0f); }

template <int KIND>
__device__ __forceinline__ float act_f(float x) {
  if constexpr (KIND == GC_ACT_GELU) {
    const float z = __builtin_fabsf(x);
    const float q = gelu_tail(z, exp2_hw(z * z * (-0.5f * kLog2e)));
    return x * (x < 0.0f ? q : 1.0f - q);
  } else if constexpr (KIND == GC_ACT_GELU_TANH) {
    const float c = __builtin_amdgcn_fmed3f(x, -11.5f, 11.5f);
    const float u = c * __builtin_fmaf(c * c, 2.0f * 0.79788456f * 0.044715f, 2.0f * 0.79788456f);
    return x * sigmoid(u);
  } else {
    return x * sigmoid(silu_arg(x));
  }
}

template <int KIND>
__device__ __forceinline__ float act_d(float x) {
  if constexpr (KIND == GC_ACT_GELU) {
    const float z = __builtin_fabsf(x);
    const float e = exp2_hw(z * z * (-0.5f * kLog2e));
    const float q = gelu_tail(z, e);
    return __builtin_fmaf(x, e * 0.39894228f, x < 0.0f ? q : 1.0f - q);
  } else if constexpr (KIND == GC_ACT_GELU_TANH) {
    const float c = __builtin_amdgcn_fmed3f(x, -11.5f, 11.5f);
    const float c2 = c * c;
    const float u = c * __builtin_fmaf(c2, 2.0f * 0.79788456f * 0.044715f, 2.0f * 0.79788456f);
    const float du = __builtin_fmaf(c2, 6.0f * 0.79788456f * 0.044715f, 2.0f * 0.79788456f);
    const float p = sigmoid(u);
    const float d = __builtin_fmaf(c * du, p * (1.0f - p), p);
    return x != x ? x : d;          // the limit above drops a NaN
  } else {
    const float p = sigmoid(silu_arg(x));
    return p * __builtin_fmaf(x, 1.0f - p, 1.0f);
  }
}

// ---------------------------------------------------------------------------------
// Chunks.  A matrix whose rows follow each other without gaps, in every array of the call,
// and whose width is a multiple of 32, is one long row (FLAT): no division, no ragged end.
// Otherwise a chunk's row comes from one 64-bit division per block (uniform) and a
// high product per lane.
// ---------------------------------------------------------------------------------
struct Grid {
  int64_t chunks;      // rows * ldc / 8
  int64_t cols;
  uint32_t per_row;    // chunks of one row
  FastDiv div;
};

struct Place {
  int64_t row, col;    // col counts elements; FLAT: row 0, col up to rows * cols
  int n;               // columns of this chunk that exist (<= 0: only padding)
};

template <bool FLAT>
__device__ __forceinline__ Place place(const Grid& g, int64_t base, uint32_t local) {
  Place p;
  if constexpr (FLAT) {
    p.row = 0;
    p.col = (base + local) * kChunk;
    p.n = kChunk;
  } else {
    const int64_t row0 = base / g.per_row;
    const uint32_t t = (uint32_t)(base - row0 * g.per_row) + local;
    const uint32_t r = fast_div(t, g.div);
    p.row = row0 + r;
    p.col = (int64_t)(t - r * g.per_row) * kChunk;
    const int64_t left = g.cols - p.col;
    p.n = left < kChunk ? (int)left : kChunk;
  }
  return p;
}

template <typename T, int KIND, bool FLAT, int U>
__device__ __forceinline__ void act_forward_tile(const ActFwdArgs& a, const Grid& g, int64_t base) {
  Raw8<T> x[U];
  Place p[U];
  bool on[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t local = u * kThreads + threadIdx.x;
    on[u] = base + local < g.chunks;      // the same for the four lanes of a block of 32
    if (!on[u]) continue;
    p[u] = place<FLAT>(g, base, local);
    x[u] = raw8w<T, FLAT>(static_cast<const T*>(a.x) + p[u].row * a.ldx + p[u].col, p[u].n, g.cols);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (!on[u]) continue;
    float v[8];
    tail8<T, FLAT>(x[u], p[u].n, g.cols);
    get8<T>(x[u], v);
    const int64_t chunk = base + u * kThreads + threadIdx.x;
    if (KIND == kNone || a.x_codes) {
      const Packed8 c = pack8<T>(v);
      reinterpret_cast<u32x2*>(a.x_codes)[chunk] = u32x2{c.lo, c.hi};
      if ((chunk & 3) == 0) a.x_exps[chunk >> 2] = (uint8_t)c.e;
    }
    if constexpr (KIND != kNone) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = act_f<KIND>(v[i]);
      store8n(static_cast<T*>(a.y) + p[u].row * a.ldy + p[u].col, FLAT ? kChunk : p[u].n, v);
      if (a.y_codes) {
        round8<T>(v);                  // f(0) = 0: the padding packs as zeros
        const Packed8 c = pack8<T>(v);
        reinterpret_cast<u32x2*>(a.y_codes)[chunk] = u32x2{c.lo, c.hi};
        if ((chunk & 3) == 0) a.y_exps[chunk >> 2] = (uint8_t)c.e;
      }
    }
  }
}

template <typename T, int KIND, bool FLAT, int U>
__global__ __launch_bounds__(kThreads) void k_act_forward(ActFwdArgs a, Grid g) {
  for (int64_t base = (int64_t)blockIdx.x * (kThreads * U); base < g.chunks; base += (int64_t)gridDim.x * (kThreads * U))
    act_forward_tile<T, KIND, FLAT, U>(a, g, base);
}

// dx = dy * f'(x) with x in full or from its checkpoint (CK); KIND == kNone: dx = the
// checkpoint's values.
template <typename T, int KIND, bool CK, bool FLAT, int U>
__device__ __forceinline__ void act_backward_tile(const ActBwdArgs& a, const Grid& g, int64_t base) {
  Raw8<T> d[U], x[U];
  u32x2 c[U];
  uint32_t e[U];
  Place p[U];
  bool on[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t local = u * kThreads + threadIdx.x;
    on[u] = base + local < g.chunks;
    if (!on[u]) continue;
    p[u] = place<FLAT>(g, base, local);
    if (!FLAT && p[u].n <= 0) { on[u] = false; continue; }
    if constexpr (CK) {
      c[u] = reinterpret_cast<const u32x2*>(a.x_codes)[base + local];
      e[u] = a.x_exps[(base + local) >> 2];
    } else {
      x[u] = raw8w<T, FLAT>(static_cast<const T*>(a.x) + p[u].row * a.ldx + p[u].col, p[u].n, g.cols);
    }
    if constexpr (KIND != kNone) d[u] = raw8w<T, FLAT>(static_cast<const T*>(a.dy) + p[u].row * a.lddy + p[u].col, p[u].n, g.cols);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (!on[u]) continue;
    float v[8];
    if constexpr (CK) {
      decode8(c[u][0], c[u][1], ckpt_step(e[u]), v);
    } else {
      tail8<T, FLAT>(x[u], p[u].n, g.cols);
      get8<T>(x[u], v);
    }
    if constexpr (KIND != kNone) {
      float t[8];
      tail8<T, FLAT>(d[u], p[u].n, g.cols);
      get8<T>(d[u], t);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = t[i] * act_d<KIND>(v[i]);
    }
    store8n(static_cast<T*>(a.dx) + p[u].row * a.lddx + p[u].col, FLAT ? kChunk : p[u].n, v);
  }
}

template <typename T, int KIND, bool CK, bool FLAT, int U>
__global__ __launch_bounds__(kThreads) void k_act_backward(ActBwdArgs a, Grid g) {
  for (int64_t base = (int64_t)blockIdx.x * (kThreads * U); base < g.chunks; base += (int64_t)gridDim.x * (kThreads * U))
    act_backward_tile<T, KIND, CK, FLAT, U>(a, g, base);
}

// A grid of at most 2^23 blocks (a dimension holds fewer than 2^32 threads); larger matrices loop.
unsigned blocks_for(int64_t chunks, int per_block) {
  const int64_t b = (chunks + per_block - 1) / per_block;
  return (unsigned)(b < (int64_t(1) << 23) ? b : (int64_t(1) << 23));
}

Grid grid_of(int64_t rows, int64_t cols, bool flat) {
  Grid g;
  g.cols = cols;
  const int64_t per_row = (cols + kBlockCols - 1) / kBlockCols * (kBlockCols / kChunk);
  g.chunks = rows * per_row;
  g.per_row = (uint32_t)(flat ? 1 : per_row);
  uint32_t s = 0;
  while ((uint64_t(1) << s) < g.per_row) ++s;
  g.div.d = g.per_row;
  g.div.magic = g.per_row > 1 ? (uint32_t)((uint64_t(1) << (31 + s)) / g.per_row + 1) : 0u;
  g.div.shift = s > 0 ? s - 1 : 0;
  return g;
}

template <typename T, int KIND>
hipError_t forward_t(const ActFwdArgs& a, hipStream_t s) {
  const bool flat = a.cols % kBlockCols == 0 && (a.rows == 1 || (a.ldx == a.cols && (!a.y || a.ldy == a.cols)));
  const Grid g = grid_of(a.rows, a.cols, flat);
  constexpr int U = 2;
  const unsigned blocks = blocks_for(g.chunks, kThreads * U);
  if (flat) k_act_forward<T, KIND, true, U><<<blocks, kThreads, 0, s>>>(a, g);
  else k_act_forward<T, KIND, false, U><<<blocks, kThreads, 0, s>>>(a, g);
  return hipGetLastError();
}

template <typename T, int KIND, bool CK>
hipError_t backward_t(const ActBwdArgs& a, hipStream_t s) {
  const bool flat = a.cols % kBlockCols == 0 &&
                    (a.rows == 1 || ((KIND == kNone || a.lddy == a.cols) && (CK || a.ldx == a.cols) && a.lddx == a.cols));
  const Grid g = grid_of(a.rows, a.cols, flat);
  constexpr int U = 2;
  const unsigned blocks = blocks_for(g.chunks, kThreads * U);
  if (flat) k_act_backward<T, KIND, CK, true, U><<<blocks, kThreads, 0, s>>>(a, g);
  else k_act_backward<T, KIND, CK, false, U><<<blocks, kThreads, 0, s>>>(a, g);
  return hipGetLastError();
}

template <typename T>
hipError_t forward_k(int kind, const ActFwdArgs& a, hipStream_t s) {
  switch (kind) {
    case GC_ACT_GELU: return forward_t<T, GC_ACT_GELU>(a, s);
    case GC_ACT_GELU_TANH: return forward_t<T, GC_ACT_GELU_TANH>(a, s);
    case GC_ACT_SILU: return forward_t<T, GC_ACT_SILU>(a, s);
    default: return forward_t<T, kNone>(a, s);
  }
}

template <typename T>
hipError_t backward_k(int kind, const ActBwdArgs& a, hipStream_t s) {
  const bool ck = a.x == nullptr;
  switch (kind) {
    case GC_ACT_GELU: return ck ? backward_t<T, GC_ACT_GELU, true>(a, s) : backward_t<T, GC_ACT_GELU, false>(a, s);
    case GC_ACT_GELU_TANH:
      return ck ? backward_t<T, GC_ACT_GELU_TANH, true>(a, s) : backward_t<T, GC_ACT_GELU_TANH, false>(a, s);
    case GC_ACT_SILU: return ck ? backward_t<T, GC_ACT_SILU, true>(a, s) : backward_t<T, GC_ACT_SILU, false>(a, s);
    default: return backward_t<T, kNone, true>(a, s);
  }
}

}  // namespace

hipError_t launch_act_forward(int dtype, int kind, const ActFwdArgs& a, hipStream_t s) {
  switch (dtype) {
    case GC_F32: return forward_k<float>(kind, a, s);
    case GC_F16: return forward_k<f16>(kind, a, s);
    default: return forward_k<bf16>(kind, a, s);
  }
}

hipError_t launch_act_backward(int dtype, int kind, const ActBwdArgs& a, hipStream_t s) {
  switch (dtype) {
    case GC_F32: return backward_k<float>(kind, a, s);
    case GC_F16: return backward_k<f16>(kind, a, s);
    default: return backward_k<bf16>(kind, a, s);
  }
}

}  // namespace gc
