// The weight gradient of a linear layer from the 8-bit checkpoint of its input
// (gc_linear_wgrad): dw = dy^T x, out x in, summed over the rows (tokens) on the matrix cores.
//
// Both factors have the summed dimension as their slow one, so their tiles go to LDS as they
// lie in memory ([row][column], 16 bits) and the fragments come out through the transposing
// LDS read of gfx950 (ds_read_b64_tr_b16: 16 lanes read 4 rows of 16 columns, each lane
// receives one column's 4 rows).  Rows k .. k + 3 of a read lie at the same bank offset, so
// the 64-byte segments of row k are permuted by xor with k % 4: the four rows then cover all
// 64 banks.
//
// Exactness.  A code times its power of two is exact in bf16 (8 significant bits; in fp16 for
// checkpoints of fp16 values), so the products are exact and the only rounding is the fp32
// accumulation.  An fp32 dy is cut into three bf16 parts whose sum is dy (8 significant bits each, down to 2^-133): three
// matrix instructions at the bf16 rate instead of one at the fp32 rate, which is a sixteenth of it.
//
// Measured, with db (fastest of repeated calls, 8-bit checkpoint of the same type; the range is that of several cards):
//   bf16  rows 4096, 4096 x 4096:   123 to 131 us, 1050 to 1120 TFLOP/s      rows 8192, 11008 x 4096:  642 to 703 us, 1050 to 1150 TFLOP/s
//   fp32  rows 4096, 4096 x 4096:   335 to 355 us,  390 to 410 TFLOP/s (three times that of bf16 products)
//   bf16  rows 32, 1024 x 1024:     10 us, a launch and its call      fp32  rows 1000, 1333 x 999:  29 us
// Added to what is there, the first two take 187 and 933 us: every row of a wave's tile waits for its own read.
// Large products use half of the matrix cycles, at the clock that the card holds under them (about 2.1 GHz of 2.4).  By the
// counters, of the time of the one wave of a SIMD, products take 58%; for 19% it waits for memory, LDS or the barrier, and for 27% it
// has an instruction that does not issue, partly behind a product.  Beside each product it issues 2.6 vector, 1.25 LDS and one
// other instruction.  LDS is not the limit by its rate: it is active in a quarter of the cycles, without bank conflicts.
// All-zero inputs run 15% faster for their power alone, and inputs that stay in the caches 5% faster.  Small
// products are bound by the latency of a stage's loads and by storing the shares' sums.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "ckpt_core.hpp"
#include "gc_train.h"
#include "internal.hpp"
#include "train_internal.hpp"

namespace gc {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kThreads = 256;

template <typename T>
constexpr int parts() { return sizeof(T) == 4 ? 3 : 1; }

template <typename T>
__device__ __forceinline__ f32x16 mfma(s16x8 a, s16x8 b, f32x16 c) {
  if constexpr (__is_same(T, f16))
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// 8 codes as 16-bit values of the product's type.
template <typename T>
__device__ __forceinline__ u32x4 decode16(u32x2 c, uint32_t e) {
  typedef typename std::conditional<__is_same(T, f16), f16, bf16>::type H;
  typedef H h8 __attribute__((ext_vector_type(8)));
  float v[8];
  decode8(c[0], c[1], ckpt_step(e), v);
  h8 h;
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = (H)v[i];
  return __builtin_bit_cast(u32x4, h);
}

// dy's chunk as the product's planes of 16-bit values.  fp32: each part is the value's
// leading 8 bits cut off (no rounding), so the remainders are exact.  A chunk with an Inf or a NaN, which would leave
// NaN remainders of an Inf, is taken apart again with those values whole in the first part.
template <typename T>
__device__ __forceinline__ void planes(const Raw8<T>& r, u32x4 out[parts<T>()]) {
  if constexpr (sizeof(T) == 2) {
    out[0] = r.q[0];
  } else {
    float v[8];
    get8<T>(r, v);
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) most = max(most, mag_key(v[i]));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float r0 = v[2 * i] - bitsf(fbits(v[2 * i]) & 0xFFFF0000u), r1 = v[2 * i + 1] - bitsf(fbits(v[2 * i + 1]) & 0xFFFF0000u);
      const float l0 = r0 - bitsf(fbits(r0) & 0xFFFF0000u), l1 = r1 - bitsf(fbits(r1) & 0xFFFF0000u);
      // the upper halves of two words, which are the parts themselves
      out[0][i] = __builtin_amdgcn_perm(fbits(v[2 * i + 1]), fbits(v[2 * i]), 0x07060302u);
      out[1][i] = __builtin_amdgcn_perm(fbits(r1), fbits(r0), 0x07060302u);
      out[2][i] = __builtin_amdgcn_perm(fbits(l1), fbits(l0), 0x07060302u);
    }
    if (__ballot(most >= 0x7F800000u)) {        // the same for the wave: skipped, not masked
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t keep = (i & 1) ? 0x0000FFFFu : 0xFFFF0000u;        // the other value of the word
        if (mag_key(v[i]) >= 0x7F800000u) {
          const uint32_t top = v[i] != v[i] ? 0x7FC0u : fbits(v[i]) >> 16;
          out[0][i >> 1] = (out[0][i >> 1] & keep) | ((i & 1) ? top << 16 : top);
          out[1][i >> 1] &= keep;
          out[2][i >> 1] &= keep;
        }
      }
    }
  }
}

// Byte offset of columns [8 c, 8 c + 8) of row k in a staged tile COLS wide.
template <int COLS>
__device__ __forceinline__ int stage_at(int k, int c) {
  return k * (2 * COLS) + ((c * 16) ^ ((COLS >= 128 ? k & 3 : (k >> 1) & 1) << 6));
}

__device__ __forceinline__ s16x4 read_tr(const char* lds, int at) {
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lds + at));
}

// Tile and share of the rows of block b.  Blocks go to the 8 XCDs in turn; every XCD gets a contiguous run of
// the tiles, share by share, ordered in bands of `band` output tiles, so that its L2 serves a compact patch.  (In
// plain order every XCD would read all of dy.)
struct TileMap {
  int tiles_i, tiles_o, band, shares;
};
struct Tile {
  int i, o, share;
};
__device__ __forceinline__ Tile tile_of(const TileMap& m, int b) {
  const int tiles = m.tiles_i * m.tiles_o, total = tiles * m.shares, q = total >> 3, r = total & 7, x = b & 7;
  const int at = x * q + (x < r ? x : r) + (b >> 3), t = at % tiles;
  const int width = m.band * m.tiles_i, first = t / width * m.band, in = t % width;
  const int high = m.tiles_o - first < m.band ? m.tiles_o - first : m.band;
  // the divisions run in vector registers
  return {__builtin_amdgcn_readfirstlane(in / high), __builtin_amdgcn_readfirstlane(first + in % high),
          __builtin_amdgcn_readfirstlane(at / tiles)};
}

// Row stride of the shares' sums: whole cache lines, and a ragged last tile of the large kernel stores its padding too.
__host__ __device__ __forceinline__ int64_t part_ld(int64_t in) { return (in + kBlockCols - 1) / kBlockCols * kBlockCols; }

// ---- any product ----------------------------------------------------------------------------
//
// TILE x TILE outputs per block of four waves, ROWS rows per stage, one stage in LDS and the next one in flight
// in registers.  Products that come here are small: what they wait for is memory, once per stage, so the
// stages are as long as LDS allows, 64 rows of a 128 tile or 128 rows of a 64 tile: 32 KB, and 64 KB
// with fp32's three planes, for two blocks per CU and more.  (Stages of 32 rows took 17 us, not 11, for 300 rows of
// 400 x 400.)
//
// One block per tile and share of the rows (`share` rows each).  With more than one share, share z writes its
// sums to part + z * out * part_ld(in) (and its db to dbpart + z * out) for k_wgrad_join.
template <int TILE>
constexpr int stage_rows() { return 8192 / TILE; }

template <typename T, int TILE>
__global__ __launch_bounds__(kThreads, 2) void k_wgrad(WgradArgs a, TileMap map, int64_t share, float* part, float* dbpart) {
  constexpr int P = parts<T>(), ROWS = stage_rows<TILE>(), CH = TILE / kChunk, STEP = kThreads / CH, N = ROWS / STEP;
  constexpr int W = TILE / 64;         // 32 x 32 products of a wave, each way
  __shared__ __attribute__((aligned(16))) char s_a[P][ROWS * TILE * 2];
  __shared__ __attribute__((aligned(16))) char s_b[ROWS * TILE * 2];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const Tile tile = tile_of(map, blockIdx.x);
  const int64_t i0 = (int64_t)tile.i * TILE, o0 = (int64_t)tile.o * TILE;
  const int64_t m_begin = (int64_t)tile.share * share;
  const int64_t m_end = m_begin + share < a.rows ? m_begin + share : a.rows;
  const int64_t ldc = (a.in + kBlockCols - 1) / kBlockCols * kBlockCols;
  const bool with_db = tile.i == 0 && a.db;
  const bool whole = o0 + TILE <= a.out && i0 + TILE <= ldc;

  // staging: thread t moves chunk t % CH of rows t / CH + STEP u of both tiles
  const int k0 = tid / CH, c0 = tid % CH;
  const int64_t o = o0 + c0 * kChunk, i = i0 + c0 * kChunk;
  const int n = a.out - o < kChunk ? (int)(a.out - o) : kChunk;
  Raw8<T> ra[N];
  u32x2 rb[N];
  uint32_t re[N];
  const auto fetch = [&](int64_t m0) {
    const T* pa = static_cast<const T*>(a.dy) + (m0 + k0) * a.lddy + o;
    const int8_t* pb = a.codes + (m0 + k0) * ldc + i;
    const uint8_t* pe = a.exps + (m0 + k0) * (ldc >> 5) + (i >> 5);
    if (whole && m0 + ROWS <= m_end) {
#pragma unroll
      for (int u = 0; u < N; ++u) {
        ra[u] = raw8(pa + u * STEP * a.lddy);
        rb[u] = *reinterpret_cast<const u32x2*>(pb + u * STEP * ldc);
        re[u] = pe[u * STEP * (ldc >> 5)];
      }
    } else {
#pragma unroll
      for (int u = 0; u < N; ++u) {
        const bool on = m0 + k0 + u * STEP < m_end;
        ra[u] = raw8n(pa + u * STEP * a.lddy, on ? n : 0, a.out);
        rb[u] = u32x2{0u, 0u};
        re[u] = 7u;
        if (on && i < ldc) {
          rb[u] = *reinterpret_cast<const u32x2*>(pb + u * STEP * ldc);
          re[u] = pe[u * STEP * (ldc >> 5)];
        }
      }
    }
  };
  const auto stage = [&]() {
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int at = stage_at<TILE>(k0 + STEP * u, c0);
      u32x4 pl[P];
      if (!whole) tail8<T>(ra[u], n, a.out);      // a cleared row stays cleared
      planes<T>(ra[u], pl);
#pragma unroll
      for (int p = 0; p < P; ++p) *reinterpret_cast<u32x4*>(&s_a[p][at]) = pl[p];
      *reinterpret_cast<u32x4*>(&s_b[at]) = decode16<T>(rb[u], re[u]);
    }
  };

  // fragments: lane l of a 32 x 32 x 16 product holds column l % 32 and rows 8 (l / 32) ..
  // + 7; its 16-lane group reads 4 of those rows at a time
  const int wo = (wave & 1) * 32 * W, wi = (wave >> 1) * 32 * W;
  const int g = lane >> 4, r4 = (lane & 15) >> 2, col = (g & 1) * 16 + (lane & 3) * 4;
  int at_a[W], at_b[W];                // of the first 16 rows; 16 rows on the permutation is the same
#pragma unroll
  for (int t = 0; t < W; ++t) {
    at_a[t] = stage_at<TILE>((g >> 1) * 8 + r4, (wo + 32 * t + col) >> 3) + (col & 4) * 2;
    at_b[t] = stage_at<TILE>((g >> 1) * 8 + r4, (wi + 32 * t + col) >> 3) + (col & 4) * 2;
  }
  const auto frag = [&](const char* lds, int at, int kk) -> s16x8 {
    const s16x4 lo = read_tr(lds, at + kk * 16 * (2 * TILE)), hi = read_tr(lds, at + (kk * 16 + 4) * (2 * TILE));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };

  f32x16 acc[W][W] = {}, accb[W] = {};
  const uint16_t one16 = __is_same(T, f16) ? 0x3C00 : 0x3F80;
  s16x8 ones;
#pragma unroll
  for (int k = 0; k < 8; ++k) ones[k] = (short)one16;

  fetch(m_begin);
  for (int64_t m0 = m_begin; m0 < m_end; m0 += ROWS) {
    __syncthreads();
    stage();
    __syncthreads();
    if (m0 + ROWS < m_end) fetch(m0 + ROWS);
#pragma unroll(W == 1 ? ROWS / 16 : 2)
    for (int kk = 0; kk < ROWS / 16; ++kk) {
      s16x8 b[W];
#pragma unroll
      for (int u = 0; u < W; ++u) b[u] = frag(s_b, at_b[u], kk);
#pragma unroll
      for (int p = 0; p < P; ++p) {
#pragma unroll
        for (int t = 0; t < W; ++t) {
          const s16x8 f = frag(s_a[p], at_a[t], kk);
#pragma unroll
          for (int u = 0; u < W; ++u) acc[t][u] = mfma<T>(f, b[u], acc[t][u]);
          if (with_db && wi == 0) accb[t] = mfma<T>(f, ones, accb[t]);
        }
      }
    }
  }

  float* out = part ? part + (int64_t)tile.share * a.out * part_ld(a.in) : a.dw;
  const int64_t ld = part ? part_ld(a.in) : a.lddw;
  const bool add = !part && a.accumulate;
#pragma unroll
  for (int t = 0; t < W; ++t) {
#pragma unroll
    for (int u = 0; u < W; ++u) {
      const int64_t ii = i0 + wi + 32 * u + (lane & 31);
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int64_t oo = o0 + wo + 32 * t + (r >> 2) * 8 + (lane >> 5) * 4 + (r & 3);
        if (oo < a.out && ii < a.in) {
          float* d = out + oo * ld + ii;
          *d = add ? *d + acc[t][u][r] : acc[t][u][r];
        }
      }
    }
    if (with_db && wi == 0 && (lane & 31) == 0) {
      float* db = dbpart ? dbpart + (int64_t)tile.share * a.out : a.db;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int64_t oo = o0 + wo + 32 * t + (r >> 2) * 8 + (lane >> 5) * 4 + (r & 3);
        if (oo < a.out) db[oo] = add ? db[oo] + accb[t][r] : accb[t][r];
      }
    }
  }
}

// ---- large products ------------------------------------------------------------------------
//
// 256 x 256 outputs per block of four waves, one wave per SIMD with a 128 x 128 quarter in 256
// accumulation registers: each fragment read from LDS feeds four products, which
// is what keeps LDS (128 fragment reads and 64 KB written and read per stage) below the
// matrix cores' time.  With one wave per SIMD nothing else fills a stall, so the order of the instructions is
// fixed by hand (the compiler's own order took 151 us, not 123, for 4096 rows of 4096 x 4096, and 256 x 128 tiles with
// two blocks per CU 158): a stage of 32 rows is two halves of 16 slots of one 32 x 32 x 16 product (32 cycles),
// and every slot carries a share of the rest (about five instructions, four cycles each).
//
// fp32: 128 outputs x 256 inputs, 24 slots a half, since each product of a pair of tiles is three (one per
// plane of dy); the cutting of dy into planes is part of the slots' other work.
constexpr int kBigI = 256;
template <typename T>
constexpr int big_o() { return sizeof(T) == 4 ? 128 : 256; }
constexpr int kRows = 32;                   // rows of one stage
constexpr int kBufs = 3;

// Byte offset of columns [8 c, 8 c + 8) of row k in a staged tile COLS wide.  Segments of 64 bytes are
// permuted by k % 4 for the transposing reads.  Inside a segment the chunks are permuted by the pair of
// segments they are in: 8 lanes write their chunk j of 8 consecutive segments at a time (128 bytes a cycle), which
// then lie in 8 different 16-byte columns of the banks.
template <int COLS>
__device__ __forceinline__ int big_at(int k, int c) {
  return k * (2 * COLS) + ((c ^ ((k & 3) << 2) ^ ((c >> 3) & 3)) << 4);
}

// No load of this kernel is conditional, so that a stage is one run of straight code that
// the products can be spread over: the last tile of either side is moved back to end with the matrix (its
// overlap is computed twice and stored once), and so is the last stage (its rows that
// were already taken are cleared).  The launcher asks for at least one tile and one stage.
struct BigPlace {          // rows and features fit 32 bits, and stay scalar there
  int i0, o0;              // where the tile reads
  int skip_i, skip_o;      // outputs before these belong to the tile before
  int m_begin, m_end;
};

// db: the tiles of one band of outputs read the same part of dy, so they share its sums out by stages: tile
// ti adds up the stages ti, ti + tiles_i, ...  A stage's sums are 64 vector instructions apart from the
// slots, paid by a block once in tiles_i stages; all of them on one block of the band made that block, and a launch
// of one round of blocks with it, 6 to 8% longer.  k_wgrad_join adds the tiles' sums.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_wgrad_big(WgradArgs a, TileMap map, int64_t share, float* part, float* dbpart) {
  constexpr bool F32 = sizeof(T) == 4;
  constexpr int P = parts<T>(), BO = big_o<T>(), TO = BO / 64, TI = kBigI / 64;   // 32 x 32 products of a wave
  constexpr int CA = BO / kChunk, RA = kThreads / CA, NA = kRows / RA, QA = sizeof(T) / 2;
  constexpr int kStageA = kRows * BO * 2, kStageB = kRows * kBigI * 2;            // bytes of a staged plane
  __shared__ __attribute__((aligned(16))) char s_a[kBufs * P * kStageA];
  __shared__ __attribute__((aligned(16))) char s_b[kBufs * kStageB];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Tile tile = tile_of(map, blockIdx.x);
  const int ti = tile.i, to = tile.o;
  const int ldc = (int)(a.in + kBlockCols - 1) / kBlockCols * kBlockCols, rows = (int)a.rows;
  BigPlace at;
  at.i0 = min(ti * kBigI, ldc - kBigI);
  at.o0 = min(to * BO, (int)a.out - BO);
  at.skip_i = ti * kBigI - at.i0;
  at.skip_o = to * BO - at.o0;
  at.m_begin = tile.share * (int)share;
  at.m_end = rows - at.m_begin < (int)share ? rows : at.m_begin + (int)share;
  const int stages = (at.m_end - at.m_begin + kRows - 1) / kRows;

  // Staging: thread t moves chunk t % CA of dy in rows t / CA + RA u (QA 16-byte loads each, four in all), and
  // the block of 32 codes t % 8 of row t / 8, which has one exponent.  Stage 0 is the last 32 rows; the others start
  // at the first row and stop short of it, so stage 0 alone has rows to clear.
  const int ka = tid / CA, ca = tid % CA, kb = tid >> 3, gb = tid & 7;
  uint32_t off_a[4], off_b, off_e;
#pragma unroll
  for (int n = 0; n < 4; ++n) off_a[n] = (uint32_t)((ka + RA * (n / QA)) * a.lddy + ca * kChunk) * (uint32_t)sizeof(T) + 16u * (n % QA);
  off_b = (uint32_t)(kb * ldc + gb * kBlockCols);
  off_e = (uint32_t)(kb * (ldc >> 5) + gb);
  int put_b[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) put_b[j] = big_at<kBigI>(kb, 4 * gb + j);
  const int put_a = big_at<BO>(ka, ca);      // RA rows on, k % 4 is the same
  typedef const __attribute__((address_space(1))) char* Global;
  Global pa = (Global)(static_cast<const T*>(a.dy) + (int64_t)(at.m_end - kRows) * a.lddy + at.o0);
  Global pb = (Global)(a.codes + (int64_t)(at.m_end - kRows) * ldc + at.i0);
  Global pe = (Global)(a.exps + (int64_t)(at.m_end - kRows) * (ldc >> 5) + (at.i0 >> 5));
  struct Stage {
    u32x4 a[4], b[2];
    uint32_t e;
  };
  // load n = 0 .. 6 of the stage that the pointers are at.  The uniform bases stay in scalar registers and
  // the offsets 32 bits wide: the compiler would otherwise keep seven 64-bit lane addresses.
  const auto load = [&](Stage& s, int n) {
    if (n < 4) {
      asm volatile("" : "+s"(pa), "+v"(off_a[n]));
      s.a[n] = ((const __attribute__((address_space(1))) Quad<sizeof(T)>*)(pa + off_a[n]))->v;
    } else if (n < 6) {
      asm volatile("" : "+s"(pb), "+v"(off_b));
      s.b[n - 4] = *(const __attribute__((address_space(1))) u32x4*)(pb + off_b + 16 * (n - 4));
    } else {
      asm volatile("" : "+s"(pe), "+v"(off_e));
      s.e = *(const __attribute__((address_space(1))) uint8_t*)(pe + off_e);
    }
  };
  const auto fetch = [&](Stage& s) {
#pragma unroll
    for (int n = 6; n >= 0; --n) load(s, n);
  };
  const uint32_t step_a = (uint32_t)(kRows * a.lddy) * (uint32_t)sizeof(T), step_b = (uint32_t)(kRows * ldc), step_e = (uint32_t)ldc;
  const auto advance = [&](bool more) {      // to the next stage; past the last one, nowhere
    pa += more ? step_a : 0u;
    pb += more ? step_b : 0u;
    pe += more ? step_e : 0u;
  };
  const auto rewind = [&]() {                // from stage 0 to stage 1
    const int64_t back = at.m_end - kRows - at.m_begin;
    pa -= back * a.lddy * (int64_t)sizeof(T);
    pb -= back * ldc;
    pe -= back * (ldc >> 5);
  };

  // The pieces of a stage's way to LDS: codes 2 p and 2 p + 1 of the thread's 32, the write of chunk j of
  // them, the write of dy's chunk u, two of that chunk's values into the sums.
  typedef typename std::conditional<__is_same(T, f16), f16, bf16>::type H;
  typedef H h2 __attribute__((ext_vector_type(2)));
  float step = 0.0f;
  u32x4 piece;
  const auto decode2 = [&](const Stage& s, int p) {
    const uint32_t c = s.b[p >> 3][(p >> 1) & 3];
    const int sh = 16 * (p & 1);
    h2 h;
    h[0] = (H)((float)(int)__builtin_amdgcn_sbfe(c, sh, 8) * step);
    h[1] = (H)((float)(int)__builtin_amdgcn_sbfe(c, sh + 8, 8) * step);
    piece[p & 3] = __builtin_bit_cast(uint32_t, h);
  };
  const auto write_b = [&](int buf, int j) { *reinterpret_cast<u32x4*>(&s_b[buf * kStageB + put_b[j]]) = piece; };
  // fp32: values 2 i and 2 i + 1 of dy's chunk u, cut as in planes(); the remainder of an Inf is 0, and that of a
  // NaN, whose upper half alone may read as an Inf, a NaN.
  u32x4 cut[P];
  const auto cut2 = [&](const Stage& s, int u, int i) {
    if constexpr (F32) {
      uint32_t w[3][2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float x = bitsf(s.a[2 * u + (i >> 1)][2 * (i & 1) + k]);
        const float d = x - bitsf(fbits(x) & 0xFFFF0000u);
        const float r = __builtin_fabsf(x) == __builtin_inff() ? 0.0f : d;
        w[0][k] = fbits(x);
        w[1][k] = fbits(r);
        w[2][k] = fbits(r - bitsf(fbits(r) & 0xFFFF0000u));
      }
#pragma unroll
      for (int p = 0; p < 3; ++p) cut[p][i] = __builtin_amdgcn_perm(w[p][1], w[p][0], 0x07060302u);
    }
  };
  const auto write_a = [&](const Stage& s, int buf, int u, int p) {
    *reinterpret_cast<u32x4*>(&s_a[(buf * P + p) * kStageA + put_a + u * RA * 2 * BO]) = F32 ? cut[p] : s.a[u];
  };
  float sums[8] = {};
  const auto add_up = [&](const Stage& s) {
#pragma unroll
    for (int u = 0; u < NA; ++u) {
      Raw8<T> r;
#pragma unroll
      for (int q = 0; q < QA; ++q) r.q[q] = s.a[u * QA + q];
      float v[8];
      get8<T>(r, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) sums[i] += v[i];
    }
  };

  const int wo = (wave & 1) * 32 * TO, wi = (wave >> 1) * 32 * TI;
  const int g = lane >> 4, r4 = (lane & 15) >> 2;
  const int row = (g >> 1) * 8 + r4, col = (g & 1) * 16 + (lane & 3) * 4;
  int at_a[TO], at_b[TI];
#pragma unroll
  for (int t = 0; t < TO; ++t) at_a[t] = big_at<BO>(row, (wo + 32 * t + col) >> 3) + (col & 4) * 2;
#pragma unroll
  for (int t = 0; t < TI; ++t) at_b[t] = big_at<kBigI>(row, (wi + 32 * t + col) >> 3) + (col & 4) * 2;
  struct Frags {
    s16x4 a[TO][P][2], b[TI][2];
  };
  // read n of the fragments of half kk: the inputs' first, then the outputs', plane by plane
  constexpr int READS = 2 * TI + 2 * TO * P;
  const auto read = [&](Frags& f, int buf, int kk, int n) {
    if (n < 2 * TI) {
      f.b[n >> 1][n & 1] = read_tr(s_b, at_b[n >> 1] + buf * kStageB + (kk * 16 + (n & 1) * 4) * (2 * kBigI));
    } else {
      const int m = n - 2 * TI, t = m / (2 * P), p = (m >> 1) % P;
      f.a[t][p][m & 1] = read_tr(s_a, at_a[t] + (buf * P + p) * kStageA + (kk * 16 + (m & 1) * 4) * (2 * BO));
    }
  };
  f32x16 acc[TO][TI] = {};
  const auto product = [&](const Frags& f, int t, int p, int u) {
    acc[t][u] = mfma<T>(__builtin_shufflevector(f.a[t][p][0], f.a[t][p][1], 0, 1, 2, 3, 4, 5, 6, 7),
                        __builtin_shufflevector(f.b[u][0], f.b[u][1], 0, 1, 2, 3, 4, 5, 6, 7), acc[t][u]);
  };

  // Half a round: the SLOTS products of `use`; the reads of `get`; the half h of `st` (its codes 16 h .. + 15, half
  // of dy's chunks) to buffer `to`; and, with `into`, the loads of a later stage.
  constexpr int SLOTS = TO * TI * P, EACH = SLOTS / 8;
  const auto half = [&](const Frags& use, Frags& get, int from, int kk, const Stage& st, int h, int to, Stage* into) {
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      product(use, i / (TI * P), (i / TI) % P, i % TI);
      if (i < 4) {
        read(get, from, kk, 2 * i);
        read(get, from, kk, 2 * i + 1);
      } else if (i + 4 < READS) {
        read(get, from, kk, i + 4);
      }
      if (h == 0 && i == 0) step = ckpt_step(st.e);
      if (i % EACH == 0) decode2(st, 8 * h + i / EACH);
      if (i % (4 * EACH) == 3 * EACH) write_b(to, 2 * h + i / (4 * EACH));
      if constexpr (F32) {
        if (i % 3 == 1 && i <= 10) cut2(st, h, i / 3);
        if (i % 3 == 1 && i >= 13 && i <= 19) write_a(st, to, h, (i - 13) / 3);
      } else {
        if ((i & 7) == 3) write_a(st, to, 2 * h + (i >> 3), 0);
      }
      if (into && i >= SLOTS - 8 && i <= SLOTS - 2) load(*into, SLOTS - 2 - i);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  const auto put = [&](const Stage& st, int to) {       // a whole stage, before the first round
    step = ckpt_step(st.e);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int p = 0; p < 4; ++p) decode2(st, 4 * j + p);
      write_b(to, j);
    }
#pragma unroll
    for (int u = 0; u < NA; ++u) {
#pragma unroll
      for (int i = 0; i < 4; ++i) cut2(st, u, i);
#pragma unroll
      for (int p = 0; p < P; ++p) write_a(st, to, u, p);
    }
  };

  // Stage s has register set and LDS buffer s % 3.  Round s multiplies stage s, writes stage s + 2 and loads
  // s + 4, which has two rounds (about 2000 cycles) to arrive.  Its one barrier, between the halves, says that
  // every wave has read stage s, whose buffer the next round overwrites, and has written stage s + 1.
  // What is loaded and written of stages past the last is the last one again, never multiplied or summed.
  int turn = dbpart ? ti : -1;       // the next stage that this tile adds up; never, without db
  Stage st0, st1, st2;
  Frags f0, f1;
  fetch(st0);
  if (stages > 1) rewind();
  fetch(st1);
  advance(2 < stages);
  fetch(st2);
  const int taken = stages * kRows - (at.m_end - at.m_begin);   // of stage 0's rows, by the stages after it
#pragma unroll
  for (int n = 0; n < 4; ++n) st0.a[n] = ka + RA * (n / QA) >= taken ? st0.a[n] : u32x4{0u, 0u, 0u, 0u};
  if (turn == 0) {
    add_up(st0);
    turn += map.tiles_i;
  }
  put(st0, 0);
  advance(3 < stages);
  fetch(st0);
  if (turn == 1 && 1 < stages) {
    add_up(st1);
    turn += map.tiles_i;
  }
  put(st1, 1);
  __syncthreads();
#pragma unroll
  for (int n = 0; n < READS; ++n) read(f0, 0, 0, n);
  const auto round = [&](Stage& put2, Stage& load4, int s, int buf) {
    if (turn == s + 2 && turn < stages) {
      add_up(put2);
      turn += map.tiles_i;
    }
    advance(s + 4 < stages);
    __builtin_amdgcn_sched_barrier(0);
    half(f0, f1, buf, 1, put2, 0, (buf + 2) % 3, &load4);
    __syncthreads();
    __builtin_amdgcn_sched_barrier(0);
    half(f1, f0, (buf + 1) % 3, 0, put2, 1, (buf + 2) % 3, nullptr);
  };
  int s = 0;
  for (; s + 3 <= stages; s += 3) {
    round(st2, st1, s, 0);
    round(st0, st2, s + 1, 1);
    round(st1, st0, s + 2, 2);
  }
  if (s < stages) round(st2, st1, s, 0);
  if (s + 1 < stages) round(st0, st2, s + 1, 1);

  // The lane's four columns of a row are 32 apart; rows follow the accumulators' layout.  A tile that lies
  // whole in the matrix is stored without a condition (the address: uniform row + lane offset + constant).
  const bool add = !part && a.accumulate;
  const int64_t ld = part ? part_ld(a.in) : a.lddw;
  typedef __attribute__((address_space(1))) char* GlobalOut;
  typedef __attribute__((address_space(1))) float* GlobalF32;
  const int64_t first = (int64_t)(at.o0 + wo) * ld + at.i0;
  float* out = part ? part + (int64_t)tile.share * a.out * part_ld(a.in) : a.dw;
  GlobalOut at_row = (GlobalOut)(out + first);      // the wave's 128 rows, this stride apart
  uint32_t off = (uint32_t)((lane >> 5) * 4 * ld + wi + (lane & 31)) * 4u;
  const auto rows_out = [&](auto&& store4) {
#pragma unroll
    for (int t = 0; t < TO; ++t) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int o = 32 * t + (r >> 2) * 8 + (r & 3);
        GlobalOut p = at_row + (int64_t)o * ld * 4;
        asm volatile("" : "+s"(p), "+v"(off));
        store4(p, o, t, r);
      }
    }
  };
  if (at.skip_i == 0 && at.skip_o == 0 && at.i0 + kBigI <= (part ? ldc : (int)a.in)) {
    if (!add) {
      rows_out([&](GlobalOut p, int, int t, int r) {
#pragma unroll
        for (int u = 0; u < TI; ++u) *(GlobalF32)(p + off + 128 * u) = acc[t][u][r];
      });
    } else {
      rows_out([&](GlobalOut p, int, int t, int r) {
        float v[TI];
#pragma unroll
        for (int u = 0; u < TI; ++u) v[u] = *(GlobalF32)(p + off + 128 * u);
#pragma unroll
        for (int u = 0; u < TI; ++u) *(GlobalF32)(p + off + 128 * u) = v[u] + acc[t][u][r];
      });
    }
  } else {
    const int o_lane = wo + (lane >> 5) * 4, i_lane = wi + (lane & 31);
    rows_out([&](GlobalOut p, int o, int t, int r) {
#pragma unroll
      for (int u = 0; u < TI; ++u) {
        const int i = i_lane + 32 * u;
        GlobalF32 d = (GlobalF32)(p + off + 128 * u);
        float v = acc[t][u][r];
        asm volatile("" : "+v"(v));            // out of the accumulators here, not all of them at the branch
        if (o_lane + o >= at.skip_o && i >= at.skip_i && at.i0 + i < (int)a.in) *d = add ? *d + v : v;
      }
    });
  }
  if (dbpart) {
    // the RA threads of a column chunk through LDS, added in order
    float* x = reinterpret_cast<float*>(s_a);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) x[ka * BO + ca * kChunk + j] = sums[j];
    __syncthreads();
    if (tid < BO && tid >= at.skip_o) {
      float sum = x[tid];
#pragma unroll
      for (int k = 1; k < RA; ++k) sum += x[k * BO + tid];
      dbpart[((int64_t)tile.share * map.tiles_i + ti) * a.out + at.o0 + tid] = sum;
    }
  }
}

// dw[r][c] (row stride ld) = (add ? dw : 0) + the shares' sums in order, in the first dw_blocks blocks (four columns a
// thread), and db = (add ? db : 0) + its parts in order in the others: one launch for both.  Bound by the shares'
// bytes.
__global__ __launch_bounds__(256) void k_wgrad_join(const float* part, int shares, uint32_t dw_blocks, int64_t out, uint32_t in,
                                                    float* dw, int64_t ld, const float* dbpart, int64_t dbs, float* db, int add) {
  if (blockIdx.x < dw_blocks) {
    const uint32_t quads = (in + 3) / 4, g = blockIdx.x * 256u + threadIdx.x, r = g / quads, c = 4 * (g - r * quads);
    if (r >= out) return;
    const int64_t ldp = part_ld(in), n = out * ldp;
    const float* p = part + r * ldp + c;
    float* d = dw + r * ld + c;
    if (c + 4 <= in) {
      const auto quad = [](const float* q) { return __builtin_bit_cast(f32x4, reinterpret_cast<const Quad<4>*>(q)->v); };
      f32x4 sum = quad(p);
#pragma unroll 8
      for (int z = 1; z < shares; ++z) sum += quad(p + z * n);
      if (add) sum = quad(d) + sum;
      reinterpret_cast<Quad<4>*>(d)->v = __builtin_bit_cast(u32x4, sum);
    } else {
      for (uint32_t j = 0; j < in - c; ++j) {
        float sum = p[j];
#pragma unroll 8
        for (int z = 1; z < shares; ++z) sum += p[z * n + j];
        d[j] = add ? d[j] + sum : sum;
      }
    }
  } else {
    const int64_t e = (int64_t)(blockIdx.x - dw_blocks) * 256 + threadIdx.x;
    if (e >= out) return;
    float sum = dbpart[e];
#pragma unroll 8
    for (int64_t z = 1; z < dbs; ++z) sum += dbpart[z * out + e];
    db[e] = add ? db[e] + sum : sum;
  }
}

__global__ __launch_bounds__(256) void k_wgrad_clear(float* dw, int64_t ld, int64_t out, int64_t in, float* db) {
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < out * in; e += (int64_t)gridDim.x * 256) {
    const int64_t r = e / in;
    dw[r * ld + (e - r * in)] = 0.0f;
    if (db && e < out) db[e] = 0.0f;     // in >= 1, so e covers [0, out)
  }
}

constexpr int64_t kMaxSpan = int64_t(1) << 40;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// How a product is cut: which kernel and tile, and shares of the rows.  stride: the larger of dy's and dw's; the
// large kernel's lane offsets have 32 bits.
//  - The large kernel from 128 of its tiles on, with one or two shares for its 256 places (one block per CU), and
//    with more shares where the rows are long enough for 160 of the places and the product is past 2^32
//    multiply-adds (2^30 for fp32, whose three planes triple them).  In us, the large kernel first:
//      bf16  4096 x 2048 x 2048:  59 and 92;   2048 x 1500 x 1500: 38 and 46;   8192 x 512 x 1024 (2^32): 35 and 33
//      fp32  4096 x 1024 x 1024:  39 and 61;   600 x 1300 x 1500:  30 and 42;   1024 x 1024 x 1024 (2^30): 28 and 26
//  - Otherwise tiles of 128 where they fill half of the card, else tiles of 64, and shares until there are about
//    512 blocks, each share at least four stages long: a share less saves four waits on memory, and the
//    joining launch costs about as much.
struct Plan {
  bool big;
  int tile;             // of the inputs, and unless big of the outputs
  int64_t tiles_i, tiles_o, shares, share;
};
Plan plan_for(int dtype, int64_t rows, int64_t in, int64_t out, int64_t stride) {
  Plan p;
  const int64_t wide_o = dtype == GC_F32 ? big_o<float>() : big_o<bf16>();
  const auto tiles = [&](int64_t ti, int64_t to) { return ceil_div(in, ti) * ceil_div(out, to); };
  const double products = (double)rows * (double)in * (double)out;
  const int64_t of_big = tiles(kBigI, wide_o), places = 256, long_rows = ceil_div(rows, 8 * kRows);
  const int64_t blocks = of_big >= places ? of_big : of_big * (places / of_big < long_rows ? places / of_big : long_rows);
  p.big = in > kBigI - kBlockCols && out >= wide_o && rows >= kRows && stride <= (int64_t(1) << 24) &&
          (of_big >= 128 || (blocks >= 160 && products > (dtype == GC_F32 ? 1073741824.0 : 4294967296.0)));
  p.tile = p.big ? kBigI : tiles(128, 128) >= 128 ? 128 : 64;
  p.tiles_i = ceil_div(in, p.tile);
  p.tiles_o = ceil_div(out, p.big ? wide_o : p.tile);
  const int64_t unit = p.big ? kRows : 8192 / p.tile, least = p.big ? 8 * kRows : 4 * unit;
  const int64_t want = (p.big ? 256 : 512) / (p.tiles_i * p.tiles_o), most = ceil_div(rows, least);
  int64_t n = want < most ? want : most;
  n = n < 1 ? 1 : n > 64 ? 64 : n;
  p.share = ceil_div(ceil_div(rows, n), unit) * unit;
  p.shares = ceil_div(rows, p.share);
  return p;
}

unsigned grid_for(int64_t n) {
  const int64_t b = ceil_div(n, 256);
  return (unsigned)(b < (int64_t(1) << 20) ? b : (int64_t(1) << 20));
}

// Sums of db that are joined at the end: one per share, and in the large kernel one per tile of the inputs.
int64_t db_parts(const Plan& p) { return p.big ? p.shares * p.tiles_i : p.shares; }

size_t workspace_of(const Plan& p, int64_t in, int64_t out) {
  const size_t dw = p.shares > 1 ? align256((size_t)p.shares * (size_t)out * (size_t)part_ld(in) * 4) : 0;
  return dw + (db_parts(p) > 1 || p.big ? align256((size_t)db_parts(p) * (size_t)out * 4) : 0);
}

template <typename T>
hipError_t wgrad_t(int dtype, const WgradArgs& a, hipStream_t s) {
  const Plan p = plan_for(dtype, a.rows, a.in, a.out, a.lddy > a.lddw ? a.lddy : a.lddw);
  char* ws = static_cast<char*>(a.ws);
  float* part = p.shares > 1 ? reinterpret_cast<float*>(ws) : nullptr;
  const int64_t dbs = a.db ? db_parts(p) : 0;
  float* dbpart = dbs > 1 || (a.db && p.big) ? reinterpret_cast<float*>(ws + (part ? align256((size_t)p.shares * (size_t)a.out * (size_t)part_ld(a.in) * 4) : 0)) : nullptr;
  // bands four tiles high for the large kernel, whose 32 blocks of an XCD then span 4 x 8 tiles of 2 and 1 bytes
  // per value; eight high for the others, with two to four blocks per CU
  const TileMap map{(int)p.tiles_i, (int)p.tiles_o, p.big ? 4 : 8, (int)p.shares};
  const unsigned blocks = (unsigned)(p.tiles_i * p.tiles_o * p.shares);
  if (p.big) {
    k_wgrad_big<T><<<blocks, kThreads, 0, s>>>(a, map, p.share, part, dbpart);
  } else if (p.tile == 128) {
    k_wgrad<T, 128><<<blocks, kThreads, 0, s>>>(a, map, p.share, part, dbpart);
  } else {
    k_wgrad<T, 64><<<blocks, kThreads, 0, s>>>(a, map, p.share, part, dbpart);
  }
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && (part || dbpart)) {
    // a product in shares has at most 256 tiles of 128 x 128 or 128 of 256 x 256, so its quads fit 32 bits
    const unsigned dw_blocks = part ? (unsigned)ceil_div(a.out * ceil_div(a.in, 4), 256) : 0u;
    const unsigned db_blocks = dbpart ? (unsigned)ceil_div(a.out, 256) : 0u;
    k_wgrad_join<<<dw_blocks + db_blocks, 256, 0, s>>>(part, (int)p.shares, dw_blocks, a.out, (uint32_t)a.in, a.dw, a.lddw,
                                                       dbpart, dbs, a.db, a.accumulate);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace

// The strides are not known here; they change the plan only past 2^24, and the larger need is taken.
size_t wgrad_workspace(int dtype, int64_t rows, int64_t in, int64_t out) {
  if (rows == 0) return 0;
  const size_t near = workspace_of(plan_for(dtype, rows, in, out, out), in, out);
  const size_t far = workspace_of(plan_for(dtype, rows, in, out, kMaxSpan), in, out);
  return near > far ? near : far;
}

hipError_t launch_wgrad(int dtype, const WgradArgs& a, hipStream_t s) {
  if (a.rows == 0) {
    k_wgrad_clear<<<grid_for(a.out * a.in), 256, 0, s>>>(a.dw, a.lddw, a.out, a.in, a.db);
    return hipGetLastError();
  }
  if (dtype == GC_F32) return wgrad_t<float>(dtype, a, s);
  if (dtype == GC_F16) return wgrad_t<f16>(dtype, a, s);
  return wgrad_t<bf16>(dtype, a, s);
}

}  // namespace gc
