// Dense layer y = act(x w^T + bias) + residual and its backward products.
//
// All products are C[m][n] = sum_k A(m, k) B(n, k), m the rows of x (of gz, of
// gz^T) and n the rows of w (the columns of w, of x):
//   forward  A = x  [m][k],  B = w  [n][k];
//   gx       A = gz [m][k],  B = w  [k][n];
//   gw       A = gz [k][m],  B = x  [k][n].
#include <algorithm>
#include <type_traits>

#include "dense.hpp"
#include "eec_internal.hpp"

namespace eec {
namespace {
using namespace dense;

// ------------------------------------------------------------------ epilogue

struct Epilogue {
  const void *bias, *residual;
  int64_t ldr;
  const float *x_scale, *w_scale;
  int32_t act;
  void *y, *preact;
  int64_t M, N;
  float* part;  // split sums [split][M][N] instead of all of the above, or NULL
};

// What L adjacent columns, `left` of which exist, have in common over the rows.
template <typename O, int L>
struct Columns {
  int64_t n, left;
  float bias[L], scale[L];
  __device__ __forceinline__ Columns(const Epilogue& e, int64_t n_, int64_t left_) : n(n_), left(left_) {
    if (e.bias) load_run((const O*)e.bias + n, left, bias);
    if (e.w_scale) load_run(e.w_scale + n, left, scale);
  }
};
// What a row's L columns bring from memory to their epilogue.  It is loaded ahead,
// for several rows at a time: the compiler keeps loads behind stores, and the wait
// for a load is a wait for the stores before it.
template <typename O, int L>
struct Incoming {
  O residual[L];
  float scale;
  __device__ __forceinline__ void load(const Epilogue& e, int64_t m, const Columns<O, L>& c) {
    if (m >= e.M) return;
    if (e.residual) load_raw<true>((const O*)e.residual + m * e.ldr + c.n, c.left, residual);
    if (e.x_scale) scale = e.x_scale[m];
  }
};

// v x_scale w_scale.  Scales of ordinary size (2^-50 to 2^51) are multiplied with each
// other first; others could leave float32's range there, or with the sum, where the
// result does not (1e-30 and 1e-15, 1e35 and 1e-35; an infinity would make a sum of 0
// a NaN), so their mantissas and powers of two are taken apart.  Telling the two apart
// takes 2 us of 138 (8192 x 4096 x 4096 e4m3).
__device__ __forceinline__ bool ordinary(float scale) { return (__float_as_uint(scale) >> 23) - 77u <= 100u; }
template <int L>
__device__ __forceinline__ void scale_run(float (&v)[L], float row, const float (&columns)[L]) {
  bool plain = ordinary(row);
#pragma unroll
  for (int i = 0; i < L; ++i) plain = plain && ordinary(columns[i]);
  if (plain) {
#pragma unroll
    for (int i = 0; i < L; ++i) v[i] *= row * columns[i];
  } else {
    const float m = __builtin_amdgcn_frexp_mantf(row);
    const int p = __builtin_amdgcn_frexp_expf(row);
#pragma unroll
    for (int i = 0; i < L; ++i) {
      float c = columns[i];
      asm volatile("" : "+v"(c));  // taken apart here, not ahead of the loop over rows (16 registers)
      v[i] = ldexpf(v[i] * (m * __builtin_amdgcn_frexp_mantf(c)), p + __builtin_amdgcn_frexp_expf(c));
    }
  }
}

// L adjacent columns of one row, from their sums over k.
template <typename O, int L>
__device__ __forceinline__ void finish_run(const Epilogue& e, int64_t m, const Columns<O, L>& c, const Incoming<O, L>& in,
                                           float (&v)[L]) {
  if (m >= e.M) return;
  if (e.x_scale) scale_run(v, in.scale, c.scale);
  if (e.bias) {
#pragma unroll
    for (int i = 0; i < L; ++i) v[i] += c.bias[i];
  }
  // rows that do not start on cache lines leave parts of lines for the L2 to join
  const bool once = e.N * (int64_t)sizeof(O) % 128 == 0;
  if (e.preact) store_run((O*)e.preact + m * e.N + c.n, c.left, v, once);
  act_values<O>(v, e.act);
  if (e.residual) {
#pragma unroll
    for (int i = 0; i < L; ++i) v[i] += (float)in.residual[i];
  }
  store_run((O*)e.y + m * e.N + c.n, c.left, v, once);
}

typedef float f32x16 __attribute__((ext_vector_type(16)));

// Chunk c (four adjacent columns) of a row of a wave's sums.
__device__ __forceinline__ void put_sums(char* rows, int row, int c, const f32x4& v) {
  __builtin_memcpy(__builtin_assume_aligned(rows + (row * 256 + (c ^ (row & 15)) * 16), 16), &v, 16);
}
// The tiles as the matrix instructions leave them: 16 rows x 4 x 16 columns, 32 x 2 x 32.
__device__ __forceinline__ void put_tile(const f32x4 (&acc)[4], char* rows) {
#pragma unroll
  for (int j = 0; j < 4; ++j) put_sums(rows, threadIdx.x & 15, j * 4 + (threadIdx.x >> 4 & 3), acc[j]);
}
__device__ __forceinline__ void put_tile(const f32x16 (&acc)[2], char* rows) {
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const f32x4 v = {acc[j][4 * a], acc[j][4 * a + 1], acc[j][4 * a + 2], acc[j][4 * a + 3]};
      put_sums(rows, threadIdx.x & 31, j * 8 + a * 2 + (threadIdx.x >> 5 & 1), v);
    }
}

// Finishes (or, split, stores) all of a wave's GROUPS matrix tiles of HIGH rows x 64
// columns, PER of them at a time through its own LDS: put_tile writes a tile's
// sums there, row by row of 256 bytes, the 16-byte chunk c of row r at c ^ (r & 15),
// and the tiles move up, so that the registers of those that are done are free.
// From there each access takes 16 bytes a lane of whole rows, and the code is short
// whatever a lane's registers hold: written out for every register it no longer
// fits the instruction cache (8192 x 8192 x 32 bf16: 64 us, this 46 us).
// What up to four rows a lane need from memory is on its way before the stores of the
// four ahead of them (8192 x 2048 x 8192 bf16 with residual, bias and SiLU 299 us with
// the loads behind those stores, 287 so; 2048 x 1024 x 2048 float32 60 and 48; with
// nothing to load and no activation it costs 1 to 4 %).
template <typename O, int HIGH, int PER, typename Acc, int GROUPS, int NB>
__device__ __forceinline__ void finish_wave(const Epilogue& e, char* lds, int64_t m0, int64_t n0, int split,
                                            Acc (&acc)[GROUPS][NB]) {
  constexpr int ROWS = PER * HIGH, ALL = GROUPS * HIGH;
  constexpr int L = 16 / (int)sizeof(O), APART = L;  // columns of a lane, rows of one access
  constexpr int TOGETHER = ROWS / APART < 4 ? ROWS / APART : 4, BATCH = TOGETHER * APART;
  static_assert(ROWS % BATCH == 0, "whole accesses");
  const int lane = threadIdx.x & 63, columns = (int)min((int64_t)64, e.N - n0);
  float* part = e.part ? e.part + split * e.M * e.N : nullptr;
  const int r0 = lane / (64 / L), col = lane % (64 / L) * L;
  const bool whole = col + L <= columns;
  const Columns<O, L> c(e, n0 + col, whole ? L : 0);
  Incoming<O, L> next[TOGETHER];
  const auto load = [&](int row) {
    if (!whole || part != nullptr || row - r0 >= ALL) return;
#pragma unroll
    for (int i = 0; i < TOGETHER; ++i) next[i].load(e, m0 + row + i * APART, c);
  };
  load(r0);
#pragma unroll 1
  for (int g = 0; g < GROUPS; g += PER) {
#pragma unroll
    for (int i = 0; i < PER; ++i) put_tile(acc[i], lds + i * HIGH * 256);
#pragma unroll
    for (int i = 0; i < GROUPS; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = i + PER < GROUPS ? acc[i + PER < GROUPS ? i + PER : 0][j] : Acc{};
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const int64_t top = m0 + g * HIGH;
    if (whole) {
#pragma unroll 1
      for (int r = r0; r < ROWS; r += BATCH) {
        Incoming<O, L> in[TOGETHER];
#pragma unroll
        for (int i = 0; i < TOGETHER; ++i) in[i] = next[i];
        load(g * HIGH + r + BATCH);
#pragma unroll
        for (int i = 0; i < TOGETHER; ++i) {
          const int row = r + i * APART;
          float v[L];
#pragma unroll
          for (int u = 0; u < L; u += 4)
            __builtin_memcpy(&v[u], __builtin_assume_aligned(lds + (row * 256 + (((col + u) / 4) ^ (row & 15)) * 16), 16), 16);
          if (part == nullptr)
            finish_run<O, L>(e, top + row, c, in[i], v);
          else if (top + row < e.M)
            store_run(part + (top + row) * e.N + n0 + col, L, v);
        }
      }
    }
    // the last columns of C that make no whole run: a row a lane, a column at a time
    if (columns % L > 0 && lane < ROWS) {
      const int64_t m = top + lane;
#pragma unroll 1
      for (int at = columns / L * L; at < columns; ++at) {
        const Columns<O, 1> one(e, n0 + at, 1);
        Incoming<O, 1> in;
        in.load(e, m, one);
        float v[1];
        __builtin_memcpy(v, lds + (lane * 256 + ((at / 4) ^ (lane & 15)) * 16 + at % 4 * 4), 4);
        if (part == nullptr)
          finish_run<O, 1>(e, m, one, in, v);
        else if (m < e.M)
          part[m * e.N + n0 + at] = v[0];
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
}
// Adds the splits in order and finishes: 4 columns a thread.
template <typename O>
__global__ void __launch_bounds__(256) k_join_splits(Epilogue e, int splits) {
  const int64_t per_row = (e.N + 3) / 4, total = e.M * per_row;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t m = i / per_row, n = i % per_row * 4;
    float v[4] = {};
    for (int s0 = 0; s0 < splits; s0 += 8) {  // eight loads on their way
      float t[8][4];
#pragma unroll
      for (int s = 0; s < 8; ++s)
        load_run(e.part + ((int64_t)(s0 + s) * e.M + m) * e.N + n, s0 + s < splits ? e.N - n : 0, t[s]);
#pragma unroll
      for (int s = 0; s < 8; ++s)
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] += t[s][c];
    }
    const Columns<O, 4> c(e, n, e.N - n);
    Incoming<O, 4> in;
    in.load(e, m, c);
    finish_run<O, 4>(e, m, c, in, v);
  }
}

// ------------------------------------------------------------------ matrix instructions

// float32 as the exact sum of three bf16 parts (8 + 8 + 8 significant bits, cut
// towards zero, so that no part overflows and all have the sign of x).  A part that
// would be 0 beside a value that is not takes the smallest bf16, 2^-133: an
// infinity times any part of the other operand is then an infinity of the right
// sign, never the NaN of an infinity times 0, and the sums of part products need no
// care.  So a value is held to 2^-131, exactly above 2^-100 but for that.
__device__ __forceinline__ void split3(float x, bf16& h, bf16& m, bf16& l) {
  const uint32_t u = __float_as_uint(x), sign = u >> 16 & 0x8000u, least = x != 0.f ? 1u : 0u;
  const bool finite = (u & 0x7f800000u) != 0x7f800000u;
  const uint32_t hi = (u & 0xffff0000u) | (x != x ? 0x400000u : 0u);  // a NaN keeps a bit of its fraction
  const float r = finite ? x - __uint_as_float(hi) : 0.f;
  const uint32_t mid = __float_as_uint(r) & 0xffff0000u;
  const uint32_t low = __float_as_uint(r - __uint_as_float(mid));
  auto part = [&](uint32_t bits) {
    const uint32_t size = max(bits >> 16 & 0x7fffu, least);
    return __builtin_bit_cast(bf16, (uint16_t)(size | sign));
  };
  h = part(hi);
  m = part(mid);
  l = part(low);
}

template <typename T>
struct Mat;  // operand planes in LDS (element type, count), and the product of 8-element fragments
template <>
struct Mat<f16> {
  using E = f16;
  static constexpr int PLANES = 1;
  using Frag = f16x8;
  static __device__ __forceinline__ f32x4 mul(const Frag (&b)[1], const Frag (&a)[1], f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(b[0], a[0], c, 0, 0, 0);
  }
};
template <>
struct Mat<bf16> {
  using E = bf16;
  static constexpr int PLANES = 1;
  using Frag = bf16x8;
  static __device__ __forceinline__ f32x4 mul(const Frag (&b)[1], const Frag (&a)[1], f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[0], a[0], c, 0, 0, 0);
  }
};
// The 8-bit instructions align the products of eight adjacent k before they add them:
// each is cut towards zero at 2^-13 of the power of two of the largest, in this
// instruction and in the 32 x 32 x 64 one alike, so a sum is off by 7 2^-13 of
// sum |a||b| at worst.  Beyond an f16 output's rounding up to 1.6e-4 of it was seen over
// all codes at k = 64 and 1.7e-5 at 4096, 1.8e-5 and 1.3e-6 for normally distributed
// values; the bf16 instruction on the same values was exact to 1e-7.  Taken for 16-bit
// outputs all the same: the operands' own rounding to e4m3, 2^-4 of each product, is far
// more than that, and the bf16 instructions take twice the time.  A float32 output is
// computed from the same codes widened to bf16 (exact, e4m3_wide).
template <>
struct Mat<e4m3> {
  using E = e4m3;
  static constexpr int PLANES = 1;
  using Frag = long;
  static __device__ __forceinline__ f32x4 mul(const Frag (&b)[1], const Frag (&a)[1], f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_fp8_fp8(b[0], a[0], c, 0, 0, 0);
  }
};
struct e4m3_wide : e4m3 {};
template <>
struct Mat<e4m3_wide> : Mat<bf16> {};
template <>
struct Mat<float> {
  using E = bf16;
  static constexpr int PLANES = 3;
  using Frag = bf16x8;
  // The part products in rising size.  The three left out have the sign of the whole: each
  // product is cut towards zero by up to 2^-21 of it (m reaches 2^-7 of a value's power of
  // two, l 2^-15), 0.6 x 2^-24 on average over mantissas.
  static __device__ __forceinline__ f32x4 mul(const Frag (&b)[3], const Frag (&a)[3], f32x4 c) {
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[2], a[0], c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[0], a[2], c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[1], a[1], c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[1], a[0], c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[0], a[1], c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[0], a[0], c, 0, 0, 0);
  }
};

// 8 elements of T as they come from memory.
template <typename T>
struct Raw {
  T v[8];
};

// Writes one 8-element chunk into its planes, `stride` bytes apart.
template <typename T>
__device__ __forceinline__ void put_chunk(char* at, int stride, const Raw<T>& r) {
  if constexpr (std::is_same<T, float>::value) {
    bf16 p[3][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) split3(r.v[i], p[0][i], p[1][i], p[2][i]);
#pragma unroll
    for (int q = 0; q < 3; ++q) __builtin_memcpy(__builtin_assume_aligned(at + q * stride, 16), p[q], 16);
  } else if constexpr (std::is_same<T, e4m3_wide>::value) {
    int q[2];
    __builtin_memcpy(q, &r, 8);
    bf16x8 w;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(q[i], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(q[i], true);
      w[4 * i] = (bf16)lo[0];
      w[4 * i + 1] = (bf16)lo[1];
      w[4 * i + 2] = (bf16)hi[0];
      w[4 * i + 3] = (bf16)hi[1];
    }
    __builtin_memcpy(__builtin_assume_aligned(at, 16), &w, 16);
  } else {
    __builtin_memcpy(__builtin_assume_aligned(at, sizeof(r)), &r, sizeof(r));
  }
}

// ------------------------------------------------------------------ general product

struct Product {
  const void *a, *b;
  int64_t lda, ldb;
  int64_t M, N, K;
  int64_t k_split;           // k of one split, a multiple of 128
  int64_t a_plane, b_plane;  // bytes between an operand's parts (float32 in planes)
};

constexpr int GBK = 32;  // k of a step of the general kernel

// Tile and split of k of a workgroup.  Workgroups go to the 8 XCDs in turn, each
// with an L2 of its own: an XCD takes a contiguous share of the work, split after
// split (the tiles of a split read the same k), each in strips of 8 tiles of m that
// run along n, so that what its CUs hold at one time reuses few rows of A and B.
// (32768 x 512 x 512 gw in float32, 16 splits of 16 tiles: 190 us with a split's
// tiles dealt over all XCDs, 169 us so.)
struct Place {
  int64_t m, n;
  int split;
};
template <int BM, int BN>
__device__ __forceinline__ Place place_of(int64_t M, int64_t N) {
  const uint32_t tiles_m = (uint32_t)((M + BM - 1) / BM), tiles_n = (uint32_t)((N + BN - 1) / BN);
  const uint32_t total = gridDim.x, b = blockIdx.x, xcd = b & 7;
  const uint32_t all = xcd * (total >> 3) + min(xcd, total & 7) + (b >> 3);
  const uint32_t split = all / (tiles_m * tiles_n), t = all - split * tiles_m * tiles_n;
  const uint32_t first = t / (8 * tiles_n) * 8, in = t - first * tiles_n;
  const uint32_t high = min(8u, tiles_m - first);
  return Place{(int64_t)(first + in % high) * BM, (int64_t)(in / high) * BN, (int)split};
}

// A tile of LINES lines x 32 k of one operand, an 8-element chunk per thread (two
// with 128 lines).  KC: k runs along memory (a chunk is one run), otherwise the
// lines do (a chunk is 8 runs of R lines).
template <typename T, bool KC, int LINES>
struct Stage {
  static constexpr int R = LINES / 64;
  static constexpr int ROW = GBK * sizeof(typename Mat<T>::E) + 8 * sizeof(typename Mat<T>::E);
  static constexpr int PLANE = LINES * ROW;
  Raw<T> r[R];

  __device__ __forceinline__ void load(const T* __restrict__ p, int64_t ld, int64_t line0, int64_t lines, int64_t k0,
                                       int64_t k_end) {
    if constexpr (KC) {
      const int64_t k = k0 + (threadIdx.x & 3) * 8, left = k_end - k;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const int64_t line = min(line0 + (threadIdx.x >> 2) + 64 * i, lines - 1);  // lines past the end: not stored
        load_raw(p + line * ld + k, left, r[i].v);
      }
    } else {
      const int64_t line = line0 + (threadIdx.x & 63) * R;
      const int64_t k = k0 + (threadIdx.x >> 6) * 8;
      const T* s = p + k * ld + line;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        T some[R];
        load_raw(s + j * ld, k + j < k_end ? lines - line : 0, some);
#pragma unroll
        for (int i = 0; i < R; ++i) r[i].v[j] = some[i];
      }
    }
  }
  __device__ __forceinline__ void store(char* lds) const {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int line = KC ? (threadIdx.x >> 2) + 64 * i : (threadIdx.x & 63) * R + i;
      const int kc = KC ? threadIdx.x & 3 : threadIdx.x >> 6;
      put_chunk<T>(lds + line * ROW + kc * 8 * sizeof(typename Mat<T>::E), PLANE, r[i]);
    }
  }
};

// Any size, stride and alignment: WM x WN waves with MI * 16 x 64 of C each.
// Operands pass through registers (where float32 is split into its parts and
// k-major ones are turned) into LDS rows of 32 k; the next two steps' loads are in
// flight while the present one is multiplied.  B is the first factor of the matrix
// instruction, so a lane holds four adjacent columns of one row of C.
template <typename T, typename O, bool A_KC, bool B_KC, int WM, int WN, int MI>
__global__ void __launch_bounds__(256) k_product(Product g, Epilogue e) {
  static_assert(WM * WN == 4, "four waves");
  constexpr int BM = WM * MI * 16, BN = WN * 64;
  using M_ = Mat<T>;
  constexpr int P = M_::PLANES;
  using SA = Stage<T, A_KC, BM>;
  using SB = Stage<T, B_KC, BN>;
  // sums: 4 KB of each wave for a matrix tile, two tiles at a time
  constexpr int PER = MI > 1 ? 2 : 1, TILES = P * (SA::PLANE + SB::PLANE), SUMS = 4 * PER * 4096;
  __shared__ __attribute__((aligned(16))) char lds[TILES > SUMS ? TILES : SUMS];
  char* lds_b = lds + P * SA::PLANE;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const Place place = place_of<BM, BN>(e.M, e.N);
  const int64_t m0 = place.m, n0 = place.n;
  const int64_t kb = place.split * g.k_split, ke = min(g.K, kb + g.k_split);
  const int wm = wave / WN * MI * 16, wn = wave % WN * 64;
  f32x4 acc[MI][4] = {};
  SA sa[2];
  SB sb[2];
  auto load = [&](int s, int64_t k) {
    if (k >= ke) return;
    sa[s].load((const T*)g.a, g.lda, m0, g.M, k, ke);
    sb[s].load((const T*)g.b, g.ldb, n0, g.N, k, ke);
  };
  // the step from k, staged in registers s; then s is loaded for the step after the next
  auto step = [&](int s, int64_t k) {
    __syncthreads();
    sa[s].store(lds);
    sb[s].store(lds_b);
    __syncthreads();
    load(s, k + 2 * GBK);
    typename M_::Frag fa[MI][P], fb[P];
    const int at = (lane & 15) * SA::ROW + (lane >> 4) * 8 * (int)sizeof(typename M_::E);
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int p = 0; p < P; ++p)
        __builtin_memcpy(&fa[i][p], __builtin_assume_aligned(lds + p * SA::PLANE + (wm + 16 * i) * SA::ROW + at, 8),
                         sizeof(fb[p]));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int p = 0; p < P; ++p)
        __builtin_memcpy(&fb[p], __builtin_assume_aligned(lds_b + p * SB::PLANE + (wn + 16 * j) * SB::ROW + at, 8),
                         sizeof(fb[p]));
#pragma unroll
      for (int i = 0; i < MI; ++i) acc[i][j] = M_::mul(fb, fa[i], acc[i][j]);
    }
  };
  load(0, kb);
  load(1, kb + GBK);
  for (int64_t k = kb; k < ke; k += 2 * GBK) {
    step(0, k);
    if (k + GBK < ke) step(1, k + GBK);
  }
  __syncthreads();
  finish_wave<O, 16, PER>(e, lds + wave * PER * 4096, m0 + wm, n0 + wn, place.split, acc);
}

// ------------------------------------------------------------------ tiled product (16- and 8-bit, aligned)

// The wave's number in its workgroup, in a scalar register.
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

typedef int i32x8 __attribute__((ext_vector_type(8)));

// One operand's LDS tile of 64 bytes of k, filled by direct loads of 16 bytes a
// lane (no registers, so later tiles' loads run under the present one's products).
// A direct load writes its 64 lanes' data one after another, 1024 bytes; against
// bank conflicts the address each lane loads from is permuted within them:
//   KC  (k along memory): LINES rows of 64 bytes, the 16-byte chunk c of row r at
//       slot c ^ (r >> 2 & 3);  fragments by ds_read_b128;
//   else (lines along memory, 16-bit): 32 rows (k) of LINES elements, PER_LOAD of
//       them a load, the 32-byte chunk c of row k at c ^ (k % PER_LOAD), and PAD
//       bytes after each load's 1024; the loads in an order (block_of) in which the
//       8 rows x 32 bytes that half a wave reads at once fill the 256 bytes of all
//       banks.  Only the low bits of a chunk's place depend on the lane, so a few
//       address registers serve all fragments.
// Neither has a bank conflict by the counter.
template <typename T, bool KC, int LINES, int WAVES>
struct Tile {
  static constexpr int BK = 64 / (int)sizeof(T);          // k of a tile
  static constexpr int LOADS = LINES / 16 / WAVES;        // direct loads of one wave
  static constexpr int PER_LOAD = 512 / LINES;            // k rows of one load (not KC)
  static constexpr int CHUNKS = 64 / PER_LOAD;            // 16-byte chunks of a k row (not KC)
  static constexpr int PAD = KC ? 0 : 16384 / LINES, STRIDE = 1024 + PAD;
  static constexpr int BYTES = LINES / 16 * STRIDE;
  static constexpr int READS = KC && sizeof(T) == 2 ? 1 : 2;  // LDS reads of one fragment
  static constexpr uint32_t NOWHERE = 0x80000000u;        // past every buffer: reads as zero
  const char* base;  // of the next tile, uniform
  int64_t step;      // bytes from tile to tile
  uint32_t off[LOADS];

  // Load i of this wave: its place among the tile's loads.
  static __device__ __forceinline__ int place(int i) { return wave_id() * LOADS + i; }
  // First k of this lane's chunk of load i within a tile.
  static __device__ __forceinline__ int at_k(int i) {
    const int lane = threadIdx.x & 63;
    if constexpr (KC)
      return ((lane & 3) ^ (lane >> 4 & 3)) * (16 / (int)sizeof(T));
    else
      return block_of(place(i)) * PER_LOAD + lane / CHUNKS;
  }
  // The k rows of load u are PER_LOAD from PER_LOAD * block_of(u), and the other way
  // round: bit 3 of k next to the lowest one, bit 2 (which tells a fragment's first
  // read from its second) above it.
  static __device__ __forceinline__ int block_of(int u) {
    return PER_LOAD == 2 ? (u & 9) | (u & 2) << 1 | (u >> 1 & 2) : (u & 4) | (u & 1) << 1 | (u >> 1 & 1);
  }
  __device__ __forceinline__ void init(const void* p, int64_t ld, int64_t line0, int64_t lines, int64_t k0) {
    const int lane = threadIdx.x & 63;
    base = (const char*)p + (KC ? (line0 * ld + k0) : (k0 * ld + line0)) * (int64_t)sizeof(T);
    step = (KC ? (int64_t)BK : (int64_t)BK * ld) * (int64_t)sizeof(T);
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      if constexpr (KC) {
        const int r = place(i) * 16 + (lane >> 2), c = (lane & 3) ^ (r >> 2 & 3);
        const int64_t line = min((int64_t)r, lines - 1 - line0);  // lines past the end: not stored
        off[i] = (uint32_t)(line * ld * (int64_t)sizeof(T)) + c * 16;
      } else {
        const int k = at_k(i), c = (lane % CHUNKS) ^ (k % PER_LOAD * 2);
        off[i] = line0 + c * 8 < lines ? (uint32_t)(k * ld * (int64_t)sizeof(T)) + c * 16 : NOWHERE;
      }
    }
  }
  // Loads the next tile, of which `left` k exist (none, perhaps): what lies past the
  // end reads as zero.
  __device__ __forceinline__ void load(char* lds, int left) {
    load_from(lds, base, left);
    base += step;
  }
  // The next tile of all three planes (BYTES apart in LDS), of a whole number of tiles.
  __device__ __forceinline__ void load_planes(char* lds, int64_t plane, int left) {
#pragma unroll
    for (int p = 0; p < 3; ++p) load_from(lds + p * BYTES, base + p * plane, left);
    base += step;
  }
  __device__ __forceinline__ void load_from(char* lds, const char* from, int left) {
    const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc((void*)from, 0, 0x7fffffff, 0x00020000);
#pragma unroll
    for (int i = 0; i < LOADS; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rsrc, (__attribute__((address_space(3))) void*)(lds + place(i) * STRIDE), 16, at_k(i) < left ? off[i] : NOWHERE,
          0, 0, 0);
  }
  // Fragment i of the lines from `line` (a multiple of 64).  Each address is one
  // addition to the buffer: through a longer chain the compiler loses sight of the
  // buffer and waits for every direct load before it reads.
  // 8-bit: 32 lines; a lane's 32 k are two of its row's 16-byte chunks, which two
  // is free as long as both operands agree.
  static __device__ __forceinline__ void fragment(i32x8& f, const char* lds, int line, int i) {
    const int lane = threadIdx.x & 63, r = line + (lane & 31);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = r * 64 + (((lane >> 5) * 2 + h) ^ (r >> 2 & 3)) * 16 + i * 2048;
      __builtin_memcpy((char*)&f + 16 * h, __builtin_assume_aligned(lds + at, 16), 16);
    }
  }
  // 16-bit: 16 lines.
  template <typename F>
  static __device__ __forceinline__ void fragment(F& f, const char* lds, int line, int i) {
    const int lane = threadIdx.x & 63;
    if constexpr (KC) {
      const int r = line + (lane & 15), at = r * 64 + ((lane >> 4) ^ (r >> 2 & 3)) * 16 + i * 1024;
      __builtin_memcpy(&f, __builtin_assume_aligned(lds + at, 16), 16);
    } else {
      // rows k and k + 4 (4 of them per 16 lanes), 8 bytes of 4 lines a lane
      typedef short s16x4 __attribute__((ext_vector_type(4)));
      const int k = (lane >> 4) * 8 + (lane >> 2 & 3), low = k % PER_LOAD;
      const int at = block_of(k / PER_LOAD) * STRIDE + low * (LINES * 2) + ((i % PER_LOAD) ^ low) * 32 + line * 2 +
                     (lane & 3) * 8 + i / PER_LOAD * PER_LOAD * 32;
      s16x4 h[2];
#pragma unroll
      for (int u = 0; u < 2; ++u)
        h[u] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (__attribute__((address_space(3))) s16x4*)(lds + (at + u * block_of(4 / PER_LOAD) * STRIDE)));
      __builtin_memcpy(&f, h, 16);
    }
  }
};

// A wave's share of C, MI * 16 rows x 64 columns, and a tile's products into it.
// `fb` and the first AHEAD of `fa` are read one tile ahead, under the products of
// the tile before, so that a tile begins with what it needs in registers.
template <typename T, int MI>
struct Share {
  static constexpr int ROWS = 16, GROUPS = MI;  // rows of a matrix tile, tiles along m
  static constexpr int NB = 4, AHEAD = 2;
  using Frag = typename Mat<T>::Frag;
  f32x4 acc[GROUPS][NB] = {};
  __device__ __forceinline__ void mul(int i, int j, const Frag& b, const Frag& a) {
    const Frag fb[1] = {b}, fa[1] = {a};
    acc[i][j] = Mat<T>::mul(fb, fa, acc[i][j]);
  }
};
template <int MI>
struct Share<e4m3, MI> {
  static constexpr int ROWS = 32, GROUPS = MI / 2;
  static constexpr int NB = 2, AHEAD = 1;
  using Frag = i32x8;
  f32x16 acc[GROUPS][NB] = {};
  __device__ __forceinline__ void mul(int i, int j, const Frag& b, const Frag& a) {  // block scales of 2^0
    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, acc[i][j], 0, 0, 0, 0x7f7f7f7f, 0, 0x7f7f7f7f);
  }
};
template <typename S>
struct Ahead {
  typename S::Frag b[S::NB], a[S::AHEAD];
};
template <typename S, typename TA, typename TB>
__device__ __forceinline__ void read_ahead(Ahead<S>& f, const char* la, const char* lb, int wm, int wn) {
#pragma unroll
  for (int j = 0; j < S::NB; ++j) TB::fragment(f.b[j], lb, wn, j);
#pragma unroll
  for (int i = 0; i < S::AHEAD; ++i) TA::fragment(f.a[i], la, wm, i);
}
// One tile's products from `f` and `la`, the next tile's `next` from `na` and
// `nb`.  The scheduling groups spread the tile's direct loads and LDS reads
// between the products; left alone the compiler gathers each read next to its use.
template <typename S, typename TA, typename TB>
__device__ __forceinline__ void multiply(S& c, const Ahead<S>& f, const char* la, int wm, Ahead<S>& next, const char* na,
                                         const char* nb, int wn) {
  constexpr int LOADS = TA::LOADS + TB::LOADS;
  typename S::Frag a[S::GROUPS];
#pragma unroll
  for (int i = 0; i < S::GROUPS; ++i) {
    constexpr int LATE = S::GROUPS - S::NB;  // the last groups read one fragment of B each
    if (i < S::AHEAD) a[i] = f.a[i];
    if (i + S::AHEAD < S::GROUPS)
      TA::fragment(a[i + S::AHEAD], la, wm, i + S::AHEAD);
    else
      TA::fragment(next.a[i + S::AHEAD - S::GROUPS], na, wm, i + S::AHEAD - S::GROUPS);
    if (i >= LATE) TB::fragment(next.b[i - LATE], nb, wn, i - LATE);
#pragma unroll
    for (int j = 0; j < S::NB; ++j) c.mul(i, j, f.b[j], a[i]);
  }
  constexpr int EACH = (LOADS + S::GROUPS - 1) / S::GROUPS;
#pragma unroll
  for (int i = 0; i < S::GROUPS; ++i) {
    if (i * EACH < LOADS) __builtin_amdgcn_sched_group_barrier(0x020, EACH, 0);  // direct loads
    if (i < S::GROUPS - S::NB)                                                   // LDS reads
      __builtin_amdgcn_sched_group_barrier(0x100, TA::READS, 0);
    else
      __builtin_amdgcn_sched_group_barrier(0x100, TA::READS + TB::READS, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, S::NB, 0);  // products
  }
}

// Waits until at most N of this wave's loads are on their way and its LDS reads
// are done, then for the workgroup.
template <int N>
__device__ __forceinline__ void tile_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | 7 << 4 | 0 << 8 | (N >> 4) << 14);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// BM x BN of C per workgroup of WM x WN waves, MI * 16 x 64 of it per wave.  BUFS
// LDS buffers: at the barrier before a tile the next one is there, to be read ahead
// from, BUFS - 3 more are on their way, and another is started into the buffer that
// everybody left at that barrier.  A load takes about 1900 cycles, a tile's products
// 1030 at 256 x 256, where two on their way do, and 258 at 128 x 128, where it takes
// six and the whole LDS (1024 x 4096 x 4096 bf16: 58 us with four buffers, 43 with
// eight).
// Needs 16-byte aligned rows and lengths (see tiled_operand).
template <typename T, typename O, bool A_KC, bool B_KC, int WM, int WN, int MI, int BUFS>
__global__ void __launch_bounds__(64 * WM * WN) k_tiled(Product g, Epilogue e) {
#ifdef __HIP_DEVICE_COMPILE__  // the host pass needs the stub alone, and drops some of them where it parses the body
  constexpr int BM = WM * MI * 16, BN = WN * 64, WAVES = WM * WN;
  using TA = Tile<T, A_KC, BM, WAVES>;
  using TB = Tile<T, B_KC, BN, WAVES>;
  constexpr int BK = TA::BK, LOADS = TA::LOADS + TB::LOADS;
  // The buffers are variables of their own: the compiler then sees that loads into
  // one do not touch the others, and does not wait for them before it reads.
  constexpr int A2 = BUFS == 8 ? TA::BYTES : 16, B2 = BUFS == 8 ? TB::BYTES : 16;
  __shared__ __attribute__((aligned(1024))) char a0[TA::BYTES], a1[TA::BYTES], a2[TA::BYTES], a3[TA::BYTES];
  __shared__ __attribute__((aligned(1024))) char b0[TB::BYTES], b1[TB::BYTES], b2[TB::BYTES], b3[TB::BYTES];
  __shared__ __attribute__((aligned(16))) char a4[A2], a5[A2], a6[A2], a7[A2], b4[B2], b5[B2], b6[B2], b7[B2];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const Place place = place_of<BM, BN>(e.M, e.N);
  const int64_t m0 = place.m, n0 = place.n;
  const int64_t kb = place.split * g.k_split, ke = min(g.K, kb + g.k_split);
  const int wm = wave / WN * MI * 16, wn = wave % WN * 64;
  using S = Share<T, MI>;
  S c;
  Ahead<S> f0, f1;
  TA ta;
  TB tb;
  ta.init(g.a, g.lda, m0, g.M, kb);
  tb.init(g.b, g.ldb, n0, g.N, kb);
  // k left from the present tile; groups of BUFS tiles, of which those past the end
  // are zeros, read from nowhere.
  int left = (int)(ke - kb);
#define EEC_LOAD(T, A, B)         \
  ta.load(A, left - (T) * BK);    \
  tb.load(B, left - (T) * BK)
#define EEC_TILE(T, F, A, NEXT, NA, NB, FREE_A, FREE_B) \
  tile_barrier<(BUFS - 3) * LOADS>();                   \
  EEC_LOAD(T + BUFS - 1, FREE_A, FREE_B);               \
  multiply<S, TA, TB>(c, F, A, wm, NEXT, NA, NB, wn)
  EEC_LOAD(0, a0, b0);
  EEC_LOAD(1, a1, b1);
  EEC_LOAD(2, a2, b2);
  if constexpr (BUFS == 8) {
    EEC_LOAD(3, a3, b3);
    EEC_LOAD(4, a4, b4);
    EEC_LOAD(5, a5, b5);
    EEC_LOAD(6, a6, b6);
  }
  tile_barrier<(BUFS - 2) * LOADS>();
  read_ahead<S, TA, TB>(f0, a0, b0, wm, wn);
  for (; left > 0; left -= BUFS * BK) {
    if constexpr (BUFS == 8) {
      EEC_TILE(0, f0, a0, f1, a1, b1, a7, b7);
      EEC_TILE(1, f1, a1, f0, a2, b2, a0, b0);
      EEC_TILE(2, f0, a2, f1, a3, b3, a1, b1);
      EEC_TILE(3, f1, a3, f0, a4, b4, a2, b2);
      EEC_TILE(4, f0, a4, f1, a5, b5, a3, b3);
      EEC_TILE(5, f1, a5, f0, a6, b6, a4, b4);
      EEC_TILE(6, f0, a6, f1, a7, b7, a5, b5);
      EEC_TILE(7, f1, a7, f0, a0, b0, a6, b6);
    } else {
      EEC_TILE(0, f0, a0, f1, a1, b1, a3, b3);
      EEC_TILE(1, f1, a1, f0, a2, b2, a0, b0);
      EEC_TILE(2, f0, a2, f1, a3, b3, a1, b1);
      EEC_TILE(3, f1, a3, f0, a0, b0, a2, b2);
    }
  }
#undef EEC_TILE
#undef EEC_LOAD
  tile_barrier<0>();  // nobody's loads or reads are left in the buffers
  // a buffer of its own for each wave: 64 rows of sums in 16 KB, or 32 in 8
  constexpr int SUMS = TA::BYTES >= 16384 && TB::BYTES >= 16384 ? 64 : 32;
  static_assert(TA::BYTES >= SUMS * 256 && TB::BYTES >= SUMS * 256 && WAVES <= 8, "room for the sums");
  const int pair = wave >> 1;
  char *even = pair == 0 ? a0 : pair == 1 ? a1 : pair == 2 ? a2 : a3, *odd = pair == 0 ? b0 : pair == 1 ? b1 : pair == 2 ? b2 : b3;
  finish_wave<O, S::ROWS, SUMS / S::ROWS>(e, wave & 1 ? odd : even, m0 + wm, n0 + wn, place.split, c.acc);
#endif
}

// ------------------------------------------------------------------ tiled product (float32 in parts)

// 256 x 128 of C per workgroup, 64 x 64 per wave, from planes of bf16 parts
// (k_pack: k in whole groups of four tiles).  A step is 32 k of all six planes,
// 72 KB of LDS, and does all six part products, so a plane is loaded once; two
// buffers: a step's 96 products a wave take 3100 cycles, the next one's loads 1900.
template <bool A_KC, bool B_KC>
__global__ void __launch_bounds__(512) k_parted(Product g, Epilogue e) {
#ifdef __HIP_DEVICE_COMPILE__  // see k_tiled
  using TA = Tile<bf16, A_KC, 256, 8>;
  using TB = Tile<bf16, B_KC, 128, 8>;
  __shared__ __attribute__((aligned(1024))) char a0[3 * TA::BYTES], a1[3 * TA::BYTES], b0[3 * TB::BYTES], b1[3 * TB::BYTES];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const Place place = place_of<256, 128>(e.M, e.N);
  const int64_t m0 = place.m, n0 = place.n;
  const int64_t kb = place.split * g.k_split, ke = min(g.K, kb + g.k_split);
  const int wm = wave / 2 * 64, wn = wave % 2 * 64;
  f32x4 acc[4][4] = {};
  TA ta;
  TB tb;
  ta.init(g.a, g.lda, m0, g.M, kb);
  tb.init(g.b, g.ldb, n0, g.N, kb);
  auto step = [&](const char* la, const char* lb) {
    bf16x8 b[3][4];
#pragma unroll
    for (int p = 0; p < 3; ++p)
#pragma unroll
      for (int j = 0; j < 4; ++j) TB::fragment(b[p][j], lb + p * TB::BYTES, wn, j);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      bf16x8 a[3];
#pragma unroll
      for (int p = 0; p < 3; ++p) TA::fragment(a[p], la + p * TA::BYTES, wm, i);
      // in rising size: (l, h), (h, l), (m, m), (m, h), (h, m), (h, h)
      constexpr int pa[6] = {2, 0, 1, 1, 0, 0}, pb[6] = {0, 2, 1, 0, 1, 0};
#pragma unroll
      for (int t = 0; t < 6; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[pb[t]][j], a[pa[t]], acc[i][j], 0, 0, 0);
    }
  };
// The scheduler would put the loads next to the wait at the step's end.
#define EEC_LOAD(A, B, LEFT)          \
  ta.load_planes(A, g.a_plane, LEFT); \
  tb.load_planes(B, g.b_plane, LEFT); \
  __builtin_amdgcn_sched_barrier(0)
  int left = (int)(ke - kb);
  EEC_LOAD(a0, b0, left);
  for (; left > 0; left -= 2 * TA::BK) {  // two steps; k is whole groups of four
    tile_barrier<0>();
    EEC_LOAD(a1, b1, left - TA::BK);
    step(a0, b0);
    tile_barrier<0>();
    EEC_LOAD(a0, b0, left - 2 * TA::BK);
    step(a1, b1);
  }
#undef EEC_LOAD
  tile_barrier<0>();
  // 64 rows of sums in 16 KB for each wave: three in an A buffer, one in a B buffer
  char* mine = wave < 3 ? a0 + wave * 16384 : wave < 6 ? a1 + (wave - 3) * 16384 : wave == 6 ? b0 : b1;
  finish_wave<float, 16, 4>(e, mine, m0 + wm, n0 + wn, place.split, acc);
#endif
}

// ------------------------------------------------------------------ few rows

// Up to 16 MT rows of x against 16 columns (rows of w) per workgroup: w goes from
// memory straight into the first factor of the matrix instruction, once, x (a few
// rows, in the L2) into the second.  The 8 waves deal runs of 128 bytes of k in
// turn and are joined in LDS, in wave order, so one launch does it all.
template <typename T, typename O, int MT>
__global__ void __launch_bounds__(512) k_few(Product g, Epilogue e) {
  using M_ = Mat<T>;
  constexpr int WAVES = 8, P = M_::PLANES;
  constexpr int CHUNK = sizeof(T) == 4 ? 32 : sizeof(T) == 2 ? 64 : 128;  // k of one run
  constexpr int STEPS = CHUNK / 32;                                      // matrix steps of one run
  constexpr int TOGETHER = MT == 1 ? 4 : 2;                              // runs in flight
  __shared__ f32x4 join[WAVES][MT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const T* w = (const T*)g.b + min(n0 + (lane & 15), g.N - 1) * g.ldb;
  const T* x[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) x[t] = (const T*)g.a + min((int64_t)(t * 16 + (lane & 15)), g.M - 1) * g.lda;
  f32x4 acc[MT] = {};
  // the epilogue's inputs set out first, and are there when the sums are
  const int64_t m = wave * 16 + (lane & 15);
  const Columns<O, 4> columns(e, n0 + q * 4, wave < MT ? e.N - n0 - q * 4 : 0);
  Incoming<O, 4> in;
  if (wave < MT) in.load(e, m, columns);
  // A run of CHUNK k: lane group q holds STEPS * 8 adjacent ones, of which step s
  // multiplies the s-th 8 (the same k of both operands meet, which is all a sum asks).
  struct Run {
    Raw<T> v[STEPS];
  };
  auto parts = [](const Raw<T>& r, typename M_::Frag (&f)[P]) {
    if constexpr (P == 3) {
      bf16 h[3][8];
#pragma unroll
      for (int i = 0; i < 8; ++i) split3(r.v[i], h[0][i], h[1][i], h[2][i]);
      __builtin_memcpy(f, h, sizeof(h));
    } else {
      put_chunk<T>((char*)f, 0, r);
    }
  };
  auto product = [&](const Run& wr, const Run (&xr)[MT]) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      typename M_::Frag fw[P], fx[P];
      parts(wr.v[s], fw);
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        parts(xr[t].v[s], fx);
        acc[t] = M_::mul(fw, fx, acc[t]);
      }
    }
  };
  const int64_t full = g.K / CHUNK;
  const int own = q * STEPS * 8;
  int64_t c = wave;
  for (; c + WAVES * (TOGETHER - 1) < full; c += WAVES * TOGETHER) {
    Run wr[TOGETHER], xr[TOGETHER][MT];
#pragma unroll
    for (int i = 0; i < TOGETHER; ++i) {
      const int64_t k = (c + WAVES * i) * CHUNK + own;
      __builtin_memcpy(&wr[i], w + k, sizeof(Run));
#pragma unroll
      for (int t = 0; t < MT; ++t) __builtin_memcpy(&xr[i][t], x[t] + k, sizeof(Run));
    }
#pragma unroll
    for (int i = 0; i < TOGETHER; ++i) product(wr[i], xr[i]);
  }
  for (; c * CHUNK < g.K; c += WAVES) {
    Run wr, xr[MT];
    const int64_t k = c * CHUNK + own, left = g.K - k;
    if (c < full) {
      __builtin_memcpy(&wr, w + k, sizeof(Run));
#pragma unroll
      for (int t = 0; t < MT; ++t) __builtin_memcpy(&xr[t], x[t] + k, sizeof(Run));
    } else {
#pragma unroll
      for (int s = 0; s < STEPS; ++s)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const bool is = s * 8 + i < left;
          wr.v[s].v[i] = is ? w[k + s * 8 + i] : T{};
#pragma unroll
          for (int t = 0; t < MT; ++t) xr[t].v[s].v[i] = is ? x[t][k + s * 8 + i] : T{};
        }
    }
    product(wr, xr);
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    join[wave][t][lane] = acc[t];
  }
  __syncthreads();
  if (wave < MT) {
    f32x4 v = join[0][wave][lane];
#pragma unroll
    for (int i = 1; i < WAVES; ++i) v += join[i][wave][lane];
    float r[4] = {v[0], v[1], v[2], v[3]};
    if (n0 + q * 4 < e.N) finish_run<O, 4>(e, m, columns, in, r);
  }
}

// ------------------------------------------------------------------ packing

// A matrix laid out for the tiled product: rows padded with zeros to a multiple of
// 128 elements, whole cache lines (at a stride of 2064 bytes a tile's 64-byte pieces
// cross lines: 1536 x 2768 x 1032 bf16 37 us, 29 us at 4096); float32 as three planes
// of bf16 parts, the number of rows padded alike (either may be k).
struct Packing {
  const void* from;
  int64_t ld, rows, cols;        // of the source
  char* to;                      // NULL: nothing to do
  int64_t to_ld, to_rows;        // elements
  int64_t plane;                 // bytes
};
struct Packings {
  Packing p[2];
};

template <typename T>
__global__ void __launch_bounds__(256) k_pack(Packings all) {
  constexpr int V = sizeof(T) == 1 ? 16 : 8;
  const Packing p = all.p[blockIdx.y];
  if (p.to == nullptr) return;
  const uint32_t chunks = (uint32_t)(p.to_ld / V), per = max(1u, 512u / chunks);  // rows of a workgroup's turn
  for (int64_t r0 = (int64_t)blockIdx.x * per; r0 < p.to_rows; r0 += (int64_t)gridDim.x * per) {
    const uint32_t total = chunks * (uint32_t)min((int64_t)per, p.to_rows - r0);
    for (uint32_t i = threadIdx.x; i < total; i += 256) {
      const int64_t row = r0 + i / chunks, col = (int64_t)(i % chunks) * V;
      T v[V];
      load_raw((const T*)p.from + row * p.ld + col, row < p.rows ? p.cols - col : 0, v);
      if constexpr (std::is_same<T, float>::value) {
        bf16 q[3][V];
#pragma unroll
        for (int c = 0; c < V; ++c) split3(v[c], q[0][c], q[1][c], q[2][c]);
#pragma unroll
        for (int k = 0; k < 3; ++k)
          __builtin_memcpy(__builtin_assume_aligned(p.to + k * p.plane + (row * p.to_ld + col) * 2, 16), q[k], 16);
      } else {
        __builtin_memcpy(__builtin_assume_aligned(p.to + (row * p.to_ld + col) * (int64_t)sizeof(T), 16), v, 16);
      }
    }
  }
}

constexpr int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }
// Element size of `dtype`'s packed form, its stride, rows and bytes.
int packed_size(int32_t dtype) { return dtype == EEC_E4M3 ? 1 : 2; }
Packing packing(int32_t dtype, const void* from, int64_t ld, int64_t rows, int64_t cols, char* to) {
  Packing p{from, ld, rows, cols, to, 0, 0, 0};
  p.to_ld = up(cols, 128);
  p.to_rows = dtype == EEC_F32 ? up(rows, 128) : rows;
  p.plane = p.to_rows * p.to_ld * packed_size(dtype);
  return p;
}
size_t packed_bytes(int32_t dtype, int64_t rows, int64_t cols) {
  return align256((size_t)packing(dtype, nullptr, 0, rows, cols, nullptr).plane * (dtype == EEC_F32 ? 3 : 1));
}
template <typename T>
void pack(hipStream_t st, const Packings& all) {
  int64_t most = 0;
  for (const Packing& p : all.p)
    if (p.to) most = std::max(most, p.to_rows * p.to_ld);
  if (most > 0) k_pack<T><<<dim3((unsigned)std::min<int64_t>((most + 4095) / 4096, 4096), 2), 256, 0, st>>>(all);
}

// ------------------------------------------------------------------ gradient of the activation

struct ActGrad {
  const void *gy, *preact;
  int64_t ldgy, rows, cols, per;  // rows of one strip
  int32_t act;
  void* gz;        // [rows][cols], or NULL
  Packing packed;  // or gz packed (packed.to not NULL)
  float* part;     // [strips][cols] column sums of gz before its rounding, or NULL
  void* gbias;     // with one strip the sums themselves instead, or NULL
};

// 16-bit types: gz is rounded to the type, as the matrix instructions take it (its column
// sums are not); two parts of it would double both products.  With the rounded preact that
// leaves gx and gw 2.4e-3 off in norm against 64 bits (8192 x 2048 x 8192 bf16), where
// products of gz in float32 are 1.7e-3 off by their own rounding.
//
// gz = gy act'(preact), as it is or packed, and its column sums: a wave takes 64 x 8
// (float32: 4) columns, a workgroup's waves deal the rows of a strip in turn.
template <typename T>
__global__ void __launch_bounds__(256) k_act_grad(ActGrad a) {
  constexpr int V = VEC<T>;
  __shared__ float join[3][64 * V];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t col = ((int64_t)blockIdx.x * 64 + lane) * V, left = a.cols - col;
  const int64_t r0 = (int64_t)blockIdx.y * a.per, r1 = min(a.packed.to ? a.packed.to_rows : a.rows, r0 + a.per);
  float sum[V] = {};
  for (int64_t r = r0 + wave; r < r1; r += 4) {
    float g[V], z[V];
    const int64_t here = r < a.rows ? left : 0;  // rows and columns of the padding are zeros
    load_run<true>((const T*)a.gy + r * a.ldgy + col, here, g);
    if (a.act != EEC_ACT_NONE) {
      load_run<true>((const T*)a.preact + r * a.cols + col, here, z);
      act_slopes<T>(g, z, a.act);
    }
    if (a.gz) store_run((T*)a.gz + r * a.cols + col, left, g);
    if (a.packed.to && col < a.packed.to_ld) {
      char* to = a.packed.to + (r * a.packed.to_ld + col) * 2;
      if constexpr (std::is_same<T, float>::value) {
        bf16 q[3][V];
#pragma unroll
        for (int i = 0; i < V; ++i) split3(g[i], q[0][i], q[1][i], q[2][i]);
#pragma unroll
        for (int k = 0; k < 3; ++k) __builtin_memcpy(__builtin_assume_aligned(to + k * a.packed.plane, 8), q[k], 2 * V);
      } else {
        store_run((T*)to, V, g);
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) sum[i] += g[i];
  }
  if (a.part == nullptr && a.gbias == nullptr) return;
  if (wave > 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) join[wave - 1][lane * V + i] = sum[i];
  }
  __syncthreads();
  if (wave == 0) {
    for (int k = 0; k < 3; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) sum[i] += join[k][lane * V + i];
    if (a.gbias)
      store_run((T*)a.gbias + col, left, sum);
    else
      store_run(a.part + (int64_t)blockIdx.y * a.cols + col, left, sum);
  }
}

// ------------------------------------------------------------------ plans

enum Kind { SMALL, GENERAL, TILE128, TILE128X2, TILE256, PARTED, FEW };  // SMALL: the general kernel in 64 x 64 tiles
struct Plan {
  Kind kind;
  bool packed;  // operands through k_pack
  int64_t tiles, splits, k_split;
};

int64_t tiles_of(int64_t M, int64_t N, int b) { return ((M + b - 1) / b) * ((N + b - 1) / b); }

// Rows up to which the forward product reads w straight into the matrix
// instructions (4096 x 4096 bf16: 14 us at 32 rows, where tiles take 17 us; 21 us
// at 64, where they take 18 us).
constexpr int64_t FEW_ROWS = 32;
// And its columns: 16 a workgroup of 512, threads that a launch counts in 32 bits (the widest layer is one workgroup past that).
constexpr int64_t FEW_COLUMNS = 16 * ((int64_t(1) << 23) - 1);

// Whether a product is worth packing for.  Packing reads and writes the operands
// once, in proportion to (M + N) K, and costs a launch; what it gains over the general
// kernel goes with M N K.  Kernel times, packed against general:
//   bf16 forward, odd k     1024^3 26 us, 20;  1531 x 2771 x 1029 42, 41;  2048 x 4096 x
//   (GELU, bias, residual)  1025 44, 42;  4096 x 4096 x 513 45, 52;  2048^3 43, 55
//   (so 16-bit forwards start between 4.4e9 and 8.6e9 products, where one of three sizes
//   still loses 2 us and two gain 7 and 12)
//   e4m3 forward, likewise  1024^3 21 us, 18;  1536^3 26, 26;  2048^3 32, 44
//   bf16 gx + gw, odd rows  700^3 36, 31;  1024^3 35, 53;  8192 x 128 x 512 32, 35
//   float32 forward         700^3 62, 25;  1024^3 37, 45;  2048 x 2048 x 512 51, 68;
//                           8192 x 128 x 512 53, 27
// In float32 the kernel behind it needs enough of its 256 x 128 tiles and splits.
bool worth_packing(int64_t M, int64_t N, int64_t K, int32_t dtype, bool forward) {
  if (M <= FEW_ROWS || N <= FEW_ROWS) return false;
  if (M > 1 << 20 || N > 1 << 20 || K > 1 << 20) return false;  // lanes' offsets within a tile fit 31 bits
  if (dtype == EEC_F32) {
    const int64_t tiles = ((M + 255) / 256) * ((N + 127) / 128);
    if (tiles * (K >= 1024 ? K / 256 : 1) < 100) return false;
  }
  const double least = !forward || dtype == EEC_F32 ? 4e8 : dtype == EEC_E4M3 ? 3e9 : 5e9;
  return (double)M * N >= 96.0 * (M + N) && (double)M * N * K >= least;
}

// How a product is run: a rule on sizes and on whether the operands take the tiled
// kernel (aligned, or packed).  k is split where the tiles alone leave most of the
// 256 CUs idle: joining the sums costs about 5 us, in which a 128 x 128 tile gets
// through 1200 k and the general kernel, which waits for memory at every step,
// through some 200.
Plan plan_product(int64_t M, int64_t N, int64_t K, int32_t dtype, bool tiled, bool packed, bool forward) {
  Plan p{};
  if (forward && M <= FEW_ROWS && N <= FEW_COLUMNS) {
    p.kind = FEW;
    p.splits = 1;
    return p;
  }
  const int64_t t256 = tiles_of(M, N, 256), t128 = tiles_of(M, N, 128);
  p.packed = packed;
  // One round of the 256 CUs takes 128 x 128 tiles about 10 us and 0.25 us for every
  // 64 bytes of k, 256 x 256 tiles 20 us and 0.49 us.  Between one and two rounds of
  // the small ones, two workgroups with four buffers share a CU instead: bf16 with
  // bias, GELU and residual, 1536 x 2816 x 1024 24 us (large tiles 35), 2048 x 4096 x
  // 1024 31 (38), x 4096 87 (99, split); beyond, split large tiles are even.
  const double steps = (double)K * (dtype == EEC_E4M3 ? 1 : 2) / 64;
  const double us128 = (double)((t128 + 255) / 256) * (10 + 0.25 * steps);
  const double us256 = (double)((t256 + 255) / 256) * (20 + 0.49 * steps);
  const bool shared = t128 > 256 && t128 <= 512 && steps <= 128;
  p.kind = packed && dtype == EEC_F32 ? PARTED
           : tiled || packed ? (shared ? TILE128X2 : us256 < us128 ? TILE256 : TILE128)
           : t128 >= 256     ? GENERAL
                             : SMALL;
  p.tiles = p.kind == TILE256  ? t256
            : p.kind == PARTED ? ((M + 255) / 256) * ((N + 127) / 128)
            : p.kind == SMALL  ? tiles_of(M, N, 64)
                               : t128;
  const bool general = p.kind == GENERAL || p.kind == SMALL;
  const int64_t step = 128;  // k of a split is a multiple of every kernel's tiles
  const int64_t least = general ? 128 : p.kind == PARTED ? 256 : 512;  // k of a split
  int64_t s = K < 4 * least ? 1 : std::min<int64_t>((p.kind == SMALL ? 512 : 256) / p.tiles, K / least);
  s = std::max<int64_t>(1, s);
  p.k_split = std::max<int64_t>(step, up((K + s - 1) / s, step));
  p.splits = std::max<int64_t>(1, (K + p.k_split - 1) / p.k_split);
  return p;
}
// Room for the split sums, however the operands turn out to be aligned.
size_t split_workspace(int64_t M, int64_t N, int64_t K, int32_t dtype, bool packed, bool forward) {
  if (M == 0 || N == 0) return 0;
  int64_t s = plan_product(M, N, K, dtype, true, packed, forward).splits;
  if (!packed) s = std::max(s, plan_product(M, N, K, dtype, false, packed, forward).splits);
  return s > 1 ? align256(4 * (size_t)s * (size_t)M * (size_t)N) : 0;
}

// Whether an operand of `size`-byte elements goes into LDS by 16-byte direct
// loads: aligned rows, a whole number of 16-byte chunks along memory, and lanes'
// offsets within a tile (256 lines or 32 k) that fit 31 bits.
bool tiled_operand(const void* p, int64_t ld, int64_t along, int size) {
  return ((uintptr_t)p & 15) == 0 && ld * size % 16 == 0 && along * size % 16 == 0 && ld * size < (1 << 22);
}

// Rows of C of one launch: with at most 2^36 outputs its tiles then stay below 2^24, and
// its threads (256 for a 128 x 128 tile, 512 for a 256 x 256 one) are counted in 32 bits.
constexpr int64_t LAUNCH_ROWS = int64_t(1) << 30;

// One product; packed_*: the operand is as k_pack leaves it.
template <typename T, typename O, bool A_KC, bool B_KC>
void product(hipStream_t st, Product g, Epilogue e, float* ws, int32_t dtype, bool packed_a, bool packed_b) {
  if (g.M == 0 || g.N == 0) return;
  if constexpr (A_KC) {  // the rows of gw are columns, at most 2^27
    if (g.M > LAUNCH_ROWS) {  // k is not split there, and at most a 16-bit gz is packed: row after row, as it is
      const int64_t first = g.M / 2;
      Product rest = g;
      Epilogue to = e;
      g.M = first;
      rest.M -= first;
      rest.a = (const T*)g.a + first * g.lda;
      to.y = (O*)e.y + first * g.N;
      if (e.preact) to.preact = (O*)e.preact + first * g.N;
      if (e.residual) to.residual = (const O*)e.residual + first * e.ldr;
      if (e.x_scale) to.x_scale = e.x_scale + first;
      product<T, O, A_KC, B_KC>(st, g, e, ws, dtype, packed_a, packed_b);
      return product<T, O, A_KC, B_KC>(st, rest, to, ws, dtype, packed_a, packed_b);
    }
  }
  const bool packed = packed_a && packed_b;
  const bool aligned = dtype != EEC_F32 && !std::is_same<T, e4m3_wide>::value &&
                       (packed_a || tiled_operand(g.a, g.lda, A_KC ? g.K : g.M, sizeof(T))) &&
                       (packed_b || tiled_operand(g.b, g.ldb, B_KC ? g.K : g.N, sizeof(T)));
  const Plan p = plan_product(g.M, g.N, g.K, dtype, aligned, packed, A_KC && B_KC);
  g.k_split = p.k_split;
  e.M = g.M;
  e.N = g.N;
  e.part = p.splits > 1 ? ws : nullptr;
  const dim3 grid((unsigned)(p.tiles * p.splits));
  Product t = g;
  // what is loaded along memory may run into the padding, which is there and zero
  if (packed_a && !A_KC) t.M = t.lda;
  if (packed_b && !B_KC) t.N = t.ldb;
  if constexpr (std::is_same<T, float>::value) {
    t.K = up(g.K, 128);
    if (p.kind == PARTED) k_parted<A_KC, B_KC><<<grid, 512, 0, st>>>(t, e);
  } else if constexpr (!std::is_same<T, e4m3_wide>::value) {
    if (p.kind == TILE256) k_tiled<T, O, A_KC, B_KC, 2, 4, 8, 4><<<grid, 512, 0, st>>>(t, e);
    if (p.kind == TILE128X2) k_tiled<T, O, A_KC, B_KC, 2, 2, 4, 4><<<grid, 256, 0, st>>>(t, e);
    if (p.kind == TILE128) k_tiled<T, O, A_KC, B_KC, 2, 2, 4, 8><<<grid, 256, 0, st>>>(t, e);
  }
  if constexpr (A_KC && B_KC) {
    const dim3 columns((unsigned)((g.N + 15) / 16));
    if (p.kind == FEW && g.M <= 16) k_few<T, O, 1><<<columns, 512, 0, st>>>(g, e);
    if (p.kind == FEW && g.M > 16) k_few<T, O, 2><<<columns, 512, 0, st>>>(g, e);
  }
  if (p.kind == GENERAL) k_product<T, O, A_KC, B_KC, 2, 2, 4><<<grid, 256, 0, st>>>(g, e);
  if (p.kind == SMALL) k_product<T, O, A_KC, B_KC, 4, 1, 1><<<grid, 256, 0, st>>>(g, e);
  if (p.splits > 1) {
    const int64_t runs = g.M * ((g.N + 3) / 4);
    k_join_splits<O><<<dim3((unsigned)std::min<int64_t>((runs + 255) / 256, 4096)), 256, 0, st>>>(e, (int)p.splits);
  }
}

template <typename F>
void by_type(int32_t dtype, F&& f) {
  if (dtype == EEC_F32) return f(float());
  if (dtype == EEC_F16) return f(f16());
  f(bf16());
}

// The forward's workspace: x and w packed, split sums.
struct FwdPlan {
  bool packed;
  size_t off_x, off_w, off_split, bytes;
};
FwdPlan fwd_plan(int64_t rows, int64_t outer, int64_t inner, int32_t dtype, int32_t out_dtype) {
  FwdPlan p{};
  const bool exact = dtype == EEC_E4M3 && out_dtype == EEC_F32;  // widened by the general kernel
  p.packed = !exact && worth_packing(rows, outer, inner, dtype, true) &&
             (dtype == EEC_F32 || inner * packed_size(dtype) % 16 != 0);
  size_t at = 0;
  p.off_x = at;
  if (p.packed) at += packed_bytes(dtype, rows, inner);
  p.off_w = at;
  if (p.packed) at += packed_bytes(dtype, outer, inner);
  p.off_split = at;
  p.bytes = at + split_workspace(rows, outer, inner, dtype, p.packed, true);
  return p;
}

// Rows of a strip at least: four for each wave, so that a few rows are one strip and
// their column sums need no second launch.
constexpr int STRIP_ROWS = 16;
int64_t act_grad_strips(int64_t rows, int64_t cols, int32_t dtype) {
  const int64_t per = 64 * (dtype == EEC_F32 ? 4 : 8), wide = (cols + per - 1) / per;
  return std::max<int64_t>(1, std::min<int64_t>((rows + STRIP_ROWS - 1) / STRIP_ROWS, 1024 / std::max<int64_t>(1, wide)));
}

// The backward's: gz (packed or not), column sums, x and w packed, split sums.
struct BwdPlan {
  bool gz, others;  // packed
  size_t off_gz, off_part, off_xp, off_wp, off_split, bytes;
};
BwdPlan bwd_plan(int64_t rows, int64_t outer, int64_t inner, int32_t dtype, int32_t act) {
  BwdPlan p{};
  if (dtype == EEC_F32) {
    p.gz = p.others = worth_packing(rows, inner, outer, dtype, false) && worth_packing(outer, inner, rows, dtype, false);
  } else {
    p.others = inner % 8 != 0 && worth_packing(rows, inner, outer, dtype, false) && worth_packing(outer, inner, rows, dtype, false);
    // gz passes through k_act_grad anyway, or is small beside what gx and gw take.  Not so
    // where its rows of 128 columns would be mostly padding and more than four times x:
    // 10^6 x 8 -> 1 with SiLU 572 us and 256 MB packed, 490 and 2 as it is (-> 33: 680, 609;
    // -> 63: 788, 796); 32768 rows of it 45 and 54 us, in 8 MB, stay packed.
    const bool padding = rows > 1 << 19 && up(outer, 128) > std::max(2 * outer, 4 * inner);
    p.gz = outer % 8 != 0 && (p.others || inner % 8 == 0) && rows > FEW_ROWS && outer < 1 << 20 && !padding &&
           (act != EEC_ACT_NONE || (double)rows * outer * inner >= 4e8);
  }
  size_t at = 0;
  p.off_gz = at;
  if (p.gz)
    at += packed_bytes(dtype, rows, outer);
  else if (act != EEC_ACT_NONE)
    at += align256((size_t)rows * (size_t)outer * (dtype == EEC_F32 ? 4 : 2));
  p.off_part = at;
  at += align256(4 * (size_t)act_grad_strips(rows, outer, dtype) * (size_t)outer);
  p.off_xp = at;
  if (p.others) at += packed_bytes(dtype, rows, inner);
  p.off_wp = at;
  if (p.others) at += packed_bytes(dtype, outer, inner);
  p.off_split = at;
  const bool both = p.gz && p.others;
  at += std::max(split_workspace(rows, inner, outer, dtype, both, false),
                 split_workspace(outer, inner, rows, dtype, both, false));
  p.bytes = at;
  return p;
}

}  // namespace

size_t linear_workspace(int64_t rows, int64_t outer, int64_t inner, int32_t dtype, int32_t out_dtype) {
  return fwd_plan(rows, outer, inner, dtype, out_dtype).bytes;
}

void launch_linear(hipStream_t st, const LinearArgs& a, char* ws) {
  const FwdPlan p = fwd_plan(a.rows, a.outer, a.inner, a.dtype, a.out_dtype);
  const Epilogue e{a.bias, a.residual, a.ldr, a.x_scale, a.w_scale, a.act, a.y, a.preact, 0, 0, nullptr};
  by_type(a.out_dtype, [&](auto zero) {
    using O = decltype(zero);
    using E = std::conditional_t<std::is_same<O, float>::value, e4m3_wide, e4m3>;
    Product g{a.x, a.w, a.ldx, a.ldw, a.rows, a.outer, a.inner, 0, 0, 0};
    if (p.packed) {
      const Packing x = packing(a.dtype, a.x, a.ldx, a.rows, a.inner, ws + p.off_x);
      const Packing w = packing(a.dtype, a.w, a.ldw, a.outer, a.inner, ws + p.off_w);
      const Packings both{{x, w}};
      if (a.dtype == EEC_E4M3)
        pack<e4m3>(st, both);
      else
        pack<O>(st, both);
      g = Product{x.to, w.to, x.to_ld, w.to_ld, a.rows, a.outer, a.inner, 0, x.plane, w.plane};
    }
    float* split = (float*)(ws + p.off_split);
    if (a.dtype == EEC_E4M3)
      product<E, O, true, true>(st, g, e, split, a.dtype, p.packed, p.packed);
    else
      product<O, O, true, true>(st, g, e, split, a.dtype, p.packed, p.packed);
  });
}

size_t linear_bwd_workspace(int64_t rows, int64_t outer, int64_t inner, int32_t dtype, int32_t act) {
  return bwd_plan(rows, outer, inner, dtype, act).bytes;
}

void launch_linear_bwd(hipStream_t st, const LinearBwdArgs& a, char* ws) {
  const BwdPlan p = bwd_plan(a.rows, a.outer, a.inner, a.dtype, a.act);
  by_type(a.dtype, [&](auto zero) {
    using T = decltype(zero);
    const bool products = a.gx != nullptr || a.gw != nullptr;
    const bool packed = p.gz && products, shaped = a.act != EEC_ACT_NONE && products && !packed;
    const Packing z = packing(a.dtype, nullptr, 0, a.rows, a.outer, packed ? ws + p.off_gz : nullptr);
    if (a.outer > 0 && ((shaped && a.rows > 0) || a.gbias || packed)) {
      const int64_t strips = act_grad_strips(a.rows, a.outer, a.dtype), cols = 64 * VEC<T>;
      const int64_t rows = packed ? z.to_rows : a.rows, width = packed ? z.to_ld : a.outer;
      const ActGrad q{a.gy,  a.preact, a.ldgy, a.rows, a.outer, (rows + strips - 1) / strips,
                      a.act, shaped ? ws + p.off_gz : nullptr, z,
                      a.gbias && strips > 1 ? (float*)(ws + p.off_part) : nullptr, strips == 1 ? a.gbias : nullptr};
      k_act_grad<T><<<dim3((unsigned)((width + cols - 1) / cols), (unsigned)strips), 256, 0, st>>>(q);
      if (a.gbias && strips > 1)
        launch_column_sum(st, a.dtype, (const float*)(ws + p.off_part), (int)strips, a.outer, a.gbias);
    }
    const void* gz = packed ? z.to : shaped ? ws + p.off_gz : (const char*)a.gy;
    const int64_t ldgz = packed ? z.to_ld : shaped ? a.outer : a.ldgy;
    Product gx{gz, a.w, ldgz, a.ldw, a.rows, a.inner, a.outer, 0, z.plane, 0};
    Product gw{gz, a.x, ldgz, a.ldx, a.outer, a.inner, a.rows, 0, z.plane, 0};
    if (p.others && products) {
      const Packing x = packing(a.dtype, a.x, a.ldx, a.rows, a.inner, a.gw ? ws + p.off_xp : nullptr);
      const Packing w = packing(a.dtype, a.w, a.ldw, a.outer, a.inner, a.gx ? ws + p.off_wp : nullptr);
      pack<T>(st, Packings{{x, w}});
      gx.b = w.to;
      gx.ldb = w.to_ld;
      gx.b_plane = w.plane;
      gw.b = x.to;
      gw.ldb = x.to_ld;
      gw.b_plane = x.plane;
    }
    float* split = (float*)(ws + p.off_split);
    Epilogue e{};
    if (a.gx) {
      e.y = a.gx;
      product<T, T, true, false>(st, gx, e, split, a.dtype, packed, p.others);
    }
    if (a.gw) {
      e.y = a.gw;
      product<T, T, false, false>(st, gw, e, split, a.dtype, packed, p.others);
    }
  });
}

}  // namespace eec
