// An update brought near the nearest matrix with orthonormal rows or columns:
//
//   X = g / (|g| + eps);   A = X X^T,  B = b A + c A^2,  X <- a X + B X   (a step)
//
// with A the Gram matrix of the shorter side (rows <= cols as above; otherwise A = X^T X and
// X <- a X + X B).  Three products a step: A and B are symmetric, so only tiles on and above
// the diagonal are computed and written twice.
//
// Numbers.  Everything is held 2^12 times its value in float16 planes: X as hi + lo (22 bits),
// so that a X carries no rounding of 11 bits from step to step, where small singular values
// grow 3.4-fold each.  Two planes: hi hi + hi lo + lo hi in every product, as exact as float32
// products (2e-7 to 1e-5 off in norm, those 1e-6 to 2e-5).  One plane, for large bf16 updates:
// hi alone in the products, 1e-3 to 2e-3 off, which is the output's own size (bf16 operands: 1e-2
// for normal g, up to 0.3 where a few directions dominate; float16 ones without X's lo 4e-2
// there).  B is computed from A as rounded: the errors of b A and c A^2 then cancel at singular
// values near 1.  These stay below 3.5 (checked on the host), so that 2^12 of them fit float16;
// elements of X keep 11 bits in hi down to 2^-26, and are held to 2^-37.
#include "product.hpp"

namespace eec {
namespace {

constexpr float SCALE = 4096.f;

// What g is multiplied with, SCALE / (|g| + eps), from its sum of squares.  Only beside a norm of zero (others are 2^-149 at
// least) can that pass float64's range: bounded, it leaves a matrix of zeros one.  A NaN stays.
__device__ __forceinline__ double scale_of(double sum, double eps) {
  const double scale = (double)SCALE / (sqrt(sum) + eps);
  return scale > 1e300 ? 1e300 : scale;
}

// Where a product's results go: alpha from + beta C, rounded into two planes or one, or (Y a
// type) into rows of y.
struct Planes {};
struct NewtonTo {
  const f16* from;     // or NULL
  int64_t from_plane;  // elements to its low part, 0: none
  f16* to;
  int64_t to_plane;    // 0: no low part
  int64_t ld;          // of from and to, a multiple of 8
  int64_t from_batch, to_batch;  // elements to the next matrix
};
// SYM: C is symmetric, tiles below the diagonal are not computed.  TURN: C's transpose goes to
// `turned` as well (SYM: into C's own lower half, without TURN).
template <typename Y, bool SYM, bool TURN = false>
struct NewtonEpilogue {
  static constexpr bool SYMMETRIC = SYM, ACROSS = SYM || TURN, IN_PLANES = std::is_same<Y, Planes>::value;
  __device__ __forceinline__ const NewtonTo& across() const { return TURN ? turned : rows; }
  int64_t M, N;  // of the product
  float alpha, beta;
  NewtonTo rows, turned;
  Y* y;  // [M][N] instead of rows.to
  int64_t y_batch, a_batch, b_batch;
  // Split over k (grid.z): sums [split][matrix][part_ld][part_ld], joined by k_join_newton, instead of all of the
  // above; or NULL.
  float* part;
  int64_t part_ld;
  bool k_along;  // k along memory, in both operands
};

template <typename Y, bool SYM, bool TURN>
__device__ __forceinline__ void of_batch(Product& g, NewtonEpilogue<Y, SYM, TURN>& e) {
  const int64_t i = blockIdx.y;
  g.a = (const f16*)g.a + i * e.a_batch;
  g.b = (const f16*)g.b + i * e.b_batch;
  const auto next = [&](NewtonTo& s) {
    if (s.from) s.from += i * s.from_batch;
    s.to += i * s.to_batch;
  };
  next(e.rows);
  if constexpr (TURN) next(e.turned);
  if constexpr (!NewtonEpilogue<Y, SYM, TURN>::IN_PLANES) e.y += i * e.y_batch;
  if constexpr (SYM) {
    if (e.part) {
      e.part += ((int64_t)blockIdx.z * gridDim.y + i) * e.part_ld * e.part_ld;
      const int64_t first = blockIdx.z * g.k_split;
      const bool kc = e.k_along;
      g.a = (const f16*)g.a + (kc ? first : first * g.lda);
      g.b = (const f16*)g.b + (kc ? first : first * g.ldb);
      g.K = min(g.k_split, g.K - first);
      g.k_split = g.K;
    }
  }
}

// Symmetric: the tiles that reach above the diagonal, row of tiles after row of tiles.
template <int BM, int BN, typename Y, bool SYM, bool TURN>
__device__ __forceinline__ Place place_of(const NewtonEpilogue<Y, SYM, TURN>& e) {
  static_assert(BM % BN == 0, "a row of tiles starts at its diagonal");
  if constexpr (SYM) {
    const uint32_t tiles_n = (uint32_t)((e.N + BN - 1) / BN);
    uint32_t t = dealt(), i = 0;
    for (uint32_t row = tiles_n; t >= row; row = tiles_n - i * (BM / BN)) t -= row, ++i;
    return Place{(int64_t)i * BM, (int64_t)(i * (BM / BN) + t) * BN, 0};
  } else {
    Epilogue plain{};
    plain.M = e.M;
    plain.N = e.N;
    return place_of<BM, BN>(plain);
  }
}
template <int BM, int BN>
int64_t newton_tiles(int64_t M, int64_t N, bool symmetric) {
  const int64_t m = (M + BM - 1) / BM, n = (N + BN - 1) / BN;
  if (!symmetric) return m * n;
  int64_t all = 0;
  for (int64_t i = 0; i < m; ++i) all += n - i * (BM / BN);
  return all;
}

// Both parts from one float32 number: left to itself the compiler fuses the sum that makes v with
// its rounding to hi, and where that differs from the rounding of v, lo belongs to another hi (one value in 8192).
__device__ __forceinline__ void split2(float v, f16& hi, f16& lo) {
  asm("" : "+v"(v));
  hi = (f16)v;
  lo = (f16)(v - (float)hi);
}

// What alpha multiplies of eight adjacent elements of one row, from a multiple of 8 on; zeros where there is none.
struct Run8 {
  f16 hi[8], lo[8];
  // `at`: elements from (row m0, column n0), both uniform, where the wave's sums start.  No branch, so that nothing
  // waits for these loads before their use; what does not exist is read past every buffer, as zero.
  __device__ __forceinline__ void load(const NewtonTo& s, int64_t m0, int64_t n0, uint32_t at, bool exists) {
    constexpr uint32_t NOWHERE = 0x80000000u;
    const f16* p = s.from + m0 * s.ld + n0;
    const auto part = [&](const f16* from, bool is, f16 (&v)[8]) {
      const auto q = __builtin_amdgcn_raw_buffer_load_b128(
          __builtin_amdgcn_make_buffer_rsrc((void*)from, 0, 0x7fffffff, 0x00020000), is && exists ? at * 2 : NOWHERE, 0, 0);
      __builtin_memcpy(v, &q, 16);
    };
    part(p, s.from != nullptr, hi);
    part(p + s.from_plane, s.from_plane != 0, lo);
  }
  __device__ __forceinline__ void value(float alpha, float beta, float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = alpha * ((float)hi[i] + (float)lo[i]) + beta * v[i];
  }
};
// Rows of planes are whole runs, whose end (all but `left` of the last) is kept at zero, so that each run is one store.
__device__ __forceinline__ void store_planes(const NewtonTo& s, int64_t m, int64_t n, int64_t left, const float (&v)[8]) {
  f16 h[8], l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) split2(i < left ? v[i] : 0.f, h[i], l[i]);
  f16* p = s.to + m * s.ld + n;
  __builtin_memcpy(__builtin_assume_aligned(p, 16), h, 16);
  if (s.to_plane) __builtin_memcpy(__builtin_assume_aligned(p + s.to_plane, 16), l, 16);
}

__device__ __forceinline__ float sum_at(const char* lds, int r, int c) {
  float v;
  __builtin_memcpy(&v, lds + (r * 256 + ((c / 4) ^ (r & 15)) * 16 + c % 4 * 4), 4);
  return v;
}

// Finishing a wave's sums, row by row of 256 bytes (64 columns) in its LDS as put_sums leaves them.
// Symmetric: 8 x 8 blocks on and above the diagonal are stored, and those above it once more
// across it, from columns of the same sums; a block on the diagonal takes its lower half from its
// upper one.  So each element is written once, by one lane, and C is symmetric to the bit.
//
// N rows a lane, 8 columns each: rows r + 8 i of the wave's, r its eighth's.
template <int N>
struct RowRuns {
  Run8 run[N];
  template <typename E>
  static __device__ __forceinline__ int64_t left(const E& e, int64_t m, int64_t n) {
    return m < e.M && !(E::SYMMETRIC && n + 7 < m) ? e.N - n : 0;
  }
  template <typename E>
  __device__ __forceinline__ void load(const E& e, int64_t top, int64_t n0, int r) {
    const int col = (threadIdx.x & 7) * 8;
#pragma unroll
    for (int i = 0; i < N; ++i, r += 8)
      run[i].load(e.rows, top, n0, (uint32_t)(r * (int)e.rows.ld + col), left(e, top + r, n0 + col) > 0);
  }
  // `lds`: the sums of row `from` on.
  template <typename E>
  __device__ __forceinline__ void finish(const E& e, const char* lds, int64_t top, int64_t n0, int r, int from) const {
    const int col = (threadIdx.x & 7) * 8;
    const int64_t n = n0 + col;
#pragma unroll
    for (int i = 0; i < N; ++i, r += 8) {
      const int64_t m = top + r, some = left(e, m, n);
      if (some <= 0) continue;
      const int at = r - from;
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; u += 4)
        __builtin_memcpy(&v[u], __builtin_assume_aligned(lds + (at * 256 + (((col + u) / 4) ^ (at & 15)) * 16), 16), 16);
      if (E::SYMMETRIC && n < m) {
#pragma unroll
        for (int u = 0; u < 8; ++u)
          if (n + u < m) v[u] = sum_at(lds, (at & ~7) + u, col + (at & 7));
      }
      run[i].value(e.alpha, e.beta, v);
      if constexpr (E::IN_PLANES) {
        store_planes(e.rows, m, n, some, v);
      } else {
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] *= 1.f / SCALE;
        store_run(e.y + m * e.N + n, some, v);
      }
    }
  }
};
// Row n0 + lane of the transpose: rows r to r + 8 N - 1 of the wave's.
template <int N>
struct TurnedRuns {
  Run8 run[N];
  template <typename E>
  static __device__ __forceinline__ int64_t left(const E& e, int64_t m, int64_t n) {  // symmetric: blocks above the diagonal
    return m < e.N && !(E::SYMMETRIC && n + 7 >= m) ? e.M - n : 0;
  }
  template <typename E>
  __device__ __forceinline__ void load(const E& e, int64_t top, int64_t n0, int r) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < N; ++i, r += 8)
      run[i].load(e.across(), n0, top, (uint32_t)(lane * (int)e.across().ld + r), left(e, n0 + lane, top + r) > 0);
  }
  template <typename E>
  __device__ __forceinline__ void finish(const E& e, const char* lds, int64_t top, int64_t n0, int r, int from) const {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < N; ++i, r += 8) {
      const int64_t m = n0 + lane, n = top + r, some = left(e, m, n);
      if (some <= 0) continue;
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = sum_at(lds, r - from + u, lane);
      run[i].value(e.alpha, e.beta, v);
      store_planes(e.across(), m, n, some, v);
    }
  }
};
// As finish_wave: what a batch of rows needs from memory is loaded before any of it is stored, and where registers are
// left (not in symmetric products, which finish two blocks at a time) before the stores of the batch ahead of it.
template <bool G, typename O, int HIGH, int PER, typename Y, bool SYM, bool TURN, typename Acc, int GROUPS, int NB>
__device__ __forceinline__ void finish(const NewtonEpilogue<Y, SYM, TURN>& e, char* lds, int64_t m0, int64_t n0, int,
                                       Acc (&acc)[GROUPS][NB]) {
  static_assert(!TURN, "large tiles have no transposes");
  constexpr int ROWS = PER * HIGH;
  static_assert(ROWS % 32 == 0, "whole batches");
  const int r0 = threadIdx.x >> 3 & 7;
  const bool whole = SYM && e.part;
  RowRuns<4> next;
  if constexpr (!SYM) next.load(e, m0, n0, r0);
#pragma unroll 1
  for (int g = 0; g < GROUPS; g += PER) {
#pragma unroll
    for (int i = 0; i < PER; ++i) put_tile(acc[i], lds + i * HIGH * 256);
#pragma unroll
    for (int i = 0; i < GROUPS; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j) acc[i][j] = i + PER < GROUPS ? acc[i + PER < GROUPS ? i + PER : 0][j] : Acc{};
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const int from = g * HIGH;
    if (whole) {
      if (n0 + 63 >= m0 + from) {  // below the diagonal nobody reads them
#pragma unroll 1
        for (int r = threadIdx.x >> 4 & 3; r < ROWS; r += 4) {
          f32x4 v;
          const int c = threadIdx.x & 15;
          __builtin_memcpy(&v, __builtin_assume_aligned(lds + (r * 256 + (c ^ (r & 15)) * 16), 16), 16);
          __builtin_memcpy(__builtin_assume_aligned(e.part + (m0 + from + r) * e.part_ld + n0 + c * 4, 16), &v, 16);
        }
      }
    } else {
#pragma unroll 1
      for (int r = from; r < from + ROWS; r += SYM ? 16 : 32) {
        if constexpr (SYM) {
          RowRuns<2> rows;
          TurnedRuns<2> turned;
          rows.load(e, m0, n0, r + r0);
          turned.load(e, m0, n0, r);
          rows.finish(e, lds, m0, n0, r + r0, from);
          turned.finish(e, lds, m0, n0, r, from);
        } else {
          const RowRuns<4> rows = next;
          if (r + 32 < GROUPS * HIGH) next.load(e, m0, n0, r + 32 + r0);
          rows.finish(e, lds, m0, n0, r + r0, from);
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
}

// Products of two planes each, BM x 128 of C per workgroup and 64 x 64 per wave, as k_parted: a
// step is 32 k of all four planes, 48 KB of LDS (32 KB at 128 x 128), and does lo hi, hi lo and
// hi hi; three (four) buffers, so that two (three) steps' loads run under the present one's 48
// products a wave (float32 2048 x 4096: X's product 103 us, 1.0 PFLOP/s of float16).
template <bool A_KC, bool B_KC, int BM, typename E>
__global__ void __launch_bounds__(2 * BM) k_pairs(Product g, E e) {
#ifdef __HIP_DEVICE_COMPILE__  // see k_tiled
  of_batch(g, e);
  constexpr int WAVES = BM / 32, BUFS = BM == 256 ? 3 : 4;
  using TA = Tile<f16, A_KC, BM, WAVES>;
  using TB = Tile<f16, B_KC, 128, WAVES>;
  constexpr int LOADS = 2 * (TA::LOADS + TB::LOADS);
  constexpr int A3 = BUFS == 4 ? 2 * TA::BYTES : 16, B3 = BUFS == 4 ? 2 * TB::BYTES : 16;
  __shared__ __attribute__((aligned(1024))) char a0[2 * TA::BYTES], a1[2 * TA::BYTES], a2[2 * TA::BYTES];
  __shared__ __attribute__((aligned(1024))) char b0[2 * TB::BYTES], b1[2 * TB::BYTES], b2[2 * TB::BYTES];
  __shared__ __attribute__((aligned(16))) char a3[A3], b3[B3];
  const int wave = wave_id();
  const Place place = place_of<BM, 128>(e);
  const int64_t m0 = place.m, n0 = place.n;
  const int wm = wave / 2 * 64, wn = wave % 2 * 64;
  f32x4 acc[4][4] = {};
  TA ta;
  TB tb;
  ta.init(g.a, g.lda, m0, g.M, 0);
  tb.init(g.b, g.ldb, n0, g.N, 0);
  auto load = [&](char* a, char* b, int left) {
    ta.load_from(a, ta.base, left);
    ta.load_from(a + TA::BYTES, ta.base + g.a_plane, left);
    ta.base += ta.step;
    tb.load_from(b, tb.base, left);
    tb.load_from(b + TB::BYTES, tb.base + g.b_plane, left);
    tb.base += tb.step;
    __builtin_amdgcn_sched_barrier(0);
  };
  auto step = [&](const char* la, const char* lb) {
    f16x8 b[2][4];
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int j = 0; j < 4; ++j) TB::fragment(b[p][j], lb + p * TB::BYTES, wn, j);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f16x8 a[2];
#pragma unroll
      for (int p = 0; p < 2; ++p) TA::fragment(a[p], la + p * TA::BYTES, wm, i);
      constexpr int pa[3] = {1, 0, 0}, pb[3] = {0, 1, 0};
#pragma unroll
      for (int t = 0; t < 3; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(b[pb[t]][j], a[pa[t]], acc[i][j], 0, 0, 0);
    }
  };
  int left = (int)g.K;
// Of a group of BUFS steps, those past the end are zeros.
#define EEC_STEP(T, A, B, FREE_A, FREE_B)                  \
  tile_barrier<(BUFS - 2) * LOADS>();                      \
  load(FREE_A, FREE_B, left - (T + BUFS - 1) * TA::BK);    \
  step(A, B)
  load(a0, b0, left);
  load(a1, b1, left - TA::BK);
  if constexpr (BUFS == 4) load(a2, b2, left - 2 * TA::BK);
  for (; left > 0; left -= BUFS * TA::BK) {
    if constexpr (BUFS == 4) {
      EEC_STEP(0, a0, b0, a3, b3);
      EEC_STEP(1, a1, b1, a0, b0);
      EEC_STEP(2, a2, b2, a1, b1);
      EEC_STEP(3, a3, b3, a2, b2);
    } else {
      EEC_STEP(0, a0, b0, a2, b2);
      EEC_STEP(1, a1, b1, a0, b0);
      EEC_STEP(2, a2, b2, a1, b1);
    }
  }
#undef EEC_STEP
  tile_barrier<0>();
  // 64 rows of sums in 16 KB for each wave: an A buffer holds one or two, a B buffer one
  char* mine;
  if constexpr (BUFS == 4)
    mine = wave == 0 ? a0 : wave == 1 ? a1 : wave == 2 ? a2 : a3;
  else
    mine = wave < 2 ? a0 + wave * 16384 : wave < 4 ? a1 + (wave - 2) * 16384 : wave < 6 ? a2 + (wave - 4) * 16384 : wave == 6 ? b0 : b1;
  finish<false, float, 16, 4>(e, mine, m0 + wm, n0 + wn, 0, acc);
#endif
}

// ------------------------------------------------------------------ small tiles

// 64 x 64 of C per workgroup, P planes, both operands with k along memory: for products whose
// large tiles would leave most CUs idle.  A step is 64 k of all planes, both halves of its
// operands' cache lines, four waves (32 x 32 each) for each half, joined in LDS at the end; three
// steps are on their way at a time, and what the epilogue reads is loaded before them (771 x 1025 float32: 13 us for A,
// 11 for A A and 12 for X's product, of which a launch and a tile's begin and end take 4).
template <int P, typename E>
__global__ void __launch_bounds__(512) k_small(Product g, E e) {
#ifdef __HIP_DEVICE_COMPILE__  // see k_tiled
  of_batch(g, e);
  using T = Tile<f16, true, 64, 4>;  // one plane of one half of one operand
  constexpr int LOADS = 2 * P, B = T::BYTES;
  // of each half P planes of A, then of B
  __shared__ __attribute__((aligned(1024))) char a0[4 * P * B], a1[4 * P * B], a2[4 * P * B], a3[4 * P * B];
  const int lane = threadIdx.x & 63, wave = wave_id() & 3, half = wave_id() >> 2;
  const Place place = place_of<64, 64>(e);
  const int64_t m0 = place.m, n0 = place.n;
  const int wm = wave / 2 * 32, wn = wave % 2 * 32, row = wave_id() * 8;
  f32x4 acc[2][2] = {};
  const char *pa = (const char*)g.a + m0 * g.lda * 2 + half * 64, *pb = (const char*)g.b + n0 * g.ldb * 2 + half * 64;
  const int line = wave * 16 + (lane >> 2), k = T::at_k(0);
  // lines past the end: not stored
  const uint32_t oa = (uint32_t)(min((int64_t)line, g.M - 1 - m0) * g.lda * 2) + k * 2;
  const uint32_t ob = (uint32_t)(min((int64_t)line, g.N - 1 - n0) * g.ldb * 2) + k * 2;
  auto load = [&](char* to, int left) {
    const bool is = half * 32 + k < left;
    const auto one = [&](char* at, const char* from, uint32_t off) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          __builtin_amdgcn_make_buffer_rsrc((void*)from, 0, 0x7fffffff, 0x00020000),
          (__attribute__((address_space(3))) void*)(at + wave * 1024), 16, is ? off : T::NOWHERE, 0, 0, 0);
    };
#pragma unroll
    for (int p = 0; p < P; ++p) {
      one(to + (half * 2 * P + p) * B, pa + p * g.a_plane, oa);
      one(to + (half * 2 * P + P + p) * B, pb + p * g.b_plane, ob);
    }
    pa += 128;
    pb += 128;
    __builtin_amdgcn_sched_barrier(0);
  };
  auto step = [&](const char* from) {
    const char* la = from + half * 2 * P * B;
    f16x8 a[2][P], b[2][P];
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        T::fragment(a[i][p], la + p * B, wm, i);
        T::fragment(b[i][p], la + (P + p) * B, wn, i);
      }
    // in rising size: (lo, hi), (hi, lo), (hi, hi)
#pragma unroll
    for (int t = P == 2 ? 0 : 2; t < 3; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(b[j][t == 1 ? P - 1 : 0], a[i][t == 0 ? P - 1 : 0], acc[i][j], 0, 0, 0);
  };
  RowRuns<1> rows;
  TurnedRuns<1> turned;
  rows.load(e, m0, n0, row + (lane >> 3));
  if constexpr (E::ACROSS) turned.load(e, m0, n0, row);
  int left = (int)g.K;
  load(a0, left);
  load(a1, left - 64);
  load(a2, left - 128);
#define EEC_STEP(T, NOW, FREE)     \
  tile_barrier<2 * LOADS>();       \
  load(FREE, left - (T + 3) * 64); \
  step(NOW);                       \
  if (left <= (T + 1) * 64) break
  for (;; left -= 256) {
    EEC_STEP(0, a0, a3);
    EEC_STEP(1, a1, a0);
    EEC_STEP(2, a2, a1);
    EEC_STEP(3, a3, a2);
  }
#undef EEC_STEP
  tile_barrier<0>();
  // sums of the first half of every step: 64 rows in a buffer of 16 KB; of the second in the next
  static_assert(4 * P * B >= 16384, "room for the sums");
  char* mine = (half == 0 ? a0 : a1) + wave / 2 * 8192;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) put_sums(mine, 16 * i + (lane & 15), wn / 4 + 4 * j + (lane >> 4), acc[i][j]);
  __syncthreads();
  const int at = threadIdx.x * 32;
  char *first = a0 + at, *second = a1 + at;
  f32x4 u[2], v[2];
  __builtin_memcpy(u, __builtin_assume_aligned(first, 16), 32);
  __builtin_memcpy(v, __builtin_assume_aligned(second, 16), 32);
  u[0] += v[0];
  u[1] += v[1];
  if constexpr (E::SYMMETRIC) {
    if (e.part) {
      const int r = threadIdx.x >> 3, c = (threadIdx.x & 7) * 2;  // 16-byte chunks c and c + 1, as put_sums permutes them
      float* to = e.part + (m0 + r) * e.part_ld + n0;
      __builtin_memcpy(__builtin_assume_aligned(to + (c ^ (r & 15)) * 4, 16), &u[0], 16);
      __builtin_memcpy(__builtin_assume_aligned(to + ((c + 1) ^ (r & 15)) * 4, 16), &u[1], 16);
      return;
    }
  }
  __builtin_memcpy(__builtin_assume_aligned(first, 16), u, 32);
  __syncthreads();
  rows.finish(e, a0, m0, n0, row + (lane >> 3), 0);
  if constexpr (E::ACROSS) turned.finish(e, a0, m0, n0, row, 0);
#endif
}

// Adds the splits of a symmetric product in order and finishes it: a block of 64 x 64 on or above the
// diagonal a workgroup.
template <typename E>
__global__ void __launch_bounds__(512) k_join_newton(E e, int splits, int64_t split_stride) {
#ifdef __HIP_DEVICE_COMPILE__
  __shared__ __attribute__((aligned(16))) char sums[16384];
  const int64_t i = blockIdx.y;
  e.rows.to += i * e.rows.to_batch;
  e.part += i * e.part_ld * e.part_ld;
  const Place place = place_of<64, 64>(e);
  const int r = threadIdx.x >> 3, c = (threadIdx.x & 7) * 2, row = wave_id() * 8;
  const float* from = e.part + (place.m + r) * e.part_ld + place.n + c * 4;
  f32x4 v[2] = {};
  for (int s0 = 0; s0 < splits; s0 += 4) {  // four splits on their way
    f32x4 t[4][2] = {};
#pragma unroll
    for (int s = 0; s < 4; ++s)
      if (s0 + s < splits) __builtin_memcpy(t[s], __builtin_assume_aligned(from + (s0 + s) * split_stride, 16), 32);
#pragma unroll
    for (int s = 0; s < 4; ++s) v[0] += t[s][0], v[1] += t[s][1];
  }
  put_sums(sums, r, c, v[0]);
  put_sums(sums, r, c + 1, v[1]);
  __syncthreads();
  RowRuns<1> rows;
  TurnedRuns<1> turned;
  rows.load(e, place.m, place.n, row + (threadIdx.x >> 3 & 7));
  turned.load(e, place.m, place.n, row);
  rows.finish(e, sums, place.m, place.n, row + (threadIdx.x >> 3 & 7), 0);
  turned.finish(e, sums, place.m, place.n, row, 0);
#endif
}

// ------------------------------------------------------------------ whole updates in one workgroup

// An update whose planes fit the LDS of one CU: every step of it in one launch, a workgroup of
// 16 waves a matrix (4 of 256 x 64 float32, five steps: 31 us).  X lies there by rows of the shorter side, two planes
// of HIGH rows (those past the end are zeros, and so are columns past the end), with one
// square that holds A, then B.  Two planes in every product.  TILES: rows of 16 in the shorter side.
constexpr int ONE_BYTES = 158 * 1024;
constexpr int one_high(int tiles) { return tiles < 2 ? 32 : 16 * tiles; }
// Bytes of the square, or of one matrix tile of each wave.
constexpr int one_square(int tiles) { return std::max(4 * one_high(tiles) * (one_high(tiles) + 8), 16 * 1024); }
struct NewtonOne {
  const void* g;
  int64_t ldg, stride;
  int rows, cols, length;  // length: of the longer side
  int xs;                  // elements from row to row of X
  int steps;
  double eps;
  void* y;
  float c[64][3];
};
template <typename T, int TILES>
__global__ void __launch_bounds__(1024) k_one(NewtonOne s) {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr int HIGH = one_high(TILES), AS = HIGH + 8, A_PLANE = HIGH * AS, KS = HIGH / 32;
  constexpr int PAIRS = TILES * (TILES + 1) / 2, EACH = (PAIRS + 15) / 16;  // tiles of A on and above the diagonal
  __shared__ __attribute__((aligned(16))) char lds[ONE_BYTES];
  __shared__ double join[16];
  const int lane = threadIdx.x & 63, wave = wave_id(), line = lane & 15, q = lane >> 4;
  f16* x = (f16*)lds;
  const int xs = s.xs, x_plane = HIGH * xs;
  f16* a = x + 2 * x_plane;
  const T* g = (const T*)s.g + blockIdx.x * s.stride;
  T* y = (T*)s.y + (int64_t)blockIdx.x * s.rows * s.cols;
  const bool wide = s.rows <= s.cols;
  for (int i = threadIdx.x; i < (x_plane + A_PLANE) / 4; i += 1024) ((i32x4*)lds)[i] = i32x4{};  // 2 planes, 8 a store
  __syncthreads();
  // g in runs of four elements of a row, dealt to the threads in turn; its float32 values wait
  // for their scale where X's two parts will be, half in each
  double sum = 0.0;
  {
    const int per_row = (s.cols + 3) / 4, down = 1024 / per_row, along = 1024 % per_row;
    const int dr = wide ? xs : 1, dc = wide ? 1 : xs;
    int r = threadIdx.x / per_row, c = threadIdx.x % per_row;
#pragma unroll 2
    for (int i = threadIdx.x; i < s.rows * per_row; i += 1024) {
      float v[4];
      load_run(g + (int64_t)r * s.ldg + c * 4, s.cols - c * 4, v);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c * 4 + j < s.cols) {
          const int at = r * dr + (c * 4 + j) * dc;
          const uint32_t u = __float_as_uint(v[j]);
          ((uint16_t*)x)[at] = (uint16_t)(u >> 16);
          ((uint16_t*)x)[at + x_plane] = (uint16_t)u;
          sum += (double)v[j] * v[j];
        }
      r += down, c += along;
      if (c >= per_row) c -= per_row, ++r;
    }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
  if (lane == 0) join[wave] = sum;
  __syncthreads();
  sum = 0.0;
  for (int i = 0; i < 16; ++i) sum += join[i];
  const double scale = scale_of(sum, s.eps);
  for (int i = threadIdx.x; i < x_plane / 8; i += 1024) {
    uint16_t h[8], l[8];
    f16 hi[8], lo[8];
    __builtin_memcpy(h, __builtin_assume_aligned(x + i * 8, 16), 16);
    __builtin_memcpy(l, __builtin_assume_aligned(x + x_plane + i * 8, 16), 16);
#pragma unroll
    for (int j = 0; j < 8; ++j) split2((float)(__uint_as_float((uint32_t)h[j] << 16 | l[j]) * scale), hi[j], lo[j]);
    __builtin_memcpy(__builtin_assume_aligned(x + i * 8, 16), hi, 16);
    __builtin_memcpy(__builtin_assume_aligned(x + x_plane + i * 8, 16), lo, 16);
  }
  __syncthreads();
  const auto row8 = [](const f16* p) {
    f16x8 v;
    __builtin_memcpy(&v, __builtin_assume_aligned(p, 16), 16);
    return v;
  };
  const auto pair4 = [](const f16* p, int plane) {  // four values from their parts
    f16 h[4], l[4];
    __builtin_memcpy(h, __builtin_assume_aligned(p, 8), 8);
    __builtin_memcpy(l, __builtin_assume_aligned(p + plane, 8), 8);
    return f32x4{(float)h[0] + (float)l[0], (float)h[1] + (float)l[1], (float)h[2] + (float)l[2], (float)h[3] + (float)l[3]};
  };
  // 16 rows from row 16 i and 16 from 16 j of a matrix, multiplied over every `by`-th 32 of n x 32 columns from the k-th on;
  // the columns' operand first, so that a lane has 4 adjacent columns of a row
  const auto gram = [&](const f16* p, int plane, int ld, int i, int j, int n, int k, int by) {
    f32x4 acc = {}, low = {};
    const f16 *pi = p + (16 * i + line) * ld + q * 8 + 32 * k, *pj = p + (16 * j + line) * ld + q * 8 + 32 * k;
#pragma unroll 2
    for (; k < n; k += by, pi += 32 * by, pj += 32 * by) {
      const f16x8 mh = row8(pi), ml = row8(pi + plane), ch = row8(pj), cl = row8(pj + plane);
      low = __builtin_amdgcn_mfma_f32_16x16x32_f16(ch, ml, low, 0, 0, 0);
      acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(ch, mh, acc, 0, 0, 0);
      low = __builtin_amdgcn_mfma_f32_16x16x32_f16(cl, mh, low, 0, 0, 0);
    }
    return acc + low;
  };
  // row 16 i + line, columns 16 j + 4 q and three more, and the same across the diagonal
  const auto put = [&](int i, int j, const f32x4& v) {
    const int r = 16 * i + line, c = 16 * j + 4 * q;
    f16 hi[4], lo[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) split2(v[u], hi[u], lo[u]);
    __builtin_memcpy(__builtin_assume_aligned(a + r * AS + c, 8), hi, 8);
    __builtin_memcpy(__builtin_assume_aligned(a + r * AS + c + A_PLANE, 8), lo, 8);
    if (i == j) return;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      a[(c + u) * AS + r] = hi[u];
      a[(c + u) * AS + r + A_PLANE] = lo[u];
    }
  };
  // the n-th tile on or above the diagonal
  const auto tile_at = [&](int n, int& i, int& j) {
    for (i = 0; n >= TILES - i; ++i) n -= TILES - i;
    j = i + n;
  };
  const int length32 = (s.length + 31) / 32, strips = (s.length + 15) / 16;
  const int parts = PAIRS >= 16 ? 1 : max(1, min(16 / PAIRS, length32));  // waves of a tile of A
  for (int step = 0; step < s.steps; ++step) {
    const float ca = s.c[step][0], cb = s.c[step][1], cc = s.c[step][2] / SCALE;
    int i, j;
    if (parts == 1) {  // A
      for (int n = wave; n < PAIRS; n += 16) {
        tile_at(n, i, j);
        put(i, j, gram(x, x_plane, xs, i, j, length32, 0, 1) * (1.f / SCALE));
      }
    } else {  // every tile by several waves, joined in order; where A will be, the old B is read no more
      f32x4* joined = (f32x4*)a;
      const int n = wave % PAIRS;
      tile_at(n, i, j);
      if (wave < parts * PAIRS) joined[wave * 64 + lane] = gram(x, x_plane, xs, i, j, length32, wave / PAIRS, parts);
      __syncthreads();
      f32x4 all = joined[n * 64 + lane];
      for (int t = 1; t < parts; ++t) all += joined[(n + t * PAIRS) * 64 + lane];
      __syncthreads();
      // a square of 32 whose second half of rows and columns is padding
      if (TILES * 16 < HIGH)
        for (int t = threadIdx.x; t < A_PLANE / 4; t += 1024) ((i32x4*)a)[t] = i32x4{};
      if (TILES * 16 < HIGH) __syncthreads();
      if (wave < PAIRS) put(i, j, all * (1.f / SCALE));
    }
    __syncthreads();
    f32x4 b[EACH];  // B, in A's place when everybody has read A
#pragma unroll
    for (int t = 0; t < EACH; ++t) {
      const int n = wave + 16 * t;
      if (n >= PAIRS) break;
      tile_at(n, i, j);
      b[t] = gram(a, A_PLANE, AS, i, j, KS, 0, 1) * cc + pair4(a + (16 * i + line) * AS + 16 * j + 4 * q, A_PLANE) * cb;
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < EACH; ++t) {
      const int n = wave + 16 * t;
      if (n >= PAIRS) break;
      tile_at(n, i, j);
      put(i, j, b[t]);
    }
    __syncthreads();
    // X: 16 columns of it depend on these alone, so a wave replaces them as soon as it has them;
    // rows and columns past the end stay zeros
    const bool last = step + 1 == s.steps;
    for (int n = wave; n < strips; n += 16) {
      typedef short s16x4 __attribute__((ext_vector_type(4)));
      f32x4 acc[TILES] = {};
#pragma unroll TILES < 8 ? KS : 1  // 128 registers a lane
      for (int k = 0; k < KS; ++k) {
        f16x8 c[2];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          s16x4 h[2];
#pragma unroll
          for (int u = 0; u < 2; ++u)
            h[u] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (__attribute__((address_space(3))) s16x4*)(x + p * x_plane + (k * 32 + q * 8 + (lane >> 2 & 3) + 4 * u) * xs + n * 16 +
                                                           (lane & 3) * 4));
          __builtin_memcpy(&c[p], h, 16);
        }
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
          const f16* p = a + (16 * t + line) * AS + k * 32 + q * 8;
          const f16x8 mh = row8(p), ml = row8(p + A_PLANE);
          acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(c[0], ml, acc[t], 0, 0, 0);
          acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(c[1], mh, acc[t], 0, 0, 0);
          acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(c[0], mh, acc[t], 0, 0, 0);
        }
      }
#pragma unroll
      for (int t = 0; t < TILES; ++t) {
        const int r = 16 * t + line, c = n * 16 + 4 * q;
        f16* p = x + r * xs + c;
        const f32x4 v = pair4(p, x_plane) * ca + acc[t] * (1.f / SCALE);
        if (!last) {
          f16 hi[4], lo[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) split2(v[u], hi[u], lo[u]);
          __builtin_memcpy(__builtin_assume_aligned(p, 8), hi, 8);
          __builtin_memcpy(__builtin_assume_aligned(p + x_plane, 8), lo, 8);
        } else if (r < (wide ? s.rows : s.cols)) {
          T* to = y + (wide ? r * s.cols + c : c * s.cols + r);
#pragma unroll
          for (int u = 0; u < 4; ++u, to += wide ? 1 : s.cols)
            if (c + u < s.length) *to = (T)(v[u] * (1.f / SCALE));
        }
      }
    }
    __syncthreads();
  }
#endif
}

// ------------------------------------------------------------------ norm and scaled planes

constexpr int SUMS = 256;  // partial sums of one matrix

template <typename T>
__global__ void __launch_bounds__(256) k_square_sums(const T* __restrict__ g, int64_t ldg, int64_t stride, int64_t rows,
                                                     int64_t cols, double* __restrict__ part) {
  constexpr int V = VEC<T>;
  __shared__ double join[4];
  const T* p = g + blockIdx.y * stride;
  // runs of 16 bytes dealt to the threads in turn, four at a time on their way
  const uint32_t per_row = (uint32_t)((cols + V - 1) / V), all = gridDim.x * 256, first = blockIdx.x * 256 + threadIdx.x;
  const uint32_t down = all / per_row, along = all % per_row;
  int64_t r = first / per_row;
  uint32_t c = first % per_row;
  double sum = 0.0;
  const auto next = [&] {
    r += down, c += along;
    if (c >= per_row) c -= per_row, ++r;
  };
  if (cols >= V) {
    while (r < rows) {
      // no branch, so that all four are on their way: a run past the row's end starts earlier, and one past the last row
      // is the last run again; what they read twice counts once
      T v[4][V];
      int from[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int64_t at = (int64_t)c * V, there = min(at, cols - V);
        from[t] = r < rows ? (int)(at - there) : V;
        __builtin_memcpy(v[t], p + min(r, rows - 1) * ldg + there, 16);
        next();
      }
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float u = j >= from[t] ? (float)v[t][j] : 0.f;
          sum += (double)u * u;
        }
    }
  } else {
    for (; r < rows; next()) {
      float v[V];
      load_run(p + r * ldg, cols, v);
#pragma unroll
      for (int j = 0; j < V; ++j) sum += (double)v[j] * v[j];
    }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
  if ((threadIdx.x & 63) == 0) join[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) part[blockIdx.y * SUMS + blockIdx.x] = (join[0] + join[1]) + (join[2] + join[3]);
}

struct Scaling {
  const void* g;
  int64_t ldg, stride, rows, cols;
  const double* part;
  int groups;  // of partial sums
  double eps;
  f16* x;
  int64_t ldx, plane, batch;  // elements from row to row, to the low part, to the next matrix
  f16* turned;                // X's transpose, or NULL
  int64_t ldt, turned_plane, turned_batch;
};
// X = SCALE g / (|g| + eps) as two planes, whose rows are padded with zeros to whole runs of 8.
template <typename T>
__global__ void __launch_bounds__(256) k_scaled(Scaling s) {
  __shared__ double join[4];
  const int64_t batch = blockIdx.y;
  double sum = (int)threadIdx.x < s.groups ? s.part[batch * SUMS + threadIdx.x] : 0.0;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
  if ((threadIdx.x & 63) == 0) join[threadIdx.x >> 6] = sum;
  __syncthreads();
  const double scale = scale_of((join[0] + join[1]) + (join[2] + join[3]), s.eps);
  const T* g = (const T*)s.g + batch * s.stride;
  f16 *x = s.x + batch * s.batch, *turned = s.turned + batch * s.turned_batch;
  __shared__ float tile[64][65];
  const int64_t across = (s.cols + 63) / 64, tiles = across * ((s.rows + 63) / 64);
  const int line = threadIdx.x >> 3, run = (threadIdx.x & 7) * 8;
  const auto put = [](f16* to, int64_t plane, const float (&v)[8]) {
    f16 hi[8], lo[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) split2(v[j], hi[j], lo[j]);
    __builtin_memcpy(__builtin_assume_aligned(to, 16), hi, 16);
    __builtin_memcpy(__builtin_assume_aligned(to + plane, 16), lo, 16);
  };
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int64_t r0 = t / across * 64, c0 = t % across * 64;
#pragma unroll
    for (int h = 0; h < 64; h += 32) {
      const int64_t r = r0 + line + h, c = c0 + run;
      float v[8];
      load_run<true>(g + r * s.ldg + c, r < s.rows ? s.cols - c : 0, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = r < s.rows && c + j < s.cols ? (float)(v[j] * scale) : 0.f;  // a NaN makes none of the padding
      if (r < s.rows && c < s.cols) put(x + r * s.ldx + c, s.plane, v);
      if (s.turned) {
#pragma unroll
        for (int j = 0; j < 8; ++j) tile[line + h][run + j] = v[j];
      }
    }
    if (!s.turned) continue;
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 64; h += 32) {
      const int64_t c = c0 + line + h, r = r0 + run;
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = tile[run + j][line + h];
      if (c < s.cols && r < s.rows) put(turned + c * s.ldt + r, s.turned_plane, v);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ host

// us of products of pairs on 256 x 128 tiles and on half of these: a round of the 256 CUs for every step of 32 k, and
// for a tile's begin and end (float32 2048 x 4096, A A: 72 wide tiles 85 us, 136
// of the others 62).
double pairs_us(int64_t tiles, int64_t K, bool wide) {
  return (double)((tiles + 255) / 256) * (wide ? 30 + 0.8 * K / 32 : 15 + 0.75 * K / 32);
}
bool wide_pairs(int64_t t256, int64_t t128, int64_t K) { return pairs_us(t256, K, true) <= pairs_us(t128, K, false); }

// How a call is run, and its workspace: partial sums, X and the next X (two planes each; with
// small tiles their transposes too), A and B.
enum Way { ONE, SMALL_TILES, LARGE_TILES };
struct OrthoPlan {
  Way way;
  bool wide;
  int64_t side, length, ldx, ldt, lds, x_plane, t_plane, ab_plane;  // elements
  int planes;                                                      // of A and B, and of the products' operands
  int splits;        // of A = X X^T over k
  int64_t k_split;   // a multiple of 64
  int64_t split_ld;  // of their sums
  size_t off_part, off_x, off_next, off_t, off_next_t, off_a, off_b, off_split, bytes;
};
// Rows of 16 that k_one holds the shorter side in, and the stride of X's rows there: 16 bytes more than
// whole steps, so that rows start in different banks.
int one_tiles(int64_t side) { return side <= 16 ? 1 : side <= 32 ? 2 : side <= 64 ? 4 : 8; }
int64_t one_stride(int64_t length) { return up(length, 32) + 8; }
OrthoPlan ortho_plan(int64_t batch, int64_t rows, int64_t cols, int32_t dtype) {
  OrthoPlan p{};
  p.wide = rows <= cols;
  p.side = std::min(rows, cols);
  p.length = std::max(rows, cols);
  if (p.side <= 128) {
    const int tiles = one_tiles(p.side);
    if (4 * one_high(tiles) * one_stride(p.length) + one_square(tiles) <= ONE_BYTES) {
      p.way = ONE;
      return p;
    }
  }
  // large tiles where they fill the chip
  p.way = batch * tiles_of(p.side, p.length, 128) >= 200 ? LARGE_TILES : SMALL_TILES;
  // one plane where its error is of the output's size: 2.1e-3 to 2.5e-3 with the output's rounding below a side of 256, where
  // two cost little (small products wait for memory), 1.9e-3 to 2.1e-3 above; a float16 output would show it eightfold
  p.planes = dtype != EEC_BF16 || p.side < 256 ? 2 : 1;
  if (p.planes == 2 && dtype == EEC_BF16) p.way = SMALL_TILES;
  p.ldx = up(cols, 128);
  p.lds = up(p.side, 128);
  p.x_plane = rows * p.ldx;
  p.ab_plane = p.side * p.lds;
  if (p.way == SMALL_TILES) {
    p.ldt = up(rows, 128);
    p.t_plane = cols * p.ldt;
  }
  // The sum of A's tiles is split where that gains: us of a step of 32 k, of a tile's begin and end, and of the join
  // with its 5 TB/s (53 x 5616 float16, six steps: 303 us whole, 146 so).
  const bool small = p.way == SMALL_TILES, two = p.planes == 2;
  const int64_t t64 = batch * newton_tiles<64, 64>(p.side, p.side, true), t128 = batch * newton_tiles<128, 128>(p.side, p.side, true);
  const int64_t t256 = batch * newton_tiles<256, 128>(p.side, p.side, true);
  const auto product_us = [&](int64_t s) {
    const int64_t K = p.length / s;
    if (!small && two) return std::min(pairs_us(t256 * s, K, true), pairs_us(t128 * s, K, false));
    return (double)(((small ? t64 : t128) * s + 255) / 256) * (small ? 4 + (two ? 0.36 : 0.22) * K / 32 : 10 + 0.25 * K / 32);
  };
  p.split_ld = up(p.side, 256);
  double best = 1e30;
  for (int s = 1; s == 1 || (s <= 64 && p.length / s >= 512 && t64 * s <= 8192); s = s < 8 ? s + 1 : s * 2) {
    const double us = product_us(s) + (s > 1 ? 9 + 2.0 * batch * p.side * p.side * s / 5e6 : 0);
    if (us < best) best = us, p.splits = s;
  }
  p.k_split = up((p.length + p.splits - 1) / p.splits, 64);
  p.splits = (int)((p.length + p.k_split - 1) / p.k_split);
  size_t at = 0;
  const auto take = [&](size_t& off, int64_t elements, int size) {
    off = at;
    at += align256((size_t)batch * (size_t)elements * (size_t)size);
  };
  take(p.off_part, SUMS, 8);
  take(p.off_x, 2 * p.x_plane, 2);
  take(p.off_next, 2 * p.x_plane, 2);
  take(p.off_t, 2 * p.t_plane, 2);
  take(p.off_next_t, 2 * p.t_plane, 2);
  take(p.off_a, p.planes * p.ab_plane, 2);
  take(p.off_b, p.planes * p.ab_plane, 2);
  take(p.off_split, p.splits > 1 ? p.splits * p.split_ld * p.split_ld : 0, 4);
  p.bytes = at;
  return p;
}

// One product on large tiles.
template <bool A_KC, bool B_KC, typename Y, bool SYM>
void large_product(hipStream_t st, int64_t batch, const Product& g, const NewtonEpilogue<Y, SYM>& e, int planes, unsigned splits = 1) {
  using E = NewtonEpilogue<Y, SYM>;
  // only bf16 takes one plane
  if constexpr (std::is_same<Y, float>::value || std::is_same<Y, f16>::value || std::is_same<Y, Planes>::value) {
    if (planes == 2) {
      const int64_t t256 = newton_tiles<256, 128>(e.M, e.N, SYM), t128 = newton_tiles<128, 128>(e.M, e.N, SYM);
      if (wide_pairs(t256 * batch * splits, t128 * batch * splits, g.K / splits))
        k_pairs<A_KC, B_KC, 256, E><<<dim3((unsigned)t256, (unsigned)batch, splits), 512, 0, st>>>(g, e);
      else
        k_pairs<A_KC, B_KC, 128, E><<<dim3((unsigned)t128, (unsigned)batch, splits), 256, 0, st>>>(g, e);
      return;
    }
  }
  if constexpr (std::is_same<Y, bf16>::value || std::is_same<Y, Planes>::value) {
    const int64_t t256 = newton_tiles<256, 256>(e.M, e.N, SYM), t128 = newton_tiles<128, 128>(e.M, e.N, SYM);
    const double steps = (double)g.K / 32 / splits;  // as plan_product
    const double us128 = (double)((t128 * batch * splits + 255) / 256) * (10 + 0.25 * steps);
    const double us256 = (double)((t256 * batch * splits + 255) / 256) * (20 + 0.49 * steps);
    if (us256 < us128)
      k_tiled<f16, float, A_KC, B_KC, 2, 4, 8, 4, false, E><<<dim3((unsigned)t256, (unsigned)batch, splits), 512, 0, st>>>(g, e);
    else
      k_tiled<f16, float, A_KC, B_KC, 2, 2, 4, 8, false, E><<<dim3((unsigned)t128, (unsigned)batch, splits), 256, 0, st>>>(g, e);
  }
}
template <typename Y, bool SYM, bool TURN>
void small_product(hipStream_t st, int64_t batch, const Product& g, const NewtonEpilogue<Y, SYM, TURN>& e, int planes, unsigned splits = 1) {
  using E = NewtonEpilogue<Y, SYM, TURN>;
  const dim3 grid((unsigned)newton_tiles<64, 64>(e.M, e.N, SYM), (unsigned)batch, splits);
  if constexpr (std::is_same<Y, bf16>::value || std::is_same<Y, Planes>::value) {
    if (planes == 1) {
      k_small<1, E><<<grid, 512, 0, st>>>(g, e);
      return;
    }
  }
  k_small<2, E><<<grid, 512, 0, st>>>(g, e);
}

}  // namespace

size_t ortho_workspace(int64_t batch, int64_t rows, int64_t cols, int32_t dtype) {
  return rows > 0 && cols > 0 ? ortho_plan(batch, rows, cols, dtype).bytes : 0;
}

void launch_ortho(hipStream_t st, const OrthoArgs& a, char* ws) {
  const OrthoPlan p = ortho_plan(a.batch, a.rows, a.cols, a.dtype);
  by_type(a.dtype, [&](auto zero) {
    using T = decltype(zero);
    if (p.way == ONE) {
      NewtonOne s{a.g,     a.ldg, a.stride, (int)a.rows, (int)a.cols, (int)p.length, (int)one_stride(p.length),
                  a.steps, a.eps, a.y,      {}};
      for (int i = 0; i < 3 * a.steps; ++i) s.c[i / 3][i % 3] = (float)a.coefficients[i];
      const dim3 grid((unsigned)a.batch);
      const int tiles = one_tiles(p.side);
      if (tiles == 1) k_one<T, 1><<<grid, 1024, 0, st>>>(s);
      if (tiles == 2) k_one<T, 2><<<grid, 1024, 0, st>>>(s);
      if (tiles == 4) k_one<T, 4><<<grid, 1024, 0, st>>>(s);
      if (tiles == 8) k_one<T, 8><<<grid, 1024, 0, st>>>(s);
      return;
    }
    double* part = (double*)(ws + p.off_part);
    f16 *x = (f16*)(ws + p.off_x), *next = (f16*)(ws + p.off_next), *A = (f16*)(ws + p.off_a), *B = (f16*)(ws + p.off_b);
    f16 *xt = (f16*)(ws + p.off_t), *next_t = (f16*)(ws + p.off_next_t);
    const bool small = p.way == SMALL_TILES;
    const int64_t x_batch = 2 * p.x_plane, t_batch = 2 * p.t_plane, ab_batch = p.planes * p.ab_plane;
    const int64_t low = p.planes == 2 ? p.ab_plane : 0;
    const int64_t xp = 2 * p.x_plane, tp = 2 * p.t_plane, ap = 2 * p.ab_plane;  // bytes from plane to plane
    const int groups = (int)std::min<int64_t>(SUMS, (a.rows * a.cols + 4095) / 4096);
    k_square_sums<T><<<dim3((unsigned)groups, (unsigned)a.batch), 256, 0, st>>>((const T*)a.g, a.ldg, a.stride, a.rows, a.cols, part);
    const Scaling s{a.g, a.ldg, a.stride, a.rows, a.cols, part, groups, a.eps, x, p.ldx, p.x_plane, x_batch,
                    small ? xt : nullptr, p.ldt, p.t_plane, t_batch};
    const int64_t tiles = tiles_of(a.rows, a.cols, 64);
    k_scaled<T><<<dim3((unsigned)std::min<int64_t>(tiles, 4096), (unsigned)a.batch), 256, 0, st>>>(s);
    for (int32_t i = 0; i < a.steps; ++i) {
      const double* c = a.coefficients + 3 * i;
      const bool last = i + 1 == a.steps;
      // A = X X^T (X^T X)
      NewtonEpilogue<Planes, true> e{};
      e.M = e.N = p.side;
      e.beta = 1.f / SCALE;
      e.rows = NewtonTo{nullptr, 0, A, low, p.lds, 0, ab_batch};
      const bool by_rows = p.wide || !small;  // the operand is X itself
      e.a_batch = e.b_batch = by_rows ? x_batch : t_batch;
      const f16* of = by_rows ? x : xt;
      const int64_t ld = by_rows ? p.ldx : p.ldt, plane = by_rows ? xp : tp;
      const Product gram{of, of, ld, ld, p.side, p.side, p.length, p.k_split, plane, plane};
      const unsigned splits = (unsigned)p.splits;
      e.part = splits > 1 ? (float*)(ws + p.off_split) : nullptr;
      e.part_ld = p.split_ld;
      e.k_along = small || p.wide;
      if (small)
        small_product(st, a.batch, gram, e, p.planes, splits);
      else if (p.wide)
        large_product<true, true>(st, a.batch, gram, e, p.planes, splits);
      else
        large_product<false, false>(st, a.batch, gram, e, p.planes, splits);
      if (splits > 1) {
        const dim3 grid((unsigned)newton_tiles<64, 64>(p.side, p.side, true), (unsigned)a.batch);
        k_join_newton<<<grid, 512, 0, st>>>(e, p.splits, a.batch * p.split_ld * p.split_ld);
        e.part = nullptr;
      }
      // B = b A + c A A
      const Product square{A, A, p.lds, p.lds, p.side, p.side, p.side, p.side, ap, ap};
      e.alpha = (float)c[1];
      e.beta = (float)(c[2] / SCALE);
      e.a_batch = e.b_batch = ab_batch;
      e.rows = NewtonTo{A, low, B, low, p.lds, ab_batch, ab_batch};
      if (small)
        small_product(st, a.batch, square, e, p.planes);
      else
        large_product<true, true>(st, a.batch, square, e, p.planes);
      // X <- a X + B X (X B); small tiles multiply rows of B, and of X, with those of X's transpose, and of B
      const Product update = p.wide ? Product{B, small ? xt : x, p.lds, small ? p.ldt : p.ldx, a.rows, a.cols, p.side, p.side, ap, small ? tp : xp}
                                    : Product{x, B, p.ldx, p.lds, a.rows, a.cols, p.side, p.side, xp, ap};
      const auto fill = [&](auto u) {
        u.M = a.rows;
        u.N = a.cols;
        u.alpha = (float)c[0];
        u.beta = 1.f / SCALE;
        u.rows = NewtonTo{x, p.x_plane, next, p.x_plane, p.ldx, x_batch, x_batch};
        u.a_batch = p.wide ? ab_batch : x_batch;
        u.b_batch = !p.wide ? ab_batch : small ? t_batch : x_batch;
        return u;
      };
      if (last) {
        auto u = fill(NewtonEpilogue<T, false>{});
        u.y = (T*)a.y;
        u.y_batch = a.rows * a.cols;
        if (small)
          small_product(st, a.batch, update, u, p.planes);
        else if (p.wide)
          large_product<true, false>(st, a.batch, update, u, p.planes);
        else
          large_product<true, true>(st, a.batch, update, u, p.planes);
      } else if (small) {
        auto u = fill(NewtonEpilogue<Planes, false, true>{});
        u.turned = NewtonTo{xt, p.t_plane, next_t, p.t_plane, p.ldt, t_batch, t_batch};
        small_product(st, a.batch, update, u, p.planes);
      } else {
        const auto u = fill(NewtonEpilogue<Planes, false>{});
        if (p.wide)
          large_product<true, false>(st, a.batch, update, u, p.planes);
        else
          large_product<true, true>(st, a.batch, update, u, p.planes);
      }
      std::swap(x, next);
      std::swap(xt, next_t);
    }
  });
}

}  // namespace eec
