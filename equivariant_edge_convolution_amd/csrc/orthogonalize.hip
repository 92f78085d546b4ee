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
// grow 3.4-fold each.  The products take hi alone for 16-bit types, where their error, 1e-3 to
// 2e-3 of the result in norm, is of the output's own size (bf16 operands: 1e-2 for normal g,
// up to 0.3 where a few directions dominate; without lo 4e-2 there), and hi hi + hi lo + lo hi
// for float32, as exact as float32 products (2e-7 to 1e-5, those 1e-6 to 2e-5).  B is
// computed from A as rounded: the errors of b A and c A^2 then cancel at singular values near 1.
// Singular values stay below 3.5 (checked on the host), so 2^12 of them fit float16, and
// elements down to 2^-26 of the largest possible keep 11 bits.
#include "product.hpp"

namespace eec {
namespace {

constexpr float SCALE = 4096.f;

struct NewtonEpilogue {
  int64_t M, N;         // of the product
  int64_t ld;           // of from and to
  const f16* from;      // alpha from + beta C, or NULL
  int64_t from_plane;   // elements to its low part, 0: none
  f16* to;
  int64_t to_plane;     // 0: no low part
  float alpha, beta;
  bool symmetric;
  int32_t dtype;        // of y
  void* y;              // [M][N] instead of `to`, or NULL
  int64_t a_batch, b_batch, from_batch, to_batch, y_batch;  // elements to the next matrix
};

__device__ __forceinline__ void of_batch(Product& g, NewtonEpilogue& e) {
  const int64_t i = blockIdx.y;
  g.a = (const f16*)g.a + i * e.a_batch;
  g.b = (const f16*)g.b + i * e.b_batch;
  if (e.from) e.from += i * e.from_batch;
  if (e.to) e.to += i * e.to_batch;
  if (e.y) e.y = (char*)e.y + i * e.y_batch * (e.dtype == EEC_F32 ? 4 : 2);
}

// Symmetric: the tiles that reach above the diagonal, row of tiles after row of tiles.
template <int BM, int BN>
__device__ __forceinline__ Place place_of(const NewtonEpilogue& e) {
  static_assert(BM % BN == 0, "a row of tiles starts at its diagonal");
  if (!e.symmetric) {
    Epilogue plain{};
    plain.M = e.M;
    plain.N = e.N;
    return place_of<BM, BN>(plain);
  }
  const uint32_t tiles_n = (uint32_t)((e.N + BN - 1) / BN);
  uint32_t t = dealt(), i = 0;
  for (uint32_t row = tiles_n; t >= row; row = tiles_n - i * (BM / BN)) t -= row, ++i;
  return Place{(int64_t)i * BM, (int64_t)(i * (BM / BN) + t) * BN, 0};
}
template <int BM, int BN>
int64_t newton_tiles(int64_t M, int64_t N, bool symmetric) {
  const int64_t m = (M + BM - 1) / BM, n = (N + BN - 1) / BN;
  if (!symmetric) return m * n;
  int64_t all = 0;
  for (int64_t i = 0; i < m; ++i) all += n - i * (BM / BN);
  return all;
}

// Eight adjacent columns of one row, `left` of which exist and are stored from column `first` on.
__device__ __forceinline__ void finish_newton(const NewtonEpilogue& e, int64_t m, int64_t n, int64_t left, int first,
                                              float (&v)[8]) {
  float was[8] = {};
  if (e.from) {
    const f16* p = e.from + m * e.ld + n;
    load_run(p, left, was);
    if (e.from_plane) {
      float low[8];
      load_run(p + e.from_plane, left, low);
#pragma unroll
      for (int i = 0; i < 8; ++i) was[i] += low[i];
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = e.alpha * was[i] + e.beta * v[i];
  if (e.y) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= 1.f / SCALE;
    if (e.dtype == EEC_F32) store_run((float*)e.y + m * e.N + n, left, v);
    if (e.dtype == EEC_F16) store_run((f16*)e.y + m * e.N + n, left, v);
    if (e.dtype == EEC_BF16) store_run((bf16*)e.y + m * e.N + n, left, v);
    return;
  }
  f16 hi[8], lo[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    hi[i] = (f16)v[i];
    lo[i] = (f16)(v[i] - (float)hi[i]);
  }
  f16* p = e.to + m * e.ld + n;
  if (left >= 8 && first <= 0) {
    __builtin_memcpy(p, hi, 16);
    if (e.to_plane) __builtin_memcpy(p + e.to_plane, lo, 16);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left && i >= first) {
        p[i] = hi[i];
        if (e.to_plane) p[i + e.to_plane] = lo[i];
      }
  }
}

// As finish_wave.  Symmetric: elements above the diagonal (and on it) are stored, and those above
// it once more across it, from columns of the same sums: each is written once, by one lane.
template <bool G, typename O, int HIGH, int PER, typename Acc, int GROUPS, int NB>
__device__ __forceinline__ void finish(const NewtonEpilogue& e, char* lds, int64_t m0, int64_t n0, int,
                                       Acc (&acc)[GROUPS][NB]) {
  constexpr int ROWS = PER * HIGH;
  const int lane = threadIdx.x & 63;
  const int r0 = lane >> 3, col = (lane & 7) * 8;
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
#pragma unroll 1
    for (int r = r0; r < ROWS; r += 8) {
      const int64_t m = top + r, n = n0 + col;
      const int64_t first = e.symmetric ? m - n : 0;
      if (m < e.M && n < e.N && first < 8) {
        float v[8];
#pragma unroll
        for (int u = 0; u < 8; u += 4)
          __builtin_memcpy(&v[u], __builtin_assume_aligned(lds + (r * 256 + (((col + u) / 4) ^ (r & 15)) * 16), 16), 16);
        finish_newton(e, m, n, e.N - n, (int)max(first, (int64_t)0), v);
      }
    }
    if (e.symmetric) {  // row n0 + lane of the other side: eight of this side's rows at a time
      const int64_t m = n0 + lane;
#pragma unroll 1
      for (int r = 0; r < ROWS; r += 8) {
        const int64_t n = top + r;
        const int64_t left = min(m, e.N) - n;  // those above the diagonal
        if (m < e.N && left > 0) {
          float v[8];
#pragma unroll
          for (int u = 0; u < 8; ++u)
            __builtin_memcpy(&v[u], lds + ((r + u) * 256 + ((lane / 4) ^ (r + u & 15)) * 16 + lane % 4 * 4), 4);
          finish_newton(e, m, n, left, 0, v);
        }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
}

// Products of two planes each, 256 x 128 of C per workgroup and 64 x 64 per wave, as k_parted:
// a step is 32 k of all four planes, 48 KB of LDS, and does lo hi, hi lo and hi hi; three
// buffers, so that two steps' loads run under the present one's 48 products a wave.
template <bool A_KC, bool B_KC>
__global__ void __launch_bounds__(512) k_pairs(Product g, NewtonEpilogue e) {
#ifdef __HIP_DEVICE_COMPILE__  // see k_tiled
  of_batch(g, e);
  using TA = Tile<f16, A_KC, 256, 8>;
  using TB = Tile<f16, B_KC, 128, 8>;
  constexpr int LOADS = 2 * (TA::LOADS + TB::LOADS);
  __shared__ __attribute__((aligned(1024))) char a0[2 * TA::BYTES], a1[2 * TA::BYTES], a2[2 * TA::BYTES];
  __shared__ __attribute__((aligned(1024))) char b0[2 * TB::BYTES], b1[2 * TB::BYTES], b2[2 * TB::BYTES];
  const int wave = wave_id();
  const Place place = place_of<256, 128>(e);
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
  load(a0, b0, left);
  load(a1, b1, left - TA::BK);
  for (; left > 0; left -= 3 * TA::BK) {  // three steps, of which those past the end are zeros
    tile_barrier<LOADS>();
    load(a2, b2, left - 2 * TA::BK);
    step(a0, b0);
    tile_barrier<LOADS>();
    load(a0, b0, left - 3 * TA::BK);
    step(a1, b1);
    tile_barrier<LOADS>();
    load(a1, b1, left - 4 * TA::BK);
    step(a2, b2);
  }
  tile_barrier<0>();
  // 64 rows of sums in 16 KB for each wave: two in an A buffer, one in a B buffer
  char* mine = wave < 2 ? a0 + wave * 16384 : wave < 4 ? a1 + (wave - 2) * 16384 : wave < 6 ? a2 + (wave - 4) * 16384 : wave == 6 ? b0 : b1;
  finish<false, float, 16, 4>(e, mine, m0 + wm, n0 + wn, 0, acc);
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
  const int64_t per_row = (cols + V - 1) / V, total = rows * per_row;
  double sum = 0.0;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / per_row, c = i % per_row * V;
    float v[V];
    load_run(p + r * ldg + c, cols - c, v);
#pragma unroll
    for (int j = 0; j < V; ++j) sum += (double)v[j] * v[j];
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
  f16 *x, *other;             // X, and the buffer of the next step's
  int64_t ldx, plane, batch;  // elements from row to row, to the low part, to the next matrix
  f16 *a, *b;                 // A and B
  int64_t side, lds, ab_plane, ab_batch;  // ab_plane 0: one plane
};
// X = SCALE g / (|g| + eps) as two planes; the columns that pad its rows are zeros, here and in
// the next step's buffer, and so are those that pad A and B to whole loads.
template <typename T>
__global__ void __launch_bounds__(256) k_scaled(Scaling s) {
  __shared__ double join[4];
  const int64_t batch = blockIdx.y;
  double sum = (int)threadIdx.x < s.groups ? s.part[batch * SUMS + threadIdx.x] : 0.0;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
  if ((threadIdx.x & 63) == 0) join[threadIdx.x >> 6] = sum;
  __syncthreads();
  const double scale = (double)SCALE / (sqrt((join[0] + join[1]) + (join[2] + join[3])) + s.eps);
  const T* g = (const T*)s.g + batch * s.stride;
  f16 *x = s.x + batch * s.batch, *other = s.other + batch * s.batch;
  const int64_t per_row = s.ldx / 8, total = s.rows * per_row, all = (int64_t)gridDim.x * 256;
  const int64_t first = (int64_t)blockIdx.x * 256 + threadIdx.x;
  for (int64_t i = first; i < total; i += all) {
    const int64_t r = i / per_row, c = i % per_row * 8, at = r * s.ldx + c;
    float v[8];
    load_run<true>(g + r * s.ldg + c, s.cols - c, v);
    f16 hi[8], lo[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float u = (float)(v[j] * scale);
      hi[j] = c + j < s.cols ? (f16)u : (f16)0.f;  // an infinite scale makes no NaN of the padding
      lo[j] = c + j < s.cols ? (f16)(u - (float)hi[j]) : (f16)0.f;
    }
    __builtin_memcpy(__builtin_assume_aligned(x + at, 16), hi, 16);
    __builtin_memcpy(__builtin_assume_aligned(x + at + s.plane, 16), lo, 16);
    if (c + 8 > s.cols) {  // real columns are written by the first step
      const f16 none[8] = {};
      __builtin_memcpy(__builtin_assume_aligned(other + at, 16), none, 16);
      __builtin_memcpy(__builtin_assume_aligned(other + at + s.plane, 16), none, 16);
    }
  }
  f16 *pa = s.a + batch * s.ab_batch, *pb = s.b + batch * s.ab_batch;
  for (int64_t r = first; r < s.side; r += all)
    for (int64_t c = s.side; c < up(s.side, 8); ++c) {
      pa[r * s.lds + c] = pb[r * s.lds + c] = (f16)0.f;
      if (s.ab_plane) pa[r * s.lds + c + s.ab_plane] = pb[r * s.lds + c + s.ab_plane] = (f16)0.f;
    }
}

// ------------------------------------------------------------------ host

// Workspace of one call: partial sums, X and the next X (two planes each), A and B.
struct OrthoPlan {
  bool wide;
  int64_t side, ldx, lds, x_plane, ab_plane;  // elements
  int planes;                                 // of A and B, and of the products' operands
  size_t off_part, off_x, off_next, off_a, off_b, bytes;
};
OrthoPlan ortho_plan(int64_t batch, int64_t rows, int64_t cols, int32_t dtype) {
  OrthoPlan p{};
  p.wide = rows <= cols;
  p.side = std::min(rows, cols);
  p.ldx = up(cols, 128);
  p.lds = up(p.side, 128);
  p.planes = dtype == EEC_F32 ? 2 : 1;
  p.x_plane = rows * p.ldx;
  p.ab_plane = p.side * p.lds;
  const size_t x = align256((size_t)batch * 2 * p.x_plane * 2), ab = align256((size_t)batch * p.planes * p.ab_plane * 2);
  p.off_part = 0;
  p.off_x = align256((size_t)batch * SUMS * 8);
  p.off_next = p.off_x + x;
  p.off_a = p.off_next + x;
  p.off_b = p.off_a + ab;
  p.bytes = p.off_b + ab;
  return p;
}

template <bool A_KC, bool B_KC>
void newton_product(hipStream_t st, int64_t batch, const Product& g, const NewtonEpilogue& e, int planes) {
  if (planes == 2) {
    const dim3 grid((unsigned)newton_tiles<256, 128>(e.M, e.N, e.symmetric), (unsigned)batch);
    k_pairs<A_KC, B_KC><<<grid, 512, 0, st>>>(g, e);
    return;
  }
  const int64_t t256 = newton_tiles<256, 256>(e.M, e.N, e.symmetric), t128 = newton_tiles<128, 128>(e.M, e.N, e.symmetric);
  const double steps = (double)g.K / 32;  // as plan_product
  const double us128 = (double)((t128 * batch + 255) / 256) * (10 + 0.25 * steps);
  const double us256 = (double)((t256 * batch + 255) / 256) * (20 + 0.49 * steps);
  if (us256 < us128)
    k_tiled<f16, float, A_KC, B_KC, 2, 4, 8, 4, false, NewtonEpilogue><<<dim3((unsigned)t256, (unsigned)batch), 512, 0, st>>>(g, e);
  else
    k_tiled<f16, float, A_KC, B_KC, 2, 2, 4, 8, false, NewtonEpilogue><<<dim3((unsigned)t128, (unsigned)batch), 256, 0, st>>>(g, e);
}

}  // namespace

size_t ortho_workspace(int64_t batch, int64_t rows, int64_t cols, int32_t dtype) {
  return ortho_plan(batch, rows, cols, dtype).bytes;
}

void launch_ortho(hipStream_t st, const OrthoArgs& a, char* ws) {
  const OrthoPlan p = ortho_plan(a.batch, a.rows, a.cols, a.dtype);
  double* part = (double*)(ws + p.off_part);
  f16 *x = (f16*)(ws + p.off_x), *next = (f16*)(ws + p.off_next), *A = (f16*)(ws + p.off_a), *B = (f16*)(ws + p.off_b);
  const int64_t x_batch = 2 * p.x_plane, ab_batch = p.planes * p.ab_plane, low = p.planes == 2 ? p.ab_plane : 0;
  const int groups = (int)std::min<int64_t>(SUMS, (a.rows * a.cols + 4095) / 4096);
  by_type(a.dtype, [&](auto zero) {
    using T = decltype(zero);
    k_square_sums<T><<<dim3((unsigned)groups, (unsigned)a.batch), 256, 0, st>>>((const T*)a.g, a.ldg, a.stride, a.rows, a.cols, part);
    const Scaling s{a.g, a.ldg, a.stride, a.rows, a.cols, part, groups, a.eps, x, next, p.ldx, p.x_plane, x_batch, A, B,
                    p.side, p.lds, low, ab_batch};
    const int64_t chunks = a.rows * p.ldx / 8;
    k_scaled<T><<<dim3((unsigned)std::min<int64_t>((chunks + 255) / 256, 2048), (unsigned)a.batch), 256, 0, st>>>(s);
  });
  for (int32_t i = 0; i < a.steps; ++i) {
    const double* c = a.coefficients + 3 * i;
    const bool last = i + 1 == a.steps;
    const int64_t n = std::max(a.rows, a.cols), xp = 2 * p.x_plane, ap = 2 * p.ab_plane;  // bytes from plane to plane
    // A = X X^T (X^T X)
    Product gram{x, x, p.ldx, p.ldx, p.side, p.side, n, n, xp, xp};
    NewtonEpilogue e{p.side, p.side, p.lds, nullptr, 0, A, low, 0.f, 1.f / SCALE, true, a.dtype, nullptr, x_batch, x_batch,
                     0, ab_batch, 0};
    if (p.wide)
      newton_product<true, true>(st, a.batch, gram, e, p.planes);
    else
      newton_product<false, false>(st, a.batch, gram, e, p.planes);
    // B = b A + c A A
    const Product square{A, A, p.lds, p.lds, p.side, p.side, p.side, p.side, ap, ap};
    e.from = A;
    e.from_plane = low;
    e.to = B;
    e.alpha = (float)c[1];
    e.beta = (float)(c[2] / SCALE);
    e.a_batch = e.b_batch = e.from_batch = ab_batch;
    newton_product<true, true>(st, a.batch, square, e, p.planes);
    // X <- a X + B X (X B)
    NewtonEpilogue u{a.rows, a.cols, p.ldx, x, p.x_plane, next, p.x_plane, (float)c[0], 1.f / SCALE, false, a.dtype,
                     last ? a.y : nullptr, ab_batch, x_batch, x_batch, x_batch, a.rows * a.cols};
    if (p.wide) {
      const Product update{B, x, p.lds, p.ldx, a.rows, a.cols, p.side, p.side, ap, xp};
      newton_product<true, false>(st, a.batch, update, u, p.planes);
    } else {
      const Product update{x, B, p.ldx, p.lds, a.rows, a.cols, p.side, p.side, xp, ap};
      std::swap(u.a_batch, u.b_batch);
      newton_product<true, true>(st, a.batch, update, u, p.planes);
    }
    std::swap(x, next);
  }
}

}  // namespace eec
