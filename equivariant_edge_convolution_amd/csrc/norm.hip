// Residual addition + root-mean-square norm over the last axis, and its backward.
//
//   s = x + residual (float32, unrounded),  rstd = 1 / sqrt(mean(s^2) + eps),
//   y = s rstd w;   8-bit rows: scale = max(max|y|, 2^-100) / 448,
//   q = e4m3(y / scale).
//   backward, with a = gy w and xhat = s rstd:
//   gx = rstd (a - xhat mean(a xhat)) + gsum,   gw = sum_rows gy xhat.
//
// Both passes are bound by memory: a row is read once into registers, its sums
// are taken there, and what is written is written from there.  A row belongs to
// one wave where it fits 4 accesses of 16 bytes per lane (no barrier at all),
// to a workgroup of 4 or 16 waves where it is wider, and is read twice by one
// workgroup where 16 waves cannot hold it.
#include <algorithm>

#include "dense.hpp"
#include "eec_internal.hpp"

namespace eec {
namespace {
using namespace dense;

constexpr float E4M3_MAX = 448.f;
// Floor of a quantised row's largest magnitude, so that 448 / amax is finite.
constexpr float AMAX_FLOOR = 7.8886090522101181e-31f;  // 2^-100

// Workgroups of a launch at most (a launch counts its threads in 32 bits).
constexpr int64_t MAX_GROUPS = 1 << 20;

struct NormIn {
  const void *x, *residual, *weight;
  int64_t ldx, ldr;
  int64_t rows;
  int width;
  float eps;
};
struct NormOut {
  void *sum, *y;
  float *scale, *rstd;
};

// Sum (maximum) over the TPR lanes of a row.  `red` holds one slot per wave;
// the two barriers make it reusable by the next call.
template <int TPR, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* red) {
  v = MAX ? wave_nan_max(v) : wave_sum(v);
  if constexpr (TPR > 64) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < TPR / 64; ++i) v = MAX ? nan_max(v, red[i]) : v + red[i];
  }
  return v;
}

// Rows in the registers of TPR threads, CH accesses of 16 bytes each; rows are
// dealt to the row groups of the grid in turn.
template <typename T, int TPR, int CH>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) k_norm(NormIn in, NormOut out) {
  constexpr int V = VEC<T>;
  constexpr int GROUPS = TPR < 256 ? 256 / TPR : 1;
  __shared__ float red[TPR / 64];
  const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  const int n = in.width;
  const T* w = (const T*)in.weight;
  for (int64_t row = (int64_t)blockIdx.x * GROUPS + grp; row < in.rows; row += (int64_t)gridDim.x * GROUPS) {
    const T* x = (const T*)in.x + row * in.ldx;
    const T* r = in.residual ? (const T*)in.residual + row * in.ldr : nullptr;
    float s[CH][V];
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int at = (c * TPR + t) * V;
      load_run<true>(x + at, n - at, s[c]);
      if (r) {
        float b[V];
        load_run<true>(r + at, n - at, b);
#pragma unroll
        for (int i = 0; i < V; ++i) s[c][i] += b[i];
      }
#pragma unroll
      for (int i = 0; i < V; ++i) ss += s[c][i] * s[c][i];
    }
    if (out.sum) {
      T* o = (T*)out.sum + row * n;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int at = (c * TPR + t) * V;
        store_run(o + at, n - at, s[c]);
      }
    }
    ss = row_reduce<TPR, false>(ss, red);
    const float rstd = 1.f / sqrtf(ss / n + in.eps);
    if (out.rstd && t == 0) out.rstd[row] = rstd;
    float amax = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int at = (c * TPR + t) * V;
      float g[V];
      if (w) load_run(w + at, n - at, g);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        s[c][i] = s[c][i] * rstd * (w ? g[i] : 1.f);
        amax = nan_max(amax, fabsf(s[c][i]));
      }
      if (!out.scale) store_run((T*)out.y + row * n + at, n - at, s[c]);
    }
    if (out.scale) {
      amax = row_reduce<TPR, true>(amax, red);
      amax = amax < AMAX_FLOOR ? AMAX_FLOOR : amax;
      if (t == 0) out.scale[row] = amax / E4M3_MAX;
      const float up = E4M3_MAX / amax;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int at = (c * TPR + t) * V;
#pragma unroll
        for (int i = 0; i < V; ++i) s[c][i] *= up;
        store_run_e4m3((uint8_t*)out.y + row * n + at, n - at, s[c]);
      }
    }
  }
}

// Rows too wide for registers: one workgroup of 1024 reads a row two or three times.
template <typename T>
__global__ void __launch_bounds__(1024) k_norm_wide(NormIn in, NormOut out) {
  constexpr int V = VEC<T>;
  __shared__ float red[16];
  const int n = in.width;
  const T* w = (const T*)in.weight;
  for (int64_t row = blockIdx.x; row < in.rows; row += gridDim.x) {
    const T* x = (const T*)in.x + row * in.ldx;
    const T* r = in.residual ? (const T*)in.residual + row * in.ldr : nullptr;
    auto load = [&](int64_t at, float (&s)[V]) {
      load_run(x + at, n - at, s);
      if (r) {
        float b[V];
        load_run<true>(r + at, n - at, b);
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] += b[i];
      }
    };
    float ss = 0.f;
    for (int64_t at = threadIdx.x * V; at < n; at += 1024 * V) {
      float s[V];
      load(at, s);
#pragma unroll
      for (int i = 0; i < V; ++i) ss += s[i] * s[i];
      if (out.sum) store_run((T*)out.sum + row * n + at, n - at, s);
    }
    ss = row_reduce<1024, false>(ss, red);
    const float rstd = 1.f / sqrtf(ss / n + in.eps);
    if (out.rstd && threadIdx.x == 0) out.rstd[row] = rstd;
    float amax = 0.f, up = 1.f;
    for (int pass = out.scale ? 0 : 1; pass < 2; ++pass) {
      for (int64_t at = threadIdx.x * V; at < n; at += 1024 * V) {
        float s[V], g[V];
        load(at, s);
        if (w) load_run(w + at, n - at, g);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          s[i] = s[i] * rstd * (w ? g[i] : 1.f);
          if (pass == 0) amax = nan_max(amax, fabsf(s[i]));
          s[i] *= up;
        }
        if (pass == 1) {
          if (out.scale)
            store_run_e4m3((uint8_t*)out.y + row * n + at, n - at, s);
          else
            store_run((T*)out.y + row * n + at, n - at, s);
        }
      }
      if (pass == 0) {
        amax = row_reduce<1024, true>(amax, red);
        amax = amax < AMAX_FLOOR ? AMAX_FLOOR : amax;
        if (threadIdx.x == 0) out.scale[row] = amax / E4M3_MAX;
        up = E4M3_MAX / amax;
      }
    }
  }
}

struct NormBwd {
  const void *gy, *s, *weight, *gsum;
  const float* rstd;
  int64_t ldgy, lds, ldgs;
  int64_t rows;
  int width;
  void* gx;
  float* part;    // [gridDim.x][width] sums of gy xhat, or NULL
  void* gweight;  // with one workgroup the sums themselves instead, or NULL
};

// s is read as the forward stored it: in 16 bits rounded, and so 2 bytes where float32 or
// x and the residual again would be 4 (16384 x 4096 bf16: 134 MB of 537).  Its rounding is
// of the outputs' own size: 2.5e-3 off in norm against 64 bits, 1.8e-3 with s in float32.
//
// TPR threads per row, rows dealt in turn to all row groups of the grid; each
// thread keeps the weight gradient of its columns in registers over its rows
// and the groups of a workgroup are joined in LDS at the end, so the partial
// sums are one row of `part` per workgroup and their order is fixed.
template <typename T, int TPR, int CH>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) k_norm_bwd(NormBwd a) {
  constexpr int V = VEC<T>;
  constexpr int GROUPS = TPR < 256 ? 256 / TPR : 1;
  __shared__ float red[TPR / 64];
  __shared__ float join[GROUPS > 1 ? GROUPS - 1 : 1][GROUPS > 1 ? TPR * V : 1];
  const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  const int n = a.width;
  const T* w = (const T*)a.weight;
  float g[CH][V], acc[CH][V] = {};
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int at = (c * TPR + t) * V;
    if (w) {
      load_run(w + at, n - at, g[c]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) g[c][i] = 1.f;
    }
  }
  for (int64_t row = (int64_t)blockIdx.x * GROUPS + grp; row < a.rows; row += (int64_t)gridDim.x * GROUPS) {
    const T* gy = (const T*)a.gy + row * a.ldgy;
    const T* s = (const T*)a.s + row * a.lds;
    const float rstd = a.rstd[row];
    float xh[CH][V], q[CH][V];
    float dot = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int at = (c * TPR + t) * V;
      load_run<true>(s + at, n - at, xh[c]);
      load_run<true>(gy + at, n - at, q[c]);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        xh[c][i] *= rstd;
        acc[c][i] += q[c][i] * xh[c][i];
        q[c][i] *= g[c][i];
        dot += q[c][i] * xh[c][i];
      }
    }
    dot = row_reduce<TPR, false>(dot, red) / n;
    const T* gs = a.gsum ? (const T*)a.gsum + row * a.ldgs : nullptr;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int at = (c * TPR + t) * V;
      float b[V];
      if (gs) load_run<true>(gs + at, n - at, b);
#pragma unroll
      for (int i = 0; i < V; ++i) q[c][i] = rstd * (q[c][i] - xh[c][i] * dot) + (gs ? b[i] : 0.f);
      if (a.gx) store_run((T*)a.gx + row * n + at, n - at, q[c]);
    }
  }
  if (a.part == nullptr && a.gweight == nullptr) return;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int at = (c * TPR + t) * V;
    if constexpr (GROUPS > 1) {
      __syncthreads();
      if (grp > 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) join[grp - 1][t * V + i] = acc[c][i];
      }
      __syncthreads();
      if (grp > 0) continue;
      for (int k = 0; k < GROUPS - 1; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) acc[c][i] += join[k][t * V + i];
    }
    if (a.gweight)
      store_run((T*)a.gweight + at, n - at, acc[c]);
    else
      store_run(a.part + (int64_t)blockIdx.x * n + at, n - at, acc[c]);
  }
}

// Rows too wide for registers: two reads of a row, and the weight gradient kept
// in the workgroup's own row of `part`.
template <typename T>
__global__ void __launch_bounds__(1024) k_norm_bwd_wide(NormBwd a) {
  constexpr int V = VEC<T>;
  __shared__ float red[16];
  const int n = a.width;
  const T* w = (const T*)a.weight;
  float* o = a.part ? a.part + (int64_t)blockIdx.x * n : nullptr;
  if (o && blockIdx.x >= a.rows)
    for (int64_t at = threadIdx.x; at < n; at += 1024) o[at] = 0.f;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* gy = (const T*)a.gy + row * a.ldgy;
    const T* s = (const T*)a.s + row * a.lds;
    const T* gs = a.gsum ? (const T*)a.gsum + row * a.ldgs : nullptr;
    const float rstd = a.rstd[row];
    float dot = 0.f;
    for (int64_t at = threadIdx.x * V; at < n; at += 1024 * V) {
      float xh[V], q[V], g[V], p[V];
      load_run(s + at, n - at, xh);
      load_run(gy + at, n - at, q);
      if (w) load_run(w + at, n - at, g);
      if (o && row != blockIdx.x) load_run(o + at, n - at, p);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float u = q[i] * (xh[i] * rstd);
        p[i] = row != blockIdx.x ? p[i] + u : u;
        dot += u * (w ? g[i] : 1.f);
      }
      if (o) store_run(o + at, n - at, p);
    }
    dot = row_reduce<1024, false>(dot, red) / n;
    if (a.gx == nullptr) continue;
    for (int64_t at = threadIdx.x * V; at < n; at += 1024 * V) {
      float xh[V], q[V], g[V], b[V];
      load_run(s + at, n - at, xh);
      load_run(gy + at, n - at, q);
      if (w) load_run(w + at, n - at, g);
      if (gs) load_run<true>(gs + at, n - at, b);
#pragma unroll
      for (int i = 0; i < V; ++i)
        q[i] = rstd * (q[i] * (w ? g[i] : 1.f) - xh[i] * rstd * dot) + (gs ? b[i] : 0.f);
      store_run((T*)a.gx + row * n + at, n - at, q);
    }
  }
}

// Column sums of the partial rows [parts][n]: 64 columns per workgroup, whose 16
// waves deal the rows in turn, eight of them on their way at a time (one by one
// each would wait for memory), and are joined in wave order.
template <typename T>
__global__ void __launch_bounds__(1024) k_column_sum(const float* __restrict__ part, int parts, int64_t n,
                                                     T* __restrict__ out) {
  constexpr int WAVES = 16, TOGETHER = 8;
  __shared__ float join[WAVES][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t col = (int64_t)blockIdx.x * 64 + lane;
  float v = 0.f;
  if (col < n)
    for (int p = wave; p < parts; p += WAVES * TOGETHER) {
      float t[TOGETHER];
#pragma unroll
      for (int i = 0; i < TOGETHER; ++i) t[i] = p + WAVES * i < parts ? part[(int64_t)(p + WAVES * i) * n + col] : 0.f;
#pragma unroll
      for (int i = 0; i < TOGETHER; ++i) v += t[i];
    }
  join[wave][lane] = v;
  __syncthreads();
  if (wave == 0 && col < n) {
#pragma unroll
    for (int i = 1; i < WAVES; ++i) v += join[i][lane];
    out[col] = (T)v;
  }
}

// Threads per row and accesses per thread for rows of `width` elements of T, as
// (TPR, CH); CH = 0: the row does not fit.
template <typename T, typename F>
void by_width(int64_t width, F&& f) {
  constexpr int V = VEC<T>;
  using std::integral_constant;
#define EEC_CASE(TPR, CH) \
  if (width <= (int64_t)(TPR) * (CH) * V) return f(integral_constant<int, TPR>(), integral_constant<int, CH>())
  EEC_CASE(64, 1);
  EEC_CASE(64, 2);
  EEC_CASE(64, 4);
  EEC_CASE(256, 2);
  EEC_CASE(256, 4);
  EEC_CASE(1024, 2);
  EEC_CASE(1024, 4);
#undef EEC_CASE
  f(integral_constant<int, 1024>(), integral_constant<int, 0>());
}

template <typename F>
void by_type(int32_t dtype, F&& f) {
  if (dtype == EEC_F32) return f(float());
  if (dtype == EEC_F16) return f(f16());
  f(bf16());
}

// Workgroups of the backward: enough to fill the chip twice over, and few enough
// that the partial sums of the weight gradient stay a small share of the rows.  A few
// rows take one, which needs no second launch for the sums (about 4 us).
// `at_once`: rows of one workgroup's turn (4 where a row is a wave's), so that each of them
// has some (500 x 128 float32 backward, in a graph: 5.9 us, 8.3 with 512 of which most had none).
constexpr int64_t ONE_GROUP_ROWS = 8;
int64_t norm_bwd_groups(int64_t rows, int64_t at_once) {
  return rows <= ONE_GROUP_ROWS ? 1 : std::min<int64_t>((rows + at_once - 1) / at_once, 512);
}

}  // namespace

void launch_norm(hipStream_t st, int32_t dtype, int64_t rows, int64_t width, const void* x, int64_t ldx,
                 const void* residual, int64_t ldr, const void* weight, float eps, void* sum, void* y, float* scale,
                 float* rstd) {
  const NormIn in{x, residual, weight, ldx, ldr, rows, (int)width, eps};
  const NormOut out{sum, y, scale, rstd};
  by_type(dtype, [&](auto zero) {
    using T = decltype(zero);
    by_width<T>(width, [&](auto tpr, auto ch) {
      constexpr int TPR = decltype(tpr)::value, CH = decltype(ch)::value;
      if constexpr (CH == 0) {
        k_norm_wide<T><<<dim3((unsigned)std::min<int64_t>(rows, MAX_GROUPS)), 1024, 0, st>>>(in, out);
      } else {
        constexpr int B = TPR < 256 ? 256 : TPR, PER = B / TPR;
        const int64_t groups = std::min<int64_t>((rows + PER - 1) / PER, MAX_GROUPS);
        k_norm<T, TPR, CH><<<dim3((unsigned)groups), B, 0, st>>>(in, out);
      }
    });
  });
}

size_t norm_bwd_workspace(int64_t rows, int64_t width) {
  return align256(4 * (size_t)norm_bwd_groups(rows, 1) * (size_t)width);
}

void launch_norm_bwd(hipStream_t st, int32_t dtype, int64_t rows, int64_t width, const void* gy, int64_t ldgy,
                     const void* s, int64_t lds, const void* weight, const float* rstd, const void* gsum,
                     int64_t ldgs, void* gx, void* gweight, char* ws) {
  int64_t groups = 1;
  NormBwd a{gy, s, weight, gsum, rstd, ldgy, lds, ldgs, rows, (int)width, gx, gweight ? (float*)ws : nullptr, nullptr};
  bool summed = gweight == nullptr;
  by_type(dtype, [&](auto zero) {
    using T = decltype(zero);
    by_width<T>(width, [&](auto tpr, auto ch) {
      constexpr int TPR = decltype(tpr)::value, CH = decltype(ch)::value;
      if constexpr (CH == 0) {
        groups = norm_bwd_groups(rows, 1);
        k_norm_bwd_wide<T><<<dim3((unsigned)groups), 1024, 0, st>>>(a);
      } else {
        groups = norm_bwd_groups(rows, TPR < 256 ? 256 / TPR : 1);
        if (groups == 1 && gweight) {
          a.part = nullptr;
          a.gweight = gweight;
          summed = true;
        }
        k_norm_bwd<T, TPR, CH><<<dim3((unsigned)groups), TPR < 256 ? 256 : TPR, 0, st>>>(a);
      }
    });
  });
  if (!summed) launch_column_sum(st, dtype, (const float*)ws, (int)groups, width, gweight);
}

void launch_column_sum(hipStream_t st, int32_t dtype, const float* part, int parts, int64_t n, void* out) {
  by_type(dtype, [&](auto zero) {
    using T = decltype(zero);
    k_column_sum<T><<<dim3((unsigned)((n + 63) / 64)), 1024, 0, st>>>(part, parts, n, (T*)out);
  });
}

}  // namespace eec
