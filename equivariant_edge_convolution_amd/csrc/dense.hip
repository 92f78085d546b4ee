// Dense layer y = act(x w^T + bias) + residual and its backward products.
//
// As products C[m][n] = sum_k A(m, k) B(n, k), m the rows of x (of gz, of gz^T) and n
// the rows of w (the columns of w, of x):
//   forward  A = x  [m][k],  B = w  [n][k];
//   gx       A = gz [m][k],  B = w  [k][n];
//   gw       A = gz [k][m],  B = x  [k][n].
#include "product.hpp"

namespace eec {
namespace {

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


}  // namespace

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

size_t linear_workspace(int64_t rows, int64_t outer, int64_t inner, int32_t dtype, int32_t out_dtype) {
  return fwd_plan(rows, outer, inner, dtype, out_dtype, false).bytes;
}

void launch_linear(hipStream_t st, const LinearArgs& a, char* ws) { launch_forward<false>(st, a, ws); }

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
    if (products) launch_backward_products(st, a, p, gz, ldgz, packed, z.plane, ws);
  });
}

void launch_backward_products(hipStream_t st, const LinearBwdArgs& a, const BwdPlan& p, const void* gz, int64_t ldgz,
                              bool packed, int64_t plane, char* ws) {
  by_type(a.dtype, [&](auto zero) {
    using T = decltype(zero);
    Product gx{gz, a.w, ldgz, a.ldw, a.rows, a.inner, a.outer, 0, plane, 0};
    Product gw{gz, a.x, ldgz, a.ldx, a.outer, a.inner, a.rows, 0, plane, 0};
    if (p.others) {
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
