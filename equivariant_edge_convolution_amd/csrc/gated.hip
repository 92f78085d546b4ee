// Gated layer: z = x w^T + bias, whose first `outer` columns are the gate and the others
// the value, y = act(z_gate) z_value; and its backward.
//
// Forward: one product with both halves of w and the gate's epilogue (product.hpp, G).
// Backward, from the z that the forward kept:
//   gz_gate = gy z_value act'(z_gate),  gz_value = gy act(z_gate)      one pass over gy and z
//   gx = gz w,  gw = gz^T x,  gbias = sum_rows gz                      as of a layer of 2 outer outputs
#include "product.hpp"

namespace eec {
namespace {

struct GateGrad {
  const void *gy, *preact;
  int64_t ldgy, rows, outer, per;  // per: rows of one strip
  int32_t act;
  void* gz;        // [rows][2 outer], or NULL
  Packing packed;  // or gz packed (packed.to not NULL)
  float* part;     // [strips][2 outer] column sums of gz before its rounding, or NULL
  void* gbias;     // with one strip the sums themselves instead, or NULL
};

// gz = gy (z_value act'(z_gate), act(z_gate)) and its column sums.  Bound by memory: gy and
// both halves of z are read once, both halves of gz written.  A wave takes 64 x 8 (float32: 4)
// outputs, a workgroup's waves deal the rows of a strip in turn.  16-bit types: gz is rounded to
// the type, as the matrix instructions take it (its column sums are not); two parts of it would double
// both products, 830 of 930 us.  That leaves gx and gw 2.3e-3 off in norm against 64 bits (8192 x 2048 ->
// 8192 bf16), where products of gz in float32 are 1.7e-3 off by their own rounding.  Packed, the
// threads past `outer` clear the columns that pad a row.
template <typename T>
__global__ void __launch_bounds__(256) k_gate_grad(GateGrad a) {
  constexpr int V = VEC<T>;
  __shared__ float join[3][2][64 * V];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t col = ((int64_t)blockIdx.x * 64 + lane) * V, left = a.outer - col;
  const int64_t r0 = (int64_t)blockIdx.y * a.per, r1 = min(a.packed.to ? a.packed.to_rows : a.rows, r0 + a.per);
  // the first padding column of this thread, beyond those with outputs
  const int64_t pad = 2 * a.outer + col - (a.outer + V - 1) / V * V;
  float sum[2][V] = {};
  const auto put = [&](int64_t r, int64_t at, int64_t n, const float (&g)[V]) {
    if constexpr (std::is_same<T, float>::value) {
      bf16 q[3][V];
#pragma unroll
      for (int i = 0; i < V; ++i) split3(g[i], q[0][i], q[1][i], q[2][i]);
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        bf16* to = (bf16*)(a.packed.to + k * a.packed.plane) + r * a.packed.to_ld + at;
        if (n >= V) {
          __builtin_memcpy(to, q[k], 2 * V);
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (i < n) to[i] = q[k][i];
        }
      }
    } else {
      store_run((T*)a.packed.to + r * a.packed.to_ld + at, n, g);
    }
  };
  for (int64_t r = r0 + wave; r < r1; r += 4) {
    const int64_t here = r < a.rows ? left : 0;  // rows of the padding are zeros
    float gy[V], z[V], v[V], gate[V];
    load_run<true>((const T*)a.gy + r * a.ldgy + col, here, gy);
    load_run<true>((const T*)a.preact + r * 2 * a.outer + col, here, z);
    load_run<true>((const T*)a.preact + (r * 2 + 1) * a.outer + col, here, v);
#pragma unroll
    for (int i = 0; i < V; ++i) gate[i] = gy[i] * v[i], v[i] = z[i];
    act_slopes<T>(gate, z, a.act);
    act_values<T>(v, a.act);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] *= gy[i];
    if (left > 0) {
      if (a.gz) {
        store_run((T*)a.gz + r * 2 * a.outer + col, left, gate);
        store_run((T*)a.gz + (r * 2 + 1) * a.outer + col, left, v);
      }
      if (a.packed.to) {
        put(r, col, left, gate);
        put(r, a.outer + col, left, v);
      }
    } else if (a.packed.to && pad < a.packed.to_ld) {
      put(r, pad, a.packed.to_ld - pad, gate);  // loaded as zeros
    }
#pragma unroll
    for (int i = 0; i < V; ++i) sum[0][i] += gate[i], sum[1][i] += v[i];
  }
  if (a.part == nullptr && a.gbias == nullptr) return;
  if (wave > 0) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < V; ++i) join[wave - 1][h][lane * V + i] = sum[h][i];
  }
  __syncthreads();
  if (wave == 0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) sum[h][i] += join[k][h][lane * V + i];
      if (a.gbias)
        store_run((T*)a.gbias + h * a.outer + col, left, sum[h]);
      else
        store_run(a.part + ((int64_t)blockIdx.y * 2 + h) * a.outer + col, left, sum[h]);
    }
  }
}

}  // namespace

size_t gated_workspace(int64_t rows, int64_t outer, int64_t inner, int32_t dtype, int32_t out_dtype) {
  return fwd_plan(rows, outer, inner, dtype, out_dtype, true).bytes;
}

void launch_gated(hipStream_t st, const LinearArgs& a, char* ws) { launch_forward<true>(st, a, ws); }

// That of a layer of 2 outer outputs whose gz is not gy itself.
size_t gated_bwd_workspace(int64_t rows, int64_t outer, int64_t inner, int32_t dtype) {
  return bwd_plan(rows, 2 * outer, inner, dtype, EEC_ACT_SILU).bytes;
}

void launch_gated_bwd(hipStream_t st, const LinearBwdArgs& a, char* ws) {
  const BwdPlan p = bwd_plan(a.rows, 2 * a.outer, a.inner, a.dtype, EEC_ACT_SILU);
  by_type(a.dtype, [&](auto zero) {
    using T = decltype(zero);
    const bool products = a.gx != nullptr || a.gw != nullptr, packed = p.gz && products;
    const Packing z = packing(a.dtype, nullptr, 0, a.rows, 2 * a.outer, packed ? ws + p.off_gz : nullptr);
    if (a.outer > 0 && ((products && a.rows > 0) || a.gbias)) {
      const int64_t strips = act_grad_strips(a.rows, 2 * a.outer, a.dtype), cols = 64 * VEC<T>;
      const int64_t rows = packed ? z.to_rows : a.rows;
      const int64_t width = up(a.outer, VEC<T>) + (packed ? z.to_ld - 2 * a.outer : 0);
      const GateGrad q{a.gy, a.preact, a.ldgy, a.rows, a.outer, (rows + strips - 1) / strips, a.act,
                       products && !packed ? ws + p.off_gz : nullptr, z,
                       a.gbias && strips > 1 ? (float*)(ws + p.off_part) : nullptr, strips == 1 ? a.gbias : nullptr};
      k_gate_grad<T><<<dim3((unsigned)((width + cols - 1) / cols), (unsigned)strips), 256, 0, st>>>(q);
      if (a.gbias && strips > 1)
        launch_column_sum(st, a.dtype, (const float*)(ws + p.off_part), (int)strips, 2 * a.outer, a.gbias);
    }
    LinearBwdArgs both = a;
    both.outer = 2 * a.outer;
    if (products)
      launch_backward_products(st, both, p, packed ? z.to : ws + p.off_gz, packed ? z.to_ld : 2 * a.outer, packed, z.plane, ws);
  });
}

}  // namespace eec
