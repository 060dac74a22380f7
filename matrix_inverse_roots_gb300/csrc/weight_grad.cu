// The weight gradient of a linear layer whose input is kept as an 8-bit checkpoint:
//   dW[o][i] = gamma[i] sum_t dz[t][o] n[t][i] + beta[i] db[o],   db[o] = sum_t dz[t][o],
// n the checkpoint's values, written as a matrix or as the B x B blocks of
// shampoo_accumulate.
#include "act_q8.cuh"
#include "dash_internal.h"
#include "train_internal.h"

namespace dash {

constexpr int WG_TILE = 64, WG_K = 16;

// One CTA per 64 x 64 tile, 4 x 4 outputs per thread, fp32 arithmetic.
template <typename T, int FMT>
__global__ void __launch_bounds__(256) weight_grad_kernel(const WeightGradArgs a, const float* db) {
  __shared__ float sa[WG_K][WG_TILE + 4], sb[WG_K][WG_TILE + 4];
  const long long ng = (a.cols + Q8_GROUP - 1) / Q8_GROUP;
  const long long o0 = static_cast<long long>(blockIdx.y) * WG_TILE;
  const long long i0 = static_cast<long long>(blockIdx.x) * WG_TILE;
  const int tr = threadIdx.x / 16, tc = threadIdx.x % 16;
  float acc[4][4] = {};
  for (long long t0 = 0; t0 < a.rows; t0 += WG_K) {
    for (int e = threadIdx.x; e < WG_K * WG_TILE; e += 256) {
      const int k = e / WG_TILE, j = e % WG_TILE;
      const long long t = t0 + k;
      float va = 0.0f, vb = 0.0f;
      if (t < a.rows) {
        if (o0 + j < a.outs) va = Elem<T>::to(static_cast<const T*>(a.dz)[t * a.lddz + o0 + j]);
        if (i0 + j < a.cols)
          vb = q8_value<FMT>(a.q[t * ng * Q8_GROUP + i0 + j]) *
               q8_scale(a.scale[t * ng + (i0 + j) / Q8_GROUP]);
      }
      sa[k][j] = va;
      sb[k][j] = vb;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < WG_K; ++k)
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          acc[u][v] = fmaf(sa[k][tr * 4 + u], sb[k][tc * 4 + v], acc[u][v]);
    __syncthreads();
  }
  const long long pr = a.block ? (a.outs + a.block - 1) / a.block * a.block : a.outs;
  const long long pc = a.block ? (a.cols + a.block - 1) / a.block * a.block : a.cols;
  for (int u = 0; u < 4; ++u)
    for (int v = 0; v < 4; ++v) {
      const long long o = o0 + tr * 4 + u, i = i0 + tc * 4 + v;
      if (o >= pr || i >= pc) continue;
      float d = 0.0f;
      if (o < a.outs && i < a.cols) {
        d = acc[u][v];
        if (a.gamma) d *= load_dt(a.gamma, a.wdt, i);
        if (a.beta) d = fmaf(db[o], load_dt(a.beta, a.wdt, i), d);
      }
      long long at = o * a.ldw + i;
      if (a.block) {
        const long long b = a.block;
        at = ((o / b) * (pc / b) + i / b) * b * b + (o % b) * b + i % b;
      }
      if (a.odt == DASH_DT_F32)
        static_cast<float*>(a.dw)[at] = d;
      else if (a.odt == DASH_DT_BF16)
        static_cast<__nv_bfloat16*>(a.dw)[at] = __float2bfloat16_rn(d);
      else
        static_cast<__half*>(a.dw)[at] = __float2half_rn(d);
    }
}

static size_t round256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

// Workspace: db (when only beta needs it), then the column sums' partials.
size_t weight_grad_ws(const WeightGradArgs& a) {
  const size_t outs = static_cast<size_t>(a.outs);
  return round256(outs * 4) + round256(outs * 4 * col_sum_parts(a.rows, a.outs));
}

template <typename T>
static dash_status weight_grad_t(const WeightGradArgs& a, const float* db, cudaStream_t st) {
  const long long b = a.block;
  const long long pr = b ? (a.outs + b - 1) / b * b : a.outs;
  const long long pc = b ? (a.cols + b - 1) / b * b : a.cols;
  const dim3 grid(static_cast<unsigned>((pc + WG_TILE - 1) / WG_TILE),
                  static_cast<unsigned>((pr + WG_TILE - 1) / WG_TILE));
  if (a.fmt == DASH_Q8_INT8)
    weight_grad_kernel<T, DASH_Q8_INT8><<<grid, 256, 0, st>>>(a, db);
  else
    weight_grad_kernel<T, DASH_Q8_E4M3><<<grid, 256, 0, st>>>(a, db);
  return cudaGetLastError() == cudaSuccess ? DASH_OK : DASH_ERR_CUDA;
}

dash_status launch_weight_grad(const WeightGradArgs& a, void* ws, cudaStream_t st) {
  float* db = a.db;
  if (a.db || a.beta) {
    if (!db) db = static_cast<float*>(ws);
    float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) +
                                           round256(static_cast<size_t>(a.outs) * 4));
    const dash_status s = launch_col_sum(a.dz, a.dt, a.rows, a.outs, a.lddz, part, db, st);
    if (s != DASH_OK) return s;
  }
  const int rec = trace_begin(st);
  const dash_status s = a.dt == DASH_DT_F32    ? weight_grad_t<float>(a, db, st)
                        : a.dt == DASH_DT_BF16 ? weight_grad_t<__nv_bfloat16>(a, db, st)
                                               : weight_grad_t<__half>(a, db, st);
  const double t = static_cast<double>(a.rows), o = static_cast<double>(a.outs),
               i = static_cast<double>(a.cols);
  trace_end(rec, st, DASH_TRACE_GEMM_BF16, 2.0 * t * o * i,
            t * o * dt_bytes(a.dt) + t * i * 33 / 32 + o * i * dt_bytes(a.odt));
  return s;
}

}  // namespace dash
