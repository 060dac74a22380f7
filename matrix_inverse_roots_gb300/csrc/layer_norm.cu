// The norm's forward and backward passes (layer norm, and with center = 0 the
// root-mean-square norm), with an optional 8-bit checkpoint of the normalised rows.
#include "act_q8.cuh"
#include "dash_internal.h"
#include "train_internal.h"

namespace dash {

constexpr int LN_THREADS = 256;

// Sum over the CTA, the same in every thread.
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
#pragma unroll
  for (int w = 0; w < LN_THREADS / 32; ++w) s += red[w];
  __syncthreads();
  return s;
}

// One CTA per row.  The variance is taken about the mean, in a second pass.
template <typename T, int FMT>
__global__ void __launch_bounds__(LN_THREADS) norm_forward_kernel(const NormFwdArgs a) {
  __shared__ float red[LN_THREADS / 32];
  const long long row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  const T* res = a.residual ? static_cast<const T*>(a.residual) + row * a.ldres : nullptr;
  T* r = a.r ? static_cast<T*>(a.r) + row * a.ldr : nullptr;
  T* y = static_cast<T*>(a.y) + row * a.ldy;
  const int ng = (a.cols + Q8_GROUP - 1) / Q8_GROUP;
  // The stream is carried in its own type: the norm sees the rounded sum.
  extern __shared__ float row_s[];
  float s = 0.0f;
  for (int c = threadIdx.x; c < a.cols; c += LN_THREADS) {
    float v = Elem<T>::to(x[c]);
    if (res) v = Elem<T>::to(Elem<T>::from(v + Elem<T>::to(res[c])));
    if (r) r[c] = Elem<T>::from(v);
    row_s[c] = v;
    s += v;
  }
  const float mean = a.center ? block_sum(s, red) / a.cols : 0.0f;
  float ss = 0.0f;
  for (int c = threadIdx.x; c < a.cols; c += LN_THREADS) {
    const float d = row_s[c] - mean;
    ss = fmaf(d, d, ss);
  }
  const float rstd = 1.0f / sqrtf(block_sum(ss, red) / a.cols + a.eps);
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
  for (int c = threadIdx.x; c < ng * Q8_GROUP; c += LN_THREADS) {
    const float n = c < a.cols ? (row_s[c] - mean) * rstd : 0.0f;
    if (c < a.cols) {
      float v = n;
      if (a.gamma) v *= load_dt(a.gamma, a.wdt, c);
      if (a.beta) v += load_dt(a.beta, a.wdt, c);
      y[c] = Elem<T>::from(v);
    }
    if (a.q) {
      // A warp holds one group.
      const uint32_t b = q8_scale_byte<FMT>(warp_max_u32(__float_as_uint(n) & 0x7fffffffu));
      a.q[row * ng * Q8_GROUP + c] = static_cast<uint8_t>(q8_code<FMT>(n * q8_inv_scale(b)));
      if ((threadIdx.x & 31) == 0) a.scale[row * ng + c / Q8_GROUP] = static_cast<uint8_t>(b);
    }
  }
}

// The normalised value of (row, c): from the checkpoint, or from the input.
template <typename T, int FMT>
__device__ __forceinline__ float norm_value(const NormBwdArgs& a, long long row, int c, float mean,
                                            float rstd) {
  if (a.q) {
    const long long ng = (a.cols + Q8_GROUP - 1) / Q8_GROUP;
    return q8_value<FMT>(a.q[row * ng * Q8_GROUP + c]) * q8_scale(a.scale[row * ng + c / Q8_GROUP]);
  }
  return (Elem<T>::to(static_cast<const T*>(a.x)[row * a.ldx + c]) - mean) * rstd;
}

// One CTA per row: dx = rstd (g - mean(g) - n mean(g n)) + dres, g = dy gamma.
template <typename T, int FMT>
__global__ void __launch_bounds__(LN_THREADS) norm_backward_kernel(const NormBwdArgs a) {
  __shared__ float red[LN_THREADS / 32];
  const long long row = blockIdx.x;
  const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
  const float mean = (a.x && a.center) ? a.mean[row] : 0.0f;
  const float rstd = a.rstd[row];
  float s1 = 0.0f, s2 = 0.0f;
  for (int c = threadIdx.x; c < a.cols; c += LN_THREADS) {
    float g = Elem<T>::to(dy[c]);
    if (a.gamma) g *= load_dt(a.gamma, a.wdt, c);
    s1 += g;
    s2 = fmaf(g, norm_value<T, FMT>(a, row, c, mean, rstd), s2);
  }
  const float c1 = a.center ? block_sum(s1, red) / a.cols : 0.0f;
  const float c2 = block_sum(s2, red) / a.cols;
  for (int c = threadIdx.x; c < a.cols; c += LN_THREADS) {
    float g = Elem<T>::to(dy[c]);
    if (a.gamma) g *= load_dt(a.gamma, a.wdt, c);
    float d = rstd * (g - c1 - norm_value<T, FMT>(a, row, c, mean, rstd) * c2);
    if (a.dres) d += Elem<T>::to(static_cast<const T*>(a.dres)[row * a.lddres + c]);
    static_cast<T*>(a.dx)[row * a.lddx + c] = Elem<T>::from(d);
  }
}

constexpr int CS_ROWS = 8;

// Partial column sums: CTA (x, y) sums the rows of slice y over 32 columns.
template <typename T, int FMT>
__global__ void __launch_bounds__(32 * CS_ROWS)
    norm_grads_kernel(const NormBwdArgs a, long long slice, float* pg, float* pb) {
  __shared__ float sg[CS_ROWS][33], sb[CS_ROWS][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const long long r0 = blockIdx.y * slice;
  const long long r1 = r0 + slice < a.rows ? r0 + slice : a.rows;
  float g = 0.0f, b = 0.0f;
  if (c < a.cols)
    for (long long r = r0 + w; r < r1; r += CS_ROWS) {
      const float d = Elem<T>::to(static_cast<const T*>(a.dy)[r * a.lddy + c]);
      const float mean = (a.x && a.center) ? a.mean[r] : 0.0f;
      g = fmaf(d, norm_value<T, FMT>(a, r, c, mean, a.rstd[r]), g);
      b += d;
    }
  sg[w][lane] = g;
  sb[w][lane] = b;
  __syncthreads();
  if (w == 0 && c < a.cols) {
    for (int i = 1; i < CS_ROWS; ++i) {
      g += sg[i][lane];
      b += sb[i][lane];
    }
    pg[static_cast<long long>(blockIdx.y) * a.cols + c] = g;
    pb[static_cast<long long>(blockIdx.y) * a.cols + c] = b;
  }
}

template <typename T>
__global__ void __launch_bounds__(32 * CS_ROWS)
    col_sum_kernel(const T* m, long long rows, long long cols, long long ld, long long slice,
                   float* part) {
  __shared__ float sb[CS_ROWS][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const long long c = static_cast<long long>(blockIdx.x) * 32 + lane;
  const long long r0 = blockIdx.y * slice;
  const long long r1 = r0 + slice < rows ? r0 + slice : rows;
  float b = 0.0f;
  if (c < cols)
    for (long long r = r0 + w; r < r1; r += CS_ROWS) b += Elem<T>::to(m[r * ld + c]);
  sb[w][lane] = b;
  __syncthreads();
  if (w == 0 && c < cols) {
    for (int i = 1; i < CS_ROWS; ++i) b += sb[i][lane];
    part[static_cast<long long>(blockIdx.y) * cols + c] = b;
  }
}

// out[c] = sum over p < parts of part[p][c], in order.
__global__ void part_sum_kernel(const float* part, int parts, long long cols, float* out) {
  const long long c = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (c >= cols) return;
  float s = 0.0f;
  for (int p = 0; p < parts; ++p) s += part[static_cast<long long>(p) * cols + c];
  out[c] = s;
}

int col_sum_parts(long long rows, long long cols) {
  (void)cols;
  const long long p = (rows + 63) / 64;
  return static_cast<int>(p < 1 ? 1 : (p > 128 ? 128 : p));
}

static dash_status part_sum(const float* part, int parts, long long cols, float* out,
                            cudaStream_t st) {
  part_sum_kernel<<<static_cast<unsigned>((cols + 127) / 128), 128, 0, st>>>(part, parts, cols,
                                                                             out);
  return cudaGetLastError() == cudaSuccess ? DASH_OK : DASH_ERR_CUDA;
}

dash_status launch_col_sum(const void* m, int dt, long long rows, long long cols, long long ld,
                           float* part, float* out, cudaStream_t st) {
  const int parts = col_sum_parts(rows, cols);
  const long long slice = (rows + parts - 1) / parts;
  const dim3 grid(static_cast<unsigned>((cols + 31) / 32), static_cast<unsigned>(parts));
  const int rec = trace_begin(st);
  if (dt == DASH_DT_F32)
    col_sum_kernel<float><<<grid, 32 * CS_ROWS, 0, st>>>(static_cast<const float*>(m), rows, cols,
                                                         ld, slice, part);
  else if (dt == DASH_DT_BF16)
    col_sum_kernel<__nv_bfloat16><<<grid, 32 * CS_ROWS, 0, st>>>(
        static_cast<const __nv_bfloat16*>(m), rows, cols, ld, slice, part);
  else
    col_sum_kernel<__half><<<grid, 32 * CS_ROWS, 0, st>>>(static_cast<const __half*>(m), rows,
                                                          cols, ld, slice, part);
  dash_status s = cudaGetLastError() == cudaSuccess ? DASH_OK : DASH_ERR_CUDA;
  if (s == DASH_OK) s = part_sum(part, parts, cols, out, st);
  trace_end(rec, st, DASH_TRACE_REDUCE, 0.0,
            static_cast<double>(rows) * cols * dt_bytes(dt) + 4.0 * cols);
  return s;
}

template <typename T>
static dash_status forward_t(const NormFwdArgs& a, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>(a.rows);
  const size_t smem = static_cast<size_t>(a.cols) * sizeof(float);
  auto k = a.fmt == DASH_Q8_INT8 ? norm_forward_kernel<T, DASH_Q8_INT8>
                                 : norm_forward_kernel<T, DASH_Q8_E4M3>;
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(smem)) != cudaSuccess)
    return DASH_ERR_CUDA;
  k<<<grid, LN_THREADS, smem, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? DASH_OK : DASH_ERR_CUDA;
}

dash_status launch_norm_forward(const NormFwdArgs& a, cudaStream_t st) {
  const int rec = trace_begin(st);
  const dash_status s = a.dt == DASH_DT_F32    ? forward_t<float>(a, st)
                        : a.dt == DASH_DT_BF16 ? forward_t<__nv_bfloat16>(a, st)
                                               : forward_t<__half>(a, st);
  const double n = static_cast<double>(a.rows) * a.cols;
  trace_end(rec, st, DASH_TRACE_NORM, 0.0,
            n * dt_bytes(a.dt) * (2 + (a.residual ? 1 : 0) + (a.r ? 1 : 0)) +
                (a.q ? n * 33 / 32 : 0.0));
  return s;
}

size_t norm_backward_ws(long long rows, long long cols) {
  return static_cast<size_t>(2) * col_sum_parts(rows, cols) * cols * sizeof(float);
}

template <typename T, int FMT>
static dash_status backward_t(const NormBwdArgs& a, float* ws, cudaStream_t st) {
  if (a.dgamma || a.dbeta) {
    // Before dx is written: it may take dy's place.
    const int parts = col_sum_parts(a.rows, a.cols);
    const long long slice = (a.rows + parts - 1) / parts;
    float* pg = ws;
    float* pb = ws + static_cast<long long>(parts) * a.cols;
    const dim3 grid(static_cast<unsigned>((a.cols + 31) / 32), static_cast<unsigned>(parts));
    norm_grads_kernel<T, FMT><<<grid, 32 * CS_ROWS, 0, st>>>(a, slice, pg, pb);
    if (cudaGetLastError() != cudaSuccess) return DASH_ERR_CUDA;
    dash_status s = DASH_OK;
    if (a.dgamma) s = part_sum(pg, parts, a.cols, a.dgamma, st);
    if (s == DASH_OK && a.dbeta) s = part_sum(pb, parts, a.cols, a.dbeta, st);
    if (s != DASH_OK) return s;
  }
  if (a.rows > 0)
    norm_backward_kernel<T, FMT><<<static_cast<unsigned>(a.rows), LN_THREADS, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? DASH_OK : DASH_ERR_CUDA;
}

template <typename T>
static dash_status backward_f(const NormBwdArgs& a, float* ws, cudaStream_t st) {
  return a.fmt == DASH_Q8_INT8 ? backward_t<T, DASH_Q8_INT8>(a, ws, st)
                               : backward_t<T, DASH_Q8_E4M3>(a, ws, st);
}

dash_status launch_norm_backward(const NormBwdArgs& a, void* ws, cudaStream_t st) {
  const int rec = trace_begin(st);
  float* w = static_cast<float*>(ws);
  const dash_status s = a.dt == DASH_DT_F32    ? backward_f<float>(a, w, st)
                        : a.dt == DASH_DT_BF16 ? backward_f<__nv_bfloat16>(a, w, st)
                                               : backward_f<__half>(a, w, st);
  const double n = static_cast<double>(a.rows) * a.cols;
  trace_end(rec, st, DASH_TRACE_NORM, 0.0,
            n * dt_bytes(a.dt) * (2 + (a.dres ? 1 : 0)) +
                (a.q ? n * 33 / 32 : n * dt_bytes(a.dt)));
  return s;
}

}  // namespace dash
