// 8-bit activation checkpoints: a matrix to codes and scales, and back.
#include "act_q8.cuh"
#include "dash_internal.h"
#include "train_internal.h"

namespace dash {

constexpr int Q8_THREADS = 256;

// One warp per group of 32 columns, a lane per column.
template <typename T, int FMT>
__global__ void __launch_bounds__(Q8_THREADS)
    act_compress_kernel(const T* x, long long rows, long long cols, long long ld, long long ng,
                        uint8_t* q, uint8_t* scale) {
  const int lane = threadIdx.x & 31;
  const long long total = rows * ng;
  const long long step = static_cast<long long>(gridDim.x) * (Q8_THREADS / 32);
  for (long long i = static_cast<long long>(blockIdx.x) * (Q8_THREADS / 32) + (threadIdx.x >> 5);
       i < total; i += step) {
    const long long r = i / ng;
    const long long c = (i - r * ng) * Q8_GROUP + lane;
    const float v = c < cols ? Elem<T>::to(x[r * ld + c]) : 0.0f;
    const uint32_t b = q8_scale_byte<FMT>(warp_max_u32(__float_as_uint(v) & 0x7fffffffu));
    q[i * Q8_GROUP + lane] = static_cast<uint8_t>(q8_code<FMT>(v * q8_inv_scale(b)));
    if (lane == 0) scale[i] = static_cast<uint8_t>(b);
  }
}

template <typename T, int FMT>
__global__ void __launch_bounds__(Q8_THREADS)
    act_restore_kernel(const uint8_t* q, const uint8_t* scale, long long rows, long long cols,
                       long long ng, T* x, long long ld) {
  const int lane = threadIdx.x & 31;
  const long long total = rows * ng;
  const long long step = static_cast<long long>(gridDim.x) * (Q8_THREADS / 32);
  for (long long i = static_cast<long long>(blockIdx.x) * (Q8_THREADS / 32) + (threadIdx.x >> 5);
       i < total; i += step) {
    const long long r = i / ng;
    const long long c = (i - r * ng) * Q8_GROUP + lane;
    if (c < cols)
      x[r * ld + c] = Elem<T>::from(q8_value<FMT>(q[i * Q8_GROUP + lane]) * q8_scale(scale[i]));
  }
}

// CTAs of a grid-strided launch over `items` warps' worth of work.
static unsigned warp_grid(long long items) {
  const long long need = (items + Q8_THREADS / 32 - 1) / (Q8_THREADS / 32);
  const long long cap = static_cast<long long>(device_sm_count()) * 32;
  return static_cast<unsigned>(need < cap ? need : (cap > 0 ? cap : 1));
}

template <typename T>
static void compress_t(const CompressArgs& a, long long ng, unsigned grid, cudaStream_t st) {
  const T* x = static_cast<const T*>(a.x);
  if (a.fmt == DASH_Q8_INT8)
    act_compress_kernel<T, DASH_Q8_INT8>
        <<<grid, Q8_THREADS, 0, st>>>(x, a.rows, a.cols, a.ld, ng, a.q, a.scale);
  else
    act_compress_kernel<T, DASH_Q8_E4M3>
        <<<grid, Q8_THREADS, 0, st>>>(x, a.rows, a.cols, a.ld, ng, a.q, a.scale);
}

template <typename T>
static void restore_t(const RestoreArgs& a, long long ng, unsigned grid, cudaStream_t st) {
  T* x = static_cast<T*>(a.x);
  if (a.fmt == DASH_Q8_INT8)
    act_restore_kernel<T, DASH_Q8_INT8>
        <<<grid, Q8_THREADS, 0, st>>>(a.q, a.scale, a.rows, a.cols, ng, x, a.ld);
  else
    act_restore_kernel<T, DASH_Q8_E4M3>
        <<<grid, Q8_THREADS, 0, st>>>(a.q, a.scale, a.rows, a.cols, ng, x, a.ld);
}

dash_status launch_act_compress(const CompressArgs& a, cudaStream_t st) {
  const long long ng = (a.cols + Q8_GROUP - 1) / Q8_GROUP;
  const unsigned grid = warp_grid(a.rows * ng);
  const int rec = trace_begin(st);
  if (a.dt == DASH_DT_F32)
    compress_t<float>(a, ng, grid, st);
  else if (a.dt == DASH_DT_BF16)
    compress_t<__nv_bfloat16>(a, ng, grid, st);
  else
    compress_t<__half>(a, ng, grid, st);
  const cudaError_t err = cudaGetLastError();
  trace_end(rec, st, DASH_TRACE_CHECKPOINT, 0.0,
            static_cast<double>(a.rows) * (a.cols * dt_bytes(a.dt) + ng * (Q8_GROUP + 1)));
  return err == cudaSuccess ? DASH_OK : DASH_ERR_CUDA;
}

dash_status launch_act_restore(const RestoreArgs& a, cudaStream_t st) {
  const long long ng = (a.cols + Q8_GROUP - 1) / Q8_GROUP;
  const unsigned grid = warp_grid(a.rows * ng);
  const int rec = trace_begin(st);
  if (a.dt == DASH_DT_F32)
    restore_t<float>(a, ng, grid, st);
  else if (a.dt == DASH_DT_BF16)
    restore_t<__nv_bfloat16>(a, ng, grid, st);
  else
    restore_t<__half>(a, ng, grid, st);
  const cudaError_t err = cudaGetLastError();
  trace_end(rec, st, DASH_TRACE_CHECKPOINT, 0.0,
            static_cast<double>(a.rows) * (a.cols * dt_bytes(a.dt) + ng * (Q8_GROUP + 1)));
  return err == cudaSuccess ? DASH_OK : DASH_ERR_CUDA;
}

}  // namespace dash
