// 8-bit activation checkpoints: a matrix to codes and scales, and back.
//
// Both are one pass over the data, bound by HBM.  A thread holds Q8_U vectors of eight
// columns (four neighbouring lanes share a group, so its largest magnitude takes two
// shuffles) and issues all their loads before the first use.  Q8_U is 4, about 16 to 32
// KB of reads in flight per 256 threads.
#include "act_q8.cuh"
#include "dash_internal.h"
#include "train_internal.h"

namespace dash {

constexpr int Q8_THREADS = 256;
constexpr int Q8_U = 4;

// Vector i of a (rows, nv) grid of vectors: FLAT when rows lie without gaps, so that i
// alone addresses it; else row and column come from a division, 32-bit within a CTA's
// tile, whose first vector's row and column are (row0, v0).
struct VecAt {
  long long row;
  int v;
};
template <bool FLAT>
__device__ __forceinline__ VecAt vec_at(long long i, long long row0, unsigned v0, unsigned off,
                                        unsigned nv) {
  VecAt a;
  if (FLAT) {
    a.row = 0;
    a.v = 0;
  } else {
    const unsigned k = (v0 + off) / nv;
    a.row = row0 + k;
    a.v = static_cast<int>(v0 + off - k * nv);
  }
  return a;
}

template <typename T, bool VEC, bool FLAT>
__global__ void __launch_bounds__(Q8_THREADS)
    act_compress_kernel(const CompressArgs a, unsigned nv, long long total) {
  const long long base = static_cast<long long>(blockIdx.x) * (Q8_THREADS * Q8_U);
  const long long row0 = FLAT ? 0 : base / nv;
  const unsigned v0 = FLAT ? 0 : static_cast<unsigned>(base - row0 * nv);
  const T* x = static_cast<const T*>(a.x);
  F2 v[Q8_U][4];
#pragma unroll
  for (int u = 0; u < Q8_U; ++u) {
    const unsigned off = u * Q8_THREADS + threadIdx.x;
    const long long i = base + off;
    const VecAt at = vec_at<FLAT>(i, row0, v0, off, nv);
    const int left = i >= total ? 0 : (FLAT ? 8 : static_cast<int>(min(a.cols - at.v * 8LL, 8LL)));
    load8<T, VEC>(x + (FLAT ? i * 8 : at.row * a.ld + at.v * 8LL), left, v[u]);
  }
#pragma unroll
  for (int u = 0; u < Q8_U; ++u) {
    const long long i = base + u * Q8_THREADS + threadIdx.x;
    uint2 codes;
    const uint32_t b = q8_encode8(a.fmt, group_amax(v[u]), v[u], codes);
    if (i < total) {
      // Codes lie without gaps whatever the matrix does.
      reinterpret_cast<uint2*>(a.q)[i] = codes;
      if ((threadIdx.x & 3) == 0) a.scale[i >> 2] = static_cast<uint8_t>(b);
    }
  }
}

template <typename T, bool VEC, bool FLAT>
__global__ void __launch_bounds__(Q8_THREADS)
    act_restore_kernel(const RestoreArgs a, unsigned nv, long long total) {
  const long long base = static_cast<long long>(blockIdx.x) * (Q8_THREADS * Q8_U);
  const long long row0 = FLAT ? 0 : base / nv;
  const unsigned v0 = FLAT ? 0 : static_cast<unsigned>(base - row0 * nv);
  T* x = static_cast<T*>(a.x);
  uint2 codes[Q8_U];
  uint32_t b[Q8_U];
#pragma unroll
  for (int u = 0; u < Q8_U; ++u) {
    const long long i = base + u * Q8_THREADS + threadIdx.x;
    codes[u] = make_uint2(0u, 0u);
    b[u] = 127u;
    if (i < total) {
      codes[u] = reinterpret_cast<const uint2*>(a.q)[i];
      b[u] = a.scale[i >> 2];
    }
  }
#pragma unroll
  for (int u = 0; u < Q8_U; ++u) {
    const unsigned off = u * Q8_THREADS + threadIdx.x;
    const long long i = base + off;
    const VecAt at = vec_at<FLAT>(i, row0, v0, off, nv);
    const int left = i >= total ? 0 : (FLAT ? 8 : static_cast<int>(min(a.cols - at.v * 8LL, 8LL)));
    F2 v[4];
    if (a.fmt == DASH_Q8_INT8)
      q8_decode8<DASH_Q8_INT8>(codes[u], b[u], v);
    else
      q8_decode8<DASH_Q8_E4M3>(codes[u], b[u], v);
    store8<T, VEC>(x + (FLAT ? i * 8 : at.row * a.ld + at.v * 8LL), left, v);
  }
}

// Access of a (rows, cols) matrix: eight-column vectors where address, leading dimension
// and width allow them (2); without gaps between rows of whole groups besides (3); else
// single elements (0).
static int access_mode(const void* x, int dt, long long cols, long long ld) {
  const bool vec = (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && cols % 8 == 0 &&
                   (ld * dt_bytes(dt)) % 16 == 0;
  return vec ? (ld == cols && cols % Q8_GROUP == 0 ? 3 : 2) : 0;
}

template <typename T>
static void compress_t(const CompressArgs& a, int mode, unsigned grid, unsigned nv,
                       long long total, cudaStream_t st) {
  if (mode == 3)
    act_compress_kernel<T, true, true><<<grid, Q8_THREADS, 0, st>>>(a, nv, total);
  else if (mode == 2)
    act_compress_kernel<T, true, false><<<grid, Q8_THREADS, 0, st>>>(a, nv, total);
  else
    act_compress_kernel<T, false, false><<<grid, Q8_THREADS, 0, st>>>(a, nv, total);
}

template <typename T>
static void restore_t(const RestoreArgs& a, int mode, unsigned grid, unsigned nv,
                      long long total, cudaStream_t st) {
  if (mode == 3)
    act_restore_kernel<T, true, true><<<grid, Q8_THREADS, 0, st>>>(a, nv, total);
  else if (mode == 2)
    act_restore_kernel<T, true, false><<<grid, Q8_THREADS, 0, st>>>(a, nv, total);
  else
    act_restore_kernel<T, false, false><<<grid, Q8_THREADS, 0, st>>>(a, nv, total);
}

// Vectors of the padded matrix, and the CTAs that hold them; false where the grid cannot.
static bool vec_grid(long long rows, long long cols, unsigned& nv, long long& total,
                     unsigned& grid) {
  nv = static_cast<unsigned>((cols + Q8_GROUP - 1) / Q8_GROUP * 4);
  total = rows * nv;
  const long long g = (total + Q8_THREADS * Q8_U - 1) / (Q8_THREADS * Q8_U);
  grid = static_cast<unsigned>(g);
  return g <= 0x7fffffff;
}

dash_status launch_act_compress(const CompressArgs& a, cudaStream_t st) {
  unsigned nv, grid;
  long long total;
  if (!vec_grid(a.rows, a.cols, nv, total, grid)) return DASH_ERR_UNSUPPORTED;
  const int mode = access_mode(a.x, a.dt, a.cols, a.ld);
  const int rec = trace_begin(st);
  if (a.dt == DASH_DT_F32)
    compress_t<float>(a, mode, grid, nv, total, st);
  else if (a.dt == DASH_DT_BF16)
    compress_t<__nv_bfloat16>(a, mode, grid, nv, total, st);
  else
    compress_t<__half>(a, mode, grid, nv, total, st);
  const cudaError_t err = cudaGetLastError();
  trace_end(rec, st, DASH_TRACE_CHECKPOINT, 0.0,
            static_cast<double>(a.rows) * (a.cols * dt_bytes(a.dt) + nv * 8.25));
  return err == cudaSuccess ? DASH_OK : DASH_ERR_CUDA;
}

dash_status launch_act_restore(const RestoreArgs& a, cudaStream_t st) {
  unsigned nv, grid;
  long long total;
  if (!vec_grid(a.rows, a.cols, nv, total, grid)) return DASH_ERR_UNSUPPORTED;
  const int mode = access_mode(a.x, a.dt, a.cols, a.ld);
  const int rec = trace_begin(st);
  if (a.dt == DASH_DT_F32)
    restore_t<float>(a, mode, grid, nv, total, st);
  else if (a.dt == DASH_DT_BF16)
    restore_t<__nv_bfloat16>(a, mode, grid, nv, total, st);
  else
    restore_t<__half>(a, mode, grid, nv, total, st);
  const cudaError_t err = cudaGetLastError();
  trace_end(rec, st, DASH_TRACE_CHECKPOINT, 0.0,
            static_cast<double>(a.rows) * (a.cols * dt_bytes(a.dt) + nv * 8.25));
  return err == cudaSuccess ? DASH_OK : DASH_ERR_CUDA;
}

}  // namespace dash
