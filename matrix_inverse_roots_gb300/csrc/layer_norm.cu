// The norm's forward and backward passes (layer norm, and with center = 0 the
// root-mean-square norm), with an optional 8-bit checkpoint of the normalised rows, and
// column sums.  All of it is bound by HBM, or at a few rows by the latency of one launch:
// every kernel reads its rows once and keeps them in registers.
#include "act_q8.cuh"
#include "dash_internal.h"
#include "train_internal.h"

namespace dash {

// A row is held by W warps, J vectors of eight columns per thread: thread t of the row has
// columns 8 (j 32 W + t).

// Sums of N values over the W warps of a row (W = 1: one warp; else the whole CTA, or the
// named barrier's group of warps), the same in every thread.  red holds N floats per warp.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], int W, int warp_in_row, float* red,
                                        int barrier) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
  if (W == 1) return;
  const int lane = threadIdx.x & 31;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) red[i * 32 + warp_in_row] = v[i];
  asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(W * 32) : "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = warp_sum(lane < W ? red[i * 32 + lane] : 0.0f);
}

// Largest CTA of a forward instance: J vectors per thread and at most 2048 vectors a row.
constexpr int fwd_threads(int J) { return J <= 2 ? 1024 : (J == 4 ? 512 : 256); }

// The variance is taken about the mean, in a second pass over the registers.
template <typename T, int J, bool VEC>
__global__ void __launch_bounds__(fwd_threads(J))
    norm_forward_kernel(const NormFwdArgs a, int W, bool wvec) {
  __shared__ float red[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // W = 1: a row per warp; else a row per CTA.
  const long long row =
      W == 1 ? static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + warp : blockIdx.x;
  if (row >= a.rows) return;
  const int t = W == 1 ? lane : static_cast<int>(threadIdx.x);
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  const T* res = static_cast<const T*>(a.residual) + row * a.ldres;
  float v[J][8];
  float s[1] = {0.0f};
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c = (j * 32 * W + t) * 8;
    load8<T, VEC>(x + c, a.cols - c, v[j]);
  }
  if (a.residual) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = (j * 32 * W + t) * 8;
      float u[8];
      load8<T, VEC>(res + c, a.cols - c, u);
      // The stream is carried in its own type: the norm sees the rounded sum.
#pragma unroll
      for (int k = 0; k < 8; ++k) v[j][k] = Elem<T>::to(Elem<T>::from(v[j][k] + u[k]));
    }
  }
  if (a.r) {
    T* r = static_cast<T*>(a.r) + row * a.ldr;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = (j * 32 * W + t) * 8;
      store8<T, VEC>(r + c, a.cols - c, v[j]);
    }
  }
  float mean = 0.0f;
  if (a.center) {
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) s[0] += v[j][k];
    row_sum<1>(s, W, warp, red[0], 0);
    mean = s[0] / a.cols;
  }
  s[0] = 0.0f;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int n = a.cols - (j * 32 * W + t) * 8;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      // Outside the row n stays 0, in the checkpoint's padding too.
      v[j][k] = (VEC ? n > 0 : k < n) ? v[j][k] - mean : 0.0f;
      s[0] = fmaf(v[j][k], v[j][k], s[0]);
    }
  }
  row_sum<1>(s, W, warp, red[1], 0);
  const float rstd = 1.0f / sqrtf(s[0] / a.cols + a.eps);
  if (t == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
  T* y = static_cast<T*>(a.y) + row * a.ldy;
  const int pitch = (a.cols + Q8_GROUP - 1) / Q8_GROUP * Q8_GROUP;
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c = (j * 32 * W + t) * 8;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[j][k] *= rstd;
    if (a.q) {
      uint2 codes;
      const uint32_t b = q8_encode8(a.fmt, group_amax(v[j]), v[j], codes);
      if (c < pitch) {
        *reinterpret_cast<uint2*>(a.q + row * pitch + c) = codes;
        if ((lane & 3) == 0) a.scale[(row * pitch + c) / Q8_GROUP] = static_cast<uint8_t>(b);
      }
    }
    if (c < a.cols) {
      float w[8];
      if (a.gamma) {
        load8_dt(a.gamma, a.wdt, wvec, c, a.cols - c, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[j][k] *= w[k];
      }
      if (a.beta) {
        load8_dt(a.beta, a.wdt, wvec, c, a.cols - c, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[j][k] += w[k];
      }
      store8<T, VEC>(y + c, a.cols - c, v[j]);
    }
  }
}

// ---------------------------------------------------------------- backward

constexpr int BWD_WARPS = 16;

// Eight elements as they lie in memory, so that a row waits in few registers between the
// two times it is used.
template <typename T, bool VEC>
struct Raw8 {
  alignas(16) T e[8];
  __device__ __forceinline__ void load(const T* p, int n) {
    if constexpr (!VEC) {
#pragma unroll
      for (int k = 0; k < 8; ++k) e[k] = k < n ? p[k] : Elem<T>::from(0.0f);
    } else if (n > 0) {
      reinterpret_cast<uint4*>(e)[0] = reinterpret_cast<const uint4*>(p)[0];
      if constexpr (sizeof(T) == 4)
        reinterpret_cast<uint4*>(e)[1] = reinterpret_cast<const uint4*>(p)[1];
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) e[k] = Elem<T>::from(0.0f);
    }
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = Elem<T>::to(e[k]);
  }
};

// dx = rstd (g - mean(g) - n mean(g n)) + dres, g = dy gamma, and this CTA's share of
// dgamma = sum dy n and dbeta = sum dy.  Persistent: a CTA of G groups of W warps, each
// group a row at a time; a thread keeps its columns from row to row, so their sums stay in
// registers and leave once, joined over the groups in shared memory, as row blockIdx.x of
// `part` (dgamma's sums, then dbeta's).  CK: n from the checkpoint, else from x.
template <typename T, bool CK, int J, bool VEC>
__global__ void __launch_bounds__(32 * BWD_WARPS, 1)
    norm_backward_kernel(const NormBwdArgs a, int W, int G, bool wvec, float* part) {
  __shared__ float red[BWD_WARPS][2][2][32];
  extern __shared__ float sums[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int grp = warp / W, wr = warp - grp * W;
  const int t = wr * 32 + lane;
  const int pitch = (a.cols + Q8_GROUP - 1) / Q8_GROUP * Q8_GROUP;
  float dg[J][8], db[J][8];
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int k = 0; k < 8; ++k) dg[j][k] = db[j][k] = 0.0f;
  int flip = 0;
  for (long long row = static_cast<long long>(blockIdx.x) * G + grp; row < a.rows;
       row += static_cast<long long>(gridDim.x) * G) {
    Raw8<T, VEC> dy[J], x[CK ? 1 : J];
    uint2 q[CK ? J : 1];
    uint32_t sc[CK ? J : 1];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = (j * 32 * W + t) * 8;
      dy[j].load(static_cast<const T*>(a.dy) + row * a.lddy + c, a.cols - c);
      if constexpr (CK) {
        q[j] = make_uint2(0u, 0u);
        sc[j] = 127u;
        if (c < pitch) {
          q[j] = *reinterpret_cast<const uint2*>(a.q + row * pitch + c);
          sc[j] = a.scale[(row * pitch + c) / Q8_GROUP];
        }
      } else {
        x[j].load(static_cast<const T*>(a.x) + row * a.ldx + c, a.cols - c);
      }
    }
    const float rstd = a.rstd[row];
    const float mean = (!CK && a.center) ? a.mean[row] : 0.0f;
    auto norm8 = [&](int j, float (&n)[8]) {
      if constexpr (CK) {
        q8_decode8(a.fmt, q[j], sc[j], n);
      } else {
        x[j].get(n);
#pragma unroll
        for (int k = 0; k < 8; ++k) n[k] = (n[k] - mean) * rstd;
      }
    };
    auto grad8 = [&](int j, float (&d)[8], float (&g)[8]) {
      const int c = (j * 32 * W + t) * 8;
      dy[j].get(d);
      if (a.gamma && c < a.cols) {
        load8_dt(a.gamma, a.wdt, wvec, c, a.cols - c, g);
#pragma unroll
        for (int k = 0; k < 8; ++k) g[k] *= d[k];
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) g[k] = d[k];
      }
    };
    // Columns outside the row have dy = g = 0 and add nothing, whatever n is there (it is
    // finite: the mean times rstd, or a padding code).
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < J; ++j) {
      if ((j * 32 * W + t) * 8 >= a.cols) continue;
      float d[8], g[8], n[8];
      norm8(j, n);
      grad8(j, d, g);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (!VEC && (j * 32 * W + t) * 8 + k >= a.cols) continue;
        s[0] += g[k];
        s[1] = fmaf(g[k], n[k], s[1]);
        dg[j][k] = fmaf(d[k], n[k], dg[j][k]);
        db[j][k] += d[k];
      }
    }
    // Two buffers in turn: a row's sums may still be read when the next row's are written.
    row_sum<2>(s, W, wr, red[grp][flip][0], 1 + grp);
    flip ^= 1;
    const float c1 = a.center ? s[0] / a.cols : 0.0f, c2 = s[1] / a.cols;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = (j * 32 * W + t) * 8;
      if (c >= a.cols) continue;
      float d[8], g[8], n[8];
      norm8(j, n);
      grad8(j, d, g);
#pragma unroll
      for (int k = 0; k < 8; ++k) g[k] = rstd * (g[k] - c1 - n[k] * c2);
      if (a.dres) {
        load8<T, VEC>(static_cast<const T*>(a.dres) + row * a.lddres + c, a.cols - c, d);
#pragma unroll
        for (int k = 0; k < 8; ++k) g[k] += d[k];
      }
      store8<T, VEC>(static_cast<T*>(a.dx) + row * a.lddx + c, a.cols - c, g);
    }
  }
  if (part == nullptr) return;
  float* out = part + static_cast<long long>(blockIdx.x) * 2 * a.cols;
  // Group by group, in order.
  for (int i = 0; i < G; ++i) {
    if (grp == i) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int c = (j * 32 * W + t) * 8;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (c + k >= a.cols) continue;
          if (i > 0) {
            dg[j][k] += sums[c + k];
            db[j][k] += sums[a.cols + c + k];
          }
          if (i + 1 < G) {
            sums[c + k] = dg[j][k];
            sums[a.cols + c + k] = db[j][k];
          } else {
            out[c + k] = dg[j][k];
            out[a.cols + c + k] = db[j][k];
          }
        }
      }
    }
    if (i + 1 < G) __syncthreads();
  }
}

// ---------------------------------------------------------------- column sums

constexpr int CS_WARPS = 8;

// CTA (x, y) sums the rows of slice y over 256 columns, eight per lane, rows dealt to the
// warps; the warps' sums are joined in order.
template <typename T, bool VEC>
__global__ void __launch_bounds__(32 * CS_WARPS)
    col_sum_kernel(const T* m, long long rows, long long cols, long long ld, long long slice,
                   float* part) {
  __shared__ float sb[CS_WARPS][256];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const long long c = static_cast<long long>(blockIdx.x) * 256 + lane * 8;
  const int n = static_cast<int>(cols - c < 8 ? cols - c : 8);
  const long long r0 = blockIdx.y * slice;
  const long long r1 = r0 + slice < rows ? r0 + slice : rows;
  float s[8] = {};
#pragma unroll 8
  for (long long r = r0 + w; r < r1; r += CS_WARPS) {
    float v[8];
    load8<T, VEC>(m + r * ld + c, n, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) s[k] += v[k];
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) sb[w][lane * 8 + k] = s[k];
  __syncthreads();
  const long long col = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (col < cols) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < CS_WARPS; ++i) t += sb[i][threadIdx.x];
    part[static_cast<long long>(blockIdx.y) * cols + col] = t;
  }
}

// out[y][c] = sum over p < parts of part[p][y][c], in a fixed order: lane x of warp w takes
// p = w, w + 8, ...; the warps' sums are joined in order.
__global__ void __launch_bounds__(256)
    part_sum_kernel(const float* part, int parts, long long cols, long long stride, float* out0,
                    float* out1) {
  __shared__ float sm[8][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const long long c = static_cast<long long>(blockIdx.x) * 32 + lane;
  float* out = blockIdx.y ? out1 : out0;
  if (out == nullptr) return;
  const float* p0 = part + blockIdx.y * cols + c;
  float s = 0.0f;
  if (c < cols) {
#pragma unroll 4
    for (int p = w; p < parts; p += 8) s += p0[p * stride];
  }
  sm[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < cols) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += sm[i][lane];
    out[c] = s;
  }
}

static dash_status part_sum(const float* part, int parts, long long cols, long long stride,
                            float* out0, float* out1, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>((cols + 31) / 32), out1 ? 2 : 1);
  part_sum_kernel<<<grid, 256, 0, st>>>(part, parts, cols, stride, out0, out1);
  return cudaGetLastError() == cudaSuccess ? DASH_OK : DASH_ERR_CUDA;
}

// Slices of the rows: four CTAs per SM, each warp of one with 16 rows or more.
int col_sum_parts(long long rows, long long cols) {
  const long long tiles = (cols + 255) / 256;
  const long long want = tiles > 0 ? (152 * 4 + tiles - 1) / tiles : 1;
  const long long most = (rows + 16 * CS_WARPS - 1) / (16 * CS_WARPS);
  const long long p = want < most ? want : most;
  return static_cast<int>(p < 1 ? 1 : p);
}

static bool vec_ok(const void* p, long long ld, int dt) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * dt_bytes(dt)) % 16 == 0;
}

template <typename T>
static void col_sum_t(const void* m, int dt, long long rows, long long cols, long long ld,
                      int parts, float* part, cudaStream_t st) {
  const long long slice = (rows + parts - 1) / parts;
  const dim3 grid(static_cast<unsigned>((cols + 255) / 256), static_cast<unsigned>(parts));
  const T* p = static_cast<const T*>(m);
  if (cols % 8 == 0 && vec_ok(m, ld, dt))
    col_sum_kernel<T, true><<<grid, 32 * CS_WARPS, 0, st>>>(p, rows, cols, ld, slice, part);
  else
    col_sum_kernel<T, false><<<grid, 32 * CS_WARPS, 0, st>>>(p, rows, cols, ld, slice, part);
}

dash_status launch_col_sum(const void* m, int dt, long long rows, long long cols, long long ld,
                           float* part, float* out, cudaStream_t st) {
  const int parts = col_sum_parts(rows, cols);
  const int rec = trace_begin(st);
  if (dt == DASH_DT_F32)
    col_sum_t<float>(m, dt, rows, cols, ld, parts, part, st);
  else if (dt == DASH_DT_BF16)
    col_sum_t<__nv_bfloat16>(m, dt, rows, cols, ld, parts, part, st);
  else
    col_sum_t<__half>(m, dt, rows, cols, ld, parts, part, st);
  dash_status s = cudaGetLastError() == cudaSuccess ? DASH_OK : DASH_ERR_CUDA;
  if (s == DASH_OK) s = part_sum(part, parts, cols, cols, out, nullptr, st);
  trace_end(rec, st, DASH_TRACE_REDUCE, 0.0,
            static_cast<double>(rows) * cols * dt_bytes(dt) + 4.0 * cols);
  return s;
}

// ---------------------------------------------------------------- host side

template <typename T, bool VEC>
static dash_status forward_t(const NormFwdArgs& a, bool wvec, cudaStream_t st) {
  const int nvec = (a.cols + 7) / 8;
  // Vectors per thread: as many as leave some 16 warps per SM; fewer rows take more
  // threads each, for the latency of one row.
  int J = 8;
  while (J > 1 && (nvec <= 16 * J ||
                   static_cast<double>(a.rows) * ((nvec + 32 * J - 1) / (32 * J)) < 152 * 16))
    J /= 2;
  while ((nvec + 32 * J - 1) / (32 * J) > 32) J *= 2;
  if (!VEC) J = 4;
  const int W = (nvec + 32 * J - 1) / (32 * J);
  const int warps = W > 1 ? W : (a.rows < 152 * 4 ? 1 : 4);
  const long long grid = W > 1 ? a.rows : (a.rows + warps - 1) / warps;
  const dim3 g(static_cast<unsigned>(grid)), b(32 * warps);
  if constexpr (VEC) {
    if (J == 1)
      norm_forward_kernel<T, 1, true><<<g, b, 0, st>>>(a, W, wvec);
    else if (J == 2)
      norm_forward_kernel<T, 2, true><<<g, b, 0, st>>>(a, W, wvec);
    else if (J == 4)
      norm_forward_kernel<T, 4, true><<<g, b, 0, st>>>(a, W, wvec);
    else
      norm_forward_kernel<T, 8, true><<<g, b, 0, st>>>(a, W, wvec);
  } else {
    norm_forward_kernel<T, 4, false><<<g, b, 0, st>>>(a, W, wvec);
  }
  return cudaGetLastError() == cudaSuccess ? DASH_OK : DASH_ERR_CUDA;
}

template <typename T>
static dash_status forward_v(const NormFwdArgs& a, cudaStream_t st) {
  const bool vec = a.cols % 8 == 0 && vec_ok(a.x, a.ldx, a.dt) && vec_ok(a.y, a.ldy, a.dt) &&
                   (!a.residual || vec_ok(a.residual, a.ldres, a.dt)) &&
                   (!a.r || vec_ok(a.r, a.ldr, a.dt));
  const bool wvec = a.cols % 8 == 0 && vec_ok(a.gamma, 0, a.wdt) && vec_ok(a.beta, 0, a.wdt);
  return vec ? forward_t<T, true>(a, wvec, st) : forward_t<T, false>(a, wvec, st);
}

dash_status launch_norm_forward(const NormFwdArgs& a, cudaStream_t st) {
  const int rec = trace_begin(st);
  const dash_status s = a.dt == DASH_DT_F32    ? forward_v<float>(a, st)
                        : a.dt == DASH_DT_BF16 ? forward_v<__nv_bfloat16>(a, st)
                                               : forward_v<__half>(a, st);
  const double n = static_cast<double>(a.rows) * a.cols;
  trace_end(rec, st, DASH_TRACE_NORM, 0.0,
            n * dt_bytes(a.dt) * (2 + (a.residual ? 1 : 0) + (a.r ? 1 : 0)) +
                (a.q ? n * 33 / 32 : 0.0));
  return s;
}

// How a backward pass is laid out: J vectors per thread, W warps per row, G rows at once
// per CTA, and one persistent CTA per SM.
struct BwdPlan {
  int J, W, G, grid;
};

static BwdPlan bwd_plan(long long rows, long long cols) {
  BwdPlan p;
  const int nvec = static_cast<int>((cols + 7) / 8);
  p.J = nvec > 32 * 2 * BWD_WARPS ? 4 : (nvec > 32 ? 2 : 1);
  p.W = (nvec + 32 * p.J - 1) / (32 * p.J);
  if (p.W < 1) p.W = 1;
  p.G = BWD_WARPS / p.W;
  const int sms = device_sm_count();
  const long long need = (rows + p.G - 1) / p.G, cap = sms > 0 ? sms : 152;
  p.grid = static_cast<int>(need < cap ? need : cap);
  return p;
}

size_t norm_backward_ws(long long rows, long long cols) {
  return static_cast<size_t>(2) * bwd_plan(rows, cols).grid * cols * sizeof(float);
}

template <typename T, bool CK, int J, bool VEC>
static dash_status backward_k(const NormBwdArgs& a, const BwdPlan& p, bool wvec, float* part,
                              cudaStream_t st) {
  auto k = norm_backward_kernel<T, CK, J, VEC>;
  const size_t smem = p.G > 1 && part ? static_cast<size_t>(a.cols) * 8 : 0;
  if (smem > 32 * 1024 && cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem)) != cudaSuccess)
    return DASH_ERR_CUDA;
  k<<<p.grid, 32 * p.W * p.G, smem, st>>>(a, p.W, p.G, wvec, part);
  return cudaGetLastError() == cudaSuccess ? DASH_OK : DASH_ERR_CUDA;
}

template <typename T, bool CK>
static dash_status backward_t(const NormBwdArgs& a, const BwdPlan& p, float* part,
                              cudaStream_t st) {
  const bool vec = a.cols % 8 == 0 && vec_ok(a.dy, a.lddy, a.dt) && vec_ok(a.dx, a.lddx, a.dt) &&
                   (!a.x || vec_ok(a.x, a.ldx, a.dt)) &&
                   (!a.dres || vec_ok(a.dres, a.lddres, a.dt));
  const bool wvec = a.cols % 8 == 0 && vec_ok(a.gamma, 0, a.wdt);
  if (p.J == 4)
    return vec ? backward_k<T, CK, 4, true>(a, p, wvec, part, st)
               : backward_k<T, CK, 4, false>(a, p, wvec, part, st);
  if (p.J == 2)
    return vec ? backward_k<T, CK, 2, true>(a, p, wvec, part, st)
               : backward_k<T, CK, 2, false>(a, p, wvec, part, st);
  return vec ? backward_k<T, CK, 1, true>(a, p, wvec, part, st)
             : backward_k<T, CK, 1, false>(a, p, wvec, part, st);
}

template <typename T>
static dash_status backward_c(const NormBwdArgs& a, const BwdPlan& p, float* part,
                              cudaStream_t st) {
  return a.q ? backward_t<T, true>(a, p, part, st) : backward_t<T, false>(a, p, part, st);
}

dash_status launch_norm_backward(const NormBwdArgs& a, void* ws, cudaStream_t st) {
  const BwdPlan p = bwd_plan(a.rows, a.cols);
  float* part = (a.dgamma || a.dbeta) ? static_cast<float*>(ws) : nullptr;
  const int rec = trace_begin(st);
  dash_status s = DASH_OK;
  if (a.rows > 0)
    s = a.dt == DASH_DT_F32    ? backward_c<float>(a, p, part, st)
        : a.dt == DASH_DT_BF16 ? backward_c<__nv_bfloat16>(a, p, part, st)
                               : backward_c<__half>(a, p, part, st);
  if (s == DASH_OK && part)
    s = part_sum(part, a.rows > 0 ? p.grid : 0, a.cols, 2LL * a.cols, a.dgamma, a.dbeta, st);
  const double n = static_cast<double>(a.rows) * a.cols;
  trace_end(rec, st, DASH_TRACE_NORM, 0.0,
            n * dt_bytes(a.dt) * (2 + (a.dres ? 1 : 0)) +
                (a.q ? n * 33 / 32 : n * dt_bytes(a.dt)));
  return s;
}

}  // namespace dash
