// The norm's forward and backward passes (layer norm, and with center = 0 the
// root-mean-square norm), with an optional 8-bit checkpoint of the normalised rows, and
// column sums.  All of it is bound by HBM, or at a few rows by the latency of one launch:
// every kernel reads its rows once and keeps them in registers.
#include "act_q8.cuh"
#include "dash_internal.h"
#include "train_internal.h"

namespace dash {

int norm_read_clear_error() {
  int v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_dash_error, sizeof(int)) != cudaSuccess) return -1;
  if (cudaMemcpyToSymbol(g_dash_error, &z, sizeof(int)) != cudaSuccess) return -1;
  return v;
}

// A row is held by W warps, J vectors of eight columns per thread: thread t of the row has
// columns 8 (j 32 W + t).

// Sums of N (1 or 2) values over the W warps of a row (W = 1: one warp; else the whole CTA,
// or the named barrier's group of warps), the same in every thread.  red holds 32 floats
// per value.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], int W, int warp_in_row, float* red,
                                        int barrier) {
  const int lane = threadIdx.x & 31;
  if constexpr (N == 2) {
    // The lower half-warp goes on with the first value, the upper with the second.
    const bool up = lane >= 16;
    float x = (up ? v[1] : v[0]) + __shfl_xor_sync(0xffffffffu, up ? v[0] : v[1], 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (W == 1) {
      v[0] = __shfl_sync(0xffffffffu, x, 0);
      v[1] = __shfl_sync(0xffffffffu, x, 16);
      return;
    }
    if ((lane & 15) == 0) red[(lane << 1) + warp_in_row] = x;
  } else {
    v[0] = warp_sum(v[0]);
    if (W == 1) return;
    if (lane == 0) red[warp_in_row] = v[0];
  }
  asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(W * 32) : "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (W <= 8) {
      // Up to eight partial sums: read by every thread, the missing ones as zeros.
      float t = 0.0f;
#pragma unroll
      for (int w = 0; w < 8; ++w) t += w < W ? red[i * 32 + w] : 0.0f;
      v[i] = t;
    } else {
      v[i] = warp_sum(lane < W ? red[i * 32 + lane] : 0.0f);
    }
  }
}

// Largest CTA of a forward instance: J vectors per thread, at most 2048 vectors a row.
constexpr int fwd_threads(int J) { return J <= 2 ? 1024 : 512; }

// W = 1: a row per warp, else a row per CTA; small CTAs, many per SM, cover one another's
// loads and sums.  The variance is taken about the mean, in a second pass over the
// registers.  (Measured and not taken: rows brought in by bulk copies several rows ahead,
// by persistent CTAs.  36.3 against 32.2 us at 8192 x 2048 bf16 with residual and
// checkpoint, since what bounds it is instruction issue, not the loads' latency.)
template <typename T, int J, bool VEC>
__global__ void __launch_bounds__(fwd_threads(J))
    norm_forward_kernel(const NormFwdArgs a, int W, bool wvec) {
  __shared__ float red[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long row =
      W == 1 ? static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + warp : blockIdx.x;
  if (row >= a.rows) return;
  const int t = W == 1 ? lane : static_cast<int>(threadIdx.x);
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  F2 v[J][4];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c = (j * 32 * W + t) * 8;
    load8<T, VEC>(x + c, a.cols - c, v[j]);
  }
  if (a.residual) {
    // The stream is carried in its own type: the norm sees the rounded sum.
    const T* res = static_cast<const T*>(a.residual) + row * a.ldres;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int c = (j * 32 * W + t) * 8;
      F2 u[4];
      load8<T, VEC>(res + c, a.cols - c, u);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[j][k] = round2<T>(v[j][k] + u[k]);
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
  float s[1];
  float mean = 0.0f;
  if (a.center) {
    F2 p = f2(0.0f);
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) p = p + v[j][k];
    s[0] = f2_sum(p);
    row_sum<1>(s, W, warp, red[0], 0);
    mean = s[0] / a.cols;
    const F2 less = f2(-mean);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int n = a.cols - (j * 32 * W + t) * 8;
      // Outside the row n stays 0, in the checkpoint's padding too.
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (VEC ? n > 0 : 2 * k + 1 < n) {
          v[j][k] = v[j][k] + less;
        } else if (!VEC && 2 * k < n) {
          float lo, hi;
          f2_get(v[j][k] + less, lo, hi);
          v[j][k] = f2(lo, 0.0f);
        }
      }
    }
  }
  F2 p = f2(0.0f);
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int k = 0; k < 4; ++k) p = f2_fma(v[j][k], v[j][k], p);
  s[0] = f2_sum(p);
  row_sum<1>(s, W, warp, red[1], 0);
  const float rstd = 1.0f / sqrtf(s[0] / a.cols + a.eps);
  if (t == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
  T* y = static_cast<T*>(a.y) + row * a.ldy;
  const int pitch = (a.cols + Q8_GROUP - 1) / Q8_GROUP * Q8_GROUP;
  const F2 rs = f2(rstd);
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int c = (j * 32 * W + t) * 8;
#pragma unroll
    for (int k = 0; k < 4; ++k) v[j][k] = v[j][k] * rs;
    if (a.q) {
      uint2 codes;
      const uint32_t b = q8_encode8(a.fmt, group_amax(v[j]), v[j], codes);
      if (c < pitch) {
        *reinterpret_cast<uint2*>(a.q + row * pitch + c) = codes;
        if ((lane & 3) == 0) a.scale[(row * pitch + c) / Q8_GROUP] = static_cast<uint8_t>(b);
      }
    }
    if (c < a.cols) {
      F2 w[4];
      if (a.gamma) {
        load8_dt(a.gamma, a.wdt, wvec, c, a.cols - c, w);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[j][k] = v[j][k] * w[k];
      }
      if (a.beta) {
        load8_dt(a.beta, a.wdt, wvec, c, a.cols - c, w);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[j][k] = v[j][k] + w[k];
      }
      store8<T, VEC>(y + c, a.cols - c, v[j]);
    }
  }
}

// ---------------------------------------------------------------- backward

constexpr int BWD_WARPS = 16;

// Joins the groups' column sums, in order, into row blockIdx.x of `part` (dgamma's sums,
// then dbeta's).  sums: 2 cols floats of shared memory.
template <int J>
__device__ __forceinline__ void join_groups(float* sums, float* part, int cols, int W, int G,
                                            int grp, int t, const F2 (&dg)[J][4],
                                            const F2 (&db)[J][4]) {
  float* out = part + static_cast<long long>(blockIdx.x) * 2 * cols;
  for (int i = 0; i < G; ++i) {
    if (grp == i) {
      float* to = i + 1 < G ? sums : out;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int c = (j * 32 * W + t) * 8;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float g[2], b[2];
          f2_get(dg[j][k], g[0], g[1]);
          f2_get(db[j][k], b[0], b[1]);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int col = c + 2 * k + h;
            if (col >= cols) continue;
            if (i > 0) {
              g[h] += sums[col];
              b[h] += sums[cols + col];
            }
            to[col] = g[h];
            to[cols + col] = b[h];
          }
        }
      }
    }
    if (i + 1 < G) __syncthreads();
  }
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// W warps per row, G groups of them per CTA; with the ring, S stages of `stage` bytes for
// each group.
struct RowPlan {
  int W, G, S;
  uint32_t stage;
};
constexpr int RING_MAX = 8;                                 // most stages of a group
constexpr int RING_BARS = 8 * BWD_WARPS * RING_MAX;         // their barriers

// Where n comes from.
enum NSource : int { N_FROM_X = 0, N_INT8 = 1, N_E4M3 = 2 };

// dx = rstd (g - mean(g) - n mean(g n)) + dres, g = dy gamma, and this CTA's share of
// dgamma = sum dy n and dbeta = sum dy.  Persistent, one CTA per SM: each group takes a row
// at a time, and a thread keeps its columns from row to row, so that their sums stay in
// registers and leave once, joined over the groups, as row blockIdx.x of `part`.
// A row is read twice, before and after its sums.  (Held in registers in between it was
// slower, 51.6 against 46.8 us at 8192 x 2048: the registers the sums leave are few.)
// RING: a row's inputs come by bulk copies into a ring of shared-memory stages that the
// group's first thread fills ahead, so that reads are in flight while a row's sums and
// their barrier are waited for.  A stage is refilled once every thread has read it for the
// last time, after the next row's barrier.  8192 x 2048 bf16 with int8 codes and dres: 58.5 us without,
// 45.9 us with.  Without RING (rows of odd sizes or alignment, short or few rows) the
// threads load for themselves.
// After a wait that ran out the group carries on (its threads must meet at its barriers)
// with whatever the stage holds and issues no more copies; the error flag tells.
// Named barrier 1 + grp is the group's: barrier 0 is the whole CTA's, where groups that
// have run out of rows wait while others still sum.
template <typename T, int SRC, int J, bool VEC, bool RING>
__global__ void __launch_bounds__(32 * BWD_WARPS, 1)
    norm_backward_kernel(const NormBwdArgs a, const RowPlan p, bool wvec, float* part) {
  constexpr bool CK = SRC != N_FROM_X;
  __shared__ float red[BWD_WARPS][2][2 * 32];
  __shared__ int abort_s;
  extern __shared__ __align__(16) uint8_t dyn[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int W = p.W, grp = warp / W, wr = warp - grp * W, t = wr * 32 + lane;
  const bool first = t == 0;
  const uint32_t bars = smem_u32(dyn) + 8u * (grp * p.S), data = smem_u32(dyn) + RING_BARS;
  volatile int* abort_flag = &abort_s;
  if (RING) {
    if (threadIdx.x == 0) {
      abort_s = 0;
      for (int i = 0; i < p.G * p.S; ++i) mbar_init(smem_u32(dyn) + 8u * i, 1);
      fence_barrier_init();
    }
    __syncthreads();
  }
  const long long step = static_cast<long long>(gridDim.x) * p.G;
  const long long row0 = static_cast<long long>(blockIdx.x) * p.G + grp;
  const int ng = (a.cols + Q8_GROUP - 1) / Q8_GROUP, pitch = ng * Q8_GROUP;
  const uint32_t bytes = static_cast<uint32_t>(a.cols) * sizeof(T);
  const uint32_t nbytes = CK ? static_cast<uint32_t>(pitch) : bytes;
  // A stage: dy, x or the codes, dres.
  auto fill = [&](long long row, int s) {
    if (*abort_flag) return;
    const uint32_t bar = bars + 8u * s;
    const uint32_t dst = data + (grp * p.S + s) * p.stage;
    mbar_arrive_expect_tx(bar, bytes + nbytes + (a.dres ? bytes : 0u));
    bulk_load(dst, static_cast<const T*>(a.dy) + row * a.lddy, bytes, bar);
    if (CK)
      bulk_load(dst + bytes, a.q + row * pitch, nbytes, bar);
    else
      bulk_load(dst + bytes, static_cast<const T*>(a.x) + row * a.ldx, nbytes, bar);
    if (a.dres)
      bulk_load(dst + bytes + nbytes, static_cast<const T*>(a.dres) + row * a.lddres, bytes, bar);
  };
  if (RING && first)
    for (int s = 0; s < p.S; ++s)
      if (row0 + s * step < a.rows) fill(row0 + s * step, s);
  // Up to two vectors' gamma stays in registers.
  constexpr bool HOLD = J <= 2;
  const int c0 = t * 8, cstep = 256 * W;  // columns c0 + j cstep
  F2 gm[HOLD ? J : 1][4];
  auto gamma8 = [&](int j, F2 (&g)[4]) {
    const int c = c0 + j * cstep;
    if (a.gamma) {
      load8_dt(a.gamma, a.wdt, wvec, c, a.cols - c, g);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) g[k] = f2(1.0f);
    }
  };
  if constexpr (HOLD) {
#pragma unroll
    for (int j = 0; j < J; ++j) gamma8(j, gm[j]);
  }
  F2 dg[J][4], db[J][4];
#pragma unroll
  for (int j = 0; j < J; ++j)
#pragma unroll
    for (int k = 0; k < 4; ++k) dg[j][k] = db[j][k] = f2(0.0f);
  // Scales and statistics come straight from global memory, one row ahead; the pointers
  // walk the group's rows.
  constexpr int NSC = CK ? J : 1;
  uint32_t sc[NSC] = {};
  const uint8_t* scp = a.scale + (CK ? row0 * ng + t / 4 : 0);
  const float* rsp = a.rstd + row0;
  const float* mup = a.mean + row0;
  float rstd = 0.0f, mean = 0.0f;
  auto small = [&](uint32_t (&b)[NSC], float& rs, float& mu) {
    if constexpr (CK) {
#pragma unroll
      for (int j = 0; j < J; ++j) b[j] = c0 + j * cstep < pitch ? scp[j * (cstep / 32)] : 127u;
      scp += step * ng;
    } else if (a.center) {
      mu = *mup;
      mup += step;
    }
    rs = *rsp;
    rsp += step;
  };
  if (row0 < a.rows) small(sc, rstd, mean);
  const T* dyp = static_cast<const T*>(a.dy) + (RING ? 0 : row0 * a.lddy + c0);
  const T* xp = static_cast<const T*>(a.x) + (RING || CK ? 0 : row0 * a.ldx + c0);
  const uint8_t* qp = a.q + (RING || !CK ? 0 : row0 * pitch + c0);
  const T* rp = static_cast<const T*>(a.dres) + (RING ? 0 : row0 * a.lddres + c0);
  T* dxp = static_cast<T*>(a.dx) + row0 * a.lddx + c0;
  const bool has_db = a.dbeta != nullptr;
  int s = 0, flip = 0;
  uint32_t ph = 0;
  for (long long row = row0; row < a.rows; row += step) {
    uint32_t nsc[NSC] = {};
    float nrstd = 0.0f, nmean = 0.0f;
    if (row + step < a.rows) small(nsc, nrstd, nmean);
    if (RING) {
      mbar_wait(bars + 8u * s, ph, abort_flag);
      const uint8_t* st = dyn + RING_BARS + (grp * p.S + s) * p.stage;
      dyp = reinterpret_cast<const T*>(st) + c0;
      xp = reinterpret_cast<const T*>(st + bytes) + c0;
      qp = st + bytes + c0;
      rp = reinterpret_cast<const T*>(st + bytes + nbytes) + c0;
    }
    const F2 rs = f2(rstd), less = f2(-mean);
    // Vector j: dy and n.
    auto vector8 = [&](int j, F2 (&d)[4], F2 (&m)[4]) {
      const int left = a.cols - (c0 + j * cstep);
      load8<T, VEC>(dyp + j * cstep, left, d);
      if constexpr (CK) {
        uint2 q = make_uint2(0u, 0u);
        if (left > 0) q = *reinterpret_cast<const uint2*>(qp + j * cstep);
        q8_decode8<SRC == N_INT8 ? DASH_Q8_INT8 : DASH_Q8_E4M3>(q, sc[j], m);
      } else {
        load8<T, VEC>(xp + j * cstep, left, m);
        // The difference first: x may lie far from zero.
#pragma unroll
        for (int k = 0; k < 4; ++k) m[k] = (m[k] + less) * rs;
      }
    };
    auto scale8 = [&](int j, F2 (&d)[4]) {
      F2 w[4];
      if constexpr (!HOLD) gamma8(j, w);
#pragma unroll
      for (int k = 0; k < 4; ++k) d[k] = d[k] * (HOLD ? gm[HOLD ? j : 0][k] : w[k]);
    };
    F2 s1 = f2(0.0f), s2 = f2(0.0f);
    // Columns outside the row have dy = g = 0 and add nothing to any sum: n is finite
    // there (it is -mean rstd, or a padding code), unless the row is not finite anyway.
#pragma unroll
    for (int j = 0; j < J; ++j) {
      if (c0 + j * cstep >= a.cols) continue;
      F2 gj[4], nj[4];
      vector8(j, gj, nj);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        dg[j][k] = f2_fma(gj[k], nj[k], dg[j][k]);
        if (has_db) db[j][k] = db[j][k] + gj[k];
      }
      scale8(j, gj);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        s1 = s1 + gj[k];
        s2 = f2_fma(gj[k], nj[k], s2);
      }
    }
    // The sums' buffers alternate: a slow warp may still read one row's when another
    // writes the next row's.
    float sum[2] = {f2_sum(s1), f2_sum(s2)};
    row_sum<2>(sum, W, wr, red[grp][flip], 1 + grp);
    flip ^= 1;
    if (RING) {
      if (W == 1) __syncwarp();
      if (first && row != row0 && row + (p.S - 1) * step < a.rows)
        fill(row + (p.S - 1) * step, s == 0 ? p.S - 1 : s - 1);
    }
    const F2 m1 = f2(a.center ? -(sum[0] / a.cols) : 0.0f), m2 = f2(-(sum[1] / a.cols));
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int left = a.cols - (c0 + j * cstep);
      if (left <= 0) continue;
      F2 gj[4], nj[4], rj[4];
      vector8(j, gj, nj);
      scale8(j, gj);
#pragma unroll
      for (int k = 0; k < 4; ++k) gj[k] = f2_fma(nj[k], m2, gj[k] + m1) * rs;
      if (a.dres) {
        load8<T, VEC>(rp + j * cstep, left, rj);
#pragma unroll
        for (int k = 0; k < 4; ++k) gj[k] = gj[k] + rj[k];
      }
      store8<T, VEC>(dxp + j * cstep, left, gj);
    }
    dxp += step * a.lddx;
    if (RING) {
      if (++s == p.S) {
        s = 0;
        ph ^= 1u;
      }
    } else {
      dyp += step * a.lddy;
      xp += step * a.ldx;
      qp += step * pitch;
      rp += step * a.lddres;
    }
#pragma unroll
    for (int j = 0; j < NSC; ++j) sc[j] = nsc[j];
    rstd = nrstd;
    mean = nmean;
  }
  if (part == nullptr) return;
  // Every copy has landed and been read: the groups' sums may overwrite the ring.
  if (RING) __syncthreads();
  join_groups<J>(reinterpret_cast<float*>(dyn), part, a.cols, W, p.G, grp, t, dg, db);
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
  F2 s[4] = {f2(0.0f), f2(0.0f), f2(0.0f), f2(0.0f)};
#pragma unroll 8
  for (long long r = r0 + w; r < r1; r += CS_WARPS) {
    F2 v[4];
    load8<T, VEC>(m + r * ld + c, n, v);
#pragma unroll
    for (int k = 0; k < 4; ++k) s[k] = s[k] + v[k];
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) f2_get(s[k], sb[w][lane * 8 + 2 * k], sb[w][lane * 8 + 2 * k + 1]);
  __syncthreads();
  const long long col = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (col < cols) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < CS_WARPS; ++i) t += sb[i][threadIdx.x];
    part[static_cast<long long>(blockIdx.y) * cols + col] = t;
  }
}

constexpr int PS_WARPS = 16;

// out[y][c] = sum over p < parts of part[p][y][c], in a fixed order: lane x of warp w takes
// p = w, w + 16, ...; the warps' sums are joined in order.  Launched before the kernel that
// writes `part` has ended (its launch latency then overlaps it) and waits for it here.
__global__ void __launch_bounds__(32 * PS_WARPS)
    part_sum_kernel(const float* part, int parts, long long cols, long long stride, float* out0,
                    float* out1) {
  __shared__ float sm[PS_WARPS][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const long long c = static_cast<long long>(blockIdx.x) * 32 + lane;
  float* out = blockIdx.y ? out1 : out0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (out == nullptr) return;
  const float* p0 = part + blockIdx.y * cols + c;
  float s = 0.0f;
  if (c < cols) {
#pragma unroll 8
    for (int p = w; p < parts; p += PS_WARPS) s += p0[p * stride];
  }
  sm[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < cols) {
#pragma unroll
    for (int i = 1; i < PS_WARPS; ++i) s += sm[i][lane];
    out[c] = s;
  }
}

static dash_status part_sum(const float* part, int parts, long long cols, long long stride,
                            float* out0, float* out1, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>((cols + 31) / 32), out1 ? 2 : 1);
  cfg.blockDim = dim3(32 * PS_WARPS);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, part_sum_kernel, part, parts, cols, stride, out0, out1) ==
                 cudaSuccess
             ? DASH_OK
             : DASH_ERR_CUDA;
}

dash_status launch_part_sum(const float* part, int parts, long long cols, float* out,
                            cudaStream_t st) {
  return part_sum(part, parts, cols, cols, out, nullptr, st);
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
  int J = 4;
  while (J > 1 && (nvec <= 16 * J ||
                   static_cast<double>(a.rows) * ((nvec + 32 * J - 1) / (32 * J)) < 152 * 16))
    J /= 2;
  while ((nvec + 32 * J - 1) / (32 * J) > 32) J *= 2;
  if (!VEC) J = 2;
  const int W = (nvec + 32 * J - 1) / (32 * J);
  const int warps = W > 1 ? W : (a.rows < 152 * 4 ? 1 : 4);
  const long long grid = W > 1 ? a.rows : (a.rows + warps - 1) / warps;
  const dim3 g(static_cast<unsigned>(grid)), b(32 * warps);
  if constexpr (VEC) {
    if (J == 1)
      norm_forward_kernel<T, 1, true><<<g, b, 0, st>>>(a, W, wvec);
    else if (J == 2)
      norm_forward_kernel<T, 2, true><<<g, b, 0, st>>>(a, W, wvec);
    else
      norm_forward_kernel<T, 4, true><<<g, b, 0, st>>>(a, W, wvec);
  } else {
    norm_forward_kernel<T, 2, false><<<g, b, 0, st>>>(a, W, wvec);
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

// How a backward pass is laid out: J vectors per thread (as few as the row's warps allow,
// for the registers of its sums), W warps per row, G rows at once per CTA, one persistent
// CTA per SM.
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

template <typename T, int SRC, int J, bool VEC, bool RING>
static dash_status backward_k(const NormBwdArgs& a, const BwdPlan& b, const RowPlan& p, bool wvec,
                              float* part, cudaStream_t st) {
  auto k = norm_backward_kernel<T, SRC, J, VEC, RING>;
  size_t smem = RING ? static_cast<size_t>(p.G) * p.S * p.stage + RING_BARS : 0;
  const size_t join = part && p.G > 1 ? static_cast<size_t>(a.cols) * 8 : 0;
  if (smem < join) smem = join;
  if (smem > 32 * 1024 && cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem)) != cudaSuccess)
    return DASH_ERR_CUDA;
  k<<<b.grid, 32 * p.W * p.G, smem, st>>>(a, p, wvec, part);
  return cudaGetLastError() == cudaSuccess ? DASH_OK : DASH_ERR_CUDA;
}

template <typename T, int SRC, int J>
static dash_status backward_j(const NormBwdArgs& a, const BwdPlan& b, float* part,
                              cudaStream_t st) {
  const bool vec = a.cols % 8 == 0 && vec_ok(a.dy, a.lddy, a.dt) && vec_ok(a.dx, a.lddx, a.dt) &&
                   (!a.x || vec_ok(a.x, a.ldx, a.dt)) &&
                   (!a.dres || vec_ok(a.dres, a.lddres, a.dt));
  const bool wvec = a.cols % 8 == 0 && vec_ok(a.gamma, 0, a.wdt);
  // The ring pays where every group has several rows of a KB or more, and needs two stages.
  const size_t row = static_cast<size_t>(a.cols) * sizeof(T);
  const size_t stage = row * (a.dres ? 2 : 1) +
                       (SRC != N_FROM_X ? (a.cols + Q8_GROUP - 1) / Q8_GROUP * Q8_GROUP : row);
  const size_t fit = (208 * 1024 - RING_BARS) / (stage * b.G);
  RowPlan p = {b.W, b.G, 1, 0};
  if (!vec) return backward_k<T, SRC, J, false, false>(a, b, p, wvec, part, st);
  if (fit < 2 || stage < 1024 || a.rows < 152LL * b.G * 2)
    return backward_k<T, SRC, J, true, false>(a, b, p, wvec, part, st);
  p.S = static_cast<int>(fit < RING_MAX ? fit : RING_MAX);
  p.stage = static_cast<uint32_t>(stage);
  return backward_k<T, SRC, J, true, true>(a, b, p, wvec, part, st);
}

template <typename T, int SRC>
static dash_status backward_t(const NormBwdArgs& a, const BwdPlan& b, float* part,
                              cudaStream_t st) {
  return b.J == 4   ? backward_j<T, SRC, 4>(a, b, part, st)
         : b.J == 2 ? backward_j<T, SRC, 2>(a, b, part, st)
                    : backward_j<T, SRC, 1>(a, b, part, st);
}

template <typename T>
static dash_status backward_c(const NormBwdArgs& a, const BwdPlan& p, float* part,
                              cudaStream_t st) {
  if (a.q == nullptr) return backward_t<T, N_FROM_X>(a, p, part, st);
  return a.fmt == DASH_Q8_INT8 ? backward_t<T, N_INT8>(a, p, part, st)
                               : backward_t<T, N_E4M3>(a, p, part, st);
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
