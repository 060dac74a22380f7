// The weight gradient of a linear layer whose input is kept as an 8-bit checkpoint:
//   dW[o][i] = gamma[i] sum_t dz[t][o] n[t][i] + beta[i] db[o],   db[o] = sum_t dz[t][o],
// n the checkpoint's values, written as a matrix or as the B x B blocks of
// shampoo_accumulate.
//
// The product over tokens runs on the tensor cores in bf16.  Neither operand is rounded:
// a checkpoint's value (7 or 4 bits times a power of two) is a bf16 number, and dz enters
// as bf16 parts that add up to it (one for bf16, two for fp16, three for fp32).  gamma
// and beta belong to columns of dW, so they are applied to the sums.
//
// Design (persistent, CTA pairs on 256 x 256 tiles of dW, cta_group::2; both operands lie
// in memory with the token index outermost, so both are MN-major):
//   warps 0, 3   TMA producers of A: 128 columns of dz per CTA, 64 tokens per slot, each
//                loading 64 of the columns (one thread starts about 16 KB of tiled copies
//                per 600 cycles, which the MMAs of a slot nearly take).
//   warp 2       TMA producer of the codes: 128 columns, 64 tokens (8 KB) per slot.
//   warps 4, 6-8, 10-15  converters: codes and scales (scales straight from global
//                memory, one slot ahead) to bf16, into the 128-byte-swizzled layout the MMA
//                reads.  A slot takes a warp pair about 1500 cycles from its codes to its
//                hand-over, three times its MMAs, so every ring slot has a pair of its
//                own.  Measured at 16384 x 8192 x 8192 with int8 codes and five slots:
//                three pairs 1340 TFLOP/s, four 1570, five 1600.  All but one of them
//                stay off the scheduler of the MMA warp, whose few instructions would
//                wait for theirs (hence the idle warps 5 and 9).
//                A converter warp makes its writes visible to the tensor core (proxy
//                fence) and arrives on the leader's barrier without a cluster-wide fence:
//                what the arrival orders are writes to this CTA's own shared memory, which
//                only this SM's tensor core reads, and they are complete before it.  (With
//                a release at cluster scope each hand-over took about 1400 cycles, more
//                than twice a slot's MMAs, and the product ran at 850 TFLOP/s.)
//   warp 1       of the leader issues the MMAs into one of two TMEM accumulators.
//   warps 16-19  epilogue of the previous tile.
// Tiles that do not fill a whole round of the pairs are split along the tokens; their
// fp32 partial sums are joined, in order, by a second kernel.
// Every wait is bounded (see mbar_wait); a time-out sets the device error flag, and the
// CTA drains its copies and MMAs, frees TMEM and returns.
#include <mutex>

#include "act_q8.cuh"
#include "dash_internal.h"
#include "train_internal.h"

namespace dash {

int weight_grad_read_clear_error() {
  int v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, g_dash_error, sizeof(int)) != cudaSuccess) return -1;
  if (cudaMemcpyToSymbol(g_dash_error, &z, sizeof(int)) != cudaSuccess) return -1;
  return v;
}

namespace {

constexpr int WT = 256;              // tile of dW per CTA pair (both directions)
constexpr int WK = 64;               // tokens per slot
constexpr int W_BOX = WK * 128;      // one box: 64 tokens of 64 bf16 columns or 128 codes
constexpr int W_GW = 2;              // warps of a converter group, each taking 32 of 64 rows
constexpr int W_EPI = 4, W_EPI0 = 16;  // epilogue warps
constexpr int W_THREADS = 32 * (W_EPI0 + W_EPI);

// A ring slot holds 64 tokens: PARTS tiles of A (128 columns of dz in two boxes), the
// converted B (128 columns in two boxes) and the codes (one box).
template <int PARTS>
struct WCfg {
  static constexpr int OFF_B = PARTS * 2 * W_BOX;
  static constexpr int OFF_Q = OFF_B + 2 * W_BOX;
  static constexpr int SLOT = OFF_Q + W_BOX;
  static constexpr int NS = (232448 - 1536) / SLOT;  // 5, 4, 3 slots
  static constexpr int CONV = NS * W_GW;             // converter warps
  static constexpr int BARS = 4 * NS + 4 + 1;
  static constexpr int SMEM = NS * SLOT + 1024 + 512;
  static_assert(NS >= 3 && CONV <= 10 && 8 * BARS + 16 <= 512, "ring, warps, barrier area");
};

struct WParams {
  int nkb;             // slots of 64 tokens
  int tiles_m, tiles_n;
  int full;            // tiles computed whole
  int split, kper;     // the others: `split` units of kper slots each
  int units;
  long long rows, ng;
  const uint8_t* scale;
  const float* db;     // column sums of dz (null without beta)
  float* partial;      // (units - full) x 256 x 256 sums
  WeightGradArgs a;
};

// Tile t of the raster: groups of 8 tile rows, walked column by column, so that the tiles
// in flight share few panels of both operands.
__device__ __forceinline__ void tile_at(int t, int tiles_m, int tiles_n, int& mt, int& nt) {
  constexpr int G = 8;
  const int per = G * tiles_n;
  const int g = t / per;
  const int h = tiles_m - g * G < G ? tiles_m - g * G : G;
  const int r = t - g * per;
  mt = g * G + r % h;
  nt = r / h;
}

// Whether the phase of the given parity is over, without waiting.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

struct Unit {
  int mt, nt, k0, k1, part;  // part: index of the partial tile, -1 for a whole one
};

__device__ __forceinline__ Unit unit_at(int u, const WParams& p) {
  Unit x;
  int t = u;
  x.part = -1;
  x.k0 = 0;
  x.k1 = p.nkb;
  if (u >= p.full) {
    x.part = u - p.full;
    t = p.full + x.part / p.split;
    x.k0 = (x.part % p.split) * p.kper;
    x.k1 = x.k0 + p.kper < p.nkb ? x.k0 + p.kper : p.nkb;
  }
  tile_at(t, p.tiles_m, p.tiles_n, x.mt, x.nt);
  return x;
}

// Where element (o, i) of dW is stored.
__device__ __forceinline__ long long dw_index(const WeightGradArgs& a, long long o, long long i) {
  if (a.block == 0) return o * a.ldw + i;
  const long long b = a.block, nbc = (a.cols + b - 1) / b;
  return ((o / b) * nbc + i / b) * b * b + (o % b) * b + i % b;
}
__host__ __device__ __forceinline__ long long padded(long long n, int b) {
  return b ? (n + b - 1) / b * b : n;
}

__device__ __forceinline__ void store_dt(void* p, int dt, long long i, float v) {
  if (dt == DASH_DT_F32)
    static_cast<float*>(p)[i] = v;
  else if (dt == DASH_DT_BF16)
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else
    static_cast<__half*>(p)[i] = __float2half_rn(v);
}

// Scales W consecutive sums of row o from column i on and stores them (W a power of two
// that divides i; a block's rows hold whole groups of W).  Outside the valid part a block
// is zero, whatever the sums there (a NaN code meets a zero there).
template <int W>
__device__ __forceinline__ void finish_store(const WeightGradArgs& a, const float* db, long long o,
                                             long long i, float (&v)[W]) {
  const long long pr = padded(a.outs, a.block), pc = padded(a.cols, a.block);
  if (o >= pr || i >= pc) return;
  const float dbo = (db != nullptr && o < a.outs) ? db[o] : 0.0f;
#pragma unroll
  for (int j = 0; j < W; ++j) {
    if (o < a.outs && i + j < a.cols) {
      if (a.gamma) v[j] *= load_dt(a.gamma, a.wdt, i + j);
      if (a.beta) v[j] = fmaf(dbo, load_dt(a.beta, a.wdt, i + j), v[j]);
    } else {
      v[j] = 0.0f;
    }
  }
  const long long at = dw_index(a, o, i);
  if (i + W <= pc) {
    if (a.odt == DASH_DT_F32) {
      float* p = static_cast<float*>(a.dw) + at;
      if ((reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
#pragma unroll
        for (int j = 0; j < W; j += 4)
          *reinterpret_cast<float4*>(p + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        return;
      }
    } else {
      uint16_t* p = static_cast<uint16_t*>(a.dw) + at;
      if ((reinterpret_cast<uintptr_t>(p) & (W * 2 < 16 ? W * 2 - 1 : 15u)) == 0) {
        uint32_t r[W / 2];
#pragma unroll
        for (int j = 0; j < W / 2; ++j)
          r[j] = a.odt == DASH_DT_BF16 ? pack_bf162(v[2 * j], v[2 * j + 1])
                                       : pack_half2(v[2 * j], v[2 * j + 1]);
        if constexpr (W >= 8) {
#pragma unroll
          for (int j = 0; j < W / 8; ++j)
            reinterpret_cast<uint4*>(p)[j] =
                make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
        } else {
          *reinterpret_cast<uint2*>(p) = make_uint2(r[0], r[1]);
        }
        return;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < W; ++j)
    if (i + j < pc) store_dt(a.dw, a.odt, at + j, v[j]);
}

__device__ __forceinline__ uint32_t bf2_sub(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t bf2_mul(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                   *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// 2^e as a bf16 number in both halves, from a word with the scale byte in its bytes 0 and
// 2; NaN (not the infinity that the shift alone would make) for the byte 255.
__device__ __forceinline__ uint32_t scale_bf2(uint32_t x) {
  return (x << 7) | (((x + 0x00010001u) >> 2) & 0x00400040u);
}

// 16 codes (one 16-byte word of a row) times the scale s (bf16, in both halves), as 16
// bf16 numbers in two 16-byte words.  Two at a time in packed bf16 arithmetic, of which
// every result is exact.  Every four come out in the order 0, 2, 1, 3, which a code word's
// two halves give without a permutation; the epilogue puts the columns back (tmem_col).
template <int FMT>
__device__ __forceinline__ void convert16(const uint4& c, uint32_t s, uint4& lo, uint4& hi) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t r[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (FMT == DASH_Q8_INT8) {
        // q = (128 + low seven bits) - (128, or 256 for a negative q): 128 + x is
        // 0x4300 + x in bf16 for x < 128, and 256 is 0x4380.
        const uint32_t x = h ? w[j] >> 8 : w[j];
        r[2 * j + h] = bf2_mul(
            bf2_sub((x & 0x007f007fu) | 0x43004300u, (x & 0x00800080u) | 0x43004300u), s);
      } else {
        // The code's exponent and mantissa in the bf16 fields, 2^120 too small (0x7b80 is
        // 2^120; subnormal codes are subnormal numbers).
        const uint32_t m = h ? w[j] >> 4 : w[j] << 4, g = h ? w[j] : w[j] << 8;
        r[2 * j + h] =
            bf2_mul(bf2_mul((m & 0x07f007f0u) | (g & 0x80008000u), 0x7b807b80u), s);
      }
    }
  }
  lo = make_uint4(r[0], r[1], r[2], r[3]);
  hi = make_uint4(r[4], r[5], r[6], r[7]);
}

// Accumulator column of a tile's column, within 16.
__host__ __device__ constexpr int tmem_col(int j) {
  return (j & ~3) | ((j & 1) << 1) | ((j >> 1) & 1);
}

template <int FMT, int PARTS>
__global__ void __launch_bounds__(W_THREADS, 1)
    weight_grad_kernel(const __grid_constant__ CUtensorMap tA, const __grid_constant__ CUtensorMap tQ,
                       const __grid_constant__ WParams p) {
  using C = WCfg<PARTS>;
  constexpr int NS = C::NS;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw_base & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  const uint32_t sbase = raw_base + pad;
  const uint32_t bar0 = sbase + NS * C::SLOT;
  auto full = [&](int s) { return bar0 + 8u * s; };             // A landed, B converted
  auto empty = [&](int s) { return bar0 + 8u * (NS + s); };     // the MMAs have read both
  auto qfull = [&](int s) { return bar0 + 8u * (2 * NS + s); };
  auto qempty = [&](int s) { return bar0 + 8u * (3 * NS + s); };
  auto tfull = [&](int s) { return bar0 + 8u * (4 * NS + s); };
  auto tempty = [&](int s) { return bar0 + 8u * (4 * NS + 2 + s); };
  const uint32_t fin_bar = bar0 + 8u * (C::BARS - 1);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + NS * C::SLOT + 8 * C::BARS);
  volatile int* abort_flag =
      reinterpret_cast<volatile int*>(smem + NS * C::SLOT + 8 * C::BARS + 8);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t crank = cluster_ctarank();
  const bool leader = (crank == 0);
  const int cid = blockIdx.x / 2;
  const int ncl = gridDim.x / 2;
  constexpr uint16_t kMask = 3;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      // Of the leader: its two producers (the bytes of both CTAs) and the slot's
      // converters of both CTAs.
      mbar_init(full(s), 2 + 2 * W_GW);
      mbar_init(empty(s), 1);
      mbar_init(qfull(s), 1);
      mbar_init(qempty(s), W_GW);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(tfull(s), 1);
      mbar_init(tempty(s), 2 * W_EPI);
    }
    mbar_init(fin_bar, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tA);
    tma_prefetch_desc(&tQ);
  }
  if (warp == 1) tmem_alloc_pair(smem_u32(tmem_slot), 512);
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0 || warp == 3) {
    if (lane == 0) {
      // -------------------------------------------------------- A producers
      const int half = warp == 0 ? 0 : 1;
      int s = 0;
      uint32_t ph = 0, armed = 0, armed_par = 0;
      bool ok = true;
      for (int u = cid; ok && u < p.units; u += ncl) {
        const Unit x = unit_at(u, p);
        const int o0 = x.mt * WT + static_cast<int>(crank) * 128 + half * 64;
        for (int kb = x.k0; kb < x.k1; ++kb) {
          if (!mbar_wait(empty(s), ph ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          uint32_t fb = full(s);
          if (leader) {
            mbar_arrive_expect_tx(fb, 2 * PARTS * W_BOX);
            armed |= 1u << s;
            armed_par = (armed_par & ~(1u << s)) | (ph << s);
          } else {
            fb = mapa_shared(fb, 0);
          }
          const uint32_t dst = sbase + s * C::SLOT + half * W_BOX;
#pragma unroll
          for (int part = 0; part < PARTS; ++part)
            tma_load_3d_pair(dst + part * 2 * W_BOX, &tA, fb, o0, kb * WK, part);
          if (++s == NS) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      // After a time-out, one that arms it for both CTAs waits for the copies it counts.
      // Its barrier also counts the converters, which may have stopped: the wait is
      // bounded all the same.
      if (!ok)
        for (int i = 0; i < NS; ++i)
          if (armed & (1u << i)) mbar_wait_drain(full(i), (armed_par >> i) & 1u);
    }
  } else if (warp == 2) {
    if (lane == 0) {
      // -------------------------------------------------------- codes producer
      int s = 0;
      uint32_t ph = 0, armed = 0, armed_par = 0;
      bool ok = true;
      for (int u = cid; ok && u < p.units; u += ncl) {
        const Unit x = unit_at(u, p);
        const int i0 = x.nt * WT + static_cast<int>(crank) * 128;
        for (int kb = x.k0; kb < x.k1; ++kb) {
          if (!mbar_wait(qempty(s), ph ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(qfull(s), W_BOX);
          armed |= 1u << s;
          armed_par = (armed_par & ~(1u << s)) | (ph << s);
          tma_load_3d(sbase + s * C::SLOT + C::OFF_Q, &tQ, qfull(s), i0, kb * WK, 0);
          if (++s == NS) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      if (!ok)
        for (int i = 0; i < NS; ++i)
          if (armed & (1u << i)) mbar_wait_drain(qfull(i), (armed_par >> i) & 1u);
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // -------------------------------------------------------- MMA issuer
      // The tensor cores take about 520 cycles for a slot's MMAs of one part; this
      // thread has to come round in less.  So: one barrier to wait for and one to signal
      // per slot, the next slot's barrier looked at before this slot's MMAs are issued,
      // and descriptors that are one addition away from a constant.
      const uint32_t idesc = make_idesc(1, 1, 1, 256, 256);
      const uint64_t d0 = smem_desc(sbase, W_BOX, 1024, LAYOUT_SW128);
      int s = 0, acc = 0;
      uint32_t ph = 0, pacc = 0;
      bool ok = true, ready = false;
      for (int u = cid; ok && u < p.units; u += ncl) {
        const Unit x = unit_at(u, p);
        if (!mbar_wait(tempty(acc), pacc ^ 1u, abort_flag)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + static_cast<uint32_t>(acc * WT);
        uint32_t accumulate = 0;
        for (int kb = x.k0; kb < x.k1; ++kb) {
          if (!ready && !mbar_wait(full(s), ph, abort_flag)) {
            ok = false;
            break;
          }
          const int sn = s + 1 == NS ? 0 : s + 1;
          const uint32_t pn = sn == 0 ? ph ^ 1u : ph;
          ready = mbar_test(full(sn), pn);
          tc_fence_after();
          const uint64_t da = d0 + static_cast<uint32_t>(s * (C::SLOT >> 4));
#pragma unroll
          for (int part = 0; part < PARTS; ++part)
#pragma unroll
            for (int kk = 0; kk < WK / 16; ++kk) {
              mma_f16_pair(d, da + ((part * 2 * W_BOX + kk * 16 * 128) >> 4),
                           da + ((C::OFF_B + kk * 16 * 128) >> 4), idesc, accumulate);
              accumulate = 1;
            }
          mma_commit_pair_mc(empty(s), kMask);
          s = sn;
          ph = pn;
        }
        if (!ok) break;
        mma_commit_pair_mc(tfull(acc), kMask);
        acc ^= 1;
        if (acc == 0) pacc ^= 1u;
      }
      // Every MMA issued above must be complete before TMEM is released.
      mma_commit_pair(fin_bar);
      mbar_wait_drain(fin_bar, 0);
    }
  } else if (warp < W_EPI0) {
    // ---------------------------------------------------------- converters
    // Converter number 0 .. 9 of the warp (5 and 9 have none).  Group s takes ring slot s,
    // every time: what it waits on there it has followed phase by phase, so a parity is
    // never ambiguous.  A warp takes 32 of a slot's rows, eight lanes a row of 128 columns,
    // four rows at a time.
    const int conv = (warp == 5 || warp == 9) ? -1 : warp - 4 - (warp > 5) - (warp > 9);
    const int s = conv / W_GW;
    uint32_t par = 0;
    // The lanes of the upper 64 columns (box 1) take the neighbouring row, whose swizzle
    // differs in the lowest bit: the eight lanes of an access then hit all banks once.
    const int c16 = lane & 7, odd = c16 >> 2;
    const int rl = (lane >> 3) ^ odd;  // row, of the four
    const int t0 = (conv % W_GW) * 32 + rl;
    const int w = (c16 & 3) * 2;       // its 16-byte words are w and w + 1 of the box's row
    const int qoff = C::OFF_Q + t0 * 128 + c16 * 16;
    const int boff = C::OFF_B + odd * W_BOX + t0 * 128;
    uint8_t* const slot = smem + s * C::SLOT;
    const uint32_t sel = 0x4040u | ((c16 >> 1) * 0x0101u);  // the group's byte to bytes 0, 2
    int ahead = s;  // slots from the unit's first to the group's next
    const bool words = (p.ng & 3) == 0 && (reinterpret_cast<uintptr_t>(p.scale) & 3u) == 0;
    bool ok = conv >= 0 && conv < C::CONV;
    for (int u = cid; ok && u < p.units; u += ncl) {
      const Unit x = unit_at(u, p);
      const int g0 = x.nt * (WT / Q8_GROUP) + static_cast<int>(crank) * 4;
      // The four scale bytes of row 32 (conv % W_GW) + lane of slot kb; 0 (a scale of 0)
      // outside.
      auto scales = [&](int kb) -> uint32_t {
        const long long r = static_cast<long long>(kb) * WK + (conv % W_GW) * 32 + lane;
        uint32_t v = 0;
        if (kb < x.k1 && r < p.rows && g0 < p.ng) {
          const uint8_t* sp = p.scale + r * p.ng + g0;
          if (words) {
            v = *reinterpret_cast<const uint32_t*>(sp);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (g0 + j < p.ng) v |= static_cast<uint32_t>(sp[j]) << (8 * j);
          }
        }
        return v;
      };
      int kb = x.k0 + ahead;
      uint32_t sc = scales(kb);
      for (; kb < x.k1; kb += NS) {
        const uint32_t next = scales(kb + NS);
        if (!mbar_wait(qfull(s), par, abort_flag) || !mbar_wait(empty(s), par ^ 1u, abort_flag)) {
          ok = false;
          break;
        }
        uint4 q[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          q[j] = *reinterpret_cast<const uint4*>(slot + qoff + j * 4 * 128);
        __syncwarp();
        if (lane == 0) mbar_arrive(qempty(s));
        uint8_t* dst = slot + boff;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t four = __shfl_sync(0xffffffffu, sc, j * 4 + rl);
          uint4 lo, hi;
          convert16<FMT>(q[j], scale_bf2(__byte_perm(four, 0u, sel)), lo, hi);
          const int sw = (t0 + j * 4) & 7;
          uint8_t* r0 = dst + j * 4 * 128;
          *reinterpret_cast<uint4*>(r0 + ((w ^ sw) << 4)) = lo;
          *reinterpret_cast<uint4*>(r0 + (((w + 1) ^ sw) << 4)) = hi;
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(mapa_shared(full(s), 0));
        sc = next;
        par ^= 1u;
      }
      ahead = kb - x.k1;
    }
  } else {
    // ---------------------------------------------------------- epilogue
    const int q = warp & 3;  // TMEM lane quarter
    int acc = 0;
    uint32_t pacc = 0;
    for (int u = cid; u < p.units; u += ncl) {
      const Unit x = unit_at(u, p);
      if (!mbar_wait(tfull(acc), pacc, abort_flag)) break;
      tc_fence_after();
      const int row = static_cast<int>(crank) * 128 + q * 32 + lane;  // in the tile
      const uint32_t taddr =
          tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * WT);
#pragma unroll 1
      for (int cc = 0; cc < WT / 16; ++cc) {
        uint32_t r[16];
        tmem_ld16(taddr + cc * 16, r);
        tmem_wait_ld(r);
        if (cc + 1 == WT / 16) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(mapa_shared(tempty(acc), 0));
        }
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(r[tmem_col(j)]);
        if (x.part >= 0) {
          float4* d = reinterpret_cast<float4*>(
              p.partial + (static_cast<long long>(x.part) * WT + row) * WT + cc * 16);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            d[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        } else {
          finish_store<16>(p.a, p.db, static_cast<long long>(x.mt) * WT + row,
                           static_cast<long long>(x.nt) * WT + cc * 16, v);
        }
      }
      acc ^= 1;
      if (acc == 0) pacc ^= 1u;
    }
  }

  tc_fence_before();
  __syncthreads();
  // No CTA may leave while a peer can still signal into it or use its TMEM.
  cluster_sync();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

// Joins the partial sums of the tiles split along the tokens (none at all for split 0, a
// gradient over no tokens).  A warp per 128 columns of a tile's row.
__global__ void __launch_bounds__(256) weight_grad_join_kernel(const __grid_constant__ WParams p,
                                                               int first, int ntiles) {
  const long long total = static_cast<long long>(ntiles) * WT * (WT / 4);
  for (long long e = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; e < total;
       e += static_cast<long long>(gridDim.x) * 256) {
    const int c4 = static_cast<int>(e % (WT / 4));
    const long long rr = e / (WT / 4);
    const int row = static_cast<int>(rr % WT);
    const int t = static_cast<int>(rr / WT);
    int mt, nt;
    tile_at(first + t, p.tiles_m, p.tiles_n, mt, nt);
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = 0; s < p.split; ++s) {
      const float4 f = *reinterpret_cast<const float4*>(
          p.partial + ((static_cast<long long>(t) * p.split + s) * WT + row) * WT + c4 * 4);
      v[0] += f.x;
      v[1] += f.y;
      v[2] += f.z;
      v[3] += f.w;
    }
    finish_store<4>(p.a, p.db, static_cast<long long>(mt) * WT + row,
                    static_cast<long long>(nt) * WT + c4 * 4, v);
  }
}

// Zeros in the blocks' padding that no tile reaches: rows from r0 on, and columns from c0.
__global__ void __launch_bounds__(256)
    weight_grad_pad_kernel(const WeightGradArgs a, long long r0, long long c0) {
  const long long pr = padded(a.outs, a.block), pc = padded(a.cols, a.block);
  for (long long o = blockIdx.y; o < pr; o += gridDim.y) {
    const long long from = o < r0 ? c0 : 0;
    for (long long i = from + (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) * 4; i < pc;
         i += static_cast<long long>(gridDim.x) * 1024) {
      float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      const long long at = dw_index(a, o, i);
      if (a.odt == DASH_DT_F32)
        *reinterpret_cast<float4*>(static_cast<float*>(a.dw) + at) =
            make_float4(v[0], v[1], v[2], v[3]);
      else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.dw) + at) = make_uint2(0u, 0u);
    }
  }
}

// dz as bf16 parts that add up to it, (parts, rows, ldp).  Every part but the last keeps
// the upper bits (truncated, so that no part overflows); what is left is exact.
template <typename T, int PARTS>
__global__ void __launch_bounds__(256)
    split_kernel(const T* dz, long long rows, long long outs, long long ld, long long ldp,
                 uint16_t* out) {
  for (long long r = blockIdx.y; r < rows; r += gridDim.y)
    for (long long c = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; c < outs;
         c += static_cast<long long>(gridDim.x) * 256) {
      float v = Elem<T>::to(dz[r * ld + c]);
#pragma unroll
      for (int k = 0; k < PARTS; ++k) {
        const uint32_t b = __float_as_uint(v) & 0xffff0000u;
        uint32_t h = b >> 16;
        // Non-finite: the first part carries it (a NaN keeps a mantissa bit), the others
        // are zero.
        if ((b & 0x7f800000u) == 0x7f800000u) {
          if (v != v) h = 0x7fc0u;
          v = 0.0f;
        } else {
          v -= __uint_as_float(b);
        }
        out[(k * rows + r) * ldp + c] = static_cast<uint16_t>(h);
      }
    }
}

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                             const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                             const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static EncodeFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, []() {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(ptr);
  });
  return fn;
}

// (inner, rows, planes) with the given row and plane strides in bytes.
bool make_map(CUtensorMap* m, const void* base, bool bytes, uint64_t inner, uint64_t rows,
              uint64_t planes, uint64_t row_bytes, uint64_t plane_bytes, uint32_t box_inner,
              uint32_t box_rows, bool swizzle) {
  EncodeFn enc = encode_fn();
  if (enc == nullptr) return false;
  cuuint64_t dim[3] = {inner, rows, planes};
  cuuint64_t stride[2] = {row_bytes, plane_bytes};
  cuuint32_t box[3] = {box_inner, box_rows, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(m, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 3,
             const_cast<void*>(base), dim, stride, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

typedef void (*WKernel)(CUtensorMap, CUtensorMap, WParams);

WKernel kernel_of(int fmt, int parts) {
  if (fmt == DASH_Q8_INT8)
    return parts == 1   ? weight_grad_kernel<DASH_Q8_INT8, 1>
           : parts == 2 ? weight_grad_kernel<DASH_Q8_INT8, 2>
                        : weight_grad_kernel<DASH_Q8_INT8, 3>;
  return parts == 1   ? weight_grad_kernel<DASH_Q8_E4M3, 1>
         : parts == 2 ? weight_grad_kernel<DASH_Q8_E4M3, 2>
                      : weight_grad_kernel<DASH_Q8_E4M3, 3>;
}
int smem_of(int parts) {
  return parts == 1 ? WCfg<1>::SMEM : (parts == 2 ? WCfg<2>::SMEM : WCfg<3>::SMEM);
}

// CTA pairs that can be resident at once, per device; 0 on error.
int resident_pairs() {
  static int cache[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if (cache[dev] == 0) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(512, 1, 1);
    cfg.blockDim = dim3(W_THREADS, 1, 1);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 1 << 30;
    for (int fmt : {DASH_Q8_INT8, DASH_Q8_E4M3})
      for (int parts = 1; parts <= 3; ++parts) {
        const void* k = reinterpret_cast<const void*>(kernel_of(fmt, parts));
        if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_of(parts)) !=
            cudaSuccess)
          return 0;
        cfg.dynamicSmemBytes = smem_of(parts);
        int m = 0;
        if (cudaOccupancyMaxActiveClusters(&m, k, &cfg) != cudaSuccess) return 0;
        n = m < n ? m : n;
      }
    const int sms = device_sm_count() / 2;
    cache[dev] = n < sms ? n : sms;
  }
  return cache[dev];
}

size_t round256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

// How the tiles are shared out among P pairs: whole tiles for as many full rounds as
// there are, the rest split along the tokens.  A split into S costs ceil(tail S / P)
// rounds of nkb / S slots; its partial tiles are written and read back once (about 0.1 us
// each when every pair does so) and a second launch joins them.  In units of one slot's
// 4 MMAs, about 0.3 us.
struct Plan {
  int tiles_m, tiles_n, nkb, parts, full, split, kper, units;
};

Plan make_plan(const WeightGradArgs& a, int pairs) {
  Plan p;
  p.tiles_m = static_cast<int>((a.outs + WT - 1) / WT);
  p.tiles_n = static_cast<int>((a.cols + WT - 1) / WT);
  p.nkb = static_cast<int>((a.rows + WK - 1) / WK);
  p.parts = a.dt == DASH_DT_F32 ? 3 : (a.dt == DASH_DT_F16 ? 2 : 1);
  const int tiles = p.tiles_m * p.tiles_n;
  const int tail = tiles % pairs;
  p.full = tiles;
  p.split = 1;
  p.kper = p.nkb;
  double best = tail ? static_cast<double>(p.nkb) * p.parts : 0.0;
  const int most = p.nkb / 4 < 64 ? p.nkb / 4 : 64;
  for (int s = 2; tail && s <= most; ++s) {
    const int kper = (p.nkb + s - 1) / s;
    const int se = (p.nkb + kper - 1) / kper;
    if (se < 2) continue;
    const double cost = static_cast<double>((tail * se + pairs - 1) / pairs) * kper * p.parts +
                        12.0 + 0.3 * tail * se;
    if (cost < best) {
      best = cost;
      p.full = tiles - tail;
      p.split = se;
      p.kper = kper;
    }
  }
  p.units = p.full + (p.split > 1 ? tail * p.split : 0);
  return p;
}

// Whether TMA can read dz where it lies.
bool dz_direct(const WeightGradArgs& a) {
  return a.dt == DASH_DT_BF16 && (reinterpret_cast<uintptr_t>(a.dz) & 15u) == 0 &&
         a.lddz % 8 == 0 && a.lddz > 0;
}

long long part_ld(const WeightGradArgs& a) { return (a.outs + 7) / 8 * 8; }

template <typename T, int PARTS>
cudaError_t run_split(const WeightGradArgs& a, uint16_t* out, cudaStream_t st) {
  const long long gx = (a.outs + 255) / 256;
  const dim3 grid(static_cast<unsigned>(gx < 64 ? gx : 64),
                  static_cast<unsigned>(a.rows < 65535 ? a.rows : 65535));
  split_kernel<T, PARTS><<<grid, 256, 0, st>>>(static_cast<const T*>(a.dz), a.rows, a.outs,
                                               a.lddz, part_ld(a), out);
  return cudaGetLastError();
}

}  // namespace

// Workspace: db (when only beta needs it), the column sums' partials, dz's parts, the
// partial tiles.  Without a device (sizes asked for on the host alone) the most partial
// tiles any number of pairs can need.
static size_t carve(const WeightGradArgs& a, const Plan& p, size_t& o_part, size_t& o_dz,
                    size_t& o_tiles) {
  size_t n = round256(static_cast<size_t>(a.outs) * 4);
  o_part = n;
  n += round256(static_cast<size_t>(a.outs) * 4 * col_sum_parts(a.rows, a.outs));
  o_dz = n;
  if (!dz_direct(a))
    n += round256(static_cast<size_t>(p.parts) * a.rows * part_ld(a) * 2);
  o_tiles = n;
  n += static_cast<size_t>(p.units - p.full) * WT * WT * 4;
  return n;
}

size_t weight_grad_ws(const WeightGradArgs& a) {
  const int pairs = resident_pairs();
  size_t x, y, z;
  return carve(a, make_plan(a, pairs > 0 ? pairs : 76), x, y, z);
}

dash_status launch_weight_grad(const WeightGradArgs& a, void* ws, cudaStream_t st) {
  const int pairs = resident_pairs();
  if (pairs <= 0) return DASH_ERR_CUDA;
  const Plan plan = make_plan(a, pairs);
  size_t o_part, o_dz, o_tiles;
  carve(a, plan, o_part, o_dz, o_tiles);
  uint8_t* w = static_cast<uint8_t*>(ws);
  float* db = a.db;
  if (a.db || a.beta) {
    if (!db) db = reinterpret_cast<float*>(w);
    const dash_status s = launch_col_sum(a.dz, a.dt, a.rows, a.outs, a.lddz,
                                         reinterpret_cast<float*>(w + o_part), db, st);
    if (s != DASH_OK) return s;
  }
  const int rec = trace_begin(st);
  cudaError_t err = cudaSuccess;
  WParams p = {};
  p.nkb = plan.nkb;
  p.tiles_m = plan.tiles_m;
  p.tiles_n = plan.tiles_n;
  p.full = plan.full;
  p.split = plan.split;
  p.kper = plan.kper;
  p.units = plan.units;
  p.rows = a.rows;
  p.ng = (a.cols + Q8_GROUP - 1) / Q8_GROUP;
  p.scale = a.scale;
  p.db = a.beta ? db : nullptr;
  p.partial = reinterpret_cast<float*>(w + o_tiles);
  p.a = a;
  if (a.rows > 0) {
    const void* dz = a.dz;
    uint64_t row_bytes = static_cast<uint64_t>(a.lddz) * 2, plane_bytes = row_bytes * a.rows;
    if (!dz_direct(a)) {
      uint16_t* out = reinterpret_cast<uint16_t*>(w + o_dz);
      if (a.dt == DASH_DT_F32)
        err = run_split<float, 3>(a, out, st);
      else if (a.dt == DASH_DT_F16)
        err = run_split<__half, 2>(a, out, st);
      else
        err = run_split<__nv_bfloat16, 1>(a, out, st);
      dz = out;
      row_bytes = static_cast<uint64_t>(part_ld(a)) * 2;
      plane_bytes = row_bytes * a.rows;
    }
    CUtensorMap tA, tQ;
    if (err != cudaSuccess ||
        !make_map(&tA, dz, false, a.outs, a.rows, plan.parts, row_bytes, plane_bytes, 64, WK,
                  true) ||
        !make_map(&tQ, a.q, true, p.ng * Q8_GROUP, a.rows, 1, p.ng * Q8_GROUP,
                  static_cast<uint64_t>(p.ng) * Q8_GROUP * a.rows, 128, WK, false)) {
      trace_end(rec, st, DASH_TRACE_GEMM_BF16, 0.0, 0.0);
      return DASH_ERR_CUDA;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(2 * (plan.units < pairs ? plan.units : pairs)), 1, 1);
    cfg.blockDim = dim3(W_THREADS, 1, 1);
    cfg.dynamicSmemBytes = smem_of(plan.parts);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, kernel_of(a.fmt, plan.parts), tA, tQ, p);
  }
  const int tiles = plan.tiles_m * plan.tiles_n;
  if (a.rows == 0) {
    p.full = 0;
    p.split = 0;
  }
  if (err == cudaSuccess && p.full < tiles) {
    const int n = tiles - p.full;
    const long long need = static_cast<long long>(n) * (WT * WT / 4 / 256);
    const long long cap = static_cast<long long>(device_sm_count()) * 8;
    weight_grad_join_kernel<<<static_cast<unsigned>(need < cap ? need : cap), 256, 0, st>>>(
        p, p.full, n);
    err = cudaGetLastError();
  }
  const long long r0 = static_cast<long long>(plan.tiles_m) * WT;
  const long long c0 = static_cast<long long>(plan.tiles_n) * WT;
  const long long pr = padded(a.outs, a.block), pc = padded(a.cols, a.block);
  if (err == cudaSuccess && (r0 < pr || c0 < pc)) {
    const dim3 grid(static_cast<unsigned>((pc + 1023) / 1024),
                    static_cast<unsigned>(pr < 8192 ? pr : 8192));
    weight_grad_pad_kernel<<<grid, 256, 0, st>>>(a, r0, c0);
    err = cudaGetLastError();
  }
  const double t = static_cast<double>(a.rows), o = static_cast<double>(a.outs),
               i = static_cast<double>(a.cols);
  trace_end(rec, st, DASH_TRACE_GEMM_BF16, 2.0 * t * o * i * plan.parts,
            t * o * dt_bytes(a.dt) + t * i * 33 / 32 + o * i * dt_bytes(a.odt));
  return err == cudaSuccess ? DASH_OK : DASH_ERR_CUDA;
}

}  // namespace dash
