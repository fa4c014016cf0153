// linear_tc.cu -- the products of the linear operator on the 5th-generation tensor cores.
//
// k_linear_tc: persistent, one CTA per SM or a pair of CTAs (cta_group::2) per 256-row tile.
//   warp 0     TMA producer: k-blocks of 64 into a ring of 128-byte-swizzled tiles
//   warp 1     MMA issuer: tcgen05.mma into one of two tensor-memory accumulators
//   warps 2-9  epilogue, two warps per tensor-memory lane quarter: bias, activation, residual,
//              staged through shared memory and out with TMA stores, while the next tile's
//              products run
// A pair shares its B columns: a k-block costs each CTA 16 KB of A and 16 KB of B for a
// 256 x 256 tile, 64 bytes per clock at the full MMA rate where a single CTA's 128 x 256
// tile needs 96. Ragged sizes need no padding in memory: TMA reads zeros past the end of a
// matrix and drops what is stored there. Every wait is bounded; one that runs out raises the
// status word, and the CTA lets its own copies and MMAs finish, frees its tensor memory and
// returns.
//
// Measured on random data, inputs that change from call to call: 4096 x 2048 x 8192 82 us (1.68 PFLOP/s; 90 with bias
// and gelu, 94 with the kept z as well), 8192 x 4096 x 4096 154 us (1.78), its dx and dw 345 us (1.59). After seconds of
// such calls the power limit makes that 170 and 355; between calls of other work the case with the kept z takes 102
// to 104. At the MMAs' full rate (512 cycles a k-block) operand reads and TMA writes together want 125 of shared memory's 128 bytes a clock.
//
// k_linear_split: for products with too few 128-row tiles to fill the GPU (decoding batches, a
// narrow output). The wide matrix (the weight) takes the MMA's 128 rows and the tokens its
// columns, so a product with a handful of tokens multiplies 16 of them, not 128; a cluster of
// up to eight CTAs shares one output tile, each with a part of K, and adds the parts in rank
// order through distributed shared memory, so the result does not depend on timing. Bound by the
// stream of the weight and by what stands around it: 4 x 4096 x 4096 9.9 us with weights that change from call to call
// (3.4 TB/s), 7.9 with one that stays in L2; start, first loads and the cluster's sum are 3 to 4 us of either.
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "act.cuh"
#include "common.cuh"
#include "linear_choice.h"
#include "linear_tc.h"

namespace moe {
namespace {

constexpr int kBK = 64;                  // k-block: one 128-byte swizzle row of bf16
constexpr int kChunkBytes = 64 * 128;    // an MN-major 64 (k) x 64 chunk
constexpr int kStage = 32 * 128;         // one 32 x 64 staging tile; a warp has two
constexpr int kEpiWarps = 8;

template <int CTAS, int BN>
struct Cfg {
  static constexpr int THREADS = 64 + 32 * kEpiWarps;
  static constexpr int TILE_M = 128 * CTAS;
  static constexpr int BCOLS = BN / CTAS;  // B columns this CTA loads
  static constexpr int A_BYTES = 128 * kBK * 2;
  static constexpr int B_BYTES = BCOLS * kBK * 2;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int STAGES = 163840 / STAGE_BYTES;
  static constexpr int EPI_OFF = STAGES * STAGE_BYTES;
  static constexpr int BAR_OFF = EPI_OFF + kEpiWarps * 2 * kStage;
  static constexpr int SMEM = BAR_OFF + 256 + 1024;
  static constexpr uint32_t TMEM_COLS = 2 * BN;
};

struct TcArgs {
  LinearGemm g;
  int kblocks, mt, nt;
  int items, whole;  // work items; the first `whole` are tiles, the others halves (BN / 2 columns) of one
};

// What a launch of k_linear_tc works on: one product or two.
template <int N>
struct TcWork {
  CUtensorMap A[N], B[N], Y[N];
  TcArgs p[N];
  int rem, extra;  // N = 2: see Walk
};

// The items of one unit (a CTA or a pair), in order. One product: every units-th item. Two: the one with
// more k-blocks first; where its last round is not full, the units from rem on take the first `extra`
// items of the second product meanwhile; the others of it are dealt out to all units. One launch in
// place of two saves a start, an end and a launch gap (9 us), and one of the two ragged last rounds.
template <int N>
struct Walk {
  const TcWork<N>& w;
  const int unit, units;
  int phase = 0, t, step, end;
  __device__ __forceinline__ Walk(const TcWork<N>& w_, int unit_, int units_) : w(w_), unit(unit_), units(units_) {
    t = unit;
    step = units;
    end = w.p[0].items;
  }
  // the next item: its product and its index there
  __device__ __forceinline__ bool next(int* prod, int* item) {
    if constexpr (N == 2) {
      while (t >= end) {
        if (++phase > 2) return false;
        t = phase == 1 ? (unit < w.rem ? w.extra : unit - w.rem) : w.extra + unit;
        step = phase == 1 ? units - w.rem : units;
        end = phase == 1 ? w.extra : w.p[1].items;
      }
    } else if (t >= end) {
      return false;
    }
    *prod = N == 2 && phase > 0 ? 1 : 0;
    *item = t;
    t += step;
    return true;
  }
};

// byte offset of 16-byte piece j of row r in a 128-byte-swizzled staging tile
__device__ __forceinline__ uint32_t piece(int r, int j) { return r * 128 + ((j ^ (r & 7)) << 4); }

// A warp's 32 x 64 piece of a row-major bf16 matrix into a staging tile and back, two columns a
// lane, the loads of eight rows in flight.
__device__ __forceinline__ void rows_in(uint32_t tile, const __nv_bfloat16* src, int64_t ld, int rows, int cols,
                                        int lane) {
  for (int r0 = 0; r0 < rows; r0 += 8) {
    uint16_t v[8][2];
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = lane + 32 * h;
        v[r][h] = r0 + r < rows && c < cols ? *reinterpret_cast<const uint16_t*>(src + (r0 + r) * ld + c) : (uint16_t)0;
      }
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = lane + 32 * h;
        asm volatile("st.shared.u16 [%0], %1;" ::"r"(tile + piece(r0 + r, c >> 3) + (c & 7) * 2), "h"(v[r][h]) : "memory");
      }
  }
}
__device__ __forceinline__ void rows_out(__nv_bfloat16* dst, int64_t ld, uint32_t tile, int rows, int cols, int lane) {
  for (int r0 = 0; r0 < rows; r0 += 8) {
    uint16_t v[8][2];
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = lane + 32 * h;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v[r][h]) : "r"(tile + piece(r0 + r, c >> 3) + (c & 7) * 2) : "memory");
      }
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = lane + 32 * h;
        if (r0 + r < rows && c < cols) *reinterpret_cast<uint16_t*>(dst + (r0 + r) * ld + c) = v[r][h];
      }
  }
}

// Tiles run down eight row blocks before they move to the next columns, so the tiles in flight
// share a few row and column blocks in L2. The tiles of a last round that would leave half of the
// units idle are given out as two halves each: 4096 x 4096 outputs are 256 tiles for 76 CTA pairs,
// 3.5 rounds in place of 4.
struct Item {
  int m, n0, half;  // row block, first column, whether BN / 2 columns
};
template <int BN>
__device__ __forceinline__ Item item_at(const TcArgs& a, int t) {
  constexpr int G = 8;
  Item it;
  it.half = t >= a.whole;
  const int h = t - a.whole;
  if (it.half) t = a.whole + (h >> 1);
  const int grp = t / (G * a.nt), r = t - grp * (G * a.nt);
  const int rows = min(G, a.mt - grp * G);
  const int n = r / rows;
  it.m = grp * G + (r - n * rows);
  it.n0 = n * BN + (it.half ? (h & 1) * (BN / 2) : 0);
  return it;
}

// Sixteen z of a row as bf16: one 32-byte store where `wide`, else a 16-byte store for each half that exists.
__device__ __forceinline__ void store_z16(__nv_bfloat16* p, const float* z, int left, bool wide) {
  if (left <= 0) return;
  const uint4 a = f_to_bf16x8(z), b = f_to_bf16x8(z + 8);
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z),
                 "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
  } else {
    *reinterpret_cast<uint4*>(p) = a;
    if (left > 8) *reinterpret_cast<uint4*>(p + 8) = b;
  }
}

// VEC: the rows of y, pre and the residual are multiples of 16 bytes (N % 8 == 0); else they are
// read and written element by element, still a whole row of the tile per instruction. F32: y is float, and
// the activation is evaluated in full precision, since no rounding to bf16 covers the fast forms' errors.
template <int CTAS, int BN, bool VEC, bool F32, int NP>
__global__ void __launch_bounds__(Cfg<CTAS, BN>::THREADS, 1)
    k_linear_tc(const __grid_constant__ TcWork<NP> work) {
  using C = Cfg<CTAS, BN>;
  constexpr bool PAIR = CTAS == 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  uint64_t* empty = full + C::STAGES;
  uint64_t* tfull = empty + C::STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;
  const int unit = PAIR ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
  const int units = PAIR ? (int)(gridDim.x >> 1) : (int)gridDim.x;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);   // the leader's producer arms it for both CTAs' bytes
      mbar_init(&empty[s], 1);  // one MMA commit (multicast to both CTAs of a pair)
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], kEpiWarps * CTAS);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    if constexpr (PAIR) tmem_alloc_pair(tmem_slot, C::TMEM_COLS);
    else tmem_alloc(tmem_slot, C::TMEM_COLS);
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync_all();  // both CTAs' barriers exist before any remote arrive
  tc_fence_after();
  pdl_wait();  // the set-up above touched no global memory; everything below may read the previous kernel's outputs
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t full0 = PAIR ? mapa_shared(smem_u32(full), 0) : smem_u32(full);
  const uint32_t tempty0 = PAIR ? mapa_shared(smem_u32(tempty), 0) : smem_u32(tempty);
  Walk<NP> walk(work, unit, units);
  int prod, t;

  if (warp == 0 && lane == 0) {
    // ------------------------------------------------------------ producer
    for (int i = 0; i < NP; ++i) {
      tma_prefetch_desc(&work.A[i]);
      tma_prefetch_desc(&work.B[i]);
    }
    int stage = 0;
    uint32_t phase = 0;
    int issued[C::STAGES];
#pragma unroll
    for (int s = 0; s < C::STAGES; ++s) issued[s] = -1;
    bool ok = true;
    while (ok && walk.next(&prod, &t)) {
      const TcArgs& args = work.p[prod];
      const LinearGemm& g = args.g;
      const CUtensorMap *tmA = &work.A[prod], *tmB = &work.B[prod];
      const Item it = item_at<BN>(args, t);
      const int m0 = it.m * C::TILE_M + (int)rank * 128;
      const int bcols = it.half ? C::BCOLS / 2 : C::BCOLS;
      const int n0 = it.n0 + (int)rank * bcols;
      const uint32_t bytes = C::A_BYTES + bcols * kBK * 2;
      for (int kb = 0; kb < args.kblocks; ++kb) {
        if (!mbar_wait_bounded(&empty[stage], phase ^ 1u, abort_flag)) {
          ok = false;
          break;
        }
        const uint32_t sa = smem_u32(smem + stage * C::STAGE_BYTES), sb = sa + C::A_BYTES;
        const uint32_t fb = full0 + stage * 8;
        if (leader) mbar_arrive_expect_tx(&full[stage], CTAS * bytes);
        issued[stage] = (int)phase;
        auto load = [&](uint32_t dst, const CUtensorMap* map, int c0, int c1) {
          if constexpr (PAIR) tma_load_2d_pair(dst, map, fb, c0, c1);
          else tma_load_2d(dst, map, fb, c0, c1);
        };
        if (g.a_mn) {
          load(sa, tmA, m0, kb * kBK);
          load(sa + kChunkBytes, tmA, m0 + 64, kb * kBK);
        } else {
          load(sa, tmA, kb * kBK, m0);
        }
        if (g.b_mn) {
#pragma unroll
          for (int c = 0; c < C::BCOLS / 64; ++c)
            if (c * 64 < bcols) load(sb + c * kChunkBytes, tmB, n0 + c * 64, kb * kBK);
        } else {  // boxes of BCOLS / 2 rows
          load(sb, tmB, kb * kBK, n0);
          if (!it.half) load(sb + C::B_BYTES / 2, tmB, kb * kBK, n0 + C::BCOLS / 2);
        }
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // no copy of ours may still be landing when the CTA leaves
    if (leader)
      for (int s = 0; s < C::STAGES; ++s)
        if (issued[s] >= 0) mbar_wait_timed(&full[s], (uint32_t)issued[s], 200000000ull);
  } else if (warp == 1 && lane == 0 && leader) {
    // ------------------------------------------------------------ MMA issuer
    uint32_t idesc = 0;
    const uint32_t sa0 = smem_u32(smem);
    auto mma = [&](uint32_t d, uint64_t a, uint64_t b, uint32_t acc) {
      if constexpr (PAIR) tc_mma_bf16_pair(d, a, b, idesc, acc);
      else tc_mma_bf16(d, a, b, idesc, acc);
    };
    int stage = 0, acc_i = 0;
    uint32_t phase = 0;
    bool ok = true;
    while (ok && walk.next(&prod, &t)) {
      const TcArgs& args = work.p[prod];
      const LinearGemm& g = args.g;
      const uint64_t ad0 = g.a_mn ? sdesc_sw128(sa0, kChunkBytes, 1024) : sdesc_sw128(sa0, 16, 1024);
      const uint64_t bd0 =
          g.b_mn ? sdesc_sw128(sa0 + C::A_BYTES, kChunkBytes, 1024) : sdesc_sw128(sa0 + C::A_BYTES, 16, 1024);
      const uint64_t as = g.a_mn ? 2048 >> 4 : 32 >> 4, bs = g.b_mn ? 2048 >> 4 : 32 >> 4;
      const int acc = acc_i & 1;
      const uint32_t par = (uint32_t)((acc_i >> 1) & 1);
      const bool free_acc = PAIR ? mbar_wait_bounded_cluster(&tempty[acc], par ^ 1u, abort_flag)
                                 : mbar_wait_bounded(&tempty[acc], par ^ 1u, abort_flag);
      if (!free_acc) break;
      tc_fence_after();
      const uint32_t d = tmem_base + (uint32_t)(acc * BN);
      idesc = idesc_bf16(C::TILE_M, t >= args.whole ? BN / 2 : BN, g.a_mn, g.b_mn);
      for (int kb = 0; kb < args.kblocks; ++kb) {
        if (!mbar_wait_bounded(&full[stage], phase, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t ad = ad0 + (uint64_t)(stage * (C::STAGE_BYTES >> 4));
        const uint64_t bd = bd0 + (uint64_t)(stage * (C::STAGE_BYTES >> 4));
        mma(d, ad, bd, kb != 0 ? 1u : 0u);
        mma(d, ad + as, bd + bs, 1u);
        mma(d, ad + 2 * as, bd + 2 * bs, 1u);
        mma(d, ad + 3 * as, bd + 3 * bs, 1u);
        if constexpr (PAIR) tc_commit_pair_mc(&empty[stage]);
        else tc_commit(&empty[stage]);
        if (++stage == C::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      if constexpr (PAIR) tc_commit_pair_mc(&tfull[acc]);
      else tc_commit(&tfull[acc]);
      ++acc_i;
    }
    if constexpr (PAIR) tc_commit_pair(drain);
    else tc_commit(drain);
    mbar_wait_timed(drain, 0, 200000000ull);
  } else if (warp >= 2) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;    // the tensor-memory lane quarter this warp may read
    const int ew = warp - 2;
    const uint32_t tile = smem_u32(smem + C::EPI_OFF + ew * 2 * kStage);
    int acc_i = 0;
    int sc = 0;  // chunks stored so far
    while (walk.next(&prod, &t)) {
      const TcArgs& args = work.p[prod];
      const LinearGemm& g = args.g;
      const __nv_bfloat16* bias = reinterpret_cast<const __nv_bfloat16*>(g.bias);
      const __nv_bfloat16* res = reinterpret_cast<const __nv_bfloat16*>(g.residual);
      const Item it = item_at<BN>(args, t);
      const int cw = BN / 64 / (it.half ? 4 : 2);  // 64-column chunks of this warp
      const int c0 = (ew / 4) * cw;
      const int64_t row0 = (int64_t)it.m * C::TILE_M + (int)rank * 128 + q * 32;  // this warp's first row
      const int rows = (int)min((int64_t)32, (int64_t)g.M - row0);              // rows of it that exist
      // y alternates between the two staging tiles and leaves by TMA. z goes out of the registers, 32 bytes
      // a lane: it spares shared memory, which the products need, a write and a read (4096 x 2048 x 8192 with gelu and
      // inputs that change: 98.3 -> 94.4 us back to back, 103.6 -> 101.9 between other work). Without VEC z takes the
      // first tile and y the second. ready(c) waits until the store that last used chunk c's tile has read it and sends
      // for its residual: for the first chunk while the products still run.
      const bool wide = VEC && g.N % 16 == 0 && (reinterpret_cast<uintptr_t>(g.pre) & 31) == 0;
      auto tile_of_y = [&] { return tile + (!VEC && g.pre ? kStage : (sc & 1) * kStage); };
      auto ready = [&](int c) {
        const int n0 = it.n0 + c * 64;
        if (rows <= 0 || n0 >= g.N) return;
        const uint32_t ty = tile_of_y();
        if (lane == 0) bulk_wait_read_but1();
        __syncwarp();
        if (!res) return;
        const int cols = min(64, g.N - n0);
        if constexpr (VEC) {  // eight lanes a row, 16 bytes each
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = (lane >> 3) + 4 * i, j = lane & 7;
            if (r < rows && 8 * j < cols) cp_async16(ty + piece(r, j), res + (row0 + r) * g.N + n0 + 8 * j);
          }
          cp_async_commit();
        } else {
          rows_in(ty, res + row0 * g.N + n0, g.N, rows, cols, lane);
        }
      };
      ready(c0);
      const int acc = acc_i & 1;
      if (!mbar_wait_bounded(&tfull[acc], (uint32_t)((acc_i >> 1) & 1), abort_flag)) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * BN);
      for (int c = c0; c < c0 + cw; ++c) {
        const int n0 = it.n0 + c * 64;
        if (rows <= 0 || n0 >= g.N) break;   // the same for the whole warp
        const int cols = min(64, g.N - n0);  // with VEC a multiple of 8
        const uint32_t ty = tile_of_y();
        ++sc;
        uint32_t v[2][32];
        tmem_ld32_async(taddr + c * 64, v[0]);
        tmem_ld32_async(taddr + c * 64 + 32, v[1]);
        // the bias travels beside the accumulator; every lane needs the same 64 values
        uint4 bv[8];
        if (VEC && bias) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            bv[j] = 8 * j < cols ? __ldg(reinterpret_cast<const uint4*>(bias + n0 + 8 * j)) : make_uint4(0, 0, 0, 0);
        }
        tmem_ld_wait(v[0]);
        tmem_ld_order(v[1]);
        float z[64];
#pragma unroll
        for (int i = 0; i < 64; ++i) z[i] = __uint_as_float(v[i >> 5][i & 31]);
        if (bias) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float b[8];
            if constexpr (VEC) {
              bf16x8_to_f(bv[j], b);
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i) b[i] = 8 * j + i < cols ? __bfloat162float(bias[n0 + 8 * j + i]) : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) z[8 * j + i] += b[i];
          }
        }
        if (g.pre) {
          if constexpr (VEC) {
            __nv_bfloat16* p = reinterpret_cast<__nv_bfloat16*>(g.pre) + (row0 + lane) * g.N + n0;
#pragma unroll
            for (int j = 0; j < 4; ++j) store_z16(p + 16 * j, z + 16 * j, lane < rows ? cols - 16 * j : 0, wide);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) st_shared_v4(tile + piece(lane, j), f_to_bf16x8(z + 8 * j));
          }
        }
        act_fwd<!F32, 64>(g.act, z, z);  // 64 independent chains: two warps a scheduler have little else to hide latency
        if (res) {
          if constexpr (VEC) cp_async_wait<0>();
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float b[8];
            bf16x8_to_f(ld_shared_v4(ty + piece(lane, j)), b);
#pragma unroll
            for (int i = 0; i < 8; ++i) z[8 * j + i] += b[i];
          }
        }
        if constexpr (!F32) {  // over the residual pieces this lane has just read
#pragma unroll
          for (int j = 0; j < 8; ++j) st_shared_v4(ty + piece(lane, j), f_to_bf16x8(z + 8 * j));
        } else if (lane < rows) {
          float* o = reinterpret_cast<float*>(g.y) + (row0 + lane) * g.N + n0;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            if constexpr (VEC) {
              if (4 * j < cols)
                *reinterpret_cast<float4*>(o + 4 * j) = make_float4(z[4 * j], z[4 * j + 1], z[4 * j + 2], z[4 * j + 3]);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (4 * j + i < cols) o[4 * j + i] = z[4 * j + i];
            }
          }
        }
        if constexpr (!VEC) {
          __syncwarp();
          const int64_t o = row0 * g.N + n0;
          if constexpr (!F32) rows_out(reinterpret_cast<__nv_bfloat16*>(g.y) + o, g.N, ty, rows, cols, lane);
          if (g.pre) rows_out(reinterpret_cast<__nv_bfloat16*>(g.pre) + o, g.N, tile, rows, cols, lane);
          __syncwarp();
          if (c + 1 < c0 + cw) ready(c + 1);
          continue;
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          if constexpr (!F32) tma_store_2d(&work.Y[prod], ty, n0, (int)row0);
          bulk_commit();
        }
        if (c + 1 < c0 + cw) ready(c + 1);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR) mbar_arrive_cluster(tempty0 + acc * 8);
        else mbar_arrive(&tempty[acc]);
      }
      ++acc_i;
    }
    cp_async_wait<0>();
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync_all();  // no CTA of the pair leaves while the other still uses it
  tc_fence_after();
  if (threadIdx.x == 0 && *abort_flag) set_status(work.p[0].g.status, MOE_ERR_TIMEOUT);
  if (warp == 2) {
    if constexpr (PAIR) tmem_dealloc_pair(tmem_base, C::TMEM_COLS);
    else tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

// ---------------------------------------------------------------- few tiles: K split over a cluster
template <int NB>
struct SplitCfg {
  static constexpr int THREADS = 192;  // producer, MMA issuer, four epilogue warps
  static constexpr int A_BYTES = 128 * kBK * 2;
  static constexpr int STAGE_BYTES = A_BYTES + NB * kBK * 2;
  static constexpr int STAGES = 110592 / STAGE_BYTES;  // two CTAs share an SM
  static constexpr int BAR_OFF = STAGES * STAGE_BYTES;
  static constexpr int SMEM = BAR_OFF + 256 + 1024;
  static constexpr uint32_t TMEM_COLS = NB < 32 ? 32 : NB;
  static_assert(NB * 128 * 4 <= BAR_OFF, "the partial sums reuse the ring");
};

// z -> y and pre for four neighbouring features of one token (n0 a multiple of 4). VEC: the rows of
// the outputs are multiples of 16 bytes, so the four values are one access.
template <bool VEC>
__device__ __forceinline__ void emit4(const LinearGemm& g, int64_t t, int n0, float (&z)[4], const float (&res)[4]) {
  const int64_t o = t * g.N + n0;
  float y[4];
  if (g.out_f32) act_fwd<false, 4>(g.act, z, y);  // no rounding to bf16 covers the fast forms' errors
  else act_fwd<true, 4>(g.act, z, y);
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] += res[i];
  __nv_bfloat16* pre = reinterpret_cast<__nv_bfloat16*>(g.pre) + o;
  if constexpr (VEC) {
    auto two = [](float a, float b) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
      return *reinterpret_cast<const uint32_t*>(&h);
    };
    if (g.pre) *reinterpret_cast<uint2*>(pre) = make_uint2(two(z[0], z[1]), two(z[2], z[3]));
    if (g.out_f32) *reinterpret_cast<float4*>(reinterpret_cast<float*>(g.y) + o) = make_float4(y[0], y[1], y[2], y[3]);
    else *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(g.y) + o) = make_uint2(two(y[0], y[1]), two(y[2], y[3]));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (n0 + i >= g.N) break;
      if (g.pre) pre[i] = __float2bfloat16_rn(z[i]);
      if (g.out_f32) reinterpret_cast<float*>(g.y)[o + i] = y[i];
      else reinterpret_cast<__nv_bfloat16*>(g.y)[o + i] = __float2bfloat16_rn(y[i]);
    }
  }
}

// four bf16 at p (as many as exist), VEC as above
template <bool VEC>
__device__ __forceinline__ void load4(const __nv_bfloat16* p, int left, float (&f)[4]) {
  if constexpr (VEC) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
    const float2 a = __bfloat1622float2(h[0]), b = __bfloat1622float2(h[1]);
    f[0] = a.x;
    f[1] = a.y;
    f[2] = b.x;
    f[3] = b.y;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = i < left ? __bfloat162float(p[i]) : 0.0f;
  }
}

// Tokens [a, e) of the tile from the parts' sums in the CTAs of the cluster: a warp a token, four
// features a lane, two tokens' loads in flight. The parts are added in rank order.
template <bool VEC, int S>
__device__ __forceinline__ void finish_tokens(const LinearGemm& g, const float* sums, int t0, int f0, int a, int e) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int n0 = f0 + 4 * lane;
  if (n0 >= g.N) return;
  const uint32_t base = smem_u32(sums) + lane * 16;
  uint32_t peer[S];
#pragma unroll
  for (int r = 0; r < S; ++r) peer[r] = S > 1 ? mapa_shared(base, r) : base;
  float b[4] = {0, 0, 0, 0};
  if (g.bias) load4<VEC>(reinterpret_cast<const __nv_bfloat16*>(g.bias) + n0, g.N - n0, b);
  for (int t = a + warp; t < e; t += 2 * warps) {
    float4 v[2][S];
    float res[2][4] = {};
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int tt = t + u * warps;
      if (tt < e) {
#pragma unroll
        for (int r = 0; r < S; ++r)
          asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(v[u][r].x), "=f"(v[u][r].y), "=f"(v[u][r].z), "=f"(v[u][r].w)
                       : "r"(peer[r] + tt * 512));
        if (g.residual)
          load4<VEC>(reinterpret_cast<const __nv_bfloat16*>(g.residual) + (int64_t)(t0 + tt) * g.N + n0, g.N - n0, res[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int tt = t + u * warps;
      if (tt < e) {
        float z[4] = {v[u][0].x, v[u][0].y, v[u][0].z, v[u][0].w};
#pragma unroll
        for (int r = 1; r < S; ++r) {
          z[0] += v[u][r].x;
          z[1] += v[u][r].y;
          z[2] += v[u][r].z;
          z[3] += v[u][r].w;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] += b[i];
        emit4<VEC>(g, t0 + tt, n0, z, res[u]);
      }
    }
  }
}

// Block (feature tile of 128, token tile of NB, part of K); the cluster holds the parts of one tile.
template <int NB, int S, bool VEC>
__global__ void __launch_bounds__(SplitCfg<NB>::THREADS)
    k_linear_split(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                   const TcArgs args) {
  using C = SplitCfg<NB>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  uint64_t* empty = full + C::STAGES;
  uint64_t* done = empty + C::STAGES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const LinearGemm& g = args.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = (int)blockIdx.x % S, tile = (int)blockIdx.x / S;
  const int f0 = (tile % args.nt) * 128, t0 = (tile / args.nt) * NB;
  const int kb0 = (int)((int64_t)args.kblocks * part / S), kb1 = (int)((int64_t)args.kblocks * (part + 1) / S);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 2) tmem_alloc(tmem_slot, C::TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();  // the set-up above touched no global memory; everything below may read the previous kernel's outputs
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0 && lane == 0) {
    // ------------------------------------------------------------ producer
    int stage = 0, issued = 0;
    uint32_t phase = 0;
    for (int kb = kb0; kb < kb1; ++kb, ++issued) {
      if (!mbar_wait_bounded(&empty[stage], phase ^ 1u, abort_flag)) break;
      const uint32_t sa = smem_u32(smem + stage * C::STAGE_BYTES), sb = sa + C::A_BYTES;
      const uint32_t fb = smem_u32(&full[stage]);
      mbar_arrive_expect_tx(&full[stage], C::STAGE_BYTES);
      if (g.b_mn) {
        tma_load_2d(sa, &tmW, fb, f0, kb * kBK);
        tma_load_2d(sa + kChunkBytes, &tmW, fb, f0 + 64, kb * kBK);
      } else {
        tma_load_2d(sa, &tmW, fb, kb * kBK, f0);
      }
      if (g.a_mn) {
#pragma unroll
        for (int c = 0; c < NB / 64; ++c) tma_load_2d(sb + c * kChunkBytes, &tmX, fb, t0 + c * 64, kb * kBK);
      } else {
        tma_load_2d(sb, &tmX, fb, kb * kBK, t0);
      }
      if (++stage == C::STAGES) {
        stage = 0;
        phase ^= 1u;
      }
    }
    // no copy of ours may still be landing when the CTA leaves
    for (int s = 0; s < min(C::STAGES, issued); ++s)
      mbar_wait_timed(&full[s], s < stage ? phase : phase ^ 1u, 200000000ull);
  } else if (warp == 1 && lane == 0) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t idesc = idesc_bf16(128, NB, g.b_mn, g.a_mn);
    const uint32_t sa0 = smem_u32(smem);
    const uint64_t ad0 = g.b_mn ? sdesc_sw128(sa0, kChunkBytes, 1024) : sdesc_sw128(sa0, 16, 1024);
    const uint64_t bd0 =
        g.a_mn ? sdesc_sw128(sa0 + C::A_BYTES, kChunkBytes, 1024) : sdesc_sw128(sa0 + C::A_BYTES, 16, 1024);
    const uint64_t as = g.b_mn ? 2048 >> 4 : 32 >> 4, bs = g.a_mn ? 2048 >> 4 : 32 >> 4;
    int stage = 0;
    uint32_t phase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!mbar_wait_bounded(&full[stage], phase, abort_flag)) break;
      tc_fence_after();
      const uint64_t ad = ad0 + (uint64_t)(stage * (C::STAGE_BYTES >> 4));
      const uint64_t bd = bd0 + (uint64_t)(stage * (C::STAGE_BYTES >> 4));
      tc_mma_bf16(tmem_base, ad, bd, idesc, kb != kb0 ? 1u : 0u);
      tc_mma_bf16(tmem_base, ad + as, bd + bs, idesc, 1u);
      tc_mma_bf16(tmem_base, ad + 2 * as, bd + 2 * bs, idesc, 1u);
      tc_mma_bf16(tmem_base, ad + 3 * as, bd + 3 * bs, idesc, 1u);
      tc_commit(&empty[stage]);
      if (++stage == C::STAGES) {
        stage = 0;
        phase ^= 1u;
      }
    }
    tc_commit(done);
    mbar_wait_timed(done, 0, 200000000ull);
  }
  __syncwarp();

  // ------------------------------------------------------------ epilogue
  const int ntok = min(NB, g.M - t0);
  float* sums = reinterpret_cast<float*>(smem);  // [token][128], over the ring once every MMA has read it
  if (warp >= 2 && mbar_wait_bounded(done, 0, abort_flag)) {
    tc_fence_after();
    const int f = (warp & 3) * 32 + lane;  // this thread's feature of the tile
    for (int c = 0; c * 32 < ntok; ++c) {
      float v[32];
      tmem_ld32(tmem_base + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)(c * 32), v);
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (c * 32 + i < ntok) sums[(c * 32 + i) * 128 + f] = v[i];
    }
  }
  // every part is in its CTA's shared memory; each CTA finishes its share of the tokens
  if constexpr (S > 1) cluster_sync_all();
  else __syncthreads();
  if (!*abort_flag) finish_tokens<VEC, S>(g, sums, t0, f0, ntok * part / S, ntok * (part + 1) / S);
  if constexpr (S > 1) cluster_sync_all();  // no CTA leaves while another still reads its sums

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0 && *abort_flag) set_status(g.status, MOE_ERR_TIMEOUT);
  if (warp == 2) tmem_dealloc(tmem_base, C::TMEM_COLS);
}

// ---------------------------------------------------------------- host side
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// launch attributes shared by the kernels of this file: stream order, and clusters of `cluster` CTAs
struct LaunchCfg {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[2];
  LaunchCfg(dim3 grid, int threads, int smem, cudaStream_t st, int cluster) {
    int n = 0;
    if (MOE_PDL) {
      at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      at[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
      at[n].id = cudaLaunchAttributeClusterDimension;
      at[n].val.clusterDim.x = (unsigned)cluster;
      at[n].val.clusterDim.y = 1;
      at[n++].val.clusterDim.z = 1;
    }
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = (unsigned)n;
  }
  LaunchCfg(const LaunchCfg&) = delete;
};

// bf16 [rows, cols], row stride ld elements, box 64 columns x box_rows, 128-byte swizzle
bool make_map(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  cuuint32_t es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(p), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// product g as number i of w: its maps and its tiles
template <int CTAS, int BN, bool VEC, bool F32, int N>
bool fill(TcWork<N>* w, int i, const LinearGemm& g) {
  using C = Cfg<CTAS, BN>;
  bool ok = g.a_mn ? make_map(&w->A[i], g.A, g.K, g.M, g.lda, kBK) : make_map(&w->A[i], g.A, g.M, g.K, g.lda, 128);
  ok = ok && (g.b_mn ? make_map(&w->B[i], g.B, g.K, g.N, g.ldb, kBK)
                     : make_map(&w->B[i], g.B, g.N, g.K, g.ldb, C::BCOLS / 2));
  w->Y[i] = w->A[i];  // where unused
  if (VEC && !F32) ok = ok && make_map(&w->Y[i], g.y, g.M, g.N, g.N, 32);
  TcArgs& a = w->p[i];
  a.g = g;
  a.kblocks = (g.K + kBK - 1) / kBK;
  a.mt = (g.M + C::TILE_M - 1) / C::TILE_M;
  a.nt = (g.N + BN - 1) / BN;
  const int64_t total = (int64_t)a.mt * a.nt;
  if (!ok || total >= (1ll << 30)) return false;
  a.items = a.whole = (int)total;
  return true;
}

// the tiles of a last round of `round` tiles over `units` as halves, where that leaves none waiting
void halve(TcArgs* a, int64_t round, int64_t units) {
  const int64_t last = round % units;
  if (2 * last > units) return;
  a->whole -= (int)last;
  a->items += (int)last;
}

template <int CTAS, int BN, bool VEC, bool F32, int N>
cudaError_t launch_work(const TcWork<N>& w, int64_t units, cudaStream_t st) {
  using C = Cfg<CTAS, BN>;
  static_assert(C::SMEM <= 232448, "shared memory budget");
  static_assert(CTAS == 1 || BN == 256, "the epilogue's warps need four chunks to share a half tile");
  auto kern = k_linear_tc<CTAS, BN, VEC, F32, N>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  LaunchCfg l(dim3((unsigned)(CTAS * units)), C::THREADS, C::SMEM, st, CTAS);
  return cudaLaunchKernelEx(&l.cfg, kern, w);
}

template <int CTAS, int BN, bool VEC, bool F32>
cudaError_t launch_tile_as(const LinearGemm& g, int sms, cudaStream_t st) {
  TcWork<1> w;
  if (!fill<CTAS, BN, VEC, F32>(&w, 0, g)) return cudaErrorInvalidValue;
  const int64_t units = sms / CTAS;
  if (CTAS == 2) halve(&w.p[0], w.p[0].items, units);
  w.rem = w.extra = 0;
  return launch_work<CTAS, BN, VEC, F32>(w, std::min<int64_t>(w.p[0].items, units), st);
}

template <int CTAS, int BN>
cudaError_t launch_tile(const LinearGemm& g, int sms, cudaStream_t st) {
  if (g.N % 8 == 0)
    return g.out_f32 ? launch_tile_as<CTAS, BN, true, true>(g, sms, st) : launch_tile_as<CTAS, BN, true, false>(g, sms, st);
  return g.out_f32 ? launch_tile_as<CTAS, BN, false, true>(g, sms, st) : launch_tile_as<CTAS, BN, false, false>(g, sms, st);
}

// Two products in one launch of CTA pairs, the longer k axis first (Walk).
cudaError_t launch_two(const LinearGemm& g0, const LinearGemm& g1, int sms, cudaStream_t st) {
  const LinearGemm &l = g0.K >= g1.K ? g0 : g1, &s = g0.K >= g1.K ? g1 : g0;
  TcWork<2> w;
  if (!fill<2, 256, true, false>(&w, 0, l) || !fill<2, 256, true, false>(&w, 1, s)) return cudaErrorInvalidValue;
  const int64_t units = sms / 2;
  w.rem = (int)(w.p[0].items % units);
  // a unit without a tile of the last round has time for `fit` tiles of the second product
  const int64_t fit = (2 * (int64_t)w.p[0].kblocks + w.p[1].kblocks) / (2 * (int64_t)w.p[1].kblocks);
  w.extra = w.rem ? (int)std::min<int64_t>((units - w.rem) * fit, w.p[1].items) : 0;
  halve(&w.p[1], w.p[1].items - w.extra, units);
  return launch_work<2, 256, true, false>(w, units, st);
}

template <int NB, int S, bool VEC>
cudaError_t launch_split_as(const LinearGemm& g, cudaStream_t st) {
  using C = SplitCfg<NB>;
  static_assert(C::SMEM <= 232448, "shared memory budget");
  auto kern = k_linear_split<NB, S, VEC>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  CUtensorMap mW, mX;
  bool ok = g.b_mn ? make_map(&mW, g.B, g.K, g.N, g.ldb, kBK) : make_map(&mW, g.B, g.N, g.K, g.ldb, 128);
  ok = ok && (g.a_mn ? make_map(&mX, g.A, g.K, g.M, g.lda, kBK) : make_map(&mX, g.A, g.M, g.K, g.lda, NB));
  if (!ok) return cudaErrorInvalidValue;
  TcArgs a;
  a.g = g;
  a.kblocks = (g.K + kBK - 1) / kBK;
  a.mt = (g.M + NB - 1) / NB;
  a.nt = (g.N + 127) / 128;
  const int64_t total = (int64_t)a.mt * a.nt * S;
  if (total >= (1ll << 31)) return cudaErrorInvalidValue;
  LaunchCfg l(dim3((unsigned)total), C::THREADS, C::SMEM, st, S);
  return cudaLaunchKernelEx(&l.cfg, kern, mW, mX, a);
}

template <int NB>
cudaError_t launch_split_nb(const LinearGemm& g, int S, cudaStream_t st) {
  if (g.a_mn && NB < 64) return cudaErrorInvalidValue;
  const bool vec = g.N % 8 == 0;
  switch (S) {
    case 1: return vec ? launch_split_as<NB, 1, true>(g, st) : launch_split_as<NB, 1, false>(g, st);
    case 2: return vec ? launch_split_as<NB, 2, true>(g, st) : launch_split_as<NB, 2, false>(g, st);
    case 4: return vec ? launch_split_as<NB, 4, true>(g, st) : launch_split_as<NB, 4, false>(g, st);
    default: return vec ? launch_split_as<NB, 8, true>(g, st) : launch_split_as<NB, 8, false>(g, st);
  }
}

}  // namespace

cudaError_t launch_linear_tc(const LinearGemm& g, int sms, cudaStream_t st) {
  const LinearChoice c = choose_linear(g.M, g.N, g.K, g.a_mn, sms);
  if (c.nb == 16) return launch_split_nb<16>(g, c.S, st);
  if (c.nb == 32) return launch_split_nb<32>(g, c.S, st);
  if (c.nb == 64) return launch_split_nb<64>(g, c.S, st);
  return c.S == 2 ? launch_tile<2, 256>(g, sms, st) : launch_tile<1, 128>(g, sms, st);
}

cudaError_t launch_linear_tc2(const LinearGemm& g0, const LinearGemm& g1, int sms, cudaStream_t st, int* launches) {
  const LinearChoice c0 = choose_linear(g0.M, g0.N, g0.K, g0.a_mn, sms);
  const LinearChoice c1 = choose_linear(g1.M, g1.N, g1.K, g1.a_mn, sms);
  const auto pair = [](const LinearChoice& c) { return c.nb == 0 && c.S == 2; };
  // k-blocks a unit walks through in both products. Together, in us (dx and dw, separate / in one launch):
  //   44: 2080 x 1096 x 2312 37.4 / 32.4;  54: 2048 x 2048 x 2048 32.9 / 31.1;
  //   88: 1500 x 2880 x 2880 43.2 / 42.3;  108: 1024 x 4096 x 4096 55.9 / 50.6, 4096 x 2048 x 2048 53.4 / 53.5;
  //   216: 8192 x 1024 x 4096 91.8 / 101, 8192 x 2048 x 2048 92.9 / 90.2;  862: 8192 x 4096 x 4096 328 / 341.
  // After the first product's ragged round the units no longer walk k in step, and what one reads is less
  // often in L2 for the others: longer walks lose more by that than a launch costs.
  const auto kblocks = [](const LinearGemm& g) {
    return (double)((g.M + 255) / 256) * ((g.N + 255) / 256) * ((g.K + kBK - 1) / kBK);
  };
  const double walk = (kblocks(g0) + kblocks(g1)) / (sms / 2);
  if (pair(c0) && pair(c1) && g0.N % 8 == 0 && g1.N % 8 == 0 && walk <= 128.0) {
    *launches += 1;
    return launch_two(g0, g1, sms, st);
  }
  *launches += 2;
  const cudaError_t e = launch_linear_tc(g0, sms, st);
  return e != cudaSuccess ? e : launch_linear_tc(g1, sms, st);
}

}  // namespace moe
