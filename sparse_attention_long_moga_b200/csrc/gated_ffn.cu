// Gated feed-forward product and its backward, as tcgen05 products on pairs of
// SMs (clusters of two CTAs, cta_group::2).
//
// Forward:   o = act(g) * u,   g = x Wg^T,  u = x Wu^T      (x [N][d], Wg, Wu [F][d])
//   one kernel: a tile is 256 tokens x 128 columns of F.  The leader CTA's B
//   rows are 128 rows of Wg, its peer's the same 128 rows of Wu, so the
//   256-column product of the pair holds a token's gate in columns [0, 128)
//   and its up value in [128, 256) of the same TMEM lane, and the epilogue
//   forms act(g) * u from fp32 accumulators without g or u ever leaving the SM.
//   e4m3 operands (kind::f8f6f4) keep the tile in bytes: 128 k a stage instead
//   of 64; the scales (one per token, one per weight row) are factors of the
//   accumulators, applied in fp32 in the epilogue.
// Backward, given do = dL/do:
//   dg = do * u * act'(g), du = do * act(g)      g, u computed again by the forward's product
//   dx = dg Wg + du Wu                           one product, K = 2F
//   dWg = dg^T x, dWu = du^T x                   one launch, K = N
//   g and u are recomputed (4 N d F of the 12 N d F operations) instead of
//   saved: a saved pair would hold 4 N F bytes per layer from the forward to
//   the backward and would be rounded to bf16.  dg and du are rounded to bf16
//   (the tensor core's operand type) once and live in the workspace only.
//
// 192 threads per CTA: warp 4 TMA producer, warp 5 TMEM allocator and (leader)
// MMA issuer, warps 0-3 epilogue, thread = token row = TMEM lane.  Two
// 256-column accumulators let a tile's epilogue overlap the next tile's
// products.  All waits are bounded.
#include "common.cuh"
#include "tc_common.cuh"

namespace moga {
namespace ffn {

using namespace moga::tc;

enum Mode { MODE_FWD = 0, MODE_DGDU = 1, MODE_DX = 2, MODE_DW = 3 };

constexpr int BM = 128;                      // accumulator rows per CTA (256 per pair)
constexpr int BN = 256;                      // accumulator columns of a tile
constexpr int kStages = 6;
constexpr int kThreads = 192;
constexpr int kRowBytes = 128;               // bytes of one operand row in a stage (one swizzle span)
constexpr int kOpBytes = 128 * kRowBytes;    // 16 KB: one operand of one CTA in a stage
constexpr int kStageBytes = 2 * kOpBytes;
constexpr int kBarOff = kStages * kStageBytes;
constexpr int kMiscOff = kBarOff + 32 * 8;
constexpr int kSmemBytes = kMiscOff + 64 + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory");
constexpr int kGroupM = 8;                   // row tiles per band of the tile order

constexpr int B_FULL = 0;                    // [kStages]
constexpr int B_EMPTY = kStages;             // [kStages]
constexpr int B_ACC_FULL = 2 * kStages;      // [2]
constexpr int B_ACC_EMPTY = B_ACC_FULL + 2;  // [2] (both CTAs' epilogue threads)
constexpr int B_END = B_ACC_EMPTY + 2;
static_assert(B_END < 32, "barrier area");

struct Params {
  int rows, cols;            // of the output (FWD, DGDU: N x F; DX: N x d; DW: F x d)
  int n_k;                   // k stages of a tile
  int seg_k;                 // DX: stages of the gate half (F / 64 rounded up)
  int m_tiles, n_tiles;      // 256-row tiles (DW: of one matrix), column tiles
  int total;                 // tiles
  int act;
  const float *xs, *gs, *us; // e4m3 scales
  const __nv_bfloat16* dh;   // DGDU
  __nv_bfloat16 *o0, *o1;    // FWD: o; DGDU: dg, du; DX: dx; DW: dWg, dWu
  long long timeout;
};

// Tile t -> (row tile, column tile).  Tiles run down bands of kGroupM row
// tiles, so that the pairs at work at one time share a few row tiles and a
// few column tiles in L2 instead of sweeping all of W for every row tile.
__device__ __forceinline__ void tile_of(int t, int m_tiles, int n_tiles, int* m, int* n) {
  const int band = kGroupM * n_tiles;
  const int b = t / band, r = t - b * band;
  const int gm = min(kGroupM, m_tiles - b * kGroupM);
  *n = r / gm;
  *m = b * kGroupM + (r - *n * gm);
}

__device__ __forceinline__ void mma_pair_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0;"
      " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p; }" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// instruction descriptors of a pair's M = 256, N = 256 product
constexpr uint32_t kIdescBf16 = pair_desc(instr_desc(BN, false));
constexpr uint32_t kIdescBMn = pair_desc(instr_desc(BN, true));
constexpr uint32_t kIdescABMn = kIdescBMn | (1u << 15);
constexpr uint32_t kIdescE4m3 = kIdescBf16 & ~((7u << 7) | (7u << 10));   // e4m3 x e4m3 (format 0)

// Activation and its derivative in fp32.  silu: g s, s = 1 / (1 + e^-g);
// gelu: the tanh form, 0.5 (1 + tanh z) = 1 / (1 + e^-2z),
// z = sqrt(2 / pi) (g + 0.044715 g^3).  e^-x overflows to infinity for large
// negative x, where the quotient is 0 as it should be; g * s is then -0.
__device__ __forceinline__ float sigmoid_of(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }
constexpr float kGelu2 = 1.5957691216057308f;    // 2 sqrt(2 / pi)
template <int ACT>
__device__ __forceinline__ float act_of(float g) {
  if (ACT == MOGA_ACT_SILU) return g * sigmoid_of(g);
  return g * sigmoid_of(kGelu2 * (g + 0.044715f * g * g * g));
}
template <int ACT>
__device__ __forceinline__ void act_and_grad(float g, float* a, float* da) {
  if (ACT == MOGA_ACT_SILU) {
    const float s = sigmoid_of(g);
    *a = g * s;
    *da = s + *a * (1.f - s);
  } else {
    const float s = sigmoid_of(kGelu2 * (g + 0.044715f * g * g * g));
    *a = g * s;
    *da = s + *a * (1.f - s) * (kGelu2 * (1.f + 0.134145f * g * g));
  }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 32 fp32 values to bf16 columns [col, col + 32) of a row; columns at or past
// `cols` (a multiple of 8) are skipped
__device__ __forceinline__ void store32(__nv_bfloat16* row, int col, int cols, const float* v) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (col + 8 * e < cols)
      *reinterpret_cast<uint4*>(row + col + 8 * e) =
          make_uint4(pack2(v[8 * e], v[8 * e + 1]), pack2(v[8 * e + 2], v[8 * e + 3]),
                     pack2(v[8 * e + 4], v[8 * e + 5]), pack2(v[8 * e + 6], v[8 * e + 7]));
}

template <int MODE, bool E4M3, int ACT>
__device__ __forceinline__ void epilogue_gated(const Params& p, uint32_t acc, int row, int col0) {
  const bool in = row < p.rows;
  const float xs = E4M3 && in ? __ldg(p.xs + row) : 1.f;
#pragma unroll 1
  for (int c0 = 0; c0 < BN / 2; c0 += 32) {
    float g[32], u[32];
    tmem_ld32(acc + c0, g);
    tmem_ld32(acc + BN / 2 + c0, u);
    tmem_wait_ld();
    const int col = col0 + c0;
    if (in && col < p.cols) {
      if (E4M3) {
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const int cc = min(col + j, p.cols - 1);
          g[j] *= xs * __ldg(p.gs + cc);
          u[j] *= xs * __ldg(p.us + cc);
        }
      }
      if (MODE == MODE_FWD) {
#pragma unroll
        for (int j = 0; j < 32; ++j) g[j] = act_of<ACT>(g[j]) * u[j];
        store32(p.o0 + (size_t)row * p.cols, col, p.cols, g);
      } else {
        const __nv_bfloat16* dh = p.dh + (size_t)row * p.cols + col;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint4 t = make_uint4(0, 0, 0, 0);
          if (col + 8 * e < p.cols) t = *reinterpret_cast<const uint4*>(dh + 8 * e);
          const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float d = __uint_as_float((i & 1) ? (w[i >> 1] & 0xffff0000u) : (w[i >> 1] << 16));
            float a, da;
            act_and_grad<ACT>(g[8 * e + i], &a, &da);
            g[8 * e + i] = d * u[8 * e + i] * da;
            u[8 * e + i] = d * a;
          }
        }
        store32(p.o0 + (size_t)row * p.cols, col, p.cols, g);
        store32(p.o1 + (size_t)row * p.cols, col, p.cols, u);
      }
    }
    __syncwarp();   // the next tcgen05.ld is the whole warp's
  }
}

template <int MODE, bool E4M3, int ACT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
ffn_kernel(const __grid_constant__ Params p, const __grid_constant__ CUtensorMap tm_a0,
           const __grid_constant__ CUtensorMap tm_a1, const __grid_constant__ CUtensorMap tm_b0,
           const __grid_constant__ CUtensorMap tm_b1) {
  constexpr int BK = E4M3 ? 128 : 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + kBarOff + 8u * (uint32_t)i; };
  int* misc = reinterpret_cast<int*>(smem + kMiscOff);
  volatile int* abort_flag = misc;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();          // 0: leader, 1: peer
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar(B_FULL + s), 1);
      mbar_init(bar(B_EMPTY + s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar(B_ACC_FULL + b), 1);
      mbar_init(bar(B_ACC_EMPTY + b), 2 * BM);
    }
    mbar_init(bar(B_END), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 5) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // both CTAs' barriers are initialised before any remote use
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // row tile (of both matrices in DW) and column tile of tile t
  auto decode = [&](int t, int* m, int* n) {
    tile_of(t, MODE == MODE_DW ? 2 * p.m_tiles : p.m_tiles, p.n_tiles, m, n);
  };

  if (warp == 4) {
    // ------------------------------------------------------------------ producer
    if (lane == 0) {
      int c = 0;
      bool ok = true;
      for (int t = pair; t < p.total && ok; t += n_pairs) {
        int m, n;
        decode(t, &m, &n);
        for (int kt = 0; kt < p.n_k; ++kt, ++c) {
          const int st = c % kStages;
          if (!(ok = mbar_wait(bar(B_EMPTY + st), ((c / kStages) & 1) ^ 1, abort_flag, p.timeout))) break;
          const uint32_t full = peer_addr(bar(B_FULL + st), 0);
          // the leader's barrier expects both CTAs' bytes
          if (leader) mbar_arrive_expect_tx(bar(B_FULL + st), 2 * kStageBytes);
          const uint32_t a = sbase + st * kStageBytes, b = a + kOpBytes;
          if (MODE == MODE_FWD || MODE == MODE_DGDU) {
            tma_load_2d_pair(a, &tm_a0, kt * BK, (m * 2 + (int)rank) * BM, full);
            tma_load_2d_pair(b, leader ? &tm_b0 : &tm_b1, kt * BK, n * (BN / 2), full);
          } else if (MODE == MODE_DX) {
            const bool up = kt >= p.seg_k;
            const int k0 = (up ? kt - p.seg_k : kt) * BK;
            const CUtensorMap* mb = up ? &tm_b1 : &tm_b0;
            const int c0 = n * BN + (int)rank * (BN / 2);
            tma_load_2d_pair(a, up ? &tm_a1 : &tm_a0, k0, (m * 2 + (int)rank) * BM, full);
            tma_load_2d_pair(b, mb, c0, k0, full);                       // 64 columns x 64 k rows
            tma_load_2d_pair(b + kOpBytes / 2, mb, c0 + 64, k0, full);
          } else {
            const bool up = m >= p.m_tiles;
            const CUtensorMap* ma = up ? &tm_a1 : &tm_a0;
            const int r0 = ((up ? m - p.m_tiles : m) * 2 + (int)rank) * BM;
            const int c0 = n * BN + (int)rank * (BN / 2);
            tma_load_2d_pair(a, ma, r0, kt * BK, full);
            tma_load_2d_pair(a + kOpBytes / 2, ma, r0 + 64, kt * BK, full);
            tma_load_2d_pair(b, &tm_b0, c0, kt * BK, full);
            tma_load_2d_pair(b + kOpBytes / 2, &tm_b0, c0 + 64, kt * BK, full);
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 5) {
    // ------------------------------------------------------------------ MMA issuer (leader)
    if (leader && lane == 0) {
      int c = 0, j = 0;   // stage and local tile counters
      bool ok = true;
      for (int t = pair; t < p.total && ok; t += n_pairs, ++j) {
        const int b = j & 1;
        if (!(ok = mbar_wait(bar(B_ACC_EMPTY + b), ((j >> 1) & 1) ^ 1, abort_flag, p.timeout))) break;
        tc_fence_after();
        const uint32_t acc = tmem + b * BN;
        for (int kt = 0; kt < p.n_k; ++kt, ++c) {
          const int st = c % kStages;
          if (!(ok = mbar_wait(bar(B_FULL + st), (c / kStages) & 1, abort_flag, p.timeout))) break;
          tc_fence_after();
          const uint32_t sa = sbase + st * kStageBytes, sb = sa + kOpBytes;
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            const uint32_t accum = (kt > 0 || ks > 0) ? 1u : 0u;
            // K-major operands advance 32 bytes along their rows; MN-major
            // ones 16 k rows of 128 bytes (64-column halves kOpBytes / 2 apart)
            const uint64_t ak = smem_desc(sa + ks * 32, 16, 1024), bk = smem_desc(sb + ks * 32, 16, 1024);
            const uint64_t am = smem_desc(sa + ks * 2048, kOpBytes / 2, 1024);
            const uint64_t bm = smem_desc(sb + ks * 2048, kOpBytes / 2, 1024);
            if (MODE == MODE_DW) mma_pair(acc, am, bm, kIdescABMn, accum);
            else if (MODE == MODE_DX) mma_pair(acc, ak, bm, kIdescBMn, accum);
            else if (E4M3) mma_pair_f8(acc, ak, bk, kIdescE4m3, accum);
            else mma_pair(acc, ak, bk, kIdescBf16, accum);
          }
          commit_pair(bar(B_EMPTY + st));
        }
        if (!ok) break;
        commit_pair(bar(B_ACC_FULL + b));
      }
      commit_pair(bar(B_END));
      mbar_drain(bar(B_END), 0, p.timeout);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ epilogue
    const uint32_t lane_addr = (uint32_t)(warp * 32) << 16;
    int j = 0;
    for (int t = pair; t < p.total; t += n_pairs, ++j) {
      int m, n;
      decode(t, &m, &n);
      const int b = j & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(bar(B_ACC_FULL + b), (j >> 1) & 1, abort_flag, p.timeout))) break;
      tc_fence_after();
      const uint32_t acc = tmem + lane_addr + b * BN;
      if (MODE == MODE_FWD || MODE == MODE_DGDU) {
        epilogue_gated<MODE, E4M3, ACT>(p, acc, (m * 2 + (int)rank) * BM + warp * 32 + lane, n * (BN / 2));
      } else {
        const bool up = MODE == MODE_DW && m >= p.m_tiles;
        const int row = ((up ? m - p.m_tiles : m) * 2 + (int)rank) * BM + warp * 32 + lane;
        __nv_bfloat16* out = (up ? p.o1 : p.o0) + (size_t)row * p.cols;
#pragma unroll 1
        for (int c0 = 0; c0 < BN; c0 += 32) {
          float v[32];
          tmem_ld32(acc + c0, v);
          tmem_wait_ld();
          if (row < p.rows) store32(out, n * BN + c0, p.cols, v);
          __syncwarp();
        }
      }
      tc_fence_before();
      mbar_arrive_cluster(peer_addr(bar(B_ACC_EMPTY + b), 0));
    }
  }

  // every product of the pair has completed (the leader drained them) and no
  // remote arrival is pending before either CTA frees its TMEM and exits
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (warp == 5) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

// ---------------------------------------------------------------- few tokens
//
// Up to kFewTokens tokens the weights' read is the time (2 F d elements for
// N d + N F others), and a 256-row tile would idle.  A CTA takes 8 RT columns
// of F and all tokens; its 8 warps split d, each streaming 64-byte pieces of
// 16 RT weight rows straight from global memory into mma.sync fragments: one
// 16-row A tile is 8 gate rows over the 8 up rows of the same columns, so a
// lane's accumulators hold gate and up of the same outputs.  A lane loads 16
// consecutive bytes of a row where the fragment wants four pieces spread over
// k; the sum over k does not mind the order as long as x is read in the same
// one.  No shared-memory stage, no barrier in the loop: with UN steps unrolled
// a lane keeps 2 RT UN 16-byte loads in flight.  The warps' sums meet in
// shared memory in a fixed order.
constexpr int kFewTokens = 32;

__device__ __forceinline__ uint4 ldg_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
// D += A (16 rows x 32 bytes of k) B (8 columns): one legacy tensor-core step
template <bool E4M3>
__device__ __forceinline__ void mma_16x8(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if (E4M3)
    asm volatile("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct FewParams {
  const uint8_t *x, *wg, *wu;   // rows of `row_bytes` bytes
  int N, F, row_bytes;
  const float *xs, *gs, *us;
  __nv_bfloat16* out;
};

template <bool E4M3, int ACT, int RT, int NT, int UN>
__global__ void __launch_bounds__(256) ffn_few_kernel(const FewParams p) {
  constexpr int kCols = 8 * RT, kToks = 8 * NT;
  __shared__ float red[8][RT * NT * 4][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int f0 = blockIdx.x * kCols;
  const uint8_t *wg[RT], *wu[RT], *xp[NT];
  bool won[RT], xon[NT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int f = f0 + 8 * r + g;
    won[r] = f < p.F;
    wg[r] = p.wg + (size_t)(won[r] ? f : 0) * p.row_bytes + 16 * q;
    wu[r] = p.wu + (size_t)(won[r] ? f : 0) * p.row_bytes + 16 * q;
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    xon[n] = 8 * n + g < p.N;
    xp[n] = p.x + (size_t)(xon[n] ? 8 * n + g : 0) * p.row_bytes + 16 * q;
  }
  float acc[RT][NT][4];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[r][n][i] = 0.f;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  // step s covers bytes [64 s, 64 s + 64) of every row; warp w takes s = w, w + 8, ...
  for (int s0 = warp; 64 * s0 < p.row_bytes; s0 += 8 * UN) {
    uint4 a[UN][RT], b[UN][RT], x[UN][NT];
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      const int k = 64 * (s0 + 8 * i);
      const bool on = k + 16 * q < p.row_bytes;
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        a[i][r] = on && won[r] ? ldg_stream(wg[r] + k) : zero;
        b[i][r] = on && won[r] ? ldg_stream(wu[r] + k) : zero;
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
        x[i][n] = on && xon[n] ? __ldg(reinterpret_cast<const uint4*>(xp[n] + k)) : zero;
    }
#pragma unroll
    for (int i = 0; i < UN; ++i)
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          mma_16x8<E4M3>(acc[r][n], a[i][r].x, b[i][r].x, a[i][r].y, b[i][r].y, x[i][n].x, x[i][n].y);
          mma_16x8<E4M3>(acc[r][n], a[i][r].z, b[i][r].z, a[i][r].w, b[i][r].w, x[i][n].z, x[i][n].w);
        }
  }
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) red[warp][(r * NT + n) * 4 + i][lane] = acc[r][n][i];
  __syncthreads();
  // output (column c, token t): accumulator of tile (c / 8, t / 8), lane 4 (c % 8) + (t % 8) / 2, slot t % 2 (gate),
  // 2 + t % 2 (up)
  for (int o = threadIdx.x; o < kCols * kToks; o += 256) {
    const int c = o % kCols, t = o / kCols, f = f0 + c;
    if (f >= p.F || t >= p.N) continue;
    const int slot = ((c >> 3) * NT + (t >> 3)) * 4 + (t & 1), l = 4 * (c & 7) + ((t & 7) >> 1);
    float gate = 0.f, up = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      gate += red[w][slot][l];
      up += red[w][slot + 2][l];
    }
    if (E4M3) {
      const float xs = __ldg(p.xs + t);
      gate *= xs * __ldg(p.gs + f);
      up *= xs * __ldg(p.us + f);
    }
    p.out[(size_t)t * p.F + f] = __float2bfloat16_rn(act_of<ACT>(gate) * up);
  }
}

template <bool E4M3, int ACT>
static moga_status launch_few(const FewParams& p, const char* who, cudaStream_t s) {
  if (p.N <= 8) ffn_few_kernel<E4M3, ACT, 1, 1, 8><<<ceil_div(p.F, 8), 256, 0, s>>>(p);
  else if (p.N <= 16) ffn_few_kernel<E4M3, ACT, 2, 2, 4><<<ceil_div(p.F, 16), 256, 0, s>>>(p);
  else ffn_few_kernel<E4M3, ACT, 2, 4, 4><<<ceil_div(p.F, 16), 256, 0, s>>>(p);
  return check_launch(who);
}

// Row-major [rows][cols] matrix of 1- or 2-byte elements, boxes of 128 bytes x box_rows.
static moga_status make_map(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int elem, int box_rows) {
  auto fn = route_tc::encode_fn();
  if (!fn) return fail(MOGA_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
  cuuint64_t gdim[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t gstride[1] = {(cuuint64_t)(cols * elem)};
  cuuint32_t box[2] = {(cuuint32_t)(kRowBytes / elem), (cuuint32_t)box_rows};
  cuuint32_t estride[2] = {1, 1};
  CUresult r = fn(m, elem == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                  const_cast<void*>(base), gdim, gstride, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(MOGA_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return MOGA_OK;
}

template <int MODE, bool E4M3, int ACT>
static moga_status launch(const Params& p, const CUtensorMap& a0, const CUtensorMap& a1, const CUtensorMap& b0,
                          const CUtensorMap& b1, const char* who, cudaStream_t s) {
  auto* k = ffn_kernel<MODE, E4M3, ACT>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return fail(MOGA_ERR_CUDA, "%s: cudaFuncSetAttribute: %s", who, cudaGetErrorString(e));
  // one pair of CTAs per pair of SMs (persistent), at most one pair per tile
  const int pairs = std::min(p.total, route_tc::sm_count() / 2);
  k<<<2 * pairs, kThreads, kSmemBytes, s>>>(p, a0, a1, b0, b1);
  return check_launch(who);
}

inline int64_t ceil64(int64_t a, int64_t b) { return (a + b - 1) / b; }

static moga_status check_dims(const char* who, int64_t N, int32_t d, int32_t F, int32_t act, int elem) {
  const int m = 16 / elem;   // 16-byte rows, as the TMA copies need them
  if (N <= 0 || N > INT32_MAX / 2) return fail(MOGA_ERR_INVALID_ARG, "%s: N=%lld out of range", who, (long long)N);
  if (d <= 0 || d % m != 0)
    return fail(MOGA_ERR_INVALID_ARG, "%s: d=%d must be a positive multiple of %d", who, d, m);
  if (F <= 0 || F % 8 != 0) return fail(MOGA_ERR_INVALID_ARG, "%s: F=%d must be a positive multiple of 8", who, F);
  if (d > (1 << 20) || F > (1 << 20) || ceil64(N, 256) * ceil64(F, 128) > INT32_MAX / 2)
    return fail(MOGA_ERR_INVALID_ARG, "%s: sizes out of range", who);
  if (act != MOGA_ACT_SILU && act != MOGA_ACT_GELU)
    return fail(MOGA_ERR_INVALID_ARG, "%s: activation %d unknown", who, act);
  return MOGA_OK;
}

template <int MODE, bool E4M3>
static moga_status launch_act(const Params& p, const CUtensorMap& a0, const CUtensorMap& b0, const CUtensorMap& b1,
                              const char* who, cudaStream_t s) {
  return p.act == MOGA_ACT_SILU ? launch<MODE, E4M3, MOGA_ACT_SILU>(p, a0, a0, b0, b1, who, s)
                                : launch<MODE, E4M3, MOGA_ACT_GELU>(p, a0, a0, b0, b1, who, s);
}

}  // namespace ffn
}  // namespace moga

extern "C" moga_status moga_gated_ffn(const void* x, const void* w_gate, const void* w_up, moga_dtype dt,
                                      const float* x_scale, const float* w_gate_scale, const float* w_up_scale,
                                      int64_t N, int32_t d, int32_t F, int32_t act, void* out, void* stream) {
  using namespace moga;
  using namespace moga::ffn;
  const char* who = "moga_gated_ffn";
  if (!x || !w_gate || !w_up || !out) return fail(MOGA_ERR_INVALID_ARG, "%s: null pointer", who);
  if (dt != MOGA_BF16 && dt != MOGA_E4M3) return fail(MOGA_ERR_INVALID_ARG, "%s: dtype must be bf16 or e4m3", who);
  const bool f8 = dt == MOGA_E4M3;
  if (f8 != (x_scale != nullptr) || f8 != (w_gate_scale != nullptr) || f8 != (w_up_scale != nullptr))
    return fail(MOGA_ERR_INVALID_ARG, "%s: the three scales go with e4m3 operands", who);
  const int elem = f8 ? 1 : 2;
  moga_status st = check_dims(who, N, d, F, act, elem);
  if (st != MOGA_OK) return st;
  const uintptr_t a = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(w_gate) |
                      reinterpret_cast<uintptr_t>(w_up) | reinterpret_cast<uintptr_t>(out);
  const uintptr_t a4 = reinterpret_cast<uintptr_t>(x_scale) | reinterpret_cast<uintptr_t>(w_gate_scale) |
                       reinterpret_cast<uintptr_t>(w_up_scale);
  if ((a & 15) || (a4 & 3))
    return fail(MOGA_ERR_INVALID_ARG, "%s: x, w_gate, w_up, out must be 16-byte aligned", who);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (N <= kFewTokens) {
    FewParams q = {};
    q.x = static_cast<const uint8_t*>(x);
    q.wg = static_cast<const uint8_t*>(w_gate);
    q.wu = static_cast<const uint8_t*>(w_up);
    q.N = (int)N;
    q.F = F;
    q.row_bytes = d * elem;
    q.xs = x_scale;
    q.gs = w_gate_scale;
    q.us = w_up_scale;
    q.out = static_cast<__nv_bfloat16*>(out);
    if (act == MOGA_ACT_SILU)
      return f8 ? launch_few<true, MOGA_ACT_SILU>(q, who, s) : launch_few<false, MOGA_ACT_SILU>(q, who, s);
    return f8 ? launch_few<true, MOGA_ACT_GELU>(q, who, s) : launch_few<false, MOGA_ACT_GELU>(q, who, s);
  }
  CUtensorMap mx, mg, mu;
  if ((st = make_map(&mx, x, N, d, elem, ffn::BM)) != MOGA_OK) return st;
  if ((st = make_map(&mg, w_gate, F, d, elem, ffn::BN / 2)) != MOGA_OK) return st;
  if ((st = make_map(&mu, w_up, F, d, elem, ffn::BN / 2)) != MOGA_OK) return st;
  ffn::Params p = {};
  p.rows = (int)N;
  p.cols = F;
  p.n_k = ceil_div(d, kRowBytes / elem);
  p.m_tiles = ceil_div((int)N, 2 * ffn::BM);
  p.n_tiles = ceil_div(F, ffn::BN / 2);
  p.total = p.m_tiles * p.n_tiles;
  p.act = act;
  p.xs = x_scale;
  p.gs = w_gate_scale;
  p.us = w_up_scale;
  p.o0 = static_cast<__nv_bfloat16*>(out);
  p.timeout = kWaitLimitCycles;
  return f8 ? launch_act<MODE_FWD, true>(p, mx, mg, mu, who, s) : launch_act<MODE_FWD, false>(p, mx, mg, mu, who, s);
}

extern "C" size_t moga_gated_ffn_bwd_ws_bytes(int64_t N, int32_t d, int32_t F) {
  if (N <= 0 || N > INT32_MAX / 2 || d <= 0 || d % 8 != 0 || F <= 0 || F % 8 != 0 || d > (1 << 20) || F > (1 << 20))
    return 0;
  return (size_t)2 * N * F * 2;
}

extern "C" moga_status moga_gated_ffn_bwd(const void* x, const void* w_gate, const void* w_up, int64_t N, int32_t d,
                                          int32_t F, int32_t act, const void* dout, void* dx, void* dw_gate,
                                          void* dw_up, void* ws, size_t ws_bytes, void* stream) {
  using namespace moga;
  using namespace moga::ffn;
  const char* who = "moga_gated_ffn_bwd";
  if (!x || !w_gate || !w_up || !dout || !ws) return fail(MOGA_ERR_INVALID_ARG, "%s: null pointer", who);
  if ((dw_gate != nullptr) != (dw_up != nullptr))
    return fail(MOGA_ERR_INVALID_ARG, "%s: dw_gate and dw_up go together", who);
  if (!dx && !dw_gate) return fail(MOGA_ERR_INVALID_ARG, "%s: no gradient asked for", who);
  moga_status st = check_dims(who, N, d, F, act, 2);
  if (st != MOGA_OK) return st;
  if (ceil64(N, 256) * ceil64(d, 256) > INT32_MAX / 2)
    return fail(MOGA_ERR_INVALID_ARG, "%s: sizes out of range", who);
  const uintptr_t a = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(w_gate) |
                      reinterpret_cast<uintptr_t>(w_up) | reinterpret_cast<uintptr_t>(dout) |
                      reinterpret_cast<uintptr_t>(dx) | reinterpret_cast<uintptr_t>(dw_gate) |
                      reinterpret_cast<uintptr_t>(dw_up) | reinterpret_cast<uintptr_t>(ws);
  if (a & 15) return fail(MOGA_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned", who);
  const size_t need = moga_gated_ffn_bwd_ws_bytes(N, d, F);
  if (ws_bytes < need) return fail(MOGA_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes", who, ws_bytes, need);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  __nv_bfloat16* dg = static_cast<__nv_bfloat16*>(ws);
  __nv_bfloat16* du = dg + (size_t)N * F;
  ffn::Params p = {};
  p.act = act;
  p.timeout = kWaitLimitCycles;
  {
    CUtensorMap mx, mg, mu;
    if ((st = make_map(&mx, x, N, d, 2, ffn::BM)) != MOGA_OK) return st;
    if ((st = make_map(&mg, w_gate, F, d, 2, ffn::BN / 2)) != MOGA_OK) return st;
    if ((st = make_map(&mu, w_up, F, d, 2, ffn::BN / 2)) != MOGA_OK) return st;
    p.rows = (int)N;
    p.cols = F;
    p.n_k = ceil_div(d, 64);
    p.m_tiles = ceil_div((int)N, 2 * ffn::BM);
    p.n_tiles = ceil_div(F, ffn::BN / 2);
    p.total = p.m_tiles * p.n_tiles;
    p.dh = static_cast<const __nv_bfloat16*>(dout);
    p.o0 = dg;
    p.o1 = du;
    if ((st = launch_act<MODE_DGDU, false>(p, mx, mg, mu, who, s)) != MOGA_OK) return st;
  }
  if (dx) {
    CUtensorMap ma0, ma1, mb0, mb1;
    if ((st = make_map(&ma0, dg, N, F, 2, ffn::BM)) != MOGA_OK) return st;
    if ((st = make_map(&ma1, du, N, F, 2, ffn::BM)) != MOGA_OK) return st;
    if ((st = make_map(&mb0, w_gate, F, d, 2, 64)) != MOGA_OK) return st;
    if ((st = make_map(&mb1, w_up, F, d, 2, 64)) != MOGA_OK) return st;
    p.rows = (int)N;
    p.cols = d;
    p.seg_k = ceil_div(F, 64);
    p.n_k = 2 * p.seg_k;
    p.m_tiles = ceil_div((int)N, 2 * ffn::BM);
    p.n_tiles = ceil_div(d, ffn::BN);
    p.total = p.m_tiles * p.n_tiles;
    p.o0 = static_cast<__nv_bfloat16*>(dx);
    if ((st = launch<MODE_DX, false, 0>(p, ma0, ma1, mb0, mb1, who, s)) != MOGA_OK) return st;
  }
  if (dw_gate) {
    CUtensorMap ma0, ma1, mb;
    if ((st = make_map(&ma0, dg, N, F, 2, 64)) != MOGA_OK) return st;
    if ((st = make_map(&ma1, du, N, F, 2, 64)) != MOGA_OK) return st;
    if ((st = make_map(&mb, x, N, d, 2, 64)) != MOGA_OK) return st;
    p.rows = F;
    p.cols = d;
    p.n_k = ceil_div((int)N, 64);
    p.m_tiles = ceil_div(F, 2 * ffn::BM);
    p.n_tiles = ceil_div(d, ffn::BN);
    p.total = 2 * p.m_tiles * p.n_tiles;
    p.o0 = static_cast<__nv_bfloat16*>(dw_gate);
    p.o1 = static_cast<__nv_bfloat16*>(dw_up);
    if ((st = launch<MODE_DW, false, 0>(p, ma0, ma1, mb, mb, who, s)) != MOGA_OK) return st;
  }
  return MOGA_OK;
}
