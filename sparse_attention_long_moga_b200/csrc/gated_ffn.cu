// Gated feed-forward product and its backward, as tcgen05 products on pairs of
// SMs (clusters of two CTAs, cta_group::2).
//
// Forward:   o = act(g) * u,   g = x Wg^T,  u = x Wu^T      (x [N][d], Wg, Wu [F][d])
//   one kernel: a tile is 256 tokens x BN / 2 columns of F.  The leader CTA's
//   B rows are BN / 2 rows of Wg, its peer's the same rows of Wu, so the
//   BN-column product of the pair holds a token's gate in columns [0, BN / 2)
//   and its up value in [BN / 2, BN) of the same TMEM lane, and the epilogue
//   forms act(g) * u from fp32 accumulators without g or u ever leaving the SM.
//   e4m3 operands (kind::f8f6f4) keep the tile in bytes: 128 k a stage instead
//   of 64; the scales (one per token, one per weight row) are factors of the
//   accumulators, applied in fp32 in the epilogue.
// Backward, given do = dL/do:
//   dg = do * u * act'(g), du = do * act(g)      g, u computed again by the forward's product
//   dx = dg Wg + du Wu                           K = 2F
//   dWg = dg^T x, dWu = du^T x                   K = N
//   g and u are recomputed (4 N d F of the 12 N d F operations) instead of
//   saved: a saved pair would hold 4 N F bytes per layer from the forward to
//   the backward and would be rounded to bf16.  dg and du are rounded to bf16
//   (the tensor core's operand type) once and live in the workspace only.
//   dx and dW share one launch (see "gradient units"), of 512-row tiles where
//   there are enough of them.
//
// EW + 2 warps per CTA: warps 0 to EW - 1 (4 or 8) epilogue (thread = TMEM lane
// of its warp's quarter; with 8 warps two share a quarter and halve its
// columns), one TMA producer, one TMEM allocator and (leader) MMA issuer.  Two
// accumulators of BN columns let a tile's epilogue overlap the next tile's
// products.  All waits are bounded.
//
// Measured (short runs, the same box; in brackets the bare cuBLAS product of
// the same operands): 32,760 x 1536 x 4096 bf16 forward 513 us, 1608 TFLOP/s
// (507), dg and du 575 us, gradients 1033 us (474 + 502); e4m3, 16,384 x 5120 x
// 13824: 1589 us, 2919 TFLOP/s (1464 with one scale for all, 1933 with row
// scales).  Bound by the tensor cores under the power cap and by the operand
// traffic from L2.
#include "common.cuh"
#include "tc_common.cuh"

namespace moga {
namespace ffn {

using namespace moga::tc;

enum Mode { MODE_FWD = 0, MODE_DGDU = 1, MODE_GRAD = 2 };

constexpr int BM = 128;                      // accumulator rows per CTA (256 per pair)
constexpr int kRowBytes = 128;               // bytes of one operand row in a stage (one swizzle span)
constexpr int kHalfBox = 64 * kRowBytes;     // 8 KB: a box of 64 rows
constexpr int kOutBox = 32 * kRowBytes;      // 4 KB: a warp's 32 rows x 64 bf16 columns of output

// Shared memory of a CTA: operand stages, then the epilogue's output boxes.
// Accumulators: HM = 1: 256 rows per pair, two buffers of BN columns;
// HM = 2: 512 rows, the two accumulators hold a CTA's two halves of 128 rows.
template <int BN, int HM, int BOXES = 8>
struct Tile {
  static constexpr int kABytes = HM * BM * kRowBytes;     // this CTA's rows of A
  static constexpr int kBBytes = BN / 2 * kRowBytes;      // this CTA's half of the B rows
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = HM == 2 ? 4 : BN == 128 ? 8 : BOXES > 8 ? 5 : 6;
  static constexpr int kOutOff = kStages * kStageBytes;   // output boxes of the epilogue warps
  static constexpr int kBarOff = kOutOff + BOXES * kOutBox;
  static constexpr int kMiscOff = kBarOff + 32 * 8;
  static constexpr int kSmemBytes = kMiscOff + 64 + 1024;
  static constexpr int kFull = 0, kEmpty = kStages, kAccFull = 2 * kStages, kAccEmpty = kAccFull + 2,
                       kEnd = kAccEmpty + 2;
  static_assert(kSmemBytes <= 227 * 1024 && kEnd < 32, "shared memory");
};

// dx or dW in the gradient launch
struct Kind {
  int units;                 // tiles x splits of K
  int k, unit_k;             // k stages of a tile, of a unit
  float* partial;            // fp32 sums [splits][rows][d] where K is split, else NULL
};

struct Params {
  int rows, cols;            // FWD, DGDU: N, F;  GRAD: N, d
  int n_k;                   // k stages of a forward tile
  int m_tiles, n_tiles;      // row tiles of N (256 HM rows), column tiles of F (FWD, DGDU) or d (GRAD)
  int high;                  // row tiles of a band (tile_of)
  int a_box;                 // FWD, DGDU: rows of a box of x
  int total;                 // FWD, DGDU: tiles
  int act;
  const float *xs, *gs, *us; // e4m3 scales
  const __nv_bfloat16* dh;   // DGDU
  // GRAD
  int F;
  int seg_k;                 // stages of the gate half of dx's K (F / 64 rounded up)
  int mf_tiles;              // row tiles of F
  Kind kind[2];              // dx, dW
  int first;                 // the kind whose units each pair takes first
  int hm;                    // 256-row halves of a tile (the kernel's HM)
  int n1, a, b;              // halves of units of the other kind for the first n1 pairs, for the others
  long long timeout;
};

// One piece of work of a pair: rows and columns of a tile, its k stages.
struct Unit {
  int kind;                  // 0: gated tile, 1: dx tile, 2: dW tile
  int m, n, k0, k1, split, up;
  int h0, h1;                // its halves (GRAD: [0, hm), or one of them)
};

// Tile t -> (row tile, column tile).  Tiles run down bands of `high` row tiles,
// so that the pairs at work at one time share a few row tiles and a few column
// tiles in L2 instead of sweeping all of W for every row tile.
__host__ __device__ __forceinline__ void tile_of(int t, int high, int m_tiles, int n_tiles, int* m, int* n) {
  const int band = high * n_tiles;
  const int b = t / band, r = t - b * band;
  const int gm = m_tiles - b * high < high ? m_tiles - b * high : high;
  *n = r / gm;
  *m = b * high + (r - *n * gm);
}

// Gradient units.  dW's tiles are 2 F / 256 x d / 256 with K = N, dx's N / 256
// x d / 256 with K = 2F: often few and long against many and short, and neither
// count fills the pairs' last round.  So both kinds share one launch, K is
// split where a tile would take longer than a pair's share of all the work
// (grad_shape), and the longer units go first: unit j P + pair of the first
// kind for each pair, then units of the other kind, of which the n1 pairs that
// hold one more of the first take fewer, about the length of one (plan_grad).
// 512-row tiles of the other kind are counted in halves, and a pair with an odd
// number ends on a single half: 32,760 x 1536 x 4096 takes 10.5 rounds of dx
// tiles instead of 11.
// The j-th unit of pair `pair` of `P`; false when it has no more.
template <int MODE>
__host__ __device__ __forceinline__ bool unit_of(const Params& p, int pair, int P, int j, Unit* u) {
  u->split = u->up = u->h0 = 0;
  u->h1 = MODE == MODE_GRAD ? p.hm : 1;
  if (MODE != MODE_GRAD) {
    const int t = j * P + pair;   // total < 2^30, P < 2^10: no overflow where the loop stops at the first false
    if (t >= p.total) return false;
    u->kind = 0;
    u->k0 = 0;
    u->k1 = p.n_k;
    tile_of(t, p.high, p.m_tiles, p.n_tiles, &u->m, &u->n);
    return true;
  }
  const int n_first = p.kind[p.first].units;
  const int mine = n_first / P + (pair < n_first % P ? 1 : 0);
  int which = p.first, t = j * P + pair;
  if (j >= mine) {
    which ^= 1;
    const int i = j - mine, halves = pair < p.n1 ? p.a : p.b;
    const int fa = p.a / p.hm, fb = p.b / p.hm;      // whole units of either group of pairs
    if (i < halves / p.hm) {
      t = i < fa || p.n1 == 0 ? i * P + pair : fa * P + (i - fa) * (P - p.n1) + pair - p.n1;
    } else {
      if (i > halves / p.hm || halves % p.hm == 0) return false;
      // the pair's last: one half, of the tiles that no pair takes whole
      const int rank = pair < p.n1 || p.a % 2 == 1 ? pair : pair - p.n1;
      const int h = 2 * (p.n1 * fa + (P - p.n1) * fb) + rank;
      t = h >> 1;
      u->h0 = h & 1;
      u->h1 = u->h0 + 1;
    }
    if (t >= p.kind[which].units) return false;
  }
  const Kind& kd = p.kind[which];
  const int mt = which == 0 ? p.m_tiles : 2 * p.mf_tiles, tiles = mt * p.n_tiles;
  u->kind = 1 + which;
  u->split = t / tiles;
  tile_of(t - u->split * tiles, p.high, mt, p.n_tiles, &u->m, &u->n);
  if (which == 1 && u->m >= p.mf_tiles) {
    u->up = 1;
    u->m -= p.mf_tiles;
  }
  u->k0 = u->split * kd.unit_k;
  u->k1 = u->k0 + kd.unit_k < kd.k ? u->k0 + kd.unit_k : kd.k;
  return true;
}

__device__ __forceinline__ void mma_pair_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0;"
      " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p; }" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// The backward's launches follow one another with programmatic dependent
// launch: the next one's CTAs are set up while the last of this one's finish,
// and wait for its memory where they first read it.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

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
    // g^2 is kept finite: far out the factor before it is 0
    *da = s + *a * (1.f - s) * (kGelu2 * (1.f + 0.134145f * fminf(g * g, 1e30f)));
  }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// ---- output boxes.  A thread owns a row, so its own 16-byte stores would
// touch 32 lines per warp instruction and half a sector each.  Instead a warp
// lays 32 rows x 64 columns of bf16 into shared memory (128-byte rows, the
// TMA's 128-byte swizzle: conflict-free for row-owning lanes) and one lane
// stores the box through the tensor map, which writes whole lines and clips
// rows and columns past the tensor's end.
__device__ __forceinline__ uint32_t box_addr(uint32_t box, int row, int piece) {
  return box + row * kRowBytes + ((piece ^ (row & 7)) << 4);
}
__device__ __forceinline__ void sts16(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
// 32 values of the lane's row into pieces [4 half, 4 half + 4) of a box
__device__ __forceinline__ void put32(uint32_t box, int lane, int half, const float* v) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    sts16(box_addr(box, lane, 4 * half + e),
          make_uint4(pack2(v[8 * e], v[8 * e + 1]), pack2(v[8 * e + 2], v[8 * e + 3]),
                     pack2(v[8 * e + 4], v[8 * e + 5]), pack2(v[8 * e + 6], v[8 * e + 7])));
}
// the warp's writes to the box become visible to the TMA, then one lane stores it
__device__ __forceinline__ void store_box(const CUtensorMap* map, uint32_t box, int col, int row, int lane) {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
  if (lane == 0) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(col), "r"(row), "r"(box)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
}
// the box of all but the last PENDING stores may be written again
template <int PENDING>
__device__ __forceinline__ void boxes_free(int lane) {
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(PENDING) : "memory");
  __syncwarp();
}

// A warp gives its accumulator back on the leader's barrier, once per tile:
// as soon as the last values are in registers, so that the next tile's products
// do not wait for this one's arithmetic and stores.
__device__ __forceinline__ void release_acc(uint32_t empty, int lane) {
  tc_fence_before();
  __syncwarp();
  if (lane == 0) asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(empty) : "memory");
}

// COLS columns of a gated tile from c_begin, for the warp's 32 rows from row0.
// `turn` counts the warp's stores: its BOXES boxes are filled in turn.
template <bool E4M3, int ACT, int BN, int COLS, int BOXES>
__device__ __forceinline__ void epilogue_fwd(const Params& p, const CUtensorMap* map, uint32_t acc, uint32_t boxes,
                                             int row0, int col0, int c_begin, int lane, int& turn, uint32_t empty) {
  const int row = row0 + lane;
  const float xs = E4M3 && row < p.rows ? __ldg(p.xs + row) : 1.f;
#pragma unroll 1
  for (int c0 = c_begin; c0 < c_begin + COLS; c0 += 64) {
    const int col = col0 + c0;
    if (col >= p.cols || row0 >= p.rows) {   // the whole warp
      release_acc(empty, lane);
      break;
    }
    const uint32_t box = boxes + (turn++ % BOXES) * kOutBox;
    boxes_free<BOXES - 1>(lane);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float g[32], u[32];
      tmem_ld32(acc + c0 + 32 * h, g);
      tmem_ld32(acc + BN / 2 + c0 + 32 * h, u);
      tmem_wait_ld();
      if (h == 1 && c0 + 64 >= c_begin + COLS) release_acc(empty, lane);
      if (E4M3) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int cc = min(col + 32 * h + 4 * e, p.cols - 4);   // F is a multiple of 8
          const float4 a = __ldg(reinterpret_cast<const float4*>(p.gs + cc));
          const float4 b = __ldg(reinterpret_cast<const float4*>(p.us + cc));
          g[4 * e] *= xs * a.x; g[4 * e + 1] *= xs * a.y; g[4 * e + 2] *= xs * a.z; g[4 * e + 3] *= xs * a.w;
          u[4 * e] *= xs * b.x; u[4 * e + 1] *= xs * b.y; u[4 * e + 2] *= xs * b.z; u[4 * e + 3] *= xs * b.w;
        }
      }
#pragma unroll
      for (int j = 0; j < 32; ++j) g[j] = act_of<ACT>(g[j]) * u[j];
      put32(box, lane, h, g);
    }
    store_box(map, box, col, row0, lane);
  }
}

// The warp's 32 rows x 64 columns of dout, 8 lanes a row (whole lines).
__device__ __forceinline__ void load_dout(const Params& p, int row0, int col, int lane, uint4* v) {
  const int c = col + 8 * (lane & 7);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = row0 + 4 * i + (lane >> 3);
    v[i] = r < p.rows && c < p.cols ? __ldg(reinterpret_cast<const uint4*>(p.dh + (size_t)r * p.cols + c))
                                    : make_uint4(0, 0, 0, 0);
  }
}

// dg and du of COLS columns of a gated tile from c_begin.  v holds the dout of
// the first 64, loaded before the products were waited for; the next 64 are
// loaded while these are worked on.  Box 0 takes dout, then dg, box 1 du.
template <int ACT, int BN, int COLS>
__device__ __forceinline__ void epilogue_dgdu(const Params& p, const CUtensorMap* mg, const CUtensorMap* mu,
                                              uint32_t acc, uint32_t boxes, int row0, int col0, int c_begin, int lane,
                                              uint4* v, uint32_t empty) {
#pragma unroll 1
  for (int c0 = c_begin; c0 < c_begin + COLS; c0 += 64) {
    const int col = col0 + c0;
    if (col >= p.cols || row0 >= p.rows) {   // the whole warp
      release_acc(empty, lane);
      break;
    }
    boxes_free<0>(lane);
    // dout from lanes of columns to lanes of rows
#pragma unroll
    for (int i = 0; i < 8; ++i) sts16(box_addr(boxes, 4 * i + (lane >> 3), lane & 7), v[i]);
    __syncwarp();
    if (c0 + 64 < c_begin + COLS) load_dout(p, row0, col + 64, lane, v);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t w[16];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint4 t = lds16(box_addr(boxes, lane, 4 * h + e));
        w[4 * e] = t.x; w[4 * e + 1] = t.y; w[4 * e + 2] = t.z; w[4 * e + 3] = t.w;
      }
      float g[32], u[32];
      tmem_ld32(acc + c0 + 32 * h, g);
      tmem_ld32(acc + BN / 2 + c0 + 32 * h, u);
      tmem_wait_ld();
      if (h == 1 && c0 + 64 >= c_begin + COLS) release_acc(empty, lane);
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float d = __uint_as_float((j & 1) ? (w[j >> 1] & 0xffff0000u) : (w[j >> 1] << 16));
        float a, da;
        act_and_grad<ACT>(g[j], &a, &da);
        g[j] = d * u[j] * da;
        u[j] = d * a;
      }
      put32(boxes, lane, h, g);            // the lane's own row and half, read above
      put32(boxes + kOutBox, lane, h, u);
    }
    store_box(mg, boxes, col, row0, lane);
    store_box(mu, boxes + kOutBox, col, row0, lane);
  }
}

// Columns [c_begin, c_begin + COLS) of a gradient tile for the warp's 32 rows:
// bf16 through the box, or the fp32 partial sum where K is split.
template <int BN, int COLS>
__device__ __forceinline__ void epilogue_grad(const Params& p, const CUtensorMap* map, const Unit& u, uint32_t acc,
                                              uint32_t box, int row0, int c_begin, int lane, uint32_t empty) {
  const int rows = u.kind == 1 ? p.rows : p.F;
  float* const partial = p.kind[u.kind - 1].partial;
  const bool split = partial != nullptr;
#pragma unroll 1
  for (int c0 = c_begin; c0 < c_begin + COLS; c0 += 64) {
    const int col = u.n * BN + c0;
    if (col >= p.cols || row0 >= rows) {   // the whole warp
      release_acc(empty, lane);
      break;
    }
    if (!split) boxes_free<0>(lane);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[32];
      tmem_ld32(acc + c0 + 32 * h, v);
      tmem_wait_ld();
      if (h == 1 && c0 + 64 >= c_begin + COLS) release_acc(empty, lane);
      if (!split) {
        put32(box, lane, h, v);
      } else if (row0 + lane < rows) {
        const size_t slab = u.kind == 1 ? u.split : u.split * 2 + u.up;
        float* dst = partial + (slab * rows + row0 + lane) * p.cols + col + 32 * h;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (col + 32 * h + 4 * e < p.cols)
            *reinterpret_cast<float4*>(dst + 4 * e) = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
      }
      __syncwarp();
    }
    if (!split) store_box(map, box, col, row0, lane);
  }
}

// Tensor maps.  Loads: FWD, DGDU: 0 x (a_box-row boxes), 1 w_gate, 2 w_up
// (BN / 2-row boxes); GRAD: 0 x, 1 w_gate, 2 w_up, 3 dg, 4 du (64 x 64 boxes).
// Stores (32-row boxes): FWD: out; DGDU: dg, du; GRAD: dx, dw_gate, dw_up.
struct Maps {
  CUtensorMap m[5], out[3];
};

// output boxes of a CTA: two per warp for dg and du, else eight to share
__host__ __device__ constexpr int boxes_of(int mode, int ew) { return mode == MODE_DGDU ? 2 * ew : 8; }

template <int MODE, bool E4M3, int ACT, int BN, int HM, int EW>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__((EW + 2) * 32, 1)
ffn_kernel(const __grid_constant__ Params p, const __grid_constant__ Maps maps) {
  constexpr int kBoxes = boxes_of(MODE, EW);
  using T = Tile<BN, HM, kBoxes>;
  constexpr int BK = E4M3 ? 128 : 64;
  // instruction descriptors of a pair's M = 256 product
  constexpr uint32_t kIdesc = pair_desc(instr_desc(BN, false));
  constexpr uint32_t kIdescBMn = pair_desc(instr_desc(BN, true));
  constexpr uint32_t kIdescABMn = kIdescBMn | (1u << 15);
  constexpr uint32_t kIdescE4m3 = kIdesc & ~((7u << 7) | (7u << 10));   // e4m3 x e4m3 (format 0)
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + T::kBarOff + 8u * (uint32_t)i; };
  int* misc = reinterpret_cast<int*>(smem + T::kMiscOff);
  volatile int* abort_flag = misc;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();          // 0: leader, 1: peer
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;
  if (MODE != MODE_FWD) let_next_start();

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int s = 0; s < T::kStages; ++s) {
      mbar_init(bar(T::kFull + s), 1);
      mbar_init(bar(T::kEmpty + s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar(T::kAccFull + b), 1);
      mbar_init(bar(T::kAccEmpty + b), 2 * EW);   // a warp's arrival stands for its lanes
    }
    mbar_init(bar(T::kEnd), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == EW + 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(2u * BN)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // both CTAs' barriers are initialised before any remote use
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == EW) {
    // ------------------------------------------------------------------ producer
    if (lane == 0) {
      if (MODE == MODE_GRAD) wait_for_previous();   // dg and du
      int c = 0;
      bool ok = true;
      Unit u;
      for (int j = 0; ok && unit_of<MODE>(p, pair, n_pairs, j, &u); ++j) {
        for (int kt = u.k0; kt < u.k1; ++kt, ++c) {
          const int st = c % T::kStages;
          if (!(ok = mbar_wait(bar(T::kEmpty + st), ((c / T::kStages) & 1) ^ 1, abort_flag, p.timeout))) break;
          const uint32_t full = peer_addr(bar(T::kFull + st), 0);
          // Rows of A past the last token are left unloaded (their products
          // reach no output): the peer's tile where it has no row, and all
          // but a_box rows of the leader's where there are fewer tokens.
          const bool peer_a = MODE == MODE_GRAD || (u.m * 2 + 1) * BM < p.rows;
          // the leader's barrier expects both CTAs' bytes
          if (leader) {
            const int a_bytes = MODE == MODE_GRAD ? 2 * (u.h1 - u.h0) * BM * kRowBytes
                                                  : (peer_a ? 2 : 1) * p.a_box * kRowBytes;
            mbar_arrive_expect_tx(bar(T::kFull + st), a_bytes + 2 * T::kBBytes);
          }
          const uint32_t a = sbase + st * T::kStageBytes, b = a + T::kABytes;
          if (MODE != MODE_GRAD) {
            if (leader || peer_a) tma_load_2d_pair(a, &maps.m[0], kt * BK, (u.m * 2 + (int)rank) * BM, full);
            tma_load_2d_pair(b, leader ? &maps.m[1] : &maps.m[2], kt * BK, u.n * (BN / 2), full);
          } else {
            // this CTA's rows of A, and its half of the tile's columns, in boxes of 64
            const int r0 = (u.m * 2 + (int)rank) * HM * BM, c0 = u.n * BN + (int)rank * (BN / 2);
            if (u.kind == 1) {
              const bool up = kt >= p.seg_k;
              const int k0 = (up ? kt - p.seg_k : kt) * BK;
              const CUtensorMap *ma = up ? &maps.m[4] : &maps.m[3], *mb = up ? &maps.m[2] : &maps.m[1];
              for (int i = 2 * u.h0; i < 2 * u.h1; ++i) tma_load_2d_pair(a + i * kHalfBox, ma, k0, r0 + 64 * i, full);
              tma_load_2d_pair(b, mb, c0, k0, full);
              tma_load_2d_pair(b + kHalfBox, mb, c0 + 64, k0, full);
            } else {
              const CUtensorMap* ma = u.up ? &maps.m[4] : &maps.m[3];
              for (int i = 2 * u.h0; i < 2 * u.h1; ++i)
                tma_load_2d_pair(a + i * kHalfBox, ma, r0 + 64 * i, kt * BK, full);
              tma_load_2d_pair(b, &maps.m[0], c0, kt * BK, full);
              tma_load_2d_pair(b + kHalfBox, &maps.m[0], c0 + 64, kt * BK, full);
            }
          }
        }
      }
      // A wait that ran out: the copies that nothing will wait for (both CTAs'
      // arrive on the leader's barriers) land before the CTAs leave.
      if (!ok && leader)
        for (int i = c > T::kStages ? c - T::kStages : 0; i < c; ++i)
          mbar_drain(bar(T::kFull + i % T::kStages), (i / T::kStages) & 1, p.timeout);
    }
    __syncwarp();
  } else if (warp == EW + 1) {
    // ------------------------------------------------------------------ MMA issuer (leader)
    if (leader && lane == 0) {
      int c = 0;   // stage counter
      bool ok = true;
      Unit u;
      for (int j = 0; ok && unit_of<MODE>(p, pair, n_pairs, j, &u); ++j) {
        // HM = 1: tile j's buffer j & 1; HM = 2: both, taken one after the other
        const int b = HM == 1 ? j & 1 : 0;
        const uint32_t empty_parity = (HM == 1 ? (j >> 1) & 1 : j & 1) ^ 1;
        if (!(ok = mbar_wait(bar(T::kAccEmpty + b), empty_parity, abort_flag, p.timeout))) break;
        tc_fence_after();
        for (int kt = u.k0; kt < u.k1; ++kt, ++c) {
          const int st = c % T::kStages;
          if (!(ok = mbar_wait(bar(T::kFull + st), (c / T::kStages) & 1, abort_flag, p.timeout))) break;
          tc_fence_after();
          const uint32_t sb = sbase + st * T::kStageBytes + T::kABytes;
#pragma unroll
          for (int h = 0; h < HM; ++h) {
            if (HM == 2 && (h < u.h0 || h >= u.h1)) continue;
            if (h == 1 && kt == u.k0) {
              if (!(ok = mbar_wait(bar(T::kAccEmpty + 1), empty_parity, abort_flag, p.timeout))) break;
              tc_fence_after();
            }
            const uint32_t acc = tmem + (HM == 1 ? b : h) * BN;
            const uint32_t sa = sbase + st * T::kStageBytes + h * BM * kRowBytes;
            // K-major operands advance 32 bytes along their rows; MN-major ones
            // 16 k rows of 128 bytes (their 64-column boxes are kHalfBox apart)
            if (MODE != MODE_GRAD) {
#pragma unroll
              for (int ks = 0; ks < 4; ++ks) {
                const uint64_t ad = smem_desc(sa + ks * 32, 16, 1024), bd = smem_desc(sb + ks * 32, 16, 1024);
                const uint32_t accum = (kt > u.k0 || ks > 0) ? 1u : 0u;
                if (E4M3) mma_pair_f8(acc, ad, bd, kIdescE4m3, accum);
                else mma_pair(acc, ad, bd, kIdesc, accum);
              }
            } else if (u.kind == 1) {
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                mma_pair(acc, smem_desc(sa + ks * 32, 16, 1024), smem_desc(sb + ks * 2048, kHalfBox, 1024), kIdescBMn,
                         (kt > u.k0 || ks > 0) ? 1u : 0u);
            } else {
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                mma_pair(acc, smem_desc(sa + ks * 2048, kHalfBox, 1024), smem_desc(sb + ks * 2048, kHalfBox, 1024),
                         kIdescABMn, (kt > u.k0 || ks > 0) ? 1u : 0u);
            }
          }
          if (!ok) break;
          commit_pair(bar(T::kEmpty + st));
        }
        if (!ok) break;
        commit_pair(bar(T::kAccFull + b));
      }
      commit_pair(bar(T::kEnd));
      mbar_drain(bar(T::kEnd), 0, p.timeout);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ epilogue
    const int quarter = warp & 3, half = warp >> 2;
    const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
    const uint32_t boxes = sbase + T::kOutOff + warp * (kBoxes / EW) * kOutBox;   // this warp's boxes
    int turn = 0;
    Unit u;
    for (int j = 0; unit_of<MODE>(p, pair, n_pairs, j, &u); ++j) {
      const int b = HM == 1 ? j & 1 : 0;
      const uint32_t parity = HM == 1 ? (j >> 1) & 1 : j & 1;
      const int row0 = (u.m * 2 + (int)rank) * HM * BM + quarter * 32;
      uint4 v[MODE == MODE_DGDU ? 8 : 1];
      if (MODE == MODE_DGDU) load_dout(p, row0, u.n * (BN / 2) + half * (BN * 2 / EW), lane, v);
      if (!__all_sync(0xffffffffu, mbar_wait(bar(T::kAccFull + b), parity, abort_flag, p.timeout))) break;
      tc_fence_after();
#pragma unroll 1
      for (int h = 0; h < HM; ++h) {
        if (HM == 2 && (h < u.h0 || h >= u.h1)) continue;   // a single half is its pair's last unit
        const uint32_t acc = tmem + lane_addr + (HM == 1 ? b : h) * BN;
        const uint32_t empty = peer_addr(bar(T::kAccEmpty + (HM == 1 ? b : h)), 0);
        if constexpr (MODE == MODE_FWD)
          epilogue_fwd<E4M3, ACT, BN, BN * 2 / EW, 8 / EW>(p, &maps.out[0], acc, boxes, row0, u.n * (BN / 2),
                                                           half * (BN * 2 / EW), lane, turn, empty);
        else if constexpr (MODE == MODE_DGDU)
          epilogue_dgdu<ACT, BN, BN * 2 / EW>(p, &maps.out[0], &maps.out[1], acc, boxes, row0, u.n * (BN / 2),
                                              half * (BN * 2 / EW), lane, v, empty);
        else
          epilogue_grad<BN, BN * 4 / EW>(p, &maps.out[u.kind == 1 ? 0 : 1 + u.up], u, acc, boxes, row0 + h * BM,
                                         half * (BN * 4 / EW), lane, empty);
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
  }

  // every product of the pair has completed (the leader drained them) and no
  // remote arrival is pending before either CTA frees its TMEM and exits
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  if (warp == EW + 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2u * BN) : "memory");
}

// bf16 of the sum of the K splits' partial sums, in split order.  dx is N d / 8
// groups of 8 values, dW_gate and dW_up F d / 8 each; a kind without partial
// sums has no groups here.
struct SumParams {
  const float *px, *pw;
  int sx, sw;
  int64_t nx, nw;            // groups of dx, of one dW
  uint4 *dx, *dwg, *dwu;
};
__global__ void __launch_bounds__(256) ffn_sum_kernel(const SumParams p) {
  wait_for_previous();
  int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const bool w = i >= p.nx;
  if (w) i -= p.nx;
  const int64_t n = w ? 2 * p.nw : p.nx;
  if (i >= n) return;
  const float4* q = reinterpret_cast<const float4*>(w ? p.pw : p.px) + 2 * i;
  const int splits = w ? p.sw : p.sx;
  float v[8] = {};
  for (int s = 0; s < splits; ++s, q += 2 * n) {
    const float4 x = __ldcs(q), y = __ldcs(q + 1);
    v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
    v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
  }
  (w ? i < p.nw ? p.dwg + i : p.dwu + (i - p.nw) : p.dx + i)[0] =
      make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}

// ---------------------------------------------------------------- few tokens
//
// For few tokens the weights' read is the time (2 F d elements for N d + N F
// others), a 256-row tile would idle, and a tile's k stages follow one another
// at 300 ns each however narrow it is.  Here a CTA takes 8 columns of F and
// all tokens; its W warps split d, each streaming 64-byte pieces of 16 weight
// rows straight from global memory into mma.sync fragments: the 16-row A tile
// is 8 gate rows over the 8 up rows of the same columns, so a lane's
// accumulators hold gate and up of the same outputs.  A lane loads 16
// consecutive bytes of a row where the fragment wants four pieces spread over
// k; the sum over k does not mind the order as long as x is read in the same
// one.  No shared-memory stage, no barrier in the loop: a lane keeps 2 UN
// 16-byte loads of weights under way, and many small CTAs per SM do the rest
// (up to 8 tokens UN = 4, W = 8 in bf16, UN = 8, W = 4 in e4m3; twice the
// unrolling measured 47 instead of 43.5 us, half the warps 46; one block per
// SM as the launch bound lets the loads of a pass stay in registers, 45.8
// against 50 us).  The warps' sums meet in shared memory in a fixed order.
// One token through 5120 x 13824: 43.4 us, the weights at 6.5 TB/s.

// Up to 16 tokens this kernel is always the faster (16 tokens, 5120 x 13824:
// 52 against 64 us; 1536 x 4096: 8.3 against 13.1).  Above, every CTA's read of
// x costs as much as its weights, so it pays while the CTAs are few: 32 tokens
// up to three per SM (5120 x 2048: 19 against 30 us, 1536 x 4096: 14.2 against
// 13.2), 64 tokens up to one (2048 x 1024: 8.5 against 14.9, 2048 x 2048: 15.8
// against 15.3).
inline bool few_tokens(int64_t N, int F, int sms) {
  return N <= 16 || (N <= 32 && F / 8 <= 3 * sms) || (N <= 64 && F / 8 <= sms);
}

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

template <bool E4M3, int ACT, int NT, int UN, int W>
__global__ void __launch_bounds__(32 * W, 1) ffn_few_kernel(const FewParams p) {
  __shared__ float red[W][4 * NT][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int f0 = blockIdx.x * 8;                      // F is a multiple of 8: all rows exist
  const uint8_t* wg = p.wg + (size_t)(f0 + g) * p.row_bytes + 16 * q;
  const uint8_t* wu = p.wu + (size_t)(f0 + g) * p.row_bytes + 16 * q;
  bool xon[NT];
  const uint8_t* xp[NT];
  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    xon[n] = 8 * n + g < p.N;
    xp[n] = p.x + (size_t)(xon[n] ? 8 * n + g : 0) * p.row_bytes + 16 * q;
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
  }
  const uint4 zero = make_uint4(0, 0, 0, 0);
  // step s covers bytes [64 s, 64 s + 64) of every row; warp w takes s = w, w + W, ...
  for (int s0 = warp; 64 * s0 < p.row_bytes; s0 += W * UN) {
    uint4 a[UN], b[UN], x[UN][NT];
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      const int k = 64 * (s0 + W * i);
      const bool on = k + 16 * q < p.row_bytes;
      a[i] = on ? ldg_stream(wg + k) : zero;
      b[i] = on ? ldg_stream(wu + k) : zero;
    }
#pragma unroll
    for (int i = 0; i < UN; ++i) {
      const int k = 64 * (s0 + W * i);
#pragma unroll
      for (int n = 0; n < NT; ++n)
        x[i][n] = xon[n] && k + 16 * q < p.row_bytes ? __ldg(reinterpret_cast<const uint4*>(xp[n] + k)) : zero;
    }
#pragma unroll
    for (int i = 0; i < UN; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma_16x8<E4M3>(acc[n], a[i].x, b[i].x, a[i].y, b[i].y, x[i][n].x, x[i][n].y);
        mma_16x8<E4M3>(acc[n], a[i].z, b[i].z, a[i].w, b[i].w, x[i][n].z, x[i][n].w);
      }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[warp][4 * n + i][lane] = acc[n][i];
  __syncthreads();
  // column c, token t: lane 4 c + (t % 8) / 2, slot 4 (t / 8) + t % 2 (gate), 2 more (up)
  for (int o = threadIdx.x; o < 8 * p.N; o += 32 * W) {
    const int c = o & 7, t = o >> 3, l = 4 * c + ((t & 7) >> 1), slot = 4 * (t >> 3) + (t & 1);
    float gate = 0.f, up = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      gate += red[w][slot][l];
      up += red[w][slot + 2][l];
    }
    if (E4M3) {
      const float xs = __ldg(p.xs + t);
      gate *= xs * __ldg(p.gs + f0 + c);
      up *= xs * __ldg(p.us + f0 + c);
    }
    p.out[(size_t)t * p.F + f0 + c] = __float2bfloat16_rn(act_of<ACT>(gate) * up);
  }
}

template <bool E4M3, int ACT>
static moga_status launch_few(const FewParams& p, const char* who, cudaStream_t s) {
  constexpr int UN = E4M3 ? 8 : 4, W = E4M3 ? 4 : 8;
  const int grid = p.F / 8;
  if (p.N <= 8) ffn_few_kernel<E4M3, ACT, 1, UN, W><<<grid, 32 * W, 0, s>>>(p);
  else if (p.N <= 16) ffn_few_kernel<E4M3, ACT, 2, 4, 8><<<grid, 256, 0, s>>>(p);
  else if (p.N <= 32) ffn_few_kernel<E4M3, ACT, 4, 2, 8><<<grid, 256, 0, s>>>(p);
  else ffn_few_kernel<E4M3, ACT, 8, 1, 8><<<grid, 256, 0, s>>>(p);
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

// a launch that may be set up before the one in front of it on the stream ends
template <class... Params_, class... Args>
static moga_status launch_next(void (*k)(Params_...), unsigned grid, int threads, int smem, cudaStream_t s,
                               const char* who, const Args&... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k, args...);
  if (e != cudaSuccess) return fail(MOGA_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
  return check_launch(who);
}

template <int MODE, bool E4M3, int ACT, int BN, int HM, int EW>
static moga_status launch(const Params& p, const Maps& maps, int pairs, const char* who, cudaStream_t s) {
  auto* k = ffn_kernel<MODE, E4M3, ACT, BN, HM, EW>;
  constexpr int smem = Tile<BN, HM, boxes_of(MODE, EW)>::kSmemBytes;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return fail(MOGA_ERR_CUDA, "%s: cudaFuncSetAttribute: %s", who, cudaGetErrorString(e));
  if (MODE == MODE_GRAD) return launch_next(k, 2 * pairs, (EW + 2) * 32, smem, s, who, p, maps);
  k<<<2 * pairs, (EW + 2) * 32, smem, s>>>(p, maps);
  return check_launch(who);
}

inline int64_t ceil64(int64_t a, int64_t b) { return (a + b - 1) / b; }

// one pair of CTAs per pair of SMs (persistent)
inline int pair_count(int sms) { return sms / 2 > 0 ? sms / 2 : 1; }

// tile counts stay below 2^30
inline bool sizes_ok(int64_t N, int64_t d, int64_t F) {
  return d <= (1 << 20) && F <= (1 << 20) && ceil64(N, 256) * ceil64(std::max(d, F), 64) <= INT32_MAX / 2;
}

static moga_status check_dims(const char* who, int64_t N, int32_t d, int32_t F, int32_t act, int elem) {
  const int m = 16 / elem;   // 16-byte rows, as the TMA copies need them
  if (N <= 0 || N > INT32_MAX / 2) return fail(MOGA_ERR_INVALID_ARG, "%s: N=%lld out of range", who, (long long)N);
  if (d <= 0 || d % m != 0)
    return fail(MOGA_ERR_INVALID_ARG, "%s: d=%d must be a positive multiple of %d", who, d, m);
  if (F <= 0 || F % 8 != 0) return fail(MOGA_ERR_INVALID_ARG, "%s: F=%d must be a positive multiple of 8", who, F);
  if (!sizes_ok(N, d, F)) return fail(MOGA_ERR_INVALID_ARG, "%s: sizes out of range", who);
  if (act != MOGA_ACT_SILU && act != MOGA_ACT_GELU)
    return fail(MOGA_ERR_INVALID_ARG, "%s: activation %d unknown", who, act);
  return MOGA_OK;
}

// Row tiles of a forward band.  The weights are read once per band: where both
// do not stay in L2's near half (64 MB), higher bands read them less often
// (16,380 x 5120 x 13824 in e4m3: 1681 us with 8, 1637 with 16, 1632 with 32;
// 8190 tokens in bf16: 1539, 1516, 1622), else low ones keep x closer (32,760 x
// 1536 x 4096: 551, 557, 555).
inline int band_tiles(int64_t d, int64_t F, int elem) { return 2 * F * d * elem > (64 << 20) ? 16 : 8; }

// The gated product over all tokens with tiles of BN accumulator columns.
template <int MODE, bool E4M3, int BN>
static moga_status launch_gated_bn(Params p, const void* x, const void* wg, const void* wu, int d, void* o0, void* o1,
                                   int sms, const char* who, cudaStream_t s) {
  constexpr int elem = E4M3 ? 1 : 2;
  Maps maps;
  moga_status st;
  p.a_box = std::min(BM, ceil_div(p.rows, 32) * 32);
  if ((st = make_map(&maps.m[0], x, p.rows, d, elem, p.a_box)) != MOGA_OK) return st;
  if ((st = make_map(&maps.m[1], wg, p.cols, d, elem, BN / 2)) != MOGA_OK) return st;
  if ((st = make_map(&maps.m[2], wu, p.cols, d, elem, BN / 2)) != MOGA_OK) return st;
  maps.m[3] = maps.m[4] = maps.m[0];
  if ((st = make_map(&maps.out[0], o0, p.rows, p.cols, 2, 32)) != MOGA_OK) return st;
  maps.out[1] = maps.out[2] = maps.out[0];
  if (MODE == MODE_DGDU && (st = make_map(&maps.out[1], o1, p.rows, p.cols, 2, 32)) != MOGA_OK) return st;
  p.n_k = ceil_div(d, kRowBytes / elem);
  p.m_tiles = ceil_div(p.rows, 2 * BM);
  p.n_tiles = ceil_div(p.cols, BN / 2);
  p.total = p.m_tiles * p.n_tiles;
  p.high = band_tiles(d, p.cols, elem);
  const int pairs = std::min(p.total, pair_count(sms));
  // Epilogue warps: eight, one for each 64 columns of the tile's rows.  For dg
  // and du, whose 16 boxes then cost an operand stage, only where the epilogue
  // is longer than the products (16,384 tokens, F = 1024: d = 512 40.6 against
  // 41.6 us with four, d = 768 52.3 against 46.9).
  if (BN == 256 && (MODE == MODE_FWD || p.n_k <= 8))
    return p.act == MOGA_ACT_SILU ? launch<MODE, E4M3, MOGA_ACT_SILU, BN, 1, BN / 32>(p, maps, pairs, who, s)
                                  : launch<MODE, E4M3, MOGA_ACT_GELU, BN, 1, BN / 32>(p, maps, pairs, who, s);
  constexpr int EW = 4;
  return p.act == MOGA_ACT_SILU ? launch<MODE, E4M3, MOGA_ACT_SILU, BN, 1, EW>(p, maps, pairs, who, s)
                                : launch<MODE, E4M3, MOGA_ACT_GELU, BN, 1, EW>(p, maps, pairs, who, s);
}

// Accumulator columns of a gated tile for the given sizes: 128 where that
// saves rounds.  A stage takes about as long as 600 + BN of the same unit (391
// and 333 ns at BN = 256 and 128 with few tokens: most of it does not depend
// on the width), so the narrow tile pays only where it fills idle pairs (256
// tokens, 1536 x 4096: 14.2 against 16.5 us; 5120 x 13824, whose 108 wide tiles
// fill most of two rounds: 83 against 67 us).
inline int pick_bn(int64_t N, int F, int sms) {
  const int64_t mt = ceil64(N, 2 * BM);
  const int P = pair_count(sms);
  return ceil64(mt * ceil64(F, 64), P) * (600 + 128) < ceil64(mt * ceil64(F, 128), P) * (600 + 256) ? 128 : 256;
}

// The gated product; o1 is DGDU's second output (FWD: o0 again).
template <int MODE, bool E4M3>
static moga_status launch_gated(const Params& p, const void* x, const void* wg, const void* wu, int d, void* o0,
                                void* o1, const char* who, cudaStream_t s) {
  const int sms = route_tc::sm_count();
  return pick_bn(p.rows, p.cols, sms) == 256 ? launch_gated_bn<MODE, E4M3, 256>(p, x, wg, wu, d, o0, o1, sms, who, s)
                                             : launch_gated_bn<MODE, E4M3, 128>(p, x, wg, wu, d, o0, o1, sms, who, s);
}

constexpr int kGradBN = 256;

// Tiles, units and splits of the gradient launch.  Depends on the sizes and
// the SM count alone, not on the gradients asked for, so that the workspace
// does too.
struct GradShape {
  // 512-row tiles (2) read a quarter less operand bytes per product, 256-row
  // ones (1) are twice as many: 512 where one and a half units per pair are
  // left (4096 x 1536 x 4096, 1.9 units: 157 against 164 us; 2048 x 1024 x 2048,
  // 0.6 units: 72 against 44).
  int hm;
  int m_tiles, mf_tiles, n_tiles;
  int tiles[2], k[2], unit_k[2], splits[2];   // dx, dW
};
inline GradShape grad_shape(int64_t N, int d, int F, int sms) {
  GradShape g;
  const int64_t P = pair_count(sms), nt = ceil64(d, kGradBN);
  g.hm = 2 * nt * (ceil64(N, 4 * BM) + 2 * ceil64(F, 4 * BM)) >= 3 * P ? 2 : 1;
  const int rows = 2 * g.hm * BM;
  g.m_tiles = (int)ceil64(N, rows);
  g.mf_tiles = ceil_div(F, rows);
  g.n_tiles = (int)nt;
  g.tiles[0] = g.m_tiles * g.n_tiles;
  g.tiles[1] = 2 * g.mf_tiles * g.n_tiles;
  g.k[0] = 2 * ceil_div(F, 64);
  g.k[1] = (int)ceil64(N, 64);
  // Stages of a pair's share, but 12 at least: below, the partial sums cost more
  // than the split saves (510 x 720 x 280, units of 10 and 8: 17.7 whole, 22.3 us
  // split; 5000 x 64 x 64, 79 stages of dW: 14.9 in units of 8, 16.6 of 16, 20.0
  // of 32).
  const int64_t share = ceil64((int64_t)g.tiles[0] * g.k[0] + (int64_t)g.tiles[1] * g.k[1], P);
  const int least = (int)std::max<int64_t>(12, share);
  for (int i = 0; i < 2; ++i) {
    g.unit_k[i] = ceil_div(g.k[i], ceil_div(g.k[i], least));
    g.splits[i] = ceil_div(g.k[i], g.unit_k[i]);
  }
  return g;
}
inline size_t round256(size_t n) { return (n + 255) / 256 * 256; }
inline size_t dgdu_bytes(int64_t N, int F) { return round256((size_t)2 * N * F * 2); }
inline size_t dx_partial_bytes(const GradShape& g, int64_t N, int d) {
  return g.splits[0] > 1 ? round256((size_t)g.splits[0] * N * d * sizeof(float)) : 0;
}
inline size_t grad_ws_bytes(const GradShape& g, int64_t N, int d, int F) {
  return dgdu_bytes(N, F) + dx_partial_bytes(g, N, d) +
         (g.splits[1] > 1 ? (size_t)g.splits[1] * 2 * F * d * sizeof(float) : 0);
}

// The gradient units' shares (see unit_of).  Returns the number of pairs.
inline int plan_grad(Params& p, const GradShape& g, int64_t N, int d, int F, bool need_dx, bool need_dw, int sms) {
  p.rows = (int)N;
  p.cols = d;
  p.F = F;
  p.m_tiles = g.m_tiles;
  p.mf_tiles = g.mf_tiles;
  p.n_tiles = g.n_tiles;
  p.seg_k = g.k[0] / 2;
  for (int i = 0; i < 2; ++i) {
    p.kind[i].units = (i == 0 ? need_dx : need_dw) ? g.tiles[i] * g.splits[i] : 0;
    p.kind[i].k = g.k[i];
    p.kind[i].unit_k = g.unit_k[i];
  }
  p.first = g.unit_k[1] >= g.unit_k[0] ? 1 : 0;
  const Kind &one = p.kind[p.first], &two = p.kind[p.first ^ 1];
  const int P = (int)std::min<int64_t>((int64_t)one.units + two.units, pair_count(sms));
  p.n1 = one.units % P;
  p.hm = g.hm;
  p.high = 8 / g.hm;   // 2048 rows a band (512-row tiles, 32,760 x 1536 x 4096: 1078 us with 4, 1097 with 8)
  const int lag = ceil_div(g.hm * one.unit_k, two.unit_k);   // halves of the second kind in the time of one of the first
  const int64_t all = (int64_t)g.hm * two.units;
  auto holds = [&](int64_t b) { return p.n1 * std::max<int64_t>(0, b - lag) + (P - p.n1) * b >= all; };
  int64_t lo = 0, hi = all;
  while (lo < hi) {
    const int64_t mid = lo + (hi - lo) / 2;
    if (holds(mid)) hi = mid;
    else lo = mid + 1;
  }
  p.b = (int)lo;
  p.a = p.n1 ? std::max(0, p.b - lag) : p.b;
  return P;
}

}  // namespace ffn
}  // namespace moga

extern "C" moga_status moga_gated_ffn(const void* x, const void* w_gate, const void* w_up, moga_dtype dt,
                                      const float* x_scale, const float* w_gate_scale, const float* w_up_scale,
                                      int64_t N, int32_t d, int32_t F, int32_t act, void* out, void* stream) {
  using namespace moga;
  using namespace moga::ffn;
  const char* who = "moga_gated_ffn";
  if (dt != MOGA_BF16 && dt != MOGA_E4M3) return fail(MOGA_ERR_INVALID_ARG, "%s: dtype must be bf16 or e4m3", who);
  const bool f8 = dt == MOGA_E4M3;
  const int elem = f8 ? 1 : 2;
  moga_status st = check_dims(who, N, d, F, act, elem);
  if (st != MOGA_OK) return st;
  if (!x || !w_gate || !w_up || !out) return fail(MOGA_ERR_INVALID_ARG, "%s: null pointer", who);
  if (f8 != (x_scale != nullptr) || f8 != (w_gate_scale != nullptr) || f8 != (w_up_scale != nullptr))
    return fail(MOGA_ERR_INVALID_ARG, "%s: the three scales go with e4m3 operands", who);
  const uintptr_t a = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(w_gate) |
                      reinterpret_cast<uintptr_t>(w_up) | reinterpret_cast<uintptr_t>(out);
  const uintptr_t ws = reinterpret_cast<uintptr_t>(w_gate_scale) | reinterpret_cast<uintptr_t>(w_up_scale);
  if (((a | ws) & 15) || (reinterpret_cast<uintptr_t>(x_scale) & 3))
    return fail(MOGA_ERR_INVALID_ARG, "%s: x, w_gate, w_up, their scales and out must be 16-byte aligned", who);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (few_tokens(N, F, route_tc::sm_count())) {
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
  ffn::Params p = {};
  p.rows = (int)N;
  p.cols = F;
  p.act = act;
  p.xs = x_scale;
  p.gs = w_gate_scale;
  p.us = w_up_scale;
  p.timeout = kWaitLimitCycles;
  return f8 ? launch_gated<MODE_FWD, true>(p, x, w_gate, w_up, d, out, out, who, s)
            : launch_gated<MODE_FWD, false>(p, x, w_gate, w_up, d, out, out, who, s);
}

extern "C" size_t moga_gated_ffn_bwd_ws_bytes(int64_t N, int32_t d, int32_t F) {
  using namespace moga;
  if (N <= 0 || N > INT32_MAX / 2 || d <= 0 || d % 8 != 0 || F <= 0 || F % 8 != 0 || !ffn::sizes_ok(N, d, F)) return 0;
  return ffn::grad_ws_bytes(ffn::grad_shape(N, d, F, route_tc::sm_count()), N, d, F);
}

extern "C" moga_status moga_gated_ffn_bwd(const void* x, const void* w_gate, const void* w_up, int64_t N, int32_t d,
                                          int32_t F, int32_t act, const void* dout, void* dx, void* dw_gate,
                                          void* dw_up, void* ws, size_t ws_bytes, void* stream) {
  using namespace moga;
  using namespace moga::ffn;
  const char* who = "moga_gated_ffn_bwd";
  moga_status st = check_dims(who, N, d, F, act, 2);
  if (st != MOGA_OK) return st;
  if (!x || !w_gate || !w_up || !dout || !ws) return fail(MOGA_ERR_INVALID_ARG, "%s: null pointer", who);
  if ((dw_gate != nullptr) != (dw_up != nullptr))
    return fail(MOGA_ERR_INVALID_ARG, "%s: dw_gate and dw_up go together", who);
  if (!dx && !dw_gate) return fail(MOGA_ERR_INVALID_ARG, "%s: no gradient asked for", who);
  const uintptr_t al = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(w_gate) |
                       reinterpret_cast<uintptr_t>(w_up) | reinterpret_cast<uintptr_t>(dout) |
                       reinterpret_cast<uintptr_t>(dx) | reinterpret_cast<uintptr_t>(dw_gate) |
                       reinterpret_cast<uintptr_t>(dw_up) | reinterpret_cast<uintptr_t>(ws);
  if (al & 15) return fail(MOGA_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned", who);
  const int sms = route_tc::sm_count();
  const GradShape g = grad_shape(N, d, F, sms);
  const size_t need = grad_ws_bytes(g, N, d, F);
  if (ws_bytes < need) return fail(MOGA_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes", who, ws_bytes, need);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  __nv_bfloat16* dg = static_cast<__nv_bfloat16*>(ws);
  __nv_bfloat16* du = dg + (size_t)N * F;
  ffn::Params p = {};
  p.act = act;
  p.timeout = kWaitLimitCycles;
  p.rows = (int)N;
  p.cols = F;
  p.dh = static_cast<const __nv_bfloat16*>(dout);
  if ((st = launch_gated<MODE_DGDU, false>(p, x, w_gate, w_up, d, dg, du, who, s)) != MOGA_OK) return st;
  const int pairs = plan_grad(p, g, N, d, F, dx != nullptr, dw_gate != nullptr, sms);
  uint8_t* const part = static_cast<uint8_t*>(ws) + dgdu_bytes(N, F);
  if (g.splits[0] > 1) p.kind[0].partial = reinterpret_cast<float*>(part);
  if (g.splits[1] > 1) p.kind[1].partial = reinterpret_cast<float*>(part + dx_partial_bytes(g, N, d));
  ffn::Maps maps;
  const void* base[5] = {x, w_gate, w_up, dg, du};
  const int64_t rows[5] = {N, F, F, N, N}, cols[5] = {d, d, d, F, F};
  for (int i = 0; i < 5; ++i)
    if ((st = make_map(&maps.m[i], base[i], rows[i], cols[i], 2, 64)) != MOGA_OK) return st;
  // a gradient that is not asked for has no unit: its map is never used
  void* outs[3] = {dx ? dx : dw_gate, dw_gate ? dw_gate : dx, dw_up ? dw_up : dx};
  const int64_t out_rows[3] = {dx ? N : F, dw_gate ? F : N, dw_up ? F : N};
  for (int i = 0; i < 3; ++i)
    if ((st = make_map(&maps.out[i], outs[i], out_rows[i], d, 2, 32)) != MOGA_OK) return st;
  st = g.hm == 2 ? launch<MODE_GRAD, false, 0, kGradBN, 2, 8>(p, maps, pairs, who, s)
                 : launch<MODE_GRAD, false, 0, kGradBN, 1, 8>(p, maps, pairs, who, s);
  if (st != MOGA_OK) return st;
  SumParams q = {};
  if (dx && p.kind[0].partial) q.nx = N * d / 8;
  if (dw_gate && p.kind[1].partial) q.nw = (int64_t)F * d / 8;
  if (q.nx + q.nw == 0) return MOGA_OK;
  q.px = p.kind[0].partial;
  q.pw = p.kind[1].partial;
  q.sx = g.splits[0];
  q.sw = g.splits[1];
  q.dx = static_cast<uint4*>(dx);
  q.dwg = static_cast<uint4*>(dw_gate);
  q.dwu = static_cast<uint4*>(dw_up);
  return launch_next(ffn_sum_kernel, (unsigned)ceil64(q.nx + 2 * q.nw, 256), 256, 0, s, who, q);
}

// test hook (moga_testing.h): the units of every pair of one launch
extern "C" int64_t moga_test_ffn_units(int32_t grad, int64_t N, int32_t d, int32_t F, int32_t need_dx,
                                       int32_t need_dw, int32_t bn, int32_t sms, int32_t* out, int64_t cap) {
  using namespace moga;
  using namespace moga::ffn;
  ffn::Params p = {};
  int P;
  if (grad) {
    P = plan_grad(p, grad_shape(N, d, F, sms), N, d, F, need_dx != 0, need_dw != 0, sms);
  } else {
    p.n_k = ceil_div(d, 64);
    p.m_tiles = (int)ceil64(N, 2 * ffn::BM);
    p.n_tiles = ceil_div(F, bn / 2);
    p.total = p.m_tiles * p.n_tiles;
    p.high = band_tiles(d, F, 2);
    P = std::min(p.total, pair_count(sms));
  }
  int64_t n = 0;
  ffn::Unit u;
  for (int pair = 0; pair < P; ++pair)
    for (int j = 0; grad ? unit_of<MODE_GRAD>(p, pair, P, j, &u) : unit_of<MODE_FWD>(p, pair, P, j, &u); ++j, ++n)
      if (n < cap) {
        const int32_t v[10] = {pair, u.kind, u.up, u.m, u.n, u.split, u.k0, u.k1, u.h0, u.h1};
        for (int i = 0; i < 10; ++i) out[10 * n + i] = v[i];
      }
  return n;
}
