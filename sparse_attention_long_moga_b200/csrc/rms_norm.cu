// Root-mean-square norm with the residual's addition, and its backward.
//
// Forward, per row of d elements:
//   h = x + residual                (rounded to the stream's type and stored)
//   r = 1 / sqrt(mean(h^2) + eps),  y = h * r * w
// y is taken from the stored h, so that the backward, which reads only h,
// differentiates exactly what the forward computed.  The 8-bit output is
//   scale = max(max|y|, 2^-100) / 448,  q = e4m3(y / scale)  per row;
// y / scale = (h w) * 448 / max|h w| (r cancels).  A value that fp32 puts on
// the wrong side of a rounding border is off by a whole step of the 3-bit
// mantissa; the few values that fall near one are computed again in two fp32
// words, so that q is the e4m3 value nearest to the exact ratio (but for rows
// with max|y| below 2^-100 or max|h w| outside 2^-80 to 2^80, where the second
// word may be cut short).  The second words need the remainder of the largest
// product; the row's threads look for it only where a value is near a border.
//
// Backward, with dn = dy * w and n = h * r:
//   dx = r * (dn - n * mean(dn * n)) + dres,   dw = sum over rows of dy * n
// r is recomputed: the row is in registers anyway, so nothing is saved but h.
//
// Bound: HBM.  Each row is read once into registers (8-element vectors, one
// to five per thread) and written once; sums, the row statistics and dw are
// fp32.  TPR threads share a row, 256 / TPR rows share a CTA.  32,760 x 1536,
// bf16 + bf16 to bf16: 61 us, 6.6 TB/s (the last writes are still in L2 when it
// ends); 32,760 x 5120, bf16 + fp32 to e4m3: 277 us, 6.6 TB/s (298 in long
// runs, where the chip is at its power cap and instructions cost bandwidth:
// hence the tie check in three of them, and all that follows from it only in
// rows that have a value near a tie).
#include <algorithm>

#include <cuda_fp8.h>

#include "common.cuh"

namespace moga {
namespace norm {

constexpr float kE4m3Max = 448.f;
constexpr float kScaleFloor = 7.888609052210118e-31f;   // 2^-100
constexpr int kMaxD = 16384;


template <class T> struct Vec;
template <> struct Vec<__nv_bfloat16> {
  using type = uint4;
  static __device__ __forceinline__ type load(const __nv_bfloat16* p) { return *reinterpret_cast<const uint4*>(p); }
  static __device__ __forceinline__ void widen(const type& t, float* f) {
    const uint32_t u[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
  // rounds to nearest even
  static __device__ __forceinline__ type narrow(const float* f) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const type& t) { *reinterpret_cast<uint4*>(p) = t; }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* f) { store(p, narrow(f)); }
};
template <> struct Vec<float> {
  struct type { float4 a, b; };
  static __device__ __forceinline__ type load(const float* p) {
    return {*reinterpret_cast<const float4*>(p), *reinterpret_cast<const float4*>(p + 4)};
  }
  static __device__ __forceinline__ void widen(const type& t, float* f) {
    f[0] = t.a.x; f[1] = t.a.y; f[2] = t.a.z; f[3] = t.a.w;
    f[4] = t.b.x; f[5] = t.b.y; f[6] = t.b.z; f[7] = t.b.w;
  }
  static __device__ __forceinline__ type narrow(const float* f) {
    return {make_float4(f[0], f[1], f[2], f[3]), make_float4(f[4], f[5], f[6], f[7])};
  }
  static __device__ __forceinline__ void store(float* p, const type& t) {
    *reinterpret_cast<float4*>(p) = t.a;
    *reinterpret_cast<float4*>(p + 4) = t.b;
  }
  static __device__ __forceinline__ void store(float* p, const float* f) { store(p, narrow(f)); }
};
template <> struct Vec<__nv_fp8_e4m3> {
  // values already scaled into +-448; out of range saturates, NaN stays NaN
  static __device__ __forceinline__ void store(__nv_fp8_e4m3* p, const float* f) {
    uint32_t u[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i], f[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i + 2], f[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
      u[i] = lo | (hi << 16);
    }
    *reinterpret_cast<uint2*>(p) = make_uint2(u[0], u[1]);
  }
};

// 8 weights of either type as fp32 (w is small and stays in L1)
__device__ __forceinline__ void load_w(const void* w, bool w_bf16, int col, float* f) {
  if (w_bf16) {
    Vec<__nv_bfloat16>::widen(Vec<__nv_bfloat16>::load(static_cast<const __nv_bfloat16*>(w) + col), f);
  } else {
    Vec<float>::widen(Vec<float>::load(static_cast<const float*>(w) + col), f);
  }
}

// sum over WIDTH neighbouring lanes (the whole warp takes part)
template <int WIDTH = 32>
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = WIDTH / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Barrier of the TPR threads of one row (named barrier 1 + group).
template <int TPR>
__device__ __forceinline__ void row_sync(int group) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(TPR) : "memory");
}

// Sum over the TPR threads of a row, in the same order on every thread.
// `slots`: TPR / 32 floats of the row's own.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* slots, int group, int lane_in_row) {
  v = warp_sum<(TPR < 32 ? TPR : 32)>(v);
  if (TPR <= 32) return v;
  if ((lane_in_row & 31) == 0) slots[lane_in_row >> 5] = v;
  row_sync<TPR>(group);
  float r = slots[0];
#pragma unroll
  for (int i = 1; i < TPR / 32; ++i) r += slots[i];
  return r;
}

// The largest v over the TPR threads of a row (slots as above).
template <int TPR>
__device__ __forceinline__ float row_max(float v, float* slots, int group, int lane_in_row) {
#pragma unroll
  for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  if (TPR <= 32) return v;
  if ((lane_in_row & 31) == 0) slots[lane_in_row >> 5] = v;
  row_sync<TPR>(group);
  v = slots[0];
#pragma unroll
  for (int i = 1; i < TPR / 32; ++i) v = fmaxf(v, slots[i]);
  return v;
}

// Whether any thread of the row has v not 0; rows inside a warp: any of the warp.
template <int TPR>
__device__ __forceinline__ bool row_any(uint32_t v, int group) {
  if (TPR <= 32) return __any_sync(0xffffffffu, v != 0);
  uint32_t r;
  asm volatile(
      "{ .reg .pred p, q; setp.ne.u32 p, %1, 0; bar.red.or.pred q, %2, %3, p; selp.u32 %0, 1, 0, q; }"
      : "=r"(r)
      : "r"(v), "r"(1 + group), "n"(TPR)
      : "memory");
  return r != 0;
}

// hi + lo (|lo| below an ulp or so of hi) as one fp32 value that a later
// rounding to fewer bits rounds as it would the sum: the nearest value, moved
// to its odd neighbour on the remainder's side where the sum is not exact.
__device__ __forceinline__ float round_to_odd(float hi, float lo) {
  const float s = hi + lo, rest = lo - (s - hi);
  int b = __float_as_int(s);
  if (rest != 0.f && !(b & 1)) b += (rest > 0.f) == (s > 0.f) ? 1 : -1;
  return __int_as_float(b);
}

// bits of q past a tie of the 3-bit mantissa, wrapped: at most 16 << 12 within 8 units of one
__device__ __forceinline__ uint32_t past_tie(float q) { return (__float_as_uint(q) << 12) - ((0x80000u - 8u) << 12); }
constexpr uint32_t kNearTie = 16u << 12;
constexpr float kE4m3Normal = 0.015625f;   // 2^-6, the least normal value

struct FwdParams {
  const void *x, *res, *w;
  void *h, *y;
  float* scale;
  int N, d;
  float eps;
  bool w_bf16;
};

template <int TPR>
constexpr int kCtaThreads = TPR > 256 ? TPR : 256;

// ROWS rows at a time per TPR threads: short rows need several under way per
// thread to fill the memory's latency.  The e4m3 forms of three vectors ask for
// the four CTAs an SM that their 54 to 64 registers allow: left alone the
// compiler takes 48 and more instructions (32,760 x 1536, bf16 + bf16: 86
// against 82 us).
template <int TPR, int VPT, int ROWS, class XT, class HT, bool RES, class YT>
__global__ void __launch_bounds__(kCtaThreads<TPR>, sizeof(YT) == 1 && VPT == 3 ? 4 : 0)
rms_norm_kernel(const FwdParams p) {
  static_assert(TPR <= 32 || ROWS == 1, "rows that share a barrier go one at a time");
  constexpr int kGroups = kCtaThreads<TPR> / TPR;
  constexpr bool kQuant = sizeof(YT) == 1;
  __shared__ float red[3][kGroups][TPR > 32 ? TPR / 32 : 1];
  const int group = threadIdx.x / TPR, li = threadIdx.x % TPR;
  const int row0 = (blockIdx.x * kGroups + group) * ROWS;
  // A row's own barrier wants all of its threads, and they leave together; rows
  // inside a warp stay for its shuffles.
  if (TPR > 32 && row0 >= p.N) return;
  const int nv = p.d >> 3;
  // vector v of row r
  auto on = [&](int r, int v) { return v < nv && (TPR > 32 || row0 + r < p.N); };
  auto at = [&](int r, int v) { return (size_t)(row0 + r) * p.d + 8 * v; };
  float f[ROWS][VPT][8];
  typename Vec<XT>::type xv[ROWS][VPT];
  typename Vec<HT>::type rv[ROWS][VPT];
#pragma unroll
  for (int r = 0; r < ROWS; ++r)
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = li + i * TPR;
      if (on(r, v)) {
        xv[r][i] = Vec<XT>::load(static_cast<const XT*>(p.x) + at(r, v));
        if (RES) rv[r][i] = Vec<HT>::load(static_cast<const HT*>(p.res) + at(r, v));
      }
    }
  float rstd[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = li + i * TPR;
      if (on(r, v)) {
        Vec<XT>::widen(xv[r][i], f[r][i]);
        if (RES) {
          float t[8];
          Vec<HT>::widen(rv[r][i], t);
#pragma unroll
          for (int j = 0; j < 8; ++j) f[r][i][j] += t[j];
          const typename Vec<HT>::type stored = Vec<HT>::narrow(f[r][i]);
          Vec<HT>::store(static_cast<HT*>(p.h) + at(r, v), stored);
          Vec<HT>::widen(stored, f[r][i]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) ss += f[r][i][j] * f[r][i][j];
      }
    }
    ss = row_sum<TPR>(ss, red[0][group], group, li);
    rstd[r] = 1.f / sqrtf(ss / (float)p.d + p.eps);
  }
  if constexpr (!kQuant) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = li + i * TPR;
      if (v < nv) {
        float w[8];
        load_w(p.w, p.w_bf16, 8 * v, w);
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
          if (on(r, v)) {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[r][i][j] = f[r][i][j] * rstd[r] * w[j];
            Vec<YT>::store(static_cast<YT*>(p.y) + at(r, v), f[r][i]);
          }
      }
    }
  } else {
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      // f becomes t = h w rounded
      float mine = 0.f;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = li + i * TPR;
        if (on(r, v)) {
          float w[8];
          load_w(p.w, p.w_bf16, 8 * v, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            f[r][i][j] *= w[j];
            mine = fmaxf(mine, fabsf(f[r][i][j]));
          }
        }
      }
      const float mx = row_max<TPR>(mine, red[1][group], group, li);
      const float amax = mx * rstd[r];                          // max|y|; NaN if the row holds NaN or infinity
      const float top = amax < kScaleFloor ? kScaleFloor : amax;
      // the short way where neither 448 / max|h w| nor the floor matters
      const bool direct = amax >= kScaleFloor && mx >= kScaleFloor;
      const float k2 = kE4m3Max / (direct ? mx : top);
      if (!direct) {   // t 448 / max|h w| = (t r) 448 / top
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) f[r][i][j] *= rstd[r];
      }
      uint32_t near = 0;   // vectors with a value near a tie
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = li + i * TPR;
        if (on(r, v)) {
          float q[8], least = kE4m3Normal;
          uint32_t past = ~0u;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            q[j] = f[r][i][j] * k2;
            // the four roundings above (t, mx, 448 / mx, q) are worth 4 units at most
            past = min(past, past_tie(q[j]));
            least = fminf(least, fabsf(q[j]));
          }
          // Subnormal values are spaced as those of [2^-6, 2^-5): with 2^-6 added, whose unit is at
          // least twice theirs (their 4 are 2, and the sum's own rounding half a one), their ties
          // are ties of the mantissa.
          if (least < kE4m3Normal)
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (fabsf(q[j]) < kE4m3Normal) past = min(past, past_tie(fabsf(q[j]) + kE4m3Normal));
          near |= (past <= kNearTie ? 1u : 0u) << i;
          Vec<YT>::store(static_cast<YT*>(p.y) + at(r, v), q);
        }
      }
      if (!direct) near = 0;
      if (row_any<TPR>(near, group)) {   // 1 vector in 8000: in two words, max|h w| = mx + me
        auto reload = [&](int i, float* h, float* w) {   // vector i of this thread
          const int v = li + i * TPR;
          if (RES) Vec<HT>::widen(Vec<HT>::load(static_cast<const HT*>(p.h) + at(r, v)), h);
          else Vec<XT>::widen(Vec<XT>::load(static_cast<const XT*>(p.x) + at(r, v)), h);
          load_w(p.w, p.w_bf16, 8 * v, w);
        };
        float h[8], w[8], me = -mx;
        if (direct && mine == mx) {   // this thread has the largest product, or one of several
#pragma unroll 1
          for (int i = 0; i < VPT && on(r, li + i * TPR); ++i) {
            reload(i, h, w);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (fabsf(h[j] * w[j]) == mx) me = fmaxf(me, fmaf(fabsf(h[j]), fabsf(w[j]), -mx));
          }
        }
        me = row_max<TPR>(me, red[2][group], group, li);
        const float k2lo = (fmaf(-k2, mx, kE4m3Max) - k2 * me) / mx;
#pragma unroll 1
        for (; near; near &= near - 1) {
          const int i = __ffs(near) - 1;
          reload(i, h, w);
          float q[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float t = h[j] * w[j], hi = t * k2;
            const float lo = fmaf(t, k2, -hi) + fmaf(t, k2lo, fmaf(h[j], w[j], -t) * k2);
            q[j] = lo == 0.f ? hi : round_to_odd(hi, lo);   // a zero keeps its sign
          }
          Vec<YT>::store(static_cast<YT*>(p.y) + at(r, li + i * TPR), q);
        }
      }
      if (li == 0 && row0 + r < p.N) p.scale[row0 + r] = top / kE4m3Max;
    }
  }
}

struct BwdParams {
  const void *dy, *h, *w, *dres;
  void* dx;
  __nv_bfloat16* dx_branch;
  float* partial;    // [gridDim.x][d] sums of dy * h * r, or NULL
  int N, d;
  float eps;
  bool w_bf16;
};

// Residence of the backward's forms, which the kernel's launch bounds and the
// launch rule (bwd_shape) both take from here.  Of the forms with a warp a row
// or less (256 threads) an SM holds this many CTAs,
__host__ __device__ constexpr int bwd_warp_ctas(int vpt) { return vpt == 1 ? 3 : 2; }
// and of those with a row a CTA as many as these threads make up.
__host__ __device__ constexpr int bwd_sm_threads(int vpt, bool h_f32, bool ahead) {
  return vpt == 4 || ahead ? 512 : vpt == 2 && h_f32 ? 640 : 1024;
}

// Persistent: a CTA walks its rows with a fixed stride and keeps its share of
// dw in registers (each thread always sees the same columns), then adds its
// row groups in shared memory and writes one partial row.  No atomics: every
// sum runs in a fixed order, so dw is the same from run to run.
// TPR threads a row (0: the CTA), VPT vectors a thread.  Rows of up to 768
// elements: a warp a row, 8 rows a CTA; of up to 128 and 64, half and a quarter
// of a warp, so that no lane is idle.  Wider rows: a row a CTA of just enough
// threads, so that an SM holds many rows in different phases and the loads of
// some are under way while others are at their sums (bwd_shape).  63,960 x
// 1536, bf16 dy, fp32 h: 233 us, 6.7 TB/s, against 276 us of four rows a CTA
// with three vectors a thread; bf16 h: 129 us, 6.1 TB/s.  393,120 heads of 128,
// bf16: 62 us, of 64: 34 us, against 129 and 127 us of a warp a row.
template <int TPR, int VPT, class DT, class HT, bool AHEAD = false>
__global__ void __launch_bounds__(TPR > 0 ? 256 : bwd_sm_threads(VPT, sizeof(HT) == 4, AHEAD),
                                  TPR > 0 ? bwd_warp_ctas(VPT) : 1)
rms_norm_bwd_kernel(const BwdParams p) {
  constexpr int GROUPS = TPR > 0 ? 256 / TPR : 1;
  extern __shared__ float s_dw[];                 // [d] when there is more than one group
  __shared__ float2 red[2][32];
  const int tpr = TPR > 0 ? TPR : blockDim.x;
  const int group = TPR > 0 ? threadIdx.x / tpr : 0, li = TPR > 0 ? threadIdx.x % tpr : threadIdx.x;
  // rows of a warp's width of threads and less: the warp's rows go through the
  // loop together, those past the last one as zeros
  constexpr int kInWarp = TPR > 0 && TPR < 32 ? 32 / TPR : 1;
  const int sub = group % kInWarp;
  const int nv = p.d >> 3;
  float acc[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
  // AHEAD: the next row's vectors, on their way while this one is worked on
  typename Vec<DT>::type dn[AHEAD ? VPT : 1];
  typename Vec<HT>::type hn[AHEAD ? VPT : 1], sn[AHEAD ? VPT : 1];
  auto load = [&](int row, typename Vec<DT>::type* dt, typename Vec<HT>::type* ht, typename Vec<HT>::type* st) {
    const size_t base = (size_t)row * p.d;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = li + i * tpr;
      if (v < nv && (kInWarp == 1 || row < p.N)) {
        dt[i] = Vec<DT>::load(static_cast<const DT*>(p.dy) + base + 8 * v);
        ht[i] = Vec<HT>::load(static_cast<const HT*>(p.h) + base + 8 * v);
        if (p.dres) st[i] = Vec<HT>::load(static_cast<const HT*>(p.dres) + base + 8 * v);
      }
    }
  };
  const int step = gridDim.x * GROUPS;
  if constexpr (AHEAD) {
    if (blockIdx.x * GROUPS + group < p.N) load(blockIdx.x * GROUPS + group, dn, hn, sn);
  }
  int par = 0;
  for (int row = blockIdx.x * GROUPS + group; row - sub < p.N; row += gridDim.x * GROUPS, par ^= 1) {
    const size_t base = (size_t)row * p.d;
    const bool in = kInWarp == 1 || row < p.N;
    typename Vec<DT>::type dv[VPT];
    typename Vec<HT>::type hv[VPT], sv[VPT];
    if constexpr (AHEAD) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        dv[i] = dn[i];
        hv[i] = hn[i];
        sv[i] = sn[i];
      }
      if (row + step < p.N) load(row + step, dn, hn, sn);
    } else {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = li + i * tpr;
        if (v < nv && in) {
          dv[i] = Vec<DT>::load(static_cast<const DT*>(p.dy) + base + 8 * v);
          hv[i] = Vec<HT>::load(static_cast<const HT*>(p.h) + base + 8 * v);
          if (p.dres) sv[i] = Vec<HT>::load(static_cast<const HT*>(p.dres) + base + 8 * v);
        }
      }
    }
    float ss = 0.f, dot = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = li + i * tpr;
      if (v < nv && in) {
        float dy[8], h[8], w[8];
        Vec<DT>::widen(dv[i], dy);
        Vec<HT>::widen(hv[i], h);
        load_w(p.w, p.w_bf16, 8 * v, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          ss += h[j] * h[j];
          dot += dy[j] * h[j] * w[j];
        }
      }
    }
    ss = warp_sum<(TPR > 0 ? TPR : 32)>(ss);
    dot = warp_sum<(TPR > 0 ? TPR : 32)>(dot);
    if (TPR == 0) {   // both sums of the CTA's warps cross one barrier; the slots alternate, so one is enough
      if ((threadIdx.x & 31) == 0) red[par][threadIdx.x >> 5] = make_float2(ss, dot);
      __syncthreads();
      const bool on = (threadIdx.x & 31) < (blockDim.x >> 5);
      const float2 t = on ? red[par][threadIdx.x & 31] : make_float2(0.f, 0.f);
      ss = warp_sum(t.x);
      dot = warp_sum(t.y);
    }
    const float inv_d = 1.f / (float)p.d;
    const float rstd = 1.f / sqrtf(ss * inv_d + p.eps);
    // r (dn - n mean(dn n)) as r dn - n c, c = r mean(dn n): no power of r is
    // formed, so nothing leaves the fp32 range before the result does (r^3 would
    // for rows of rms 4e12 and more and for an eps of 1e-26 and less)
    const float c = rstd * (rstd * (dot * inv_d));
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = li + i * tpr;
      if (v < nv && in) {
        float dy[8], h[8], w[8], o[8];
        Vec<DT>::widen(dv[i], dy);
        Vec<HT>::widen(hv[i], h);
        load_w(p.w, p.w_bf16, 8 * v, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float n = h[j] * rstd;
          acc[i][j] += dy[j] * n;
          o[j] = rstd * (dy[j] * w[j]) - n * c;
        }
        if (p.dres) {
          float s[8];
          Vec<HT>::widen(sv[i], s);
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] += s[j];
        }
        Vec<HT>::store(static_cast<HT*>(p.dx) + base + 8 * v, o);
        if (p.dx_branch) Vec<__nv_bfloat16>::store(p.dx_branch + base + 8 * v, o);
      }
    }
  }
  if (!p.partial) return;
  float* dst = p.partial + (size_t)blockIdx.x * p.d;
  if constexpr (kInWarp > 1) {   // the warp's rows first, then its TPR lanes stand for it
#pragma unroll
    for (int o = 16; o >= TPR; o >>= 1)
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] += __shfl_xor_sync(0xffffffffu, acc[i][j], o);
  }
  constexpr int kParts = TPR > 0 ? 8 : 1;
  for (int g = 0; g < kParts; ++g) {
    if (group == g * kInWarp) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = li + i * tpr;
        if (v < nv) {
          if (g > 0) {
            float s[8];
            Vec<float>::widen(Vec<float>::load(s_dw + 8 * v), s);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[i][j] += s[j];
          }
          Vec<float>::store(g == kParts - 1 ? dst + 8 * v : s_dw + 8 * v, acc[i]);
        }
      }
    }
    if (kParts > 1) __syncthreads();
  }
}

// dw[c] = sum of the partial rows: 32 columns a CTA, 32 strided row slices
// added in order.
__global__ void __launch_bounds__(1024) rms_norm_dw_kernel(const float* __restrict__ partial, int rows, int d,
                                                           float* __restrict__ dw) {
  __shared__ float s[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x, j = threadIdx.y;
  float a = 0.f;
  if (c < d) {
    const float* q = partial + c;
    int r = j;
    for (; r + 7 * 32 < rows; r += 8 * 32) {   // eight loads under way (up to 37 rows a slice: 8 CTAs an SM)
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = q[(size_t)(r + 32 * i) * d];
#pragma unroll
      for (int i = 0; i < 8; ++i) a += v[i];
    }
    for (; r < rows; r += 32) a += q[(size_t)r * d];
  }
  s[j][threadIdx.x] = a;
  __syncthreads();
  if (j == 0 && c < d) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += s[i][threadIdx.x];
    dw[c] = t;
  }
}

// Forward layout (threads a row, vectors a thread): the first whose capacity
// holds the row, so that few lanes idle.  For few rows (up to the
// SM count) a row's own latency counts, not the lanes left idle, so wider rows
// are taken, up to one vector a thread (1 x 5120: 2.5 against 3.1 us, most of it
// the launch, 148 x 5120: 2.9 against 3.7; 300 x 5120: 5.9 against 4.4).
// Short rows of many (more than 64 per SM) go four at a time, up to 128 elements
// also two or four of them to a warp's width (393,120 heads of 128, bf16: 35
// against 81 us of a row a warp, one at a time; 100,000 x 256: 33.2 against
// 36.3, to e4m3 32.2 against 39.5; 60,000 x 512: no difference).
inline int pick_config(int d, int64_t N, int sms) {
  static const int cap[6] = {32 * 3, 64 * 3, 64 * 5, 128 * 5, 256 * 5, 512 * 5};
  const int nv = d >> 3;
  if (nv <= 32 && N > 64 * (int64_t)sms) return nv <= 8 ? 6 : nv <= 16 ? 7 : 8;
  int i = 0;
  while (cap[i] < nv) ++i;
  if (N <= sms) {
    static const int one[6] = {32, 64, 64, 128, 256, 512};
    while (i < 5 && one[i] < nv) ++i;
  }
  return i;
}

inline int sm_count_of_current() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 148;
  return n > 0 ? n : 148;
}

template <class XT, class HT, bool RES, class YT>
static moga_status launch_fwd(const FwdParams& p, cudaStream_t s) {
  switch (pick_config(p.d, p.N, sm_count_of_current())) {
#define MOGA_NORM_CASE(I, TPR, VPT, ROWS)                                                                      \
  case I: {                                                                                                    \
    constexpr int g = kCtaThreads<TPR> / TPR * ROWS;                                                           \
    rms_norm_kernel<TPR, VPT, ROWS, XT, HT, RES, YT><<<(p.N - 1) / g + 1, kCtaThreads<TPR>, 0, s>>>(p);        \
    break;                                                                                                     \
  }
    MOGA_NORM_CASE(0, 32, 3, 1)
    MOGA_NORM_CASE(1, 64, 3, 1)
    MOGA_NORM_CASE(2, 64, 5, 1)
    MOGA_NORM_CASE(3, 128, 5, 1)
    MOGA_NORM_CASE(4, 256, 5, 1)
    MOGA_NORM_CASE(5, 512, 5, 1)
    MOGA_NORM_CASE(6, 8, 1, 4)
    MOGA_NORM_CASE(7, 16, 1, 4)
    MOGA_NORM_CASE(8, 32, 1, 4)
#undef MOGA_NORM_CASE
  }
  return check_launch("moga_rms_norm");
}

template <class XT, class HT, bool RES>
static moga_status launch_fwd_y(const FwdParams& p, moga_dtype y_dt, cudaStream_t s) {
  if (y_dt == MOGA_E4M3) return launch_fwd<XT, HT, RES, __nv_fp8_e4m3>(p, s);
  if (y_dt == MOGA_BF16) return launch_fwd<XT, HT, RES, __nv_bfloat16>(p, s);
  if constexpr (sizeof(HT) == 4) return launch_fwd<XT, HT, RES, float>(p, s);
  return fail(MOGA_ERR_UNSUPPORTED, "moga_rms_norm: an fp32 output needs an fp32 stream");
}

// Backward launch shape: threads of a CTA, vectors a thread, CTAs an SM holds.
// All CTAs have to be resident at once (a second round of them costs a third),
// so the last is what the kernels' launch bounds hold their registers to
// (bwd_warp_ctas, bwd_sm_threads): 64 a thread (one vector; two with a bf16 h),
// 96 (two, fp32 h), 128 (three, four, and with the next row under way), 80 (a
// warp a row or less, one).  Without a bound three vectors with an fp32 h take
// 138 to 152, one CTA an SM and a second round (40,000 rows, bf16 dy, of 264:
// 61 against 42 us, of 512: 70 against 52, of 768: 88 against 73).
// Short rows keep the next one under way, but for a warp's width of fp32 h,
// where registers spill and enough bytes are on their way without (256
// columns: bf16 h 73 against 84 us for 200,000 rows, fp32 249 against 238 us
// for 400,000).
// Bytes on the way decide between one and two vectors: two where a bf16 row's
// vectors are small or where one would leave an SM's threads unused
// (32,760 x 5120, fp32 h: 526 us with one vector, 367 with two).
// A bf16 row's vectors are small: where 512 threads fill up, they keep the next
// row's under way as well (at 110 registers; 63,960 x 1536: 129 against 138 us
// with 1024 threads that do not, 20,000 x 8192: 210 against 231; 5120, of whose
// 320-thread CTAs only one would fit: 266 against 236).  So do the fp32 rows of
// which an SM holds one either way (20,000 x 8192, bf16 dy: 367 against 466 us;
// fp32 dy: 474 against 472 with dres, 411 against 442 without).
struct BwdShape {
  int threads, vpt, per_sm;
  bool ahead;
};
constexpr int kWarpRow = 768;
inline int bwd_rows(int d) { return d <= 64 ? 32 : d <= 128 ? 16 : d <= kWarpRow ? 8 : 1; }   // of a CTA
inline BwdShape bwd_shape(int d, bool h_f32) {
  if (d <= 256) return {256, 1, bwd_warp_ctas(1), !h_f32 || d <= 128};
  if (d <= kWarpRow) return {256, 3, bwd_warp_ctas(3), false};
  auto threads = [d](int vpt) { return (ceil_div(d / 8, vpt) + 31) / 32 * 32; };
  const int t1 = threads(1), t2 = threads(2);
  auto shape = [h_f32](int threads, int vpt, bool ahead) {
    return BwdShape{threads, vpt, std::max(1, bwd_sm_threads(vpt, h_f32, ahead) / threads), ahead};
  };
  if ((!h_f32 || t2 >= 448) && t2 <= 512 && 512 / t2 * t2 >= 448) return shape(t2, 2, true);
  if (!h_f32) return shape(t2, 2, false);
  if (d > 8192) return shape(threads(4), 4, false);
  if (1024 / t1 * t1 >= 896) return shape(t1, 1, false);
  return shape(t2, 2, false);
}
inline int bwd_ctas(int64_t N, int d, bool h_f32, int sms) {
  const int rows = bwd_rows(d);
  return (int)std::min<int64_t>((N + rows - 1) / rows, (int64_t)sms * bwd_shape(d, h_f32).per_sm);
}

// the kernel of bwd_shape's form
template <class DT, class HT>
static auto bwd_kernel(int d) -> void (*)(const BwdParams) {
  const BwdShape k = bwd_shape(d, sizeof(HT) == 4);
  if (d <= 64) return rms_norm_bwd_kernel<8, 1, DT, HT, true>;
  if (d <= 128) return rms_norm_bwd_kernel<16, 1, DT, HT, true>;
  if (d <= 256) return rms_norm_bwd_kernel<32, 1, DT, HT, sizeof(HT) == 2>;
  if (d <= kWarpRow) return rms_norm_bwd_kernel<32, 3, DT, HT>;
  if constexpr (sizeof(HT) == 4) {
    if (k.vpt == 1) return rms_norm_bwd_kernel<0, 1, DT, HT>;
    if (k.vpt == 4) return rms_norm_bwd_kernel<0, 4, DT, HT>;
  }
  return k.ahead ? rms_norm_bwd_kernel<0, 2, DT, HT, true> : rms_norm_bwd_kernel<0, 2, DT, HT>;
}

// its columns' sums, shared by a CTA's rows where it has several
inline size_t bwd_smem(int d) { return d <= kWarpRow ? d * sizeof(float) : 0; }

template <class DT, class HT>
static moga_status launch_bwd(const BwdParams& p, int ctas, cudaStream_t s) {
  bwd_kernel<DT, HT>(p.d)<<<ctas, bwd_shape(p.d, sizeof(HT) == 4).threads, bwd_smem(p.d), s>>>(p);
  return check_launch("moga_rms_norm_bwd");
}

static moga_status check_dims(const char* who, int64_t N, int32_t d, float eps) {
  if (N <= 0 || N > INT32_MAX / 2) return fail(MOGA_ERR_INVALID_ARG, "%s: N=%lld out of range", who, (long long)N);
  if (d <= 0 || d % 8 != 0) return fail(MOGA_ERR_INVALID_ARG, "%s: d=%d must be a positive multiple of 8", who, d);
  if (d > kMaxD) return fail(MOGA_ERR_UNSUPPORTED, "%s: d=%d above %d", who, d, kMaxD);
  if (!(eps > 0.f && eps < 1e30f)) return fail(MOGA_ERR_INVALID_ARG, "%s: eps must be positive and finite", who);
  return MOGA_OK;
}

inline bool is_float_dt(moga_dtype t) { return t == MOGA_F32 || t == MOGA_BF16; }

}  // namespace norm
}  // namespace moga

extern "C" moga_status moga_rms_norm(const void* x, moga_dtype x_dt, const void* residual, moga_dtype res_dt,
                                     const void* w, moga_dtype w_dt, int64_t N, int32_t d, float eps, void* h,
                                     void* y, moga_dtype y_dt, float* scale, void* stream) {
  using namespace moga;
  using namespace moga::norm;
  moga_status st = check_dims("moga_rms_norm", N, d, eps);
  if (st != MOGA_OK) return st;
  if (!x || !w || !y) return fail(MOGA_ERR_INVALID_ARG, "moga_rms_norm: null pointer");
  if ((residual != nullptr) != (h != nullptr))
    return fail(MOGA_ERR_INVALID_ARG, "moga_rms_norm: residual and h go together");
  if (!is_float_dt(x_dt) || !is_float_dt(w_dt) || (residual && !is_float_dt(res_dt)) ||
      (!is_float_dt(y_dt) && y_dt != MOGA_E4M3))
    return fail(MOGA_ERR_INVALID_ARG, "moga_rms_norm: bad dtype");
  if ((y_dt == MOGA_E4M3) != (scale != nullptr))
    return fail(MOGA_ERR_INVALID_ARG, "moga_rms_norm: scale goes with an e4m3 output");
  if (residual && x_dt == MOGA_F32 && res_dt == MOGA_BF16)
    return fail(MOGA_ERR_UNSUPPORTED, "moga_rms_norm: an fp32 x needs an fp32 residual");
  const uintptr_t a = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(residual) |
                      reinterpret_cast<uintptr_t>(w) | reinterpret_cast<uintptr_t>(h);
  if ((a & 15) || (reinterpret_cast<uintptr_t>(y) & 15) || (reinterpret_cast<uintptr_t>(scale) & 3))
    return fail(MOGA_ERR_INVALID_ARG, "moga_rms_norm: pointers must be 16-byte aligned");
  norm::FwdParams p;
  p.x = x;
  p.res = residual;
  p.w = w;
  p.h = h;
  p.y = y;
  p.scale = scale;
  p.N = (int)N;
  p.d = d;
  p.eps = eps;
  p.w_bf16 = w_dt == MOGA_BF16;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  using B = __nv_bfloat16;
  if (!residual)
    return x_dt == MOGA_BF16 ? launch_fwd_y<B, B, false>(p, y_dt, s) : launch_fwd_y<float, float, false>(p, y_dt, s);
  if (res_dt == MOGA_BF16) return launch_fwd_y<B, B, true>(p, y_dt, s);
  return x_dt == MOGA_BF16 ? launch_fwd_y<B, float, true>(p, y_dt, s) : launch_fwd_y<float, float, true>(p, y_dt, s);
}

extern "C" size_t moga_rms_norm_bwd_ws_bytes(int64_t N, int32_t d) {
  using namespace moga::norm;
  if (N <= 0 || N > INT32_MAX / 2 || d <= 0 || d % 8 != 0 || d > kMaxD) return 0;
  const int sms = sm_count_of_current();
  return (size_t)std::max(bwd_ctas(N, d, false, sms), bwd_ctas(N, d, true, sms)) * d * sizeof(float);
}

extern "C" moga_status moga_rms_norm_bwd(const void* dy, moga_dtype dy_dt, const void* h, moga_dtype h_dt,
                                         const void* w, moga_dtype w_dt, const void* dres, int64_t N, int32_t d,
                                         float eps, void* dx, void* dx_branch, float* dw, void* ws, size_t ws_bytes,
                                         void* stream) {
  using namespace moga;
  using namespace moga::norm;
  moga_status st = check_dims("moga_rms_norm_bwd", N, d, eps);
  if (st != MOGA_OK) return st;
  if (!dy || !h || !w || !dx) return fail(MOGA_ERR_INVALID_ARG, "moga_rms_norm_bwd: null pointer");
  if (!is_float_dt(dy_dt) || !is_float_dt(h_dt) || !is_float_dt(w_dt))
    return fail(MOGA_ERR_INVALID_ARG, "moga_rms_norm_bwd: bad dtype");
  if (dy_dt == MOGA_F32 && h_dt == MOGA_BF16)
    return fail(MOGA_ERR_UNSUPPORTED, "moga_rms_norm_bwd: an fp32 dy needs an fp32 h");
  if (dx_branch && h_dt == MOGA_BF16)
    return fail(MOGA_ERR_INVALID_ARG, "moga_rms_norm_bwd: dx_branch is for an fp32 h (dx is bf16 already)");
  const uintptr_t a = reinterpret_cast<uintptr_t>(dy) | reinterpret_cast<uintptr_t>(h) |
                      reinterpret_cast<uintptr_t>(w) | reinterpret_cast<uintptr_t>(dres) |
                      reinterpret_cast<uintptr_t>(dx) | reinterpret_cast<uintptr_t>(dx_branch) |
                      reinterpret_cast<uintptr_t>(dw) | reinterpret_cast<uintptr_t>(ws);
  if (a & 15) return fail(MOGA_ERR_INVALID_ARG, "moga_rms_norm_bwd: pointers must be 16-byte aligned");
  const int ctas = bwd_ctas(N, d, h_dt == MOGA_F32, sm_count_of_current());
  if (dw) {
    const size_t need = moga_rms_norm_bwd_ws_bytes(N, d);
    if (!ws) return fail(MOGA_ERR_INVALID_ARG, "moga_rms_norm_bwd: null workspace");
    if (ws_bytes < need)
      return fail(MOGA_ERR_WORKSPACE, "moga_rms_norm_bwd: workspace %zu < %zu bytes", ws_bytes, need);
  }
  norm::BwdParams p;
  p.dy = dy;
  p.h = h;
  p.w = w;
  p.dres = dres;
  p.dx = dx;
  p.dx_branch = static_cast<__nv_bfloat16*>(dx_branch);
  p.partial = dw ? static_cast<float*>(ws) : nullptr;
  p.N = (int)N;
  p.d = d;
  p.eps = eps;
  p.w_bf16 = w_dt == MOGA_BF16;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  using B = __nv_bfloat16;
  if (h_dt == MOGA_BF16) st = launch_bwd<B, B>(p, ctas, s);
  else if (dy_dt == MOGA_BF16) st = launch_bwd<B, float>(p, ctas, s);
  else st = launch_bwd<float, float>(p, ctas, s);
  if (st != MOGA_OK || !dw) return st;
  rms_norm_dw_kernel<<<ceil_div(d, 32), dim3(32, 32), 0, s>>>(p.partial, ctas, d, dw);
  return check_launch("moga_rms_norm_bwd/dw");
}

// test hook (moga_testing.h): CTAs an SM asked for, and resident
extern "C" int64_t moga_test_norm_bwd_ctas(int32_t d, moga_dtype h_dt, moga_dtype dy_dt, int32_t* resident) {
  using namespace moga;
  using namespace moga::norm;
  if (check_dims("moga_test_norm_bwd_ctas", 1, d, 1.f) != MOGA_OK || !is_float_dt(h_dt) || !is_float_dt(dy_dt) ||
      (dy_dt == MOGA_F32 && h_dt == MOGA_BF16))
    return -1;
  using B = __nv_bfloat16;
  const BwdShape k = bwd_shape(d, h_dt == MOGA_F32);
  auto* f = h_dt == MOGA_BF16    ? bwd_kernel<B, B>(d)
            : dy_dt == MOGA_BF16 ? bwd_kernel<B, float>(d)
                                 : bwd_kernel<float, float>(d);
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, f, k.threads, bwd_smem(d)) != cudaSuccess) return -1;
  *resident = n;
  return k.per_sm;
}
