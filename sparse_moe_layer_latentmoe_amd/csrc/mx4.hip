// Matrices in microscaled 4-bit floating point (MXFP4: E2M1 elements, a
// power-of-two scale for each block of 32 along k): quantisation of
// activations, the way back, and products of two such matrices.
//
//   value = code * 2^(scale - 127);  y[m][n] = sum_k x[m][k] w[n][k]
//
// The matrix instructions take the codes and the scales as they are stored
// (a lane's 16 bytes are one block of 32, its scale one byte of a register)
// and add into fp32.  Products of codes are multiples of 1/4 up to 36, so a
// block's sum is exact; blocks of different scales and the running sum are
// added to about 2^-23 of the sum of the magnitudes (measured: exact where all
// scales are equal, at worst 2^-22.3 with scales spread over 2^24), which is
// an fp32 sum.  So results of either type take the same instructions.
// Weights are the A operand and tokens the B operand: a lane's results are
// consecutive columns of one token.
#include <type_traits>

#include "fp8_copies.h"
#include "fp8_device.h"
#include "gemm_device.h"
#include "kernels.h"
#include "wave_device.h"

namespace lmoe {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// ---- quantisation ------------------------------------------------------------

// 2^(byte - 127); 255 stands for NaN.
__device__ __forceinline__ float e8m0_value(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7FC00000u)
                      : (byte ? __uint_as_float(byte << 23) : __uint_as_float(0x00400000u));
}

// E2M1 magnitude code of a >= 0: nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6, ties to
// the even code, larger ones 6.
__device__ __forceinline__ uint32_t e2m1_code(float a) {
  return (a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) + (a >= 3.5f) +
         (a > 5.0f);
}

// Eight values of a row from column c; columns from `cols` on read as 0.
template <bool VEC>
__device__ __forceinline__ void mx4_load8(const uint16_t* p, int c, int cols, float (&v)[8]) {
  if (VEC && c + 8 <= cols) {
    const u16x8 a = *reinterpret_cast<const u16x8*>(p + c);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = bf16_to_f32(a[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < cols ? bf16_to_f32(p[c + i]) : 0.f;
  }
}
template <bool VEC>
__device__ __forceinline__ void mx4_load8(const float* p, int c, int cols, float (&v)[8]) {
  if (VEC && c + 8 <= cols) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(p + c);
    const f32x4 b = *reinterpret_cast<const f32x4*>(p + c + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < cols ? p[c + i] : 0.f;
  }
}

// Scale exponent of a block whose largest magnitude is amax: floor(log2 amax)
// - 2, so that the largest element lies in [4, 8), at least -127 (zeros,
// denormals).
__device__ __forceinline__ int mx4_exponent(float amax) {
  int ex;
  (void)frexpf(amax, &ex);  // amax = m 2^ex, 0.5 <= m < 1
  return amax > 0.f ? max(ex - 3, -127) : -127;
}

// Eight values / 2^e as codes, the first in the lowest four bits; a value that
// rounds to 0 loses its sign.
__device__ __forceinline__ uint32_t mx4_pack8(const float (&v)[8], int e) {
  uint32_t w = 0;
  if (e >= -100) {
    const float s = __uint_as_float((uint32_t)(e + 127) << 23);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], s, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], s, 3);
  } else {
    // denormal numbers among them: the comparisons themselves
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t c = e2m1_code(ldexpf(fabsf(v[i]), -e));
      w |= (c | (v[i] < 0.f ? 8u : 0u)) << (4 * i);
    }
  }
  const uint32_t m = w & 0x77777777u;
  const uint32_t some = (m | (m >> 1) | (m >> 2)) & 0x11111111u;
  return m | (w & (some << 3));
}

}  // namespace

// Rows [rows, cols], `stride` elements apart: four lanes to a block of 32, eight
// values a lane; codes of nb blocks a row (those past cols are 0).
template <class T, bool VEC>
__global__ __launch_bounds__(256) void mx4_quantize_kernel(const T* __restrict__ x, long rows,
                                                           int cols, long stride, int nb,
                                                           uint32_t* __restrict__ codes,
                                                           uint8_t* __restrict__ scales) {
  const long b = (long)blockIdx.x * 64 + threadIdx.x / 4;
  if (b >= rows * nb) return;  // whole groups of four lanes
  const long row = b / nb;
  const int i = threadIdx.x & 3;
  float v[8];
  mx4_load8<VEC>(x + row * stride, (int)(b - row * nb) * 32 + i * 8, cols, v);
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[j]));
  m = fmaxf(m, __shfl_xor(m, 1, 64));
  m = fmaxf(m, __shfl_xor(m, 2, 64));
  const int e = mx4_exponent(m);
  codes[b * 4 + i] = mx4_pack8(v, e);
  if (i == 0) scales[b] = (uint8_t)(e + 127);
}

// The values, rounded once to T where they do not fit it: eight a lane.
template <class T, bool VEC>
__global__ __launch_bounds__(256) void mx4_dequantize_kernel(const uint32_t* __restrict__ codes,
                                                             const uint8_t* __restrict__ scales,
                                                             long rows, int cols, int nb,
                                                             T* __restrict__ y) {
  const long b = (long)blockIdx.x * 64 + threadIdx.x / 4;
  if (b >= rows * nb) return;
  const long row = b / nb;
  const int i = threadIdx.x & 3;
  const int c = (int)(b - row * nb) * 32 + i * 8;
  if (c >= cols) return;
  const uint32_t w = codes[b * 4 + i];
  const float s = e8m0_value(scales[b]);
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t q = (w >> (4 * j)) & 15u, ex = (q >> 1) & 3u;
    // exponent bits and one mantissa bit; 0.5 is the only subnormal
    const float a = ex ? __uint_as_float(((ex + 126u) << 23) | ((q & 1u) << 22))
                       : ((q & 1u) ? 0.5f : 0.f);
    v[j] = ((q & 8u) ? -a : a) * s;
  }
  T* yp = y + row * cols + c;
  if constexpr (std::is_same<T, float>::value) {
    if (VEC && c + 8 <= cols) {
      *reinterpret_cast<f32x4*>(yp) = f32x4{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4*>(yp + 4) = f32x4{v[4], v[5], v[6], v[7]};
      return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j < cols) yp[j] = v[j];
  } else {
    u16x8 o;
#pragma unroll
    for (int j = 0; j < 8; ++j)  // (a NaN stays one: f32_to_bf16 is for numbers)
      o[j] = v[j] == v[j] ? f32_to_bf16(v[j]) : (uint16_t)0x7FC0u;
    if (VEC && c + 8 <= cols) {
      *reinterpret_cast<u16x8*>(yp) = o;
      return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j < cols) yp[j] = o[j];
  }
}

// ---- products -------------------------------------------------------------------

namespace {

// A lane's 16 bytes as the instructions' operand (they take the low half).
__device__ __forceinline__ i32x8 low(i32x4 a) {
  return __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
}

// Row of x that row m of the product reads, and whether there is one.
__device__ __forceinline__ long mx4_x_row(const Mx4Gemm& p, int m, bool& ok) {
  ok = true;
  if (!p.rows) return m;
  const int r = p.rows[m];
  ok = r >= 0 && r < p.x_rows;
  return ok ? r : 0;
}

template <class OUT>
__device__ __forceinline__ void mx4_store4(const Mx4Gemm& p, int m, int n, f32x4 v) {
  OUT* y = static_cast<OUT*>(p.y) + (size_t)m * p.N + n;
  if constexpr (std::is_same<OUT, float>::value)
    *reinterpret_cast<f32x4*>(y) = v;
  else
    store4_bf16(y, v);
}

// 16-byte piece c of row r of 16 rows loaded as whole lines: a holds rows 0-7,
// b rows 8-15, lane 8 (r % 8) + c the piece.
__device__ __forceinline__ i32x4 mx4_permute(const i32x4& a, const i32x4& b, int src4, bool lo) {
  i32x4 r;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const int va = __builtin_amdgcn_ds_bpermute(src4, a[d]);
    const int vb = __builtin_amdgcn_ds_bpermute(src4, b[d]);
    r[d] = lo ? va : vb;
  }
  return r;
}

}  // namespace

// Few tokens: every weight byte is read once, as whole cache lines, and k is
// split over the NW waves of a work-group, whose sums are added in LDS in a
// fixed order.  Work-group: 16 RG weight rows x 16 token rows.  A step is a line
// of 128 bytes of each row (256 k, eight blocks): lane (r, q) (r = lane % 16,
// q = lane / 16) takes blocks q and 4 + q of row r, whose scales are byte q of
// the line's two scale words.
template <bool GROUPED, int NW, int RG, int U, class OUT>
__global__ __launch_bounds__(NW * 64) void mx4_stream_kernel(Mx4Gemm p, const Tile* tiles,
                                                             const int* ntiles) {
  __shared__ f32x4 red[NW][RG][64];
  const int nblocks = (p.N + 16 * RG - 1) / (16 * RG);
  const int nb = blockIdx.x % nblocks;
  const int tm = blockIdx.x / nblocks;
  int e = 0, m0 = tm * 16, mcount = min(16, p.M - m0);
  if (GROUPED) {
    if (tm >= *ntiles) return;
    e = uniform(tiles[tm].expert);
    m0 = uniform(tiles[tm].row0);
    mcount = uniform(tiles[tm].nrows);
  }
  const int n0 = nb * (16 * RG);
  const int lane = threadIdx.x & 63;
  const int w = uniform(threadIdx.x >> 6);
  const int r16 = lane & 15, kq = lane >> 4;
  const int RB = p.K / 2, SW = p.K / 128;  // bytes and scale words of a row
  const int lines = (SW + 1) / 2;
  const int kbeg = w * lines / NW, kend = (w + 1) * lines / NW;

  const int lrow = lane >> 3;
  const uint8_t* wa[RG];
  const uint32_t* wsp[RG];
#pragma unroll
  for (int g = 0; g < RG; ++g) {
    // 16-row groups past N read the last one (N is a multiple of 16)
    const size_t n = (size_t)e * p.N + min(n0 + g * 16, p.N - 16);
    wa[g] = p.w + (n + lrow) * RB;
    wsp[g] = reinterpret_cast<const uint32_t*>(p.ws) + (n + r16) * SW;
  }
  bool xok;
  const long row = mx4_x_row(p, m0 + (r16 < mcount ? r16 : 0), xok);
  const uint8_t* xp = p.x + row * RB + kq * 16;
  const uint32_t* xsp = reinterpret_cast<const uint32_t*>(p.xs) + row * SW;
  const int src0 = (((r16 & 7) << 3) | kq) * 4;
  const int src1 = (((r16 & 7) << 3) | (4 + kq)) * 4;
  const bool lo = r16 < 8;

  f32x4 acc[RG];
#pragma unroll
  for (int g = 0; g < RG; ++g) acc[g] = f32x4{0.f, 0.f, 0.f, 0.f};

  struct Stage {
    i32x4 l[U][RG][2], x[U][2];
    uint32_t s[U][RG][2], xs[U][2];
  };
  // Half a line ends the row where K is an odd multiple of 128: its second
  // half reads the first one's bytes again and is not multiplied.
  auto load = [&](Stage& S, int kb) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (U > 1 && kb + u >= kend) break;
      const int k = kb + u;
      const bool half = 2 * k + 2 > SW;
      const int ch = half ? (lane & 3) : (lane & 7);
#pragma unroll
      for (int g = 0; g < RG; ++g) {
        const uint8_t* at = wa[g] + (size_t)k * 128 + ch * 16;
        S.l[u][g][0] = __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(at));
        S.l[u][g][1] =
            __builtin_nontemporal_load(reinterpret_cast<const i32x4*>(at + (size_t)8 * RB));
        S.s[u][g][0] = wsp[g][2 * k];
        S.s[u][g][1] = wsp[g][2 * k + (half ? 0 : 1)];
      }
      S.x[u][0] = *reinterpret_cast<const i32x4*>(xp + (size_t)k * 128);
      S.x[u][1] = *reinterpret_cast<const i32x4*>(xp + (size_t)k * 128 + (half ? 0 : 64));
      S.xs[u][0] = xsp[2 * k];
      S.xs[u][1] = xsp[2 * k + (half ? 0 : 1)];
    }
  };
  auto compute = [&](const Stage& S, int kb) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (U > 1 && kb + u >= kend) break;
      const bool half = 2 * (kb + u) + 2 > SW;
      // a row index outside x: zeros (codes 0, scale 1)
      const i32x4 none = {0, 0, 0, 0};
      const i32x4 x0 = xok ? S.x[u][0] : none, x1 = xok ? S.x[u][1] : none;
      const int s0 = xok ? (int)(S.xs[u][0] >> (8 * kq)) : 127;
      const int s1 = xok ? (int)(S.xs[u][1] >> (8 * kq)) : 127;
#pragma unroll
      for (int g = 0; g < RG; ++g) {
        const i32x4 w0 = mx4_permute(S.l[u][g][0], S.l[u][g][1], src0, lo);
        acc[g] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            low(w0), low(x0), acc[g], 4, 4, 0, (int)(S.s[u][g][0] >> (8 * kq)), 0, s0);
        if (!half) {
          const i32x4 w1 = mx4_permute(S.l[u][g][0], S.l[u][g][1], src1, lo);
          acc[g] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              low(w1), low(x1), acc[g], 4, 4, 0, (int)(S.s[u][g][1] >> (8 * kq)), 0, s1);
        }
      }
    }
  };
  Stage A, B;
  if (kbeg < kend) load(A, kbeg);
  for (int kb = kbeg; kb < kend; kb += 2 * U) {
    if (kb + U < kend) load(B, kb + U);
    compute(A, kb);
    if (kb + U < kend) {
      if (kb + 2 * U < kend) load(A, kb + 2 * U);
      compute(B, kb + U);
    }
  }

#pragma unroll
  for (int g = 0; g < RG; ++g) red[w][g][lane] = acc[g];
  __syncthreads();
  for (int g = w; g < RG; g += NW) {
    f32x4 sm = red[0][g][lane];
#pragma unroll
    for (int v = 1; v < NW; ++v) sm += red[v][g][lane];
    const int n = n0 + g * 16;
    if (r16 < mcount && n < p.N) mx4_store4<OUT>(p, m0 + r16, n + kq * 4, sm);
  }
}

// ---- launchers ---------------------------------------------------------------------

namespace {

template <class F>
void with_type(bool bf16, bool vec, F f) {
  if (bf16 && vec) f(uint16_t{}, std::true_type{});
  else if (bf16) f(uint16_t{}, std::false_type{});
  else if (vec) f(float{}, std::true_type{});
  else f(float{}, std::false_type{});
}

bool wide(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// A launch has fewer than 2^32 threads.
bool too_many(long grid, int threads) { return grid >= (1L << 32) / threads; }

struct Plan {
  bool stream;  // weight streaming, else LDS-tiled
  int bm;       // token rows of a tile
  int splits;   // of k (dense tiles)
};

Plan make_plan(int M, int N, int K, int groups) {
  (void)M, (void)N, (void)K, (void)groups;
  return {true, kStreamTileM, 1};
}

int grouped_tiles(int rows, int groups, int tile_m) {
  return (rows < groups ? rows : groups) + rows / tile_m + 1;
}

// Work-groups and threads of a product's launch.
constexpr int kGroupedWaves = 4, kGroupedRG = 4, kDenseWaves = 8, kDenseRG = 1;
long grid_of(const Plan& plan, int M, int N, int groups, int* threads) {
  const int rg = groups ? kGroupedRG : kDenseRG;
  *threads = 64 * (groups ? kGroupedWaves : kDenseWaves);
  const long tiles = groups ? grouped_tiles(M, groups, plan.bm) : (M + plan.bm - 1) / plan.bm;
  return tiles * ((N + 16 * rg - 1) / (16 * rg));
}

template <class OUT>
hipError_t launch(const Mx4Gemm& p, const Plan& plan, const Tile* tiles, const int* ntiles,
                  hipStream_t s) {
  int threads;
  const long grid = grid_of(plan, p.M, p.N, p.groups, &threads);
  if (too_many(grid, threads)) return hipErrorInvalidConfiguration;
  if (p.groups)
    mx4_stream_kernel<true, kGroupedWaves, kGroupedRG, 1, OUT><<<grid, threads, 0, s>>>(p, tiles,
                                                                                       ntiles);
  else
    mx4_stream_kernel<false, kDenseWaves, kDenseRG, 2, OUT><<<grid, threads, 0, s>>>(p, nullptr,
                                                                                    nullptr);
  return hipGetLastError();
}

}  // namespace

hipError_t mx4_quantize(const void* x, bool bf16, long rows, int cols, long stride,
                        uint8_t* codes, uint8_t* scales, hipStream_t s) {
  const int nb = (cols + 31) / 32;
  const long grid = (rows * nb + 63) / 64;
  const bool vec = stride % (bf16 ? 8 : 4) == 0 && wide(x, 16);
  with_type(bf16, vec, [&](auto t, auto v) {
    using T = decltype(t);
    mx4_quantize_kernel<T, decltype(v)::value><<<grid, 256, 0, s>>>(
        static_cast<const T*>(x), rows, cols, stride, nb, reinterpret_cast<uint32_t*>(codes),
        scales);
  });
  return hipGetLastError();
}

hipError_t mx4_dequantize(const uint8_t* codes, const uint8_t* scales, long rows, int cols,
                          void* y, bool bf16, hipStream_t s) {
  const int nb = (cols + 31) / 32;
  const long grid = (rows * nb + 63) / 64;
  const bool vec = cols % (bf16 ? 8 : 4) == 0 && wide(y, 16);
  with_type(bf16, vec, [&](auto t, auto v) {
    using T = decltype(t);
    mx4_dequantize_kernel<T, decltype(v)::value><<<grid, 256, 0, s>>>(
        reinterpret_cast<const uint32_t*>(codes), scales, rows, cols, nb, static_cast<T*>(y));
  });
  return hipGetLastError();
}

bool mx4_matmul_fits(int M, int N, int K, int groups) {
  int threads;
  const long grid = grid_of(make_plan(M, N, K, groups), M, N, groups, &threads);
  return !too_many(grid, threads);
}

size_t mx4_matmul_workspace(int M, int N, int K, int groups) {
  const Plan plan = make_plan(M, N, K, groups);
  if (groups) return 256 + (size_t)grouped_tiles(M, groups, plan.bm) * sizeof(Tile);
  return plan.splits > 1 ? (size_t)plan.splits * M * N * sizeof(float) : 0;
}

hipError_t mx4_matmul(Mx4Gemm p, const int32_t* offsets, bool out_bf16, void* ws, hipStream_t s) {
  const Plan plan = make_plan(p.M, p.N, p.K, p.groups);
  const Tile* tiles = nullptr;
  const int32_t* ntiles = nullptr;
  if (p.groups) {
    const int max_tiles = grouped_tiles(p.M, p.groups, plan.bm);
    int32_t* n = static_cast<int32_t*>(ws);
    Tile* t = reinterpret_cast<Tile*>(static_cast<char*>(ws) + 256);
    const hipError_t e = group_tiles(offsets, p.groups, p.M, plan.bm, max_tiles, t, n, s);
    if (e != hipSuccess) return e;
    tiles = t;
    ntiles = n;
  }
  return out_bf16 ? launch<uint16_t>(p, plan, tiles, ntiles, s)
                  : launch<float>(p, plan, tiles, ntiles, s);
}

}  // namespace lmoe
