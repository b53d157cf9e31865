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
// scales are equal, at worst 2^-22.3 with scales from 2^-20 to 2^20), which is
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
// values a lane (16 or 32 bytes read, 4 written, in order); codes of nb blocks a row
// (those past cols are 0).  HBM: 8192 x 8192 bf16 in 32 us, 5.3 TB/s.
template <class T, bool VEC>
__global__ __launch_bounds__(256) void mx4_quantize_kernel(const T* __restrict__ x, long rows,
                                                           int cols, long stride, int nb,
                                                           uint32_t* __restrict__ codes,
                                                           uint8_t* __restrict__ scales) {
  const uint32_t b = blockIdx.x * 64 + threadIdx.x / 4;  // (fewer than 2^30)
  if (b >= (uint32_t)(rows * nb)) return;                // whole groups of four lanes
  const uint32_t row = b / (uint32_t)nb;
  const int i = threadIdx.x & 3;
  float v[8];
  mx4_load8<VEC>(x + row * stride, (int)(b - row * nb) * 32 + i * 8, cols, v);
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[j]));
  m = fmaxf(m, __shfl_xor(m, 1, 64));
  m = fmaxf(m, __shfl_xor(m, 2, 64));
  const int e = mx4_exponent(m);
  codes[(size_t)b * 4 + i] = mx4_pack8(v, e);
  if (i == 0) scales[b] = (uint8_t)(e + 127);
}

// The values, rounded once to T where they do not fit it: eight a lane.  HBM's writes:
// 8192 x 8192 to bf16 in 42 us, 4.0 TB/s (2, 4 or 8 blocks in flight a lane: the same).
template <class T, bool VEC>
__global__ __launch_bounds__(256) void mx4_dequantize_kernel(const uint32_t* __restrict__ codes,
                                                             const uint8_t* __restrict__ scales,
                                                             long rows, int cols, int nb,
                                                             T* __restrict__ y) {
  const uint32_t b = blockIdx.x * 64 + threadIdx.x / 4;
  if (b >= (uint32_t)(rows * nb)) return;
  const uint32_t row = b / (uint32_t)nb;
  const int i = threadIdx.x & 3;
  const int c = (int)(b - row * nb) * 32 + i * 8;
  if (c >= cols) return;
  const uint32_t w = codes[(size_t)b * 4 + i];
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
  T* yp = y + (size_t)row * cols + c;
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

template <class V>
__device__ __forceinline__ V pick(bool c, V a, V b) {
  return c ? a : b;
}

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
// the line's two scale words.  HBM and latency: 1 x 10240 x 8192 in 12.1 us (44 MB, 3.7
// TB/s: all of it is asked for at once, then a launch's start and end); 1 x 16384 x 16384
// in 30 us (4.7 TB/s).  Two or four row groups a work-group, 4 or 16 waves: 11.5 to 16.4
// us, and slower where N or K is small.
template <int NW, int RG, int U, class OUT>
__global__ __launch_bounds__(NW * 64) void mx4_stream_kernel(Mx4Gemm p) {
  __shared__ f32x4 red[NW][RG][64];
  const int nblocks = (p.N + 16 * RG - 1) / (16 * RG);
  const int nb = blockIdx.x % nblocks;
  const int tm = blockIdx.x / nblocks;
  const int m0 = tm * 16, mcount = min(16, p.M - m0);
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
    const size_t n = min(n0 + g * 16, p.N - 16);
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

// Few tokens a group: as above, but each of the NW waves takes 16 RG weight rows of
// its own over the whole of k, and everything comes through LDS by direct copies
// one line (256 values) ahead: a wave's codes (8 rows x 128 bytes a copy, with the
// non-temporal hint) into its own two slots, the 16 token rows' by the first two
// waves.  Scales come two lines at a time, 16 bytes of a row, into registers.  One
// barrier a line.  LDS rows are XOR-swizzled: row r keeps its 16-byte chunk c at c ^
// (r % 8), rows 8 to 15 of sixteen at c ^ (r % 8) ^ 1.  Work items (tile, row block) are
// taken XCD-major.  HBM: 704 rows over 512 groups of 5120 x 2048, 394 of which have any, in
// 308 us, 7.1 TB/s (into registers, as above: 480 us).
template <int NW, int RG, class OUT>
__global__ __launch_bounds__(NW * 64) void mx4_lines_kernel(Mx4Gemm p, const Tile* tiles,
                                                            const int* ntiles) {
  constexpr int ROWS = NW * 16 * RG, CSLOT = 16 * RG * 128, TSLOT = 16 * 128;
  __shared__ __attribute__((aligned(1024))) char smem[NW * 2 * CSLOT + 2 * TSLOT];
  const int nblocks = (p.N + ROWS - 1) / ROWS;
  const int nwork = uniform(*ntiles) * nblocks;
  const int b = blockIdx.x;
  if (b >= nwork) return;
  const int per = nwork / kXcds;
  const int item = b < per * kXcds ? (b % kXcds) * per + b / kXcds : b;
  const int nb = item % nblocks, tix = item / nblocks;
  const int e = uniform(tiles[tix].expert), m0 = uniform(tiles[tix].row0);
  const int mcount = uniform(tiles[tix].nrows);
  const int lane = threadIdx.x & 63;
  const int w = uniform(threadIdx.x >> 6);
  const int r16 = lane & 15, kq = lane >> 4;
  const int RB = p.K / 2, SW = p.K / 128, LT = (SW + 1) / 2;
  const int n0 = nb * ROWS + w * 16 * RG;
  constexpr uint32_t kNone = 0x80000000u;

  // Offsets are from the wave's first row (a matrix may be larger than a buffer).
  // 16-row groups past N read the last one (their columns are not stored).
  const int base = min(n0, p.N - 16);
  const __amdgpu_buffer_rsrc_t rc = buffer_rsrc(p.w + ((size_t)e * p.N + base) * RB);
  const uint32_t piece = (lane & 7) ^ (lane >> 3);
  const uint32_t clane = (uint32_t)(lane >> 3) * (uint32_t)RB + piece * 16;
  char* const cslots = smem + w * 2 * CSLOT;
  const size_t srow = ((size_t)e * p.N + base) * SW * 4;
  const __amdgpu_buffer_rsrc_t rs =
      buffer_rsrc(p.ws + srow, (size_t)p.groups * p.N * SW * 4 - srow);
  uint32_t soff[RG];
#pragma unroll
  for (int g = 0; g < RG; ++g)
    soff[g] = (uint32_t)(min(n0 + g * 16, p.N - 16) - base + r16) * (uint32_t)SW * 4u;

  // tokens: rows past the tile's count and indices outside x read as 0
  const bool gather = p.rows != nullptr;
  const uint8_t* const xbase = gather ? p.x : p.x + (size_t)m0 * RB;
  const size_t xs0 = gather ? 0 : (size_t)m0 * SW * 4;
  const __amdgpu_buffer_rsrc_t rx = buffer_rsrc(xbase);
  const __amdgpu_buffer_rsrc_t rxs = buffer_rsrc(p.xs + xs0, (size_t)p.x_rows * SW * 4 - xs0);
  auto x_row = [&](int i, bool& ok) -> uint32_t {
    ok = i < mcount;
    if (!ok) return 0;
    return gather ? (uint32_t)mx4_x_row(p, m0 + i, ok) : (uint32_t)i;
  };
  char* const tslots = smem + NW * 2 * CSLOT;
  uint32_t toff = kNone, xsoff = kNone;
  {
    bool ok;
    uint32_t row = x_row(8 * w + (lane >> 3), ok);
    if (w < 2 && ok) toff = row * (uint32_t)RB + (w ? piece ^ 1u : piece) * 16;
    row = x_row(r16, ok);
    if (ok) xsoff = row * (uint32_t)SW * 4u;
  }
  auto issue = [&](int l) __attribute__((always_inline)) {
    // the second half of a half line reads as 0
    const bool half = 2 * l + 2 > SW;
    char* const cs = cslots + (l & 1) * CSLOT;
    const uint32_t a = half && (piece & 4) ? kNone : clane;
    const uint32_t c = half && (piece & 4) ? kNone : clane ^ 16u;
#pragma unroll
    for (int g = 0; g < RG; ++g) {
      const int row = min(n0 + g * 16, p.N - 16) - base;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rc, (lds_void*)(cs + g * 2048), 16, a,
                                               row * RB + l * 128, 0, 2 /* nt */);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rc, (lds_void*)(cs + g * 2048 + 1024), 16, c,
                                               (row + 8) * RB + l * 128, 0, 2);
    }
    if (w < 2) {
      const bool none = half && ((w ? piece ^ 1u : piece) & 4);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rx, (lds_void*)(tslots + (l & 1) * TSLOT + w * 1024), 16, none ? kNone : toff, l * 128, 0,
          0);
    }
  };
  u32x4 scur[RG], snext[RG], xcur, xnext;
  auto scales = [&](int l) __attribute__((always_inline)) {
#pragma unroll
    for (int g = 0; g < RG; ++g)
      snext[g] = __builtin_amdgcn_raw_buffer_load_b128(rs, soff[g] + l * 8, 0, 0);
    xnext = __builtin_amdgcn_raw_buffer_load_b128(rxs, xsoff + l * 8, 0, 0);
  };
  f32x4 acc[RG];
#pragma unroll
  for (int g = 0; g < RG; ++g) acc[g] = f32x4{0.f, 0.f, 0.f, 0.f};

  scales(0);
  issue(0);
  const int at = (r16 >> 3) * 1024 + (r16 & 7) * 128, sz = (r16 & 7) ^ (r16 >> 3);
  const int a0 = at + ((kq ^ sz) << 4), a1 = at + (((4 + kq) ^ sz) << 4);
  for (int l = 0; l < LT; ++l) {
    // this line's copies (every wave's) have landed, and every wave is done with
    // the slots that the next line's overwrite
    wait_vmcnt<0>();
    stage_barrier_hard();
    if ((l & 1) == 0) {
#pragma unroll
      for (int g = 0; g < RG; ++g) scur[g] = snext[g];
      xcur = xnext;
    }
    if (l + 1 < LT) {
      issue(l + 1);
      if (l & 1) scales(l + 1);
    }
    const char* const cs = cslots + (l & 1) * CSLOT;
    const char* const ts = tslots + (l & 1) * TSLOT;
    const i32x4 x0 = *reinterpret_cast<const i32x4*>(ts + a0);
    const i32x4 x1 = *reinterpret_cast<const i32x4*>(ts + a1);
    const uint32_t xw0 = l & 1 ? xcur[2] : xcur[0], xw1 = l & 1 ? xcur[3] : xcur[1];
    // (a half line's second word is another row's: its values are 0, 1 will do)
    const bool half = 2 * l + 2 > SW;
    const int t0 = (int)(xw0 >> (8 * kq)), t1 = half ? 127 : (int)(xw1 >> (8 * kq));
#pragma unroll
    for (int g = 0; g < RG; ++g) {
      const i32x4 c0 = *reinterpret_cast<const i32x4*>(cs + g * 2048 + a0);
      const i32x4 c1 = *reinterpret_cast<const i32x4*>(cs + g * 2048 + a1);
      const uint32_t w0 = l & 1 ? scur[g][2] : scur[g][0], w1 = l & 1 ? scur[g][3] : scur[g][1];
      acc[g] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
          low(c0), low(x0), acc[g], 4, 4, 0, (int)(w0 >> (8 * kq)), 0, t0);
      acc[g] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
          low(c1), low(x1), acc[g], 4, 4, 0, half ? 127 : (int)(w1 >> (8 * kq)), 0, t1);
    }
  }
#pragma unroll
  for (int g = 0; g < RG; ++g) {
    const int n = n0 + g * 16;
    if (r16 < mcount && n < p.N) mx4_store4<OUT>(p, m0 + r16, n + kq * 4, acc[g]);
  }
}

// Many tokens: MFMA tiles of BM token rows x BN weight rows fed through LDS by
// direct global -> LDS copies.  A step is a line of k (128 bytes of a row, 256
// values) in two halves of the tile's weight rows; each wave owns 32 TM token
// rows and 32 TH weight rows of each half, and holds the fragments it multiplies
// in registers: a 32x32x64 MFMA takes 16 bytes of a row and lane, lane (r, h) (r =
// lane % 32, h = lane / 32) of step s the block 4 h + s of row r, whose scale is
// byte s of word h of the line's two.  A fragment's registers are read anew from
// LDS, for the next half (one set of them where there are two groups, two where
// there is one), right after their last use, so no LDS read is waited for at
// the top of a step.  During step k, LDS holds what is read in it (weight half 1 of
// k, half 0 of k + 1, token rows of k + 1), and copies run into the places of what
// step k - 1 read: token rows of k + 2 and, with a ring of WD lines of weights,
// half 1 of line k + WD - 1 and half 0 of k + WD.  One barrier a step; the copy
// instructions are spread over the MFMAs.
//
// Scales come two lines at a time (16 bytes of a row), half of the tile's rows with
// each step.
//
// Bound by the matrix instructions at the clock that the card runs them at:
// 8192 x 10240 x 8192 in 309 to 317 us (4.4 PFLOP/s; they are busy in 65% of the
// cycles, at 1.6 GHz), and by what a tile costs beside its steps, about 11 us (start
// and scales 3 to 4, first lines 3, the results' way out 4 to 6).  180224 rows over 512
// groups of 2048 x 5120: 1.33 to 1.43 ms (2.7 PFLOP/s).  Four waves with half the LDS reads,
// twice the registers: the same.  Tiles of half as many columns, two work-groups a CU: 2%
// to 29% slower in groups of 8 to 128 rows.
//
// Split over k (dense, few tiles): work-group (x, y) computes tile x over the
// y-th part of the lines and writes fp32 partial sums to part y of `y`.
template <bool GROUPED, int NW, int BM, int BN, int WM, int WD, class OUT>
__global__ __launch_bounds__(NW * 64) void mx4_pipe_kernel(Mx4Gemm p, const Tile* tiles,
                                                           const int* ntiles) {
  constexpr int BH = BN / 2, WN = NW / WM;
  constexpr int TM = BM / WM / 32, TH = BH / WN / 32, SETS = TH == 1 ? 2 : 1;
  constexpr int RPI = kFp8CopyRows, ROWB = 128;
  constexpr int NIA = BM / RPI / NW, NIH = BH / RPI / NW;  // copies a wave and unit
  constexpr int ABUF = BM * ROWB, HBUF = BH * ROWB;
  constexpr int SROWS = BM + BN;       // rows of scales
  constexpr int NST = BM / 32, NSB = BN / 32;  // copies of half of two lines' scales
  constexpr int NSW = 2;               // a wave's with each step (some twice)
  static_assert(NST <= NW && NSB <= NW, "one of each a wave");
  static_assert(TM * 32 * WM == BM && TH * 32 * WN == BH, "whole groups");
  static_assert(NIA * RPI * NW == BM && NIH * RPI * NW == BH, "rows per unit");
  // One LDS array: with several, the compiler tells them apart and then waits
  // for all copies in flight before every LDS read.
  constexpr int W00 = 2 * ABUF, S00 = W00 + 2 * WD * HBUF, LDS = S00 + 2 * SROWS * 16;
  static_assert(LDS <= 160 * 1024, "LDS");
  __shared__ __attribute__((aligned(1024))) char smem[LDS];

  int tm, nb;
  const int nblocks = (p.N + BN - 1) / BN;
  if (!work_item_uniform<GROUPED>(nblocks, p.M, BM, tiles, ntiles, tm, nb)) return;
  int e = 0, m0, mcount;
  if (GROUPED) {
    e = uniform(tiles[tm].expert);
    m0 = uniform(tiles[tm].row0);
    mcount = uniform(tiles[tm].nrows);
  } else {
    m0 = tm * BM;
    mcount = min(BM, p.M - m0);
  }
  const int n0 = nb * BN;
  const int lane = threadIdx.x & 63;
  const int w = uniform(threadIdx.x >> 6);
  const int wm = w / WN, wn = w % WN;
  const int RB = p.K / 2, SW = p.K / 128;  // bytes and scale words of a row
  const int LT = (SW + 1) / 2;             // lines of a whole row
  int k0 = 0, KL = LT;                     // this work-group's: k0 .. k0 + KL - 1
  if (!GROUPED && p.splits > 1) {
    k0 = blockIdx.y * LT / p.splits;
    KL = (blockIdx.y + 1) * LT / p.splits - k0;
    p.y = static_cast<float*>(p.y) + (size_t)blockIdx.y * p.M * p.N;
  }
  // the last line is half a line (and this work-group's)
  const int half_line = SW % 2 && k0 + KL == LT ? KL - 1 : -1;

  // Copy sources: instruction j of wave w fills rows RPI (w + NW j) .. + 7 of its
  // buffer, written already swizzled (16-byte chunk c of row r in place c ^ (r / 2)
  // % 8).  Token rows past the tile's count, rows whose index is outside x and the
  // second half of a half line are past the buffer's bound and read as 0.  Weight
  // rows past N read the matrix's last rows again (their columns are not stored).
  constexpr uint32_t kNone = 0x80000000u;
  const int lr = lane >> 3;
  const int sw = ((4 * (w & 1)) + (lr >> 1)) & 7;
  static_assert(NW % 2 == 0, "the swizzle of a wave's rows");
  const uint32_t chunk = (uint32_t)(((lane & 7) ^ sw) * 16);
  const bool gather = p.rows != nullptr;
  const __amdgpu_buffer_rsrc_t ra =
      buffer_rsrc((gather ? p.x : p.x + (size_t)m0 * RB) + k0 * ROWB);
  const size_t w0 = ((size_t)e * p.N + n0) * RB + k0 * ROWB;
  const __amdgpu_buffer_rsrc_t rb = buffer_rsrc(p.w + w0);
  auto x_row = [&](int i, bool& ok) -> uint32_t {
    ok = i < mcount;
    if (!ok) return 0;
    return gather ? (uint32_t)mx4_x_row(p, m0 + i, ok) : (uint32_t)i;
  };
  uint32_t ao[NIA], bo = fp8_weight_lane(lane, chunk, (uint32_t)RB);
#pragma unroll
  for (int j = 0; j < NIA; ++j) {
    bool ok;
    const uint32_t row = x_row(RPI * (w + NW * j) + lr, ok);
    ao[j] = ok ? row * (uint32_t)RB + chunk : kNone;
    asm volatile("" : "+v"(ao[j]));  // one register: not half of a 64-bit product
  }
  asm volatile("" : "+v"(bo));
  const bool upper = chunk >= 64;  // of a half line, what is not there
  auto copy_x = [&](int k, int j) __attribute__((always_inline)) {
    const uint32_t at = k == half_line && upper ? kNone : ao[j];
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        ra, (lds_void*)(smem + (k & 1) * ABUF + (w + NW * j) * RPI * ROWB), 16, at, k * ROWB, 0, 0);
  };
  // weight half h of line k, to ring offset r
  auto copy_w = [&](int k, int h, int r, int j) __attribute__((always_inline)) {
    const uint32_t at = k == half_line && upper ? kNone : bo;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        rb, (lds_void*)(smem + W00 + r + h * HBUF + (w + NW * j) * RPI * ROWB), 16, at,
        fp8_weight_scalar(h * BH + (w + NW * j) * RPI, p.N - n0, k, RB), 0, 0);
  };
  // Scales of lines 2 g and 2 g + 1: rows 0 .. BM - 1 are the tokens', then the
  // weights'.  A copy fills 16 rows, lane l row l / 4, place l % 4, which holds word
  // (l % 4) ^ 2 (i % 2) of the four, i the row / 16 (so that 32 rows' reads of a line
  // meet no bank twice).  With half j a wave copies the (w % NST)-th of that half of
  // the tokens' rows and the (w % NSB)-th of the weights'.  Words past K and rows
  // that are not there read as 0.
  const __amdgpu_buffer_rsrc_t rxs = buffer_rsrc(gather ? p.xs : p.xs + (size_t)m0 * SW * 4);
  const __amdgpu_buffer_rsrc_t rws = buffer_rsrc(p.ws + ((size_t)e * p.N + n0) * SW * 4);
  const int wt = w % NST, wb = w % NSB;
  uint32_t so[2];  // the token row's offset
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    bool ok;
    const uint32_t row = x_row(16 * (j * NST + wt) + (lane >> 2), ok);
    so[j] = ok ? row * (uint32_t)SW * 4u : kNone;
    asm volatile("" : "+v"(so[j]));
  }
  // (words from the row's start; lines are counted from k0)
  auto word_of = [&](int g, int id) __attribute__((always_inline)) {
    return (uint32_t)(2 * k0 + 4 * g) + (uint32_t)((lane & 3) ^ ((id & 1) << 1));
  };
  auto copy_st = [&](int g, int j, uint32_t off) __attribute__((always_inline)) {
    const int id = j * NST + wt;
    // (past the bound: kNone and whatever is added to it)
    const uint32_t word = word_of(g, id), sum = off + word * 4u;
    const uint32_t at = word < (uint32_t)SW ? sum : kNone;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        rxs, (lds_void*)(smem + S00 + ((g & 1) * SROWS + 16 * id) * 16), 4, at, 0, 0, 0);
  };
  auto copy_sw = [&](int g, int j) __attribute__((always_inline)) {
    const int id = j * NSB + wb, row = 16 * id + (lane >> 2);
    const uint32_t word = word_of(g, id);
    const uint32_t sum = ((uint32_t)row * (uint32_t)SW + word) * 4u;
    const uint32_t at = ((n0 + row < p.N) & (word < (uint32_t)SW)) ? sum : kNone;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        rws, (lds_void*)(smem + S00 + ((g & 1) * SROWS + BM + 16 * id) * 16), 4, at, 0, 0, 0);
  };
  // what the first MFMAs need, then what step 0 reads, then what it need not
  // wait for
  constexpr int R = 2 * HBUF;  // a line's place in the ring of weights
#pragma unroll
  for (int j = 0; j < NIA; ++j) copy_x(0, j);
#pragma unroll
  for (int j = 0; j < NIH; ++j) copy_w(0, 0, 0, j);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    copy_st(0, j, so[j]);
    copy_sw(0, j);
  }
#pragma unroll
  for (int j = 0; j < NIH; ++j) copy_w(0, 1, 0, j);
  if (KL > 1) {
#pragma unroll
    for (int j = 0; j < NIH; ++j) copy_w(1, 0, R, j);
#pragma unroll
    for (int j = 0; j < NIA; ++j) copy_x(1, j);
    copy_st(1, 0, so[0]);
    copy_sw(1, 0);
    if constexpr (WD == 3) {
#pragma unroll
      for (int j = 0; j < NIH; ++j) copy_w(1, 1, R, j);
      if (KL > 2) {
#pragma unroll
        for (int j = 0; j < NIH; ++j) copy_w(2, 0, 2 * R, j);
      }
    }
  }

  const int r32 = lane & 31, kh = lane >> 5;
  uint32_t lo[4];  // a lane's place of block 4 h + s in a 32-row group
#pragma unroll
  for (int s = 0; s < 4; ++s) lo[s] = r32 * ROWB + (((4 * kh + s) ^ ((r32 >> 1) & 7)) << 4);
  const uint32_t aw = (uint32_t)(wm * (BM / WM)) * ROWB;
  const uint32_t bw = (uint32_t)(W00 + wn * (BH / WN) * ROWB);
  f32x16 acc[2 * TH][TM];
#pragma unroll
  for (int a = 0; a < 2 * TH; ++a)
#pragma unroll
    for (int b = 0; b < TM; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[a][b][i] = 0.f;

  struct Frag {
    i32x4 v[4];
  };
  // fragments: token group t of line k, weight group g at ring offset r
  auto read_x1 = [&](int k, int t, int s) __attribute__((always_inline)) {
    return *reinterpret_cast<const i32x4*>(smem + (k & 1) * ABUF + aw + t * 32 * ROWB + lo[s]);
  };
  auto read_w1 = [&](int r, int g, int s) __attribute__((always_inline)) {
    return *reinterpret_cast<const i32x4*>(smem + bw + r + g * 32 * ROWB + lo[s]);
  };
  auto read_x = [&](int k, int t) __attribute__((always_inline)) {
    Frag f;
#pragma unroll
    for (int s = 0; s < 4; ++s) f.v[s] = read_x1(k, t, s);
    return f;
  };
  auto read_w = [&](int r, int g) __attribute__((always_inline)) {
    Frag f;
#pragma unroll
    for (int s = 0; s < 4; ++s) f.v[s] = read_w1(r, g, s);
    return f;
  };
  // the word of scales of row `row` (a multiple of 32 and the lane's) for line k
  const uint32_t sl = (uint32_t)(S00 + r32 * 16 + kh * 4), sx = r32 >> 4;
  auto read_s = [&](int k, int row) __attribute__((always_inline)) {
    return *reinterpret_cast<const int*>(smem + sl + ((k >> 1) & 1) * (SROWS * 16) + row * 16 +
                                         (((k & 1) ^ sx) << 3));
  };
  Frag xf[TM], wf[SETS][TH];
  int xs[TM], ws[2 * TH];

  int r0 = 0;  // ring offset of line k
  // Step k.  COPY: 2 copies everything (k + WD < KL), 1 all but the weights of
  // line k + WD (the last step with copies), 0 nothing.
  auto step = [&](auto copy_c, int k) __attribute__((always_inline)) {
    constexpr int COPY = decltype(copy_c)::value;
    const int r1 = r0 + R == WD * R ? 0 : r0 + R;
    const int r2 = r1 + R == WD * R ? 0 : r1 + R;  // r0 when WD = 2
    // what this step reads has landed (with WD = 3 the weight copies of the
    // last step may be in flight), and this wave's LDS reads of the last step
    // are done; then the same for every wave
    if (WD == 3 && COPY) wait_vmcnt<2 * NIH>();
    else wait_vmcnt<0>();
    wait_lgkmcnt0();
    stage_barrier_hard();
    // half j of group g of the scales comes with step 2 g - 3 + j, so that group g,
    // first read in step 2 g - 1, is whole then, and what it replaces, group g - 2,
    // was last read in step 2 g - 4
    constexpr bool XC = COPY == 2 || (COPY == 1 && WD == 3);  // line k + 2 exists
    constexpr int NX = XC ? NIA + NSW : 0;
    constexpr int NC = NX + (COPY == 2 ? 2 * NIH : (COPY == 1 ? NIH : 0));
    constexpr int X0 = WD == 2 ? NC - NX : 0, W0 = WD == 2 ? 0 : NX;
    const int part = (k + 1) & 1;
    const uint32_t sof = pick(part != 0, so[1], so[0]);
    auto copy = [&](int c) __attribute__((always_inline)) {
      if (c >= X0 && c < X0 + NIA && XC) copy_x(k + 2, c - X0);
      else if (XC && c == X0 + NIA) copy_st((k + 3) >> 1, part, sof);
      else if (XC && c == X0 + NIA + 1) copy_sw((k + 3) >> 1, part);
      else if (c < W0 + NIH) copy_w(k + WD - 1, 1, WD == 2 ? r1 : r2, c - W0);
      else copy_w(k + WD, 0, r0, c - W0 - NIH);
    };
    constexpr int NP = TM * TH * 4;  // MFMAs of a half
    constexpr int EVERY = NC <= NP ? 2 : 1;
    static_assert(NC <= 2 * NP, "copies");
#pragma unroll
    for (int i = 0; i < 2 * NP; ++i) {
      // (neighbouring products go to different sums)
      const int h = i / NP, g = i % NP / (4 * TM), s = i % (4 * TM) / TM, t = i % TM;
      const int a = h * TH + g;
      if (SETS == 2 && i % NP == 0) wf[1 - h][0] = read_w(h == 0 ? r0 + HBUF : r1, 0);
      const i32x8 av = low(wf[SETS == 2 ? h : 0][g].v[s]), bv = low(xf[t].v[s]);
#define LMOE_MFMA(S) \
  __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, acc[a][t], 4, 4, S, ws[a], S, xs[t])
      acc[a][t] = s == 0 ? LMOE_MFMA(0) : s == 1 ? LMOE_MFMA(1) : s == 2 ? LMOE_MFMA(2) : LMOE_MFMA(3);
#undef LMOE_MFMA
      // keeps the product here
      asm volatile("" : "+v"(acc[a][t]));
      if (SETS == 1 && t == TM - 1) wf[0][g].v[s] = read_w1(h == 0 ? r0 + HBUF : r1, g, s);
      if (h == 1 && g == TH - 1) {
        xf[t].v[s] = read_x1(k + 1, t, s);
        if (s == 3) xs[t] = read_s(k + 1, wm * (BM / WM) + t * 32);
      }
      if (t == TM - 1 && s == 3) ws[a] = read_s(k + 1, BM + h * BH + wn * (BH / WN) + g * 32);
      if (i % EVERY == 0 && i / EVERY < NC) copy(i / EVERY);
      __builtin_amdgcn_sched_barrier(0);
    }
    r0 = r1;
  };
  if (KL > 2) wait_vmcnt<(WD == 3 ? 4 : 2) * NIH + NIA + NSW>();
  else wait_vmcnt<0>();
  stage_barrier_hard();
#pragma unroll
  for (int t = 0; t < TM; ++t) {
    xf[t] = read_x(0, t);
    xs[t] = read_s(0, wm * (BM / WM) + t * 32);
  }
#pragma unroll
  for (int g = 0; g < TH; ++g) wf[0][g] = read_w(0, g);
#pragma unroll
  for (int b = 0; b < 2 * TH; ++b)
    ws[b] = read_s(0, BM + (b / TH) * BH + wn * (BH / WN) + (b % TH) * 32);
  int k = 0;
  for (; k + WD < KL; ++k) step(std::integral_constant<int, 2>{}, k);
  if (k + WD - 1 < KL) step(std::integral_constant<int, 1>{}, k++);
  for (; k < KL; ++k) step(std::integral_constant<int, 0>{}, k);
  // the last step read ahead (values that are not used): let the reads end
  // before the buffers are written below
  wait_lgkmcnt0();
  stage_barrier_hard();

  // Lane (r, h) holds, in registers 4 v .. + 3 of a group, columns 8 v + 4 h .. + 3 of
  // token r.  They leave through LDS, in the wave's own region, as whole pieces of
  // rows of 32 columns (16-byte chunk c of row r in place c ^ r % chunks).
  constexpr int EL = std::is_same<OUT, float>::value ? 4 : 2;
  constexpr int RBO = 32 * EL, CH = RBO / 16, RPS = 64 / CH;  // row bytes, chunks; rows a store
  static_assert(NW * 32 * RBO <= 2 * ABUF + 2 * WD * HBUF, "staging room");
  char* const reg = smem + w * 32 * RBO;
#pragma unroll
  for (int a = 0; a < 2 * TH; ++a)
#pragma unroll
    for (int t = 0; t < TM; ++t) {
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const f32x4 q = {acc[a][t][4 * v], acc[a][t][4 * v + 1], acc[a][t][4 * v + 2],
                         acc[a][t][4 * v + 3]};
        const int c = EL == 4 ? 2 * v + kh : v;
        char* const to = reg + r32 * RBO + ((c ^ (r32 & (CH - 1))) << 4);
        if constexpr (EL == 4) *reinterpret_cast<f32x4*>(to) = q;
        else *reinterpret_cast<u16x4*>(to + kh * 8) = pack4_bf16(q);
      }
      const int n = n0 + (a / TH) * BH + wn * (BH / WN) + (a % TH) * 32;
      const int c = lane & (CH - 1);
#pragma unroll
      for (int j = 0; j < 32 / RPS; ++j) {
        const int row = j * RPS + lane / CH, i = wm * (BM / WM) + t * 32 + row;
        const u32x4 q =
            *reinterpret_cast<const u32x4*>(reg + row * RBO + ((c ^ (row & (CH - 1))) << 4));
        if (i < mcount && n + c * (16 / EL) < p.N)
          *reinterpret_cast<u32x4*>(static_cast<OUT*>(p.y) + (size_t)(m0 + i) * p.N + n +
                                    c * (16 / EL)) = q;
      }
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

// How a product runs.
struct Plan {
  bool stream;  // weight streaming, else LDS-tiled
  int bm;       // token rows of a tile
  int splits;   // of k (dense tiles)
};

// Grouped: rows per group on average decide.  512 groups of 5120 x 2048, Poisson counts:
// 16 rows at a time 438 us at 6 rows on average, 490 at 10, 533 at 12, 689 at 16; tiles of
// 64 rows 521, 558, 557, 575.  Tiles of 64, 128 and 192 rows take times like `cost`, and
// a group's last one is wasted in part: 0.4 of one on average, at least one a group.
Plan grouped_plan(int rows, int groups) {
  if (rows <= 10L * groups) return {true, kStreamTileM, 1};
  const double r = (double)rows / groups;
  const int bm[3] = {64, 128, 192};
  const double cost[3] = {1.0, 1.25, 1.675};
  int best = 0;
  double least = 0;
  for (int i = 0; i < 3; ++i) {
    const double n = r / bm[i] + 0.4;
    const double c = (n > 1 ? n : 1.0) * cost[i];
    if (i == 0 || c < least) best = i, least = c;
  }
  return {false, bm[best], 1};
}

// Dense: the tile shape and the split of k with the least estimated time, or, up to
// 16 rows, the stream where that is less.  Estimates are lines of measurements (N x K
// weights in MB, a call of M rows): the stream 42 MB 12.1 us at M = 1, 16.5 at 8, 20.2
// at 16; 134 MB (16384 x 16384) 30.1, 40.9, 50.0 (each work-group reads all tokens for 16
// weight rows); 8 MB 7.6 to 8.6.  The tiles at any M up to 64: 42 MB 16.2, 134 MB 27.4,
// 8 MB 10.7 to 11.8 (k split in most, and added up by a second kernel).
struct DenseTile {
  int bm, bn;
};
constexpr DenseTile kDenseTiles[3] = {{256, 256}, {128, 256}, {64, 128}};
// A line of 256 k of n tiles, us: of 256 tiles at a time 1.7 and 1.0; of the smallest 0.6,
// two work-groups a CU, and no less than 0.8.
double tile_us(const DenseTile& t, long n) {
  if (t.bm == 64) return n * (0.6 / 256) > 0.8 ? n * (0.6 / 256) : 0.8;
  return (double)((n + 255) / 256) * (t.bm == 256 ? 1.7 : 1.0);
}
double stream_us(int M, int N, int K) {
  return 7.5 + 0.5e-6 * N * K * (0.196 + 0.011 * (M - 1));
}
Plan dense_plan(int M, int N, int K) {
  const int lines = (K + 255) / 256;
  Plan best{};
  double least = 0;
  for (const DenseTile& t : kDenseTiles) {
    for (int s = 1; s <= 8; s *= 2) {
      if (s > 1 && lines / s < 4) continue;  // a part is at least four lines
      const long n = (long)((M + t.bm - 1) / t.bm) * ((N + t.bn - 1) / t.bn) * s;
      double us = tile_us(t, n) * ((lines + s - 1) / s) + 8.0;
      if (s > 1) us += 4.0 + (double)s * M * N * 8 / 4e6;
      if (best.bm == 0 || us < least) best = {false, t.bm, s}, least = us;
    }
  }
  if (M <= 16 && stream_us(M, N, K) < least) best = {true, kStreamTileM, 1};
  return best;
}

Plan make_plan(int M, int N, int K, int groups) {
  return groups ? grouped_plan(M, groups) : dense_plan(M, N, K);
}

int grouped_tiles(int rows, int groups, int tile_m) {
  return (rows < groups ? rows : groups) + rows / tile_m + 1;
}

long xcd_grid(long work) { return kXcds * ((work + kXcds - 1) / kXcds); }

// Work-groups and threads of a product's launch.
constexpr int kGroupedWaves = 4, kGroupedRG = 2, kDenseWaves = 8, kDenseRG = 1;
long grid_of(const Plan& plan, int M, int N, int groups, int* threads) {
  const long tiles = groups ? grouped_tiles(M, groups, plan.bm) : (M + plan.bm - 1) / plan.bm;
  if (plan.stream) {
    const int rows = groups ? 16 * kGroupedWaves * kGroupedRG : 16 * kDenseRG;
    *threads = 64 * (groups ? kGroupedWaves : kDenseWaves);
    return tiles * ((N + rows - 1) / rows);
  }
  const bool small = !groups && plan.bm == 64;
  *threads = small ? 256 : 512;
  const int bn = small ? 128 : 256;
  return xcd_grid(tiles * ((N + bn - 1) / bn));
}

template <class OUT>
hipError_t launch(const Mx4Gemm& p, const Plan& plan, const Tile* tiles, const int* ntiles,
                  hipStream_t s) {
  int threads;
  const long grid = grid_of(plan, p.M, p.N, p.groups, &threads);
  if (too_many(grid, threads)) return hipErrorInvalidConfiguration;
  const dim3 g(grid, p.splits);
  if (plan.stream) {
    if (p.groups)
      mx4_lines_kernel<kGroupedWaves, kGroupedRG, OUT><<<g, threads, 0, s>>>(p, tiles, ntiles);
    else
      mx4_stream_kernel<kDenseWaves, kDenseRG, 2, OUT><<<g, threads, 0, s>>>(p);
  } else if (p.groups) {
    if (plan.bm == 64)
      mx4_pipe_kernel<true, 8, 64, 256, 2, 3, OUT><<<g, threads, 0, s>>>(p, tiles, ntiles);
    else if (plan.bm == 128)
      mx4_pipe_kernel<true, 8, 128, 256, 2, 3, OUT><<<g, threads, 0, s>>>(p, tiles, ntiles);
    else
      mx4_pipe_kernel<true, 8, 192, 256, 2, 3, OUT><<<g, threads, 0, s>>>(p, tiles, ntiles);
  } else {
    if (plan.bm == 64)
      mx4_pipe_kernel<false, 4, 64, 128, 2, 3, OUT><<<g, threads, 0, s>>>(p, nullptr, nullptr);
    else if (plan.bm == 128)
      mx4_pipe_kernel<false, 8, 128, 256, 2, 3, OUT><<<g, threads, 0, s>>>(p, nullptr, nullptr);
    else
      mx4_pipe_kernel<false, 8, 256, 256, 4, 2, OUT><<<g, threads, 0, s>>>(p, nullptr, nullptr);
  }
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
  p.splits = plan.splits;
  if (plan.splits > 1) {
    void* const y = p.y;
    p.y = ws;
    const hipError_t e = launch<float>(p, plan, nullptr, nullptr, s);
    if (e != hipSuccess) return e;
    return add_parts(static_cast<const float*>(ws), plan.splits, (long)p.M * p.N, y, out_bf16, s);
  }
  return out_bf16 ? launch<uint16_t>(p, plan, tiles, ntiles, s)
                  : launch<float>(p, plan, tiles, ntiles, s);
}

}  // namespace lmoe
