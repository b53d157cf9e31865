// What the FP4 matrix instructions do: their sums against 64 bits, and their rate
// in a loop of registers.
//
//   hipcc --offload-arch=gfx950 -O3 -Xclang -target-feature -Xclang -packed-fp32-ops
//       profiles/mxfp4_instruction.hip -o mxfp4_instruction && ./mxfp4_instruction
//
// Sums: 4096 products of a 16 x 128 and a 128 x 16 matrix of random codes, each block
// of 32 with a scale of its own, 2^-s to 2^s, onto a C of 0 or of random numbers, twice
// each; the error of each of the 256 results over the sum of its terms' magnitudes.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstdio>
#include <random>
#include <string>
#include <vector>

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

#define CHECK(x)                                             \
  do {                                                       \
    const hipError_t e = (x);                                \
    if (e != hipSuccess) {                                   \
      std::printf("%s: %s\n", #x, hipGetErrorString(e));     \
      return 1;                                              \
    }                                                        \
  } while (0)

__device__ i32x8 low(i32x4 a) { return __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1); }

// Work-group t (64 threads): D = A B + C of the t-th matrices.  Lane (r, q), r = lane %
// 16, q = lane / 16, holds block q of row r of A and of column r of B, and rows 4 q ..
// + 3 of column r of C and D.
__global__ void sums(const uint8_t* a, const uint8_t* b, const uint8_t* sa, const uint8_t* sb,
                     const float* c, float* d) {
  const int lane = threadIdx.x, r = lane & 15, q = lane >> 4;
  const size_t t = blockIdx.x;
  const i32x4 av = *reinterpret_cast<const i32x4*>(a + t * 1024 + r * 64 + q * 16);
  const i32x4 bv = *reinterpret_cast<const i32x4*>(b + t * 1024 + r * 64 + q * 16);
  const f32x4 cv = *reinterpret_cast<const f32x4*>(c + t * 256 + lane * 4);
  *reinterpret_cast<f32x4*>(d + t * 256 + lane * 4) =
      __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(low(av), low(bv), cv, 4, 4, 0,
                                                       sa[t * 64 + r * 4 + q], 0,
                                                       sb[t * 64 + r * 4 + q]);
}

// n rounds of four (32 x 32 x 64) or eight (16 x 16 x 128) products of each wave's own.
template <bool WIDE>
__global__ __launch_bounds__(256) void rate(float* out, int n) {
  const i32x4 a = {(int)threadIdx.x * 0x1234567, 0x11223344, 0x51525354, 0x22222222}, b = a + 1;
  const int s = 0x7f7f7f7f;
  float r = 0.f;
  if constexpr (WIDE) {
    f32x16 c[4] = {};
    for (int k = 0; k < n; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        c[i] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(low(a), low(b), c[i], 4, 4, 0, s, 0, s);
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 16; ++j) r += c[i][j];
  } else {
    f32x4 c[8] = {};
    for (int k = 0; k < n; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        c[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(low(a), low(b), c[i], 4, 4, 0, s, 0, s);
    for (int i = 0; i < 8; ++i) r += c[i][0] + c[i][1] + c[i][2] + c[i][3];
  }
  out[blockIdx.x * 256 + threadIdx.x] = r;
}

int main() {
  constexpr int T = 4096;
  static const double mag[8] = {0, .5, 1, 1.5, 2, 3, 4, 6};
  std::mt19937 g(1);
  std::normal_distribution<double> normal;
  uint8_t *da, *db, *dsa, *dsb;
  float *dc, *dd;
  CHECK(hipMalloc(&da, T * 1024));
  CHECK(hipMalloc(&db, T * 1024));
  CHECK(hipMalloc(&dsa, T * 64));
  CHECK(hipMalloc(&dsb, T * 64));
  CHECK(hipMalloc(&dc, T * 1024));
  CHECK(hipMalloc(&dd, T * 1024));
  const int spread[5] = {0, 2, 8, 12, 20};
  for (int mode = 0; mode < 20; ++mode) {
    std::vector<uint8_t> a(T * 1024), b(T * 1024), sa(T * 64), sb(T * 64);
    std::vector<float> c(T * 256), d(T * 256);
    for (auto& v : a) v = (uint8_t)g();
    for (auto& v : b) v = (uint8_t)g();
    const int w = spread[mode / 4];
    const bool onto = mode % 2;
    for (auto* s : {&sa, &sb})
      for (auto& v : *s) v = (uint8_t)(127 - w + (int)(g() % (2 * w + 1)));
    for (auto& v : c) v = onto ? (float)(normal(g) * 200) : 0.f;
    CHECK(hipMemcpy(da, a.data(), a.size(), hipMemcpyHostToDevice));
    CHECK(hipMemcpy(db, b.data(), b.size(), hipMemcpyHostToDevice));
    CHECK(hipMemcpy(dsa, sa.data(), sa.size(), hipMemcpyHostToDevice));
    CHECK(hipMemcpy(dsb, sb.data(), sb.size(), hipMemcpyHostToDevice));
    CHECK(hipMemcpy(dc, c.data(), c.size() * 4, hipMemcpyHostToDevice));
    sums<<<T, 64>>>(da, db, dsa, dsb, dc, dd);
    CHECK(hipGetLastError());
    CHECK(hipMemcpy(d.data(), dd, d.size() * 4, hipMemcpyDeviceToHost));
    double worst = 0;
    long exact = 0, n = 0;
    for (int t = 0; t < T; ++t)
      for (int l = 0; l < 64; ++l)
        for (int v = 0; v < 4; ++v, ++n) {
          const int row = 4 * (l >> 4) + v, col = l & 15;
          double s = c[t * 256 + l * 4 + v], m = std::fabs(s);
          for (int k = 0; k < 128; ++k) {
            const int p = a[t * 1024 + row * 64 + k / 2] >> 4 * (k & 1) & 15;
            const int q = b[t * 1024 + col * 64 + k / 2] >> 4 * (k & 1) & 15;
            const int e = sa[t * 64 + row * 4 + k / 32] + sb[t * 64 + col * 4 + k / 32] - 254;
            const double x = std::ldexp(mag[p & 7] * mag[q & 7], e);
            s += (p ^ q) & 8 ? -x : x;
            m += x;
          }
          const double err = std::fabs(d[t * 256 + l * 4 + v] - s);
          exact += (float)s == d[t * 256 + l * 4 + v];
          if (err > worst * m) worst = err / m;
        }
    std::printf("scales 2^%d to 2^%d, C %s: worst error %s of the magnitudes, correctly rounded %.2f%%\n",
                -w, w, onto ? "normal x 200" : "0",
                worst > 0 ? ("2^" + std::to_string(std::log2(worst))).c_str() : "0", 100.0 * exact / n);
    std::fflush(stdout);
  }
  hipEvent_t e0, e1;
  CHECK(hipEventCreate(&e0));
  CHECK(hipEventCreate(&e1));
  for (int wide = 0; wide < 2; ++wide)
    for (int rep = 0; rep < 3; ++rep) {
      const int n = 20000;
      CHECK(hipEventRecord(e0));
      if (wide) rate<true><<<512, 256>>>(dd, n);
      else rate<false><<<512, 256>>>(dd, n);
      CHECK(hipEventRecord(e1));
      CHECK(hipEventSynchronize(e1));
      float ms;
      CHECK(hipEventElapsedTime(&ms, e0, e1));
      const double flops = 512.0 * 4 * n * (wide ? 4 * 2.0 * 32 * 32 * 64 : 8 * 2.0 * 16 * 16 * 128);
      std::printf("%s: %.2f ms, %.2f PFLOP/s\n", wide ? "32 x 32 x 64" : "16 x 16 x 128", ms,
                  flops / ms / 1e12);
      std::fflush(stdout);
    }
  return 0;
}
