// Host-side launchers of the gfx950 kernels (each defined next to its kernel).
// All launchers enqueue on `s` and return hipGetLastError() of the launch.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace lmoe {

struct ProjIn;
struct ProjOut;
struct ExpUp;
struct ExpDown;
struct ExpUpMx;
struct ExpDownMx;
struct Tile;

// Weight-streaming GEMMs (few tokens; expert tiles of 16 rows).
hipError_t stream_proj_in(const ProjIn& p, hipStream_t s);
hipError_t stream_proj_out(const ProjOut& p, hipStream_t s);
hipError_t stream_exp_up(const ExpUp& p, const Tile* tiles, const int* ntiles, int max_tiles,
                         hipStream_t s);
// rows_per_expert: the batch's average rows per expert, ceil(T K / E) (it
// picks the launch shape)
hipError_t stream_exp_down(const ExpDown& p, const Tile* tiles, const int* ntiles, int max_tiles,
                           int rows_per_expert, hipStream_t s);
constexpr int kStreamTileM = 16;
// Dense GEMMs stream weights for batches of at most this many tokens.
constexpr int kStreamDenseMaxTokens = 64;

// LDS-tiled MFMA GEMMs (many tokens; expert tiles of tiled_block_m() rows;
// every N must be a multiple of tiled_block_n()).
hipError_t tiled_proj_in(const ProjIn& p, hipStream_t s);
hipError_t tiled_proj_out(const ProjOut& p, hipStream_t s);
// tokens: the batch's token count (every gathered latent row index is below it)
hipError_t tiled_exp_up(const ExpUp& p, const Tile* tiles, const int* ntiles, int max_tiles,
                        int tokens, hipStream_t s);
hipError_t tiled_exp_down(const ExpDown& p, const Tile* tiles, const int* ntiles, int max_tiles,
                          hipStream_t s);
int tiled_block_m();
int tiled_block_n();

// Split-k LDS-tiled dense GEMMs for mid-sized batches (T <= kSplitMaxTokens):
// up to kSplitMax fp32 partial [T, N] arrays in `part`, then a fixed-order
// reduction that runs the problem's epilogue.  Same dimension requirements as
// the tiled GEMMs.
constexpr int kSplitMax = 8;
constexpr int kSplitMaxTokens = 256;
hipError_t split_proj_in(const ProjIn& p, float* part, hipStream_t s);
hipError_t split_proj_out(const ProjOut& p, float* part, hipStream_t s);

// MXFP4 expert weights: quantiser (rows x cols bf16 -> codes rows x cols/2,
// scales rows x cols/32; cols a multiple of 32) and the weight-streaming
// expert GEMMs (K a multiple of 128, N a multiple of 64).
hipError_t mxfp4_quantize(const uint16_t* w, long rows, int cols, uint8_t* codes,
                          uint8_t* scales, hipStream_t s);
// tokens as for tiled_exp_up, rows_per_expert as for stream_exp_down
hipError_t stream_mx_exp_up(const ExpUpMx& p, const Tile* tiles, const int* ntiles,
                            int max_tiles, int tokens, int rows_per_expert, hipStream_t s);
hipError_t stream_mx_exp_down(const ExpDownMx& p, const Tile* tiles, const int* ntiles,
                              int max_tiles, hipStream_t s);
// The LDS-tiled expert GEMMs with MXFP4 weights (large batches; same
// dimension requirements and tile list as tiled_exp_up / tiled_exp_down).
hipError_t tiled_mx_exp_up(const ExpUpMx& p, const Tile* tiles, const int* ntiles, int max_tiles,
                           int tokens, hipStream_t s);
hipError_t tiled_mx_exp_down(const ExpDownMx& p, const Tile* tiles, const int* ntiles,
                             int max_tiles, hipStream_t s);

// Router: fp32 logits, then per token sigmoid / bias / top-K / weights.  The
// logits GEMM may split k over router_splits(T, E, R) partial [T, E] arrays
// (logits must hold that many); router_select adds them in split order.
// Splitting happens only for T <= router_split_max_tokens(), into at most
// router_max_splits() parts.
constexpr int router_max_splits() { return 8; }
constexpr int router_split_max_tokens() { return 1024; }
int router_splits(int T, int E, int R);
hipError_t router_logits(const float* z, const float* wg, float* logits, int T, int E, int R,
                         hipStream_t s);
// n_group > 1: group-limited selection (at most 64 groups, one per lane).
hipError_t router_select(const float* logits, const float* bias, int T, int E, int R, int K,
                         int n_group, int topk_group, float rho, int32_t* idx, float* w,
                         hipStream_t s);

// Routing from given logits [T, E] (rows `stride` elements apart, fp32 or
// bf16) and the gradient of its weights; T >= 1, E <= 1024, K <= 64,
// n_group <= 64 equal groups, best 1 or 2 (with best 2 and n_group > 1,
// groups of at least two).
struct RouteProblem {
  int T, E, K, n_group, topk_group, best, softmax, renorm;
  float rho;
  long stride;
};
hipError_t route_logits(const RouteProblem& r, const void* logits, bool bf16, const float* bias,
                        int32_t* idx, float* w, hipStream_t s);
hipError_t route_logits_backward(const RouteProblem& r, const void* logits, bool bf16,
                                 const int32_t* idx, const float* dw, void* dlogits,
                                 hipStream_t s);

// Grouping by expert: counts[E], offsets[E+1], rows_tok[T*K], inv[T*K] and
// the tile list (tiles of at most tile_m rows) with its length in *ntiles.
// blockcnt is scratch of ceil(T/64) * E ints.
hipError_t dispatch(const int32_t* idx, int T, int K, int E, int32_t* blockcnt, int32_t* counts,
                    int32_t* offsets, int32_t* rows_tok, int32_t* inv, Tile* tiles,
                    int32_t* ntiles, int tile_m, hipStream_t s);

// The block's pre-norm for T tokens of width D (a multiple of 8): xt =
// bf16(gamma * h) [T, D] and rn = 1 / sqrt(mean(h^2) + eps) [T].
hipError_t prenorm(const uint16_t* h, const uint16_t* gamma, int T, int D, float eps,
                   uint16_t* xt, float* rn, hipStream_t s);

// The norms around a block with its gate and residual scale, and their
// gradients.  T >= 1, 1 <= D <= block_norm_max_width(); h and y may have row
// strides, every other [T, D] array is dense.  A null y is 0; null post: y is
// not normalised; null x / dx: no second norm; null alpha, pre: ones.
struct NormParam {
  const void* p;
  int bf16;
};
struct BlockNormProblem {
  const void* h;
  const void* y;
  long h_stride, y_stride;
  bool h_bf16, y_bf16;
  NormParam pre, post, alpha, gate;
  int gate_kind;  // 0 none, 1 [D], 2 [T], 3 [T, D]
  int T, D;
  float eps;
};
struct BlockNormGrads {
  const float* stats;  // [T, 2] of the forward
  const void* dh_out;
  const void* dx;
  // wanted gradients, in their inputs' types; null: not computed
  void *dh, *dy, *dpre, *dpost, *dalpha, *dgate;
};
int block_norm_max_width();
hipError_t block_norm(const BlockNormProblem& b, void* h_out, void* x, float* stats,
                      hipStream_t s);
// bytes of the partial column sums of `nsums` column outputs
size_t block_norm_backward_part(int T, int D, int nsums);
hipError_t block_norm_backward(const BlockNormProblem& b, const BlockNormGrads& g, float* part,
                               hipStream_t s);

// 8-bit floating point (e4m3) with fp32 scales of blocks of 128 along k.
// Activations [rows, cols] (rows `stride` apart): a scale for each block of a
// row, scales [rows, ceil(cols / 128)].  Weights [matrices, rows, cols]: a
// scale for each 128 x 128 block, scales [matrices, ceil(rows / 128),
// ceil(cols / 128)].
hipError_t fp8_quantize(const void* x, bool bf16, long rows, int cols, long stride,
                        uint8_t* codes, float* scales, hipStream_t s);
hipError_t fp8_quantize_weight(const void* w, bool bf16, long matrices, int rows, int cols,
                               uint8_t* codes, float* scales, hipStream_t s);
// y[m] = x[rows ? rows[m] : m] w^T, K a multiple of 128, N of 16.  groups = 0:
// one weight matrix for all M rows; else row m takes the matrix of the group
// whose range offsets[g] .. offsets[g + 1] - 1 holds it (rows of no group are
// not written).
constexpr int kFp8MaxBlocks = 256;  // blocks of k that the LDS-tiled product takes
struct Fp8Gemm {
  const uint8_t* x;     // [x_rows, K]
  const float* xs;      // [x_rows, KB]
  const uint8_t* w;     // [groups or 1, N, K]
  const float* ws;      // [groups or 1, NB, KB]
  const int32_t* rows;  // [M] or null
  void* y;              // [M, N], bf16 or fp32
  int M, N, K, KB, NB, x_rows, groups;
  int splits = 1;       // of k: set by fp8_matmul
  float* ys = nullptr;  // [M, NB]: the scales of a quantised output
};
// whether the product's launches stay below 2^32 threads
bool fp8_matmul_fits(int M, int N, int KB, int groups, bool out_bf16);
// bytes of `ws`: the groups' row tiles, or the partial sums of a split of k
size_t fp8_matmul_workspace(int M, int N, int KB, int groups, bool out_bf16);
hipError_t fp8_matmul(Fp8Gemm p, const int32_t* offsets, bool out_bf16, void* ws,
                      hipStream_t s);

// The row tiles (at most tile_m rows each) of the groups offsets[g] ..
// offsets[g + 1] - 1 of `rows` rows, at most 1024 groups, and their number.
hipError_t group_tiles(const int32_t* offsets, int groups, int rows, int tile_m, int max_tiles,
                       Tile* tiles, int32_t* ntiles, hipStream_t s);
// y = the sum of `splits` arrays of n fp32 numbers (a multiple of 4), in order.
hipError_t add_parts(const float* part, int splits, long n, void* y, bool bf16, hipStream_t s);

// The layer's expert projections in that format, on the dispatch's tile list
// (tiles of plan.bm rows; groups = experts, N and K multiples of 128):
//   up    y = e4m3 codes and ys = scales of relu(z[rows] Wup[e]^T)^2
//   down  y = H Wdn[e]^T in bf16
// path: lmoe_path; KB: blocks of the longer of the two k ranges.
struct Fp8Plan {
  bool stream;  // weight streaming, else LDS-tiled
  int bm;       // token rows of a tile
  int splits;   // of k (dense tiles)
};
Fp8Plan fp8_expert_plan(int rows, int experts, int KB, int path);
// whether both projections (F hidden, R latent columns) can be launched
bool fp8_experts_fit(const Fp8Plan& plan, long max_tiles, int F, int R);
hipError_t fp8_exp_up(const Fp8Gemm& p, const Fp8Plan& plan, const Tile* tiles, const int* ntiles,
                      int max_tiles, hipStream_t s);
hipError_t fp8_exp_down(const Fp8Gemm& p, const Fp8Plan& plan, const Tile* tiles,
                        const int* ntiles, int max_tiles, hipStream_t s);

// Microscaled 4-bit floating point (layout: lmoe_quantize_mxfp4).  Rows [rows,
// cols] `stride` apart -> codes [rows, 16 ceil(cols / 32)] and scales [rows,
// ceil(cols / 32)], and back to dense rows.
hipError_t mx4_quantize(const void* x, bool bf16, long rows, int cols, long stride,
                        uint8_t* codes, uint8_t* scales, hipStream_t s);
hipError_t mx4_dequantize(const uint8_t* codes, const uint8_t* scales, long rows, int cols,
                          void* y, bool bf16, hipStream_t s);
// The product of two such matrices, as fp8_matmul's (K a multiple of 128, N of
// 16).
struct Mx4Gemm {
  const uint8_t* x;     // [x_rows, K / 2]
  const uint8_t* xs;    // [x_rows, K / 32]
  const uint8_t* w;     // [groups or 1, N, K / 2]
  const uint8_t* ws;    // [groups or 1, N, K / 32]
  const int32_t* rows;  // [M] or null
  void* y;              // [M, N], bf16 or fp32
  int M, N, K, x_rows, groups;
  int splits = 1;  // of k: set by mx4_matmul
};
// whether the product's launches stay below 2^32 threads
bool mx4_matmul_fits(int M, int N, int K, int groups);
size_t mx4_matmul_workspace(int M, int N, int K, int groups);
hipError_t mx4_matmul(Mx4Gemm p, const int32_t* offsets, bool out_bf16, void* ws, hipStream_t s);

// A whole sparse layer for 1 <= T <= 16 tokens (T K <= 1024): router, experts,
// weighted sum, shared expert (S > 0).  D, F and S multiples of 64, or of 128
// where the format is not bf16; a matrix is smaller than 2^31 - 16 bytes.
struct MoeTokens {
  const void* x;                                 // [T, D], rows x_stride apart
  const void* gate;                              // [E, D]
  const float* bias;                             // [E] or null
  const void *up, *down, *sup, *sdown;           // codes: [E, F or 2 F, D], [E, D, F], ...
  const void *up_s, *down_s, *sup_s, *sdown_s;   // scales (not for bf16)
  void* y;                                       // [T, D]
  int32_t* idx;                                  // [T, K]
  float* weights;                                // [T, K]
  long x_stride;
  int x_bf16, gate_bf16, y_bf16, format, gated;  // format: lmoe_expert_format
  int T, D, F, S;
  RouteProblem r;
};
size_t moe_tokens_workspace(const MoeTokens& m);
hipError_t moe_tokens(const MoeTokens& m, void* workspace, hipStream_t s);
// How often a work-group looks for an entry's hidden rows before it gives up.
extern int moe_tokens_looks;

// r = sum_k w[t][k] O[inv[t][k]] -> r16 (bf16) and, if r32 != NULL, fp32.
hipError_t combine(const uint16_t* o, const int32_t* inv, const float* w, int T, int K, int R,
                   uint16_t* r16, float* r32, hipStream_t s);

}  // namespace lmoe
