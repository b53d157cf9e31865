// C ABI of the operators around the layer (routing from logits, the norms
// around a block, 8-bit block-scaled matrices): argument checks and launches.
// See include/lmoe.h for the contract.  Every check runs on the host before
// any HIP call.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "../../include/lmoe.h"
#include "kernels.h"

using namespace lmoe;

namespace {

constexpr int64_t kMaxTokens = int64_t{1} << 22;

bool is_type(int32_t t) { return t == LMOE_F32 || t == LMOE_BF16; }
int64_t type_size(int32_t t) { return t == LMOE_BF16 ? 2 : 4; }
bool aligned(const void* p, int64_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

struct Span {
  const void* p;
  int64_t bytes;
};
bool overlap(const Span& a, const Span& b) {
  if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
  const char* x = static_cast<const char*>(a.p);
  const char* y = static_cast<const char*>(b.p);
  return x < y + b.bytes && y < x + a.bytes;
}
// No output overlaps an input or another output.
bool disjoint(std::initializer_list<Span> in, std::initializer_list<Span> out) {
  for (const Span& o : out) {
    for (const Span& i : in)
      if (overlap(o, i)) return false;
    for (const Span& q : out)
      if (&q != &o && overlap(o, q)) return false;
  }
  return true;
}
// Bytes from the first element to the end of the last of `rows` rows.
int64_t strided(int64_t rows, int64_t stride, int64_t width, int64_t el) {
  return rows > 0 ? ((rows - 1) * stride + width) * el : 0;
}

lmoe_status check_router(const lmoe_router* r) {
  if (!r) return LMOE_ERR_INVALID_ARG;
  if (r->n_experts <= 0 || r->top_k <= 0 || r->n_group <= 0 || !std::isfinite(r->scale))
    return LMOE_ERR_INVALID_ARG;
  if (r->score != LMOE_SCORE_SIGMOID && r->score != LMOE_SCORE_SOFTMAX)
    return LMOE_ERR_INVALID_ARG;
  if (r->renormalise != 0 && r->renormalise != 1) return LMOE_ERR_INVALID_ARG;
  if (r->group_score != 1 && r->group_score != 2) return LMOE_ERR_INVALID_ARG;
  if (r->topk_group < 1 || r->topk_group > r->n_group || r->n_experts % r->n_group)
    return LMOE_ERR_INVALID_ARG;
  const int32_t per = r->n_experts / r->n_group;
  if (r->n_group > 1 && r->group_score > per) return LMOE_ERR_INVALID_ARG;
  if (r->top_k > static_cast<int64_t>(r->topk_group) * per) return LMOE_ERR_INVALID_ARG;
  if (r->n_experts > 1024 || r->top_k > 64 || r->n_group > 64) return LMOE_ERR_UNSUPPORTED;
  return LMOE_OK;
}

lmoe_status check_route(const lmoe_router* r, int32_t type, int64_t stride, int32_t T) {
  const lmoe_status st = check_router(r);
  if (st != LMOE_OK) return st;
  if (!is_type(type) || T < 0 || stride < r->n_experts) return LMOE_ERR_INVALID_ARG;
  if (T > kMaxTokens || stride > (int64_t{1} << 31)) return LMOE_ERR_UNSUPPORTED;
  return LMOE_OK;
}

RouteProblem route_problem(const lmoe_router& r, int64_t stride, int32_t T) {
  return {T,       r.n_experts,   r.top_k,       r.n_group, r.topk_group,
          r.group_score, r.score == LMOE_SCORE_SOFTMAX, r.renormalise, r.scale,
          static_cast<long>(stride)};
}

lmoe_status check_norm(const lmoe_block_norm_args* a) {
  if (!a) return LMOE_ERR_INVALID_ARG;
  if (a->T < 0 || a->D <= 0 || !std::isfinite(a->eps) || !(a->eps > 0.f))
    return LMOE_ERR_INVALID_ARG;
  for (int32_t t : {a->h_type, a->y_type, a->pre_type, a->post_type, a->res_scale_type,
                    a->gate_type})
    if (!is_type(t)) return LMOE_ERR_INVALID_ARG;
  if (a->gate_kind < LMOE_GATE_NONE || a->gate_kind > LMOE_GATE_FULL ||
      (a->gate != nullptr) != (a->gate_kind != LMOE_GATE_NONE && (a->T > 0 || a->gate)))
    return LMOE_ERR_INVALID_ARG;
  // a launch has fewer than 2^32 threads, up to 1024 of them to a token
  if (a->D > block_norm_max_width() || a->T >= kMaxTokens) return LMOE_ERR_UNSUPPORTED;
  if (a->T == 0) return LMOE_OK;
  if (!a->h || a->h_stride < a->D) return LMOE_ERR_INVALID_ARG;
  if (a->y ? a->y_stride < a->D : (a->post_weight || a->gate)) return LMOE_ERR_INVALID_ARG;
  if (a->h_stride > (int64_t{1} << 31) || (a->y && a->y_stride > (int64_t{1} << 31)))
    return LMOE_ERR_UNSUPPORTED;
  if (!aligned(a->h, type_size(a->h_type)) || !aligned(a->y, type_size(a->y_type)) ||
      !aligned(a->pre_weight, type_size(a->pre_type)) ||
      !aligned(a->post_weight, type_size(a->post_type)) ||
      !aligned(a->res_scale, type_size(a->res_scale_type)) ||
      !aligned(a->gate, type_size(a->gate_type)))
    return LMOE_ERR_INVALID_ARG;
  return LMOE_OK;
}

int64_t gate_bytes(const lmoe_block_norm_args& a) {
  const int64_t n = a.gate_kind == LMOE_GATE_CHANNEL ? a.D
                    : a.gate_kind == LMOE_GATE_TOKEN ? a.T
                    : a.gate_kind == LMOE_GATE_FULL  ? static_cast<int64_t>(a.T) * a.D
                                                     : 0;
  return n * type_size(a.gate_type);
}

int norm_sums(const lmoe_block_norm_args& a, const lmoe_block_norm_grads& g) {
  return (g.dpre_weight != nullptr) + (g.dpost_weight != nullptr) + (g.dres_scale != nullptr) +
         (g.dgate != nullptr && a.gate_kind == LMOE_GATE_CHANNEL);
}

BlockNormProblem norm_problem(const lmoe_block_norm_args& a) {
  auto par = [](const void* p, int32_t t) { return NormParam{p, p && t == LMOE_BF16}; };
  return {a.h,
          a.y,
          static_cast<long>(a.h_stride),
          static_cast<long>(a.y_stride),
          a.h_type == LMOE_BF16,
          a.y_type == LMOE_BF16,
          par(a.pre_weight, a.pre_type),
          par(a.post_weight, a.post_type),
          par(a.res_scale, a.res_scale_type),
          par(a.gate, a.gate_type),
          a.gate_kind,
          a.T,
          a.D,
          a.eps};
}

lmoe_status check_quantize(const void* x, int32_t type, int64_t rows, int64_t cols, int64_t stride,
                           int64_t nscales, const uint8_t* codes, const float* scales) {
  const int64_t el = type_size(type);
  if (!x || !codes || !scales || !aligned(x, el) || !aligned(scales, 4))
    return LMOE_ERR_INVALID_ARG;
  if (!disjoint({{x, strided(rows, stride, cols, el)}},
                {{codes, rows * cols}, {scales, nscales * 4}}))
    return LMOE_ERR_INVALID_ARG;
  return LMOE_OK;
}

// Largest element count of an array whose work-groups a launch can number.
constexpr int64_t kMaxElements = int64_t{1} << 40;

// Host-side checks that do not need the workspace.
lmoe_status check_fp8(const lmoe_fp8_matmul_args* a) {
  if (!a) return LMOE_ERR_INVALID_ARG;
  if (a->M < 0 || a->N <= 0 || a->K <= 0 || a->n_groups < 0 || !is_type(a->y_type) ||
      (a->M > 0 && a->x_rows < 1))
    return LMOE_ERR_INVALID_ARG;
  if (a->N % 16 || a->K % 128 || a->N > (1 << 20) || a->K > 65536 ||
      a->n_groups > 1024 || a->M > (1 << 24))
    return LMOE_ERR_UNSUPPORTED;
  if (a->M == 0) return LMOE_OK;
  if (!a->x || !a->x_scales || !a->w || !a->w_scales || !a->y || !aligned(a->x, 16) ||
      !aligned(a->w, 16) || !aligned(a->y, 16) || !aligned(a->x_scales, 4) ||
      !aligned(a->w_scales, 4) || !aligned(a->rows, 4) || !aligned(a->offsets, 4))
    return LMOE_ERR_INVALID_ARG;
  if ((a->n_groups > 0) != (a->offsets != nullptr)) return LMOE_ERR_INVALID_ARG;
  if (!a->rows && a->x_rows < a->M) return LMOE_ERR_INVALID_ARG;
  if (a->rows && static_cast<int64_t>(a->x_rows) * a->K >= (int64_t{1} << 31))
    return LMOE_ERR_UNSUPPORTED;
  if (!fp8_matmul_fits(a->M, a->N, a->K / 128, a->n_groups, a->y_type == LMOE_BF16))
    return LMOE_ERR_UNSUPPORTED;
  const int64_t G = a->n_groups ? a->n_groups : 1, kb = a->K / 128, nb = (a->N + 127) / 128;
  if (!disjoint({{a->x, static_cast<int64_t>(a->x_rows) * a->K},
                 {a->x_scales, a->x_rows * kb * 4},
                 {a->w, G * a->N * a->K},
                 {a->w_scales, G * nb * kb * 4},
                 {a->rows, static_cast<int64_t>(a->M) * 4},
                 {a->offsets, (G + 1) * 4}},
                {{a->y, static_cast<int64_t>(a->M) * a->N * type_size(a->y_type)}}))
    return LMOE_ERR_INVALID_ARG;
  return LMOE_OK;
}

lmoe_status status(hipError_t e) { return e == hipSuccess ? LMOE_OK : LMOE_ERR_HIP; }

}  // namespace

extern "C" {

lmoe_status lmoe_route_logits(const lmoe_router* router, const void* logits, int32_t logits_type,
                              int64_t logits_stride, const float* bias, int32_t T,
                              int32_t* topk_idx, float* topk_w, void* stream) {
  const lmoe_status st = check_route(router, logits_type, logits_stride, T);
  if (st != LMOE_OK) return st;
  if (T == 0) return LMOE_OK;
  const int64_t el = type_size(logits_type), E = router->n_experts, K = router->top_k;
  if (!logits || !topk_idx || !topk_w || !aligned(logits, el) || !aligned(bias, 4) ||
      !aligned(topk_idx, 4) || !aligned(topk_w, 4))
    return LMOE_ERR_INVALID_ARG;
  if (!disjoint({{logits, strided(T, logits_stride, E, el)}, {bias, E * 4}},
                {{topk_idx, T * K * 4}, {topk_w, T * K * 4}}))
    return LMOE_ERR_INVALID_ARG;
  return status(route_logits(route_problem(*router, logits_stride, T), logits,
                             logits_type == LMOE_BF16, bias, topk_idx, topk_w,
                             static_cast<hipStream_t>(stream)));
}

lmoe_status lmoe_route_logits_backward(const lmoe_router* router, const void* logits,
                                       int32_t logits_type, int64_t logits_stride,
                                       const int32_t* topk_idx, const float* dw, int32_t T,
                                       void* dlogits, void* stream) {
  const lmoe_status st = check_route(router, logits_type, logits_stride, T);
  if (st != LMOE_OK) return st;
  if (T == 0) return LMOE_OK;
  const int64_t el = type_size(logits_type), E = router->n_experts, K = router->top_k;
  if (!logits || !topk_idx || !dw || !dlogits || !aligned(logits, el) || !aligned(topk_idx, 4) ||
      !aligned(dw, 4) || !aligned(dlogits, el))
    return LMOE_ERR_INVALID_ARG;
  if (!disjoint({{logits, strided(T, logits_stride, E, el)}, {topk_idx, T * K * 4},
                 {dw, T * K * 4}},
                {{dlogits, T * E * el}}))
    return LMOE_ERR_INVALID_ARG;
  return status(route_logits_backward(route_problem(*router, logits_stride, T), logits,
                                      logits_type == LMOE_BF16, topk_idx, dw, dlogits,
                                      static_cast<hipStream_t>(stream)));
}

lmoe_status lmoe_block_norm(const lmoe_block_norm_args* a, void* h_out, void* x, float* stats,
                            void* stream) {
  const lmoe_status st = check_norm(a);
  if (st != LMOE_OK) return st;
  if (a->T == 0) return LMOE_OK;
  const int64_t T = a->T, D = a->D, he = type_size(a->h_type), ye = type_size(a->y_type);
  if (!h_out || !aligned(h_out, he) || !aligned(x, ye) || !aligned(stats, 4))
    return LMOE_ERR_INVALID_ARG;
  if (!disjoint({{a->h, strided(T, a->h_stride, D, he)},
                 {a->y, strided(T, a->y_stride, D, ye)},
                 {a->pre_weight, D * type_size(a->pre_type)},
                 {a->post_weight, D * type_size(a->post_type)},
                 {a->res_scale, D * type_size(a->res_scale_type)},
                 {a->gate, gate_bytes(*a)}},
                {{h_out, T * D * he}, {x, T * D * ye}, {stats, T * 8}}))
    return LMOE_ERR_INVALID_ARG;
  return status(block_norm(norm_problem(*a), h_out, x, stats, static_cast<hipStream_t>(stream)));
}

size_t lmoe_block_norm_workspace_size(const lmoe_block_norm_args* a,
                                      const lmoe_block_norm_grads* g) {
  if (!g || check_norm(a) != LMOE_OK) return 0;
  const int n = norm_sums(*a, *g);
  return n ? block_norm_backward_part(a->T, a->D, n) : 0;
}

lmoe_status lmoe_block_norm_backward(const lmoe_block_norm_args* a, const float* stats,
                                     const void* dh_out, const void* dx,
                                     const lmoe_block_norm_grads* g, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  const lmoe_status st = check_norm(a);
  if (st != LMOE_OK) return st;
  if (!g) return LMOE_ERR_INVALID_ARG;
  const int64_t T = a->T, D = a->D, he = type_size(a->h_type), ye = type_size(a->y_type);
  if ((g->dpost_weight && !a->post_weight) || (g->dres_scale && !a->res_scale) ||
      (g->dgate && a->gate_kind == LMOE_GATE_NONE) || (g->dpre_weight && !a->pre_weight) ||
      (T > 0 && g->dy && !a->y))
    return LMOE_ERR_INVALID_ARG;
  if (!aligned(g->dh, he) || !aligned(g->dy, ye) ||
      !aligned(g->dpre_weight, type_size(a->pre_type)) ||
      !aligned(g->dpost_weight, type_size(a->post_type)) ||
      !aligned(g->dres_scale, type_size(a->res_scale_type)) ||
      !aligned(g->dgate, type_size(a->gate_type)) || !aligned(dh_out, he) || !aligned(dx, ye) ||
      !aligned(stats, 4))
    return LMOE_ERR_INVALID_ARG;
  const int sums = norm_sums(*a, *g);
  if (T == 0 && sums == 0) return LMOE_OK;
  if (T > 0 && !stats) return LMOE_ERR_INVALID_ARG;
  const size_t need = lmoe_block_norm_workspace_size(a, g);
  if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
    return LMOE_ERR_WORKSPACE;
  if (!disjoint({{a->h, strided(T, a->h_stride, D, he)},
                 {a->y, strided(T, a->y_stride, D, ye)},
                 {a->pre_weight, D * type_size(a->pre_type)},
                 {a->post_weight, D * type_size(a->post_type)},
                 {a->res_scale, D * type_size(a->res_scale_type)},
                 {a->gate, gate_bytes(*a)},
                 {stats, T * 8},
                 {dh_out, T * D * he},
                 {dx, T * D * ye}},
                {{g->dh, T * D * he},
                 {g->dy, T * D * ye},
                 {g->dpre_weight, D * type_size(a->pre_type)},
                 {g->dpost_weight, D * type_size(a->post_type)},
                 {g->dres_scale, D * type_size(a->res_scale_type)},
                 {g->dgate, gate_bytes(*a)},
                 {workspace, static_cast<int64_t>(need)}}))
    return LMOE_ERR_INVALID_ARG;
  BlockNormGrads q{stats, dh_out, dx, g->dh, g->dy, g->dpre_weight, g->dpost_weight,
                   g->dres_scale, g->dgate};
  return status(block_norm_backward(norm_problem(*a), q, static_cast<float*>(workspace),
                                    static_cast<hipStream_t>(stream)));
}

lmoe_status lmoe_quantize_fp8(const void* x, int32_t x_type, int64_t rows, int32_t cols,
                              int64_t x_stride, uint8_t* codes, float* scales, void* stream) {
  if (rows < 0 || cols <= 0 || !is_type(x_type) || x_stride < cols) return LMOE_ERR_INVALID_ARG;
  if (rows > kMaxElements / cols || x_stride > (int64_t{1} << 31)) return LMOE_ERR_UNSUPPORTED;
  if (rows == 0) return LMOE_OK;
  const int64_t nb = (static_cast<int64_t>(cols) + 127) / 128;
  // a launch has fewer than 2^32 threads: 16 to a block
  if (rows * nb >= (int64_t{1} << 28)) return LMOE_ERR_UNSUPPORTED;
  const lmoe_status st =
      check_quantize(x, x_type, rows, cols, x_stride, rows * nb, codes, scales);
  if (st != LMOE_OK) return st;
  return status(fp8_quantize(x, x_type == LMOE_BF16, rows, cols, x_stride, codes, scales,
                             static_cast<hipStream_t>(stream)));
}

lmoe_status lmoe_quantize_fp8_weight(const void* w, int32_t w_type, int64_t matrices, int32_t rows,
                                     int32_t cols, uint8_t* codes, float* scales, void* stream) {
  if (matrices < 0 || rows <= 0 || cols <= 0 || !is_type(w_type)) return LMOE_ERR_INVALID_ARG;
  const int64_t nb = ((static_cast<int64_t>(rows) + 127) / 128) *
                     ((static_cast<int64_t>(cols) + 127) / 128);
  // a launch has fewer than 2^32 threads: 256 to a block
  if (matrices > ((int64_t{1} << 24) - 1) / nb) return LMOE_ERR_UNSUPPORTED;
  if (matrices == 0) return LMOE_OK;
  const lmoe_status st =
      check_quantize(w, w_type, matrices * rows, cols, cols, matrices * nb, codes, scales);
  if (st != LMOE_OK) return st;
  return status(fp8_quantize_weight(w, w_type == LMOE_BF16, matrices, rows, cols, codes, scales,
                                    static_cast<hipStream_t>(stream)));
}

size_t lmoe_fp8_matmul_workspace_size(const lmoe_fp8_matmul_args* a) {
  if (check_fp8(a) != LMOE_OK || a->M == 0) return 0;
  return fp8_matmul_workspace(a->M, a->N, a->K / 128, a->n_groups,
                              a->y_type == LMOE_BF16);
}

lmoe_status lmoe_fp8_matmul(const lmoe_fp8_matmul_args* a, void* workspace, size_t workspace_bytes,
                            void* stream) {
  const lmoe_status st = check_fp8(a);
  if (st != LMOE_OK) return st;
  if (a->M == 0) return LMOE_OK;
  const size_t need = fp8_matmul_workspace(a->M, a->N, a->K / 128, a->n_groups,
                              a->y_type == LMOE_BF16);
  if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
    return LMOE_ERR_WORKSPACE;
  const int64_t G = a->n_groups ? a->n_groups : 1, kb = a->K / 128, nb = (a->N + 127) / 128;
  if (!disjoint({{a->x, static_cast<int64_t>(a->x_rows) * a->K},
                 {a->x_scales, a->x_rows * kb * 4},
                 {a->w, G * a->N * a->K},
                 {a->w_scales, G * nb * kb * 4},
                 {a->rows, static_cast<int64_t>(a->M) * 4},
                 {a->offsets, (G + 1) * 4},
                 {a->y, static_cast<int64_t>(a->M) * a->N * type_size(a->y_type)}},
                {{workspace, static_cast<int64_t>(need)}}))
    return LMOE_ERR_INVALID_ARG;
  const Fp8Gemm p{a->x,    a->x_scales, a->w,
                  a->w_scales, a->rows, a->y,
                  a->M,    a->N,        a->K,
                  a->K / 128, (a->N + 127) / 128, a->x_rows, a->n_groups};
  return status(fp8_matmul(p, a->offsets, a->y_type == LMOE_BF16, workspace,
                           static_cast<hipStream_t>(stream)));
}

}  // extern "C"
