// A whole sparse layer for a few tokens (up to 16).
//
//   l_t = x_t Wg^T;  (I_t, w_t) = route(l_t)
//   h_p = act(x_t Wup[e]^T)            for each pair p = (t, k), e = I_t[k]
//   y_t = sum_k w_tk h_p Wdown[e]^T  (+ the shared expert's, weight 1)
//   act: relu(u)^2, or silu(u_gate) u_up of two halves of the up rows
//
// Bound by HBM: each used expert's weights are read once (where more than five
// tokens use it, once for each five), and everything else is small; so what counts
// is that the weights' stream starts early and never pauses.  Two kernels: the first
// computes the logits (64-bit sums, rounded once to fp32) and clears the second
// one's counters and flags.  The second one's work-groups each route all tokens
// by themselves, a wave a token (for many experts and more than four tokens
// route_logits's kernel does it before them), list the used experts, and then draw
// items: first blocks of rows of the up projections, expert by expert, then of the
// down projections.
//
// Measured, the second kernel: 22 experts of 2048 x 5120 for one token, bf16 162 us
// (923 MB, 5.7 TB/s), MXFP4 74 (245 MB, 3.3 TB/s); 97 experts for six tokens, FP8 340
// (2035 MB, 6.0 TB/s).  A card that only reads reaches 7.0.  What small layers add to
// that is latency, one thing after the other: 5 to 9 us until the first weights are
// asked for, 2 to 4 for the first lines and rows, 3 to 6 for an expert's hidden rows
// to be written, seen and read, 3 for the last output rows: 29 us for a layer of 35 MB.
//
// Items are drawn from kQueues counters a projection (one counter for all took
// 25 ns an item, whatever its size), each work-group from its own until that is
// empty and then from the others.  A down item waits until its expert's hidden
// rows are written.  No work-group draws a down item before all up items are
// drawn, and who holds an up item does not wait, so whatever is waited for is
// being worked on, whichever work-groups run.  The pairs' output rows are added
// by the wave that finishes a block of columns last, in a fixed order: the same
// bits every time.
//
// Weights are the MFMA's A operand, read from HBM as whole lines into registers,
// kAhead lines ahead (on into the next block), brought into its layout through LDS
// and decoded exactly to bf16 (8-bit: the block's scale on its sum).  The tokens'
// operand is bf16, too: a value that is no bf16 number (fp32 x, the hidden rows)
// is the sum of three such parts (24 bits: an fp32 number's), each a column of its
// own of the operand, of which one token leaves 15 free; their results are added at
// the end.  (Two parts for results in bf16, 16 bits, were not enough: what cancels
// between experts, or in a row of weights, leaves their error.)  The 16 columns hold
// five tokens, or all of them where x is bf16 and the projection up; an expert with
// more is taken as several entries, and its weights are read again for each (blocks
// of such entries next to each other, for a cache to hold them: 3% to 13% slower).
//
// The loop is kept small and rolled: unrolled over the forms of an item, its 40 KB
// of code did not stay in the instruction cache and it ran three times as long.
// So did rings of lines in LDS: their copies took as long to issue as to arrive.
#include <type_traits>

#include "fp8_device.h"
#include "gemm_device.h"
#include "kernels.h"
#include "mxfp4_device.h"
#include "route_device.h"

namespace lmoe {

namespace {

constexpr int kWaves = 8, kThreads = kWaves * 64;
constexpr int kQueues = 16, kSpread = 64;  // counters, ints apart
constexpr int kAhead = 3;                  // lines that a wave loads ahead
constexpr int kParts = 3;                  // bf16 numbers of an fp32 operand
constexpr int kTurn = 16 / kParts;         // rows of an entry
constexpr int kLogitTokens = 4;            // tokens of a work-group of the first kernel
constexpr float kBf16Max = 0x1.FEp127f;

// Formats: k values in a line of 128 bytes, fragments of 8 values in 16 bytes,
// waves that share a row group of 16 (each takes every WK-th line).  Items are 16
// kWaves / WK rows: 128 KB at K = 2048 in each format; a line of each wave is 256
// values of x.
template <int FMT>
struct Fmt;
template <>
struct Fmt<0> {  // bf16
  static constexpr int LK = 64, NF = 1, WK = 4;
};
template <>
struct Fmt<1> {  // MXFP4
  static constexpr int LK = 256, NF = 4, WK = 1;
};
template <>
struct Fmt<2> {  // FP8
  static constexpr int LK = 128, NF = 2, WK = 2;
};

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

// c ? a : b of values.  (A conditional of variables chooses between their
// addresses, which keeps all that a kernel's lambdas share in memory.)
template <class V>
__device__ __forceinline__ V pick(bool c, V a, V b) {
  return c ? a : b;
}

struct MoeParams {
  MoeTokens m;
  float *logits, *h, *hs, *o;
  int32_t *queues, *up_done, *down_done;
  int looks;   // for an entry's hidden rows, before a work-group gives up
  int xbytes;  // LDS for the tokens' rows (then the waves' sums)
  int turn_at; // where in LDS lines change their layout
  int early;   // LDS of one token's x, which is there before the first block; or 0
  int misc;    // where in LDS what is not of the loop begins
};

__device__ __forceinline__ f32x4 load4(const float* p) { return *reinterpret_cast<const f32x4*>(p); }
__device__ __forceinline__ f32x4 load4(const uint16_t* p) {
  const u16x4 v = *reinterpret_cast<const u16x4*>(p);
  return f32x4{bf16_to_f32(v[0]), bf16_to_f32(v[1]), bf16_to_f32(v[2]), bf16_to_f32(v[3])};
}

// What work-groups hand each other (hidden rows, output rows) is stored and
// loaded past the XCDs' own L2 caches, by relaxed atomics of the whole device:
// a finished store is then visible everywhere, and no cache has to be written
// back or emptied.  (With plain stores and agent fences instead, which do that
// for a whole L2 at every item, the kernel took five times as long.)
__device__ __forceinline__ void put4_shared(float* p, f32x4 v) {
  uint64_t u[2];
  __builtin_memcpy(u, &v, 16);
  uint64_t* q = reinterpret_cast<uint64_t*>(p);
  __hip_atomic_store(q, u[0], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __hip_atomic_store(q + 1, u[1], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ f32x4 get4_shared(const float* p) {
  const uint64_t* q = reinterpret_cast<const uint64_t*>(p);
  const uint64_t u[2] = {__hip_atomic_load(q, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT),
                         __hip_atomic_load(q + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)};
  f32x4 v;
  __builtin_memcpy(&v, u, 16);
  return v;
}
__device__ __forceinline__ float get1_shared(const float* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// Four values as `parts` bf16 numbers each, `pitch` bytes apart.
__device__ __forceinline__ void put_parts(f32x4 u, char* to, int pitch, int parts) {
  // what is rounded to infinity, or is infinite, is the last part's
#pragma unroll 1
  for (int q = 1; q < parts; ++q, to += pitch) {
    f32x4 c;
#pragma unroll
    for (int n = 0; n < 4; ++n) c[n] = __builtin_amdgcn_fmed3f(u[n], -kBf16Max, kBf16Max);
    const bf16x4 b = __builtin_convertvector(c, bf16x4);
    *reinterpret_cast<bf16x4*>(to) = b;
    u -= __builtin_convertvector(b, f32x4);
  }
  *reinterpret_cast<bf16x4*>(to) = __builtin_convertvector(u, bf16x4);
}
// This wave's stores are done (and none of its later accesses begins before).
__device__ __forceinline__ void stores_done() {
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  wait_vmcnt<0>();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

}  // namespace

// Logits: a work-group an expert and four tokens, products and sums in 64 bits.
template <class GT, class XT>
__global__ __launch_bounds__(256) void moe_logits_kernel(const XT* __restrict__ x, long x_stride,
                                                         const GT* __restrict__ gate, int T, int E,
                                                         int D, float* __restrict__ logits,
                                                         int32_t* __restrict__ sync, int nsync) {
  constexpr int TB = kLogitTokens;
  __shared__ double part[4][TB];
  const int e = blockIdx.x, tid = threadIdx.x, t0 = blockIdx.y * TB;
  if (t0 == 0)
    for (int i = e * 256 + tid; i < nsync; i += E * 256) sync[i] = 0;
  double acc[TB];
#pragma unroll
  for (int u = 0; u < TB; ++u) acc[u] = 0.0;
  for (int k = tid * 4; k < D; k += 1024) {
    const f32x4 g = load4(gate + (size_t)e * D + k);
#pragma unroll
    for (int u = 0; u < TB; ++u) {
      if (t0 + u >= T) break;
      const f32x4 v = load4(x + (t0 + u) * x_stride + k);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[u] = fma((double)g[i], (double)v[i], acc[u]);
    }
  }
#pragma unroll
  for (int u = 0; u < TB; ++u) {
    if (t0 + u >= T) break;
    const double s = wave_sum(acc[u]);
    if ((tid & 63) == 0) part[tid >> 6][u] = s;
  }
  __syncthreads();
  if (tid < TB && t0 + tid < T)
    logits[(size_t)(t0 + tid) * E + e] =
        (float)(part[0][tid] + part[1][tid] + part[2][tid] + part[3][tid]);
}

namespace {

// What a work-group works on: block `blk` of rows of the projection's entry u, K
// long.
struct Item {
  int down, u, blk, K;
};

// What a wave loads: its rows' lines in an item's matrix.
struct Source {
  const uint8_t* codes;
  const uint32_t* scales;
  uint32_t lane, slane;  // a lane's offset in eight rows, in the scales
  int first, second;     // offsets of the first and the last eight rows
  int lines, odd;        // of the item; the last is half a line
};

struct Line {
  u32x4 l[2];  // of the first and the last eight rows
  uint32_t s[2];
};

constexpr int kShared = 0xFFFF;  // an entry of the shared expert

}  // namespace

// NJ: E is at most 64 NJ and the tokens are routed here; 0: they have been.
template <int FMT, int NJ>
__global__ __launch_bounds__(kThreads, 4) void moe_tokens_kernel(MoeParams p) {
  using C = Fmt<FMT>;
  constexpr int LK = C::LK, NF = C::NF, WK = C::WK, WR = kWaves / WK, NL = kAhead + 1;
  extern __shared__ __attribute__((aligned(16))) char smem[];

  const MoeTokens& m = p.m;
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = uniform(tid >> 6), wk = w % WK, wr = w / WK;
  const int T = m.T, E = m.r.E, K = m.r.K, D = m.D, F = m.F, S = m.S, gated = m.gated;
  const int P = T * K;
  int queue = blockIdx.x % kQueues;  // (wave 0's, as is the phase)
  int phase = 0;

  // ---- routing and the list of used experts, in every work-group ----
  int pending = 0;
  if (tid == 0) {
    int at = queue * kSpread;
    asm volatile("" : "+v"(at));  // (of one known address, the result is waited for here)
    pending = __hip_atomic_fetch_add(p.queues + at, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  int* const stick = reinterpret_cast<int*>(smem + p.misc);     // [2][2] drawn runs
  int* const scount = stick + 4;                                // [kWaves]
  float* const sw = reinterpret_cast<float*>(scount + kWaves);  // [P] pairs' weights
  uint16_t* const slist = reinterpret_cast<uint16_t*>(sw + P);  // [P] pairs by expert
  // entries: expert, first of its pairs in the list, their number and, from bit 5 on,
  // its entry in the projection up.  The down projection's, then (from upto on; the
  // same ones where x is fp32) the up projection's.
  const bool own_up = m.x_bf16 && T > kTurn;
  const int upto = own_up ? P + 16 : 0;
  uint16_t* const sexp = slist + P;
  uint16_t* const sstart = sexp + P + 16 + upto;
  uint16_t* const srows = sstart + P + 16 + upto;
  constexpr int ROUTE = kWaves * (256 + NJ * 512);
  char* const scratch = smem + p.early;
  uint32_t* const smask = reinterpret_cast<uint32_t*>(scratch + ROUTE);  // [E] tokens
  uint32_t* const sfirst = smask + E;                                 // [E]
  int32_t* const sidx = reinterpret_cast<int32_t*>(sfirst + E);       // [P]
  for (int i = tid; i < E; i += kThreads) smask[i] = 0;
  // One token: its x is brought into LDS, as put_rows below does it, by the waves that
  // do not route.
  if (p.early && w > 0) {
    const int parts = m.x_bf16 ? 1 : kParts, pitch = p.early / parts;
    constexpr int N = 3, step = (kThreads - 64) * 4;
#pragma unroll 1
    for (int k = (tid - 64) * 4; k * 2 < pitch - 16; k += N * step) {
      f32x4 v[N];
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int at = min(k + j * step, D - 4);
        v[j] = m.x_bf16 ? load4(static_cast<const uint16_t*>(m.x) + at)
                        : load4(static_cast<const float*>(m.x) + at);
      }
#pragma unroll
      for (int j = 0; j < N; ++j)
        if ((k + j * step) * 2 < pitch - 16)
          put_parts(k + j * step < D ? v[j] : f32x4{0.f, 0.f, 0.f, 0.f}, smem + (k + j * step) * 2,
                    pitch, parts);
    }
  }
  if constexpr (NJ > 0) {
    for (int t = w; t < T; t += kWaves) {
      route_token<float, NJ>(p.logits + (size_t)t * E, m.bias, m.r, lane,
                             reinterpret_cast<float*>(scratch + w * 256),
                             scratch + kWaves * 256 + w * NJ * 512, sidx + t * K, sw + t * K);
      if (NJ > 2) break;  // (up to four tokens)
      wave_lds_fence();
    }
  } else {
    for (int i = tid; i < P; i += kThreads) {
      sidx[i] = m.idx[i];
      sw[i] = m.weights[i];
    }
  }
  __syncthreads();
  for (int i = tid; i < P; i += kThreads) {
    // (whatever a bias that is no number made of it: an expert)
    const int e = (int)min((uint32_t)sidx[i], (uint32_t)E - 1u);
    sidx[i] = e;
    atomicOr(&smask[e], 1u << (i / K));
    if (NJ > 0 && blockIdx.x == 0) {
      m.idx[i] = sidx[i];
      m.weights[i] = sw[i];
    }
  }
  __syncthreads();
  // Entries: the shared expert's first, then the used experts', each of up to kTurn of
  // the tokens that take it, or (up, x in bf16) of all of them.
  const int nsh = S > 0 ? (T + kTurn - 1) / kTurn : 0;
  const int nshu = S > 0 && own_up ? 1 : nsh;
  auto put_entry = [&](int u, int e, int first, int n, int ue) __attribute__((always_inline)) {
    sexp[u] = (uint16_t)e;
    sstart[u] = (uint16_t)first;
    srows[u] = (uint16_t)(n | ue << 5);
  };
  if (tid < nsh)
    put_entry(tid, kShared, tid * kTurn, min(kTurn, T - tid * kTurn), own_up ? 0 : tid);
  if (tid < nshu && own_up) put_entry(upto, kShared, 0, T, 0);
  int nexp, nexpu;
  {
    // thread i: experts 4 i to 4 i + 3.  Sums of three numbers each: experts used (11
    // bits), their further entries (10), their pairs.
    uint32_t v[4], inc = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t n = 4 * tid + j < E ? __popc(smask[4 * tid + j]) : 0;
      v[j] = n ? 1u | ((n - 1) / kTurn) << 11 | n << 21 : 0u;
      inc += v[j];
    }
    const uint32_t own = inc;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const uint32_t o = __shfl_up(inc, off, 64);
      if (lane >= off) inc += o;
    }
    if (lane == 63) scount[w] = (int)inc;
    __syncthreads();
    uint32_t at = inc - own, all = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
      if (i < w) at += (uint32_t)scount[i];
      all += (uint32_t)scount[i];
    }
    const int used = uniform((int)(all & 0x7FF)), more = uniform((int)(all >> 11 & 0x3FF));
    nexp = nsh + used + more;
    nexpu = nshu + used + (own_up ? 0 : more);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = (int)(v[j] >> 21), first = (int)(at >> 21), x = (int)(at & 0x7FF);
      if (n) {
        sfirst[4 * tid + j] = first;
        if (own_up) put_entry(upto + nshu + x, 4 * tid + j, first, n, 0);
      }
      for (int r = 0, u = nsh + x + (int)(at >> 11 & 0x3FF); r < n; r += kTurn, ++u)
        put_entry(u, 4 * tid + j, first + r, min(kTurn, n - r), own_up ? nshu + x : u);
      at += v[j];
    }
  }
  __syncthreads();
  for (int i = tid; i < P; i += kThreads) {
    const int e = sidx[i], t = i / K;
    slist[sfirst[e] + __popc(smask[e] & ((1u << t) - 1u))] = (uint16_t)i;
  }
  const int fr = 16 * WR >> gated;  // hidden columns of an up item
  const int nf = F / fr, ns = S / fr, nd = D / (16 * WR), nsup = nshu * ns;
  const int nup = nsup + (nexpu - nshu) * nf, ndown = nexp * nd, total = nup + ndown;

  // Runs of blocks: the first gridDim.x of a projection are long and cover three
  // quarters of it, the others are short.
  auto long_run = [&](int ph) __attribute__((always_inline)) {
    return min(max(pick(ph != 0, ndown, nup) * 3 / 4 / (int)gridDim.x, 1), 64);
  };
  auto run_at = [&](int ph, int n) __attribute__((always_inline)) {  // first block of run n
    const int g = (int)gridDim.x, len = long_run(ph), over = max(n - g, 0);
    return min(n, g) * len + over * ((len + 3) / 4);
  };
  // Wave 0: the run of draw t of the queue, or from a queue that is not empty.
  auto draw = [&](int t, int* to) __attribute__((always_inline)) {
    for (;;) {
      const int end = pick(phase != 0, ndown, nup), base = pick(phase != 0, nup, 0);
      const int n = t * kQueues + queue, from = run_at(phase, min(n, end));
      if (from < end) {
        if (lane == 0) {
          to[0] = base + from;
          to[1] = base + min(run_at(phase, n + 1), end);
        }
        return;
      }
      uint64_t some;
      for (;;) {
        const int q = lane & (kQueues - 1);
        const int at = __hip_atomic_load(p.queues + (phase * kQueues + q) * kSpread,
                                         __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        const int end = pick(phase != 0, ndown, nup);
        some = __ballot(lane < kQueues && run_at(phase, min(at * kQueues + q, end)) < end);
        if (some || phase == 1) break;
        phase = 1;
      }
      if (!some) {
        if (lane == 0) to[0] = to[1] = total;
        return;
      }
      // the next one after the own
      const uint64_t later = some & (~0ull << queue);
      queue = __builtin_ctzll(later ? later : some);
      int got = 0;
      if (lane == 0)
        got = __hip_atomic_fetch_add(p.queues + (phase * kQueues + queue) * kSpread, 1,
                                     __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      t = uniform(got);
    }
  };
  if (w == 0) draw(uniform(pending), stick);
  __syncthreads();  // (the lists, too; the room before them is free)
  int cur = uniform(stick[0]), end = uniform(stick[1]);  // the run

  auto item_of = [&](int i) __attribute__((always_inline)) {
    Item it;
    it.down = i >= nup;
    const bool sh = i < nsup;
    const int j = i - pick(it.down != 0, nup, pick(sh, 0, nsup));
    const int n = pick(it.down != 0, nd, pick(sh, ns, nf));
    const int u = j / n;
    it.blk = j - u * n;
    it.u = u + pick(it.down != 0, 0, upto + pick(sh, 0, nshu));
    it.K = pick(it.down != 0, pick(it.u < nsh, S, F), D);
    return it;
  };
  auto of_shared = [&](const Item& it) __attribute__((always_inline)) {
    return it.u < pick(it.down != 0, nsh, upto + nshu);
  };
  auto lines_of = [&](int k) __attribute__((always_inline)) { return (k + LK - 1) / LK; };
  const int r16 = lane & 15, kq = lane >> 4;

  Source src;
  auto enter = [&](const Item& it) __attribute__((always_inline)) {
    const bool sh = of_shared(it), down = it.down, two = gated && !down;
    const int rows = pick(down, D, pick(sh, S, F));  // of one half where gated
    const int ex = uniform(sexp[it.u]);
    const size_t e = sh ? 0 : (size_t)ex * ((size_t)rows << two);
    const uint32_t rb = FMT == 0 ? it.K * 2 : FMT == 1 ? it.K / 2 : it.K;
    const void* const w0 = pick(sh, pick(down, m.sdown, m.sup), pick(down, m.down, m.up));
    const void* const s0 = pick(sh, pick(down, m.sdown_s, m.sup_s), pick(down, m.down_s, m.up_s));
    src.codes = static_cast<const uint8_t*>(w0) + e * rb;
    // the wave's 16 rows; where gated, eight of the gate's half and the same of
    // the other
    const int group = it.blk * WR + wr, first = group * (two ? 8 : 16);
    const int second = two ? rows + first : first + 8;
    src.first = first * rb;
    src.second = second * rb;
    src.lane = (uint32_t)(lane >> 3) * rb + (lane & 7) * 16;
    const int sr = it.K / 128;  // scale words of a row (FP8: of 128 rows)
    if (FMT == 1) {
      src.scales = static_cast<const uint32_t*>(s0) + e * sr;
      src.slane = (uint32_t)((r16 < 8 ? first + r16 : second + r16 - 8) * sr) * 4;
    }
    if (FMT == 2) {  // of the rows of the lane's results
      src.scales = static_cast<const uint32_t*>(s0) + e / 128 * sr;
      src.slane = (uint32_t)(pick(kq < 2, first, second) / 128 * sr) * 4;
    }
    src.lines = lines_of(it.K);
    src.odd = FMT == 1 && it.K % LK != 0;
  };
  // Line j of the wave's: wk + WK j of its rows.  (MXFP4: where K ends in half a
  // line, its second half reads the first one's bytes and scales again, and x is
  // 0 there.)  The loads are always issued, out of the buffers' bounds where there
  // is no such line (nothing is fetched then): behind a branch, the compiler
  // would have to wait for all loads in flight wherever it waits for one.
  auto load = [&](Line& A, int j, bool some) __attribute__((always_inline)) {
    const int l = wk + WK * j;
    const bool on = some && l < src.lines;
    const __amdgpu_buffer_rsrc_t codes = buffer_rsrc(src.codes);
    const bool half = FMT == 1 && src.odd && l == src.lines - 1;
    const uint32_t at = on ? (half && (lane & 4) ? src.lane - 64 : src.lane) : 0x80000000u;
    const int to = pick(on, l, 0) * 128;
    A.l[0] = __builtin_amdgcn_raw_buffer_load_b128(codes, at, src.first + to, 2 /* nt */);
    A.l[1] = __builtin_amdgcn_raw_buffer_load_b128(codes, at, src.second + to, 2);
    if (FMT != 0) {
      const __amdgpu_buffer_rsrc_t scales = buffer_rsrc(src.scales);
      const uint32_t sat = on ? src.slane : 0x80000000u;
      const int st = pick(on, l, 0) * (FMT == 1 ? 8 : 4);
      A.s[0] = __builtin_amdgcn_raw_buffer_load_b32(scales, sat, st, 0);
      if (FMT == 1)
        A.s[1] = __builtin_amdgcn_raw_buffer_load_b32(scales, sat, st + (half ? 0 : 4), 0);
    }
  };

  // A line's way into the instruction's layout, through 2 KB of LDS of the wave's
  // own: lane l writes piece l % 8 of row l / 8 (and of row 8 + l / 8), lane (r, q)
  // reads pieces q and 4 + q of row r, places exchanged so that neither meets a
  // bank twice.
  char* const turn_in = smem + p.turn_at + w * 2048 + (lane >> 3) * 128 +
                        (((lane & 7) ^ (lane >> 3)) << 4);
  char* const turn_in2 = smem + p.turn_at + w * 2048 + 1024 + (lane >> 3) * 128 +
                         (((lane & 7) ^ (lane >> 3) ^ 1) << 4);
  const char* const turn_row =
      smem + p.turn_at + w * 2048 + (r16 >> 3) * 1024 + (r16 & 7) * 128;
  const char* const turn_out = turn_row + ((kq ^ (r16 & 7) ^ (r16 >> 3)) << 4);
  const char* const turn_out2 = turn_row + (((4 + kq) ^ (r16 & 7) ^ (r16 >> 3)) << 4);
  // Adds line j to acc; x0: the lane's place in LDS of the first value of its
  // column's row in line `l0`.  (A line past the last is zeros times the last's x.)
  auto compute = [&](const Line& A, f32x4& acc, int j, int lines, const char* x0, int l0)
                     __attribute__((always_inline)) {
    u32x4 c[2];
    *reinterpret_cast<u32x4*>(turn_in) = A.l[0];
    *reinterpret_cast<u32x4*>(turn_in2) = A.l[1];
    c[0] = *reinterpret_cast<const u32x4*>(turn_out);
    c[1] = *reinterpret_cast<const u32x4*>(turn_out2);
    const char* const xl = x0 + (min(wk + WK * j, lines - 1) - l0) * (LK * 2);
    f32x4 sum = FMT == 2 ? f32x4{0.f, 0.f, 0.f, 0.f} : acc;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < NF; ++i) {
        bf16x8 wf;
        if (FMT == 0) {
          wf = __builtin_bit_cast(bf16x8, c[h]);
        } else if (FMT == 1) {
          wf = mx_decode8(c[h][i], mx_scale((A.s[h] >> (8 * kq)) & 255u));
        } else {
#pragma unroll
          for (int d = 0; d < 2; ++d) {
            const auto v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[h][2 * i + d], 1.f, false);
            const auto v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[h][2 * i + d], 1.f, true);
            wf[4 * d] = v0[0], wf[4 * d + 1] = v0[1];
            wf[4 * d + 2] = v1[0], wf[4 * d + 3] = v1[1];
          }
        }
        sum = mfma_bf16(wf, *reinterpret_cast<const bf16x8*>(xl + h * 64 * NF + i * 16), sum);
      }
    acc = FMT == 2 ? acc + sum * __uint_as_float(A.s[0]) : sum;
  };

  // The item's tokens' rows (x, or hidden rows), values k0 .. k0 + kn - 1, into
  // LDS as `parts` bf16 numbers each; zeros from K on.  A wave takes 256 values of a
  // row at a time and has N such pieces, of whichever rows, in flight (one row
  // after the other would wait for memory once a row).
  auto put_rows = [&](const Item& it, int r0, int rows, int k0, int kn, int pitch, int parts)
                      __attribute__((always_inline)) {
    const bool sh = of_shared(it), down = it.down;
    constexpr int N = 5;
    const uint32_t pieces = (kn + 255) >> 8, all = rows * pieces;  // at most 2^11
    const uint32_t per_row = 0xFFFFFFFFu / pieces + 1;             // (0 of one piece)
    auto row_of = [&](uint32_t c) __attribute__((always_inline)) {
      return pieces == 1 ? c : __umulhi(c, per_row);
    };
#pragma unroll 1
    for (uint32_t c0 = w; c0 < all; c0 += N * kWaves) {
      f32x4 v[N];
      const float* hp[N];
      size_t xo[N];
      uint32_t at[N];
#pragma unroll
      for (int j = 0; j < N; ++j) {
        // (past the last: the last again, which is not put)
        const uint32_t c = min(c0 + j * kWaves, all - 1), r = row_of(c);
        const int pair = uniform(sh ? r0 + (int)r : (int)slist[r0 + r]);
        hp[j] = pick(sh, p.hs, p.h) + (size_t)pair * it.K;
        xo[j] = (size_t)(sh ? pair : pair / K) * m.x_stride;
        at[j] = min(k0 + (int)(c - r * pieces) * 256 + lane * 4, it.K - 4);
      }
      if (down) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = get4_shared(hp[j] + at[j]);
      } else if (m.x_bf16) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = load4(static_cast<const uint16_t*>(m.x) + xo[j] + at[j]);
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = load4(static_cast<const float*>(m.x) + xo[j] + at[j]);
      }
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const uint32_t c = c0 + j * kWaves, r = row_of(c);
        const int k = (int)(c - r * pieces) * 256 + lane * 4;
        if (c >= all || k >= kn) continue;
        char* const to = smem + r * parts * pitch + k * 2;
        put_parts(k0 + k < it.K ? v[j] : f32x4{0.f, 0.f, 0.f, 0.f}, to, pitch, parts);
      }
    }
  };
  // Until the flags of an up entry's hidden rows are all set.  Bounded (about ten
  // seconds; once it has run out, one look an entry): should one ever be lost, the
  // kernel ends, and what it adds to y for that entry is NaN.
  auto flags_of = [&](int u) __attribute__((always_inline)) {
    return pick(u < nshu, u * ns, nsup + (u - nshu) * nf) * WR;
  };
  int looks = p.looks;
  auto wait_hidden = [&](int u) __attribute__((always_inline)) {
    const int n = pick(u < nshu, ns, nf) * WR;
    const int32_t* const flags = p.up_done + flags_of(u);
#pragma unroll 1
    for (int look = 0; look < looks; ++look) {
      int ok = 1;
      for (int i = tid; i < n; i += kThreads)
        ok &= __hip_atomic_load(flags + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (__syncthreads_and(ok)) return 1.f;
    }
    looks = min(looks, 1);
    return __uint_as_float(0x7FC00000u);
  };

  Line buf[NL];
  Item it = item_of(cur);
  if (cur < total) {
    enter(it);
#pragma unroll
    for (int q = 0; q < kAhead; ++q) load(buf[q], q, true);
  }
  int run = cur;             // the first of the run's blocks
  int next = -1, nend = -1;  // the run after it; -1: not drawn, total: none
  int staged = p.early ? 0 : -1;  // whose rows are in LDS, all of them
  int waited = -1;           // the up entry whose hidden rows are known to be written,
  float there = 1.f;         // and 1, or NaN where they were waited for in vain
  int parity = 1;  // (the first run's place is still being read)
#pragma unroll 1
  while (cur < total) {
    // A run is drawn (its number is here by the end of a block) when fewer than two
    // blocks after this one are known, so that the next one's weights are always
    // on the way; no earlier, for the long ones to be shared out evenly.
    const bool last = cur + 1 == end;
    const bool draws = next < 0 ? cur + 2 >= end : last && nend - next == 1;
    if (draws && tid == 0)
      pending = __hip_atomic_fetch_add(p.queues + (phase * kQueues + queue) * kSpread, 1,
                                       __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const int coming = last ? next : cur + 1;  // the block after this one
    const bool known = coming >= 0 && coming < total;
    const bool sh = of_shared(it);
    const int r0 = uniform(sstart[it.u]), info = uniform(srows[it.u]);
    const int rows = info & 31, above = info >> 5;
    const int parts = !it.down && m.x_bf16 ? 1 : kParts;
    const int cols = rows * parts;
    // turns of NL lines a wave, and how many of them have their rows in LDS at a
    // time (at least one)
    constexpr int per = NL * WK * LK * 2;
    const int lines = src.lines, turns = (lines + NL * WK - 1) / (NL * WK);
    const int chunk = min((p.xbytes / cols - 16) / per, turns);
    const int pitch = min(chunk * per, lines * LK * 2) + 16;
    // one token's x is the same for every expert
    const bool all = chunk == turns;
    const int whose = it.down ? it.u + 1 : (T == 1 ? 0 : -2 - it.u);
    const bool keep = all && whose == staged;
    f32x4 acc[2] = {};  // of every other line
    const char* const xat = smem + (r16 < cols ? r16 : 0) * pitch + kq * NF * 16;
    Item nit = it;

    int in = 0, l0 = 0;  // turns in this chunk, its first line
#pragma unroll 1
    for (int j = 0; j < turns; ++j) {
      if (in == 0 && !keep) {
        if (it.down && above != waited) there = wait_hidden(above);
        else if (j > 0) __syncthreads();  // what is there has been read
        waited = pick(it.down != 0, above, waited);
        l0 = j * NL * WK;
        put_rows(it, r0, rows, l0 * LK, min(chunk * (per / 2), (lines - l0) * LK), pitch, parts);
        __syncthreads();
      }
      in = in + 1 == chunk ? 0 : in + 1;
      const bool ends = j + 1 == turns;
#pragma unroll
      for (int q = 0; q < NL; ++q) {
        // kAhead lines ahead, in the last turn the next block's
        if (q == 1 && ends && known) {
          nit = item_of(coming);
          enter(nit);
        }
        const bool over = q > 0 && ends;
        load(buf[(q + kAhead) % NL], pick(over, q - 1, j * NL + q + kAhead), !over || known);
        compute(buf[q], acc[q & 1], j * NL + q, lines, xat, l0);
      }
    }
    staged = all ? whose : -1;

    // the waves' sums (two places in turn: the last item's may still be read)
    f32x4* const red = reinterpret_cast<f32x4*>(smem + p.xbytes) + parity * kThreads;
    int* const drawn = stick + 2 * parity;
    parity ^= 1;
    red[tid] = acc[0] + acc[1];
    if (draws && w == 0) draw(uniform(pending), drawn);
    __syncthreads();
    if (wk == 0) {
      // lane (r, q): columns 4 q .. + 3 of token row r
      const int r = lane >> 2, q = lane & 3;
      const bool live = r < rows;
      f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
      for (int i = 0; i < parts; ++i) {
#pragma unroll
        for (int j = 0; j < WK; ++j)
          v += red[(w + j) * 64 + q * 16 + (live ? r * parts + i : 0)];
      }
      const int pair = live ? (sh ? r0 + r : slist[r0 + r]) : 0;
      const int group = it.blk * WR + wr;
      if (!it.down) {
        float* const hrow = pick(sh, p.hs, p.h) + (size_t)pair * pick(sh, S, F);
        f32x4 o;
        if (gated) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            o[i] = v[i] / (1.f + expf(-v[i])) * __shfl_xor(v[i], 2, 64);
          if (live && q < 2) put4_shared(hrow + group * 8 + 4 * q, o);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = v[i] < 0.f ? 0.f : v[i] * v[i];
          if (live) put4_shared(hrow + group * 16 + 4 * q, o);
        }
      } else if (live) {
        put4_shared(p.o + (size_t)(sh ? P + pair : pair) * D + group * 16 + 4 * q,
                    v * ((sh ? 1.f : sw[pair]) * there));
      }
      if (last) {
        // the run is written: a lane tells of each of its blocks
        stores_done();
        const int i = run + lane;
        if (!it.down) {
          if (i < end)
            __hip_atomic_store(p.up_done + i * WR + wr, 1, __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_AGENT);
        } else {
          int before = 0;
          if (i < end)
            before = __hip_atomic_fetch_add(p.down_done + ((i - nup) % nd * WR + wr) * kSpread, 1,
                                            __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          // Where all pairs' rows of a block's columns are there, they are added: a
          // lane a column of one of four tokens, or every second or fourth row of it
          // where there are two tokens or one.
          const int G = T == 1 ? 4 : T == 2 ? 2 : 1, part = kq & (G - 1);
          for (uint64_t done = __ballot(i < end && before == nexp - 1); done; done &= done - 1) {
            const int n0 = ((run + __builtin_ctzll(done) - nup) % nd * WR + wr) * 16;
            const float* const at = p.o + n0 + r16;
#pragma unroll 1
            for (int t0 = 0; t0 < T; t0 += 4 / G) {
              const int t = t0 + (G == 1 ? kq : G == 2 ? kq >> 1 : 0), tr = min(t, T - 1);
              float s = S > 0 && part == 0 ? get1_shared(at + (size_t)(P + tr) * D) : 0.f;
#pragma unroll 1
              for (int k0 = part; k0 - part < K; k0 += 8 * G) {
                float a[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  a[i] = get1_shared(at + (size_t)(tr * K + min(k0 + G * i, K - 1)) * D);
#pragma unroll
                for (int i = 0; i < 8; ++i) s += k0 + G * i < K ? a[i] : 0.f;
              }
              if (G > 1) s += __shfl_xor(s, 16, 64);
              if (G > 2) s += __shfl_xor(s, 32, 64);
              if (part == 0 && t < T) {
                const size_t to = (size_t)t * D + n0 + r16;
                if (m.y_bf16) static_cast<uint16_t*>(m.y)[to] = f32_to_bf16(s);
                else static_cast<float*>(m.y)[to] = s;
              }
            }
          }
        }
      }
    }
    const int db = draws ? uniform(drawn[0]) : -1, de = draws ? uniform(drawn[1]) : -1;
    if (!last) {
      cur += 1;
      if (draws) next = db, nend = de;
    } else {
      const bool had = next >= 0;
      cur = run = pick(had, next, db);
      end = pick(had, nend, de);
      next = pick(had, db, -1);
      nend = pick(had, de, -1);
    }
    it = nit;
    if (!known && cur < total) {
      it = item_of(cur);
      enter(it);
#pragma unroll
      for (int q = 0; q < kAhead; ++q) load(buf[q], q, true);
    }
  }
}

namespace {

template <class F>
void with_format(int format, F f) {
  if (format == 0) f(std::integral_constant<int, 0>{});
  else if (format == 1) f(std::integral_constant<int, 1>{});
  else f(std::integral_constant<int, 2>{});
}

struct Layout {
  size_t sync, logits, h, hs, o, total;
  int nsync, up_done, down_done;  // ints: counters and flags, and where they begin
};
Layout layout(const MoeTokens& m) {
  Layout l{};
  auto take = [&](size_t bytes) {
    const size_t at = l.total;
    l.total += (bytes + 255) / 256 * 256;
    return at;
  };
  const size_t pairs = (size_t)m.T * m.r.K;
  const size_t used = pairs < (size_t)m.r.E ? pairs : m.r.E;
  l.down_done = 2 * kQueues * kSpread;
  l.up_done = l.down_done + m.D / 16 * kSpread;
  // a flag for each 8 (gated) or 16 hidden columns of an entry (an expert has one for
  // every kTurn rows, and one more)
  const size_t entries = used + pairs / kTurn, shared = m.S ? 1 + m.T / kTurn : 0;
  l.nsync = l.up_done + (int)((entries * m.F + shared * m.S) / (m.gated ? 8 : 16));
  l.sync = take((size_t)l.nsync * 4);
  l.logits = take((size_t)m.T * m.r.E * 4);
  l.h = take(pairs * m.F * 4);
  l.hs = take((size_t)m.T * m.S * 4);
  l.o = take((pairs + (m.S ? m.T : 0)) * m.D * 4);
  return l;
}

}  // namespace

int moe_tokens_looks = 1 << 22;

size_t moe_tokens_workspace(const MoeTokens& m) { return layout(m).total; }

hipError_t moe_tokens(const MoeTokens& m, void* workspace, hipStream_t s) {
  const Layout l = layout(m);
  char* const ws = static_cast<char*>(workspace);
  int32_t* const sync = reinterpret_cast<int32_t*>(ws + l.sync);
  const int P = m.T * m.r.K, E = m.r.E;
  // LDS: the tokens' rows and the waves' sums, in whose room the tokens are
  // routed before; then the lists
  // Routed here: a second pass of a wave, or eight tokens' logits of 512 experts in every
  // work-group, cost more than a launch (T = 6 of 512 experts: 368 us against 341 + 5; T =
  // 13 of 128: 68 against 64 + 5 and the gap between two kernels).
  const bool here = E <= 128 || (E <= 512 && m.T <= 4);
  const int nj = !here ? 0 : (E <= 128 ? 2 : 8);
  const int route = kWaves * (256 + nj * 512) + 8 * E + 4 * P;
  const int down_cols = (m.T < kTurn ? m.T : kTurn) * kParts;
  const int cols = m.x_bf16 && m.T > down_cols ? m.T : down_cols;
  const int red = 2 * kThreads * 16, lists = m.x_bf16 && m.T > kTurn ? 18 * P + 288 : 12 * P + 192;
  // One work-group a CU or two.  One starts sooner (each routes and stages for itself),
  // two keep more on the way.  512 experts top-22 of 2048 x 5120, one against two: MXFP4 T = 1
  // (245 MB) 78 us and 91, T = 2 (460 MB) 130 and 146, T = 4 (840 MB) 210 and 208; FP8 T = 1 105
  // and 112, T = 2 (860 MB) 184 and 180, T = 6 405 and 364; bf16 T = 1 (920 MB) 162 and 167, T =
  // 2 308 and 294, T = 4 625 and 583.  Many tokens, 128 experts top-8 (T = 13, MXFP4, 168 MB): 79
  // and 71.
  // The shared expert is not counted: of one of 1.07 GB (bf16, 8192 x 32768) T = 2 takes
  // 291 us and 283, T = 4 323 and 340.
  const double mb = 1e-6 * (P < E ? P : E) * m.D * m.F * (m.gated ? 3 : 2) *
                    (m.format == 0 ? 2.0 : m.format == 1 ? 0.53 : 1.0);
  const bool few = m.T <= 4 && mb < (m.T == 1 ? 1200 : 700);
  const int room = (few ? 156 : 79) * 1024;
  const int least = cols * (2048 + 16), left = room - red - lists - kWaves * 2048;
  const int xbytes = (left > least ? left : least) / 16 * 16;
  const int turned = kWaves * 2048, work = xbytes + red + turned;
  // One token's x comes before the first block if all of it fits (in turns of 2048
  // bytes, as the kernel counts it) beside what routing takes.
  const int line = m.format == 1 ? 512 : m.format == 2 ? 256 : 128;  // bytes of x
  const int xparts = m.x_bf16 ? 1 : kParts, xrow = (m.D * 2 + line - 1) / line * line;
  const bool fits = (xbytes / xparts - 16) / 2048 >= (xrow + 2047) / 2048 &&
                    xparts * (xrow + 16) + route <= work;
  const int early = m.T == 1 && fits ? xparts * (xrow + 16) : 0;
  MoeParams p{m,
              reinterpret_cast<float*>(ws + l.logits),
              reinterpret_cast<float*>(ws + l.h),
              reinterpret_cast<float*>(ws + l.hs),
              reinterpret_cast<float*>(ws + l.o),
              sync,
              sync + l.up_done,
              sync + l.down_done,
              moe_tokens_looks,
              xbytes,
              xbytes + red,
              early,
              ((early + route > work ? early + route : work) + 15) / 16 * 16};
  const int lds = p.misc + lists;
  auto logits = [&](auto g, auto x) {
    using GT = decltype(g);
    using XT = decltype(x);
    moe_logits_kernel<GT, XT><<<dim3(E, (m.T + kLogitTokens - 1) / kLogitTokens), 256, 0, s>>>(
        static_cast<const XT*>(m.x), m.x_stride, static_cast<const GT*>(m.gate), m.T, E, m.D,
        p.logits, sync, l.nsync);
  };
  if (m.gate_bf16 && m.x_bf16) logits(uint16_t{}, uint16_t{});
  else if (m.gate_bf16) logits(uint16_t{}, float{});
  else if (m.x_bf16) logits(float{}, uint16_t{});
  else logits(float{}, float{});
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (!here) {
    e = route_logits(m.r, p.logits, false, m.bias, m.idx, m.weights, s);
    if (e != hipSuccess) return e;
  }
  const int grid = few ? 256 : 512;
  with_format(m.format, [&](auto fmt) {
    constexpr int FMT = decltype(fmt)::value;
    if (nj == 0) moe_tokens_kernel<FMT, 0><<<grid, kThreads, lds, s>>>(p);
    else if (nj == 2) moe_tokens_kernel<FMT, 2><<<grid, kThreads, lds, s>>>(p);
    else moe_tokens_kernel<FMT, 8><<<grid, kThreads, lds, s>>>(p);
  });
  return hipGetLastError();
}

}  // namespace lmoe
