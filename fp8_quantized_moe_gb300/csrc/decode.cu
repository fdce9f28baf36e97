// The expert FFN of a decoding step (sm_103a): moe_ffn_decode
//   y[t] = bf16( sum_j w[t, j] Wo[e] (silu(W0[e] x[t]) * (W1[e] x[t])) ),  e = ids[t, j]
// for a few tokens, on bf16 activations and quantised expert weights (e4m3 or
// int8 with per-channel, blockwise or static scales, MXFP8, MXFP4).
//
// With a few tokens the weights of the chosen experts are all that matters:
// 3 D F bytes an expert (half for MXFP4), read once, against a few flops a
// byte.  So nothing is quantised here, the weights stream through shared
// memory at the rate of HBM, and everything else has to fit beside that
// stream.  Two kernels, each one persistent CTA per SM:
//   kernel 1 (PHASE 1)  h = silu(W0 x) * (W1 x) of every (token, expert) pair,
//                       fp32, into the workspace;
//   kernel 2 (PHASE 2)  o = Wo h of every pair, fp32, into the workspace; the
//                       CTA that finishes the last expert of a block of output
//                       columns sums the block's pairs with their weights, in
//                       ascending j, and writes y.
// Kernel 2 is launched while kernel 1 runs (programmatic launch): as a CTA of
// kernel 1 leaves its SM, one of kernel 2 fills its ring with the first
// weights of wo and only then waits for kernel 1's results.
//
// Every CTA first sorts the pairs by expert for itself (at most 1024): a
// chunk is up to `cap` pairs of one expert, a unit of work one chunk and one
// block of RB weight rows (PHASE 1: RB/2 channels of wi_0 and the same of
// wi_1), all of K.  Units of the same rows are adjacent, so that two chunks of
// one expert read its weights together.
//
// Roles: warp 0 moves the stages (TMA boxes of 128-byte weight rows, 16 KB a
// stage; bulk copies of the activations' rows and of the weight scales).
// Warps 1..4 turn the stage's activations into f16, each (row, 128-byte span
// of the weights) scaled by the power of two that puts its largest value in
// [2^14, 2^15): f16 then holds every bf16 value to within 2^-39 of the span's
// largest, and h to 2^-12 relative (against 2^-9 of the result's bf16).
// Warps 5..12 contract: ldmatrix brings 16 rows x 32 bytes of weights, one
// conversion makes two f16 weights (exact for e4m3, int8 and e2m1, NaN codes
// included), and mma.m16n8k16 multiplies them with eight tokens.  The tensor
// core is nowhere near its limit, so the plain warp-wide MMA serves: its
// operands come from registers, where the weights are converted, and its M is
// only 16.  In PHASE 1 rows 0..7 of a fragment are wi_0 channels and rows
// 8..15 the same wi_1 channels, so a thread holds both factors of its h.
// Span sums are scaled (weight block scale, activation span scale) into fp32
// accumulators.
//
// RB = 32 (8 warps = 2 row tiles x 4 spans of K, summed at the end) makes
// small units, for few of them; RB = 128 (8 row tiles) reads the activations
// a quarter as often.
//
// Every wait is bounded; on expiry the kernel raises MOE_DEVERR_TIMEOUT, lets
// its copies land and returns.
#include <cudaTypedefs.h>

#include <mutex>

#include "mx4.cuh"

namespace moe {
namespace {

__device__ unsigned int g_err;

constexpr int kConvWarps = 4, kMmaWarps = 8;
constexpr int kThreads = 32 * (1 + kConvWarps + kMmaWarps);
constexpr int kStageW = 16384;  // weight bytes of a stage
constexpr int kMaxStages = 10;
constexpr int kMaxPairs = 1024;
constexpr int kMaxTokens = 64;
constexpr int kMaxExperts = 1024;
constexpr int kSmemLimit = 232448;

enum { kE4M3 = 0, kInt8 = 1, kMx8 = 2, kMx4 = 3 };
enum { kScaleChannel = 0, kScaleBlock = 1, kScaleTensor = 2, kScaleMx = 3 };

struct Params {
  const void* act;  // PHASE 1: x bf16 [T, K]; PHASE 2: h fp32 [slots, K]
  const int32_t* ids;
  const float* topk_w;
  const float* scale;  // fp32 scales, or the MX scale words
  float* out;          // PHASE 1: h [slots, F]; PHASE 2: o [slots, D]
  uint16_t* y;
  unsigned int* count;  // finished units of every block of output rows (PHASE 1 clears them)
  int ncount;
  int T, k, E, g0, El;
  int K, N;  // N: channels (PHASE 1: F, PHASE 2: D)
  int mode;
  int cap, stages, pitch;  // pairs a chunk; bytes of an activation row in shared memory
};

struct Ctl {
  uint64_t full[kMaxStages], xfull[kMaxStages], empty[kMaxStages];
  int abort_flag, no_abort, err, nchunk, last;
  int pad[3];
  uint16_t pos[kMaxPairs];     // slot of pair i (pairs sorted by expert), 0xFFFF: not local
  uint16_t order[kMaxPairs];   // pair of slot s
  uint16_t cexp[kMaxPairs], cstart[kMaxPairs], cnum[kMaxPairs];
  uint16_t num[kMaxExperts];
};

template <int WT, int PHASE, int RB>
struct Cfg {
  static constexpr int ROWTILES = RB / 16, SUBS = kMmaWarps / ROWTILES;
  static constexpr int KE = WT == kMx4 ? 256 : 128;   // values of K in 128 bytes of weights
  static constexpr int KC = KE / 8;                   // and in a 16-byte chunk
  static constexpr int ES = PHASE == 1 ? 2 : 4;       // bytes of an activation as it arrives
  static constexpr int STAGE_K = SUBS * KE;
  static constexpr int SPANS = KE / 128;              // scale words of a row and sub-tile
  static constexpr int SCALE_BYTES = SUBS * SPANS * RB * 4;
  static constexpr int PAD = WT == kMx4 ? 64 : 32;    // keeps eight rows' fragments in different banks
  static constexpr int PITCH = STAGE_K * ES + PAD;
  static constexpr int RED_BYTES = SUBS > 1 ? 2 * kMmaWarps * 32 * 16 : 0;
  static_assert(SUBS * RB * 128 == kStageW, "stage");
};

constexpr size_t kCtlBytes = (sizeof(Ctl) + 127) / 128 * 128;

__device__ __forceinline__ void grid_dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts64(uint32_t a, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void sts32f(uint32_t a, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Four weights (one 32-bit word of codes) -> two f16 pairs.
template <int WT>
__device__ __forceinline__ void weights4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (WT == kInt8) {
    // b + 128 under the exponent of 1024 is the f16 1152 + b
    const uint32_t u = w ^ 0x80808080u;
    asm("{\n\t.reg .b32 a, b;\n\t"
        "prmt.b32 a, %2, 0x64646464, 0x4140;\n\t"
        "prmt.b32 b, %2, 0x64646464, 0x4342;\n\t"
        "sub.rn.f16x2 %0, a, %3;\n\t"
        "sub.rn.f16x2 %1, b, %3;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(u), "r"(0x64806480u));
  } else {
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}

// Eight e2m1 weights -> four f16 pairs.
__device__ __forceinline__ void weights8(uint32_t w, uint32_t (&v)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
      : "r"(w));
}

// ---- the pairs by expert ---------------------------------------------------
// A stable counting sort by warp 0: 32 pairs at a time, the rank of a pair
// among its expert's earlier ones from a warp-wide match and a running count.
// Every CTA of both kernels gets the same tables.
__device__ void build_chunks(const Params& p, Ctl* c) {
  const int lane = threadIdx.x & 31;
  const int R = p.T * p.k;
  // c->order holds the local expert of every pair (0xFFFF: none) until the slots are known
  for (int i0 = 0; i0 < R; i0 += 32) {
    const int i = i0 + lane;
    const int e = i < R ? c->order[i] : 0xFFFF;
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    const int rank = __popc(same & ((1u << lane) - 1u));
    if (e != 0xFFFF) {
      const int before = c->num[e];
      c->pos[i] = static_cast<uint16_t>(before + rank);
    }
    __syncwarp();
    if (e != 0xFFFF && (same >> lane) == 1u)  // the last of its expert in this batch
      c->num[e] = static_cast<uint16_t>(c->pos[i] + 1);
    __syncwarp();
  }
  int slots = 0, chunks = 0;
  for (int e0 = 0; e0 < p.El; e0 += 32) {
    const int e = e0 + lane;
    const int n = e < p.El ? c->num[e] : 0;
    const int nc = (n + p.cap - 1) / p.cap;
    int in = n, ic = nc;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, in, o), b = __shfl_up_sync(0xffffffffu, ic, o);
      if (lane >= o) {
        in += a;
        ic += b;
      }
    }
    const int off = slots + in - n, c0 = chunks + ic - nc;
    for (int j = 0; j < nc; ++j) {
      c->cexp[c0 + j] = static_cast<uint16_t>(e);
      c->cstart[c0 + j] = static_cast<uint16_t>(off + j * p.cap);
      c->cnum[c0 + j] = static_cast<uint16_t>(min(p.cap, n - j * p.cap));
    }
    if (e < p.El) c->num[e] = static_cast<uint16_t>(off);
    slots += __shfl_sync(0xffffffffu, in, 31);
    chunks += __shfl_sync(0xffffffffu, ic, 31);
  }
  if (lane == 0) c->nchunk = chunks;
  __syncwarp();
  for (int i0 = 0; i0 < R; i0 += 32) {
    const int i = i0 + lane;
    if (i < R) {
      const int e = c->order[i];
      c->pos[i] = e == 0xFFFF ? 0xFFFF : static_cast<uint16_t>(c->num[e] + c->pos[i]);
    }
  }
  __syncwarp();
  for (int i0 = 0; i0 < R; i0 += 32) {  // (the experts in `order` are no longer needed)
    const int i = i0 + lane;
    if (i < R && c->pos[i] != 0xFFFF) c->order[c->pos[i]] = static_cast<uint16_t>(i);
  }
}

template <int WT, int PHASE, int RB, int NT>
struct Mma {
  using C = Cfg<WT, PHASE, RB>;

  // One sub-tile: 16 rows x nch 16-byte chunks (at most 8) of weights at `wt`
  // (row A + lane / 4 and row B + lane / 4 of the fragment), activations at
  // `xb` (already this lane's), the weights' scale words of this lane's two
  // rows at sA, sB and the activations' span scales at `xs`.
  static __device__ __forceinline__ void sub_tile(float (&acc)[NT][4], uint32_t wt, uint32_t swz, uint32_t xb,
                                                  int pitch8, int nch, uint32_t sA, uint32_t sB, uint32_t xs,
                                                  int mode) {
    float blk[NT][4], sum[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) blk[n][i] = sum[n][i] = 0.0f;
    const int hi = (threadIdx.x >> 4) & 1;  // lanes 16..31 address the second chunk of a pair
    uint32_t wA = 0, wB = 0;
#pragma unroll
    for (int c = 0; c < 8; c += 2) {
      if (c >= nch) break;
      if (WT == kMx8 || WT == kMx4) {
        if (c == 0 || (WT == kMx4 && c == 4)) {
          wA = lds32(sA + (c == 4 ? RB * 4 : 0));
          wB = lds32(sB + (c == 4 ? RB * 4 : 0));
        }
      }
      uint32_t r[4];
      ldmatrix_x4(wt + (((c + hi) * 16) ^ swz), r);
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        if (WT != kMx8 && WT != kMx4 && c + cc >= nch) break;
        if (WT == kMx4) {
          uint32_t va[4], vb[4];
          weights8(r[2 * cc], va);
          weights8(r[2 * cc + 1], vb);
          const uint32_t a0[4] = {va[0], vb[0], va[1], vb[1]}, a1[4] = {va[2], vb[2], va[3], vb[3]};
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint4 b = lds128(xb + n * pitch8 + (c + cc) * 64);
            mma_f16(blk[n], a0, b.x, b.y);
            mma_f16(blk[n], a1, b.z, b.w);
          }
        } else {
          uint32_t a[4];
          weights4<WT>(r[2 * cc], a[0], a[2]);
          weights4<WT>(r[2 * cc + 1], a[1], a[3]);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint2 b = lds64(xb + n * pitch8 + (c + cc) * 32);
            mma_f16(blk[n], a, b.x, b.y);
          }
        }
        if (WT == kMx4 || (WT == kMx8 && cc == 1)) {  // a 32-wide block is done: its scales
          const int b = WT == kMx4 ? (c + cc) & 3 : c / 2;
          const float fa = e8m0_value((wA >> (8 * b)) & 0xFFu), fb = e8m0_value((wB >> (8 * b)) & 0xFFu);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            sum[n][0] = __fmaf_rn(blk[n][0], fa, sum[n][0]);
            sum[n][1] = __fmaf_rn(blk[n][1], fa, sum[n][1]);
            sum[n][2] = __fmaf_rn(blk[n][2], fb, sum[n][2]);
            sum[n][3] = __fmaf_rn(blk[n][3], fb, sum[n][3]);
            blk[n][0] = blk[n][1] = blk[n][2] = blk[n][3] = 0.0f;
          }
        }
      }
    }
    float fa = 1.0f, fb = 1.0f;
    if (WT == kE4M3 || WT == kInt8) {
      if (mode == kScaleBlock) {
        fa = __uint_as_float(lds32(sA));
        fb = __uint_as_float(lds32(sB));
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint2 s = lds64(xs + n * 32);
      const float s0 = __uint_as_float(s.x), s1 = __uint_as_float(s.y);
      if (WT == kMx8 || WT == kMx4) {
        acc[n][0] = __fmaf_rn(sum[n][0], s0, acc[n][0]);
        acc[n][1] = __fmaf_rn(sum[n][1], s1, acc[n][1]);
        acc[n][2] = __fmaf_rn(sum[n][2], s0, acc[n][2]);
        acc[n][3] = __fmaf_rn(sum[n][3], s1, acc[n][3]);
      } else {
        acc[n][0] = __fmaf_rn(blk[n][0], s0 * fa, acc[n][0]);
        acc[n][1] = __fmaf_rn(blk[n][1], s1 * fa, acc[n][1]);
        acc[n][2] = __fmaf_rn(blk[n][2], s0 * fb, acc[n][2]);
        acc[n][3] = __fmaf_rn(blk[n][3], s1 * fb, acc[n][3]);
      }
    }
  }
};

template <int WT, int PHASE, int RB>
__global__ void __launch_bounds__(kThreads, 1) decode_kernel(const __grid_constant__ CUtensorMap tmW, const Params p) {
  using C = Cfg<WT, PHASE, RB>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* bp = smem_raw + (base - raw);
  // stages of weights | activations | weight scales | activation span scales | control | partial sums
  const uint32_t S = p.stages;
  const int cap = p.cap;
  const uint32_t x_ring = base + S * kStageW;
  const uint32_t x_bytes = cap * C::PITCH;
  const uint32_t s_ring = x_ring + S * x_bytes;
  const uint32_t v_ring = s_ring + S * C::SCALE_BYTES;  // [stage][sub][cap] floats
  const uint32_t v_bytes = C::SUBS * cap * 4;
  Ctl* ctl = reinterpret_cast<Ctl*>(bp + (v_ring + S * v_bytes - base));
  float* red = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(ctl) + kCtlBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int R = p.T * p.k;

  if (PHASE == 1) {
    grid_dep_launch();
    if (blockIdx.x == 0)
      for (int i = threadIdx.x; i < p.ncount; i += kThreads) p.count[i] = 0;
  }
  if (threadIdx.x == 0) {
    for (uint32_t s = 0; s < S; ++s) {
      mbar_init(smem_u32(&ctl->full[s]), 1);
      mbar_init(smem_u32(&ctl->xfull[s]), kConvWarps);
      mbar_init(smem_u32(&ctl->empty[s]), kMmaWarps);
    }
    ctl->abort_flag = 0;
    ctl->no_abort = 0;
    ctl->err = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmW);
  }
  for (int i = threadIdx.x; i < R; i += kThreads) {
    const int id = __ldg(p.ids + i), e = id - p.g0;
    if (PHASE == 1 && blockIdx.x == 0 && (id < 0 || id >= p.E)) raise_error(&g_err, MOE_DEVERR_BAD_EXPERT_ID);
    ctl->order[i] = (id >= 0 && id < p.E && e >= 0 && e < p.El) ? static_cast<uint16_t>(e) : 0xFFFF;
  }
  for (int i = threadIdx.x; i < p.El; i += kThreads) ctl->num[i] = 0;
  __syncthreads();
  if (warp == 0) build_chunks(p, ctl);
  __syncthreads();

  const int nchunk = ctl->nchunk;
  const int rows_per = PHASE == 1 ? RB / 2 : RB;  // channels of a unit
  const int nblock = (p.N + rows_per - 1) / rows_per;
  const int total = nchunk * nblock;
  const int nst = (p.K + C::STAGE_K - 1) / C::STAGE_K;
  volatile int* abort_flag = &ctl->abort_flag;
  bool timed_out = false;

  if (PHASE == 2 && nchunk == 0) {  // no local expert was chosen at all
    grid_dep_wait();
    const int64_t n = static_cast<int64_t>(p.T) * p.N;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * kThreads)
      p.y[i] = 0;
    return;
  }

  if (warp == 0) {
    // ------------------------------------------------------------- producer
    const bool words = p.mode == kScaleBlock || p.mode == kScaleMx;  // scales along K, one word a row and 128 values
    const int nkb = p.K / 128;                                        // (only used with such scales: K % 128 == 0)
    const int64_t scale_rows = static_cast<int64_t>(PHASE == 1 ? 2 * p.N : p.N);
    // bytes of stage kst of a chunk of n pairs
    auto valid_subs = [&](int kst) { return min(C::SUBS, (p.K - kst * C::STAGE_K + C::KE - 1) / C::KE); };
    auto valid_kb = [&](int kst) { return min(C::SUBS * C::SPANS, nkb - kst * C::SUBS * C::SPANS); };
    auto x_len = [&](int kst) { return min(C::STAGE_K, p.K - kst * C::STAGE_K) * C::ES; };
    auto load_weights = [&](int s, int ch, int blk, int kst) {
      const int e = ctl->cexp[ch], n = ctl->cnum[ch], c0 = blk * rows_per;
      const uint32_t fb = smem_u32(&ctl->full[s]);
      const int subs = valid_subs(kst), kbs = words ? valid_kb(kst) : 0;
      if (lane == 0)
        mbar_arrive_expect_tx(fb, subs * RB * 128 + n * x_len(kst) + kbs * RB * 4);
      __syncwarp();
      const uint32_t dst = base + s * kStageW;
      constexpr int kBoxes = PHASE == 1 ? 2 : 1;
      if (lane < subs * kBoxes) {
        const int sub = lane / kBoxes, half = lane % kBoxes;
        const int row = PHASE == 1 ? e * 2 * p.N + half * p.N + c0 : e * p.N + c0;
        tma_load_2d(dst + sub * RB * 128 + half * (RB / 2) * 128, &tmW, (kst * C::SUBS + sub) * 128, row, fb);
      }
      if (lane < kbs * kBoxes) {
        const int kb = lane / kBoxes, half = lane % kBoxes;
        const int64_t gkb = kst * C::SUBS * C::SPANS + kb;
        const int64_t n0 = (PHASE == 1 ? half * p.N : 0) + c0;
        const float* src = p.mode == kScaleMx ? p.scale + gkb * (p.El * scale_rows) + e * scale_rows + n0
                                              : p.scale + (static_cast<int64_t>(e) * nkb + gkb) * scale_rows + n0;
        bulk_load(s_ring + s * C::SCALE_BYTES + (kb * RB + half * (RB / 2)) * 4, src, rows_per * 4, fb);
      }
    };
    auto load_acts = [&](int s, int ch, int kst) {
      const int n = ctl->cnum[ch], st = ctl->cstart[ch];
      const uint32_t fb = smem_u32(&ctl->full[s]);
      const uint32_t len = x_len(kst);
      for (int i = lane; i < n; i += 32) {
        const int64_t row = PHASE == 1 ? ctl->order[st + i] / p.k : st + i;
        bulk_load(x_ring + s * x_bytes + i * C::PITCH,
                  static_cast<const uint8_t*>(p.act) + (row * p.K + static_cast<int64_t>(kst) * C::STAGE_K) * C::ES,
                  len, fb);
      }
    };
    // the steps of this CTA in order: unit u, its chunk and row block, K stage kst
    struct Step {
      int u, ch, blk, kst;
    };
    auto begin = [&] {
      const int u = blockIdx.x;
      return Step{u, total ? u % nchunk : 0, total ? u / nchunk : 0, 0};
    };
    auto next = [&](Step& q) {
      if (++q.kst == nst) {
        q.kst = 0;
        q.u += gridDim.x;
        q.blk = q.u / nchunk;
        q.ch = q.u - q.blk * nchunk;
      }
    };
    uint32_t issued = 0;
    uint32_t s = 0, ph = 0;
    Step q = begin();
    if (PHASE == 2) {
      // the ring's first weights do not depend on kernel 1; its h does
      Step w = q;
      for (uint32_t i = 0; i < S && w.u < total; ++i, next(w)) load_weights(i, w.ch, w.blk, w.kst);
      grid_dep_wait();
      // h was written through the generic proxy and is read by bulk copies
      asm volatile("fence.proxy.async;" ::: "memory");
      for (; issued < S && q.u < total; ++issued, next(q)) load_acts(issued, q.ch, q.kst);
      ph = 1;  // a full ring is out; where it is not full, no step is left
    }
    for (; q.u < total; next(q), ++issued) {
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(&ctl->empty[s]), ph ^ 1, abort_flag, kWaitLimitNs))) {
        timed_out = true;
        break;
      }
      load_weights(s, q.ch, q.blk, q.kst);
      load_acts(s, q.ch, q.kst);
      if (++s == S) {
        s = 0;
        ph ^= 1;
      }
    }
    if (timed_out) {
      if (lane == 0) {
        *abort_flag = 1;
        ctl->err = 2;
        for (uint32_t j = issued > S ? issued - S : 0; j < issued; ++j)  // copies in flight land before the CTA exits
          mbar_wait_bounded(smem_u32(&ctl->full[j % S]), (j / S) & 1, &ctl->no_abort, kWaitLimitNs);
      }
      __syncwarp();
    }
  } else if (warp <= kConvWarps) {
    // ------------------------------------------------- activations to f16
    constexpr int PER = C::KE / 32;  // values a lane: 4 or 8
    uint32_t s = 0, ph = 0;
    for (int u = blockIdx.x; u < total && !timed_out; u += gridDim.x) {
      const int n = ctl->cnum[u % nchunk];
      for (int kst = 0; kst < nst; ++kst) {
        if (!mbar_wait_bounded_warp(smem_u32(&ctl->full[s]), ph, abort_flag, kWaitLimitNs)) {
          timed_out = true;
          break;
        }
        const int left = p.K - kst * C::STAGE_K;
        const int subs = min(C::SUBS, (left + C::KE - 1) / C::KE);
        for (int i = warp - 1; i < n * subs; i += kConvWarps) {
          const int sub = i / n, row = i - sub * n;
          const uint32_t at = x_ring + s * x_bytes + row * C::PITCH + sub * C::KE * C::ES;
          const bool ok = sub * C::KE + lane * PER < left;  // K is a multiple of 16: a lane's values are all in or out
          float v[PER];
#pragma unroll
          for (int j = 0; j < PER; ++j) v[j] = 0.0f;
          if (ok) {
            if (PHASE == 1) {
              uint32_t w[PER / 2];
              if (PER == 4) {
                const uint2 d = lds64(at + lane * 8);
                w[0] = d.x;
                w[1] = d.y;
              } else {
                const uint4 d = lds128(at + lane * 16);
                w[0] = d.x;
                w[1] = d.y;
                w[PER / 2 - 2] = d.z;
                w[PER / 2 - 1] = d.w;
              }
#pragma unroll
              for (int j = 0; j < PER / 2; ++j) {
                v[2 * j] = bf16lo(w[j]);
                v[2 * j + 1] = bf16hi(w[j]);
              }
            } else {
#pragma unroll
              for (int j = 0; j < PER / 4; ++j) {
                const uint4 d = lds128(at + lane * 4 * PER + 16 * j);
                v[4 * j] = __uint_as_float(d.x);
                v[4 * j + 1] = __uint_as_float(d.y);
                v[4 * j + 2] = __uint_as_float(d.z);
                v[4 * j + 3] = __uint_as_float(d.w);
              }
            }
          }
          // largest finite magnitude of the span; infinities and NaN pass through
          uint32_t m = 0;
#pragma unroll
          for (int j = 0; j < PER; ++j) {
            const uint32_t b = __float_as_uint(v[j]) & 0x7FFFFFFFu;
            m = max(m, b < 0x7F800000u ? b : 0u);
          }
          m = __reduce_max_sync(0xffffffffu, m);  // (all lanes have read the span, too)
          // 2^(14 - e), e = floor(log2(m)) held at or above -100
          const int e = max(static_cast<int>(m >> 23) - 127, -100);
          const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
#pragma unroll
          for (int j = 0; j < PER; ++j) v[j] = __fmul_rn(v[j], up);
          if (PER == 4)
            sts64(at + lane * 8, f16x2(v[0], v[1]), f16x2(v[2], v[3]));
          else
            sts128(at + lane * 16, make_uint4(f16x2(v[0], v[1]), f16x2(v[2], v[3]), f16x2(v[PER - 4], v[PER - 3]),
                                              f16x2(v[PER - 2], v[PER - 1])));
          if (lane == 0)
            sts32f(v_ring + s * v_bytes + (sub * cap + row) * 4, __uint_as_float(static_cast<uint32_t>(127 - 14 + e) << 23));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl->xfull[s]));
        if (++s == S) {
          s = 0;
          ph ^= 1;
        }
      }
    }
    if (timed_out) {
      *abort_flag = 1;
      ctl->err = 2;
    }
  } else {
    // ----------------------------------------------------------- contraction
    const int mw = warp - 1 - kConvWarps;
    const int tile = mw % C::ROWTILES, sub = mw / C::ROWTILES;
    const int g = lane >> 2, t4 = lane & 3;
    // rows of the fragment: 0..7 from row A, 8..15 from row B
    const int rowA = PHASE == 1 ? 8 * tile : 16 * tile, rowB = PHASE == 1 ? RB / 2 + 8 * tile : 16 * tile + 8;
    const int lrow = ((lane >> 3) & 1 ? rowB : rowA) + (lane & 7);  // the row this lane addresses for ldmatrix
    const uint32_t w_off = sub * RB * 128 + lrow * 128, swz = (lrow & 7) * 16;
    const uint32_t x_off = g * C::PITCH + sub * C::KE * C::ES + t4 * (WT == kMx4 ? 16 : 8);
    const uint32_t s_off = sub * C::SPANS * RB * 4;
    uint32_t s = 0, ph = 0;
    int parity = 0;
    if (PHASE == 2) grid_dep_wait();  // before o and the counters are touched

    auto unit = [&](auto nt_tag, int ch, int blk) {
      constexpr int NT = decltype(nt_tag)::value;
      float acc[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
      for (int kst = 0; kst < nst && !timed_out; ++kst) {
        if (!mbar_wait_bounded_warp(smem_u32(&ctl->full[s]), ph, abort_flag, kWaitLimitNs) ||
            !mbar_wait_bounded_warp(smem_u32(&ctl->xfull[s]), ph, abort_flag, kWaitLimitNs)) {
          timed_out = true;
          *abort_flag = 1;
          break;
        }
        const int left = p.K - (kst * C::SUBS + sub) * C::KE;
        const int nch = min(8, left / C::KC);  // K is a multiple of 16 (e2m1: 128): whole chunks
        if (nch > 0) {
          const uint32_t st = s_ring + s * C::SCALE_BYTES + s_off;
          Mma<WT, PHASE, RB, NT>::sub_tile(acc, base + s * kStageW + w_off, swz, x_ring + s * x_bytes + x_off,
                                           8 * C::PITCH, nch, st + (rowA + g) * 4, st + (rowB + g) * 4,
                                           v_ring + s * v_bytes + sub * cap * 4 + t4 * 8, p.mode);
        }
        fence_proxy_async_smem();  // this warp's reads of the stage before the next copies into it
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl->empty[s]));
        if (++s == S) {
          s = 0;
          ph ^= 1;
        }
      }
      if (C::SUBS > 1) {  // the spans of K meet in ascending order
        float4* r4 = reinterpret_cast<float4*>(red) + parity * kMmaWarps * 32;
        r4[mw * 32 + lane] = make_float4(acc[0][0], acc[0][1], acc[0][2], acc[0][3]);
        named_barrier_sync(1, kMmaWarps * 32);
        if (sub == 0) {
#pragma unroll
          for (int q = 1; q < C::SUBS; ++q) {
            const float4 v = r4[(q * C::ROWTILES + tile) * 32 + lane];
            acc[0][0] += v.x;
            acc[0][1] += v.y;
            acc[0][2] += v.z;
            acc[0][3] += v.w;
          }
        }
        parity ^= 1;  // the other half is free: every warp has passed this barrier since it was read
      }
      if (sub == 0) {
        const int e = ctl->cexp[ch], n = ctl->cnum[ch], st = ctl->cstart[ch];
        const int ca = blk * rows_per + (PHASE == 1 ? 8 * tile : 16 * tile) + g;  // channel of row A
        const int cb = PHASE == 1 ? ca : ca + 8;
        float fa = 1.0f, fb = 1.0f;
        if (p.mode == kScaleChannel) {
          const float* sc = p.scale + static_cast<int64_t>(e) * (PHASE == 1 ? 2 * p.N : p.N);
          if (ca < p.N) fa = __ldg(sc + ca);
          if (cb < p.N) fb = __ldg(sc + (PHASE == 1 ? p.N : 0) + cb);
        } else if (p.mode == kScaleTensor) {
          fa = fb = __ldg(p.scale);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int col = nt * 8 + 2 * t4 + j;
            if (col < n) {
              const float va = acc[nt][j] * fa, vb = acc[nt][2 + j] * fb;
              float* o = p.out + static_cast<int64_t>(st + col) * p.N;
              if (PHASE == 1) {
                if (ca < p.N) o[ca] = silu_f32(va) * vb;
              } else {
                if (ca < p.N) o[ca] = va;
                if (cb < p.N) o[cb] = vb;
              }
            }
          }
      }
    };

    // (a warp that gave up waiting still walks the units, without waits: the
    // other warps count on it at the barriers)
    for (int u = blockIdx.x; u < total; u += gridDim.x) {
      const int blk = u / nchunk, ch = u - blk * nchunk;
      const int n = ctl->cnum[ch];
      if (RB == 32 || n <= 8)
        unit(std::integral_constant<int, 1>{}, ch, blk);
      else if (n <= 16)
        unit(std::integral_constant<int, RB == 32 ? 1 : 2>{}, ch, blk);
      else
        unit(std::integral_constant<int, RB == 32 ? 1 : 4>{}, ch, blk);
      if (PHASE == 2) {
        // the block's last unit (over all CTAs) sums its pairs into y
        __threadfence();
        named_barrier_sync(1, kMmaWarps * 32);
        if (mw == 0 && lane == 0) ctl->last = atomicAdd(p.count + blk, 1u) == static_cast<unsigned>(nchunk - 1);
        named_barrier_sync(1, kMmaWarps * 32);
        if (ctl->last) {
          __threadfence();
          const int th = mw * 32 + lane, d0 = blk * RB;
          for (int i = th; i < p.T * RB; i += kMmaWarps * 32) {
            const int t = i / RB, d = d0 + i % RB;
            if (d >= p.N) continue;
            float a = 0.0f;
            for (int j = 0; j < p.k; ++j) {
              const int q = t * p.k + j;
              if (ctl->pos[q] == 0xFFFF) continue;
              const float w = p.topk_w ? __ldg(p.topk_w + q) : 1.0f;
              a = __fmaf_rn(w, __ldcg(p.out + static_cast<int64_t>(ctl->pos[q]) * p.N + d), a);
            }
            p.y[static_cast<int64_t>(t) * p.N + d] = static_cast<uint16_t>(pack_bf16x2(a, 0.0f) & 0xFFFFu);
          }
        }
      }
    }
    if (timed_out) {
      *abort_flag = 1;
      ctl->err = 2;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && ctl->err) raise_error(&g_err, MOE_DEVERR_TIMEOUT);
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// Weight rows as bytes: boxes of box_rows x 128 bytes, 128-byte swizzle;
// reads past the extents return zeros.
bool make_map(CUtensorMap* m, const void* ptr, uint64_t bytes, uint64_t rows, uint32_t box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {bytes, rows}, strides[1] = {bytes};
  cuuint32_t box[2] = {128, box_rows}, estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int WT, int PHASE, int RB>
moe_status launch(const void* w, Params p, int sms, cudaStream_t st) {
  using C = Cfg<WT, PHASE, RB>;
  CUtensorMap tm;
  const uint64_t bytes = WT == kMx4 ? p.K / 2 : p.K;
  if (!make_map(&tm, w, bytes, static_cast<uint64_t>(p.El) * (PHASE == 1 ? 2 : 1) * p.N, PHASE == 1 ? RB / 2 : RB))
    return MOE_ERR_CUDA;
  p.cap = RB == 32 || p.T <= 8 ? 8 : (p.T <= 16 ? 16 : 32);
  const size_t stage = kStageW + static_cast<size_t>(p.cap) * C::PITCH + C::SCALE_BYTES + C::SUBS * p.cap * 4;
  const size_t fixed = 1024 + kCtlBytes + C::RED_BYTES;
  p.stages = static_cast<int>((kSmemLimit - fixed) / stage);
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  const size_t smem = fixed + p.stages * stage;
  auto kernel = decode_kernel<WT, PHASE, RB>;
  MOE_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)));
  const int per = PHASE == 1 ? RB / 2 : RB;
  const int64_t units = static_cast<int64_t>(p.T) * p.k * ((p.N + per - 1) / per);  // at most: a chunk a pair
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(units < sms ? units : sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = PHASE == 2 ? 1 : 0;
  MOE_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, tm, p));
  return MOE_OK;
}

template <int WT, int PHASE>
moe_status launch_rb(const void* w, const Params& p, int rb, int sms, cudaStream_t st) {
  return rb == 32 ? launch<WT, PHASE, 32>(w, p, sms, st) : launch<WT, PHASE, 128>(w, p, sms, st);
}

template <int PHASE>
moe_status launch_type(int wt, const void* w, const Params& p, int rb, int sms, cudaStream_t st) {
  switch (wt) {
    case kE4M3: return launch_rb<kE4M3, PHASE>(w, p, rb, sms, st);
    case kInt8: return launch_rb<kInt8, PHASE>(w, p, rb, sms, st);
    case kMx8: return launch_rb<kMx8, PHASE>(w, p, rb, sms, st);
    default: return launch_rb<kMx4, PHASE>(w, p, rb, sms, st);
  }
}

// Workspace: h fp32 [R, F] | o fp32 [R, D] | a counter for every 32 output
// columns, each part 256-byte aligned.
int64_t align256(int64_t b) { return (b + 255) / 256 * 256; }
int64_t counters(int64_t D) { return (D + 31) / 32; }

bool shape_ok(int64_t T, int k, int64_t D, int64_t F) {
  return T >= 0 && T <= kMaxTokens && k > 0 && k <= 32 && T * k <= kMaxPairs && D > 0 && F > 0 && D % 16 == 0 &&
         F % 16 == 0 && D <= 32768 && F <= 32768;
}

// Scale mode of one weight tensor in the kernel's terms, -1 if it is not taken.
int scale_kind(int wt, int mode, int64_t K, int64_t N) {
  if (wt == kMx8 || wt == kMx4) return K % 128 == 0 && N % 128 == 0 ? kScaleMx : -1;
  if (mode == MOE_SCALE_PER_ROW) return kScaleChannel;
  if (mode == MOE_SCALE_PER_TENSOR) return kScaleTensor;
  return mode == MOE_SCALE_PER_ROW_BLOCK128 && K % 128 == 0 && N % 128 == 0 ? kScaleBlock : -1;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" __attribute__((visibility("hidden"))) cudaError_t moe_detail_take_error_decode(unsigned int* out) {
  unsigned int v = 0, z = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_err, sizeof(v));
  if (e == cudaSuccess && v) e = cudaMemcpyToSymbol(g_err, &z, sizeof(z));
  *out = v;
  return e;
}

extern "C" size_t moe_ffn_decode_workspace_bytes(int64_t T, int k, int64_t D, int64_t F) {
  if (!shape_ok(T, k, D, F)) return 0;
  return static_cast<size_t>(align256(T * k * F * 4) + align256(T * k * D * 4) + align256(counters(D) * 4));
}

extern "C" moe_status moe_ffn_decode(const uint16_t* x, const int32_t* topk_ids, const float* topk_w, int64_t T, int k,
                                     int E, int group_offset, int E_local, int64_t D, int64_t F,
                                     moe_weight_type type, const void* w_in, const void* s_in, moe_scale_mode in_mode,
                                     const void* w_out, const void* s_out, moe_scale_mode out_mode, uint16_t* y,
                                     void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  MOE_HOST_CHECK(x && topk_ids && w_in && s_in && w_out && s_out && y && workspace, MOE_ERR_INVALID_ARG);
  MOE_HOST_CHECK(shape_ok(T, k, D, F), MOE_ERR_INVALID_ARG);
  MOE_HOST_CHECK(E > 0 && E <= kMaxExperts && group_offset >= 0 && E_local > 0 && E_local <= E - group_offset,
                 MOE_ERR_INVALID_ARG);
  MOE_HOST_CHECK(type == MOE_WEIGHT_E4M3 || type == MOE_WEIGHT_INT8 || type == MOE_WEIGHT_MXFP8 ||
                     type == MOE_WEIGHT_MXFP4,
                 MOE_ERR_INVALID_ARG);
  const int kin = scale_kind(type, in_mode, D, F), kout = scale_kind(type, out_mode, F, D);
  MOE_HOST_CHECK(kin >= 0 && kout >= 0, MOE_ERR_INVALID_ARG);
  MOE_HOST_CHECK(static_cast<int64_t>(E_local) * 2 * F < (1ll << 31) && static_cast<int64_t>(E_local) * D < (1ll << 31),
                 MOE_ERR_INVALID_ARG);
  MOE_HOST_CHECK(aligned16(x) && aligned16(w_in) && aligned16(w_out) && aligned16(s_in) && aligned16(s_out) &&
                     aligned16(y) && aligned16(workspace),
                 MOE_ERR_INVALID_ARG);
  MOE_HOST_CHECK(workspace_bytes >= moe_ffn_decode_workspace_bytes(T, k, D, F), MOE_ERR_INVALID_ARG);
  int dev = 0, major = 0, minor = 0, sms = 0;
  MOE_CUDA_TRY(cudaGetDevice(&dev));
  MOE_CUDA_TRY(cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev));
  MOE_CUDA_TRY(cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev));
  MOE_CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  if (major != 10 || minor != 3) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  cudaStream_t st = as_stream(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const int64_t R = T * k;
  float* h = reinterpret_cast<float*>(ws);
  float* o = reinterpret_cast<float*>(ws + align256(R * F * 4));
  unsigned int* count = reinterpret_cast<unsigned int*>(ws + align256(R * F * 4) + align256(R * D * 4));
  Params p{};
  p.ids = topk_ids;
  p.topk_w = topk_w;
  p.y = y;
  p.count = count;
  p.ncount = static_cast<int>(counters(D));
  p.T = static_cast<int>(T);
  p.k = k;
  p.E = E;
  p.g0 = group_offset;
  p.El = E_local;
  const int64_t active = R < E_local ? R : E_local;
  p.act = x;
  p.scale = static_cast<const float*>(s_in);
  p.out = h;
  p.K = static_cast<int>(D);
  p.N = static_cast<int>(F);
  p.mode = kin;
  const int rb1 = T <= 8 && active * ((F + 63) / 64) < 8ll * sms ? 32 : 128;
  moe_status s = launch_type<1>(type, w_in, p, rb1, sms, st);
  if (s != MOE_OK) return s;
  p.act = h;
  p.scale = static_cast<const float*>(s_out);
  p.out = o;
  p.K = static_cast<int>(F);
  p.N = static_cast<int>(D);
  p.mode = kout;
  const int rb2 = T <= 8 && active * ((D + 127) / 128) < 8ll * sms ? 32 : 128;
  return launch_type<2>(type, w_out, p, rb2, sms, st);
}
