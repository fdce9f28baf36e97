// The expert FFN of a decoding step (sm_103a): moe_ffn_decode
//   y[t] = bf16( sum_j w[t, j] Wo[e] (silu(W0[e] x[t]) * (W1[e] x[t])) ),  e = ids[t, j]
// for a few tokens, on bf16 activations and quantised expert weights (e4m3 or
// int8 with per-channel, blockwise or static scales, MXFP8, MXFP4).
//
// With a few tokens the weights of the chosen experts are all that matters:
// 3 D F bytes an expert (half for MXFP4), read once, against a few flops a
// byte.  So nothing is quantised here, the weights stream through shared
// memory at the rate of HBM, and everything else has to fit beside that
// stream.  One cooperative kernel, a persistent CTA per SM, in two phases:
//   phase 1  h = silu(W0 x) * (W1 x) of every (token, expert) pair, fp32, into
//            the workspace;
//   phase 2  o = Wo h of every pair, fp32, into the workspace; the warp that
//            finishes the last unit of 16 output columns sums their pairs with
//            the choices' weights, in ascending j, and writes y.
// Between them every CTA's h has to be there.  Weights do not wait for that: a
// ring of wo's goes out while the last of phase 1 is at work.
//
// Every CTA first sorts the pairs by expert for itself (at most 1024): a
// chunk is up to `cap` pairs of one expert.  A unit of work is one chunk, one
// block of 128 weight rows (phase 1: 64 channels of wi_0 and the same of wi_1)
// and one segment of K (more than one segment where there are too few blocks
// to fill the SMs evenly; the segments' sums meet in fp32 in ascending order,
// phase 1's where phase 2 reads them).  Units run expert-major: the CTAs then
// read a few experts at a time, long runs of memory each.  (64 tokens over 256
// experts: with the blocks of all experts side by side the bare stream ran at
// 1.1 TB/s, expert-major at 3.9.)
//
// Roles:
//   warp 0       the weights, a TMA box of 128 rows x 128 bytes each (two a stage),
//                and by cp.async the activations' rows and the scale words.  TMA
//                for the boxes alone: single 16 KB boxes stream at 7.2 TB/s here,
//                with four small bulk copies beside each at 5.1.
//   CONV warps   turn a stage's activations into f16 in place, each (row, span of
//                a box's K) scaled by the power of two that puts its largest value
//                in [2^14, 2^15).  f16 then holds a bf16 value exactly down to
//                2^-28 of the span's largest and to 2^-39 of that below, and h to
//                2^-11 relative down to there.  (The result's bf16 has 2^-8: with
//                h in fp32 it would be 1.659e-3 from exact, with f16 it is 1.671e-3,
//                relative Frobenius, one result in ten off by one bf16 step.)
//                A sum over MX blocks grows to 2^23 times the largest weight's
//                magnitude before the span scale comes off: weights to 2^104.
//   8 warps a group contract, 16 weight rows each: ldmatrix brings 16 rows x 32
//                bytes, one conversion makes two f16 weights (exact for e4m3, int8
//                and e2m1, NaN codes included), mma.m16n8k16 multiplies them with
//                eight tokens.  At a few tokens the tensor core is far from its
//                limit (16 % busy), so the warp-wide MMA serves: its operands come
//                from registers, where the weights are converted anyway, and its M
//                is only 16.  In phase 1 rows 0..7 of a fragment are wi_0 channels
//                and rows 8..15 the same wi_1 channels, so a thread holds both
//                factors of its h.  Span sums are scaled (weight block scale,
//                activation span scale) into fp32 accumulators.
//
// Measured with warm code and cold weights, TB/s of weights and scales (of the
// measured 6.79): 64 tokens, 218 experts of 7168 x 2048, blockwise e4m3 1.57 ms, 6.3;
// 7 tokens, 8 experts of 4096 x 14336, int8 0.203 ms, 6.1; one token, 2 of these,
// e4m3 61 us, 6.0 (about 8 us of it start, phase change and end); 16 tokens, 103
// experts of 7168 x 2048, MXFP4 0.65 ms, 3.7 (bound by issue: 3200 warp instructions
// a 16 KB box, ALU pipe 47 % and issue slots 52 % busy); one token of 8 experts of
// 2048 x 768 17 us, where start, phase change and end are most of it.
//
// Every wait is bounded; on expiry the kernel raises MOE_DEVERR_TIMEOUT, lets
// its copies land, marks the workspace, whose counters it leaves as they are, and
// returns.
#include <cudaTypedefs.h>

#include <mutex>

#include "mx4.cuh"

namespace moe {
namespace {

__device__ unsigned int g_err;

constexpr int kMmaWarps = 8;  // contracting warps of a group
constexpr int kMaxNT = 2;     // two groups: eight tokens times this a chunk (registers)
// e2m1's stage holds twice the values of the other types' bytes and takes longer
// to convert and to multiply than to arrive: two groups of contracting warps, on
// alternate stages, and five warps that convert (16 tokens over 256 experts: 703 us
// with one group and three warps, 689 with two groups, 656 with five warps, too).
__host__ __device__ constexpr int groups_of(int wt) { return wt == 3 ? 2 : 1; }
__host__ __device__ constexpr int conv_of(int wt) { return wt == 3 ? 5 : 3; }
__host__ __device__ constexpr int threads_of(int wt) { return 32 * (1 + conv_of(wt) + kMmaWarps * groups_of(wt)); }
constexpr int kRows = 128;              // weight rows of a unit
constexpr int kBoxW = kRows * 128;      // weight bytes of a TMA box
constexpr int kMaxStages = 10;
constexpr int kMaxSegs = 8;
constexpr int kMaxPairs = 1024;
constexpr int kMaxTokens = 64;
constexpr int kMaxExperts = 1024;
constexpr int kMaxDim = 32768;  // D and F
constexpr int kSmemLimit = 232448;
// Set in the workspace's first counter by a call that timed out: the counters
// then hold what it left, and the calls after it stop instead of counting on.
constexpr unsigned int kBroken = 0x80000000u;

enum { kE4M3 = 0, kInt8 = 1, kMx8 = 2, kMx4 = 3 };
enum { kScaleChannel = 0, kScaleBlock = 1, kScaleTensor = 2, kScaleMx = 3 };

struct PhaseParams {
  const void* act;     // phase 1: x bf16 [T, K]; phase 2: h fp32 [slots, K], or partial a [segs][slots, 2K]
  const float* scale;  // fp32 scales, or the MX scale words
  float* out;          // phase 1: h [slots, N], or partial a [segs][slots, 2N]; phase 2: o [segs][slots, N]
  int K, N;            // N: channels (phase 1: F, phase 2: D)
  int mode;
  int nblock, nst;     // row blocks, K stages
};

struct Params {
  PhaseParams f[2];
  const int32_t* ids;
  const float* topk_w;
  uint16_t* y;
  unsigned int* sync;   // [0] warps done with phase 1 (or kBroken), [1] CTAs that have seen all of them; zero between calls
  unsigned int* count;  // finished units of every 16 output columns; zero between calls
  int T, k, E, g0, El;
  int cap, stages;  // pairs a chunk; ring stages
  int smax;         // segments of K at most
  uint64_t stall_ns;  // test hook (moe_test_stall_consumers): 0, or the wait limit in ns
};

struct Ctl {
  uint64_t full[kMaxStages], xraw[kMaxStages], xfull[kMaxStages], empty[kMaxStages];
  uint64_t rfull[kMmaWarps], rempty[kMmaWarps];  // a warp's sums have been left for its partner, and taken
  uint64_t never;  // test hook: a barrier that nothing arrives on
  int abort_flag, no_abort, err, nchunk, segs1, segs2;
  uint16_t pos[kMaxPairs];     // slot of pair i (pairs sorted by expert), 0xFFFF: not local
  uint16_t order[kMaxPairs];   // pair of slot s
  uint16_t cexp[kMaxPairs], cstart[kMaxPairs], cnum[kMaxPairs];
  uint16_t cfirst[kMaxPairs], ccount[kMaxPairs];  // the first chunk of the chunk's expert, and how many it has
  uint16_t num[kMaxExperts];
};

template <int WT, int PHASE>
struct Cfg {
  static constexpr bool MX = WT == kMx8 || WT == kMx4;
  // Boxes (128 bytes of each weight row) a stage: two, so that a warp has two
  // boxes' loads in flight and half the hand-offs; one for e2m1, whose box
  // holds twice the values and whose activations take the space
  static constexpr int BOXES = WT == kMx4 ? 1 : 2;
  static constexpr int BOX_K = WT == kMx4 ? 256 : 128;  // values of K in a box: a span of an activation row
  static constexpr int KE = BOXES * BOX_K;              // and in a stage
  static constexpr int STAGE_W = BOXES * kBoxW;
  static constexpr int WORDS = BOX_K / 128;             // scale words of a row and box
  // a row's scale word as it is used: one float, or (MX) its four blocks' powers
  // of two as bf16, which holds them all
  static constexpr int SCALE_ROW = MX ? 8 : 4;
  static constexpr int SCALE_BYTES = BOXES * WORDS * kRows * SCALE_ROW;
  static constexpr int PER = BOX_K / 32;  // values of a span a lane converts
  // bytes of an activation row as it arrives (bf16 x, fp32 h; the f16 form takes
  // the front of each span's place), padded so that eight rows' fragments lie
  // in different banks
  static constexpr int SPAN_BYTES = BOX_K * (PHASE == 1 ? 2 : 4);
  static constexpr int ROW_BYTES = BOXES * SPAN_BYTES;
  static constexpr int PITCH = ROW_BYTES + (WT == kMx4 ? 64 : 32);
};

// How many segments of K: the fewest stages on the busiest CTA, a unit's
// start and end counted as two stages.  One warp, a lane a choice (at most
// 2^19 units x 8 segments x 130 stages: 32 bits hold the cost).
__device__ __forceinline__ int pick_segs(int units, int nst, int grid, int smax) {
  const int s = (threadIdx.x & 31) + 1;
  const unsigned int cost = s <= smax && s <= nst ? static_cast<unsigned>((units * s + grid - 1) / grid * ((nst + s - 1) / s + 2))
                                                  : 0xFFFFFFFFu;
  return __ffs(__ballot_sync(0xffffffffu, cost == __reduce_min_sync(0xffffffffu, cost)));
}

constexpr size_t kCtlBytes = (sizeof(Ctl) + 127) / 128 * 128;

__device__ __forceinline__ unsigned int load_acquire(const unsigned int* p) {
  unsigned int v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The first product of a sum: c = a b.
__device__ __forceinline__ void mma_f16_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
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

// 16-byte asynchronous copy; with src_bytes 0 the destination is zero-filled.
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}
// One of the barrier's arrivals, made when this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(bar) : "memory");
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
// Every CTA sorts for itself, to the same tables.

__device__ __forceinline__ int local_expert(const Params& p, int i) {
  const int id = __ldg(p.ids + i);
  if (id < 0 || id >= p.E) {
    raise_error(&g_err, MOE_DEVERR_BAD_EXPERT_ID);
    return 0xFFFF;
  }
  const int e = id - p.g0;
  return e >= 0 && e < p.El ? e : 0xFFFF;
}

// Up to 32 pairs, one a lane: a pair's slot is the number of pairs before it
// in (expert, pair) order, its chunk the number of chunks of smaller experts
// and of earlier pairs of its own.
__device__ __forceinline__ void build_chunks_warp(const Params& p, Ctl* c) {
  const int lane = threadIdx.x & 31;
  const int R = p.T * p.k;
  const int e = lane < R ? local_expert(p, lane) : 0xFFFF;
  const uint32_t same = __match_any_sync(0xffffffffu, e);
  const bool mine = e != 0xFFFF;
  const int rank = __popc(same & ((1u << lane) - 1u)), n = __popc(same);
  const int nc = mine && rank == 0 ? (n + p.cap - 1) / p.cap : 0;  // a group's first pair counts its chunks
  int start = 0, chunk = 0, total = 0;
#pragma unroll 8
  for (int j = 0; j < 32; ++j) {
    const int ej = __shfl_sync(0xffffffffu, e, j), cj = __shfl_sync(0xffffffffu, nc, j);
    start += ej < e;
    chunk += ej < e ? cj : 0;
    total += cj;
  }
  if (mine) {
    c->pos[lane] = static_cast<uint16_t>(start + rank);
    c->order[start + rank] = static_cast<uint16_t>(lane);
    if (rank % p.cap == 0) {
      const int q = chunk + rank / p.cap;
      c->cexp[q] = static_cast<uint16_t>(e);
      c->cstart[q] = static_cast<uint16_t>(start + rank);
      c->cnum[q] = static_cast<uint16_t>(min(p.cap, n - rank));
      c->cfirst[q] = static_cast<uint16_t>(chunk);
      c->ccount[q] = static_cast<uint16_t>((n + p.cap - 1) / p.cap);
    }
  } else if (lane < R) {
    c->pos[lane] = 0xFFFF;
  }
  if (lane == 0) c->nchunk = total;
}

// More than 32 pairs, by the whole CTA.  `bits` (shared memory that the ring
// does not use yet) holds a bit a pair for every local expert: a pair's rank is
// the number of its expert's bits below its own, so that the order does not
// depend on when the atomics come.  Behind it, a word an expert: its first
// chunk and slot.
__device__ void build_chunks(const Params& p, Ctl* c, uint32_t* bits) {
  const int tid = threadIdx.x, lane = tid & 31;
  const int R = p.T * p.k, W = (R + 31) / 32;
  uint32_t* first = bits + p.El * W;
  for (int i = tid; i < p.El * W; i += blockDim.x) bits[i] = 0;
  __syncthreads();
  for (int i = tid; i < R; i += blockDim.x) {
    const int e = local_expert(p, i);
    c->order[i] = static_cast<uint16_t>(e);
    if (e != 0xFFFF) atomicOr(bits + e * W + i / 32, 1u << (i & 31));
  }
  __syncthreads();
  for (int e = tid; e < p.El; e += blockDim.x) {
    int n = 0;
    for (int w = 0; w < W; ++w) n += __popc(bits[e * W + w]);
    c->num[e] = static_cast<uint16_t>(n);
  }
  __syncthreads();
  if (tid < 32) {  // a lane: a run of consecutive experts
    const int per = (p.El + 31) / 32, e0 = lane * per, e1 = min(e0 + per, p.El);
    uint32_t sum = 0;  // chunks above 16 bits of pairs: at most 1024 of either
    for (int e = e0; e < e1; ++e) sum += c->num[e] | ((c->num[e] + p.cap - 1) / p.cap) << 16;
    uint32_t at = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t a = __shfl_up_sync(0xffffffffu, at, o);
      if (lane >= o) at += a;
    }
    if (lane == 31) c->nchunk = at >> 16;
    at -= sum;
    for (int e = e0; e < e1; ++e) {
      first[e] = at;
      at += c->num[e] | ((c->num[e] + p.cap - 1) / p.cap) << 16;
    }
  }
  __syncthreads();
  for (int e = tid; e < p.El; e += blockDim.x) {
    const int n = c->num[e], nc = (n + p.cap - 1) / p.cap, off = first[e] & 0xFFFF, c0 = first[e] >> 16;
    for (int j = 0; j < nc; ++j) {
      c->cexp[c0 + j] = static_cast<uint16_t>(e);
      c->cstart[c0 + j] = static_cast<uint16_t>(off + j * p.cap);
      c->cnum[c0 + j] = static_cast<uint16_t>(min(p.cap, n - j * p.cap));
      c->cfirst[c0 + j] = static_cast<uint16_t>(c0);
      c->ccount[c0 + j] = static_cast<uint16_t>(nc);
    }
  }
  for (int i = tid; i < R; i += blockDim.x) {
    const int e = c->order[i];
    int at = 0xFFFF;
    if (e != 0xFFFF) {
      at = (first[e] & 0xFFFF) + __popc(bits[e * W + i / 32] & ((1u << (i & 31)) - 1u));
      for (int w = 0; w < i / 32; ++w) at += __popc(bits[e * W + w]);
    }
    c->pos[i] = static_cast<uint16_t>(at);
  }
  __syncthreads();
  for (int i = tid; i < R; i += blockDim.x)  // (the experts in `order` are no longer needed)
    if (c->pos[i] != 0xFFFF) c->order[c->pos[i]] = static_cast<uint16_t>(i);
}

struct BoxAt {
  uint32_t wt, xb, sA, sB, xs;
};

template <int WT, int PHASE, int NT>
struct Box {
  using C = Cfg<WT, PHASE>;
  static constexpr int DEPTH = WT == kMx4 ? (NT == 1 ? 4 : 1) : (NT <= 2 ? 4 : 2);
  static constexpr int BW = WT == kMx4 ? 4 : 2;  // words of a chunk's activation fragment
  uint32_t r[4][4];
  uint32_t b[DEPTH][2][NT][BW];
  float fA[4], fB[4];
  uint2 xv[NT];

  __device__ __forceinline__ void load_b(const BoxAt& at, int c) {
#pragma unroll
    for (int cc = 0; cc < 2; ++cc)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (WT == kMx4) {
          const uint4 v = lds128(at.xb + n * 8 * C::PITCH + (2 * c + cc) * 64);
          b[c % DEPTH][cc][n][0] = v.x;
          b[c % DEPTH][cc][n][1] = v.y;
          b[c % DEPTH][cc][n][BW - 2] = v.z;
          b[c % DEPTH][cc][n][BW - 1] = v.w;
        } else {
          const uint2 v = lds64(at.xb + n * 8 * C::PITCH + (2 * c + cc) * 32);
          b[c % DEPTH][cc][n][0] = v.x;
          b[c % DEPTH][cc][n][1] = v.y;
        }
      }
  }
  __device__ __forceinline__ void load_f(const BoxAt& at, int v) {
    const uint2 a = lds64(at.sA + v * kRows * C::SCALE_ROW), d = lds64(at.sB + v * kRows * C::SCALE_ROW);
    fA[0] = bf16lo(a.x);
    fA[1] = bf16hi(a.x);
    fA[2] = bf16lo(a.y);
    fA[3] = bf16hi(a.y);
    fB[0] = bf16lo(d.x);
    fB[1] = bf16hi(d.x);
    fB[2] = bf16lo(d.y);
    fB[3] = bf16hi(d.y);
  }
  __device__ __forceinline__ void load(const BoxAt& at, uint32_t swz, bool block_scale) {
    const int hi = (threadIdx.x >> 4) & 1;  // lanes 16..31 address the second chunk of a pair
#pragma unroll
    for (int c = 0; c < 4; ++c) ldmatrix_x4(at.wt + (((2 * c + hi) * 16) ^ swz), r[c]);
#pragma unroll
    for (int c = 0; c < DEPTH; ++c) load_b(at, c);
#pragma unroll
    for (int i = 0; i < 4; ++i) fA[i] = fB[i] = 1.0f;
    if (C::MX) {
      load_f(at, 0);
    } else if (block_scale) {
      fA[0] = __uint_as_float(lds32(at.sA));
      fB[0] = __uint_as_float(lds32(at.sB));
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) xv[n] = lds64(at.xs + n * 32);
  }
  __device__ __forceinline__ void contract(float (&acc)[NT][4], const BoxAt& at) {
    // Without block scales, two chains of sums, s0 and blk[0].  MX: s0 sums the
    // scaled 32-wide blocks; a block is scaled into it one block late, while the
    // next one's products run.
    float s0[NT][4], blk[2][NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) s0[n][i] = 0.0f;
    auto fold = [&](int k, float fa, float fb) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        s0[n][0] = __fmaf_rn(blk[k][n][0], fa, s0[n][0]);
        s0[n][1] = __fmaf_rn(blk[k][n][1], fa, s0[n][1]);
        s0[n][2] = __fmaf_rn(blk[k][n][2], fb, s0[n][2]);
        s0[n][3] = __fmaf_rn(blk[k][n][3], fb, s0[n][3]);
      }
    };
    float pa = 0.0f, pb = 0.0f;  // the scales of the block before
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (WT == kMx4 && c == 2) load_f(at, 1);
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        if (WT == kMx4) {
          uint32_t va[4], vb[4];
          weights8(r[c][2 * cc], va);
          weights8(r[c][2 * cc + 1], vb);
          const uint32_t a0[4] = {va[0], vb[0], va[1], vb[1]}, a1[4] = {va[2], vb[2], va[3], vb[3]};
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_f16_first(blk[cc][n], a0, b[c % DEPTH][cc][n][0], b[c % DEPTH][cc][n][1]);
            mma_f16(blk[cc][n], a1, b[c % DEPTH][cc][n][BW - 2], b[c % DEPTH][cc][n][BW - 1]);
          }
          if (c > 0 || cc > 0) fold(cc ^ 1, pa, pb);
          pa = fA[(2 * c + cc) & 3];
          pb = fB[(2 * c + cc) & 3];
        } else {
          uint32_t a[4];
          weights4<WT>(r[c][2 * cc], a[0], a[2]);
          weights4<WT>(r[c][2 * cc + 1], a[1], a[3]);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint32_t b0 = b[c % DEPTH][cc][n][0], b1 = b[c % DEPTH][cc][n][1];
            if (C::MX) {
              if (cc == 0)
                mma_f16_first(blk[c & 1][n], a, b0, b1);
              else
                mma_f16(blk[c & 1][n], a, b0, b1);
            } else if (cc == 0) {
              if (c == 0)
                mma_f16_first(s0[n], a, b0, b1);
              else
                mma_f16(s0[n], a, b0, b1);
            } else {
              if (c == 0)
                mma_f16_first(blk[0][n], a, b0, b1);
              else
                mma_f16(blk[0][n], a, b0, b1);
            }
          }
          if (C::MX && cc == 1) {
            if (c > 0) fold((c & 1) ^ 1, pa, pb);
            pa = fA[c];
            pb = fB[c];
          }
        }
      }
      if (c + DEPTH < 4) load_b(at, c + DEPTH);
    }
    if (C::MX) fold(1, pa, pb);  // the last block
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float x0 = __uint_as_float(xv[n].x), x1 = __uint_as_float(xv[n].y);
      if (C::MX) {
        acc[n][0] = __fmaf_rn(s0[n][0], x0, acc[n][0]);
        acc[n][1] = __fmaf_rn(s0[n][1], x1, acc[n][1]);
        acc[n][2] = __fmaf_rn(s0[n][2], x0, acc[n][2]);
        acc[n][3] = __fmaf_rn(s0[n][3], x1, acc[n][3]);
      } else {
        acc[n][0] = __fmaf_rn(s0[n][0] + blk[0][n][0], x0 * fA[0], acc[n][0]);
        acc[n][1] = __fmaf_rn(s0[n][1] + blk[0][n][1], x1 * fA[0], acc[n][1]);
        acc[n][2] = __fmaf_rn(s0[n][2] + blk[0][n][2], x0 * fB[0], acc[n][2]);
        acc[n][3] = __fmaf_rn(s0[n][3] + blk[0][n][3], x1 * fB[0], acc[n][3]);
      }
    }
  }
};

// One span of an activation row, PER values a lane: scaled to f16 in shared
// memory at `at`, the scale to put back at `sc`.
template <int PER>
__device__ __forceinline__ void store_span(float (&v)[PER], uint32_t at, uint32_t sc, int lane) {
  // largest finite magnitude of the span; infinities and NaN pass through
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const uint32_t b = __float_as_uint(v[j]) & 0x7FFFFFFFu;
    m = max(m, b < 0x7F800000u ? b : 0u);
  }
  m = __reduce_max_sync(0xffffffffu, m);
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
  if (lane == 0) sts32f(sc, __uint_as_float(static_cast<uint32_t>(127 - 14 + e) << 23));
}

// The weights pass through L2 once: marked to leave it first, they do not push
// out what is needed again soon (activations, h, o, the kernels' own code).
__device__ __forceinline__ uint64_t evict_first_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, int x, int y, int z, uint32_t bar,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, "
      "%3, %4}], [%5], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(policy)
      : "memory");
}

// Where a CTA is: unit u = (chunk, row block, segment), stages [kst, end) of
// it left.  Units are numbered by expert, row block, segment and last by the
// expert's chunks, so that these read the same weights together.
struct Step {
  int u, ch, blk, seg, kst, end;
};
struct Walk {
  int nblock, segs, nst, total;
  const Ctl* ctl;
  __device__ __forceinline__ void open(Step& q) const {
    const int per = nblock * segs;
    const int any = q.u / per;  // a chunk of the expert
    const int first = ctl->cfirst[any], count = ctl->ccount[any];
    int r = q.u - first * per;
    if (count > 1) {
      q.ch = first + r % count;
      r /= count;
    } else {
      q.ch = first;
    }
    q.blk = r / segs;
    q.seg = r - q.blk * segs;
    q.kst = q.seg * nst / segs;
    q.end = (q.seg + 1) * nst / segs;
  }
  __device__ __forceinline__ Step begin() const {
    Step q{static_cast<int>(blockIdx.x), 0, 0, 0, 0, 0};
    if (q.u < total) open(q);
    return q;
  }
  __device__ __forceinline__ bool done(const Step& q) const { return q.u >= total; }
  __device__ __forceinline__ void next(Step& q) const {
    if (++q.kst == q.end) {
      q.u += gridDim.x;
      if (q.u < total) open(q);
    }
  }
  __device__ __forceinline__ int skip(Step& q, int n) const {  // n stages on; returns how many lie past the end
    while (n > 0 && q.u < total) {
      if (q.kst + n < q.end) {
        q.kst += n;
        return 0;
      }
      n -= q.end - q.kst;
      q.u += gridDim.x;
      if (q.u < total) open(q);
    }
    return n;
  }
};

template <int WT>
__global__ void __launch_bounds__(threads_of(WT), 1)
    decode_kernel(const __grid_constant__ CUtensorMap tm1, const __grid_constant__ CUtensorMap tm2,
                  const __grid_constant__ Params p) {
  using G = Cfg<WT, 2>;  // the ring's geometry: phase 2's, whose activations are the wider
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* bp = smem_raw + (base - raw);
  // stages of weights | f16 activations | weight scales | activation span scales | control
  const uint32_t S = p.stages;
  const int cap = p.cap;
  const uint32_t x_ring = base + S * G::STAGE_W;
  const uint32_t x_bytes = cap * G::PITCH;
  const uint32_t s_ring = x_ring + S * x_bytes;
  const uint32_t v_ring = s_ring + S * G::SCALE_BYTES;
  const uint32_t v_bytes = G::BOXES * cap * 4;
  Ctl* ctl = reinterpret_cast<Ctl*>(bp + (v_ring + S * v_bytes - base));
  float* red = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(ctl) + kCtlBytes);  // two groups: sums on their way
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int R = p.T * p.k;

  if (threadIdx.x == 0) {
    for (int w = 0; w < kMmaWarps; ++w) {
      mbar_init(smem_u32(&ctl->rfull[w]), 32);
      mbar_init(smem_u32(&ctl->rempty[w]), 32);
    }
    mbar_init(smem_u32(&ctl->never), 1);
    for (uint32_t s = 0; s < S; ++s) {
      mbar_init(smem_u32(&ctl->full[s]), 1);
      mbar_init(smem_u32(&ctl->xraw[s]), 32);
      mbar_init(smem_u32(&ctl->xfull[s]), 1);
      mbar_init(smem_u32(&ctl->empty[s]), kMmaWarps * groups_of(WT));
    }
    ctl->abort_flag = 0;
    ctl->no_abort = 0;
    ctl->err = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm1);
    tma_prefetch_desc(&tm2);
  }
  if (R <= 32) {
    if (warp == 1) build_chunks_warp(p, ctl);
  } else {
    build_chunks(p, ctl, reinterpret_cast<uint32_t*>(bp));
    // the ring is written by asynchronous copies next
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    __syncwarp();
    const int segs1 = pick_segs(ctl->nchunk * p.f[0].nblock, p.f[0].nst, gridDim.x, p.smax);
    const int segs2 = pick_segs(ctl->nchunk * p.f[1].nblock, p.f[1].nst, gridDim.x, p.smax);
    if (lane == 0) {
      ctl->segs1 = segs1;
      ctl->segs2 = segs2;
    }
  }
  __syncthreads();

  const int nchunk = ctl->nchunk;
  const int segs1 = ctl->segs1;
  const int slots = nchunk > 0 ? ctl->cstart[nchunk - 1] + ctl->cnum[nchunk - 1] : 0;  // local pairs
  volatile int* abort_flag = &ctl->abort_flag;
  bool timed_out = false;

  if (nchunk == 0) {  // no local expert was chosen at all
    const int64_t n = static_cast<int64_t>(p.T) * p.f[1].N;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * blockDim.x)
      p.y[i] = 0;
    return;
  }

  auto walk_of = [&](int phase) {
    Walk w;
    w.nblock = p.f[phase - 1].nblock;
    w.nst = p.f[phase - 1].nst;
    w.segs = phase == 1 ? segs1 : ctl->segs2;
    w.total = nchunk * w.nblock * w.segs;
    w.ctl = ctl;
    return w;
  };
  auto has_words = [](const PhaseParams& f) {  // one scale word a row and 128 values of K
    return f.mode == kScaleBlock || f.mode == kScaleMx;
  };
  const bool partial = segs1 > 1;  // phase 1 leaves sums of K segments
  // where the raw scale words v of stage s arrive: the end of their place
  auto raw_words = [&](uint32_t s, int v) {
    return s_ring + s * G::SCALE_BYTES + (v + 1) * kRows * G::SCALE_ROW - kRows * 4;
  };

  if (warp == 0) {
    // ------------------------- weights by TMA; activations and scales by cp.async
    const uint64_t policy = evict_first_policy();
    uint32_t s = 0, ph = 0, issued = 0;  // the ring goes on from phase 1 to phase 2
    auto advance = [&] {
      if (++s == S) {
        s = 0;
        ph ^= 1;
      }
    };
    auto wait_empty = [&] {
      if (!mbar_wait_bounded_warp(smem_u32(&ctl->empty[s]), ph ^ 1, abort_flag, kWaitLimitNs)) timed_out = true;
      return !timed_out;
    };
    // All of phase 1, from every CTA: its warps count themselves.  The last CTA to
    // have seen it sets the counters back for the next call.
    auto wait_phase1 = [&] {
      int ok = 1;
      if (lane == 0) {
        const unsigned int all = gridDim.x * kMmaWarps;
        const uint64_t t0 = globaltimer_ns();
        for (unsigned int v; (v = load_acquire(p.sync)) != all;) {
          if ((v & kBroken) || *abort_flag || globaltimer_ns() - t0 > kWaitLimitNs) {
            ok = 0;
            break;
          }
        }
        if (ok && atomicAdd(p.sync + 1, 1u) == gridDim.x - 1) {
          atomicSub(p.sync, all);  // (kBroken stays, if another CTA has set it since)
          p.sync[1] = 0;
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      __syncwarp();  // what lane 0 has seen holds for every lane's copies
      return ok != 0;
    };
    auto run = [&](auto phase_tag) {
      constexpr int PHASE = decltype(phase_tag)::value;
      using C = Cfg<WT, PHASE>;
      constexpr int kPer = PHASE == 1 ? kRows / 2 : kRows;  // channels of a unit
      const PhaseParams& f = p.f[PHASE - 1];
      const Walk walk = walk_of(PHASE);
      const int nbox = (f.K + C::BOX_K - 1) / C::BOX_K;  // boxes along K
      const bool words = has_words(f), joined = PHASE == 2 && partial;
      const int nkb = f.K / 128;  // (used with scale words: K % 128 == 0)
      const int64_t scale_rows = static_cast<int64_t>(PHASE == 1 ? 2 * f.N : f.N);
      auto load_weights = [&](uint32_t s, const Step& q) {
        if (lane == 0) {
          const uint32_t fb = smem_u32(&ctl->full[s]);
          const int e = ctl->cexp[q.ch];
          const int boxes = min(C::BOXES, nbox - q.kst * C::BOXES);
          mbar_arrive_expect_tx(fb, boxes * kBoxW);
          // rows past the tensor's channels or K arrive as zeros
          for (int v = 0; v < boxes; ++v)
            tma_load_3d(base + s * C::STAGE_W + v * kBoxW, PHASE == 1 ? &tm1 : &tm2, (q.kst * C::BOXES + v) * 128, q.blk * kPer,
                        PHASE == 1 ? 2 * e : e, fb, policy);
        }
      };
      // This lane's sources at a unit's first stage, kept over the unit: its part
      // of the scale words, and of the first kKept x 32 chunks of activations.
      constexpr int kChunks = C::ROW_BYTES / 16, kVals = PHASE == 1 ? 8 : 4;  // 16-byte chunks of a row, values in one
      constexpr int kKept = 4;
      constexpr int kWords = C::BOXES * C::WORDS;
      int unit = -1, n = 0, st = 0;
      const float* sc = f.scale;
      const uint8_t* xsrc[kKept];
      const int64_t kb_pitch = f.mode == kScaleMx ? p.El * scale_rows : scale_rows;  // from one 128-wide block to the next
      auto row_src = [&](int i) {  // chunk i of the unit's activations at K = 0
        const int r = i / kChunks, c = i % kChunks;
        const int64_t row = PHASE == 1 ? ctl->order[st + r] / p.k : st + r;
        return static_cast<const uint8_t*>(f.act) + (row * f.K + c * kVals) * (PHASE == 1 ? 2 : 4);
      };
      auto load_rest = [&](uint32_t s, const Step& q) {
        if (q.u != unit) {
          unit = q.u;
          n = ctl->cnum[q.ch];
          st = ctl->cstart[q.ch];
          const int e = ctl->cexp[q.ch];
          if (words) {
            const int64_t n0 = q.blk * kPer + (PHASE == 1 ? (lane & 15) * 4 + (lane >> 4) * f.N : lane * 4);
            sc = f.scale + (f.mode == kScaleMx ? e * scale_rows : static_cast<int64_t>(e) * nkb * scale_rows) + n0;
          }
#pragma unroll
          for (int j = 0; j < kKept; ++j)
            xsrc[j] = lane + 32 * j < n * kChunks && !joined ? row_src(lane + 32 * j) : static_cast<const uint8_t*>(f.act);
        }
        if (words) {
#pragma unroll
          for (int v = 0; v < kWords; ++v) {
            const int64_t kb = q.kst * kWords + v;
            const bool ok = kb < nkb;
            cp_async_16(raw_words(s, v) + lane * 16, ok ? sc + kb * kb_pitch : f.scale, ok ? 16u : 0u);
          }
        }
        if (!joined) {
          const int64_t k0 = static_cast<int64_t>(q.kst) * C::ROW_BYTES;
          const uint32_t dst = x_ring + s * x_bytes;
          // K is a multiple of 16: a chunk is all in or out
#pragma unroll
          for (int j = 0; j < kKept; ++j) {
            const int i = lane + 32 * j;
            if (i < n * kChunks) {
              const int r = i / kChunks, c = i % kChunks;
              const bool ok = q.kst * C::KE + c * kVals < f.K;
              cp_async_16(dst + r * C::PITCH + c * 16, ok ? xsrc[j] + k0 : xsrc[j], ok ? 16u : 0u);
            }
          }
          for (int i = lane + 32 * kKept; i < n * kChunks; i += 32) {
            const int r = i / kChunks, c = i % kChunks;
            const bool ok = q.kst * C::KE + c * kVals < f.K;
            cp_async_16(dst + r * C::PITCH + c * 16, ok ? row_src(i) + k0 : static_cast<const uint8_t*>(f.act), ok ? 16u : 0u);
          }
        }
        cp_async_arrive(smem_u32(&ctl->xraw[s]));
      };

      Step q = walk.begin();
      if (PHASE == 2) {
        // weights do not depend on phase 1: a ring of them goes out as its stages
        // come back, then every CTA's h has to be there
        const uint32_t s0 = s, ph0 = ph;
        uint32_t ahead = 0;
        for (Step w = q; ahead < S && !walk.done(w) && wait_empty(); walk.next(w), ++ahead) {
          load_weights(s, w);
          ++issued;
          advance();
        }
        if (!timed_out) timed_out = !wait_phase1();
        if (timed_out) return;
        s = s0;
        ph = ph0;
        for (; ahead > 0; --ahead, walk.next(q)) {
          load_rest(s, q);
          advance();
        }
      }
      for (; !walk.done(q) && wait_empty(); walk.next(q)) {
        load_weights(s, q);
        ++issued;
        load_rest(s, q);
        advance();
      }
    };
    run(std::integral_constant<int, 1>{});
    if (!timed_out) run(std::integral_constant<int, 2>{});
    if (timed_out) {
      *abort_flag = 1;
      ctl->err = 2;
    }
    // Copies in flight land before the CTA exits, whichever warp's wait ran out
    // (this one may have issued them all and be done).
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (lane == 0)
      for (uint32_t j = issued > S ? issued - S : 0; j < issued; ++j)
        mbar_wait_bounded(smem_u32(&ctl->full[j % S]), (j / S) & 1, &ctl->no_abort, kWaitLimitNs);
    __syncwarp();
  } else if (warp <= conv_of(WT)) {
    // ---------------------- activations to f16 and MX scale codes to bf16, in place
    uint32_t step = warp - 1;  // this warp's next stage of the CTA's,
    int left = warp - 1;       // and how many stages of the phase lie before it
    auto run = [&](auto phase_tag) {
      constexpr int PHASE = decltype(phase_tag)::value;
      using C = Cfg<WT, PHASE>;
      constexpr int PER = C::PER;
      const PhaseParams& f = p.f[PHASE - 1];
      const Walk walk = walk_of(PHASE);
      // h of phase 1's segments: their sums in ascending order, then SwiGLU
      auto join = [&](int slot, int col, bool ok, float (&v)[PER]) {
        float a0[PER], a1[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j) a0[j] = a1[j] = 0.0f;
        if (ok)
          for (int g = 0; g < segs1; ++g) {
            const float* src = static_cast<const float*>(f.act) + (static_cast<int64_t>(g) * slots + slot) * 2 * f.K + col;
#pragma unroll
            for (int j = 0; j < PER; j += 4) {
              const float4 u = __ldcg(reinterpret_cast<const float4*>(src + j));
              const float4 w = __ldcg(reinterpret_cast<const float4*>(src + f.K + j));
              a0[j] += u.x;
              a0[j + 1] += u.y;
              a0[j + 2] += u.z;
              a0[j + 3] += u.w;
              a1[j] += w.x;
              a1[j + 1] += w.y;
              a1[j + 2] += w.z;
              a1[j + 3] += w.w;
            }
          }
#pragma unroll
        for (int j = 0; j < PER; ++j) v[j] = ok ? __fmul_rn(silu_f32(a0[j]), a1[j]) : 0.0f;
      };
      // a lane's PER values of the raw row at `at`
      auto raw = [&](uint32_t at, float (&v)[PER]) {
#pragma unroll
        for (int j = 0; j < PER; j += 4) {
          if (PHASE == 1) {
            const uint2 d = lds64(at + (lane * PER + j) * 2);
            v[j] = bf16lo(d.x);
            v[j + 1] = bf16hi(d.x);
            v[j + 2] = bf16lo(d.y);
            v[j + 3] = bf16hi(d.y);
          } else {
            const uint4 d = lds128(at + (lane * PER + j) * 4);
            v[j] = __uint_as_float(d.x);
            v[j + 1] = __uint_as_float(d.y);
            v[j + 2] = __uint_as_float(d.z);
            v[j + 3] = __uint_as_float(d.w);
          }
        }
      };

      Step q = walk.begin();
      left = walk.skip(q, left);
      for (; !walk.done(q); step += conv_of(WT), left = walk.skip(q, conv_of(WT))) {
        const uint32_t s = step % S, ph = (step / S) & 1;
        if (!mbar_wait_bounded_warp(smem_u32(&ctl->xraw[s]), ph, abort_flag, kWaitLimitNs)) {
          timed_out = true;
          break;
        }
        if (C::MX) {  // a lane: four rows' words of four codes, as bf16
          auto pair = [](uint32_t w) {  // the low two codes of w
            return pack_bf16x2(e8m0_value(w & 0xFFu), e8m0_value((w >> 8) & 0xFFu));
          };
#pragma unroll
          for (int v = 0; v < C::BOXES * C::WORDS; ++v) {
            const uint4 u = lds128(raw_words(s, v) + lane * 16);
            const uint32_t dst = s_ring + s * C::SCALE_BYTES + (v * kRows + lane * 4) * C::SCALE_ROW;
            __syncwarp();  // the bf16 go over the words
            sts128(dst, make_uint4(pair(u.x), pair(u.x >> 16), pair(u.y), pair(u.y >> 16)));
            sts128(dst + 16, make_uint4(pair(u.z), pair(u.z >> 16), pair(u.w), pair(u.w >> 16)));
          }
        }
        const int n = ctl->cnum[q.ch];
        const uint32_t at = x_ring + s * x_bytes, av = v_ring + s * v_bytes;
        if (PHASE == 2 && partial) {
          const int st = ctl->cstart[q.ch];
          for (int i = 0; i < n; ++i)
            for (int b = 0; b < C::BOXES; ++b) {
              const int col = q.kst * C::KE + b * C::BOX_K + lane * PER;
              float v[PER];
              join(st + i, col, col < f.K, v);
              store_span<PER>(v, at + i * C::PITCH + b * C::SPAN_BYTES, av + (b * cap + i) * 4, lane);
            }
        } else {
          // two spans' latencies together: a row's two, or (one a row) two rows' (an odd last one twice)
          constexpr int kRowsAtOnce = C::BOXES == 2 ? 1 : 2;
          for (int i = 0; i < n; i += kRowsAtOnce) {
            const int i1 = C::BOXES == 2 ? i : (i + 1 < n ? i + 1 : i), b1 = C::BOXES - 1;
            const uint32_t at0 = at + i * C::PITCH, at1 = at + i1 * C::PITCH + b1 * C::SPAN_BYTES;
            float v[PER], w[PER];
            raw(at0, v);
            raw(at1, w);
            store_span<PER>(v, at0, av + i * 4, lane);
            store_span<PER>(w, at1, av + (b1 * cap + i1) * 4, lane);
          }
        }
        // Two groups: each waits for every stage, the other's too, so one barrier
        // stands for weights and activations
        if (groups_of(WT) == 2 && !mbar_wait_bounded_warp(smem_u32(&ctl->full[s]), ph, abort_flag, kWaitLimitNs)) {
          timed_out = true;
          break;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&ctl->xfull[s]));
      }
    };
    run(std::integral_constant<int, 1>{});
    if (!timed_out) run(std::integral_constant<int, 2>{});
    if (timed_out) {
      *abort_flag = 1;
      ctl->err = 2;
    }
  } else {
    // ----------------------------------------------------------- contraction
    const int mw = (warp - 1 - conv_of(WT)) % kMmaWarps, group = (warp - 1 - conv_of(WT)) / kMmaWarps;
    uint32_t handed = 0;  // two groups: units whose sums went from the second to the first
    const int g = lane >> 2, t4 = lane & 3;
    uint32_t s = 0, ph = 0;
    auto run = [&](auto phase_tag) {
      constexpr int PHASE = decltype(phase_tag)::value;
      using C = Cfg<WT, PHASE>;
      constexpr int kPer = PHASE == 1 ? kRows / 2 : kRows;  // channels of a unit
      const PhaseParams& f = p.f[PHASE - 1];
      const Walk walk = walk_of(PHASE);
      const int nbox = (f.K + C::BOX_K - 1) / C::BOX_K;  // boxes along K
      // rows of the fragment: 0..7 from row A, 8..15 from row B
      const int rowA = PHASE == 1 ? 8 * mw : 16 * mw, rowB = PHASE == 1 ? kRows / 2 + 8 * mw : 16 * mw + 8;
      const int lrow = ((lane >> 3) & 1 ? rowB : rowA) + (lane & 7);  // the row this lane addresses for ldmatrix
      const uint32_t w_off = lrow * 128, swz = (lrow & 7) * 16;
      const uint32_t x_off = g * C::PITCH + t4 * (WT == kMx4 ? 16 : 8);
      auto unit = [&](auto nt_tag, const Step& q) {
        constexpr int NT = decltype(nt_tag)::value;
        float acc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
        // what the unit's end needs, asked for before its products
        const int e = ctl->cexp[q.ch], n = ctl->cnum[q.ch], st = ctl->cstart[q.ch];
        const int ca = q.blk * kPer + (PHASE == 1 ? 8 * mw : 16 * mw) + g;  // channel of row A
        const int cb = PHASE == 1 ? ca : ca + 8;
        float fa = 1.0f, fb = 1.0f;
        if (f.mode == kScaleChannel) {
          const float* sc = f.scale + static_cast<int64_t>(e) * (PHASE == 1 ? 2 * f.N : f.N);
          if (ca < f.N) fa = __ldg(sc + ca);
          if (cb < f.N) fb = __ldg(sc + (PHASE == 1 ? f.N : 0) + cb);
        } else if (f.mode == kScaleTensor) {
          fa = fb = __ldg(f.scale);
        }

        // Up to eight tokens: boxes alternate between two register sets, one box's
        // loads in flight while the other's products run.  A stage goes back as
        // soon as its last box is done; the next is waited for before that only if
        // it is already there.
        const int first = q.kst * C::BOXES, last = min(q.end * C::BOXES, nbox);
        uint32_t ls = s, lph = ph;  // the stage that the next load reads
        auto ready = [&] {
          return __all_sync(0xffffffffu, mbar_try_wait(smem_u32(&ctl->xfull[ls]), lph) &&
                                             mbar_try_wait(smem_u32(&ctl->full[ls]), lph));
        };
        auto wait = [&] {
          if (!mbar_wait_bounded_warp(smem_u32(&ctl->xfull[ls]), lph, abort_flag, kWaitLimitNs) ||
              (groups_of(WT) == 1 && !mbar_wait_bounded_warp(smem_u32(&ctl->full[ls]), lph, abort_flag, kWaitLimitNs))) {
            timed_out = true;
            *abort_flag = 1;
          }
        };
        auto box_at = [&](uint32_t sg, int v) {
          BoxAt a;
          a.wt = base + sg * C::STAGE_W + v * kBoxW + w_off;
          a.xb = x_ring + sg * x_bytes + v * C::SPAN_BYTES + x_off;
          a.sA = s_ring + sg * C::SCALE_BYTES + (v * C::WORDS * kRows + rowA + g) * C::SCALE_ROW;
          a.sB = a.sA + (rowB - rowA) * C::SCALE_ROW;
          a.xs = v_ring + sg * v_bytes + v * cap * 4 + t4 * 8;
          return a;
        };
        // box j of the unit: its loads, and what follows when its products are done
        auto load = [&](Box<WT, PHASE, NT>& b, int j) {
          b.load(box_at(ls, C::BOXES == 2 ? j & 1 : 0), swz, f.mode == kScaleBlock);
          if (C::BOXES == 1 || (j & 1) || j + 1 == last) {
            if (++ls == S) {
              ls = 0;
              lph ^= 1;
            }
          }
        };
        auto work = [&](Box<WT, PHASE, NT>& b, int j) {
          b.contract(acc, box_at(s, C::BOXES == 2 ? j & 1 : 0));
          if (C::BOXES == 1 || (j & 1) || j + 1 == last) {
            fence_proxy_async_smem();  // this warp's reads of the stage before the next copy into it
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ctl->empty[s]));
            if (++s == S) {
              s = 0;
              ph ^= 1;
            }
          }
        };
        if constexpr (groups_of(WT) == 2) {
          // Every other stage; the ring position moves on over the partner's, too.  A
          // stage is given back by both groups: a barrier tells only the parity of
          // its last round, so the slot may not be filled again before this warp
          // has seen the partner's round.
          auto step_on = [&](uint32_t& a, uint32_t& b) {
            if (++a == S) {
              a = 0;
              b ^= 1;
            }
          };
          for (int j = first; j < last; ++j) {
            wait();
            if (timed_out) break;
            if (((j - first) & 1) == group) {
              Box<WT, PHASE, NT> b;
              load(b, j);
              work(b, j);
            } else {
              if (lane == 0) mbar_arrive(smem_u32(&ctl->empty[s]));
              step_on(ls, lph);
              step_on(s, ph);
            }
          }
          if (!timed_out) {
            float* r = red + mw * 32 * 4 * kMaxNT + lane;
            if (group == 1) {
              if (!mbar_wait_bounded_warp(smem_u32(&ctl->rempty[mw]), (handed & 1) ^ 1, abort_flag, kWaitLimitNs)) timed_out = true;
              if (!timed_out) {
#pragma unroll
                for (int i = 0; i < 4 * NT; ++i) r[32 * i] = acc[i / 4][i % 4];
                mbar_arrive(smem_u32(&ctl->rfull[mw]));
              }
            } else {
              if (!mbar_wait_bounded_warp(smem_u32(&ctl->rfull[mw]), handed & 1, abort_flag, kWaitLimitNs)) timed_out = true;
              if (!timed_out) {
#pragma unroll
                for (int i = 0; i < 4 * NT; ++i) acc[i / 4][i % 4] += r[32 * i];
                mbar_arrive(smem_u32(&ctl->rempty[mw]));
              }
            }
            if (timed_out) *abort_flag = 1;
            ++handed;
          }
        } else if constexpr (NT == 1) {
          Box<WT, PHASE, NT> b0, b1;
          wait();
          if (!timed_out) load(b0, first);
          for (int j = first; j < last && !timed_out; j += 2) {  // first is even (two boxes a stage) or any (one)
            if (j + 1 < last) {
              if (C::BOXES == 1) {
                if (ready()) {
                  load(b1, j + 1);
                  work(b0, j);
                } else {
                  work(b0, j);
                  wait();
                  if (timed_out) break;
                  load(b1, j + 1);
                }
              } else {
                load(b1, j + 1);
                work(b0, j);
              }
              if (j + 2 < last) {
                if (ready()) {
                  load(b0, j + 2);
                  work(b1, j + 1);
                } else {
                  work(b1, j + 1);
                  wait();
                  if (timed_out) break;
                  load(b0, j + 2);
                }
              } else {
                work(b1, j + 1);
              }
            } else {
              work(b0, j);
            }
          }
        } else {  // (two sets of more tokens' fragments do not fit in the registers)
          for (int j = first; j < last; ++j) {
            if (C::BOXES == 1 || !(j & 1)) wait();
            if (timed_out) break;
            Box<WT, PHASE, NT> b;
            load(b, j);
            work(b, j);
          }
        }
        if (timed_out || group > 0) return;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int col = nt * 8 + 2 * t4 + j;
            if (col >= n) continue;
            const float va = acc[nt][j] * fa, vb = acc[nt][2 + j] * fb;
            if (PHASE == 1) {
              if (ca >= f.N) continue;
              if (walk.segs == 1) {
                f.out[static_cast<int64_t>(st + col) * f.N + ca] = __fmul_rn(silu_f32(va), vb);
              } else {
                float* o = f.out + (static_cast<int64_t>(q.seg) * slots + st + col) * 2 * f.N;
                o[ca] = va;
                o[f.N + ca] = vb;
              }
            } else {
              float* o = f.out + (static_cast<int64_t>(q.seg) * slots + st + col) * f.N;
              if (ca < f.N) o[ca] = va;
              if (cb < f.N) o[cb] = vb;
            }
          }
      };

      for (Step q = walk.begin(); !walk.done(q) && !timed_out;) {
        const int n = ctl->cnum[q.ch];
        if (n <= 8)
          unit(std::integral_constant<int, 1>{}, q);
        else if (n <= 16)
          unit(std::integral_constant<int, 2>{}, q);
        else
          unit(std::integral_constant<int, groups_of(WT) == 2 ? 2 : 4>{}, q);
        if (PHASE == 2 && !timed_out && group == 0) {
          // the last unit (over all CTAs) that gets to these 16 columns sums their
          // pairs into y: each warp for the rows of its own, without its neighbours
          __threadfence();
          __syncwarp();
          unsigned int done = 0;
          if (lane == 0) done = atomicAdd(p.count + q.blk * kMmaWarps + mw, 1u);
          done = __shfl_sync(0xffffffffu, done, 0);
          const int d = q.blk * kRows + 16 * mw + 4 * (lane & 3);
          const bool all = done == static_cast<unsigned>(nchunk * walk.segs - 1);
          if (all && lane == 0) p.count[q.blk * kMmaWarps + mw] = 0;  // for the next call
          if (all && d < f.N) {  // (N % 16 == 0: for all lanes or none)
            __threadfence();
            __syncwarp();
            const int64_t seg_pitch = static_cast<int64_t>(slots) * f.N;
            for (int t = lane >> 2; t < p.T; t += 8) {
              float a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
              for (int j0 = 0; j0 < p.k; j0 += 8) {
                float4 o[8];
                bool ok[8];
                float w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {  // eight pairs' loads first
                  const int pr = t * p.k + j0 + j;
                  const int slot = j0 + j < p.k ? ctl->pos[pr] : 0xFFFF;
                  ok[j] = slot != 0xFFFF;
                  o[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                  w[j] = 1.0f;
                  if (ok[j]) {
                    const float* src = f.out + static_cast<int64_t>(slot) * f.N + d;
                    o[j] = __ldcg(reinterpret_cast<const float4*>(src));
                    if (p.topk_w) w[j] = __ldg(p.topk_w + pr);
                  }
                }
                for (int sg = 1; sg < walk.segs; ++sg)
#pragma unroll
                  for (int j = 0; j < 8; ++j)
                    if (ok[j]) {
                      const float4 v = __ldcg(reinterpret_cast<const float4*>(
                          f.out + sg * seg_pitch + static_cast<int64_t>(ctl->pos[t * p.k + j0 + j]) * f.N + d));
                      o[j].x += v.x;
                      o[j].y += v.y;
                      o[j].z += v.z;
                      o[j].w += v.w;
                    }
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  if (ok[j]) {
                    a[0] = __fmaf_rn(w[j], o[j].x, a[0]);
                    a[1] = __fmaf_rn(w[j], o[j].y, a[1]);
                    a[2] = __fmaf_rn(w[j], o[j].z, a[2]);
                    a[3] = __fmaf_rn(w[j], o[j].w, a[3]);
                  }
              }
              *reinterpret_cast<uint2*>(p.y + static_cast<int64_t>(t) * f.N + d) =
                  make_uint2(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]));
            }
          }
          __syncwarp();
        }
        q.u += gridDim.x;
        if (!walk.done(q)) walk.open(q);
      }
    };
    if (p.stall_ns && !mbar_wait_bounded_warp(smem_u32(&ctl->never), 0, abort_flag, p.stall_ns)) {
      timed_out = true;
      *abort_flag = 1;
    }
    if (!timed_out) run(std::integral_constant<int, 1>{});
    if (!timed_out) {
      __threadfence();
      __syncwarp();
      if (lane == 0 && group == 0) atomicAdd(p.sync, 1u);
      run(std::integral_constant<int, 2>{});
    }
    if (timed_out) {
      *abort_flag = 1;
      ctl->err = 2;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && ctl->err) {
    atomicOr(p.sync, kBroken);
    raise_error(&g_err, MOE_DEVERR_TIMEOUT);
  }
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

// The weights as bytes [slabs][rows][bytes] (wi: two slabs of F rows an
// expert; wo: one of D rows), boxes of 128 bytes x box_rows x box_slabs with
// the 128-byte swizzle; reads past the extents return zeros.
bool make_map(CUtensorMap* m, const void* ptr, uint64_t bytes, uint64_t rows, uint64_t slabs, uint32_t box_rows,
              uint32_t box_slabs) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {bytes, rows, slabs}, strides[2] = {bytes, bytes * rows};
  cuuint32_t box[3] = {128, box_rows, box_slabs}, estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(ptr), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int64_t kSyncWords = 64;
int64_t align256(int64_t b) { return (b + 255) / 256 * 256; }
int64_t blocks(int64_t n, int64_t per) { return (n + per - 1) / per; }

// Segments of K at most: their sums take workspace, and only a few pairs need them.
int max_segs(int64_t R) {
  const int64_t s = R > 0 ? 128 / R : 1;
  return static_cast<int>(s < 1 ? 1 : (s > kMaxSegs ? kMaxSegs : s));
}

// Workspace: the sync words and a counter for every 16 output columns (zero
// between calls; room for the largest D, so that calls of other shapes may
// follow on the same workspace) | h fp32 [R, F] or partial a [segs][R, 2F] | o fp32
// [segs][R, D], each part 256-byte aligned.
constexpr int64_t kCountBytes = (kSyncWords + kMaxDim / kRows * kMmaWarps) * 4;
static_assert(kCountBytes % 256 == 0, "h starts 256-byte aligned");
int64_t h_bytes(int64_t R, int64_t F) {
  const int64_t s = max_segs(R);
  return align256(R * F * 4 * (s > 1 ? 2 * s : 1));
}
int64_t o_bytes(int64_t R, int64_t D) { return align256(R * D * 4 * max_segs(R)); }

bool shape_ok(int64_t T, int k, int64_t D, int64_t F) {
  return T >= 0 && T <= kMaxTokens && k > 0 && k <= 32 && T * k <= kMaxPairs && D > 0 && F > 0 && D % 16 == 0 &&
         F % 16 == 0 && D <= kMaxDim && F <= kMaxDim;
}

template <int WT>
moe_status launch(const void* w_in, const void* w_out, Params p, int sms, cudaStream_t st) {
  using C = Cfg<WT, 2>;
  const PhaseParams &f1 = p.f[0], &f2 = p.f[1];
  CUtensorMap tm1, tm2;
  const int half = WT == kMx4 ? 2 : 1;
  if (!make_map(&tm1, w_in, f1.K / half, f1.N, 2ull * p.El, kRows / 2, 2) ||
      !make_map(&tm2, w_out, f2.K / half, f2.N, p.El, kRows, 1))
    return MOE_ERR_CUDA;
  if (groups_of(WT) == 2 && p.cap > 8 * kMaxNT) p.cap = 8 * kMaxNT;
  const size_t stage = C::STAGE_W + static_cast<size_t>(p.cap) * (C::PITCH + 4 * C::BOXES) + C::SCALE_BYTES;
  const size_t red = groups_of(WT) == 2 ? kMmaWarps * 32 * 4 * kMaxNT * 4 : 0;
  const size_t fixed = 1024 + kCtlBytes + red;
  p.stages = static_cast<int>((kSmemLimit - fixed) / stage);
  if (p.stages > kMaxStages) p.stages = kMaxStages;
  // the ring holds the pair sort's bits and words first (at most 136 KB; the smallest ring has 160)
  const size_t sort = (static_cast<size_t>((p.T * p.k + 31) / 32) + 1) * p.El * 4;
  // (a converting warp waits for one stage of its own at a time: a ring shorter
  // than their number would let one mistake a slot's last round for its next)
  MOE_HOST_CHECK(p.stages >= conv_of(WT) && p.stages * stage >= sort, MOE_ERR_UNSUPPORTED);
  const size_t smem = fixed + p.stages * stage;
  // no more CTAs than units (a chunk a pair, all segments)
  const int64_t u = static_cast<int64_t>(p.T) * p.k * p.smax * (f1.nblock > f2.nblock ? f1.nblock : f2.nblock);
  auto kernel = decode_kernel<WT>;
  MOE_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit));
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;  // all CTAs at once: they wait for one another between the phases
  attr[0].val.cooperative = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(u < sms ? u : sms));
  cfg.blockDim = dim3(threads_of(WT));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  MOE_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, tm1, tm2, p));
  return MOE_OK;
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

// The most that any batch of up to T tokens needs: a few pairs' sums of segments
// can take more than more pairs' whole sums (h: 1024 F bytes for 16 pairs in eight
// segments, 260 F for 65 pairs in one).
extern "C" size_t moe_ffn_decode_workspace_bytes(int64_t T, int k, int64_t D, int64_t F) {
  if (!shape_ok(T, k, D, F)) return 0;
  int64_t most = 0;
  for (int64_t t = 1; t <= T; ++t) {
    const int64_t b = h_bytes(t * k, F) + o_bytes(t * k, D);
    most = b > most ? b : most;
  }
  return static_cast<size_t>(kCountBytes + most);
}

extern "C" __attribute__((visibility("hidden"))) uint64_t moe_detail_stall_ns();

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
  float* h = reinterpret_cast<float*>(ws + kCountBytes);
  float* o = reinterpret_cast<float*>(ws + kCountBytes + h_bytes(R, F));
  const int ke = 256;  // values of K in a stage, of either width
  const int d = static_cast<int>(D), f = static_cast<int>(F);
  Params p{};
  p.f[0] = {x, static_cast<const float*>(s_in), h, d, f, kin, static_cast<int>(blocks(F, kRows / 2)),
            static_cast<int>(blocks(D, ke))};
  p.f[1] = {h, static_cast<const float*>(s_out), o, f, d, kout, static_cast<int>(blocks(D, kRows)),
            static_cast<int>(blocks(F, ke))};
  p.ids = topk_ids;
  p.topk_w = topk_w;
  p.y = y;
  p.sync = reinterpret_cast<unsigned int*>(ws);
  p.count = p.sync + kSyncWords;
  p.T = static_cast<int>(T);
  p.k = k;
  p.E = E;
  p.g0 = group_offset;
  p.El = E_local;
  // Pairs a chunk.  A narrow one leaves the ring more of shared memory; an
  // expert with more pairs takes several chunks and is read again (from L2: its
  // chunks run side by side), so it has to be rare: the mean number of pairs an
  // expert is at most 2 (for 8; Poisson: 1 expert in 4000 has more) or 6 (for 16).
  p.cap = T <= 8 || R <= 2 * static_cast<int64_t>(E_local) ? 8
                                                           : (T <= 16 || R <= 6 * static_cast<int64_t>(E_local) ? 16 : 32);
  p.smax = max_segs(R);
  p.stall_ns = moe_detail_stall_ns();
  switch (type) {
    case MOE_WEIGHT_E4M3: return launch<kE4M3>(w_in, w_out, p, sms, st);
    case MOE_WEIGHT_INT8: return launch<kInt8>(w_in, w_out, p, sms, st);
    case MOE_WEIGHT_MXFP8: return launch<kMx8>(w_in, w_out, p, sms, st);
    default: return launch<kMx4>(w_in, w_out, p, sms, st);
  }
}
