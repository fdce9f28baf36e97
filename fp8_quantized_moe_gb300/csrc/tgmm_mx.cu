// Weight gradient of a grouped matmul on block-scaled 8-bit operands (sm_103a):
//   tgmm_fp8_mx  out[e, k, n] = sum_{m in e} r(lhs)[m, k] r(rhs)[m, n]   (fp32 out)
// from bf16 lhs and rhs, each rounded (r) to e4m3 with one power-of-two scale for
// every 32 consecutive rows of an expert and column: the contracted dimension is the
// row, so the tensor core's block-scaled MMA (tcgen05.mma.kind::mxf8f6f4, one E8M0
// scale per 32 values of K) applies both scales and one fp32 accumulator runs over all
// of an expert's rows.
//
// The scale of a block is the smallest power of two, 2^-127 at least, with
// amax <= 448 * 2^X, so no value saturates (the MX formats' own rule, floor(log2 amax) - 8,
// cuts off up to an eighth of the largest value; a gradient sums such values, all cut
// off to the same side).  Division by it is exact: the code is e4m3's rounding of the
// value alone.
//
// e4m3 has no infinity.  A block with one gets the scale kInfCode, which no other block has,
// and its infinities the code 448, far above the block's finite values but not above what a
// small value of the other operand brings back into fp32's range.  So that an overflow in a
// gradient is never lost, the product's epilogue warps read the bf16 operands again where the
// scales say that there is an infinity, and add its products with values other than zero to
// the sums (add_infinities).  Where there is none this costs a word for each CTA that rounds,
// read while the first tile's MMAs run.
//
// Two kernels:
//   round_rows_kernel  both operands to codes in the workspace, transposed: for 128 rows
//     of an expert (padded with zeros) and 128 columns a 16 KB tile, the image that the MMA
//     reads from shared memory (128 lines of 128 rows' codes, 128-byte swizzle); the scale
//     codes as the 32 x 16-byte atoms that go to tensor memory.  Line p of a tile holds column
//     64 (p / 8 % 2) + 8 (p % 8) + p / 16: a lane has 8 columns of 8 consecutive rows, and in
//     this order the 8-byte pieces of a warp's lanes fall on different banks.  A tile goes out
//     as one bulk copy (stored by the lanes, 8 bytes each, L1 was the busiest unit).  Maxima
//     of 32 rows are among 4 lanes.  Bound by memory: 2 bytes read, 1 written.
//   tgmm_mx_kernel  persistent pairs of CTAs, 256 (k) x 256 (n) tiles, 128 rows of
//     k and half of B a CTA (16 warps, one CTA per SM):
//     warp 0       TMA producer: per stage one block of 128 rows, A 16 KB and half of B
//                  16 KB, and the scale atoms of this CTA's k rows and of all of n.
//     warp 1       of the pair's even CTA: MMA issuer, an M = 256, N = 256 MMA for each 32
//                  rows that the block holds.
//     warps 4..7   the scale atoms from shared to tensor memory, each to its quarter of the
//                  lanes (tcgen05.st; copied by tcgen05.cp they would stand in the tensor
//                  core's own queue, in front of the products).
//     warps 8..15  epilogue: the accumulator to 128 registers a thread, accumulator
//                  handed back, then whole 32-byte sectors to memory, beside the next
//                  tile's MMAs.
//     Tiles run expert-major, then n tile, then k tile.
//     One CTA per 128 x 256 tile needs 48 KB a block and SM, some 640 clocks (the 77 bytes a
//     clock that gmm_block.cu's loads reach alone); a pair needs 32 KB.
//     Measured with the rounding, back to back: 16384 rows, 4096 x 28672, 8 experts 1.68 to
//     1.76 ms (rounding 0.26; in bursts 1.55: the power limit lowers the clock); there without
//     the stores 1.33, without the MMAs 1.35, with neither 0.96: loads, MMAs and stores (3.8
//     GB) overlap only in part.  49152 rows, 4096 x 2816, 64 experts: 780 to 820 us (rounding
//     166, stores alone 475); 16384 rows, 2048 x 1536, 128 experts: 302 to 319 us (39, 260).  One CTA a
//     128 x 256 tile, its issuing loops run by one lane and its scales by tcgen05.cp: 1.87 ms,
//     980, 376 us; the pair with such loops: 1.75 ms; tiles stored by the lanes 3 % more
//     (rounding 0.28 ms, 187, 47 us).  Gradients by TMA from shared memory instead of the
//     transpose: 1.69 ms and 855 us where it gave 1.60 and 835.
//
// Every wait is bounded; on expiry the kernel raises MOE_DEVERR_TIMEOUT, lets what
// it issued finish and returns.
#include <algorithm>

#include "grouped.cuh"

namespace moe {
namespace {

__device__ unsigned int g_err;

constexpr int kRB = 128;  // rows of a block (four scales a column)
constexpr int kAtom = 512;
constexpr int kTileBytes = 128 * kRB;

// ---- local groups --------------------------------------------------------
struct Tables {
  int start[kMaxGroups + 1];   // first row of each local group; the last: their end
  int kstart[kMaxGroups + 1];  // first 128-row block of each
};

// Filled by all threads of the block (256 at least); false when a size is negative
// or they do not add up to M.  Ends with a barrier.
__device__ bool build_tables(const int32_t* sizes, int E, int g0, int El, int64_t M, Tables* t) {
  __shared__ int64_t wrows[8];
  __shared__ int wblk[8];
  __shared__ int bad_any;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) bad_any = 0;
  __syncthreads();
  int sz[4] = {0, 0, 0, 0};
  int64_t rows = 0;
  int blk = 0;
  bool bad = false;
  if (tid < 256) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int g = 4 * tid + i;
      if (g < E) sz[i] = __ldg(sizes + g);
      bad = bad || sz[i] < 0;
      rows += sz[i];
      if (g >= g0 && g < g0 + El && sz[i] > 0) blk += (sz[i] + kRB - 1) / kRB;
    }
    if (bad) bad_any = 1;
  }
  int64_t ir = rows;
  int ib = blk;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t r = __shfl_up_sync(0xffffffffu, ir, o);
    const int b = __shfl_up_sync(0xffffffffu, ib, o);
    if (lane >= o) {
      ir += r;
      ib += b;
    }
  }
  if (warp < 8 && lane == 31) {
    wrows[warp] = ir;
    wblk[warp] = ib;
  }
  __syncthreads();
  int64_t total = 0;
  if (tid < 256) {
    int64_t r = ir - rows;
    int b = ib - blk;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      if (w < warp) {
        r += wrows[w];
        b += wblk[w];
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int local = 4 * tid + i - g0;
      if (4 * tid + i < E && local >= 0 && local < El) {
        t->start[local] = static_cast<int>(r);
        t->kstart[local] = b;
        if (sz[i] > 0) b += (sz[i] + kRB - 1) / kRB;
        if (local == El - 1) {
          t->start[El] = static_cast<int>(r + sz[i]);
          t->kstart[El] = b;
        }
      }
      r += sz[i];
    }
  }
#pragma unroll
  for (int w = 0; w < 8; ++w) total += wrows[w];
  __syncthreads();
  return !bad_any && total == M;
}

// ---- rounding ------------------------------------------------------------
struct Operand {
  const uint16_t* x;   // [src_rows, C]
  const int32_t* idx;  // row m is x[idx[m] / k], or x[m] without
  int k;
  int64_t src_rows;
  int C, ncb, nrb;     // columns; 128-column blocks; atoms a row block (a multiple of what a tile reads)
  uint8_t* q;          // [row blocks][ncb][kTileBytes]
  uint8_t* sf;         // [row blocks][nrb][512]
};

constexpr int kInfCode = 253;  // (finite values: 247 at the most; NaN among them: 248)
// What stands for an infinity's bits, 0x7F80, in block_scale: one test for a lane's eight
// columns, and block_scale gives kInfCode without one of its own.
constexpr uint32_t kInfBits = 0x7F80, kInfMark = (kInfCode + 8) << 7;
constexpr int kRoundCtas = 1024;       // CTAs that round, at the most: each has a word for "an infinity seen"

// Power-of-two scale of a block from the bf16 bits of its largest magnitude:
// the E8M0 code X + 127 and, through inv, 2^-X.
__device__ __forceinline__ uint32_t block_scale(uint32_t amax_bits, float& inv) {
  const int field = static_cast<int>(amax_bits >> 7), mant = static_cast<int>(amax_bits & 0x7F);
  const int code = max(field - 8 + (mant > 0x60 ? 1 : 0), 0);  // X = field - 127 - 8 (+ 1 above 1.75 * 2^8)
  inv = __uint_as_float(static_cast<uint32_t>(254 - code) << 23);
  return static_cast<uint32_t>(code);
}

__global__ void __launch_bounds__(256, 4) round_rows_kernel(const Operand oa, const Operand ob, const int32_t* sizes,
                                                            int E, int g0, int El, int64_t M, int* inf_seen) {
  __shared__ Tables t;
  __shared__ __align__(16) uint8_t sfs[2][kAtom];
  __shared__ __align__(128) uint8_t tile[2][kTileBytes];
  grid_release_next();  // (the product's kernel takes over the SMs as they come free)
  if (!build_tables(sizes, E, g0, El, M, &t)) return;  // (the product's kernel raises the error)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // warp: 32 rows (warp & 3) of 64 columns (warp >> 2); lane: 8 rows, 8 columns
  const int j = warp & 3, rl = lane >> 3, cu = (warp >> 2) * 64 + (lane & 7) * 8;
  const int per = oa.ncb + ob.ncb;
  const int64_t total = static_cast<int64_t>(t.kstart[El]) * per;
  int sel = 0;
  bool inf = false;
  for (int64_t w = blockIdx.x; w < total; w += gridDim.x, sel ^= 1) {
    const int kb = static_cast<int>(w / per);
    int cb = static_cast<int>(w - static_cast<int64_t>(kb) * per);
    const bool second = cb >= oa.ncb;
    if (second) cb -= oa.ncb;
    const Operand& o = second ? ob : oa;
    int lo = 0, hi = El;  // the last group whose first block is <= kb: it is not empty
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (t.kstart[mid] <= kb) lo = mid; else hi = mid;
    }
    const int r0 = t.start[lo] + (kb - t.kstart[lo]) * kRB + 32 * j + 8 * rl;  // this thread's first row
    const int nr = t.start[lo + 1] - r0;                                       // rows of the group from there on
    const int c0 = cb * 128 + cu;
    // lane (rl, i) finds the source of row i of its eight, the others take it from there
    int src = r0 + (lane & 7);
    if (o.idx && (lane & 7) < nr) {
      const int pick = __ldg(o.idx + src);
      const uint32_t row = static_cast<uint32_t>(pick) / static_cast<uint32_t>(o.k);
      src = static_cast<int>(row);
      if (pick < 0 || row >= o.src_rows) {
        raise_error(&g_err, MOE_DEVERR_BAD_POSITION);
        src = -1;
      }
    }
    uint4 d[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = __shfl_sync(0xffffffffu, src, (lane & 24) + i);
      d[i] = make_uint4(0, 0, 0, 0);
      if (i < nr && row >= 0 && c0 < o.C)
        d[i] = __ldg(reinterpret_cast<const uint4*>(o.x + static_cast<int64_t>(row) * o.C + c0));
    }
    // largest magnitude of each column over the 32 rows: bf16 magnitudes order
    // like their bits
    uint32_t m[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      m[0] = __vmaxu2(m[0], d[i].x & 0x7FFF7FFFu);
      m[1] = __vmaxu2(m[1], d[i].y & 0x7FFF7FFFu);
      m[2] = __vmaxu2(m[2], d[i].z & 0x7FFF7FFFu);
      m[3] = __vmaxu2(m[3], d[i].w & 0x7FFF7FFFu);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      m[c] = __vmaxu2(m[c], __shfl_xor_sync(0xffffffffu, m[c], 8));
      m[c] = __vmaxu2(m[c], __shfl_xor_sync(0xffffffffu, m[c], 16));
    }
    const uint32_t top = __vmaxu2(__vmaxu2(m[0], m[1]), __vmaxu2(m[2], m[3]));
    if (max(top >> 16, top & 0xFFFFu) >= kInfBits) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if ((m[c] & 0xFFFFu) == kInfBits) {
          m[c] ^= kInfBits ^ kInfMark;
          inf = true;
        }
        if (m[c] >> 16 == kInfBits) {
          m[c] ^= (kInfBits ^ kInfMark) << 16;
          inf = true;
        }
      }
    }
    // column 64 (warp / 4) + 8 (lane % 8) + c is line 16 c + 8 (warp / 4) + lane % 8
    const int line0 = 8 * (warp >> 2) + (lane & 7);
    uint8_t* t0 = tile[sel] + line0 * 128 + (((2 * j + (rl >> 1)) ^ (lane & 7)) << 4) + 8 * (rl & 1);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      float inv;
      const uint32_t code = block_scale((c & 1) ? m[c >> 1] >> 16 : m[c >> 1] & 0xFFFFu, inv);
      const int line = 16 * c + line0;
      if (rl == 0) sfs[sel][16 * (line & 31) + 4 * (line >> 5) + j] = static_cast<uint8_t>(code);
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t x = (c >> 1) == 0 ? d[i].x : (c >> 1) == 1 ? d[i].y : (c >> 1) == 2 ? d[i].z : d[i].w;
        v[i] = __fmul_rn((c & 1) ? bf16hi(x) : bf16lo(x), inv);  // exact: a power of two
      }
      *reinterpret_cast<uint2*>(t0 + 16 * 128 * c) = pack_e4m3x8(v);
    }
    fence_proxy_async_smem();
    if (tid == 0) bulk_wait_read<0>();  // the last tile's copy has read the other buffer, which is written next
    __syncthreads();                    // (one barrier a tile: the buffers alternate)
    if (tid == 0) {
      bulk_store(o.q + (static_cast<int64_t>(kb) * o.ncb + cb) * kTileBytes, smem_u32(tile[sel]), kTileBytes);
      bulk_commit();
    }
    if (tid < 32)
      *reinterpret_cast<uint4*>(o.sf + (static_cast<int64_t>(kb) * o.nrb + cb) * kAtom + 16 * tid) =
          *reinterpret_cast<const uint4*>(&sfs[sel][16 * tid]);
  }
  const int any = __syncthreads_or(inf);
  if (tid == 0) {
    inf_seen[blockIdx.x] = any;
    bulk_wait_all();
  }
}

// ---- product -------------------------------------------------------------
constexpr int kBM = 128, kBN = 256;
constexpr int kStages = 6;
constexpr int kABytes = kBM * kRB, kBBytes = kBN / 2 * kRB;
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kSfBytes = 3 * kAtom;  // a stage's scale atoms: A's, B's two
constexpr int kSfCols = 16, kSfCol0 = kBN;  // tensor-memory columns of a stage's scales: A's 4, B's 8, 4 unused
constexpr int kCtrlWarps = 8, kEpiWarps = 8;
constexpr int kSfWarp = 4;  // the first of the four that move scales
constexpr int kThreads = 32 * (kCtrlWarps + kEpiWarps);
// registers a thread: 128 at launch (a 512-thread CTA alone on its SM), handed from the
// first two warpgroups to the epilogue
constexpr uint32_t kCtrlRegs = 56, kEpiRegs = 200;
static_assert(256 * kCtrlRegs + 256 * kEpiRegs <= 128 * kThreads, "register split");
static_assert(kSfCol0 + kStages * kSfCols <= 512, "tensor memory");

struct Params {
  const int32_t* group_sizes;
  int E, g0, El;
  int64_t M;
  int K, N, ktiles, ntiles;
  int ncb_a, ncb_b;  // 128-column blocks
  int nrb_a, nrb_b;
  const uint8_t* sf_a;
  const uint8_t* sf_b;
  const int* inf_seen;  // a word for each CTA that rounded
  int round_ctas;
  const uint16_t* lhs;  // the operands themselves, for add_infinities
  const int32_t* lhs_index;
  int lhs_k;
  int64_t lhs_rows;
  const uint16_t* rhs;
  float* out;
  uint64_t stall_ns;  // test hook (moe_test_stall_consumers): 0, or the wait limit in ns
};

struct Ctl {
  uint64_t full[kStages], empty[kStages];  // full: the even CTA's counts both CTAs
  uint64_t sfull[kStages];                 // this CTA's scale atoms have landed
  uint64_t tfull, tempty, drain;
  uint64_t never;  // test hook: a barrier that nothing arrives on
  uint32_t tmem_base;
  int abort_flag, no_abort, err;
  Tables t;
};
constexpr size_t kCtlBytes = (sizeof(Ctl) + 127) / 128 * 128;
constexpr size_t kSmem = 1024 + static_cast<size_t>(kStages) * (kStageBytes + kSfBytes) + kCtlBytes;
static_assert(kSmem <= 232448, "shared memory per CTA");

struct Tile {
  int el, kb0, rows, k0, n0;  // rows: of the expert
};

// (ktiles: pairs of 128 rows of k)
__device__ __forceinline__ Tile get_tile(const Params& p, const Ctl* c, int t, int rank) {
  const int per = p.ktiles * p.ntiles;
  Tile tl;
  tl.el = t / per;
  const int r = t - tl.el * per, nt = r / p.ktiles;
  tl.k0 = (2 * (r - nt * p.ktiles) + rank) * kBM;  // (K or more: an odd CTA without rows)
  tl.n0 = nt * kBN;
  tl.kb0 = c->t.kstart[tl.el];
  tl.rows = c->t.start[tl.el + 1] - c->t.start[tl.el];
  return tl;
}

__device__ __forceinline__ void store8(float* o, const uint32_t* v, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(o), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    *reinterpret_cast<uint4*>(o) = make_uint4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<uint4*>(o + 4) = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

// D (+)= (A 2^(sfa - 127)) (B 2^(sfb - 127))^T over a CTA pair: M = 256 rows, 128 from each
// CTA; each CTA's tensor memory holds the scales of its own rows of A and of all of B.
__device__ __forceinline__ void mma_mx_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                            uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// Whether 16 bytes of scale codes hold kInfCode.
__device__ __forceinline__ bool has_inf(const uint4& v) {
  constexpr uint32_t c = kInfCode * 0x01010101u;
  return (__vcmpeq4(v.x, c) | __vcmpeq4(v.y, c) | __vcmpeq4(v.z, c) | __vcmpeq4(v.w, c)) != 0;
}

// Row k of the output that the accumulator's row l of warp quarter q4 is.
__device__ __forceinline__ int row_of_lane(int k0, int q4, int l) {
  return k0 + 64 * ((l >> 3) & 1) + 8 * (l & 7) + (l >> 4) + 2 * q4;
}

// The products that an infinity enters with a value other than zero, added to the 32 x 128 sums
// that this warp has stored for a tile.  A lane keeps its four columns' signs as masks over
// the rows k, so that any number of infinities costs the same: the bf16 operands of the row
// blocks that hold one are read again.  16384 x 4096 x 28672 over 8 experts, 1.58 ms without:
// 3.1 ms with one infinity, 0.21 s with nothing else (a step to be skipped).
__device__ __noinline__ void add_infinities(const Params& p, const Ctl* c, const Tile& tl, int q4, int n0) {
  const int lane = threadIdx.x & 31, k = row_of_lane(tl.k0, q4, lane), n4 = n0 + 4 * lane;
  const int nkb = (tl.rows + kRB - 1) / kRB;
  const bool k_in = k < p.K, n_in = n4 < p.N;
  if (tl.k0 >= p.K || n0 >= p.N) return;
  const uint8_t* fa = p.sf_a + (static_cast<int64_t>(tl.kb0) * p.nrb_a + tl.k0 / 128) * kAtom + 16 * lane;
  const uint8_t* fb = p.sf_b + (static_cast<int64_t>(tl.kb0) * p.nrb_b + n0 / 128) * kAtom + 16 * lane;
  uint32_t pos[4] = {0, 0, 0, 0}, neg[4] = {0, 0, 0, 0};  // bit l: row_of_lane(l)
  for (int kb0 = 0; kb0 < nkb; kb0 += 8) {
    uint32_t found = 0;  // blocks with an infinity, of eight (written while this kernel waited: not __ldg)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (kb0 + i < nkb &&
          (has_inf(__ldcg(reinterpret_cast<const uint4*>(fa + static_cast<int64_t>(kb0 + i) * p.nrb_a * kAtom))) |
           has_inf(__ldcg(reinterpret_cast<const uint4*>(fb + static_cast<int64_t>(kb0 + i) * p.nrb_b * kAtom)))))
        found |= 1u << i;
    found = __reduce_or_sync(0xffffffffu, found);
    for (; found; found &= found - 1) {
      const int r0 = (kb0 + __ffs(found) - 1) * kRB, left = min(tl.rows - r0, kRB);
      const int64_t first = c->t.start[tl.el] + r0;
      for (int h = 0; h < left; h += 32) {
        int src = -1;  // lane: the lhs row of row h + lane (-1: zeros, reported where they were rounded)
        if (h + lane < left) {
          src = static_cast<int>(first) + h + lane;
          if (p.lhs_index) {
            const int pick = __ldg(p.lhs_index + src);
            src = pick < 0 || pick / p.lhs_k >= p.lhs_rows ? -1 : pick / p.lhs_k;
          }
        }
#pragma unroll 1
        for (int i0 = h; i0 < min(left, h + 32); i0 += 8) {
          float a[8];
          uint2 d[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int row = __shfl_sync(0xffffffffu, src, (i0 + i) & 31);
            a[i] = 0.0f;
            d[i] = make_uint2(0, 0);
            if (k_in && row >= 0)
              a[i] = __uint_as_float(static_cast<uint32_t>(__ldg(p.lhs + static_cast<int64_t>(row) * p.K + k)) << 16);
            if (n_in && i0 + i < left) d[i] = __ldg(reinterpret_cast<const uint2*>(p.rhs + (first + i0 + i) * p.N + n4));
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t up = __ballot_sync(0xffffffffu, a[i] > 0.0f), down = __ballot_sync(0xffffffffu, a[i] < 0.0f);
            const uint32_t up_inf = __ballot_sync(0xffffffffu, a[i] == INFINITY);
            const uint32_t down_inf = __ballot_sync(0xffffffffu, a[i] == -INFINITY);
            const float b[4] = {bf16lo(d[i].x), bf16hi(d[i].x), bf16lo(d[i].y), bf16hi(d[i].y)};
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // (an infinity with any sign of the other, any sign with its infinity)
              const uint32_t u = isinf(b[j]) ? up : up_inf, w = isinf(b[j]) ? down : down_inf;
              pos[j] |= b[j] > 0.0f ? u : b[j] < 0.0f ? w : 0u;
              neg[j] |= b[j] > 0.0f ? w : b[j] < 0.0f ? u : 0u;
            }
          }
        }
      }
    }
  }
  __syncwarp();  // the other lanes' stores of the tile
  if (!n_in || !(pos[0] | pos[1] | pos[2] | pos[3] | neg[0] | neg[1] | neg[2] | neg[3])) return;
  float* out = p.out + static_cast<int64_t>(tl.el) * p.K * p.N + n4;
  for (int l = 0; l < 32; ++l) {
    const int64_t row = row_of_lane(tl.k0, q4, l);
    if (row >= p.K) continue;
    float4* o = reinterpret_cast<float4*>(out + row * p.N);
    const auto add = [&](float x, int j) {  // (both signs: NaN)
      return x + (pos[j] >> l & 1 ? INFINITY : 0.0f) - (neg[j] >> l & 1 ? INFINITY : 0.0f);
    };
    const float4 x = *o;
    *o = make_float4(add(x.x, 0), add(x.y, 1), add(x.z, 2), add(x.w, 3));
  }
}

// Four 32-bit columns of this warp's lane quarter.
__device__ __forceinline__ void tmem_st_x4(uint32_t taddr, const uint4& v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w));
}

__global__ void __launch_bounds__(kThreads, 1)
    tgmm_mx_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* bp = smem_raw + (base - raw);
  const uint32_t sf_ring = base + kStages * kStageBytes;
  Ctl* ctl = reinterpret_cast<Ctl*>(bp + kStages * (kStageBytes + kSfBytes));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // a pair works on one sequence of tiles; its even CTA (rank 0) issues the MMAs
  // and owns the full and accumulator-empty barriers
  const int rank = static_cast<int>(__clusterRelativeBlockRank());
  const int t0 = static_cast<int>(__clusterIdx().x), step = static_cast<int>(__clusterGridDimInClusters().x);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&ctl->full[s]), 1 + 2 * 4);  // the producer's announcement, four scale warps a CTA
      mbar_init(smem_u32(&ctl->empty[s]), 1);
      mbar_init(smem_u32(&ctl->sfull[s]), 1);
    }
    mbar_init(smem_u32(&ctl->tfull), 1);
    mbar_init(smem_u32(&ctl->tempty), 2 * kEpiWarps);
    mbar_init(smem_u32(&ctl->drain), 1);
    mbar_init(smem_u32(&ctl->never), 1);
    ctl->abort_flag = 0;
    ctl->no_abort = 0;
    ctl->err = 0;
    fence_mbar_init();
  }
  // (both CTAs of a pair read the same group sizes, so they leave here together)
  if (!build_tables(p.group_sizes, p.E, p.g0, p.El, p.M, &ctl->t)) {
    grid_wait_previous();  // (this kernel never ends before the one it overlaps)
    if (threadIdx.x == 0) raise_error(&g_err, MOE_DEVERR_GROUP_SIZES);
    return;
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&ctl->tmem_base), 512);
    tmem_relinquish_pair();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  tc_fence_before();
  // the peer's barriers are initialised and its columns allocated before any
  // operand, commit or release crosses between the two CTAs
  cluster_sync_all();
  tc_fence_after();
  grid_wait_previous();  // the codes are complete (all but the group sizes, which round_rows_kernel did not write)
  const uint32_t tmem = ctl->tmem_base;
  if (rank == 1 && threadIdx.x == 0 &&
      ld_shared_cluster_u32(mapa_shared(smem_u32(&ctl->tmem_base), 0)) != tmem)
    raise_error(&g_err, MOE_DEVERR_TMEM);  // the pair's accumulators would not line up
  const int total = p.El * p.ktiles * p.ntiles;
  volatile int* abort_flag = &ctl->abort_flag;
  bool timed_out = false;

  if (warp < kCtrlWarps) {
    setmaxnreg_dec<kCtrlRegs>();
    if (warp == 0) {
      const bool leader = elect_one();
      uint32_t it = 0, s = 0, ph = 1;
      const uint32_t full0 = mapa_shared(smem_u32(&ctl->full[0]), 0), full_l = smem_u32(&ctl->full[0]), empty0 = smem_u32(&ctl->empty[0]), sfull0 = smem_u32(&ctl->sfull[0]);
      for (int t = t0; t < total && !timed_out; t += step) {
        const Tile tl = get_tile(p, ctl, t, rank);
        const int nkb = (tl.rows + kRB - 1) / kRB;
        const uint8_t* fa = p.sf_a + (static_cast<int64_t>(tl.kb0) * p.nrb_a + tl.k0 / 128) * kAtom;
        const uint8_t* fbp = p.sf_b + (static_cast<int64_t>(tl.kb0) * p.nrb_b + tl.n0 / 128) * kAtom;
        // lines of the tiles (past an operand's last block: the next row block's, never stored)
        int ya = (tl.kb0 * p.ncb_a + tl.k0 / 128) * 128, yb = (tl.kb0 * p.ncb_b + tl.n0 / 128 + rank) * 128;
        for (int kb = 0; kb < nkb; ++kb, ++it) {
          if (!wait_uniform(empty0 + 8 * s, ph, abort_flag)) {
            timed_out = true;
            break;
          }
          if (leader) {
            const uint32_t sa = base + s * kStageBytes, sf = sf_ring + s * kSfBytes, sb = sfull0 + 8 * s, fb = full0 + 8 * s;
            mbar_arrive_expect_tx(sb, kSfBytes);
            if (rank == 0) mbar_arrive_expect_tx(full_l + 8 * s, 2 * kStageBytes);
            bulk_load(sf, fa, kAtom, sb);
            bulk_load(sf + kAtom, fbp, 2 * kAtom, sb);
            tma_load_2d_pair(sa, &tmA, 0, ya, fb);
            tma_load_2d_pair(sa + kABytes, &tmB, 0, yb, fb);
          }
          fa += p.nrb_a * kAtom;
          fbp += p.nrb_b * kAtom;
          ya += p.ncb_a * 128;
          yb += p.ncb_b * 128;
          if (++s == kStages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      __syncwarp();
      if (lane == 0) {
        if (timed_out) {
          *abort_flag = 1;
          ctl->err = 2;
        }
        // The last loads land before the CTAs can exit, whichever role's wait ran out:
        // the scales of either CTA here; the codes are complete once the MMAs that
        // read them are, and otherwise (a wait ran out) within microseconds.
        for (uint32_t j = it > kStages ? it - kStages : 0; j < it; ++j)
          mbar_wait_bounded(smem_u32(&ctl->sfull[j % kStages]), (j / kStages) & 1, &ctl->no_abort, kWaitLimitNs);
        if (*abort_flag) mbar_wait_bounded(smem_u32(&ctl->never), 0, &ctl->no_abort, 1000000ull);
      }
      __syncwarp();
    } else if (warp == 1) {
      if (rank == 0) {
        const bool leader = elect_one();
        uint32_t acc = 0, s = 0, ph = 0;
        bool ready = false;  // the next stage is full: asked while a block's products are queued
        const uint32_t full0 = smem_u32(&ctl->full[0]), empty0 = smem_u32(&ctl->empty[0]);
        const uint64_t da0 = smem_desc_sw128(base), db0 = smem_desc_sw128(base + kABytes);
        for (int t = t0; t < total && !timed_out; t += step) {
          const Tile tl = get_tile(p, ctl, t, rank);
          const int nkb = (tl.rows + kRB - 1) / kRB;
          if (nkb == 0) continue;
          if (!wait_uniform(smem_u32(&ctl->tempty), (acc & 1) ^ 1, abort_flag)) {
            timed_out = true;
            break;
          }
          tc_fence_after();
          for (int kb = 0; kb < nkb; ++kb) {
            if (!ready && !wait_uniform(full0 + 8 * s, ph, abort_flag)) {
              timed_out = true;
              break;
            }
            tc_fence_after();
            const uint32_t sft = tmem + kSfCol0 + s * kSfCols;
            const uint64_t da = da0 + s * (kStageBytes >> 4), db = db0 + s * (kStageBytes >> 4);
            const int left = tl.rows - kb * kRB;  // rows of the block: an MMA for each 32
            if (leader) {
#pragma unroll
              for (int k4 = 0; k4 < 4; ++k4)
                if (k4 == 0 || left > 32 * k4)
                  mma_mx_pair(tmem, da + 2 * k4, db + 2 * k4, idesc_mx_e4m3(2 * kBM, kBN, k4, k4), sft, sft + 4,
                              kb > 0 || k4 > 0);
              mma_commit_pair_mc(empty0 + 8 * s, 0x3);
            }
            if (++s == kStages) {
              s = 0;
              ph ^= 1;
            }
            ready = __all_sync(0xffffffffu, mbar_test(full0 + 8 * s, ph));
          }
          if (timed_out) break;
          if (leader) mma_commit_pair_mc(smem_u32(&ctl->tfull), 0x3);
          ++acc;
        }
        __syncwarp();
        if (leader) {
        mma_commit_pair(smem_u32(&ctl->drain));
        if (!mbar_wait_bounded(smem_u32(&ctl->drain), 0, &ctl->no_abort, kWaitLimitNs)) timed_out = true;
        if (timed_out) {
          *abort_flag = 1;
          ctl->err = 2;
        }
        }
      }
      __syncwarp();
    } else if (warp >= kSfWarp) {
      // The stage was empty when the producer announced its scales, and so were their
      // columns: the same MMAs read both.
      const uint32_t tq = tmem + kSfCol0 + (static_cast<uint32_t>((warp & 3) * 32) << 16);
      uint32_t s = 0, ph = 0;
      const uint32_t sfull0 = smem_u32(&ctl->sfull[0]), full0 = mapa_shared(smem_u32(&ctl->full[0]), 0);
      for (int t = t0; t < total && !timed_out; t += step) {
        const Tile tl = get_tile(p, ctl, t, rank);
        const int nkb = (tl.rows + kRB - 1) / kRB;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!wait_uniform(sfull0 + 8 * s, ph, abort_flag)) {
            timed_out = true;
            break;
          }
          tc_fence_after();  // (behind the MMAs that read the columns: commit, empty, producer, sfull)
          const uint8_t* sf = bp + kStages * kStageBytes + s * kSfBytes + 16 * lane;
          tmem_st_x4(tq + s * kSfCols, *reinterpret_cast<const uint4*>(sf));
          tmem_st_x4(tq + s * kSfCols + 4, *reinterpret_cast<const uint4*>(sf + kAtom));
          tmem_st_x4(tq + s * kSfCols + 8, *reinterpret_cast<const uint4*>(sf + 2 * kAtom));
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          // (relaxed: it orders only tensor-memory stores that have completed)
          if (lane == 0) mbar_arrive_cluster_relaxed(full0 + 8 * s);
          if (++s == kStages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      if (timed_out) {
        *abort_flag = 1;
        ctl->err = 2;
      }
    }
  } else {
    setmaxnreg_inc<kEpiRegs>();
    const int q4 = warp & 3, half = (warp - kCtrlWarps) >> 2;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(q4 * 32) << 16) + half * (kBN / 2);
    const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
    uint32_t acc = 0;
    int inf = 0;
    for (int i = lane; i < p.round_ctas; i += 32) inf |= __ldcg(p.inf_seen + i);
    if (p.stall_ns && !mbar_wait_bounded_warp(smem_u32(&ctl->never), 0, abort_flag, p.stall_ns)) timed_out = true;
    for (int t = t0; t < total && !timed_out; t += step) {
      const Tile tl = get_tile(p, ctl, t, rank);
      uint32_t v[4][32];
      if (tl.rows > 0) {
        if (!__all_sync(0xffffffffu,
                        mbar_wait_bounded_idle(smem_u32(&ctl->tfull), acc & 1, abort_flag, kWaitLimitNs))) {
          timed_out = true;
          break;
        }
        ++acc;
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld_32x32b_x32(taddr + 32 * i, v[i]);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&ctl->tempty), 0));
      } else {  // an expert without rows: zeros
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int c = 0; c < 32; ++c) v[i][c] = 0;
      }
      // The accumulator's rows and columns are lines of the operands' tiles: column 16 c + b of
      // this warp's 128 is n = 8 b + c, lane l of the warp k = 64 (l / 8 % 2) + 8 (l % 8) +
      // l / 16 + 2 q4.  A lane has a row; after a transpose of 8-column pieces in each four lanes it
      // has columns 8 q.. (q = l % 4) of four rows 8 apart, so that a store instruction writes
      // 8 rows x 128 bytes and not 32 rows x 32 (370 -> 331 us on 128 small experts).
      const int k = tl.k0 + 64 * ((lane >> 3) & 1) + 8 * (lane & 4) + (lane >> 4) + 2 * q4;
      const int n = tl.n0 + half * (kBN / 2) + (lane & 3) * 8;
      const bool odd = lane & 1, high = lane & 2;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t y[4][8];  // pieces 4 i + j of the lane's row
#pragma unroll
        for (int c = 0; c < 8; ++c) {
#pragma unroll
          for (int j = 0; j < 4; ++j) y[j][c] = v[(16 * c + 4 * i + j) >> 5][(16 * c + 4 * i + j) & 31];
          const uint32_t s01 = __shfl_xor_sync(0xffffffffu, odd ? y[0][c] : y[1][c], 1);
          const uint32_t s23 = __shfl_xor_sync(0xffffffffu, odd ? y[2][c] : y[3][c], 1);
          if (odd) {
            y[0][c] = s01;
            y[2][c] = s23;
          } else {
            y[1][c] = s01;
            y[3][c] = s23;
          }
          const uint32_t s02 = __shfl_xor_sync(0xffffffffu, high ? y[0][c] : y[2][c], 2);
          const uint32_t s13 = __shfl_xor_sync(0xffffffffu, high ? y[1][c] : y[3][c], 2);
          if (high) {
            y[0][c] = s02;
            y[1][c] = s13;
          } else {
            y[2][c] = s02;
            y[3][c] = s13;
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (k + 8 * j < p.K && n + 32 * i < p.N)
            store8(p.out + (static_cast<int64_t>(tl.el) * p.K + k + 8 * j) * p.N + n + 32 * i, y[j], wide);
      }
    }
    if (__any_sync(0xffffffffu, inf) && !timed_out) {  // (after all tiles: no role waits for it)
      for (int t = t0; t < total; t += step) {
        const Tile tl = get_tile(p, ctl, t, rank);
        add_infinities(p, ctl, tl, q4, tl.n0 + half * (kBN / 2));
      }
    }
    if (timed_out) {
      *abort_flag = 1;
      ctl->err = 2;
    }
  }

  tc_fence_before();
  // neither CTA leaves (or frees its columns) while the other may still write its
  // tensor memory or arrive on its barriers
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
  if (threadIdx.x == 0 && ctl->err) raise_error(&g_err, MOE_DEVERR_TIMEOUT);
}

// ---- workspace -----------------------------------------------------------
// 128-row blocks that any M rows in El groups can take, then both operands' codes
// and scale atoms.
struct Layout {
  int64_t blocks;
  int ncb_a, ncb_b, nrb_a, nrb_b;
  int64_t q_a, q_b, sf_a, sf_b, inf, bytes;
};

bool make_layout(int64_t M, int64_t K, int64_t N, int El, Layout* l) {
  if (M < 0 || M >= (1ll << 31) - (1 << 18) || K <= 0 || K % 16 || K >= (1 << 30) || N <= 0 || N % 16 ||
      N >= (1 << 30) || El <= 0 || El > kMaxGroups)
    return false;
  l->blocks = M == 0 ? 0 : (M - 1) / kRB + El;  // sum of ceil(size / 128), at the most
  l->ncb_a = static_cast<int>((K + 127) / 128);
  l->ncb_b = static_cast<int>((N + 127) / 128);
  const int64_t most = 128ll * std::max(l->ncb_a, l->ncb_b);
  if (l->blocks > ((1ll << 31) - 1) / most - 2) return false;  // (a tile's lines are counted in 32 bits)
  l->nrb_a = static_cast<int>((K + 255) / 256) * 2;  // (a tile reads two of either)
  l->nrb_b = static_cast<int>((N + 255) / 256) * 2;
  l->q_a = 0;
  l->q_b = l->q_a + l->blocks * l->ncb_a * kTileBytes;
  l->sf_a = l->q_b + l->blocks * l->ncb_b * kTileBytes;
  l->sf_b = l->sf_a + l->blocks * l->nrb_a * kAtom;
  l->inf = l->sf_b + l->blocks * l->nrb_b * kAtom;
  l->bytes = l->inf + kRoundCtas * 4;
  return true;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" __attribute__((visibility("hidden"))) cudaError_t moe_detail_take_error_tgmm_mx(unsigned int* out) {
  unsigned int v = 0, z = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_err, sizeof(v));
  if (e == cudaSuccess && v) e = cudaMemcpyToSymbol(g_err, &z, sizeof(z));
  *out = v;
  return e;
}

extern "C" __attribute__((visibility("hidden"))) uint64_t moe_detail_stall_ns();

extern "C" size_t tgmm_fp8_mx_workspace_bytes(int64_t M, int64_t K, int64_t N, int E_local) {
  Layout l;
  return make_layout(M, K, N, E_local, &l) ? static_cast<size_t>(std::max<int64_t>(l.bytes, 16)) : 0;
}

extern "C" moe_status tgmm_fp8_mx(const uint16_t* lhs, int64_t lhs_rows, const int32_t* lhs_index, int k,
                                  const uint16_t* rhs, const int32_t* group_sizes, int E, int group_offset,
                                  int E_local, int64_t M, int64_t K, int64_t N, float* out, void* workspace,
                                  size_t workspace_bytes, moe_stream_t stream) {
  MOE_HOST_CHECK(lhs && rhs && group_sizes && out && workspace, MOE_ERR_INVALID_ARG);
  MOE_HOST_CHECK(E > 0 && E <= kMaxGroups && group_offset >= 0 && E_local > 0 && E_local <= E - group_offset,
                 MOE_ERR_INVALID_ARG);
  MOE_HOST_CHECK(k > 0 && lhs_rows >= 0 && (lhs_index || (k == 1 && lhs_rows == M)), MOE_ERR_INVALID_ARG);
  Layout l;
  MOE_HOST_CHECK(make_layout(M, K, N, E_local, &l), MOE_ERR_INVALID_ARG);
  MOE_HOST_CHECK(aligned16(lhs) && aligned16(rhs) && aligned16(out) && aligned16(workspace) &&
                     workspace_bytes >= static_cast<size_t>(l.bytes),
                 MOE_ERR_INVALID_ARG);
  const int64_t ktiles = (K + 2 * kBM - 1) / (2 * kBM), ntiles = (N + kBN - 1) / kBN, total = E_local * ktiles * ntiles;
  MOE_HOST_CHECK(total < (1ll << 31), MOE_ERR_INVALID_ARG);
  int sms = 0;
  const int dev = sm103_device(&sms);
  if (dev < 0) return MOE_ERR_UNSUPPORTED;
  cudaStream_t st = as_stream(stream);
  if (M == 0) {
    MOE_CUDA_TRY(cudaMemsetAsync(out, 0, static_cast<size_t>(E_local) * K * N * 4, st));
    return MOE_OK;
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  CUtensorMap A, B;
  constexpr auto plain = CU_TENSOR_MAP_SWIZZLE_NONE;  // (a tile is the swizzled image already)
  if (!make_map_u8(&A, ws + l.q_a, kRB, static_cast<uint64_t>(l.blocks) * l.ncb_a * 128, kRB, kBM, plain) ||
      !make_map_u8(&B, ws + l.q_b, kRB, static_cast<uint64_t>(l.blocks) * l.ncb_b * 128, kRB, kBN / 2, plain))
    return MOE_ERR_CUDA;
  const Operand oa{lhs, lhs_index, k, lhs_rows, static_cast<int>(K), l.ncb_a, l.nrb_a,
                   ws + l.q_a, ws + l.sf_a};
  const Operand ob{rhs, nullptr, 1, M, static_cast<int>(N), l.ncb_b, l.nrb_b,
                   ws + l.q_b, ws + l.sf_b};
  const int64_t rounds = l.blocks * (oa.ncb + ob.ncb);
  const int round_ctas = static_cast<int>(std::min<int64_t>(rounds, std::min(sms * 4, kRoundCtas)));
  int* inf_seen = reinterpret_cast<int*>(ws + l.inf);
  round_rows_kernel<<<static_cast<unsigned>(round_ctas), 256, 0, st>>>(oa, ob, group_sizes, E, group_offset, E_local, M,
                                                                       inf_seen);
  MOE_CUDA_TRY(cudaGetLastError());
  const Params p{group_sizes, E, group_offset, E_local, M, static_cast<int>(K), static_cast<int>(N),
                 static_cast<int>(ktiles), static_cast<int>(ntiles), l.ncb_a, l.ncb_b, l.nrb_a, l.nrb_b, ws + l.sf_a, ws + l.sf_b,
                 inf_seen, round_ctas, lhs, lhs_index, k, lhs_rows, rhs, out, moe_detail_stall_ns()};
  static SmemLimit limit;
  MOE_CUDA_TRY(limit.set(tgmm_mx_kernel, kSmem, dev));
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // pairs that are resident at once, per device (fewer than half of the SMs where a
  // cluster of SMs has an odd number: a pair more than that would run after all others)
  static std::atomic<int> resident[kMaxDevices];
  int pairs = resident[dev].load(std::memory_order_relaxed);
  if (pairs == 0) {
    cfg.gridDim = dim3(2 * (sms / 2));
    MOE_CUDA_TRY(cudaOccupancyMaxActiveClusters(&pairs, tgmm_mx_kernel, &cfg));
    if (pairs <= 0) return MOE_ERR_UNSUPPORTED;
    resident[dev].store(pairs, std::memory_order_relaxed);
  }
  cfg.gridDim = dim3(2 * static_cast<unsigned>(std::min<int64_t>(total, pairs)));
  cfg.numAttrs = 2;
  MOE_CUDA_TRY(cudaLaunchKernelEx(&cfg, tgmm_mx_kernel, A, B, p));
  return MOE_OK;
}
