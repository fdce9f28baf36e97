// Grouped MXFP4 matmul on the block-scaled 4-bit tensor-core MMA (sm_103a):
//   gmm_fp4_mx  out[m, n] = sum_k deq(lhs)[m, k] deq(rhs)[g(m), n, k]  (bf16 out)
// with both operands packed e2m1 codes and one E8M0 scale per 32 values of K
// (mx4.cuh).  tcgen05.mma.kind::mxf4 multiplies 64 values of K an instruction
// and applies both scales itself, so one fp32 accumulator runs over all of K.
//
// One persistent CTA per SM, 128 x 256 tiles:
//   warp 0      TMA producer: per stage 256 values of K (128 packed bytes a
//               row, 128-byte swizzle), 128 A rows and 256 B rows: 48 KB,
//               four stages; and B's scale words.
//   warp 1      MMA issuer: copies the stage's scale atoms into tensor memory
//               (tcgen05.cp), then four M = 128, N = 256, K = 64 MMAs.
//   warp 2      gatherer of A's scale words, by 4-byte cp.async, into a ring
//               of its own that runs further ahead than the stages.
//   warps 4..11 epilogue: accumulator -> bf16 in registers, accumulator
//               released, then row segments to memory.
// The tensor core takes the scales of 128 rows as an atom of 32 x 16 bytes, whose
// 16 bytes l are the words of rows l, 32 + l, 64 + l and 96 + l.  In memory the
// words of consecutive rows are adjacent.  B's rows can come in any order, since
// its rows are output columns: TMA brings channel 4 l + c of each 128 to row 32 c
// + l of the tile, so that B's scale words are an atom as they lie, one 512-byte
// bulk copy, and the epilogue undoes the order when it packs columns.  A's rows
// start anywhere (a group's first row), so its words are gathered.  (With all
// scale words gathered the stage's 24 copies an element of the warp held the MMAs
// up: 980 us at 16384 x 28672 x 4096 over 8 groups.)
// The 256-column accumulator and the scale slots share the 512 columns, so
// there is one accumulator; the epilogue hands it back as soon as its 128
// columns a warp sit packed in 64 registers, before any of them is stored.
//
// Tiles run expert-major, then N tile, then M tile: CTAs that run together
// share an expert's weights.  A group's M tiles start at its first row; rows
// past its end are computed and not stored.
//
// Measured: 16384 x 28672 x 4096 over 8 groups 841 us (4.6 PFLOP/s), 16384 x 1536
// x 2048 over 128 groups 51 us (5.5 TB/s), 32 of 64 groups of 12000 x 4096 x 7168
// 135 us (4.6 TB/s).  Of the large one's 1145 clocks a stage the six scale
// copies take some 215 (682 us without them).  What holds the other 930 is not
// known: four such MMAs take 512 at their nominal rate.  (Pairs of CTAs, each with
// half of B, read a third less through shared memory and L2: 657 us without the
// copies, 898 with them.)
//
// Every wait is bounded; on expiry
// the kernel raises MOE_DEVERR_TIMEOUT, lets what it issued finish and returns.
#include <cudaTypedefs.h>

#include <mutex>

#include "mx4.cuh"

namespace moe {
namespace {

__device__ unsigned int g_err;

constexpr int kBM = 128, kBN = 256;
constexpr int kStages = 4;
constexpr int kRowBytes = 128;       // a stage's bytes of one operand row: 256 values
constexpr int kABytes = kBM * kRowBytes, kBBytes = kBN * kRowBytes;
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kAtom = 512;           // scale words of 128 rows and 128 values of K: 32 rows of 16 bytes
constexpr int kSfBBytes = 4 * kAtom; // a stage's: two halves of B, each for two 128-wide K blocks
constexpr int kSfABytes = 2 * kAtom; // a slot of A's ring
constexpr int kSfSlots = 8;
constexpr int kSfCols = 24;          // tensor-memory columns of a stage's scales: 4 an atom
constexpr int kSfCol0 = kBN;
constexpr int kLag = 4;              // stages of A's scale copies in flight
constexpr int kCtrlWarps = 4, kEpiWarps = 8;
constexpr int kThreads = 32 * (kCtrlWarps + kEpiWarps);
constexpr int kMaxGroups = 1024;
constexpr int kStgPitch = 80, kStgBytes = 8 * kStgPitch;
static_assert(kSfCol0 + kStages * kSfCols <= 512, "tensor memory");
static_assert(kLag < kSfSlots, "the gatherer announces a slot before it needs the last one back");

struct Params {
  const int32_t* group_sizes;
  int E, g0, El;
  int64_t M;
  int N, nkb;  // nkb: 128-wide K blocks
  int ntiles;
  const uint32_t* lhs_sf;
  const uint32_t* rhs_sf;
  uint16_t* out;
  uint64_t stall_ns;  // test hook (moe_test_stall_consumers): 0, or the wait limit in ns
};

struct Ctl {
  uint64_t full[kStages], empty[kStages], sffull[kSfSlots], sfempty[kSfSlots];
  uint64_t tfull, tempty, drain;
  uint64_t never;  // test hook: a barrier that nothing arrives on
  uint32_t tmem_base;
  int abort_flag, no_abort, err, total;
  int start[kMaxGroups + 1], prefix[kMaxGroups + 1];  // local groups' first rows and tiles; the last: their ends
};
constexpr size_t kCtlBytes = (sizeof(Ctl) + 127) / 128 * 128;
constexpr size_t kSmem = 1024 + static_cast<size_t>(kStages) * (kStageBytes + kSfBBytes) + kSfSlots * kSfABytes + kCtlBytes +
                         static_cast<size_t>(kEpiWarps) * kStgBytes;
static_assert(kSmem <= 232448, "shared memory per CTA");

// kind::mxf4 instruction descriptor: A and B e2m1 (format 1), scale type
// E8M0; sf_id (0 or 2) selects the low or high two bytes of each scale cell:
// the scales of the first or second 64 values of a 128-wide K block.
__device__ __forceinline__ constexpr uint32_t idesc_mx4(int m, int n, int sf_id) {
  return (static_cast<uint32_t>(sf_id) << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
         (1u << 23) | (static_cast<uint32_t>(m >> 4) << 24) | (static_cast<uint32_t>(sf_id) << 29);
}

__device__ __forceinline__ void mma_mx4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// Local groups' first rows and first tiles, by warp 0 (any size
// negative or a sum other than M: err).
__device__ void build_tables(const Params& p, Ctl* c) {
  const int lane = threadIdx.x & 31;
  int64_t rows = 0;
  int tiles = 0;
  bool bad = false;
  for (int g0 = 0; g0 < p.E; g0 += 32) {
    const int g = g0 + lane, local = g - p.g0;
    const int sz = g < p.E ? __ldg(p.group_sizes + g) : 0;
    bad = bad || sz < 0;
    const bool mine = g < p.E && local >= 0 && local < p.El;
    int64_t ir = sz;
    const int nt = mine && sz > 0 ? (sz + kBM - 1) / kBM * p.ntiles : 0;
    int it = nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t r = __shfl_up_sync(0xffffffffu, ir, o);
      const int t = __shfl_up_sync(0xffffffffu, it, o);
      if (lane >= o) {
        ir += r;
        it += t;
      }
    }
    if (mine) {
      c->start[local] = static_cast<int>(rows + ir - sz);
      if (local == p.El - 1) c->start[p.El] = static_cast<int>(rows + ir);
      c->prefix[local] = tiles + it - nt;
    }
    rows += __shfl_sync(0xffffffffu, ir, 31);
    tiles += __shfl_sync(0xffffffffu, it, 31);
  }
  bad = __any_sync(0xffffffffu, bad);
  if (lane == 0) {
    c->prefix[p.El] = tiles;
    c->total = tiles;
    c->err = (bad || rows != p.M) ? 1 : 0;
  }
}

struct Tile {
  int el, row0, rows, n0;
};

__device__ __forceinline__ Tile get_tile(const Params& p, const Ctl* c, int t) {
  int lo = 0, hi = p.El;  // the last group whose first tile is <= t: it is not empty
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (c->prefix[mid] <= t) lo = mid; else hi = mid;
  }
  Tile tl;
  tl.el = lo;
  const int sz = c->start[lo + 1] - c->start[lo], mt = (sz + kBM - 1) / kBM, local = t - c->prefix[lo];
  const int nt = local / mt, mi = local - nt * mt;
  tl.row0 = c->start[lo] + mi * kBM;
  tl.rows = min(kBM, sz - mi * kBM);
  tl.n0 = nt * kBN;
  return tl;
}

__global__ void __launch_bounds__(kThreads, 1)
    gmm_mx4_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* bp = smem_raw + (base - raw);
  const uint32_t sfb_ring = base + kStages * kStageBytes, sfa_ring = sfb_ring + kStages * kSfBBytes;
  Ctl* ctl = reinterpret_cast<Ctl*>(bp + kStages * (kStageBytes + kSfBBytes) + kSfSlots * kSfABytes);
  uint8_t* stg_base = reinterpret_cast<uint8_t*>(ctl) + kCtlBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (warp == 0) build_tables(p, ctl);
  if (threadIdx.x == 32) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&ctl->full[s]), 1);
      mbar_init(smem_u32(&ctl->empty[s]), 1);
    }
    for (int q = 0; q < kSfSlots; ++q) {
      mbar_init(smem_u32(&ctl->sffull[q]), 32);
      mbar_init(smem_u32(&ctl->sfempty[q]), 1);
    }
    mbar_init(smem_u32(&ctl->tfull), 1);
    mbar_init(smem_u32(&ctl->tempty), kEpiWarps);
    mbar_init(smem_u32(&ctl->drain), 1);
    mbar_init(smem_u32(&ctl->never), 1);
    ctl->abort_flag = 0;
    ctl->no_abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  if (ctl->err) {
    if (threadIdx.x == 0) raise_error(&g_err, MOE_DEVERR_GROUP_SIZES);
    return;
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&ctl->tmem_base), 512);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  const int total = ctl->total, nstep = (p.nkb + 1) / 2;
  volatile int* abort_flag = &ctl->abort_flag;
  bool timed_out = false;

  if (warp == 0) {
    if (lane == 0) {
      uint32_t it = 0;
      const int64_t brows = static_cast<int64_t>(p.El) * p.N;
      for (int t = blockIdx.x; t < total && !timed_out; t += gridDim.x) {
        const Tile tl = get_tile(p, ctl, t);
        const int brow = tl.el * p.N + tl.n0;
        for (int kb = 0; kb < nstep; ++kb, ++it) {
          const int s = it % kStages;
          if (!mbar_wait_bounded(smem_u32(&ctl->empty[s]), ((it / kStages) & 1) ^ 1, abort_flag, kWaitLimitNs)) {
            timed_out = true;
            break;
          }
          const uint32_t fb = smem_u32(&ctl->full[s]), sa = base + s * kStageBytes;
          const int nh = min(2, p.nkb - 2 * kb);                // 128-wide K blocks of this stage
          const int words = min(kBN, p.N - tl.n0);              // channels of the tile (a multiple of 16)
          mbar_arrive_expect_tx(fb, kStageBytes + nh * words * 4);
          tma_load_2d(sa, &tmA, kb * kRowBytes, tl.row0, fb);
          tma_load_3d(sa + kABytes, &tmB, kb * kRowBytes, brow / 4, 0, fb);
          tma_load_3d(sa + kABytes + kBBytes / 2, &tmB, kb * kRowBytes, brow / 4 + 32, 0, fb);
          // channels past N keep what lay there: their columns are not stored
          for (int h = 0; h < nh; ++h)
            bulk_load(sfb_ring + s * kSfBBytes + 2 * kAtom * h, p.rhs_sf + (2 * kb + h) * brows + brow, words * 4, fb);
        }
      }
      if (timed_out) {
        *abort_flag = 1;
        ctl->err = 2;
      }
      // The last loads land before the CTA can exit, whichever role's wait ran out
      // (this one may have issued them all and be done).
      for (uint32_t j = it > kStages ? it - kStages : 0; j < it; ++j)
        mbar_wait_bounded(smem_u32(&ctl->full[j % kStages]), (j / kStages) & 1, &ctl->no_abort, kWaitLimitNs);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      uint32_t it = 0, acc = 0;
      for (int t = blockIdx.x; t < total && !timed_out; t += gridDim.x, ++acc) {
        if (!mbar_wait_bounded(smem_u32(&ctl->tempty), (acc & 1) ^ 1, abort_flag, kWaitLimitNs)) {
          timed_out = true;
          break;
        }
        tc_fence_after();
        for (int kb = 0; kb < nstep; ++kb, ++it) {
          const int s = it % kStages;
          const uint32_t ph = (it / kStages) & 1, q = it % kSfSlots;
          if (!mbar_wait_bounded(smem_u32(&ctl->full[s]), ph, abort_flag, kWaitLimitNs) ||
              !mbar_wait_bounded(smem_u32(&ctl->sffull[q]), (it / kSfSlots) & 1, abort_flag, kWaitLimitNs)) {
            timed_out = true;
            break;
          }
          tc_fence_after();
          const uint32_t sa = base + s * kStageBytes, sfa_sm = sfa_ring + q * kSfABytes, sfb_sm = sfb_ring + s * kSfBBytes;
          const uint32_t sft = tmem + kSfCol0 + s * kSfCols;  // per K block: A's 4 columns, then B's 8
          const uint64_t da = smem_desc_sw128(sa), db = smem_desc_sw128(sa + kABytes);
          const int nh = min(2, p.nkb - 2 * kb);  // 128-wide K blocks of this stage
          auto copy = [&](int h, int c) {  // atom c of K block h: A's, B's two
            tmem_cp_32x128b_warpx4(sft + 12 * h + 4 * c, smem_desc_plain(c == 0 ? sfa_sm + kAtom * h
                                                                                : sfb_sm + 2 * kAtom * h + kAtom * (c - 1)));
          };
          auto multiply = [&](int h, int half) {
            mma_mx4(tmem, da + 4 * h + 2 * half, db + 4 * h + 2 * half, idesc_mx4(kBM, kBN, 2 * half), sft + 12 * h,
                    sft + 12 * h + 4, kb > 0 || h > 0 || half > 0);
          };
          // The second block's copies between the first one's products: a product
          // that follows its copies directly waits for them (907 us with each
          // block's copies before its two products, 841 this way; all six first,
          // or the next stage's ahead of this one's products, are slower still)
          copy(0, 0);
          copy(0, 1);
          copy(0, 2);
          multiply(0, 0);
          if (nh > 1) {
            copy(1, 0);
            copy(1, 1);
          }
          multiply(0, 1);
          if (nh > 1) {
            copy(1, 2);
            multiply(1, 0);
            multiply(1, 1);
          }
          mma_commit(smem_u32(&ctl->empty[s]));
          mma_commit(smem_u32(&ctl->sfempty[q]));
        }
        if (timed_out) break;
        mma_commit(smem_u32(&ctl->tfull));
      }
      mma_commit(smem_u32(&ctl->drain));
      if (!mbar_wait_bounded(smem_u32(&ctl->drain), 0, &ctl->no_abort, kWaitLimitNs)) timed_out = true;
      if (timed_out) {
        *abort_flag = 1;
        ctl->err = 2;
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    // Lane l copies the words of tile rows 32 c + l: the words of a tile's rows
    // for one K block are adjacent, so an instruction reads one 128-byte line.  A
    // slot is announced kLag stages later, once its copies have landed and are
    // visible to the tensor core's (async-proxy) reads.
    uint32_t it = 0;
    for (int t = blockIdx.x; t < total && !timed_out; t += gridDim.x) {
      const Tile tl = get_tile(p, ctl, t);
      for (int kb = 0; kb < nstep; ++kb, ++it) {
        const int q = it % kSfSlots;
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(&ctl->sfempty[q]), ((it / kSfSlots) & 1) ^ 1, abort_flag,
                                                       kWaitLimitNs))) {
          timed_out = true;
          break;
        }
        const uint32_t dst = sfa_ring + q * kSfABytes + lane * 16;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int64_t k = 2 * kb + h;
#pragma unroll
          for (int c = 0; c < 4; ++c) {  // rows past M read as zeros
            const int64_t row = static_cast<int64_t>(tl.row0) + 32 * c + lane;
            const bool ok = k < p.nkb && row < p.M;
            cp_async_4(dst + kAtom * h + 4 * c, ok ? p.lhs_sf + k * p.M + row : p.lhs_sf, ok ? 4u : 0u);
          }
        }
        cp_async_commit();
        if (it >= kLag) {
          cp_async_wait<kLag>();
          fence_proxy_async_smem();
          mbar_arrive(smem_u32(&ctl->sffull[(it - kLag) % kSfSlots]));
        }
      }
    }
    cp_async_wait<0>();
    fence_proxy_async_smem();
    for (uint32_t j = it > kLag ? it - kLag : 0; j < it; ++j) mbar_arrive(smem_u32(&ctl->sffull[j % kSfSlots]));
    if (timed_out) {
      *abort_flag = 1;
      ctl->err = 2;
    }
  } else if (warp >= kCtrlWarps) {
    const int q4 = warp & 3, half = (warp - kCtrlWarps) >> 2;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(q4 * 32) << 16) + half * (kBN / 2);
    uint8_t* stg = stg_base + (warp - kCtrlWarps) * kStgBytes;
    uint32_t acc = 0;
    if (p.stall_ns && !mbar_wait_bounded_warp(smem_u32(&ctl->never), 0, abort_flag, p.stall_ns)) timed_out = true;
    for (int t = blockIdx.x; t < total && !timed_out; t += gridDim.x, ++acc) {
      const Tile tl = get_tile(p, ctl, t);
      if (!mbar_wait_bounded_warp(smem_u32(&ctl->tfull), acc & 1, abort_flag, kWaitLimitNs)) {
        timed_out = true;
        break;
      }
      tc_fence_after();
      // column 32 c + l of the warp's 128 holds channel 4 l + c
      uint32_t w[4][16];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t u[32], v[32];
        tmem_ld_32x32b_x32(taddr + 64 * i, u);
        tmem_ld_32x32b_x32(taddr + 64 * i + 32, v);
        tmem_wait_ld();
#pragma unroll
        for (int l = 0; l < 32; ++l)
          w[l / 8][2 * (l % 8) + i] = pack_bf16x2(__uint_as_float(u[l]), __uint_as_float(v[l]));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&ctl->tempty));
      const int nrows = tl.rows - q4 * 32;
      const int64_t row = static_cast<int64_t>(tl.row0) + q4 * 32;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = tl.n0 + half * (kBN / 2) + 32 * i;
        // 8 rows at a time through a small staging buffer, so that a store
        // instruction writes 64 contiguous bytes of each of 8 rows
        uint8_t* out = reinterpret_cast<uint8_t*>(p.out + row * p.N + n);
        const int rr = lane >> 2, q = lane & 3;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          if ((lane >> 3) == s) {
            uint4* d = reinterpret_cast<uint4*>(stg + (lane & 7) * kStgPitch);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              d[j] = make_uint4(w[i][4 * j], w[i][4 * j + 1], w[i][4 * j + 2], w[i][4 * j + 3]);
          }
          __syncwarp();
          const int r = 8 * s + rr;
          if (r < nrows && n + 8 * q < p.N)
            *reinterpret_cast<uint4*>(out + static_cast<int64_t>(r) * p.N * 2 + 16 * q) =
                *reinterpret_cast<const uint4*>(stg + rr * kStgPitch + 16 * q);
          __syncwarp();
        }
      }
    }
    if (timed_out) {
      *abort_flag = 1;
      ctl->err = 2;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && ctl->err) raise_error(&g_err, MOE_DEVERR_TIMEOUT);
}

// Rows of out before the first and after the last local group: zeros.
__global__ void __launch_bounds__(256) zero_rows_kernel(uint16_t* out, int64_t M, int64_t N, const int32_t* sizes,
                                                        int E, int g0, int El) {
  __shared__ int64_t bound[2];
  if (threadIdx.x < 32) {
    int64_t lo = 0, hi = 0;
    for (int g = threadIdx.x; g < E; g += 32) {
      const int64_t sz = __ldg(sizes + g);
      lo += g < g0 ? sz : 0;
      hi += g < g0 + El ? sz : 0;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      lo += __shfl_xor_sync(0xffffffffu, lo, o);
      hi += __shfl_xor_sync(0xffffffffu, hi, o);
    }
    if (threadIdx.x == 0) {
      bound[0] = min(max(lo, static_cast<int64_t>(0)), M);
      bound[1] = min(max(hi, bound[0]), M);
    }
  }
  __syncthreads();
  const int64_t n16 = N / 8, head = bound[0] * n16, gap = (bound[1] - bound[0]) * n16;
  const int64_t all = M * n16 - gap, step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  uint4* o = reinterpret_cast<uint4*>(out);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < all; i += step)
    o[i < head ? i : i + gap] = make_uint4(0, 0, 0, 0);
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

// Packed codes as bytes, 128-byte swizzle; reads past the extents return
// zeros.  A: boxes of 128 rows x 128 bytes.  B: row 4 l + c of the matrix is
// (l, c), and a box of 32 l x 4 c puts it at row 32 c + l of the tile.
bool make_map(CUtensorMap* m, const void* ptr, uint64_t bytes, uint64_t rows, bool b) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {bytes, b ? rows / 4 : rows, 4}, strides[2] = {b ? 4 * bytes : bytes, bytes};
  cuuint32_t box[3] = {kRowBytes, b ? 32u : static_cast<cuuint32_t>(kBM), 4}, estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, b ? 3 : 2, const_cast<void*>(ptr), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" __attribute__((visibility("hidden"))) cudaError_t moe_detail_take_error_gmm_mx4(unsigned int* out) {
  unsigned int v = 0, z = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_err, sizeof(v));
  if (e == cudaSuccess && v) e = cudaMemcpyToSymbol(g_err, &z, sizeof(z));
  *out = v;
  return e;
}

extern "C" __attribute__((visibility("hidden"))) uint64_t moe_detail_stall_ns();

extern "C" moe_status gmm_fp4_mx(const uint8_t* lhs_q, const uint8_t* lhs_sf, const uint8_t* rhs_q,
                                 const uint8_t* rhs_sf, const int32_t* group_sizes, int E, int group_offset,
                                 int E_local, int64_t M, int64_t K, int64_t N, uint16_t* out, moe_stream_t stream) {
  MOE_HOST_CHECK(lhs_q && lhs_sf && rhs_q && rhs_sf && group_sizes && out, MOE_ERR_INVALID_ARG);
  MOE_HOST_CHECK(E > 0 && E <= kMaxGroups && group_offset >= 0 && E_local > 0 && E_local <= E - group_offset,
                 MOE_ERR_INVALID_ARG);
  MOE_HOST_CHECK(M >= 0 && M < (1ll << 31) - kBM && K > 0 && K % 128 == 0 && K < (1 << 30) && N > 0 && N % 16 == 0 &&
                     N <= ((1ll << 31) - kBN) / E_local,
                 MOE_ERR_INVALID_ARG);
  MOE_HOST_CHECK(aligned16(lhs_q) && aligned16(rhs_q) && aligned16(out) &&
                     (reinterpret_cast<uintptr_t>(lhs_sf) & 3) == 0 && aligned16(rhs_sf),
                 MOE_ERR_INVALID_ARG);
  const int64_t ntiles = (N + kBN - 1) / kBN;
  const int64_t units = ((M + kBM - 1) / kBM + E_local) * ntiles;
  MOE_HOST_CHECK(units < (1ll << 31), MOE_ERR_INVALID_ARG);
  int dev = 0, major = 0, minor = 0, sms = 0;
  MOE_CUDA_TRY(cudaGetDevice(&dev));
  MOE_CUDA_TRY(cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev));
  MOE_CUDA_TRY(cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev));
  MOE_CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  if (major != 10 || minor != 3) return MOE_ERR_UNSUPPORTED;
  if (M == 0) return MOE_OK;
  cudaStream_t st = as_stream(stream);
  if (E_local < E) {
    zero_rows_kernel<<<sms * 4, 256, 0, st>>>(out, M, N, group_sizes, E, group_offset, E_local);
    MOE_CUDA_TRY(cudaGetLastError());
  }
  CUtensorMap A, B;
  if (!make_map(&A, lhs_q, K / 2, M, false)) return MOE_ERR_CUDA;
  if (!make_map(&B, rhs_q, K / 2, static_cast<uint64_t>(E_local) * N, true)) return MOE_ERR_CUDA;
  Params p{group_sizes, E, group_offset, E_local, M, static_cast<int>(N), static_cast<int>(K / 128),
           static_cast<int>(ntiles), reinterpret_cast<const uint32_t*>(lhs_sf),
           reinterpret_cast<const uint32_t*>(rhs_sf), out, moe_detail_stall_ns()};
  MOE_CUDA_TRY(cudaFuncSetAttribute(gmm_mx4_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(kSmem)));
  gmm_mx4_kernel<<<static_cast<unsigned>(units < sms ? units : sms), kThreads, kSmem, st>>>(A, B, p);
  MOE_CUDA_TRY(cudaGetLastError());
  return MOE_OK;
}
