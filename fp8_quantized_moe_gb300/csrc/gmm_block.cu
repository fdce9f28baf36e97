// Grouped matmul of e4m3 operands with a scale for each block of 128 (sm_103a):
//   gmm_fp8_block  out[m, n] = bf16( sum_kb sa[m, kb] sb[g(m), n / 128, kb] *
//                                    sum_{k in block kb} a[m, k] w[g(m), n, k] )
// sa: one fp32 scale per row and 128 values of K; sb: one per 128 x 128 block
// of an expert's weights.  The input gradient is the same product on the
// transposed weights (codes and block scales transposed: nothing is rounded again).
//
// Mathematics.  The scale of a K block cannot leave the sum over blocks, so each
// 128-wide block is one tensor-core accumulation that starts fresh, P, and the
// epilogue warps keep the running sum in fp32 registers: acc += s P.  With the
// weights' scale constant over 128 channels, s = sa sb is one number for a thread
// (its row, its warp's 128 channels): one fused multiply-add an element and block,
// and no scale is read per element.
//
// Layout of a CTA (12 warps, one CTA per SM, 128 x 256 tiles):
//   warp 0      TMA producer: 128 A rows and 256 B rows of 128 bytes per stage, 48 KB,
//               four stages, 128-byte swizzle.
//   warp 1      MMA issuer: four M = 128, N = 256, K = 32 tcgen05.mma.kind::f8f6f4 a block.
//   warps 2, 3  zeros for the rows of no local group.
//   warps 4..11 epilogue: warp w has tensor-memory lanes 32 (w % 4).. (rows) and
//               128 of the tile's columns: 128 running sums a thread.
// The producing and issuing warps run with all lanes (wait_uniform).  Two 256-column accumulators take alternate K blocks.
//
// Tiles run expert-major, then N tile, then M tile: CTAs that run together share
// an expert's weights.  A group's M tiles start at its first row; rows past its end
// are computed and not stored.
//
// Few tiles (SPLIT): a cluster of 2, 4 or 8 CTAs
// shares a tile, each with a part of the K blocks; the partial tiles meet in shared
// memory (the stages', which are done with) and every CTA adds up and stores a slice of
// the columns, in the order of the CTAs.
//
// Bound and measurements.  A block's four MMAs take 523 clocks with their operands in place,
// whatever their N (520 to 525 for N = 32, 64, 96, 128, 192 and 256).  On 16384 x 4096 x 28672
// over 8 groups, some 3136 blocks an SM, in bursts (1.94 GHz): 1.38 ms, 854 clocks a block; the
// same loop without any fold 798 clocks (1.29 ms, both accumulators handed back and forth),
// without fold and MMAs 637 (1.03 ms: loads, 77 bytes a clock and SM), the hand-over alone 501
// (0.81 ms).  So loads, MMAs and hand-over are each well below the whole and overlap only in part;
// no unit is at its limit (8192 x 4096 x 7168, one group: tensor pipe 61 % busy, L1 and shared
// memory 51, L2 41, DRAM 23).  Back to back the power limit lowers the clock: 1.53 to 1.67 ms,
// 2.3 to 2.5 PFLOP/s; the plain product of gmm_fp8 (one accumulator a tile, no fold) 1.40.
// 64 of 96 groups of 49152 x 4096 x 7168: 939 to 969 us (a last tile of some 60 of 128 rows
// in each group of 512); 16384 x 1536 x 2048 over 128 groups: 90 us, its bytes 72.
// On the way there (burst or back to back alike):
//   - tensor-memory loads of 16 columns, two at a time, against 32 columns: 2.4 against
//     1.7 PFLOP/s (32 registers in a row cost moves and spills);
//   - the epilogue's waits sleeping in the barrier (a suspend-time hint) against polling:
//     5 %; polling without pause made even the loop without a fold 20 % slower: the
//     polls take shared memory's time from the MMA's operands;
//   - scales two blocks ahead against one, and the issuing warp's early look at the next
//     stage: 6 and 3 %;
//   - pairs of CTAs on 256 x 256 tiles (half of B each; these issuing loops and 16-column loads,
//     scales one block ahead): 3 % slower on the large groups and on 64 of 96, 22 % on 128
//     small ones (256-row tiles leave more rows empty);
//   - four accumulators of 128 columns: 25 % slower (twice as many MMAs, each as long);
//   - 16 epilogue warps of 64 columns: 10 % slower; the next block's first columns loaded
//     before a block's last sums: 12 %.
//
// Every wait is bounded; on expiry the kernel raises MOE_DEVERR_TIMEOUT, lets what
// it issued finish and returns.
#include "grouped.cuh"

namespace moe {
namespace {

__device__ unsigned int g_err;

constexpr int kBM = 128, kBN = 256, kBK = 128;
constexpr int kStages = 4;
constexpr int kABytes = kBM * kBK, kBBytes = kBN * kBK;
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kCtrlWarps = 4, kEpiWarps = 8;
constexpr int kThreads = 32 * (kCtrlWarps + kEpiWarps);
// registers a thread: 168 at launch (a 384-thread CTA alone on its SM), handed from the
// control warpgroup to the epilogue
constexpr uint32_t kCtrlRegs = 40, kEpiRegs = 232;
static_assert(128 * kCtrlRegs + 256 * kEpiRegs <= 168 * kThreads, "register split");

struct Params {
  const int32_t* group_sizes;  // or null: one group of all M rows
  int E, g0, El;
  int64_t M;
  int N, nkb, ntiles, nblk;  // nkb: K blocks; ntiles: 256-column tiles; nblk: 128-channel blocks
  const float* lhs_s;
  const float* rhs_s;
  uint16_t* out;
  uint64_t stall_ns;  // test hook (moe_test_stall_consumers): 0, or the wait limit in ns
};

struct Ctl {
  uint64_t full[kStages], empty[kStages];
  uint64_t tfull[2], tempty[2], drain;
  uint64_t pfull;  // SPLIT: every CTA's partial tile is in its shared memory
  uint64_t never;  // test hook: a barrier that nothing arrives on
  uint32_t tmem_base;
  int abort_flag, no_abort, err, total;
  int start[kMaxGroups + 1], prefix[kMaxGroups + 1];  // local groups' first rows and tiles; the last: their ends
};
constexpr size_t kCtlBytes = (sizeof(Ctl) + 127) / 128 * 128;
constexpr size_t kSmem = 1024 + static_cast<size_t>(kStages) * kStageBytes + kCtlBytes;
static_assert(kSmem <= 232448, "shared memory per CTA");
static_assert(kStages * kStageBytes >= kBM * kBN * 4, "SPLIT: a partial tile in the stages");

// Local groups' first rows and first tiles, by warp 0 (any size
// negative or a sum other than M: err).
__device__ void build_tables(const Params& p, Ctl* c) {
  const int lane = threadIdx.x & 31;
  int64_t rows = 0;
  int units = 0;
  bool bad = false;
  for (int g0 = 0; g0 < p.E; g0 += 32) {
    const int g = g0 + lane, local = g - p.g0;
    const int sz = g < p.E ? (p.group_sizes ? __ldg(p.group_sizes + g) : static_cast<int>(p.M)) : 0;
    bad = bad || sz < 0;
    const bool mine = g < p.E && local >= 0 && local < p.El;
    int64_t ir = sz;
    const int nu = mine && sz > 0 ? (sz + kBM - 1) / kBM * p.ntiles : 0;
    int iu = nu;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t r = __shfl_up_sync(0xffffffffu, ir, o);
      const int t = __shfl_up_sync(0xffffffffu, iu, o);
      if (lane >= o) {
        ir += r;
        iu += t;
      }
    }
    if (mine) {
      c->start[local] = static_cast<int>(rows + ir - sz);
      if (local == p.El - 1) c->start[p.El] = static_cast<int>(rows + ir);
      c->prefix[local] = units + iu - nu;
    }
    rows += __shfl_sync(0xffffffffu, ir, 31);
    units += __shfl_sync(0xffffffffu, iu, 31);
  }
  bad = __any_sync(0xffffffffu, bad);
  if (lane == 0) {
    c->prefix[p.El] = units;
    c->total = units;
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

// The epilogue's wait: one outcome for the whole warp, asleep in the barrier.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, const volatile int* abort_flag) {
  return __all_sync(0xffffffffu, mbar_wait_bounded_idle(bar, parity, abort_flag, kWaitLimitNs));
}

// The same for writes of other CTAs of the cluster (acquire at cluster scope).
__device__ __forceinline__ bool wait_warp_cluster(uint32_t bar, uint32_t parity, const volatile int* abort_flag) {
  auto attempt = [&] {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
  };
  bool ok = attempt();
  const uint64_t t0 = globaltimer_ns();
  while (!ok && !*abort_flag && globaltimer_ns() - t0 <= kWaitLimitNs) ok = attempt();
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// 16-byte unit u (columns 4 u..) of row r of a partial tile: units swizzled by row, so that
// eight rows' (a thread's each) stores meet no bank twice.
__device__ __forceinline__ uint32_t part_offset(int r, int u) {
  return static_cast<uint32_t>(r * (kBN * 4) + ((u ^ (r & 7)) << 4));
}

// Rows of no local group, zeroed by two warps of every CTA.
__device__ void zero_outside(const Params& p, const Ctl* c, int cta, int ctas) {
  const int64_t n16 = p.N / 8, head = c->start[0] * n16, gap = (c->start[p.El] - c->start[0]) * n16;
  const int64_t all = p.M * n16 - gap, step = 64ll * ctas;
  uint4* o = reinterpret_cast<uint4*>(p.out);
  for (int64_t i = 64ll * cta + (threadIdx.x & 63); i < all; i += step) o[i < head ? i : i + gap] = make_uint4(0, 0, 0, 0);
}

template <bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    gmm_block_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  uint8_t* bp = smem_raw + (base - raw);
  Ctl* ctl = reinterpret_cast<Ctl*>(bp + kStages * kStageBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // SPLIT: a cluster has one tile, this CTA the K blocks [kb_lo, kb_hi) of it
  const int rank = SPLIT ? static_cast<int>(__clusterRelativeBlockRank()) : 0;
  const int parts = SPLIT ? static_cast<int>(__clusterSizeInBlocks()) : 1;
  const int t0 = SPLIT ? static_cast<int>(__clusterIdx().x) : static_cast<int>(blockIdx.x);
  const int step = SPLIT ? (1 << 30) : static_cast<int>(gridDim.x);
  const int kb_lo = SPLIT ? rank * p.nkb / parts : 0, kb_hi = SPLIT ? (rank + 1) * p.nkb / parts : p.nkb;

  if (warp == 0) build_tables(p, ctl);
  if (threadIdx.x == 32) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&ctl->full[s]), 1);
      mbar_init(smem_u32(&ctl->empty[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&ctl->tfull[a]), 1);
      mbar_init(smem_u32(&ctl->tempty[a]), kEpiWarps);
    }
    mbar_init(smem_u32(&ctl->pfull), static_cast<uint32_t>(parts * kEpiWarps));
    mbar_init(smem_u32(&ctl->drain), 1);
    mbar_init(smem_u32(&ctl->never), 1);
    ctl->abort_flag = 0;
    ctl->no_abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  // the CTAs of a cluster read the same group sizes, so they leave here together
  if (ctl->err) {
    if (threadIdx.x == 0) raise_error(&g_err, MOE_DEVERR_GROUP_SIZES);
    return;
  }
  const bool zeroes = p.El < p.E && (warp == 2 || warp == 3);
  if (SPLIT) {
    if (zeroes) zero_outside(p, ctl, blockIdx.x, gridDim.x);
    if (t0 >= ctl->total) return;  // (and here)
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
  if (SPLIT) cluster_sync_all(); else __syncthreads();  // (a peer's pfull is initialised before it is arrived on)
  tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  const int total = ctl->total;
  volatile int* abort_flag = &ctl->abort_flag;
  bool timed_out = false;

  if (warp < kCtrlWarps) {
    setmaxnreg_dec<kCtrlRegs>();
    if (warp == 0) {
      const bool leader = elect_one();
      const uint32_t full0 = smem_u32(&ctl->full[0]), empty0 = smem_u32(&ctl->empty[0]);
      uint32_t it = 0, s = 0, ph = 1;
      for (int t = t0; t < total && !timed_out; t += step) {
        const Tile tl = get_tile(p, ctl, t);
        const int brow = tl.el * p.N + tl.n0;
        for (int kb = kb_lo; kb < kb_hi; ++kb, ++it) {
          if (!wait_uniform(empty0 + 8 * s, ph, abort_flag)) {
            timed_out = true;
            break;
          }
          if (leader) {
            const uint32_t sa = base + s * kStageBytes, fb = full0 + 8 * s;
            mbar_arrive_expect_tx(fb, kStageBytes);
            tma_load_2d(sa, &tmA, kb * kBK, tl.row0, fb);
            tma_load_2d(sa + kABytes, &tmB, kb * kBK, brow, fb);
          }
          if (++s == kStages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      __syncwarp();
      if (timed_out && lane == 0) {
        *abort_flag = 1;
        ctl->err = 2;
      }
      // the last loads land before the CTA can exit, whichever role's wait ran out
      if (lane == 0)
        for (uint32_t j = it > kStages ? it - kStages : 0; j < it; ++j)
          mbar_wait_bounded(full0 + 8 * (j % kStages), (j / kStages) & 1, &ctl->no_abort, kWaitLimitNs);
      __syncwarp();
    } else if (warp == 1) {
      const bool leader = elect_one();
      const uint32_t full0 = smem_u32(&ctl->full[0]), empty0 = smem_u32(&ctl->empty[0]);
      const uint32_t tfull0 = smem_u32(&ctl->tfull[0]), tempty0 = smem_u32(&ctl->tempty[0]);
      const uint64_t da0 = smem_desc_sw128(base), db0 = smem_desc_sw128(base + kABytes);
      uint32_t s = 0, ph = 0, a = 0, aph = 1;
      bool ready = false;  // the next stage is full: asked while a block's products are queued (1.59 -> 1.54 ms)
      for (int t = t0; t < total && !timed_out; t += step) {
        for (int kb = kb_lo; kb < kb_hi; ++kb) {
          if ((!ready && !wait_uniform(full0 + 8 * s, ph, abort_flag)) ||
              !wait_uniform(tempty0 + 8 * a, aph, abort_flag)) {
            timed_out = true;
            break;
          }
          tc_fence_after();
          const uint64_t da = da0 + s * (kStageBytes >> 4), db = db0 + s * (kStageBytes >> 4);
          if (leader) {
#pragma unroll
            for (int k4 = 0; k4 < 4; ++k4)  // 32 bytes of K: 2 in the descriptors' 16-byte units
              mma_f8(tmem + a * kBN, da + 2 * k4, db + 2 * k4, idesc_e4m3_f32(kBM, kBN), k4 > 0);
            mma_commit(empty0 + 8 * s);
            mma_commit(tfull0 + 8 * a);
          }
          if (++s == kStages) {
            s = 0;
            ph ^= 1;
          }
          ready = __all_sync(0xffffffffu, mbar_test(full0 + 8 * s, ph));
          a ^= 1;
          aph ^= a == 0;
        }
      }
      __syncwarp();
      if (leader) {
        mma_commit(smem_u32(&ctl->drain));
        if (!mbar_wait_bounded(smem_u32(&ctl->drain), 0, &ctl->no_abort, kWaitLimitNs)) timed_out = true;
        if (timed_out) {
          *abort_flag = 1;
          ctl->err = 2;
        }
      }
      __syncwarp();
    } else if (!SPLIT && zeroes) {
      zero_outside(p, ctl, blockIdx.x, gridDim.x);
    }
  } else {
    setmaxnreg_inc<kEpiRegs>();
    const int q4 = warp & 3, half = (warp - kCtrlWarps) >> 2, r = q4 * 32 + lane;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(q4 * 32) << 16) + half * (kBN / 2);
    const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
    uint32_t it = 0;
    if (p.stall_ns && !mbar_wait_bounded_warp(smem_u32(&ctl->never), 0, abort_flag, p.stall_ns)) timed_out = true;
    for (int t = t0; t < total && !timed_out; t += step) {
      const Tile tl = get_tile(p, ctl, t);
      // (a row past the group's end takes its last one's scales, channels past N the last block's)
      const float* sa = p.lhs_s + static_cast<int64_t>(tl.row0 + min(r, tl.rows - 1)) * p.nkb;
      const float* sb = p.rhs_s + (static_cast<int64_t>(tl.el) * p.nblk + min(tl.n0 / kBK + half, p.nblk - 1)) * p.nkb;
      uint64_t acc[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) acc[j] = 0;
      // a block's scales are asked for two blocks ahead (one ahead: 1.69 instead of 1.59 ms on
      // the large groups)
      float next = __fmul_rn(__ldg(sa + kb_lo), __ldg(sb + kb_lo)), na = 0.f, nw = 0.f;
      if (kb_lo + 1 < kb_hi) {
        na = __ldg(sa + kb_lo + 1);
        nw = __ldg(sb + kb_lo + 1);
      }
#pragma unroll 1
      for (int kb = kb_lo; kb < kb_hi; ++kb) {
        const uint64_t s2 = f2_pack(next, next);
        const float ma = na, mw = nw;
        if (kb + 2 < kb_hi) {
          na = __ldg(sa + kb + 2);
          nw = __ldg(sb + kb + 2);
        }
        next = __fmul_rn(ma, mw);
        const uint32_t a = it & 1;
        if (!wait_warp(smem_u32(&ctl->tfull[a]), (it >> 1) & 1, abort_flag)) {
          timed_out = true;
          break;
        }
        ++it;
        tc_fence_after();
        const uint32_t ta = taddr + a * kBN;
        // two loads of 16 columns in flight while two are added up; the accumulator
        // goes back before the last two are
        uint64_t u[4][8];
        tmem_ld_32x32b_x16_pairs(ta, u[0]);
        tmem_ld_32x32b_x16_pairs(ta + 16, u[1]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int x = 2 * (c & 1), y = 2 - x;
          if (c < 3) {
            tmem_ld_32x32b_x16_pairs(ta + 32 * (c + 1), u[y]);
            tmem_ld_32x32b_x16_pairs(ta + 32 * (c + 1) + 16, u[y + 1]);
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&ctl->tempty[a]));
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[16 * c + i] = f2_fma(u[x][i], s2, acc[16 * c + i]);
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[16 * c + 8 + i] = f2_fma(u[x + 1][i], s2, acc[16 * c + 8 + i]);
          if (c < 3) tmem_wait_ld();
        }
      }
      if (timed_out) break;
      if (SPLIT) {
        // Partial tiles into the stages (every load has landed and every MMA read them:
        // the last accumulator was full), then slices of columns from all of them.
        if (r < tl.rows) {
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            float x, y, z, w;
            f2_unpack(acc[2 * j], x, y);
            f2_unpack(acc[2 * j + 1], z, w);
            *reinterpret_cast<float4*>(bp + part_offset(r, 32 * half + j)) = make_float4(x, y, z, w);
          }
        }
        __syncwarp();
        if (lane < parts) mbar_arrive_cluster(mapa_shared(smem_u32(&ctl->pfull), lane));
        if (!wait_warp_cluster(smem_u32(&ctl->pfull), 0, abort_flag)) {
          timed_out = true;
          break;
        }
        const int cols = kBN / parts, per = cols / 8;  // 8 columns: 16 bytes of bf16
        for (int i = threadIdx.x - 32 * kCtrlWarps; i < tl.rows * per; i += 32 * kEpiWarps) {
          const int row = i / per, c = rank * cols + 8 * (i - row * per);
          if (tl.n0 + c >= p.N) continue;
          float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
          for (int q0 = 0; q0 < parts; q0 += 4) {  // four CTAs' loads in flight, added in order
            float4 lo[4], hi[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (q0 + q < parts) {
                lo[q] = ld_cluster_f4(mapa_shared(base + part_offset(row, c / 4), q0 + q));
                hi[q] = ld_cluster_f4(mapa_shared(base + part_offset(row, c / 4 + 1), q0 + q));
              }
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (q0 + q < parts) {
                v[0] += lo[q].x;
                v[1] += lo[q].y;
                v[2] += lo[q].z;
                v[3] += lo[q].w;
                v[4] += hi[q].x;
                v[5] += hi[q].y;
                v[6] += hi[q].z;
                v[7] += hi[q].w;
              }
          }
          *reinterpret_cast<uint4*>(p.out + static_cast<int64_t>(tl.row0 + row) * p.N + tl.n0 + c) =
              make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                         pack_bf16x2(v[6], v[7]));
        }
      } else if (r < tl.rows) {
        uint16_t* o = p.out + static_cast<int64_t>(tl.row0 + r) * p.N + tl.n0 + half * (kBN / 2);
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // 16 columns: one 32-byte sector of the row
          if (tl.n0 + half * (kBN / 2) + 16 * i >= p.N) break;
          uint32_t w[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float x, y;
            f2_unpack(acc[8 * i + j], x, y);
            w[j] = pack_bf16x2(x, y);
          }
          if (wide) {
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(o + 16 * i), "r"(w[0]),
                         "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                         : "memory");
          } else {
            *reinterpret_cast<uint4*>(o + 16 * i) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4*>(o + 16 * i + 8) = make_uint4(w[4], w[5], w[6], w[7]);
          }
        }
      }
    }
    if (timed_out) {
      *abort_flag = 1;
      ctl->err = 2;
    }
  }

  tc_fence_before();
  if (SPLIT) cluster_sync_all(); else __syncthreads();  // (no CTA leaves while a peer reads its part)
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0 && ctl->err) raise_error(&g_err, MOE_DEVERR_TIMEOUT);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" __attribute__((visibility("hidden"))) cudaError_t moe_detail_take_error_gmm_block(unsigned int* out) {
  unsigned int v = 0, z = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_err, sizeof(v));
  if (e == cudaSuccess && v) e = cudaMemcpyToSymbol(g_err, &z, sizeof(z));
  *out = v;
  return e;
}

extern "C" __attribute__((visibility("hidden"))) uint64_t moe_detail_stall_ns();

extern "C" moe_status gmm_fp8_block(const uint8_t* lhs_q, const float* lhs_scale, const uint8_t* rhs_q,
                                    const float* rhs_scale, const int32_t* group_sizes, int E, int group_offset,
                                    int E_local, int64_t M, int64_t K, int64_t N, uint16_t* out, moe_stream_t stream) {
  MOE_HOST_CHECK(lhs_q && lhs_scale && rhs_q && rhs_scale && out && (group_sizes || E == 1), MOE_ERR_INVALID_ARG);
  MOE_HOST_CHECK(E > 0 && E <= kMaxGroups && group_offset >= 0 && E_local > 0 && E_local <= E - group_offset,
                 MOE_ERR_INVALID_ARG);
  MOE_HOST_CHECK(M >= 0 && M < (1ll << 31) - 2 * kBM && K > 0 && K % 128 == 0 && K < (1 << 30) && N > 0 &&
                     N % 16 == 0 && N <= ((1ll << 31) - kBN) / E_local,
                 MOE_ERR_INVALID_ARG);
  MOE_HOST_CHECK(aligned16(lhs_q) && aligned16(lhs_scale) && aligned16(rhs_q) && aligned16(rhs_scale) && aligned16(out),
                 MOE_ERR_INVALID_ARG);
  const int64_t ntiles = (N + kBN - 1) / kBN;
  const int64_t most = ((M + kBM - 1) / kBM + E_local) * ntiles;  // tiles, at the most
  MOE_HOST_CHECK(most < (1ll << 31), MOE_ERR_INVALID_ARG);
  int sms = 0;
  const int dev = sm103_device(&sms);
  if (dev < 0) return MOE_ERR_UNSUPPORTED;
  if (M == 0) return MOE_OK;
  cudaStream_t st = as_stream(stream);
  CUtensorMap A, B;
  if (!make_map_u8(&A, lhs_q, K, M, K, kBM)) return MOE_ERR_CUDA;
  if (!make_map_u8(&B, rhs_q, K, static_cast<uint64_t>(E_local) * N, K, kBN)) return MOE_ERR_CUDA;
  const Params p{group_sizes, E, group_offset, E_local, M, static_cast<int>(N), static_cast<int>(K / 128),
                 static_cast<int>(ntiles), static_cast<int>((N + 127) / 128), lhs_scale, rhs_scale, out,
                 moe_detail_stall_ns()};
  // CTAs a tile: twice as many while the device holds them and the K blocks that are saved
  // (0.4 us each) take longer than the joining: 1.5 us and 2.3 us for 128 rows with the first
  // two, 0.4 and 2.4 for each doubling after that.  Measured on one row x 1536 x 2048: 9.9, 8.2,
  // 6.9, 6.6 us with 1, 2, 4, 8; on 128 rows 11.7, 12.3, 13.2, 15.2, with K = 4096 17.9, 15.5, 14.8, 16.1.
  const int64_t rows = M < kBM ? M : kBM;
  int parts = 1;
  while (parts < 8 && 2 * parts * most <= sms && 128ll * p.nkb > 2 * parts * ((parts == 1 ? 512 : 128) + 6 * rows))
    parts *= 2;
  auto kernel = parts > 1 ? gmm_block_kernel<true> : gmm_block_kernel<false>;
  static SmemLimit limit[2];
  MOE_CUDA_TRY(limit[parts > 1].set(kernel, kSmem, dev));
  if (parts == 1) {
    kernel<<<static_cast<unsigned>(most < sms ? most : sms), kThreads, kSmem, st>>>(A, B, p);
    MOE_CUDA_TRY(cudaGetLastError());
    return MOE_OK;
  }
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(parts);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(parts * most));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  MOE_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, A, B, p));
  return MOE_OK;
}
