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
// Bound.  A pair of CTAs works on 256 x 256 tiles, 128 rows a CTA; a K block is
// four M = 256, N = 256, K = 32 tcgen05.mma.kind::f8f6f4 of the pair, 554 clocks at
// their measured rate, and the fold takes 256 clocks of each SM's fp32 pipes and the
// reading of 128 KB of tensor memory beside it.
//
// Layout of a CTA (12 warps, one CTA per SM, persistent):
//   warp 0      TMA producer: this CTA's 128 A rows and its half (128 rows) of the
//               B tile per stage, 32 KB, six stages, 128-byte swizzle.
//   warp 1      of the pair's even CTA: MMA issuer.
//   warps 4..11 epilogue: warp w has tensor-memory lanes 32 (w % 4).. (rows) and
//               128 of the tile's columns: 128 running sums a thread.
// Two 256-column accumulators take alternate K blocks.  Row and block scales come
// straight to registers, four K blocks at a time and four blocks ahead.
//
// Tiles run expert-major, then N tile, then M tile: CTAs that run together share
// an expert's weights.  A group's M tiles start at its first row; rows past its end
// are computed and not stored.
//
// Every wait is bounded; on expiry the kernel raises MOE_DEVERR_TIMEOUT, lets what
// it issued finish and returns.
#include "grouped.cuh"

namespace moe {
namespace {

__device__ unsigned int g_err;

constexpr int kBM = 128, kBN = 256, kBK = 128;
constexpr int kStages = 6;
constexpr int kABytes = kBM * kBK, kBBytes = kBN / 2 * kBK;
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kCtrlWarps = 4, kEpiWarps = 8;
constexpr int kThreads = 32 * (kCtrlWarps + kEpiWarps);
// registers a thread: 168 at launch, handed from the control warpgroup to the epilogue
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
  uint64_t never;  // test hook: a barrier that nothing arrives on
  uint32_t tmem_base;
  int abort_flag, no_abort, err, total;
  int start[kMaxGroups + 1], prefix[kMaxGroups + 1];  // local groups' first rows and units; the last: their ends
};
constexpr size_t kCtlBytes = (sizeof(Ctl) + 127) / 128 * 128;
constexpr size_t kSmem = 1024 + static_cast<size_t>(kStages) * kStageBytes + kCtlBytes;
static_assert(kSmem <= 232448, "shared memory per CTA");

// Local groups' first rows and first units (pairs of M tiles times N tiles), by
// warp 0 (any size negative or a sum other than M: err).
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
    const int nu = mine && sz > 0 ? (sz + 2 * kBM - 1) / (2 * kBM) * p.ntiles : 0;
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
  int el, row0, rows, n0;  // rows <= 0: the odd CTA of a pair past the group's end
};

__device__ __forceinline__ Tile get_tile(const Params& p, const Ctl* c, int t, int rank) {
  int lo = 0, hi = p.El;  // the last group whose first unit is <= t: it is not empty
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (c->prefix[mid] <= t) lo = mid; else hi = mid;
  }
  Tile tl;
  tl.el = lo;
  const int sz = c->start[lo + 1] - c->start[lo], mp = (sz + 2 * kBM - 1) / (2 * kBM), local = t - c->prefix[lo];
  const int nt = local / mp, mi = 2 * (local - nt * mp) + rank;
  tl.row0 = c->start[lo] + mi * kBM;
  tl.rows = min(kBM, sz - mi * kBM);
  tl.n0 = nt * kBN;
  return tl;
}

// 32 lanes x 32 columns of tensor memory as 16 packed fp32 pairs a thread.
__device__ __forceinline__ void tmem_ld_x32_pairs(uint32_t taddr, uint64_t (&r)[16]) {
  asm volatile(
      "{\n\t.reg .b32 t<32>;\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {t0, t1, t2, t3, t4, t5, t6, t7, t8, t9, t10, t11, t12, t13, t14, t15, "
      "t16, t17, t18, t19, t20, t21, t22, t23, t24, t25, t26, t27, t28, t29, t30, t31}, [%16];\n\t"
      "mov.b64 %0, {t0, t1};\n\tmov.b64 %1, {t2, t3};\n\tmov.b64 %2, {t4, t5};\n\tmov.b64 %3, {t6, t7};\n\t"
      "mov.b64 %4, {t8, t9};\n\tmov.b64 %5, {t10, t11};\n\tmov.b64 %6, {t12, t13};\n\tmov.b64 %7, {t14, t15};\n\t"
      "mov.b64 %8, {t16, t17};\n\tmov.b64 %9, {t18, t19};\n\tmov.b64 %10, {t20, t21};\n\tmov.b64 %11, {t22, t23};\n\t"
      "mov.b64 %12, {t24, t25};\n\tmov.b64 %13, {t26, t27};\n\tmov.b64 %14, {t28, t29};\n\tmov.b64 %15, {t30, t31};\n\t}"
      : "=l"(r[0]), "=l"(r[1]), "=l"(r[2]), "=l"(r[3]), "=l"(r[4]), "=l"(r[5]), "=l"(r[6]), "=l"(r[7]), "=l"(r[8]),
        "=l"(r[9]), "=l"(r[10]), "=l"(r[11]), "=l"(r[12]), "=l"(r[13]), "=l"(r[14]), "=l"(r[15])
      : "r"(taddr)
      : "memory");
}
// The loads have landed; the values are used only after it.
__device__ __forceinline__ void tmem_wait_ld_pairs(uint64_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+l"(r[0]), "+l"(r[1]), "+l"(r[2]), "+l"(r[3]), "+l"(r[4]), "+l"(r[5]), "+l"(r[6]), "+l"(r[7]),
                 "+l"(r[8]), "+l"(r[9]), "+l"(r[10]), "+l"(r[11]), "+l"(r[12]), "+l"(r[13]), "+l"(r[14]), "+l"(r[15])
               :
               : "memory");
}

// Scales of K blocks kb .. kb + 3 (past the last: not read).
__device__ __forceinline__ void load_scales4(const float* s, int kb, int nkb, bool vec, float (&v)[4]) {
  if (vec) {
    const float4 f = __ldg(reinterpret_cast<const float4*>(s + kb));
    v[0] = f.x;
    v[1] = f.y;
    v[2] = f.z;
    v[3] = f.w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = kb + j < nkb ? __ldg(s + kb + j) : 0.f;
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    gmm_block_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
  Ctl* ctl = reinterpret_cast<Ctl*>(smem_raw + (base - raw) + kStages * kStageBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // a pair works on one sequence of units; its even CTA (rank 0) issues the MMAs
  // and owns the full and accumulator-empty barriers
  const int rank = static_cast<int>(__clusterRelativeBlockRank());
  const int unit0 = static_cast<int>(__clusterIdx().x), units = static_cast<int>(__clusterGridDimInClusters().x);

  if (warp == 0) build_tables(p, ctl);
  if (threadIdx.x == 32) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&ctl->full[s]), 1);
      mbar_init(smem_u32(&ctl->empty[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&ctl->tfull[a]), 1);
      mbar_init(smem_u32(&ctl->tempty[a]), 2 * kEpiWarps);
    }
    mbar_init(smem_u32(&ctl->drain), 1);
    mbar_init(smem_u32(&ctl->never), 1);
    ctl->abort_flag = 0;
    ctl->no_abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  // both CTAs of a pair read the same group sizes, so they leave here together
  if (ctl->err) {
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
  const uint32_t tmem = ctl->tmem_base;
  if (rank == 1 && threadIdx.x == 0 &&
      ld_shared_cluster_u32(mapa_shared(smem_u32(&ctl->tmem_base), 0)) != tmem)
    raise_error(&g_err, MOE_DEVERR_TMEM);  // the pair's accumulators would not line up
  const int total = ctl->total;
  volatile int* abort_flag = &ctl->abort_flag;
  bool timed_out = false;

  if (warp < kCtrlWarps) {
    setmaxnreg_dec<kCtrlRegs>();
    if (warp == 0) {
      if (lane == 0) {
        uint32_t it = 0;
        for (int t = unit0; t < total && !timed_out; t += units) {
          const Tile tl = get_tile(p, ctl, t, rank);
          const int brow = tl.el * p.N + tl.n0 + rank * (kBN / 2);
          for (int kb = 0; kb < p.nkb; ++kb, ++it) {
            const int s = it % kStages;
            if (!mbar_wait_bounded_idle(smem_u32(&ctl->empty[s]), ((it / kStages) & 1) ^ 1, abort_flag, kWaitLimitNs)) {
              timed_out = true;
              break;
            }
            const uint32_t sa = base + s * kStageBytes;
            // both CTAs' boxes complete on the even CTA's full barrier
            const uint32_t fb = mapa_shared(smem_u32(&ctl->full[s]), 0);
            if (rank == 0) mbar_arrive_expect_tx(smem_u32(&ctl->full[s]), 2 * kStageBytes);
            tma_load_2d_pair(sa, &tmA, kb * kBK, tl.row0, fb);
            tma_load_2d_pair(sa + kABytes, &tmB, kb * kBK, brow, fb);
          }
        }
        if (timed_out) {
          *abort_flag = 1;
          ctl->err = 2;
        }
        // The last loads land before the CTAs can exit, whichever role's wait ran
        // out.  The even CTA's barriers count both CTAs' loads; a load of the odd
        // one that the even one never announced lands within microseconds.
        if (rank == 0) {
          for (uint32_t j = it > kStages ? it - kStages : 0; j < it; ++j)
            mbar_wait_bounded(smem_u32(&ctl->full[j % kStages]), (j / kStages) & 1, &ctl->no_abort,
                              ctl->err ? kWaitLimitNs / 8 : kWaitLimitNs);
        } else if (timed_out) {
          mbar_wait_bounded(smem_u32(&ctl->never), 0, &ctl->no_abort, 1000000ull);
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      if (lane == 0 && rank == 0) {
        uint32_t it = 0;
        for (int t = unit0; t < total && !timed_out; t += units) {
          for (int kb = 0; kb < p.nkb; ++kb, ++it) {
            const int s = it % kStages;
            const uint32_t a = it & 1;
            if (!mbar_wait_bounded(smem_u32(&ctl->full[s]), (it / kStages) & 1, abort_flag, kWaitLimitNs) ||
                !mbar_wait_bounded(smem_u32(&ctl->tempty[a]), ((it >> 1) & 1) ^ 1, abort_flag, kWaitLimitNs)) {
              timed_out = true;
              break;
            }
            tc_fence_after();
            const uint32_t sa = base + s * kStageBytes;
            const uint64_t da = smem_desc_sw128(sa), db = smem_desc_sw128(sa + kABytes);
#pragma unroll
            for (int k4 = 0; k4 < 4; ++k4)  // 32 bytes of K: 2 in the descriptors' 16-byte units
              mma_f8_pair(tmem + a * kBN, da + 2 * k4, db + 2 * k4, idesc_e4m3_f32(2 * kBM, kBN), k4 > 0);
            mma_commit_pair_mc(smem_u32(&ctl->empty[s]), 0x3);  // frees the stage in both CTAs
            mma_commit_pair_mc(smem_u32(&ctl->tfull[a]), 0x3);
          }
        }
        mma_commit_pair(smem_u32(&ctl->drain));
        if (!mbar_wait_bounded(smem_u32(&ctl->drain), 0, &ctl->no_abort, kWaitLimitNs)) timed_out = true;
        if (timed_out) {
          *abort_flag = 1;
          ctl->err = 2;
        }
      }
      __syncwarp();
    }
  } else {
    setmaxnreg_inc<kEpiRegs>();
    const int q4 = warp & 3, half = (warp - kCtrlWarps) >> 2;
    const uint32_t taddr = tmem + (static_cast<uint32_t>(q4 * 32) << 16) + half * (kBN / 2);
    const bool vec = (p.nkb & 3) == 0;  // every row's scales start on 16 bytes
    const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
    uint32_t it = 0;
    if (p.stall_ns && !mbar_wait_bounded_warp(smem_u32(&ctl->never), 0, abort_flag, p.stall_ns)) timed_out = true;
    for (int t = unit0; t < total && !timed_out; t += units) {
      const Tile tl = get_tile(p, ctl, t, rank);
      const int r = q4 * 32 + lane, nb = min(tl.n0 / kBK + half, p.nblk - 1);
      const bool work = tl.rows > q4 * 32 && tl.n0 + half * (kBN / 2) < p.N;  // (of the warp)
      // a row past the group's end takes the scales of its last one (an odd CTA past
      // it: of any row)
      const int64_t srow = tl.rows > 0 ? tl.row0 + min(r, tl.rows - 1) : 0;
      const float* sa = p.lhs_s + srow * p.nkb;
      const float* sb = p.rhs_s + (static_cast<int64_t>(tl.el) * p.nblk + nb) * p.nkb;
      uint64_t acc[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) acc[j] = 0;
      float na[4], nw[4];
      load_scales4(sa, 0, p.nkb, vec, na);
      load_scales4(sb, 0, p.nkb, vec, nw);
      for (int kb0 = 0; kb0 < p.nkb && !timed_out; kb0 += 4) {
        float s4[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) s4[j] = __fmul_rn(na[j], nw[j]);
        if (kb0 + 4 < p.nkb) {
          load_scales4(sa, kb0 + 4, p.nkb, vec, na);
          load_scales4(sb, kb0 + 4, p.nkb, vec, nw);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (kb0 + j >= p.nkb) break;
          const uint32_t a = it & 1;
          if (!mbar_wait_bounded_warp(smem_u32(&ctl->tfull[a]), (it >> 1) & 1, abort_flag, kWaitLimitNs)) {
            timed_out = true;
            break;
          }
          ++it;
          tc_fence_after();
          const uint32_t ta = taddr + a * kBN;
          const uint64_t s2 = f2_pack(s4[j], s4[j]);
          uint64_t u[16], v[16];
          if (work) {
            tmem_ld_x32_pairs(ta, u);
            tmem_wait_ld_pairs(u);
            tmem_ld_x32_pairs(ta + 32, v);
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[i] = f2_fma(u[i], s2, acc[i]);
            tmem_wait_ld_pairs(v);
            tmem_ld_x32_pairs(ta + 64, u);
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[16 + i] = f2_fma(v[i], s2, acc[16 + i]);
            tmem_wait_ld_pairs(u);
            tmem_ld_x32_pairs(ta + 96, v);
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[32 + i] = f2_fma(u[i], s2, acc[32 + i]);
            tmem_wait_ld_pairs(v);
          }
          tc_fence_before();
          __syncwarp();
          // (relaxed: it orders only tensor-memory loads that have completed)
          if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&ctl->tempty[a]), 0));
          if (work) {
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[48 + i] = f2_fma(v[i], s2, acc[48 + i]);
          }
        }
      }
      if (timed_out) break;
      if (r < tl.rows) {
        uint16_t* o = p.out + (tl.row0 + r) * static_cast<int64_t>(p.N) + tl.n0 + half * (kBN / 2);
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
  // neither CTA leaves (or frees its columns) while the other may still write its
  // tensor memory or arrive on its barriers
  cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
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
  const int64_t max_units = ((M + 2 * kBM - 1) / (2 * kBM) + E_local) * ntiles;
  MOE_HOST_CHECK(max_units < (1ll << 31), MOE_ERR_INVALID_ARG);
  const int sms = sm103_count();
  if (sms <= 0) return MOE_ERR_UNSUPPORTED;
  if (M == 0) return MOE_OK;
  cudaStream_t st = as_stream(stream);
  CUtensorMap A, B;
  if (!make_map_u8(&A, lhs_q, K, M, K, kBM)) return MOE_ERR_CUDA;
  if (!make_map_u8(&B, rhs_q, K, static_cast<uint64_t>(E_local) * N, K, kBN / 2)) return MOE_ERR_CUDA;
  Params p{group_sizes, E, group_offset, E_local, M, static_cast<int>(N), static_cast<int>(K / 128),
           static_cast<int>(ntiles), static_cast<int>((N + 127) / 128), lhs_scale, rhs_scale, out,
           moe_detail_stall_ns()};
  MOE_CUDA_TRY(cudaFuncSetAttribute(gmm_block_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(kSmem)));
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // pairs that are resident at once, per device
  static std::mutex mu;
  static int resident[kMaxDevices] = {};
  int dev = 0, pairs = 0;
  MOE_CUDA_TRY(cudaGetDevice(&dev));
  if (dev < 0 || dev >= kMaxDevices) return MOE_ERR_UNSUPPORTED;
  {
    std::lock_guard<std::mutex> lock(mu);
    pairs = resident[dev];
  }
  if (pairs == 0) {
    // the register split may only hand out what the CTA is launched with
    cudaFuncAttributes fa{};
    MOE_CUDA_TRY(cudaFuncGetAttributes(&fa, gmm_block_kernel));
    if (static_cast<int64_t>(fa.numRegs) * kThreads < 128ll * kCtrlRegs + 256ll * kEpiRegs) return MOE_ERR_UNSUPPORTED;
    cfg.gridDim = dim3(2 * (sms / 2));
    MOE_CUDA_TRY(cudaOccupancyMaxActiveClusters(&pairs, gmm_block_kernel, &cfg));
    if (pairs <= 0) return MOE_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lock(mu);
    resident[dev] = pairs;
  }
  if (E_local < E) {
    zero_outside_rows_kernel<<<sms * 4, 256, 0, st>>>(out, M, N, group_sizes, E, group_offset, E_local);
    MOE_CUDA_TRY(cudaGetLastError());
  }
  cfg.gridDim = dim3(2 * static_cast<unsigned>(max_units < pairs ? max_units : pairs));
  MOE_CUDA_TRY(cudaLaunchKernelEx(&cfg, gmm_block_kernel, A, B, p));
  return MOE_OK;
}
