// MXFP4 quantisation and reading back (OCP MX v1.0, see mx4.cuh):
//   moe_quantize_rows_mx4      bf16 rows -> packed e2m1 codes + E8M0 codes
//   moe_quantize_sort_mx4      the same for token rows, written to the k
//                              expert-sorted rows of each token
//   moe_swiglu_quant_mx4       h = bf16(silu(a0) a1) -> codes
//   moe_dequantize_rows_mx4    codes -> bf16 values
//
// 2^X is a power of two, so x / 2^X is exact in fp32 and each code is the
// correctly rounded e2m1 value of the quotient.
//
// All are HBM-bound (2 B read and 17/32 B written a value, or the reverse), the
// quantiser not by far from its instructions: about 75 a lane and 16 values.
// Rows are whole numbers of 128-column blocks, so a dense matrix is one run
// of such blocks: eight lanes take a block, each 16 adjacent values (one
// 32-byte load, one 8-byte store of codes), and no lane idles whatever the row
// length.  A 32-column scale block is two lanes (one shuffle for amax); two
// more shuffles put the block's four scale codes into the one word that the
// K-block-major scale layout stores.  A warp keeps the loads of kUnits times
// four blocks in flight.
#include "mx4.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// Units of 32 lanes that a warp loads before it works on the first.  Measured at
// 90112 x 4096 (floor 138 us): quantising 150 / 142 / 142 / 158 us with 1 / 2 / 4
// / 8, reading back 228 / 169 / 154 / 146 us.
constexpr int kUnits = 2;
constexpr int kBackUnits = 8;
constexpr int64_t kMaxCols = 32768;

__device__ __forceinline__ uint4 ldg16(const void* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

struct Pack16 {  // 16 bf16 values
  uint32_t w[8];
};
// 32 bytes (32-byte aligned) in one load
__device__ __forceinline__ Pack16 ldg32(const void* p) {
  Pack16 r;
  asm("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]), "=r"(r.w[6]), "=r"(r.w[7])
      : "l"(p));
  return r;
}
// Two 16-byte loads, where the address is only 16-byte aligned.
__device__ __forceinline__ Pack16 ldg16x2(const void* p) {
  const uint4 a = ldg16(p), b = ldg16(static_cast<const uint4*>(p) + 1);
  return Pack16{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}

// The larger magnitude of each half (bf16 pairs; NaN where either is NaN),
// with some sign.
__device__ __forceinline__ uint32_t maxabs2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Row and 128-column block of block b: 32-bit division where it holds every
// block (a 64-bit one takes as long as the work on a block).
__device__ __forceinline__ void split_block(int64_t b, int64_t blocks, int nkb, int64_t& row, int& kb) {
  if (blocks <= 0xFFFFFFFFll) {
    const uint32_t r = static_cast<uint32_t>(b) / static_cast<uint32_t>(nkb);
    row = r;
    kb = static_cast<int>(static_cast<uint32_t>(b) - r * static_cast<uint32_t>(nkb));
  } else {
    row = b / nkb;
    kb = static_cast<int>(b - row * nkb);
  }
}

// ---- producers: 16 bf16 values (packed) of a row, from column c on ----

struct Mx4RowsOp {  // plain bf16 rows
  const uint16_t* x;
  int64_t cols;
  bool wide;  // x is 32-byte aligned
  __device__ __forceinline__ Pack16 load(int64_t row, int c) const {
    const uint16_t* p = x + row * cols + c;
    return wide ? ldg32(p) : ldg16x2(p);
  }
  __device__ __forceinline__ int ndst() const { return 1; }
  __device__ __forceinline__ int64_t dst(int64_t row, int) const { return row; }
};

struct Mx4GatherOp {  // token rows: the codes go to the token's k sorted rows
  const uint16_t* x;
  int64_t cols;
  bool wide;
  const int32_t* pos;
  int k;
  int64_t R;
  __device__ __forceinline__ Pack16 load(int64_t row, int c) const {
    const uint16_t* p = x + row * cols + c;
    return wide ? ldg32(p) : ldg16x2(p);
  }
  __device__ __forceinline__ int ndst() const { return k; }
  __device__ __forceinline__ int64_t dst(int64_t row, int j) const {
    const int64_t p = __ldg(pos + row * k + j);
    return (p >= 0 && p < R) ? p : -1;
  }
};

struct Mx4SwigluOp {  // h = bf16(silu(a0) a1), a = [a0 | a1] of width 2F
  const uint16_t* a;
  int64_t F;
  __device__ __forceinline__ Pack16 load(int64_t row, int c) const {
    const Pack16 p0 = ldg16x2(a + row * 2 * F + c), p1 = ldg16x2(a + row * 2 * F + F + c);
    float a0[16], a1[16], h[16];
    Pack16 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a0[2 * i] = bf16lo(p0.w[i]);
      a0[2 * i + 1] = bf16hi(p0.w[i]);
      a1[2 * i] = bf16lo(p1.w[i]);
      a1[2 * i + 1] = bf16hi(p1.w[i]);
    }
    swiglu_h_x2<16>(a0, a1, h, r.w);
    return r;
  }
  __device__ __forceinline__ int ndst() const { return 1; }
  __device__ __forceinline__ int64_t dst(int64_t row, int) const { return row; }
};

// q [nrows, 64 nkb] bytes, sf words [nkb][nrows]; `rows` source rows of nkb
// 128-column blocks.
template <class Op>
__global__ void __launch_bounds__(kThreads) quant_mx4_kernel(Op op, int64_t rows, int nkb, int64_t nrows, uint8_t* q,
                                                             uint32_t* sf) {
  const int lane = threadIdx.x & 31;
  const int l8 = lane & 7;
  const int64_t blocks = rows * nkb;
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * (4 * kUnits) + (lane >> 3);
  int64_t row[kUnits];
  int kb[kUnits];
  Pack16 d[kUnits];
  split_block(first, blocks, nkb, row[0], kb[0]);
#pragma unroll
  for (int u = 1; u < kUnits; ++u) {  // four blocks further each
    row[u] = row[u - 1];
    kb[u] = kb[u - 1] + 4;
    while (kb[u] >= nkb) {
      kb[u] -= nkb;
      ++row[u];
    }
  }
#pragma unroll
  for (int u = 0; u < kUnits; ++u)
    d[u] = first + 4 * u < blocks ? op.load(row[u], kb[u] * 128 + l8 * 16) : Pack16{{0, 0, 0, 0, 0, 0, 0, 0}};
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    uint32_t* w = d[u].w;
    uint32_t m2 = maxabs2(maxabs2(maxabs2(w[0], w[1]), maxabs2(w[2], w[3])),
                          maxabs2(maxabs2(w[4], w[5]), maxabs2(w[6], w[7])));
    m2 = maxabs2(m2, __shfl_xor_sync(0xffffffffu, m2, 1)) & 0x7FFF7FFFu;
    const uint32_t code = mx4_scale_code(max(m2 & 0xFFFFu, m2 >> 16));
    // 2^-X as a bf16 pair.  The products are exact, but for those far below the
    // smallest code's half step, whose code is 0 all the same
    const uint32_t inv = __float_as_uint(mx4_inv_scale(code)) >> 16, inv2 = inv | inv << 16;
    float v[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t t = code == kE8M0NaN ? w[i] & 0x80008000u  // the signs alone: infinity times zero is no value to round
                                          : mul2(w[i], inv2);
      v[2 * i] = bf16lo(t);
      v[2 * i + 1] = bf16hi(t);
    }
    const uint2 codes = make_uint2(pack_e2m1x8(v), pack_e2m1x8(v + 8));
    uint32_t word = code << (8 * (l8 >> 1));
    word |= __shfl_xor_sync(0xffffffffu, word, 2);
    word |= __shfl_xor_sync(0xffffffffu, word, 4);
    if (first + 4 * u < blocks) {
      for (int j = 0; j < op.ndst(); ++j) {
        const int64_t dr = op.dst(row[u], j);
        if (dr < 0) continue;
        *reinterpret_cast<uint2*>(q + (dr * nkb + kb[u]) * 64 + l8 * 8) = codes;
        if (l8 == 0) sf[kb[u] * nrows + dr] = word;
      }
    }
  }
}

template <class Op>
moe_status launch_quant(const Op& op, int64_t rows, int64_t cols, int64_t nrows, uint8_t* q, uint8_t* sf,
                        cudaStream_t st) {
  const int nkb = static_cast<int>(cols / 128);
  const int64_t per = kWarps * 4 * kUnits;
  const int64_t grid = (rows * nkb + per - 1) / per;
  if (grid == 0) return MOE_OK;
  MOE_HOST_CHECK(grid < (1ll << 31), MOE_ERR_INVALID_ARG);
  quant_mx4_kernel<<<static_cast<unsigned>(grid), kThreads, 0, st>>>(op, rows, nkb, nrows, q,
                                                                     reinterpret_cast<uint32_t*>(sf));
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// One 8-value group (4 bytes of codes, a 16-byte store) a lane and unit: half a
// warp takes a 128-column block.
__global__ void __launch_bounds__(kThreads) dequant_mx4_kernel(const uint8_t* q, const uint8_t* sf, int64_t rows,
                                                               int nkb, uint16_t* out) {
  const int lane = threadIdx.x & 31;
  const int l16 = lane & 15;
  const int64_t blocks = rows * nkb;
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * (2 * kBackUnits) + (lane >> 4);
  int64_t row;
  int kb;
  split_block(first, blocks, nkb, row, kb);
  uint32_t c[kBackUnits], s[kBackUnits];
#pragma unroll
  for (int u = 0; u < kBackUnits; ++u) {
    const bool ok = first + 2 * u < blocks;
    c[u] = ok ? __ldg(reinterpret_cast<const uint32_t*>(q + (first + 2 * u) * 64 + l16 * 4)) : 0u;
    s[u] = ok ? __ldg(sf + (kb * rows + row) * 4 + (l16 >> 2)) : 0u;
    kb += 2;
    while (kb >= nkb) {
      kb -= nkb;
      ++row;
    }
  }
#pragma unroll
  for (int u = 0; u < kBackUnits; ++u) {
    const float sc = e8m0_value(s[u]);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = pack_bf16x2(__fmul_rn(e2m1_value(c[u] >> (8 * i)), sc), __fmul_rn(e2m1_value(c[u] >> (8 * i + 4)), sc));
    if (first + 2 * u < blocks)
      *reinterpret_cast<uint4*>(out + (first + 2 * u) * 128 + l16 * 8) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

bool shape_ok(int64_t rows, int64_t cols) {
  return rows >= 0 && rows < (1ll << 31) && cols > 0 && cols % 128 == 0 && cols <= kMaxCols;
}

bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_quantize_rows_mx4(const uint16_t* x, int64_t rows, int64_t cols, uint8_t* q, uint8_t* sf,
                                            moe_stream_t stream) {
  MOE_HOST_CHECK(x && q && sf && shape_ok(rows, cols), MOE_ERR_INVALID_ARG);
  MOE_HOST_CHECK(aligned16(x) && aligned16(q) && aligned4(sf), MOE_ERR_INVALID_ARG);
  return launch_quant(Mx4RowsOp{x, cols, aligned32(x)}, rows, cols, rows, q, sf, as_stream(stream));
}

// Called by sort.cu once the sort indices exist (moe_quantize_sort_mx4).
extern "C" __attribute__((visibility("hidden"))) moe_status moe_detail_quantize_gather_mx4(
    const uint16_t* x, const int32_t* pos, int64_t T, int k, int64_t D, uint8_t* xs_q, uint8_t* xs_sf,
    cudaStream_t st) {
  MOE_HOST_CHECK(shape_ok(T, D), MOE_ERR_INVALID_ARG);
  return launch_quant(Mx4GatherOp{x, D, aligned32(x), pos, k, T * k}, T, D, T * k, xs_q, xs_sf, st);
}

extern "C" moe_status moe_swiglu_quant_mx4(const uint16_t* a, int64_t R, int64_t F, uint8_t* h_q, uint8_t* h_sf,
                                           moe_stream_t stream) {
  MOE_HOST_CHECK(a && h_q && h_sf && shape_ok(R, F), MOE_ERR_INVALID_ARG);
  MOE_HOST_CHECK(aligned16(a) && aligned16(h_q) && aligned4(h_sf), MOE_ERR_INVALID_ARG);
  return launch_quant(Mx4SwigluOp{a, F}, R, F, R, h_q, h_sf, as_stream(stream));
}

extern "C" moe_status moe_dequantize_rows_mx4(const uint8_t* q, const uint8_t* sf, int64_t rows, int64_t cols,
                                              uint16_t* x, moe_stream_t stream) {
  MOE_HOST_CHECK(q && sf && x && shape_ok(rows, cols), MOE_ERR_INVALID_ARG);
  MOE_HOST_CHECK(aligned16(q) && aligned16(x) && aligned4(sf), MOE_ERR_INVALID_ARG);
  const int64_t nkb = cols / 128, per = kWarps * 2 * kBackUnits;
  const int64_t grid = (rows * nkb + per - 1) / per;
  if (grid == 0) return MOE_OK;
  MOE_HOST_CHECK(grid < (1ll << 31), MOE_ERR_INVALID_ARG);
  dequant_mx4_kernel<<<static_cast<unsigned>(grid), kThreads, 0, as_stream(stream)>>>(q, sf, rows,
                                                                                     static_cast<int>(nkb), x);
  MOE_CUDA_TRY(cudaGetLastError());
  return MOE_OK;
}
