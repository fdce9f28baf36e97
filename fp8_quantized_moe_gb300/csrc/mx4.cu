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
// All are HBM-bound (2 B read and 17/32 B written a value, or the reverse).
// Rows are whole numbers of 128-column blocks, so a dense matrix is one run
// of such blocks: half a warp takes a block, each lane 8 adjacent values (one
// 16-byte load, one 4-byte store of codes), and no lane idles whatever the
// row length.  A 32-column scale block is four lanes (two shuffles for amax);
// two more shuffles put the block's four scale codes into the one word that
// the K-block-major scale layout stores.  A warp keeps the loads of kUnits
// pairs of blocks in flight.
#include "mx4.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnits = 4;  // 256-value units a warp loads before it works on the first
constexpr int64_t kMaxCols = 32768;

__device__ __forceinline__ uint4 ldg16(const void* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

// ---- producers: 8 bf16 values (packed) of 128-column block kb of a row ----

struct Mx4RowsOp {  // plain bf16 rows
  const uint16_t* x;
  int64_t cols;
  __device__ __forceinline__ uint4 load(int64_t row, int c) const { return ldg16(x + row * cols + c); }
  __device__ __forceinline__ int ndst() const { return 1; }
  __device__ __forceinline__ int64_t dst(int64_t row, int) const { return row; }
};

struct Mx4GatherOp {  // token rows: the codes go to the token's k sorted rows
  const uint16_t* x;
  int64_t cols;
  const int32_t* pos;
  int k;
  int64_t R;
  __device__ __forceinline__ uint4 load(int64_t row, int c) const { return ldg16(x + row * cols + c); }
  __device__ __forceinline__ int ndst() const { return k; }
  __device__ __forceinline__ int64_t dst(int64_t row, int j) const {
    const int64_t p = __ldg(pos + row * k + j);
    return (p >= 0 && p < R) ? p : -1;
  }
};

struct Mx4SwigluOp {  // h = bf16(silu(a0) a1), a = [a0 | a1] of width 2F
  const uint16_t* a;
  int64_t F;
  __device__ __forceinline__ uint4 load(int64_t row, int c) const {
    const uint4 d0 = ldg16(a + row * 2 * F + c), d1 = ldg16(a + row * 2 * F + F + c);
    const uint32_t w0[4] = {d0.x, d0.y, d0.z, d0.w}, w1[4] = {d1.x, d1.y, d1.z, d1.w};
    float a0[8], a1[8], h[8];
    uint32_t hb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a0[2 * i] = bf16lo(w0[i]);
      a0[2 * i + 1] = bf16hi(w0[i]);
      a1[2 * i] = bf16lo(w1[i]);
      a1[2 * i + 1] = bf16hi(w1[i]);
    }
    swiglu_h_x2<8>(a0, a1, h, hb);
    return make_uint4(hb[0], hb[1], hb[2], hb[3]);
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
  const int l16 = lane & 15;
  const int64_t blocks = rows * nkb;
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * (2 * kUnits) + (lane >> 4);
  int64_t row[kUnits];
  int kb[kUnits];
  uint4 d[kUnits];
  row[0] = first / nkb;
  kb[0] = static_cast<int>(first - row[0] * nkb);
#pragma unroll
  for (int u = 1; u < kUnits; ++u) {  // two blocks further each
    row[u] = row[u - 1];
    kb[u] = kb[u - 1] + 2;
    while (kb[u] >= nkb) {
      kb[u] -= nkb;
      ++row[u];
    }
  }
#pragma unroll
  for (int u = 0; u < kUnits; ++u)
    d[u] = first + 2 * u < blocks ? op.load(row[u], kb[u] * 128 + l16 * 8) : make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const uint32_t w[4] = {d[u].x, d[u].y, d[u].z, d[u].w};
    // bf16 magnitudes order like their bit patterns, infinities and NaN last
    uint32_t m2 = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                           __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
    m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, 1));
    m2 = __vmaxu2(m2, __shfl_xor_sync(0xffffffffu, m2, 2));
    const uint32_t code = mx4_scale_code(max(m2 & 0xFFFFu, m2 >> 16));
    const float inv = mx4_inv_scale(code);
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __fmul_rn(bf16lo(w[i]), inv);
      v[2 * i + 1] = __fmul_rn(bf16hi(w[i]), inv);
    }
    if (code == kE8M0NaN) {  // the signs alone (an infinity or a NaN times zero is no value to round)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16 & 0x80000000u);
        v[2 * i + 1] = __uint_as_float(w[i] & 0x80000000u);
      }
    }
    const uint32_t codes = pack_e2m1x8(v);
    uint32_t word = code << (8 * (l16 >> 2));
    word |= __shfl_xor_sync(0xffffffffu, word, 4);
    word |= __shfl_xor_sync(0xffffffffu, word, 8);
    if (first + 2 * u < blocks) {
      for (int j = 0; j < op.ndst(); ++j) {
        const int64_t dr = op.dst(row[u], j);
        if (dr < 0) continue;
        *reinterpret_cast<uint32_t*>(q + (dr * nkb + kb[u]) * 64 + l16 * 4) = codes;
        if (l16 == 0) sf[kb[u] * nrows + dr] = word;
      }
    }
  }
}

template <class Op>
moe_status launch_quant(const Op& op, int64_t rows, int64_t cols, int64_t nrows, uint8_t* q, uint8_t* sf,
                        cudaStream_t st) {
  const int nkb = static_cast<int>(cols / 128);
  const int64_t per = kWarps * 2 * kUnits;
  const int64_t grid = (rows * nkb + per - 1) / per;
  if (grid == 0) return MOE_OK;
  MOE_HOST_CHECK(grid < (1ll << 31), MOE_ERR_INVALID_ARG);
  quant_mx4_kernel<<<static_cast<unsigned>(grid), kThreads, 0, st>>>(op, rows, nkb, nrows, q,
                                                                     reinterpret_cast<uint32_t*>(sf));
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// One 8-value group (4 bytes of codes) a lane and unit, as in the quantiser.
__global__ void __launch_bounds__(kThreads) dequant_mx4_kernel(const uint8_t* q, const uint8_t* sf, int64_t rows,
                                                               int nkb, uint16_t* out) {
  const int lane = threadIdx.x & 31;
  const int l16 = lane & 15;
  const int64_t blocks = rows * nkb;
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * (2 * kUnits) + (lane >> 4);
  int64_t row = first / nkb;
  int kb = static_cast<int>(first - row * nkb);
  uint32_t c[kUnits], s[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
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
  for (int u = 0; u < kUnits; ++u) {
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

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_quantize_rows_mx4(const uint16_t* x, int64_t rows, int64_t cols, uint8_t* q, uint8_t* sf,
                                            moe_stream_t stream) {
  MOE_HOST_CHECK(x && q && sf && shape_ok(rows, cols), MOE_ERR_INVALID_ARG);
  MOE_HOST_CHECK(aligned16(x) && aligned16(q) && aligned4(sf), MOE_ERR_INVALID_ARG);
  return launch_quant(Mx4RowsOp{x, cols}, rows, cols, rows, q, sf, as_stream(stream));
}

// Called by sort.cu once the sort indices exist (moe_quantize_sort_mx4).
extern "C" __attribute__((visibility("hidden"))) moe_status moe_detail_quantize_gather_mx4(
    const uint16_t* x, const int32_t* pos, int64_t T, int k, int64_t D, uint8_t* xs_q, uint8_t* xs_sf,
    cudaStream_t st) {
  MOE_HOST_CHECK(shape_ok(T, D), MOE_ERR_INVALID_ARG);
  return launch_quant(Mx4GatherOp{x, D, pos, k, T * k}, T, D, T * k, xs_q, xs_sf, st);
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
  const int64_t nkb = cols / 128, per = kWarps * 2 * kUnits;
  const int64_t grid = (rows * nkb + per - 1) / per;
  if (grid == 0) return MOE_OK;
  MOE_HOST_CHECK(grid < (1ll << 31), MOE_ERR_INVALID_ARG);
  dequant_mx4_kernel<<<static_cast<unsigned>(grid), kThreads, 0, as_stream(stream)>>>(q, sf, rows,
                                                                                     static_cast<int>(nkb), x);
  MOE_CUDA_TRY(cudaGetLastError());
  return MOE_OK;
}
