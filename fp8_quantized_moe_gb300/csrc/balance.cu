// Balance loss of the router with per-expert counts, and its gradient.
//
// The T rows are S sequences of L = T / S rows, n_s of them valid.  With p the
// softmax of a row's logits, for every sequence s and expert e:
//   counts[s, e] = pairs of valid rows routed to e      mean[s, e] = (1/n_s) sum of p[t, e]
//   f[s, e]      = counts[s, e] E / (k n_s)
//   loss         = coef / S * sum_s sum_e f[s, e] mean[s, e]
// and, counts being constants, for a valid row of s
//   dlogits[t, e] = p_e (c_e - sum_j p_j c_j),   c_e = grad coef E / (S k n_s^2) counts[s, e].
//
// Both passes read the logits once (the second from L2 where they fit), so they
// are bound by memory, or by latency where there are few rows.  A row is held by
// LPR lanes, four columns a load and lane: its maximum and sum are shuffles.
// Column sums stay in registers over a warp's rows, are added over the block's warps
// and then over the blocks of a sequence in a fixed order (no floating-point atomics:
// the result does not depend on timing); counts are integers.
//
// Measured, both passes back to back: 24 rows of 128 experts 6.8 us, 4 x 4096 of 256 experts
// 20 us (12 for the sums, 8 for the gradient; bytes 5), 32 x 8192 of 64 experts 53 us (19, 34;
// bytes 21): the small ones are launches and round trips.  The last one's kernels keep their issue slots
// 66 and 57 % busy and DRAM 45 and 34 % (L2 30 and 21), and their warps wait for loads most: a
// warp asks for its rows, then computes them, and the other warps cover that only in part.
// (exp_f32 and one load a lane: 84 us when the rest took 57.)
//
// The gradient takes counts relative to the row's most probable expert e*: with
// c'_e = c_e - c_{e*} the formula is the same, and where p_{e*} is near 1 the two terms
// of the difference no longer cancel (the integers' difference is exact).
#include <algorithm>
#include <type_traits>

#include "common.cuh"

namespace moe {
namespace {

__device__ unsigned int g_err;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxE = 1024, kMaxK = 32;

struct Shape {
  int64_t L;      // rows a sequence
  int S, E, k;
  int chunk;      // rows a block
  int per;        // blocks a sequence
  bool vec;       // 16-byte loads: rows start on 16 bytes
};

// The four columns 4 (lane + LPR i) .. of a row; past E: -inf.  (Plain loads: the gradient may be
// written over the logits, each row by the lanes that have read it whole.)
template <int LPR>
__device__ __forceinline__ float4 load4(const float* row, int i, int sub, const Shape& s, bool on) {
  const int c = 4 * (sub + LPR * i);
  float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
  if (!on || c >= s.E) return v;
  if (s.vec) return *reinterpret_cast<const float4*>(row + c);
  v.x = row[c];
  if (c + 1 < s.E) v.y = row[c + 1];
  if (c + 2 < s.E) v.z = row[c + 2];
  if (c + 3 < s.E) v.w = row[c + 3];
  return v;
}

template <int LPR>
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// e^x for x <= 0 (0 from -150 on, -inf among it; NaN stays): 2^t, t = x log2 e, by the
// hardware's exponential (2^-22 relative), times 1 + ln 2 of what rounding t lost.  Seven
// instructions; exp_f32's twenty would take as long as the memory does.
__device__ __forceinline__ float exp_nonpos(float x) {
  x = x < -150.0f ? -150.0f : x;
  const float t = __fmul_rn(x, 1.44269502162933349609375f);
  float r = __fmaf_rn(x, 1.44269502162933349609375f, -t);
  r = __fmaf_rn(x, 1.925963033500011e-8f, r);  // log2 e less the constant above
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(t));
  return __fmaf_rn(y, __fmul_rn(r, 0.693147182464599609375f), y);
}

// Logits of this lane to probabilities, in place.  A row of -inf alone has p = 0; m: its maximum.
template <int LPR, int N>
__device__ __forceinline__ void softmax(float (&v)[N], float& m) {
  m = v[0];
#pragma unroll
  for (int j = 1; j < N; ++j) m = fmaxf(m, v[j]);
  m = row_max<LPR>(m);
  const float sub = m == -INFINITY ? 0.0f : m;
  float z = 0.0f;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    v[j] = exp_nonpos(__fsub_rn(v[j], sub));
    z = __fadd_rn(z, v[j]);
  }
  z = row_sum<LPR>(z);
  const float inv = z == 0.0f ? 0.0f : __frcp_rn(z);  // (NaN stays)
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = __fmul_rn(v[j], inv);
}

struct Sums {    // one entry a block of rows
  float* p;      // [blocks, E]
  int* counts;   // [blocks, E]
  int* tokens;   // [blocks]
  unsigned int* ticket;
  float* loss;   // [S * expert blocks]
};

__device__ __forceinline__ float term(int count, float sum, int n, const Shape& s, float* mean) {
  const float r = n > 0 ? __frcp_rn(static_cast<float>(n)) : 0.0f;
  *mean = __fmul_rn(sum, r);
  return static_cast<float>(count) * *mean * r;  // f mean k / E
}

// WHOLE: the one block of the one sequence also finishes (few rows: one launch).
template <int LPR, int NV, bool WHOLE>
__global__ void __launch_bounds__(kThreads) balance_rows_kernel(const float* logits, const int32_t* ids,
                                                                const uint8_t* valid, Shape s, Sums w, float coef,
                                                                float* loss, int* counts, float* mean, int* tokens) {
  constexpr int RPW = 32 / LPR, N = 4 * NV;
  constexpr int U = NV > 4 ? 1 : 8 / NV;  // rows a lane holds at once
  extern __shared__ float smem[];     // [kWarps][E] sums, then [E] counts
  int* cnt = reinterpret_cast<int*>(smem + kWarps * s.E);
  if (!WHOLE) grid_release_next();
  __shared__ int n_tok;
  __shared__ float red[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, sub = lane & (LPR - 1);
  for (int e = tid; e < s.E; e += kThreads) cnt[e] = 0;
  if (tid == 0) {
    n_tok = 0;
    if (!WHOLE && blockIdx.x == 0) *w.ticket = 0;
  }
  __syncthreads();
  const int seq = blockIdx.x / s.per, part = blockIdx.x - seq * s.per;
  const int64_t lo = static_cast<int64_t>(part) * s.chunk, hi = min(lo + s.chunk, s.L), row0 = seq * s.L;
  // pairs
  int mine = 0;
  const uint32_t pairs = hi > lo ? static_cast<uint32_t>((hi - lo) * s.k) : 0u, k = static_cast<uint32_t>(s.k);
  constexpr int P = 4;  // pairs whose loads are in flight together
  for (uint32_t i0 = tid; i0 < pairs; i0 += kThreads * P) {
    int e[P];
    bool on[P];
#pragma unroll
    for (int q = 0; q < P; ++q) {
      const uint32_t i = i0 + q * kThreads, r = i / k;
      on[q] = i < pairs && (!valid || __ldg(valid + row0 + lo + r));
      mine += on[q] && i - r * k == 0;
    }
#pragma unroll
    for (int q = 0; q < P; ++q) e[q] = on[q] ? __ldg(ids + (row0 + lo) * s.k + i0 + q * kThreads) : 0;
#pragma unroll
    for (int q = 0; q < P; ++q) {
      if (!on[q]) continue;
      if (e[q] >= 0 && e[q] < s.E) atomicAdd(cnt + e[q], 1);
      else raise_error(&g_err, MOE_DEVERR_BAD_EXPERT_ID);
    }
  }
  if (mine) atomicAdd(&n_tok, mine);
  // probabilities
  float acc[N];
#pragma unroll
  for (int j = 0; j < N; ++j) acc[j] = 0.0f;
  for (int64_t b = lo + warp * RPW * U; b < hi; b += kWarps * RPW * U) {
    float v[U][N];
    bool on[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = b + u * RPW + lane / LPR;
      on[u] = r < hi && (!valid || __ldg(valid + row0 + r));
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const float4 f = load4<LPR>(logits + (row0 + r) * s.E, i, sub, s, on[u]);
        v[u][4 * i] = f.x;
        v[u][4 * i + 1] = f.y;
        v[u][4 * i + 2] = f.z;
        v[u][4 * i + 3] = f.w;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float m;
      softmax<LPR>(v[u], m);  // (a row that does not count: p = 0)
#pragma unroll
      for (int j = 0; j < N; ++j) acc[j] = __fadd_rn(acc[j], v[u][j]);
    }
  }
#pragma unroll
  for (int o = LPR; o < 32; o <<= 1)
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] = __fadd_rn(acc[j], __shfl_xor_sync(0xffffffffu, acc[j], o));
  if (lane < LPR) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int c = 4 * (sub + LPR * (j >> 2)) + (j & 3);
      if (c < s.E) smem[warp * s.E + c] = acc[j];
    }
  }
  __syncthreads();
  const int n = n_tok;
  float part_loss = 0.0f;
  for (int e = tid; e < s.E; e += kThreads) {
    float sum = 0.0f;
#pragma unroll
    for (int q = 0; q < kWarps; ++q) sum = __fadd_rn(sum, smem[q * s.E + e]);
    if (WHOLE) {
      float me;
      part_loss += term(cnt[e], sum, n, s, &me);
      counts[e] = cnt[e];
      mean[e] = me;
    } else {
      w.p[static_cast<int64_t>(blockIdx.x) * s.E + e] = sum;
      w.counts[static_cast<int64_t>(blockIdx.x) * s.E + e] = cnt[e];
    }
  }
  if (WHOLE) {
    part_loss = row_sum<32>(part_loss);
    if (lane == 0) red[warp] = part_loss;
    __syncthreads();
    if (tid == 0) {
      float t = 0.0f;
#pragma unroll
      for (int q = 0; q < kWarps; ++q) t += red[q];
      *loss = t * coef * (static_cast<float>(s.E) / s.k);
      *tokens = n;
    }
  } else if (tid == 0) {
    w.tokens[blockIdx.x] = n;
  }
}

// Block (sequence, 32 experts): sums over the sequence's blocks of rows, warp q those of
// q, q + 32, ..; the last block to finish adds up the loss in order.
constexpr int kFinishWarps = 32;
__global__ void __launch_bounds__(32 * kFinishWarps) balance_finish_kernel(Shape s, Sums w, float coef, float* loss,
                                                                           int* counts, float* mean, int* tokens) {
  __shared__ float ps[kFinishWarps][32];
  __shared__ int cs[kFinishWarps][32], ts[kFinishWarps];
  __shared__ bool last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int seq = blockIdx.x, e = blockIdx.y * 32 + lane;
  grid_wait_previous();
  // (not __ldg: the kernel before wrote these while this one lived)
  const int64_t b0 = static_cast<int64_t>(seq) * s.per;
  float p = 0.0f;
  int c = 0, n = 0;
#pragma unroll 8
  for (int b = warp; b < s.per; b += kFinishWarps) {
    if (e < s.E) {
      p = __fadd_rn(p, __ldcg(w.p + (b0 + b) * s.E + e));
      c += __ldcg(w.counts + (b0 + b) * s.E + e);
    }
  }
  for (int b = threadIdx.x; b < s.per; b += 32 * kFinishWarps) n += __ldcg(w.tokens + b0 + b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  ps[warp][lane] = p;
  cs[warp][lane] = c;
  if (lane == 0) ts[warp] = n;
  __syncthreads();
  if (warp == 0) {
    p = 0.0f;
    c = 0;
    n = 0;
#pragma unroll
    for (int q = 0; q < kFinishWarps; ++q) {
      p = __fadd_rn(p, ps[q][lane]);
      c += cs[q][lane];
      n += ts[q];
    }
    float me = 0.0f;
    float t = term(c, p, n, s, &me);
    if (e < s.E) {
      counts[static_cast<int64_t>(seq) * s.E + e] = c;
      mean[static_cast<int64_t>(seq) * s.E + e] = me;
    } else {
      t = 0.0f;
    }
    t = row_sum<32>(t);
    if (lane == 0) {
      w.loss[seq * gridDim.y + blockIdx.y] = t;
      if (blockIdx.y == 0) tokens[seq] = n;
      __threadfence();
      last = atomicAdd(w.ticket, 1u) == gridDim.x * gridDim.y - 1;
    }
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  float t = 0.0f;
  for (int i = threadIdx.x; i < static_cast<int>(gridDim.x * gridDim.y); i += 32 * kFinishWarps) t += __ldcg(w.loss + i);
  t = row_sum<32>(t);
  if (lane == 0) ps[0][warp] = t;
  __syncthreads();
  if (threadIdx.x == 0) {
    t = 0.0f;
#pragma unroll
    for (int q = 0; q < kFinishWarps; ++q) t += ps[0][q];
    *loss = t * (coef / s.S) * (static_cast<float>(s.E) / s.k);
  }
}

// (NV == 6: 80 registers, so that three blocks are resident as in the other pass; 67 us for
// 65536 rows of 768 experts.)
template <int LPR, int NV>
__global__ void __launch_bounds__(kThreads, NV == 6 ? 3 : 1)
    balance_grad_kernel(const float* logits, const uint8_t* valid, Shape s, const int* counts, const int* tokens,
                        const float* grad, float coef, float* dlogits) {
  constexpr int RPW = 32 / LPR, N = 4 * NV;
  constexpr int U = NV > 2 ? 1 : 2;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane & (LPR - 1);
  const int seq = blockIdx.x / s.per, part = blockIdx.x - seq * s.per;
  const int64_t lo = static_cast<int64_t>(part) * s.chunk, hi = min(lo + s.chunk, s.L), row0 = seq * s.L;
  int cnt[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int c = 4 * (sub + LPR * (j >> 2)) + (j & 3);
    cnt[j] = c < s.E ? __ldg(counts + static_cast<int64_t>(seq) * s.E + c) : 0;
  }
  const float n = static_cast<float>(__ldg(tokens + seq));
  const float rn = n > 0.0f ? __frcp_rn(n) : 0.0f;
  const float factor = (grad ? __ldg(grad) : 1.0f) * (coef / s.S) * (static_cast<float>(s.E) / s.k) * rn * rn;
  for (int64_t b = lo + warp * RPW * U; b < hi; b += kWarps * RPW * U) {
    float v[U][N];
    bool on[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = b + u * RPW + lane / LPR;
      on[u] = r < hi && (!valid || __ldg(valid + row0 + r));
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const float4 f = load4<LPR>(logits + (row0 + r) * s.E, i, sub, s, on[u]);
        v[u][4 * i] = f.x;
        v[u][4 * i + 1] = f.y;
        v[u][4 * i + 2] = f.z;
        v[u][4 * i + 3] = f.w;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = b + u * RPW + lane / LPR;
      // the lane's own largest logit's count, then the row's (equal ones: the larger count)
      float x = v[u][0];
      int ref = cnt[0];
#pragma unroll
      for (int j = 1; j < N; ++j)
        if (v[u][j] > x) {
          x = v[u][j];
          ref = cnt[j];
        }
      float m;
      softmax<LPR>(v[u], m);
      ref = x == m ? ref : -1;
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) ref = max(ref, __shfl_xor_sync(0xffffffffu, ref, o));
      float d[N], t = 0.0f;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        d[j] = static_cast<float>(cnt[j] - ref);
        t = __fmaf_rn(v[u][j], d[j], t);
      }
      t = row_sum<LPR>(t);
      if (r >= hi) continue;
      float* out = dlogits + (row0 + r) * s.E;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = 4 * (sub + LPR * i);
        float o4[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          o4[j] = on[u] ? __fmul_rn(__fmul_rn(v[u][4 * i + j], __fsub_rn(d[4 * i + j], t)), factor) : 0.0f;
        if (s.vec) {
          if (c < s.E) *reinterpret_cast<float4*>(out + c) = make_float4(o4[0], o4[1], o4[2], o4[3]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (c + j < s.E) out[c + j] = o4[j];
        }
      }
    }
  }
}

// Lanes a row and loads a lane.  Two loads a lane where they do: half the lanes, so fewer
// shuffles a row and more rows an instruction than with one (32 x 8192 rows of 64 experts, both
// passes: 53 against 59 us).  Three between the powers of two, for lanes past the last expert do
// all the work of the others (65536 rows of 192 experts: 43 against 49 us; 131072 of 96: 43
// against 54; 32768 of 384: 45 against 53; six loads, 65536 of 768: 117 against 191).
template <class F>
cudaError_t by_width(int E, F&& f) {
  if (E <= 32) return f(std::integral_constant<int, 4>{}, std::integral_constant<int, 2>{});
  if (E <= 64) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 2>{});
  if (E <= 96) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 3>{});
  if (E <= 128) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 2>{});
  if (E <= 192) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 3>{});
  if (E <= 256) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 2>{});
  if (E <= 384) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 3>{});
  if (E <= 512) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 4>{});
  if (E <= 768) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 6>{});
  return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 8>{});
}

// Blocks at most: those that 152 multiprocessors hold at once, by the registers of a row's
// columns (both passes: 32768 rows of 512 experts 57 us with three a multiprocessor, 59 with
// four; 65536 of 768 117 and 144; 65536 of 1000 189 with two, 201 with four).
int blocks_for(int E) { return 152 * (E <= 384 ? 4 : E <= 768 ? 3 : 2); }
constexpr int kMinChunk = 32;

bool make_shape(int64_t T, int E, int k, int64_t S, Shape* s) {
  if (T < 0 || S < 1 || S > (1 << 20) || T % S || E < 1 || E > kMaxE || k < 1 || k > kMaxK || T > ((1ll << 31) - 1) / k) return false;
  s->L = T / S;
  s->S = static_cast<int>(S);
  s->E = E;
  s->k = k;
  const int64_t per = std::max<int64_t>(1, std::min<int64_t>(blocks_for(E) / S, (s->L + kMinChunk - 1) / kMinChunk));
  s->chunk = static_cast<int>(std::max<int64_t>(1, (s->L + per - 1) / per));
  s->per = static_cast<int>(std::max<int64_t>(1, (s->L + s->chunk - 1) / s->chunk));
  return true;
}

size_t workspace(const Shape& s, Sums* w, void* base) {
  const int64_t blocks = static_cast<int64_t>(s.S) * s.per, eb = (s.E + 31) / 32;
  const int64_t n[5] = {blocks * s.E, blocks * s.E, blocks, s.S * eb, 1};
  int64_t off[6] = {0};
  for (int i = 0; i < 5; ++i) off[i + 1] = off[i] + (n[i] + 3) / 4 * 4;
  if (w) {
    int* b = static_cast<int*>(base);
    *w = Sums{reinterpret_cast<float*>(b), b + off[1], b + off[2], reinterpret_cast<unsigned int*>(b + off[4]),
              reinterpret_cast<float*>(b + off[3])};
  }
  return static_cast<size_t>(off[5]) * 4;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" __attribute__((visibility("hidden"))) cudaError_t moe_detail_take_error_balance(unsigned int* out) {
  unsigned int v = 0, z = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_err, sizeof(v));
  if (e == cudaSuccess && v) e = cudaMemcpyToSymbol(g_err, &z, sizeof(z));
  *out = v;
  return e;
}

extern "C" size_t moe_router_balance_workspace_bytes(int64_t T, int E, int k, int64_t seqs) {
  Shape s;
  return make_shape(T, E, k, seqs, &s) ? workspace(s, nullptr, nullptr) : 0;
}

extern "C" moe_status moe_router_balance(const float* logits, const int32_t* topk_ids, const uint8_t* valid, int64_t T,
                                         int E, int k, int64_t seqs, float coef, float* loss, int32_t* counts,
                                         float* mean, int32_t* tokens, void* ws, size_t ws_bytes,
                                         moe_stream_t stream) {
  MOE_HOST_CHECK(loss && counts && mean && tokens && ws && (T == 0 || (logits && topk_ids)), MOE_ERR_INVALID_ARG);
  Shape s;
  MOE_HOST_CHECK(make_shape(T, E, k, seqs, &s), MOE_ERR_INVALID_ARG);
  MOE_HOST_CHECK(aligned16(logits) && aligned16(ws) && ws_bytes >= workspace(s, nullptr, nullptr), MOE_ERR_INVALID_ARG);
  cudaStream_t st = as_stream(stream);
  s.vec = E % 4 == 0;
  Sums w;
  workspace(s, &w, ws);
  const size_t smem = static_cast<size_t>(kWarps + 1) * E * 4;
  const bool whole = s.S == 1 && s.per == 1;
  const unsigned blocks = static_cast<unsigned>(s.S) * s.per;
  MOE_CUDA_TRY(by_width(E, [&](auto lpr, auto nv) {
    constexpr int LPR = decltype(lpr)::value, NV = decltype(nv)::value;
    if (whole)
      balance_rows_kernel<LPR, NV, true>
          <<<blocks, kThreads, smem, st>>>(logits, topk_ids, valid, s, w, coef, loss, counts, mean, tokens);
    else
      balance_rows_kernel<LPR, NV, false>
          <<<blocks, kThreads, smem, st>>>(logits, topk_ids, valid, s, w, coef, loss, counts, mean, tokens);
    return cudaGetLastError();
  }));
  if (!whole) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(s.S, (E + 31) / 32);
    cfg.blockDim = dim3(32 * kFinishWarps);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    MOE_CUDA_TRY(cudaLaunchKernelEx(&cfg, balance_finish_kernel, s, w, coef, loss, counts, mean, tokens));
  }
  return MOE_OK;
}

extern "C" moe_status moe_router_balance_backward(const float* logits, const uint8_t* valid, int64_t T, int E, int k,
                                                  int64_t seqs, float coef, const int32_t* counts,
                                                  const int32_t* tokens, const float* grad, float* dlogits,
                                                  moe_stream_t stream) {
  Shape s;
  MOE_HOST_CHECK(make_shape(T, E, k, seqs, &s), MOE_ERR_INVALID_ARG);
  MOE_HOST_CHECK(counts && tokens && (T == 0 || (logits && dlogits)) && aligned16(logits) && aligned16(dlogits),
                 MOE_ERR_INVALID_ARG);
  if (T == 0) return MOE_OK;
  s.vec = E % 4 == 0;
  cudaStream_t st = as_stream(stream);
  MOE_CUDA_TRY(by_width(E, [&](auto lpr, auto nv) {
    balance_grad_kernel<decltype(lpr)::value, decltype(nv)::value><<<static_cast<unsigned>(s.S) * s.per, kThreads, 0, st>>>(
        logits, valid, s, counts, tokens, grad, coef, dlogits);
    return cudaGetLastError();
  }));
  return MOE_OK;
}
