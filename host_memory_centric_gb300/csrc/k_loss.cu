// k_loss.cu -- losses of the training step and their gradients (sm_103a).
//
// Linear cross-entropy (the LM head and its loss without the logits),
// distillation from a teacher's top logits, and the balance loss of a routed
// mixture of experts.  Statistics, sums and losses are FP32; gradients are
// rounded to BF16 once, where they are written.  No sum depends on the order
// of atomics, so the same inputs give the same bits.
#include "mt_kernels.h"

namespace mt {
namespace {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ void unpack8(const uint4& q, float (&f)[8]) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&q);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 t = __bfloat1622float2(h[k]);
    f[2 * k] = t.x;
    f[2 * k + 1] = t.y;
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint4 q;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&q);
#pragma unroll
  for (int k = 0; k < 4; ++k) h[k] = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
  return q;
}
// Sum and maximum over a block of NT threads, the warps' parts combined in
// warp order; every thread gets the result.  red: NT / 32 floats.
template <int NT>
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.f;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) t += red[w];
  return t;
}
template <int NT>
__device__ __forceinline__ float block_max(float v, float* red) {
  v = warp_max(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = -INFINITY;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) t = fmaxf(t, red[w]);
  return t;
}

// ------------------------------------------------------------------ linear cross-entropy
// One block per row: joins the row's pieces (m_p, s_p), whose sums leave the
// target out, with M = max m_p:
//   rest = sum_p s_p exp(m_p - M),  S = rest + exp(z_target - M),
//   loss = (M - z_target) + log S,
// and, with E, turns the stored exp(z - m_p) into the logits' gradient in
// place: d = E exp(m_p - M) / S g, one factor per piece of 256 columns, and
// d = -rest / S g (= (p - 1) g) at the target, so that loss and gradient of a
// confident row (p near 1) keep their digits.  Rows without a target get zeros.
constexpr int JOIN_THREADS = 256;

__global__ void __launch_bounds__(JOIN_THREADS) ce_join_k(const float2* __restrict__ stat, int npieces,
                                                          const int32_t* __restrict__ target,
                                                          const float* __restrict__ zt, int V, float g,
                                                          float* __restrict__ row_loss, bf16* __restrict__ E,
                                                          int64_t ldE) {
  extern __shared__ float f[];  // [npieces]
  __shared__ float red[JOIN_THREADS / 32];
  const int64_t row = blockIdx.x;
  const int tgt = target[row];
  const bool has = tgt >= 0 && tgt < V;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (!has) {
    if (threadIdx.x == 0) row_loss[row] = 0.f;
    if (E)
      for (int64_t c = threadIdx.x * 8; c < V; c += JOIN_THREADS * 8)
        *reinterpret_cast<uint4*>(E + row * ldE + c) = make_uint4(0, 0, 0, 0);
    return;
  }
  const float2* st = stat + row * npieces;
  float m = -INFINITY;
  for (int p = threadIdx.x; p < npieces; p += JOIN_THREADS) m = fmaxf(m, st[p].x);
  const float M = block_max<JOIN_THREADS>(m, red);
  float s = 0.f;
  for (int p = threadIdx.x; p < npieces; p += JOIN_THREADS) s += st[p].y * expf(st[p].x - M);
  const float rest = block_sum<JOIN_THREADS>(s, red);
  const float z = zt[row], et = expf(z - M), S = rest + et;
  if (threadIdx.x == 0) row_loss[row] = z == M ? log1pf(rest) : (M - z) + logf(S);
  if (!E) return;
  for (int p = threadIdx.x; p < npieces; p += JOIN_THREADS) f[p] = expf(st[p].x - M) / S * g;
  __syncthreads();
  const float dt = -rest / S * g;
  bf16* e = E + row * ldE;
  for (int p = warp; p < npieces; p += JOIN_THREADS / 32) {  // a warp's 32 vectors are one piece
    const int c = p * 256 + lane * 8;
    if (c >= V) continue;
    float v[8];
    unpack8(*reinterpret_cast<const uint4*>(e + c), v);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = c + k == tgt ? dt : v[k] * f[p];
    *reinterpret_cast<uint4*>(e + c) = pack8(v);
  }
}

// ------------------------------------------------------------------ distillation
// One block per row of student logits z, teacher logits y at ids i:
//   q = softmax over the filled slots of y / tau, p = softmax(z / tau),
//   kd = sum_j q_j (log q_j - log p_{i_j}),  ce = lse(z) - z_target,
//   dz_v = w_ce (softmax(z)_v - [v = target]) + w_kd / tau (p_v - sum_{i_j = v} q_j).
// The row is read twice (the second time from L2): statistics at both
// temperatures, then the dense part of the gradient; the at most K + 1 columns
// with a teacher entry or the target are then written again from their logits
// kept in FP32, each by one thread, so that no element is rounded twice and an
// id that appears in several slots gets the sum of their q.
constexpr int KD_THREADS = 512;
constexpr int KD_MAX_K = 1024;

struct RunningSum {  // sum of exp(a (z - m)) at two scales a around one running maximum m
  float m = -INFINITY, s1 = 0.f, st = 0.f;
  __device__ __forceinline__ void add(float z, float it) {
    if (z > m) {
      s1 = m == -INFINITY ? 1.f : s1 * expf(m - z) + 1.f;
      st = m == -INFINITY ? 1.f : st * expf((m - z) * it) + 1.f;
      m = z;
    } else if (m != -INFINITY || z != z) {
      s1 += expf(z - m);
      st += expf((z - m) * it);
    }
  }
};

__global__ void __launch_bounds__(KD_THREADS) distill_k(const bf16* logits, const int32_t* __restrict__ target,
                                                        const float* __restrict__ t_val,
                                                        const int32_t* __restrict__ t_idx, int V, int K, float tau,
                                                        float w_ce, float w_kd, float* __restrict__ row_ce,
                                                        float* __restrict__ row_kd, bf16* dlogits) {
  __shared__ float red[KD_THREADS / 32];
  __shared__ int id[KD_MAX_K];
  __shared__ float y[KD_MAX_K], q[KD_MAX_K], zj[KD_MAX_K];
  const int64_t row = blockIdx.x;
  const bf16* z = logits + row * V;
  const float it = 1.f / tau;
  const int tid = threadIdx.x;
  const int tgt = target ? target[row] : -1;
  const bool hard = tgt >= 0 && tgt < V;
  const float zt = hard ? __bfloat162float(z[tgt]) : 0.f;
  float ym = -INFINITY;
  for (int j = tid; j < K; j += KD_THREADS) {
    const int i = t_idx[row * K + j];
    const bool in = i >= 0 && i < V;
    const float v = in ? t_val[row * K + j] * it : -INFINITY;
    id[j] = in ? i : -1;
    y[j] = v;
    zj[j] = in ? __bfloat162float(z[i]) : 0.f;
    ym = fmaxf(ym, v);
  }
  ym = block_max<KD_THREADS>(ym, red);
  const bool soft = ym != -INFINITY;
  float ys = 0.f;
  for (int j = tid; j < K; j += KD_THREADS) {
    const float v = id[j] < 0 || !soft ? 0.f : expf(y[j] - ym);
    q[j] = v;
    ys += v;
  }
  ys = block_sum<KD_THREADS>(ys, red);
  const float yl = logf(ys);

  RunningSum r;
  for (int c = tid; c < V; c += KD_THREADS) r.add(__bfloat162float(z[c]), it);
  const float m = block_max<KD_THREADS>(r.m, red);
  const float f1 = r.m == -INFINITY ? 0.f : expf(r.m - m), ft = r.m == -INFINITY ? 0.f : expf((r.m - m) * it);
  // log p = (z - m) / tau - log sum exp((z - m) / tau): differences first, so
  // that the size of the logits costs no digits
  const float l1 = logf(block_sum<KD_THREADS>(r.s1 * f1, red));
  const float lt = logf(block_sum<KD_THREADS>(r.st * ft, red));

  float kd = 0.f;
  for (int j = tid; j < K; j += KD_THREADS) {
    if (id[j] < 0 || !soft || q[j] == 0.f) continue;
    q[j] /= ys;
    kd += q[j] * ((y[j] - ym - yl) - ((zj[j] - m) * it - lt));
  }
  kd = block_sum<KD_THREADS>(kd, red);
  if (tid == 0) {
    row_kd[row] = soft ? kd : 0.f;
    if (row_ce) row_ce[row] = hard ? l1 - (zt - m) : 0.f;
  }
  if (!dlogits) return;
  bf16* d = dlogits + row * V;
  const float a1 = hard ? w_ce : 0.f, at = soft ? w_kd * it : 0.f;
  auto grad = [&](float x) {
    float v = 0.f;
    if (hard) v += a1 * expf((x - m) - l1);
    if (soft) v += at * expf((x - m) * it - lt);
    return v;
  };
  for (int c = tid; c < V; c += KD_THREADS) d[c] = __float2bfloat16_rn(grad(__bfloat162float(z[c])));
  __syncthreads();
  for (int j = tid; j <= K; j += KD_THREADS) {  // slot K: the target, if no slot names it
    const int i = j < K ? id[j] : (hard ? tgt : -1);
    if (i < 0 || (j < K && !soft && i != tgt)) continue;
    bool first = true;
    float qs = 0.f;
    for (int u = 0; u < K; ++u) {
      if (id[u] != i) continue;
      if (u < j) first = false;
      qs += q[u];
    }
    if (!first) continue;
    const float x = j < K ? zj[j] : zt;
    float v = 0.f;
    if (hard) v += a1 * (i == tgt ? expm1f((x - m) - l1) : expf((x - m) - l1));
    if (soft) v += at * (expf((x - m) * it - lt) - qs);
    d[i] = __float2bfloat16_rn(v);
  }
}

// ------------------------------------------------------------------ router balance
// Groups of S tokens, n valid ones each, c[e] of their n k choices going to expert e, f = c / (n k):
//   balance = alpha E / G sum_g sum_e f_e P_e, P_e = mean over valid t of p_te = softmax(logits_t)_e,
//   z loss  = zc / G sum_g mean over valid t of lse_t^2,
//   dlogit_te = alpha E / (G n) p_te (f_e - sum_j f_j p_tj) + 2 zc / (G n) lse_t p_te.
constexpr int BAL_THREADS = 256;
constexpr int BAL_MAX_E = 512;

// Choices per expert and valid tokens of one group per block.
__global__ void __launch_bounds__(BAL_THREADS) balance_count_k(const int32_t* __restrict__ idx,
                                                               const uint8_t* __restrict__ valid, int S, int E, int k,
                                                               int32_t* __restrict__ counts, int32_t* __restrict__ n) {
  __shared__ int c[BAL_MAX_E + 1];
  const int64_t g = blockIdx.x;
  for (int e = threadIdx.x; e <= E; e += BAL_THREADS) c[e] = 0;
  __syncthreads();
  for (int64_t i = threadIdx.x; i < (int64_t)S * k; i += BAL_THREADS) {
    const int64_t t = g * S + i / k;
    if (valid && !valid[t]) continue;
    if (i % k == 0) atomicAdd(&c[E], 1);
    const int e = idx[g * S * k + i];
    if (e >= 0 && e < E) atomicAdd(&c[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += BAL_THREADS) counts[g * E + e] = c[e];
  if (threadIdx.x == 0) n[g] = c[E];
}

// Rows [b rows, (b + 1) rows) of a group per block: the rows' gradient, one warp
// per row, and the block's sums of p and lse^2 (partial: [G][blocks][E + 1]).
__global__ void __launch_bounds__(BAL_THREADS) balance_grad_k(const float* __restrict__ logits,
                                                              const uint8_t* __restrict__ valid, int S, int E, int k,
                                                              int rows, float alpha_g, float zc_g,
                                                              const int32_t* __restrict__ counts,
                                                              const int32_t* __restrict__ n, bf16* __restrict__ dlogits,
                                                              float* __restrict__ partial) {
  __shared__ float f[BAL_MAX_E];
  __shared__ float acc[BAL_THREADS / 32][BAL_MAX_E + 1];
  const int64_t g = blockIdx.y;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float inv_n = n[g] > 0 ? 1.f / (float)n[g] : 0.f;
  for (int e = threadIdx.x; e < E; e += BAL_THREADS) f[e] = (float)counts[g * E + e] * inv_n / (float)k;
  for (int e = lane; e <= E; e += 32) acc[warp][e] = 0.f;
  __syncthreads();
  const float cb = alpha_g * (float)E * inv_n, cz = 2.f * zc_g * inv_n;
  const int r1 = min(S, (int)(blockIdx.x + 1) * rows);
  for (int r = blockIdx.x * rows + warp; r < r1; r += BAL_THREADS / 32) {
    const int64_t t = g * S + r;
    const float* z = logits + t * E;
    bf16* d = dlogits ? dlogits + t * E : nullptr;
    if (valid && !valid[t]) {
      if (d)
        for (int e = lane; e < E; e += 32) d[e] = __float2bfloat16_rn(0.f);
      continue;
    }
    float v[BAL_MAX_E / 32], m = -INFINITY, s = 0.f, mean = 0.f;
#pragma unroll
    for (int j = 0; j < BAL_MAX_E / 32; ++j) {
      v[j] = j * 32 + lane < E ? z[j * 32 + lane] : -INFINITY;
      m = fmaxf(m, v[j]);
    }
    m = warp_max(m);
#pragma unroll
    for (int j = 0; j < BAL_MAX_E / 32; ++j)
      if (j * 32 + lane < E) {
        v[j] = expf(v[j] - m);
        s += v[j];
      }
    s = warp_sum(s);
    const float lse = m + logf(s), is = 1.f / s;
#pragma unroll
    for (int j = 0; j < BAL_MAX_E / 32; ++j)
      if (j * 32 + lane < E) {
        v[j] *= is;
        mean += f[j * 32 + lane] * v[j];
        acc[warp][j * 32 + lane] += v[j];
      }
    mean = warp_sum(mean);
    if (lane == 0) acc[warp][E] += lse * lse;
    if (d) {
#pragma unroll
      for (int j = 0; j < BAL_MAX_E / 32; ++j)
        if (j * 32 + lane < E)
          d[j * 32 + lane] = __float2bfloat16_rn(v[j] * (cb * (f[j * 32 + lane] - mean) + cz * lse));
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += BAL_THREADS) {
    float a = 0.f;
#pragma unroll
    for (int w = 0; w < BAL_THREADS / 32; ++w) a += acc[w][e];
    partial[(g * gridDim.x + blockIdx.x) * (E + 1) + e] = a;
  }
}

// Group sums of the blocks' partials in block order: prob, and the group's two losses.
__global__ void __launch_bounds__(BAL_THREADS) balance_group_k(const float* __restrict__ partial, int nblk, int E, int k,
                                                               const int32_t* __restrict__ counts,
                                                               const int32_t* __restrict__ n, float* __restrict__ prob,
                                                               float2* __restrict__ gloss) {
  __shared__ float red[BAL_THREADS / 32];
  const int64_t g = blockIdx.x;
  const float inv_n = n[g] > 0 ? 1.f / (float)n[g] : 0.f;
  float lb = 0.f, lz = 0.f;
  for (int e = threadIdx.x; e <= E; e += BAL_THREADS) {
    float a = 0.f;
    for (int b = 0; b < nblk; ++b) a += partial[(g * nblk + b) * (E + 1) + e];
    a *= inv_n;
    if (e < E) {
      prob[g * E + e] = a;
      lb += (float)counts[g * E + e] * inv_n / (float)k * a;
    } else {
      lz = a;
    }
  }
  lb = block_sum<BAL_THREADS>(lb, red);
  lz = block_sum<BAL_THREADS>(lz, red);
  if (threadIdx.x == 0) gloss[g] = make_float2(lb, lz);
}

__global__ void __launch_bounds__(BAL_THREADS) balance_loss_k(const float2* __restrict__ gloss, int64_t G,
                                                              float scale_b, float scale_z, float* __restrict__ loss) {
  __shared__ float red[BAL_THREADS / 32];
  float b = 0.f, z = 0.f;
  for (int64_t g = threadIdx.x; g < G; g += BAL_THREADS) {
    b += gloss[g].x;
    z += gloss[g].y;
  }
  b = block_sum<BAL_THREADS>(b, red);
  z = block_sum<BAL_THREADS>(z, red);
  if (threadIdx.x == 0) {
    loss[0] = b * scale_b;
    loss[1] = z * scale_z;
  }
}

inline bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
inline int64_t up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

// Tokens a linear cross-entropy call keeps the exponentials of at a time: as
// many as fit kPieceBytes, at least 1024 (a chunk re-reads the weights for
// every product, so short chunks are bound by memory), the chunks of one call
// equal up to the 256-row tile.
constexpr int64_t kPieceBytes = (int64_t)1 << 30;
int64_t ce_chunk(int64_t T, int V) {
  int64_t most = kPieceBytes / (2 * up(V, 64)) / 256 * 256;
  if (most < 1024) most = 1024;
  if (T <= most) return T;
  const int64_t n = (T + most - 1) / most;
  return up((T + n - 1) / n, 256);
}

struct CeScratch {
  int* ctr;
  float2* stat;
  float* zt;
  bf16* E;
  float* dWacc;
  int64_t ldE, chunk;
  int npieces;
};
size_t ce_carve(int64_t T, int H, int V, bool grads, uint8_t* base, CeScratch* w) {
  size_t off = 0;
  auto take = [&](int64_t bytes) {
    uint8_t* p = base ? base + off : nullptr;
    off += (size_t)up(bytes, 256);
    return p;
  };
  w->chunk = ce_chunk(T, V);
  w->npieces = (V + 255) / 256;
  w->ldE = up(V, 64);
  w->ctr = (int*)take(256);
  w->stat = (float2*)take(w->chunk * w->npieces * 8);
  w->zt = (float*)take(w->chunk * 4);
  w->E = grads ? (bf16*)take(w->chunk * w->ldE * 2) : nullptr;
  w->dWacc = grads && w->chunk < T ? (float*)take((int64_t)V * H * 4) : nullptr;
  return off;
}
bool ce_shape_ok(int64_t T, int H, int V) {
  return T >= 0 && T <= ((int64_t)1 << 40) && H > 0 && H % 8 == 0 && V > 0 && V <= (1 << 21);
}

struct BalScratch {
  int32_t* n;
  float2* gloss;
  float* partial;
  int nblk, rows;
};
size_t bal_carve(int64_t T, int S, int E, uint8_t* base, BalScratch* w) {
  size_t off = 0;
  auto take = [&](int64_t bytes) {
    uint8_t* p = base ? base + off : nullptr;
    off += (size_t)up(bytes, 256);
    return p;
  };
  const int64_t G = T / S;
  int64_t blk = (608 + G - 1) / G;  // about four blocks per SM in all
  const int64_t most = (S + 7) / 8;
  if (blk > most) blk = most;
  w->rows = (int)((S + blk - 1) / blk);
  w->nblk = (S + w->rows - 1) / w->rows;
  w->n = (int32_t*)take(G * 4);
  w->gloss = (float2*)take(G * 8);
  w->partial = (float*)take(G * w->nblk * (E + 1) * 4);
  return off;
}
bool bal_shape_ok(int64_t T, int S, int E) {
  return T >= 0 && S > 0 && T % S == 0 && T / S <= 65535 && E >= 1 && E <= BAL_MAX_E;
}

}  // namespace

// ------------------------------------------------------------------ launchers
size_t linear_cross_entropy_scratch(int64_t T, int H, int V, bool grads) {
  if (!ce_shape_ok(T, H, V)) return 0;
  CeScratch w;
  return ce_carve(T, H, V, grads, nullptr, &w);
}

cudaError_t linear_cross_entropy(const bf16* h, const bf16* W, const int32_t* target, int64_t T, int H, int V, float g,
                                 float* row_loss, bf16* dh, bf16* dW, void* scratch, size_t scratch_bytes,
                                 cudaStream_t s) {
  const bool grads = dh || dW;
  if (!ce_shape_ok(T, H, V) || !al16(h) || !al16(W) || !al16(dh) || !al16(dW) ||
      (reinterpret_cast<uintptr_t>(scratch) & 255))
    return cudaErrorInvalidValue;
  CeScratch w;
  if (ce_carve(T, H, V, grads, (uint8_t*)scratch, &w) > scratch_bytes) return cudaErrorInvalidValue;
  if (T == 0) return cudaSuccess;
  cudaError_t e = cudaMemsetAsync(w.ctr, 0, 256, s);
  if (e != cudaSuccess) return e;
  for (int64_t c0 = 0; c0 < T; c0 += w.chunk) {
    const int rows = (int)(T - c0 < w.chunk ? T - c0 : w.chunk);
    const bool first = c0 == 0, last = c0 + rows >= T;
    const SoftmaxPieces sp{w.stat, w.npieces, target + c0, w.zt, w.E, w.ldE};
    e = gemm_softmax_pieces(h + c0 * H, W, rows, V, H, sp, w.ctr, s);
    if (e != cudaSuccess) return e;
    ce_join_k<<<rows, JOIN_THREADS, w.npieces * sizeof(float), s>>>(w.stat, w.npieces, target + c0, w.zt, V, g,
                                                                    row_loss + c0, w.E, w.ldE);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (!grads) continue;
    GemmArgs gd{w.E, w.ldE, 0, W, H, 1, rows, H, V, dh ? dh + c0 * H : nullptr, H, nullptr, 0, nullptr, 0, 0};
    GemmArgs gw{w.E, w.ldE, 1, h + c0 * H, H, 1, V, H, rows, last ? dW : nullptr, H, nullptr, 0, nullptr, H, 0};
    if (w.dWacc) {
      gw.Dacc = w.dWacc;
      gw.acc_mode = first ? 1 : 2;
    }
    if (dh && dW) e = gemm_grads(gd, gw, w.ctr, s);
    else e = gemm_one(dh ? gd : gw, w.ctr, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t distill_topk(const bf16* logits, const int32_t* target, const float* t_val, const int32_t* t_idx,
                         int64_t rows, int V, int K, float tau, float w_ce, float w_kd, float* row_ce, float* row_kd,
                         bf16* dlogits, cudaStream_t s) {
  if (rows < 0 || rows > 0x7fffffff || V < 1 || K < 1 || K > KD_MAX_K || !(tau > 0.f) || !(tau < INFINITY) || !(1.f / tau < INFINITY) || !al16(logits) ||
      !al16(dlogits))
    return cudaErrorInvalidValue;
  if (rows == 0) return cudaSuccess;
  distill_k<<<(unsigned)rows, KD_THREADS, 0, s>>>(logits, target, t_val, t_idx, V, K, tau, w_ce, w_kd, row_ce, row_kd,
                                                  dlogits);
  return cudaGetLastError();
}

size_t router_balance_scratch(int64_t T, int S, int E) {
  if (!bal_shape_ok(T, S, E) || T == 0) return 0;
  BalScratch w;
  return bal_carve(T, S, E, nullptr, &w);
}

cudaError_t router_balance(const float* logits, const int32_t* idx, const uint8_t* valid, int64_t T, int S, int E,
                           int k, float alpha, float z_coef, float* loss, int32_t* counts, float* prob, bf16* dlogits,
                           void* scratch, size_t scratch_bytes, cudaStream_t s) {
  if (!bal_shape_ok(T, S, E) || k < 1 || k > E || (int64_t)S * k > 0x7fffffff || !al16(logits) || !al16(dlogits) ||
      (reinterpret_cast<uintptr_t>(scratch) & 255))
    return cudaErrorInvalidValue;
  if (T == 0) return cudaSuccess;
  BalScratch w;
  if (bal_carve(T, S, E, (uint8_t*)scratch, &w) > scratch_bytes) return cudaErrorInvalidValue;
  const int64_t G = T / S;
  const float per_group = 1.f / (float)G;
  balance_count_k<<<(unsigned)G, BAL_THREADS, 0, s>>>(idx, valid, S, E, k, counts, w.n);
  balance_grad_k<<<dim3((unsigned)w.nblk, (unsigned)G), BAL_THREADS, 0, s>>>(
      logits, valid, S, E, k, w.rows, alpha * per_group, z_coef * per_group, counts, w.n, dlogits, w.partial);
  balance_group_k<<<(unsigned)G, BAL_THREADS, 0, s>>>(w.partial, w.nblk, E, k, counts, w.n, prob, w.gloss);
  balance_loss_k<<<1, BAL_THREADS, 0, s>>>(w.gloss, G, alpha * per_group * (float)E, z_coef * per_group, loss);
  return cudaGetLastError();
}

}  // namespace mt
