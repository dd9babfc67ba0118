// k_loss.cu -- losses of the training step and their gradients (sm_103a).
//
// Linear cross-entropy (the LM head and its loss without the logits),
// distillation from a teacher's top logits, and the balance loss of a routed
// mixture of experts.  Statistics, sums and losses are FP32; gradients are
// rounded to BF16 once, where they are written.  No sum depends on the order
// of atomics, so the same inputs give the same bits.
#include "mt_kernels.h"

#include <cuda_fp16.h>

#include <atomic>

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

__device__ __forceinline__ uint32_t su32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A kernel launched with programmatic serialisation may start while the one
// before it runs; it sees that one's writes after dep_wait().
__device__ __forceinline__ void dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void dep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Two FP32 values in a register pair: one instruction for both
// (fma / add / mul.f32x2), each rounded as the single form rounds it.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair2(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpair2(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 wide2(uint32_t w) {  // the two BF16 values of a word
  return pair2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ f32x2 ex2_2(f32x2 v) {
  const float2 t = unpair2(v);
  return pair2(ex2(t.x), ex2(t.y));
}

// A bounded wait of this file's kernels ran out (0: none did).
__device__ int g_loss_error = 0;
constexpr long long kWaitCycles = 4000000000LL;  // about 2 s at 2 GHz

__device__ __forceinline__ void mbar_init(uint64_t* b, uint32_t n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(su32(b)), "r"(n));
}
__device__ __forceinline__ void mbar_expect_tx(uint64_t* b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(su32(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(su32(b)) : "memory");
}
__device__ __forceinline__ bool mbar_test(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(su32(b)), "r"(parity)
      : "memory");
  return ok != 0;
}
// Bounded wait; once one ran out (recorded in g_loss_error: the outputs are not
// valid) this thread waits for nothing more, so that the kernel ends.
__device__ __forceinline__ void mbar_wait(uint64_t* b, uint32_t parity, bool& failed) {
  if (failed || mbar_test(b, parity)) return;
  const long long t0 = clock64();
  while (!mbar_test(b, parity)) {
    if (clock64() - t0 > kWaitCycles) {
      failed = true;
      atomicCAS(&g_loss_error, 0, 4);
      return;
    }
  }
}
// n bytes (a multiple of 16) from global to shared memory, both 16-byte
// aligned; their arrival completes on the barrier
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t n, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(su32(dst)),
               "l"(src), "r"(n), "r"(su32(bar))
               : "memory");
}
// Between this thread's loads from a stage of a ring of such copies and the
// barrier that frees it.  The barrier orders plain accesses only; without the
// fence the next copy came before loads that stood in a queue behind stores
// (8192 rows of 32000 columns: 20 to 60 thousand elements of the gradient were
// those of a later chunk).  Distillation is as fast with it; the balance loss of
// 131072 tokens of 128 experts takes 0.7 us more.
__device__ __forceinline__ void reads_before_copies() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void async_load4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(su32(dst)), "l"(src) : "memory");
}

// ------------------------------------------------------------------ linear cross-entropy
// One block per row: joins the row's pieces (m_p, s_p), whose sums leave the
// target out, with M = max m_p:
//   rest = sum_p s_p exp(m_p - M),  S = rest + exp(z_target - M),
//   loss = (M - z_target) + log S,
// and, with E, turns the stored fp16 2^15 exp(z - m_p) into the logits'
// gradient in BF16 in place: d = exp(z - m_p) exp(m_p - M) / S, one factor per
// piece of 128 columns, and d = -rest / S (= p - 1) at the target, so that loss
// and gradient of a confident row (p near 1) keep their digits.  The factor g
// of the gradients waits for the products' FP32 results: rounded here, g (p - 1)
// of most rows would be off by the same amount, and the errors would add up.
// Rows without a target get zeros, and zeros in hm too, a copy of h for dW = d^T
// h: what padding holds may be no number, and 0 times that would not be 0.
// Bound by HBM (4 bytes a logit; 8192 rows of 32000: 199 us, 5.3 TB/s).  The
// blocks of grid.y share a row; each joins the statistics for itself.
constexpr int JOIN_THREADS = 256;

__global__ void __launch_bounds__(JOIN_THREADS) ce_join_k(const float2* __restrict__ stat, int npieces,
                                                          const int32_t* __restrict__ target,
                                                          const float* __restrict__ zt, int V,
                                                          float* __restrict__ row_loss, uint16_t* __restrict__ E,
                                                          int64_t ldE, const bf16* __restrict__ h,
                                                          bf16* __restrict__ hm, int H) {
  __shared__ float red[JOIN_THREADS / 32];
  dep_launch();
  dep_wait();
  const int64_t row = blockIdx.x;
  const int tgt = target[row];
  const bool has = tgt >= 0 && tgt < V;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (hm && blockIdx.y == 0)
    for (int i = threadIdx.x; i < H / 8; i += JOIN_THREADS)
      reinterpret_cast<uint4*>(hm + row * H)[i] =
          has ? reinterpret_cast<const uint4*>(h + row * H)[i] : make_uint4(0, 0, 0, 0);
  uint4* e = reinterpret_cast<uint4*>(E + row * ldE);
  const int nvec = (V + 7) / 8, step = 32 * (JOIN_THREADS / 32) * (int)gridDim.y;
  const int first = ((int)blockIdx.y * (JOIN_THREADS / 32) + warp) * 32 + lane;
  if (!has) {
    if (threadIdx.x == 0 && blockIdx.y == 0) row_loss[row] = 0.f;
    if (E)
      for (int v = first; v < nvec; v += step) e[v] = make_uint4(0, 0, 0, 0);
    return;
  }
  // the first vectors are on their way while the statistics are joined
  const float2* st = stat + row * npieces;
  constexpr int U = 4;  // vectors of a thread on their way at a time
  uint4 q[U];
  float f[U];
  auto load = [&](int v) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int w = v + u * step;
      if (w < nvec) {
        q[u] = e[w];
        f[u] = st[w >> 4].x;
      }
    }
  };
  const float z = zt[row];
  if (E) load(first);
  float m = -INFINITY;
  for (int p = threadIdx.x; p < npieces; p += JOIN_THREADS) m = fmaxf(m, st[p].x);
  const float M = block_max<JOIN_THREADS>(m, red);
  float s = 0.f;
  for (int p = threadIdx.x; p < npieces; p += JOIN_THREADS) s += st[p].y * expf(st[p].x - M);
  const float rest = block_sum<JOIN_THREADS>(s, red);
  const float et = expf(z - M), S = rest + et;
  if (threadIdx.x == 0 && blockIdx.y == 0) row_loss[row] = z == M ? log1pf(rest) : (M - z) + logf(S);
  if (!E) return;
  const float scale = 0x1p-15f / S, dt = -rest / S;
  for (int v = first; v < nvec; v += U * step) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int w = v + u * step;
      if (w >= nvec) continue;
      const float k = expf(f[u] - M) * scale;
      const __half2* h2 = reinterpret_cast<const __half2*>(&q[u]);
      float x[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 t = __half22float2(h2[i]);
        x[2 * i] = t.x * k;
        x[2 * i + 1] = t.y * k;
      }
      if (w == tgt >> 3) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (w * 8 + i == tgt) x[i] = dt;
      }
      e[w] = pack8(x);
    }
    load(v + U * step);
  }
}

// dh = bf16(g sum over the runs of a split sum), n4 groups of four values; the 32
// warps of a block take every 32nd run, their sums join in warp order.
constexpr int RUN_WARPS = 32;
__global__ void __launch_bounds__(RUN_WARPS * 32) ce_add_runs_k(const float4* __restrict__ slabs, int64_t n4, int runs,
                                                               float g, uint2* __restrict__ dh) {
  __shared__ float4 part[RUN_WARPS][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t i = (int64_t)blockIdx.x * 32 + lane;
  dep_launch();
  dep_wait();
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (i < n4) {
#pragma unroll 8
    for (int r = warp; r < runs; r += RUN_WARPS) {
      const float4 u = slabs[r * n4 + i];
      v.x += u.x;
      v.y += u.y;
      v.z += u.z;
      v.w += u.w;
    }
  }
  part[warp][lane] = v;
  __syncthreads();
  if (warp != 0 || i >= n4) return;
#pragma unroll 8
  for (int w = 1; w < min(RUN_WARPS, runs); ++w) {
    const float4 u = part[w][lane];
    v.x += u.x;
    v.y += u.y;
    v.z += u.z;
    v.w += u.w;
  }
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x * g, v.y * g), b = __floats2bfloat162_rn(v.z * g, v.w * g);
  dh[i] = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// Up to sixteen tokens.  The products are then bound by reading W and writing
// dW, and their tiles' fixed costs weigh more than their work: of a 256-row tile
// a few per cent would be tokens, and one token on a head of 448 by 93899 took
// 137 us of which the bytes need 25 (now 41).  So W is streamed and multiplied
// by mma.sync.  Two ways:
//   one pass over W (ce_few_one_k) gives z, the statistics and the blocks' sums
//   for dh, a second kernel the losses, dh, and dW = g d^T h from z;
//   two passes, for rows that the first way does not hold or that are too narrow
//   for it: z = h W^T (ce_few_fwd_k; 16 by 8 by 16, up to eight tokens leave half
//   of its rows empty), one warp on 16 rows of W, h in shared memory; z goes to
//   scratch in FP32 (16 rows at most) beside each block's (m, s) as in the
//   softmax epilogue; then dh += d W and dW = g d^T h by the same mma, W through
//   a ring of bulk copies, 16 rows by 512 columns a stage, d in BF16 as the tiles
//   take it (with fma in FP32 it was bound by issue slots: 412 us against 160
//   for the forward with 11 tokens).
constexpr int FEW_T = 16, FEW_WARPS = 8, FEW_ROWS = FEW_WARPS * 16;
constexpr int FEW_SMEM = 200 * 1024;  // the most that h may take in shared memory
// bytes of a row of h in shared memory: whole 64-byte groups, an odd number of
// them, so that the rows an LDS.128 touches at once lie in different banks
__host__ __device__ constexpr int few_stride(int H) { return ((H + 31) / 32 | 1) * 64; }
__host__ __device__ constexpr int few_held(int T) { return T <= 8 ? 8 : 16; }  // rows of h held

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// HELD: 8 or 16 rows of h.
template <int HELD>
__global__ void __launch_bounds__(FEW_WARPS * 32) ce_few_fwd_k(const bf16* __restrict__ h, const bf16* __restrict__ W,
                                                              const int32_t* __restrict__ target, int T, int H, int V,
                                                              int ldz, float* __restrict__ z,
                                                              float2* __restrict__ stat, float* __restrict__ zt) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int NT = HELD / 8;  // tokens a lane has results of: g and g + 8
  __shared__ float2 red[FEW_WARPS][HELD];
  dep_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;  // token (and row of W) and quarter of the mma's fragments
  const int stride = few_stride(H), hv = H / 8;
  for (int i = tid; i < HELD * (stride / 16); i += FEW_WARPS * 32) {
    const int t = i / (stride / 16), v = i % (stride / 16);
    uint4 q = make_uint4(0, 0, 0, 0);
    if (t < T && v < hv) q = reinterpret_cast<const uint4*>(h + (int64_t)t * H)[v];
    *reinterpret_cast<uint4*>(smem + t * stride + v * 16) = q;
  }
  __syncthreads();
  int tgt[NT];
  float m[NT], s[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    tgt[i] = g + 8 * i < T ? target[g + 8 * i] : -1;
    m[i] = -INFINITY;
    s[i] = 0.f;
  }
  for (int v0 = (blockIdx.x * FEW_WARPS + warp) * 16; v0 < V; v0 += gridDim.x * FEW_ROWS) {
    // rows past the end repeat the last one; their results are dropped
    const uint4* w0 = reinterpret_cast<const uint4*>(W + (int64_t)min(v0 + g, V - 1) * H);
    const uint4* w1 = reinterpret_cast<const uint4*>(W + (int64_t)min(v0 + 8 + g, V - 1) * H);
    float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    // a lane takes 8 consecutive columns of every 32: two k steps of 16, the
    // same columns of h and W in the same lane's fragments
    for (int k = c; k - c < hv; k += 16) {  // 16-byte vectors; up to 4 groups of 32 columns at a time
      uint4 b0[4], b1[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        b0[u] = b1[u] = make_uint4(0, 0, 0, 0);
        if (k + 4 * u < hv) {
          b0[u] = __ldcs(w0 + k + 4 * u);
          b1[u] = __ldcs(w1 + k + 4 * u);
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (k - c + 4 * u >= hv) break;  // warp-uniform
        const uint4 a = *reinterpret_cast<const uint4*>(smem + g * stride + (k + 4 * u) * 16);
        uint4 e = make_uint4(0, 0, 0, 0);
        if (NT == 2) e = *reinterpret_cast<const uint4*>(smem + (g + 8) * stride + (k + 4 * u) * 16);
        mma_bf16(acc[0], a.x, e.x, a.y, e.y, b0[u].x, b0[u].y);
        mma_bf16(acc[1], a.x, e.x, a.y, e.y, b1[u].x, b1[u].y);
        mma_bf16(acc[0], a.z, e.z, a.w, e.w, b0[u].z, b0[u].w);
        mma_bf16(acc[1], a.z, e.z, a.w, e.w, b1[u].z, b1[u].w);
      }
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int t = g + 8 * i;
      if (t >= T) continue;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int v = v0 + 8 * j + 2 * c;
        const float x0 = acc[j][2 * i], x1 = acc[j][2 * i + 1];
        if (z && v < V) *reinterpret_cast<float2*>(z + (int64_t)t * ldz + v) = make_float2(x0, x1);  // ldz > V, even
        const float y0 = v < V ? x0 : -INFINITY, y1 = v + 1 < V ? x1 : -INFINITY;
        const float mn = fmaxf(m[i], fmaxf(y0, y1));
        const float ref = mn == -INFINITY ? 0.f : mn;
        s[i] *= m[i] == -INFINITY ? 1.f : ex2((m[i] - ref) * kLog2e);
        m[i] = mn;
        if (v == tgt[i] || v + 1 == tgt[i]) zt[t] = v == tgt[i] ? x0 : x1;
        s[i] += v < V && v != tgt[i] ? ex2((y0 - ref) * kLog2e) : 0.f;
        s[i] += v + 1 < V && v + 1 != tgt[i] ? ex2((y1 - ref) * kLog2e) : 0.f;
      }
    }
  }
  auto join = [](float& m, float& s, float m2, float s2) {
    const float M = fmaxf(m, m2);
    if (M != -INFINITY) {
      s = s * (m == -INFINITY ? 1.f : ex2((m - M) * kLog2e)) + s2 * (m2 == -INFINITY ? 1.f : ex2((m2 - M) * kLog2e));
    } else {
      s += s2;
    }
    m = M;
  };
#pragma unroll
  for (int i = 0; i < NT; ++i) {
#pragma unroll
    for (int o = 2; o > 0; o >>= 1) {  // lane 0 of the four holds the result
      const float m2 = __shfl_down_sync(0xffffffffu, m[i], o), s2 = __shfl_down_sync(0xffffffffu, s[i], o);
      join(m[i], s[i], m2, s2);
    }
    if (c == 0) red[warp][g + 8 * i] = make_float2(m[i], s[i]);
  }
  __syncthreads();
  if (tid < T) {
    float2 r = red[0][tid];
    for (int w = 1; w < FEW_WARPS; ++w) join(r.x, r.y, red[w][tid].x, red[w][tid].y);
    stat[(int64_t)tid * gridDim.x + blockIdx.x] = r;
  }
}

constexpr int FEW_THREADS = 128, FEW_COLS = 512, FEW_STAGES = 4;
// Row groups of a block: the warps have 128 columns each; narrow rows leave some
// of them free to take every second or fourth 16 rows.
__host__ __device__ constexpr int few_groups(int H) { return H <= 128 ? 4 : H <= 256 ? 2 : 1; }
__host__ __device__ constexpr int few_sub(int H) { return 16 * few_groups(H); }  // rows of a stage
// bytes from row to row of W in a stage: 16 more than the columns' own, so that
// the eight rows an ldmatrix reads lie in different banks
__host__ __device__ constexpr int few_wrow(int H) { return FEW_COLS * 2 / few_groups(H) + 16; }
// A stage: rows of W in BF16, where dh is made of them, then the tokens' z of these rows in FP32.
__host__ __device__ constexpr int few_stage(int T, int H, bool dh) {
  return ((dh ? few_sub(H) * few_wrow(H) : 0) + T * few_sub(H) * 4 + 127) / 128 * 128;
}
// After the ring, for two stages in turn: d in BF16, [rows][16 tokens] and [16 tokens][rows].
__host__ __device__ constexpr int few_d_bytes(int H) { return few_sub(H) * 16 * 2; }
__host__ __device__ constexpr int few_smem(int T, int H, bool dh) {
  return FEW_STAGES * few_stage(T, H, dh) + 4 * few_d_bytes(H);
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(su32(p))
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(su32(p))
               : "memory");
}

__device__ __forceinline__ void mma_bf16_k8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(b0));
}

// One pass over W for z, the statistics and dh:
//   dh_t = g (sum_{v != target} p_v W_v - (rest / S) W_target)
// needs p only up to a factor per token, so each block keeps sums of exp(z_v - m)
// W_v around its running maximum m, moved when m rises, and ce_few_dh adds the
// blocks' sums with their factors exp(m - M) / S.  W is then read once and dW
// written once, which is the floor: 5 tokens of 3584 by 152064 take 370 us of
// 321 (with a second pass over W 558), dh alone 198 and the losses alone 159 of
// 160.  A stage is 8 or 16 whole rows: the warps take a slice of the columns
// each, h of it in registers as the first factor of z, the sums of dh in
// registers too (their columns as the rows of the mma, tokens as its columns).
// The warps' parts of z meet in shared memory, every warp adds them for itself in
// the layout in which exp(z - m) is then its second factor of dh: one barrier a
// stage.  W comes out of shared memory twice, once transposed.  16 rows where
// rows are short (12 tokens of 1024 by 128256: 140 us, with 8 rows 157), four
// warps up to 512 columns (8 of 512: 67, with eight warps of half the columns 71).
// NT: groups of eight tokens; NW: warps; KP: groups of 32 columns that a warp has.
// RB: groups of eight rows in a stage.  Of the last OUT column groups h stays in
// shared memory, in the order of the fragments, where the registers do not reach
// (spilled, 5 tokens of 3584 by 152064 took 440 us).
__host__ __device__ constexpr int one_rows(int KP) { return KP <= 4 ? 16 : 8; }
__host__ __device__ constexpr int one_pitch(int KP, int NW) { return NW * KP * 64 + 16; }  // an ldmatrix's rows in different banks
__host__ __device__ constexpr int one_stages(int KP, int NW) { return NW == 4 ? 4 : KP == 8 ? 6 : 3; }
__host__ __device__ constexpr int one_out(int NT, int KP) { return NT == 1 && KP >= 16 ? 7 : 0; }
__host__ __device__ constexpr int one_smem(int NT, int KP, int NW) {
  return one_stages(KP, NW) * one_rows(KP) * one_pitch(KP, NW) + NW * 32 * (2 * NT * one_rows(KP) + one_out(NT, KP) * 16);
}
// blocks per SM: the registers' 12 a column group and eight tokens, and the rings
__host__ __device__ constexpr int one_blocks(int NT, int KP, int NW) { return NW == 4 ? 3 : NT * KP <= 4 ? 2 : 1; }

template <int NT, int KP, int NW>
__global__ void __launch_bounds__(NW * 32, one_blocks(NT, KP, NW))
    ce_few_one_k(const bf16* __restrict__ h, const bf16* __restrict__ W, const int32_t* __restrict__ target, int T, int H,
                 int V, int ldz, float* __restrict__ z, float2* __restrict__ stat, float* __restrict__ zt,
                 float* __restrict__ slabs) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int NS = one_stages(KP, NW), ROWS = one_rows(KP), RB = ROWS / 8, PITCH = one_pitch(KP, NW), STAGE = ROWS * PITCH;
  constexpr int OUT = one_out(NT, KP), IN = KP - OUT, NTH = NW * 32;
  float2* parts = reinterpret_cast<float2*>(smem + NS * STAGE);  // [2][RB][NT][NW][32]
  __shared__ uint64_t full[NS];
  dep_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int base = warp * KP * 32;
  const int groups = (V + ROWS - 1) / ROWS;  // of rows: the blocks take them in turn
  const int stages = (groups - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
  auto row = [&](int k) { return (k * (int)gridDim.x + (int)blockIdx.x) * ROWS; };  // the first of stage k
  bool failed = false;
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) mbar_init(&full[i], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // what no copy writes and the products read: columns past the last, and the rows that a short last stage leaves of
  // a part of the ring that no stage before it has filled
  const int pad = PITCH / 16 - H / 8;
  for (int i = tid; i < NS * ROWS * pad; i += NTH)
    *reinterpret_cast<uint4*>(smem + i / pad * PITCH + H * 2 + i % pad * 16) = make_uint4(0, 0, 0, 0);
  const int last = min(ROWS, V - row(stages - 1));
  if (stages <= NS)
    for (int i = tid; i < (ROWS - last) * (H / 8); i += NTH)
      *reinterpret_cast<uint4*>(smem + (stages - 1) * STAGE + (last + i / (H / 8)) * PITCH + i % (H / 8) * 16) =
          make_uint4(0, 0, 0, 0);
  __syncthreads();
  auto fill = [&](int k) {  // the first warp
    const int b = row(k), n = min(ROWS, V - b);
    if (lane == 0) mbar_expect_tx(&full[k % NS], (uint32_t)n * (uint32_t)H * 2);
    __syncwarp();
    if (lane < n)
      bulk_load(smem + (k % NS) * STAGE + lane * PITCH, W + (int64_t)(b + lane) * H, (uint32_t)H * 2, &full[k % NS]);
    __syncwarp();
  };
  if (warp == 0)
    for (int k = 0; k < min(stages, NS); ++k) fill(k);
  uint4* held = reinterpret_cast<uint4*>(parts + 2 * RB * NT * NTH) + tid;  // [OUT][NTH], this thread's
  uint32_t ha[IN][4 * NT];
  float dh[KP][2][NT][4];
#pragma unroll
  for (int k = 0; k < KP; ++k) {
    for (int i = 0; i < NT; ++i) {
      uint32_t x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int col = base + 32 * k + 8 * j + 2 * c, t = g + 8 * i;
        x[j] = t < T && col < H ? *reinterpret_cast<const uint32_t*>(h + (int64_t)t * H + col) : 0;
        if (k < IN) ha[k < IN ? k : 0][4 * i + j] = x[j];
        dh[k][j >> 1][i][2 * (j & 1)] = dh[k][j >> 1][i][2 * (j & 1) + 1] = 0.f;
      }
      if (k >= IN) held[(k - IN) * NTH] = make_uint4(x[0], x[1], x[2], x[3]);
    }
  }
  int tgt[NT];
  bool has[NT];
  float m[NT], s[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    tgt[i] = g + 8 * i < T ? target[g + 8 * i] : -1;
    has[i] = tgt[i] >= 0 && tgt[i] < V;
    m[i] = -INFINITY;
    s[i] = 0.f;
  }
  for (int k = 0; k < stages; ++k) {
    const uint8_t* wp = smem + (k % NS) * STAGE + (lane & 7) * PITCH + (base + (lane >> 3) * 8) * 2;
    reads_before_copies();  // those of the stage before, all used by now
    mbar_wait(&full[k % NS], (uint32_t)(k / NS) & 1, failed);
    float2* part = parts + (k & 1) * RB * NT * NTH + lane;
    float acc[RB][2][4];
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[b][0][q] = acc[b][1][q] = 0.f;
#pragma unroll
    for (int j = 0; j < KP; ++j) {
      uint4 a, a8 = make_uint4(0, 0, 0, 0);
      if (j < IN) {
        const uint32_t* f = ha[j < IN ? j : 0];
        a = make_uint4(f[0], f[1], f[2], f[3]);
        if (NT > 1) a8 = make_uint4(f[4 * NT - 4], f[4 * NT - 3], f[4 * NT - 2], f[4 * NT - 1]);
      } else {
        a = held[(j - IN) * NTH];
      }
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        uint32_t w[4];
        ldmatrix4(w, wp + b * 8 * PITCH + j * 64);
        mma_bf16(acc[b][0], a.x, a8.x, a.y, a8.y, w[0], w[1]);
        mma_bf16(acc[b][1], a.z, a8.z, a.w, a8.w, w[2], w[3]);
      }
    }
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int i = 0; i < NT; ++i)
        part[((b * NT + i) * NW + warp) * 32] =
            make_float2(acc[b][0][2 * i] + acc[b][1][2 * i], acc[b][0][2 * i + 1] + acc[b][1][2 * i + 1]);
    __syncthreads();  // also: every warp is done with the stage before, which takes a new one
    if (warp == 0 && k >= 1 && k - 1 + NS < stages) fill(k - 1 + NS);
    uint32_t e[RB][NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int t = g + 8 * i, v0 = row(k) + 2 * c;  // this lane's rows: v0 + 8 b and the next
      float2 x[RB];
      float mn = m[i];
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        const int v = v0 + 8 * b;
        x[b] = part[(b * NT + i) * NW * 32];
#pragma unroll
        for (int w = 1; w < NW; ++w) {
          const float2 y = part[((b * NT + i) * NW + w) * 32];
          x[b].x += y.x;
          x[b].y += y.y;
        }
        if (warp == (k & (NW - 1)) && t < T && v < V) {
          if (z) *reinterpret_cast<float2*>(z + (int64_t)t * ldz + v) = x[b];  // ldz > V, even
          if (has[i] && (v == tgt[i] || v + 1 == tgt[i])) zt[t] = v == tgt[i] ? x[b].x : x[b].y;
        }
        if (has[i] && v < V) mn = fmaxf(mn, x[b].x);
        if (has[i] && v + 1 < V) mn = fmaxf(mn, x[b].y);
      }
      mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, 1));
      mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, 2));
      if (__any_sync(0xffffffffu, mn > m[i])) {  // the sums so far move to the new maximum
        const float f = m[i] == -INFINITY ? 1.f : ex2((m[i] - mn) * kLog2e);
        s[i] *= f;
        m[i] = mn;
        const float f0 = __shfl_sync(0xffffffffu, f, 8 * c), f1 = __shfl_sync(0xffffffffu, f, 8 * c + 4);
#pragma unroll
        for (int j = 0; j < KP; ++j)
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            dh[j][q][i][0] *= f0;
            dh[j][q][i][1] *= f1;
            dh[j][q][i][2] *= f0;
            dh[j][q][i][3] *= f1;
          }
      }
      const float ref = mn == -INFINITY ? 0.f : mn;
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        const int v = v0 + 8 * b;
        const float e0 = has[i] && v < V && v != tgt[i] ? ex2((x[b].x - ref) * kLog2e) : 0.f;
        const float e1 = has[i] && v + 1 < V && v + 1 != tgt[i] ? ex2((x[b].y - ref) * kLog2e) : 0.f;
        s[i] += e0 + e1;
        // rounded for the mma: half a step of BF16 of each term of dh, as of d where tiles take it
        const __nv_bfloat162 p = __floats2bfloat162_rn(e0, e1);
        e[b][i] = *reinterpret_cast<const uint32_t*>(&p);
      }
    }
    if (!slabs) continue;
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int j = 0; j < KP; ++j) {
        uint32_t w[4];
        ldmatrix4_t(w, wp + b * 8 * PITCH + j * 64);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          mma_bf16_k8(dh[j][0][i], w[0], w[1], e[b][i]);
          mma_bf16_k8(dh[j][1][i], w[2], w[3], e[b][i]);
        }
      }
  }
  if (failed && tid == 0) {  // what is on its way lands before the block's memory goes
    const long long t0 = clock64();
    while (clock64() - t0 < kWaitCycles) {
    }
  }
  if (warp == 0) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      s[i] += __shfl_xor_sync(0xffffffffu, s[i], 1);
      s[i] += __shfl_xor_sync(0xffffffffu, s[i], 2);
      if (c == 0 && g + 8 * i < T) stat[(int64_t)(g + 8 * i) * gridDim.x + blockIdx.x] = make_float2(m[i], s[i]);
    }
  }
  if (!slabs) return;
  float* out = slabs + (int64_t)blockIdx.x * T * H;
#pragma unroll
  for (int k = 0; k < KP; ++k)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int col = base + 32 * k + 8 * q + g;
      if (col >= H) continue;
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int t = 8 * i + 2 * c + u;
          if (t < T) out[(int64_t)t * H + col] = dh[k][q >> 1][i][2 * (q & 1) + u];
        }
    }
}

// A token's statistics from the blocks' (m, s), as in ce_join_k; one warp.
struct FewStat {
  float M, inv, at;  // maximum, 1 / S (0: no target), p - 1 at the target
  int tgt;           // -1: none
};
__device__ __forceinline__ FewStat few_join(const float2* __restrict__ stat, int npieces, const float* __restrict__ zt,
                                            const int32_t* __restrict__ target, int t, int T, int V, int lane,
                                            float* row_loss) {
  const int tgt = t < T ? target[t] : -1;
  const bool has = tgt >= 0 && tgt < V;
  float M = -INFINITY, rest = 0.f, S = 1.f;
  if (has) {
    const float2* st = stat + (int64_t)t * npieces;
    for (int i = lane; i < npieces; i += 256) {  // eight loads at a time
      float2 p[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) p[u] = i + 32 * u < npieces ? st[i + 32 * u] : make_float2(-INFINITY, 0.f);
      float mn = M;
#pragma unroll
      for (int u = 0; u < 8; ++u) mn = fmaxf(mn, p[u].x);
      rest *= M == -INFINITY ? 1.f : expf(M - mn);
#pragma unroll
      for (int u = 0; u < 8; ++u) rest += p[u].y * (p[u].x == -INFINITY ? 1.f : expf(p[u].x - mn));
      M = mn;
    }
    const float wm = warp_max(M);
    rest = warp_sum(rest * (M == -INFINITY ? 1.f : expf(M - wm)));
    M = wm;
    S = rest + expf(zt[t] - M);
  }
  if (row_loss && lane == 0 && t < T)
    row_loss[t] = !has ? 0.f : zt[t] == M ? log1pf(rest) : (M - zt[t]) + logf(S);
  return FewStat{M, has ? 1.f / S : 0.f, has ? -rest / S : 0.f, has ? tgt : -1};
}

// Token t's loss, and dh in 128 columns from col0 on from the blocks' sums; FEW_THREADS threads.
__device__ __forceinline__ void ce_few_dh(const bf16* __restrict__ W, const int32_t* __restrict__ target, int t, int T,
                                          int H, int V, int col0, const float2* __restrict__ stat, int npieces,
                                          const float* __restrict__ zt, const float* __restrict__ slabs, float scale,
                                          float* row_loss, bf16* __restrict__ dh) {
  constexpr int NW = FEW_THREADS / 32;
  __shared__ float4 part[NW][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = col0 + lane * 4;
  const FewStat f = few_join(stat, npieces, zt, target, t, T, V, lane, warp == 0 && col0 == 0 ? row_loss : nullptr);
  if (!dh) return;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (f.tgt >= 0 && col < H) {
#pragma unroll 8
    for (int r = warp; r < npieces; r += NW) {
      const float m = stat[(int64_t)t * npieces + r].x, w = m == -INFINITY ? 1.f : expf(m - f.M);
      const float4 u = *reinterpret_cast<const float4*>(slabs + ((int64_t)r * T + t) * H + col);
      v.x += u.x * w;
      v.y += u.y * w;
      v.z += u.z * w;
      v.w += u.w * w;
    }
  }
  part[warp][lane] = v;
  __syncthreads();
  if (warp != 0 || col >= H) return;
#pragma unroll
  for (int w = 1; w < NW; ++w) {
    const float4 u = part[w][lane];
    v.x += u.x;
    v.y += u.y;
    v.z += u.z;
    v.w += u.w;
  }
  uint2 o = make_uint2(0, 0);
  if (f.tgt >= 0) {
    const uint2 q = *reinterpret_cast<const uint2*>(W + (int64_t)f.tgt * H + col);
    const __nv_bfloat162 w0 = *reinterpret_cast<const __nv_bfloat162*>(&q.x), w1 = *reinterpret_cast<const __nv_bfloat162*>(&q.y);
    const __nv_bfloat162 a = __floats2bfloat162_rn(scale * (v.x * f.inv + f.at * __low2float(w0)),
                                                   scale * (v.y * f.inv + f.at * __high2float(w0)));
    const __nv_bfloat162 b = __floats2bfloat162_rn(scale * (v.z * f.inv + f.at * __low2float(w1)),
                                                   scale * (v.w * f.inv + f.at * __high2float(w1)));
    o = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
  *reinterpret_cast<uint2*>(dh + (int64_t)t * H + col) = o;
}

// Block (x, y): rows [x per, (x + 1) per) of W, columns [512 y, 512 (y + 1)).
// DH: dh as well, from W, into slabs.  Without it W is not read, and the first
// first_y rows of blocks, if there are any, make the losses, and dh of what
// ce_few_one_k left.
template <bool DH>
__global__ void __launch_bounds__(FEW_THREADS, DH ? 3 : 6) ce_few_bwd_k(const bf16* __restrict__ h, const bf16* __restrict__ W,
                                                              const int32_t* __restrict__ target, int T, int H, int V,
                                                              int ldz, const float* __restrict__ z,
                                                              const float2* __restrict__ stat, int npieces,
                                                              const float* __restrict__ zt, int per, float scale,
                                                              float* __restrict__ row_loss, float* __restrict__ slabs,
                                                              bf16* __restrict__ dW, int first_y, bf16* __restrict__ dhout) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float sM[FEW_T], sI[FEW_T], sD[FEW_T];  // maximum, 1 / S (0: no target), p - 1 at the target
  __shared__ int sT[FEW_T];
  __shared__ uint64_t full[FEW_STAGES];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int by = (int)blockIdx.y - first_y;
  if (!DH && by < 0) {
    const int q = blockIdx.y * gridDim.x + blockIdx.x, n = dhout ? (H + 127) / 128 : 1;
    dep_launch();
    dep_wait();
    if (q < T * n) ce_few_dh(W, target, q / n, T, H, V, q % n * 128, stat, npieces, zt, slabs, scale, row_loss, dhout);
    return;
  }
  const int RG = few_groups(H), SUB = few_sub(H), WROW = few_wrow(H), STAGE = few_stage(T, H, DH);
  const int ZOFF = DH ? SUB * WROW : 0;  // the tokens' logits in a stage
  const int rg = warp / (4 / RG);  // this warp's row group
  const int col0 = by * FEW_COLS, wcol = warp % (4 / RG) * 128, base = col0 + wcol;
  const int ncol = min(128, H - base);  // this warp's columns: a multiple of 8, or none
  const int r0 = blockIdx.x * per, r1 = min(V, r0 + per), stages = (r1 - r0 + SUB - 1) / SUB;
  uint8_t* dbuf = smem + FEW_STAGES * STAGE;
  bool failed = false;
  dep_launch();
  if (tid == 0) {
    for (int i = 0; i < FEW_STAGES; ++i) mbar_init(&full[i], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // h as the second factor of dW: tile (G, j) holds columns 32 G + 8 (n / 2) + 2 j +
  // n % 2 for n = 0 .. 7, so that a lane's results of tiles j = 0 .. 3 are eight
  // neighbouring columns
  // (tokens without a target are left out: what padding holds may be no number)
  uint32_t hb[16][2];
  const uint16_t* h16 = reinterpret_cast<const uint16_t*>(h);
  bool used[2][2];
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int tok = 2 * c + 8 * k + i, tgt = tok < T ? target[tok] : -1;
      used[k][i] = tgt >= 0 && tgt < V;
    }
#pragma unroll
  for (int t = 0; t < 16; ++t) {
    const int col = base + 32 * (t >> 2) + 8 * (g >> 1) + 2 * (t & 3) + (g & 1);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int tok = 2 * c + 8 * k;
      const uint32_t lo = col < H && used[k][0] ? h16[(int64_t)tok * H + col] : 0;
      const uint32_t hi = col < H && used[k][1] ? h16[(int64_t)(tok + 1) * H + col] : 0;
      hb[t][k] = lo | (hi << 16);
    }
  }
  float dh[DH ? 16 : 1][4];
  if constexpr (DH) {
#pragma unroll
    for (int t = 0; t < 16; ++t) dh[t][0] = dh[t][1] = dh[t][2] = dh[t][3] = 0.f;
  }
  // the first warp: stage k's rows of W, and the tokens' logits of them (z's rows
  // are padded, so that whole stages may be read past V)
  auto fill = [&](int k) {
    uint8_t* to = smem + (k % FEW_STAGES) * STAGE;
    uint64_t* bar = &full[k % FEW_STAGES];
    const int b = r0 + k * SUB, n = min(SUB, r1 - b);
    const uint32_t bytes = (uint32_t)min(FEW_COLS / RG, H - col0) * 2;
    if (lane == 0) mbar_expect_tx(bar, (DH ? (uint32_t)n * bytes : 0u) + (uint32_t)(T * SUB) * 4);
    __syncwarp();
    if (DH)
      for (int r = lane; r < n; r += 32) bulk_load(to + r * WROW, W + (int64_t)(b + r) * H + col0, bytes, bar);
    if (lane < T) bulk_load(to + ZOFF + lane * SUB * 4, z + (int64_t)lane * ldz + b, (uint32_t)SUB * 4, bar);
    __syncwarp();
  };
  dep_wait();
  __syncthreads();
  if (warp == 0)
    for (int k = 0; k < min(stages, FEW_STAGES); ++k) fill(k);
  for (int t = warp; t < FEW_T; t += FEW_THREADS / 32) {
    const FewStat f = few_join(stat, npieces, zt, target, t, T, V, lane,
                               blockIdx.x == 0 && blockIdx.y == 0 ? row_loss : nullptr);
    if (lane == 0) {
      sM[t] = f.M;
      sI[t] = f.inv;
      sD[t] = f.at;
      sT[t] = f.tgt;
    }
  }
  __syncthreads();
  for (int k = 0; k < stages; ++k) {
    const uint8_t* st = smem + (k % FEW_STAGES) * STAGE;
    const int b = r0 + k * SUB, n = min(SUB, r1 - b);
    bf16* dT = reinterpret_cast<bf16*>(dbuf + (k & 1) * 2 * few_d_bytes(H));  // [SUB][16]
    bf16* dN = dT + SUB * 16;                                                 // [16][SUB]
    reads_before_copies();  // those of the stage before, all used by now
    mbar_wait(&full[k % FEW_STAGES], (uint32_t)(k / FEW_STAGES) & 1, failed);
    for (int i = tid; i < FEW_T * SUB; i += FEW_THREADS) {  // the logits' gradient
      const int t = i / SUB, r = i % SUB;
      float d = 0.f;
      if (r < n && sT[t] >= 0) {
        const float x = reinterpret_cast<const float*>(st + ZOFF)[t * SUB + r];
        d = b + r == sT[t] ? sD[t] : ex2((x - sM[t]) * kLog2e) * sI[t];
      }
      const bf16 v = __float2bfloat16_rn(d);
      dT[r * 16 + t] = v;
      dN[t * SUB + r] = v;
    }
    // rows past the last: their d is 0, but what an earlier stage left of W there
    // may be no number
    if (DH)
      for (int i = n * (WROW / 16) + tid; i < SUB * (WROW / 16); i += FEW_THREADS)
        reinterpret_cast<uint4*>(smem + (k % FEW_STAGES) * STAGE)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();  // also: every warp is done with the stage before, which takes a new one
    if (warp == 0 && k >= 1 && k - 1 + FEW_STAGES < stages) fill(k - 1 + FEW_STAGES);
    if (ncol <= 0 || rg * 16 >= n) continue;
    uint32_t aT[4], aN[DH ? 4 : 1];
    // fragments of 16 by 16: lanes 0 .. 7 give the rows of the first 8 by 8 part, and so on
    ldmatrix4(aT, dT + (rg * 16 + (lane & 15)) * 16 + (lane >> 4) * 8);
    if constexpr (DH) ldmatrix4(aN, dN + (lane & 15) * SUB + rg * 16 + (lane >> 4) * 8);
    const uint8_t* wp = st + (rg * 16 + (lane & 15)) * WROW + wcol * 2 + (lane >> 4) * 16;
#pragma unroll
    for (int G = 0; G < 4; ++G) {
      if (32 * G >= ncol) break;
      float o[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
        mma_bf16(o[j], aT[0], aT[1], aT[2], aT[3], hb[4 * G + j][0], hb[4 * G + j][1]);
      }
      if constexpr (DH) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t w[4];
          ldmatrix4_t(w, wp + G * 64 + j * 32);
          mma_bf16(dh[4 * G + 2 * j], aN[0], aN[1], aN[2], aN[3], w[0], w[1]);
          mma_bf16(dh[4 * G + 2 * j + 1], aN[0], aN[1], aN[2], aN[3], w[2], w[3]);
        }
      }
      if (dW && 32 * G + 8 * c < ncol) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = rg * 16 + g + 8 * i;
          if (r >= n) continue;
          uint32_t q[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(o[j][2 * i] * scale, o[j][2 * i + 1] * scale);
            q[j] = *reinterpret_cast<const uint32_t*>(&v);
          }
          *reinterpret_cast<uint4*>(dW + (int64_t)(b + r) * H + base + 32 * G + 8 * c) = make_uint4(q[0], q[1], q[2], q[3]);
        }
      }
    }
  }
  if (failed && tid == 0) {  // what is on its way lands before the block's memory goes
    const long long t0 = clock64();
    while (clock64() - t0 < kWaitCycles) {
    }
  }
  if constexpr (DH) {
    if (RG > 1) {  // the row groups' parts, added in order through the ring's memory
      float* part = reinterpret_cast<float*>(smem) + (int64_t)warp * 64 * 32 + lane;
      __syncthreads();
      if (rg > 0) {
#pragma unroll
        for (int t = 0; t < 64; ++t) part[t * 32] = dh[t >> 2][t & 3];
      }
      __syncthreads();
      if (rg > 0) return;
      for (int q = 1; q < RG; ++q) {
        const float* other = part + q * (4 / RG) * 64 * 32;
#pragma unroll
        for (int t = 0; t < 64; ++t) dh[t >> 2][t & 3] += other[t * 32];
      }
    }
    float* out = slabs + (int64_t)blockIdx.x * T * H + base;
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      if (8 * t >= ncol) break;
      if (g < T) *reinterpret_cast<float2*>(out + (int64_t)g * H + 8 * t + 2 * c) = make_float2(dh[t][0], dh[t][1]);
      if (g + 8 < T) *reinterpret_cast<float2*>(out + (int64_t)(g + 8) * H + 8 * t + 2 * c) = make_float2(dh[t][2], dh[t][3]);
    }
  }
}

// ------------------------------------------------------------------ distillation
// A row of student logits z, teacher logits y at ids i:
//   q = softmax over the filled slots of y / tau, p = softmax(z / tau),
//   kd = sum_j q_j (log q_j - log p_{i_j}),  ce = lse(z) - z_target,
//   dz_v = w_ce (softmax(z)_v - [v = target]) + w_kd / tau (p_v - sum_{i_j = v} q_j).
// Bound by HBM (8192 rows of 32000 at two temperatures 192 us, 4096 of 152064
// 432: 0.81 and 0.85 of the measured copy rate): the statistics need the whole
// row before the first gradient element.  A block takes one row at a time, and every n-th row: a producer
// lane streams the row through a ring of shared memory with bulk copies, always
// ahead of the warps that work on it, across row ends.  Where a row fits the
// ring it stays there until its gradient is written; a longer one is fetched a
// second time, from L2 (152 rows under work are at most 46 MB of 152064
// columns).  The working warps take running sums of exp(z - m) around each
// thread's maximum m at both temperatures, join them once per row, and write
// the dense part of the gradient.  A further warp works out the teacher's
// distribution of the next row meanwhile, and rewrites the at most K + 1
// columns with a teacher entry or the target from their FP32 values once the
// dense part stands, so that no element is rounded twice and an id that appears
// in several slots gets the sum of their q, in slot order.
constexpr int KD_MAX_K = 1024;
struct KdArgs {
  int64_t rows;
  int kcap;  // slots there is room for: K up to a power of two, at least 32
  const bf16* logits;
  const int32_t* target;
  const float* t_val;
  const int32_t* t_idx;
  int V, K;
  float tau, w_ce, w_kd;
  float *row_ce, *row_kd;
  bf16* dlogits;
};

template <int ID>
__device__ __forceinline__ void named_sync(int n) {
  asm volatile("bar.sync %0, %1;" ::"n"(ID), "r"(n) : "memory");
}
template <int ID>
__device__ __forceinline__ void named_arrive(int n) {
  asm volatile("bar.arrive %0, %1;" ::"n"(ID), "r"(n) : "memory");
}

template <int CW, int U, int NS>
constexpr size_t kd_smem(int kcap) {
  return (size_t)NS * CW * 32 * U * 16 + (size_t)kcap * (2 * 4 + 2) * 4;
}
// CW working warps, a ring of NS chunks of U 16-byte vectors a thread, BPS blocks
// per SM that the registers are to allow.  TWO: both temperatures are summed (hard targets and tau != 1);
// else one exponential serves both.  Exponentials are taken as 2^(z a - c) with
// a = log2(e) or log2(e) / tau and the reference c = fl(m a) kept as it is
// rounded, so that the fused product loses nothing.
template <int CW, int U, int NS, int BPS, bool TWO>
__global__ void __launch_bounds__((CW + 2) * 32, BPS) distill_k(const KdArgs a) {
  constexpr int CT = CW * 32, CV = CT * U;  // threads that work on the row; vectors of a chunk
  extern __shared__ __align__(128) uint8_t smem[];
  uint4* ring = reinterpret_cast<uint4*>(smem);                    // [NS][CV]
  float* slots = reinterpret_cast<float*>(smem + NS * CV * 16);    // two rows' slots, used in turn
  int* table = reinterpret_cast<int*>(slots + 2 * 4 * a.kcap);     // [2 kcap] ids seen, -1 free
  __shared__ float part[2][CW + 1][3];  // (m, s1, st) of the warps; the last one's is of the row's ends
  __shared__ int s_tgt[2];              // the row's target, -1: none
  __shared__ int s_soft[2];             // whether it has a teacher
  __shared__ uint64_t full[NS], empty[NS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int V = a.V, K = a.K;
  const float it = 1.f / a.tau, itl = it * kLog2e;
  constexpr float kLn2 = 0.6931471805599453f;
  const bool grad = a.dlogits != nullptr;
  bool failed = false;
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], CW);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  // the row in memory: up to 7 elements, whole 16-byte vectors, up to 7
  // elements.  The vectors go through the ring; the elements at the ends belong
  // to lanes of the teacher's warp.
  int head, nvec, nc;
  bool held;  // the row stays in the ring until its gradient is written
  auto place = [&](int64_t row) {
    const int skip = (int)((row * V) & 7);
    head = skip ? min(8 - skip, V) : 0;
    nvec = (V - head) >> 3;
    nc = (nvec + CV - 1) / CV;
    held = grad && nc <= NS;
  };

  if (warp == CW + 1) {  // producer
    if (lane == 0) {
      int slot = 0;
      uint32_t ph = 1;  // the ring starts empty
      for (int64_t row = blockIdx.x; row < a.rows && !failed; row += gridDim.x) {
        place(row);
        const uint4* src = reinterpret_cast<const uint4*>(a.logits + row * V + head);
        for (int pass = grad && !held ? 0 : 1; pass < 2 && !failed; ++pass)
          for (int c = 0; c < nc; ++c) {
            mbar_wait(&empty[slot], ph, failed);
            if (failed) break;
            const uint32_t bytes = (uint32_t)min(nvec - c * CV, CV) * 16;
            mbar_expect_tx(&full[slot], bytes);
            bulk_load(ring + slot * CV, src + (int64_t)c * CV, bytes, &full[slot]);
            if (++slot == NS) {
              slot = 0;
              ph ^= 1;
            }
          }
      }
      if (failed) {  // nothing more is issued; what is on its way lands before the block's memory goes
        const long long t0 = clock64();
        while (clock64() - t0 < kWaitCycles) {
        }
      }
    }
    return;
  }

  if (warp == CW) {  // the teacher
    int turn = 0;
    float zt = 0.f, ze = -INFINITY, ysum = 0.f;
    int tgt = -1, ie = -1;
    bool twice = false, listed = false, soft = false;
    // everything of a row that its statistics do not enter; its slots' arrays are those of its turn
    auto prepare = [&](int64_t row, int par) {
      place(row);
      const bf16* z = a.logits + row * V;
      int* id = reinterpret_cast<int*>(slots + par * 4 * a.kcap);
      float *y = reinterpret_cast<float*>(id) + a.kcap, *q = y + a.kcap, *zj = q + a.kcap;
      tgt = a.target ? a.target[row] : -1;
      if (tgt >= V || tgt < 0) tgt = -1;
      for (int j = lane; j < 2 * a.kcap; j += 32) table[j] = -1;
      ie = lane < head ? lane : lane >= 8 && head + nvec * 8 + lane - 8 < V ? head + nvec * 8 + lane - 8 : -1;
      ze = ie >= 0 ? __bfloat162float(z[ie]) : -INFINITY;
      float ym = -INFINITY;
      bool nan = false;
      twice = listed = false;
#pragma unroll 4
      for (int j = lane; j < K; j += 32) {
        int i = a.t_idx[row * K + j];
        if (i < 0 || i >= V) i = -1;
        const float v = i >= 0 ? a.t_val[row * K + j] * it : -INFINITY;
        zj[j] = i >= 0 ? __bfloat162float(z[i]) : 0.f;
        id[j] = i;
        y[j] = v;
        ym = fmaxf(ym, v);
        nan |= v != v;
        listed |= i >= 0 && i == tgt;
      }
      zt = tgt >= 0 ? __bfloat162float(z[tgt]) : 0.f;
      __syncwarp();
      for (int j = lane; j < K; j += 32) {
        const int i = id[j];
        if (i < 0) continue;
        uint32_t h = (uint32_t)i * 2654435761u >> 7;
        for (;;) {  // ends: the table has twice as many places as there are slots
          h &= 2u * (uint32_t)a.kcap - 1u;
          const int old = atomicCAS(&table[h], -1, i);
          if (old == i) twice = true;
          if (old == -1 || old == i) break;
          ++h;
        }
      }
      ym = warp_max(ym);
      nan = __any_sync(0xffffffffu, nan);
      twice = __any_sync(0xffffffffu, twice);
      listed = __any_sync(0xffffffffu, listed);
      if (nan && ym == -INFINITY) ym = 0.f;  // a NaN among the slots shows in the row, it does not empty it
      soft = ym != -INFINITY;
      ysum = 0.f;
      for (int j = lane; j < K; j += 32) {
        const float d = y[j] - ym, v = id[j] < 0 || !soft ? 0.f : expf(d);
        y[j] = d;
        q[j] = v;
        ysum += v;
      }
      ysum = warp_sum(ysum);
      const float wm = warp_max(ze), ref = wm == -INFINITY ? 0.f : wm;
      const float st = warp_sum(ie >= 0 ? ex2(fmaf(ze, itl, -__fmul_rn(ref, itl))) : 0.f);
      const float s1 = TWO ? warp_sum(ie >= 0 ? ex2(fmaf(ze, kLog2e, -__fmul_rn(ref, kLog2e))) : 0.f) : st;
      if (lane == 0) {
        part[par][CW][0] = wm;
        part[par][CW][1] = s1;
        part[par][CW][2] = st;
        s_tgt[par] = tgt;
        s_soft[par] = soft;
      }
    };
    if ((int64_t)blockIdx.x < a.rows) prepare(blockIdx.x, 0);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, ++turn) {
      const int par = turn & 1;
      named_sync<1>(CT + 32);  // the row's statistics
      float m = lane <= CW ? part[par][lane <= CW ? lane : 0][0] : -INFINITY;
      const float pm = m;
      m = warp_max(m);
      if (m == -INFINITY) m = 0.f;
      const float c1 = __fmul_rn(m, kLog2e), ct = __fmul_rn(m, itl);
      float s1 = 0.f, st = 0.f;
      if (lane <= CW) {
        const bool none = pm == -INFINITY;
        s1 = part[par][lane][1] * (none ? 1.f : ex2(__fmul_rn(pm, kLog2e) - c1));
        st = part[par][lane][2] * (none ? 1.f : ex2(__fmul_rn(pm, itl) - ct));
      }
      s1 = warp_sum(s1);
      st = warp_sum(st);
      const bool hard = tgt >= 0;
      const float l1 = log2f(s1), lt = log2f(st);
      const float w1 = hard ? a.w_ce : 0.f, wt = soft ? a.w_kd * it : 0.f;
      int* id = reinterpret_cast<int*>(slots + par * 4 * a.kcap);
      float *y = reinterpret_cast<float*>(id) + a.kcap, *q = y + a.kcap, *zj = q + a.kcap;
      float kd = 0.f;
      const float yl = logf(ysum);
      for (int j = lane; j < K; j += 32) {
        if (id[j] < 0 || q[j] == 0.f) continue;
        q[j] /= ysum;
        kd += q[j] * ((y[j] - yl) - kLn2 * (fmaf(zj[j], itl, -ct) - lt));
      }
      kd = warp_sum(kd);
      if (lane == 0) {
        a.row_kd[row] = soft ? kd : 0.f;
        if (a.row_ce) a.row_ce[row] = hard ? kLn2 * (l1 - fmaf(zt, kLog2e, -c1)) : 0.f;
      }
      const float zt0 = zt;
      const int tgt0 = tgt;
      const bool soft0 = soft, twice0 = twice, listed0 = listed;
      if (grad && ie >= 0) {  // the row's ends
        float v = 0.f;
        if (hard) v += w1 / s1 * ex2(fmaf(ze, kLog2e, -c1));
        if (soft) v += wt / st * ex2(fmaf(ze, itl, -ct));
        a.dlogits[row * V + ie] = __float2bfloat16_rn(v);
      }
      if (row + gridDim.x < a.rows) prepare(row + gridDim.x, par ^ 1);
      if (!grad) continue;
      named_sync<2>(CT + 32);  // the dense part of the row is written
      bf16* d = a.dlogits + row * V;
      for (int j = lane; j <= K; j += 32) {  // slot K: the target, if no slot names it
        const int i = j < K ? id[j] : (listed0 ? -1 : tgt0);
        if (i < 0) continue;
        bool first = true;
        float qs = j < K ? q[j] : 0.f;
        if (twice0) {
          qs = 0.f;
          for (int u = 0; u < K; ++u) {
            if (id[u] != i) continue;
            if (u < j) first = false;
            qs += q[u];
          }
        }
        if (!first) continue;
        const float x = j < K ? zj[j] : zt0;
        float v = 0.f;
        if (hard) {
          const float lp = kLn2 * (fmaf(x, kLog2e, -c1) - l1);
          v += w1 * (i == tgt0 ? expm1f(lp) : expf(lp));
        }
        if (soft0) v += wt * (ex2(fmaf(x, itl, -ct) - lt) - qs);
        d[i] = __float2bfloat16_rn(v);
      }
      __syncwarp();
    }
    return;
  }

  // the working warps
  int slot = 0, turn = 0;
  uint32_t ph = 0;
  auto step = [&] {
    if (++slot == NS) {
      slot = 0;
      ph ^= 1;
    }
  };
  auto free_slot = [&] {
    reads_before_copies();
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[slot]);
  };
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, ++turn) {
    const int par = turn & 1;
    place(row);
    const int slot0 = slot;
    const uint32_t ph0 = ph;
    float m = -INFINITY;
    f32x2 t0 = 0, t1 = 0, u0 = 0, u1 = 0;
    const f32x2 at2 = pair2(itl, itl), a12 = pair2(kLog2e, kLog2e);
    for (int c = 0; c < nc; ++c) {
      mbar_wait(&full[slot], ph, failed);
      const uint4* b = ring + slot * CV;
      uint4 r[U];
      if (c * CV + CV <= nvec) {
#pragma unroll
        for (int j = 0; j < U; ++j) r[j] = b[j * CT + tid];
      } else {
#pragma unroll
        for (int j = 0; j < U; ++j) {
          r[j] = make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);  // -inf: no probability
          if (c * CV + j * CT + tid < nvec) r[j] = b[j * CT + tid];
        }
      }
      if (!held) free_slot();
      step();
      // packed maxima: exact, and NaN passes by (it shows in the sums)
      __nv_bfloat162 mx = __halves2bfloat162(__ushort_as_bfloat16(0xFF80), __ushort_as_bfloat16(0xFF80));
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&r[j]);
#pragma unroll
        for (int k = 0; k < 4; ++k) mx = __hmax2(mx, h[k]);
      }
      const float mc = fmaxf(__low2float(mx), __high2float(mx));
      if (mc > m) {  // a new maximum: the sums so far move to it
        if (m != -INFINITY) {
          const float ft = ex2(__fmul_rn(m, itl) - __fmul_rn(mc, itl));
          t0 = mul2(t0, pair2(ft, ft));
          t1 = mul2(t1, pair2(ft, ft));
          if (TWO) {
            const float f1 = ex2(__fmul_rn(m, kLog2e) - __fmul_rn(mc, kLog2e));
            u0 = mul2(u0, pair2(f1, f1));
            u1 = mul2(u1, pair2(f1, f1));
          }
        }
        m = mc;
      }
      const float ref = m == -INFINITY ? 0.f : m;
      const float nct = -__fmul_rn(ref, itl), nc1 = -__fmul_rn(ref, kLog2e);
      const f32x2 ct2 = pair2(nct, nct), c12 = pair2(nc1, nc1);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const uint32_t w[4] = {r[j].x, r[j].y, r[j].z, r[j].w};
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
          const f32x2 x0 = wide2(w[k]), x1 = wide2(w[k + 1]);
          t0 = add2(t0, ex2_2(fma2(x0, at2, ct2)));
          t1 = add2(t1, ex2_2(fma2(x1, at2, ct2)));
          if (TWO) {
            u0 = add2(u0, ex2_2(fma2(x0, a12, c12)));
            u1 = add2(u1, ex2_2(fma2(x1, a12, c12)));
          }
        }
      }
    }
    {
      const float2 t = unpair2(add2(t0, t1)), u = unpair2(add2(u0, u1));
      const float wm = warp_max(m), M = wm == -INFINITY ? 0.f : wm;
      const bool none = m == -INFINITY;  // its sums are 0 (or NaN)
      const float st = warp_sum((t.x + t.y) * (none ? 1.f : ex2(__fmul_rn(m, itl) - __fmul_rn(M, itl))));
      const float s1 = TWO ? warp_sum((u.x + u.y) * (none ? 1.f : ex2(__fmul_rn(m, kLog2e) - __fmul_rn(M, kLog2e)))) : st;
      if (lane == 0) {
        part[par][warp][0] = wm;
        part[par][warp][1] = s1;
        part[par][warp][2] = st;
      }
    }
    named_sync<1>(CT + 32);
    if (!grad) continue;
    m = lane <= CW ? part[par][lane <= CW ? lane : 0][0] : -INFINITY;
    const float pm = m;
    m = warp_max(m);
    if (m == -INFINITY) m = 0.f;
    const float c1 = __fmul_rn(m, kLog2e), ct = __fmul_rn(m, itl);
    float s1 = 0.f, st = 0.f;
    if (lane <= CW) {
      const bool none = pm == -INFINITY;
      s1 = part[par][lane][1] * (none ? 1.f : ex2(__fmul_rn(pm, kLog2e) - c1));
      st = part[par][lane][2] * (none ? 1.f : ex2(__fmul_rn(pm, itl) - ct));
    }
    s1 = warp_sum(s1);
    st = warp_sum(st);
    const bool hard = s_tgt[par] >= 0, soft = s_soft[par];
    const float f1 = hard ? __fdividef(a.w_ce, s1) : 0.f, ft = soft ? __fdividef(a.w_kd * it, st) : 0.f;
    const float fs = TWO ? ft : f1 + ft;
    uint4* dv = reinterpret_cast<uint4*>(a.dlogits + row * V + head);
    const f32x2 ct2 = pair2(-ct, -ct), ft2 = pair2(fs, fs), c12 = pair2(-c1, -c1), f12 = pair2(f1, f1);
    if (held) {
      slot = slot0;
      ph = ph0;
    }
    for (int c = 0; c < nc; ++c) {
      if (!held) mbar_wait(&full[slot], ph, failed);
      const uint4* b = ring + slot * CV;
      uint4 r[U];  // beyond the row: whatever the ring holds, not stored
#pragma unroll
      for (int j = 0; j < U; ++j) r[j] = b[j * CT + tid];
      free_slot();
      step();
      if (hard || soft) {
#pragma unroll
        for (int j = 0; j < U; ++j) {
          const uint32_t w[4] = {r[j].x, r[j].y, r[j].z, r[j].w};
          uint32_t o[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const f32x2 x = wide2(w[k]);
            f32x2 v = mul2(ex2_2(fma2(x, at2, ct2)), ft2);
            if (TWO) v = fma2(ex2_2(fma2(x, a12, c12)), f12, v);
            const float2 t = unpair2(v);
            const __nv_bfloat162 h = __floats2bfloat162_rn(t.x, t.y);
            o[k] = *reinterpret_cast<const uint32_t*>(&h);
          }
          r[j] = make_uint4(o[0], o[1], o[2], o[3]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < U; ++j) r[j] = make_uint4(0, 0, 0, 0);
      }
      uint4* out = dv + c * CV + tid;
      if (c * CV + CV <= nvec) {
#pragma unroll
        for (int j = 0; j < U; ++j) out[j * CT] = r[j];
      } else {
#pragma unroll
        for (int j = 0; j < U; ++j)
          if (c * CV + j * CT + tid < nvec) out[j * CT] = r[j];
      }
    }
    named_arrive<2>(CT + 32);
  }
}

// ------------------------------------------------------------------ router balance
// Groups of S tokens, n valid ones each, c[e] of their n k choices going to expert e, f = c / (n k):
//   balance = alpha E / G sum_g sum_e f_e P_e, P_e = mean over valid t of p_te = softmax(logits_t)_e,
//   z loss  = zc / G sum_g mean over valid t of lse_t^2,
//   dlogit_te = alpha E / (G n) p_te (f_e - sum_j f_j p_tj) + 2 zc / (G n) lse_t p_te.
// f needs every choice of the group before the first gradient, but only the
// choices (4 k bytes a token): a first kernel counts them, a second reads the
// logits once and does everything else (131072 tokens of 128: 28 us captured, of
// which the bytes need 15).  The second starts while the first
// runs (programmatic launch) and waits for the counts only after its first
// rows are loaded and their softmax is taken.
constexpr int BAL_MAX_E = 512;
constexpr int BAL_COUNT_THREADS = 512;
constexpr int BAL_THREADS = 512;

// Choices per expert and valid tokens of one part of a group per block:
// parts[g][part][e], the valid tokens at e = E.  A thread takes whole tokens,
// four at a time so that their loads overlap.  The counters are laid out
// [expert][lane], so that the lanes of a warp never meet in one bank or one
// address; integer sums do not depend on the order of the atomics.
__global__ void __launch_bounds__(BAL_COUNT_THREADS) balance_count_k(const int32_t* __restrict__ idx,
                                                                     const uint8_t* __restrict__ valid, int S, int E,
                                                                     int k, int per, int ldp,
                                                                     int32_t* __restrict__ parts,
                                                                     int* __restrict__ ticket) {
  extern __shared__ int hist[];  // [E][32]
  __shared__ int wn[BAL_COUNT_THREADS / 32];
  dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t g = blockIdx.y;
  for (int i = threadIdx.x; i < E * 32; i += BAL_COUNT_THREADS) hist[i] = 0;
  __syncthreads();
  int live = 0;
  auto add = [&](int e) {
    if (e >= 0 && e < E) atomicAdd(&hist[e * 32 + lane], 1);
  };
  const int t1 = min(S, (int)(blockIdx.x + 1) * per);
  for (int t0 = (int)blockIdx.x * per + threadIdx.x; t0 < t1; t0 += 4 * BAL_COUNT_THREADS) {
    bool on[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int t = t0 + u * BAL_COUNT_THREADS;
      on[u] = t < t1 && (!valid || valid[g * S + t]);
      live += on[u];
    }
    for (int i = 0; i < k; i += 4) {
      int4 q[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int32_t* p = idx + (g * S + t0 + u * BAL_COUNT_THREADS) * k + i;
        q[u] = make_int4(-1, -1, -1, -1);
        if (!on[u]) continue;
        if ((k & 3) == 0) {
          q[u] = *reinterpret_cast<const int4*>(p);
        } else {
          q[u].x = p[0];
          if (i + 1 < k) q[u].y = p[1];
          if (i + 2 < k) q[u].z = p[2];
          if (i + 3 < k) q[u].w = p[3];
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        add(q[u].x);
        add(q[u].y);
        add(q[u].z);
        add(q[u].w);
      }
    }
  }
  live = __reduce_add_sync(0xffffffffu, live);
  if (lane == 0) wn[warp] = live;
  __syncthreads();
  int32_t* out = parts + (g * gridDim.x + blockIdx.x) * ldp;
  for (int e = warp; e < E; e += BAL_COUNT_THREADS / 32) {
    const int c = __reduce_add_sync(0xffffffffu, hist[e * 32 + lane]);
    if (lane == 0) out[e] = c;
  }
  if (threadIdx.x == 0) {
    int c = 0;
#pragma unroll
    for (int w = 0; w < BAL_COUNT_THREADS / 32; ++w) c += wn[w];
    out[E] = c;
    if (blockIdx.x == 0) {
      ticket[1 + g] = 0;
      if (g == 0) ticket[0] = 0;
    }
  }
}

struct BalArgs {
  const float* logits;
  const uint8_t* valid;
  int64_t G;
  int S, E, k, rows, nblk, ldp;
  float alpha, z_coef;  // both over G
  int nparts;
  const int32_t* parts;  // [G][nparts][ldp] of the counting kernel
  int32_t* counts;
  bf16* dlogits;
  float *prob, *loss;
  float* partial;  // [G][nblk][ldp]: E sums of p, the sum of lse^2, zeros
  float2* gloss;   // [G]
  int* ticket;     // [1 + G], zeroed by the counting kernel
};

// LPR lanes share a row, each holding NV vectors of 8 logits (vector j of a
// lane: elements 8 (j LPR + lane) ..).  A block takes a.rows rows of one group,
// as many at a time as it has lanes for.  VEC: E is a multiple of 8; rows are
// written as 16-byte vectors and come through a ring of BAL_STAGES chunks of
// shared memory, filled by bulk copies (one register set ahead, a block had 16
// KB on its way and an SM 4 of the 7 TB/s' worth; the ring holds four times
// that).  The block that finishes a group last adds the blocks' sums in block
// order, and the one that finishes the last group adds the groups' losses.
constexpr int BAL_STAGES = 4;

// Lanes that share a row, vectors a lane holds, rows a block has at a time.
// With many long rows that come as vectors a lane holds two of them: the shuffles
// and logarithms of a row weigh half as much (131072 rows of 128: 28.3 us against
// 30.6, but 4096: 11.3 against 10.1).
constexpr bool bal_wide(int64_t T, int E) { return E % 8 == 0 && (E > 256 || (E > 64 && T >= 32768)); }
constexpr int bal_lanes(int64_t T, int E) {
  const int e = bal_wide(T, E) ? E / 2 : E;
  return e <= 8 ? 1 : e <= 16 ? 2 : e <= 32 ? 4 : e <= 64 ? 8 : e <= 128 ? 16 : 32;
}
constexpr int bal_rows(int64_t T, int E) { return BAL_THREADS / bal_lanes(T, E); }

template <int LPR, int NV, bool VEC>
__global__ void __launch_bounds__(BAL_THREADS, NV == 1 ? 2 : 1) balance_grad_k(const BalArgs a) {
  constexpr int RPB = BAL_THREADS / LPR;  // rows in flight per block
  constexpr int WARPS = BAL_THREADS / 32;
  constexpr int NE = LPR * NV * 8;        // columns the lanes of a row cover
  __shared__ float acc[WARPS][NE + 1];
  __shared__ __align__(16) float tree[4 * BAL_THREADS];
  __shared__ float red[WARPS];
  __shared__ int last;
  __shared__ int cnt[NE + 1];  // the group's choices per expert, its valid tokens at E
  extern __shared__ __align__(128) float ring[];  // VEC: [BAL_STAGES][RPB][E]
  __shared__ uint64_t full[BAL_STAGES];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int sub = tid % LPR, slot = tid / LPR;
  const int64_t g = blockIdx.y;
  const int E = a.E;
  const int r1 = min(a.S, (int)(blockIdx.x + 1) * a.rows);
  const int first = (int)blockIdx.x * a.rows + slot;
  constexpr int NP = NV * 4;  // pairs of columns a lane holds
  f32x2 x[NP], f[NP], P[NP];
  float zz = 0.f;
  const int r0 = (int)blockIdx.x * a.rows, chunks = (r1 - r0 + RPB - 1) / RPB;
  const float* src = a.logits + (g * a.S + first) * E + sub * 8;
  bf16* dst = a.dlogits + (g * a.S + first) * E + sub * 8;
  const uint8_t* val = a.valid ? a.valid + g * a.S + first : nullptr;
  bool failed = false;
  auto fill = [&](int c) {  // one thread: chunk c into its stage of the ring
    const uint32_t bytes = (uint32_t)min(RPB, r1 - r0 - c * RPB) * (uint32_t)E * 4;
    mbar_expect_tx(&full[c % BAL_STAGES], bytes);
    bulk_load(ring + (c % BAL_STAGES) * RPB * E, a.logits + (g * a.S + r0 + c * RPB) * E, bytes, &full[c % BAL_STAGES]);
  };
  if (VEC) {
    if (tid == 0) {
      for (int i = 0; i < BAL_STAGES; ++i) mbar_init(&full[i], 1);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
      for (int c = 0; c < min(chunks, BAL_STAGES); ++c) fill(c);
    }
    __syncthreads();
  }
  const f32x2 nothing = pair2(-INFINITY, -INFINITY);
  auto load = [&](int c, bool on) {  // this lane's part of its row of chunk c
    const float* in = VEC ? ring + ((c % BAL_STAGES) * RPB + slot) * E + sub * 8 : src;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e = (j * LPR + sub) * 8;
      if (VEC) {
        x[4 * j] = x[4 * j + 1] = x[4 * j + 2] = x[4 * j + 3] = nothing;
        if (on && e < E) {
          const ulonglong2* p = reinterpret_cast<const ulonglong2*>(in + j * LPR * 8);
          const ulonglong2 u = p[0], w = p[1];
          x[4 * j] = u.x;
          x[4 * j + 1] = u.y;
          x[4 * j + 2] = w.x;
          x[4 * j + 3] = w.y;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[4 * j + i] = pair2(on && e + 2 * i < E ? in[j * LPR * 8 + 2 * i] : -INFINITY,
                               on && e + 2 * i + 1 < E ? in[j * LPR * 8 + 2 * i + 1] : -INFINITY);
      }
    }
  };
  auto over_row = [&](float v, auto op) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  };
  auto sum = [](float u, float w) { return u + w; };
  auto mx = [](float u, float w) { return fmaxf(u, w); };
#pragma unroll
  for (int i = 0; i < NP; ++i) P[i] = f[i] = 0;
  float cz = 0.f, cb = 0.f, inv_n = 0.f;
  bool started = false;
  const f32x2 l2e = pair2(kLog2e, kLog2e);
  constexpr float kLn2 = 0.6931471805599453f;
  int r = first;
  bool on = r < r1 && (!val || *val);
  // the same number of turns for every lane of a warp: the shuffles are warp-wide
  for (int turn = 0; turn < chunks; ++turn, r += RPB) {
    const bool now = on;
    if (VEC) mbar_wait(&full[turn % BAL_STAGES], (uint32_t)(turn / BAL_STAGES) & 1, failed);
    load(turn, now);
    src += (int64_t)RPB * E;
    if (val) val += RPB;
    on = r + RPB < r1 && (!val || *val);
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const float2 t = unpair2(x[i]);
      m = fmaxf(m, fmaxf(t.x, t.y));
    }
    m = over_row(m, mx);
    if (VEC) {
      reads_before_copies();
      __syncthreads();  // every lane has its part: the stage takes the next chunk
      if (tid == 0 && turn + BAL_STAGES < chunks) fill(turn + BAL_STAGES);
    }
    // 2^(x log2(e) - c) with c = fl(m log2(e)): the rounding of c cancels.  Padded
    // rows and lanes beyond E hold -inf, whose exponential is 0.
    const float c = m == -INFINITY ? 0.f : __fmul_rn(m, kLog2e);
    const f32x2 nc = pair2(-c, -c);
    f32x2 e2[NP], s2 = 0, f2 = 0;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      e2[i] = ex2_2(fma2(x[i], l2e, nc));
      s2 = add2(s2, e2[i]);
    }
    if (!started) {
      started = true;
      dep_wait();  // the counts and the tickets
      for (int i = tid; i <= E; i += BAL_THREADS) cnt[i] = 0;
      __syncthreads();
      const int32_t* pc = a.parts + g * a.nparts * a.ldp;
      const int lanes = max(1, BAL_THREADS / (E + 1));  // threads that share a column, each taking every lanes-th part
      for (int i = tid; i < lanes * (E + 1); i += BAL_THREADS) {
        const int e = i % (E + 1);
        int n = 0;
#pragma unroll 8
        for (int q = i / (E + 1); q < a.nparts; q += lanes) n += pc[q * a.ldp + e];
        atomicAdd(&cnt[e], n);
      }
      __syncthreads();
      const int n = cnt[E];
      if (blockIdx.x == 0)
        for (int e = tid; e < E; e += BAL_THREADS) a.counts[g * E + e] = cnt[e];
      inv_n = n > 0 ? 1.f / (float)n : 0.f;
      cb = a.alpha * (float)E * inv_n;
      cz = 2.f * a.z_coef * inv_n;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int e = ((i >> 2) * LPR + sub) * 8 + 2 * (i & 3);
        f[i] = pair2(e < E ? (float)cnt[e] * inv_n / (float)a.k : 0.f,
                     e + 1 < E ? (float)cnt[e + 1] * inv_n / (float)a.k : 0.f);
      }
    }
#pragma unroll
    for (int i = 0; i < NP; ++i) f2 = fma2(f[i], e2[i], f2);
    const float2 st = unpair2(s2), ft = unpair2(f2);
    const float s = over_row(st.x + st.y, sum), fe = over_row(ft.x + ft.y, sum);
    const float is = now ? __fdividef(1.f, s) : 0.f;
    const float lse = now ? kLn2 * (__log2f(s) + c) : 0.f;
    const float shift = cz * lse - cb * (fe * is);
    const f32x2 is2 = pair2(is, is), cb2 = pair2(cb, cb), sh2 = pair2(shift, shift);
    if (sub == 0) zz += lse * lse;
    uint32_t o[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const f32x2 p = mul2(e2[i], is2);
      P[i] = add2(P[i], p);
      const float2 t = unpair2(mul2(p, fma2(f[i], cb2, sh2)));
      const __nv_bfloat162 h = __floats2bfloat162_rn(t.x, t.y);
      o[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    if (a.dlogits && r < r1) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int e = (j * LPR + sub) * 8;
        if (VEC) {
          if (e < E)
            *reinterpret_cast<uint4*>(dst + j * LPR * 8) = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (e + i < E)
              dst[j * LPR * 8 + i] = __ushort_as_bfloat16((unsigned short)(o[4 * j + (i >> 1)] >> (16 * (i & 1))));
        }
      }
    }
    dst += (int64_t)RPB * E;
  }
  if (VEC && failed && tid == 0) {  // what is on its way lands before the block's memory goes
    const long long t0 = clock64();
    while (clock64() - t0 < kWaitCycles) {
    }
  }
  // the block's sums: rows of a warp by shuffles, warps in warp order
#pragma unroll
  for (int i = 0; i < NP; ++i) {
#pragma unroll
    for (int o = 16; o >= LPR; o >>= 1) P[i] = add2(P[i], __shfl_xor_sync(0xffffffffu, P[i], o));
    const float2 t = unpair2(P[i]);
    if (lane < LPR) {
      acc[warp][((i >> 2) * LPR + sub) * 8 + 2 * (i & 3)] = t.x;
      acc[warp][((i >> 2) * LPR + sub) * 8 + 2 * (i & 3) + 1] = t.y;
    }
  }
  zz = warp_sum(zz);
  if (lane == 0) acc[warp][NE] = zz;
  __syncthreads();
  // (a group of one block has its sums at hand: no trip through memory)
  float* part = a.nblk == 1 ? tree : a.partial + (g * a.nblk + blockIdx.x) * a.ldp;
  for (int e = tid; e < a.ldp; e += BAL_THREADS) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) v += e <= E ? acc[w][e < E ? e : NE] : 0.f;
    part[e] = v;
  }
  int C = 1;
  if (a.nblk > 1) {
    __threadfence();
    __syncthreads();
    if (tid == 0) last = atomicAdd(&a.ticket[1 + g], 1) == a.nblk - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
    // the group: thread (c, q) adds the four columns q of blocks c, c + C, ... in order, then the C parts in order
    const int c4 = a.ldp / 4;
    C = max(1, min(a.nblk, BAL_THREADS / c4));
    const float4* all = reinterpret_cast<const float4*>(a.partial + g * a.nblk * a.ldp);
    if (tid < C * c4) {
      const int c = tid / c4, q = tid % c4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
      for (int b = c; b < a.nblk; b += C) {
        const float4 u = __ldcg(all + (int64_t)b * c4 + q);
        v.x += u.x;
        v.y += u.y;
        v.z += u.z;
        v.w += u.w;
      }
      reinterpret_cast<float4*>(tree)[tid] = v;
    }
  }
  __syncthreads();
  float lb = 0.f, lz = 0.f;
  for (int e = tid; e <= E; e += BAL_THREADS) {
    float v = 0.f;
    for (int c = 0; c < C; ++c) v += tree[c * a.ldp + e];
    v *= inv_n;
    if (e < E) {
      a.prob[g * E + e] = v;
      lb += (float)cnt[e] * inv_n / (float)a.k * v;
    } else {
      lz = v;
    }
  }
  lb = block_sum<BAL_THREADS>(lb, red);
  lz = block_sum<BAL_THREADS>(lz, red);
  if (a.G > 1) {
    if (tid == 0) {
      a.gloss[g] = make_float2(lb, lz);
      __threadfence();
      last = atomicAdd(&a.ticket[0], 1) == a.G - 1;
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    lb = lz = 0.f;
    for (int64_t i = tid; i < a.G; i += BAL_THREADS) {
      const float2 v = __ldcg(a.gloss + i);
      lb += v.x;
      lz += v.y;
    }
    lb = block_sum<BAL_THREADS>(lb, red);
    lz = block_sum<BAL_THREADS>(lz, red);
  }
  if (tid == 0) {
    a.loss[0] = lb * a.alpha * (float)E;
    a.loss[1] = lz * a.z_coef;
  }
}

inline bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
inline int64_t up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

// Tokens a linear cross-entropy call keeps the exponentials of at a time: as
// many as fit kPieceBytes, at least 1024 (a chunk re-reads the weights for
// every product, so short chunks are bound by memory), the chunks of one call
// equal up to the 256-row tile.
// the blocks of 512 threads that the SMs hold at once
constexpr int64_t bal_blocks(int64_t T, int E) { return bal_wide(T, E) && E <= 256 ? 152 : 304; }
constexpr int64_t kPieceBytes = (int64_t)3 << 30;
int64_t ce_chunk(int64_t T, int V) {
  int64_t most = kPieceBytes / (2 * up(V, 64)) / 256 * 256;
  if (most < 2048) most = 2048;
  if (T <= most) return T;
  const int64_t n = (T + most - 1) / most;
  return up((T + n - 1) / n, 256);
}

// Runs that the sum over V of a chunk's dh is cut into.  Its tiles are long (V
// / 64 K blocks each) and few (rows / 256 by H / 256); they go first and dW's
// short tiles fill up behind them, so a cut is needed only where the last long
// tile would end after its share of all work: 76 CTA pairs, a K block as the
// unit, 10 of them for an epilogue that no main loop hides (few rows).  A cut
// has to save 24 units (about 8 us), what adding the runs costs.
int ce_runs(int64_t rows, int H, int V, bool dW) {
  const int64_t pairs = 76, nh = (H + 255) / 256, n = (rows + 255) / 256 * nh, nk = (V + 63) / 64;
  if (n >= 2 * pairs) return 1;  // two waves and more even out
  const int64_t w = (rows + 63) / 64 < 10 ? 10 : (rows + 63) / 64;
  const double share = ((double)n * nk + (dW ? (double)((V + 255) / 256) * nh * w : 0.0)) / pairs;
  auto end = [&](int64_t k) { return (double)((n * k + pairs - 1) / pairs * ((nk + k - 1) / k)); };
  int best = 1;
  for (int k = 2; k <= 32 && nk / k >= 8 && end(best) > 1.05 * share; ++k) {
    const int64_t per = (nk + k - 1) / k;
    if ((nk + per - 1) / per != k) continue;  // the last run would be empty
    if (end(k) < end(best) - (best == 1 ? 24.0 : 0.0)) best = k;
  }
  return best;
}

struct CeScratch {
  int* ctr;
  float2* stat;
  float* zt;
  uint16_t* E;
  bf16* hm;
  float *dWacc, *slabs;
  int64_t ldE, chunk;
  int npieces, runs, per;  // per: rows of W of a backward block, few tokens
  float* z;
  int ldz;
  int one;               // few tokens: the form that reads W once (0: it is read twice)
  int dw_x, dw_per;      // blocks that make dW alone, and their rows of W
};
bool ce_few(int64_t T, int H) { return T <= FEW_T && (int64_t)few_held((int)T) * few_stride(H) <= FEW_SMEM; }
// The form of ce_few_one_k, its column groups of a warp times its warps: the
// least that holds a row of H; 0: W is read twice, because no form does, or
// because rows are so narrow that the barrier of a stage outweighs its work (7
// tokens of 88 by 48042, losses alone: 7.0 us against 14.6 in one pass).
int few_one(int64_t T, int H) {
  const int groups = (H + 31) / 32;
  return groups <= 4    ? 0
         : groups <= 16 ? 4 * 4
         : groups <= 32 ? 4 * 8
         : groups <= 64 ? 8 * 8
                        : groups <= 128 && T <= 8 ? 16 * 8 : 0;
}
size_t ce_carve(int64_t T, int H, int V, bool grads, bool dW, uint8_t* base, CeScratch* w) {
  size_t off = 0;
  auto take = [&](int64_t bytes) {
    uint8_t* p = base ? base + off : nullptr;
    off += (size_t)up(bytes, 256);
    return p;
  };
  if (ce_few(T, H)) {
    // forward blocks: what shared memory lets an SM hold, at most four; backward
    // blocks: the two or three per SM that run at once, of at least one stage of
    // rows each
    const int64_t smem = few_held((int)T) * few_stride(H), fit = FEW_SMEM / smem < 4 ? FEW_SMEM / smem : 4;
    const int sub = few_sub(H);
    const int64_t most = (V + FEW_ROWS - 1) / FEW_ROWS, ny = (H + FEW_COLS - 1) / FEW_COLS;
    w->npieces = (int)(most < 152 * fit ? most : 152 * fit);  // where W is read twice
    const int64_t bps = 226 * 1024 / (few_smem((int)T, H, true) + 1024) < 3 ? 2 : 3;
    int64_t nx = 152 * bps / ny > 0 ? 152 * bps / ny : 1;
    if (nx > (V + sub - 1) / sub) nx = (V + sub - 1) / sub;
    w->per = (int)up((V + nx - 1) / nx, sub);
    w->runs = (V + w->per - 1) / w->per;
    w->chunk = T;
    w->ldz = (int)up(V + sub, 64);
    w->one = few_one(T, H);
    if (w->one) {
      // as many blocks as run at once, of at least 32 rows each: each leaves a
      // slab of dh to add (16 tokens of 256 by 8192: 16.7 us, with 16 rows 25.2)
      const int nw = w->one == 16 ? 4 : 8;
      const int64_t nb = 152 * one_blocks(few_held((int)T) / 8, w->one / nw, nw), most = (V + 31) / 32;
      w->npieces = (int)(most < nb ? most : nb);
    }
    int64_t dx = 152 * 6 / ny > 0 ? 152 * 6 / ny : 1;
    if (dx > (V + 2 * sub - 1) / (2 * sub)) dx = (V + 2 * sub - 1) / (2 * sub);
    w->dw_per = (int)up((V + dx - 1) / dx, sub);
    w->dw_x = (V + w->dw_per - 1) / w->dw_per;
    w->stat = (float2*)take(T * w->npieces * 8);
    w->zt = (float*)take(T * 4);
    w->z = grads ? (float*)take(T * w->ldz * 4) : nullptr;
    w->slabs = grads ? (float*)take((int64_t)(w->one ? w->npieces : w->runs) * T * H * 4) : nullptr;
    return off;
  }
  w->chunk = ce_chunk(T, V);
  w->npieces = (V + 127) / 128;
  w->ldE = up(V, 64);
  w->ctr = (int*)take(256);
  w->stat = (float2*)take(w->chunk * w->npieces * 8);
  w->zt = (float*)take(w->chunk * 4);
  w->E = grads ? (uint16_t*)take(w->chunk * w->ldE * 2) : nullptr;
  w->hm = grads ? (bf16*)take(w->chunk * H * 2) : nullptr;
  w->dWacc = grads && w->chunk < T ? (float*)take((int64_t)V * H * 4) : nullptr;
  // the runs with dW beside them or without: room for the larger number
  const int a = grads ? ce_runs(w->chunk, H, V, true) : 1, b = grads ? ce_runs(w->chunk, H, V, false) : 1;
  w->runs = dW ? a : b;
  const int most = a > b ? a : b;
  w->slabs = most > 1 ? (float*)take((int64_t)most * w->chunk * H * 4) : nullptr;
  return off;
}
bool ce_shape_ok(int64_t T, int H, int V) {
  return T >= 0 && T <= ((int64_t)1 << 40) && H > 0 && H % 8 == 0 && V > 0 && V <= (1 << 21);
}

struct BalScratch {
  int32_t* parts;
  int* ticket;
  float2* gloss;
  float* partial;
  int nblk, rows, ldp, nparts;
};
size_t bal_carve(int64_t T, int S, int E, uint8_t* base, BalScratch* w) {
  size_t off = 0;
  auto take = [&](int64_t bytes) {
    uint8_t* p = base ? base + off : nullptr;
    off += (size_t)up(bytes, 256);
    return p;
  };
  const int64_t G = T / S;
  int64_t blk = (bal_blocks(T, E) + G - 1) / G;
  const int64_t most = (S + bal_rows(T, E) - 1) / bal_rows(T, E);  // a block has all its lanes' rows to take
  if (blk > most) blk = most;
  w->rows = (int)((S + blk - 1) / blk);
  w->nblk = (S + w->rows - 1) / w->rows;
  // counting blocks of a group: at least 512 tokens each, 64 at most in all
  const int64_t parts = (S + 511) / 512, cap = (64 + G - 1) / G;
  w->nparts = (int)(parts < cap ? parts : cap);
  w->ldp = (int)up(E + 1, 4);
  w->parts = (int32_t*)take(G * w->nparts * w->ldp * 4);
  w->ticket = (int*)take((1 + G) * 4);
  w->gloss = (float2*)take(G * 8);
  w->partial = (float*)take(G * w->nblk * w->ldp * 4);
  return off;
}
bool bal_shape_ok(int64_t T, int S, int E) {
  return T >= 0 && S > 0 && T % S == 0 && T / S <= 65535 && E >= 1 && E <= BAL_MAX_E;
}

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, int cluster, bool dependent,
                   cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  unsigned n = 0;
  if (cluster > 0) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = (unsigned)cluster;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (dependent) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int LPR, int NV, bool VEC>
cudaError_t launch_balance_grad(const BalArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)a.nblk, (unsigned)a.G);
  if (!VEC) return launch(balance_grad_k<LPR, NV, VEC>, grid, BAL_THREADS, 0, 0, true, s, a);
  constexpr int DEV = 16;
  static std::atomic<int> done[DEV];  // room for the whole ring, set once per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev >= DEV || !done[dev].load(std::memory_order_acquire))) {
    e = cudaFuncSetAttribute(balance_grad_k<LPR, NV, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(BAL_STAGES * (size_t)BAL_THREADS * NV * 32));
    if (e == cudaSuccess && dev < DEV) done[dev].store(1, std::memory_order_release);
  }
  if (e != cudaSuccess) return e;
  // no more stages than the block has chunks for
  const int chunks = (a.rows + BAL_THREADS / LPR - 1) / (BAL_THREADS / LPR);
  const size_t smem = (size_t)(BAL_THREADS / LPR) * a.E * 4 * (chunks < BAL_STAGES ? chunks : BAL_STAGES);
  return launch(balance_grad_k<LPR, NV, VEC>, grid, BAL_THREADS, smem, 0, true, s, a);
}

// The join and the sum of runs stand between two GEMMs that use nearly all
// shared memory: they ask for the same split of it and the L1 cache, which an
// SM changes only when it is empty.  Set once per device.
cudaError_t share_memory_config() {
  constexpr int DEV = 16;
  static std::atomic<int> done[DEV];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < DEV && done[dev].load(std::memory_order_acquire))) return e;
  e = cudaFuncSetAttribute(ce_join_k, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(ce_add_runs_k, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
  if (e == cudaSuccess && dev < DEV) done[dev].store(1, std::memory_order_release);
  return e;
}

// Blocks of a distillation kernel that are resident at once, looked up once per
// device, form and slot room.
template <int CW, int U, int NS, int BPS, bool TWO>
cudaError_t distill_resident(int kcap, int* out) {
  constexpr int DEV = 16;
  static std::atomic<int> known[DEV][6];
  int dev = 0, ki = 0, sms = 0, n = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  while ((32 << ki) < kcap) ++ki;
  std::atomic<int>* slot = dev < DEV ? &known[dev][ki] : nullptr;
  if (slot && (*out = slot->load(std::memory_order_acquire)) > 0) return cudaSuccess;
  // room for the most slots, so that the setting never shrinks under another call
  e = cudaFuncSetAttribute(distill_k<CW, U, NS, BPS, TWO>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)kd_smem<CW, U, NS>(KD_MAX_K));
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess)
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, distill_k<CW, U, NS, BPS, TWO>, (CW + 2) * 32,
                                                      kd_smem<CW, U, NS>(kcap));
  if (e != cudaSuccess) return e;
  if (n < 1) return cudaErrorInvalidConfiguration;
  *out = n * sms;
  if (slot) slot->store(*out, std::memory_order_release);
  return cudaSuccess;
}

template <int CW, int U, int NS, int BPS, bool TWO>
cudaError_t launch_distill2(const KdArgs& a, cudaStream_t s) {
  int n = 0;
  const cudaError_t e = distill_resident<CW, U, NS, BPS, TWO>(a.kcap, &n);
  if (e != cudaSuccess) return e;
  if (n > a.rows) n = (int)a.rows;
  return launch(distill_k<CW, U, NS, BPS, TWO>, dim3((unsigned)n), (CW + 2) * 32, kd_smem<CW, U, NS>(a.kcap), 0, false, s, a);
}
template <int CW, int U, int NS, int BPS>
cudaError_t launch_distill(const KdArgs& a, cudaStream_t s) {
  return a.target && a.tau != 1.f ? launch_distill2<CW, U, NS, BPS, true>(a, s) : launch_distill2<CW, U, NS, BPS, false>(a, s);
}

// Room for a kernel's shared memory, set once per device.
template <auto KERNEL>
cudaError_t allow_smem(int bytes) {
  constexpr int DEV = 16;
  static std::atomic<int> done[DEV];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev >= DEV || !done[dev].load(std::memory_order_acquire))) {
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < DEV) done[dev].store(1, std::memory_order_release);
  }
  return e;
}

template <int NT, int KP, int NW>
cudaError_t launch_few_one(const bf16* h, const bf16* W, const int32_t* target, int T, int H, int V, bool dh,
                           const CeScratch& w, cudaStream_t s) {
  const cudaError_t e = allow_smem<ce_few_one_k<NT, KP, NW>>(one_smem(NT, KP, NW));
  if (e != cudaSuccess) return e;
  return launch(ce_few_one_k<NT, KP, NW>, dim3((unsigned)w.npieces), NW * 32, (size_t)one_smem(NT, KP, NW), 0, false, s, h,
                W, target, T, H, V, w.ldz, w.z, w.stat, w.zt, dh ? w.slabs : nullptr);
}

// Losses and gradients from z and the blocks' statistics.
cudaError_t launch_few_bwd(const bf16* h, const bf16* W, const int32_t* target, int T, int H, int V, float g,
                           float* row_loss, bf16* dh, bf16* dW, const CeScratch& w, cudaStream_t s) {
  const unsigned ny = (unsigned)((H + FEW_COLS - 1) / FEW_COLS);
  if (dh && !w.one) {
    constexpr int a = few_smem(FEW_T, 8, true), b = few_smem(FEW_T, 512, true);  // the largest ring
    const cudaError_t e = allow_smem<ce_few_bwd_k<true>>(a > b ? a : b);
    if (e != cudaSuccess) return e;
    return launch(ce_few_bwd_k<true>, dim3((unsigned)w.runs, ny), FEW_THREADS, (size_t)few_smem(T, H, true), 0, true, s, h,
                  W, target, T, H, V, w.ldz, (const float*)w.z, (const float2*)w.stat, w.npieces, (const float*)w.zt, w.per,
                  g, row_loss, w.slabs, dW, 0, (bf16*)nullptr);
  }
  const unsigned first = dh ? (unsigned)T * (unsigned)((H + 127) / 128) : dW ? 0u : (unsigned)T;
  const unsigned nx = dW ? (unsigned)w.dw_x : first, fy = (first + nx - 1) / nx;
  return launch(ce_few_bwd_k<false>, dim3(nx, fy + (dW ? ny : 0u)), FEW_THREADS, (size_t)few_smem(T, H, false), 0, true, s,
                h, W, target, T, H, V, w.ldz, (const float*)w.z, (const float2*)w.stat, w.npieces, (const float*)w.zt,
                w.dw_per, g, row_loss, w.slabs, dW, (int)fy, dh);
}

template <int HELD>
cudaError_t launch_few_fwd(const bf16* h, const bf16* W, const int32_t* target, int T, int H, int V, const CeScratch& w,
                           cudaStream_t s) {
  const cudaError_t e = allow_smem<ce_few_fwd_k<HELD>>(FEW_SMEM);  // the widest h
  if (e != cudaSuccess) return e;
  return launch(ce_few_fwd_k<HELD>, dim3((unsigned)w.npieces), FEW_WARPS * 32, (size_t)HELD * few_stride(H), 0, false, s,
                h, W, target, T, H, V, w.ldz, w.z, w.stat, w.zt);
}

// Linear cross-entropy of up to sixteen tokens.
cudaError_t linear_ce_few(const bf16* h, const bf16* W, const int32_t* target, int T, int H, int V, float g,
                          float* row_loss, bf16* dh, bf16* dW, const CeScratch& w, cudaStream_t s) {
  cudaError_t e = cudaErrorInvalidValue;
  const bool d = dh != nullptr;
  switch (T <= 8 ? w.one : w.one + 1) {
    case 0: e = launch_few_fwd<8>(h, W, target, T, H, V, w, s); break;
    case 1: e = launch_few_fwd<16>(h, W, target, T, H, V, w, s); break;
    case 16: e = launch_few_one<1, 4, 4>(h, W, target, T, H, V, d, w, s); break;
    case 17: e = launch_few_one<2, 4, 4>(h, W, target, T, H, V, d, w, s); break;
    case 32: e = launch_few_one<1, 4, 8>(h, W, target, T, H, V, d, w, s); break;
    case 33: e = launch_few_one<2, 4, 8>(h, W, target, T, H, V, d, w, s); break;
    case 64: e = launch_few_one<1, 8, 8>(h, W, target, T, H, V, d, w, s); break;
    case 65: e = launch_few_one<2, 8, 8>(h, W, target, T, H, V, d, w, s); break;
    case 128: e = launch_few_one<1, 16, 8>(h, W, target, T, H, V, d, w, s); break;
  }
  if (e == cudaSuccess) e = launch_few_bwd(h, W, target, T, H, V, g, row_loss, dh, dW, w, s);
  if (e != cudaSuccess || !dh || w.one) return e;
  const int64_t n4 = (int64_t)T * H / 4;
  return launch(ce_add_runs_k, dim3((unsigned)((n4 + 31) / 32)), RUN_WARPS * 32, 0, 0, true, s,
                reinterpret_cast<const float4*>(w.slabs), n4, w.runs, g, reinterpret_cast<uint2*>(dh));
}

}  // namespace

// ------------------------------------------------------------------ launchers
size_t linear_cross_entropy_scratch(int64_t T, int H, int V, bool grads) {
  if (!ce_shape_ok(T, H, V)) return 0;
  CeScratch w;
  return ce_carve(T, H, V, grads, true, nullptr, &w);
}

cudaError_t linear_cross_entropy(const bf16* h, const bf16* W, const int32_t* target, int64_t T, int H, int V, float g,
                                 float* row_loss, bf16* dh, bf16* dW, void* scratch, size_t scratch_bytes,
                                 cudaStream_t s) {
  const bool grads = dh || dW;
  if (!ce_shape_ok(T, H, V) || !al16(h) || !al16(W) || !al16(dh) || !al16(dW) ||
      (reinterpret_cast<uintptr_t>(scratch) & 255))
    return cudaErrorInvalidValue;
  CeScratch w;
  if (ce_carve(T, H, V, grads, dW != nullptr, (uint8_t*)scratch, &w) > scratch_bytes) return cudaErrorInvalidValue;
  if (T == 0) return cudaSuccess;
  if (ce_few(T, H)) return linear_ce_few(h, W, target, (int)T, H, V, g, row_loss, dh, dW, w, s);
  // tiles are drawn from a counter where some pair takes more than one
  const int64_t nt = (w.chunk + 255) / 256, nv = (V + 255) / 256, nh = (H + 255) / 256;
  const bool draw = nt * nv > 76 || nh * (nt * w.runs + nv) > 76;
  cudaError_t e = cudaSuccess;
  if (draw && (e = cudaMemsetAsync(w.ctr, 0, 256, s)) != cudaSuccess) return e;
  int* ctr = draw ? w.ctr : nullptr;
  if ((e = share_memory_config()) != cudaSuccess) return e;
  for (int64_t c0 = 0; c0 < T; c0 += w.chunk) {
    const int rows = (int)(T - c0 < w.chunk ? T - c0 : w.chunk);
    const bool first = c0 == 0, last = c0 + rows >= T;
    const SoftmaxPieces sp{w.stat, w.npieces, target + c0, w.zt, w.E, w.ldE};
    e = gemm_softmax_pieces(h + c0 * H, W, rows, V, H, sp, ctr, !first, s);
    if (e != cudaSuccess) return e;
    // few rows: several blocks share each, down to about 2048 columns a block
    const int want = 1216 / rows, most = (V + 2047) / 2048, split = want < 1 || !w.E ? 1 : want < most ? want : most;
    e = launch(ce_join_k, dim3((unsigned)rows, (unsigned)split), JOIN_THREADS, 0, 0, true, s, (const float2*)w.stat,
               w.npieces, target + c0, (const float*)w.zt, V, row_loss + c0, w.E, w.ldE, h + c0 * H,
               dW ? w.hm : nullptr, H);
    if (e != cudaSuccess) return e;
    if (!grads) continue;
    const bf16* d = reinterpret_cast<const bf16*>(w.E);
    const GemmArgs gd{d, w.ldE, 0, W, H, 1, rows, H, V, dh ? dh + c0 * H : nullptr, H, nullptr, 0, nullptr, 0, 0};
    GemmArgs gw{d, w.ldE, 1, w.hm, H, 1, V, H, rows, last ? dW : nullptr, H, nullptr, 0, nullptr, H, 0};
    if (w.dWacc) {
      gw.Dacc = w.dWacc;
      gw.acc_mode = first ? 1 : 2;
    }
    e = gemm_grads(GradArgs{dh ? &gd : nullptr, dW ? &gw : nullptr, g, w.runs, w.slabs, ctr}, s);
    if (e != cudaSuccess) return e;
    if (dh && w.runs > 1) {
      const int64_t n4 = (int64_t)rows * H / 4;
      e = launch(ce_add_runs_k, dim3((unsigned)((n4 + 31) / 32)), RUN_WARPS * 32, 0, 0, true, s,
                 reinterpret_cast<const float4*>(w.slabs), n4, w.runs, g, reinterpret_cast<uint2*>(dh + c0 * H));
      if (e != cudaSuccess) return e;
    }
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
  int kcap = 32;
  while (kcap < K) kcap *= 2;
  const KdArgs a{rows, kcap, logits, target, t_val, t_idx, V, K, tau, w_ce, w_kd, row_ce, row_kd, dlogits};
  // working warps of a block, by the row's length and the number of rows; each
  // rule with both sides measured (us, GB300)
  //   many rows: one warp and 12 blocks per SM up to 7168 columns (16384 rows of
  //   7000: 114 against 118 with two warps; 8192 rows of 10000: 81 against 67),
  //   two up to 15360 (8192 rows of 14336: 95 against 98 with four; of 16384: 110
  //   against 101), four up to 26624 (3000 rows of 26000: 58 against 69 with
  //   eight; 8192 of 28000: 177 against 170), with two temperatures, where the
  //   exponentials weigh more, up to 40960 (3000 of 36000: 84 against 97; 4096 of
  //   45000: 161 against 149), eight up to 61440 (4096 rows of 58000: 174 against
  //   176 with sixteen, of 65000: 204 against 184), with two temperatures up to
  //   73728 (of 70000: 214 against 239; of 80000: 252 against 214, where two rows
  //   per SM no longer stay in L2 until they are read again)
  const bool two = target && tau != 1.f;
  int warps = V <= 7168 ? 1 : V <= 15360 ? 2 : V <= (two ? 40960 : 26624) ? 4 : V <= (two ? 73728 : 61440) ? 8 : 16;
  //   rows for two turns of four warps' 608 blocks: four further on (1216 rows of
  //   36000: 35 against 39 with eight; 1500 of 42000: 51 against 48), for one turn
  //   too (500 rows of 58000: 24 against 27; 600 of 64000: 34 against 31)
  if (warps == 8 && V <= (rows <= 608 ? 61440 : rows <= 1216 ? 45056 : 0)) warps = 4;
  //   few rows, so that a row's own time counts: four warps while their 608
  //   blocks take all rows at once (304 rows of 4096: 4.6 against 6.7 with one;
  //   600: 7.8 against 9.2; 1200: 11.4 against 10.4), eight while 304 do (152 rows
  //   of 24000: 6.0 against 7.0 with four), sixteen while 152 do (152 rows of
  //   48000: 8.2 against 8.8 with eight)
  if (V > 2048 && warps < 4 && rows <= 608) warps = 4;
  if (V > 16384 && warps < 8 && rows <= 304) warps = 8;
  if (V > 32768 && rows <= 152) warps = 16;
  if (warps == 1) return launch_distill<1, 4, 6, 12>(a, s);
  if (warps == 2) return launch_distill<2, 4, 6, 8>(a, s);
  if (warps == 4) return launch_distill<4, 4, 6, 4>(a, s);
  if (warps == 8) return launch_distill<8, 4, 6, 2>(a, s);
  return launch_distill<16, 4, 5, 1>(a, s);
}

size_t router_balance_scratch(int64_t T, int S, int E) {
  if (!bal_shape_ok(T, S, E) || T == 0) return 0;
  BalScratch w;
  return bal_carve(T, S, E, nullptr, &w);
}

cudaError_t router_balance(const float* logits, const int32_t* idx, const uint8_t* valid, int64_t T, int S, int E,
                           int k, float alpha, float z_coef, float* loss, int32_t* counts, float* prob, bf16* dlogits,
                           void* scratch, size_t scratch_bytes, cudaStream_t s) {
  if (!bal_shape_ok(T, S, E) || k < 1 || k > E || (int64_t)S * k > (1 << 30) || !al16(logits) || !al16(dlogits) || !al16(idx) ||
      (reinterpret_cast<uintptr_t>(scratch) & 255))
    return cudaErrorInvalidValue;
  if (T == 0) return cudaSuccess;
  BalScratch w;
  if (bal_carve(T, S, E, (uint8_t*)scratch, &w) > scratch_bytes) return cudaErrorInvalidValue;
  const int64_t G = T / S;
  const size_t smem = (size_t)E * 32 * sizeof(int);
  cudaError_t e = cudaSuccess;
  if (smem > 48 * 1024)  // per device, so set on every call that needs it
    e = cudaFuncSetAttribute(balance_count_k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const int per = (S + w.nparts - 1) / w.nparts;
  balance_count_k<<<dim3((unsigned)w.nparts, (unsigned)G), BAL_COUNT_THREADS, smem, s>>>(idx, valid, S, E, k, per, w.ldp,
                                                                                        w.parts, w.ticket);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const BalArgs a{logits, valid, G, S, E, k, w.rows, w.nblk, w.ldp, alpha / (float)G, z_coef / (float)G, w.nparts,
                  w.parts, counts, dlogits, prob, loss, w.partial, w.gloss, w.ticket};
  const int lanes = bal_lanes(T, E);
  if (bal_wide(T, E)) {
    if (lanes == 8) return launch_balance_grad<8, 2, true>(a, s);
    if (lanes == 16) return launch_balance_grad<16, 2, true>(a, s);
    return launch_balance_grad<32, 2, true>(a, s);
  }
  if (E % 8 == 0) {
    if (lanes == 1) return launch_balance_grad<1, 1, true>(a, s);
    if (lanes == 2) return launch_balance_grad<2, 1, true>(a, s);
    if (lanes == 4) return launch_balance_grad<4, 1, true>(a, s);
    if (lanes == 8) return launch_balance_grad<8, 1, true>(a, s);
    if (lanes == 16) return launch_balance_grad<16, 1, true>(a, s);
    return launch_balance_grad<32, 1, true>(a, s);
  }
  if (lanes == 1) return launch_balance_grad<1, 1, false>(a, s);
  if (lanes == 2) return launch_balance_grad<2, 1, false>(a, s);
  if (lanes == 4) return launch_balance_grad<4, 1, false>(a, s);
  if (lanes == 8) return launch_balance_grad<8, 1, false>(a, s);
  if (lanes == 16) return launch_balance_grad<16, 1, false>(a, s);
  return E <= 256 ? launch_balance_grad<32, 1, false>(a, s) : launch_balance_grad<32, 2, false>(a, s);
}

cudaError_t loss_error_read(int* code, int clear) {
  cudaError_t e = cudaMemcpyFromSymbol(code, g_loss_error, sizeof(int));
  if (e == cudaSuccess && clear) {
    const int z = 0;
    e = cudaMemcpyToSymbol(g_loss_error, &z, sizeof(int));
  }
  return e;
}

}  // namespace mt
