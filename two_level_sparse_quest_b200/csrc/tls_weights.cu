// tls_weights.cu -- the attention weight that each cached token received in a
// decode step, added to one fp32 number per (sequence, KV head, token):
//
//   weights[b][g][t] += sum over the group's heads h of exp(tau q_h . K_t - lse_h)
//
// for the listed tokens, or for every token of each sequence, with lse_h the
// log-sum-exp that the step's attention returned.  It is what a cache is
// evicted by (tls_evict.cu).
//
// A token is read once for all heads of its group: d elements of K (or half a
// 4-bit record) and 8 bytes of its sum, against 2 G d flop, so HBM bounds it up to the latent
// shape's 64 heads.  The tokens are the MMA rows (16 a tile), the heads its
// columns; K goes from global memory straight into the A fragments: the order
// of the contraction is free, so lane c of a quad takes 16 neighbouring bytes
// of a row's every 64 (bf16), or a quarter of the row's codes (4 bits).  The
// queries sit in shared memory as B fragments, in the same order.  fp32 keys
// take CUDA cores, four lanes a token.
//
// Measured (one B200): 64 groups of 4096 listed tokens, 4 heads, bf16 14.0 us
// (14.8 with inputs past the L2), every token of 98304 267 us (6.2 TB/s), 4-bit
// keys 11.1 (11.8) and 147 us; the latent's 64 heads over 4 x 2048 tokens 7.1 us
// (8.6), most of it the 73 KB of queries that each SM fetches, 128 heads 10.4.
//
// The exponent is formed as tau s - lse in natural units, rounded once, before
// it is scaled for exp2: the weights that matter have it near zero.  Each
// token's sum over the heads has a fixed order and is added once, by one
// atomic, so the result does not depend on the order of the CTAs; a list that
// holds a token twice adds it twice.
#include <algorithm>

#include "tls_cache.h"
#include "tls_kv4.cuh"
#include "tls_mma.cuh"

namespace tls {
namespace {

constexpr int kWThreads = 256;  // at most; fewer where the tiles do not reach every SM
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ int n_tokens(const WeightsArgs &a, int b) {
  return a.token_idx ? a.k_t : min(max(a.seq_lens[b], 0), a.max_ctx);
}
// Token at position j of the group's list (or the j-th token), -1 if none; n > 0.
// Without a branch of single lanes, so that a warp stays together for its matrix
// instructions.
__device__ __forceinline__ int token_at(const WeightsArgs &a, int group, int j, int n) {
  const int at = min(j, n - 1);
  const int t = a.token_idx ? a.token_idx[static_cast<size_t>(group) * a.k_t + at] : at;
  return (j < n && t >= 0 && t < a.max_ctx) ? t : -1;
}
// *p += v where on: predicated, for the same reason.
__device__ __forceinline__ void add_weight(float *p, float v, bool on) {
  asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %2, 0;\n @p red.global.add.f32 [%0], %1;\n}\n" ::"l"(p), "f"(v),
               "r"(static_cast<uint32_t>(on))
               : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
// exp(x) for the sum; a head whose attention saw no token (lse = -inf) gives 0.
__device__ __forceinline__ float weight_of(float s, float tau, float lse) {
  return lse == -INFINITY ? 0.f : ex2(fmaf(s, tau, -lse) * kLog2e);
}

// KIND 1: bf16 rows, 2: 4-bit records.  NT: column blocks of 8 heads.
template <int D, int NT, int KIND>
struct WeightsSmem {
  static constexpr int KS = D / 16;
  static constexpr int kQ = NT * KS * 32 * 8;
  static constexpr int kBytes = kQ + NT * 8 * 8;
};

template <int D, int NT, int KIND>
__global__ void __launch_bounds__(kWThreads, NT == 1 && D <= 128 ? 5 : 1) weights_mma_kernel(WeightsArgs a) {
  using L = WeightsSmem<D, NT, KIND>;
  constexpr int KS = L::KS;
  extern __shared__ __align__(16) unsigned char smem[];
  uint4 *qs = reinterpret_cast<uint4 *>(smem);                  // [NT][KS / 2][32 lanes]: two MMA steps a read
  float2 *hp = reinterpret_cast<float2 *>(smem + L::kQ);        // [8 NT] (tau, lse) of each head
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int group = blockIdx.y, b = group / a.n_kv_heads, gk = group % a.n_kv_heads;
  const int G = a.n_q_heads / a.n_kv_heads;
  const size_t head0 = static_cast<size_t>(b) * a.n_q_heads + static_cast<size_t>(gk) * G;
  grid_dependency_wait();
  const int n = n_tokens(a, b);
  const int tiles = (n + 15) / 16;
  if (static_cast<int>(blockIdx.x) * warps >= tiles) return;

  const int row_bytes = KIND == 1 ? 2 * D : Kv4Rec<KIND == 1 ? 128 : D>::kBytes;
  const unsigned char *base =
      static_cast<const unsigned char *>(a.keys) + static_cast<size_t>(group) * a.max_ctx * row_bytes;
  float *out = a.weights + static_cast<size_t>(group) * a.max_ctx;
  const int step = gridDim.x * warps;
  int tile = blockIdx.x * warps + warp;
  int t0 = token_at(a, group, tile * 16 + g, n), t1 = token_at(a, group, tile * 16 + 8 + g, n);

  // B fragments: lane (g, c) of block nt: the 8 channels 32 i + 8 c of head 8 nt + g, steps 2 i and 2 i + 1
  if constexpr (KIND == 1) {
    const uint16_t *q0 = static_cast<const uint16_t *>(a.q);
    const uint16_t *qp = q0 + (head0 + g) * D + 8 * c;  // a lane's column is the same in every fragment
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const bool ok = nt * 8 + g < G;
#pragma unroll 3
      for (int i = warp; i < KS / 2; i += warps)
        cp_async16(qs + (nt * (KS / 2) + i) * 32 + lane, ok ? qp + nt * 8 * D + 32 * i : q0, ok);
    }
    cp_async_commit();
    for (int h = threadIdx.x; h < NT * 8; h += blockDim.x)
      hp[h] = make_float2(a.scale, h < G ? a.lse[head0 + h] : -INFINITY);
    if constexpr (D == 576) {  // long rows: on their way while the queries arrive
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (c + 4 * i < 9) {
          prefetch_l2(base + static_cast<size_t>(max(t0, 0)) * row_bytes + (c + 4 * i) * 128);
          prefetch_l2(base + static_cast<size_t>(max(t1, 0)) * row_bytes + (c + 4 * i) * 128);
        }
    }
    cp_async_wait<0>();
  } else {
    for (int h = warp; h < NT * 8; h += warps) {  // one warp a head: its row as fp16, scaled by a power of two
      uint2 w = make_uint2(0u, 0u);
      const bool mine = lane * 4 < D;
      if (h < G && mine) w = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(a.q) + (head0 + h) * D + 4 * lane);
      const uint32_t ex = __reduce_max_sync(0xffffffffu, max(bf16_exps(w.x), bf16_exps(w.y)));
      float undo;
      const float mult = q_norm(ex, &undo);
      // channels 4 lane .. + 3: quarter lane / KS of the row, step lane % KS
      const int ks = lane % KS;
      if (mine)
        reinterpret_cast<uint2 *>(qs + ((h >> 3) * (KS / 2) + ks / 2) * 32 + (h & 7) * 4 + lane / KS)[ks & 1] =
            make_uint2(q_to_f16(w.x, mult), q_to_f16(w.y, mult));
      if (lane == 0) hp[h] = make_float2(a.scale * undo, h < G ? a.lse[head0 + h] : -INFINITY);
    }
  }
  __syncthreads();

  for (; tile < tiles; tile += step) {
    const unsigned char *r0 = base + static_cast<size_t>(max(t0, 0)) * row_bytes;
    const unsigned char *r1 = base + static_cast<size_t>(max(t1, 0)) * row_bytes;
    float s[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
    const int n0 = token_at(a, group, (tile + step) * 16 + g, n), n1 = token_at(a, group, (tile + step) * 16 + 8 + g, n);
    if constexpr (KIND == 1) {
      constexpr int NL = D / 32;              // 16-byte reads per row and lane
      constexpr int U = NL < 6 ? NL : 6;      // pairs of reads in flight
      static_assert(NL % U == 0, "whole batches of reads");
#pragma unroll
      for (int i0 = 0; i0 < NL; i0 += U) {
        uint4 x[U], y[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          x[i] = ld_stream16(r0 + (i0 + i) * 64 + 16 * c);
          y[i] = ld_stream16(r1 + (i0 + i) * 64 + 16 * c);
        }
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint4 q = qs[(nt * (KS / 2) + i0 + i) * 32 + lane];
            mma_full(s[nt], x[i].x, y[i].x, x[i].y, y[i].y, q.x, q.y);
            mma_full(s[nt], x[i].z, y[i].z, x[i].w, y[i].w, q.z, q.w);
          }
      }
    } else {
      using R = Kv4Rec<D>;
      constexpr int CW = D / 32;
      uint32_t w0[CW], w1[CW], sc0, sc1;
      if constexpr (D == 128) {
        *reinterpret_cast<uint4 *>(w0) = *reinterpret_cast<const uint4 *>(r0 + 16 * c);
        *reinterpret_cast<uint4 *>(w1) = *reinterpret_cast<const uint4 *>(r1 + 16 * c);
        sc0 = *reinterpret_cast<const uint16_t *>(r0 + R::kKS + 2 * c);
        sc1 = *reinterpret_cast<const uint16_t *>(r1 + R::kKS + 2 * c);
      } else {
        *reinterpret_cast<uint2 *>(w0) = *reinterpret_cast<const uint2 *>(r0 + 8 * c);
        *reinterpret_cast<uint2 *>(w1) = *reinterpret_cast<const uint2 *>(r1 + 8 * c);
        sc0 = r0[R::kKS + c];
        sc1 = r1[R::kKS + c];
      }
#pragma unroll
      for (int w = 0; w < CW; ++w) {
        const uint32_t f0 = (w < 2 ? sc0 & 0xffu : sc0 >> 8) * 0x00800080u;
        const uint32_t f1 = (w < 2 ? sc1 & 0xffu : sc1 >> 8) * 0x00800080u;
        uint32_t x[4], y[4];
        e2m1_unpack(w0[w], x[0], x[1], x[2], x[3]);
        e2m1_unpack(w1[w], y[0], y[1], y[2], y[3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = hmul2(x[e], f0);
          y[e] = hmul2(y[e], f1);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint4 q = qs[(nt * (KS / 2) + w) * 32 + lane];
          mma_f16(s[nt], x[0], y[0], x[1], y[1], q.x, q.y);
          mma_f16(s[nt], x[2], y[2], x[3], y[3], q.z, q.w);
        }
      }
    }
    float w0 = 0.f, w1 = 0.f;  // this lane's heads: tokens of rows g, g + 8
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float2 p = hp[nt * 8 + 2 * c + e];
        w0 += weight_of(s[nt][e], p.x, p.y);
        w1 += weight_of(s[nt][e + 2], p.x, p.y);
      }
    float v = c & 1 ? w1 : w0;  // even lanes sum row g's token, odd ones row g + 8's
    v += __shfl_xor_sync(0xffffffffu, c & 1 ? w0 : w1, 1);
    v += __shfl_xor_sync(0xffffffffu, v, 2);
    const int tt = c & 1 ? t1 : t0;
    add_weight(out + tt, v, c < 2 && tt >= 0);
    t0 = n0;
    t1 = n1;
  }
}

// fp32 keys: four lanes share a token (lane c takes float4 c of every four),
// eight tokens a warp, the heads one after another from shared memory.
template <int D>
__global__ void __launch_bounds__(kWThreads) weights_f32_kernel(WeightsArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  float4 *qs = reinterpret_cast<float4 *>(smem);  // [G][D / 4]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int group = blockIdx.y, b = group / a.n_kv_heads, gk = group % a.n_kv_heads;
  const int G = a.n_q_heads / a.n_kv_heads;
  const size_t head0 = static_cast<size_t>(b) * a.n_q_heads + static_cast<size_t>(gk) * G;
  grid_dependency_wait();
  const int n = n_tokens(a, b);
  const int tiles = (n + 7) / 8;
  if (static_cast<int>(blockIdx.x) * warps >= tiles) return;
  const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(a.q) + head0 * D);
  float *lse = reinterpret_cast<float *>(qs + G * (D / 4));
  for (int i = threadIdx.x; i < G * (D / 4); i += blockDim.x) qs[i] = q[i];
  for (int i = threadIdx.x; i < G; i += blockDim.x) lse[i] = a.lse[head0 + i];
  __syncthreads();
  const float *K = static_cast<const float *>(a.keys) + static_cast<size_t>(group) * a.max_ctx * D;
  float *out = a.weights + static_cast<size_t>(group) * a.max_ctx;
  for (int tile = blockIdx.x * warps + warp; tile < tiles; tile += gridDim.x * warps) {
    const int t = token_at(a, group, tile * 8 + g, n);
    const float4 *row = reinterpret_cast<const float4 *>(K + static_cast<size_t>(max(t, 0)) * D);
    float4 k[D / 16];
#pragma unroll
    for (int i = 0; i < D / 16; ++i) k[i] = row[4 * i + c];
    float w = 0.f;
    for (int h = 0; h < G; ++h) {
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const float4 v = qs[h * (D / 4) + 4 * i + c];
        s0 = fmaf(v.x, k[i].x, s0);
        s1 = fmaf(v.y, k[i].y, s1);
        s0 = fmaf(v.z, k[i].z, s0);
        s1 = fmaf(v.w, k[i].w, s1);
      }
      s0 += s1;
      s0 += __shfl_xor_sync(0xffffffffu, s0, 1);
      s0 += __shfl_xor_sync(0xffffffffu, s0, 2);
      w += weight_of(s0, a.scale, lse[h]);
    }
    add_weight(out + t, w, c == 0 && t >= 0);
  }
}

// Threads of a CTA and CTAs of a group: as many as run at once (per_sm of 256
// threads), no more than there are tiles; half-size CTAs while each still gets
// an SM of its own (latent, 64 heads, 4 x 2048 tokens 8.0 -> 7.1 us).  Not
// beyond that: each CTA fetches all queries again (4 x 4096 tokens, 128
// against 256 CTAs: 8.5 us and 9.3; with 128 heads, one CTA an SM, 12.2 and
// 20.8).  No quarters: over 192 shapes (latent, bf16, 4-bit, fp32; 1 to 16
// groups, 128 to 4096 tokens) they gain 0.2 us at most, and the choice here is
// within 1 % of the best of all sizes on average, within 5 % for 183 of them.
struct Split {
  int threads, ctas;
};
Split split_of(const WeightsArgs &a, int tokens_per_warp, int per_sm) {
  const long long n = a.token_idx ? a.k_t : a.max_ctx;
  const long long groups = static_cast<long long>(a.batch) * a.n_kv_heads;
  const long long sms = a.num_sms > 0 ? a.num_sms : 148;
  const long long tiles = (n + tokens_per_warp - 1) / tokens_per_warp;
  int warps = kWThreads / 32;
  if (groups * ((tiles + warps / 2 - 1) / (warps / 2)) <= sms) warps /= 2;
  const long long fill = std::max<long long>(1, sms * per_sm / groups);
  return {warps * 32, static_cast<int>(std::max<long long>(1, std::min((tiles + warps - 1) / warps, fill)))};
}

template <int D, int NT, int KIND>
cudaError_t run_mma(const WeightsArgs &a, cudaStream_t st) {
  using L = WeightsSmem<D, NT, KIND>;
  auto kern = weights_mma_kernel<D, NT, KIND>;
  if (L::kBytes > 48 * 1024) {
    static bool configured[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64 || !configured[dev]) {
      cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
      if (e != cudaSuccess) return e;
      if (dev >= 0 && dev < 64) configured[dev] = true;
    }
  }
  // resident CTAs an SM, by registers (the latent's 128 heads: by shared memory)
  const Split sp = split_of(a, 16, D == 576 ? (NT == 16 ? 1 : 2) : NT == 1 ? 5 : NT <= 4 ? 4 : 3);
  return launch_pdl(kern, dim3(sp.ctas, a.batch * a.n_kv_heads), dim3(sp.threads), L::kBytes, st, a);
}

template <int D, int KIND>
cudaError_t dispatch_mma(const WeightsArgs &a, cudaStream_t st) {
  const int G = a.n_q_heads / a.n_kv_heads;
  if (G <= 8) return run_mma<D, 1, KIND>(a, st);
  if (G <= 16) return run_mma<D, 2, KIND>(a, st);
  if (G <= 32) return run_mma<D, 4, KIND>(a, st);
  if (G <= 64) return run_mma<D, 8, KIND>(a, st);
  if constexpr (D == 576) return run_mma<D, 16, KIND>(a, st);
  return cudaErrorInvalidValue;
}

template <int D>
cudaError_t run_f32(const WeightsArgs &a, cudaStream_t st) {
  const int G = a.n_q_heads / a.n_kv_heads;
  const size_t smem = static_cast<size_t>(G) * (D + 1) * 4;  // at most 33 KB (64 heads of 128 channels)
  const Split sp = split_of(a, 8, 4);
  return launch_pdl(weights_f32_kernel<D>, dim3(sp.ctas, a.batch * a.n_kv_heads), dim3(sp.threads), smem, st, a);
}

}  // namespace

cudaError_t launch_accum_weights(const WeightsArgs &a, cudaStream_t st) {
  if (a.keys_kind == 0) return a.d == 128 ? run_f32<128>(a, st) : run_f32<64>(a, st);
  if (a.keys_kind == 1) {
    if (a.d == 576) return dispatch_mma<576, 1>(a, st);
    return a.d == 128 ? dispatch_mma<128, 1>(a, st) : dispatch_mma<64, 1>(a, st);
  }
  return a.d == 128 ? dispatch_mma<128, 2>(a, st) : dispatch_mma<64, 2>(a, st);
}

}  // namespace tls
