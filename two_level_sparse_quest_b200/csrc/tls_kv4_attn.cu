// tls_kv4_attn.cu -- exact softmax attention of one decode step over the
// 4-bit KV cache: over listed tokens (in the cache, or in a slot cache of
// blocks), or over every token of each sequence.
//
// For query head h of a group: a_t = tau q_h . K_t, o_h = sum_t softmax(a)_t V_t,
// lse_h = log sum_t exp(a_t), with K_t and V_t the values the record stands for.
//
// Bound: a token is 9 d / 8 bytes (144 at d 128), against 4 G d flop, so HBM
// is the floor; at that rate an SM has 6.4 cycles for a token, and it is the
// instructions that widen the codes (two for each pair of channels: e2m1 ->
// fp16, times the scale, each at half rate) that come near it, not the tensor
// pipe.  Measured (one B200): 64 groups of 98304 tokens, 4 heads, 174 us (5.2
// TB/s, 0.80 of the measured copy rate), 8 heads 199, 16 heads 338; of 4096
// listed ones 19.3 us, 8 heads 20.6, 16 heads 29.6.
//
// Layout: the tokens are the MMA rows.  S^T[16 tokens x 8 heads] = K q^T takes
// one m16n8k16 per 16 channels, O^T[16 channels x 8 heads] += V^T P^T one per
// 16 channels and 16 tokens: up to 8 heads cost one MMA column block, half of
// what heads as rows would.  The order of the contraction is free, so lane c
// of a quad takes 32 neighbouring channels of K (one 16-byte read of codes
// and two scales) and lane group g takes 16 neighbouring channels of V (8
// bytes and one scale) and no operand passes through another lane, except P:
// its two fp16 parts turn from S^T's accumulator layout into the B operand
// with movmatrix.  V's pairs (two tokens of one channel) are formed on the
// codes, a nibble of each token in a byte, before they are widened.
//
// Numerics: K and V are exact in fp16; q is (tls_kv4.cuh, q_norm); sums are
// fp32.  P is 2^(s - m + 14), at most 2^15, as two fp16 parts, high and low
// (22 bits; what falls below 2^-38 of the largest weight is dropped), whatever
// the output's type, and the sum l is of the unrounded weights: with the high
// part alone each weight would be off by up to 2^-11, which moves a bf16
// output by a step now and then.  m is a running reference that moves only
// when a score exceeds it by more than one (log2).  A unit of at most four
// heads leaves four of the eight columns free: they repeat the heads' queries
// and carry the low parts, so that P's second part costs no MMA (every token
// of 8 x 96k, 4 heads: 174 us against 192 with two MMAs; 8 heads 200 with two,
// 177 with the high part alone).
//
// Work split: a unit is one group (or 16 of its heads).  A thread-block
// cluster of up to 8 CTAs takes a unit, every warp 32-token tiles in turn
// through its own ring in shared memory; the warps' and then the CTAs' partial
// (m, l, O) are joined in shared memory, the CTAs' over distributed shared
// memory, so that one launch does the whole step.  Long calls are cut into
// parts that leave their partials in the workspace for a second launch
// (kv4_plan).
#include <algorithm>

#include "tls_cache.h"
#include "tls_kv4.cuh"
#include "tls_mma.cuh"

namespace tls {
namespace {

constexpr int kTile = 32;   // tokens per ring stage
constexpr int kWarps = 8;   // per CTA
constexpr int kRing = 3;
constexpr int kMaxCluster = 8;
constexpr int kMaxSplit = 148;
constexpr float kPShift = 14.f;     // P is scaled by 2^14
constexpr float kNoMax = -3e38f;    // a warp's m before its first token: finite, so that a masked score stays -inf

template <int D, int NT>
struct Kv4Smem {
  using R = Kv4Rec<D>;
  static constexpr int kStage = kTile * R::kBytes;
  // A warp's partial O [8 NT heads][D channels] overlays its ring.  Two words
  // of padding per lane group's channels and a head stride of 4 mod 16 keep
  // the 8-byte stores of a half warp in distinct banks.
  static constexpr int kCpl = D / 8;  // channels per lane group
  static constexpr int kHead = 8 * (kCpl + 2) + 4;
  static_assert(kHead % 16 == 4, "bank spread of the partial's heads");
  static constexpr int kPartial = 8 * NT * kHead * 4;
  static constexpr int kWarpBytes = kRing * kStage > kPartial ? kRing * kStage : kPartial;
  static constexpr int kSmem = kWarps * kWarpBytes;
  static_assert(kWarpBytes % 16 == 0, "every ring starts on 16 bytes");
  static __device__ __forceinline__ int at(int head, int ch) { return head * kHead + ch + 2 * (ch / kCpl); }
};

template <int BYTES>
__device__ __forceinline__ void cp_async_chunk(uint32_t dst, const void *src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(dst), "l"(src) : "memory");
}
template <int BYTES>
__device__ __forceinline__ void cp_async_chunk(uint32_t dst, const void *src, bool ok) {
  const int n = ok ? BYTES : 0;  // 0 source bytes: zero-filled
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;\n" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

__device__ __forceinline__ uint32_t movmatrix(uint32_t a) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}

__device__ __forceinline__ float2 ld_cluster(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr));
  return v;
}

// The token (0..15 of a half) in MMA row `row` (0..7; rows 8..15 are 8 more).
// Halves take even and odd tokens of a stage; with this order neither the
// 16-byte reads of K (row pairs two tokens apart) nor the 8-byte reads of V
// (rows 2c) collide in shared memory at d 128.
__device__ __forceinline__ int row_token(int row) { return (0x57463120u >> (4 * row)) & 15; }

template <int D, int NT, bool LOCOL, bool LIST, bool PAGED>
__global__ void __launch_bounds__(kWarps * 32, NT == 1 ? 2 : 1) kv4_attn_kernel(Kv4AttnArgs a) {
  using R = Kv4Rec<D>;
  using L = Kv4Smem<D, NT>;
  constexpr int OT = D / 16;   // 16-channel tiles of O
  constexpr int CW = D / 32;   // 32-bit words of K codes per lane and token
  constexpr int VW = D / 64;   // 32-bit words of V codes per lane and token
  constexpr bool kBulk = !LIST && R::kBytes % 16 == 0;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) float s_ml[kWarps][8 * NT][2];
  __shared__ __align__(8) float s_cta[8 * NT][2];
  __shared__ uint4 s_q[NT][D / 32][32];
  __shared__ float s_scale[8 * NT];
  __shared__ uint64_t s_full[kWarps][kRing];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  unsigned char *ring = smem + warp * L::kWarpBytes;
  const uint32_t ring_s = smem_addr(ring);

  const int CS = a.cluster;
  const int rank = static_cast<int>(blockIdx.x) % CS;
  const int part = (static_cast<int>(blockIdx.x) / CS) % a.n_split;
  const int unit = static_cast<int>(blockIdx.x) / (CS * a.n_split);
  const int group = unit / a.n_head_chunks, hc = unit % a.n_head_chunks;
  const int b = group / a.n_kv_heads, gk = group % a.n_kv_heads;
  const int G = a.n_q_heads / a.n_kv_heads;
  const int HG = a.head_chunk;
  const int head0 = gk * G + hc * HG;

  grid_dependency_wait();

  const int n = LIST ? a.k_t : min(max(a.seq_lens[b], 0), a.max_ctx);
  const int n_tiles = (n + kTile - 1) / kTile;
  const int per_part = (n_tiles + a.n_split - 1) / a.n_split;
  const int t_end = min(n_tiles, (part + 1) * per_part);
  const int stride = CS * kWarps;
  int t_issue = part * per_part + rank * kWarps + warp;
  const int my_tiles = t_issue < t_end ? (t_end - t_issue + stride - 1) / stride : 0;

  const unsigned char *base = static_cast<const unsigned char *>(a.cache);
  if constexpr (PAGED) base += static_cast<size_t>(group) * a.n_slots * a.block_size * R::kBytes;
  else base += static_cast<size_t>(group) * a.max_ctx * R::kBytes;
  const int32_t *ids = LIST ? a.token_idx + static_cast<size_t>(group) * a.k_t : nullptr;
  const int32_t *slots = PAGED ? a.slot_of_block + static_cast<size_t>(group) * a.n_blocks_max : nullptr;

  // Cache row of this lane's token of tile t, or -1.
  auto row_of = [&](int t) -> int {
    const int j = t * kTile + lane;
    if (t >= t_end || j >= n) return -1;
    if constexpr (!LIST) return j;
    const int tok = ids[j];
    if (tok < 0 || tok >= a.max_ctx) return -1;
    if constexpr (!PAGED) return tok;
    const int blk = tok / a.block_size;
    const int slot = slots[blk];
    return (slot >= 0 && slot < a.n_slots) ? slot * a.block_size + (tok - blk * a.block_size) : -1;
  };

  // The ring.  Neighbouring tokens at d 128 (a record is a multiple of 16
  // bytes) come with one bulk copy a stage, counted by the stage's mbarrier;
  // tokens past the end get zero scales, so that stale bytes stay finite.
  // Listed tokens come with cp.async, nine chunks of d / 8 bytes a record; where
  // some are missing, eight lanes bring a record's first eight chunks and every
  // lane its own record's ninth, zero-filled.  (One bulk copy per listed record
  // was slower: 24.0 us against 20.4 for 8 x 96k, 4096 tokens.)
  // The queries' loads go out first (warps below NT, one block of 8 columns each).
  uint4 qv[D / 32];
  if (warp < NT) {
    const int h = LOCOL ? g & 3 : warp * 8 + g;  // LOCOL: columns 4 .. 7 repeat the heads of 0 .. 3
    const uint4 *qp = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q) +
                                                      (static_cast<size_t>(b) * a.n_q_heads + head0 + h) * D + c * (D / 4));
#pragma unroll
    for (int i = 0; i < D / 32; ++i) qv[i] = h < HG ? qp[i] : make_uint4(0u, 0u, 0u, 0u);
  }
  uint32_t valid[kRing];  // valid tokens of the stages in flight, oldest first
#pragma unroll
  for (int s = 0; s < kRing; ++s) valid[s] = 0;
  // rows of the next two tiles: their ids are on the way while earlier tiles are copied and computed
  int row_next = kBulk ? 0 : row_of(t_issue), row_after = kBulk ? 0 : row_of(t_issue + stride), stage_issue = 0;
  if constexpr (kBulk) {
    if (lane == 0) {
#pragma unroll
      for (int s = 0; s < kRing; ++s) mbarrier_init(&s_full[warp][s], 1);
      mbarrier_init_fence();
    }
    __syncwarp();
  }
  auto issue = [&]() -> uint32_t {
    uint32_t mask;
    if constexpr (kBulk) {
      const int left = t_issue < t_end ? n - t_issue * kTile : 0;  // tokens of this stage, at least; the same in every lane
      mask = left >= kTile ? 0xffffffffu : (1u << max(left, 0)) - 1u;
      if (left > 0) {
        unsigned char *dst = ring + stage_issue * L::kStage;
        if (lane == 0) {
          const uint32_t bytes = min(left, kTile) * R::kBytes;
          mbarrier_expect_tx(&s_full[warp][stage_issue], bytes);
          bulk_load(dst, base + static_cast<size_t>(t_issue) * (kTile * R::kBytes), bytes, &s_full[warp][stage_issue]);
        }
        if (lane >= left)  // the last stage of all: nothing is copied over these zeros
          *reinterpret_cast<uint4 *>(dst + lane * R::kBytes + R::kKS) = make_uint4(0u, 0u, 0u, 0u);
      }
      t_issue += stride;
    } else {
      const int row = row_next;
      mask = __ballot_sync(0xffffffffu, row >= 0);
      if (mask != 0u) {
        constexpr int CB = R::kChunk;
        const uint32_t dst = ring_s + stage_issue * L::kStage;
        if (mask == 0xffffffffu) {
#pragma unroll
          for (int i = 0; i < 9; ++i) {  // neighbouring lanes on neighbouring bytes
            const int idx = i * 32 + lane, tk = (idx * 57) >> 9;  // idx / 9 for idx < 288
            const long long u = __shfl_sync(0xffffffffu, row, tk);
            cp_async_chunk<CB>(dst + idx * CB, base + (u - tk) * R::kBytes + idx * CB);
          }
        } else {
          const unsigned char *src = base + (lane & 7) * CB;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const long long u = __shfl_sync(0xffffffffu, row, 4 * i + (lane >> 3));
            cp_async_chunk<CB>(dst + (4 * i + (lane >> 3)) * R::kBytes + (lane & 7) * CB,
                               u >= 0 ? src + u * R::kBytes : base, u >= 0);
          }
          cp_async_chunk<CB>(dst + lane * R::kBytes + 8 * CB,
                             row >= 0 ? base + static_cast<long long>(row) * R::kBytes + 8 * CB : base, row >= 0);
        }
      }
      t_issue += stride;
      row_next = row_after;
      row_after = row_of(t_issue + stride);
    }
    if (++stage_issue == kRing) stage_issue = 0;
    return mask;
  };

  valid[1] = issue();
  if constexpr (!kBulk) cp_async_commit();

  // Queries: B fragments of S^T = K q^T in shared memory, two MMA steps a
  // read.  Lane (g, c) holds head 8 nt + g's channels c D/4 .. + D/4 - 1, four
  // per step.
  if (warp < NT) {
    const int h = warp * 8 + g;
    uint32_t w[D / 8];
    uint32_t ex = 0;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      w[4 * i] = qv[i].x;
      w[4 * i + 1] = qv[i].y;
      w[4 * i + 2] = qv[i].z;
      w[4 * i + 3] = qv[i].w;
    }
#pragma unroll
    for (int i = 0; i < D / 8; ++i) ex = max(ex, bf16_exps(w[i]));
    ex = max(ex, __shfl_xor_sync(0xffffffffu, ex, 1));
    ex = max(ex, __shfl_xor_sync(0xffffffffu, ex, 2));
    float undo;
    const float mult = q_norm(ex, &undo);
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
      s_q[warp][i][lane] = make_uint4(q_to_f16(w[4 * i], mult), q_to_f16(w[4 * i + 1], mult),
                                      q_to_f16(w[4 * i + 2], mult), q_to_f16(w[4 * i + 3], mult));
    if (c == 0) s_scale[h] = a.scale_log2 * undo;
  }
  __syncthreads();
  // the second stage once every warp has asked for its first: its bytes would only delay theirs
#pragma unroll
  for (int s = 1; s < kRing - 1; ++s) {
    valid[s + 1] = issue();
    if constexpr (!kBulk) cp_async_commit();
  }
  float sl[NT][2];  // score scale of this lane's columns (heads 8 nt + 2c, + 1)
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    sl[nt][0] = s_scale[nt * 8 + 2 * c];
    sl[nt][1] = s_scale[nt * 8 + 2 * c + 1];
  }

  float o[NT][OT][4];
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int j = 0; j < OT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[nt][j][e] = 0.f;
    m[nt][0] = m[nt][1] = kNoMax;
    l[nt][0] = l[nt][1] = 0.f;
  }

  const int ktok = 2 * row_token(g);  // this lane's K rows: tokens ktok + half, ktok + 16 + half
  const int vtok0 = 2 * row_token(2 * c), vtok1 = 2 * row_token(2 * c + 1);

  int st = 0;
  uint32_t phase = 0;  // mbarrier parity of the ring's current round (every stage is used once a round until the last tile)
  bool alive = true;
  for (int it = 0; it < my_tiles; ++it) {
#pragma unroll
    for (int s = 0; s + 1 < kRing; ++s) valid[s] = valid[s + 1];
    valid[kRing - 1] = alive ? issue() : 0u;
    if constexpr (!kBulk) {
      cp_async_commit();
      cp_async_wait<kRing - 1>();
      __syncwarp();
    }
    const uint32_t vm = valid[0];
    if constexpr (kBulk) {
      if (vm != 0u) {  // a wait that gives up (which a correct run never sees): no further copies, those in flight are
                       // waited for, the result is undefined
        const bool arrived = mbarrier_wait(&s_full[warp][st], phase);
        if (!__all_sync(0xffffffffu, arrived)) {
          alive = false;
          if (lane == 0 && a.err) atomicOr(a.err, kErrAttnWait);
          (void)mbarrier_wait(&s_full[warp][st], phase);  // its bytes may still land: not while the ring holds partials
        }
      }
    }
    if (vm != 0u && alive) {
      const unsigned char *S = ring + st * L::kStage;
      // (both halves in one body where the registers allow it: every token 174 us against 179, lists the same)
#pragma unroll NT == 1 ? 2 : 1
      for (int hf = 0; hf < 2; ++hf, S += R::kBytes) {  // even tokens of the stage, then odd ones
        // ---- S^T = K q^T: rows g, g + 8 of heads 2c, 2c + 1
        float s[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
        const unsigned char *k0 = S + ktok * R::kBytes, *k1 = k0 + 16 * R::kBytes;
        uint32_t w0[CW], w1[CW], sc0, sc1;
        if constexpr (D == 128) {
          *reinterpret_cast<uint4 *>(w0) = *reinterpret_cast<const uint4 *>(k0 + 16 * c);
          *reinterpret_cast<uint4 *>(w1) = *reinterpret_cast<const uint4 *>(k1 + 16 * c);
          sc0 = *reinterpret_cast<const uint16_t *>(k0 + R::kKS + 2 * c);
          sc1 = *reinterpret_cast<const uint16_t *>(k1 + R::kKS + 2 * c);
        } else {
          *reinterpret_cast<uint2 *>(w0) = *reinterpret_cast<const uint2 *>(k0 + 8 * c);
          *reinterpret_cast<uint2 *>(w1) = *reinterpret_cast<const uint2 *>(k1 + 8 * c);
          sc0 = k0[R::kKS + c];
          sc1 = k1[R::kKS + c];
        }
        // a word is widened while the one before it is scaled and multiplied: the three take different pipes
        uint32_t x[2][4], y[2][4];
        auto widen = [&](int w) {
          e2m1_unpack(w0[w], x[w & 1][0], x[w & 1][1], x[w & 1][2], x[w & 1][3]);
          e2m1_unpack(w1[w], y[w & 1][0], y[w & 1][1], y[w & 1][2], y[w & 1][3]);
        };
        widen(0);
#pragma unroll
        for (int w = 0; w < CW; ++w) {
          if (w + 1 < CW) widen(w + 1);
          // words 0, 1 of a row lie in the lane's first group of 16 channels, 2, 3 in its second
          const uint32_t f0 = (w < 2 ? sc0 & 0xffu : sc0 >> 8) * 0x00800080u;
          const uint32_t f1 = (w < 2 ? sc1 & 0xffu : sc1 >> 8) * 0x00800080u;
          uint32_t (&X)[4] = x[w & 1], (&Y)[4] = y[w & 1];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            X[e] = hmul2(X[e], f0);
            Y[e] = hmul2(Y[e], f1);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint4 qf = s_q[nt][w][lane];
            mma_f16(s[nt], X[0], Y[0], X[1], Y[1], qf.x, qf.y);
            mma_f16(s[nt], X[2], Y[2], X[3], Y[3], qf.z, qf.w);
          }
        }
        // ---- online softmax in the log2 domain: t = score - m + 14
        if (vm != 0xffffffffu) {
          const bool ok0 = (vm >> (ktok + hf)) & 1u, ok1 = (vm >> (ktok + 16 + hf)) & 1u;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!(e < 2 ? ok0 : ok1)) s[nt][e] = -INFINITY;
        }
        float top = -INFINITY;
        float t[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            t[nt][e] = fmaf(s[nt][e], sl[nt][e & 1], kPShift - m[nt][e & 1]);
            top = fmaxf(top, t[nt][e]);
          }
        if (__any_sync(0xffffffffu, top > kPShift + 1.f)) {  // some score exceeds its head's m by more than one
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float mx = fmaxf(s[nt][e], s[nt][e + 2]) * sl[nt][e];
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
              if (mx > m[nt][e]) {
                const float alpha = ex2(m[nt][e] - mx);  // 0 for the first tokens
                m[nt][e] = mx;
                l[nt][e] *= alpha;
#pragma unroll
                for (int j = 0; j < OT; ++j) {
                  o[nt][j][e] *= alpha;
                  o[nt][j][e + 2] *= alpha;
                }
                t[nt][e] = fmaf(s[nt][e], sl[nt][e], kPShift - mx);
                t[nt][e + 2] = fmaf(s[nt][e + 2], sl[nt][e], kPShift - mx);
              }
            }
          __syncwarp();  // a head's lanes branch alone; movmatrix and mma take the whole warp
        }
        // ---- O^T += V^T P^T
        uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[e] = ex2(t[nt][e]);
            l[nt][e & 1] += p[e];
          }
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const __half2 hi = __floats2half2_rn(p[2 * r], p[2 * r + 1]);
            const float2 hf2 = __half22float2(hi);
            const __half2 lo = __floats2half2_rn(p[2 * r] - hf2.x, p[2 * r + 1] - hf2.y);
            const uint32_t uh = *reinterpret_cast<const uint32_t *>(&hi), ul = *reinterpret_cast<const uint32_t *>(&lo);
            if constexpr (LOCOL) {
              ph[nt][r] = movmatrix(c < 2 ? uh : ul);
            } else {
              ph[nt][r] = movmatrix(uh);
              pl[nt][r] = movmatrix(ul);
            }
          }
        }
        const unsigned char *v0 = S + vtok0 * R::kBytes, *v1 = S + vtok1 * R::kBytes;
        constexpr int V8 = 16 * R::kBytes;  // rows 8 more: 16 tokens on
        uint32_t w[4][VW], sc[2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const unsigned char *v = (i & 1 ? v1 : v0) + (i >> 1) * V8;
          if constexpr (D == 128) *reinterpret_cast<uint2 *>(w[i]) = *reinterpret_cast<const uint2 *>(v + R::kVC + 8 * g);
          else w[i][0] = *reinterpret_cast<const uint32_t *>(v + R::kVC + 4 * g);
        }
        // a lane group's channels share one scale (d 64: half of one)
        constexpr int SD = D == 128 ? 1 : 2;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t a0 = v0[r * V8 + R::kVS + g / SD], a1 = v1[r * V8 + R::kVS + g / SD];
          sc[r] = (a0 << 7) | (a1 << 23);
        }
#pragma unroll
        for (int q = 0; q < VW; ++q) {
          // bytes of one channel from two tokens: even channels, odd channels
          uint32_t ev[2][4], od[2][4];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint32_t x = w[2 * r][q], y = w[2 * r + 1][q];
            e2m1_unpack((x & 0x0f0f0f0fu) | ((y << 4) & 0xf0f0f0f0u), ev[r][0], ev[r][1], ev[r][2], ev[r][3]);
            e2m1_unpack(((x >> 4) & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u), od[r][0], od[r][1], od[r][2], od[r][3]);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t a0 = hmul2(ev[0][j], sc[0]), a1 = hmul2(od[0][j], sc[0]);
            const uint32_t a2 = hmul2(ev[1][j], sc[1]), a3 = hmul2(od[1][j], sc[1]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_f16(o[nt][4 * q + j], a0, a1, a2, a3, ph[nt][0], ph[nt][1]);
              if constexpr (!LOCOL) mma_f16(o[nt][4 * q + j], a0, a1, a2, a3, pl[nt][0], pl[nt][1]);
            }
          }
        }
      }
    }
    __syncwarp();
    if (++st == kRing) {
      st = 0;
      phase ^= 1u;
    }
  }
  if constexpr (!kBulk) cp_async_wait<0>();
  __syncwarp();

  if constexpr (LOCOL) {  // a head's sum over the high parts (lane c) and over the low parts (lane c + 2)
#pragma unroll
    for (int j = 0; j < OT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[0][j][e] += __shfl_xor_sync(0xffffffffu, o[0][j][e], 2);
  }
  // ---- the warp's partial into its own ring
  float *po = reinterpret_cast<float *>(ring);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float t = l[nt][e];
      t += __shfl_xor_sync(0xffffffffu, t, 4);
      t += __shfl_xor_sync(0xffffffffu, t, 8);
      t += __shfl_xor_sync(0xffffffffu, t, 16);
      const int h = nt * 8 + 2 * c + e;
      if (g == 0) {
        s_ml[warp][h][0] = m[nt][e] == kNoMax ? -INFINITY : m[nt][e];
        s_ml[warp][h][1] = t;
      }
#pragma unroll
      for (int j = 0; j < OT; ++j)
        *reinterpret_cast<float2 *>(po + L::at(h, g * L::kCpl + 2 * j)) = make_float2(o[nt][j][e], o[nt][j][e + 2]);
    }
  }
  __syncthreads();

  // ---- joined over the CTA's warps (a warp without a token has m = -inf, l = 0), two channels a thread
  float *cta_o = reinterpret_cast<float *>(smem);
  const int n_pairs = HG * (D / 2);
  for (int i = threadIdx.x; i < n_pairs; i += kWarps * 32) {
    const int h = i / (D / 2), ch = 2 * (i % (D / 2));
    float2 ml[kWarps], ow[kWarps];
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      ml[w] = *reinterpret_cast<const float2 *>(s_ml[w][h]);
      ow[w] = *reinterpret_cast<const float2 *>(reinterpret_cast<const float *>(smem + w * L::kWarpBytes) + L::at(h, ch));
      M = fmaxf(M, ml[w].x);
    }
    const float Mu = M == -INFINITY ? 0.f : M;
    float ls = 0.f;
    float2 acc = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = ex2(ml[w].x - Mu);
      ls = fmaf(f, ml[w].y, ls);
      acc.x = fmaf(f, ow[w].x, acc.x);
      acc.y = fmaf(f, ow[w].y, acc.y);
    }
    *reinterpret_cast<float2 *>(cta_o + L::at(h, ch)) = acc;  // warp 0's elements (h, ch ..): read by this thread only
    if (ch == 0) *reinterpret_cast<float2 *>(s_cta[h]) = make_float2(M, ls);
  }
  if (CS > 1) {
    cluster_arrive_release();
    cluster_wait();
  } else {
    __syncthreads();
  }

  // ---- joined over the cluster: each CTA writes a share of the outputs
  const size_t n_units = static_cast<size_t>(a.batch) * a.n_kv_heads * a.n_head_chunks;
  const int share = (n_pairs + CS - 1) / CS, i_end = min(n_pairs, (rank + 1) * share);
  for (int i = rank * share + threadIdx.x; i < i_end; i += kWarps * 32) {
    const int h = i / (D / 2), ch = 2 * (i % (D / 2));
    float M, ls;
    float2 acc;
    if (CS == 1) {
      const float2 t = *reinterpret_cast<const float2 *>(s_cta[h]);
      M = t.x;
      ls = t.y;
      acc = *reinterpret_cast<const float2 *>(cta_o + L::at(h, ch));
    } else {
      const uint32_t am = smem_addr(s_cta[h]), ao = smem_addr(cta_o + L::at(h, ch));
      float2 mr[kMaxCluster], orr[kMaxCluster];  // all loads first: one round trip
      M = -INFINITY;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        mr[r] = r < CS ? ld_cluster(cluster_map(am, r)) : make_float2(-INFINITY, 0.f);
        orr[r] = r < CS ? ld_cluster(cluster_map(ao, r)) : make_float2(0.f, 0.f);
      }
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) M = fmaxf(M, mr[r].x);
      const float Mu = M == -INFINITY ? 0.f : M;
      ls = 0.f;
      acc = make_float2(0.f, 0.f);
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        const float f = ex2(mr[r].x - Mu);
        ls = fmaf(f, mr[r].y, ls);
        acc.x = fmaf(f, orr[r].x, acc.x);
        acc.y = fmaf(f, orr[r].y, acc.y);
      }
    }
    if (a.n_split > 1) {
      float *ml = a.part + (static_cast<size_t>(unit) * a.n_split + part) * HG * 2;
      float *pp = a.part + n_units * a.n_split * HG * 2 + (static_cast<size_t>(unit) * a.n_split + part) * HG * D;
      *reinterpret_cast<float2 *>(pp + 2 * i) = acc;
      if (ch == 0) *reinterpret_cast<float2 *>(ml + 2 * h) = make_float2(M, ls);
    } else {
      const float2 res = ls == 0.f ? make_float2(0.f, 0.f) : make_float2(acc.x / ls, acc.y / ls);
      const size_t head = static_cast<size_t>(b) * a.n_q_heads + head0 + h;
      if (a.out_dtype == 1)
        *reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(a.out) + head * D + ch) = __floats2bfloat162_rn(res.x, res.y);
      else *reinterpret_cast<float2 *>(static_cast<float *>(a.out) + head * D + ch) = res;
      if (a.lse && ch == 0) a.lse[head] = ls == 0.f ? -INFINITY : (M + (log2f(ls) - kPShift)) * 0.69314718055994531f;
    }
  }
  if (CS > 1) {  // no CTA leaves while another reads its shared memory
    cluster_arrive_release();
    cluster_wait();
  }
}

// Joins the n_split partials of one (unit, head): eight groups of D threads
// take every eighth part, the groups are joined in shared memory.
constexpr int kMergeGroups = 8;
template <int D>
__global__ void __launch_bounds__(kMergeGroups * D) kv4_merge_kernel(Kv4AttnArgs a) {
  __shared__ float s_o[kMergeGroups][D], s_m[kMergeGroups], s_l[kMergeGroups];
  grid_dependency_wait();
  const int HG = a.head_chunk;
  const int unit = blockIdx.x / HG, h = blockIdx.x % HG;
  const int ch = threadIdx.x % D, grp = threadIdx.x / D;
  const size_t n_units = static_cast<size_t>(a.batch) * a.n_kv_heads * a.n_head_chunks;
  const float *ml = a.part + static_cast<size_t>(unit) * a.n_split * HG * 2 + 2 * h;
  const float *po = a.part + n_units * a.n_split * HG * 2 + static_cast<size_t>(unit) * a.n_split * HG * D + h * D + ch;
  constexpr int U = 8;  // parts in flight
  float M = -INFINITY, ls = 0.f, acc = 0.f;
  for (int p0 = grp; p0 < a.n_split; p0 += U * kMergeGroups) {
    float mv[U], lv[U], ov[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int p = p0 + u * kMergeGroups;
      const bool ok = p < a.n_split;
      mv[u] = ok ? ml[static_cast<size_t>(p) * HG * 2] : -INFINITY;
      lv[u] = ok ? ml[static_cast<size_t>(p) * HG * 2 + 1] : 0.f;
      ov[u] = ok ? po[static_cast<size_t>(p) * HG * D] : 0.f;
    }
    float Mn = M;
#pragma unroll
    for (int u = 0; u < U; ++u) Mn = fmaxf(Mn, mv[u]);
    const float Mu = Mn == -INFINITY ? 0.f : Mn;
    const float f0 = ex2(M - Mu);
    ls *= f0;
    acc *= f0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float f = ex2(mv[u] - Mu);
      ls = fmaf(f, lv[u], ls);
      acc = fmaf(f, ov[u], acc);
    }
    M = Mn;
  }
  s_o[grp][ch] = acc;
  if (ch == 0) {
    s_m[grp] = M;
    s_l[grp] = ls;
  }
  __syncthreads();
  if (grp != 0) return;
#pragma unroll
  for (int i = 0; i < kMergeGroups; ++i) M = fmaxf(M, s_m[i]);
  const float Mu = M == -INFINITY ? 0.f : M;
  ls = acc = 0.f;
#pragma unroll
  for (int i = 0; i < kMergeGroups; ++i) {
    const float f = ex2(s_m[i] - Mu);
    ls = fmaf(f, s_l[i], ls);
    acc = fmaf(f, s_o[i][ch], acc);
  }
  const int group = unit / a.n_head_chunks, hc = unit % a.n_head_chunks;
  const int b = group / a.n_kv_heads, gk = group % a.n_kv_heads;
  const size_t head = static_cast<size_t>(b) * a.n_q_heads + gk * (a.n_q_heads / a.n_kv_heads) + hc * HG + h;
  const float res = ls == 0.f ? 0.f : acc / ls;
  if (a.out_dtype == 1) static_cast<__nv_bfloat16 *>(a.out)[head * D + ch] = __float2bfloat16_rn(res);
  else static_cast<float *>(a.out)[head * D + ch] = res;
  if (a.lse && ch == 0) a.lse[head] = ls == 0.f ? -INFINITY : (M + (log2f(ls) - kPShift)) * 0.69314718055994531f;
}

// Partials that a call may leave in the workspace, over all units.
int max_parts(int sms) { return 4 * sms; }

// How a call is cut: heads per unit, and either CTAs per cluster or parts per
// unit (joined by a second launch), whichever this estimate in tenths of a
// microsecond finds cheapest.  A warp takes 1.9 us for a tile when two CTAs
// share an SM and 1.1 us alone, a wave of CTAs costs 3.5 us around its tiles;
// 16 heads, always alone on their SM, 1.7 us and 15 us (nothing covers a wave's
// start and its joins); a cluster 1 us, the second launch 3.  It is a rule to
// choose by and no prediction: fitted at d 128, it counts a wave that is hardly
// begun as a whole one and so misjudges cuts that it does not take.  Measured
// over 680 shapes (both d; 4, 8 and 16 heads; 1 to 256 units; lists of 128 to
// 8192 tokens and every one of up to 98304) its choice is within 1.1 % of the
// best cut on average and within 5 % for 94 of 100; the worst is 16 units of
// 8192 listed tokens (16.7 us with clusters of 8, 13.2 as 18 parts).  Some of
// them: 64 units of 4096 listed tokens 19.6 us with clusters of 4 (one wave),
// 22.5 with 2, 22.9 as 4 parts, 24.7 with 8, 25.7 as 9 parts; 64 units of 98304
// tokens 173 us as 9 parts (two full waves), 189 with clusters of 4, 200 with 8;
// with 16 heads 338 with clusters of 2, 348 as 9 parts, and 96 units of 32768
// tokens 187 us as 3 parts, 229 whole.
void kv4_plan(Kv4AttnArgs &a, int n_max) {
  const int G = a.n_q_heads / a.n_kv_heads;
  a.head_chunk = std::min(G, 16);
  a.n_head_chunks = G / a.head_chunk;
  const int units = a.batch * a.n_kv_heads * a.n_head_chunks;
  const int sms = a.num_sms > 0 ? a.num_sms : 148;
  const int resident = a.head_chunk > 8 ? sms : 2 * sms;              // 16 heads: one CTA an SM (registers)
  const int tiles = std::max(1, (n_max + kTile - 1) / kTile);         // of one unit
  const int most = (tiles + kWarps - 1) / kWarps;                     // CTAs of a unit that still have a tile for every warp
  // clusters of 4 and 8 do not fill every GPC: 7/8 and 13/16 of the places (at one CTA an SM 132 and 120 of 148 run at once)
  auto places = [&](int cluster) { return cluster == 8 ? resident * 13 / 16 : cluster == 4 ? resident * 7 / 8 : resident; };
  a.cluster = a.n_split = 1;
  long long best = -1;
  auto consider = [&](int cluster, int n_split) {
    const int per_unit = cluster * n_split;
    const long long ctas = static_cast<long long>(units) * per_unit;
    const int rounds = (tiles + per_unit * kWarps - 1) / (per_unit * kWarps);
    const long long waves = (ctas + places(cluster) - 1) / places(cluster);
    const int wave = resident == sms ? 150 : 35, tile = resident == sms ? 17 : ctas <= sms ? 11 : 19;
    const long long cost = waves * (wave + rounds * tile) + (cluster > 1 ? 10 : 0) + (n_split > 1 ? 30 : 0);
    if (best < 0 || cost < best) {
      best = cost;
      a.cluster = cluster;
      a.n_split = n_split;
    }
  };
  for (int c = 1; c <= kMaxCluster && (c == 1 || c <= most); c *= 2) consider(c, 1);
  for (int c : {1, kMaxCluster})  // as many parts as fill one to four waves
    for (int w = 1; w <= 4; ++w) {
      const int p = std::min({static_cast<int>(static_cast<long long>(w) * places(c) / (static_cast<long long>(units) * c)),
                              most / c, kMaxSplit, max_parts(sms) / units});
      if (p >= 2) consider(c, p);
    }
}

template <int D, int NT, bool LOCOL, bool LIST, bool PAGED>
cudaError_t run(const Kv4AttnArgs &a, cudaStream_t st) {
  using L = Kv4Smem<D, NT>;
  auto kern = kv4_attn_kernel<D, NT, LOCOL, LIST, PAGED>;
  static bool configured[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) configured[dev] = true;
  }
  const long long ctas = static_cast<long long>(a.batch) * a.n_kv_heads * a.n_head_chunks * a.n_split * a.cluster;
  return launch_pdl_cluster(kern, dim3(static_cast<unsigned>(ctas)), dim3(kWarps * 32), L::kSmem, st, a.cluster, a);
}

template <int D, int NT, bool LOCOL>
cudaError_t dispatch(const Kv4AttnArgs &a, cudaStream_t st) {
  if (!a.token_idx) return run<D, NT, LOCOL, false, false>(a, st);
  return a.slot_of_block ? run<D, NT, LOCOL, true, true>(a, st) : run<D, NT, LOCOL, true, false>(a, st);
}
template <int D>
cudaError_t dispatch(const Kv4AttnArgs &a, cudaStream_t st) {
  if (a.head_chunk <= 4) return dispatch<D, 1, true>(a, st);
  return a.head_chunk <= 8 ? dispatch<D, 1, false>(a, st) : dispatch<D, 2, false>(a, st);
}

}  // namespace

size_t kv4_attn_part_floats(int heads_per_group, int d, int num_sms) {
  return static_cast<size_t>(max_parts(num_sms > 0 ? num_sms : 148)) * std::min(heads_per_group, 16) * (2 + d);
}

cudaError_t launch_kv4_attention(Kv4AttnArgs a, cudaStream_t st) {
  kv4_plan(a, a.token_idx ? a.k_t : a.max_ctx);
  const cudaError_t e = a.d == 128 ? dispatch<128>(a, st) : dispatch<64>(a, st);
  if (e != cudaSuccess || a.n_split == 1) return e;
  const dim3 grid(a.batch * a.n_q_heads);  // units times their heads
  if (a.d == 128) return launch_pdl(kv4_merge_kernel<128>, grid, dim3(kMergeGroups * 128), 0, st, a);
  return launch_pdl(kv4_merge_kernel<64>, grid, dim3(kMergeGroups * 64), 0, st, a);
}

}  // namespace tls
