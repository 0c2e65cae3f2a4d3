// tls_evict.cu -- eviction from a KV cache by accumulated attention weight
// (tls_weights.cu): which tokens stay, and the cache's rows moved together.
//
// select: per (sequence, KV head) the first n_sink tokens, the last n_recent,
//   and of the rest those with the largest weights, `budget` in all, ties to
//   the lower index, ids ascending.  One thread-block cluster per group; each
//   CTA reads its slice of the weights once, into shared memory as ordered
//   keys (a slice beyond that room is read again from L2), and three radix
//   passes of 11, 11 and 10 bits find the budget-th largest key: every CTA
//   counts its slice and adds its non-zero counts into every CTA's sums with
//   remote shared-memory reductions (few: weights share their exponents), so
//   that after one cluster barrier each finds the same digit from its own
//   shared memory (reading everyone's 2048 counts took 2.3 us a pass with
//   eight CTAs).  The second pass sets the keys of the found bin apart, the
//   third reads only those.  The compaction counts per warp, CTA and cluster,
//   and writes ids at their ranks.  Tokens that no step selected share the
//   weight zero, so that key is counted in registers instead of by atomics on
//   one bin.
// compact: row keep[j] moves to row j.  As keep ascends, a chunk of rows only
//   overwrites rows that no later chunk reads, so chunk by chunk -- all loads,
//   a barrier, all stores -- is in place without a copy.  A CTA takes a column
//   slice of one array of one group; where such slices are few, a cluster takes
//   it, a chunk for each of its CTAs at a time, so that a single sequence still
//   fills the GPU.
// Both are bound by HBM: 4 bytes a token, and each kept row once in and out.
// Half of 8 x 8 caches of 98304 tokens, K and V in bf16: 567 us in all, the
// selection 28 to 33 of them (by the weights' spread; the moves 6.0 TB/s); one
// sequence of 49152 tokens in 4 bits 34 us, the selection 12 to 15.
#include <algorithm>

#include "tls_cache.h"
#include "tls_device.cuh"

namespace tls {
namespace {

// ---------------------------------------------------------------- select
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kSelCap = 49152;          // keys of one CTA in shared memory (192 KB), a multiple of 128
constexpr int kCandCap = 2048;          // of them, those that share the first digit of the threshold, kept apart
constexpr uint32_t kZeroKey = 0x80000000u;
constexpr uint32_t kProtected = 0xffffffffu;  // above +inf
static_assert(kBins == 2 * kSelThreads, "a thread owns two bins");

__device__ __forceinline__ void red_cluster(uint32_t addr, int v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_v2(uint32_t addr, int2 v) {
  asm volatile("st.shared::cluster.v2.s32 [%0], {%1, %2};" ::"r"(addr), "r"(v.x), "r"(v.y) : "memory");
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(EvictArgs a, int CS, int cap) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ __align__(16) int hist[kBins];      // this CTA's counts of the current digit
  __shared__ __align__(16) int sums[2][kBins];   // the cluster's (CS > 1): every CTA adds its counts into everyone's
  __shared__ uint32_t cand[kCandCap];
  __shared__ __align__(8) int2 s_tot[kMaxCluster];  // each CTA's keys above and equal to the threshold
  __shared__ int s_gt[kSelWarps], s_eq[kSelWarps], s_scan[33], s_found[3], s_cand;
  grid_dependency_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(blockIdx.x) % CS, group = static_cast<int>(blockIdx.x) / CS;
  const int b = group / a.n_kv_heads;
  const int len = min(max(a.seq_lens[b], 0), a.max_ctx);
  const int k = min(len, a.budget);
  int32_t *keep = a.keep_idx + static_cast<size_t>(group) * a.budget;
  if (rank == 0 && tid == 0 && group % a.n_kv_heads == 0) a.new_lens[b] = k;
  for (int i = k + rank * kSelThreads + tid; i < a.budget; i += CS * kSelThreads) keep[i] = -1;
  if (len <= a.budget) {  // every token stays
    for (int i = rank * kSelThreads + tid; i < len; i += CS * kSelThreads) keep[i] = i;
    return;
  }
  const int slice = ((len + CS - 1) / CS + 127) & ~127;
  const int t0 = min(rank * slice, len), n = min(slice, len - t0);
  const float *w = a.weights + static_cast<size_t>(group) * a.max_ctx + t0;
  // keys i .. i + 3 of the slice from their weights; 0, below every key, past its end
  const int free_lo = a.n_sink - t0, free_hi = len - a.n_recent - t0;  // [free_lo, free_hi): ranked by weight
  auto key_of = [&](int i, float v) -> uint32_t {
    if (i >= n) return 0u;
    if (i < free_lo || i >= free_hi) return kProtected;
    return score_key(v != v ? -INFINITY : v);  // a NaN ranks as -inf
  };
  auto keys_of = [&](int i, const float4 &v) {
    return make_uint4(key_of(i, v.x), key_of(i + 1, v.y), key_of(i + 2, v.z), key_of(i + 3, v.w));
  };
  const bool wide = (reinterpret_cast<size_t>(w) & 15) == 0;
  auto weights_at = [&](int i) -> float4 {
    if (wide && i + 4 <= n) return *reinterpret_cast<const float4 *>(w + i);
    return make_float4(i < n ? w[i] : 0.f, i + 1 < n ? w[i + 1] : 0.f, i + 2 < n ? w[i + 2] : 0.f, i + 3 < n ? w[i + 3] : 0.f);
  };
  auto keys_at = [&](int i) -> uint4 {
    return i < cap ? *reinterpret_cast<const uint4 *>(keys + i) : keys_of(i, weights_at(i));
  };

  hist[2 * tid] = hist[2 * tid + 1] = 0;
  if (CS > 1) sums[0][2 * tid] = sums[0][2 * tid + 1] = sums[1][2 * tid] = sums[1][2 * tid + 1] = 0;
  if (tid == 0) s_cand = 0;
  __syncthreads();
  if (CS > 1) cluster_arrive_release();  // waited for before the first add into another CTA's sums

  // the weights, once: keys into shared memory, counts of the first digit
  constexpr int U = 4;  // reads of four weights in flight per thread
  int zeros = 0;        // keys of weight zero seen by this thread
  auto count = [&](uint32_t key) {
    if (key == kZeroKey) ++zeros;
    else if (key != 0u) atomicAdd(&hist[key >> 21], 1);
  };
  for (int i0 = 4 * tid; i0 < n; i0 += 4 * U * kSelThreads) {
    float4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + 4 * u * kSelThreads;
      if (i < n) v[u] = weights_at(i);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + 4 * u * kSelThreads;
      if (i < n) {
        const uint4 key = keys_of(i, v[u]);
        if (i < cap) *reinterpret_cast<uint4 *>(keys + i) = key;
        count(key.x);
        count(key.y);
        count(key.z);
        count(key.w);
      }
    }
  }
  __syncwarp();
  zeros = __reduce_add_sync(0xffffffffu, zeros);
  if (lane == 0 && zeros) atomicAdd(&hist[kZeroKey >> 21], zeros);
  __syncwarp();
  if (CS > 1) cluster_wait();

  uint32_t thr = 0;
  int krem = k;
#pragma unroll 1
  for (int p = 0; p < 3; ++p) {
    const int shift = p == 0 ? 21 : p == 1 ? 10 : 0;
    __syncthreads();  // this CTA's counts are complete
    // thread t owns the bins kBins - 2 - 2 t and the next, from the top
    const int b0 = kBins - 2 - 2 * tid;
    int2 s = *reinterpret_cast<const int2 *>(hist + b0);
    *reinterpret_cast<int2 *>(hist + b0) = make_int2(0, 0);  // for the next digit
    if (CS > 1) {
      int *sum = sums[p & 1] + b0;
      const uint32_t sa = smem_addr(sum);
      if (s.x | s.y)
        for (int r = 0; r < CS; ++r) {
          if (s.x) red_cluster(cluster_map(sa, r), s.x);
          if (s.y) red_cluster(cluster_map(sa, r) + 4, s.y);
        }
      __syncwarp();
      cluster_arrive_release();
      cluster_wait();
      s = *reinterpret_cast<const int2 *>(sum);
      *reinterpret_cast<int2 *>(sum) = make_int2(0, 0);  // pass 2 adds here again, after pass 1's barrier
    }
    int total;
    int acc = block_excl_scan<kSelThreads>(s.x + s.y, s_scan, total);
    const int cnt[2] = {s.y, s.x};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (acc < krem && acc + cnt[j] >= krem) {  // exactly one bin of the cluster's sum satisfies this
        s_found[0] = b0 + 1 - j;
        s_found[1] = acc;
        s_found[2] = cnt[j];
      }
      acc += cnt[j];
    }
    __syncthreads();
    thr |= static_cast<uint32_t>(s_found[0]) << shift;
    krem -= s_found[1];
    if (krem == s_found[2] && thr != 0u) {  // the whole bin is kept: every key from the bin's lowest up
      thr -= 1u;
      krem = 0;
      break;
    }
    if (p == 2) break;
    const uint32_t want = thr >> shift;
    if (p == 0) {  // the second digit of the keys that share the first, and those keys apart where they fit
      auto take = [&](uint32_t key) {
        if ((key >> 21) == want && key != kZeroKey && key != 0u) {
          atomicAdd(&hist[(key >> 10) & 2047u], 1);
          const int at = atomicAdd(&s_cand, 1);
          if (at < kCandCap) cand[at] = key;
        }
      };
      for (int i = 4 * tid; i < n; i += 4 * kSelThreads) {
        const uint4 key = keys_at(i);
        take(key.x);
        take(key.y);
        take(key.z);
        take(key.w);
      }
      if (lane == 0 && zeros && (kZeroKey >> 21) == want) atomicAdd(&hist[(kZeroKey >> 10) & 2047u], zeros);
    } else {
      const int nc = s_cand;
      auto take = [&](uint32_t key) {
        if ((key >> 10) == want && key != kZeroKey && key != 0u) atomicAdd(&hist[key & 1023u], 1);
      };
      if (nc <= kCandCap) {
        for (int i = tid; i < nc; i += kSelThreads) take(cand[i]);
      } else {
        for (int i = 4 * tid; i < n; i += 4 * kSelThreads) {
          const uint4 key = keys_at(i);
          take(key.x);
          take(key.y);
          take(key.z);
          take(key.w);
        }
      }
      if (lane == 0 && zeros && (kZeroKey >> 10) == want) atomicAdd(&hist[kZeroKey & 1023u], zeros);
    }
    __syncwarp();
  }

  // ---- ids at their ranks: warp w owns a contiguous run of the slice, a lane four neighbours a step
  const int seg = ((n + kSelWarps - 1) / kSelWarps + 127) & ~127;
  const int i_begin = warp * seg, i_end = min(i_begin + seg, n);
  int ngt = 0, neq = 0;
#pragma unroll 2
  for (int i = i_begin + 4 * lane; i < i_end; i += 128) {
    const uint4 key = keys_at(i);
    ngt += (key.x > thr) + (key.y > thr) + (key.z > thr) + (key.w > thr);
    neq += (key.x == thr) + (key.y == thr) + (key.z == thr) + (key.w == thr);
  }
  __syncwarp();
  ngt = __reduce_add_sync(0xffffffffu, ngt);
  neq = __reduce_add_sync(0xffffffffu, neq);
  if (lane == 0) {
    s_gt[warp] = ngt;
    s_eq[warp] = neq;
  }
  __syncthreads();
  const int vg = s_gt[lane], ve = s_eq[lane];
  int gt_before = __reduce_add_sync(0xffffffffu, lane < warp ? vg : 0);
  int eq_before = __reduce_add_sync(0xffffffffu, lane < warp ? ve : 0);
  if (CS > 1) {
    if (warp == 0) {  // this CTA's totals to every CTA
      const int2 tot = make_int2(__reduce_add_sync(0xffffffffu, vg), __reduce_add_sync(0xffffffffu, ve));
      if (lane < CS) st_cluster_v2(cluster_map(smem_addr(&s_tot[rank]), lane), tot);
      __syncwarp();
    }
    cluster_arrive_release();
    cluster_wait();  // nothing is sent to another CTA after this: each may leave when it is done
    for (int r = 0; r < rank; ++r) {
      gt_before += s_tot[r].x;
      eq_before += s_tot[r].y;
    }
  }
  for (int i0 = i_begin; i0 < i_end; i0 += 128) {
    const int i = i0 + 4 * lane;
    uint4 q = make_uint4(0u, 0u, 0u, 0u);
    if (i < i_end) q = keys_at(i);
    const uint32_t key[4] = {q.x, q.y, q.z, q.w};
    int c = 0;  // this lane's keys above (low half) and equal to (high half) the threshold: at most 128 a step
#pragma unroll
    for (int e = 0; e < 4; ++e) c += (key[e] > thr ? 1 : 0) + (key[e] == thr ? 1 << 16 : 0);
    const int incl = warp_incl_scan(c), excl = incl - c, all = __shfl_sync(0xffffffffu, incl, 31);
    int eq = eq_before + (excl >> 16);
    int pos = gt_before + (excl & 0xffff) + min(krem, eq);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool same = key[e] == thr;
      if (key[e] > thr || (same && eq < krem)) {
        if (pos < k) keep[pos] = t0 + i + e;  // always holds; keeps the write in bounds
        ++pos;
      }
      eq += same;
    }
    gt_before += all & 0xffff;
    eq_before += all >> 16;
  }
}

// ---------------------------------------------------------------- compact
constexpr int kMoveUnroll = 8;

template <typename V, int kMoveThreads>
__device__ void move_rows(const CompactArgs &a, int arr, int vec0, int n_vec, int group, int len, int rank, int CS) {
  // columns vec0 .. vec0 + n_vec - 1 (in units of V) of array arr
  const size_t row_vecs = a.row_bytes[arr] / sizeof(V);
  V *base = static_cast<V *>(a.rows[arr]) + static_cast<size_t>(group) * a.max_ctx * row_vecs + vec0;
  const bool zero_tail = a.weights && a.rows[arr] == a.weights;
  const int32_t *keep = a.keep_idx + static_cast<size_t>(group) * a.budget;
  const int per_pass = kMoveThreads / n_vec;             // rows of one pass of the CTA
  const int r = threadIdx.x / n_vec, v = threadIdx.x % n_vec;
  const bool on = r < per_pass;
  const int chunk = per_pass * kMoveUnroll;
  const int rows = min(a.budget, len);
  const int step = chunk * CS;  // int: max_ctx is below 2^28 (the shape checks)
  auto sources = [&](int first, int (&src)[kMoveUnroll]) {  // this thread's rows: where they come from
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int j = first + u * per_pass;
      src[u] = on && j < rows ? keep[j] : j;
    }
  };
  int src[kMoveUnroll];
  sources(rank * chunk + r, src);
  for (int j0 = 0; j0 < rows; j0 += step) {
    const int first = j0 + rank * chunk + r;
    V x[kMoveUnroll];
    int next[kMoveUnroll];
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int j = first + u * per_pass;
      if (src[u] >= a.max_ctx) src[u] = j;  // out of range: the row stays
      if (src[u] >= 0 && src[u] != j) x[u] = base[static_cast<size_t>(src[u]) * row_vecs + v];
    }
    sources(first + step, next);  // on their way while the rows arrive
    if (CS > 1) {
      cluster_arrive_release();
      cluster_wait();
    } else {
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int j = first + u * per_pass;
      if (src[u] >= 0 && src[u] != j) base[static_cast<size_t>(j) * row_vecs + v] = x[u];
      if constexpr (sizeof(V) == 4)
        if (zero_tail && src[u] < 0) base[static_cast<size_t>(j) * row_vecs + v] = V(0);
      src[u] = next[u];
    }
  }
  if constexpr (sizeof(V) == 4)
    if (zero_tail)  // every load of this cluster is done (the last barrier, or there was none)
      for (int j = a.budget + rank * kMoveThreads + threadIdx.x; j < len; j += CS * kMoveThreads) base[j] = V(0);
}

struct MovePlan {
  int vec_bytes[kMaxEvictRows + 1];  // load width of each array
  int slice[kMaxEvictRows + 1];      // columns of a slice, in vectors
  int first[kMaxEvictRows + 2];      // first slice index of each array
  int cluster;
};

template <int kMoveThreads>
__global__ void __launch_bounds__(kMoveThreads, kMoveThreads == 256 ? 3 : 1) evict_compact_kernel(CompactArgs a, MovePlan p) {
  grid_dependency_wait();
  const int CS = p.cluster;
  const int rank = static_cast<int>(blockIdx.x) % CS, slice = static_cast<int>(blockIdx.x) / CS;
  const int group = blockIdx.y;
  int arr = 0;
  while (slice >= p.first[arr + 1]) ++arr;
  const int len = min(max(a.seq_lens[group / a.n_kv_heads], 0), a.max_ctx);
  const int vb = p.vec_bytes[arr];
  const int vec0 = (slice - p.first[arr]) * p.slice[arr];
  const int n_vec = min(p.slice[arr], a.row_bytes[arr] / vb - vec0);
  switch (vb) {
    case 16: move_rows<uint4, kMoveThreads>(a, arr, vec0, n_vec, group, len, rank, CS); break;
    case 8: move_rows<uint2, kMoveThreads>(a, arr, vec0, n_vec, group, len, rank, CS); break;
    case 4: move_rows<uint32_t, kMoveThreads>(a, arr, vec0, n_vec, group, len, rank, CS); break;
    case 2: move_rows<uint16_t, kMoveThreads>(a, arr, vec0, n_vec, group, len, rank, CS); break;
    default: move_rows<uint8_t, kMoveThreads>(a, arr, vec0, n_vec, group, len, rank, CS); break;
  }
}

}  // namespace

cudaError_t launch_evict_select(const EvictArgs &a, cudaStream_t st) {
  // One CTA an SM.  More CTAs a group while they find room and still have 4096
  // keys each; a slice beyond kSelCap keys is read again from L2.
  const int groups = a.batch * a.n_kv_heads;
  int cs = 1;
  while (cs < kMaxCluster && static_cast<long long>(cs) * 4096 < a.max_ctx &&
         static_cast<long long>(groups) * cs * 2 <= a.num_sms)
    cs *= 2;
  const long long slice = ((static_cast<long long>(a.max_ctx) + cs - 1) / cs + 127) / 128 * 128;
  const int cap = static_cast<int>(std::min<long long>(slice, kSelCap));
  const size_t smem = static_cast<size_t>(cap) * 4;
  static bool configured[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelCap * 4);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) configured[dev] = true;
  }
  return launch_pdl_cluster(evict_select_kernel, dim3(groups * cs), dim3(kSelThreads), smem, st, cs, a,
                            cs, cap);
}

cudaError_t launch_evict_compact(const CompactArgs &a, cudaStream_t st) {
  MovePlan p{};
  const int groups = a.batch * a.n_kv_heads;
  const int sms = a.num_sms > 0 ? a.num_sms : 148;
  // Column slices of whole rows up to 256 bytes, or narrower (64 bytes at
  // least) while clusters of eight do not reach two CTAs an SM; then the
  // largest cluster with which all CTAs run at once, three an SM.
  int slices = 0;
  for (int wide = 256; wide >= 64; wide /= 2) {
    slices = 0;
    for (int i = 0; i < a.n_rows; ++i) {
      // the widest access that divides the row and that every row starts on
      const size_t addr = reinterpret_cast<size_t>(a.rows[i]);
      int v = 16;
      while (v > 1 && (a.row_bytes[i] % v || addr % v)) v /= 2;
      const int vecs = a.row_bytes[i] / v;
      const int n_slices = (a.row_bytes[i] + wide - 1) / wide;
      p.vec_bytes[i] = v;
      p.slice[i] = std::min((vecs + n_slices - 1) / n_slices, 256);
      p.first[i] = slices;
      slices += (vecs + p.slice[i] - 1) / p.slice[i];
    }
    if (static_cast<long long>(groups) * slices * kMaxCluster >= 2 * sms) break;
  }
  p.first[a.n_rows] = slices;
  // Slices that nearly fill the SMs by themselves take a large CTA each: its
  // barrier is cheaper than a cluster's.  Half of 32768 tokens a group, large
  // CTAs against clusters: K, V in bf16 and weights 32 groups (96 slices) 126 us
  // against 114, 40 (120) 136 against 166, 64 184 against 197; 4-bit records and
  // weights 48 groups (96) 77 against 62, 64 (128) 83 against 98.  Over 65 such
  // counts (six row layouts, 4 to 256 groups) the rule is within 1 % of the
  // better of the two on average; it is furthest off where the slices are one and
  // a bit or nearly two waves (96 groups of d 64 rows 158 against 145).
  const long long units = static_cast<long long>(groups) * slices;
  if (units * 5 >= 4LL * sms) {
    p.cluster = 1;
    return launch_pdl(evict_compact_kernel<512>, dim3(slices, groups), dim3(512), 0, st, a, p);
  }
  int cs = 1;
  while (cs < kMaxCluster && units * cs * 2 <= 3 * sms) cs *= 2;
  p.cluster = cs;
  return launch_pdl_cluster(evict_compact_kernel<256>, dim3(slices * cs, groups), dim3(256), 0, st, cs, a, p);
}

}  // namespace tls
