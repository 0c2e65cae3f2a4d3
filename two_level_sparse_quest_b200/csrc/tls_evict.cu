// tls_evict.cu -- eviction from a KV cache by accumulated attention weight
// (tls_weights.cu): which tokens stay, and the cache's rows moved together.
//
// select: per (sequence, KV head) the first n_sink tokens, the last n_recent,
//   and of the rest those with the largest weights, `budget` in all, ties to
//   the lower index, ids ascending.  One thread-block cluster per group; each
//   CTA reads its slice of the weights once into shared memory as ordered
//   keys (a slice beyond that room is read again from L2), then three radix
//   passes of 11, 11 and 10 bits find the budget-th largest key: every CTA
//   histograms its slice, one cluster barrier, every CTA sums the cluster's
//   histograms over distributed shared memory and finds the same digit.  The
//   compaction counts per warp, then per CTA, then over the cluster, and
//   writes ids at their ranks.  Tokens that no step selected share the weight
//   zero, so that key is counted in registers instead of by atomics on one bin.
// compact: row keep[j] moves to row j.  As keep ascends, a chunk of rows only
//   overwrites rows that no later chunk reads, so chunk by chunk -- all loads,
//   a barrier, all stores -- is in place without a copy.  A cluster takes a
//   column slice of one array of one group and a super-chunk of rows at a
//   time, so a single sequence still fills the GPU.
// Both are bound by HBM: 4 bytes a token, and each kept row once in and out.
#include <algorithm>

#include "tls_device.cuh"
#include "tls_internal.h"

namespace tls {
namespace {

// ---------------------------------------------------------------- select
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kSelCap = 49152;          // keys of one CTA in shared memory (192 KB)
constexpr uint32_t kZeroKey = 0x80000000u;
constexpr uint32_t kProtected = 0xffffffffu;  // above +inf

__device__ __forceinline__ int4 ld_cluster_v4(uint32_t addr) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ int2 ld_cluster_v2(uint32_t addr) {
  int2 v;
  asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(EvictArgs a, int CS, int cap) {
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ __align__(16) int hist[2][kBins];
  __shared__ __align__(8) int2 s_tot;   // this CTA's keys above and equal to the threshold
  __shared__ int s_gt[kSelWarps], s_eq[kSelWarps], s_scan[33], s_found[3];
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
  const int slice = ((len + CS - 1) / CS + 31) & ~31;
  const int t0 = min(rank * slice, len), n = min(slice, len - t0);
  const float *w = a.weights + static_cast<size_t>(group) * a.max_ctx + t0;
  auto key_of = [&](int i, float v) -> uint32_t {
    const int t = t0 + i;
    if (t < a.n_sink || t >= len - a.n_recent) return kProtected;
    return score_key(v != v ? -INFINITY : v);  // a NaN ranks as -inf
  };
  auto key_at = [&](int i) -> uint32_t { return i < cap ? keys[i] : key_of(i, w[i]); };

  // pass 0 reads the weights; U loads in flight per thread
  constexpr int U = 8;
  int zeros = 0;  // keys of weight zero seen by this thread
  for (int i = tid; i < kBins; i += kSelThreads) hist[0][i] = hist[1][i] = 0;
  __syncthreads();
  for (int i0 = tid; i0 < n; i0 += U * kSelThreads) {
    float v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kSelThreads;
      v[u] = i < n ? w[i] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kSelThreads;
      if (i < n) {
        const uint32_t key = key_of(i, v[u]);
        if (i < cap) keys[i] = key;
        if (key == kZeroKey) ++zeros;
        else atomicAdd(&hist[0][key >> 21], 1);
      }
    }
  }
  zeros = __reduce_add_sync(0xffffffffu, zeros);
  if (lane == 0 && zeros) atomicAdd(&hist[0][kZeroKey >> 21], zeros);
  __syncwarp();

  uint32_t thr = 0;
  int krem = k;
#pragma unroll 1
  for (int p = 0; p < 3; ++p) {
    const int shift = p == 0 ? 21 : p == 1 ? 10 : 0;
    int *h = hist[p & 1];
    // every CTA's histogram is complete (and its previous one no longer read)
    if (CS > 1) {
      cluster_arrive_release();
      cluster_wait();
    } else {
      __syncthreads();
    }
    // thread t owns the four bins kBins - 4 - 4 t .. + 3, from the top
    const int b0 = kBins - 4 - 4 * tid;
    int4 s = make_int4(0, 0, 0, 0);
    const uint32_t ha = smem_addr(h + b0);
    for (int r = 0; r < CS; ++r) {
      const int4 x = CS > 1 ? ld_cluster_v4(cluster_map(ha, r)) : *reinterpret_cast<const int4 *>(h + b0);
      s.x += x.x;
      s.y += x.y;
      s.z += x.z;
      s.w += x.w;
    }
    int total;
    int acc = block_excl_scan<kSelThreads>(s.x + s.y + s.z + s.w, s_scan, total);
    const int cnt[4] = {s.w, s.z, s.y, s.x};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (acc < krem && acc + cnt[j] >= krem) {  // exactly one bin of the cluster's sum satisfies this
        s_found[0] = b0 + 3 - j;
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
    // the other buffer for the next digit (pass 2 clears pass 0's first: every CTA has read it by now)
    int *hn = hist[(p + 1) & 1];
    if (p == 1) {
      for (int i = tid; i < kBins; i += kSelThreads) hn[i] = 0;
    }
    __syncthreads();
    const int nshift = p == 0 ? 10 : 0;
    const uint32_t nmask = p == 0 ? 2047u : 1023u;
    const uint32_t want = thr >> shift;
    for (int i = tid; i < n; i += kSelThreads) {
      const uint32_t key = key_at(i);
      if (key != kZeroKey && (key >> shift) == want) atomicAdd(&hn[(key >> nshift) & nmask], 1);
    }
    if (lane == 0 && zeros && (kZeroKey >> shift) == want) atomicAdd(&hn[(kZeroKey >> nshift) & nmask], zeros);
    __syncwarp();
  }

  // ---- ids at their ranks: warp w owns a contiguous run of the slice
  const int seg = ((n + kSelWarps - 1) / kSelWarps + 31) & ~31;
  const int i_begin = warp * seg, i_end = min(i_begin + seg, n);
  int ngt = 0, neq = 0;
  for (int i0 = i_begin; i0 < i_end; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t key = i < i_end ? key_at(i) : 0u;  // 0 is below every key
    ngt += __popc(__ballot_sync(0xffffffffu, key > thr));
    neq += __popc(__ballot_sync(0xffffffffu, i < i_end && key == thr));
  }
  if (lane == 0) {
    s_gt[warp] = ngt;
    s_eq[warp] = neq;
  }
  __syncthreads();
  int gt_before = 0, eq_before = 0, gt_all = 0, eq_all = 0;
  for (int v = 0; v < kSelWarps; ++v) {
    if (v < warp) {
      gt_before += s_gt[v];
      eq_before += s_eq[v];
    }
    gt_all += s_gt[v];
    eq_all += s_eq[v];
  }
  if (CS > 1) {
    if (tid == 0) s_tot = make_int2(gt_all, eq_all);
    cluster_arrive_release();
    cluster_wait();
    for (int r = 0; r < rank; ++r) {
      const int2 x = ld_cluster_v2(cluster_map(smem_addr(&s_tot), r));
      gt_before += x.x;
      eq_before += x.y;
    }
    cluster_arrive_release();  // waited for at the end: no CTA leaves while its counts are read
  }
  int pos = gt_before + min(krem, eq_before);
  const unsigned below = (1u << lane) - 1u;
  for (int i0 = i_begin; i0 < i_end; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t key = i < i_end ? key_at(i) : 0u;
    const unsigned eq = __ballot_sync(0xffffffffu, i < i_end && key == thr);
    const bool sel = i < i_end && (key > thr || (key == thr && eq_before + __popc(eq & below) < krem));
    const unsigned m = __ballot_sync(0xffffffffu, sel);
    if (sel) {
      const int at = pos + __popc(m & below);
      if (at < k) keep[at] = t0 + i;  // always holds; keeps the write in bounds
    }
    pos += __popc(m);
    eq_before += __popc(eq);
  }
  if (CS > 1) cluster_wait();
}

// ---------------------------------------------------------------- compact
constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 8;

template <typename V>
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
  // the first rows usually stay where they are: nothing to load or store there
  for (long long j0 = 0; j0 < rows; j0 += static_cast<long long>(chunk) * CS) {
    const long long first = j0 + static_cast<long long>(rank) * chunk + r;
    V x[kMoveUnroll];
    int src[kMoveUnroll];
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const long long j = first + u * per_pass;
      src[u] = on && j < rows ? keep[j] : static_cast<int>(min(j, 0x7fffffffLL));
      if (src[u] >= a.max_ctx) src[u] = static_cast<int>(j);  // out of range: the row stays
    }
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const long long j = first + u * per_pass;
      if (src[u] >= 0 && src[u] != j) x[u] = base[static_cast<size_t>(src[u]) * row_vecs + v];
    }
    if (CS > 1) {
      cluster_arrive_release();
      cluster_wait();
    } else {
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const long long j = first + u * per_pass;
      if (src[u] >= 0 && src[u] != j) base[static_cast<size_t>(j) * row_vecs + v] = x[u];
      if constexpr (sizeof(V) == 4)
        if (zero_tail && src[u] < 0) base[static_cast<size_t>(j) * row_vecs + v] = V(0);
    }
  }
  if constexpr (sizeof(V) == 4)
    if (zero_tail)  // every load of this cluster is done (the last barrier, or there was none)
      for (long long j = static_cast<long long>(a.budget) + rank * kMoveThreads + threadIdx.x; j < len; j += static_cast<long long>(CS) * kMoveThreads)
        base[j] = V(0);
}

struct MovePlan {
  int vec_bytes[kMaxEvictRows + 1];  // load width of each array
  int slice[kMaxEvictRows + 1];      // columns of a slice, in vectors
  int first[kMaxEvictRows + 2];      // first slice index of each array
  int cluster;
};

__global__ void __launch_bounds__(kMoveThreads) evict_compact_kernel(CompactArgs a, MovePlan p) {
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
    case 16: move_rows<uint4>(a, arr, vec0, n_vec, group, len, rank, CS); break;
    case 8: move_rows<uint2>(a, arr, vec0, n_vec, group, len, rank, CS); break;
    case 4: move_rows<uint32_t>(a, arr, vec0, n_vec, group, len, rank, CS); break;
    case 2: move_rows<uint16_t>(a, arr, vec0, n_vec, group, len, rank, CS); break;
    default: move_rows<uint8_t>(a, arr, vec0, n_vec, group, len, rank, CS); break;
  }
}

}  // namespace

cudaError_t launch_evict_select(const EvictArgs &a, cudaStream_t st) {
  // about 4096 keys a CTA or more; beyond eight CTAs the slices grow
  int cs = 1;
  while (cs < kMaxCluster && static_cast<long long>(cs) * 4096 < a.max_ctx) cs *= 2;
  const long long slice = ((static_cast<long long>(a.max_ctx) + cs - 1) / cs + 31) / 32 * 32;
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
  return launch_pdl_cluster(evict_select_kernel, dim3(a.batch * a.n_kv_heads * cs), dim3(kSelThreads), smem, st, cs, a,
                            cs, cap);
}

cudaError_t launch_evict_compact(const CompactArgs &a, cudaStream_t st) {
  MovePlan p{};
  const int groups = a.batch * a.n_kv_heads;
  const int want = 4 * (a.num_sms > 0 ? a.num_sms : 148);  // CTAs that keep HBM busy
  int slices = 0;
  for (int i = 0; i < a.n_rows; ++i) {
    // the widest access that divides the row and that every row starts on
    const size_t addr = reinterpret_cast<size_t>(a.rows[i]);
    int v = 16;
    while (v > 1 && (a.row_bytes[i] % v || addr % v)) v /= 2;
    const int vecs = a.row_bytes[i] / v;
    // whole rows up to 256 bytes where the groups alone are many, else columns of 64 bytes or a little less
    const int wide = static_cast<long long>(groups) * a.n_rows * kMaxCluster >= want ? 256 : 64;
    const int n_slices = (a.row_bytes[i] + wide - 1) / wide;
    p.vec_bytes[i] = v;
    p.slice[i] = std::min((vecs + n_slices - 1) / n_slices, kMoveThreads);
    p.first[i] = slices;
    slices += (vecs + p.slice[i] - 1) / p.slice[i];
  }
  p.first[a.n_rows] = slices;
  int cs = 1;
  while (cs < kMaxCluster && static_cast<long long>(groups) * slices * cs < want) cs *= 2;
  p.cluster = cs;
  return launch_pdl_cluster(evict_compact_kernel, dim3(slices * cs, groups), dim3(kMoveThreads), 0, st, cs, a, p);
}

}  // namespace tls
