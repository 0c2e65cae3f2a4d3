// tls_kv4.cu -- rows in and out of the 4-bit KV cache (record: tls_kv4.cuh).
//
// append: a CTA owns the appended rows of a few whole blocks of one group.  A
//   thread quantises sixteen channels of one row (32 bytes in, 8 code bytes
//   and a scale byte out): scale = amax / 6 rounded to e5m3, code = x / scale
//   rounded to e2m1, both to nearest even, quotients with one residual step so
//   that a tie is a tie.  While the rows
//   are in L1 the CTA also brings the block summary up to date (max / min are
//   associative and the summary holds stored values, so merging the new rows
//   into it gives the bits of a rebuild) and writes the label slab's rows.
// read: a thread widens eight channels of one row to bf16 (exact).
// Both are one pass over the rows.  A 48k prompt of 8 KV heads at d 128 (393k
// rows, 258 MB each way): append 66 us, bound by its instructions (130 per row
// and warp, DRAM at 0.43 of its peak); read 41 us, bound by HBM (6.3 TB/s).
#include <algorithm>

#include "tls_cache.h"
#include "tls_kv4.cuh"

namespace tls {
namespace {

constexpr int kRowThreads = 256;
constexpr int kReadRows = 4;  // rows of a thread in flight

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Elementwise max / min of two bf16 pairs (a NaN gives way, +0 above -0, as fmaxf / fminf).
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Sixteen bf16 (two 16-byte chunks) -> eight code bytes and a scale byte.
__device__ __forceinline__ uint2 quantise16(const uint4 &u, const uint4 &v, int *scale_byte) {
  const uint32_t lo[4] = {u.x, u.y, u.z, u.w}, hi[4] = {v.x, v.y, v.z, v.w};
  uint32_t m2 = 0;  // bf16 magnitudes order like their bits
#pragma unroll
  for (int i = 0; i < 4; ++i) m2 = max_u16x2(m2, max_u16x2(lo[i] & 0x7fff7fffu, hi[i] & 0x7fff7fffu));
  const uint32_t m = max(m2 & 0xffffu, m2 >> 16);
  if (m >= 0x7f80u) {
    *scale_byte = kKv4NanScale;
    return make_uint2(0u, 0u);
  }
  const int b = kv4_scale_byte(__uint_as_float(m << 16));
  *scale_byte = b;
  if (b == 0) return make_uint2(0u, 0u);
  const float s = kv4_scale_value(b), r = rcp_approx(s);
  return make_uint2(e2m1_codes(lo, s, r), e2m1_codes(hi, s, r));
}

__device__ __forceinline__ bool kv4_range(const Kv4RowsArgs &a, int b, int *old_len, int *new_len) {
  *old_len = a.old_lens[b];
  *new_len = a.new_lens[b];
  return *old_len >= 0 && *new_len >= *old_len && *new_len <= a.max_ctx && *new_len - *old_len <= a.row_stride;
}

template <int D>
__global__ void __launch_bounds__(kRowThreads) kv4_append_kernel(Kv4RowsArgs a) {
  using R = Kv4Rec<D>;
  constexpr int TPR = D / 8;                // threads of one row: K groups, then V groups
  constexpr int RPP = kRowThreads / TPR;    // rows per pass
  constexpr int NW = kRowThreads / 32;
  constexpr int U = 2;                      // passes in flight
  // each warp's max, then min, of a block's channels (pairs); two blocks in turn, so one barrier a block
  __shared__ __align__(16) uint32_t part[2][NW][2][D / 2];
  grid_dependency_wait();
  const int group = blockIdx.y, b = group / a.n_kv_heads;
  int old_len, new_len;
  if (!kv4_range(a, b, &old_len, &new_len)) {
    if (blockIdx.x == 0 && threadIdx.x == 0 && a.err) atomicOr(a.err, kErrAppendRange);
    return;
  }
  const int bs = a.block_size;
  const int first = old_len / bs + static_cast<int>(blockIdx.x) * a.blocks_per_cta;
  if (new_len == old_len || static_cast<long long>(first) * bs >= new_len) return;
  const size_t src0 = static_cast<size_t>(group) * a.row_stride;  // source row of token old_len
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gi = tid % TPR, rr = tid / TPR;
  const bool is_v = gi >= D / 16;
  const int ch = (is_v ? gi - D / 16 : gi) * 16;
  const uint16_t *src = static_cast<const uint16_t *>(is_v ? a.V : a.K) + src0 * D + ch;
  uint8_t *cache = static_cast<uint8_t *>(a.cache) + (static_cast<size_t>(group) * a.max_ctx + old_len) * R::kBytes;
  const int code_at = (is_v ? R::kVC : 0) + ch / 2, scale_at = (is_v ? R::kVS : R::kKS) + ch / 16;
  // rows and blocks as int: max_ctx + block_size fits (the shape checks); rows count from old_len
  for (int i = 0, blk = first; i < a.blocks_per_cta && blk * bs < new_len; ++i, ++blk) {
    const int r0 = max(old_len, blk * bs) - old_len, r1 = min(new_len, blk * bs + bs) - old_len;
    uint32_t hi[8], lo[8];  // of this thread's sixteen channels of K
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      hi[e] = 0xff80ff80u;  // -inf
      lo[e] = 0x7f807f80u;  // +inf
    }
    for (int t0 = r0 + rr; t0 < r1; t0 += U * RPP) {
      uint4 x[U][2];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (t0 + u * RPP < r1) {
          const uint4 *p = reinterpret_cast<const uint4 *>(src + static_cast<size_t>(t0 + u * RPP) * D);
          x[u][0] = p[0];
          x[u][1] = p[1];
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (t0 + u * RPP < r1) {
          int sb;
          const uint2 c = quantise16(x[u][0], x[u][1], &sb);
          uint8_t *rec = cache + static_cast<size_t>(t0 + u * RPP) * R::kBytes;
          *reinterpret_cast<uint2 *>(rec + code_at) = c;
          rec[scale_at] = static_cast<uint8_t>(sb);
          const uint32_t v[8] = {x[u][0].x, x[u][0].y, x[u][0].z, x[u][0].w, x[u][1].x, x[u][1].y, x[u][1].z, x[u][1].w};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            hi[e] = max_bf16x2(hi[e], v[e]);
            lo[e] = min_bf16x2(lo[e], v[e]);
          }
        }
      }
    }
    if (a.meta) {
      __syncwarp();
#pragma unroll
      for (int o = TPR; o < 32; o <<= 1)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          hi[e] = max_bf16x2(hi[e], __shfl_xor_sync(0xffffffffu, hi[e], o));
          lo[e] = min_bf16x2(lo[e], __shfl_xor_sync(0xffffffffu, lo[e], o));
        }
      if (lane < TPR / 2) {  // the lanes of K, of the warp's first row
        uint4 *ph = reinterpret_cast<uint4 *>(&part[i & 1][warp][0][gi * 8]);
        uint4 *pl = reinterpret_cast<uint4 *>(&part[i & 1][warp][1][gi * 8]);
        ph[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        ph[1] = make_uint4(hi[4], hi[5], hi[6], hi[7]);
        pl[0] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        pl[1] = make_uint4(lo[4], lo[5], lo[6], lo[7]);
      }
      __syncthreads();
      if (tid < D) {
        const bool min_row = tid >= D / 2;
        uint32_t *m = static_cast<uint32_t *>(a.meta) + (static_cast<size_t>(group) * a.n_blocks_max + blk) * D + tid;
        const uint32_t *p = &part[i & 1][0][0][tid];
        uint32_t v = blk * bs < old_len ? *m : p[0];  // the block had rows already
#pragma unroll
        for (int w = 0; w < NW; ++w) v = min_row ? min_bf16x2(v, p[w * D]) : max_bf16x2(v, p[w * D]);
        *m = v;
      }
    }
  }
  const uint16_t *K = static_cast<const uint16_t *>(a.K) + src0 * D;
  const int t_begin = max(old_len, first * bs);
  const int t_end = static_cast<int>(min(static_cast<long long>(new_len), (static_cast<long long>(first) + a.blocks_per_cta) * bs));
  if (a.slab) {
    uint16_t *slab = static_cast<uint16_t *>(a.slab) + (static_cast<size_t>(group) * a.max_ctx + t_begin) * a.n_label;
    const int log_r = 31 - __clz(a.n_label);  // a power of two
    const int l = tid & (a.n_label - 1), k = a.label_idx[l];
    const bool ok = k >= 0 && k < D;
    const int rows = kRowThreads >> log_r;
    for (int t0 = t_begin + (tid >> log_r); t0 < t_end; t0 += 4 * rows) {
      uint16_t v[4];  // the loads first: one round trip
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int t = t0 + u * rows;
        v[u] = ok && t < t_end ? K[static_cast<size_t>(t - old_len) * D + k] : static_cast<uint16_t>(0);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (t0 + u * rows < t_end) slab[(static_cast<size_t>(t0 + u * rows - t_begin) << log_r) + l] = v[u];
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kRowThreads) kv4_read_kernel(Kv4RowsArgs a) {
  using R = Kv4Rec<D>;
  constexpr int TPR = D / 4;  // threads of one row: eight channels each, K then V, so that stores are whole lines
  constexpr int RPP = kRowThreads / TPR;
  constexpr int U = kReadRows;
  grid_dependency_wait();
  const int group = blockIdx.y, b = group / a.n_kv_heads;
  int old_len, new_len;
  if (!kv4_range(a, b, &old_len, &new_len)) {
    if (blockIdx.x == 0 && threadIdx.x == 0 && a.err) atomicOr(a.err, kErrAppendRange);
    return;
  }
  const int gi = threadIdx.x % TPR, rr = threadIdx.x / TPR;
  const bool is_v = gi >= D / 8;
  const int ch = (is_v ? gi - D / 8 : gi) * 8;
  uint16_t *dst0 = static_cast<uint16_t *>(const_cast<void *>(is_v ? a.V : a.K));
  if (!dst0) return;
  const uint8_t *cache = static_cast<const uint8_t *>(a.cache) + static_cast<size_t>(group) * a.max_ctx * R::kBytes;
  const int n = new_len - old_len;
  for (int r0 = static_cast<int>(blockIdx.x) * (U * RPP) + rr; r0 < n; r0 += static_cast<int>(gridDim.x) * (U * RPP)) {
    uint32_t c[U], s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * RPP;
      if (r < n) {
        const uint8_t *rec = cache + static_cast<size_t>(old_len + r) * R::kBytes;
        c[u] = *reinterpret_cast<const uint32_t *>(rec + (is_v ? R::kVC : 0) + ch / 2);
        s[u] = rec[(is_v ? R::kVS : R::kKS) + ch / 16];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * RPP;
      if (r < n) {
        uint32_t h[4], o[4];
        e2m1_unpack(c[u], h[0], h[1], h[2], h[3]);
        const uint32_t s2 = s[u] * 0x00800080u;  // the scale twice, as fp16 (b << 7)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t v = hmul2(h[i], s2);
          const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&v));
          o[i] = __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x7632);  // exact
        }
        *reinterpret_cast<uint4 *>(dst0 + (static_cast<size_t>(group) * a.row_stride + r) * D + ch) =
            make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

}  // namespace

cudaError_t launch_kv4_append(Kv4RowsArgs a, cudaStream_t st) {
  // whole blocks of about 64 rows a CTA (32 rows: 512 threads' worth of 16-channel groups)
  a.blocks_per_cta = std::max(1, 64 / a.block_size);
  const long long touched = static_cast<long long>(a.row_stride + a.block_size - 1LL) / a.block_size + 1;
  const long long gx = (touched + a.blocks_per_cta - 1) / a.blocks_per_cta;
  const dim3 grid(static_cast<unsigned>(gx), a.batch * a.n_kv_heads);
  if (a.d == 128) return launch_pdl(kv4_append_kernel<128>, grid, dim3(kRowThreads), 0, st, a);
  return launch_pdl(kv4_append_kernel<64>, grid, dim3(kRowThreads), 0, st, a);
}

cudaError_t launch_kv4_read(const Kv4RowsArgs &a, cudaStream_t st) {
  const int per = kReadRows * kRowThreads / (a.d / 4);
  const long long gx = std::min<long long>((static_cast<long long>(a.row_stride) + per - 1) / per, 65535);
  const dim3 grid(static_cast<unsigned>(gx), a.batch * a.n_kv_heads);
  if (a.d == 128) return launch_pdl(kv4_read_kernel<128>, grid, dim3(kRowThreads), 0, st, a);
  return launch_pdl(kv4_read_kernel<64>, grid, dim3(kRowThreads), 0, st, a);
}

}  // namespace tls
