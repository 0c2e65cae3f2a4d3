// tls_kv4.cu -- rows in and out of the 4-bit KV cache (record: tls_kv4.cuh).
//
// append: a CTA owns the appended rows of a few whole blocks of one group.  A
//   thread quantises sixteen channels of one row (32 bytes in, 8 code bytes
//   and a scale byte out): scale = amax / 6 rounded to e5m3, code = x / scale
//   rounded to e2m1, both to nearest even and decided in fp32.  The quotient
//   is x * (1 / scale) with one residual step, fma(fma(-q, s, x), r, q)
//   (Markstein, "Computation of elementary functions on the IBM RISC
//   System/6000 processor", 1990), so that a tie is a tie.  While the rows
//   are in L1 the CTA also brings the block summary up to date (max / min are
//   associative and the summary holds stored values, so merging the new rows
//   into it gives the bits of a rebuild) and writes the label slab's rows.
// read: a thread widens sixteen channels of one row to bf16 (exact).
// Both are one pass over the rows, bound by HBM.
#include <algorithm>

#include "tls_internal.h"
#include "tls_kv4.cuh"

namespace tls {
namespace {

constexpr int kRowThreads = 256;

// Sixteen bf16 (two 16-byte chunks) -> eight code bytes and a scale byte.
__device__ __forceinline__ uint2 quantise16(const uint4 &u, const uint4 &v, int *scale_byte) {
  const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
  uint32_t m = 0;  // bf16 magnitudes order like their bits
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
  if (m >= 0x7f80u) {
    *scale_byte = kKv4NanScale;
    return make_uint2(0u, 0u);
  }
  const int b = kv4_scale_byte(__uint_as_float(m << 16));
  *scale_byte = b;
  if (b == 0) return make_uint2(0u, 0u);
  const float s = kv4_scale_value(b), r = __frcp_rn(s);
  uint32_t c[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x0 = bf16_lo(w[i]), x1 = bf16_hi(w[i]);
    float q0 = x0 * r, q1 = x1 * r;
    q0 = fmaf(fmaf(-q0, s, x0), r, q0);
    q1 = fmaf(fmaf(-q1, s, x1), r, q1);
    c[i >> 2] |= e2m1_pack(q0, q1) << (8 * (i & 3));
  }
  return make_uint2(c[0], c[1]);
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
  constexpr int U = 2;                      // passes in flight
  __shared__ uint4 part_hi[kRowThreads], part_lo[kRowThreads];
  grid_dependency_wait();
  const int group = blockIdx.y, b = group / a.n_kv_heads;
  int old_len, new_len;
  if (!kv4_range(a, b, &old_len, &new_len)) {
    if (blockIdx.x == 0 && threadIdx.x == 0 && a.err) atomicOr(a.err, kErrAppendRange);
    return;
  }
  const int bs = a.block_size;
  const long long first = static_cast<long long>(old_len / bs) + static_cast<long long>(blockIdx.x) * a.blocks_per_cta;
  if (new_len == old_len || first * bs >= new_len) return;
  const int t_begin = max(old_len, static_cast<int>(first * bs));
  const int t_end = static_cast<int>(min(static_cast<long long>(new_len), (first + a.blocks_per_cta) * bs));
  const size_t src0 = static_cast<size_t>(group) * a.row_stride;  // source row of token old_len
  const int tid = threadIdx.x, gi = tid % TPR, rr = tid / TPR;
  const bool is_v = gi >= D / 16;
  const int ch = (is_v ? gi - D / 16 : gi) * 16;
  const uint16_t *src = static_cast<const uint16_t *>(is_v ? a.V : a.K) + ch;
  uint8_t *cache = static_cast<uint8_t *>(a.cache) + static_cast<size_t>(group) * a.max_ctx * R::kBytes;
  for (int t0 = t_begin + rr; t0 < t_end; t0 += U * RPP) {
    uint4 x[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = t0 + u * RPP;
      if (t < t_end) {
        const uint4 *p = reinterpret_cast<const uint4 *>(src + (src0 + (t - old_len)) * D);
        x[u][0] = p[0];
        x[u][1] = p[1];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = t0 + u * RPP;
      if (t < t_end) {
        int sb;
        const uint2 c = quantise16(x[u][0], x[u][1], &sb);
        uint8_t *rec = cache + static_cast<size_t>(t) * R::kBytes;
        *reinterpret_cast<uint2 *>(rec + (is_v ? R::kVC : 0) + ch / 2) = c;
        rec[(is_v ? R::kVS : R::kKS) + ch / 16] = static_cast<uint8_t>(sb);
      }
    }
  }
  const uint16_t *K = static_cast<const uint16_t *>(a.K) + src0 * D;
  if (a.meta) {
    constexpr int CH = D / 8;                 // 16-byte chunks of a row
    constexpr int P = kRowThreads / CH;       // threads that share a chunk
    const int c = tid % CH, p = tid / CH;
    for (long long blk = first; blk < first + a.blocks_per_cta && blk * bs < new_len; ++blk) {
      const int r0 = max(old_len, static_cast<int>(blk * bs));
      const int r1 = static_cast<int>(min(static_cast<long long>(new_len), (blk + 1) * bs));
      float hi[8], lo[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        hi[e] = -INFINITY;
        lo[e] = INFINITY;
      }
      auto merge = [&](const uint4 &vh, const uint4 &vl) {
        float f[8], g[8];
        chunk_to_f32<BF16>(vh, f);
        chunk_to_f32<BF16>(vl, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          hi[e] = fmaxf(hi[e], f[e]);
          lo[e] = fminf(lo[e], g[e]);
        }
      };
      auto pack = [](const float (&f)[8]) {  // exact: every value came from a bf16
        uint4 v;
        v.x = __byte_perm(__float_as_uint(f[0]), __float_as_uint(f[1]), 0x7632);
        v.y = __byte_perm(__float_as_uint(f[2]), __float_as_uint(f[3]), 0x7632);
        v.z = __byte_perm(__float_as_uint(f[4]), __float_as_uint(f[5]), 0x7632);
        v.w = __byte_perm(__float_as_uint(f[6]), __float_as_uint(f[7]), 0x7632);
        return v;
      };
      for (int t = r0 + p; t < r1; t += P) {
        const uint4 v = *reinterpret_cast<const uint4 *>(K + static_cast<size_t>(t - old_len) * D + c * 8);
        merge(v, v);
      }
      part_hi[tid] = pack(hi);
      part_lo[tid] = pack(lo);
      __syncthreads();
      if (p == 0) {
        for (int i = 1; i < P; ++i) merge(part_hi[i * CH + c], part_lo[i * CH + c]);
        uint4 *m = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.meta) +
                                             (static_cast<size_t>(group) * a.n_blocks_max + blk) * 2 * D) + c;
        if (blk * bs < old_len) merge(m[0], m[CH]);  // the block had rows already
        m[0] = pack(hi);
        m[CH] = pack(lo);
      }
      __syncthreads();
    }
  }
  if (a.slab) {
    uint16_t *slab = static_cast<uint16_t *>(a.slab) + static_cast<size_t>(group) * a.max_ctx * a.n_label;
    const long long n = static_cast<long long>(t_end - t_begin) * a.n_label;
    for (long long i = tid; i < n; i += kRowThreads) {
      const int t = t_begin + static_cast<int>(i / a.n_label), l = static_cast<int>(i % a.n_label);
      const int k = a.label_idx[l];
      slab[static_cast<size_t>(t) * a.n_label + l] =
          (k >= 0 && k < D) ? K[static_cast<size_t>(t - old_len) * D + k] : static_cast<uint16_t>(0);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kRowThreads) kv4_read_kernel(Kv4RowsArgs a) {
  using R = Kv4Rec<D>;
  constexpr int TPR = D / 8;
  constexpr int RPP = kRowThreads / TPR;
  constexpr int U = 4;
  grid_dependency_wait();
  const int group = blockIdx.y, b = group / a.n_kv_heads;
  int old_len, new_len;
  if (!kv4_range(a, b, &old_len, &new_len)) {
    if (blockIdx.x == 0 && threadIdx.x == 0 && a.err) atomicOr(a.err, kErrAppendRange);
    return;
  }
  const int gi = threadIdx.x % TPR, rr = threadIdx.x / TPR;
  const bool is_v = gi >= D / 16;
  const int ch = (is_v ? gi - D / 16 : gi) * 16;
  uint16_t *dst0 = static_cast<uint16_t *>(const_cast<void *>(is_v ? a.V : a.K));
  if (!dst0) return;
  const uint8_t *cache = static_cast<const uint8_t *>(a.cache) + static_cast<size_t>(group) * a.max_ctx * R::kBytes;
  const int n = new_len - old_len;
  for (long long r0 = static_cast<long long>(blockIdx.x) * (U * RPP) + rr; r0 < n;
       r0 += static_cast<long long>(gridDim.x) * (U * RPP)) {
    uint2 c[U];
    uint32_t s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long r = r0 + u * RPP;
      if (r < n) {
        const uint8_t *rec = cache + static_cast<size_t>(old_len + r) * R::kBytes;
        c[u] = *reinterpret_cast<const uint2 *>(rec + (is_v ? R::kVC : 0) + ch / 2);
        s[u] = rec[(is_v ? R::kVS : R::kKS) + ch / 16];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long r = r0 + u * RPP;
      if (r < n) {
        uint32_t h[8], o[8];
        e2m1_unpack(c[u].x, h[0], h[1], h[2], h[3]);
        e2m1_unpack(c[u].y, h[4], h[5], h[6], h[7]);
        const uint32_t s2 = s[u] * 0x00800080u;  // the scale twice, as fp16 (b << 7)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t v = hmul2(h[i], s2);
          const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&v));
          o[i] = __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x7632);  // exact
        }
        uint4 *d = reinterpret_cast<uint4 *>(dst0 + (static_cast<size_t>(group) * a.row_stride + r) * D + ch);
        d[0] = make_uint4(o[0], o[1], o[2], o[3]);
        d[1] = make_uint4(o[4], o[5], o[6], o[7]);
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
  const int per = 4 * kRowThreads / (a.d / 8);
  const long long gx = std::min<long long>((static_cast<long long>(a.row_stride) + per - 1) / per, 65535);
  const dim3 grid(static_cast<unsigned>(gx), a.batch * a.n_kv_heads);
  if (a.d == 128) return launch_pdl(kv4_read_kernel<128>, grid, dim3(kRowThreads), 0, st, a);
  return launch_pdl(kv4_read_kernel<64>, grid, dim3(kRowThreads), 0, st, a);
}

}  // namespace tls
