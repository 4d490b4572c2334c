// paged_attention.cu - attention of one token per sequence over a paged cache
// (svdq_attention_decode).
//
//   out = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale q . k_j - m),   m = a running maximum
//
// Every key and value is read once: 4 bytes per cached element pair, 4 flops per byte and
// head of a group, so HBM bounds it. The work is cut without regard to heads and
// sequences: the keys of all (sequence, key head) segments, in units of 16, form one
// line that is dealt evenly to two blocks per SM, so that ragged batches and single long
// sequences both fill the GPU. Up to eight segments of a sequence share the line, each with a
// block of its own per range: blocks that run side by side then read rows of the same
// tokens, which lie side by side. Inside a block four warps take a piece's units in turn,
// each with its own ring of asynchronous copies and its own running softmax, without any
// barrier until the piece ends.
//
// Both products run on the warp tensor instructions with the keys as rows: S^T = K Q^T
// (16 keys x 8 heads) and O^T = V^T P^T (16 elements x 8 heads), so that a group of up
// to 8 query heads fills the eight columns of m16n8k16; with the queries as rows, half
// of the 16 rows would be padding for such a group. P^T passes from the accumulator layout
// of the first product to the operand layout of the second by a transposing register move.
//
// A segment that one block finishes is written at once. Pieces of a segment cut by a
// block boundary go to the workspace (sums in fp32, maximum, total) and a second kernel,
// launched as a dependent of the first, joins them in the order of the blocks: the
// result depends on the lengths alone.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace svdq {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kUnit = 16;          // keys per unit of work
constexpr int kBlocksPerSm = 2;
constexpr int kRow = 8;            // heads per column tile of the products
constexpr int kMaxRanges = 512;    // of the line: at most kBlocksPerSm per SM

struct PagedArgs {
  svdq_heads q, out;
  svdq_kv_cache cache;
  const int32_t* page_table;
  int64_t table_ld;
  const int32_t* kv_len;
  int batch;
  int group;        // query heads per key head
  int row_groups;   // segments per (sequence, key head): ceil(group / (8 * kNt))
  float scale_log2; // scale * log2(e)
  float* scratch;
  unsigned* status;
  int abreast;      // segments of a sequence that share the line: 8, 4, 2 or 1
  int grid;         // ranges of the line at most: blocks of the first kernel / abreast
};

// Floats of one partial result: sums [rows][kDim], then maxima and totals [rows].
template <int kDim, int kNt>
__host__ __device__ constexpr int partial_floats() {
  return kRow * kNt * (kDim + 2);
}

__device__ __forceinline__ int clamped_len(const PagedArgs& a, int s) {
  const int64_t most = min(a.table_ld * a.cache.page_size, static_cast<int64_t>(0x7FFFFFFF - kUnit));
  return static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(a.kv_len[s]), most)));
}

__device__ __forceinline__ int units_of(int len) { return (len + kUnit - 1) / kUnit; }

__device__ __forceinline__ void ldmatrix_x4(uint32_t saddr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(saddr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t saddr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(saddr)
               : "memory");
}
// Transpose of an 8x8 tile of 16-bit elements held one row per four lanes.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// exp2 of a difference to a maximum; a score of -inf counts nothing, even while the
// maximum is -inf itself (no key yet).
__device__ __forceinline__ float exp2_from(float x, float top) { return x == -INFINITY ? 0.0f : exp2f(x - top); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Ranges that share `total` units: none has less than a unit for each warp unless
// there is no more than that altogether. 0 without any unit.
__device__ __forceinline__ int blocks_for(long long total, int grid) {
  return static_cast<int>(min(static_cast<long long>(grid), (total + kWarps - 1) / kWarps));
}

// Sum of v over the block, to all threads. Two calls need a barrier between them.
__device__ __forceinline__ long long block_sum(long long v, long long* sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  long long t = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) t += sh[w];
  return t;
}

template <int kDim, int kNt, int kStages>
struct PagedShared {
  static constexpr int kTile = kUnit * kDim * 2;                       // bytes of 16 keys
  static constexpr int kRing = kWarps * kStages * 2 * kTile;
  static constexpr int kMerge = kWarps * kRow * kNt * (kDim + 4) * 4;  // reuses the ring
  static constexpr int kBytes = (kRing > kMerge ? kRing : kMerge);
};

template <int kDim, int kNt, int kStages>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) paged_split_kernel(const PagedArgs a) {
  using Sh = PagedShared<kDim, kNt, kStages>;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ long long sh_sum[kWarps];
  __shared__ long long sh_base;
  __shared__ int sh_seq;
  __shared__ float sh_m[kWarps][kRow * kNt], sh_l[kWarps][kRow * kNt];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_trigger();

  // this block's range [lo, hi) of the line of units, and the sequence it begins in
  const int segs = a.cache.heads * a.row_groups / a.abreast;   // of the line, per sequence
  const int range = blockIdx.x / a.abreast, beside = blockIdx.x - range * a.abreast;
  long long mine = 0;
  for (int s = tid; s < a.batch; s += kThreads) {
    const int len = clamped_len(a, s);
    if (blockIdx.x == 0 && len != a.kv_len[s]) record_status(a.status, kStatusEinval);
    mine += units_of(len);
  }
  const long long total = block_sum(mine, sh_sum) * segs;
  const int blocks = blocks_for(total, a.grid);
  if (range >= blocks) return;
  const long long lo = total * range / blocks, hi = total * (range + 1) / blocks;
  long long before = 0;
  for (int s0 = 0; s0 < a.batch; s0 += kThreads) {
    __syncthreads();
    const int s = s0 + tid;
    const long long n = s < a.batch ? units_of(clamped_len(a, s)) : 0;
    long long incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    if (lane == 31) sh_sum[warp] = incl;
    __syncthreads();
    long long chunk = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) incl += sh_sum[w];
      chunk += sh_sum[w];
    }
    const long long first = (before + incl - n) * segs, end = (before + incl) * segs;
    if (first <= lo && lo < end) {
      sh_seq = s;
      sh_base = first;
    }
    before += chunk;
    if (before * segs > lo) break;   // the same for all threads
  }
  __syncthreads();
  int seq = sh_seq;
  long long base = sh_base;

  unsigned char* ring = smem + warp * kStages * 2 * Sh::kTile;
  const uint32_t ring_u = smem_u32(ring);
  const int dim = a.cache.head_dim;
  const __nv_bfloat16* kc = static_cast<const __nv_bfloat16*>(a.cache.k);
  const __nv_bfloat16* vc = static_cast<const __nv_bfloat16*>(a.cache.v);

  long long cur = lo;
  while (cur < hi) {
    const int len = clamped_len(a, seq);
    const int nu = units_of(len);
    if (cur >= base + static_cast<long long>(nu) * segs) {   // past this sequence (or it is empty)
      base += static_cast<long long>(nu) * segs;
      ++seq;
      continue;
    }
    const int in_line = static_cast<int>((cur - base) / nu);
    const int u0 = static_cast<int>((cur - base) - static_cast<long long>(in_line) * nu);
    const int seg = in_line * a.abreast + beside;
    const int u1 = static_cast<int>(min(static_cast<long long>(nu), u0 + (hi - cur)));
    const int kvh = seg / a.row_groups, h0 = (seg - kvh * a.row_groups) * kRow * kNt;   // first head of the group
    const int32_t* table = a.page_table + seq * a.table_ld;

    // unit u of this warp: u0 + warp + 4 i
    const int count = (u1 - u0 - warp + kWarps - 1) / kWarps;
    auto unit_at = [&](int i) { return u0 + warp + kWarps * i; };
    auto lookup = [&](int i) {   // the page of key (lane % 16) of unit i
      const int key = unit_at(i) * kUnit + (lane & 15);
      return (i < count && key < len) ? table[key / a.cache.page_size] : -1;
    };
    auto issue = [&](int i, int page) {
      const int key = unit_at(i) * kUnit + (lane & 15);
      long long off = -1;
      if (key < len) {
        if (page >= 0 && page < a.cache.pages)
          off = page * a.cache.page_ld + static_cast<long long>(key % a.cache.page_size) * a.cache.slot_ld +
                kvh * a.cache.head_ld;
        else
          record_status(a.status, kStatusEinval);
      }
      unsigned char* kt = ring + (i % kStages) * 2 * Sh::kTile;
      unsigned char* vt = kt + Sh::kTile;
#pragma unroll
      for (int rr = 0; rr < kUnit / 4; ++rr) {
        const int row = rr * 4 + (lane >> 3);
        const long long o = __shfl_sync(0xffffffffu, off, row);
#pragma unroll
        for (int cc = 0; cc < kDim / 64; ++cc) {
          const int c = cc * 8 + (lane & 7);
          const bool on = o >= 0 && c * 8 < dim;
          const int at = row * kDim * 2 + ((c ^ (row & 7)) << 4);
          const long long src = on ? o + c * 8 : 0;
          cp_async16(kt + at, kc + src, on ? 16 : 0);
          cp_async16(vt + at, vc + src, on ? 16 : 0);
        }
      }
      return off >= 0;
    };

    // the group's queries as the column operand of S^T = K Q^T
    uint32_t qf[kNt][kDim / 16][2];
#pragma unroll
    for (int n = 0; n < kNt; ++n) {
      const int h = h0 + n * kRow + (lane >> 2);
      const bool on = h < a.group;
      const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(a.q.data) + seq * a.q.token_ld +
                                (static_cast<long long>(kvh) * a.group + (on ? h : 0)) * a.q.head_ld;
#pragma unroll
      for (int kk = 0; kk < kDim / 16; ++kk)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int e = kk * 16 + b * 8 + 2 * (lane & 3);
          qf[n][kk][b] = on && e < dim ? *reinterpret_cast<const uint32_t*>(qp + e) : 0u;
        }
    }

    float o[kNt][kDim / 16][4];
    float m[kNt][2], l[kNt][2];
#pragma unroll
    for (int n = 0; n < kNt; ++n) {
#pragma unroll
      for (int i = 0; i < kDim / 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[n][i][j] = 0.0f;
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.0f;
    }

    // bit i of `good`: which keys of the unit in stage i take part (by lane % 16)
    unsigned good[kStages];
    int page = lookup(0);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      const int next = lookup(i + 1);
      good[i] = 0;
      if (i < count) good[i] = __ballot_sync(0xffffffffu, issue(i, page)) & 0xFFFFu;
      cp_async_commit();
      page = next;
    }
    good[kStages - 1] = 0;

    for (int i = 0; i < count; ++i) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      {
        const int j = i + kStages - 1;   // into the stage that the last turn has read
        const int next = lookup(j + 1);
        unsigned g = 0;
        if (j < count) g = __ballot_sync(0xffffffffu, issue(j, page)) & 0xFFFFu;
        cp_async_commit();
        page = next;
        good[kStages - 1] = g;
      }
      const uint32_t kt = ring_u + (i % kStages) * 2 * Sh::kTile, vt = kt + Sh::kTile;

      float s[kNt][4];
#pragma unroll
      for (int n = 0; n < kNt; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
      {
        const int row = (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
        for (int kk = 0; kk < kDim / 16; ++kk) {
          uint32_t kf[4];
          const int c = 2 * kk + (lane >> 4);
          ldmatrix_x4(kt + row * kDim * 2 + ((c ^ (row & 7)) << 4), kf);
#pragma unroll
          for (int n = 0; n < kNt; ++n) mma_bf16_16816(s[n], kf, qf[n][kk]);
        }
      }
      // keys lane / 4 and lane / 4 + 8; columns (heads) 2 (lane % 4) and the next
      const bool on0 = (good[0] >> (lane >> 2)) & 1, on1 = (good[0] >> ((lane >> 2) + 8)) & 1;
      bool grow = false;
#pragma unroll
      for (int n = 0; n < kNt; ++n)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          s[n][j] = on0 ? s[n][j] * a.scale_log2 : -INFINITY;
          s[n][2 + j] = on1 ? s[n][2 + j] * a.scale_log2 : -INFINITY;
          // The maximum is renewed only when a score passes it by 2^8: the terms
          // then stay below 2^8, far inside the range of bf16 and fp32.
          grow |= fmaxf(s[n][j], s[n][2 + j]) > (m[n][j] == -INFINITY ? -INFINITY : m[n][j] + 8.0f);
        }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int n = 0; n < kNt; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float top = fmaxf(s[n][j], s[n][2 + j]);
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            top = fmaxf(top, m[n][j]);
            const float f = exp2_from(m[n][j], top);
            m[n][j] = top;
            l[n][j] *= f;
#pragma unroll
            for (int i2 = 0; i2 < kDim / 16; ++i2) {
              o[n][i2][j] *= f;
              o[n][i2][2 + j] *= f;
            }
          }
      }
      uint32_t pf[kNt][2];
#pragma unroll
      for (int n = 0; n < kNt; ++n) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          s[n][j] = exp2_from(s[n][j], m[n][j]);
          s[n][2 + j] = exp2_from(s[n][2 + j], m[n][j]);
          l[n][j] += s[n][j] + s[n][2 + j];
        }
        pf[n][0] = transpose8x8(pack_bf16(s[n][0], s[n][1]));
        pf[n][1] = transpose8x8(pack_bf16(s[n][2], s[n][3]));
      }
      {
        const int row = (lane & 7) + (lane >> 4) * 8;
#pragma unroll
        for (int mt = 0; mt < kDim / 16; ++mt) {
          uint32_t vf[4];
          const int c = 2 * mt + ((lane >> 3) & 1);
          ldmatrix_x4_trans(vt + row * kDim * 2 + ((c ^ (row & 7)) << 4), vf);
#pragma unroll
          for (int n = 0; n < kNt; ++n) mma_bf16_16816(o[n][mt], vf, pf[n]);
        }
      }
#pragma unroll
      for (int j = 0; j + 1 < kStages; ++j) good[j] = good[j + 1];
      __syncwarp();
    }
    cp_async_wait<0>();

    // join the four warps
    __syncthreads();
    float* osh = reinterpret_cast<float*>(smem) + warp * kRow * kNt * (kDim + 4);
#pragma unroll
    for (int n = 0; n < kNt; ++n)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = n * kRow + 2 * (lane & 3) + j;
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], x);
        if (lane < 4) sh_m[warp][r] = m[n][j], sh_l[warp][r] = l[n][j];
#pragma unroll
        for (int mt = 0; mt < kDim / 16; ++mt) {
          osh[r * (kDim + 4) + mt * 16 + (lane >> 2)] = o[n][mt][j];
          osh[r * (kDim + 4) + mt * 16 + 8 + (lane >> 2)] = o[n][mt][2 + j];
        }
      }
    __syncthreads();
    const bool whole = u0 == 0 && u1 == nu;
    float* part = a.scratch + (static_cast<long long>(blockIdx.x) * 2 + (cur == lo ? 0 : 1)) * partial_floats<kDim, kNt>();
    for (int idx = tid; idx < kRow * kNt * kDim; idx += kThreads) {
      const int r = idx / kDim, d = idx - r * kDim;
      if (h0 + r >= a.group || d >= dim) continue;
      float top = sh_m[0][r];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) top = fmaxf(top, sh_m[w][r]);
      float sum = 0.0f, tot = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = exp2_from(sh_m[w][r], top);
        sum = fmaf(f, reinterpret_cast<const float*>(smem)[w * kRow * kNt * (kDim + 4) + r * (kDim + 4) + d], sum);
        tot = fmaf(f, sh_l[w][r], tot);
      }
      if (whole) {
        static_cast<__nv_bfloat16*>(a.out.data)[seq * a.out.token_ld +
                                                (static_cast<long long>(kvh) * a.group + h0 + r) * a.out.head_ld + d] =
            __float2bfloat16(tot == 0.0f ? 0.0f : sum / tot);
      } else {
        part[r * kDim + d] = sum;
        if (d == 0) {
          part[kRow * kNt * kDim + r] = top;
          part[kRow * kNt * (kDim + 1) + r] = tot;
        }
      }
    }
    __syncthreads();   // the ring and the statistics are free again
    cur += u1 - u0;
  }
}

// Joins the pieces of one segment's row: grid (batch * segments, rows of a segment).
template <int kDim, int kNt>
__global__ void __launch_bounds__(kThreads) paged_join_kernel(const PagedArgs a) {
  constexpr int kShares = kThreads / kDim;   // threads per element: each takes every kShares-th piece
  __shared__ long long sh[2][kWarps];
  __shared__ float sh_red[kWarps];
  __shared__ float sh_weight[kMaxRanges];
  __shared__ float sh_sum[kShares][kDim];
  const int tid = threadIdx.x;
  const int per_seq = a.cache.heads * a.row_groups, segs = per_seq / a.abreast;
  const int seq = blockIdx.x / per_seq, seg = blockIdx.x - seq * per_seq;
  const int kvh = seg / a.row_groups, h = (seg - kvh * a.row_groups) * kRow * kNt + blockIdx.y;
  long long mine = 0, all = 0;
  for (int s = threadIdx.x; s < a.batch; s += kThreads) {
    const int n = units_of(clamped_len(a, s));
    all += n;
    if (s < seq) mine += n;
  }
  const long long total = block_sum(all, sh[0]) * segs;
  const long long nu = units_of(clamped_len(a, seq));
  const long long first = block_sum(mine, sh[1]) * segs + seg / a.abreast * nu;
  pdl_wait();
  if (h >= a.group) return;
  const int d = tid % kDim, share = tid / kDim;
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out.data) + seq * a.out.token_ld +
                       (static_cast<long long>(kvh) * a.group + h) * a.out.head_ld + d;
  const bool writes = share == 0 && d < a.cache.head_dim;
  if (nu == 0) {
    if (writes) *dst = __float2bfloat16(0.0f);
    return;
  }
  // range b holds units [total b / blocks, total (b + 1) / blocks)
  const int blocks = blocks_for(total, a.grid);
  const long long b0 = ((first + 1) * blocks - 1) / total, b1 = ((first + nu) * blocks - 1) / total;
  if (b0 == b1) return;   // written by that block
  const int pieces = static_cast<int>(b1 - b0) + 1;
  // the first block's piece is its last one, unless its range begins there
  const int slot0 = total * b0 / blocks != first ? 1 : 0;
  auto piece = [&](int i) {
    return a.scratch +
           (((b0 + i) * a.abreast + seg % a.abreast) * 2 + (i == 0 ? slot0 : 0)) * partial_floats<kDim, kNt>();
  };
  // all maxima and totals at once, then the weighted sums in independent loads
  float top = -INFINITY;
  for (int i = tid; i < pieces; i += kThreads) {
    sh_weight[i] = piece(i)[kRow * kNt * kDim + blockIdx.y];
    top = fmaxf(top, sh_weight[i]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((tid & 31) == 0) sh_red[tid >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sh_red[w]);
  __syncthreads();
  float tot = 0.0f;
  for (int i = tid; i < pieces; i += kThreads) {
    const float f = exp2_from(sh_weight[i], top);
    sh_weight[i] = f;
    tot = fmaf(f, piece(i)[kRow * kNt * (kDim + 1) + blockIdx.y], tot);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
  if ((tid & 31) == 0) sh_red[tid >> 5] = tot;
  __syncthreads();
  tot = 0.0f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) tot += sh_red[w];
  float sum = 0.0f;
#pragma unroll 8
  for (int i = share; i < pieces; i += kShares) sum = fmaf(sh_weight[i], d < a.cache.head_dim ? piece(i)[blockIdx.y * kDim + d] : 0.0f, sum);
  sh_sum[share][d] = sum;
  __syncthreads();
  if (!writes) return;
  sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kShares; ++i) sum += sh_sum[i][d];
  *dst = __float2bfloat16(tot == 0.0f ? 0.0f : sum / tot);
}

template <int kDim, int kNt, int kStages>
cudaError_t launch_one(PagedArgs a, cudaStream_t st) {
  constexpr int smem = PagedShared<kDim, kNt, kStages>::kBytes;
  a.row_groups = (a.group + kRow * kNt - 1) / (kRow * kNt);
  const int per_seq = a.cache.heads * a.row_groups;
  a.abreast = per_seq % 8 == 0 ? 8 : (per_seq % 4 == 0 ? 4 : (per_seq % 2 == 0 ? 2 : 1));
  a.grid = std::min(kBlocksPerSm * num_sms() / a.abreast, kMaxRanges);
  cudaError_t e = cudaFuncSetAttribute(paged_split_kernel<kDim, kNt, kStages>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  paged_split_kernel<kDim, kNt, kStages><<<a.grid * a.abreast, kThreads, smem, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(a.batch) * a.cache.heads * a.row_groups,
                     static_cast<unsigned>(std::min(a.group, kRow * kNt)));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_join_kernel<kDim, kNt>, a);
}

}  // namespace

size_t paged_scratch_bytes(int heads, int kv_heads, int head_dim) {
  const size_t one = heads / kv_heads <= kRow ? (head_dim <= 64 ? partial_floats<64, 1>() : partial_floats<128, 1>())
                                              : (head_dim <= 64 ? partial_floats<64, 2>() : partial_floats<128, 2>());
  return static_cast<size_t>(kBlocksPerSm) * num_sms() * 2 * one * sizeof(float);
}

cudaError_t launch_paged(const svdq_heads& q, const svdq_kv_cache& cache, const int32_t* page_table,
                         int64_t table_ld, const int32_t* kv_len, int batch, float scale, const svdq_heads& out,
                         void* scratch, cudaStream_t stream) {
  PagedArgs a{};
  a.q = q, a.out = out, a.cache = cache;
  a.page_table = page_table, a.table_ld = table_ld, a.kv_len = kv_len;
  a.batch = batch;
  a.group = q.heads / cache.heads;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.scratch = static_cast<float*>(scratch);
  a.status = device_status_word();
  // Up to 8 query heads per key head fill one column tile; more take two, which
  // halves the reads of the cache.
  if (cache.head_dim <= 64) return a.group <= kRow ? launch_one<64, 1, 6>(a, stream) : launch_one<64, 2, 6>(a, stream);
  return a.group <= kRow ? launch_one<128, 1, 3>(a, stream) : launch_one<128, 2, 3>(a, stream);
}

}  // namespace svdq
