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
// P is rounded to bf16 there, because the product takes two operands of one 16-bit type and V is
// bf16: at most 2^-8 of sum p |v| / sum p, as much as the rounding of the result. The sums of the
// weights take the unrounded fp32 values.
//
// A segment that one block finishes is written at once. Pieces of a segment cut by a
// block boundary go to the workspace (sums in fp32, maximum, total), with a note of the first
// and the last range of the segment, and a second kernel, launched as a dependent of the
// first, joins them in the order of the ranges: the result depends on the lengths alone.
//
// One sequence alone costs latency: lengths, pages, keys and the join wait for one another.
// So both kernels keep to 32-bit arithmetic and few barriers (64-bit divisions and a loop
// over pieces whose loads waited for one another took 14 of 24 us).
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
  float* scratch;   // partial results: [range][segment beside][2]
  int2* ends;       // [sequence][segment]: twice the first range with a piece of it, plus that
                    // piece's slot, and twice the last
  int page_shift;   // log2(page_size), or -1
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

// Ranges that share `total` units: none has less than a unit for each warp unless there is
// no more than that altogether. 0 without any unit.
__device__ __forceinline__ int ranges_for(unsigned total, int grid) {
  return static_cast<int>(min(static_cast<unsigned>(grid), (total + kWarps - 1) / kWarps));
}

// Inclusive scan over the block. Two calls need a barrier between them.
__device__ __forceinline__ unsigned block_scan(unsigned v, unsigned* sh, unsigned* sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned up = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += up;
  }
  if (lane == 31) sh[warp] = v;
  __syncthreads();
  *sum = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) v += sh[w];
    *sum += sh[w];
  }
  return v;
}

template <int kDim, int kNt, int kStages>
struct PagedShared {
  static constexpr int kTile = kUnit * kDim * 2;                       // bytes of 16 keys
  static constexpr int kRing = kWarps * kStages * 2 * kTile;
  static constexpr int kMerge = kWarps * kRow * kNt * (kDim + 4) * 4;  // reuses the ring
  static constexpr int kBytes = (kRing > kMerge ? kRing : kMerge);
};

template <int kDim, int kNt, int kStages>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) paged_split_kernel(const __grid_constant__ PagedArgs a) {
  using Sh = PagedShared<kDim, kNt, kStages>;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ unsigned sh_scan[2][kWarps];
  __shared__ unsigned sh_base;
  __shared__ int sh_seq;
  __shared__ float sh_m[kWarps][kRow * kNt], sh_l[kWarps][kRow * kNt];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_trigger();

  // this block's range [lo, hi) of the line of units, and the sequence it begins in; all
  // units together are below 2^31
  const unsigned segs = a.cache.heads * a.row_groups / a.abreast;   // of the line, per sequence
  const int range = blockIdx.x / a.abreast, beside = blockIdx.x - range * a.abreast;
  unsigned total = 0, upto = 0, here = 0;   // in sequences' units: all, those before thread's next, its own
  for (int s0 = 0; s0 < a.batch; s0 += kThreads) {
    const int s = s0 + tid;
    here = 0;
    if (s < a.batch) {
      const int len = clamped_len(a, s);
      if (blockIdx.x == 0 && len != a.kv_len[s]) record_status(a.status, kStatusEinval);
      here = units_of(len);
    }
    unsigned sum;
    if (s0 > 0) __syncthreads();
    upto = total + block_scan(here, sh_scan[0], &sum);
    total += sum;
  }
  total *= segs;
  const int ranges = ranges_for(total, a.grid);
  if (range >= ranges) return;
  // the first total % ranges of them are one unit longer
  const unsigned share = total / ranges, longer = total - share * ranges;
  const unsigned lo = share * range + min(static_cast<unsigned>(range), longer);
  const unsigned hi = lo + share + (range < longer ? 1 : 0);
  if (a.batch <= kThreads) {
    if ((upto - here) * segs <= lo && lo < upto * segs) sh_seq = tid, sh_base = (upto - here) * segs;
  } else {
    unsigned before = 0;
    for (int s0 = 0; s0 < a.batch; s0 += kThreads) {
      const int s = s0 + tid;
      here = s < a.batch ? units_of(clamped_len(a, s)) : 0;
      unsigned sum;
      __syncthreads();
      upto = before + block_scan(here, sh_scan[1], &sum);
      if ((upto - here) * segs <= lo && lo < upto * segs) sh_seq = s, sh_base = (upto - here) * segs;
      before += sum;
      if (before * segs > lo) break;   // the same for all threads
    }
  }
  __syncthreads();
  int seq = sh_seq;
  unsigned base = sh_base;

  unsigned char* ring = smem + warp * kStages * 2 * Sh::kTile;
  const uint32_t ring_u = smem_u32(ring);
  const int dim = a.cache.head_dim;
  const __nv_bfloat16* kc = static_cast<const __nv_bfloat16*>(a.cache.k);
  const __nv_bfloat16* vc = static_cast<const __nv_bfloat16*>(a.cache.v);

  unsigned cur = lo;
  while (cur < hi) {
    const int len = clamped_len(a, seq);
    const unsigned nu = units_of(len);
    if (cur >= base + nu * segs) {   // past this sequence (or it is empty)
      base += nu * segs;
      ++seq;
      continue;
    }
    const unsigned in_line = (cur - base) / nu;
    const int u0 = static_cast<int>(cur - base - in_line * nu);
    const int u1 = static_cast<int>(min(nu, u0 + (hi - cur)));
    const int seg = static_cast<int>(in_line) * a.abreast + beside;
    const int kvh = seg / a.row_groups, h0 = (seg - kvh * a.row_groups) * kRow * kNt;   // first head of the group
    const int32_t* table = a.page_table + seq * a.table_ld;

    // unit u of this warp: u0 + warp + 4 i
    const int count = (u1 - u0 - warp + kWarps - 1) / kWarps;
    auto unit_at = [&](int i) { return u0 + warp + kWarps * i; };
    auto page_of = [&](int key) { return a.page_shift >= 0 ? key >> a.page_shift : key / a.cache.page_size; };
    auto lookup = [&](int i) {   // the page of key (lane % 16) of unit i
      const int key = unit_at(i) * kUnit + (lane & 15);
      return (i < count && key < len) ? table[page_of(key)] : -1;
    };
    auto issue = [&](int i, int page) {
      const int key = unit_at(i) * kUnit + (lane & 15);
      long long off = -1;
      if (key < len) {
        if (page >= 0 && page < a.cache.pages)
          off = page * a.cache.page_ld + static_cast<long long>(key - page_of(key) * a.cache.page_size) * a.cache.slot_ld +
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
    const bool whole = u0 == 0 && u1 == static_cast<int>(nu);
    float* part = a.scratch + ((static_cast<long long>(range) * a.abreast + beside) * 2 + (cur == lo ? 0 : 1)) *
                                  partial_floats<kDim, kNt>();
    if (tid == 0) {
      int2* ends = a.ends + static_cast<long long>(seq) * a.cache.heads * a.row_groups + seg;
      if (u0 == 0) ends->x = 2 * range + (cur == lo ? 0 : 1);
      if (u1 == static_cast<int>(nu)) ends->y = 2 * range;
    }
    if (tid < kRow * kNt) {   // the warps' weights, and with them the total
      float top = sh_m[0][tid];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) top = fmaxf(top, sh_m[w][tid]);
      float tot = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = exp2_from(sh_m[w][tid], top);
        tot = fmaf(f, sh_l[w][tid], tot);
        sh_m[w][tid] = f;
      }
      sh_l[0][tid] = tot;
      if (!whole) {
        part[kRow * kNt * kDim + tid] = top;
        part[kRow * kNt * (kDim + 1) + tid] = tot;
      }
    }
    __syncthreads();
    for (int idx = tid; idx < kRow * kNt * kDim; idx += kThreads) {
      const int r = idx / kDim, d = idx - r * kDim;
      if (h0 + r >= a.group || d >= dim) continue;
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        sum = fmaf(sh_m[w][r], reinterpret_cast<const float*>(smem)[w * kRow * kNt * (kDim + 4) + r * (kDim + 4) + d], sum);
      if (whole) {
        const float tot = sh_l[0][r];
        static_cast<__nv_bfloat16*>(a.out.data)[seq * a.out.token_ld +
                                                (static_cast<long long>(kvh) * a.group + h0 + r) * a.out.head_ld + d] =
            __float2bfloat16(tot == 0.0f ? 0.0f : sum / tot);
      } else {
        part[r * kDim + d] = sum;
      }
    }
    __syncthreads();   // the ring and the statistics are free again
    cur += u1 - u0;
  }
}

// Joins the pieces of one segment's row: grid (batch * segments, rows of a segment).
constexpr int kJoinThreads = 256;
template <int kDim, int kNt>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const __grid_constant__ PagedArgs a) {
  constexpr int kShares = kJoinThreads / kDim;   // threads per element: each takes every kShares-th piece
  __shared__ float sh_red[2][kJoinThreads / 32];
  __shared__ float sh_weight[kMaxRanges];
  __shared__ float sh_sum[kShares][kDim];
  const int tid = threadIdx.x;
  const int per_seq = a.cache.heads * a.row_groups;
  const int seq = blockIdx.x / per_seq, seg = blockIdx.x - seq * per_seq;
  const int kvh = seg / a.row_groups, h = (seg - kvh * a.row_groups) * kRow * kNt + blockIdx.y;
  const int d = tid % kDim, share = tid / kDim;
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out.data) + seq * a.out.token_ld +
                       (static_cast<long long>(kvh) * a.group + h) * a.out.head_ld + d;
  const bool writes = share == 0 && d < a.cache.head_dim && h < a.group;
  const bool empty = clamped_len(a, seq) == 0;
  pdl_wait();
  if (empty && writes) *dst = __float2bfloat16(0.0f);
  if (empty || h >= a.group) return;
  const int2 ends = a.ends[blockIdx.x];
  const int first = ends.x >> 1, slot0 = ends.x & 1, pieces = (ends.y >> 1) - first + 1;
  if (pieces == 1) return;   // written by the block of that range
  // all pieces but the first begin their range, and are in slot 0
  const float* mine =
      a.scratch + static_cast<long long>(first * a.abreast + seg % a.abreast) * 2 * partial_floats<kDim, kNt>();
  const int step = 2 * a.abreast * partial_floats<kDim, kNt>();
  auto piece = [&](int i) {
    return mine + static_cast<long long>(i) * step + (i == 0 ? slot0 * partial_floats<kDim, kNt>() : 0);
  };
  // all maxima and totals at once, then the weighted sums in independent loads
  constexpr int kMine = (kMaxRanges + kJoinThreads - 1) / kJoinThreads;
  float top = -INFINITY, tot = 0.0f, m[kMine], l[kMine];
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    const int i = tid + j * kJoinThreads;
    m[j] = -INFINITY, l[j] = 0.0f;
    if (i < pieces) {
      m[j] = piece(i)[kRow * kNt * kDim + blockIdx.y];
      l[j] = piece(i)[kRow * kNt * (kDim + 1) + blockIdx.y];
    }
    top = fmaxf(top, m[j]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((tid & 31) == 0) sh_red[0][tid >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) top = fmaxf(top, sh_red[0][w]);
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    const int i = tid + j * kJoinThreads;
    const float f = exp2_from(m[j], top);
    if (i < pieces) sh_weight[i] = f;
    tot = fmaf(f, l[j], tot);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
  if ((tid & 31) == 0) sh_red[1][tid >> 5] = tot;
  __syncthreads();
  tot = 0.0f;
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) tot += sh_red[1][w];
  float sum = 0.0f;
  if (d < a.cache.head_dim) {
#pragma unroll 10
    for (int i = share; i < pieces; i += kShares) sum = fmaf(sh_weight[i], piece(i)[blockIdx.y * kDim + d], sum);
  }
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
  a.ends = reinterpret_cast<int2*>(a.scratch + static_cast<size_t>(a.grid) * a.abreast * 2 * partial_floats<kDim, kNt>());
  cudaError_t e = cudaFuncSetAttribute(paged_split_kernel<kDim, kNt, kStages>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  e = launch_behind(paged_split_kernel<kDim, kNt, kStages>, dim3(a.grid * a.abreast), kThreads, smem, st, a);
  if (e != cudaSuccess) return e;
  const dim3 rows(static_cast<unsigned>(a.batch) * a.cache.heads * a.row_groups,
                  static_cast<unsigned>(std::min(a.group, kRow * kNt)));
  return launch_behind(paged_join_kernel<kDim, kNt>, rows, kJoinThreads, 0, st, a);
}

}  // namespace

namespace {

int row_groups_of(int heads, int kv_heads) {
  const int group = heads / kv_heads, rows = group <= kRow ? kRow : 2 * kRow;
  return (group + rows - 1) / rows;
}

}  // namespace

size_t paged_scratch_bytes(int batch, int heads, int kv_heads, int head_dim) {
  const size_t one = heads / kv_heads <= kRow ? (head_dim <= 64 ? partial_floats<64, 1>() : partial_floats<128, 1>())
                                              : (head_dim <= 64 ? partial_floats<64, 2>() : partial_floats<128, 2>());
  return static_cast<size_t>(kBlocksPerSm) * num_sms() * 2 * one * sizeof(float) +
         static_cast<size_t>(batch) * kv_heads * row_groups_of(heads, kv_heads) * sizeof(int2);
}

bool paged_fits(int batch, int heads, int kv_heads, int64_t most_keys) {
  const double units = static_cast<double>(batch) * kv_heads * row_groups_of(heads, kv_heads) *
                       (static_cast<double>(most_keys) / kUnit + 1);
  return units < 2147483648.0;
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
  a.page_shift = (cache.page_size & (cache.page_size - 1)) == 0 ? __builtin_ctz(cache.page_size) : -1;
  // Up to 8 query heads per key head fill one column tile; more take two, which
  // halves the reads of the cache.
  if (cache.head_dim <= 64) return a.group <= kRow ? launch_one<64, 1, 6>(a, stream) : launch_one<64, 2, 6>(a, stream);
  return a.group <= kRow ? launch_one<128, 1, 3>(a, stream) : launch_one<128, 2, 3>(a, stream);
}

}  // namespace svdq
