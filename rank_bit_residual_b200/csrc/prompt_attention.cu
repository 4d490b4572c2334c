// prompt_attention.cu - attention over packed prompts (svdq_attention_prompt).
//
//   out = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale q . k_j - m),   m = the running maximum
//
// A block takes 64 rows of one head; four warps of 16 rows walk over the keys in
// tiles of 64 with a running maximum and sum, products on the warp tensor instructions.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"

namespace svdq {

namespace {

constexpr int kThreads = 128;
constexpr int kRows = 64;   // query rows of a block
constexpr int kKeys = 64;   // keys of a tile

struct PromptArgs {
  svdq_heads q, k, v, out;
  const int32_t* cu_q;
  const int32_t* cu_k;
  int batch;
  int64_t q_tokens, k_tokens;
  int dim, causal;
  float scale_log2;
  unsigned* status;
};

// Start of sequence s (no list: one sequence of all rows).
__device__ __forceinline__ long long cu_at(const int32_t* cu, int s, long long tokens) {
  if (!cu) return s == 0 ? 0 : tokens;
  return max(0ll, min(static_cast<long long>(cu[s]), tokens));
}

__device__ __forceinline__ bool bad_cu(const int32_t* cu, int s, long long tokens) {
  return cu && (cu[s] < 0 || cu[s + 1] < cu[s] || cu[s + 1] > tokens);
}

struct Tile {
  int seq;        // -1: past the last tile
  int row0;       // first row of the tile in its sequence
  long long q0;   // first row of the sequence in q
  int rows;       // rows of the sequence
  long long k0;
  int keys;
};

// The tile `index` of the line of all sequences' row tiles; every thread of the block calls it.
__device__ Tile find_tile(const PromptArgs& a, long long index) {
  __shared__ int sh_warp[kThreads / 32];
  __shared__ Tile sh_tile;
  if (threadIdx.x == 0) sh_tile.seq = -1;
  long long before = 0;
  for (int s0 = 0; s0 < a.batch; s0 += kThreads) {
    const int s = s0 + threadIdx.x;
    int n = 0;
    long long q0 = 0, q1 = 0;
    if (s < a.batch) {
      q0 = cu_at(a.cu_q, s, a.q_tokens), q1 = cu_at(a.cu_q, s + 1, a.q_tokens);
      n = static_cast<int>(max(0ll, q1 - q0 + kRows - 1) / kRows);
      if (index == 0 && (bad_cu(a.cu_q, s, a.q_tokens) || bad_cu(a.cu_k, s, a.k_tokens)))
        record_status(a.status, kStatusEinval);
    }
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if ((threadIdx.x & 31) >= o) incl += up;
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 31) sh_warp[threadIdx.x >> 5] = incl;
    __syncthreads();
    int chunk = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < (threadIdx.x >> 5)) incl += sh_warp[w];
      chunk += sh_warp[w];
    }
    if (before + incl - n <= index && index < before + incl) {
      sh_tile.seq = s;
      sh_tile.row0 = static_cast<int>(index - (before + incl - n)) * kRows;
      sh_tile.q0 = q0;
      sh_tile.rows = static_cast<int>(q1 - q0);
      sh_tile.k0 = cu_at(a.cu_k, s, a.k_tokens);
      sh_tile.keys = static_cast<int>(max(0ll, cu_at(a.cu_k, s + 1, a.k_tokens) - sh_tile.k0));
    }
    before += chunk;
    if (before > index) break;
  }
  __syncthreads();
  return sh_tile;
}

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

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// exp2 of a difference to a maximum; a score of -inf counts nothing, even while the
// maximum is -inf itself (no key yet).
__device__ __forceinline__ float exp2_from(float x, float top) { return x == -INFINITY ? 0.0f : exp2f(x - top); }

// The bf16 pairs of a word, infinities and NaN replaced by zero; sets *found then.
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t w, bool* found) {
  if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u, *found = true;
  if ((w & 0x7F800000u) == 0x7F800000u) w &= 0xFFFFu, *found = true;
  return w;
}

template <int kDim>
__global__ void __launch_bounds__(kThreads) prompt_kernel(const PromptArgs a) {
  __shared__ __align__(128) unsigned char sh_k[kKeys * kDim * 2], sh_v[kKeys * kDim * 2];
  __shared__ int sh_odd;   // a value that is not finite behind some row's place
  if (threadIdx.x == 0) sh_odd = 0;
  const Tile t = find_tile(a, blockIdx.x);
  if (t.seq < 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.y, kvh = h / (a.q.heads / a.k.heads);
  const int r0 = t.row0 + warp * 16 + (lane >> 2);   // this lane's rows: r0 and r0 + 8

  const __nv_bfloat16* qp = static_cast<const __nv_bfloat16*>(a.q.data) + t.q0 * a.q.token_ld + h * a.q.head_ld;
  const __nv_bfloat16* kp = static_cast<const __nv_bfloat16*>(a.k.data) + t.k0 * a.k.token_ld + kvh * a.k.head_ld;
  const __nv_bfloat16* vp = static_cast<const __nv_bfloat16*>(a.v.data) + t.k0 * a.v.token_ld + kvh * a.v.head_ld;

  uint32_t qf[kDim / 16][4];
#pragma unroll
  for (int kk = 0; kk < kDim / 16; ++kk)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = r0 + (i & 1) * 8, e = kk * 16 + (i >> 1) * 8 + 2 * (lane & 3);
      qf[kk][i] = row < t.rows && e < a.dim ? *reinterpret_cast<const uint32_t*>(qp + row * a.q.token_ld + e) : 0u;
    }
  float o[kDim / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < kDim / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;

  const int shift = t.keys - t.rows;   // row r sees keys 0 .. shift + r
  const int last = a.causal ? min(t.keys, min(t.rows, t.row0 + kRows) + shift) : t.keys;
  // Tiles from here on hold keys that some row does not see. A value there that is not
  // finite must not meet that row's zero weight (0 * NaN): it is taken out of the product
  // and added at the end to the rows that see it.
  const int cut = a.causal ? max(0, t.row0 + shift + 1) / kKeys * kKeys : last;
  for (int key0 = 0; key0 < last; key0 += kKeys) {
    __syncthreads();
    for (int i = threadIdx.x; i < kKeys * (kDim / 8); i += kThreads) {
      const int row = i / (kDim / 8), c = i % (kDim / 8);
      const bool on = key0 + row < t.keys && c * 8 < a.dim;
      const int at = row * kDim * 2 + ((c ^ (row & 7)) << 4);
      cp_async16(sh_k + at, on ? kp + (key0 + row) * a.k.token_ld + c * 8 : kp, on ? 16 : 0);
      cp_async16(sh_v + at, on ? vp + (key0 + row) * a.v.token_ld + c * 8 : vp, on ? 16 : 0);
    }
    cp_async_commit();
    cp_async_wait<0>();
    if (key0 >= cut) {
      bool found = false;
      for (int i = threadIdx.x; i < kKeys * (kDim / 8); i += kThreads) {   // what this thread has copied
        const int row = i / (kDim / 8), c = i % (kDim / 8);
        uint4* w = reinterpret_cast<uint4*>(sh_v + row * kDim * 2 + ((c ^ (row & 7)) << 4));
        uint4 x = *w;
        x.x = finite_or_zero(x.x, &found), x.y = finite_or_zero(x.y, &found);
        x.z = finite_or_zero(x.z, &found), x.w = finite_or_zero(x.w, &found);
        *w = x;
      }
      if (found) sh_odd = 1;
    }
    __syncthreads();

    float s[kKeys / 8][4];
#pragma unroll
    for (int n = 0; n < kKeys / 8; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.0f;
#pragma unroll
    for (int n = 0; n < kKeys / 16; ++n)
#pragma unroll
      for (int kk = 0; kk < kDim / 16; ++kk) {
        uint32_t f[4];
        const int row = n * 16 + (lane & 7) + (lane >> 4) * 8, c = 2 * kk + ((lane >> 3) & 1);
        ldmatrix_x4(smem_u32(sh_k) + row * kDim * 2 + ((c ^ (row & 7)) << 4), f);
        const uint32_t b0[2] = {f[0], f[1]}, b1[2] = {f[2], f[3]};
        mma_bf16_16816(s[2 * n], qf[kk], b0);
        mma_bf16_16816(s[2 * n + 1], qf[kk], b1);
      }
    float top[2] = {m[0], m[1]};
#pragma unroll
    for (int n = 0; n < kKeys / 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = key0 + n * 8 + 2 * (lane & 3) + (i & 1), row = r0 + (i >> 1) * 8;
        const bool on = key < t.keys && (!a.causal || key <= row + shift);
        s[n][i] = on ? s[n][i] * a.scale_log2 : -INFINITY;
        top[i >> 1] = fmaxf(top[i >> 1], s[n][i]);
      }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
      top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
      const float f = exp2_from(m[i], top[i]);
      m[i] = top[i];
      l[i] *= f;
#pragma unroll
      for (int d = 0; d < kDim / 8; ++d) o[d][2 * i] *= f, o[d][2 * i + 1] *= f;
    }
#pragma unroll
    for (int n = 0; n < kKeys / 16; ++n) {
#pragma unroll
      for (int j = 2 * n; j < 2 * n + 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[j][i] = exp2_from(s[j][i], m[i >> 1]);
          l[i >> 1] += s[j][i];
        }
      const uint32_t pf[4] = {pack_bf16(s[2 * n][0], s[2 * n][1]), pack_bf16(s[2 * n][2], s[2 * n][3]),
                              pack_bf16(s[2 * n + 1][0], s[2 * n + 1][1]), pack_bf16(s[2 * n + 1][2], s[2 * n + 1][3])};
#pragma unroll
      for (int d = 0; d < kDim / 16; ++d) {
        uint32_t f[4];
        const int row = n * 16 + (lane & 15), c = 2 * d + (lane >> 4);
        ldmatrix_x4_trans(smem_u32(sh_v) + row * kDim * 2 + ((c ^ (row & 7)) << 4), f);
        const uint32_t b0[2] = {f[0], f[1]}, b1[2] = {f[2], f[3]};
        mma_bf16_16816(o[2 * d], pf, b0);
        mma_bf16_16816(o[2 * d + 1], pf, b1);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    const int row = r0 + 8 * i;
    if (row >= t.rows) continue;
    const float inv = l[i] == 0.0f ? 0.0f : 1.0f / l[i];
    if (sh_odd) {
      for (int j = cut; j <= row + shift && j < t.keys; ++j)
#pragma unroll
        for (int d = 0; d < kDim / 8; ++d)
          for (int b = 0; b < 2; ++b) {
            const int e = d * 8 + 2 * (lane & 3) + b;
            const float x = e < a.dim ? __bfloat162float(vp[j * a.v.token_ld + e]) : 0.0f;
            if (!isfinite(x)) o[d][2 * i + b] += x;
          }
    }
    __nv_bfloat16* dst =
        static_cast<__nv_bfloat16*>(a.out.data) + (t.q0 + row) * a.out.token_ld + h * a.out.head_ld + 2 * (lane & 3);
#pragma unroll
    for (int d = 0; d < kDim / 8; ++d)
      if (d * 8 < a.dim) *reinterpret_cast<uint32_t*>(dst + d * 8) = pack_bf16(o[d][2 * i] * inv, o[d][2 * i + 1] * inv);
  }
}

}  // namespace

cudaError_t launch_prompt(const svdq_heads& q, const svdq_heads& k, const svdq_heads& v, const int32_t* cu_q,
                          const int32_t* cu_k, int batch, int64_t q_tokens, int64_t k_tokens, int head_dim,
                          bool causal, float scale, const svdq_heads& out, cudaStream_t stream, bool* bad_args) {
  PromptArgs a{q, k, v, out, cu_q, cu_k, batch, q_tokens, k_tokens, head_dim, causal ? 1 : 0,
               scale * 1.4426950408889634f, device_status_word()};
  *bad_args = false;
  const dim3 grid(static_cast<unsigned>(q_tokens / kRows + batch), static_cast<unsigned>(q.heads));
  if (head_dim <= 64)
    prompt_kernel<64><<<grid, kThreads, 0, stream>>>(a);
  else
    prompt_kernel<128><<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace svdq
