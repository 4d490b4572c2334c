// head_norm.cu - RMS norm and rotation of query and key heads, with the rows of a
// paged cache written on the way (svdq_qk_norm_rope, svdq_kv_append).
//
//   y = x * rsqrt(mean(x^2) + eps) * w,   then per pair  A (a cos - b sin, b cos + a sin)
//
// Every row is read once and written once; nothing else moves, so the pass is bound by
// HBM (a few tokens: by the latency of one load, one reduction and one store). A group of
// 8, 16 or 32 lanes (head_dim up to 64, 128, 256) holds a row, eight consecutive
// elements per lane (16-byte loads of bf16). The cosines of a token are the same for
// all its heads: a block computes them once (fp64 product and reduction to one turn, fp32
// sincospi) into shared memory, and each group keeps the eight pairs of its lanes in
// registers while it walks over the heads of one token. The partner of an element
// in the half layout sits in another lane at the same place (one shuffle) when
// rot_dim / 2 is a multiple of 8, else the row goes through shared memory.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "internal.h"
#include "ptx.cuh"

namespace svdq {

namespace {

constexpr int kThreads = 256;
constexpr int kVec = 8;           // elements per lane
constexpr int kMaxTokens = 4;     // tokens per block
constexpr int kMaxDim = 256;

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[kVec]);
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&x)[kVec]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&x)[kVec]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[kVec]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&x)[kVec]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

struct HeadsTile {
  int tokens_per_block;   // power of two, 1 .. kMaxTokens
  int rows;               // heads of q, k and (with a cache) v per token
};

// kLanes lanes per row. Blocks: x over tiles of tokens_per_block tokens, y over ranges of
// a token's rows.
template <typename T, int kLanes>
__global__ void __launch_bounds__(kThreads) heads_kernel(const HeadsArgs a, const HeadsTile tile) {
  constexpr int kGroups = kThreads / kLanes;
  __shared__ float2 sh_cs[kMaxTokens][kMaxDim / 2];
  __shared__ float sh_row[kGroups][kLanes * kVec];

  const int lane = threadIdx.x % kLanes;
  const int group = threadIdx.x / kLanes;
  const int groups_per_token = kGroups / tile.tokens_per_block;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tile.tokens_per_block;
  const int tl = group / groups_per_token;
  const int64_t t = t0 + tl;
  const bool live = t < a.tokens;
  const int half = a.rope.rot_dim / 2;

  for (int i = threadIdx.x; i < half * tile.tokens_per_block; i += kThreads) {
    const int tt = i / half, j = i - tt * half;
    if (t0 + tt < a.tokens) {
      const double turn = static_cast<double>(a.positions[t0 + tt]) * a.rope.turns[j];
      float s, c;
      sincospif(static_cast<float>(2.0 * (turn - rint(turn))), &s, &c);
      sh_cs[tt][j] = make_float2(a.rope.amplitude * c, a.rope.amplitude * s);
    }
  }
  __syncthreads();

  const int e0 = lane * kVec;
  const bool in_row = e0 < a.head_dim;
  // this lane's pairs: element e0 + i turns with (cs[i].x, cs[i].y), sin negated for the
  // first of a pair; elements past rot_dim with (1, 0)
  float cs[kVec], sn[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int e = e0 + i;
    cs[i] = 1.0f, sn[i] = 0.0f;
    if (e < a.rope.rot_dim) {
      const int j = a.rope.interleaved ? e >> 1 : (e < half ? e : e - half);
      const bool first = a.rope.interleaved ? (e & 1) == 0 : e < half;
      const float2 v = sh_cs[tl][j];
      cs[i] = v.x;
      sn[i] = first ? -v.y : v.y;
    }
  }
  const bool by_shuffle = half % kVec == 0;
  const int partner = e0 < half ? lane + half / kVec : (e0 < a.rope.rot_dim ? lane - half / kVec : lane);

  int64_t slot = -1;
  if (a.cache.k && live) {
    slot = a.slots[t];
    if (slot >= a.cache.pages * a.cache.page_size) {
      if (group % groups_per_token == 0 && lane == 0 && blockIdx.y == 0) record_status(a.status, kStatusEinval);
      slot = -1;
    }
  }
  int64_t cache_row = 0;
  if (slot >= 0) cache_row = slot / a.cache.page_size * a.cache.page_ld + slot % a.cache.page_size * a.cache.slot_ld;

  const int stride = groups_per_token * gridDim.y;
  const int r_first = blockIdx.y * groups_per_token + group % groups_per_token;
  const int trips = (tile.rows + stride - 1) / stride;
  for (int trip = 0; trip < trips; ++trip) {
    const int r = r_first + trip * stride;
    const bool on = live && r < tile.rows && in_row;
    const bool is_q = r < a.q.heads, is_k = !is_q && r < a.q.heads + a.k.heads;
    const int h = is_q ? r : (is_k ? r - a.q.heads : r - a.q.heads - a.k.heads);
    const svdq_heads& src = is_q ? a.q : (is_k ? a.k : a.v);
    float x[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) x[i] = 0.0f;
    if (on) load8(static_cast<const T*>(src.data) + t * src.token_ld + h * src.head_ld + e0, x);

    const void* w = is_q ? a.q_weight : (is_k ? a.k_weight : nullptr);
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < kVec; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (w && in_row) {
      const float inv = rsqrtf(ss / static_cast<float>(a.head_dim) + a.eps);
      float wv[kVec];
      if (a.weight_bf16)
        load8(static_cast<const __nv_bfloat16*>(w) + e0, wv);
      else
        load8(static_cast<const float*>(w) + e0, wv);
#pragma unroll
      for (int i = 0; i < kVec; ++i) x[i] *= inv * wv[i];
    }

    if (half > 0) {
      float other[kVec];
      if (a.rope.interleaved) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) other[i] = x[i ^ 1];
      } else if (by_shuffle) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) other[i] = __shfl_sync(0xffffffffu, x[i], partner, kLanes);
      } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) sh_row[group][e0 + i] = x[i];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const int e = e0 + i;
          other[i] = e < a.rope.rot_dim ? sh_row[group][e < half ? e + half : e - half] : 0.0f;
        }
        __syncwarp();
      }
      if (is_q || is_k) {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
          if (e0 + i < a.rope.rot_dim) x[i] = fmaf(other[i], sn[i], x[i] * cs[i]);
      }
    }

    if (!on) continue;
    if (is_q) {
      store8(static_cast<T*>(a.q_out.data) + t * a.q_out.token_ld + h * a.q_out.head_ld + e0, x);
    } else {
      if (is_k && a.k_out.data)
        store8(static_cast<T*>(a.k_out.data) + t * a.k_out.token_ld + h * a.k_out.head_ld + e0, x);
      if (slot >= 0)
        store8(static_cast<T*>(is_k ? a.cache.k : a.cache.v) + cache_row + h * a.cache.head_ld + e0, x);
    }
  }
}

template <typename T, int kLanes>
cudaError_t launch_lanes(const HeadsArgs& a, cudaStream_t st) {
  HeadsTile tile;
  tile.rows = a.q.heads + a.k.heads + (a.cache.k ? a.v.heads : 0);
  // Four tokens per block share nothing but the launch; a block per token and more blocks
  // per token only when there are too few to fill the GPU.
  tile.tokens_per_block = kMaxTokens;
  const int64_t want = 4 * num_sms();
  while (tile.tokens_per_block > 1 && ceil_div(a.tokens, tile.tokens_per_block) < want) tile.tokens_per_block /= 2;
  const int64_t bx = ceil_div(a.tokens, tile.tokens_per_block);
  const int per_block = kThreads / kLanes / tile.tokens_per_block;
  const int64_t by = std::max<int64_t>(1, std::min<int64_t>(ceil_div(tile.rows, per_block), want / bx));
  heads_kernel<T, kLanes><<<dim3(static_cast<unsigned>(bx), static_cast<unsigned>(by)), kThreads, 0, st>>>(a, tile);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_type(const HeadsArgs& a, cudaStream_t st) {
  if (a.head_dim <= 64) return launch_lanes<T, 8>(a, st);
  if (a.head_dim <= 128) return launch_lanes<T, 16>(a, st);
  return launch_lanes<T, 32>(a, st);
}

}  // namespace

cudaError_t launch_heads(const HeadsArgs& a, svdq_dtype dtype, cudaStream_t stream) {
  return dtype == SVDQ_BF16 ? launch_type<__nv_bfloat16>(a, stream) : launch_type<float>(a, stream);
}

}  // namespace svdq
