// head_norm.cu - RMS norm and rotation of query and key heads, with the rows of a
// paged cache written on the way (svdq_qk_norm_rope, svdq_kv_append).
//
//   y = x * rsqrt(mean(x^2) + eps) * w,   then per pair  A (a cos - b sin, b cos + a sin)
//
// Every row is read once and written once; nothing else moves, so the pass is bound by
// HBM (a few tokens: by the latency of one load, one reduction and one store). A group of
// 8, 16 or 32 lanes (head_dim up to 64, 128, 256) holds a row, eight consecutive
// elements per lane (16-byte loads of bf16). A warp takes a token, or a share of its heads:
// the cosines are the same for all heads, so its lanes compute them once, and each lane
// keeps what it needs of them in registers while the rows go by, the next ones in flight behind these:
//   y_i = inv (x_i A_i + x_partner B_i),   A = w cos,   B = -+ w_partner sin
// The partner of an element in the half layout sits in another lane at the same place
// (exchanged as it lies in memory, two bf16 per shuffle) when rot_dim / 2 is a multiple
// of 8, else the row goes through shared memory. Angles are exact to 2^-32 of a turn at
// any position: a frequency is a 64-bit fraction of a turn, and its integer product with
// the position wraps at whole turns by itself. (fp64 products cost more than the rows of
// two heads: 69 -> 47 us for 8192 tokens came from halving their number.) Warps wait for nothing but their own loads;
// with blocks of four tokens that shared their cosines behind a barrier, that start of every
// block took as long as its rows.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "encode.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace svdq {

namespace {

constexpr int kThreads = 256;
constexpr int kVec = 8;           // elements per lane
constexpr int kWarps = kThreads / 32;
constexpr int kBlocksPerSm = 3;
constexpr int kMaxDim = 256;
constexpr int kFlight = 2;        // rows of a group that are loaded together, one such set ahead

// How the partner of a rotated element is found.
enum Pairing { kShuffle = 0, kNeighbour = 1, kThroughShared = 2 };

// Eight elements as they lie in memory.
template <typename T>
struct Raw {
  static constexpr int kWords = kVec * sizeof(T) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) {
      const uint4 u = reinterpret_cast<const uint4*>(p)[i];
      w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i)
      reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
  // the eight values as four pairs
  __device__ __forceinline__ void get(uint64_t (&x)[kVec / 2]) const {
#pragma unroll
    for (int i = 0; i < kVec / 2; ++i) {
      if (sizeof(T) == 2)
        x[i] = pk2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
      else
        x[i] = pk2(__uint_as_float(w[(2 * i) % kWords]), __uint_as_float(w[(2 * i + 1) % kWords]));
    }
  }
  __device__ __forceinline__ void put(const uint64_t (&x)[kVec / 2]) {
#pragma unroll
    for (int i = 0; i < kVec / 2; ++i) {
      float lo, hi;
      upk2(x[i], lo, hi);
      if (sizeof(T) == 2) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        w[i] = *reinterpret_cast<const uint32_t*>(&v);
      } else {
        w[(2 * i) % kWords] = __float_as_uint(lo), w[(2 * i + 1) % kWords] = __float_as_uint(hi);
      }
    }
  }
};

__device__ __forceinline__ void take8(const float* p, float (&x)[kVec]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

// kLanes lanes per row. A unit is a share of a token's heads; the warps of the grid take
// units in turn.
template <typename T, int kLanes, int kPairing>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) heads_kernel(const __grid_constant__ HeadsArgs a, const int shares) {
  constexpr int kGroups = 32 / kLanes;   // rows of a warp at a time
  __shared__ __align__(16) float sh_w[2][kMaxDim];
  __shared__ unsigned long long sh_turns[kMaxDim / 2];   // in 2^-64 of a turn
  __shared__ __align__(16) float sh_cos[kWarps][kMaxDim / 2], sh_sin[kWarps][kMaxDim / 2];
  __shared__ __align__(16) T sh_row[kPairing == kThroughShared ? kThreads * kVec : 1];

  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % kLanes;                 // in the row
  const int group = threadIdx.x % 32 / kLanes;
  const int half = a.rope.rot_dim / 2;
  const int e0 = lane * kVec;
  const bool in_row = e0 < a.head_dim;
  const float inv_dim = 1.0f / static_cast<float>(a.head_dim);

  for (int i = threadIdx.x; i < a.head_dim; i += kThreads) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const void* w = s == 0 ? a.q_weight : a.k_weight;
      sh_w[s][i] = !w ? 1.0f
                      : a.weight_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i])
                                      : static_cast<const float*>(w)[i];
    }
  }
  for (int j = threadIdx.x; j < half; j += kThreads) {
    const double turn = a.rope.turns[j];
    sh_turns[j] = __double2ull_rd((turn - floor(turn)) * 18446744073709551616.0);
  }
  __syncthreads();

  // the partner of element e of a head, and its lane here
  auto partner_of = [&](int e) {
    if (e >= a.rope.rot_dim) return e;
    return kPairing == kNeighbour ? e ^ 1 : (e < half ? e + half : e - half);
  };
  const int partner = partner_of(e0) / kVec;
  const unsigned units = static_cast<unsigned>(a.tokens) * shares;   // below 2^31
  const unsigned warps = gridDim.x * kWarps;
  const int stride = kGroups * shares;

  // what a unit needs first is loaded while the one before it is worked on
  int64_t next_position = 0, next_slot = -1;
  auto look_ahead = [&](unsigned unit) {
    if (unit >= units) return;
    const unsigned t = shares == 1 ? unit : unit / shares;
    if (half > 0) next_position = a.positions[t];
    if (a.cache.k) next_slot = a.slots[t];
  };
  Raw<T> now[kFlight], next[kFlight];
#pragma unroll
  for (int u = 0; u < kFlight; ++u) now[u].zero(), next[u].zero();   // lanes past head_dim stay so

  unsigned unit = blockIdx.x * kWarps + warp;
  look_ahead(unit);
  for (; unit < units; unit += warps) {
    const int64_t t = shares == 1 ? unit : unit / shares;
    const int share = static_cast<int>(unit - static_cast<unsigned>(t) * shares);
    const int h0 = share * kGroups + group;   // heads h0, h0 + stride, ... are this group's
    const int64_t position_now = next_position, slot = next_slot;
    look_ahead(unit + warps);

    // The rows of this group in one tensor, a set of kFlight at a time, the next set in
    // flight. start() loads the first set; every lane makes the same number of turns.
    auto load_set = [&](const svdq_heads& src, Raw<T> (&set)[kFlight], const T*& p, int first) {
      const int64_t step = stride * src.head_ld;
      const int left = in_row ? src.heads - h0 : 0;
#pragma unroll
      for (int u = 0; u < kFlight; ++u, p += step)
        if (first + u * stride < left) set[u].load(p);
    };
    auto start = [&](const svdq_heads& src) {
      const T* p = static_cast<const T*>(src.data) + t * src.token_ld + h0 * src.head_ld + e0;
      load_set(src, now, p, 0);
      return p;
    };
    auto walk = [&](const svdq_heads& src, const T* p, auto&& use) {
      const int left = in_row ? src.heads - h0 : 0;
      for (int first = 0; first < src.heads; first += kFlight * stride) {
        load_set(src, next, p, first + kFlight * stride);
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
          if (first + u * stride < src.heads) use(now[u], first + u * stride < left);
          now[u] = next[u];
        }
      }
    };
    // a running pointer to where rows go
    auto row_of = [&](void* data, int64_t token_row, int64_t head_ld) {
      return static_cast<T*>(data) + token_row + h0 * head_ld + e0;
    };
    const T* from = start(a.q.heads > 0 ? a.q : a.k);

    // where the token's key and value go in the cache
    int64_t cache_row = -1;
    if (a.cache.k && slot >= 0) {
      const int64_t slots = a.cache.pages * a.cache.page_size;
      if (slot >= slots) {
        if (threadIdx.x % 32 == 0 && share == 0) record_status(a.status, kStatusEinval);
      } else {
        // (a division of 64 bits takes as long as several rows)
        const int64_t page = slots <= 0x7FFFFFFF ? static_cast<unsigned>(slot) / static_cast<unsigned>(a.cache.page_size)
                                                 : slot / a.cache.page_size;
        cache_row = page * a.cache.page_ld + (slot - page * a.cache.page_size) * a.cache.slot_ld;
      }
    }
    if (half > 0) {
      const unsigned long long position = static_cast<unsigned long long>(position_now);
      for (int j = threadIdx.x % 32; j < half; j += 32) {
        // the upper half of the product as a signed number of 2^-31 half turns
        const int turned = static_cast<int>((position * sh_turns[j]) >> 32);
        float s, c;
        sincospif(static_cast<float>(turned) * 4.656612873077393e-10f, &s, &c);
        sh_cos[warp][j] = a.rope.amplitude * c;
        sh_sin[warp][j] = a.rope.amplitude * s;
      }
      __syncwarp();
    }

    auto turn_heads = [&](const svdq_heads& src, const T* p, const void* weight, const float* w, auto&& store) {
      uint64_t own[kVec / 2], theirs[kVec / 2];   // A and B
      uint32_t mask[Raw<T>::kWords];              // 0 where no partner takes part
      // eight consecutive floats, or those of the pairs of eight consecutive elements
      float we[kVec], wp[kVec], co[kVec], si[kVec];
      const bool turns0 = e0 < a.rope.rot_dim;
      const int ew = in_row ? e0 : 0;
      take8(w + ew, we);
      if (kPairing == kNeighbour) {
#pragma unroll
        for (int i = 0; i < kVec; i += 2) {
          wp[i] = we[i + 1], wp[i + 1] = we[i];
          const int j = e0 + i < a.rope.rot_dim ? (e0 + i) >> 1 : 0;
          co[i] = co[i + 1] = sh_cos[warp][j];
          si[i + 1] = sh_sin[warp][j];
          si[i] = -si[i + 1];
        }
      } else if (kPairing == kShuffle) {   // all eight turn, or none
        const int j = turns0 ? (e0 < half ? e0 : e0 - half) : 0;
        take8(w + (turns0 ? partner * kVec : 0), wp);
        take8(sh_cos[warp] + j, co);
        take8(sh_sin[warp] + j, si);
        if (e0 < half) {
#pragma unroll
          for (int i = 0; i < kVec; ++i) si[i] = -si[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const int e = e0 + i, j = e < half ? e : e - half;
          const bool turns = e < a.rope.rot_dim;
          wp[i] = w[turns ? partner_of(e) : 0];
          co[i] = sh_cos[warp][turns ? j : 0];
          si[i] = sh_sin[warp][turns ? j : 0];
          if (e < half) si[i] = -si[i];
        }
      }
#pragma unroll
      for (int i = 0; i < kVec; i += 2) {
        // rot_dim is even: both of two consecutive elements turn, or neither
        const bool turns = e0 + i < a.rope.rot_dim;
        own[i / 2] = turns ? pk2(we[i] * co[i], we[i + 1] * co[i + 1]) : pk2(we[i], we[i + 1]);
        theirs[i / 2] = turns ? pk2(wp[i] * si[i], wp[i + 1] * si[i + 1]) : 0;
        if (sizeof(T) == 2)
          mask[i / 2] = turns ? 0xFFFFFFFFu : 0u;
        else
          mask[i % Raw<T>::kWords] = mask[(i + 1) % Raw<T>::kWords] = turns ? 0xFFFFFFFFu : 0u;
      }
      walk(src, p, [&](Raw<T>& raw, bool live) {
        uint64_t x[kVec / 2];
        raw.get(x);
        uint64_t inv2 = pk2(1.0f, 1.0f);
        if (weight) {
          uint64_t s2 = fmul2_rn(x[0], x[0]);
#pragma unroll
          for (int i = 1; i < kVec / 2; ++i) s2 = ffma2_rn(x[i], x[i], s2);
          float ss, s1;
          upk2(s2, ss, s1);
          ss += s1;
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          const float inv = rsqrtf(fmaf(ss, inv_dim, a.eps));
          inv2 = pk2(inv, inv);
        }
        if (half > 0) {
          Raw<T> raw2;
          if (kPairing == kNeighbour) {
#pragma unroll
            for (int i = 0; i < Raw<T>::kWords; ++i)
              raw2.w[i] = sizeof(T) == 2 ? __byte_perm(raw.w[i], 0, 0x1032) : raw.w[(i ^ 1) % Raw<T>::kWords];
          } else if (kPairing == kShuffle) {
#pragma unroll
            for (int i = 0; i < Raw<T>::kWords; ++i) raw2.w[i] = __shfl_sync(0xffffffffu, raw.w[i], partner, kLanes);
          } else {
            T* row = sh_row + (kPairing == kThroughShared ? (threadIdx.x - lane) * kVec : 0);
            raw.store(row + e0);
            __syncwarp();
            T mine[kVec];
#pragma unroll
            for (int i = 0; i < kVec; ++i) mine[i] = row[partner_of(e0 + i)];
            __syncwarp();
#pragma unroll
            for (int i = 0; i < Raw<T>::kWords; ++i) raw2.w[i] = reinterpret_cast<const uint32_t*>(mine)[i];
          }
          if (2 * half < a.head_dim) {
            // a value that takes no part must not meet B = 0 as an infinity
#pragma unroll
            for (int i = 0; i < Raw<T>::kWords; ++i) raw2.w[i] &= mask[i];
          }
          uint64_t y[kVec / 2];
          raw2.get(y);
#pragma unroll
          for (int i = 0; i < kVec / 2; ++i) x[i] = ffma2_rn(y[i], theirs[i], fmul2_rn(x[i], own[i]));
        } else {
#pragma unroll
          for (int i = 0; i < kVec / 2; ++i) x[i] = fmul2_rn(x[i], own[i]);
        }
        if (weight) {
#pragma unroll
          for (int i = 0; i < kVec / 2; ++i) x[i] = fmul2_rn(x[i], inv2);
        }
        Raw<T> out;
        out.put(x);
        store(out, live);
      });
    };

    if (a.q.heads > 0) {
      T* q = row_of(a.q_out.data, t * a.q_out.token_ld, a.q_out.head_ld);
      const int64_t step = stride * a.q_out.head_ld;
      turn_heads(a.q, from, a.q_weight, sh_w[0], [&](const Raw<T>& y, bool live) {
        if (live) y.store(q);
        q += step;
      });
      from = start(a.k);
    }
    {
      T* k = a.k_out.data ? row_of(a.k_out.data, t * a.k_out.token_ld, a.k_out.head_ld) : nullptr;
      T* c = cache_row >= 0 ? row_of(a.cache.k, cache_row, a.cache.head_ld) : nullptr;
      const int64_t step = stride * a.k_out.head_ld, c_step = stride * a.cache.head_ld;
      turn_heads(a.k, from, a.k_weight, sh_w[1], [&](const Raw<T>& y, bool live) {
        if (live && a.k_out.data) y.store(k);
        if (live && cache_row >= 0) y.store(c);
        k += step, c += c_step;
      });
    }
    if (a.cache.k) {
      T* c = cache_row >= 0 ? row_of(a.cache.v, cache_row, a.cache.head_ld) : nullptr;
      const int64_t c_step = stride * a.cache.head_ld;
      walk(a.v, start(a.v), [&](const Raw<T>& y, bool live) {
        if (live && cache_row >= 0) y.store(c);
        c += c_step;
      });
    }
    __syncwarp();   // the cosines may be written again
  }
}

template <typename T, int kLanes, int kPairing>
cudaError_t launch_pairing(const HeadsArgs& a, cudaStream_t st) {
  const int64_t warps = static_cast<int64_t>(kBlocksPerSm) * num_sms() * kWarps;
  // A token's heads are divided only when there are fewer tokens than warps, down to one row
  // per group: every share computes the cosines again (4 units per warp instead of one
  // or two: 37 -> 57 us for an append of 6007 tokens).
  const int64_t most = ceil_div(std::max({a.q.heads, a.k.heads, 1}), 32 / kLanes);
  const int64_t shares = std::max<int64_t>(1, std::min<int64_t>(most, ceil_div(warps, a.tokens)));
  const int64_t blocks = std::min<int64_t>(ceil_div(a.tokens * shares, kWarps), warps / kWarps);
  heads_kernel<T, kLanes, kPairing><<<static_cast<unsigned>(blocks), kThreads, 0, st>>>(a, static_cast<int>(shares));
  return cudaGetLastError();
}

template <typename T, int kLanes>
cudaError_t launch_lanes(const HeadsArgs& a, cudaStream_t st) {
  if (a.rope.interleaved) return launch_pairing<T, kLanes, kNeighbour>(a, st);
  if (a.rope.rot_dim / 2 % kVec == 0) return launch_pairing<T, kLanes, kShuffle>(a, st);
  return launch_pairing<T, kLanes, kThroughShared>(a, st);
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
