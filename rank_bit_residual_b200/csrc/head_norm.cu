// head_norm.cu - RMS norm and rotation of query and key heads, with the rows of a
// paged cache written on the way (svdq_qk_norm_rope, svdq_kv_append).
//
//   y = x * rsqrt(mean(x^2) + eps) * w,   then per pair  A (a cos - b sin, b cos + a sin)
//
// Every row is read once and written once; nothing else moves, so the pass is bound by
// HBM, if it issues few enough instructions (a few tokens: by the latency of one load, one
// reduction and one store). A group of 4, 8 or 16 lanes (head_dim up to 64, 128, 256)
// holds a row, each lane two chunks of eight consecutive elements (16-byte loads of bf16).
// In the half layout a lane's two chunks are partners when rot_dim / 2 is a multiple of 8,
// so that a rotation needs no exchange:
//   y_i = inv (x_i A_i + x_partner B_i),   A = w cos,   B = -+ w_partner sin
// and the norm three shuffles for four rows of 128. (With one chunk per lane: 150
// instructions for two rows of 128 elements, 47 us for 8192 tokens of 40 heads.) Other
// half layouts pass the row through shared memory. A warp takes a token, or a share of its heads:
// the cosines are the same for all heads, so its lanes compute them once, and each lane
// keeps what it needs of them in registers while the rows go by, the next ones in flight
// behind these. A frequency is a 64-bit fraction of a turn (cut there), and its integer
// product with the position wraps at whole turns by itself: angles are within 2^-32 + |position| 2^-64
// of a turn, and are then rounded to the 24 bits of a float (of half a turn at most). Warps
// wait for nothing but their own loads.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "encode.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace svdq {

namespace {

constexpr int kThreads = 256;
constexpr int kVec = 8;           // elements of a chunk; a lane has two
constexpr int kWarps = kThreads / 32;
constexpr int kBlocksPerSm = 2;
constexpr int kMaxDim = 256;

// How the partner of a rotated element is found.
enum Pairing { kHalves = 0, kNeighbour = 1, kThroughShared = 2 };

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
  // sets of rows that are loaded together, one set ahead: as many as the registers hold
  // (two sets of bf16 rows: 41 -> 37 us for 8192 tokens of 40 heads)
  constexpr int kFlight = sizeof(T) == 2 ? 2 : 1;
  __shared__ __align__(16) float sh_w[2][kMaxDim];
  __shared__ unsigned long long sh_turns[kMaxDim / 2];   // in 2^-64 of a turn
  __shared__ __align__(16) float sh_cos[kWarps][kMaxDim / 2], sh_sin[kWarps][kMaxDim / 2];
  __shared__ __align__(16) T sh_row[kPairing == kThroughShared ? kThreads * 2 * kVec : 1];

  pdl_wait();
  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % kLanes;                 // in the row
  const int group = threadIdx.x % 32 / kLanes;
  const int half = a.rope.rot_dim / 2;
  const float inv_dim = 1.0f / static_cast<float>(a.head_dim);

  // the two chunks of this lane, by their first element
  int e[2] = {2 * lane * kVec, (2 * lane + 1) * kVec};
  const bool partners = kPairing == kHalves && lane < half / kVec;   // the two are each other's
  if (partners) e[0] = lane * kVec, e[1] = lane * kVec + half;
  const bool on[2] = {e[0] < a.head_dim, e[1] < a.head_dim};

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
  Raw<T> now[kFlight][2], next[kFlight][2];
#pragma unroll
  for (int u = 0; u < kFlight; ++u)   // chunks past head_dim stay zero
#pragma unroll
    for (int c = 0; c < 2; ++c) now[u][c].zero(), next[u][c].zero();

  unsigned unit = blockIdx.x * kWarps + warp;
  int64_t t = 0;
  int share = 0, h0 = 0;   // heads h0, h0 + stride, ... are this group's
  // The rows of this group in one tensor, a set of kFlight at a time, the next set in
  // flight. start() loads the first set; every lane makes the same number of turns.
  auto load_set = [&](const svdq_heads& src, Raw<T> (&set)[kFlight][2], const T*& p, int first) {
    const int64_t step = stride * src.head_ld;
#pragma unroll
    for (int u = 0; u < kFlight; ++u, p += step)
      if (first + u * stride + h0 < src.heads) {
        if (on[0]) set[u][0].load(p + e[0]);
        if (on[1]) set[u][1].load(p + e[1]);
      }
  };
  auto start = [&](const svdq_heads& src) {
    const T* p = static_cast<const T*>(src.data) + t * src.token_ld + h0 * src.head_ld;
    load_set(src, now, p, 0);
    return p;
  };
  auto start_unit = [&]() -> const T* {
    if (unit >= units) return nullptr;
    t = shares == 1 ? unit : unit / shares;
    share = static_cast<int>(unit - static_cast<unsigned>(t) * shares);
    h0 = share * kGroups + group;
    return start(a.q.heads > 0 ? a.q : a.k);
  };
  look_ahead(unit);
  const T* from = start_unit();

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

  while (unit < units) {
    const int64_t position_now = next_position, slot = next_slot;
    look_ahead(unit + warps);
    auto walk = [&](const svdq_heads& src, const T* p, auto&& use) {
      for (int first = 0; first < src.heads; first += kFlight * stride) {
        load_set(src, next, p, first + kFlight * stride);
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
          if (first + u * stride < src.heads) use(now[u], first + u * stride + h0 < src.heads);
          now[u][0] = next[u][0];
          now[u][1] = next[u][1];
        }
      }
    };
    // a running pointer to where rows go
    auto row_of = [&](void* data, int64_t token_row, int64_t head_ld) {
      return static_cast<T*>(data) + token_row + h0 * head_ld;
    };
    auto put_row = [&](T* p, const Raw<T> (&y)[2]) {
      if (on[0]) y[0].store(p + e[0]);
      if (on[1]) y[1].store(p + e[1]);
    };

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

    // the partner of an element that turns, and its pair
    auto partner_of = [&](int i) { return kPairing == kNeighbour ? i ^ 1 : (i < half ? i + half : i - half); };
    auto pair_of = [&](int i) { return kPairing == kNeighbour ? i >> 1 : (i < half ? i : i - half); };

    auto turn_heads = [&](const svdq_heads& src, const T* p, const void* weight, const float* w, auto&& store) {
      uint64_t own[2][kVec / 2], theirs[2][kVec / 2];   // A and B
      uint32_t mask[2][Raw<T>::kWords];                 // 0 where no partner takes part
      {
        float we[2][kVec];
#pragma unroll
        for (int c = 0; c < 2; ++c) take8(w + (on[c] ? e[c] : 0), we[c]);
        if (kPairing == kHalves) {
          float co[kVec], si[kVec];
          take8(sh_cos[warp] + (partners ? e[0] : 0), co);
          take8(sh_sin[warp] + (partners ? e[0] : 0), si);
#pragma unroll
          for (int i = 0; i < kVec; ++i) {
            if (!partners) co[i] = 1.0f, si[i] = 0.0f;
          }
#pragma unroll
          for (int i = 0; i < kVec; i += 2) {
            own[0][i / 2] = pk2(we[0][i] * co[i], we[0][i + 1] * co[i + 1]);
            own[1][i / 2] = pk2(we[1][i] * co[i], we[1][i + 1] * co[i + 1]);
            theirs[0][i / 2] = pk2(-we[1][i] * si[i], -we[1][i + 1] * si[i + 1]);
            theirs[1][i / 2] = pk2(we[0][i] * si[i], we[0][i + 1] * si[i + 1]);
          }
#pragma unroll
          for (int i = 0; i < Raw<T>::kWords; ++i) mask[0][i] = mask[1][i] = partners ? 0xFFFFFFFFu : 0u;
        } else {
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < kVec; i += 2) {
              // rot_dim is even: both of two consecutive elements turn, or neither
              const bool turns = e[c] + i < a.rope.rot_dim;
              float own2[2] = {we[c][i], we[c][i + 1]}, theirs2[2] = {0.0f, 0.0f};
              if (turns) {
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                  const int el = e[c] + i + b, j = pair_of(el);
                  const bool first = kPairing == kNeighbour ? b == 0 : el < half;
                  const float si = sh_sin[warp][j];
                  own2[b] *= sh_cos[warp][j];
                  theirs2[b] = w[partner_of(el)] * (first ? -si : si);
                }
              }
              own[c][i / 2] = pk2(own2[0], own2[1]);
              theirs[c][i / 2] = pk2(theirs2[0], theirs2[1]);
              if (sizeof(T) == 2)
                mask[c][i / 2] = turns ? 0xFFFFFFFFu : 0u;
              else
                mask[c][i % Raw<T>::kWords] = mask[c][(i + 1) % Raw<T>::kWords] = turns ? 0xFFFFFFFFu : 0u;
            }
        }
      }
      walk(src, p, [&](Raw<T> (&raw)[2], bool live) {
        uint64_t x[2][kVec / 2];
        raw[0].get(x[0]);
        raw[1].get(x[1]);
        uint64_t inv2 = pk2(1.0f, 1.0f);
        if (weight) {
          uint64_t s2[2] = {fmul2_rn(x[0][0], x[0][0]), fmul2_rn(x[1][0], x[1][0])};
#pragma unroll
          for (int i = 1; i < kVec / 2; ++i)
#pragma unroll
            for (int c = 0; c < 2; ++c) s2[c] = ffma2_rn(x[c][i], x[c][i], s2[c]);
          float ss, s1;
          upk2(fadd2_rn(s2[0], s2[1]), ss, s1);
          ss += s1;
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          const float inv = rsqrtf(fmaf(ss, inv_dim, a.eps));
          inv2 = pk2(inv, inv);
        }
        if (half > 0) {
          uint64_t y[2][kVec / 2];
          const bool partial = 2 * half < a.head_dim;   // then some values take no part, and must
                                                        // not meet B = 0 as infinities
          Raw<T> other[2];
          if (kPairing == kHalves) {
            other[0] = raw[1], other[1] = raw[0];
          } else if (kPairing == kNeighbour) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int i = 0; i < Raw<T>::kWords; ++i)
                other[c].w[i] =
                    sizeof(T) == 2 ? __byte_perm(raw[c].w[i], 0, 0x1032) : raw[c].w[(i ^ 1) % Raw<T>::kWords];
          } else {
            T* row = sh_row + (kPairing == kThroughShared ? (threadIdx.x - lane) * 2 * kVec : 0);
            raw[0].store(row + e[0]);
            raw[1].store(row + e[1]);
            __syncwarp();
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              T mine[kVec];
#pragma unroll
              for (int i = 0; i < kVec; ++i) mine[i] = row[e[c] + i < a.rope.rot_dim ? partner_of(e[c] + i) : 0];
#pragma unroll
              for (int i = 0; i < Raw<T>::kWords; ++i) other[c].w[i] = reinterpret_cast<const uint32_t*>(mine)[i];
            }
            __syncwarp();
          }
          if (kPairing == kHalves && !partial) {
#pragma unroll
            for (int i = 0; i < kVec / 2; ++i) y[0][i] = x[1][i], y[1][i] = x[0][i];
          } else {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              if (partial) {
#pragma unroll
                for (int i = 0; i < Raw<T>::kWords; ++i) other[c].w[i] &= mask[c][i];
              }
              other[c].get(y[c]);
            }
          }
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < kVec / 2; ++i) x[c][i] = ffma2_rn(y[c][i], theirs[c][i], fmul2_rn(x[c][i], own[c][i]));
        } else {
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < kVec / 2; ++i) x[c][i] = fmul2_rn(x[c][i], own[c][i]);
        }
        if (weight) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < kVec / 2; ++i) x[c][i] = fmul2_rn(x[c][i], inv2);
        }
        Raw<T> out[2];
        out[0].put(x[0]);
        out[1].put(x[1]);
        store(out, live);
      });
    };

    if (a.q.heads > 0) {
      T* q = row_of(a.q_out.data, t * a.q_out.token_ld, a.q_out.head_ld);
      const int64_t step = stride * a.q_out.head_ld;
      turn_heads(a.q, from, a.q_weight, sh_w[0], [&](const Raw<T> (&y)[2], bool live) {
        if (live) put_row(q, y);
        q += step;
      });
      from = start(a.k);
    }
    {
      T* k = a.k_out.data ? row_of(a.k_out.data, t * a.k_out.token_ld, a.k_out.head_ld) : nullptr;
      T* c = cache_row >= 0 ? row_of(a.cache.k, cache_row, a.cache.head_ld) : nullptr;
      const int64_t step = stride * a.k_out.head_ld, c_step = stride * a.cache.head_ld;
      turn_heads(a.k, from, a.k_weight, sh_w[1], [&](const Raw<T> (&y)[2], bool live) {
        if (live && a.k_out.data) put_row(k, y);
        if (live && cache_row >= 0) put_row(c, y);
        k += step, c += c_step;
      });
    }
    if (a.cache.k) {
      T* c = cache_row >= 0 ? row_of(a.cache.v, cache_row, a.cache.head_ld) : nullptr;
      const int64_t c_step = stride * a.cache.head_ld;
      walk(a.v, start(a.v), [&](const Raw<T> (&y)[2], bool live) {
        if (live && cache_row >= 0) put_row(c, y);
        c += c_step;
      });
    }
    __syncwarp();   // the cosines may be written again
    unit += warps;
    from = start_unit();
  }
}

template <typename T, int kLanes, int kPairing>
cudaError_t launch_pairing(const HeadsArgs& a, cudaStream_t st) {
  const int64_t warps = static_cast<int64_t>(kBlocksPerSm) * num_sms() * kWarps;
  // A token's heads are divided only as far as that leaves no warp a second unit, and down
  // to one row per group: every share computes the cosines again, and a few units in a second
  // turn double the time (1237 tokens in two shares: 12.3 us, whole 10.7).
  const int64_t most = ceil_div(std::max({a.q.heads, a.k.heads, 1}), 32 / kLanes);
  const int64_t shares = std::max<int64_t>(1, std::min<int64_t>(most, warps / a.tokens));
  const int64_t blocks = std::min<int64_t>(ceil_div(a.tokens * shares, kWarps), warps / kWarps);
  return launch_behind(heads_kernel<T, kLanes, kPairing>, dim3(static_cast<unsigned>(blocks)), kThreads, 0, st, a,
                       static_cast<int>(shares));
}

template <typename T, int kLanes>
cudaError_t launch_lanes(const HeadsArgs& a, cudaStream_t st) {
  if (a.rope.interleaved) return launch_pairing<T, kLanes, kNeighbour>(a, st);
  if (a.rope.rot_dim / 2 % kVec == 0) return launch_pairing<T, kLanes, kHalves>(a, st);
  return launch_pairing<T, kLanes, kThroughShared>(a, st);
}

template <typename T>
cudaError_t launch_type(const HeadsArgs& a, cudaStream_t st) {
  if (a.head_dim <= 64) return launch_lanes<T, 4>(a, st);
  if (a.head_dim <= 128) return launch_lanes<T, 8>(a, st);
  return launch_lanes<T, 16>(a, st);
}

}  // namespace

cudaError_t launch_heads(const HeadsArgs& a, svdq_dtype dtype, cudaStream_t stream) {
  return dtype == SVDQ_BF16 ? launch_type<__nv_bfloat16>(a, stream) : launch_type<float>(a, stream);
}

}  // namespace svdq
