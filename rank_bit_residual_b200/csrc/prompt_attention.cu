// prompt_attention.cu - attention over packed prompts (svdq_attention_prompt).
//
//   out = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale q . k_j - m),   m = the running maximum
//
// One pass over the keys with a running maximum and sum. A block works on an item of two
// tiles of 128 rows that share their keys: consecutive rows of a sequence, each with the
// heads of a key head's group (the largest power of two of them) side by side. Per tile
// and 64 keys, S = Q K^T goes to tensor memory, four warps (one row per thread, so row
// maxima and sums need no exchange) turn it into P = 2^(S c - m) in bf16 and put it back
// over S, and O += P V accumulates in tensor memory with P as the operand from there. Each
// tile has two S buffers: the products of the next 64 keys run while softmax works on
// these. (With one buffer of 128 keys, softmax waited for P V and the next S in turn: 3400
// cycles per 128 keys of both tiles against 2048 of products.)
//
// With 128-element heads a row tile and 128 keys cost 1280 cycles of products (S in two parts
// of 64 keys 768, P V 512) and 1024 of exponentials at 16 a cycle, 768 of them left after the
// quarter that the FMA pipe takes, so both bound the kernel.
//
// P is rounded to bf16 because the product takes two operands of one 16-bit type and V is bf16:
// at most 2^-8 of sum p |v| / sum p, as much as the rounding of the result. The sums of the
// weights take the unrounded fp32 values.
//
// The maximum is renewed (and O rescaled, by the softmax warps themselves) only when a
// score passes it by 2^8; P then stays below 2^8, and both sums are fp32. O is at rest for
// that once the products of the next S are complete, because products run in order and
// that S follows P V of the keys before these.
//
// Warps: 0-3 and 4-7 softmax and output of the two tiles, 8 and 11 their products, 9 the loads and the
// choice of items (blocks that have not started are taken over, so that long and short
// items balance), 10 cleans values: in tiles that hold a key some row does not see,
// rows behind the sequence's end become zero, and infinities and NaN too (a zero weight
// must not meet them); the latter are added at the end to the rows that do see them.
//
// Few rows over many keys would leave most SMs idle: the keys of an item are then divided
// among several items, whose unfinished sums a second kernel joins (301 rows over 7501 keys,
// 40 items: 102 us with one share, 53 with three).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "encode.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace svdq {

namespace {

constexpr int kRows = 128;      // query rows of a tile
constexpr int kKeys = 128;      // keys of a loaded tile
constexpr int kPart = 64;       // keys of a part: what softmax takes at a time
constexpr int kThreads = 384;
constexpr int kMaxFold = 5;     // 32 heads in a tile: a warp's rows
constexpr int kMaxShares = 8;   // items that divide an item's keys
constexpr int kItems = 4;       // items between the chooser and the slowest reader

struct PromptArgs {
  svdq_heads q, k, v, out;
  const int32_t* cu_q;
  const int32_t* cu_k;
  int batch;
  int64_t q_tokens, k_tokens;
  int dim, causal;
  int fold;         // log2 of the heads that lie side by side in a tile
  int pairs;        // items per row range: heads >> fold
  int shares;       // items that divide an item's keys
  int group;        // query heads per key head
  float* partial;   // with several shares: [item][share][tile] sums [dim][128], maxima [128], totals [128]
  float scale_log2;
  unsigned* status;
};

struct Item {
  int valid;        // 0: no more
  int keys, k0;     // keys of the sequence and their first row
  int kvh;
  int n[2];         // parts of each row tile
  int cut;          // first loaded tile with a key that some row does not see
  int row[2];       // first row in q and out
  int rows[2];      // rows inside the sequence, 0 .. 128 >> fold
  int head;         // the first
  int seen[2];      // keys that the tile's first row sees (causal; row r sees r more)
  int index;        // of the item and its share
};

// Start of sequence s (no list: one sequence of all rows).
__device__ __forceinline__ long long cu_at(const int32_t* cu, int s, long long tokens) {
  if (!cu) return s == 0 ? 0 : tokens;
  return max(0ll, min(static_cast<long long>(cu[s]), tokens));
}

__device__ __forceinline__ bool bad_cu(const int32_t* cu, int s, long long tokens) {
  return cu && (cu[s] < 0 || cu[s + 1] < cu[s] || cu[s + 1] > tokens);
}

// 32 sequences of the line, one per lane.
struct Window {
  int first = -32;          // sequence of lane 0; below 0: nothing loaded yet
  int before = 0;           // row ranges of the sequences in front
  int q0, rows, k0, keys;   // first rows and counts
  int n, upto;              // row ranges, and those of the lanes up to this one
};

__device__ __forceinline__ void load_window(const PromptArgs& a, int first, int before, Window& w) {
  const int lane = threadIdx.x & 31, s = first + lane;
  w.first = first, w.before = before;
  w.q0 = w.rows = w.k0 = w.keys = w.n = 0;
  if (s < a.batch) {
    w.q0 = static_cast<int>(cu_at(a.cu_q, s, a.q_tokens));
    w.rows = max(0, static_cast<int>(cu_at(a.cu_q, s + 1, a.q_tokens)) - w.q0);
    w.k0 = static_cast<int>(cu_at(a.cu_k, s, a.k_tokens));
    w.keys = max(0, static_cast<int>(cu_at(a.cu_k, s + 1, a.k_tokens)) - w.k0);
    w.n = (w.rows + (2 * kRows >> a.fold) - 1) >> (8 - a.fold);   // of 256 >> fold rows
  }
  w.upto = w.n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, w.upto, o);
    if (lane >= o) w.upto += up;
  }
}

// Item `index` of the line: row ranges of all sequences, each with its `pairs` heads. The
// whole warp calls it; valid = 0 past the last range. A block's items come in order, so the
// window of the last one is kept, and moves on only when it must (from the
// start each time, 6000 sequences of 7 rows took 42.6 ms instead of 2.8).
__device__ Item find_item(const PromptArgs& a, int index, Window& w) {
  const int lane = threadIdx.x & 31;
  // every index of the grid passes here, and there are at least as many as sequences
  if (index < a.batch && lane == 0 && (bad_cu(a.cu_q, index, a.q_tokens) || bad_cu(a.cu_k, index, a.k_tokens)))
    record_status(a.status, kStatusEinval);
  const int whole = a.shares == 1 ? index : index / a.shares, part = index - whole * a.shares;
  const int range = whole / a.pairs, pair = whole - range * a.pairs;
  Item it;
  it.valid = 0;
  it.index = index;
  if (w.first < 0 || range < w.before) load_window(a, 0, 0, w);
  while (true) {
    const int before = w.before, n = w.n, incl = w.upto;
    const unsigned hit = __ballot_sync(0xffffffffu, before + incl > range);
    if (hit != 0) {
      int src = __ffs(hit) - 1;
      // Ranges far down a causal sequence see the most keys and go first: of one sequence
      // among many, or, when a warp holds all sequences, of all of them, so that the last items
      // to start are the short ones.
      int place = __shfl_sync(0xffffffffu, n - 1 - (range - before - (incl - n)), src);
      if (a.batch > 1 && a.batch <= 32) {
        // the farthest place with more than `range` ranges at it or behind it
        int end = __reduce_max_sync(0xffffffffu, n), skipped = 0;   // ranges at `end` or behind it
        place = 0;
        while (end - place > 1) {
          const int middle = (place + end) / 2;
          const int behind = __reduce_add_sync(0xffffffffu, max(0, n - middle));
          if (behind > range)
            place = middle;
          else
            end = middle, skipped = behind;
        }
        unsigned has = __ballot_sync(0xffffffffu, n > place);   // sequences that reach this place
        for (int i = range - skipped; i > 0; --i) has &= has - 1;
        src = __ffs(has) - 1;
      }
      const int q0 = __shfl_sync(0xffffffffu, w.q0, src), rows = __shfl_sync(0xffffffffu, w.rows, src);
      int k0 = __shfl_sync(0xffffffffu, w.k0, src), keys = __shfl_sync(0xffffffffu, w.keys, src);
      it.valid = 1;
      it.head = pair << a.fold;
      int last = 0;   // keys that any row sees
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int row = (2 * place + t) * (kRows >> a.fold);
        it.row[t] = q0 + row;
        it.rows[t] = max(0, min(kRows >> a.fold, rows - row));
        it.seen[t] = a.causal ? keys - rows + row + 1 : keys;
        if (it.rows[t] > 0) last = max(last, a.causal ? min(keys, it.seen[t] + it.rows[t] - 1) : keys);
      }
      if (a.shares > 1) {   // this share's keys become the item's own
        const int tiles = (last + kKeys - 1) / kKeys;
        const int from = tiles * part / a.shares * kKeys, to = tiles * (part + 1) / a.shares * kKeys;
        k0 += from;
        keys = min(keys, to) - from;
        it.seen[0] -= from, it.seen[1] -= from;
      }
      it.keys = keys, it.k0 = k0;
      it.cut = 0x7FFFFFFF;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int end = a.causal ? min(keys, it.seen[t] + it.rows[t] - 1) : keys;
        it.n[t] = it.rows[t] > 0 ? max(0, end + kPart - 1) / kPart : 0;
        it.cut = min(it.cut, max(0, min(keys, it.seen[t])) / kKeys);
      }
      it.kvh = it.head / a.group;
      return it;
    }
    if (w.first + 32 >= a.batch) return it;
    load_window(a, w.first + 32, before + __shfl_sync(0xffffffffu, incl, 31), w);
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float max3_nan(float x, float y, float z) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}

// 2^x of a pair on the FMA pipe, for x from -126 (and below, as -126) to 126: x = n + f with n
// the nearest integer (added and subtracted 1.5 * 2^23 leaves it in the low bits), 2^f on
// [-1/2, 1/2] by the cubic of least maximal relative error (7.5e-5, from an exchange
// iteration; bf16 rounds to 2^-9 afterwards), and n added to the exponent.
__device__ __forceinline__ uint64_t exp2_poly(uint64_t x) {
  constexpr float kShift = 12582912.0f;
  float lo, hi;
  upk2(x, lo, hi);
  x = pk2(fmaxf(lo, -126.0f), fmaxf(hi, -126.0f));
  const uint64_t r = fadd2_rn(x, pk2(kShift, kShift));
  const uint64_t f = fsub2_rn(x, fsub2_rn(r, pk2(kShift, kShift)));
  uint64_t p = ffma2_rn(pk2(0.05517167f, 0.05517167f), f, pk2(0.24261112f, 0.24261112f));
  p = ffma2_rn(p, f, pk2(0.69326099f, 0.69326099f));
  p = ffma2_rn(p, f, pk2(0.99992807f, 0.99992807f));
  float nl, nh, pl, ph;
  upk2(r, nl, nh);
  upk2(p, pl, ph);
  return pk2(__uint_as_float((__float_as_uint(nl) << 23) + __float_as_uint(pl)),
             __uint_as_float((__float_as_uint(nh) << 23) + __float_as_uint(ph)));
}

// The bf16 pair of a word, infinities and NaN replaced by zero.
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t w) {
  if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
  if ((w & 0x7F800000u) == 0x7F800000u) w &= 0xFFFFu;
  return w;
}

// Floats of an unfinished row tile: sums, maxima and totals.
template <int kDim>
__host__ __device__ constexpr int partial_floats() {
  return (kDim + 2) * kRows;
}

template <int kDim>
struct Shape {
  static constexpr int kTile = kKeys * kDim * 2;         // bytes of 128 rows of a head
  static constexpr int kRing = kDim == 128 ? 4 : 10;     // tiles of keys and values in flight
  static constexpr int kSmem = 2 * kTile + kRing * kTile + 8 * 4096 + 1024;   // and 32 rows of 64 outputs per warp
  static constexpr int kPoly = kDim == 128 ? 2 : 3;      // pairs of eight whose exponentials go to the FMA pipe
  static constexpr int kO = 256;                         // tensor memory columns: S0, S1, O0, O1
};

template <int kRing>
struct Barriers {
  uint64_t q_full, q_empty;
  uint64_t full[kRing], empty[kRing];
  uint64_t raw[kRing];   // loaded, for the cleaning warp, which then completes `full`
  uint64_t s_full[2][2], p_full[2][2], o_full[2];   // by row tile and buffer
  uint64_t item_full[kItems], item_empty[kItems];
  uint64_t answer;
};

// A ring position and its phase.
template <int kN>
struct Turn {
  int i = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++i == kN) i = 0, phase ^= 1;
  }
};

// kShared: the keys of an item are divided, and its sums stay unfinished.
template <int kDim, bool kShared>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v, const __grid_constant__ PromptArgs a) {
  using Sz = Shape<kDim>;
  extern __shared__ unsigned char smem_raw[];
  __shared__ Barriers<Sz::kRing> bar;
  __shared__ Item items[kItems];
  __shared__ int odd[2 * kItems];        // by item number (from 1): the number, if values were taken out
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  __shared__ __align__(16) uint4 answer;

  unsigned char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  unsigned char* sq = smem;              // two tiles of Q
  unsigned char* ring = smem + 2 * Sz::kTile;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  volatile int* abort = &abort_flag;

  if (threadIdx.x == 0) {
    abort_flag = 0;
    mbar_init(&bar.q_full, 1);
    mbar_init(&bar.q_empty, 2);
    for (int i = 0; i < Sz::kRing; ++i) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.empty[i], 2);
      mbar_init(&bar.raw[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(&bar.s_full[t][b], 1);
        mbar_init(&bar.p_full[t][b], 4);
      }
      mbar_init(&bar.o_full[t], 1);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&bar.item_full[i], 1);
      mbar_init(&bar.item_empty[i], 11);   // 8 softmax warps, 2 for the products, the cleaning warp
      odd[i] = odd[kItems + i] = 0;
    }
    mbar_init(&bar.answer, 1);
    fence_mbar_init();
    tma_prefetch_desc(&map_q);
    tma_prefetch_desc(&map_k);
    tma_prefetch_desc(&map_v);
  }
  if (warp == 8) {
    tmem_alloc(&tmem_base, 512);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  __syncwarp();   // .aligned instructions follow in every role

  if (warp >= 8) {
    if (warp == 9) {
      // ---------------------------------------------------------- items and loads
      Turn<kItems> slot;
      Turn<Sz::kRing> r;
      uint32_t q_phase = 0, answer_phase = 0, last_raw = 0, raw_phase = 0;   // the last two by ring position
      int index = blockIdx.x;
      Window window;
      bool ok = true;
      while (ok) {
        // ask for the next item while this one is worked on
        if (lane == 0 && index >= 0) {
          mbar_arrive_expect_tx(&bar.answer, 16);
          block_request(&answer, &bar.answer);
        }
        Item it;
        it.valid = 0;
        if (index >= 0) it = find_item(a, index, window);
        if (index < 0 || it.valid) {
          ok = mbar_wait_warp(&bar.item_empty[slot.i], slot.phase ^ 1, a.status, abort);
          if (ok && lane == 0) {
            items[slot.i] = it;
            mbar_arrive(&bar.item_full[slot.i]);
          }
          slot.next();
        }
        if (index < 0) break;
        const int n = it.valid ? (max(it.n[0], it.n[1]) + 1) / 2 : 0;   // tiles of two parts
        if (ok && n > 0 && lane == 0) {
          ok = mbar_wait_soon(&bar.q_empty, q_phase ^ 1, a.status, abort);
          q_phase ^= 1;
          if (ok) {
            mbar_arrive_expect_tx(&bar.q_full, 2 * Sz::kTile);
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int c = 0; c < kDim / 64; ++c)
                tma_load_3d(sq + t * Sz::kTile + c * kRows * 128, &map_q, &bar.q_full, c * 64, it.head, it.row[t]);
          }
          for (int j = 0; ok && j < 2 * n; ++j) {   // K0, V0, K1, V1, ...
            ok = mbar_wait_soon(&bar.empty[r.i], r.phase ^ 1, a.status, abort);
            if (!ok) break;
            const bool raw = (j & 1) && (j >> 1) >= it.cut;
            uint64_t* to = raw ? &bar.raw[r.i] : &bar.full[r.i];
            last_raw = (last_raw & ~(1u << r.i)) | (raw ? 1u << r.i : 0u);
            if (raw) raw_phase ^= 1u << r.i;
            mbar_arrive_expect_tx(to, Sz::kTile);
#pragma unroll
            for (int c = 0; c < kDim / 64; ++c)
              tma_load_3d(ring + r.i * Sz::kTile + c * kKeys * 128, (j & 1) ? &map_v : &map_k, to, c * 64, it.kvh,
                          it.k0 + (j >> 1) * kKeys);
            r.next();
          }
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        int got = -1;
        if (lane == 0) {
          // also on an abort: the answer must have landed before the block ends
          if (mbar_wait(&bar.answer, answer_phase, a.status, nullptr)) got = block_answer(&answer);
          fence_proxy_async_smem();
        }
        answer_phase ^= 1;
        index = __shfl_sync(0xffffffffu, got, 0);
      }
      // nothing may still be in flight when the block ends
      if (lane == 0 && *abort) {
        mbar_wait(&bar.q_full, q_phase ^ 1, a.status, nullptr);
        Turn<Sz::kRing> w = r;
        for (int i = 0; i < Sz::kRing; ++i) {
          if ((last_raw >> w.i) & 1)
            mbar_wait(&bar.raw[w.i], ((raw_phase >> w.i) & 1) ^ 1, a.status, nullptr);
          else
            mbar_wait(&bar.full[w.i], w.phase ^ 1, a.status, nullptr);
          w.next();
        }
      }
    } else if (warp == 8 || warp == 11) {
      // ------------------------------------------------------------------ products
      // One warp for each row tile, so that one's waits do not hold up the other's products.
      // The whole warp walks through this part and one lane issues; what the instructions
      // take is broadcast from lane 0, so that the compiler keeps it in uniform registers
      // (an instruction whose operands it has to move there first takes about 60 cycles
      // to issue, as long as it takes to run).
      auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
      constexpr uint32_t idesc_o = idesc_bf16_bmn(kRows, kDim);
      // a negative scale negates Q in the product (bit 13), so that softmax sees a positive one
      const uint32_t idesc_s = idesc_bf16(kRows, kPart) | (a.scale_log2 < 0.0f ? 1u << 13 : 0u);
      const int t = warp == 8 ? 0 : 1;
      const uint32_t tm = uniform(tmem);
      const uint32_t q0 = uniform(smem_u32(sq)) + t * Sz::kTile, ring0 = uniform(smem_u32(ring));
      const uint32_t ts = tm + t * kKeys, to = tm + Sz::kO + t * kDim;
      const bool leader = elect_one() != 0;
      Turn<kItems> slot;
      Turn<Sz::kRing> r;
      uint32_t q_phase = 0, p_phase = 0;   // the latter with a bit per buffer
      bool ok = true;
      auto commit = [&](uint64_t* b) {
        if (leader) mma_commit(b);
        __syncwarp();
      };
      // S of part i, from the keys in ring position buf
      auto scores = [&](int i, int buf) {
        const uint64_t qd = smem_desc_sw128(q0);
        const uint64_t kd = smem_desc_sw128(ring0 + buf * Sz::kTile + (i & 1) * (kPart * 128));
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < kDim / 16; ++kk) {
            const uint64_t off = ((kk >> 2) * (kRows * 128) + (kk & 3) * 32) >> 4;
            mma_f16(ts + (i & 1) * kPart, qd + off, kd + off, idesc_s, kk > 0);
          }
          mma_commit(&bar.s_full[t][i & 1]);
        }
        __syncwarp();
      };
      while (true) {
        if (!mbar_wait_soon_warp(&bar.item_full[slot.i], slot.phase, a.status, abort)) break;
        const int valid = uniform(items[slot.i].valid);
        const int n = uniform(items[slot.i].n[t]);                                // parts of this tile
        const int both = uniform(max(items[slot.i].n[0], items[slot.i].n[1]));   // parts that are loaded
        if (leader) mbar_arrive(&bar.item_empty[slot.i]);
        __syncwarp();
        slot.next();
        if (!valid) break;
        if (both == 0) continue;
        ok = mbar_wait_soon_warp(&bar.q_full, q_phase, a.status, abort) &&
             mbar_wait_soon_warp(&bar.full[r.i], r.phase, a.status, abort);
        q_phase ^= 1;
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (i < n) scores(i, r.i);
        commit(&bar.empty[r.i]);
        if (both <= 2) commit(&bar.q_empty);
        r.next();
        int vbuf = 0, kbuf = 0;
        for (int i = 0; i < both; ++i) {
          if ((i & 1) == 0) {
            vbuf = r.i;
            ok = mbar_wait_soon_warp(&bar.full[vbuf], r.phase, a.status, abort);
            r.next();
            if (ok && i + 2 < both) {
              kbuf = r.i;
              ok = mbar_wait_soon_warp(&bar.full[kbuf], r.phase, a.status, abort);
              r.next();
            }
            if (!ok) break;
          }
          if (i < n) {
            ok = mbar_wait_soon_warp(&bar.p_full[t][i & 1], (p_phase >> (i & 1)) & 1, a.status, abort);
            if (!ok) break;
            p_phase ^= 1u << (i & 1);
            tc_fence_after();
            const uint64_t vd = smem_desc_sw128_mn(ring0 + vbuf * Sz::kTile + (i & 1) * (kPart * 128), kKeys * 128);
            if (leader) {
#pragma unroll
              for (int kk = 0; kk < kPart / 16; ++kk)
                mma_f16_ta(to, ts + (i & 1) * kPart + kk * 8, vd + ((kk * 2048) >> 4), idesc_o, i > 0 || kk > 0);
              if (i == n - 1) mma_commit(&bar.o_full[t]);
              // in the place of the S that would come next: O is at rest for the last part
              if (i == n - 2) mma_commit(&bar.s_full[t][i & 1]);
            }
            __syncwarp();
            if (i + 2 < n) scores(i + 2, kbuf);
          }
          if ((i & 1) == 1 || i == both - 1) commit(&bar.empty[vbuf]);
          if (i + 2 < both && ((i & 1) == 1 || i + 3 == both)) commit(&bar.empty[kbuf]);
          if (i + 3 == both) commit(&bar.q_empty);
        }
        if (!ok) break;
      }
    } else if (warp == 10) {
      // ----------------------------------------------------------------- cleaning
      Turn<kItems> slot;
      Turn<Sz::kRing> r;
      int number = 0;
      uint32_t raw_phase = 0;              // by ring position
      while (true) {
        if (!mbar_wait_warp(&bar.item_full[slot.i], slot.phase, a.status, abort)) break;
        const Item it = items[slot.i];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.item_empty[slot.i]);
        slot.next();
        if (!it.valid) break;
        ++number;
        const int n = (max(it.n[0], it.n[1]) + 1) / 2;
        bool ok = true;
        for (int j = 0; ok && j < n; ++j) {
          r.next();                        // the keys
          if (j >= it.cut) {
            ok = mbar_wait_warp(&bar.raw[r.i], (raw_phase >> r.i) & 1, a.status, abort);
            if (!ok) break;
            raw_phase ^= 1u << r.i;
            // 16-byte pieces in memory order: 8 to a row of 64 elements, whatever the swizzle
            uint4* piece = reinterpret_cast<uint4*>(ring + r.i * Sz::kTile);
            const int inside = min(kKeys, it.keys - j * kKeys);   // rows of this sequence
            for (int c = 0; c < kDim / 64; ++c)
              for (int i = inside * 8 + lane; i < kKeys * 8; i += 32) piece[c * kKeys * 8 + i] = make_uint4(0, 0, 0, 0);
            __syncwarp();
            // an exponent of all ones carries into the sign bit
            constexpr int kBatch = 8;
            uint32_t carried = 0;
            for (int i = lane; i < Sz::kTile / 16; i += 32 * kBatch) {
              uint4 x[kBatch];
#pragma unroll
              for (int b = 0; b < kBatch; ++b) x[b] = piece[i + 32 * b];
#pragma unroll
              for (int b = 0; b < kBatch; ++b)
                carried |= ((x[b].x & 0x7F807F80u) + 0x00800080u) | ((x[b].y & 0x7F807F80u) + 0x00800080u) |
                           ((x[b].z & 0x7F807F80u) + 0x00800080u) | ((x[b].w & 0x7F807F80u) + 0x00800080u);
            }
            if (__any_sync(0xffffffffu, (carried & 0x80008000u) != 0)) {   // hardly ever
              for (int i = lane; i < Sz::kTile / 16; i += 32) {
                const uint4 x = piece[i];
                piece[i] = make_uint4(finite_or_zero(x.x), finite_or_zero(x.y), finite_or_zero(x.z), finite_or_zero(x.w));
              }
              odd[number % (2 * kItems)] = number;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.full[r.i]);
          }
          r.next();
        }
        if (!ok) break;
      }
    }
  } else {
    // ------------------------------------------------------------ softmax and output
    const int t = warp >> 2;
    const int row = (warp & 3) * 32 + lane;   // of the tile
    const int down = row >> a.fold;           // of the sequence, from the tile's first
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t to = tmem + lanes + Sz::kO + t * kDim;
    // The product takes the sign. A scale of zero is one so small that all weights are 1, and
    // a masked -inf still comes out as a weight of 0.
    const float scale = fmaxf(fabsf(a.scale_log2), 1e-30f);
    Turn<kItems> slot;
    uint32_t s_phase = 0, o_phase = 0;   // the former with a bit per buffer
    int number = 0;
    while (true) {
      if (!mbar_wait_warp(&bar.item_full[slot.i], slot.phase, a.status, abort)) break;
      // only what the loop needs is kept over it (its registers are full); the rest of the item
      // is read behind it
      const Item& it = items[slot.i];
      if (!it.valid) break;
      const int n = it.n[t];
      const int all_see = min(it.keys, it.seen[t]);
      ++number;
      float m = -INFINITY;
      uint64_t sums[2] = {0, 0};   // two pairs of partial sums
      bool ok = true;
      // S of the next part was complete in time: its first half is being loaded already. (A
      // wait takes some 200 cycles even when there is nothing to wait for.)
      bool ahead = false;
      uint32_t s[2][32];
      for (int j = 0; j < n; ++j) {
        const int buf = j & 1;
        const uint32_t ts = tmem + lanes + t * kKeys + buf * kPart;
        if (!ahead) {
          ok = mbar_wait_soon_warp(&bar.s_full[t][buf], (s_phase >> buf) & 1, a.status, abort);
          if (!ok) break;
          tc_fence_after();
          tmem_ld_32x32b_x32(ts, s[0]);
        }
        s_phase ^= 1u << buf;
        ahead = false;
        tmem_ld_wait_regs(s[0]);
        tmem_ld_32x32b_x32(ts + 32, s[1]);
        // weights of half a part with the maximum m; kPoly pairs of eight by polynomial
        auto weights = [&](int c, auto poly, uint64_t scale2, uint64_t base2, uint64_t (&add)[2]) {
          uint32_t p[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint64_t x =
                ffma2_rn(pk2(__uint_as_float(s[c][2 * i]), __uint_as_float(s[c][2 * i + 1])), scale2, base2);
            uint64_t e;
            float lo, hi;
            if (i % 8 >= 8 - decltype(poly)::value) {
              e = exp2_poly(x);
            } else {
              upk2(x, lo, hi);
              e = pk2(ex2(lo), ex2(hi));
            }
            add[i & 1] = fadd2_rn(add[i & 1], e);
            upk2(e, lo, hi);
            p[i] = pack_bf16(lo, hi);
          }
          tmem_st_32x32b_x16(ts + c * 16, p);
        };
        auto largest = [&](int c, float (&tops)[2]) {
#pragma unroll
          for (int i = 0; i < 32; i += 2)
            tops[(i >> 1) & 1] = max3_nan(tops[(i >> 1) & 1], __uint_as_float(s[c][i]), __uint_as_float(s[c][i + 1]));
        };
        const uint64_t scale2 = pk2(scale, scale);
        bool done = false;
        if (j > 0 && (j + 1) * kPart <= all_see) {
          // Most parts leave the maximum as it is: their weights are taken with it while their
          // own largest score is found, and taken again in the rare case that it is too large (or NaN).
          const uint64_t base2 = pk2(-m, -m);
          uint64_t add[2] = {sums[0], sums[1]};
          float tops[2] = {-INFINITY, -INFINITY};
          largest(0, tops);
          weights(0, std::integral_constant<int, Sz::kPoly>{}, scale2, base2, add);
          tmem_ld_wait_regs(s[1]);
          const bool there = j + 1 < n && mbar_test(&bar.s_full[t][buf ^ 1], (s_phase >> (buf ^ 1)) & 1);
          largest(1, tops);
          weights(1, std::integral_constant<int, Sz::kPoly>{}, scale2, base2, add);
          const float top = max3_nan(tops[0], tops[1], tops[1]) * scale;
          // Not where a row has seen nothing but -inf (m = -inf). Both forms say so; the compiler finds
          // better registers with the first for heads of 128 elements (512 sequences of 128 rows:
          // 286 us, with the second 310) and with the second for 64 (2 x 2048 rows: 117.5 us, with
          // the first 121).
          const bool small = kDim == 128 ? top <= m + 8.0f && m > -INFINITY : top - m <= 8.0f;
          // Rows behind the sequence's end hold whatever lies there and are never stored: they
          // decide nothing for the rows beside them in the warp.
          done = __all_sync(0xffffffffu, small || row >= it.rows[t] << a.fold);
          if (done) {
            sums[0] = add[0], sums[1] = add[1];
            ahead = __all_sync(0xffffffffu, there);
            if (ahead) {
              tc_fence_after();
              tmem_ld_32x32b_x32(ts ^ kPart, s[0]);
            }
          }
        } else {
          tmem_ld_wait_regs(s[1]);
        }
        if (!done) {
          const int left = (a.causal ? min(it.keys, it.seen[t] + down) : it.keys) - j * kPart;   // keys of this row
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (c * 32 + i >= left) s[c][i] = 0xFF800000u;   // -inf
          float tops[2] = {-INFINITY, -INFINITY};
          largest(0, tops);
          largest(1, tops);
          const float up = fmaxf(m, max3_nan(tops[0], tops[1], tops[1]) * scale);
          const float f = m == -INFINITY ? 0.0f : ex2(m - up);
          m = up;
          sums[0] = fmul2_rn(sums[0], pk2(f, f));
          sums[1] = fmul2_rn(sums[1], pk2(f, f));
          if (j > 0 && __any_sync(0xffffffffu, f != 1.0f)) {
            // O is at rest once the next S (or what stands for it) is complete
            ok = mbar_wait_soon_warp(&bar.s_full[t][buf ^ 1], (s_phase >> (buf ^ 1)) & 1, a.status, abort);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < kDim / 16; ++c) {
              uint32_t o[16];
              tmem_ld_32x32b_x16(to + c * 16, o);
              tmem_ld_wait_regs(o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tmem_st_32x32b_x16(to + c * 16, o);
            }
          }
          const float base = m == -INFINITY ? 0.0f : -m;
          weights(0, std::integral_constant<int, 0>{}, scale2, pk2(base, base), sums);
          weights(1, std::integral_constant<int, 0>{}, scale2, pk2(base, base), sums);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_full[t][buf]);
      }
      if (!ok) break;
      const int seen = a.causal ? min(it.keys, it.seen[t] + down) : it.keys;   // keys of this row
      const int k0 = it.k0, kvh = it.kvh, cut = it.cut, row0 = it.row[t], rows = it.rows[t] << a.fold, head = it.head;
      const int index = it.index;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.item_empty[slot.i]);
      slot.next();
      if (n >= 2) s_phase ^= 1u << (n & 1);   // what stood for the S after the last
      if (n > 0) {
        ok = mbar_wait_soon_warp(&bar.o_full[t], o_phase, a.status, abort);
        if (!ok) break;
        o_phase ^= 1;
        tc_fence_after();
      }
      float l4[4];
      upk2(sums[0], l4[0], l4[1]);
      upk2(sums[1], l4[2], l4[3]);
      const float l = (l4[0] + l4[1]) + (l4[2] + l4[3]);
      float inv = l == 0.0f ? 0.0f : 1.0f / l;
      float* partial = nullptr;
      if (kShared) {
        inv = 1.0f;
        partial = a.partial + (static_cast<long long>(index) * 2 + t) * partial_floats<kDim>() + row;
        partial[kDim * kRows] = m;
        partial[(kDim + 1) * kRows] = l;
      }
      const bool extra = n > 0 && odd[number % (2 * kItems)] == number;
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out.data) + row0 * a.out.token_ld + head * a.out.head_ld;
      if (extra) {   // hardly ever, so short rather than fast: the values taken out are added
        const __nv_bfloat16* vp = static_cast<const __nv_bfloat16*>(a.v.data) + kvh * a.v.head_ld;
        dst += down * a.out.token_ld + (row & ((1 << a.fold) - 1)) * a.out.head_ld;
#pragma unroll 1
        for (int c = 0; c < a.dim; c += 16) {
          uint32_t o[16];
          __syncwarp();
          tmem_ld_32x32b_x16(to + c, o);
          tmem_ld_wait_regs(o);
          if (row >= rows) continue;
          for (int key = cut * kKeys; key < seen; ++key)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float x = c + i < a.dim ? __bfloat162float(vp[(k0 + key) * a.v.token_ld + c + i]) : 0.0f;
              if (!isfinite(x)) o[i] = __float_as_uint(__uint_as_float(o[i]) + x);
            }
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (c + i >= a.dim) continue;
            if (kShared)
              partial[(c + i) * kRows] = __uint_as_float(o[i]);
            else
              dst[c + i] = __float2bfloat16_rn(__uint_as_float(o[i]) * inv);
          }
        }
        __syncwarp();
        tc_fence_before();
        continue;
      }
      unsigned char* stage = ring + Sz::kRing * Sz::kTile + warp * 4096;
      // Short code: a block runs through it once per item, so it waits for instructions (unrolled,
      // and with the rare case above in it, 1000 sequences of 30 rows took 277 us instead of 242).
#pragma unroll 1
      for (int pair = 0; pair < kDim / 64; ++pair)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int c = 2 * pair + half;
        uint32_t o[32];
        __syncwarp();
        if (n > 0) {
          tmem_ld_32x32b_x32(to + c * 32, o);
          tmem_ld_wait_regs(o);
        }
        if (kShared) {
#pragma unroll
          for (int i = 0; i < 32; ++i) partial[(c * 32 + i) * kRows] = n > 0 ? __uint_as_float(o[i]) : 0.0f;
          continue;
        }
        // A lane has a row; stored from there, one instruction would touch 32 lines. 64 columns
        // at a time go through shared memory, and 8 lanes store 128 bytes of a row.
        unsigned char* mine = stage + lane * 128;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t w[4];
#pragma unroll
          for (int b = 0; b < 4; ++b)
            w[b] = n > 0 ? pack_bf16(__uint_as_float(o[8 * i + 2 * b]) * inv, __uint_as_float(o[8 * i + 2 * b + 1]) * inv)
                         : 0u;
          *reinterpret_cast<uint4*>(mine + ((((c & 1) * 4 + i) ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if ((c & 1) == 0) continue;
        __syncwarp();
        const int col = (c - 1) * 32 + (lane & 7) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = i * 4 + (lane >> 3), at = (warp & 3) * 32 + r;   // of the warp, of the tile
          const uint4 v = *reinterpret_cast<const uint4*>(stage + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
          if (at < rows && col < a.dim)
            *reinterpret_cast<uint4*>(dst + ((at >> a.fold) * a.out.token_ld + (at & ((1 << a.fold) - 1)) * a.out.head_ld) +
                                      col) = v;
        }
      }
      tc_fence_before();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    __syncwarp();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the shares of one row tile: grid (items, 2, 4), a thread per row and eighth of the elements.
constexpr int kJoinThreads = 256;
template <int kDim>
__global__ void __launch_bounds__(kJoinThreads) prompt_join_kernel(const __grid_constant__ PromptArgs a) {
  __shared__ Item sh_item;
  if (threadIdx.x < 32) {
    Window window;
    const Item it = find_item(a, blockIdx.x * a.shares, window);
    if (threadIdx.x == 0) sh_item = it;
  }
  __syncthreads();
  pdl_wait();
  const int t = blockIdx.y, row = threadIdx.x % kRows, eighth = blockIdx.z * 2 + threadIdx.x / kRows;
  if (!sh_item.valid || row >= sh_item.rows[t] << a.fold) return;
  const int step = 2 * partial_floats<kDim>();   // from share to share
  const float* p = a.partial + (static_cast<long long>(blockIdx.x) * a.shares * 2 + t) * partial_floats<kDim>() + row;
  float top = -INFINITY;
  for (int s = 0; s < a.shares; ++s) top = fmaxf(top, p[s * step + kDim * kRows]);
  float weight[kMaxShares], total = 0.0f;
#pragma unroll
  for (int s = 0; s < kMaxShares; ++s) {
    const float m = s < a.shares ? p[s * step + kDim * kRows] : -INFINITY;
    weight[s] = m == -INFINITY ? 0.0f : exp2f(m - top);
    if (weight[s] != 0.0f) total = fmaf(weight[s], p[s * step + (kDim + 1) * kRows], total);
  }
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.out.data) +
                       (sh_item.row[t] + (row >> a.fold)) * a.out.token_ld +
                       (sh_item.head + (row & ((1 << a.fold) - 1))) * a.out.head_ld;
  for (int d = eighth * (kDim / 8); d < (eighth + 1) * (kDim / 8) && d < a.dim; d += 8) {
    float x[8] = {};
#pragma unroll
    for (int s = 0; s < kMaxShares; ++s)
      if (weight[s] != 0.0f) {   // a share that saw no key holds nothing
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = fmaf(weight[s], p[s * step + (d + i) * kRows], x[i]);
      }
    *reinterpret_cast<uint4*>(dst + d) =
        make_uint4(pack_bf16(x[0] * inv, x[1] * inv), pack_bf16(x[2] * inv, x[3] * inv),
                   pack_bf16(x[4] * inv, x[5] * inv), pack_bf16(x[6] * inv, x[7] * inv));
  }
}

// How an item is made up, and how many there are at most.
struct PromptPlan {
  int fold, pairs, shares;
  int64_t items;
};

PromptPlan plan_prompt(int heads, int kv_heads, int batch, int64_t q_tokens, int64_t k_tokens) {
  PromptPlan p;
  // Heads that share their keys lie side by side in a tile, a power of two of them: fewer rows
  // of the sequence then are in it, of which fewer lie behind its end or beside the diagonal
  // (32 on 8 heads, with one, two and all four of a group side by side: 9 ragged prompts 110, 94 and
  // 92 us, 1000 sequences of 30 rows 883, 458 and 248, 128 of 100 rows 152, 84 and 90).
  const int group = heads / kv_heads;
  for (p.fold = 0; p.fold < kMaxFold && group % (2 << p.fold) == 0;) ++p.fold;
  p.pairs = heads >> p.fold;
  p.items = (q_tokens / (2 * kRows >> p.fold) + batch) * p.pairs;
  // As many shares as fill the SMs once, each of a thousand keys or more on average: below
  // that the join takes what the shares gain.
  const int64_t fill = num_sms() / std::max<int64_t>(p.items, 1), keys = k_tokens / std::max(batch, 1) / 1024;
  p.shares = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({fill, keys, kMaxShares})));
  return p;
}

template <int kDim>
cudaError_t launch_dim(const PromptArgs& a, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                       int64_t items, cudaStream_t st) {
  constexpr int smem = Shape<kDim>::kSmem;
  auto* kernel = a.shares > 1 ? prompt_kernel<kDim, true> : prompt_kernel<kDim, false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kernel<<<static_cast<unsigned>(items * a.shares), kThreads, smem, st>>>(mq, mk, mv, a);
  e = cudaGetLastError();
  if (e != cudaSuccess || a.shares == 1) return e;
  return launch_behind(prompt_join_kernel<kDim>, dim3(static_cast<unsigned>(items), 2, 4), kJoinThreads, 0, st, a);
}

}  // namespace

size_t prompt_scratch_bytes(int heads, int kv_heads, int head_dim, int batch, int64_t q_tokens, int64_t k_tokens) {
  const PromptPlan p = plan_prompt(heads, kv_heads, batch, q_tokens, k_tokens);
  if (p.shares == 1) return 0;
  return static_cast<size_t>(p.items) * p.shares * 2 * sizeof(float) *
         (head_dim <= 64 ? partial_floats<64>() : partial_floats<128>());
}

cudaError_t launch_prompt(const svdq_heads& q, const svdq_heads& k, const svdq_heads& v, const int32_t* cu_q,
                          const int32_t* cu_k, int batch, int64_t q_tokens, int64_t k_tokens, int head_dim,
                          bool causal, float scale, const svdq_heads& out, void* scratch, cudaStream_t stream,
                          bool* bad_args) {
  const PromptPlan p = plan_prompt(q.heads, k.heads, batch, q_tokens, k_tokens);
  PromptArgs a{q, k, v, out, cu_q, cu_k, batch, q_tokens, k_tokens, head_dim, causal ? 1 : 0,
               p.fold, p.pairs, p.shares, q.heads / k.heads, static_cast<float*>(scratch), scale * 1.4426950408889634f,
               device_status_word()};
  CUtensorMap mq, mk, mv;
  // without any key no tile of k or v is ever loaded
  *bad_args = !make_tmap_heads(&mq, q, head_dim, q_tokens, kRows >> p.fold, 1u << p.fold) ||
              !make_tmap_heads(&mk, k_tokens > 0 ? k : q, head_dim, k_tokens > 0 ? k_tokens : q_tokens, kKeys) ||
              !make_tmap_heads(&mv, k_tokens > 0 ? v : q, head_dim, k_tokens > 0 ? k_tokens : q_tokens, kKeys);
  if (*bad_args) return cudaSuccess;
  return head_dim <= 64 ? launch_dim<64>(a, mq, mk, mv, p.items, stream)
                        : launch_dim<128>(a, mq, mk, mv, p.items, stream);
}

}  // namespace svdq
