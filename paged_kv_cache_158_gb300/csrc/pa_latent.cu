// Latent attention over a paged latent cache: the cache write of latent rows
// and single-token attention in absorbed form, on the sm_103a tensor cores.
//
// What is computed: a token's row r_i has 576 values, 512 latent and 64
// rotary; head h of sequence s has the query q (576 values, the key projection
// folded in) and
//   out[s][h] = sum_i p_i r_i[0:512],  p = softmax_{i < c_s}(scale * q . r_i),
// the ordinary attention formula ("vLLM推理加速深度解读：PagedAttention如何提升10x吞吐量"
// §2.1, through the block table of §2.3) with one key and one value for all
// heads.
//
// Bound: a token is 1152 bytes and 2 * 1088 flops a head.  With 64 heads that
// is 121 flops a byte, below the card's ratio (288 of measured peaks): HBM;
// with 128 heads 242: HBM and tensor cores together.
//
// Design (GB300):
//  * One persistent CTA per SM takes (64 heads) x (a range of 64-token tiles):
//    the batch's tiles, numbered sequence by sequence, are cut into equal
//    ranges, one for each worker, so ragged batches and single long contexts
//    alike load every SM to within a tile.  More than 64 heads: the CTAs of
//    one worker (one for each 64 heads) walk the same range at the same time,
//    so the rows come from HBM once and from L2 for the others.
//  * Worker w's part of sequence s is at most one segment; its partial result
//    (m, l, o) goes to slot s + w of the workspace (along the walk either s or
//    w grows, so the slots are distinct and there are at most S + W), and a
//    merge kernel joins a sequence's segments.  A sequence inside one range is
//    written directly.
//  * 64 heads are the rows of the products (M = 64) because of the memories:
//    the output of 128 heads x 512 fp32 would fill the tensor memory with no
//    room for logits, and 128 query rows the shared memory with no room for
//    two tiles.  With M = 64 an accumulator uses 16 of every 32 lanes: the
//    output's first 256 values sit in lanes 0-15 and the last 256 in lanes
//    16-31 of the same 256 columns.
//  * A tile is 64 rows of 576 values (nine 64-value swizzle atoms), copied by
//    TMA one box a block and atom into a two-stage ring; it is the K operand
//    of S = Q K^T (N = 64) and, its first eight atoms read the other way
//    round, the V operand of O += P V (N = 256, twice).
//  * Four softmax warps (one head row a lane) read S from tensor memory, keep
//    the running reference and sum in fp32 and write P, rounded once to fp16
//    (the sum adds the rounded weights), to shared memory.  The reference
//    moves only when the tile's maximum is more than 2^8 above it, so the
//    output in tensor memory is seldom rescaled.
//  * S is double-buffered: S(t+1) is computed while the softmax works on S(t).
#include <cuda.h>
#include <cuda_fp16.h>

#include <atomic>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_launch.cuh"
#include "pa_tensormap.cuh"
#include "pa_umma.cuh"

namespace pa {
namespace {

// ---- cache write ----------------------------------------------------------
// Thread i moves 16-byte vector i % 72 of token i / 72.  Bound: HBM, 2304
// bytes and a slot a token.

constexpr int kRowVecs = kLatentRow / 8, kLatVecs = kLatentDim / 8;

__global__ void __launch_bounds__(256)
    latent_write_kernel(const uint4* __restrict__ latent, long long latent_stride,
                        const uint4* __restrict__ rope, long long rope_stride,
                        uint4* __restrict__ cache, const int64_t* __restrict__ slot_mapping,
                        int num_tokens, long long num_slots, unsigned int* err) {
  pdl_wait();
  pdl_launch_dependents();
  const long long total = (long long)num_tokens * kRowVecs;
  const long long stride = (long long)gridDim.x * blockDim.x;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += stride) {
    const int t = (int)(i / kRowVecs);
    const int v = (int)(i - (long long)t * kRowVecs);
    const long long slot = slot_mapping[t];
    const uint4 x = v < kLatVecs ? latent[t * latent_stride + v] : rope[t * rope_stride + v - kLatVecs];
    if (slot < 0) continue;  // padding token
    if (slot >= num_slots) {
      if (v == 0) atomicOr(err, PA_ERRBIT_SLOT);
      continue;
    }
    cache[slot * kRowVecs + v] = x;
  }
}

// ---- decode -----------------------------------------------------------------

constexpr int kRows = 64;              // head rows of a CTA (MMA M)
constexpr int kTile = 64;              // tokens of a tile
constexpr int kAtoms = kLatentRow / 64;
constexpr int kAtomBytes = 64 * 128;   // 64 rows x 64 fp16
constexpr int kTileBytes = kAtoms * kAtomBytes;
constexpr int kThreads = 192;          // four softmax warps, TMA, MMA
constexpr int kSeqsPerLaunch = 1024;

constexpr int kOffQ = 0;
constexpr int kOffK = kTileBytes;      // stage s at kOffK + s * kTileBytes
constexpr int kOffP = 3 * kTileBytes;
constexpr int kOffBar = kOffP + kAtomBytes;
constexpr int kSmem = kOffBar + 256 + 1024;  // + alignment slack
static_assert(kSmem <= 232448, "beyond the opt-in shared memory of one CTA");

constexpr uint32_t kTmemCols = 512;    // O: [0, 256); S: 64 columns each
constexpr uint32_t kColS = 256;
constexpr uint32_t kLaneHi = 16u << 16;  // the output's upper 256 values

constexpr float kRescale = 8.f;        // base-2 logits above the reference that move it

struct LatentParams {
  void* out;
  const int32_t* block_tables;
  const int32_t* context_lens;
  float* ws_o;       // [slots][H][512]
  float2* ws_ml;     // [slots][H]
  int* cum;          // [S + 1] first tile of each sequence (for the merge)
  unsigned int* err;
  int seq_begin, num_seqs, num_heads, head_tiles, workers;
  int block_size, num_blocks, max_blocks, max_context_len;
  int oob_row;
  float scale_log2;
};

__device__ __forceinline__ int context_of(const LatentParams& a, int s, bool report) {
  int c = a.context_lens[a.seq_begin + s], e = 0;
  const long long cap = (long long)a.max_blocks * a.block_size;
  if (c < 0) { c = 0; e = 1; }
  if (c > cap) { c = (int)cap; e = 1; }
  if (c > a.max_context_len) { c = a.max_context_len; e = 1; }
  if (report && e) atomicOr(a.err, PA_ERRBIT_CONTEXT);
  return c;
}

__device__ __forceinline__ int tiles_of(int c) { return (c + kTile - 1) / kTile; }

// First tile of worker w of W over n tiles, and the worker of tile x.  No
// more workers take part than there are tiles, so every one of them has some.
__device__ __forceinline__ int active_workers(const LatentParams& a, int n) {
  return max(1, min(a.workers, n));
}
__device__ __forceinline__ int worker_begin(int w, int W, int n) {
  return (int)((long long)w * n / W);
}
__device__ __forceinline__ int worker_of(int x, int W, int n) {
  return (int)((((long long)x + 1) * W - 1) / n);
}

// A worker's walk over its range: the next sequence with tiles and the tiles
// of it that fall in the range.  Every warp role walks by itself.
struct Walk {
  int s, t, left;                // next sequence, its first tile, tiles left
  int c, n, t_begin, t_end;      // the current segment
  int cur;
  __device__ bool next(const LatentParams& a) {
    while (left > 0 && s < a.num_seqs) {
      cur = s;
      c = context_of(a, s, false);
      n = tiles_of(c);
      t_begin = t;
      t_end = min(n, t + left);
      ++s;
      t = 0;
      if (t_end > t_begin) {
        left -= t_end - t_begin;
        return true;
      }
    }
    return false;
  }
};

__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n"
      "  .reg .pred p;\n"
      "  mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      "  selp.u32 %0, 1, 0, p;\n"
      "}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Polls two barriers (for at most the bounded wait's time): true when the
// second one's phase is complete and the first one's is not.  Warp-uniform.
__device__ __forceinline__ bool pv_first(uint32_t tile, uint32_t tile_parity, uint32_t p,
                                         uint32_t p_parity) {
  const uint64_t t0 = global_timer_ns();
  while (true) {
    int r = mbar_test(tile, tile_parity) ? 1 : mbar_test(p, p_parity) ? 2 : 0;
    if (r == 0 && global_timer_ns() - t0 > kWaitLimitNs) r = 1;  // the wait that follows reports it
    r = __shfl_sync(kFullMask, r, 0);
    if (r != 0) return r == 2;
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    latent_decode_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tc,
                         const LatentParams a) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t s_base = smem_u32(sm);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + kOffBar);
  // 0 q_full, 1 q_empty, 2,3 k_full, 4,5 k_empty, 6,7 s_full, 8 p_full, 9 o_full, 10 done
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + kOffBar + 128);
  volatile int* fail = reinterpret_cast<volatile int*>(sm + kOffBar + 132);
  int* start = reinterpret_cast<int*>(sm + kOffBar + 136);  // first sequence, its first tile, tiles

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 160) {
    for (int i = 0; i < 10; ++i) mbar_init(bar(i), i == 8 ? 128 : 1);
    mbar_init(bar(10), kThreads);
    *fail = 0;
    fence_mbar_init();
    prefetch_tensormap(&tq);
    prefetch_tensormap(&tc);
  }
  if (warp == 4) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_launch_dependents();
  // Tiles of every sequence and this worker's first: warp 0 scans 32 lengths
  // at a time.
  const int worker = (int)blockIdx.x / a.head_tiles, ht = (int)blockIdx.x % a.head_tiles;
  if (warp == 0) {
    int total = 0;
    const bool first = blockIdx.x == 0;
    for (int b = 0; b < a.num_seqs; b += 32)
      total += b + lane < a.num_seqs ? tiles_of(context_of(a, b + lane, first)) : 0;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) total += __shfl_xor_sync(kFullMask, total, o);
    const int W = active_workers(a, total);
    const int r0 = worker < W ? worker_begin(worker, W, total) : 0;
    const int r1 = worker < W ? worker_begin(worker + 1, W, total) : 0;
    int run = 0;
    if (lane == 0) {
      start[0] = a.num_seqs;
      start[1] = 0;
      start[2] = r1 - r0;
    }
    __syncwarp();
    for (int b = 0; b < a.num_seqs; b += 32) {
      const int n = b + lane < a.num_seqs ? tiles_of(context_of(a, b + lane, false)) : 0;
      int x = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFullMask, x, o);
        if (lane >= o) x += y;
      }
      const int c0 = run + x - n;
      if (r1 > r0 && c0 <= r0 && r0 < c0 + n) {
        start[0] = b + lane;
        start[1] = r0 - c0;
      }
      if (first && b + lane < a.num_seqs) a.cum[b + lane] = c0;
      run += __shfl_sync(kFullMask, x, 31);
    }
    if (first && lane == 0) a.cum[a.num_seqs] = run;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Walk w;
  w.s = start[0];
  w.t = start[1];
  w.left = start[2];
  const int h0 = ht * kRows;

  if (warp == 4) {
    // ---------------- TMA: the queries of a segment, then its tiles
    const int nb = kTile / a.block_size;
    int g = 0, seg = 0;
    bool ok = true;
    while (ok && w.next(a)) {
      if (seg > 0) ok = __all_sync(kFullMask, mbar_wait_bounded(bar(1), (seg - 1) & 1));
      if (!ok) break;
      if (lane == 0) mbar_arrive_expect_tx(bar(0), kTileBytes);
      __syncwarp();
      if (lane < kAtoms)
        tma_load_2d(s_base + kOffQ + lane * kAtomBytes, &tq, lane * 64,
                    (a.seq_begin + w.cur) * a.num_heads + h0, bar(0));
      ++seg;
      const int32_t* bt = a.block_tables + (size_t)(a.seq_begin + w.cur) * a.max_blocks;
      const int b = lane % nb;
      // The cache row of this lane's block of tile t, one tile ahead.
      auto tile_row = [&](int t) {
        const int lb = t * nb + b;
        int row = a.oob_row;
        if (t < w.t_end && lb * a.block_size < w.c) {
          const int phys = bt[lb];
          if (phys >= 0 && phys < a.num_blocks)
            row = phys * a.block_size;
          else if (lane < nb)
            atomicOr(a.err, PA_ERRBIT_BLOCK_ID);
        }
        return row;
      };
      int row = tile_row(w.t_begin);
      for (int t = w.t_begin; t < w.t_end; ++t, ++g) {
        const int st = g & 1;
        if (g >= 2) ok = __all_sync(kFullMask, mbar_wait_bounded(bar(4 + st), ((g >> 1) - 1) & 1));
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(bar(2 + st), kTileBytes);
        __syncwarp();
        const uint32_t dst = s_base + kOffK + st * kTileBytes + b * a.block_size * 128;
        for (int i = lane; i < kAtoms * nb; i += 32) {
          const int at = i / nb;
          tma_load_2d(dst + at * kAtomBytes, &tc, at * 64, row, bar(2 + st));
        }
        row = tile_row(t + 1);
      }
    }
    if (!ok && lane == 0) {
      *fail = 1;
      // The copies in flight land (bounded) before the shared memory goes.
      if (seg > 0) mbar_wait_bounded(bar(0), (seg - 1) & 1);
      for (int u = max(0, g - 2); u < g; ++u) mbar_wait_bounded(bar(2 + (u & 1)), (u >> 1) & 1);
    }
  } else if (warp == 5) {
    // ---------------- MMA: S(t + 1) before P.V of t, so the softmax of t
    // overlaps a product
    constexpr uint32_t kIdQK = umma_idesc_f16(kRows, kTile, false, false);
    constexpr uint32_t kIdPV = umma_idesc_f16(kRows, 256, false, true);
    const bool leader = lane == 0;
    const uint64_t q_desc = umma_desc_sw128(s_base + kOffQ, 16, 1024);
    const uint64_t k_desc = umma_desc_sw128(s_base + kOffK, 16, 1024);
    const uint64_t v_desc = umma_desc_sw128(s_base + kOffK, kAtomBytes, 1024);
    const uint64_t p_desc = umma_desc_sw128(s_base + kOffP, 16, 1024);
    constexpr uint64_t kStageStep = (uint64_t)kTileBytes >> 4;
    auto uni = [&](bool v) { return __all_sync(kFullMask, v); };
    // P.V of tile g; `first`: it starts a segment.
    int qk = 0, pv = 0;
    auto pv_mma = [&](int g, bool first) {
      const uint64_t vd = v_desc + (g & 1) * kStageStep;
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < kTile / 16; ++k)
#pragma unroll
        for (int half = 0; half < 2; ++half)
          umma_f16_if(leader, tmem + (half ? kLaneHi : 0u), p_desc + (uint64_t)((k * 32) >> 4),
                      vd + (uint64_t)((half * 4 * kAtomBytes + k * 16 * 128) >> 4), kIdPV,
                      !first || k > 0);
      umma_commit_if(leader, bar(4 + (g & 1)));
      umma_commit_if(leader, bar(9));
      ++pv;
    };
    int g = 0, seg = 0;
    bool ok = true, prev_first = false;
    while (ok && w.next(a)) {
      ok = uni(mbar_wait_bounded(bar(0), seg & 1));
      for (int t = w.t_begin; ok && t < w.t_end; ++t, ++g) {
        const int st = g & 1;
        // Of S(t) and P.V of the tile before, the one that can start first: a
        // tile that is still on its way must not hold back the product that
        // frees the other stage.
        if (g > 0 && pv_first(bar(2 + st), (g >> 1) & 1, bar(8), (g - 1) & 1)) {
          ok = uni(mbar_wait_bounded(bar(8), (g - 1) & 1));
          if (ok) pv_mma(g - 1, prev_first);
        }
        ok = ok && uni(mbar_wait_bounded(bar(2 + st), (g >> 1) & 1));
        if (!ok) break;
        // Rows past the context: stale slots may hold anything, and 0 * NaN
        // would poison O (their logits are masked).
        const int live = w.c - t * kTile;
        if (live < kTile) {
          unsigned char* v = sm + kOffK + st * kTileBytes;
          const int chunks = (kTile - live) * 8;
          for (int i = lane; i < chunks * kAtoms; i += 32) {
            const int at = i / chunks, r = live + (i % chunks) / 8, ch = i % 8;
            *reinterpret_cast<uint4*>(v + at * kAtomBytes + r * 128 + ch * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        tc_fence_after();
        const uint64_t kd = k_desc + st * kStageStep;
#pragma unroll
        for (int k = 0; k < kLatentRow / 16; ++k) {
          const uint64_t off = (uint64_t)(((k / 4) * kAtomBytes + (k % 4) * 32) >> 4);
          umma_f16_if(leader, tmem + kColS + 64 * st, q_desc + off, kd + off, kIdQK, k > 0);
        }
        umma_commit_if(leader, bar(6 + st));
        ++qk;
        if (t + 1 == w.t_end) umma_commit_if(leader, bar(1));  // the queries' last reader
        if (pv < g) {
          ok = uni(mbar_wait_bounded(bar(8), (g - 1) & 1));
          if (ok) pv_mma(g - 1, prev_first);
        }
        prev_first = t == w.t_begin;
      }
      ++seg;
    }
    if (ok && g > 0) {
      ok = uni(mbar_wait_bounded(bar(8), (g - 1) & 1));
      if (ok) pv_mma(g - 1, prev_first);
    }
    if (!ok && lane == 0) {
      atomicOr(a.err, PA_ERRBIT_TIMEOUT);
      *fail = 1;
      // Every product started ends (bounded) before its memory goes.
      if (qk > 0) mbar_wait_bounded(bar(6 + ((qk - 1) & 1)), ((qk - 1) >> 1) & 1);
      if (pv > 0) mbar_wait_bounded(bar(9), (pv - 1) & 1);
    }
  } else {
    // ---------------- softmax: lane l < 16 of warp i owns head row 16 i + l;
    // lanes 16-31 hold the upper output values of the same rows
    const uint32_t t_lane = (uint32_t)(warp * 32) << 16;
    const int row = 16 * warp + (lane & 15);
    const int h = h0 + row;
    const bool live_warp = h0 + 16 * warp < a.num_heads;
    unsigned char* p_row = sm + kOffP + row * 128;
    int g = 0;
    bool ok = true;
    while (ok && w.next(a)) {
      float m = -INFINITY, l = 0.f;
      for (int t = w.t_begin; t < w.t_end; ++t, ++g) {
        const int st = g & 1;
        ok = __all_sync(kFullMask, mbar_wait_bounded(bar(6 + st), (g >> 1) & 1) && !*fail);
        if (!ok) break;
        tc_fence_after();
        uint32_t pk[kTile / 2];
        float alpha = 1.f;
        if (live_warp) {
          uint32_t sr[kTile];
          tmem_ld32(tmem + t_lane + kColS + 64 * st, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
          tmem_ld32(tmem + t_lane + kColS + 64 * st + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
          tmem_wait_ld();
          float x[kTile];
#pragma unroll
          for (int j = 0; j < kTile; ++j) x[j] = __uint_as_float(sr[j]) * a.scale_log2;
          const int live = w.c - t * kTile;
          if (live < kTile) {
#pragma unroll
            for (int j = 0; j < kTile; ++j)
              if (j >= live) x[j] = -INFINITY;
          }
          float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int j = 0; j < kTile; j += 8)
#pragma unroll
            for (int u = 0; u < 4; ++u) mq[u] = fmax3(mq[u], x[j + 2 * u], x[j + 2 * u + 1]);
          const float mx = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3]));
          if (mx > m + kRescale || m == -INFINITY) {
            alpha = m == -INFINITY ? 1.f : exp2_approx(m - mx);
            m = mx;
          }
          const float ref = m == -INFINITY ? 0.f : m;
          float sq[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < kTile / 2; ++j) {
            pk[j] = exp2_f32_to_f16x2(x[2 * j] - ref, x[2 * j + 1] - ref);
            sq[j & 3] = add_f16x2_f32(pk[j], sq[j & 3]);
          }
          l = l * alpha + ((sq[0] + sq[1]) + (sq[2] + sq[3]));
        }
        // P and O are free once P.V of the tile before is done (a segment's
        // epilogue has waited for its last).
        if (t > w.t_begin) {
          ok = __all_sync(kFullMask, mbar_wait_bounded(bar(9), (g - 1) & 1) && !*fail);
          if (!ok) break;
          tc_fence_after();
        }
        if (live_warp) {
          // Lanes 16-31 saw no logits of their own: the row's factor comes
          // from the lane that did.
          const float al = __shfl_sync(kFullMask, alpha, lane & 15);
          if (t > w.t_begin && __any_sync(kFullMask, al != 1.f)) {
#pragma unroll
            for (int cb = 0; cb < 8; ++cb) {
              uint32_t r[32];
              tmem_ld32(tmem + t_lane + cb * 32, r);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * al);
              tmem_st32(tmem + t_lane + cb * 32, r);
            }
            tmem_wait_st();
          }
          if (lane < 16) {
#pragma unroll
            for (int ch = 0; ch < 8; ++ch)
              *reinterpret_cast<uint4*>(p_row + ((ch ^ (row & 7)) << 4)) =
                  make_uint4(pk[4 * ch], pk[4 * ch + 1], pk[4 * ch + 2], pk[4 * ch + 3]);
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        mbar_arrive(bar(8));
      }
      if (!ok) break;
      // The segment's output: to `out` when it is the whole sequence, else a
      // partial.
      ok = __all_sync(kFullMask, mbar_wait_bounded(bar(9), (g - 1) & 1) && !*fail);
      if (!ok) break;
      tc_fence_after();
      if (live_warp) {
        const float lr = __shfl_sync(kFullMask, l, lane & 15);
        const float inv = lr > 0.f ? 1.f / lr : 0.f;
        const bool whole = w.t_begin == 0 && w.t_end == w.n;
        const size_t sh = (size_t)(a.seq_begin + w.cur) * a.num_heads + h;
        const size_t ph = (size_t)(w.cur + worker) * a.num_heads + h;
        if (!whole && lane < 16 && h < a.num_heads) a.ws_ml[ph] = make_float2(m, l);
        const int d0 = lane < 16 ? 0 : 256;
        __half* orow = static_cast<__half*>(a.out) + sh * kLatentDim + d0;
        float* prow = a.ws_o + ph * kLatentDim + d0;
#pragma unroll
        for (int cb = 0; cb < 8; ++cb) {
          uint32_t r[32];
          tmem_ld32(tmem + t_lane + cb * 32, r);
          tmem_wait_ld();
          if (h < a.num_heads) {
            if (whole) {
#pragma unroll
              for (int j8 = 0; j8 < 4; ++j8) {
                uint32_t o[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                  const __half2 hv = __floats2half2_rn(__uint_as_float(r[8 * j8 + 2 * u]) * inv,
                                                       __uint_as_float(r[8 * j8 + 2 * u + 1]) * inv);
                  o[u] = *reinterpret_cast<const uint32_t*>(&hv);
                }
                *reinterpret_cast<uint4*>(orow + cb * 32 + j8 * 8) = make_uint4(o[0], o[1], o[2], o[3]);
              }
            } else {
#pragma unroll
              for (int j = 0; j < 32; j += 4)
                *reinterpret_cast<uint4*>(prow + cb * 32 + j) = make_uint4(r[j], r[j + 1], r[j + 2], r[j + 3]);
            }
          }
        }
      }
      tc_fence_before();
    }
    if (!ok && lane == 0) *fail = 1;
  }
  tc_fence_before();
  mbar_arrive(bar(10));
  if (warp == 4) {
    if (!mbar_wait_bounded(bar(10), 0) && lane == 0) atomicOr(a.err, PA_ERRBIT_TIMEOUT);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the segments of each (sequence, head): with M = max m_i,
//   out = sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i.
// 128 threads, four values each; a sequence of no tokens gets zeros, one that
// a single worker covered is already written.
__global__ void __launch_bounds__(128) latent_merge_kernel(const LatentParams a) {
  pdl_wait();
  pdl_launch_dependents();
  const int s = (int)blockIdx.x / a.num_heads, h = (int)blockIdx.x - s * a.num_heads;
  const int c0 = a.cum[s], c1 = a.cum[s + 1], total = a.cum[a.num_seqs];
  __half* out = static_cast<__half*>(a.out) +
                ((size_t)(a.seq_begin + s) * a.num_heads + h) * kLatentDim + 4 * threadIdx.x;
  if (c0 == c1) {
    *reinterpret_cast<uint2*>(out) = make_uint2(0, 0);
    return;
  }
  const int W = active_workers(a, total);
  const int w0 = worker_of(c0, W, total), w1 = worker_of(c1 - 1, W, total);
  if (w0 == w1) return;
  const size_t base = (size_t)(s + w0) * a.num_heads + h;
  float M = -INFINITY;
  for (int i = 0; i <= w1 - w0; ++i) M = fmaxf(M, a.ws_ml[base + (size_t)i * a.num_heads].x);
  float L = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int i = 0; i <= w1 - w0; ++i) {
    const size_t at = base + (size_t)i * a.num_heads;
    const float2 ml = a.ws_ml[at];
    const float4 v = *reinterpret_cast<const float4*>(a.ws_o + at * kLatentDim + 4 * threadIdx.x);
    const float wt = ml.x == -INFINITY ? 0.f : exp2_approx(ml.x - M);
    L = fmaf(wt, ml.y, L);
    o[0] = fmaf(wt, v.x, o[0]);
    o[1] = fmaf(wt, v.y, o[1]);
    o[2] = fmaf(wt, v.z, o[2]);
    o[3] = fmaf(wt, v.w, o[3]);
  }
  const float inv = L > 0.f ? 1.f / L : 0.f;
  const __half2 x = __floats2half2_rn(o[0] * inv, o[1] * inv), y = __floats2half2_rn(o[2] * inv, o[3] * inv);
  *reinterpret_cast<uint2*>(out) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
}

struct LatentLayout {
  int head_tiles, workers;
  size_t cum, ml, o, total;
};

LatentLayout latent_layout(int num_seqs, int num_heads, int sms) {
  LatentLayout l{};
  l.head_tiles = (num_heads + kRows - 1) / kRows;
  l.workers = sms / l.head_tiles > 0 ? sms / l.head_tiles : 1;
  const int seqs = num_seqs < kSeqsPerLaunch ? num_seqs : kSeqsPerLaunch;
  const size_t slots = (size_t)seqs + l.workers;
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  l.cum = 0;
  l.ml = up((size_t)(seqs + 1) * 4);
  l.o = up(l.ml + slots * num_heads * sizeof(float2));
  l.total = up(l.o + slots * num_heads * kLatentDim * sizeof(float));
  return l;
}

}  // namespace

cudaError_t launch_latent_write(const void* latent, long long latent_stride, const void* rope,
                                long long rope_stride, void* cache, const int64_t* slot_mapping,
                                int num_tokens, int block_size, int num_blocks, unsigned int* err,
                                cudaStream_t stream) {
  const long long vecs = (long long)num_tokens * kRowVecs;
  long long blocks = (vecs + 255) / 256;
  if (blocks > 152 * 16) blocks = 152 * 16;
  return launch_pdl(latent_write_kernel, dim3((unsigned)blocks), dim3(256), 0, stream,
                    static_cast<const uint4*>(latent), latent_stride, static_cast<const uint4*>(rope),
                    rope_stride, static_cast<uint4*>(cache), slot_mapping, num_tokens,
                    (long long)num_blocks * block_size, err);
}

size_t latent_workspace_bytes(int num_seqs, int num_heads, int sms) {
  return latent_layout(num_seqs, num_heads, sms).total;
}

cudaError_t launch_latent_decode(const LatentArgs& g, cudaStream_t stream) {
  // Once per device: the shared-memory opt-in.
  static std::atomic<unsigned long long> prepared{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev > 63 || !(prepared.load(std::memory_order_acquire) >> dev & 1)) {
    e = cudaFuncSetAttribute(latent_decode_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    if (dev <= 63) prepared.fetch_or(1ull << dev, std::memory_order_release);
  }
  const LatentLayout l = latent_layout(g.num_seqs, g.num_heads, g.sms);
  const long long rows = (long long)g.num_blocks * g.block_size;
  CUtensorMap tq, tc;
  const cuuint64_t str[1] = {(cuuint64_t)kLatentRow * 2};
  const cuuint64_t qdims[2] = {(cuuint64_t)kLatentRow, (cuuint64_t)g.num_seqs * g.num_heads};
  const cuuint64_t cdims[2] = {(cuuint64_t)kLatentRow, (cuuint64_t)rows};
  const cuuint32_t qbox[2] = {64, (cuuint32_t)kRows}, cbox[2] = {64, (cuuint32_t)g.block_size};
  if (!encode_tensor_map(&tq, g.query, 2, qdims, str, qbox) ||
      !encode_tensor_map(&tc, g.cache, 2, cdims, str, cbox))
    return cudaErrorInvalidValue;
  LatentParams p{};
  p.out = g.out;
  p.block_tables = g.block_tables;
  p.context_lens = g.context_lens;
  p.cum = reinterpret_cast<int*>(g.workspace + l.cum);
  p.ws_ml = reinterpret_cast<float2*>(g.workspace + l.ml);
  p.ws_o = reinterpret_cast<float*>(g.workspace + l.o);
  p.err = g.err;
  p.num_heads = g.num_heads;
  p.head_tiles = l.head_tiles;
  p.workers = l.workers;
  p.block_size = g.block_size;
  p.num_blocks = g.num_blocks;
  p.max_blocks = g.max_blocks;
  p.max_context_len = g.max_context_len;
  p.oob_row = (int)rows;
  p.scale_log2 = g.scale_log2;
  for (int b = 0; b < g.num_seqs; b += kSeqsPerLaunch) {
    p.seq_begin = b;
    p.num_seqs = g.num_seqs - b < kSeqsPerLaunch ? g.num_seqs - b : kSeqsPerLaunch;
    e = launch_pdl(latent_decode_kernel, dim3((unsigned)(l.workers * l.head_tiles)), dim3(kThreads),
                   kSmem, stream, tq, tc, p);
    if (e != cudaSuccess) return e;
    e = launch_pdl(latent_merge_kernel, dim3((unsigned)((long long)p.num_seqs * p.num_heads)),
                   dim3(128), 0, stream, p);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace pa
