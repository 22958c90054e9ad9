// Attention of several queries per sequence over the quantised cache
// (kv_tree_attn, kv_cross_attn): the split kernel for up to 32 query rows a KV
// head (internal template; the instantiations live in multi_d{64,128}_k{2,3,4,8}.cu).
#pragma once

#include "multi_attn.cuh"

namespace kvq {

namespace narrow {

// Split kernel: one persistent CTA per SM walks an equal share of all units'
// blocks in tiles of up to four blocks (128 columns); for each unit it meets
// it leaves one partial (running max, sum and unnormalised output of every
// row), or the output itself where its share holds the whole unit.
//
// Both products run on tcgen05 with the columns of the cache as the long
// side, so that their time goes with the number of query rows N (16 or 32)
// and not with a padded 128:
//   S^T [128 columns x N] = K [128 x D] . Q^T [D x N]
//   O^T [D channels x N] += V^T [D x 128] . P^T [128 x N]
// K and V^T are the A operands, in tensor memory: the packed codes lie in the
// order of the A fragments, so a lane turns its words into f16 pairs in
// registers and stores them there, without a pass through shared memory. Q
// and P^T are B operands in shared memory (128-byte swizzle; Q k-major, P^T
// as written by the threads, one column's N weights in a row, n-major).
//
// Roles: warps 0-7 softmax (a thread owns one column of a tile), 8-23 dequantise
// (two sets of eight, one for the even and one for the odd tiles, each four
// warps for the keys of one block each and four for the values of 32 channels
// each), 24 issues the score products, 25 the value products, 26 the bulk
// copies of the groups' chunks. K, V and P are double buffered by tile, S has
// four buffers. The hand-offs of a tile cost each role hundreds of cycles of
// latency, so every role but the issuers has two tiles' time for a tile: the
// first four softmax warps take the even tiles and the other four the odd
// ones, each with references, sums and an O of its own that are joined at the
// segment's end.
//
// Softmax with the columns across lanes: every row's weights are taken
// against a reference that all its columns share and that moves only when
// some score exceeds it by 2^kLag (one vote a tile); the max over the
// columns, and the rescale of O, are paid only then.
//
// What bounds it: instruction issue (some 4000 warp instructions a tile at
// D = 128, three quarters of them dequantisation), and fetching them: every
// role's loop body is longer than a scheduler's instruction cache. 16
// sequences of 32768 tokens, 32 rows a head, K2/V4: 198 us on the device (546 MB,
// 2.8 TB/s); four of 131072, 12 rows, K2/V2: 142 us (403 MB, 2.8 TB/s). The
// compiler spills 208 to 312 bytes a thread in every instance.
//
// Every wait is bounded; a role that gives up raises the CTA's abort flag,
// the others leave at their next wait, and the softmax warps leave together
// at a segment's end, so that none is left at a barrier.
constexpr int kSoftmaxWarps = 8, kDequantWarp = 8, kScoreWarp = 24, kOutWarp = 25, kCopyWarp = 26;
constexpr int kSplitThreads = 28 * 32;  // (the last warp is idle: registers are shared out by fours)

template <int D, int N>
struct MultiTile {
  static constexpr int NS = 4;                 // buffers of S
  static constexpr int QBYTES = N * D * 2;     // [D / 64 panels][N rows][128 B]
  static constexpr int PBYTES = 128 * 128;     // [128 columns][128 B], the first 2 N of each used
  // tensor memory columns
  static constexpr int KCOLS = D / 2, VCOLS = 64;
  static constexpr int TK = 0, TV = TK + 2 * KCOLS, TS = TV + 2 * VCOLS, TO = TS + NS * N, TEND = TO + 2 * N;
  static constexpr int TCOLS = TEND <= 256 ? 256 : 512;
  static_assert(TEND <= 512, "tensor memory");
  // shared memory: Q | P | row scales and references | reductions | barriers | chunk stages
  static constexpr int OFF_P = QBYTES;
  static constexpr int OFF_ROW = OFF_P + 2 * PBYTES;    // float [2][2][N]: scales, then bias - reference
  static constexpr int OFF_FAC = OFF_ROW + 2 * N * 8;   // float [2][N]: rescale factors, at the end those of the join
  static constexpr int OFF_SUM = OFF_FAC + 2 * N * 4;   // float [2][N]: the sums
  static constexpr int OFF_SCALE = OFF_SUM + 2 * N * 4; // float [N]: scales of the segment's queries
  static constexpr int OFF_RED = OFF_SCALE + N * 4;     // float [8 warps][N]
  static constexpr int OFF_BAR = OFF_RED + 8 * N * 4;
  static constexpr int NBAR = 2 * kMaxStages + 23;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;   // abort flag, tensor memory address, bad[8][8]
  static constexpr int OFF_RAW = (OFF_MISC + 16 + 256 + 127) / 128 * 128;
};

// Stages of kTileBlocks chunks: as many as fit, at most kMaxStages, and an
// even number, so that a stage always serves the same set of dequantising
// warps (a set that skipped a stage's phase would take the phase before it
// for the one it waits for). The block takes more than half of an SM's shared
// memory in any case, so that two calls that overlap never share an SM's
// tensor memory.
template <int D, int N>
int multi_stages(int chunk) {
  const int room = 227 * 1024 - MultiTile<D, N>::OFF_RAW;
  const int n = room / (kTileBlocks * chunk);
  return (n < kMaxStages ? n : kMaxStages) & ~1;
}
template <int D, int N>
int multi_smem(int chunk) {
  const int n = MultiTile<D, N>::OFF_RAW + multi_stages<D, N>(chunk) * kTileBlocks * chunk;
  return n > 120 * 1024 ? n : 120 * 1024;
}

template <int D, int N, int KB, int VB>
__global__ void __launch_bounds__(kSplitThreads, 1)
    multi_split_kernel(const __grid_constant__ MultiAttnArgs a, int n_stages) {
  using T = MultiTile<D, N>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* raw_full = reinterpret_cast<uint64_t*>(smem + T::OFF_BAR);
  uint64_t* raw_empty = raw_full + kMaxStages;
  uint64_t* k_full = raw_empty + kMaxStages;
  uint64_t *k_empty = k_full + 2, *v_full = k_full + 4, *v_empty = k_full + 6;
  uint64_t *p_full = k_full + 8, *o_done = k_full + 10, *q_full = k_full + 12, *drain = k_full + 13;
  uint64_t *s_full = k_full + 15, *s_empty = k_full + 19;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + T::OFF_MISC);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(smem + T::OFF_MISC + 4);
  // columns of segment i's draft block k with a value that is not finite in f16:
  // bad[8 (i & 7) + k]. The value warps write it and clear the place of
  // segment i + 3 when they begin segment i: they are never more than two
  // tiles apart, nor more than two ahead of what the softmax warps read.
  uint32_t* bad = reinterpret_cast<uint32_t*>(smem + T::OFF_MISC + 16);
  // (through a shuffle: the compiler then knows that it is the warp's)
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int cta = blockIdx.x;

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < n_stages; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 8);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 4);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 4);
      mbar_init(&v_empty[i], 1);
      mbar_init(&p_full[i], kSoftmaxWarps / 2);
      mbar_init(&o_done[i], 2);  // the MMA, and its issuer: what the value warps wrote before is visible too
    }
    for (int i = 0; i < T::NS; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], kSoftmaxWarps / 2);
    }
    mbar_init(q_full, kSoftmaxWarps);
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    mbar_fence_init();
  }
  if (threadIdx.x < 64) bad[threadIdx.x] = 0u;
  if (warp == kScoreWarp) tc_alloc(tmem_at, T::TCOLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_at, 0);

  SegmentCursor seg;
  seg.begin(a, cta);
  bool ok = true;
  uint32_t tile = 0;  // tiles so far, over all segments: buffer tile & 1, stage tile % n_stages
  uint32_t n_seg = 0; // segments begun

  // 72 registers a thread at launch, shared out again by fours of warps: 2 x 104 + 4 x 64 + 40
  if (warp < kSoftmaxWarps) {
    registers_up<104>();
    float* scale = reinterpret_cast<float*>(smem + T::OFF_SCALE);
    const int grp = warp >> 2, quarter = warp & 3, bar_id = 1 + grp;
    const int tid = threadIdx.x & 127, col = quarter * 32 + lane;  // column of the tile, channel of O^T
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t o_at = tmem + lanes + T::TO + grp * N;
    float* offs = reinterpret_cast<float*>(smem + T::OFF_ROW) + 2 * N;
    float *my_scale = offs + (grp - 2) * N, *my_off = offs + grp * N;
    float* fac = reinterpret_cast<float*>(smem + T::OFF_FAC);
    float* my_fac = fac + grp * N;
    float* sums = reinterpret_cast<float*>(smem + T::OFF_SUM);
    float* red = reinterpret_cast<float*>(smem + T::OFF_RED) + grp * 4 * N;
    while (ok && seg.next(a, cta)) {
      const int h = seg.h, b = seg.b;
      // queries of the segment (the scores of the last one are done: their
      // barriers were waited for) and fresh references
      query_rows<D, 256 / N>(a, b, h, seg.rt, threadIdx.x, scale, [&](int n, int ch, uint4 x) {
        // the keys' k order: channel t D/4 + 4s + 2p + e at 16s + 8p + 2t + e
        const int t = ch / (D / 4), k0 = 4 * (ch % (D / 4)) + 2 * t;
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int k = k0 + 8 * i, piece = ((k & 63) >> 3) ^ (n & 7);
          *reinterpret_cast<uint32_t*>(smem + (k >> 6) * (N * 128) + n * 128 + piece * 16 + (k & 7) * 2) = w[i];
        }
      });
      fence_async_proxy();
      named_barrier_sync(3, kSoftmaxWarps * 32);  // scale[] is written
      mbar_arrive_if(lane == 0, q_full);
      if (tid < N) my_scale[tid] = scale[tid], my_off[tid] = INFINITY;
      named_barrier_sync(bar_id, 128);
      float l[N];
#pragma unroll
      for (int n = 0; n < N; ++n) l[n] = 0.0f;
      const uint32_t seg_tile = tile;
      int last0 = -1, last1 = -1;  // the segment's last tile of each buffer
      bool failed = false;
#pragma unroll 1
      for (int blk = seg.blk0; blk < seg.blk1; blk += kTileBlocks, ++tile) {
        const uint32_t buf = tile & 1, sb = tile % T::NS;
        if (buf) last1 = static_cast<int>(tile);
        else last0 = static_cast<int>(tile);
        if (buf != static_cast<uint32_t>(grp)) continue;
        // which rows may see this thread's column: all, none, or, drafted, some
        uint32_t hide = 0u;
        int kind = kGroupBlock;
        const bool plain = blk + kTileBlocks <= seg.blk1 && seg.plain(blk, kTileBlocks);
        if (!plain) {
          uint32_t cols = 0u;
          if (blk + quarter < seg.blk1) {
            int idx;
            kind = block_kind(seg.seq, blk + quarter, &idx);
            cols = column_mask(a, seg.seq, b, kind, idx);
            if (kind == kDraftBlock) {
#pragma unroll 1
              for (int n = 0; n < N; ++n) {
                const int r = n;
                const uint32_t m = r < a.rows ? draft_bits(a, b, r % a.T, idx) : 0u;
                if (!(m >> lane & 1u)) hide |= 1u << n;
              }
            }
          }
          if (!(cols >> lane & 1u)) hide = 0xffffffffu;
        }
        if (!failed) failed = !pipe_wait(&s_full[sb], tile / T::NS & 1, abort_flag);
        tc_fence_after();
        float s[N];
        tc_ld<N>(tmem + lanes + T::TS + sb * N, s);
        tc_wait_ld();
#pragma unroll
        for (int n = 0; n < N; n += 4) {
          const float4 f = *reinterpret_cast<const float4*>(my_scale + n), o = *reinterpret_cast<const float4*>(my_off + n);
          const float2 x = __ffma2_rn(make_float2(s[n], s[n + 1]), make_float2(f.x, f.y), make_float2(o.x, o.y));
          const float2 y = __ffma2_rn(make_float2(s[n + 2], s[n + 3]), make_float2(f.z, f.w), make_float2(o.z, o.w));
          s[n] = x.x, s[n + 1] = x.y, s[n + 2] = y.x, s[n + 3] = y.y;
        }
        if (!plain) {
#pragma unroll
          for (int n = 0; n < N; ++n)
            if (hide >> n & 1u) s[n] = -INFINITY;
        }
        float top4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int n = 4; n < N; n += 4) {
#pragma unroll
          for (int k = 0; k < 4; ++k) top4[k] = fmaxf(top4[k], s[n + k]);
        }
        const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
        // lane 0 votes for its warp's wish to move the reference, the others for its failure
        const bool move = __any_sync(0xffffffffu, top > kBias + kLag);
        const int votes = named_barrier_count(bar_id, 128, lane == 0 ? move : failed);
        if (votes > 4) failed = true;
        const bool later = tile - seg_tile >= 2;  // O holds tiles of this segment
        if (votes && votes <= 4) {
          // the rows' maxima over the tile (scores again: against a
          // reference of -inf they are infinite)
          tc_ld<N>(tmem + lanes + T::TS + sb * N, s);
          tc_wait_ld();
#pragma unroll
          for (int n = 0; n < N; ++n) {
            s[n] = hide >> n & 1u ? -INFINITY : s[n] * my_scale[n];
            const float m = warp_max(s[n]);
            if (lane == 0) red[quarter * N + n] = m;
          }
          named_barrier_sync(bar_id, 128);
          if (tid < N) {
            const float old = kBias - my_off[tid];  // -inf at first
            const float m = fmaxf(fmaxf(red[tid], red[N + tid]), fmaxf(red[2 * N + tid], red[3 * N + tid]));
            const float now = fmaxf(old, m), was = my_off[tid], is = kBias - now;
            my_fac[tid] = now == -INFINITY ? 1.0f : exp2f(is - was);
            my_off[tid] = is;
          }
          named_barrier_sync(bar_id, 128);
#pragma unroll
          for (int n = 0; n < N; ++n) l[n] *= my_fac[n];
          if (later) {  // every value product so far into this O is done once the last one is
            if (!failed) failed = !pipe_wait(&o_done[buf], ((tile - 2) >> 1) & 1, abort_flag);
            tc_fence_after();
#pragma unroll
            for (int n = 0; n < N; n += 8) {
              float o[8];
              tc_ld<8>(o_at + n, o);
              tc_wait_ld();
#pragma unroll
              for (int k = 0; k < 8; ++k) o[k] *= my_fac[n + k];
              tc_st<8>(o_at + n, o);
            }
            tc_wait_st();
          }
#pragma unroll
          for (int n = 0; n < N; ++n) s[n] = hide >> n & 1u ? -INFINITY : s[n] + my_off[n];
        }
        tc_fence_before();
        __syncwarp();
        mbar_arrive_if(lane == 0, &s_empty[sb]);
        // the weights; buffer `buf` of P is free when the tile before the last is done
        if (tile - seg_tile >= 2 && !failed) failed = !pipe_wait(&o_done[buf], ((tile - 2) >> 1) & 1, abort_flag);
        uint8_t* p_row = smem + T::OFF_P + buf * T::PBYTES + col * 128;
#pragma unroll
        for (int n = 0; n < N; n += 8) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float p0 = fast_exp2(s[n + 2 * k]), p1 = fast_exp2(s[n + 2 * k + 1]);
            const float2 sum = __fadd2_rn(make_float2(l[n + 2 * k], l[n + 2 * k + 1]), make_float2(p0, p1));
            l[n + 2 * k] = sum.x, l[n + 2 * k + 1] = sum.y;
            w[k] = f2_to_h2(p0, p1);
          }
          const int piece = (n / 8) ^ (col & 7);
          *reinterpret_cast<uint4*>(p_row + piece * 16) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        fence_async_proxy();
        tc_fence_before();
        __syncwarp();
        mbar_arrive_if(lane == 0, &p_full[buf]);
      }
      // the rows' sums over the columns
#pragma unroll
      for (int n = 0; n < N; ++n) {
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) l[n] += __shfl_xor_sync(0xffffffffu, l[n], off);
        if (lane == 0) red[quarter * N + n] = l[n];
      }
      const bool whole = seg.blk0 == 0 && seg.blk1 == seg.seq.total;
      named_barrier_sync(bar_id, 128);
      if (tid < N) sums[grp * N + tid] = (red[tid] + red[N + tid]) + (red[2 * N + tid] + red[3 * N + tid]);
      named_barrier_sync(3, kSoftmaxWarps * 32);
      if (threadIdx.x < N) {  // row n of the tile: its sum and max, and what its O's count
        const int n = threadIdx.x, r = n;
        // (the reference less the bias: what the weights are relative to)
        const float m0 = -offs[n], m1 = -offs[N + n], m = fmaxf(m0, m1);
        const float f0 = m0 == -INFINITY ? 0.0f : exp2f(m0 - m), f1 = m1 == -INFINITY ? 0.0f : exp2f(m1 - m);
        const float sum = f0 * sums[n] + f1 * sums[N + n];
        fac[N + n] = f1 * a.v_scale;
        if (r < a.rows) {
          if (!whole) {
            reinterpret_cast<float2*>(a.part_ml)[static_cast<size_t>(seg.slot) * N + n] = make_float2(m, sum);
          } else if (a.lse) {
            const size_t at = (static_cast<size_t>(b) * a.geo.Hq + static_cast<size_t>(h) * a.geo.gqa) * a.T + r;
            a.lse[at] = sum == 0.0f ? -INFINITY : (m + log2f(sum)) * 0.69314718055994530942f;
          }
        }
        fac[n] = f0 * a.v_scale;
        scale[n] = whole ? (sum == 0.0f ? 0.0f : 1.0f / sum) : 1.0f;
      }
      named_barrier_sync(3, kSoftmaxWarps * 32);
      if (last0 >= 0 && !failed) failed = !pipe_wait(&o_done[0], (last0 >> 1) & 1, abort_flag);
      if (last1 >= 0 && !failed) failed = !pipe_wait(&o_done[1], (last1 >> 1) & 1, abort_flag);
      tc_fence_after();
      if (!failed && col < D) {
        const int half = grp * (N / 2);  // these warps write half of the rows
        const size_t orow = (static_cast<size_t>(b) * a.geo.Hq + static_cast<size_t>(h) * a.geo.gqa) * a.T;
        float* part = a.part_o + static_cast<size_t>(seg.slot) * N * D + col;
#pragma unroll 1
        for (int n = half; n < half + N / 2; n += 8) {
          float o[8];
          tc_ld<8>(tmem + lanes + T::TO + n, o);
          tc_wait_ld();
          float o1[8];
          tc_ld<8>(tmem + lanes + T::TO + N + n, o1);
          tc_wait_ld();
#pragma unroll
          for (int i = 0; i < 8; ++i)  // (an O without a tile holds anything)
            o[i] = (last0 >= 0 ? o[i] * fac[n + i] : 0.0f) + (last1 >= 0 ? o1[i] * fac[N + n + i] : 0.0f);
          for (int k = 0; k < a.draft_blocks; ++k) {  // values that are not finite, in the rows that see them
            for (uint32_t left = bad[8 * (n_seg & 7) + k]; left; left &= left - 1) {
              const int j = __ffs(left) - 1;
              const size_t at = ((static_cast<size_t>(b) * a.geo.H + h) * a.T + kGroup * k + j) * D + col;
              const uint16_t x = a.vd[at];
              const float y = act_to_float(x, a.geo.act_bf16) * INFINITY;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int r = n + i;
                if ((x & 0x7fffu) >= a.v_top && r < a.rows && (draft_bits(a, b, r % a.T, k) >> j & 1u)) o[i] += y;
              }
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (n + i >= a.rows) continue;
            if (whole)
              a.out[(orow + n + i) * D + col] = float_to_act(o[i] * scale[n + i], a.geo.act_bf16);
            else
              part[(n + i) * D] = o[i];
          }
          __syncwarp();
        }
      }
      tc_fence_before();
      // the next segment's queries and references go over this one's when
      // every softmax warp is here; a failure makes all of them leave
      if (named_barrier_count(3, kSoftmaxWarps * 32, failed)) ok = false;
      ++n_seg;
    }
  } else if (warp < kScoreWarp) {
    registers_down<64>();
    const uint32_t set = (warp - kDequantWarp) >> 3;
    const bool keys = ((warp - kDequantWarp) & 4) == 0;
    const int quarter = warp & 3;
    const uint32_t at = tmem + (static_cast<uint32_t>(quarter * 32) << 16) +
                        (keys ? T::TK + set * T::KCOLS : T::TV + set * T::VCOLS);
    uint64_t* full_bar = keys ? &k_full[set] : &v_full[set];
    uint64_t* empty_bar = keys ? &k_empty[set] : &v_empty[set];
    const uint8_t* raw = smem + T::OFF_RAW;
    const int chunk = a.geo.chunk.bytes;
    uint32_t st = 0, st_par = 0;
    while (ok && seg.next(a, cta)) {
      if (!keys && a.draft_blocks) {
        if (lane < 8) bad[8 * ((n_seg + 3) & 7) + lane] = 0u;
        __syncwarp();
      }
#pragma unroll 1
      for (int blk = seg.blk0; blk < seg.blk1; blk += kTileBlocks, ++tile) {
        const uint8_t* src = raw + st * kTileBlocks * chunk;
        uint64_t *raw_bar = &raw_full[st], *raw_free = &raw_empty[st];
        const uint32_t raw_par = st_par;
        if (++st == static_cast<uint32_t>(n_stages)) st = 0, st_par ^= 1;
        if ((tile & 1) != set) continue;
        ok = pipe_wait(raw_bar, raw_par, abort_flag) && pipe_wait(empty_bar, ((tile >> 1) & 1) ^ 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const int nb = min(kTileBlocks, seg.blk1 - blk);
        if (keys) {
          if (quarter < nb) {
            block_keys<D, KB, 2>(a, seg, blk + quarter, src + quarter * chunk, 0, lane,
                             [&](int s, int mt, const uint32_t(&v)[8]) {
                               tc_st_frag2(at + (static_cast<uint32_t>(mt * 16) << 16) + 8 * s, v);
                             });
          }
        } else if (quarter < D / 32) {
          block_values<D, VB, kTileBlocks>(a, seg, blk, src, quarter, lane, bad + 8 * (n_seg & 7),
                                       [&](int q, int mm, const uint32_t(&v)[8]) {
                                         tc_st_frag2(at + (static_cast<uint32_t>(mm * 16) << 16) + 16 * q, v);
                                       });
        }
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        mbar_arrive_if(lane == 0, raw_free);
        mbar_arrive_if(lane == 0, full_bar);
      }
      ++n_seg;
    }
  } else if (warp == kScoreWarp) {
    registers_down<40>();
    const uint64_t q_desc = smem_operand(smem_u32(smem), 1024);
    uint32_t seg_par = 0;
    while (ok && seg.next(a, cta)) {
      if (!(ok = pipe_wait(q_full, seg_par, abort_flag))) break;
      seg_par ^= 1;
#pragma unroll 1
      for (int blk = seg.blk0; blk < seg.blk1; blk += kTileBlocks, ++tile) {
        const uint32_t buf = tile & 1, sb = tile % T::NS;
        if (!(ok = pipe_wait(&k_full[buf], (tile >> 1) & 1, abort_flag) &&
                   pipe_wait(&s_empty[sb], (tile / T::NS & 1) ^ 1, abort_flag)))
          break;
        tc_fence_after();
        const uint32_t sc = tmem + T::TS + sb * N, k = tmem + T::TK + buf * T::KCOLS;
        if (elect_one()) {
#pragma unroll
          for (int s = 0; s < D / 16; ++s)
            tc_mma(sc, k + 8 * s, q_desc + (((s >> 2) * (N * 128) + (s & 3) * 32) >> 4), tc_instr(N, false), s != 0);
          tc_commit(&k_empty[buf]);
          tc_commit(&s_full[sb]);
        }
        __syncwarp();
      }
    }
    if (!ok) {  // let what was issued finish before the memory goes
      if (elect_one()) {
        tc_commit(&drain[0]);
        (void)mbar_wait_bounded(&drain[0], 0);
      }
      __syncwarp();
    }
  } else if (warp == kOutWarp) {
    registers_down<40>();
    const uint64_t p_desc = smem_operand(smem_u32(smem + T::OFF_P), 1024);
    while (ok && seg.next(a, cta)) {
      const uint32_t first = tile;
#pragma unroll 1
      for (int blk = seg.blk0; blk < seg.blk1; blk += kTileBlocks, ++tile) {
        const uint32_t buf = tile & 1, par = (tile >> 1) & 1;
        if (!(ok = pipe_wait(&v_full[buf], par, abort_flag) && pipe_wait(&p_full[buf], par, abort_flag))) break;
        tc_fence_after();
        const int steps = 2 * min(kTileBlocks, seg.blk1 - blk);
        const bool fresh = tile - first < 2;  // its O's first in the segment
        const uint32_t o = tmem + T::TO + buf * N, v = tmem + T::TV + buf * T::VCOLS;
        const uint64_t p = p_desc + buf * (T::PBYTES >> 4);
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < 2 * kTileBlocks; ++j)
            if (j < steps) tc_mma(o, v + 8 * j, p + j * (2048 >> 4), tc_instr(N, true), !(fresh && j == 0));
          tc_commit(&v_empty[buf]);
          tc_commit(&o_done[buf]);
          mbar_arrive(&o_done[buf]);
        }
        __syncwarp();
      }
    }
    if (!ok) {
      if (elect_one()) {
        tc_commit(&drain[1]);
        (void)mbar_wait_bounded(&drain[1], 0);
      }
      __syncwarp();
    }
  } else if (warp == kCopyWarp) {
    registers_down<40>();
    ok = copy_chunks(a, seg, cta, smem + T::OFF_RAW, n_stages, raw_full, raw_empty, abort_flag);
  } else {
    registers_down<40>();
  }
  pdl_launch_dependents();  // the merge is scheduled from here on
  if (!ok && lane == 0) set_error(a.tab.err_flag, kErrTimeout);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kScoreWarp) tc_dealloc(tmem, T::TCOLS);
}

}  // namespace narrow

template <int D, int N, int KB, int VB>
cudaError_t launch_narrow(const MultiAttnArgs& a, cudaStream_t s) {
  using namespace narrow;
  static int configured[kMaxDevices] = {};  // per device and instance: the attribute is per device
  const int smem = multi_smem<D, N>(a.geo.chunk.bytes);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (smem > configured[dev]) {
    e = cudaFuncSetAttribute(multi_split_kernel<D, N, KB, VB>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    configured[dev] = smem;
  }
  multi_split_kernel<D, N, KB, VB><<<a.n_ctas, kSplitThreads, smem, s>>>(a, multi_stages<D, N>(a.geo.chunk.bytes));
  return cudaGetLastError();
}

}  // namespace kvq
