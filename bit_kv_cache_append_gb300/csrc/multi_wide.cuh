// Attention of several queries per sequence over the quantised cache
// (kv_tree_attn, kv_cross_attn): the split kernel for tiles of 128 query rows
// (internal template; the instantiations live in multi_d{64,128}_k{2,3,4,8}.cu).
#pragma once

#include "multi_attn.cuh"

namespace kvq {

namespace wide {

// One persistent CTA per SM walks an equal share of all units' blocks in
// tiles of up to four blocks (128 columns), as the kernel for few rows does
// (multi_narrow.cuh), with the query rows as the products' long side:
//   S [128 rows x 128 columns] = Q [128 x D] . K^T [D x 128]
//   O [128 rows x D] += P [128 x 128] . V [128 x D]
// Q, K and V^T are in shared memory (128-byte swizzle, k-major), P takes the
// place of S in tensor memory: a thread owns a row, so the softmax needs no
// exchange between threads, and a weight goes from the score's registers to
// tensor memory without a pass through shared memory.
//
// The dequantised fragments are put so that every store is one 16-byte piece
// and a quarter warp's eight pieces fall into different banks:
//   columns of a block: position 8t + 4kb + 2h + e holds token 16kb + 8h + 2t
//     + e, so that a lane's tokens of one channel are adjacent in V^T;
//   k of K and Q: channels t D/4 + 8u .. + 7 are piece 2t + (u & 1) of the
//     128-byte row in panel u / 2;
//   rows of V^T, columns of O: channel 8c + g is row 8c + 4 (g & 1) + g / 2.
//
// Roles: warps 0-7 softmax (0-3 the even tiles, 4-7 the odd ones, each with an
// S, references, sums and an O of its own that are joined at the segment's
// end), 8-15 keys (half a block each), 16-23 values (32 channels of two blocks
// each, of one at D = 64), 24 issues the score products, 25 the value
// products, 26 the bulk copies of the chunks. K is double buffered, V where
// there is room.
//
// Up to 64 rows are held twice (COPIES = 2): the first copy's weights are
// those of a tile's first two blocks, the second's of the last two, and zero
// elsewhere, so that all four schedulers share the softmax of a tile (64
// sequences of 4133 tokens, 61 rows a head: 232 -> 208 us). The copies are
// joined at the end of a segment that is a whole unit, else they are partials
// of their own for the merge.
//
// What bounds it: the instruction issue of dequantisation and softmax
// together, then shared memory (per tile 64 KB written and 96 KB read by the
// products), then the tensor cores (1024 cycles a tile at D = 128).
// Those 64 sequences take 155 us on the device (321 MB, 2.1 TB/s), eight of up
// to 4001 tokens with 1536 rows a head 188 us (101 GFLOP, 0.54 PFLOP/s); some
// 5 us of a segment are its queries and its output, in which dequantisation is
// two tiles ahead at most.
//
// Every wait is bounded, as in multi_narrow.cuh.
constexpr int kSoftmaxWarps = 8, kValueWarp = 16, kScoreWarp = 24, kOutWarp = 25, kCopyWarp = 26;
constexpr int kWideThreads = 28 * 32;  // (the last warp is idle: registers are shared out by fours)
constexpr int kRows = 128;

// Token of column position p of a block.
__device__ __forceinline__ constexpr int token_of_position(int p) {
  return 16 * ((p >> 2) & 1) + 8 * ((p >> 1) & 1) + 2 * (p >> 3) + (p & 1);
}

template <int D>
struct WideTile {
  static constexpr int QBYTES = kRows * D * 2;    // [D / 64 panels][128 rows][128 B]
  static constexpr int KBYTES = 128 * D * 2;      // [D / 64 panels][128 columns][128 B]
  static constexpr int VBYTES = D * 128 * 2;      // [2 panels of 64 columns][D channels][128 B]
  // tensor memory columns: S (P in its first 64) twice, O twice
  static constexpr int TS = 0, TO = 256, TCOLS = 512;
  // shared memory: Q | K twice | V (n_v times) | row exchange | barriers | chunk stages
  static constexpr int OFF_K = QBYTES, OFF_V = OFF_K + 2 * KBYTES;
  // the rest begins behind V (n_v VBYTES from OFF_V)
  static constexpr int ROW = 0;                    // float2 [2][128]: max and sum
  static constexpr int SCALE = ROW + 2 * kRows * 8;  // float [128]
  static constexpr int BAR = SCALE + kRows * 4;
  static constexpr int NBAR = 2 * kMaxStages + 17;
  static constexpr int MISC = BAR + NBAR * 8;      // abort flag, tensor memory address, bad[8][8]
  static constexpr int RAW = (MISC + 16 + 256 + 127) / 128 * 128;
  static constexpr int kRoom = 227 * 1024 - OFF_V - RAW;  // for V and the stages
};

// Two buffers of V where two stages of chunks fit beside them (all but 8-bit
// keys and values at D = 128), else one.
template <int D>
int wide_v_buffers(int chunk) {
  return WideTile<D>::kRoom - 2 * WideTile<D>::VBYTES >= 2 * kTileBlocks * chunk ? 2 : 1;
}
template <int D>
int wide_stages(int chunk) {
  const int n = (WideTile<D>::kRoom - wide_v_buffers<D>(chunk) * WideTile<D>::VBYTES) / (kTileBlocks * chunk);
  return n < kMaxStages ? n : kMaxStages;
}
// (more than half of an SM's shared memory in any case: two calls that
// overlap never share an SM's tensor memory)
template <int D>
int wide_smem(int chunk) {
  const int n = WideTile<D>::OFF_V + wide_v_buffers<D>(chunk) * WideTile<D>::VBYTES + WideTile<D>::RAW +
                wide_stages<D>(chunk) * kTileBlocks * chunk;
  return n > 120 * 1024 ? n : 120 * 1024;
}

template <int D, int KB, int VB, int COPIES>
__global__ void __launch_bounds__(kWideThreads, 1)
    multi_wide_kernel(const __grid_constant__ MultiAttnArgs a, int n_stages, int n_v) {
  using T = WideTile<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* rest = smem + T::OFF_V + n_v * T::VBYTES;
  uint64_t* raw_full = reinterpret_cast<uint64_t*>(rest + T::BAR);
  uint64_t* raw_empty = raw_full + kMaxStages;
  uint64_t* k_full = raw_empty + kMaxStages;
  uint64_t *k_empty = k_full + 2, *v_full = k_full + 4, *v_empty = k_full + 6, *s_full = k_full + 8;
  uint64_t *p_full = k_full + 10, *o_done = k_full + 12, *q_full = k_full + 14, *drain = k_full + 15;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(rest + T::MISC);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(rest + T::MISC + 4);
  // columns of segment i's draft blocks with a value that is not finite in f16, as in
  // multi_narrow.cuh: bad[8 (i & 7) + block], cleared three segments ahead
  uint32_t* bad = reinterpret_cast<uint32_t*>(rest + T::MISC + 16);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int cta = blockIdx.x;

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < n_stages; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 16);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 8);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 8);
      mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], kSoftmaxWarps / 2);
      mbar_init(&o_done[i], 2);  // the MMA, and its issuer: what the value warps wrote before is visible too
      mbar_init(&drain[i], 1);
    }
    mbar_init(q_full, kSoftmaxWarps);
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
  uint32_t tile = 0;   // tiles so far, over all segments
  uint32_t n_seg = 0;  // segments begun

  // 72 registers a thread at launch, shared out again by fours of warps: 2 x 104 + 4 x 64 + 40
  if (warp < kSoftmaxWarps) {
    registers_up<104>();
    float2* state = reinterpret_cast<float2*>(rest + T::ROW);
    float* scales = reinterpret_cast<float*>(rest + T::SCALE);
    constexpr int ROWS = kRows / COPIES, NQ = kTileBlocks / COPIES;  // rows of the tile, blocks of a copy
    const int grp = warp >> 2, row = (warp & 3) * 32 + lane;  // row of the tile, lane of tensor memory
    const int copy = row / ROWS, q_lo = copy * NQ;            // (the warp's)
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + T::TS + grp * 128, o_at = tmem + lanes + T::TO + grp * D;
    while (ok && seg.next(a, cta)) {
      const int h = seg.h, b = seg.b, r = seg.rt * ROWS + row % ROWS;
      const bool live = r < a.rows, idle = __all_sync(0xffffffffu, !live);
      // queries of the segment (the scores of the last one are done: their
      // barriers were waited for)
      query_rows<D, 2>(a, b, h, seg.rt, threadIdx.x, scales, [&](int n, int ch, uint4 x) {
        const int t = ch / (D / 4), u = ch % (D / 4) / 8, piece = (2 * t + (u & 1)) ^ (n & 7);
        *reinterpret_cast<uint4*>(smem + (u >> 1) * (kRows * 128) + n * 128 + piece * 16) = x;
      });
      fence_async_proxy();
      named_barrier_sync(3, kSoftmaxWarps * 32);  // scales[] is written
      mbar_arrive_if(lane == 0, q_full);
      const float scale = scales[row];
      float ref = -INFINITY, sum = 0.0f;  // reference in log2 units, bias included in neither
      const uint32_t seg_tile = tile;
      int last0 = -1, last1 = -1;  // the segment's last tile of each buffer
      bool failed = false;
#pragma unroll 1
      for (int blk = seg.blk0; blk < seg.blk1; blk += kTileBlocks, ++tile) {
        const uint32_t buf = tile & 1;
        if (buf) last1 = static_cast<int>(tile);
        else last0 = static_cast<int>(tile);
        if (buf != static_cast<uint32_t>(grp)) continue;
        const int nb = min(kTileBlocks, seg.blk1 - blk);
        // the columns each block shows this row, in token order
        uint32_t see[NQ];
        const bool plain = seg.plain(blk, nb);
#pragma unroll
        for (int q = 0; q < NQ; ++q) see[q] = 0xffffffffu;
        if (!plain) {
#pragma unroll 1
          for (int q = 0; q < NQ && q_lo + q < nb; ++q) {
            int idx;
            const int kind = block_kind(seg.seq, blk + q_lo + q, &idx);
            uint32_t m = column_mask(a, seg.seq, b, kind, idx);
            if (kind == kDraftBlock) m = live ? draft_bits(a, b, r % a.T, idx) : 0u;
#pragma unroll
            for (int k = 0; k < NQ; ++k)
              if (k == q) see[k] = m;
          }
        }
        if (!failed) failed = !pipe_wait_short(&s_full[buf], (tile >> 1) & 1, abort_flag);
        if (idle) {  // no row to weigh: whatever lies in these lanes stays in them
          mbar_arrive_if(lane == 0, &p_full[buf]);
          continue;
        }
        tc_fence_after();
        float top = -INFINITY;
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
          if (q_lo + q >= nb) continue;
          float s[32];
          tc_ld<32>(s_at + 32 * (q_lo + q), s);
          tc_wait_ld();
          if (plain) {
#pragma unroll
            for (int p = 0; p < 32; ++p) top = fmaxf(top, s[p]);
          } else {
#pragma unroll
            for (int p = 0; p < 32; ++p) top = see[q] >> token_of_position(p) & 1u ? fmaxf(top, s[p]) : top;
          }
        }
        top *= scale;
        if (__any_sync(0xffffffffu, top > ref + kLag)) {
          const float now = fmaxf(ref, top), f = now == -INFINITY ? 1.0f : exp2f(ref - now);
          ref = now;
          sum *= f;
          if (tile - seg_tile >= 2) {  // (these scores were issued behind O's last value product)
#pragma unroll 1
            for (int n = 0; n < D; n += 16) {
              float o[16];
              tc_ld<16>(o_at + n, o);
              tc_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] *= f;
              tc_st<16>(o_at + n, o);
            }
          }
        }
        const float off = ref == -INFINITY ? 0.0f : kBias - ref;
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
          if (q_lo + q >= nb) continue;
          float s[32];
          tc_ld<32>(s_at + 32 * (q_lo + q), s);
          tc_wait_ld();
          uint32_t w[16];
#pragma unroll
          for (int p = 0; p < 32; p += 2) {
            float2 d = __ffma2_rn(make_float2(s[p], s[p + 1]), make_float2(scale, scale), make_float2(off, off));
            if (!plain) {
              if (!(see[q] >> token_of_position(p) & 1u)) d.x = -INFINITY;
              if (!(see[q] >> token_of_position(p + 1) & 1u)) d.y = -INFINITY;
            }
            s[p] = fast_exp2(d.x);
            s[p + 1] = fast_exp2(d.y);
            w[p / 2] = f2_to_h2(s[p], s[p + 1]);
          }
          float2 part = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int p = 0; p < 32; p += 2) part = __fadd2_rn(part, make_float2(s[p], s[p + 1]));
          sum += part.x + part.y;
          // over scores of columns before the block's, which are read or not this copy's
          tc_st8(s_at + 16 * (q_lo + q), w);
          tc_st8(s_at + 16 * (q_lo + q) + 8, w + 8);
        }
        if (COPIES == 2) {  // the other copy's blocks
          const uint32_t zero[8] = {};
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            tc_st8(s_at + 16 * (NQ - q_lo + q), zero);
            tc_st8(s_at + 16 * (NQ - q_lo + q) + 8, zero);
          }
        }
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        mbar_arrive_if(lane == 0, &p_full[buf]);
      }
      // the two groups' states of every row, joined
      state[grp * kRows + row] = make_float2(ref == -INFINITY ? -INFINITY : ref - kBias, sum);
      named_barrier_sync(3, kSoftmaxWarps * 32);
      const bool whole = seg.blk0 == 0 && seg.blk1 == seg.seq.total;
      const bool joined = COPIES == 2 && whole;  // the copies' outputs are joined here
      const float2 s0 = state[row], s1 = state[kRows + row];
      float m = fmaxf(s0.x, s1.x);
      if (joined) m = fmaxf(m, fmaxf(state[row ^ ROWS].x, state[kRows + (row ^ ROWS)].x));
      const float f0 = s0.x == -INFINITY ? 0.0f : exp2f(s0.x - m), f1 = s1.x == -INFINITY ? 0.0f : exp2f(s1.x - m);
      float total = f0 * s0.y + f1 * s1.y;
      if (joined) {
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const float2 t = state[g * kRows + (row ^ ROWS)];
          if (t.x != -INFINITY) total = fmaf(exp2f(t.x - m), t.y, total);
        }
      }
      const size_t orow = (static_cast<size_t>(b) * a.geo.Hq + static_cast<size_t>(h) * a.geo.gqa) * a.T + r;
      const size_t prow = static_cast<size_t>(seg.slot) * kRows + row;
      if (grp == 0 && live) {
        if (!whole)
          reinterpret_cast<float2*>(a.part_ml)[prow] = make_float2(m, total);
        else if (a.lse && copy == 0)
          a.lse[orow] = total == 0.0f ? -INFINITY : (m + log2f(total)) * 0.69314718055994530942f;
      }
      if (last0 >= 0 && !failed) failed = !pipe_wait_short(&o_done[0], (last0 >> 1) & 1, abort_flag);
      if (last1 >= 0 && !failed) failed = !pipe_wait_short(&o_done[1], (last1 >> 1) & 1, abort_flag);
      tc_fence_after();
      const float inv = a.v_scale * (whole ? (total == 0.0f ? 0.0f : 1.0f / total) : 1.0f);
      const float c0 = f0 * inv, c1 = f1 * inv;
      auto output = [&](int n, float (&o)[8]) {  // channels n .. n + 7 of the row
        float o0[8], o1[8];
        tc_ld<8>(tmem + lanes + T::TO + n, o0);
        tc_ld<8>(tmem + lanes + T::TO + D + n, o1);
        tc_wait_ld();
#pragma unroll
        for (int j = 0; j < 8; ++j)  // column 4 (g & 1) + g / 2 is channel g; an O without a tile holds anything
          o[2 * (j & 3) + (j >> 2)] = (last0 >= 0 ? o0[j] * c0 : 0.0f) + (last1 >= 0 ? o1[j] * c1 : 0.0f);
      };
      // the second copy's part of the output goes through the queries' place (their products are done)
      float* other = reinterpret_cast<float*>(smem) + row % ROWS;
      if (joined) {
        if (copy == 1 && !failed) {
#pragma unroll 1
          for (int n = grp * (D / 2); n < (grp + 1) * (D / 2); n += 8) {
            float o[8];
            output(n, o);
#pragma unroll
            for (int j = 0; j < 8; ++j) other[(n + j) * ROWS] = o[j];
          }
        }
        named_barrier_sync(3, kSoftmaxWarps * 32);
      }
      if (!failed && !(joined && copy == 1)) {
#pragma unroll 1
        for (int n = grp * (D / 2); n < (grp + 1) * (D / 2); n += 8) {  // these warps write half of the channels
          float o[8];
          output(n, o);
          if (joined) {
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] += other[(n + j) * ROWS];
          }
          if (live) {
            for (int k = 0; k < a.draft_blocks; ++k) {  // values that are not finite, in the rows that see them
              uint32_t left = bad[8 * (n_seg & 7) + k];
              if (left) left &= draft_bits(a, b, r % a.T, k);
              for (; left; left &= left - 1) {
                const uint16_t* v =
                    a.vd + ((static_cast<size_t>(b) * a.geo.H + h) * a.T + kGroup * k + __ffs(left) - 1) * D + n;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  if ((v[j] & 0x7fffu) >= a.v_top) o[j] = fmaf(act_to_float(v[j], a.geo.act_bf16), INFINITY, o[j]);
              }
            }
            if (whole) {
              uint32_t w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                w[j] = static_cast<uint32_t>(float_to_act(o[2 * j], a.geo.act_bf16)) |
                       static_cast<uint32_t>(float_to_act(o[2 * j + 1], a.geo.act_bf16)) << 16;
              *reinterpret_cast<uint4*>(a.out + orow * D + n) = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
              // four channels of all rows together: a warp's store is 512 adjacent bytes
              float4* dst = reinterpret_cast<float4*>(a.part_o + static_cast<size_t>(seg.slot) * kRows * D) + n / 4 * kRows + row;
              dst[0] = make_float4(o[0], o[1], o[2], o[3]);
              dst[kRows] = make_float4(o[4], o[5], o[6], o[7]);
            }
          }
          __syncwarp();
        }
      }
      tc_fence_before();
      // the next segment's queries go over this one's when every softmax warp
      // is here; a failure makes all of them leave
      if (named_barrier_count(3, kSoftmaxWarps * 32, failed)) ok = false;
      ++n_seg;
    }
  } else if (warp < kScoreWarp) {
    registers_down<64>();
    const bool keys = warp < kValueWarp;
    const int w = warp & 7, g = lane >> 2, t = lane & 3;
    const uint8_t* raw = rest + T::RAW;
    const int chunk = a.geo.chunk.bytes;
    uint32_t st = 0, st_par = 0, vb = 0, v_par = 0;
    while (ok && seg.next(a, cta)) {
      if (!keys && a.draft_blocks) {
        if (lane < 8) bad[8 * ((n_seg + 3) & 7) + lane] = 0u;
        __syncwarp();
      }
#pragma unroll 1
      for (int blk = seg.blk0; blk < seg.blk1; blk += kTileBlocks, ++tile) {
        const uint32_t buf = tile & 1;
        ok = pipe_wait_short(&raw_full[st], st_par, abort_flag) &&
             (keys ? pipe_wait_short(&k_empty[buf], ((tile >> 1) & 1) ^ 1, abort_flag) : pipe_wait_short(&v_empty[vb], v_par ^ 1, abort_flag));
        if (!ok) break;
        const uint8_t* src = raw + st * kTileBlocks * chunk;
        if (keys) {  // m-tile w & 1 of block w / 2
          const int q = w >> 1, mt = w & 1;
          if (blk + q < seg.blk1) {
            uint8_t* at = smem + T::OFF_K + buf * T::KBYTES + (32 * q + 8 * (g >> 1) + 4 * mt + (g & 1)) * 128;
            block_keys<D, KB, 1>(a, seg, blk + q, src + q * chunk, mt, lane, [&](int s, int, const uint32_t(&v)[8]) {
              const int u = s >> 1;
#pragma unroll
              for (int r0 = 0; r0 < 2; ++r0) {
                const int piece = (2 * t + (u & 1)) ^ (4 * mt + 2 * r0 + (g & 1));
                *reinterpret_cast<uint4*>(at + (u >> 1) * (128 * 128) + r0 * 256 + piece * 16) =
                    make_uint4(v[r0], v[2 + r0], v[4 + r0], v[6 + r0]);
              }
            });
          }
        } else {  // channels 32 vg .. + 31 of NB blocks from q0 on
          constexpr int VG = D / 32, NB = kTileBlocks * VG / 8;
          const int vg = w % VG, q0 = w / VG * NB, rho = 4 * (g & 1) + (g >> 1);
          if (blk + q0 < seg.blk1) {
            uint8_t* at = smem + T::OFF_V + vb * T::VBYTES + (q0 >> 1) * (D * 128) + (32 * vg + rho) * 128;
            block_values<D, VB, NB>(a, seg, blk + q0, src + q0 * chunk, vg, lane, bad + 8 * (n_seg & 7),
                                    [&](int q, int mm, const uint32_t(&v)[8]) {
                                      const int piece = (4 * ((q0 + q) & 1) + t) ^ rho;
#pragma unroll
                                      for (int r0 = 0; r0 < 2; ++r0)
                                        *reinterpret_cast<uint4*>(at + (16 * mm + 8 * r0) * 128 + piece * 16) =
                                            make_uint4(v[r0], v[2 + r0], v[4 + r0], v[6 + r0]);
                                    });
          }
        }
        fence_async_proxy();
        __syncwarp();
        mbar_arrive_if(lane == 0, &raw_empty[st]);
        mbar_arrive_if(lane == 0, keys ? &k_full[buf] : &v_full[vb]);
        if (++st == static_cast<uint32_t>(n_stages)) st = 0, st_par ^= 1;
        if (++vb == static_cast<uint32_t>(n_v)) vb = 0, v_par ^= 1;
      }
      ++n_seg;
    }
  } else if (warp == kScoreWarp) {
    registers_down<40>();
    const uint64_t q_desc = smem_operand(smem_u32(smem), 1024), k_desc = smem_operand(smem_u32(smem + T::OFF_K), 1024);
    uint32_t seg_par = 0;
    while (ok && seg.next(a, cta)) {
      if (!(ok = pipe_wait_short(q_full, seg_par, abort_flag))) break;
      seg_par ^= 1;
#pragma unroll 1
      for (int blk = seg.blk0; blk < seg.blk1; blk += kTileBlocks, ++tile) {
        const uint32_t buf = tile & 1, par = (tile >> 1) & 1;
        // S holds the weights of tile - 2 until their value product is done
        if (!(ok = pipe_wait_short(&k_full[buf], par, abort_flag) && pipe_wait_short(&o_done[buf], par ^ 1, abort_flag))) break;
        tc_fence_after();
        const uint32_t instr = tc_instr(32 * min(kTileBlocks, seg.blk1 - blk), false);
        const uint32_t sc = tmem + T::TS + buf * 128;
        const uint64_t k = k_desc + buf * (T::KBYTES >> 4);
        if (elect_one()) {
#pragma unroll
          for (int s = 0; s < D / 16; ++s)
            tc_mma_ss(sc, q_desc + (((s >> 2) * (kRows * 128) + (s & 3) * 32) >> 4),
                      k + (((s >> 2) * (128 * 128) + (s & 3) * 32) >> 4), instr, s != 0);
          tc_commit(&k_empty[buf]);
          tc_commit(&s_full[buf]);
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
    const uint64_t v_desc = smem_operand(smem_u32(smem + T::OFF_V), 1024);
    uint32_t vb = 0, v_par = 0;
    while (ok && seg.next(a, cta)) {
      const uint32_t first = tile;
#pragma unroll 1
      for (int blk = seg.blk0; blk < seg.blk1; blk += kTileBlocks, ++tile) {
        const uint32_t buf = tile & 1, par = (tile >> 1) & 1;
        if (!(ok = pipe_wait_short(&v_full[vb], v_par, abort_flag) && pipe_wait_short(&p_full[buf], par, abort_flag))) break;
        tc_fence_after();
        const int steps = 2 * min(kTileBlocks, seg.blk1 - blk);
        const bool fresh = tile - first < 2;  // its O's first in the segment
        const uint32_t o = tmem + T::TO + buf * D, p = tmem + T::TS + buf * 128;
        const uint64_t v = v_desc + vb * (T::VBYTES >> 4);
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < 2 * kTileBlocks; ++j)
            if (j < steps)
              tc_mma(o, p + 8 * j, v + (((j >> 2) * (D * 128) + (j & 3) * 32) >> 4), tc_instr(D, false), !(fresh && j == 0));
          tc_commit(&v_empty[vb]);
          tc_commit(&o_done[buf]);
          mbar_arrive(&o_done[buf]);
        }
        __syncwarp();
        if (++vb == static_cast<uint32_t>(n_v)) vb = 0, v_par ^= 1;
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
    ok = copy_chunks(a, seg, cta, rest + T::RAW, n_stages, raw_full, raw_empty, abort_flag);
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

}  // namespace wide

template <int D, int KB, int VB, int COPIES>
cudaError_t launch_wide(const MultiAttnArgs& a, cudaStream_t s) {
  using namespace wide;
  static int configured[kMaxDevices] = {};  // per device and instance: the attribute is per device
  const int chunk = a.geo.chunk.bytes, smem = wide_smem<D>(chunk);
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (smem > configured[dev]) {
    e = cudaFuncSetAttribute(multi_wide_kernel<D, KB, VB, COPIES>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    configured[dev] = smem;
  }
  multi_wide_kernel<D, KB, VB, COPIES><<<a.n_ctas, kWideThreads, smem, s>>>(a, wide_stages<D>(chunk), wide_v_buffers<D>(chunk));
  return cudaGetLastError();
}

}  // namespace kvq
