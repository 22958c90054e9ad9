// Pieces of the attention of several queries per sequence (kv_tree_attn,
// kv_cross_attn): the blocks of 32 columns a (sequence, KV head) reads, the
// equal split of all units' blocks over the CTAs, the turning of a block of
// any kind into f16 tensor-core operands in registers, and the tcgen05
// wrappers.
#pragma once

#include "decode_kivi.cuh"

namespace kvq {

// The f16x2 pair 1024.0 of the 8-bit code conversion (decode_kivi.cuh).
constexpr uint32_t kH2Magic = 0x64006400u;

constexpr int kTileBlocks = 4;      // blocks of a tile: 128 columns
constexpr int kMaxStages = 8;       // tiles whose chunks may be in flight
// Weights are taken against a reference that moves only when a score exceeds
// it by 2^kLag, and carry a factor of 2^kBias (taken off the partial's max,
// exactly): in f16 (to 2^15 above; 11 bits down to 2^-14, 2^-25 rounds to
// zero) a weight keeps its bits to 2^-21 of the reference and is lost below
// 2^-32.
constexpr float kBias = 7.0f, kLag = 8.0f;

enum BlockKind { kGroupBlock = 0, kSinkBlock = 1, kTailBlock = 2, kDraftBlock = 3 };

// Blocks of one sequence: those of the quantised segment and of the tail end
// at its length. Blocks [plain0, plain1) are groups every token of which is
// read from its codes.
struct SeqBlocks {
  int64_t len;
  int groups, sinks, tail, total;
  int plain0, plain1;
};

__device__ __forceinline__ SeqBlocks seq_blocks(const MultiAttnArgs& a, int b) {
  SeqBlocks s;
  s.len = a.L;
  s.groups = a.n_groups;
  s.sinks = a.n_sink > 0;
  s.tail = a.tail_blocks;
  if (a.lens) {
    int64_t n = a.lens[b];
    n = n < 0 ? 0 : n > a.L ? a.L : n;
    s.len = n;
    const int64_t in = n - kGroup * a.g_begin, ex = n - a.F;
    s.groups = in <= 0 ? 0 : min(s.groups, static_cast<int>((in + kGroup - 1) / kGroup));
    s.tail = ex <= 0 ? 0 : min(s.tail, static_cast<int>((ex + kGroup - 1) / kGroup));
  }
  s.total = s.groups + s.sinks + s.tail + a.draft_blocks;
  const int64_t end = s.len < a.F ? s.len : a.F;
  s.plain0 = a.qlo > kGroup * a.g_begin;
  s.plain1 = a.geo.n_dyn || s.groups == 0 ? 0 : static_cast<int>(end / kGroup - a.g_begin);
  return s;
}

__device__ __forceinline__ int block_kind(const SeqBlocks& s, int i, int* idx) {
  if (i < s.groups) return *idx = i, kGroupBlock;
  i -= s.groups;
  if (i < s.sinks) return *idx = i, kSinkBlock;
  i -= s.sinks;
  if (i < s.tail) return *idx = i, kTailBlock;
  return *idx = i - s.tail, kDraftBlock;
}

// The flat list of items that the CTAs share out equally (fewer than 2^31: the
// host checks): sequences in order, each with H * row_tiles units of
// seq_blocks().total blocks, every unit led by a.seg_cost items that stand for
// what a segment costs beside its blocks (queries, joining, output), so that
// a CTA with many short units gets fewer blocks. `first_item` is the index of
// sequence b's first item, or with b = B the length of the list. Whole warps
// call it.
__device__ __forceinline__ int unit_items(const MultiAttnArgs& a, int total) { return total ? total + a.seg_cost : 0; }

__device__ __forceinline__ int first_item(const MultiAttnArgs& a, int b) {
  const int per = a.geo.H * a.row_tiles;
  if (!a.lens) return per * b * unit_items(a, seq_blocks(a, 0).total);
  int sum = 0;
#pragma unroll 1
  for (int i = threadIdx.x & 31; i < b; i += 32) sum += unit_items(a, seq_blocks(a, i).total);
  return per * __reduce_add_sync(0xffffffffu, sum);
}

// The sequence that holds item i of the list, and its first item. Whole warps.
__device__ __forceinline__ int find_sequence(const MultiAttnArgs& a, int i, int* first) {
  const int per = a.geo.H * a.row_tiles;
  if (!a.lens) {
    const int n = per * unit_items(a, seq_blocks(a, 0).total), b = i / n;
    *first = b * n;
    return b;
  }
  const int lane = threadIdx.x & 31;
  int base = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < a.geo.B; b0 += 32) {
    const int n = b0 + lane < a.geo.B ? per * unit_items(a, seq_blocks(a, b0 + lane).total) : 0;
    int incl = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += o;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, i < base + incl);
    if (hit) {
      const int l = __ffs(hit) - 1;
      *first = base + __shfl_sync(0xffffffffu, incl - n, l);
      return b0 + l;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  *first = base;
  return a.geo.B;
}

// CTAs that share a list of `work` items: lengths on the device may leave
// fewer items than the launch has CTAs, and every sharing CTA has one.
__device__ __forceinline__ int sharing_ctas(const MultiAttnArgs& a, int work) {
  return work < a.n_ctas ? work : a.n_ctas;
}
// The shares: CTA c's begins at item floor(c work / n), in 32 bits (a 64-bit
// division takes a kernel's start a quarter of a microsecond).
struct Shares {
  unsigned q, r, n;
  __device__ __forceinline__ Shares(int work, int ctas)
      : q(static_cast<unsigned>(work) / static_cast<unsigned>(ctas)),
        r(static_cast<unsigned>(work) % static_cast<unsigned>(ctas)), n(static_cast<unsigned>(ctas)) {}
  __device__ __forceinline__ int begin(int c) const {
    return static_cast<int>(static_cast<unsigned>(c) * q + static_cast<unsigned>(c) * r / n);
  }
  // the CTA that has item i: a guess that rounding leaves at most one off
  __device__ __forceinline__ int owner(int i) const {
    const float per = static_cast<float>(q) + static_cast<float>(r) / static_cast<float>(n);
    int c = min(static_cast<int>(n) - 1, static_cast<int>(static_cast<float>(i) / per));
    while (begin(c) > i) --c;
    while (begin(c + 1) <= i) ++c;
    return c;
  }
};

// Slot of a CTA's partial of a unit (kvq_internal.h): whether it begins the unit.
__device__ __forceinline__ int partial_slot(const MultiAttnArgs& a, int cta, int unit, bool begins) {
  return begins ? a.n_ctas + (a.cuts ? cta : unit) : cta;
}

// Walks a CTA's share [i0, i1) of the list one segment (the blocks of a unit
// inside the share) at a time.
struct SegmentCursor {
  int i0, i1;       // what is left of the share
  int first;        // first item of sequence b
  SeqBlocks seq;
  int b, h, rt;     // sequence, KV head, row tile of the current segment
  int blk0, blk1;   // its blocks
  int slot;         // its partial

  __device__ __forceinline__ void begin(const MultiAttnArgs& a, int cta) {
    const int work = first_item(a, a.geo.B), n = sharing_ctas(a, work);
    i0 = i1 = first = 0;
    b = 0;
    if (cta < n) {
      const Shares shares(work, n);
      i0 = shares.begin(cta);
      i1 = shares.begin(cta + 1);
      b = find_sequence(a, i0, &first);
      seq = seq_blocks(a, b);
    }
  }
  __device__ __forceinline__ bool next(const MultiAttnArgs& a, int cta) {
    const int per = a.geo.H * a.row_tiles;
#pragma unroll 1
    while (i0 < i1) {
      const int items = unit_items(a, seq.total);
      if (i0 >= first + per * items) {  // on to the next sequence
        first += per * items;
        seq = seq_blocks(a, ++b);
        continue;
      }
      const unsigned u = static_cast<unsigned>(i0 - first) / static_cast<unsigned>(items);
      const int in = i0 - first - static_cast<int>(u) * items, take = min(items - in, i1 - i0);
      i0 += take;
      blk0 = max(0, in - a.seg_cost);
      blk1 = max(0, in + take - a.seg_cost);
      if (blk0 == blk1) continue;  // only the unit's lead
      h = static_cast<int>(u / static_cast<unsigned>(a.row_tiles));
      rt = static_cast<int>(u) - h * a.row_tiles;
      slot = partial_slot(a, cta, (b * a.geo.H + h) * a.row_tiles + rt, blk0 == 0);
      return true;
    }
    return false;
  }
  // whether blocks [blk, blk + n) are plain groups
  __device__ __forceinline__ bool plain(int blk, int n) const { return blk >= seq.plain0 && blk + n <= seq.plain1; }
};

// Up to 32 polls of phase `parity` of `bar` by a whole warp, three instructions
// each; true once it is complete. A poll that finds it incomplete is suspended
// until it completes, or for the hardware's own limit, 7860 cycles as
// multi_wait_probe_kernel measures them: a round that fails takes 0.25 M cycles,
// an eighth of a millisecond. (With a limit of a microsecond given the hardware
// waits as long, and the ring shape takes 163 us instead of 155.)
__device__ __forceinline__ bool pipe_poll(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
      "mov.u32 n, 32;\n"
      "again:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "@p bra over;\n\t"
      "sub.u32 n, n, 1;\n\t"
      "setp.ne.u32 q, n, 0;\n\t"
      "@q bra again;\n"
      "over:\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return __all_sync(0xffffffffu, done != 0);
}

// Wait of a whole warp for phase `parity` of `bar`, bounded and abortable as
// warp_wait is. Many warps wait at any time here and share the schedulers with
// those that work, so the clock and the abort flag are looked at once a round
// of polls: a third of all instructions were polls with warp_wait.
__device__ __forceinline__ bool pipe_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                          long long budget = kWaitCycles) {
  const uint32_t addr = smem_u32(bar);
  if (pipe_poll(addr, parity)) return true;
  const long long t0 = clock64();
  while (true) {
    if (pipe_poll(addr, parity)) return true;
    if (__any_sync(0xffffffffu, *abort_flag != 0)) return false;
    if (__any_sync(0xffffffffu, clock64() - t0 > budget)) {
      *abort_flag = 1;
      return false;
    }
  }
}

// The same with less code, for the kernel of 128-row tiles, whose roles do not
// fit the instruction cache together otherwise (ring shape 208 -> 191 us, 384
// queries 218 -> 211 us; in the other kernel batch 16 went from 202 to 219 us
// with it): the bound is a count of rounds, 2^13 of them 2.06 G cycles, about a
// second. (With the clock read in every round the ring shape takes 157 us
// instead of 155, 384 queries 187.7 instead of 186.3.)
constexpr int kWaitRounds = 1 << 13;
__device__ __forceinline__ bool pipe_wait_short(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                                int rounds = kWaitRounds) {
  const uint32_t addr = smem_u32(bar);
#pragma unroll 1
  for (int i = 0; i < rounds; ++i) {
    if (pipe_poll(addr, parity)) return true;
    if (__any_sync(0xffffffffu, *abort_flag != 0)) return false;
  }
  *abort_flag = 1;
  return false;
}

// Which columns of a block every row of the sequence may see (bit j: column
// j); of a draft block, those that exist. Whole warps.
__device__ __forceinline__ uint32_t column_mask(const MultiAttnArgs& a, const SeqBlocks& s, int b, int kind, int idx) {
  const int lane = threadIdx.x & 31;
  bool ok;
  if (kind == kGroupBlock) {
    const int64_t grp = a.g_begin + idx, pos = kGroup * grp;
    ok = pos + lane >= a.qlo && pos + lane < a.F && pos + lane < s.len;
    if (a.geo.n_dyn)
      ok = ok && !(a.lay.sink_mask[static_cast<size_t>(b) * a.geo.n_slots + grp % a.geo.n_slots] >> lane & 1u);
  } else if (kind == kSinkBlock) {
    const int64_t pos = lane >= a.n_sink ? a.L : a.geo.n_dyn ? a.lay.sink_pos[b * kMaxSinks + lane] : lane;
    ok = lane < a.n_sink && pos < a.F && pos < s.len;  // a sink still in the tail is read there
  } else if (kind == kTailBlock) {
    const int64_t pos = a.F + kGroup * idx + lane;
    ok = pos < a.L && pos < s.len;
  } else {
    ok = kGroup * idx + lane < a.T;
  }
  return __ballot_sync(0xffffffffu, ok);
}

// Drafted tokens of block idx that query i of sequence b sees.
__device__ __forceinline__ uint32_t draft_bits(const MultiAttnArgs& a, int b, int i, int idx) {
  const uint64_t w = a.mask[(static_cast<size_t>(b) * a.T + i) * a.mask_words + (idx >> 1)];
  const uint32_t m = static_cast<uint32_t>(idx & 1 ? w >> 32 : w);
  const int left = a.T - kGroup * idx;
  return left >= kGroup ? m : m & ((1u << left) - 1u);
}

// Position of drafted token i behind the layer's end: the drafted tokens it
// sees, less itself.
__device__ __forceinline__ int draft_depth(const MultiAttnArgs& a, int b, int i) {
  int n = 0;
  for (int k = 0; k < a.draft_blocks; ++k) n += __popc(draft_bits(a, b, i, k));
  return n > 0 ? n - 1 : 0;
}

// f16x2 of two activations times a unit: exact in f16's normal range.
__device__ __forceinline__ uint32_t act2_to_h2(uint32_t x, int bf16, float unit) {
  if (!bf16) return as_u32(__hmul2(as_h2(x), __float2half2_rn(unit)));
  return f2_to_h2(__uint_as_float(x << 16) * unit, __uint_as_float(x & 0xffff0000u) * unit);
}

// Keys and values are held times a unit, 2^-unit_shift: 1/2 and 1/8 for 2- and
// 3-bit codes, whose conversions give code / 2 and code / 8, else 1. The
// score's scale and the output's take it off again (powers of two: only a value
// below 2^-11 can lose bits, and no more than 2^-22). 4-bit codes come as
// code / 512: there the unit would cost small values their bits, and the
// multiplication stays with the code.
__host__ __device__ constexpr int unit_shift(int bits) { return bits == 2 ? 1 : bits == 3 ? 3 : 0; }

// The code pair P of a lane's words as an f16x2 of code * unit (exact).
template <int BITS>
__device__ __forceinline__ uint32_t code_units(const uint32_t* w, int P) {
  CodeConsts<BITS> cc;
  cc.magic = kH2Magic;
  const uint32_t x = pair_at<BITS>(cc, w, P);
  return BITS == 4 ? as_u32(__hmul2(as_h2(x), as_h2(h2pow2(9)))) : x;
}
// A zero point (pair) times the unit.
template <int BITS>
__device__ __forceinline__ uint32_t zero_units(uint32_t z) {
  return unit_shift(BITS) ? as_u32(__hmul2(as_h2(z), as_h2(h2pow2(-unit_shift(BITS))))) : z;
}

// The keys of a group as the tensor core's A fragments (rows = tokens, k =
// channels in the order of kvq_layout.h): put(first k-step, m-tile, 8 words)
// with the four words of each of two k-steps. Each value is
// RN((code * s + z) * unit) in f16: one rounding, as of a key held in f16. (A
// single query takes the scales and zeros itself, with a residual, against
// exact codes; for many that is a copy of all of them per group. Where a few
// channels are ten times the others the rounding is the largest error of the
// result, 6e-4 to 1.4e-3 of it; keys in two f16 terms would double these loops
// and the score products.)
template <int D, int KB, class Put>
__device__ __forceinline__ void group_keys(const uint8_t* chunk, int lane, Put put) {
  constexpr int S = D / 16, KW = D * KB / 32, PW = piece_words(KW);
  const int t = lane & 3;
  const uint8_t* meta = chunk + kGroup * D * KB / 8;
  uint32_t w[KW];
  load_lane_words<KW, PW>(chunk, lane, w);
#pragma unroll
  for (int u = 0; u < S / 2; ++u) {
    const uint4 s4 = reinterpret_cast<const uint4*>(meta)[u * 4 + t];
    const uint32_t sc[4] = {s4.x, s4.y, s4.z, s4.w};  // q = 2 ds + p: k-step 2u + ds, k-half p
    uint32_t z[4];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      z[q] = zero_units<KB>(
          *reinterpret_cast<const uint32_t*>(meta + 2 * D + 2 * ((2 * u + (q >> 1)) * 16 + 2 * t + 8 * (q & 1))));
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      uint32_t v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {  // i = 4 ds + r: row half r & 1, k-half r >> 1
        const int q = 2 * (i >> 2) + ((i & 3) >> 1);
        v[i] = hfma2_bits(code_units<KB>(w, (m * S + 2 * u) * 4 + i), sc[q], z[q]);
      }
      put(2 * u, m, v);
    }
  }
}

// m-tile mt (16 tokens) of a group's keys, as group_keys. The loop stays a loop:
// the roles of the kernel of 128-row tiles share the instruction cache with
// less of it (ring shape 191 -> 187 us).
template <int D, int KB, class Put>
__device__ __forceinline__ void group_keys_half(const uint8_t* chunk, int mt, int lane, Put put) {
  constexpr int S = D / 16, KW = D * KB / 32, PW = piece_words(KW);
  constexpr int UU = KB == 3 ? 2 : 1;  // pairs of k-steps to an iteration: a 3-bit block of 32 codes is two
  constexpr int W = UU * KB / 2;       // words of a lane and iteration
  const int t = lane & 3;
  const uint8_t* meta = chunk + kGroup * D * KB / 8;
#pragma unroll 1
  for (int u0 = 0; u0 < S / 2; u0 += UU) {
    uint32_t w[W];
    const int first = mt * (KW / 2) + u0 / UU * W;
    if constexpr (W == 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(chunk + code_word_offset(lane, first, PW));
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (W == 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(chunk + code_word_offset(lane, first, PW));
      w[0] = v.x, w[1] = v.y;
    } else {
#pragma unroll
      for (int k = 0; k < W; ++k)
        w[k] = *reinterpret_cast<const uint32_t*>(chunk + code_word_offset(lane, first + k, PW));
    }
#pragma unroll
    for (int du = 0; du < UU; ++du) {
      const int u = u0 + du;
      const uint4 s4 = reinterpret_cast<const uint4*>(meta)[u * 4 + t];
      const uint32_t sc[4] = {s4.x, s4.y, s4.z, s4.w};  // q = 2 ds + p: k-step 2u + ds, k-half p
      uint32_t z[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        z[q] = zero_units<KB>(
            *reinterpret_cast<const uint32_t*>(meta + 2 * D + 2 * ((2 * u + (q >> 1)) * 16 + 2 * t + 8 * (q & 1))));
      uint32_t v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {  // i = 4 ds + r: row half r & 1, k-half r >> 1
        const int q = 2 * (i >> 2) + ((i & 3) >> 1);
        v[i] = hfma2_bits(code_units<KB>(w, 8 * du + i), sc[q], z[q]);
      }
      put(2 * u, mt, v);
    }
  }
}

// Values of one group and the 32 channels of channel group vg as A fragments
// (rows = channels, k = tokens): put(m-tile of the two, 8 words) with the four
// words of each of the group's two k-steps. Columns outside `cols` become
// zero whatever their scale holds.
template <int D, int VB, class Put>
__device__ __forceinline__ void group_values(const uint8_t* region, int vg, int lane, uint32_t cols, Put put) {
  constexpr int PW = piece_words(D * VB / 32);
  const int t = lane & 3;
  const uint8_t* meta = region + kGroup * D * VB / 8;
  uint32_t w[VB];  // the lane's words of the two m-tiles
  if constexpr (VB == 4 || VB == 8) {
#pragma unroll
    for (int k = 0; k < VB / 4; ++k) {
      const uint4 v = *reinterpret_cast<const uint4*>(region + code_word_offset(lane, vg * VB + 4 * k, PW));
      w[4 * k] = v.x, w[4 * k + 1] = v.y, w[4 * k + 2] = v.z, w[4 * k + 3] = v.w;
    }
  } else if constexpr (VB == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(region + code_word_offset(lane, vg * VB, PW));
    w[0] = v.x, w[1] = v.y;
  } else {
#pragma unroll
    for (int k = 0; k < VB; ++k)
      w[k] = *reinterpret_cast<const uint32_t*>(region + code_word_offset(lane, vg * VB + k, PW));
  }
  const uint4 s4 = *reinterpret_cast<const uint4*>(meta + 2 * (vg * 32 + 8 * t));
  const uint32_t sc[4] = {s4.x, s4.y, s4.z, s4.w};  // k = 2 kb + h: tokens 16 kb + 8 h + 2 t, + 1
  uint32_t z[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    z[k] = zero_units<VB>(*reinterpret_cast<const uint32_t*>(meta + 2 * (D + vg * 32 + 8 * k + 2 * t)));
#pragma unroll
  for (int mm = 0; mm < 2; ++mm) {
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // i = 4 kb + r: channel half r & 1, token half r >> 1
      const int k = 2 * (i >> 2) + ((i & 3) >> 1);
      v[i] = hfma2_bits(code_units<VB>(w, mm * 8 + i), sc[k], z[k]);
    }
    if (cols != 0xffffffffu) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t two = cols >> (16 * (i >> 2) + 8 * ((i & 3) >> 1) + 2 * t);
        v[i] &= (two & 1u ? 0x0000ffffu : 0u) | (two & 2u ? 0xffff0000u : 0u);
      }
    }
    put(mm, v);
  }
}

// The rows of an exact block: row j at base + ((first + j) & wrap) * D.
struct ExactRows {
  size_t base;   // elements, from the start of the sinks', the tail's or the drafted keys (values)
  int first, wrap;
};
__device__ __forceinline__ ExactRows exact_rows(const MultiAttnArgs& a, int b, int h, int kind, int idx) {
  const size_t bh = static_cast<size_t>(b) * a.geo.H + h;
  const int D = a.geo.D;
  if (kind == kSinkBlock) return {bh * a.geo.n_sink_slots * D, 0, ~0};
  if (kind == kTailBlock) {
    const int wrap = a.geo.tail_cap - 1;
    return {bh * a.geo.tail_cap * D, static_cast<int>((a.F + kGroup * idx) & wrap), wrap};
  }
  return {bh * a.T * D, kGroup * idx, ~0};
}

// m-tile mt of an exact block's keys (rows outside `cols`, a mask of those
// that exist and count, are zero): put as group_keys. Drafted keys are
// rotated at their position when the cache applies RoPE and rounded to the
// activation type, as an append would store them.
template <int D, class Put>
__device__ __forceinline__ void exact_keys(const MultiAttnArgs& a, int b, int h, int kind, int idx, uint32_t cols,
                                           int mt, int lane, Put put) {
  constexpr int S = D / 16;
  const int g = lane >> 2, t = lane & 3, bf = a.geo.act_bf16;
  const uint16_t* src = kind == kSinkBlock ? a.lay.sink_k : kind == kTailBlock ? a.lay.tail_k : a.kd;
  const ExactRows rows = exact_rows(a, b, h, kind, idx);
  src += rows.base;
  const bool rot = kind == kDraftBlock && a.tab.rope;
  const uint16_t* row[2];
  const float* tab[2] = {};
#pragma unroll
  for (int r0 = 0; r0 < 2; ++r0) {
    const int j = 16 * mt + g + 8 * r0;
    row[r0] = cols >> j & 1u ? src + ((rows.first + j) & rows.wrap) * D : nullptr;
    if (rot && row[r0]) tab[r0] = a.tab.rope + static_cast<size_t>(a.L + draft_depth(a, b, kGroup * idx + j)) * D;
  }
#pragma unroll 2
  for (int u = 0; u < S / 2; ++u) {  // the lane's channels t D / 4 + 8u .. + 7: two k-steps
    uint32_t v[8];
#pragma unroll
    for (int r0 = 0; r0 < 2; ++r0) {
      uint4 x = make_uint4(0u, 0u, 0u, 0u);
      const int c = t * (D / 4) + 8 * u;
      if (row[r0]) {
        x = *reinterpret_cast<const uint4*>(row[r0] + c);
        if (rot) {
          uint4 y = *reinterpret_cast<const uint4*>(row[r0] + (c < D / 2 ? c + D / 2 : c - D / 2));
          if (c < D / 2) {
            rotate8(x, y, tab[r0], c, bf);
          } else {
            rotate8(y, x, tab[r0], c - D / 2, bf);
          }
        }
      }
      v[r0] = act2_to_h2(x.x, bf, a.k_unit), v[2 + r0] = act2_to_h2(x.y, bf, a.k_unit);
      v[4 + r0] = act2_to_h2(x.z, bf, a.k_unit), v[6 + r0] = act2_to_h2(x.w, bf, a.k_unit);
    }
    __syncwarp();
    put(2 * u, mt, v);
  }
}

// The same with all of a lane's loads in flight together, for 33 and more rows
// (ring shape 178 -> 155 us; up to 32 rows, where the code of all roles is
// longer than the instruction cache takes, batch 16 went from 201 to 224 us).
template <int D, class Put>
__device__ __forceinline__ void exact_keys_at_once(const MultiAttnArgs& a, int b, int h, int kind, int idx,
                                                   uint32_t cols, int mt, int lane, Put put) {
  constexpr int S = D / 16;
  const int g = lane >> 2, t = lane & 3, bf = a.geo.act_bf16;
  const uint16_t* src = kind == kSinkBlock ? a.lay.sink_k : kind == kTailBlock ? a.lay.tail_k : a.kd;
  const ExactRows rows = exact_rows(a, b, h, kind, idx);
  src += rows.base;
  const bool rot = kind == kDraftBlock && a.tab.rope;
  const uint16_t* row[2];
  const float* tab[2] = {};
#pragma unroll
  for (int r0 = 0; r0 < 2; ++r0) {
    const int j = 16 * mt + g + 8 * r0;
    row[r0] = cols >> j & 1u ? src + ((rows.first + j) & rows.wrap) * D : nullptr;
    if (rot && row[r0]) tab[r0] = a.tab.rope + static_cast<size_t>(a.L + draft_depth(a, b, kGroup * idx + j)) * D;
  }
  // the lane's channels t D / 4 + 8u .. + 7 are two k-steps
  auto place = [&](int u, const uint4 (&x)[2]) {
    const uint32_t v[8] = {act2_to_h2(x[0].x, bf, a.k_unit), act2_to_h2(x[1].x, bf, a.k_unit),
                           act2_to_h2(x[0].y, bf, a.k_unit), act2_to_h2(x[1].y, bf, a.k_unit),
                           act2_to_h2(x[0].z, bf, a.k_unit), act2_to_h2(x[1].z, bf, a.k_unit),
                           act2_to_h2(x[0].w, bf, a.k_unit), act2_to_h2(x[1].w, bf, a.k_unit)};
    put(2 * u, mt, v);
  };
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  if (rot) {
#pragma unroll 1
    for (int u = 0; u < S / 2; ++u) {
      const int c = t * (D / 4) + 8 * u, pair = c < D / 2 ? D / 2 : -(D / 2);
      uint4 x[2] = {zero, zero};
#pragma unroll 1
      for (int r0 = 0; r0 < 2; ++r0) {
        const uint16_t* from = r0 ? row[1] : row[0];
        if (!from) continue;
        uint4 lo = *reinterpret_cast<const uint4*>(from + c), hi = *reinterpret_cast<const uint4*>(from + c + pair);
        if (pair < 0) {
          const uint4 swap = lo;
          lo = hi, hi = swap;
        }
        rotate8(lo, hi, r0 ? tab[1] : tab[0], pair < 0 ? c - D / 2 : c, bf);
        if (r0) x[1] = pair < 0 ? hi : lo;
        else x[0] = pair < 0 ? hi : lo;
      }
      __syncwarp();
      place(u, x);
    }
    return;
  }
  uint4 x[S / 2][2];  // all in flight together
#pragma unroll
  for (int u = 0; u < S / 2; ++u)
#pragma unroll
    for (int r0 = 0; r0 < 2; ++r0)
      x[u][r0] = row[r0] ? *reinterpret_cast<const uint4*>(row[r0] + t * (D / 4) + 8 * u) : zero;
  __syncwarp();
#pragma unroll
  for (int u = 0; u < S / 2; ++u) place(u, x[u]);
}

// Values of an exact block and channel group vg: put as group_values; columns
// outside `cols` are zero. A lane loads a channel pair of every eighth row,
// and eight rows by eight channels are transposed at a time. In a draft block
// a value that is not finite in f16 (a bf16 value from 65536 / v_unit on among
// them) is put as zero too, so that it cannot meet the zero weight of a row
// that does not see it; returns the columns that had one (in every lane).
template <int D, class Put>
__device__ __forceinline__ uint32_t exact_values(const MultiAttnArgs& a, int b, int h, int kind, int idx, int vg,
                                                 uint32_t cols, int lane, Put put) {
  const int g = lane >> 2, t = lane & 3, bf = a.geo.act_bf16;
  const uint16_t* src = kind == kSinkBlock ? a.lay.sink_v : kind == kTailBlock ? a.lay.tail_v : a.vd;
  const ExactRows rows = exact_rows(a, b, h, kind, idx);
  src += rows.base + 32 * vg + 2 * t;
  uint32_t x[4][4];  // [row 8k + g][channels 32 vg + 8i + 2t, + 1]
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int j = 8 * k + g;
    const uint16_t* row = src + ((rows.first + j) & rows.wrap) * D;
    const bool in = cols >> j & 1u;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[k][i] = in ? *reinterpret_cast<const uint32_t*>(row + 8 * i) : 0u;
  }
  uint32_t bad = 0;
  if (kind == kDraftBlock) {
    const uint32_t top = a.v_top;
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if ((x[k][i] & 0x7fffu) >= top) x[k][i] &= 0xffff0000u, bad |= 1u << (8 * k + g);
        if ((x[k][i] & 0x7fff0000u) >= top << 16) x[k][i] &= 0x0000ffffu, bad |= 1u << (8 * k + g);
      }
  }
  __syncwarp();
#pragma unroll
  for (int mm = 0; mm < 2; ++mm) {
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)  // i = 4 kb + r: channel half r & 1, token half r >> 1
      v[i] = act2_to_h2(movmatrix_t(x[2 * (i >> 2) + ((i & 3) >> 1)][2 * mm + (i & 1)]), bf, a.v_unit);
    put(mm, v);
  }
  if (kind != kDraftBlock) return 0u;
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) bad |= __shfl_xor_sync(0xffffffffu, bad, off);
  return bad;
}

// The keys of NM m-tiles from mt on of block blk of a segment; `chunk`: its
// group's, if it is one. Columns that do not count come out as anything.
template <int D, int KB, int NM, class Put>
__device__ __forceinline__ void block_keys(const MultiAttnArgs& a, const SegmentCursor& seg, int blk, const uint8_t* chunk,
                                           int mt, int lane, Put put) {
  if (blk < seg.seq.groups) {
    if constexpr (NM == 2) group_keys<D, KB>(chunk, lane, put);
    else group_keys_half<D, KB>(chunk, mt, lane, put);
  } else {
    int idx;
    const int kind = block_kind(seg.seq, blk, &idx);
    const uint32_t cols = column_mask(a, seg.seq, seg.b, kind, idx);
#pragma unroll 1
    for (int m = 0; m < NM; ++m) {
      if constexpr (NM == 2) exact_keys<D>(a, seg.b, seg.h, kind, idx, cols, mt + m, lane, put);
      else exact_keys_at_once<D>(a, seg.b, seg.h, kind, idx, cols, mt + m, lane, put);
    }
  }
}

// Values of channel group vg of NB blocks from blk on, put(block, m-tile of
// the two, 8 words); `src`: the blocks' chunks, where they are groups. Columns
// that do not count are zero. Draft blocks' columns that held a value that is
// not finite in f16 go to bad[].
template <int D, int VB, int NB, class Put>
__device__ __forceinline__ void block_values(const MultiAttnArgs& a, const SegmentCursor& seg, int blk, const uint8_t* src,
                                             int vg, int lane, uint32_t* bad, Put put) {
  const int chunk = a.geo.chunk.bytes;
  src += a.geo.chunk.vc_off;
  if (blk + NB <= seg.blk1 && seg.plain(blk, NB)) {
    // (all blocks' words are in flight together: a warp alone hides no latency)
#pragma unroll
    for (int q = 0; q < NB; ++q)
      group_values<D, VB>(src + q * chunk, vg, lane, 0xffffffffu,
                          [&](int mm, const uint32_t(&v)[8]) { put(q, mm, v); });
    return;
  }
#pragma unroll 1
  for (int q = 0; q < NB && blk + q < seg.blk1; ++q) {
    auto one = [&](int mm, const uint32_t(&v)[8]) { put(q, mm, v); };
    int idx;
    const int kind = block_kind(seg.seq, blk + q, &idx);
    const uint32_t cols = seg.plain(blk + q, 1) ? 0xffffffffu : column_mask(a, seg.seq, seg.b, kind, idx);
    if (kind == kGroupBlock) {
      group_values<D, VB>(src + q * chunk, vg, lane, cols, one);
    } else {
      const uint32_t x = exact_values<D>(a, seg.b, seg.h, kind, idx, vg, cols, lane, one);
      if (x && lane == 0) atomicOr(&bad[idx], x);
    }
  }
}

// The copy warp: the groups' chunks of every tile into its stage, in one bulk
// copy where they are adjacent in the ring. Returns false when a wait gave up
// (its copies have landed by then).
__device__ __forceinline__ bool copy_chunks(const MultiAttnArgs& a, SegmentCursor& seg, int cta, uint8_t* raw, int n_stages,
                                            uint64_t* full, uint64_t* empty, volatile int* abort_flag) {
  const int chunk = a.geo.chunk.bytes, n_slots = a.geo.n_slots;
  const int slot0 = static_cast<int>(a.g_begin % n_slots);
  uint32_t st = 0, st_par = 0, issued = 0;
  bool ok = true;
  while (ok && seg.next(a, cta)) {
    const uint8_t* unit = a.lay.chunks + (static_cast<size_t>(seg.b) * a.geo.H + seg.h) * n_slots * chunk;
    int slot = static_cast<int>((static_cast<unsigned>(slot0) + seg.blk0) % n_slots);  // ring slot of block blk
#pragma unroll 1
    for (int blk = seg.blk0; blk < seg.blk1; blk += kTileBlocks) {
      if (!(ok = warp_wait(&empty[st], st_par ^ 1, abort_flag))) break;  // (tiles ahead: it may sleep)
      const int n = max(0, min(min(kTileBlocks, seg.blk1 - blk), seg.seq.groups - blk));  // groups come first
      const int n0 = min(n, n_slots - slot);
      if ((threadIdx.x & 31) == 0) {
        uint8_t* dst = raw + st * kTileBlocks * chunk;
        mbar_expect_tx(&full[st], static_cast<uint32_t>(n * chunk));
        if (n0 > 0) bulk_g2s(dst, unit + static_cast<size_t>(slot) * chunk, n0 * chunk, &full[st]);
        for (int i = n0; i < n; ++i)  // (a ring shorter than a tile wraps more than once)
          bulk_g2s(dst + i * chunk, unit + static_cast<size_t>((slot + i) % n_slots) * chunk, chunk, &full[st]);
      }
      __syncwarp();
      slot = (slot + kTileBlocks) % n_slots;
      ++issued;
      if (++st == static_cast<uint32_t>(n_stages)) st = 0, st_par ^= 1;
    }
  }
  if (!ok && (threadIdx.x & 31) == 0) {
    const uint32_t n = min(issued, static_cast<uint32_t>(n_stages));
    for (uint32_t i = 1; i <= n; ++i) {
      const uint32_t t = issued - i;
      (void)mbar_wait_bounded(&full[t % n_stages], (t / n_stages) & 1);
    }
  }
  __syncwarp();
  return ok;
}

// Queries of a row tile in f16 (and over again where the threads are for more
// rows): TPR threads a row, put(row of the tile, first of eight channels, those
// as f16). A row is rotated in fp32 when the cache applies RoPE, scaled by a
// power of two that brings its largest value near one, so that bf16 queries
// keep their bits in f16 whatever their size, and rounded once; scale[row]
// turns a dot product into a score in log2 units. Rows that do not exist are
// zero. Threads of a row are adjacent lanes of one warp.
template <int D, int TPR, class Put>
__device__ __forceinline__ void query_rows(const MultiAttnArgs& a, int b, int h, int rt, int tid, float* scale, Put put) {
  constexpr int HC = D / 16, NP = (HC + TPR - 1) / TPR;  // chunk pairs of a row, and of a thread
  const int n = tid / TPR, sub = tid % TPR, r = rt * a.tile_rows + n % a.tile_rows, bf = a.geo.act_bf16;
  const bool live = r < a.rows;
  const uint16_t* row = a.q + (static_cast<size_t>(b) * a.geo.Hq + static_cast<size_t>(h) * a.geo.gqa) * a.T * D +
                        static_cast<size_t>(r) * D;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  auto chunk = [&](int c) { return live ? reinterpret_cast<const uint4*>(row)[c] : zero; };
  // the largest magnitude, by its bits
  uint32_t top2 = 0u;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int c = sub + i * TPR;
    const uint4 lo = c < HC ? chunk(c) : zero, hi = c < HC ? chunk(c + HC) : zero;
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) top2 = __vmaxu2(top2, w[k] & 0x7fff7fffu);
  }
#pragma unroll
  for (int off = TPR / 2; off >= 1; off >>= 1) top2 = __vmaxu2(top2, __shfl_xor_sync(0xffffffffu, top2, off));
  const float top = act_to_float(static_cast<uint16_t>(max(top2 & 0xffffu, top2 >> 16)), bf);
  int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
  e = e < -100 ? -100 : e > 100 ? 100 : e;
  const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  const float* tab = nullptr;
  if (live && a.tab.rope) tab = a.tab.rope + static_cast<size_t>(a.L + draft_depth(a, b, r % a.T)) * D;
  // (a loop, over rows read again: as fast as unrolled, with less code)
#pragma unroll 1
  for (int i = 0; i < NP; ++i) {
    const int c = sub + i * TPR;
    if (c >= HC) continue;
    const uint4 lo = chunk(c), hi = chunk(c + HC);
    const uint32_t w8[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    float x[16];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      x[2 * k] = act_to_float(static_cast<uint16_t>(w8[k] & 0xffffu), bf);
      x[2 * k + 1] = act_to_float(static_cast<uint16_t>(w8[k] >> 16), bf);
    }
    if (tab) {
#pragma unroll
      for (int k = 0; k < 8; k += 2) {
        const float4 cs = *reinterpret_cast<const float4*>(tab + 2 * (8 * c + k));
        rope_pair(x[k], x[8 + k], cs.x, cs.y, &x[k], &x[8 + k]);
        rope_pair(x[k + 1], x[9 + k], cs.z, cs.w, &x[k + 1], &x[9 + k]);
      }
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = f2_to_h2(x[8 * half + 2 * k] * down, x[8 * half + 2 * k + 1] * down);
      put(n, 8 * c + half * (D / 2), make_uint4(w[0], w[1], w[2], w[3]));
    }
  }
  if (sub == 0) scale[n] = a.qscale * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
}

// ------------------------------------------------------------------ tcgen05
// Tensor memory addresses: lane in bits 16 .. 31, 32-bit column in 0 .. 15. A
// warp reaches the 32 lanes of its quarter (warp index mod 4).

__device__ __forceinline__ void tc_alloc(uint32_t* smem_addr, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(smem_addr)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_dealloc(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// The generic proxy's shared-memory writes become visible to the tensor core.
__device__ __forceinline__ void fence_async_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Two A fragments (16 rows x 32 k, 8 words a lane) into 16 lanes x 16 columns:
// word (row g + 8 i, column t + 4 j) from lane 4 g + t, register 2 j + i.
__device__ __forceinline__ void tc_st_frag2(uint32_t addr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// Eight words a thread into eight columns of its lane.
__device__ __forceinline__ void tc_st8(uint32_t addr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// N consecutive columns of the warp's 32 lanes, one lane a thread.
template <int N>
__device__ __forceinline__ void tc_ld(uint32_t addr, float (&v)[N]) {
  static_assert(N % 8 == 0, "eights");
#pragma unroll
  for (int i = 0; i < N; i += 8) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(addr + i));
#pragma unroll
    for (int k = 0; k < 8; ++k) v[i + k] = __uint_as_float(r[k]);
  }
}
template <int N>
__device__ __forceinline__ void tc_st(uint32_t addr, const float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 8)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr + i),
                 "r"(__float_as_uint(v[i])), "r"(__float_as_uint(v[i + 1])), "r"(__float_as_uint(v[i + 2])),
                 "r"(__float_as_uint(v[i + 3])), "r"(__float_as_uint(v[i + 4])), "r"(__float_as_uint(v[i + 5])),
                 "r"(__float_as_uint(v[i + 6])), "r"(__float_as_uint(v[i + 7]))
                 : "memory");
}

// Shared-memory operand with the 128-byte swizzle: eight rows of 128 bytes
// to an atom of 1024 bytes (16-byte piece c of row r at piece c ^ (r & 7)),
// atoms `sbo` bytes apart.
__device__ __forceinline__ uint64_t smem_operand(uint32_t addr, uint32_t sbo) {
  return static_cast<uint64_t>((addr & 0x3ffffu) >> 4) | 1ull << 16 | static_cast<uint64_t>(sbo >> 4) << 32 |
         1ull << 46 | 2ull << 61;
}
// kind::f16, f16 operands, fp32 sums, A 128 rows k-major, B n columns; `mn`:
// B is stored n-major (k rows of n contiguous values).
__host__ __device__ constexpr uint32_t tc_instr(int n, bool mn) {
  return 1u << 4 | (mn ? 1u << 16 : 0u) | static_cast<uint32_t>(n >> 3) << 17 | (128u >> 4) << 24;
}
// One thread of the (converged) warp. The MMAs are issued inside a branch on
// it: their operands then stay in uniform registers, and an MMA of N = 32
// takes 17 cycles to issue and run; under `lane == 0`, or predicated, 58 to 140.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
// D (+)= A B, A in tensor memory.
__device__ __forceinline__ void tc_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t instr, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(instr), "r"(static_cast<uint32_t>(add))
      : "memory");
}
// The same with A in shared memory.
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t instr, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(instr), "r"(static_cast<uint32_t>(add))
      : "memory");
}
// One arrival on `bar` when every MMA this thread has issued is complete.
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void mbar_arrive_if(bool leader, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(static_cast<uint32_t>(leader))
      : "memory");
}

// The registers a thread of this warp (with the three others of its four) may
// use from here on.
template <int R>
__device__ __forceinline__ void registers_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void registers_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// The largest of a warp's values (NaN left out).
__device__ __forceinline__ float warp_max(float x) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
  return m;
}

// Barrier `id` over `threads` threads that counts those whose `p` holds.
__device__ __forceinline__ int named_barrier_count(int id, int threads, bool p) {
  int n;
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %3, 0;\n\t"
      "barrier.cta.red.popc.u32 %0, %1, %2, q;\n\t}"
      : "=r"(n)
      : "r"(id), "r"(threads), "r"(static_cast<int>(p))
      : "memory");
  return n;
}

}  // namespace kvq
