// Attention of several queries per sequence over the quantised cache
// (kv_tree_attn, kv_cross_attn): the merge of the split kernels' partials and
// the dispatch. The split kernels are in multi_narrow.cuh (up to 32 query rows
// a KV head) and multi_wide.cuh (more).
#include "multi_attn.cuh"

namespace kvq {

// Launchers of the split kernels, instantiated in multi_d{64,128}_k{2,3,4,8}.cu.
template <int D, int KB>
cudaError_t launch_multi_split(const MultiAttnArgs& a, cudaStream_t s);

namespace {

// Merge: combines the partials of a row's unit by log-sum-exp (M = max m,
// o = sum 2^(m - M) o / sum 2^(m - M) l). It is short and bound by latency: a
// warp has four partials' loads in flight, and where a unit has more (few
// units on many SMs) `share` of the CTA's warps take a part of them each and
// are joined through shared memory.
//
// Partials lie as the split kernels write them: WIDE (128-row tiles), four
// channels of all 128 rows together, and a warp combines eight rows' 16
// channels; else a row's channels together, and a warp combines a row.
//
// Blocks go by units, or where these are more than the split kernel's CTAs by
// the cuts between the CTAs' shares: a unit that none cuts is written already
// (384 queries a sequence, 768 units on 152 CTAs: 235 us with blocks by units,
// 191 by cuts). Sequences without a column have no cut; a block each writes
// their zeros. What a block looks up first takes longer than a row, so a large
// grid's blocks walk over rows instead of each having eight warps' (384
// queries: 191 us with 2544 blocks, 187 with 477).
constexpr int kMultiMergeWarps = 8;

template <int D, bool WIDE>
__global__ void __launch_bounds__(kMultiMergeWarps * 32, 4)
    multi_merge_kernel(const __grid_constant__ MultiAttnArgs a, int items, int share) {
  constexpr int NC = WIDE ? 4 : D / 32;  // channels a lane holds
  __shared__ float joint[kMultiMergeWarps][NC + 2][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = warp % share;
  const int work = first_item(a, a.geo.B), n = sharing_ctas(a, work), per = a.geo.H * a.row_tiles;
  // sequence, unit in it, its first item, the unit's blocks, the CTAs that had some
  int b = 0, in = 0, first = 0, nb = 0, c0 = 0, c1 = -1;
  const int x = blockIdx.x;
  const bool cuts = a.cuts;
  bool mine = true;
  if (!cuts) {
    b = x / per;
    in = x - b * per;
    first = first_item(a, b);
    nb = seq_blocks(a, b).total;
  } else if (x < a.n_ctas - 1) {  // the unit that the end of CTA x's share cuts
    mine = x + 1 < n;
    if (mine) {
      const int i = Shares(work, n).begin(x + 1);
      b = find_sequence(a, i, &first);
      nb = seq_blocks(a, b).total;
      in = (i - first) / (nb + a.seg_cost);
    }
  } else {  // a sequence without a column
    b = x - (a.n_ctas - 1);
    mine = seq_blocks(a, b).total == 0;
  }
  if (nb) {
    const int i0 = first + in * (nb + a.seg_cost) + a.seg_cost;
    const Shares shares(work, n);
    c0 = shares.owner(i0);
    c1 = shares.owner(i0 + nb - 1);
    // one CTA had the whole unit and wrote its output; or another cut's block has it
    if (c0 == c1 || (cuts && c0 != x)) mine = false;
  }
  pdl_wait_primary();  // the partials are complete and visible from here on
  if (!mine) return;
  const int begin = partial_slot(a, c0, b * per + in, true), stride = a.copies * a.tile_rows;
  const int twice = a.copies - 1;                 // (one copy or two)
  const int r0 = in % a.row_tiles * a.tile_rows;  // first row of the unit
#pragma unroll 1
  for (int item = blockIdx.y * (kMultiMergeWarps / share) + warp / share; item - warp / share < items;
       item += gridDim.y * (kMultiMergeWarps / share)) {
    const int row = WIDE ? item / (D / 16) * 8 + (lane & 7) : item;
    const int ch = WIDE ? item % (D / 16) * 16 + (lane >> 3) * 4 : NC * lane;
    const bool live = item < items && row < a.tile_rows && r0 + row < a.rows;
    // partial p: copy p % copies of the row in segment c0 + p / copies
    const int parts = live ? (c1 - c0 + 1) * a.copies : 0;
    float M = -INFINITY, l = 0.0f, o[NC];
#pragma unroll
    for (int k = 0; k < NC; ++k) o[k] = 0.0f;
    auto add = [&](float m, float sum, const float (&x)[NC], float ref) {
      // A partial that saw nothing takes no part. One that did does with any
      // weight, zero too: where all its scores were NaN its maximum is -inf,
      // and its sum is what carries the NaN.
      const bool none = m == -INFINITY && sum == 0.0f;
      const float w = none ? 0.0f : fast_exp2(m - ref);
      l = fmaf(sum, w, l);
#pragma unroll
      for (int k = 0; k < NC; ++k) o[k] = none ? o[k] : fmaf(x[k], w, o[k]);
    };
    auto rescale = [&](float top) {  // to the larger maximum; returns what weights are taken against
      const float now = fmaxf(M, top), ref = now == -INFINITY ? 0.0f : now;
      const float f = M == -INFINITY ? 0.0f : fast_exp2(M - ref);
      M = now;
      l *= f;
#pragma unroll
      for (int k = 0; k < NC; ++k) o[k] *= f;
      return ref;
    };
    constexpr int NF = 4;  // partials in flight
#pragma unroll 1
    for (int p0 = sub; p0 < parts; p0 += NF * share) {
      float2 ml[NF];
      float x[NF][NC];
#pragma unroll
      for (int i = 0; i < NF; ++i) {
        const int p = p0 + i * share;
        ml[i] = make_float2(-INFINITY, 0.0f);
#pragma unroll
        for (int k = 0; k < NC; ++k) x[i][k] = 0.0f;
        if (p < parts) {
          const int c = c0 + (p >> twice);
          const size_t slot = static_cast<size_t>(c == c0 ? begin : c) * stride;
          const int at = (p & twice) * a.tile_rows + row;
          ml[i] = reinterpret_cast<const float2*>(a.part_ml)[slot + at];
          const float* src = a.part_o + slot * D + (WIDE ? static_cast<size_t>(ch) * stride + 4 * at : at * D + ch);
          if (NC == 4) {
            const float4 v = *reinterpret_cast<const float4*>(src);
            x[i][0] = v.x, x[i][1] = v.y, x[i][NC - 2] = v.z, x[i][NC - 1] = v.w;
          } else {
            const float2 v = *reinterpret_cast<const float2*>(src);
            x[i][0] = v.x, x[i][1] = v.y;
          }
        }
      }
      float top = ml[0].x;
#pragma unroll
      for (int i = 1; i < NF; ++i) top = fmaxf(top, ml[i].x);
      const float ref = rescale(top);
#pragma unroll
      for (int i = 0; i < NF; ++i) add(ml[i].x, ml[i].y, x[i], ref);
    }
    if (share > 1) {
      joint[warp][0][lane] = M;
      joint[warp][1][lane] = l;
#pragma unroll
      for (int k = 0; k < NC; ++k) joint[warp][2 + k][lane] = o[k];
      __syncthreads();
#pragma unroll 1
      for (int j = 1; sub == 0 && j < share; ++j) {
        float x[NC];
#pragma unroll
        for (int k = 0; k < NC; ++k) x[k] = joint[warp + j][2 + k][lane];
        const float m = joint[warp + j][0][lane];
        add(m, joint[warp + j][1][lane], x, rescale(m));
      }
      __syncthreads();
    }
    if (sub) continue;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // a row that saw nothing is zero
    auto write = [&](int h, int r) {
      const size_t orow = (static_cast<size_t>(b) * a.geo.Hq + static_cast<size_t>(h) * a.geo.gqa) * a.T + r;
#pragma unroll
      for (int k = 0; k < NC; k += 2)
        *reinterpret_cast<uint32_t*>(a.out + orow * D + ch + k) =
            static_cast<uint32_t>(float_to_act(o[k] * inv, a.geo.act_bf16)) |
            static_cast<uint32_t>(float_to_act(o[k + 1] * inv, a.geo.act_bf16)) << 16;
      if (a.lse && ch == 0) a.lse[orow] = l == 0.0f ? -INFINITY : (M + log2f(l)) * 0.69314718055994530942f;
    };
    if (live) write(in / a.row_tiles, r0 + row);
    if (cuts && !nb && item < items && row < a.tile_rows) {  // a sequence without a column: its other units
#pragma unroll 1
      for (int v = 1; v < per; ++v)
        if (v % a.row_tiles * a.tile_rows + row < a.rows) write(v / a.row_tiles, v % a.row_tiles * a.tile_rows + row);
    }
  }
}

template <int D>
cudaError_t launch_d(const MultiAttnArgs& a, cudaStream_t s, int64_t* launches) {
  cudaError_t e = cudaErrorInvalidValue;
  switch (a.geo.kb) {
    case 2: e = launch_multi_split<D, 2>(a, s); break;
    case 3: e = launch_multi_split<D, 3>(a, s); break;
    case 4: e = launch_multi_split<D, 4>(a, s); break;
    case 8: e = launch_multi_split<D, 8>(a, s); break;
  }
  if (e != cudaSuccess) return e;
  ++*launches;
  const int rows = a.rows < a.tile_rows ? a.rows : a.tile_rows;
  const bool wide = a.tile_rows > 32;
  const int units = a.geo.B * a.geo.H * a.row_tiles;
  if (!a.lens && units == a.n_ctas) return cudaSuccess;  // every share is a whole unit
  const int items = wide ? (rows + 7) / 8 * (D / 16) : rows;
  // warps that share a unit's partials: so many that each has four at most
  // (where all sequences have one length)
  const int parts = ((a.n_ctas + units - 1) / units + 1) * a.copies;
  const int share = parts <= 4 ? 1 : parts <= 8 ? 2 : parts <= 16 ? 4 : kMultiMergeWarps;
  const int across = a.cuts ? a.n_ctas - 1 + a.geo.B : units;
  const int down = (items * share + kMultiMergeWarps - 1) / kMultiMergeWarps, fill = 4 * a.n_ctas / across;
  const dim3 grid(static_cast<unsigned>(across), static_cast<unsigned>(down < fill ? down : fill > 1 ? fill : 1));
  // scheduled as the split kernel drains (programmatic dependent launch)
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kMultiMergeWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = wide ? cudaLaunchKernelEx(&cfg, multi_merge_kernel<D, true>, a, items, share)
           : cudaLaunchKernelEx(&cfg, multi_merge_kernel<D, false>, a, items, share);
  if (e != cudaSuccess) return e;
  ++*launches;
  return cudaSuccess;
}

// The split kernels' waits made to run out, as wait_probe_kernel does with the
// decode's: four barriers that nothing arrives at. Warp 0 (pipe_wait) gives up
// after `budget` cycles, warp 2 (pipe_wait_short) after kProbeRounds rounds, and
// both raise an abort flag; warps 1 and 3 wait with the kernels' own bounds and
// must leave through that flag. res[w]: 1 if warp w's wait returned "completed"
// (must be 0), res[4 + w]: the SM clock cycles it took.
constexpr int kProbeRounds = 8;
__global__ void __launch_bounds__(128) multi_wait_probe_kernel(int* err_flag, long long* res, long long budget) {
  __shared__ __align__(8) uint64_t bars[4];
  __shared__ int abort_flags[2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x < 4) mbar_init(&bars[threadIdx.x], 1);
  if (threadIdx.x < 2) abort_flags[threadIdx.x] = 0;
  mbar_fence_init();
  __syncthreads();
  volatile int* ab = &abort_flags[warp >> 1];
  const long long t0 = clock64();
  bool ok;
  if (warp == 0) ok = pipe_wait(&bars[0], 0, ab, budget);
  else if (warp == 1) ok = pipe_wait(&bars[1], 0, ab);
  else if (warp == 2) ok = pipe_wait_short(&bars[2], 0, ab, kProbeRounds);
  else ok = pipe_wait_short(&bars[3], 0, ab);
  if (lane == 0) {
    res[warp] = ok ? 1 : 0;
    res[4 + warp] = clock64() - t0;
    if (!ok) set_error(err_flag, kErrTimeout);
  }
}

}  // namespace

// Rows of a tile: up to 32 rows the columns are the products' long side and
// the tile is as narrow as holds them; more rows are the long side themselves,
// up to 64 twice over (128 of the tensor core's). 4 x 32768 tokens, D 128, K2/V4:
// 16 rows take 64 us in a tile of 16, 70 in 32 and 83 in 64; 32 rows 73 in 32 and
// 86 in 64; 64 rows 90 in 64 and 100 in 128.
int multi_tile_rows(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }

// A segment's start and end take what some 32 blocks of a long one take (up to
// 32 rows; cross step 22.5 us with 16, 21.5 with 32) or 20 (more rows).
int multi_seg_cost(int tile_rows) { return tile_rows > 32 ? 20 : 32; }

int multi_unit_shift(int bits) { return unit_shift(bits); }

// CTAs of the split kernel: one per SM where there is a tile for each. But
// units that SMs are enough for, all of one length, have a CTA each and no
// merge where sharing them out would take few tiles off a CTA's time: it costs
// a second kernel, and a second segment for most CTAs where the units are not
// few (up to 32 rows: 5 tiles and 24 times the share of the SMs that have a
// unit; more rows: 3 and 8). Shared and not, up to 32 rows, D 128, K2/V4: 128
// units of 3900 columns 50 and 34 us, of 16000 110 and 95, of 32768 195 and 210;
// 64 units of 2700 28 and 25, of 6000 38 and 42; two of 512 as long, with one
// launch less. 61 rows and more: 128 units of 2000 56 and 41, 64 of 900 28 and
// 24, of 2700 37 and 46.
int multi_attn_ctas(int64_t units, int64_t blocks, bool wide, bool ragged, int sm_count) {
  const int64_t tiles = (units * blocks + kTileBlocks - 1) / kTileBlocks;
  const int64_t few = wide ? 3 * sm_count + 8 * units : 5 * sm_count + 24 * units;
  if (!ragged && units <= sm_count && blocks * (sm_count - units) <= kTileBlocks * few)
    return static_cast<int>(units);
  return static_cast<int>(tiles < sm_count ? tiles : sm_count);
}

cudaError_t launch_multi_wait_probe(int* err_flag, long long* res, long long budget, cudaStream_t s,
                                    int64_t* launches) {
  multi_wait_probe_kernel<<<1, 128, 0, s>>>(err_flag, res, budget);
  ++*launches;
  return cudaGetLastError();
}

cudaError_t launch_multi_attn(MultiAttnArgs& a, cudaStream_t s, int64_t* launches) {
  return a.geo.D == 128 ? launch_d<128>(a, s, launches) : launch_d<64>(a, s, launches);
}

}  // namespace kvq
