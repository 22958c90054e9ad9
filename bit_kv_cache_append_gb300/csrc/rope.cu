// Rotary positions and per-head norms in front of the cache: kv_rope_apply
// and kv_qk_norm_rope (one kernel, with and without the norm).
//
// Angles. A pair turns by f_i radians a position (f_i built in double on the
// host with the configured scaling). The kernel holds f_i / 2 pi as a 64-bit
// fraction of a turn and multiplies it by the position modulo 2^64: whole
// turns fall away exactly, and the phase is off by at most |position| times
// 2^-55 turns (the double's rounding), 2^-35 at a million positions, where an
// fp32 angle would have lost all but four bits. What is left, a phase in
// [-1/2, 1/2) turn, goes through sincospif.
//
// Bound: HBM bandwidth. A row of D channels is read and written once (4 D
// bytes); a warp takes one token and holds the token's cosines and sines in
// registers while it walks over the heads, so the angle work is paid once
// per token and not per head. A lane owns two 16-byte chunks of a row, the
// two that hold each other's rotation partners (half layout: chunks j and
// j + rot / 16; interleaved: 2j and 2j + 1), so a rotation needs no
// exchange between lanes; the norm's sum crosses the row's lanes in shuffles.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <new>
#include <string>

#include "kvq.h"
#include "kvq_device.cuh"

namespace {

constexpr int kMaxPairs = 128;  // rot_dim / 2 at head_dim 256

struct FreqTable {
  uint64_t turn[kMaxPairs];  // turns a position, times 2^64
};

struct RowsDev {
  uint16_t* data;
  int64_t sb, sh, st;
};

struct RopeArgs {
  RowsDev in[2], out[2];     // queries (or the only tensor), keys
  const uint16_t* weight[2];
  const int64_t* pos;
  int64_t pos_sb, first_pos;
  int H[2];                  // heads of each
  int n_tokens;              // T
  int64_t rows;              // B * T
  int D, rot, inverse;
  int heads_per_warp;        // a multiple of the rows a warp takes at once
  float att, eps, inv_d;
  FreqTable f;
};

constexpr int kWarps = 4;    // warps of a CTA, one token each
constexpr int kDepth = 4;    // passes whose loads are in flight together

// Two activations as floats, and back.
template <bool BF>
__device__ __forceinline__ float2 unpack2(uint32_t x) {
  if (BF) return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
  return __half22float2(*reinterpret_cast<__half2*>(&x));
}
template <bool BF>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if (BF) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
  }
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// The eight words of a lane's two chunks as the first (x0) and second (x1)
// channels of its eight pairs, two pairs to a float2.
template <bool INTER, bool BF>
__device__ __forceinline__ void to_pairs(const uint32_t* w, float2 (&x0)[4], float2 (&x1)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (INTER) {  // word 2i is pair 2i
      const float2 p = unpack2<BF>(w[2 * i]), q = unpack2<BF>(w[2 * i + 1]);
      x0[i] = make_float2(p.x, q.x), x1[i] = make_float2(p.y, q.y);
    } else {      // words i of the two chunks hold pairs 2i, 2i + 1
      x0[i] = unpack2<BF>(w[i]), x1[i] = unpack2<BF>(w[4 + i]);
    }
  }
}

// LPR: lanes per head row (each two chunks of 8 channels). INTER: interleaved
// pairs. A warp takes the token blockIdx.x * kWarps + warp and the heads
// [blockIdx.y * heads_per_warp, + heads_per_warp) of queries and keys in one
// list. The norm's weights are folded into the token's cosines and sines, so
// a pair costs three packed operations for each of its channels.
// (with the norm four CTAs an SM, 128 registers: 125 us for 4 x 8192 tokens of
// 32 + 8 heads of 128 channels; 150 us with the 162 the compiler would take)
template <bool NORM, int LPR, bool INTER, bool BF>
__global__ void __launch_bounds__(kWarps * 32, NORM ? 4 : 1) rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int RPP = 32 / LPR;              // rows per pass
  constexpr int PPL = RPP >= 8 ? 1 : 8 / RPP;  // pairs whose angle a lane works out
  __shared__ uint64_t turn[kMaxPairs];
  for (int i = threadIdx.x; i < a.rot / 2; i += kWarps * 32) turn[i] = a.f.turn[i];
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  if (row >= a.rows) return;
  const int64_t b = row / a.n_tokens, t = row - b * a.n_tokens;
  const int j = lane % LPR, rg = lane / LPR;
  const int nch = a.D / 8, nrot = a.rot / 8;  // chunks of a row; rotated ones (half layout: whole and even in number)
  // this lane's chunks; -1: none
  int c0, c1;
  if (INTER || 2 * j >= nrot) {
    c0 = 2 * j < nch ? 2 * j : -1;
    c1 = 2 * j + 1 < nch ? 2 * j + 1 : -1;
  } else {
    c0 = j;
    c1 = j + nrot / 2;
  }
  // cosines and sines of the lane's eight pairs (pair i: frequency 8j + i, in
  // either layout); the row groups of the warp work out a share each
  float2 co[4], si[4];
  uint32_t turned = 0;  // which of the lane's pairs rotate
  {
    const int64_t p = a.pos ? a.pos[b * a.pos_sb + t] : a.first_pos + t;
    float c[PPL], s[PPL];
#pragma unroll
    for (int k = 0; k < PPL; ++k) {
      const int fi = 8 * j + (rg * PPL + k) % 8;
      c[k] = 1.0f, s[k] = 0.0f;
      if (2 * fi < a.rot) {
        const int64_t ph = static_cast<int64_t>(static_cast<uint64_t>(p) * turn[fi]);
        // 2 * phase in turns, from the upper 32 bits (2^-31 of half a turn)
        sincospif(static_cast<float>(static_cast<int>(ph >> 32)) * 0x1p-31f, &s[k], &c[k]);
        c[k] *= a.att;
        s[k] *= a.inverse ? -a.att : a.att;
      }
    }
    float* cf = reinterpret_cast<float*>(co);
    float* sf = reinterpret_cast<float*>(si);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      cf[i] = __shfl_sync(0xffffffffu, c[i % PPL], (i / PPL) * LPR + j);
      sf[i] = __shfl_sync(0xffffffffu, s[i % PPL], (i / PPL) * LPR + j);
      if (2 * (8 * j + i) < a.rot) turned |= 1u << i;
    }
  }
  const int h0 = blockIdx.y * a.heads_per_warp, h_all = h0 + a.heads_per_warp;
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {  // queries, then keys
    const int lo = max(h0 - (part ? a.H[0] : 0), 0), hi = min(h_all - (part ? a.H[0] : 0), a.H[part]);
    if (lo >= hi) continue;
    const uint16_t* in = a.in[part].data + b * a.in[part].sb + t * a.in[part].st;
    uint16_t* out = a.out[part].data + b * a.out[part].sb + t * a.out[part].st;
    const int64_t in_h = a.in[part].sh, out_h = a.out[part].sh;
    // the weights of the lane's pairs
    auto weights = [&](float2(&w0)[4], float2(&w1)[4]) {
      const uint32_t one = BF ? 0x3f803f80u : 0x3c003c00u;
      uint4 w[2] = {make_uint4(one, one, one, one), make_uint4(one, one, one, one)};
      const uint4* src = reinterpret_cast<const uint4*>(a.weight[part]);
      if (src && c0 >= 0) w[0] = src[c0];
      if (src && c1 >= 0) w[1] = src[c1];
      to_pairs<INTER, BF>(reinterpret_cast<const uint32_t*>(w), w0, w1);
    };
    float2 w0[4], w1[4], wc0[4], ws0[4], wc1[4], ws1[4];
    if (NORM) weights(w0, w1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      wc0[i] = NORM ? __fmul2_rn(w0[i], co[i]) : co[i], ws0[i] = NORM ? __fmul2_rn(w0[i], si[i]) : si[i];
      wc1[i] = NORM ? __fmul2_rn(w1[i], co[i]) : co[i], ws1[i] = NORM ? __fmul2_rn(w1[i], si[i]) : si[i];
      ws1[i].x = -ws1[i].x, ws1[i].y = -ws1[i].y;
    }
#pragma unroll 1
    for (int base = lo; base < hi; base += RPP * kDepth) {
      uint4 x[kDepth][2];
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        const int h = base + d * RPP + rg;
        x[d][0] = x[d][1] = make_uint4(0u, 0u, 0u, 0u);
        if (h < hi) {
          const uint4* src = reinterpret_cast<const uint4*>(in + h * in_h);
          if (c0 >= 0) x[d][0] = src[c0];
          if (c1 >= 0) x[d][1] = src[c1];
        }
      }
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        if (base + d * RPP >= hi) break;
        const int h = base + d * RPP + rg;
        const uint32_t* xw = reinterpret_cast<const uint32_t*>(&x[d][0]);
        float2 x0[4], x1[4], y0[4], y1[4];
        to_pairs<INTER, BF>(xw, x0, x1);
        float2 r = make_float2(1.0f, 1.0f);
        if (NORM) {
          float2 ss = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int i = 0; i < 4; ++i) ss = __ffma2_rn(x1[i], x1[i], __ffma2_rn(x0[i], x0[i], ss));
          float sum = ss.x + ss.y;
#pragma unroll
          for (int off = LPR / 2; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
          r.x = r.y = 1.0f / sqrtf(fmaf(sum, a.inv_d, a.eps));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          y0[i] = __ffma2_rn(x1[i], ws1[i], __fmul2_rn(x0[i], wc0[i]));
          y1[i] = __ffma2_rn(x1[i], wc1[i], __fmul2_rn(x0[i], ws0[i]));
          if (NORM) y0[i] = __fmul2_rn(y0[i], r), y1[i] = __fmul2_rn(y1[i], r);
        }
        if (NORM && turned != 0xffu) {  // pairs that do not turn: a partner must not reach them, infinite or not
          weights(w0, w1);  // (again: sixteen registers that the other heads do not hold)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (turned >> i & 1u) continue;
            float& o0 = i & 1 ? y0[i / 2].y : y0[i / 2].x;
            float& o1 = i & 1 ? y1[i / 2].y : y1[i / 2].x;
            o0 = (i & 1 ? x0[i / 2].y * w0[i / 2].y : x0[i / 2].x * w0[i / 2].x) * r.x;
            o1 = (i & 1 ? x1[i / 2].y * w1[i / 2].y : x1[i / 2].x * w1[i / 2].x) * r.x;
          }
        }
        if (h < hi) {
          uint4 o[2];
          uint32_t* ow = reinterpret_cast<uint32_t*>(&o[0]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (INTER) {
              ow[2 * i] = pack2<BF>(y0[i].x, y1[i].x), ow[2 * i + 1] = pack2<BF>(y0[i].y, y1[i].y);
            } else {
              ow[i] = pack2<BF>(y0[i].x, y0[i].y), ow[4 + i] = pack2<BF>(y1[i].x, y1[i].y);
            }
          }
          if (!NORM && turned != 0xffu) {  // channels that are only copied keep their bits
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (!(turned >> i & 1u)) ow[i] = xw[i];  // (half layout: all of a lane's pairs turn, or none)
          }
          uint4* dst = reinterpret_cast<uint4*>(out + h * out_h);
          if (c0 >= 0) dst[c0] = o[0];
          if (c1 >= 0) dst[c1] = o[1];
        }
      }
    }
  }
}

kv_status fail(kv_status s, const std::string& msg) { return kvq::report(s, msg.c_str()); }

template <bool NORM, int LPR>
void launch(const RopeArgs& a, bool inter, bool bf, dim3 grid, cudaStream_t s) {
  const dim3 block(kWarps * 32);
  if (inter) {
    if (bf) rope_kernel<NORM, LPR, true, true><<<grid, block, 0, s>>>(a);
    else rope_kernel<NORM, LPR, true, false><<<grid, block, 0, s>>>(a);
  } else {
    if (bf) rope_kernel<NORM, LPR, false, true><<<grid, block, 0, s>>>(a);
    else rope_kernel<NORM, LPR, false, false><<<grid, block, 0, s>>>(a);
  }
}

}  // namespace

struct kv_rope {
  kv_rope_config cfg;
  double att;
  FreqTable f;
};

namespace {

constexpr int kMaxHeads = 1 << 29;  // (queries' and keys' together, and a pass more, stay an int)

kv_status check_rows(const kv_rows* r, const char* what) {
  if (!r || !r->data) return fail(KV_ERR_INVALID_ARG, std::string(what) + " is NULL");
  if (reinterpret_cast<uintptr_t>(r->data) & 15u)
    return fail(KV_ERR_INVALID_ARG, std::string(what) + " must be 16-byte aligned");
  if (r->stride_b % 8 || r->stride_h % 8 || r->stride_t % 8)
    return fail(KV_ERR_INVALID_ARG, std::string(what) + "'s strides must be multiples of 8 elements");
  return KV_OK;
}

RowsDev rows_dev(const kv_rows* r) {
  return RowsDev{static_cast<uint16_t*>(r->data), r->stride_b, r->stride_h, r->stride_t};
}

// SMs of the current device, asked for once per device.
cudaError_t sm_count(int* n) {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> known[kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < kMaxDevices && (*n = known[dev].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
  e = cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess && dev < kMaxDevices) known[dev].store(*n, std::memory_order_relaxed);
  return e;
}

constexpr int kFillCtas = 4;  // CTAs on every SM that the launch should come to

// Launch over queries and keys (H[1] = 0: one tensor).
kv_status run_rope(const kv_rope* rope, kv_dtype dtype, int64_t batch, RopeArgs& a, bool norm, void* stream) {
  const kv_rope_config& c = rope->cfg;
  a.rows = batch * a.n_tokens;
  a.D = c.head_dim;
  a.rot = c.rot_dim;
  a.att = static_cast<float>(rope->att);
  a.inv_d = 1.0f / static_cast<float>(c.head_dim);
  a.f = rope->f;
  int lpr = 1;
  while (16 * lpr < a.D) lpr *= 2;
  const int rpp = 32 / lpr, n_heads = a.H[0] + a.H[1];
  const int64_t blocks = (a.rows + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffff) return fail(KV_ERR_INVALID_ARG, "batch * n_tokens too large");
  // one warp takes all of a token's heads where there are tokens enough to
  // fill the GPU, else as few as one pass
  int sms = 0;
  const cudaError_t asked = sm_count(&sms);
  if (asked != cudaSuccess) return fail(KV_ERR_CUDA, std::string("SM count: ") + cudaGetErrorString(asked));
  int split = 1;
  const int passes = (n_heads + rpp - 1) / rpp;
  while (split < passes && blocks * split < sms * kFillCtas) ++split;
  if (split > 65535) split = 65535;
  const int per = (passes + split - 1) / split;
  a.heads_per_warp = per * rpp;
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((n_heads + a.heads_per_warp - 1) / a.heads_per_warp));
  const bool inter = c.layout == KV_ROPE_INTERLEAVED, bf = dtype == KV_DT_BF16;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
#define KVQ_ROPE_CASE(N)                              \
  case N:                                             \
    if (norm) launch<true, N>(a, inter, bf, grid, s); \
    else launch<false, N>(a, inter, bf, grid, s);     \
    break;
  switch (lpr) {
    KVQ_ROPE_CASE(1)
    KVQ_ROPE_CASE(2)
    KVQ_ROPE_CASE(4)
    KVQ_ROPE_CASE(8)
    KVQ_ROPE_CASE(16)
  }
#undef KVQ_ROPE_CASE
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(KV_ERR_CUDA, std::string("rope launch: ") + cudaGetErrorString(e));
  kvq::count_launches(1);
  return KV_OK;
}

kv_status check_common(const kv_rope* rope, kv_dtype dtype, int batch, int n_tokens, const int64_t* positions) {
  if (!rope) return fail(KV_ERR_INVALID_ARG, "rope is NULL");
  if (dtype != KV_DT_F16 && dtype != KV_DT_BF16) return fail(KV_ERR_INVALID_ARG, "dtype must be F16 or BF16");
  if (batch < 1 || n_tokens < 1) return fail(KV_ERR_INVALID_ARG, "batch and token counts must be positive");
  if (reinterpret_cast<uintptr_t>(positions) & 7u) return fail(KV_ERR_INVALID_ARG, "positions must be 8-byte aligned");
  return KV_OK;
}

}  // namespace

extern "C" {

kv_status kv_rope_create(const kv_rope_config* cfg, kv_rope** out) {
  if (!cfg || !out) return fail(KV_ERR_INVALID_ARG, "config or out is NULL");
  const kv_rope_config& c = *cfg;
  if (c.head_dim < 16 || c.head_dim > 256 || c.head_dim % 8)
    return fail(KV_ERR_INVALID_ARG, "head_dim must be a multiple of 8 in 16 .. 256");
  if (c.layout != KV_ROPE_HALF && c.layout != KV_ROPE_INTERLEAVED) return fail(KV_ERR_INVALID_ARG, "unknown layout");
  if (c.rot_dim < 0 || c.rot_dim > c.head_dim || c.rot_dim % 2)
    return fail(KV_ERR_INVALID_ARG, "rot_dim must be even and in 0 .. head_dim");
  if (c.layout == KV_ROPE_HALF && c.rot_dim % 16)
    return fail(KV_ERR_UNSUPPORTED, "rot_dim must be a multiple of 16 in the half layout");
  if (c.scaling < KV_ROPE_SCALE_NONE || c.scaling > KV_ROPE_SCALE_WAVELENGTH)
    return fail(KV_ERR_INVALID_ARG, "unknown scaling");
  if (!(c.base > 1.0) || !std::isfinite(c.base)) return fail(KV_ERR_INVALID_ARG, "base must be above 1");
  if (!(c.factor >= 1.0) || !std::isfinite(c.factor)) return fail(KV_ERR_INVALID_ARG, "factor must be >= 1");
  if (c.scaling == KV_ROPE_SCALE_NTK && c.rot_dim == 2)
    return fail(KV_ERR_INVALID_ARG, "NTK scaling needs more than one pair");
  const bool banded = c.scaling == KV_ROPE_SCALE_YARN || c.scaling == KV_ROPE_SCALE_WAVELENGTH;
  const bool yarn = c.scaling == KV_ROPE_SCALE_YARN;
  const double fast = c.fast == 0.0 ? (yarn ? 32.0 : 4.0) : c.fast, slow = c.slow == 0.0 ? 1.0 : c.slow;
  if (banded) {
    if (c.orig_max_pos < 1) return fail(KV_ERR_INVALID_ARG, "orig_max_pos must be >= 1");
    if (!(fast > slow) || !(slow > 0.0) || !std::isfinite(fast))
      return fail(KV_ERR_INVALID_ARG, "fast must be above slow, and slow above 0");
  }
  if (!(c.attn_factor >= 0.0) || !std::isfinite(c.attn_factor))
    return fail(KV_ERR_INVALID_ARG, "attn_factor must be >= 0");
  kv_rope* r = new (std::nothrow) kv_rope();
  if (!r) return fail(KV_ERR_INVALID_ARG, "out of host memory");
  r->cfg = c;
  r->att = c.attn_factor > 0.0 ? c.attn_factor : yarn ? 0.1 * std::log(c.factor) + 1.0 : 1.0;
  const double pi = 3.14159265358979323846;
  const double rot = c.rot_dim, orig = static_cast<double>(c.orig_max_pos);
  double base = c.base;
  if (c.scaling == KV_ROPE_SCALE_NTK) base *= std::pow(c.factor, rot / (rot - 2.0));
  // YaRN: the (fractional) pair that makes `turns` turns over orig_max_pos
  auto pair_of = [&](double turns) { return rot * std::log(orig / (turns * 2.0 * pi)) / (2.0 * std::log(base)); };
  double low = 0.0, high = 0.0;
  if (yarn && c.rot_dim) {
    low = std::fmax(std::floor(pair_of(fast)), 0.0);
    high = std::fmin(std::ceil(pair_of(slow)), rot - 1.0);
  }
  for (int i = 0; i < c.rot_dim / 2; ++i) {
    double inv = std::pow(base, -2.0 * i / rot);
    if (c.scaling == KV_ROPE_SCALE_LINEAR) {
      inv /= c.factor;
    } else if (yarn) {
      const double ramp = std::fmin(std::fmax((i - low) / (high > low ? high - low : 0.001), 0.0), 1.0);
      inv = inv / c.factor * ramp + inv * (1.0 - ramp);
    } else if (c.scaling == KV_ROPE_SCALE_WAVELENGTH) {
      const double turns = orig * inv / (2.0 * pi);  // orig_max_pos / wavelength
      const double keep = std::fmin(std::fmax((turns - slow) / (fast - slow), 0.0), 1.0);
      inv = (1.0 - keep) * inv / c.factor + keep * inv;
    }
    r->f.turn[i] = static_cast<uint64_t>(std::ldexp(inv / (2.0 * pi), 64));  // inv <= 1: below 2^62
  }
  *out = r;
  return KV_OK;
}

kv_status kv_rope_destroy(kv_rope* rope) {
  if (!rope) return fail(KV_ERR_INVALID_ARG, "rope is NULL");
  delete rope;
  return KV_OK;
}

kv_status kv_rope_apply(const kv_rope* rope, kv_dtype dtype, int batch, int n_heads, int n_tokens, const kv_rows* x,
                        const kv_rows* y, const int64_t* positions, int64_t pos_stride_b, int64_t first_pos,
                        int inverse, void* cuda_stream) {
  kv_status st = check_common(rope, dtype, batch, n_tokens, positions);
  if (st != KV_OK) return st;
  if (n_heads < 1 || n_heads > kMaxHeads) return fail(KV_ERR_INVALID_ARG, "n_heads must be in 1 .. 2^29");
  if ((st = check_rows(x, "x")) != KV_OK || (st = check_rows(y, "y")) != KV_OK) return st;
  RopeArgs a{};
  a.in[0] = rows_dev(x);
  a.out[0] = rows_dev(y);
  a.H[0] = n_heads;
  a.n_tokens = n_tokens;
  a.pos = positions;
  a.pos_sb = pos_stride_b;
  a.first_pos = first_pos;
  a.inverse = inverse ? 1 : 0;
  return run_rope(rope, dtype, batch, a, false, cuda_stream);
}

kv_status kv_qk_norm_rope(const kv_rope* rope, kv_dtype dtype, int batch, int n_q_heads, int n_kv_heads, int n_tokens,
                          const kv_rows* q, const kv_rows* k, const void* q_weight, const void* k_weight, float eps,
                          const int64_t* positions, int64_t pos_stride_b, int64_t first_pos, const kv_rows* q_out,
                          const kv_rows* k_out, void* cuda_stream) {
  kv_status st = check_common(rope, dtype, batch, n_tokens, positions);
  if (st != KV_OK) return st;
  if (n_q_heads < 1 || n_kv_heads < 0 || n_q_heads > kMaxHeads || n_kv_heads > kMaxHeads)
    return fail(KV_ERR_INVALID_ARG, "head counts must be in 1 .. 2^29 (keys: 0 .. 2^29)");
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(KV_ERR_INVALID_ARG, "eps must be >= 0");
  if ((st = check_rows(q, "q")) != KV_OK || (st = check_rows(q_out, "q_out")) != KV_OK) return st;
  if ((reinterpret_cast<uintptr_t>(q_weight) | reinterpret_cast<uintptr_t>(k_weight)) & 15u)
    return fail(KV_ERR_INVALID_ARG, "weights must be 16-byte aligned");
  RopeArgs a{};
  a.in[0] = rows_dev(q);
  a.out[0] = rows_dev(q_out);
  a.H[0] = n_q_heads;
  if (n_kv_heads) {
    if ((st = check_rows(k, "k")) != KV_OK || (st = check_rows(k_out, "k_out")) != KV_OK) return st;
    a.in[1] = rows_dev(k);
    a.out[1] = rows_dev(k_out);
    a.H[1] = n_kv_heads;
  }
  a.weight[0] = static_cast<const uint16_t*>(q_weight);
  a.weight[1] = static_cast<const uint16_t*>(k_weight);
  a.n_tokens = n_tokens;
  a.pos = positions;
  a.pos_sb = pos_stride_b;
  a.first_pos = first_pos;
  a.eps = eps;
  return run_rope(rope, dtype, batch, a, true, cuda_stream);
}

}  // extern "C"
