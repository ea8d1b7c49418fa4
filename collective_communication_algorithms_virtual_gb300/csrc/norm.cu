// ReduceScatter + residual + RMS norm of the virtual ranks' partial sums, and
// its gradient (see vc.h).
//
// Both stream: every input is read once and every output written once, and
// the norm's mean is taken while the row is on chip, in the registers of one
// block (rows too long for them: in shared memory, in fp32).  Memory bounds
// them; on a GB300, copy rate 6.69 TB/s:
//   forward, 8 ranks, 2048 tokens of 8192 bf16 to 8 bits: 352 MB, 57.9 us, 6.1 TB/s
//   backward, 4 ranks, 4096 tokens of 4096 bf16: 268 MB, 50.6 us, 5.3 TB/s
//   forward, 1 rank, 4096 tokens of 4096 bf16: 134 MB, 24.0 us, 5.6 TB/s
//   forward, 8 ranks, one token of 4096 each: 3.0 us, launch and latency
#include "layer.cuh"

namespace vc {
namespace layer {
namespace {

// Most threads of a block that holds a row in registers, `vpt` units a thread.
__host__ __device__ constexpr int norm_threads(bool vec, int vpt) { return vec && vpt == 2 ? 1024 : 512; }
// Blocks of that size per SM that its registers are kept low enough for.
__host__ __device__ constexpr int norm_blocks(bool vec, bool few, int vpt) {
  return vec && !few && vpt == 1 ? 3 : vec && vpt == 2 ? 1 : vpt <= 3 ? 2 : 1;
}

struct NormParams {
  const void* send[VC_MAX_RANKS];
  const void* residual[VC_MAX_RANKS];
  const void* weight[VC_MAX_RANKS];
  void* residual_out[VC_MAX_RANKS];
  void* out[VC_MAX_RANKS];
  float* scale[VC_MAX_RANKS];
  float* rstd[VC_MAX_RANKS];
  int nranks, has_residual, has_residual_out, has_rstd;
  uint32_t rows;
  int32_t hidden;
  float eps;
};

// The larger magnitude; a NaN stays one.
__device__ __forceinline__ float max_magnitude(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(fabsf(b)));
  return m;
}
// Quantiser of a row whose largest magnitude has the bits `top`.  Added to
// 1.5 * 2^23, whose neighbours are whole numbers, a number's nearest whole one
// (ties to even) is left in the low bits of the sum: one operation for the
// product, the rounding and the conversion, and no clamping, since no |y| is
// above the largest (one rank, 4096 x 4096 bf16 to 8 bits: 25.1 us; with two
// products, a conversion and a clamp 27.4).
struct Quant {
  float inv, scale;
  bool none, tiny;  // none: zeros, or an infinity or NaN, whose row is zeros too; tiny: 127 / max would overflow
  __device__ __forceinline__ explicit Quant(uint32_t top) {
    const float most = __uint_as_float(top);
    none = top == 0 || top >= 0x7f800000u;
    tiny = most < 1e-30f;
    inv = none ? 0.f : 127.f / (tiny ? most * 0x1p64f : most);
    scale = most / 127.f;
  }
  __device__ __forceinline__ uint32_t byte(float y) const {  // in the low byte
    return __float_as_uint(__fmaf_rn(tiny ? y * 0x1p64f : y, inv, 12582912.f));
  }
  __device__ __forceinline__ uint32_t four(const float* y) const {
    const uint32_t lo = __byte_perm(byte(y[0]), byte(y[1]), 0x0040), hi = __byte_perm(byte(y[2]), byte(y[3]), 0x0040);
    return none ? 0 : __byte_perm(lo, hi, 0x5410);
  }
};

// A block works a row, VPT units of it in each thread.  The sum over the ranks
// is in rank order in fp32.
//   FEW (one or two ranks): so little is read for a row that its loads alone
// do not keep memory busy; a block takes rows blockIdx.x, + gridDim.x, ... and
// asks for the next row's units while it works one (4096 tokens of 4096 bf16,
// one rank: 36.4 us with a block per row, 24.0 so).
//   Otherwise a block per row, and a thread asks for several ranks' units, the
// residual and the weight before it uses the first (8 ranks, 2048 x 8192 bf16
// to 8 bits: 91 us before it did, 57.7 so): up to 512 units one of them a
// thread, four ranks at a time and three blocks of 512 per SM (8 ranks, 4096 x
// 4096: 56.8 us; eight at a time and two blocks 60.9), then two units a
// thread (1024 threads of one: 63.3 against 62.4), to 1536 three (8 ranks,
// 1024 x 10240: 42.1 us, with four 52.9), to 2048 two in blocks of 1024.
template <int DT, bool VEC, bool FEW, int VPT, bool I8>
__global__ void __launch_bounds__(norm_threads(VEC, VPT), norm_blocks(VEC, FEW, VPT))
    norm_kernel(const __grid_constant__ NormParams p) {
  using E = El<DT>;
  using R = Row<E::kSize, VEC>;
  using Out = Span<E::kSize, 16, VEC>;
  constexpr int kN = E::kVec;
  using Quants = Span<1, kN, VEC>;
  // ranks whose loads are in flight together
  constexpr int kBatch = FEW ? 2 : VPT == 1 ? 4 : (VEC ? 8 : 4) / VPT > 0 ? (VEC ? 8 : 4) / VPT : 1;
  // the residual and the weight are asked for well before they are used,
  // where registers allow it
  constexpr bool kAhead = VPT <= (VEC ? 4 : 2);
  __shared__ float part[2][32];
  __shared__ uint32_t most[2][32];
  __shared__ __align__(16) unsigned char room[norm_threads(VEC, VPT) / 32][Out::kRoom];
  stream_order();
  const uint32_t r = blockIdx.y;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t width = static_cast<int64_t>(p.hidden) * E::kSize;
  const int nu = (p.hidden + kN - 1) / kN;
  const int64_t sent = static_cast<int64_t>(p.nranks) * p.rows;
  // a row from its place in a buffer of `rows` rows
  const auto row_of = [&](const void* buffer, int64_t at, int64_t rows) {
    const char* b = static_cast<const char*>(buffer);
    return R(b + at, nu, Bytes{b, b + rows * width});
  };
  const int64_t block = static_cast<int64_t>(r) * p.rows * width;  // where rank r's rows begin in each send buffer
  const R weights = row_of(p.weight[r], 0, 1);
  struct Loaded {
    typename R::Raw res[VPT], v[kBatch][VPT];
  };
  const auto load_res = [&](int64_t own, Loaded& l) {
    const R residual = row_of(p.has_residual ? p.residual[r] : p.out[r], own, p.rows);
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      const int c = threadIdx.x + u * blockDim.x;
      l.res[u] = R::zero();
      if (p.has_residual && c < nu) l.res[u] = residual.load_plain(c);
    }
  };
  const auto load_ranks = [&](int q0, int64_t at, Loaded& l) {
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (q0 + b >= p.nranks) break;
      const R from = row_of(p.send[q0 + b], at, sent);
#pragma unroll
      for (int u = 0; u < VPT; ++u) {
        const int c = threadIdx.x + u * blockDim.x;
        l.v[b][u] = R::zero();
        if (c < nu) l.v[b][u] = from.load(c);
      }
    }
  };
  typename R::Raw weight[VPT];
  const auto load_weight = [&] {
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      const int c = threadIdx.x + u * blockDim.x;
      weight[u] = R::zero();
      if (c < nu) weight[u] = weights.load_kept(c);
    }
  };
  // One row, of which the residual (kAhead or FEW) and the ranks' units (FEW) are there.
  const auto work = [&](uint32_t t, int flip, Loaded& now) {
    const int64_t own = t * width, at = block + own;  // the row's place in rank r's buffers, and in the send buffers
    const R residual = row_of(p.has_residual ? p.residual[r] : p.out[r], own, p.rows);
    float h[VPT][kN];
#pragma unroll
    for (int u = 0; u < VPT; ++u)
#pragma unroll
      for (int i = 0; i < kN; ++i) h[u][i] = 0.f;
    for (int q0 = 0; q0 < p.nranks; q0 += kBatch) {
      if (!FEW) load_ranks(q0, at, now);
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (q0 + b >= p.nranks) break;
        const R from = row_of(p.send[q0 + b], at, sent);
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
          const int c = threadIdx.x + u * blockDim.x;
          if (c < nu) {
            float f[kN];
            E::widen(from.finish(now.v[b][u], c, p.hidden), f);
#pragma unroll
            for (int i = 0; i < kN; ++i) h[u][i] += f[i];
          }
        }
      }
      if (FEW) break;
    }
    if (!FEW && !kAhead) load_res(own, now);
    if (!FEW && kAhead) load_weight();
    char* sums = p.has_residual_out ? static_cast<char*>(p.residual_out[r]) + own : nullptr;
    float ss = 0.f;
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      const int c = threadIdx.x + u * blockDim.x;
      if (p.has_residual && c < nu) {
        float f[kN];
        E::widen(residual.finish(now.res[u], c, p.hidden), f);
#pragma unroll
        for (int i = 0; i < kN; ++i) h[u][i] += f[i];
      }
      mask_unit<E::kSize, VEC>(c, p.hidden, h[u]);
#pragma unroll
      for (int i = 0; i < kN; ++i) ss += h[u][i] * h[u][i];
      if (sums) Out(room[warp], E::narrow(h[u])).write(sums, c - lane, p.hidden);
    }
    const float rs = 1.f / sqrtf(block_sum(ss, part[flip]) / static_cast<float>(p.hidden) + p.eps);
    if (p.has_rstd && threadIdx.x == 0) p.rstd[r][t] = rs;
    if (!FEW && !kAhead) load_weight();
    float top = 0.f;
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      const int c = threadIdx.x + u * blockDim.x;
      float w[kN];
#pragma unroll
      for (int i = 0; i < kN; ++i) w[i] = 0.f;
      if (c < nu) E::widen(weights.finish(weight[u], c, p.hidden), w);
#pragma unroll
      for (int i = 0; i < kN; ++i) h[u][i] = h[u][i] * rs * w[i];
      if (I8) {
        mask_unit<E::kSize, VEC>(c, p.hidden, h[u]);
        if (c < nu) {
#pragma unroll
          for (int i = 0; i < kN; ++i) top = max_magnitude(top, h[u][i]);
        }
      } else {
        Out(room[warp], E::narrow(h[u])).write(static_cast<char*>(p.out[r]) + own, c - lane, p.hidden);
      }
    }
    if (I8) {
      const Quant quant(block_max_bits(__float_as_uint(top), most[flip]));
      if (threadIdx.x == 0) p.scale[r][t] = quant.scale;
      int8_t* to = static_cast<int8_t*>(p.out[r]) + static_cast<int64_t>(t) * p.hidden;
#pragma unroll
      for (int u = 0; u < VPT; ++u) {
        const int c = threadIdx.x + u * blockDim.x;
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < kN / 4; ++i) w[i] = quant.four(h[u] + 4 * i);
        if constexpr (kN == 8) Quants(room[warp], make_uint2(w[0], w[1])).write(to, c - lane, p.hidden);
        else Quants(room[warp], w[0]).write(to, c - lane, p.hidden);
      }
    }
  };
  if constexpr (FEW) {
    load_weight();
    Loaded next;
    load_res(blockIdx.x * width, next);
    load_ranks(0, block + blockIdx.x * width, next);
    int flip = 0;
    for (uint32_t t = blockIdx.x; t < p.rows; t += gridDim.x, flip ^= 1) {
      Loaded now = next;
      if (t + gridDim.x < p.rows) {
        const int64_t own = (t + gridDim.x) * width;
        load_res(own, next);
        load_ranks(0, block + own, next);
      }
      work(t, flip, now);
    }
  } else {
    Loaded now;
    if (kAhead) load_res(blockIdx.x * width, now);
    work(blockIdx.x, 0, now);
  }
}

// Any row, element by element, held in shared memory.
template <int DT, bool I8>
__global__ void __launch_bounds__(1024) norm_any_kernel(const __grid_constant__ NormParams p) {
  using E = El<DT>;
  extern __shared__ float h[];
  __shared__ float part[32];
  __shared__ uint32_t most[32];
  stream_order();
  const uint32_t r = blockIdx.y, t = blockIdx.x;
  const int64_t row = static_cast<int64_t>(r) * p.rows + t;
  const int64_t at = row * p.hidden, own = static_cast<int64_t>(t) * p.hidden;
  float ss = 0.f;
  for (int c = threadIdx.x; c < p.hidden; c += blockDim.x) {
    float x = 0.f;
#pragma unroll 4
    for (int q = 0; q < p.nranks; ++q) x += E::load(p.send[q], at + c);
    if (p.has_residual) x += E::load(p.residual[r], own + c);
    if (p.has_residual_out) E::store(p.residual_out[r], own + c, x);
    h[c] = x;
    ss += x * x;
  }
  const float rs = 1.f / sqrtf(block_sum(ss, part) / static_cast<float>(p.hidden) + p.eps);
  if (p.has_rstd && threadIdx.x == 0) p.rstd[r][t] = rs;
  float top = 0.f;
  for (int c = threadIdx.x; c < p.hidden; c += blockDim.x) {  // each thread reads back what it wrote
    const float y = h[c] * rs * E::load(p.weight[r], c);
    if (I8) {
      h[c] = y;
      top = max_magnitude(top, y);
    } else {
      E::store(p.out[r], own + c, y);
    }
  }
  if (I8) {
    const Quant quant(block_max_bits(__float_as_uint(top), most));
    if (threadIdx.x == 0) p.scale[r][t] = quant.scale;
    for (int c = threadIdx.x; c < p.hidden; c += blockDim.x)
      static_cast<int8_t*>(p.out[r])[own + c] = static_cast<int8_t>(quant.none ? 0 : quant.byte(h[c]));
  }
}

struct GradParams {
  const void* dout[VC_MAX_RANKS];
  const void* dres_out[VC_MAX_RANKS];
  const void* h[VC_MAX_RANKS];
  const void* weight[VC_MAX_RANKS];
  const float* rstd[VC_MAX_RANKS];
  void* dsend[VC_MAX_RANKS];
  void* dres[VC_MAX_RANKS];
  float* part;  // [nranks * per][hidden] sums of the weight's gradient over each block's rows
  int nranks, has_dres_out, has_dsend, has_dres, has_dweight;
  uint32_t rows, per;  // tokens, blocks of each rank
  int32_t hidden;
};

// Most threads of a block of the gradient whose threads hold `vpt` units (4
// ranks x 1024 x 4096 bf16, 512 units: 256 threads of 2 50.1 us, 512 of 1
// 50.2, 128 of 4 59).
__host__ __device__ constexpr int grad_threads(int vpt) { return 128 * vpt; }

// Block b of rank r takes the rank's rows b, b + per, ...; each thread keeps
// the weight's gradient of its columns over them, so that it leaves the chip
// once a block instead of once a row: 152 blocks, 2.5 MB for 4096 columns,
// summed by norm_weight_kernel in a fixed order (3.3 us of the 50.1; adding to
// one array with atomics would make the last bits depend on the order).
// Without the weight's gradient the call takes 46.8 us.
template <int DT, bool VEC, int VPT>
__global__ void __launch_bounds__(grad_threads(VPT), VEC ? 1 : VPT == 1 ? 6 : 2) norm_grad_kernel(const __grid_constant__ GradParams p) {
  using E = El<DT>;
  constexpr int kN = E::kVec;
  using R = Row<E::kSize, VEC>;
  using Out = Span<E::kSize, 16, VEC>;
  __shared__ float part[2][32];
  __shared__ __align__(16) unsigned char room[grad_threads(VPT) / 32][Out::kRoom];
  stream_order();
  const uint32_t r = blockIdx.x / p.per, b = blockIdx.x - r * p.per;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nu = (p.hidden + kN - 1) / kN;
  const int64_t width = static_cast<int64_t>(p.hidden) * E::kSize;
  const auto row_of = [&](const void* buffer, int64_t at_byte, int64_t rows) {
    const char* b = static_cast<const char*>(buffer);
    return R(b + at_byte, nu, Bytes{b, b + rows * width});
  };
  const R weights = row_of(p.weight[r], 0, 1);
  float dw[VPT][kN];
#pragma unroll
  for (int u = 0; u < VPT; ++u)
#pragma unroll
    for (int i = 0; i < kN; ++i) dw[u][i] = 0.f;
  typename R::Raw wraw[VPT];
#pragma unroll
  for (int u = 0; u < VPT; ++u) {
    const int c = threadIdx.x + u * blockDim.x;
    wraw[u] = R::zero();
    if (c < nu) wraw[u] = weights.load_kept(c);
  }
  // A row's loads are asked for while the row before is worked, where
  // registers allow it (4 ranks x 1024 x 4096 bf16: 51.7 with, 53.2 us without).
  constexpr bool kAhead = VEC && VPT <= 2;
  struct Loaded {
    typename R::Raw g[VPT], h[VPT], d[VPT];
    float rs;
  };
  const auto rows_at = [&](uint32_t t, const void* buffer) { return row_of(buffer, static_cast<int64_t>(t) * width, p.rows); };
  const void* dres_out = p.has_dres_out ? p.dres_out[r] : p.h[r];
  const auto fetch = [&](uint32_t t, Loaded& l) {
    const R dout = rows_at(t, p.dout[r]), hs = rows_at(t, p.h[r]), dres = rows_at(t, dres_out);
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      const int c = threadIdx.x + u * blockDim.x;
      l.g[u] = l.h[u] = l.d[u] = R::zero();
      if (c < nu) {
        l.g[u] = dout.load(c);
        l.h[u] = hs.load(c);
        if (p.has_dres_out) l.d[u] = dres.load_plain(c);
      }
    }
    l.rs = p.rstd[r][t];
  };
  const float inv = 1.f / static_cast<float>(p.hidden);
  Loaded next;
  if (kAhead) fetch(b, next);
  int flip = 0;
  for (uint32_t t = b; t < p.rows; t += p.per, flip ^= 1) {
    const int64_t own = static_cast<int64_t>(t) * width;
    const R dout = rows_at(t, p.dout[r]), hs = rows_at(t, p.h[r]), dres = rows_at(t, dres_out);
    Loaded now;
    if (kAhead) {
      now = next;
      if (t + p.per < p.rows) fetch(t + p.per, next);
    } else {
      fetch(t, now);
    }
    const float rs = now.rs;
    float g[VPT][kN], h[VPT][kN], gh = 0.f;
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      const int c = threadIdx.x + u * blockDim.x;
#pragma unroll
      for (int i = 0; i < kN; ++i) g[u][i] = h[u][i] = 0.f;
      if (c >= nu) continue;
      float w[kN];
      E::widen(dout.finish(now.g[u], c, p.hidden), g[u]);
      E::widen(hs.finish(now.h[u], c, p.hidden), h[u]);
      E::widen(weights.finish(wraw[u], c, p.hidden), w);
      mask_unit<E::kSize, VEC>(c, p.hidden, g[u]);
      mask_unit<E::kSize, VEC>(c, p.hidden, h[u]);
      mask_unit<E::kSize, VEC>(c, p.hidden, w);
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        dw[u][i] += g[u][i] * h[u][i] * rs;
        g[u][i] *= w[i];
        gh += g[u][i] * h[u][i];
      }
    }
    const float mean = block_sum(gh, part[flip]) * inv * rs * rs;
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      const int c = threadIdx.x + u * blockDim.x;
      float d[kN];
#pragma unroll
      for (int i = 0; i < kN; ++i) d[i] = rs * (g[u][i] - h[u][i] * mean);
      if (p.has_dres_out && c < nu) {
        float f[kN];
        E::widen(dres.finish(now.d[u], c, p.hidden), f);
#pragma unroll
        for (int i = 0; i < kN; ++i) d[i] += f[i];
      }
      if (p.has_dres || p.has_dsend) {
        const Out v(room[warp], E::narrow(d));
        if (p.has_dres) v.template write<true>(static_cast<char*>(p.dres[r]) + own, c - lane, p.hidden);
        if (p.has_dsend) {
          const int64_t at = (static_cast<int64_t>(r) * p.rows + t) * width;
          for (int q = 0; q < p.nranks; ++q) v.template write<true>(static_cast<char*>(p.dsend[q]) + at, c - lane, p.hidden);
        }
      }
    }
  }
  if (p.has_dweight) {
    float* to = p.part + static_cast<int64_t>(blockIdx.x) * p.hidden;
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      const int c = threadIdx.x + u * blockDim.x;
      if (c < nu) {
        if constexpr (VEC) {
#pragma unroll
          for (int i = 0; i < kN; i += 4)
            *reinterpret_cast<float4*>(to + c * kN + i) = make_float4(dw[u][i], dw[u][i + 1], dw[u][i + 2], dw[u][i + 3]);
        } else {
#pragma unroll
          for (int i = 0; i < kN; ++i)
            if (c * kN + i < p.hidden) to[c * kN + i] = dw[u][i];
        }
      }
    }
  }
}

// Any row, element by element; the weight's gradient in shared memory.
template <int DT>
__global__ void __launch_bounds__(1024) norm_grad_any_kernel(const __grid_constant__ GradParams p) {
  using E = El<DT>;
  extern __shared__ float dw[];
  __shared__ float part[2][32];
  stream_order();
  const uint32_t r = blockIdx.x / p.per, b = blockIdx.x - r * p.per;
  for (int c = threadIdx.x; c < p.hidden; c += blockDim.x) dw[c] = 0.f;  // only its own thread uses a column
  int flip = 0;
  for (uint32_t t = b; t < p.rows; t += p.per, flip ^= 1) {
    const int64_t own = static_cast<int64_t>(t) * p.hidden;
    const float rs = p.rstd[r][t];
    float gh = 0.f;
    for (int c = threadIdx.x; c < p.hidden; c += blockDim.x) {
      const float dy = E::load(p.dout[r], own + c), h = E::load(p.h[r], own + c);
      dw[c] += dy * h * rs;
      gh += dy * E::load(p.weight[r], c) * h;
    }
    const float mean = block_sum(gh, part[flip]) / static_cast<float>(p.hidden) * rs * rs;
    const int64_t at = (static_cast<int64_t>(r) * p.rows + t) * p.hidden;
    for (int c = threadIdx.x; c < p.hidden; c += blockDim.x) {
      const float g = E::load(p.dout[r], own + c) * E::load(p.weight[r], c);
      float d = rs * (g - E::load(p.h[r], own + c) * mean);
      if (p.has_dres_out) d += E::load(p.dres_out[r], own + c);
      if (p.has_dres) E::store(p.dres[r], own + c, d);
      if (p.has_dsend)
        for (int q = 0; q < p.nranks; ++q) E::store(p.dsend[q], at + c, d);
    }
  }
  if (p.has_dweight)
    for (int c = threadIdx.x; c < p.hidden; c += blockDim.x) p.part[static_cast<int64_t>(blockIdx.x) * p.hidden + c] = dw[c];
}

struct WeightParams {
  const float* part;
  float* dweight[VC_MAX_RANKS];
  uint32_t per, chunks;  // parts of each rank; blocks of each rank
  int32_t hidden;
};
constexpr int kSumAhead = 8;   // parts of a thread whose loads are in flight together
constexpr int kSumWarps = 16;  // of a block, at most

// dweight[r] = the sum of rank r's parts: 32 columns a block, its warps take
// the parts in turn, and the warps' sums are added in warp order.
__global__ void __launch_bounds__(kSumWarps * 32) norm_weight_kernel(const __grid_constant__ WeightParams p) {
  __shared__ float sums[kSumWarps][32];
  stream_order();
  const uint32_t r = blockIdx.x / p.chunks, chunk = blockIdx.x - r * p.chunks;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int c = static_cast<int>(chunk) * 32 + lane;
  float x = 0.f;
  if (c < p.hidden) {
    const float* from = p.part + static_cast<int64_t>(r) * p.per * p.hidden + c;
    for (uint32_t b0 = warp; b0 < p.per; b0 += warps * kSumAhead) {  // loads in flight together
      float v[kSumAhead];
#pragma unroll
      for (int i = 0; i < kSumAhead; ++i) {
        const uint32_t b = b0 + i * warps;
        v[i] = b < p.per ? from[static_cast<int64_t>(b) * p.hidden] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < kSumAhead; ++i) x += v[i];
    }
  }
  sums[warp][lane] = x;
  __syncthreads();
  if (warp == 0 && c < p.hidden) {
    x = 0.f;
    for (int w = 0; w < warps; ++w) x += sums[w][lane];
    p.dweight[r][c] = x;
  }
}

unsigned threads_for(int64_t n, int per_thread, int most) {
  const int64_t t = (n + per_thread - 1) / per_thread;
  return static_cast<unsigned>(std::min<int64_t>(most, (t + 31) / 32 * 32));
}
// Threads of a block that takes a row element by element.
unsigned any_threads(int64_t hidden) { return threads_for(hidden, 4, 1024); }

// Blocks of each rank: enough to fill the GPU, at most one per row.
uint32_t blocks_per_rank(int64_t resident, int nranks, uint32_t rows) {
  return static_cast<uint32_t>(std::max<int64_t>(1, std::min<int64_t>(rows, resident / nranks)));
}

template <int DT, bool VEC, bool FEW, int VPT, bool I8>
vc_status_t launch_norm(DeviceState* st, int dev, int64_t n, cudaStream_t s, const NormParams& p, int64_t bytes) {
  constexpr auto kKernel = norm_kernel<DT, VEC, FEW, VPT, I8>;
  Shape shape{p.rows, threads_for(n, VPT, norm_threads(VEC, VPT)), 0, 1, static_cast<unsigned>(p.nranks)};
  if (FEW) shape.grid = blocks_per_rank(int64_t(st->nsm) * resident_blocks<kKernel>(dev, static_cast<int>(shape.block), 0), p.nranks, p.rows);
  return launch<kKernel>(dev, shape, s, p, kNorm, 0, bytes);
}
template <int DT, bool VEC, bool FEW, int VPT>
vc_status_t launch_norm(DeviceState* st, int dev, int64_t n, bool i8, cudaStream_t s, const NormParams& p, int64_t bytes) {
  return i8 ? launch_norm<DT, VEC, FEW, VPT, true>(st, dev, n, s, p, bytes) : launch_norm<DT, VEC, FEW, VPT, false>(st, dev, n, s, p, bytes);
}

vc_status_t norm(const void* const* send, const void* const* residual, const void* const* weight,
                 void* const* residual_out, void* const* out, float* const* scale, float* const* rstd, int nranks,
                 size_t rows, size_t hidden, double eps, vc_dtype_t dtype, vc_dtype_t out_dtype, cudaStream_t stream) {
  vc_status_t rc = check_ranks(nranks);
  if (rc == VC_SUCCESS) rc = check_float(dtype);
  if (rc != VC_SUCCESS) return rc;
  const bool i8 = out_dtype == VC_INT8;
  if (!i8 && out_dtype != dtype) return fail(VC_ERR_UNSUPPORTED, "out_dtype must be the data's or VC_INT8");
  if (!(eps >= 0) || !std::isfinite(eps)) return fail(VC_ERR_INVALID_ARG, "eps must be finite and not negative");
  if (hidden > VC_NORM_MAX_HIDDEN) return fail(VC_ERR_UNSUPPORTED, "hidden above VC_NORM_MAX_HIDDEN");
  rc = check_tokens(nranks, rows, hidden);
  if (rc != VC_SUCCESS) return rc;
  const int64_t es = dtype_size(dtype), n = static_cast<int64_t>(rows) * static_cast<int64_t>(hidden);
  const int os = dtype_size(out_dtype);
  Buffers b;
  rc = b.add(send, nranks, n * nranks * es, static_cast<int>(es), false, "send");
  if (rc == VC_SUCCESS) rc = b.add(weight, nranks, static_cast<int64_t>(hidden) * es, static_cast<int>(es), false, "weight");
  if (rc == VC_SUCCESS && residual)
    rc = b.add(residual, nranks, n * es, static_cast<int>(es), false, "residual", residual_out);
  if (rc == VC_SUCCESS && residual_out) rc = b.add(residual_out, nranks, n * es, static_cast<int>(es), true, "residual_out");
  if (rc == VC_SUCCESS) rc = b.add(out, nranks, n * os, os, true, "out");
  const bool aligned = b.aligned16();
  if (rc == VC_SUCCESS && i8) rc = b.add(const_cast<const void* const*>(reinterpret_cast<void* const*>(scale)), nranks, static_cast<int64_t>(rows) * 4, 4, true, "scale");
  if (rc == VC_SUCCESS && rstd) rc = b.add(const_cast<const void* const*>(reinterpret_cast<void* const*>(rstd)), nranks, static_cast<int64_t>(rows) * 4, 4, true, "rstd");
  if (rc == VC_SUCCESS) rc = b.disjoint();
  if (rc != VC_SUCCESS || n == 0) return rc;

  DeviceState* st = nullptr;
  int dev = 0;
  rc = device_state(&st, &dev);
  if (rc != VC_SUCCESS) return rc;
  NormParams p = {};
  for (int r = 0; r < nranks; ++r) {
    p.send[r] = send[r];
    p.weight[r] = weight[r];
    p.out[r] = out[r];
    if (residual) p.residual[r] = residual[r];
    if (residual_out) p.residual_out[r] = residual_out[r];
    if (i8) p.scale[r] = scale[r];
    if (rstd) p.rstd[r] = rstd[r];
  }
  p.nranks = nranks;
  p.has_residual = residual != nullptr;
  p.has_residual_out = residual_out != nullptr;
  p.has_rstd = rstd != nullptr;
  p.rows = static_cast<uint32_t>(rows);
  p.hidden = static_cast<int32_t>(hidden);
  p.eps = static_cast<float>(eps);
  const int64_t tokens = static_cast<int64_t>(rows) * nranks;
  const int64_t bytes = n * nranks * (es * (nranks + p.has_residual + p.has_residual_out) + os) +
                        static_cast<int64_t>(hidden) * es * nranks + tokens * 4 * (p.has_rstd + i8);
  return for_dtype(dtype, [&](auto code) {
    constexpr int DT = code();
    // VC_ERR_UNSUPPORTED: too long for registers
    const auto go = [&](auto vec, auto few) -> vc_status_t {
      constexpr bool VEC = vec(), FEW = few();
      const int64_t n = units_of(static_cast<int64_t>(hidden), El<DT>::kSize);
      if (n <= 512) return launch_norm<DT, VEC, FEW, 1>(st, dev, n, i8, stream, p, bytes);
      if (n <= 1024) return launch_norm<DT, VEC, FEW, 2>(st, dev, n, i8, stream, p, bytes);
      if constexpr (VEC) {
        if (n <= 1536) return launch_norm<DT, VEC, false, 3>(st, dev, n, i8, stream, p, bytes);
        if (n <= 2048) return launch_norm<DT, VEC, false, 2>(st, dev, n, i8, stream, p, bytes);
        if (n <= 4096) return launch_norm<DT, VEC, false, 8>(st, dev, n, i8, stream, p, bytes);
      } else {
        if (n <= 2048) return launch_norm<DT, VEC, false, 4>(st, dev, n, i8, stream, p, bytes);
      }
      return VC_ERR_UNSUPPORTED;
    };
    const bool whole = aligned && hidden % El<DT>::kVec == 0;
    const vc_status_t rc = !whole        ? go(std::false_type{}, std::false_type{})
                           : nranks <= 2 ? go(std::true_type{}, std::true_type{})
                                         : go(std::true_type{}, std::false_type{});
    if (rc != VC_ERR_UNSUPPORTED) return rc;
    const Shape shape{p.rows, any_threads(static_cast<int64_t>(hidden)), hidden * sizeof(float), 1,
                      static_cast<unsigned>(nranks)};
    return i8 ? launch<norm_any_kernel<DT, true>>(dev, shape, stream, p, kNorm, 0, bytes)
              : launch<norm_any_kernel<DT, false>>(dev, shape, stream, p, kNorm, 0, bytes);
  });
}

template <auto K>
vc_status_t launch_grad(DeviceState* st, int dev, unsigned threads, size_t smem, cudaStream_t s, GradParams& p, int64_t bytes,
                        float** scratch) {
  vc_status_t rc = allow<K>(dev, smem, false);
  if (rc != VC_SUCCESS) return rc;
  p.per = blocks_per_rank(int64_t(st->nsm) * resident_blocks<K>(dev, static_cast<int>(threads), smem), p.nranks, p.rows);
  const unsigned blocks = p.per * static_cast<unsigned>(p.nranks);
  if (p.has_dweight) {
    cudaMemPool_t pool;
    rc = scratch_pool(st, dev, &pool);
    if (rc != VC_SUCCESS) return rc;
    const size_t need = static_cast<size_t>(blocks) * p.hidden * sizeof(float);
    cudaError_t e = cudaMallocFromPoolAsync(reinterpret_cast<void**>(scratch), need, pool, s);
    if (e == cudaErrorMemoryAllocation) {
      cudaGetLastError();
      return fail(VC_ERR_NOMEM, "scratch allocation of " + std::to_string(need) + " bytes failed");
    }
    if (e != cudaSuccess) return cuda_fail(e, "cudaMallocFromPoolAsync");
    p.part = *scratch;
  }
  return launch<K>(dev, Shape{blocks, threads, smem}, s, p, kNormBackward, 0, bytes);
}

vc_status_t norm_grad(const void* const* dout, const void* const* dres_out, const void* const* h,
                      const void* const* weight, const float* const* rstd, void* const* dsend, void* const* dres,
                      float* const* dweight, int nranks, size_t rows, size_t hidden, vc_dtype_t dtype,
                      cudaStream_t stream) {
  vc_status_t rc = check_ranks(nranks);
  if (rc == VC_SUCCESS) rc = check_float(dtype);
  if (rc != VC_SUCCESS) return rc;
  if (hidden > VC_NORM_MAX_HIDDEN) return fail(VC_ERR_UNSUPPORTED, "hidden above VC_NORM_MAX_HIDDEN");
  rc = check_tokens(nranks, rows, hidden);
  if (rc != VC_SUCCESS) return rc;
  if (!dsend && !dres && !dweight) return fail(VC_ERR_INVALID_ARG, "no gradient is asked for");
  const int64_t es = dtype_size(dtype), n = static_cast<int64_t>(rows) * static_cast<int64_t>(hidden);
  const int a = static_cast<int>(es);
  Buffers b;
  rc = b.add(dout, nranks, n * es, a, false, "dout");
  if (rc == VC_SUCCESS) rc = b.add(h, nranks, n * es, a, false, "h");
  if (rc == VC_SUCCESS) rc = b.add(weight, nranks, static_cast<int64_t>(hidden) * es, a, false, "weight");
  if (rc == VC_SUCCESS && dres_out) rc = b.add(dres_out, nranks, n * es, a, false, "dresidual_out", dres);
  if (rc == VC_SUCCESS && dsend) rc = b.add(dsend, nranks, n * nranks * es, a, true, "dsend");
  if (rc == VC_SUCCESS && dres) rc = b.add(dres, nranks, n * es, a, true, "dresidual");
  const bool aligned = b.aligned16();
  if (rc == VC_SUCCESS) rc = b.add(reinterpret_cast<const void* const*>(rstd), nranks, static_cast<int64_t>(rows) * 4, 4, false, "rstd");
  if (rc == VC_SUCCESS && dweight) rc = b.add(const_cast<const void* const*>(reinterpret_cast<void* const*>(dweight)), nranks, static_cast<int64_t>(hidden) * 4, 4, true, "dweight");
  if (rc == VC_SUCCESS) rc = b.disjoint();
  if (rc != VC_SUCCESS || hidden == 0) return rc;
  if (rows == 0) {  // the sum over no tokens
    for (int r = 0; dweight && r < nranks; ++r) {
      cudaError_t e = cudaMemsetAsync(dweight[r], 0, hidden * sizeof(float), stream);
      if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync");
    }
    return VC_SUCCESS;
  }

  DeviceState* st = nullptr;
  int dev = 0;
  rc = device_state(&st, &dev);
  if (rc != VC_SUCCESS) return rc;
  GradParams p = {};
  for (int r = 0; r < nranks; ++r) {
    p.dout[r] = dout[r];
    p.h[r] = h[r];
    p.weight[r] = weight[r];
    p.rstd[r] = rstd[r];
    if (dres_out) p.dres_out[r] = dres_out[r];
    if (dsend) p.dsend[r] = dsend[r];
    if (dres) p.dres[r] = dres[r];
  }
  p.nranks = nranks;
  p.has_dres_out = dres_out != nullptr;
  p.has_dsend = dsend != nullptr;
  p.has_dres = dres != nullptr;
  p.has_dweight = dweight != nullptr;
  p.rows = static_cast<uint32_t>(rows);
  p.hidden = static_cast<int32_t>(hidden);
  const int64_t bytes = n * nranks * es * (2 + p.has_dres_out + p.has_dres + (dsend ? nranks : 0)) +
                        static_cast<int64_t>(rows) * nranks * 4 + static_cast<int64_t>(hidden) * nranks * es;
  float* scratch = nullptr;
  rc = for_dtype(dtype, [&](auto code) {
    constexpr int DT = code();
    const auto go = [&](auto vec) {
      constexpr bool VEC = vec();
      const int64_t n = units_of(static_cast<int64_t>(hidden), El<DT>::kSize);
      if (n <= grad_threads(1))
        return launch_grad<norm_grad_kernel<DT, VEC, 1>>(st, dev, threads_for(n, 1, grad_threads(1)), 0, stream, p, bytes, &scratch);
      if (n <= 2 * grad_threads(2))
        return launch_grad<norm_grad_kernel<DT, VEC, 2>>(st, dev, threads_for(n, 2, grad_threads(2)), 0, stream, p, bytes, &scratch);
      if constexpr (VEC) {
        if (n <= 4 * grad_threads(4))
          return launch_grad<norm_grad_kernel<DT, VEC, 4>>(st, dev, threads_for(n, 4, grad_threads(4)), 0, stream, p, bytes, &scratch);
      }
      return VC_ERR_UNSUPPORTED;
    };
    const vc_status_t rc = aligned && hidden % El<DT>::kVec == 0 ? go(std::true_type{}) : go(std::false_type{});
    if (rc != VC_ERR_UNSUPPORTED) return rc;
    return launch_grad<norm_grad_any_kernel<DT>>(st, dev, any_threads(static_cast<int64_t>(hidden)),
                                                 hidden * sizeof(float), stream, p, bytes, &scratch);
  });
  if (rc == VC_SUCCESS && dweight) {
    WeightParams w = {};
    w.part = scratch;
    for (int r = 0; r < nranks; ++r) w.dweight[r] = dweight[r];
    w.per = p.per;
    w.chunks = static_cast<uint32_t>((hidden + 31) / 32);
    w.hidden = p.hidden;
    // warps enough to have every part in flight at once
    const unsigned warps = std::min<unsigned>(kSumWarps, (p.per + kSumAhead - 1) / kSumAhead);
    rc = launch<norm_weight_kernel>(dev, Shape{w.chunks * static_cast<unsigned>(nranks), warps * 32}, stream, w, kNormWeight, 1,
                                    static_cast<int64_t>(hidden) * nranks * 4 * (1 + static_cast<int64_t>(p.per)));
  }
  if (scratch) {
    cudaError_t e = cudaFreeAsync(scratch, stream);
    if (e != cudaSuccess && rc == VC_SUCCESS) rc = cuda_fail(e, "cudaFreeAsync");
  }
  return rc;
}

}  // namespace
}  // namespace layer
}  // namespace vc

using namespace vc;

VC_EXPORT vc_status_t vc_reduce_scatter_norm(const void* const* send, const void* const* residual,
                                             const void* const* weight, void* const* residual_out, void* const* out,
                                             float* const* scale, float* const* rstd, int nranks, size_t rows,
                                             size_t hidden, double eps, vc_dtype_t dtype, vc_dtype_t out_dtype,
                                             vc_stream_t stream) {
  return entry([&] {
    return layer::norm(send, residual, weight, residual_out, out, scale, rstd, nranks, rows, hidden, eps, dtype,
                       out_dtype, reinterpret_cast<cudaStream_t>(stream));
  });
}

VC_EXPORT vc_status_t vc_reduce_scatter_norm_backward(const void* const* dout, const void* const* dresidual_out,
                                                      const void* const* h, const void* const* weight,
                                                      const float* const* rstd, void* const* dsend,
                                                      void* const* dresidual, float* const* dweight, int nranks,
                                                      size_t rows, size_t hidden, vc_dtype_t dtype,
                                                      vc_stream_t stream) {
  return entry([&] {
    return layer::norm_grad(dout, dresidual_out, h, weight, rstd, dsend, dresidual, dweight, nranks, rows, hidden,
                            dtype, reinterpret_cast<cudaStream_t>(stream));
  });
}
