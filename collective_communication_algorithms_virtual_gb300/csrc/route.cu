// Choice of experts for each token, and its gradient (see vc.h).
//
// One warp takes one token: lane l holds experts l*V .. l*V + V - 1 in
// registers, V the power of 2 that covers all experts, so that the lowest
// lane, and in it the lowest register, is the lowest index of a tie.  What is
// compared is computed with the same roundings in the same order everywhere
// (single operations, and a softmax sum that adds neighbours first), so that
// the choice is one and the same for any V.
//
// Instruction issue bounds it: 16384 tokens of 256 bf16 logits, sigmoid scores
// with a bias, 4 of 8 groups, 8 experts chosen, take 14.7 us for 870
// instructions a token, 82% of the issue slots (the 9.4 MB would take 1.4 us):
// 490 for the row, the choice of 8 by logits and their weights (of one expert
// 370), 245 for the scores and biases, 135 for the groups.  Softmax without
// them, 505 instructions, 9.4 us.  8 tokens, 64 experts: 2.0 us, a launch.  Four
// tokens a block and 32 registers keep 64 warps per SM (8 tokens and 48
// registers: 16.8 us).
#include "layer.cuh"

namespace vc {
namespace layer {
namespace {

constexpr int kWarps = 4;  // tokens of a block
constexpr unsigned kAll = 0xffffffffu;

struct RouteParams {
  const void* logits[VC_MAX_RANKS];
  const float* bias[VC_MAX_RANKS];
  int32_t* ids[VC_MAX_RANKS];
  float* weights[VC_MAX_RANKS];
  uint32_t rows;
  int experts, topk, groups, keep_groups, group_top;
  int group_size, group_lanes;  // group_lanes: lanes of a group, where that is a power of 2 of whole lanes, else 0
  int sigmoid, renormalize, has_bias, by_score;  // by_score: experts are compared by scores, not by logits
  int vec, vec_bias;                             // each lane's experts are one aligned piece of the row
  float scale;
};
struct RouteGradParams {
  const float* dweights[VC_MAX_RANKS];
  const void* logits[VC_MAX_RANKS];
  const int32_t* ids[VC_MAX_RANKS];
  void* dlogits[VC_MAX_RANKS];
  uint32_t rows;
  int experts, topk, renormalize, vec;
  float scale;
};

constexpr float kNone = -INFINITY;
constexpr float kLowest = -3.402823466e38f;  // of the finite numbers

// Lane's V logits of a row; -inf past the last expert.
// KEPT: through L1, for what is read again: the bias by every warp (16384
// tokens with one bias of 256: 24 us with every read from L2, 17 us from L1).
template <int DT, int V, bool KEPT = false>
__device__ __forceinline__ void load_row(const void* row, int lane, int experts, int vec, float* l) {
  using E = El<DT>;
  const int e0 = lane * V;
  if (vec) {
    if (e0 < experts) {
      if constexpr (V % E::kVec == 0) {
#pragma unroll
        for (int i = 0; i < V / E::kVec; ++i) {
          const uint4* at = static_cast<const uint4*>(row) + lane * (V / E::kVec) + i;
          E::widen(KEPT ? __ldg(at) : dev::ld16(at), l + i * E::kVec);
        }
      } else if constexpr (V * E::kSize == 8) {
        const uint2 v = static_cast<const uint2*>(row)[lane];
        if constexpr (DT == VC_FLOAT32) {
          l[0] = __uint_as_float(v.x);
          l[1] = __uint_as_float(v.y);
        } else {
          dev::widen2<E::kF16>(v.x, l);
          dev::widen2<E::kF16>(v.y, l + 2);
        }
      } else if constexpr (V * E::kSize == 4 && V == 2) {
        dev::widen2<E::kF16>(static_cast<const uint32_t*>(row)[lane], l);
      } else {
        l[0] = E::load(row, lane);
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) l[i] = kNone;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = e0 + i < experts ? E::load(row, e0 + i) : kNone;
  }
}
template <int DT, int V>
__device__ __forceinline__ void store_row(void* row, int lane, int experts, int vec, const float* x) {
  using E = El<DT>;
  const int e0 = lane * V;
  if constexpr (V % E::kVec == 0) {
    if (vec) {
      if (e0 < experts) {
#pragma unroll
        for (int i = 0; i < V / E::kVec; ++i)
          dev::st16_wb(static_cast<uint4*>(row) + lane * (V / E::kVec) + i, E::narrow(x + i * E::kVec));
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (e0 + i < experts) E::store(row, e0 + i, x[i]);
}

// Sum over all lanes' V values, neighbours first.
template <int V>
__device__ __forceinline__ float pair_sum(const float* x) {
  float s[V];
#pragma unroll
  for (int i = 0; i < V; ++i) s[i] = x[i];
#pragma unroll
  for (int n = V / 2; n > 0; n /= 2)
#pragma unroll
    for (int i = 0; i < n; ++i) s[i] = __fadd_rn(s[2 * i], s[2 * i + 1]);
  float t = s[0];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) t = __fadd_rn(t, __shfl_xor_sync(kAll, t, d));
  return t;
}
// The largest over the warp (NaN is passed over).
__device__ __forceinline__ float warp_max(float x) {
  float m;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(x));
  return m;
}
template <int V>
__device__ __forceinline__ float row_max(const float* l) {  // NaN is passed over
  float m = kNone;
#pragma unroll
  for (int i = 0; i < V; ++i) m = fmaxf(m, l[i]);
  return warp_max(m);
}
__device__ __forceinline__ bool there(float l) { return l > kNone; }
// exp(l - most), with the largest itself (infinite ones too) at 1.
__device__ __forceinline__ float soft(float l, float most) {
  return !there(l) ? 0.f : l == most ? 1.f : expf(__fsub_rn(l, most));
}
__device__ __forceinline__ float sigmoid(float l) {  // not for NaN; 0 at -inf
  return __frcp_rn(__fadd_rn(1.f, expf(-l)));
}

// The two largest of a group so far, and one more value.
struct Two {
  float a = kNone, b = kNone;
  __device__ __forceinline__ void take(float x) {
    b = fmaxf(b, fminf(a, x));
    a = fmaxf(a, x);
  }
  // Of a group that has experts above kNone, whatever their sum.
  __device__ __forceinline__ float worth(int top) const { return top == 2 && b > kNone ? fmaxf(__fadd_rn(a, b), kLowest) : a; }
};

// An expert that may be among the chosen.
struct Candidate {
  float c;
  int expert;
};

// The choice proper: lane j's `place` is where its expert `id` stands among
// the chosen, best first, or -1 (some lanes hold none); returns how many are
// chosen.  With several experts a lane, the k-th best of the lanes' bests
// (equal ones counted once) is no better than the k-th best of all; what
// reaches it, a little more than k experts as a rule, is laid out one to a
// lane in index order, and each counts those before it.  More than 32 of them
// (ties, or fewer lanes with an expert than k) are taken one by one instead.
// 16384 tokens, 256 experts, 8 chosen in 4 of 8 groups: 15.8 us while each
// round of the bound also looked for its lane, 14.7 us so.
template <int V>
__device__ __forceinline__ int choose(float* c, int topk, int lane, Candidate* list, int* id, int* place) {
  float best = c[0];
#pragma unroll
  for (int i = 1; i < V; ++i) best = fmaxf(best, c[i]);
  *id = -1;
  *place = -1;
  if constexpr (V == 1) {
    int found = 0;
    for (; found < topk; ++found) {
      const float top = warp_max(best);
      if (!(top > kNone)) break;
      const int from = __ffs(__ballot_sync(kAll, best == top)) - 1;
      if (lane == from) best = kNone;
      if (lane == found) {
        *id = from;
        *place = found;
      }
    }
    return found;
  }
  float bound = kNone, rest = best;
#pragma unroll 4
  for (int j = 0; j < topk; ++j) {
    bound = warp_max(rest);
    if (rest == bound) rest = kNone;
  }
  bound = fmaxf(bound, kLowest);  // above -inf
  int mine = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) mine += c[i] >= bound;
  int upto = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int m = __shfl_up_sync(kAll, upto, d);
    if (lane >= d) upto += m;
  }
  const int n = __shfl_sync(kAll, upto, 31);
  if (n <= 32) {
    int at = upto - mine;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (c[i] >= bound) list[at++] = Candidate{c[i], lane * V + i};
    __syncwarp();
    Candidate x{kNone, -1};
    if (lane < n) x = list[lane];
    int before = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
      const float y = __shfl_sync(kAll, x.c, j);
      before += j < lane ? y >= x.c : y > x.c;
    }
    if (lane < n && before < topk) {
      *id = x.expert;
      *place = before;
    }
    return min(n, topk);
  }
  int found = 0;
  for (; found < topk; ++found) {
    const float top = warp_max(best);
    if (!(top > kNone)) break;
    const int from = __ffs(__ballot_sync(kAll, best == top)) - 1;
    int i0 = 0;
#pragma unroll
    for (int i = V - 1; i >= 0; --i)
      if (c[i] == top) i0 = i;
    const int e = __shfl_sync(kAll, lane * V + i0, from);
    if (lane == found) {
      *id = e;
      *place = found;
    }
    if (lane == from) {
      best = kNone;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (i == i0) c[i] = kNone;
        best = fmaxf(best, c[i]);
      }
    }
  }
  return found;
}

template <int DT, int V>
__global__ void __launch_bounds__(kWarps * 32, V <= 8 ? 16 : 4) route_kernel(const __grid_constant__ RouteParams p) {
  __shared__ float table[kWarps][V * 32];  // a token's c, where a group's experts are not whole lanes
  __shared__ Candidate list[kWarps][32];
  stream_order();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t r = blockIdx.y, t = blockIdx.x * kWarps + warp;
  if (t >= p.rows) return;
  const char* row = static_cast<const char*>(p.logits[r]) + static_cast<int64_t>(t) * p.experts * El<DT>::kSize;
  float c[V];  // what experts are compared by, -inf where not to be chosen
  load_row<DT, V, true>(row, lane, p.experts, p.vec, c);  // the chosen logits are read again
  float most = 0.f, sum = 1.f;
  // the softmax's maximum and sum, where a score is wanted (the sum cancels
  // in weights that are renormalised)
  if (!p.sigmoid) {
    most = row_max<V>(c);
    if (p.by_score || !p.renormalize) {
      float e[V];
#pragma unroll
      for (int i = 0; i < V; ++i) e[i] = soft(c[i], most);
      sum = pair_sum<V>(e);
      if (p.by_score) {
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] = there(c[i]) ? __fdiv_rn(e[i], sum) : kNone;
      }
    }
  } else if (p.by_score) {
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = there(c[i]) ? sigmoid(c[i]) : kNone;
  }
  if (!p.by_score) {
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = there(c[i]) ? c[i] : kNone;  // NaN
  }
  if (p.has_bias) {
    float b[V];
    load_row<VC_FLOAT32, V, true>(p.bias[r], lane, p.experts, p.vec_bias, b);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      c[i] = fmaxf(__fadd_rn(c[i], b[i]), kNone);  // a NaN is not chosen either
    }
  }
  if (p.groups > 1) {
    if (p.group_lanes) {
      Two two;
#pragma unroll
      for (int i = 0; i < V; ++i) two.take(c[i]);
      for (int d = 1; d < p.group_lanes; d <<= 1) {
        const float a = __shfl_xor_sync(kAll, two.a, d), b = __shfl_xor_sync(kAll, two.b, d);
        two.take(a);
        two.take(b);
      }
      // the best groups one by one, the lowest of equal ones first
      float rest = two.worth(p.group_top);
      bool kept = false;
      const int group = lane & -p.group_lanes;
      for (int g = 0; g < p.keep_groups; ++g) {
        const float top = warp_max(rest);
        const int best = (__ffs(__ballot_sync(kAll, rest == top)) - 1) & -p.group_lanes;
        if (group == best) {
          kept = true;
          rest = NAN;  // passed over from now on
        }
      }
      if (!kept) {
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] = kNone;
      }
    } else {
      const int size = p.group_size;
#pragma unroll
      for (int i = 0; i < V; ++i) table[warp][lane * V + i] = c[i];
      __syncwarp();
      Two two;
      if (lane < p.groups)
        for (int i = 0; i < size; ++i) two.take(table[warp][lane * size + i]);
      const float mine = two.worth(p.group_top);
      int better = 0;
      for (int g = 0; g < p.groups; ++g) {
        const float w = __shfl_sync(kAll, mine, g);
        better += g < lane ? w >= mine : w > mine;
      }
      const uint32_t kept = __ballot_sync(kAll, lane < p.groups && better < p.keep_groups);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = lane * V + i;
        if (e < p.experts && !(kept >> (e / size) & 1)) c[i] = kNone;
      }
    }
  }
  int id, place;
  const int n = choose<V>(c, p.topk, lane, list[warp], &id, &place);
  float w = 0.f;
  if (place >= 0) {  // the score, again from the logit
    const float l = El<DT>::load(row, id);
    w = p.sigmoid ? sigmoid(l) : __fdiv_rn(soft(l, most), sum);
  }
  if (p.renormalize) w = w / fmaxf(warp_sum(w), 0x1p-126f);
  const int64_t to = static_cast<int64_t>(t) * p.topk;
  if (place >= 0) {
    p.ids[r][to + place] = id;
    p.weights[r][to + place] = w * p.scale;
  }
  if (lane >= n && lane < p.topk) {
    p.ids[r][to + lane] = -1;
    p.weights[r][to + lane] = 0.f;
  }
}

// The gradient.  With sigmoid scores only the chosen logits are read; with
// renormalised softmax scores the row is read for its largest logit (16384
// tokens, 256 bf16 logits, 8 chosen: 10.2 us, 9.1 us without).  The kind of
// score is a compile-time constant: in one kernel the row's registers cost the
// sigmoid forms 3% (the same sizes, not renormalised: 8.65 us, 8.3 us so).
// 16384 tokens, 128 fp32 logits, 6 chosen: softmax 7.4 us for 350 instructions
// a token (17.6 MB, 2.6 us), renormalised 6.9 us for 300; sigmoid 6.2 us for
// 240, renormalised 7.1 us for 310.
template <int DT, int V, bool SIGMOID>
__global__ void __launch_bounds__(kWarps * 32) route_grad_kernel(const __grid_constant__ RouteGradParams p) {
  stream_order();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t r = blockIdx.y, t = blockIdx.x * kWarps + warp;
  if (t >= p.rows) return;
  const int64_t at = static_cast<int64_t>(t) * p.experts * El<DT>::kSize;
  const char* row = static_cast<const char*>(p.logits[r]) + at;
  float all[V];
  if (!SIGMOID) load_row<DT, V>(row, lane, p.experts, p.vec, all);
  // lane j: choice j's expert, its logit and the gradient of scale * (its share or score)
  int id = -1;
  float l = kNone, d = 0.f;
  if (lane < p.topk) {
    const int64_t from = static_cast<int64_t>(t) * p.topk + lane;
    id = p.ids[r][from];
    if (id >= 0 && id < p.experts) {
      l = El<DT>::load(row, id);
      d = p.dweights[r][from] * p.scale;
    } else {
      id = -1;
    }
  }
  float x[V];  // the row's gradient
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = 0.f;
  float give = 0.f;  // lane j: what its choice adds to its expert's gradient
  if (p.renormalize) {
    // shares of the chosen scores; of a softmax they depend on the chosen
    // logits alone, and the gradient stays among them
    const float most = warp_max(l);
    const float e = !there(l) ? 0.f : SIGMOID ? sigmoid(l) : soft(l, most);
    float total = warp_sum(e);
    if (!SIGMOID) {
      // `total` counts from the best chosen score.  The scores themselves sum
      // to less than 2^-126 only where that one is more than 80 below the
      // row's largest logit (exp(-80) / 1024 experts is above it).
      const float top = row_max<V>(all);
      if (!(most == top || most - top >= -80.f)) {
#pragma unroll
        for (int i = 0; i < V; ++i) all[i] = soft(all[i], top);
        const float sum = pair_sum<V>(all);
        const float s = warp_sum(there(l) ? __fdiv_rn(soft(l, top), sum) : 0.f);
        if (!(s >= 0x1p-126f)) total = 0.f;
      }
    }
    if (total >= 0x1p-126f) {
      const float share = e / total;
      give = share * (d - warp_sum(d * share));
      if (SIGMOID) give *= 1.f / (1.f + expf(l));
    }
  } else if (SIGMOID) {
    give = there(l) ? d * sigmoid(l) / (1.f + expf(l)) : 0.f;
  } else {
    const float most = row_max<V>(all);
#pragma unroll
    for (int i = 0; i < V; ++i) all[i] = soft(all[i], most);
    const float sum = pair_sum<V>(all);
    const float s = there(l) ? soft(l, most) / sum : 0.f;
    const float dot = warp_sum(d * s);
    give = d * s;
    const float by = sum > 0.f ? dot / sum : 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = -all[i] * by;
  }
  if (!there(l)) give = 0.f;
  for (int j = 0; j < p.topk; ++j) {
    const int e = __shfl_sync(kAll, id, j);
    const float g = __shfl_sync(kAll, give, j);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (e == lane * V + i) x[i] += g;
  }
  store_row<DT, V>(static_cast<char*>(p.dlogits[r]) + at, lane, p.experts, p.vec, x);
}

// Runs f with the experts a lane holds as a compile-time constant.
template <class F>
vc_status_t for_width(int experts, F&& f) {
  if (experts <= 32) return f(std::integral_constant<int, 1>{});
  if (experts <= 64) return f(std::integral_constant<int, 2>{});
  if (experts <= 128) return f(std::integral_constant<int, 4>{});
  if (experts <= 256) return f(std::integral_constant<int, 8>{});
  if (experts <= 512) return f(std::integral_constant<int, 16>{});
  return f(std::integral_constant<int, 32>{});
}

vc_status_t check_route(int nranks, size_t rows, int nexperts, const vc_route_t* how, vc_dtype_t dtype) {
  vc_status_t rc = check_ranks(nranks);
  if (rc == VC_SUCCESS) rc = check_float(dtype);
  if (rc != VC_SUCCESS) return rc;
  if (!how) return fail(VC_ERR_INVALID_ARG, "null route description");
  if (how->score != VC_SCORE_SOFTMAX && how->score != VC_SCORE_SIGMOID) return fail(VC_ERR_INVALID_ARG, "unknown score");
  if (nexperts < 1 || nexperts > VC_ROUTE_MAX_EXPERTS) return fail(VC_ERR_INVALID_ARG, "nexperts outside [1, 1024]");
  if (how->topk < 1 || how->topk > VC_ROUTE_MAX_TOPK || how->topk > nexperts)
    return fail(VC_ERR_INVALID_ARG, "topk outside [1, min(nexperts, 32)]");
  if (!std::isfinite(how->scale)) return fail(VC_ERR_INVALID_ARG, "scale must be finite");
  return check_tokens(nranks, rows, static_cast<size_t>(nexperts));
}
// Whether a lane's V experts are whole, aligned pieces of every row.
bool whole_lanes(bool aligned, int experts, int v) { return aligned && experts % v == 0; }

vc_status_t route(const void* const* logits, const float* const* bias, int32_t* const* ids, float* const* weights,
                  int nranks, size_t rows, int nexperts, const vc_route_t* how, vc_dtype_t dtype, cudaStream_t stream) {
  vc_status_t rc = check_route(nranks, rows, nexperts, how, dtype);
  if (rc != VC_SUCCESS) return rc;
  if (how->ngroups < 1 || how->ngroups > 32 || nexperts % how->ngroups)
    return fail(VC_ERR_INVALID_ARG, "ngroups must be in [1, 32] and divide nexperts");
  if (how->topk_groups < 1 || how->topk_groups > how->ngroups) return fail(VC_ERR_INVALID_ARG, "topk_groups outside [1, ngroups]");
  if (how->group_top != 1 && how->group_top != 2) return fail(VC_ERR_INVALID_ARG, "group_top must be 1 or 2");
  const int es = dtype_size(dtype);
  const int64_t n = static_cast<int64_t>(rows), k = how->topk;
  Buffers b;
  rc = b.add(logits, nranks, n * nexperts * es, es, false, "logits");
  const bool aligned = b.aligned16();
  bool bias_aligned = true;
  for (int r = 0; bias && r < nranks; ++r) bias_aligned &= (reinterpret_cast<uintptr_t>(bias[r]) & 15) == 0;
  if (rc == VC_SUCCESS && bias) rc = b.add(reinterpret_cast<const void* const*>(bias), nranks, int64_t(nexperts) * 4, 4, false, "bias");
  if (rc == VC_SUCCESS) rc = b.add(reinterpret_cast<const void* const*>(ids), nranks, n * k * 4, 4, true, "ids");
  if (rc == VC_SUCCESS) rc = b.add(reinterpret_cast<const void* const*>(weights), nranks, n * k * 4, 4, true, "weights");
  if (rc == VC_SUCCESS) rc = b.disjoint();
  if (rc != VC_SUCCESS || rows == 0) return rc;
  DeviceState* st = nullptr;
  int dev = 0;
  rc = device_state(&st, &dev);
  if (rc != VC_SUCCESS) return rc;
  RouteParams p = {};
  for (int r = 0; r < nranks; ++r) {
    p.logits[r] = logits[r];
    if (bias) p.bias[r] = bias[r];
    p.ids[r] = ids[r];
    p.weights[r] = weights[r];
  }
  p.rows = static_cast<uint32_t>(rows);
  p.experts = nexperts;
  p.topk = how->topk;
  p.groups = how->ngroups;
  p.group_size = nexperts / how->ngroups;
  p.keep_groups = how->topk_groups;
  p.group_top = how->group_top;
  p.sigmoid = how->score == VC_SCORE_SIGMOID;
  p.renormalize = how->renormalize != 0;
  p.has_bias = bias != nullptr;
  p.by_score = bias != nullptr || (how->ngroups > 1 && how->group_top == 2);
  p.scale = how->scale;
  const int64_t bytes = n * nranks * (int64_t(nexperts) * es + k * 8) + (bias ? int64_t(nexperts) * nranks * 4 : 0);
  const Shape shape{(p.rows + kWarps - 1) / kWarps, kWarps * 32, 0, 1, static_cast<unsigned>(nranks)};
  return for_dtype(dtype, [&](auto code) {
    return for_width(nexperts, [&](auto width) {
      p.vec = whole_lanes(aligned, nexperts, width());
      p.vec_bias = whole_lanes(bias_aligned, nexperts, width());
      const int lanes = p.group_size % width() ? 0 : p.group_size / width();
      p.group_lanes = lanes & (lanes - 1) ? 0 : lanes;
      return launch<route_kernel<code(), width()>>(dev, shape, stream, p, kRoute, 0, bytes);
    });
  });
}

vc_status_t route_grad(const float* const* dweights, const void* const* logits, const int32_t* const* ids,
                       void* const* dlogits, int nranks, size_t rows, int nexperts, const vc_route_t* how,
                       vc_dtype_t dtype, cudaStream_t stream) {
  vc_status_t rc = check_route(nranks, rows, nexperts, how, dtype);
  if (rc != VC_SUCCESS) return rc;
  const int es = dtype_size(dtype);
  const int64_t n = static_cast<int64_t>(rows), k = how->topk;
  Buffers b;
  rc = b.add(logits, nranks, n * nexperts * es, es, false, "logits");
  if (rc == VC_SUCCESS) rc = b.add(dlogits, nranks, n * nexperts * es, es, true, "dlogits");
  const bool aligned = b.aligned16();
  if (rc == VC_SUCCESS) rc = b.add(reinterpret_cast<const void* const*>(dweights), nranks, n * k * 4, 4, false, "dweights");
  if (rc == VC_SUCCESS) rc = b.add(reinterpret_cast<const void* const*>(ids), nranks, n * k * 4, 4, false, "ids");
  if (rc == VC_SUCCESS) rc = b.disjoint();
  if (rc != VC_SUCCESS || rows == 0) return rc;
  DeviceState* st = nullptr;
  int dev = 0;
  rc = device_state(&st, &dev);
  if (rc != VC_SUCCESS) return rc;
  RouteGradParams p = {};
  for (int r = 0; r < nranks; ++r) {
    p.dweights[r] = dweights[r];
    p.logits[r] = logits[r];
    p.ids[r] = ids[r];
    p.dlogits[r] = dlogits[r];
  }
  p.rows = static_cast<uint32_t>(rows);
  p.experts = nexperts;
  p.topk = how->topk;
  p.renormalize = how->renormalize != 0;
  p.scale = how->scale;
  const bool sigmoid = how->score == VC_SCORE_SIGMOID;
  const int64_t bytes = n * nranks * ((int64_t(nexperts) + (sigmoid ? k : nexperts)) * es + k * 8);
  const Shape shape{(p.rows + kWarps - 1) / kWarps, kWarps * 32, 0, 1, static_cast<unsigned>(nranks)};
  return for_dtype(dtype, [&](auto code) {
    return for_width(nexperts, [&](auto width) {
      p.vec = whole_lanes(aligned, nexperts, width());
      return sigmoid ? launch<route_grad_kernel<code(), width(), true>>(dev, shape, stream, p, kRouteBackward, 0, bytes)
                     : launch<route_grad_kernel<code(), width(), false>>(dev, shape, stream, p, kRouteBackward, 0, bytes);
    });
  });
}

}  // namespace
}  // namespace layer
}  // namespace vc

using namespace vc;

VC_EXPORT vc_status_t vc_route(const void* const* logits, const float* const* bias, int32_t* const* ids,
                               float* const* weights, int nranks, size_t rows, int nexperts, const vc_route_t* how,
                               vc_dtype_t dtype, vc_stream_t stream) {
  return entry([&] {
    return layer::route(logits, bias, ids, weights, nranks, rows, nexperts, how, dtype,
                        reinterpret_cast<cudaStream_t>(stream));
  });
}

VC_EXPORT vc_status_t vc_route_backward(const float* const* dweights, const void* const* logits,
                                        const int32_t* const* ids, void* const* dlogits, int nranks, size_t rows,
                                        int nexperts, const vc_route_t* how, vc_dtype_t dtype, vc_stream_t stream) {
  return entry([&] {
    return layer::route_grad(dweights, logits, ids, dlogits, nranks, rows, nexperts, how, dtype,
                             reinterpret_cast<cudaStream_t>(stream));
  });
}
