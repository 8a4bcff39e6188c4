// Routing with scores (moe_route): softmax or sigmoid scores, a balance bias for
// the selection, groups of experts, top-k, scaled weights.  One wavefront per
// token; lane l holds the P experts l * P .. l * P + P - 1 (one 4 * P or 2 * P
// byte run of the row).
//
// Everything that decides an id is computed in double, so that neighbouring
// scores fall as the definition says; fp64 runs at the fp32 rate here, and a
// score (an exponential and a division) costs about 45 of the ~700 instructions
// of a token with 256 experts.  The rest are cross-lane steps, which stay in the
// vector registers: within 16-lane rows by DPP, across them by lane reads.  A
// choice value is held as an order-preserving 64-bit key; the maximum over the
// lanes is taken over the upper halves, and over the lower ones only where
// several lanes share the upper one.
//   * P is the smallest one that fits whose groups cover whole, power-of-two runs
//     of lanes (8 groups of 32 experts: P = 4, 8 lanes a group; 8 of 20: P = 5,
//     4 lanes): the groups' values then come from the same DPP steps.  Other
//     group sizes pass their values through LDS, one lane per group.
#include <type_traits>

#include "common.h"
#include "launch.h"

namespace moe {

namespace {

constexpr int kWavesPerBlock = 4;

// Monotone map of a double to uint64; NaN as -inf, -0 as +0.  0 is below every
// key it returns and marks experts that cannot be chosen (any more).
__device__ __forceinline__ uint64_t key_of(double v) {
  if (v != v) v = -__builtin_inf();
  if (v == 0.0) v = 0.0;
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return static_cast<uint32_t>(
      __builtin_amdgcn_update_dpp(static_cast<int>(v), static_cast<int>(v), CTRL, 0xf, 0xf, false));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, static_cast<uint64_t>(dpp<CTRL>(static_cast<uint32_t>(u >> 32))) << 32 |
                                        dpp<CTRL>(static_cast<uint32_t>(u)));
}
constexpr int kXor1 = 0xb1, kXor2 = 0x4e, kHalfMirror = 0x141, kMirror = 0x140;

__device__ __forceinline__ double lane_d(double v, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double,
                            static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(u >> 32), lane))) << 32 |
                                static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(u), lane)));
}

// Maximum over the 64 lanes (all active), wave-uniform.
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = max(v, dpp<kXor1>(v));
  v = max(v, dpp<kXor2>(v));
  v = max(v, dpp<kHalfMirror>(v));
  v = max(v, dpp<kMirror>(v));
  const uint32_t a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16);
  const uint32_t c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
  return max(max(a, b), max(c, d));
}
__device__ __forceinline__ float wave_max_f(float v) {
  // non-NaN floats order as their mapped bits
  const uint32_t u = __float_as_uint(v);
  const uint32_t m = wave_max_u32((u >> 31) ? ~u : (u | 0x80000000u));
  return __uint_as_float((m >> 31) ? (m & 0x7fffffffu) : ~m);
}
__device__ __forceinline__ double wave_sum_d(double v) {
  v += dpp<kXor1>(v);
  v += dpp<kXor2>(v);
  v += dpp<kHalfMirror>(v);
  v += dpp<kMirror>(v);
  return (lane_d(v, 0) + lane_d(v, 16)) + (lane_d(v, 32) + lane_d(v, 48));
}

// The two largest of two ordered pairs.
__device__ __forceinline__ void merge2(double& v1, double& v2, double o1, double o2) {
  v2 = fmax(fmin(v1, o1), fmax(v2, o2));
  v1 = fmax(v1, o1);
}

// KS: slots per lane for the chosen (k <= 64 * KS).
template <int P, bool BF16, int KS>
__global__ __launch_bounds__(kWave * kWavesPerBlock) void route_kernel(const void* __restrict__ logits,
                                                                       const float* __restrict__ bias, RouteArgs a) {
  __shared__ double vals[kWavesPerBlock][P * kWave];   // group values by way of LDS (group_lanes == 0)
  const int w = threadIdx.x >> 6, lane = lane_id();
  const int t = blockIdx.x * kWavesPerBlock + w;
  if (t >= a.T) return;                         // whole waves leave, no block barrier below
  const int E = a.E, e0 = lane * P;

  float l[P], b[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    l[i] = -__builtin_inff();
    b[i] = 0.f;
  }
  using In = std::conditional_t<BF16, uint16_t, float>;
  const In* row = static_cast<const In*>(logits) + static_cast<size_t>(t) * E + e0;
  if (e0 + P <= E) {                            // the whole run: as few loads as its alignment allows
    In v[P];
    __builtin_memcpy(v, row, sizeof(v));
    if (bias) __builtin_memcpy(b, bias + e0, sizeof(b));
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if constexpr (BF16) l[i] = bf16_to_f32(v[i]);
      else l[i] = v[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (e0 + i >= E) continue;
      if constexpr (BF16) l[i] = bf16_to_f32(row[i]);
      else l[i] = row[i];
      if (bias) b[i] = bias[e0 + i];
    }
  }
  double s[P];
#pragma unroll
  for (int i = 0; i < P; ++i)
    if (l[i] != l[i]) l[i] = -__builtin_inff();
  if (a.sigmoid) {
#pragma unroll
    for (int i = 0; i < P; ++i) s[i] = 1.0 / (1.0 + exp(-static_cast<double>(l[i])));
  } else {
    float m = l[0];
#pragma unroll
    for (int i = 1; i < P; ++i) m = fmaxf(m, l[i]);
    m = wave_max_f(m);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      // the largest logits count 1 also where they are +inf; an all -inf row counts nothing
      s[i] = l[i] == -__builtin_inff() ? 0.0
             : l[i] == m               ? 1.0
                                       : exp(static_cast<double>(l[i]) - static_cast<double>(m));
      sum += s[i];
    }
    sum = wave_sum_d(sum);
#pragma unroll
    for (int i = 0; i < P; ++i) s[i] = sum > 0.0 ? s[i] / sum : 0.0;
  }

  uint64_t key[P];
#pragma unroll
  for (int i = 0; i < P; ++i)
    key[i] = e0 + i < E ? key_of(bias ? s[i] + static_cast<double>(b[i]) : static_cast<double>(l[i])) : 0ull;

  if (a.n_groups > 1) {
    // what a group is valued by: choice values (NaN as -inf), or scores
    double g[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      g[i] = bias ? s[i] + static_cast<double>(b[i]) : a.top2 ? s[i] : static_cast<double>(l[i]);
      if (g[i] != g[i] || e0 + i >= E) g[i] = -__builtin_inf();
    }
    const int size = E / a.n_groups;
    const bool two = a.top2 && size > 1;
    double v1 = -__builtin_inf(), v2 = -__builtin_inf();
    const int L = a.group_lanes;
    if (L > 0) {
#pragma unroll
      for (int i = 0; i < P; ++i) merge2(v1, v2, g[i], -__builtin_inf());
      // after each step every lane of the doubled run holds the run's two largest
      if (L > 1) merge2(v1, v2, dpp<kXor1>(v1), dpp<kXor1>(v2));
      if (L > 2) merge2(v1, v2, dpp<kXor2>(v1), dpp<kXor2>(v2));
      if (L > 4) merge2(v1, v2, dpp<kHalfMirror>(v1), dpp<kHalfMirror>(v2));
      if (L > 8) merge2(v1, v2, dpp<kMirror>(v1), dpp<kMirror>(v2));
      if (L > 16) merge2(v1, v2, __shfl_xor(v1, 16, kWave), __shfl_xor(v2, 16, kWave));
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) vals[w][e0 + i] = g[i];
      // the wave's own values: its writes before its reads
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      if (lane < a.n_groups)
        for (int j = 0; j < size; ++j) merge2(v1, v2, vals[w][lane * size + j], -__builtin_inf());
    }
    double v = two ? v1 + v2 : v1;
    if (v != v) v = -__builtin_inf();
    // rank of this lane's group (of its experts, or of the lane's own number) among all
    const int stride = L > 0 ? L : 1;
    int rank = 0;
    for (int o = 0; o < a.n_groups; ++o) {
      const double ov = lane_d(v, o * stride);
      const bool later = lane >= (o + 1) * stride;             // lanes of groups after o
      rank += (ov > v) | ((ov == v) & later) ? 1 : 0;
    }
    const bool stays = rank < a.top_groups;
    if (L > 0) {
#pragma unroll
      for (int i = 0; i < P; ++i) key[i] = stays ? key[i] : 0ull;
    } else {
      const uint64_t kept = __ballot(stays && lane < a.n_groups);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int gi = (e0 + i) / size;
        if (gi >= a.n_groups || !((kept >> gi) & 1)) key[i] = 0ull;
      }
    }
  }

  // k rounds: the largest key, the lowest expert that has it.  Round r is kept by lane r % 64,
  // slot r / 64.  A retired key's upper half is 0, which no other key's is.
  uint32_t hi[P], lo[P];
#pragma unroll
  for (int i = 0; i < P; ++i) hi[i] = static_cast<uint32_t>(key[i] >> 32), lo[i] = static_cast<uint32_t>(key[i]);
  int cid[KS];
#pragma unroll
  for (int i = 0; i < KS; ++i) cid[i] = 0;
  for (int r = 0; r < a.k; ++r) {
    uint32_t best = hi[0];
#pragma unroll
    for (int i = 1; i < P; ++i) best = max(best, hi[i]);
    const uint32_t top = wave_max_u32(best);
    uint64_t m[P], any = 0;
    int n = 0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      m[i] = __ballot(hi[i] == top);
      any |= m[i];
      n += __popcll(m[i]);
    }
    if (n > 1) {                                // several share the upper half: the lower ones tell
      uint32_t b = 0;
#pragma unroll
      for (int i = 0; i < P; ++i) b = max(b, hi[i] == top ? lo[i] : 0u);
      const uint32_t low = wave_max_u32(b);
      any = 0;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        m[i] = __ballot(hi[i] == top && lo[i] == low);
        any |= m[i];
      }
    }
    const int wl = __ffsll(static_cast<unsigned long long>(any)) - 1;   // the lowest lane, its lowest slot
    int ws = P - 1;
#pragma unroll
    for (int i = P - 2; i >= 0; --i) ws = (m[i] >> wl) & 1 ? i : ws;
    const bool mine = lane == wl;
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (ws == i) hi[i] = mine ? 0u : hi[i];   // ws is wave-uniform
#pragma unroll
    for (int i = 0; i < KS; ++i)
      if (KS == 1 || r / kWave == i) cid[i] = lane == r % kWave ? wl * P + ws : cid[i];
  }
  // the chosen experts' scores, from the lanes that hold them
  double cs[KS], sum = 0.0;
#pragma unroll
  for (int j = 0; j < KS; ++j) {
    const int from = cid[j] / P, slot = cid[j] - from * P;
    cs[j] = 0.0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const double v = __shfl(s[i], from, kWave);
      cs[j] = slot == i ? v : cs[j];
    }
    if (j * kWave + lane >= a.k) cs[j] = 0.0;
    sum += cs[j];
  }
  const double denom = a.renormalize ? wave_sum_d(sum) : 1.0;
  const double factor = denom > 0.0 ? static_cast<double>(a.scale) / denom : 0.0;
#pragma unroll
  for (int j = 0; j < KS; ++j) {
    const int at = j * kWave + lane;
    if (at < a.k) {
      a.topk_ids[static_cast<size_t>(t) * a.k + at] = cid[j];
      a.topk_w[static_cast<size_t>(t) * a.k + at] = static_cast<float>(cs[j] * factor);
    }
  }
}

template <int P, int KS>
void launch_k(const void* logits, const float* bias, const RouteArgs& a, hipStream_t stream) {
  dim3 grid((a.T + kWavesPerBlock - 1) / kWavesPerBlock), block(kWave * kWavesPerBlock);
  if (a.bf16)
    hipLaunchKernelGGL((route_kernel<P, true, KS>), grid, block, 0, stream, logits, bias, a);
  else
    hipLaunchKernelGGL((route_kernel<P, false, KS>), grid, block, 0, stream, logits, bias, a);
}

template <int P>
void launch_p(const void* logits, const float* bias, const RouteArgs& a, hipStream_t stream) {
  if (a.k <= kWave) launch_k<P, 1>(logits, bias, a, stream);
  else launch_k<P, P>(logits, bias, a, stream);   // k <= E <= 64 * P
}

}  // namespace

hipError_t launch_route(const void* logits, const float* bias, const RouteArgs& args, hipStream_t stream) {
  RouteArgs a = args;
  const int least = (a.E + kWave - 1) / kWave, size = a.E / a.n_groups;
  int P = least;
  a.group_lanes = 0;
  for (int p = least; a.n_groups > 1 && p <= 8; ++p) {
    const int lanes = size / p;
    if (size % p == 0 && (lanes & (lanes - 1)) == 0) {
      P = p;
      a.group_lanes = lanes;
      break;
    }
  }
  // a grid has fewer than 2^32 threads: at most 2^25 tokens of a wavefront each in a launch
  constexpr int kMost = 1 << 25;
  for (int t = 0; t < args.T; t += kMost) {
    a.T = args.T - t < kMost ? args.T - t : kMost;
    a.topk_ids = args.topk_ids + static_cast<size_t>(t) * a.k;
    a.topk_w = args.topk_w + static_cast<size_t>(t) * a.k;
    const void* row = static_cast<const char*>(logits) + static_cast<size_t>(t) * a.E * (a.bf16 ? 2 : 4);
    switch (P) {
      case 1: launch_p<1>(row, bias, a, stream); break;
      case 2: launch_p<2>(row, bias, a, stream); break;
      case 3: launch_p<3>(row, bias, a, stream); break;
      case 4: launch_p<4>(row, bias, a, stream); break;
      case 5: launch_p<5>(row, bias, a, stream); break;
      case 6: launch_p<6>(row, bias, a, stream); break;
      case 7: launch_p<7>(row, bias, a, stream); break;
      default: launch_p<8>(row, bias, a, stream); break;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (a.T < kMost) break;                     // t + kMost may pass int32
  }
  return hipSuccess;
}

}  // namespace moe
